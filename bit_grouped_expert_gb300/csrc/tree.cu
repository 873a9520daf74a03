// Attention of drafted trees over a paged cache (tree.h).
//
// The query heads of a KV head and the nodes of a tree together make the rows
// of one matrix (row = node * G + head), so that a K or V tile read once
// serves all of them: per tile of 64 positions
//   S[128 rows x 64]  = Q . K^T     tcgen05, K in shared memory
//   P = 2^(S - m)                   one thread a row, running maximum m and sum l
//   O[128 rows x D]  += P . V       tcgen05, P in tensor memory, V in shared memory
// A unit is (sequence, KV head, up to 128 rows); its tiles are the cached
// positions and then the tree's own nodes.  All units' tiles, in a row, are cut
// into one equal run per CTA, whatever the lengths: a unit that spans CTAs
// leaves partial results (m, l, O in fp32), which a second kernel joins.
//
// Roles: the first four warps own the rows (at D = 256 eight, two threads a
// row), the next loads (TMA: pages by the table's numbers, K one tile ahead of
// V, into a ring), the next issues the MMAs (S of the next tile during the
// softmax of this one; at D = 256 the last issues those of O).  Rescaling O on a new maximum
// is put off while the maximum grows by less than 2^8: P then stays within
// 2^8 and the fp32 sums lose nothing.
// Who waits on a barrier's parity must know that the phase before has passed:
// the comments at the waits say from what.  (The whole protocol was run on
// the CPU as a model, tests/test_tree_protocol.py, for overflows, stale
// slots and deadlocks.)
//
// Bound: for few rows by HBM (24 sequences of 1,100 to 9,000 positions, 5 nodes
// each, 260 MB: 58 us, 4.5 TB/s with the start, the results' way out and the join;
// 5.9 TB/s in between).  For 128 rows by shared memory: a 128-wide tile of D = 256
// moves Q 64, K 64 (both for the scores) and V 64 KB out of it and K and V in,
// 2,560 cycles at 128 bytes each of the 3,050 a tile takes; its MMAs are 2,048
// (61 nodes over 131,000 positions: 106 us, 1,240 TFLOP/s).
//
// Every wait is bounded: after one second the kernel records
// MOE_ERR_DEVICE_TIMEOUT, drains its copies and MMAs, frees tensor memory
// and exits.
#include <cuda_fp16.h>
#include <math.h>

#include "attn_join.cuh"
#include "cache.cuh"
#include "kernels.h"
#include "tc.h"
#include "tc_ptx.cuh"
#include "tree.h"

namespace moe {
namespace {

constexpr int TR_MAXN = 256;      // nodes of a tree
constexpr int TR_ROWS = 128;      // rows of a unit (MMA M)
constexpr int TR_MAX_SMS = JOIN_MAX_CTAS / 2;  // SMs used at most (the workspace is sized for them)
constexpr float TR_SLACK = 8.f;   // growth of the maximum (log2) that O is not rescaled for
constexpr unsigned long long TR_TIMEOUT_NS = 1000000000ull;

template <int D>
struct Cfg {
  static constexpr bool BIG = D == 256;             // one CTA has the SM; else two share it
  static constexpr int CTAS = BIG ? 1 : 2;
  // positions of a tile.  At D = 256 score MMAs of 64 positions would read
  // more of Q than of K from shared memory, and one thread issues an MMA every 50
  // cycles or so: 128-wide ones took 109 us where 64-wide ones took 117 (61
  // nodes over 131,000 positions), and as long for few rows.
  static constexpr int TILE = BIG ? 128 : 64;
  static constexpr int CHUNKS = D / 64;             // 128-byte columns of a row
  static constexpr int ISSUERS = BIG ? 2 : 1;       // warps that issue MMAs (scores and output apart)
  // threads of a row, each with TILE / HALVES columns of S and D / HALVES of O
  // (two CTAs have no registers for more than one)
  static constexpr int HALVES = BIG ? 2 : 1;
  static constexpr int ROW_WARPS = 4 * HALVES, LOADER = ROW_WARPS, WARPS = ROW_WARPS + 1 + ISSUERS;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int OVERHEAD = 1;                // what a unit costs besides its tiles, in tiles
  // A tile of K or V takes PARTS ring slots: K by columns (CHUNKS / PARTS of
  // them, TILE rows each), V by rows (64, all columns).
  static constexpr int PARTS = TILE / 64;
  static constexpr int SLOT = 64 * D * 2, Q_CHUNK = TR_ROWS * 128, V_CHUNK = 64 * 128, K_CHUNK = TILE * 128;
  static constexpr int K_CHUNKS = CHUNKS / PARTS;   // columns of a K slot
  static constexpr int NS = D == 256 ? 5 : D == 128 ? 4 : 10;  // ring slots: what fits next to Q in 227 KB, or half of that
  static constexpr int OFF_RING = CHUNKS * Q_CHUNK;
  static constexpr int OFF_MISC = OFF_RING + NS * SLOT;
  static constexpr int SMEM = OFF_MISC + 3 * 1024;
  static_assert(SMEM * CTAS <= 227 * 1024, "shared memory");
  // Tensor memory columns: O, one S tile, two P tiles.  The rows take a whole S
  // tile into registers first thing, so that the next one's MMAs run during
  // the softmax.  (Two S tiles turned into P in place, whose MMAs had to wait for
  // the output's, took as long within 2 %: shared memory is the bound.)
  static constexpr uint32_t S_COL = D, P_COL = D + TILE, TMEM = BIG ? 512 : 256;
  static_assert(P_COL + TILE <= TMEM, "tensor memory");
};

struct TreeMaps {
  CUtensorMap q;             // {64, Hq, nodes, chunks}, boxes of G heads x nt nodes
  CUtensorMap k, v;          // {64, pool rows, chunks}: boxes of one page's rows of a slot
  CUtensorMap k_new, v_new;  // {64, nodes, chunks}: boxes of a slot
};

struct TreeArgs {
  CacheView c;
  const uint16_t *v_new;
  const int32_t *slots, *offsets, *parent;
  uint16_t *o;
  JoinArgs j;
  int B, n_nodes, max_nodes, Hq, Hkv, G;
  int nt;           // nodes of a unit
  int nt_mul, g_mul;  // 2^16 / nt + 1 and 2^16 / G + 1: x / nt = x nt_mul >> 16 for x < 2^9 (nt, G <= 128)
  int page_box;     // rows of a box (min(page, 64))
  float scale_log2;
};

struct Seq {
  int slot, L, lo, n;  // n == 0: nothing to do
};

struct Count {
  long long team, alone;  // with one row tile of a (sequence, KV head), with all
};

struct Misc {
  uint64_t full[10], empty[10];
  uint64_t q_full, q_free, s_full, s_free, p_ready[2], pv_done[2], o_free, rows_bar, pair_bar[4], final_bar;
  uint32_t tmem;
  int abort_flag, nonfinite;
  int b0;
  Seq s0;
  long long off0;
  int16_t parent[TR_MAXN];
  union {
    struct {
      Count wsum[12];
      int wrts[12];
    };
    float row[2][2][TR_ROWS];  // later: what the two threads of a row exchange, [turn][half]
  };
};
static_assert(sizeof(Misc) <= 3 * 1024, "misc area");

__device__ __forceinline__ Seq load_seq(const TreeArgs &a, int b) {
  // the loads first: none of them waits for another's check
  Seq s;
  s.slot = a.slots ? a.slots[b] : b;
  s.lo = a.offsets[b];
  const int hi = a.offsets[b + 1];
  const bool in = s.slot >= 0 && s.slot < a.c.n_slots;
  s.L = in ? slot_len(a.c, s.slot) : -1;
  s.n = hi - s.lo;
  if (s.L < 0 || s.lo < 0 || hi < s.lo || s.n > a.max_nodes || hi > a.n_nodes) {
    set_status(a.c.status, MOE_ERR_DEVICE_BOUNDS);
    s.n = s.L = s.lo = 0;
  }
  return s;
}

template <int TILE>
__device__ __forceinline__ int tiles_of(int n) {
  return (n + TILE - 1) / TILE;
}

// A sequence's count for one row tile of every KV head, and its row tiles.
template <typename C>
__device__ __forceinline__ long long seq_tiles(const TreeArgs &a, const Seq &s) {
  return s.n == 0 ? 0 : (long long)a.Hkv * (C::OVERHEAD + tiles_of<C::TILE>(s.L) + tiles_of<C::TILE>(s.n));
}
__device__ __forceinline__ int row_tiles(const TreeArgs &a, const Seq &s) {
  return (s.n + a.nt - 1) * a.nt_mul >> 16;
}

// x y / z, in 32 bits where that is enough (a 64-bit division takes hundreds of cycles).
// (its many instructions apart: a CTA's start is mostly their fetching)
__device__ __noinline__ long long div_long(long long p, long long z) { return p / z; }
__device__ __forceinline__ long long mul_div(long long x, int y, long long z) {
  const long long p = x * y;
  return (p | z) < (1ll << 31) ? (long long)((uint32_t)p / (uint32_t)z) : div_long(p, z);
}

// A CTA's walk over the units of its run.  A unit counts OVH + its tiles, the
// overhead first, so that a CTA with more units has fewer tiles.  Alone, CTAs
// cut the row of all units (sequence, KV head, row tile); in teams, a team cuts
// the row of all (sequence, KV head) and its member i has row tile i of each.
template <typename C>
struct Walk {
  static constexpr int OVH = C::OVERHEAD;
  const TreeArgs &a;
  int b;
  long long left;  // of the run, still to come
  Seq s;
  int member;      // the row tile of a team's member, -1 alone
  int g, rt, off;  // unit, and where in its count the run's part begins
  int nt_all;      // tiles of the unit
  int t0, n;       // this CTA's: the first, and how many
  bool fresh;

  __device__ Walk(const TreeArgs &a_, int b0, const Seq &s0, long long off0, long long count, int member_)
      : a(a_), b(b0), left(count), s(s0), member(member_), fresh(true) {
    nt_all = tiles_of<C::TILE>(s.L) + tiles_of<C::TILE>(s.n);
    const int rts = member < 0 ? row_tiles(a, s) : 1, u = (int)mul_div(off0, 1, OVH + nt_all);
    g = u / rts;
    rt = member < 0 ? u - g * rts : member;
    off = (int)(off0 - (long long)u * (OVH + nt_all));
  }
  // the next unit with tiles for this CTA; false when the run is done
  __device__ bool next() {
    while (left > 0) {
      if (!fresh) {
        off = 0;
        if (member >= 0 || ++rt * a.nt >= s.n) {
          rt = max(member, 0);
          if (++g >= a.Hkv) {
            g = 0;
            do {  // left > 0: a later sequence has tiles
              s = load_seq(a, ++b);
            } while (s.n == 0 && b + 1 < a.B);
            if (s.n == 0) return false;
            nt_all = tiles_of<C::TILE>(s.L) + tiles_of<C::TILE>(s.n);
          }
        }
      }
      fresh = false;
      const int take = (int)(left < OVH + nt_all - off ? left : (long long)(OVH + nt_all - off));
      left -= take;
      t0 = max(0, off - OVH);
      n = max(0, off + take - OVH) - t0;
      if (n > 0 && rt * a.nt < s.n) return true;  // a smaller tree has nothing for some members
    }
    return false;
  }
  __device__ int node0() const { return rt * a.nt; }
  __device__ int nodes() const { return min(a.nt, s.n - rt * a.nt); }
};

__device__ __forceinline__ bool tr_wait(uint64_t *bar, uint32_t parity, Misc *m, int32_t *status) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  uint32_t n = 0;
  while (!ptx::mbar_try_wait_sleep(bar, parity, 20000u)) {
    if ((++n & 7u) == 0) {
      if (*reinterpret_cast<volatile int *>(&m->abort_flag)) return false;
      if (ptx::globaltimer() - t0 > TR_TIMEOUT_NS) {
        *reinterpret_cast<volatile int *>(&m->abort_flag) = 1;
        set_status(status, MOE_ERR_DEVICE_TIMEOUT);
        return false;
      }
    }
  }
  return true;
}

// The same for a whole warp: one answer for all lanes, and the lanes together again.
__device__ __forceinline__ bool tr_wait_warp(uint64_t *bar, uint32_t parity, Misc *m, int32_t *status) {
  return __all_sync(0xffffffffu, tr_wait(bar, parity, m, status));
}

// Bounded wait used while draining after an abort.
__device__ __forceinline__ void tr_drain(uint64_t *bar, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity))
    if (ptx::globaltimer() - t0 > TR_TIMEOUT_NS) return;
}

template <bool FP16>
__device__ __forceinline__ float value(uint32_t bits) {
  if constexpr (FP16)
    return __half2float(__ushort_as_half((uint16_t)bits));
  else
    return __uint_as_float(bits << 16);
}
template <bool FP16>
constexpr uint32_t EXP_MASK = FP16 ? 0x7C00u : 0x7F80u;  // all ones: infinity or NaN

// Position of K(j) / V(j) of a unit of n tiles in the ring's load order
// K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1), PARTS slots each.
template <typename C>
__device__ __forceinline__ uint32_t k_pos(int j) {
  return C::PARTS * (j == 0 ? 0u : 2u * j - 1u);
}
template <typename C>
__device__ __forceinline__ uint32_t v_pos(int j, int n) {
  return C::PARTS * (j == n - 1 ? 2u * n - 1u : 2u * j + 2u);
}

template <int D, bool FP16>
__global__ void __launch_bounds__(Cfg<D>::THREADS, Cfg<D>::CTAS)
    tree_kernel(const __grid_constant__ TreeMaps maps, const __grid_constant__ TreeArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzled tiles want 1024
  Misc *m = reinterpret_cast<Misc *>(smem + C::OFF_MISC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the joining kernel may be scheduled now; it waits for this grid to finish
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (ptx::smem_u32(smem) & 1023u) {  // not placed as declared: no kernel then, rather than wrong tiles
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
      set_status(a.c.status, MOE_ERR_UNSUPPORTED);
      a.j.desc[blockIdx.x].parts = 0;
    }
    return;
  }
  if (warp == C::LOADER && lane == 0) {
    ptx::prefetch_tmap(&maps.q);
    ptx::prefetch_tmap(&maps.k);
    ptx::prefetch_tmap(&maps.v);
    ptx::prefetch_tmap(&maps.k_new);
    ptx::prefetch_tmap(&maps.v_new);
  }
  if (warp == C::LOADER + 1) {
    ptx::tmem_alloc(&m->tmem, C::TMEM);
    ptx::tmem_relinquish();
  }
  // what the kernel before writes (lengths, tables, rows, queries) from here on,
  // by ordinary loads: a read-only one may look at what was there before
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // This CTA's run: every thread adds up some sequences' units, a scan gives
  // their places, and the thread whose sequences hold the run's start writes
  // down where that is.
  const int per = (a.B + C::THREADS - 1) / C::THREADS, sb = min(a.B, tid * per), se = min(a.B, sb + per);
  Seq seq{0, 0, 0, 0};
  Count mine{0, 0};
  int rts = 0;  // most row tiles
  for (int b = sb; b < se; ++b) {
    seq = load_seq(a, b);
    const long long t = seq_tiles<C>(a, seq);
    mine.team += t;
    mine.alone += t * row_tiles(a, seq);
    rts = max(rts, row_tiles(a, seq));
  }
  if (tid >= 32 && tid < 32 + C::NS) {
    ptx::mbar_init(&m->full[tid - 32], 1);
    ptx::mbar_init(&m->empty[tid - 32], 1);
    ptx::fence_mbar_init();
  } else if (tid == 64) {
    m->abort_flag = 0;
    ptx::mbar_init(&m->q_full, 1);
    ptx::mbar_init(&m->q_free, 1);
    ptx::mbar_init(&m->final_bar, C::ISSUERS);
    ptx::fence_mbar_init();
  } else if (tid == 96) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&m->p_ready[i], C::ROW_WARPS);
      ptx::mbar_init(&m->pv_done[i], 1);
    }
    ptx::mbar_init(&m->s_full, 1);
    ptx::mbar_init(&m->s_free, C::ROW_WARPS);
    ptx::mbar_init(&m->o_free, C::ROW_WARPS);
    ptx::mbar_init(&m->rows_bar, C::ROW_WARPS);
    for (int i = 0; i < 4; ++i) ptx::mbar_init(&m->pair_bar[i], C::HALVES);
    ptx::fence_mbar_init();
  }
  Count inc = mine;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc.team, o), u = __shfl_up_sync(0xffffffffu, inc.alone, o);
    rts = max(rts, __shfl_xor_sync(0xffffffffu, rts, o));
    if (lane >= o) {
      inc.team += t;
      inc.alone += u;
    }
  }
  if (lane == 31) {
    m->wsum[warp] = inc;
    m->wrts[warp] = rts;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = m->tmem;
  // the warps' counts, a lane each
  Count upto = lane < C::WARPS ? m->wsum[lane] : Count{0, 0};
  rts = (int)__reduce_max_sync(0xffffffffu, lane < C::WARPS ? (unsigned)m->wrts[lane] : 0u);
#pragma unroll 1
  for (int o = 1; o < 16; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, upto.team, o), u = __shfl_up_sync(0xffffffffu, upto.alone, o);
    if (lane >= o) {
      upto.team += t;
      upto.alone += u;
    }
  }
  static_assert(C::WARPS <= 16, "four steps");
  const Count all{__shfl_sync(0xffffffffu, upto.team, 15), __shfl_sync(0xffffffffu, upto.alone, 15)};
  // Teams of one CTA a row tile read a tile of K and V at the same time, so
  // that it comes from DRAM once: 16 trees of 61 nodes over 8,000 positions each
  // (268 MB, more than L2) take 182 us alone and 108 in teams.  Not where trees of
  // different sizes would leave a fifth of the members without work.  Alone and
  // in teams, by the share of the members with work: eight trees of 61 nodes and
  // eight of 40 (7/8) 149 and 107 us, of 30 (3/4) 142 and 105, of 10 (5/8) 84 and
  // 104; over 2,000 positions, which L2 holds, 51 and 50 us (all), 49 and 48 (7/8),
  // 45.8 and 47.3 (3/4).
  const int grid = gridDim.x, cta = blockIdx.x;
  const bool teams = rts > 1 && rts <= grid && 4 * all.team * grid <= 5 * all.alone * (grid / rts);
  const int size = teams ? rts : 1;
  const long long T = teams ? all.team : all.alone;
  long long before = __shfl_sync(0xffffffffu, teams ? upto.team : upto.alone, max(warp - 1, 0));
  if (warp == 0) before = 0;
  const long long held = teams ? mine.team : mine.alone;
  before += (teams ? inc.team : inc.alone) - held;
  const int runs = (int)(T < (long long)(grid / size) ? T : (long long)(grid / size)), run = cta / size;
  if (run >= runs) {  // less to do than CTAs
    if (tid == 0) a.j.desc[cta].parts = 0;
    if (warp == C::LOADER + 1) ptx::tmem_dealloc(tmem, C::TMEM);
    return;
  }
  const long long first = mul_div(T, run, runs), end = mul_div(T, run + 1, runs);
  if (first >= before && first < before + held) {
    long long at = before;
    int b = sb;
    if (per > 1)
      for (;; ++b) {
        seq = load_seq(a, b);
        const long long t = seq_tiles<C>(a, seq) * (teams ? 1 : row_tiles(a, seq));
        if (first < at + t) break;
        at += t;
      }
    m->b0 = b;
    m->s0 = seq;
    m->off0 = first - at;
  }
  __syncthreads();
  Walk<C> w(a, m->b0, m->s0, m->off0, end - first, teams ? cta - run * size : -1);
  uint8_t *ring = smem + C::OFF_RING;
  int32_t *status = a.c.status;

  if (warp == C::LOADER) {
    // ---------------------------------------------------------------- loads
    const int pool_rows = a.c.n_pages << a.c.page_shift, in_page = (1 << a.c.page_shift) - 1;
    // boxes of a slot: this lane's rows and column of it.  A K slot of one
    // column span and a V slot go in one box where a page holds all of its rows
    // (one box a column: 61 nodes over 131,000 positions 108 us for 102, few rows the same).
    const int v_boxes = 64 / a.page_box, k_boxes = C::TILE / a.page_box;
    const bool whole = v_boxes == 1;
    const int v_box = whole ? 0 : lane / C::CHUNKS, v_chunk = whole ? 0 : lane % C::CHUNKS;
    const bool v_issues = whole ? lane == 0 : lane < v_boxes * C::CHUNKS;
    const int k_box = C::PARTS > 1 ? lane / C::K_CHUNKS : v_box, k_chunk = C::PARTS > 1 ? lane % C::K_CHUNKS : v_chunk;
    const bool k_issues = C::PARTS > 1 ? lane < k_boxes * C::K_CHUNKS : v_issues;
    const int box_bytes = a.page_box * 128;
    uint32_t ld = 0, units = 0;
    bool ok = true;
    while (ok && w.next()) {
      const int L = w.s.L, n_old = tiles_of<C::TILE>(L), x = w.g * C::CHUNKS, blocks = pages_of(L, a.c.page_shift);
      const int32_t *table = a.c.table + (size_t)w.s.slot * a.c.max_pages;
      int eb = -64, ent = 0;  // 32 table entries from block eb on, one a lane
      // the pool row of position `pos`, lane by lane, all of them in the tile
      // that begins at `base` (past the pool, read as zeros, where there is none)
      auto locate = [&](int base, int pos) {
        constexpr int SPAN = C::TILE / 16;  // blocks of a tile at most; the tile before stays in view
        const int blk0 = base >> a.c.page_shift;
        if (blk0 < eb || blk0 + SPAN > eb + 32) {
          eb = max(0, blk0 - SPAN);
          ent = eb + lane < blocks ? table[eb + lane] : -1;
          if (eb + lane < blocks && (unsigned)ent >= (unsigned)a.c.n_pages) {
            set_status(status, MOE_ERR_DEVICE_BOUNDS);
            ent = -1;
          }
        }
        const int p = __shfl_sync(0xffffffffu, ent, ((pos >> a.c.page_shift) - eb) & 31);
        return p < 0 ? pool_rows : (p << a.c.page_shift) + (pos & in_page);
      };
      // the next ring slot, its bytes announced; null if the wait gave up
      auto take_slot = [&]() -> uint8_t * {
        const uint32_t slot = ld % C::NS;
        if (!tr_wait_warp(&m->empty[slot], ((ld / C::NS) & 1u) ^ 1u, m, status)) return nullptr;
        if (lane == 0) ptx::mbar_arrive_expect_tx(&m->full[slot], C::SLOT);
        __syncwarp();
        return ring + slot * C::SLOT;
      };
      auto load_k = [&](int t) {
        for (int part = 0; part < C::PARTS; ++part) {
          uint8_t *dst = take_slot();
          if (!dst) return false;
          uint64_t *bar = &m->full[ld % C::NS];
          const int col = x + part * C::K_CHUNKS;
          if (t >= n_old) {
            if (lane == 0) ptx::tma_load_3d(dst, &maps.k_new, bar, 0, w.s.lo + (t - n_old) * C::TILE, col);
          } else {
            const int row = locate(t * C::TILE, t * C::TILE + k_box * a.page_box);
            if (k_issues)
              ptx::tma_load_3d(dst + k_chunk * C::K_CHUNK + k_box * box_bytes, &maps.k, bar, 0, row, col + k_chunk);
          }
          ++ld;
        }
        return true;
      };
      auto load_v = [&](int t) {
        for (int part = 0; part < C::PARTS; ++part) {
          uint8_t *dst = take_slot();
          if (!dst) return false;
          uint64_t *bar = &m->full[ld % C::NS];
          if (t >= n_old) {
            if (lane == 0)
              ptx::tma_load_3d(dst, &maps.v_new, bar, 0, w.s.lo + (t - n_old) * C::TILE + part * 64, x);
          } else {
            const int row = locate(t * C::TILE, t * C::TILE + part * 64 + v_box * a.page_box);
            if (v_issues)
              ptx::tma_load_3d(dst + v_chunk * C::V_CHUNK + v_box * box_bytes, &maps.v, bar, 0, row, x + v_chunk);
          }
          ++ld;
        }
        return true;
      };
      // the unit's queries, once the last unit's scores are done
      ok = units == 0 || tr_wait_warp(&m->q_free, (units - 1) & 1u, m, status);
      if (!ok) break;
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(&m->q_full, (uint32_t)(a.j.rows_cap * 128 * C::CHUNKS));
        for (int ch = 0; ch < C::CHUNKS; ++ch)
          ptx::tma_load_4d(smem + ch * C::Q_CHUNK, &maps.q, &m->q_full, 0, w.g * a.G, w.s.lo + w.node0(), ch);
      }
      ++units;
      ok = load_k(w.t0);
      for (int j = 0; ok && j < w.n; ++j) {
        if (j + 1 < w.n) ok = load_k(w.t0 + j + 1);
        ok = ok && load_v(w.t0 + j);
      }
    }
    if (!ok && lane == 0) {  // loads of the last slots may still be in flight
      if (units) tr_drain(&m->q_full, (units - 1) & 1u);
      for (uint32_t i = ld > (uint32_t)C::NS ? ld - C::NS : 0; i < ld; ++i)
        tr_drain(&m->full[i % C::NS], (i / C::NS) & 1u);
    }
  } else if (warp > C::LOADER) {
    // ----------------------------------------------------------------- MMAs
    const bool does_s = warp == C::LOADER + 1, does_o = C::ISSUERS == 1 || !does_s;
    const uint32_t id_s = ptx::idesc_f16(C::TILE, FP16, false), id_o = ptx::idesc_f16(D, FP16, true);
    const uint64_t qd = ptx::sdesc_sw128(ptx::smem_u32(smem));
    uint32_t ld = 0, units = 0, jj = 0;  // jj: running tile count
    bool ok = true;
    auto scores = [&](uint32_t pos, uint32_t t, bool first) {  // S of running tile t from the K tile at load `pos`
      if (t >= 1 && !tr_wait_warp(&m->s_free, (t - 1) & 1u, m, status)) return false;
      // (a unit's first slots may follow the last unit's V of tile t - 2)
      if (first && t >= 2 && !tr_wait_warp(&m->pv_done[t & 1], ((t - 2) >> 1) & 1u, m, status)) return false;
      const uint32_t s_col = tmem + C::S_COL;
#pragma unroll
      for (int part = 0; part < C::PARTS; ++part, ++pos) {
        const uint32_t slot = pos % C::NS;
        if (!tr_wait_warp(&m->full[slot], (pos / C::NS) & 1u, m, status)) return false;
        ptx::tc_fence_after();
        const uint64_t kd = ptx::sdesc_sw128(ptx::smem_u32(ring + slot * C::SLOT));
        if (ptx::elect_one()) {
#pragma unroll
          for (int c = 0; c < C::K_CHUNKS; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int ch = part * C::K_CHUNKS + c;
              const uint64_t b = kd + (c * C::K_CHUNK + i * 32) / 16;
              ptx::mma_ss(s_col, qd + (ch * C::Q_CHUNK + i * 32) / 16, b, id_s, (ch | i) != 0);
            }
          ptx::mma_commit(&m->empty[slot]);
          if (part == C::PARTS - 1) ptx::mma_commit(&m->s_full);
        }
        __syncwarp();
      }
      return true;
    };
    auto values = [&](uint32_t pos, uint32_t t, bool first) {  // O += P V of running tile t
      if (!tr_wait_warp(&m->p_ready[t & 1], (t >> 1) & 1u, m, status) ||
          (first && units > 0 && !tr_wait_warp(&m->o_free, (units - 1) & 1u, m, status)))
        return false;
      const uint32_t p_col = tmem + C::P_COL + (t & 1) * (C::TILE / 2);
#pragma unroll
      for (int part = 0; part < C::PARTS; ++part, ++pos) {
        const uint32_t slot = pos % C::NS;
        if (!tr_wait_warp(&m->full[slot], (pos / C::NS) & 1u, m, status)) return false;
        ptx::tc_fence_after();
        const uint64_t vd = ptx::sdesc_sw128_mn(ptx::smem_u32(ring + slot * C::SLOT), C::V_CHUNK);
        if (ptx::elect_one()) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            ptx::mma_ts(tmem, p_col + 8 * (4 * part + i), vd + i * 2048 / 16, id_o, !first || part > 0 || i > 0);
          ptx::mma_commit(&m->empty[slot]);
          if (part == C::PARTS - 1) ptx::mma_commit(&m->pv_done[t & 1]);
        }
        __syncwarp();
      }
      return true;
    };
    while (ok && w.next()) {
      if (does_s) {
        ok = tr_wait_warp(&m->q_full, units & 1u, m, status) && scores(ld + k_pos<C>(0), jj, true);
      }
      for (int j = 0; ok && j < w.n; ++j, ++jj) {
        if (does_s) {
          if (j + 1 < w.n) ok = scores(ld + k_pos<C>(j + 1), jj + 1, false);
          // the unit's last scores are under way
          if (ok && j + 1 == max(1, w.n - 1) && ptx::elect_one()) ptx::mma_commit(&m->q_free);
          __syncwarp();
        }
        if (ok && does_o) ok = values(ld + v_pos<C>(j, w.n), jj, j == 0);
      }
      ld += 2 * C::PARTS * w.n;
      ++units;
    }
    __syncwarp();
    if (ptx::elect_one()) ptx::mma_commit(&m->final_bar);  // every MMA done before tensor memory is freed
    __syncwarp();
    tr_drain(&m->final_bar, 0);
  } else {
    // ----------------------------------------------------------------- rows
    constexpr int COLS = C::TILE / C::HALVES, OCOLS = D / C::HALVES;  // this thread's columns of S and of O
    static_assert(COLS == 64, "a thread's columns of S are one word of sees[], and its P one store");
    const int r = tid & (TR_ROWS - 1), half = tid / TR_ROWS;
    const int my_node = r * a.g_mul >> 16, my_head = r - my_node * a.G;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t ld = 0, jj = 0, syncs = 0, pairs = 0;
    bool ok = true;
    SplitDesc split{};
    // one arrival a warp, for all of its lanes
    auto arrive = [&](uint64_t *bar) {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar);
    };
    auto rows_sync = [&]() {  // all row warps meet (a wait that can give up, as all others)
      arrive(&m->rows_bar);
      return tr_wait_warp(&m->rows_bar, syncs++ & 1u, m, status);
    };
    // the value of the row's other thread; the two warps meet here (two buffers
    // in turn: who writes one again has met the other's reader since)
    auto exchange = [&](float v, bool &got) {
      const uint32_t turn = pairs++ & 1u;
      m->row[turn][half][r] = v;
      arrive(&m->pair_bar[warp & 3]);
      got = tr_wait_warp(&m->pair_bar[warp & 3], turn, m, status);
      return m->row[turn][half ^ 1][r];
    };
    // The unit whose tiles were the last: its result is taken out of tensor
    // memory while the next unit's first scores run.
    struct Unit {
      int lo, nodes, node0, rows, g, n_old, t0, n, nt_all;
      long long done;  // where this CTA's part ends in the count of all
    } un{};
    float mx = -INFINITY, sum = 0.f;
    bool in = false, real = false;
    unsigned long long sees[TR_MAXN / 64] = {};
    auto finish = [&]() {
      if (!tr_wait_warp(&m->pv_done[(jj - 1) & 1], ((jj - 1) >> 1) & 1u, m, status)) return false;
      ptx::tc_fence_after();
      if constexpr (C::HALVES == 2) {
        bool got;
        sum += exchange(sum, got);
        if (!got) return false;
      }
      const bool whole = un.n == un.nt_all, starts = un.t0 == 0;
      if (!whole && starts) {
        const long long u1 = un.done - un.n + un.nt_all;  // the unit's end in the count of all
        split = SplitDesc{(int)mul_div(u1 * runs + T - 1, 1, T) - run, size, un.rows, un.lo + un.node0, un.g * a.G, {}};
      }
      // PV has ended, and with it every write of the flag
      const bool fix = un.t0 + un.n > un.n_old && *reinterpret_cast<volatile int *>(&m->nonfinite) != 0;
      const size_t pslot = (size_t)2 * cta + (starts ? 1 : 0);
      const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      if (fix) {  // into O, apart from the usual way out
#pragma unroll 1
        for (int d = half * OCOLS; d < (half + 1) * OCOLS; d += 32) {
          uint32_t v[32];
          ptx::tmem_ld_x32(lanes + d, v);
          ptx::tmem_wait_ld();
          for (int i = 0; i < un.nodes; ++i) {
            const int t = un.n_old + i / C::TILE;
            if (!real || t < un.t0 || t >= un.t0 + un.n || !(sees[i / 64] >> (i % 64) & 1)) continue;
            const uint16_t *src = a.v_new + (size_t)(un.lo + i) * a.c.row + un.g * D + d;
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              const uint32_t h = src[q];
              if ((h & EXP_MASK<FP16>) == EXP_MASK<FP16>)
                v[q] = __float_as_uint(__uint_as_float(v[q]) + value<FP16>(h));
            }
          }
          __syncwarp();
          ptx::tmem_st_x32(lanes + d, v);
        }
        ptx::tmem_wait_st();
      }
      if ((warp & 3) * 32 < un.rows) {
        uint16_t *out = a.o + ((size_t)(un.lo + un.node0 + my_node) * a.Hq + un.g * a.G + my_head) * D;
        auto put = [&](int d, uint32_t (&v)[32]) {  // columns d .. d + 31 of this row
          if (whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint4 x;
              x.x = pack2<FP16>(__uint_as_float(v[i]) * inv, __uint_as_float(v[i + 1]) * inv);
              x.y = pack2<FP16>(__uint_as_float(v[i + 2]) * inv, __uint_as_float(v[i + 3]) * inv);
              x.z = pack2<FP16>(__uint_as_float(v[i + 4]) * inv, __uint_as_float(v[i + 5]) * inv);
              x.w = pack2<FP16>(__uint_as_float(v[i + 6]) * inv, __uint_as_float(v[i + 7]) * inv);
              if (sum == 0.f) x = make_uint4(0u, 0u, 0u, 0u);  // a row that sees nothing
              *reinterpret_cast<uint4 *>(out + d + i) = x;
            }
          } else {
            uint4 *part = reinterpret_cast<uint4 *>(a.j.part) + (pslot * (D / 4) + d / 4) * a.j.rows_cap + r;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              part[i * a.j.rows_cap] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        };
#pragma unroll 1
        for (int d = half * OCOLS; d < (half + 1) * OCOLS; d += 64) {
          uint32_t v0[32], v1[32];
          __syncwarp();
          ptx::tmem_ld_x32(lanes + d, v0);
          ptx::tmem_ld_x32(lanes + d + 32, v1);
          ptx::tmem_wait_ld();
          if (in) {
            put(d, v0);
            put(d + 32, v1);
          }
        }
        if (in && !whole && half == 0)
          *reinterpret_cast<float2 *>(a.j.ml + (pslot * a.j.rows_cap + r) * 2) = make_float2(mx, sum);
      }
      ptx::tc_fence_before();
      arrive(&m->o_free);
      return true;
    };
    while (ok) {
      const bool more = w.next();
      constexpr int UPS = 2 / C::HALVES;
      int up[UPS], own = -2;  // parents of nodes tid (and tid + 128), and of this row's node
      if (more) {
        const int32_t *parent = a.parent + w.s.lo;
#pragma unroll
        for (int i = 0; i < UPS; ++i) up[i] = tid + i * TR_ROWS < w.s.n ? parent[tid + i * TR_ROWS] : -2;
        if (my_node < w.nodes()) own = parent[w.node0() + my_node];
      }
      if (un.n > 0) ok = finish();
      if (!more || !ok) break;
      const int L = w.s.L, n_old = tiles_of<C::TILE>(L);
      un = Unit{w.s.lo, w.s.n, w.node0(), w.nodes() * a.G, w.g, n_old, w.t0, w.n, w.nt_all, end - w.left};
      in = r < un.rows;
      real = in && own >= -1 && own < un.node0 + my_node;
      const bool active = (warp & 3) * 32 < un.rows;                     // the warp has rows
      const bool all_real = __all_sync(0xffffffffu, real || !in);  // none of them is padding
#pragma unroll
      for (int q = 0; q < TR_MAXN / 64; ++q) sees[q] = 0;
      mx = -INFINITY;
      sum = 0.f;
      for (int j = 0; j < un.n; ++j, ++jj) {
        const int t = un.t0 + j;
        const bool edge = t >= n_old || (t + 1) * C::TILE > L;
        if (t >= n_old && (j == 0 || t == n_old)) {
          // the first of the tree's own tiles: its parents, and what this row's node sees of each tile
          if (!(ok = rows_sync())) break;  // the last unit's readers are done
#pragma unroll
          for (int i = 0; i < UPS; ++i)
            if (tid + i * TR_ROWS < un.nodes) {
              if (up[i] >= tid + i * TR_ROWS || up[i] < -2) {
                set_status(status, MOE_ERR_DEVICE_BOUNDS);
                up[i] = -2;
              }
              m->parent[tid + i * TR_ROWS] = (int16_t)up[i];
            }
          if (tid == 0) m->nonfinite = 0;
          if (!(ok = rows_sync())) break;
          for (int i = real ? un.node0 + my_node : -1; i >= 0; i = m->parent[i]) {
            if (m->parent[i] == -2) {  // padding has no children
              set_status(status, MOE_ERR_DEVICE_BOUNDS);
              break;
            }
#pragma unroll
            for (int q = 0; q < TR_MAXN / 64; ++q)
              if (i / 64 == q) sees[q] |= 1ull << (i % 64);
          }
          __syncwarp();
        }
        if (!(ok = tr_wait_warp(&m->s_full, jj & 1u, m, status))) break;
        // Every row warp, with rows or without, is at most two tiles ahead of O: the P
        // tile of jj is free then, and no wait below or in the other roles can take
        // a phase of its barrier for the one two before.
        if (jj >= 2 && !(ok = tr_wait_warp(&m->pv_done[jj & 1], ((jj - 2) >> 1) & 1u, m, status))) break;
        ptx::tc_fence_after();
        if (edge) {
          // V rows that nobody may see become zeros (0 x NaN is NaN), and in the
          // tree's own tiles non-finite values as well: finish() adds them to
          // the rows that see them
          const uint32_t pos = ld + v_pos<C>(j, un.n);
          // the slots' last loads have been used up (else their barriers could still be a phase behind)
          if (jj >= 1) ok = tr_wait_warp(&m->pv_done[(jj - 1) & 1], ((jj - 1) >> 1) & 1u, m, status);
          for (int part = 0; ok && part < C::PARTS; ++part)
            ok = tr_wait_warp(&m->full[(pos + part) % C::NS], ((pos + part) / C::NS) & 1u, m, status);
          if (!ok) break;
          for (int e = tid; e < C::TILE * C::CHUNKS * 8; e += TR_ROWS * C::HALVES) {  // 16-byte pieces
            const int part = e / (64 * C::CHUNKS * 8), ch = e / (64 * 8) % C::CHUNKS, q = (e / 8) % 64;
            uint4 *piece = reinterpret_cast<uint4 *>(ring + (pos + part) % C::NS * C::SLOT + ch * C::V_CHUNK + q * 128 +
                                                     (e & 7) * 16);
            const int at = (t < n_old ? t : t - n_old) * C::TILE + part * 64 + q;
            const bool hold = t < n_old ? at < L : at < un.nodes && m->parent[at] != -2;
            if (!hold) {
              *piece = make_uint4(0u, 0u, 0u, 0u);
            } else if (t >= n_old) {
              uint32_t x[4] = {piece->x, piece->y, piece->z, piece->w};
              bool bad = false;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if ((x[i] & EXP_MASK<FP16>) == EXP_MASK<FP16>) x[i] &= 0xFFFF0000u, bad = true;
                if ((x[i] >> 16 & EXP_MASK<FP16>) == EXP_MASK<FP16>) x[i] &= 0x0000FFFFu, bad = true;
              }
              if (bad) {
                *piece = make_uint4(x[0], x[1], x[2], x[3]);
                m->nonfinite = 1;
              }
            }
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
        }
        if (active) {
          uint32_t x[COLS / 32][32];
#pragma unroll
          for (int h = 0; h < COLS / 32; ++h)
            ptx::tmem_ld_x32(lanes + C::S_COL + half * COLS + 32 * h, x[h]);
          ptx::tmem_wait_ld();
          ptx::tc_fence_before();
          arrive(&m->s_free);
          if (edge || !all_real) {
            unsigned long long see = 0;  // of this thread's columns
            if (real) {
              const int pos = (t < n_old ? t : t - n_old) * C::TILE + half * COLS;
              if (t < n_old) {
                const int left = L - pos;
                see = left >= 64 ? ~0ull : left <= 0 ? 0 : (1ull << left) - 1;
              } else {
#pragma unroll
                for (int q = 0; q < TR_MAXN / 64; ++q)
                  if (pos / 64 == q) see = sees[q];
              }
            }
#pragma unroll
            for (int h = 0; h < COLS / 32; ++h) {
              const uint32_t bits = (uint32_t)(see >> (32 * h));
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(bits >> i & 1)) x[h][i] = 0xFF800000u;  // -infinity
            }
          }
          float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int h = 0; h < COLS / 32; ++h)
#pragma unroll
            for (int i = 0; i < 32; ++i) t4[i & 3] = fmaxf(t4[i & 3], __uint_as_float(x[h][i]));
          float tmax = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * a.scale_log2;
          if constexpr (C::HALVES == 2) {
            tmax = fmaxf(tmax, exchange(tmax, ok));
            if (!ok) break;
          }
          const bool grows = in && tmax > mx + TR_SLACK;  // also the first score a row sees
          if (__any_sync(0xffffffffu, grows)) {
            const float f = grows ? (mx == -INFINITY ? 0.f : ex2(mx - tmax)) : 1.f;
            if (grows) mx = tmax;
            sum *= f;
            if (j > 0) {  // O holds the earlier tiles
              if (!(ok = tr_wait_warp(&m->pv_done[(jj - 1) & 1], ((jj - 1) >> 1) & 1u, m, status))) break;
              ptx::tc_fence_after();
#pragma unroll 1
              for (int d = half * OCOLS; d < (half + 1) * OCOLS; d += 32) {
                uint32_t v[32];
                ptx::tmem_ld_x32(lanes + d, v);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                ptx::tmem_st_x32(lanes + d, v);
              }
            }
          }
          // The weights are rounded to the cache's type: a tcgen05.mma takes both factors in
          // one type, and V is the cache's.  Their sum stays in fp32, unrounded.  Each
          // weight is off by half a step at most, so o by half a step of sum p|v|:
          // against 64 bits 0.0022-0.0024 (bf16) and 0.00029 (fp16) of the output's norm, with
          // fp32 weights 0.0017 and 0.00021 from the output's own rounding alone.  (Two products, of
          // the weights' upper and lower halves, would keep them at twice the MMAs for V.)
          const float base = mx == -INFINITY ? 0.f : -mx;
          uint32_t p[COLS / 2];
          float acc[4] = {};
#pragma unroll
          for (int i = 0; i < COLS; i += 2) {
            const float p0 = ex2(fmaf(__uint_as_float(x[i / 32][i % 32]), a.scale_log2, base));
            const float p1 = ex2(fmaf(__uint_as_float(x[i / 32][i % 32 + 1]), a.scale_log2, base));
            acc[i & 2] += p0;
            acc[(i & 2) + 1] += p1;
            p[i / 2] = pack2<FP16>(p0, p1);
          }
          sum += (acc[0] + acc[1]) + (acc[2] + acc[3]);
          const uint32_t p_col = lanes + C::P_COL + (jj & 1) * (C::TILE / 2) + half * (COLS / 2);
          ptx::tmem_st_x32(p_col, p);
          ptx::tmem_wait_st();
        } else {
          arrive(&m->s_free);
        }
        ptx::tc_fence_before();
        arrive(&m->p_ready[jj & 1]);
      }
      ld += 2 * C::PARTS * un.n;
    }
    if (tid == 0) a.j.desc[cta] = split;
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == C::LOADER + 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM);
  }
}

// ---------------------------------------------------------------- host

bool row_map(CUtensorMap *map, const void *p, int64_t rows, int row, int D, int box_rows, int box_chunks) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(row / 64)};
  cuuint64_t strides[2] = {(cuuint64_t)row * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_chunks};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool query_map(CUtensorMap *map, const void *p, int nodes, int Hq, int D, int G, int nt) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {64, (cuuint64_t)Hq, (cuuint64_t)nodes, (cuuint64_t)(D / 64)};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)Hq * D * 2, 128};
  cuuint32_t box[4] = {64, (cuuint32_t)G, (cuuint32_t)nt, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int tree_ctas(int D, int sms) { return (D == 256 ? 1 : 2) * (sms < TR_MAX_SMS ? sms : TR_MAX_SMS); }

int unit_nodes(int G, int max_nodes) {
  const int nt = TR_ROWS / G;
  return nt < max_nodes ? nt : max_nodes;
}

// Workspace: the split units, then maxima and sums, then partial outputs.
size_t tree_ws(int D, int ctas, int rows_cap, size_t *ml_at, size_t *part_at) {
  *ml_at = (size_t)ctas * sizeof(SplitDesc);
  *part_at = *ml_at + ((size_t)2 * ctas * rows_cap * 8 + 255) / 256 * 256;
  return *part_at + (size_t)2 * ctas * rows_cap * D * 4;
}

template <int D, bool FP16>
cudaError_t launch_tree(const TreeMaps &maps, const TreeArgs &a, int ctas, cudaStream_t s) {
  using C = Cfg<D>;
  // per device and cheap: set on every call rather than remembered
  cudaError_t e = cudaFuncSetAttribute(tree_kernel<D, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const bool chain = prof_chain(MOE_KERNEL_ATTN_TREE), quiet = prof_quiet(MOE_KERNEL_ATTN_TREE);
  prof_before(MOE_KERNEL_ATTN_TREE, s);
  e = launch_dep(chain, tree_kernel<D, FP16>, dim3(ctas), dim3(C::THREADS), C::SMEM, s, maps, a);
  prof_after(MOE_KERNEL_ATTN_TREE, s);
  if (e != cudaSuccess) return e;
  return launch_dep(quiet, join_kernel<D, FP16>, dim3(ctas * 2 / C::CTAS), dim3(JOIN_THREADS), 0, s, a.j, ctas);
}

template <bool FP16>
cudaError_t launch_tree_d(int D, const TreeMaps &maps, const TreeArgs &a, int ctas, cudaStream_t s) {
  return D == 64    ? launch_tree<64, FP16>(maps, a, ctas, s)
         : D == 128 ? launch_tree<128, FP16>(maps, a, ctas, s)
                    : launch_tree<256, FP16>(maps, a, ctas, s);
}

}  // namespace
}  // namespace moe

extern "C" size_t attn_tree_workspace_bytes(const attn_cache *c, int32_t B, int32_t n_nodes, int32_t max_nodes,
                                            int32_t Hq) {
  moe::CacheView v;
  if (moe::cache_view(c, &v) != MOE_OK || B < 1 || n_nodes < 1 || max_nodes < 1 || max_nodes > moe::TR_MAXN || Hq < 1 ||
      Hq % c->n_kv_heads || Hq / c->n_kv_heads > moe::TR_ROWS)
    return 0;
  const int G = Hq / c->n_kv_heads;
  size_t ml, part;
  return moe::tree_ws(c->head_dim, moe::tree_ctas(c->head_dim, moe::TR_MAX_SMS),
                      G * moe::unit_nodes(G, max_nodes), &ml, &part);
}

extern "C" moe_status attn_tree(const attn_cache *c, int32_t layer, const void *q_d, const void *k_new_d,
                                const void *v_new_d, const int32_t *slots_d, const int32_t *offsets_d,
                                const int32_t *parent_d, int32_t B, int32_t n_nodes, int32_t max_nodes, int32_t Hq,
                                float scale, void *ws_d, size_t ws_bytes, void *o_d, void *stream) {
  using moe::aligned16;
  moe::TreeArgs a;
  const moe_status st = moe::cache_view(c, &a.c);
  if (st != MOE_OK) return st;
  if (layer < 0 || layer >= c->n_layers || B < 0 || n_nodes < 0 || max_nodes < 1 || Hq < 1 || !(scale >= 0.f) ||
      isinf(scale))
    return MOE_ERR_INVALID_ARGUMENT;
  const int D = c->head_dim, G = Hq / c->n_kv_heads;
  if (Hq % c->n_kv_heads || G > moe::TR_ROWS || max_nodes > moe::TR_MAXN || B > moe::CACHE_MAX_SEQS)
    return MOE_ERR_UNSUPPORTED;
  if (B == 0 || n_nodes == 0) return MOE_OK;
  if (!q_d || !k_new_d || !v_new_d || !offsets_d || !parent_d || !ws_d || !o_d) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned16(q_d) || !aligned16(k_new_d) || !aligned16(v_new_d) || !aligned16(slots_d) ||
      !aligned16(offsets_d) || !aligned16(parent_d) || !aligned16(ws_d) || !aligned16(o_d))
    return MOE_ERR_MISALIGNED;
  const size_t no = (size_t)n_nodes * Hq * D * 2, nn = (size_t)n_nodes * a.c.row * 2;
  const size_t np = (size_t)c->n_layers * c->n_pages * c->page_size * a.c.row * 2;
  if (moe::ranges_meet(o_d, no, q_d, no) || moe::ranges_meet(o_d, no, k_new_d, nn) ||
      moe::ranges_meet(o_d, no, v_new_d, nn) || moe::ranges_meet(o_d, no, c->k_d, np) ||
      moe::ranges_meet(o_d, no, c->v_d, np))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws_bytes < attn_tree_workspace_bytes(c, B, n_nodes, max_nodes, Hq)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return moe::note_cuda_error(e);
  if (scale == 0.f) scale = 1.f / sqrtf((float)D);
  const int ctas = moe::tree_ctas(D, sms);
  a.v_new = static_cast<const uint16_t *>(v_new_d);
  a.slots = slots_d;
  a.offsets = offsets_d;
  a.parent = parent_d;
  a.o = static_cast<uint16_t *>(o_d);
  a.B = B;
  a.n_nodes = n_nodes;
  a.max_nodes = max_nodes;
  a.Hq = Hq;
  a.Hkv = c->n_kv_heads;
  a.G = G;
  a.nt = moe::unit_nodes(G, max_nodes);
  a.j.rows_cap = a.nt * G;
  a.nt_mul = 65536 / a.nt + 1;
  a.g_mul = 65536 / G + 1;
  a.page_box = c->page_size < 64 ? c->page_size : 64;
  a.scale_log2 = scale * 1.4426950408889634f;
  size_t ml_at, part_at;
  moe::tree_ws(D, ctas, a.j.rows_cap, &ml_at, &part_at);
  a.j.row_major = 0;
  a.j.most_groups = 8;
  a.j.o = a.o;
  a.j.Hq = Hq;
  a.j.G = G;
  a.j.desc = static_cast<moe::SplitDesc *>(ws_d);
  a.j.ml = moe::ws_ptr<float>(ws_d, ml_at);
  a.j.part = moe::ws_ptr<float>(ws_d, part_at);
  const int64_t pool_rows = (int64_t)c->n_pages * c->page_size;
  const uint16_t *k = a.c.k + (size_t)layer * pool_rows * a.c.row, *v = a.c.v + (size_t)layer * pool_rows * a.c.row;
  const bool wide = D == 256;  // K tiles of two column spans
  const int all = D / 64, boxed = a.page_box == 64 ? all : 1;  // columns of a slot, of a box
  moe::TreeMaps maps;
  if (!moe::query_map(&maps.q, q_d, n_nodes, Hq, D, G, a.nt) ||
      !moe::row_map(&maps.k, k, pool_rows, a.c.row, D, a.page_box, wide ? 1 : boxed) ||
      !moe::row_map(&maps.v, v, pool_rows, a.c.row, D, a.page_box, boxed) ||
      !moe::row_map(&maps.k_new, k_new_d, n_nodes, a.c.row, D, wide ? 128 : 64, wide ? all / 2 : all) ||
      !moe::row_map(&maps.v_new, v_new_d, n_nodes, a.c.row, D, 64, all))
    return moe::note_cuda_error(cudaErrorInvalidValue);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp16 = c->dtype == MOE_FP16;
  e = fp16 ? moe::launch_tree_d<true>(D, maps, a, ctas, s) : moe::launch_tree_d<false>(D, maps, a, ctas, s);
  return moe::note_cuda_error(e);
}
