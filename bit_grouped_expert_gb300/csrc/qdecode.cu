// Attention over the 8-bit paged KV cache for few rows (qcache.h, qattend.cu): up
// to 16 rows (query heads of a KV head times tokens) a unit, as decoding has them.
// (Of more, a thread's share of the rows takes longer than it saves: 24 sequences of up to 9,000
// positions, D = 256, 16, 32, 40 rows: 39.7, 62, 74 us here, 43, 49.6, 50.2 as whole matrices.)
//
// There the matrices stand the other way up: positions, not rows, fill the
// 128 lanes of an MMA, so that a thread has one position and a share of the
// rows, and little work is repeated for rows that are not there:
//   S^T[128 positions x 3 R] = K . [Qh Qm Ql]^T    tcgen05 (e4m3), all in shared memory
//   P = 2^(S scales + log2 V scales - u)           a position's rows by two threads
//   O^T[D x 3 R]            += V^T . [Ph Pm Pl]^T  tcgen05 (e4m3 x e5m2), all in shared memory
// The parts of q (three e4m3 here, which keep fp16 whole too) and of the weights (qattend.cu)
// are columns of one product, added up where it is read: K and V go through the tensor
// cores once.
//
// A row's maxima (qattend.cuh) are spread over 128 threads, and are not needed as long as nothing
// passes a running one by 2^7: each tile the four warps that share the
// rows exchange one flag, and only where it is up they find the maxima and rescale.
// Sums stay in their threads until the unit ends.
//
// Units, runs, roles, waits and the joining kernel are qattend.cu's, with two S
// and two P buffers, and the row warps cutting the queries between units.
//
// HBM bounds it between the ends of a call and of its units: 48 tokens over up to 9,000 positions, 16 heads on 2
// of 256, bf16, 53.8 us (4.9 TB/s) with the join (6.4); 64 x 2 tokens over up to 3,000, 32 heads on 8 of 128, fp16, 58.2 us
// (3.9 TB/s); one token over 700 positions 14.4 us, latency.
#include <math.h>

#include "qattend.cuh"

namespace moe {
namespace {

// RT: rows of a thread; a unit's rows are two halves of RT.
template <int D, int RT>
struct DCfg {
  static constexpr int ROWB = D < 128 ? D : 128;    // bytes of a row in a column span
  static constexpr int CHUNKS = D / ROWB;           // column spans
  // (12 warps have 168 registers a thread, 13 would have 128)
  static constexpr int ROW_WARPS = 8, LOAD_K = 8, ISSUE_S = 9, ISSUE_O = 10, LOAD_V = 11, WARPS = 12, THREADS = WARPS * 32;
  // What a unit costs besides its tiles, in tiles (some 3 us: its first maxima, its queries, its result).  (The
  // second case above with 4, 5, 6: 60.8, 60.2, 61.0 us; the first with 2, 3, 4, 5: 55.6, 54.9, 54.9, 55.4.)
  static constexpr int OVERHEAD = D == 256 ? 3 : 5;
  static constexpr int SLOT = QT_TILE * D, SPAN = QT_TILE * ROWB;  // a tile of K or V, one column span of it
  // Rows, and columns of a product: a half's three parts side by side, so that what
  // a thread reads of S and writes of P lies together (the columns behind them are not looked at).
  static constexpr int R = 2 * RT, HALF = (3 * RT + 15) / 16 * 16, N = 2 * HALF;
  __device__ static int column(int r, int part) { return r / RT * HALF + part * RT + r % RT; }
  static constexpr int Q_SPAN = N * ROWB, P_TILE = QT_TILE * 128;
  static constexpr int NSK = D == 256 ? 2 : D == 128 ? 5 : 8, NSV = D == 256 ? 3 : NSK;  // ring slots of K, of V
  // Slots of the scales' ring.  Those of tile x are asked for when K of tile x - NSK has been
  // used up, so that all row warps have read the scores of the tile two before that: they
  // are past the scales of tile x - NSK - 3.
  static constexpr int SCALES = D == 64 ? 16 : 8;
  static_assert(SCALES >= NSK + 3, "scales");
  static constexpr int OFF_P = CHUNKS * Q_SPAN;
  static constexpr int OFF_RING = OFF_P + 2 * P_TILE;
  static constexpr int OFF_V = OFF_RING + NSK * SLOT, OFF_MISC = OFF_V + NSV * SLOT;
  static constexpr int MISC = (D == 64 ? 4 : 3) * 1024, SMEM = OFF_MISC + MISC;
  static_assert(SMEM <= 227 * 1024 && OFF_P % 1024 == 0 && OFF_RING % 1024 == 0, "shared memory");
  // Tensor memory columns: two S tiles, O of each 128 values of a head.
  static constexpr int O_TILES = D == 256 ? 2 : 1;
  static constexpr uint32_t O_COL = 2 * N, USED = (2 + O_TILES) * N;
  static constexpr uint32_t TMEM = USED <= 64 ? 64 : USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
  static_assert(USED <= 512 && RT % 4 == 0 && R % 8 == 0, "rows");
};

template <typename C, int RT>
struct DMisc : QRing<C> {
  uint64_t s_full[2], s_free[2], p_ready[2], pv_done[2], meet[2];
  int nonfinite[4];                  // by the unit's number: that unit, if NaN was taken out of its V
  __align__(16) float q_f[4][C::R];  // by the unit's number: what a row's scores are multiplied by
  // [half][warp], each warp its own: 2^6 over the running maximum, in log2; infinity before the first score
  __align__(16) float base[2][4][RT];
  __align__(16) float apart[2][4][RT];  // the same: the running maximum less that of score + log2 (V scale); 0 at first
  union {
    struct {
      long long wsum[C::WARPS];
      int2 wunits[C::WARPS];  // units, the longest
    };
    struct {                         // later: what the four warps of a half exchange
      int grows[2][2][4];            // [turn][half][warp]
      float most[2][4][RT];          // [half][warp][row]: scores
      float most_v[2][4][RT];        // with their V scales' log2
      float sums[2][4][RT];
    };
  };
};

// N columns of a warp's lanes, a multiple of 16.
template <int N>
__device__ __forceinline__ void read_columns(uint32_t taddr, uint32_t (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 16) {
    uint32_t x[16];
    ptx::tmem_ld_x16(taddr + i, x);
#pragma unroll
    for (int k = 0; k < 16; ++k) v[i + k] = x[k];
  }
}

// The sum (or maximum) over a warp's lanes of N values each, N a multiple of 4: two steps
// hand half of the values to the other lane, so that 1.5 N exchanges do instead of 5 N.
// Lane l is left with those of rows (l / 8) * N / 4 .. of N / 4.
template <int N, typename F>
__device__ __forceinline__ void fold(const float (&v)[N], float (&out)[N / 4], F op) {
  const int lane = threadIdx.x & 31;
  float h[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const bool up = lane & 16;
    const float keep = up ? v[N / 2 + i] : v[i], give = up ? v[i] : v[N / 2 + i];
    h[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, 16));
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const bool up = lane & 8;
    const float keep = up ? h[N / 4 + i] : h[i], give = up ? h[i] : h[N / 4 + i];
    out[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, 8));
#pragma unroll
    for (int o = 4; o; o >>= 1) out[i] = op(out[i], __shfl_xor_sync(0xffffffffu, out[i], o));
  }
}

// What a warp holds of a unit's queries: rows (u * warps + its own) * AT_ONCE + lane / LANES, u = 0 .. UPW - 1.
template <typename C, int D, int WARPS>
struct Queries {
  static constexpr int LANES = D / 8, AT_ONCE = 32 / LANES;
  static constexpr int UPW = (C::R + WARPS * AT_ONCE - 1) / (WARPS * AT_ONCE);
  uint4 x[UPW];
  __device__ __forceinline__ static int row(int u, int warp) {
    return (u * WARPS + warp) * AT_ONCE + (int)(threadIdx.x & 31) / LANES;
  }
  // (rows that are not there: zeros)
  __device__ __forceinline__ void load(const AttendArgs &a, const QWalk<C> &w, int warp) {
    const int rows = w.tokens() * a.G, d = (int)(threadIdx.x & 31) % LANES * 8;
#pragma unroll
    for (int u = 0; u < UPW; ++u) {
      const int r = row(u, warp), token = r * a.g_mul >> 16;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows)
        x[u] = *reinterpret_cast<const uint4 *>(
            a.x + ((size_t)(w.s.lo + w.token0() + token) * a.Hq + w.g * a.G + (r - token * a.G)) * D + d);
    }
  }
  __device__ __forceinline__ int cut(int u, int fp16, uint2 (&part)[3]) const {
    float f[8];
    if (fp16)
      unpack8<true>(x[u], f);
    else
      unpack8<false>(x[u], f);
    return cut_row<LANES, 3>(f, part);
  }
  // a row's parts to the operand's place, its factor to q_f
  __device__ __forceinline__ static void store(uint8_t *q_tile, float *q_f, int r, const uint2 (&part)[3], float factor) {
    const int d = (int)(threadIdx.x & 31) % LANES * 8;
    if (r >= C::R) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint32_t off = C::column(r, k) * C::ROWB + d % C::ROWB;
      off ^= (C::ROWB == 128 ? off >> 7 & 7 : off >> 7 & 3) << 4;
      *reinterpret_cast<uint2 *>(q_tile + d / C::ROWB * C::Q_SPAN + off) = part[k];
    }
    if (d == 0) q_f[r] = factor;
  }
};

template <int D, int RT>
__global__ void __launch_bounds__(DCfg<D, RT>::THREADS, 1)
    qdecode_kernel(const __grid_constant__ QMaps maps, const __grid_constant__ AttendArgs a, const int fp16) {
  using C = DCfg<D, RT>;
  using M = DMisc<C, RT>;
  static_assert(sizeof(M) <= C::MISC, "misc area");
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzled tiles want 1024
  M *m = reinterpret_cast<M *>(smem + C::OFF_MISC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const CacheView &c = a.q.c;
  // the joining kernel may be scheduled now; it waits for this grid to finish
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (ptx::smem_u32(smem) & 1023u) {  // not placed as declared: no kernel then, rather than wrong tiles
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
      set_status(c.status, MOE_ERR_UNSUPPORTED);
      a.j.desc[blockIdx.x].parts = 0;
    }
    return;
  }
  if (warp == C::LOAD_K && lane == 0) ptx::prefetch_tmap(&maps.k);
  if (warp == C::LOAD_V && lane == 0) ptx::prefetch_tmap(&maps.v);
  if (warp == C::ISSUE_S) {
    ptx::tmem_alloc(&m->tmem, C::TMEM);
    ptx::tmem_relinquish();
  }
  if (tid >= 32 && tid < 32 + C::NSK) {
    ptx::mbar_init(&m->k_full[tid - 32], 1);
    ptx::mbar_init(&m->k_empty[tid - 32], 1);
    ptx::fence_mbar_init();
  } else if (tid >= 48 && tid < 48 + C::NSV) {
    ptx::mbar_init(&m->v_full[tid - 48], 1);
    ptx::mbar_init(&m->v_empty[tid - 48], 1);
    ptx::fence_mbar_init();
  } else if (tid >= 64 && tid < 64 + C::SCALES) {
    ptx::mbar_init(&m->sc_full[tid - 64], 16);
    ptx::fence_mbar_init();
  } else if (tid >= 128 && tid < 128 + 8 * RT) {
    m->base[0][0][tid - 128] = INFINITY;
    m->apart[0][0][tid - 128] = 0.f;
  } else if (tid == 96) {
    m->abort_flag = 0;
    ptx::mbar_init(&m->q_full, C::ROW_WARPS);
    ptx::mbar_init(&m->final_bar, 2);
    ptx::mbar_init(&m->o_free, C::ROW_WARPS);
    for (int i = 0; i < 4; ++i) m->nonfinite[i] = -1;
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&m->p_ready[i], C::ROW_WARPS);
      ptx::mbar_init(&m->pv_done[i], 1);
      ptx::mbar_init(&m->s_full[i], 1);
      ptx::mbar_init(&m->s_free[i], C::ROW_WARPS);
      ptx::mbar_init(&m->meet[i], 4);
    }
    ptx::fence_mbar_init();
  }
  // what the kernel before writes (lengths, tables, codes, scales, queries) from here on,
  // by ordinary loads: a read-only one may look at what was there before
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const QRun run = find_run<C>(a, m);
  const uint32_t tmem = m->tmem;
  const int cta = blockIdx.x;
  if (run.count == 0) {  // less to do than CTAs
    if (tid == 0) a.j.desc[cta].parts = 0;
    if (warp == C::ISSUE_S) ptx::tmem_dealloc(tmem, C::TMEM);
    return;
  }
  QWalk<C> w(a, m->b0, m->s0, m->off0, run);
  uint8_t *k_ring = smem + C::OFF_RING, *v_ring = smem + C::OFF_V, *p_tiles = smem + C::OFF_P;
  int32_t *status = c.status;

  if (warp == C::LOAD_K) {
    load_tiles<C, false>(&maps.k, a, m, w, k_ring, [](uint32_t) { return true; });
  } else if (warp == C::LOAD_V) {
    load_tiles<C, true>(&maps.v, a, m, w, v_ring, [](uint32_t) { return true; });
  } else if (warp == C::ISSUE_S || warp == C::ISSUE_O) {
    // ----------------------------------------------------------------- MMAs
    const bool does_s = warp == C::ISSUE_S;
    const uint32_t id_s = ptx::idesc_f8(C::N, false, false, false, false), id_o = ptx::idesc_f8(C::N, false, true, true, true);
    const uint64_t qd = ptx::sdesc_rows(ptx::smem_u32(smem), C::ROWB, 16);
    uint32_t units = 0, jj = 0;  // jj: running tile count
    bool ok = true;
    auto scores = [&](uint32_t t) {  // S^T of running tile t
      const uint32_t slot = t % C::NSK;
      if ((t >= 2 && !q_wait_warp(&m->s_free[t & 1], ((t - 2) >> 1) & 1u, m, status)) ||
          !q_wait_warp(&m->k_full[slot], (t / C::NSK) & 1u, m, status))
        return false;
      ptx::tc_fence_after();
      const uint64_t kd = ptx::sdesc_rows(ptx::smem_u32(k_ring + slot * C::SLOT), C::ROWB, 16);
      if (ptx::elect_one()) {
#pragma unroll
        for (int ch = 0; ch < C::CHUNKS; ++ch)
#pragma unroll
          for (int i = 0; i < C::ROWB / 32; ++i)
            ptx::mma_ss_f8(tmem + (t & 1) * C::N, kd + (ch * C::SPAN + i * 32) / 16,
                             qd + (ch * C::Q_SPAN + i * 32) / 16, id_s, (ch | i) != 0);
        ptx::mma_commit(&m->k_empty[slot]);
        ptx::mma_commit(&m->s_full[t & 1]);
      }
      __syncwarp();
      return true;
    };
    auto values = [&](uint32_t t, bool first) {  // O^T += V^T P^T of running tile t
      const uint32_t slot = t % C::NSV;
      if (!q_wait_warp(&m->p_ready[t & 1], (t >> 1) & 1u, m, status) ||
          (first && units > 0 && !q_wait_warp(&m->o_free, (units - 1) & 1u, m, status)) ||
          !q_wait_warp(&m->v_full[slot], (t / C::NSV) & 1u, m, status))
        return false;
      ptx::tc_fence_after();
      const uint64_t pd = ptx::sdesc_rows(ptx::smem_u32(p_tiles + (t & 1) * C::P_TILE), 128, 16);  // a position's weights a row
      // (heads of 64 values: the product's upper 64 rows are the lower ones again)
      const uint64_t vd = ptx::sdesc_rows(ptx::smem_u32(v_ring + slot * C::SLOT), C::ROWB, D == 64 ? 0 : C::SPAN);
      if (ptx::elect_one()) {
#pragma unroll
        for (int ot = 0; ot < C::O_TILES; ++ot)
#pragma unroll
          for (int i = 0; i < QT_TILE / 32; ++i)
            ptx::mma_ss_f8(tmem + C::O_COL + ot * C::N, vd + (ot * C::SPAN + i * 32 * C::ROWB) / 16,
                           pd + i * 32 * 128 / 16, id_o, !first || i > 0);
        ptx::mma_commit(&m->v_empty[slot]);
        ptx::mma_commit(&m->pv_done[t & 1]);
      }
      __syncwarp();
      return true;
    };
    while (ok && w.next()) {
      if (does_s) ok = q_wait_warp(&m->q_full, units & 1u, m, status) && scores(jj);
      for (int j = 0; ok && j < w.n; ++j, ++jj) {
        if (!does_s)
          ok = values(jj, j == 0);
        else if (j + 1 < w.n)
          ok = scores(jj + 1);
      }
      ++units;
    }
    __syncwarp();
    if (ptx::elect_one()) ptx::mma_commit(&m->final_bar);  // every MMA done before tensor memory is freed
    __syncwarp();
    q_drain(&m->final_bar, 0);
  } else {
    // ----------------------------------------------------------------- rows
    const int half = warp >> 2, quad = warp & 3, at = quad * 32 + lane;  // this thread's position of a tile, value of O
    const int r0 = half * RT;                                            // its first row
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + half * C::HALF;
    uint32_t jj = 0, meets = 0;
    int units = 0;
    bool ok = true;
    SplitDesc split{};
    // one arrival a warp, for all of its lanes
    auto arrive = [&](uint64_t *bar) {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar);
    };
    auto meet = [&]() {  // the half's four warps (a wait that can give up, as all others)
      arrive(&m->meet[half]);
      return q_wait_warp(&m->meet[half], meets++ & 1u, m, status);
    };
    struct Unit {
      int slot, lo, token0, rows, g, t0, n, nt_all;
      int pos0;               // position of its first token
      int all_see, some_see;  // positions that all of its rows see, that its last one does
      long long done;         // where this CTA's part ends in the count of all
    } un{};
    float sum[RT];
    // the sum of a row's three parts
    auto three = [](const uint32_t(&v)[C::HALF], int i) {
      return (__uint_as_float(v[i]) + __uint_as_float(v[RT + i])) + __uint_as_float(v[2 * RT + i]);
    };
    // The unit's result out of tensor memory, while the next unit's first scores run.
    auto finish = [&]() {
      const bool whole = un.n == un.nt_all, starts = un.t0 == 0;
      const size_t pslot = (size_t)2 * cta + (starts ? 1 : 0);
      // sums over the half's positions
      float mine4[RT / 4];
      fold(sum, mine4, [](float x, float y) { return x + y; });
      if ((lane & 7) == 0)
#pragma unroll
        for (int i = 0; i < RT / 4; ++i) m->sums[half][quad][lane / 8 * (RT / 4) + i] = mine4[i];
      if (!meet()) return false;
#pragma unroll
      for (int i = 0; i < RT; ++i)
        sum[i] = (m->sums[half][0][i] + m->sums[half][1][i]) + (m->sums[half][2][i] + m->sums[half][3][i]);
      float by[RT];  // what the rows of O are to be multiplied by
#pragma unroll
      for (int i = 0; i < RT; ++i) by[i] = ex2(-m->apart[half][quad][i]) * (whole ? 1.f / sum[i] : 1.f);
      __syncwarp();
      if (lane < RT) {  // the maxima: to the joining kernel, and from the start for the next unit
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < RT; ++i)
          if (i == lane) mine = sum[i];
        if (quad == 0 && !whole && r0 + lane < un.rows)
          *reinterpret_cast<float2 *>(a.j.ml + (pslot * a.j.rows_cap + r0 + lane) * 2) =
              make_float2(QT_TOP - m->base[half][quad][lane], mine);
        m->base[half][quad][lane] = INFINITY;
        m->apart[half][quad][lane] = 0.f;
      }
      __syncwarp();
      if (!q_wait_warp(&m->pv_done[(jj - 1) & 1], ((jj - 1) >> 1) & 1u, m, status)) return false;
      ptx::tc_fence_after();
      if (!whole && starts) {
        const long long u1 = un.done - un.n + un.nt_all;  // the unit's end in the count of all
        const int ends = (int)q_mul_div(u1 * run.runs + run.T - 1, 1, run.T);
        split = SplitDesc{ends - cta, 1, un.rows, un.lo + un.token0, un.g * a.G, {}};
      }
      // PV has ended, and with it every write of the flag
      const bool fix = *reinterpret_cast<volatile int *>(&m->nonfinite[(units - 1) & 3]) == units - 1;
#pragma unroll 1
      for (int ot = 0; ot < C::O_TILES; ++ot) {
        const int d = ot * 128 + at;
        uint32_t v[C::HALF];
        __syncwarp();
        read_columns(lanes + C::O_COL + ot * C::N, v);
        ptx::tmem_wait_ld();
        if (D == 64 && at >= 64) continue;
        float o[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) o[i] = three(v, i) * by[i];
        if (fix) {  // codes NaN that were taken out of the edge's tiles, for the rows that see them
          const int p1 = min(un.some_see, (un.t0 + un.n) * QT_TILE);
          const int32_t *table = c.table + (size_t)un.slot * c.max_pages;
          for (int p = max(un.all_see, un.t0 * QT_TILE); p < p1; ++p) {
            const unsigned page = (unsigned)table[p >> c.page_shift];
            if (page >= (unsigned)c.n_pages) continue;
            const uint8_t code =
                a.v_layer[((((size_t)page << c.page_shift) + (p & ((1 << c.page_shift) - 1))) * a.Hkv + un.g) * D + d];
            if ((code & 0x7F) != 0x7F) continue;
#pragma unroll
            for (int i = 0; i < RT; ++i)
              if (p <= un.pos0 + ((r0 + i) * a.g_mul >> 16)) o[i] = NAN;
          }
        }
        uint16_t *out = a.o + ((size_t)(un.lo + un.token0) * a.Hq + un.g * a.G) * D + d;
        float *part = a.j.part + pslot * a.j.rows_cap * D + d;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const int r = r0 + i, token = r * a.g_mul >> 16;
          if (r >= un.rows) continue;
          if (whole) {
            const float y = sum[i] == 0.f ? 0.f : o[i];
            out[((size_t)token * a.Hq + (r - token * a.G)) * D] =
                fp16 ? __half_as_ushort(__float2half_rn(y)) : f32_to_bf16(y);
          } else {
            part[(size_t)r * D] = o[i];
          }
        }
      }
      ptx::tc_fence_before();
      arrive(&m->o_free);
      return true;
    };
    using Q = Queries<C, D, C::ROW_WARPS>;
    auto cut_queries = [&](const Q &q, int unit) {
#pragma unroll
      for (int u = 0; u < Q::UPW; ++u) {
        uint2 part[3];
        const int e = q.cut(u, fp16, part);
        Q::store(smem, m->q_f[unit & 3], Q::row(u, warp), part, exp2_int(e) * a.scale_log2);
      }
      ptx::fence_proxy_async_smem();
      arrive(&m->q_full);
    };
    bool more = w.next();
    if (more) {
      Q q;
      q.load(a, w, warp);
      cut_queries(q, 0);
    }
    while (ok && more) {
      const int pos0 = w.s.L - w.s.n + w.token0();
      un = Unit{w.s.slot, w.s.lo, w.token0(), w.tokens() * a.G, w.g, w.t0, w.n, w.nt_all, pos0, 0, 0, run.end - w.left};
      un.all_see = max(0, pos0 + 1);
      un.some_see = max(0, pos0 + w.tokens());
      more = w.next();  // the unit behind this one
#pragma unroll
      for (int i = 0; i < RT; ++i) sum[i] = 0.f;
      for (int j = 0; j < un.n; ++j, ++jj) {
        const int t = un.t0 + j;
        const bool edge = (t + 1) * QT_TILE > un.all_see;
        // The scores are there; the P tile of jj is free, so that no wait below or in the other
        // roles can take a phase of its barrier for the one two before (the first two
        // tiles' barrier is a phase behind: asked for the one before its first, it says yes); the
        // scales are there (this warp has waited for the slot's phase before, SCALES tiles ago).
        if (!(ok = q_wait_warp(&m->s_full[jj & 1], (jj >> 1) & 1u, &m->pv_done[jj & 1], ((jj >> 1) & 1u) ^ 1u,
                               &m->sc_full[jj % C::SCALES], (jj / C::SCALES) & 1u, m, status)))
          break;
        ptx::tc_fence_after();
        if (edge) {
          // (codes NaN that are taken out: finish() puts them where they belong)
          const uint32_t slot = jj % C::NSV;
          // (the slot's last load, of tile jj - 3 or before, has been used up: its phase has passed)
          static_assert(C::NSV >= 3, "V slots");
          if (!(ok = q_wait_warp(&m->v_full[slot], (jj / C::NSV) & 1u, m, status))) break;
          if (clear_edge<C, C::ROW_WARPS * 32>(v_ring + slot * C::SLOT, t * QT_TILE, un.all_see, un.some_see))
            m->nonfinite[units & 3] = units;
          __syncwarp();
        }
        const float(*sc)[8] = m->scales[jj % C::SCALES];
        const float ks = sc[0][at / QT_GROUP], vl = v_log2(sc[1][at / QT_GROUP]);
        // this position's scores; they and, with the V scale, the weights' exponents over the running maxima
        float s[RT], x[RT], y[RT];
        {
          uint32_t v[C::HALF];
          read_columns(lanes + (jj & 1) * C::N, v);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < RT; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(&m->q_f[units & 3][r0 + i]);
            const float qf[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) s[i + k] = three(v, i + k) * (qf[k] * ks);
          }
        }
        ptx::tc_fence_before();
        arrive(&m->s_free[jj & 1]);
        // The unit's scores are done: the next one's queries may go to their place, so
        // that its first scores run during this one's end.
        if (j == un.n - 1 && more) {
          Q q;
          q.load(a, w, warp);
          cut_queries(q, units + 1);
        }
        if (edge) {
          const int first = pos0 - (t * QT_TILE + at);  // row r sees the position if -first <= its token
#pragma unroll
          for (int i = 0; i < RT; ++i)
            if (r0 + i >= un.rows || first + ((r0 + i) * a.g_mul >> 16) < 0) s[i] = -INFINITY;
        }
        // (infinite where the maxima are still to be found)
        bool grows = false;
        auto over_maximum = [&]() {
          float most = -INFINITY;
#pragma unroll
          for (int i = 0; i < RT; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(&m->base[half][quad][i]);
            const float4 h = *reinterpret_cast<const float4 *>(&m->apart[half][quad][i]);
            const float base[4] = {f.x, f.y, f.z, f.w}, apart[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[i + k] = s[i + k] + base[k];
              y[i + k] = x[i + k] + (vl + apart[k]);
            }
          }
          if (edge)
#pragma unroll
            for (int i = 0; i < RT; ++i)
              if (s[i] == -INFINITY) x[i] = y[i] = -INFINITY;  // (and not NaN before the first score)
#pragma unroll
          for (int i = 0; i < RT; ++i) most = largest_of(most, x[i], y[i]);
          grows |= most > QT_TOP + QT_SLACK;
        };
        over_maximum();
        grows = __any_sync(0xffffffffu, grows);
        const uint32_t turn = jj & 1u;
        if (lane == 0) m->grows[turn][half][quad] = grows;
        if (!(ok = meet())) break;
        {
          const volatile int *f = m->grows[turn][half];
          grows = (f[0] | f[1] | f[2] | f[3]) != 0;
        }
        float f[RT];  // what O's earlier tiles are to be multiplied by
        if (grows) {
          float mine4[RT / 4], mine4_v[RT / 4];
          auto larger = [](float x, float y) { return fmaxf(x, y); };
          fold(s, mine4, larger);
#pragma unroll
          for (int i = 0; i < RT; ++i) y[i] = s[i] + vl;
          fold(y, mine4_v, larger);
          if ((lane & 7) == 0)
#pragma unroll
            for (int i = 0; i < RT / 4; ++i) {
              m->most[half][quad][lane / 8 * (RT / 4) + i] = mine4[i];
              m->most_v[half][quad][lane / 8 * (RT / 4) + i] = mine4_v[i];
            }
          if (!(ok = meet())) break;
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            auto of_four = [i, half](const float(&v)[2][4][RT]) {
              return fmaxf(fmaxf(v[half][0][i], v[half][1][i]), fmaxf(v[half][2][i], v[half][3][i]));
            };
            const float most = of_four(m->most), most_v = of_four(m->most_v);
            const float was = m->base[half][quad][i], apart = m->apart[half][quad][i];
            // (of a row that has seen nothing yet: any score)
            const bool up = most > -INFINITY && most + was > QT_TOP + QT_SLACK;
            const bool wider = most_v > -INFINITY && most_v + was + apart > QT_TOP + QT_SLACK;
            const float mx = up ? most : QT_TOP - was;
            if (up) sum[i] *= ex2(QT_TOP - most - was);
            f[i] = wider ? ex2(QT_TOP - was - most_v - apart) : 1.f;
            x[i] = up ? QT_TOP - most : was;
            // (the other maximum stays where it is: this one's growth comes to what is between them)
            y[i] = wider ? mx - most_v : up ? apart + (most - (QT_TOP - was)) : apart;
          }
          // (the exchanged maxima are written again after the next tile's meeting at the earliest)
          __syncwarp();
          if (lane == 0)
#pragma unroll
            for (int i = 0; i < RT; ++i) m->base[half][quad][i] = x[i], m->apart[half][quad][i] = y[i];
          __syncwarp();
          over_maximum();
        }
        // the weights: this position's row of the tile, a byte a row and part
        uint32_t p_row[C::HALF / 4] = {};
#pragma unroll
        for (int i = 0; i < RT; i += 4) {
          float p[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sum[i + k] += ex2(x[i + k]);
            p[k] = ex2(y[i + k]);
          }
          uint32_t h0, m0, l0, h1, m1, l1;
          cut_weights(p[0], p[1], h0, m0, l0);
          cut_weights(p[2], p[3], h1, m1, l1);
          p_row[i / 4] = __byte_perm(h0, h1, 0x7531);
          p_row[(RT + i) / 4] = __byte_perm(m0, m1, 0x7531);
          p_row[(2 * RT + i) / 4] = __byte_perm(l0, l1, 0x5410);
        }
        uint8_t *p_tile = p_tiles + (jj & 1) * C::P_TILE + at * 128;
#pragma unroll
        for (int i = 0; i < C::HALF; i += 16)
          *reinterpret_cast<uint4 *>(p_tile + ((half * C::HALF + i) ^ (at & 7) << 4)) =
              make_uint4(p_row[i / 4], p_row[i / 4 + 1], p_row[i / 4 + 2], p_row[i / 4 + 3]);
        // O, once the product with the tile before is done (the weights are made meanwhile)
        if (grows && j > 0) {
          if (!(ok = q_wait_warp(&m->pv_done[(jj - 1) & 1], ((jj - 1) >> 1) & 1u, m, status))) break;
          ptx::tc_fence_after();
#pragma unroll 1
          for (int ot = 0; ot < C::O_TILES; ++ot) {
            const uint32_t col = lanes + C::O_COL + ot * C::N;
            uint32_t v[C::HALF];
            read_columns(col, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 3 * RT; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f[i % RT]);
#pragma unroll
            for (int i = 0; i < C::HALF; i += 16) {
              uint32_t y[16];
#pragma unroll
              for (int q = 0; q < 16; ++q) y[q] = v[i + q];
              ptx::tmem_st_x16(col + i, y);
            }
          }
          ptx::tmem_wait_st();
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        arrive(&m->p_ready[jj & 1]);
      }
      ++units;
      if (ok) ok = finish();
    }
    if (tid == 0) a.j.desc[cta] = split;
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == C::ISSUE_S) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM);
  }
}

template <int D, int RT>
cudaError_t launch_few(bool fp16, const QMaps &maps, const AttendArgs &a, int ctas, cudaStream_t s) {
  using C = DCfg<D, RT>;
  // per device and cheap: set on every call rather than remembered
  cudaError_t e = cudaFuncSetAttribute(qdecode_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const bool chain = prof_chain(MOE_KERNEL_ATTN_QCACHE);
  prof_before(MOE_KERNEL_ATTN_QCACHE, s);
  e = launch_dep(chain, qdecode_kernel<D, RT>, dim3(ctas), dim3(C::THREADS), C::SMEM, s, maps, a, (int)fp16);
  prof_after(MOE_KERNEL_ATTN_QCACHE, s);
  return e;
}

template <int D>
cudaError_t launch_few_d(bool fp16, const QMaps &maps, const AttendArgs &a, int ctas, cudaStream_t s) {
  // (up to 8 rows as 16: one token over 700 positions 17.2 us for 15.4, 48 over up to 9,000 58.4 for 55.5, 64 over up
  // to 3,000 of 8 heads of 128 81 for 63)
  return a.j.rows_cap <= 8 ? launch_few<D, 4>(fp16, maps, a, ctas, s) : launch_few<D, 8>(fp16, maps, a, ctas, s);
}

}  // namespace

cudaError_t launch_attend_few(int D, bool fp16, const QMaps &maps, const AttendArgs &a, int ctas, cudaStream_t s) {
  return D == 64    ? launch_few_d<64>(fp16, maps, a, ctas, s)
         : D == 128 ? launch_few_d<128>(fp16, maps, a, ctas, s)
                    : launch_few_d<256>(fp16, maps, a, ctas, s);
}

}  // namespace moe
