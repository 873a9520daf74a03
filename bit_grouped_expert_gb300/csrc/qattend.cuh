// What the kernels of attention over the 8-bit paged KV cache share (qattend.cu,
// qdecode.cu): units and runs, the loading warp, bounded waits.
#pragma once
#include "attn_join.cuh"
#include "kernels.h"
#include "qcache.cuh"
#include "rotary.cuh"
#include "tc.h"
#include "tc_ptx.cuh"

namespace moe {

constexpr int QT_ROWS = 128;      // rows of a unit (MMA M)
constexpr int QT_TILE = 128;      // positions of a tile
constexpr int QT_GROUP = 16;      // positions that share scales at least (the smallest page)
constexpr int QT_MAX_SMS = JOIN_MAX_CTAS / 2;
// A row has two maxima over what it sees: m of its scores s, for the sum of its weights, and u of
// s + log2 (V scale), for what its weights are as factors of the codes:
//   l = sum 2^(s - m),   P = 2^(s + log2 (V scale) - u),   o = O 2^(u - m) / l.
// So no page takes bits from another that the row's result does not take from it.  P is cut into
// three e5m2 parts, whose range is wide: at the running maximum it is 2^6, and O is rescaled only where
// that grows by more than 2^7, so that P stays below 2^13.  (l is held the same way.)
constexpr float QT_TOP = 6.f, QT_SLACK = 7.f;
// Where units are not cut.  (One token, heads of 256, without and with it: 64 sequences of 700, 1,400, 3,000
// positions 24.7 and 19.5, 30.5 and 25.4, 45.8 and 40.8 us; one of 350 14.2 and 12.9; one of 1,400, which counts 14
// tiles more than its share, 15.0, uncut 17.7.  8 sequences' 100 rows over 1,500 41.7 and 37.8, 50 rows over 350 19.7 and 20.0.)
constexpr int QT_SPARES = 8;
constexpr unsigned long long QT_TIMEOUT_NS = 1000000000ull;

struct QMaps {
  CUtensorMap k, v;  // {ROWB, pool rows, heads * CHUNKS} bytes: boxes of one page's rows
};

struct AttendArgs {
  QCacheView q;
  const float *ks, *vs;  // the layer's scales
  const float *q_factor; // [n_rows][Hq] what a query's parts are to be multiplied by (whole matrices)
  const uint16_t *x;
  const int32_t *slots, *offsets;
  uint16_t *o;
  JoinArgs j;
  int B, n_rows, max_rows, Hq, Hkv, G;
  int nt;           // tokens of a unit
  int g_mul;        // 2^16 / G + 1: x / G = x g_mul >> 16 for x < 2^8 (G <= 128)
  int page_box;     // rows of a box (min(page, 128))
  const uint8_t *v_layer;
  float scale_log2;
};

struct QSeq {
  int slot, L, lo, n;  // n == 0: nothing to do
};

// What both kernels keep beside their tiles.
struct QShared {
  int abort_flag;
  uint32_t tmem;
  int b0;
  QSeq s0;
  long long off0;
  uint64_t q_full, o_free, final_bar;
};
template <typename C>
struct QRing : QShared {
  uint64_t k_full[C::NSK], k_empty[C::NSK], v_full[C::NSV], v_empty[C::NSV], sc_full[C::SCALES];
  float scales[C::SCALES][2][8];   // of a tile's groups: K, V
};
__device__ __forceinline__ QSeq q_load_seq(const AttendArgs &a, int b) {
  const CacheView &c = a.q.c;
  QSeq s;
  s.slot = a.slots ? a.slots[b] : b;
  s.lo = a.offsets[b];
  const int hi = a.offsets[b + 1];
  const bool in = s.slot >= 0 && s.slot < c.n_slots;
  s.L = in ? slot_len(c, s.slot) : -1;
  s.n = hi - s.lo;
  if (s.L < 0 || s.lo < 0 || hi < s.lo || s.n > a.max_rows || hi > a.n_rows) {
    set_status(c.status, MOE_ERR_DEVICE_BOUNDS);
    s.n = s.L = s.lo = 0;
  }
  return s;
}

// Positions that row tile rt's last row sees (none where that row is padding), and their tiles (one at least).
__device__ __forceinline__ int sees_of(const AttendArgs &a, const QSeq &s, int rt) {
  return max(0, s.L - s.n + min(s.n, (rt + 1) * a.nt));
}
__device__ __forceinline__ int tiles_of(const AttendArgs &a, const QSeq &s, int rt) {
  return max(1, (sees_of(a, s, rt) + QT_TILE - 1) / QT_TILE);
}
__device__ __forceinline__ int row_tiles(const AttendArgs &a, const QSeq &s) { return (s.n + a.nt - 1) / a.nt; }
// What a unit counts: its tiles and what it costs besides, or each the same (0: not).
template <typename C>
__device__ __forceinline__ int unit_count(int tiles, int each) {
  return each ? each : C::OVERHEAD + tiles;
}
// The count of a sequence's units, of one KV head.
template <typename C>
__device__ __forceinline__ long long head_count(const AttendArgs &a, const QSeq &s, int each) {
  long long t = 0;
  for (int rt = 0, rts = row_tiles(a, s); rt < rts; ++rt) t += unit_count<C>(tiles_of(a, s, rt), each);
  return t;
}

static __device__ __noinline__ long long q_div_long(long long p, long long z) { return p / z; }
__device__ __forceinline__ long long q_mul_div(long long x, int y, long long z) {
  const long long p = x * y;
  return (p | z) < (1ll << 31) ? (long long)((uint32_t)p / (uint32_t)z) : q_div_long(p, z);
}

// A CTA's run: its length (0: none) and where it ends in the count T of all units, which `runs` CTAs share.
struct QRun {
  long long count, end, T;
  int runs;
  int each;  // not 0: a unit is a run, and counts this
};

// A CTA's walk over the units of its run, in the order sequence, KV head, row
// tile.  A unit counts OVH + its tiles, the overhead first.
template <typename C>
struct QWalk {
  static constexpr int OVH = C::OVERHEAD;
  const AttendArgs &a;
  int b;
  long long left;  // of the run, still to come
  QSeq s;
  int g, rt, off;  // unit, and where in its count the run's part begins
  int nt_all;      // tiles of the unit
  int t0, n;       // this CTA's: the first, and how many
  bool fresh;
  const int each;

  __device__ QWalk(const AttendArgs &a_, int b0, const QSeq &s0, long long off0, const QRun &run)
      : a(a_), b(b0), left(run.count), s(s0), rt(0), fresh(true), each(run.each) {
    const long long head = head_count<C>(a, s, each);
    g = (int)q_mul_div(off0, 1, head);
    off0 -= g * head;
    while (off0 >= unit_count<C>(nt_all = tiles_of(a, s, rt), each)) {
      off0 -= unit_count<C>(nt_all, each);
      ++rt;
    }
    off = (int)off0;
  }
  // the next unit with tiles for this CTA; false when the run is done
  __device__ bool next() {
    while (left > 0) {
      if (!fresh) {
        off = 0;
        if (++rt * a.nt >= s.n) {
          rt = 0;
          if (++g >= a.Hkv) {
            g = 0;
            do {  // left > 0: a later sequence has tiles
              s = q_load_seq(a, ++b);
            } while (s.n == 0 && b + 1 < a.B);
            if (s.n == 0) return false;
          }
        }
        nt_all = tiles_of(a, s, rt);
      }
      fresh = false;
      const int all = unit_count<C>(nt_all, each), take = (int)(left < all - off ? left : (long long)(all - off));
      left -= take;
      t0 = max(0, off - OVH);
      n = min(nt_all, max(0, off + take - OVH)) - t0;
      if (n > 0) return true;
    }
    return false;
  }
  __device__ int token0() const { return rt * a.nt; }
  __device__ int tokens() const { return min(a.nt, s.n - rt * a.nt); }
};

__device__ __forceinline__ bool q_wait(uint64_t *bar, uint32_t parity, QShared *m, int32_t *status) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  uint32_t n = 0;
  while (!ptx::mbar_try_wait_sleep(bar, parity, 20000u)) {
    if ((++n & 7u) == 0) {
      if (*reinterpret_cast<volatile int *>(&m->abort_flag)) return false;
      if (ptx::globaltimer() - t0 > QT_TIMEOUT_NS) {
        *reinterpret_cast<volatile int *>(&m->abort_flag) = 1;
        set_status(status, MOE_ERR_DEVICE_TIMEOUT);
        return false;
      }
    }
  }
  return true;
}
// The same for a whole warp: one answer for all lanes, and the lanes together again.
__device__ __forceinline__ bool q_wait_warp(uint64_t *bar, uint32_t parity, QShared *m, int32_t *status) {
  return __all_sync(0xffffffffu, q_wait(bar, parity, m, status));
}
// Three waits at once, a lane each: a warp that finds all of them done has asked once.
__device__ __forceinline__ bool q_wait_warp(uint64_t *bar0, uint32_t parity0, uint64_t *bar1, uint32_t parity1,
                                            uint64_t *bar2, uint32_t parity2, QShared *m, int32_t *status) {
  const int which = threadIdx.x & 3;
  return q_wait_warp(which == 0 ? bar0 : which == 1 ? bar1 : bar2, which == 0 ? parity0 : which == 1 ? parity1 : parity2, m,
                     status);
}
// Bounded wait used while draining after an abort.
__device__ __forceinline__ void q_drain(uint64_t *bar, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity))
    if (ptx::globaltimer() - t0 > QT_TIMEOUT_NS) return;
}

// This CTA's run: every thread adds up some sequences' units, a scan gives
// their places, and the thread whose sequences hold the run's start writes
// down where that is.  All threads call it.
// Where there are no more units than CTAs, and the longest of them is no more than QT_SPARES
// tiles above an equal share, each is a run: the joining kernel then has nothing to do.
template <typename C, typename M>
__device__ __forceinline__ QRun find_run(const AttendArgs &a, M *m) {
  constexpr int MANY = QT_MAX_SMS + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.B + C::THREADS - 1) / C::THREADS, sb = min(a.B, tid * per), se = min(a.B, sb + per);
  QSeq seq{0, 0, 0, 0};
  long long held = 0;
  int units = 0, longest = 0;
  for (int b = sb; b < se; ++b) {
    seq = q_load_seq(a, b);
    if (seq.n == 0) continue;
    const int rts = row_tiles(a, seq);
    held += a.Hkv * head_count<C>(a, seq, 0);
    units = rts < MANY ? min(MANY, units + a.Hkv * rts) : MANY;
    longest = max(longest, C::OVERHEAD + tiles_of(a, seq, rts - 1));  // (the last rows see the most)
  }
  long long inc = held;
  int u_inc = units;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    const int u = __shfl_up_sync(0xffffffffu, u_inc, o);
    if (lane >= o) inc += t, u_inc += u;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) m->wsum[warp] = inc, m->wunits[warp] = make_int2(u_inc, longest);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  QRun run;
  long long before = inc - held;
  int u_before = u_inc - units, u_all = 0;
  run.T = 0;
  for (int w = 0; w < C::WARPS; ++w) {
    const int2 u = m->wunits[w];
    if (w < warp) before += m->wsum[w], u_before += u.x;
    run.T += m->wsum[w];
    u_all += u.x;
    longest = max(longest, u.y);
  }
  const int ctas = gridDim.x;
  run.each = u_all <= ctas && (long long)(longest - QT_SPARES) * ctas <= run.T ? longest : 0;
  if (run.each) {
    held = (long long)units * longest;
    before = (long long)u_before * longest;
    run.T = (long long)u_all * longest;
    run.runs = u_all;
  } else {
    run.runs = (int)(run.T < (long long)ctas ? run.T : (long long)ctas);
  }
  run.count = run.end = 0;
  if ((int)blockIdx.x >= run.runs) return run;
  const long long first = q_mul_div(run.T, blockIdx.x, run.runs);
  run.end = q_mul_div(run.T, blockIdx.x + 1, run.runs);
  if (first >= before && first < before + held) {
    long long at = before;
    int b = sb;
    if (per > 1)
      for (;; ++b) {
        seq = q_load_seq(a, b);
        const long long t = a.Hkv * head_count<C>(a, seq, run.each);
        if (first < at + t) break;
        at += t;
      }
    m->b0 = b;
    m->s0 = seq;
    m->off0 = first - at;
  }
  __syncthreads();
  run.count = run.end - first;
  return run;
}

// A loading warp: a unit's K tiles and the scales of K and V, or its V tiles, into their ring.
// first: what to do before the first tile of each unit (false: give up).
template <typename C, bool V, typename M, typename F>
__device__ __forceinline__ void load_tiles(const CUtensorMap *map, const AttendArgs &a, M *m, QWalk<C> &w, uint8_t *ring,
                                           F first) {
  constexpr int NS = V ? C::NSV : C::NSK;
  const CacheView &c = a.q.c;
  const int lane = threadIdx.x & 31;
  uint64_t *full = V ? m->v_full : m->k_full, *empty = V ? m->v_empty : m->k_empty;
  const int pool_rows = c.n_pages << c.page_shift, in_page = (1 << c.page_shift) - 1;
  const int boxes = QT_TILE / a.page_box;
  const bool whole = boxes == 1;  // a page holds a tile's rows: one box
  const int box = whole ? 0 : lane / C::CHUNKS, span = whole ? 0 : lane % C::CHUNKS;
  const bool issues = whole ? lane == 0 : lane < boxes * C::CHUNKS;
  const int box_at = span * C::SPAN + box * a.page_box * C::ROWB;
  uint32_t tiles = 0, units = 0;
  bool ok = true;
  while (ok && w.next()) {
    if (!(ok = first(units++))) break;
    const int z = w.g * C::CHUNKS + span, blocks = pages_of(sees_of(a, w.s, w.rt), c.page_shift);
    const int32_t *table = c.table + (size_t)w.s.slot * c.max_pages;
    // 64 table entries from block eb on, two a lane: the tile loaded next (8 blocks at most) begins in
    // the first 32, so that those fetched last are not looked at at once.
    auto entry = [&](int j) { return j < blocks ? table[j] : -1; };
    int eb = (w.t0 * QT_TILE >> c.page_shift) & ~31, ent0 = entry(eb + lane), ent1 = entry(eb + 32 + lane);
    // the page of position `pos`, lane by lane, of the tile; -1 where there is none
    auto page_at = [&](int pos) {
      const int j = (pos >> c.page_shift) - eb;
      const int p0 = __shfl_sync(0xffffffffu, ent0, j & 31), p1 = __shfl_sync(0xffffffffu, ent1, j & 31);
      const int p = j < 32 ? p0 : p1;
      if ((unsigned)p < (unsigned)c.n_pages) return p;
      if (eb + j < blocks) set_status(c.status, MOE_ERR_DEVICE_BOUNDS);
      return -1;
    };
    for (int j = 0; j < w.n; ++j, ++tiles) {
      const int t = w.t0 + j;
      if ((t * QT_TILE >> c.page_shift) >= eb + 32) {
        eb += 32;
        ent0 = ent1;
        ent1 = entry(eb + 32 + lane);
      }
      const uint32_t slot = tiles % NS;
      const int pos = t * QT_TILE + box * a.page_box, page = page_at(pos);
      if (!(ok = q_wait_warp(&empty[slot], ((tiles / NS) & 1u) ^ 1u, m, c.status))) break;
      if (lane == 0) ptx::mbar_arrive_expect_tx(&full[slot], C::SLOT);
      __syncwarp();
      // (past the pool, read as zeros, where there is no page)
      if (issues)
        ptx::tma_load_3d(ring + slot * C::SLOT + box_at, map, &full[slot], 0,
                         page < 0 ? pool_rows : (page << c.page_shift) + (pos & in_page), z);
      // The tile's scales: a lane a group, K's in the first eight lanes, V's in the next; zero where
      // there is no page.  (Straight to shared memory: a load into a register, even one
      // used a tile later, held this warp up for its latency, 0.5 us a tile.)
      if (!V) {
        const uint32_t at = tiles % C::SCALES;
        const int group = page_at(t * QT_TILE + (lane & 7) * QT_GROUP);
        if (lane < 16) {
          const float *src = (lane < 8 ? a.ks : a.vs) + (group < 0 ? 0 : (size_t)group * a.Hkv + w.g);
          ptx::cp_async_4(&m->scales[at][lane >> 3][lane & 7], src, group < 0 ? 0 : 4);
          ptx::cp_async_arrive_noinc(&m->sc_full[at]);
        }
        __syncwarp();
      }
    }
  }
  if (!V) ptx::cp_async_wait_all();
  if (!ok && lane == 0)  // loads of the last slots may still be in flight
    for (uint32_t i = tiles > (uint32_t)NS ? tiles - NS : 0; i < tiles; ++i) q_drain(&full[i % NS], (i / NS) & 1u);
}

// Two of a kind in one instruction (an issue slot for both).
__device__ __forceinline__ float2 fma_both(float x, float y, float a, float b) {  // x a + b, y a + b
  float2 r;
  asm("{\n\t.reg .b64 p, q, s;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\tmov.b64 s, {%5, %5};\n\t"
      "fma.rn.f32x2 p, p, q, s;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x), "f"(y), "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 mul_both(float2 x, float a) {
  float2 r;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(a));
  return r;
}
__device__ __forceinline__ float2 add_both(float2 x, float2 y) {
  float2 r;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tadd.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ float largest_of(float a, float b, float c) {  // (passes over NaN)
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two weights (P) in three e5m2 parts, each the nearest to what the ones before leave: as
// fp16, of which an e5m2 value is the upper byte.  Off by 2^-11 of a weight (and fp16's 2^-11), or half
// of e5m2's least step, 2^-17, which is 2^-23 of the one at the running maximum.
// The first two parts are the bytes 1 and 3 of hi and mid, the third those of lo, 0 and 1.
// (NaN leaves the first two by the addition, but not the third.)
__device__ __forceinline__ void cut_weights(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  auto upper = [](uint32_t a) { return (a + 0x00800080u) & 0xFF00FF00u; };
  auto minus = [](uint32_t a, uint32_t b) {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&d);
  };
  const uint32_t whole = half_pair<true>(x, y);
  hi = upper(whole);
  const uint32_t rest = minus(whole, hi);
  mid = upper(rest);
  const uint32_t last = minus(rest, mid);
  uint16_t codes;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(codes) : "r"(last));
  lo = codes;
}

// log2 of a page's V scale.  Always finite, so that it adds to -infinity, the score of what is not seen: zero
// as -300 (below the least scale), infinity and NaN, which only pages that no row sees may hold, as 300.
__device__ __forceinline__ float v_log2(float scale) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(fabsf(scale)));
  return fmaxf(fminf(y, 300.f), -300.f);
}

// A code that is NaN among the four of a word: 0x7F or 0xFF.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {  // 0x80 in every such byte
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// The exponent and the codes of eight values of a row, LANES lanes a row: the
// parts add up to the values times 2^-e, each being the nearest e4m3 to what the ones before leave.
template <int LANES, int PARTS>
__device__ __forceinline__ int cut_row(const float (&f)[8], uint2 (&part)[PARTS]) {
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (fabsf(f[i]) < INFINITY) most = fmaxf(most, fabsf(f[i]));
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  const int e = scale_exp(most);
  const float back = exp2_int(-e);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = f[i] * back;
    if (!(fabsf(v[i]) < INFINITY)) v[i] = NAN;  // (its rests are NaN as well)
  }
#pragma unroll
  for (int k = 0; k < PARTS; ++k) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = to_codes(v[2 * i], v[2 * i + 1]);
      const float2 got = from_codes(h[i]);
      v[2 * i] -= got.x;
      v[2 * i + 1] -= got.y;
    }
    part[k] = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  }
  return e;
}

// V of an edge's tile, in shared memory: rows that no row of the unit sees become zeros
// (0 x NaN is NaN), and among those that only some see the code NaN as well; true if there was one.
template <typename C, int THREADS>
__device__ __forceinline__ bool clear_edge(uint8_t *tile, int pos, int all_see, int some_see) {
  constexpr int PIECES = C::ROWB / 16;  // of a row in a span
  bool found = false;
  for (int e = threadIdx.x; e < QT_TILE * C::CHUNKS * PIECES; e += THREADS) {
    const int at = pos + e / PIECES % QT_TILE;
    if (at < all_see) continue;
    uint4 *piece = reinterpret_cast<uint4 *>(tile + e * 16);
    if (at >= some_see) {
      *piece = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const uint4 x = *piece;
      const uint32_t b0 = nan_codes(x.x), b1 = nan_codes(x.y), b2 = nan_codes(x.z), b3 = nan_codes(x.w);
      if (b0 | b1 | b2 | b3) {
        auto clear = [](uint32_t v, uint32_t bad) { return v & ~((bad >> 7) * 255u); };
        *piece = make_uint4(clear(x.x, b0), clear(x.y, b1), clear(x.z, b2), clear(x.w, b3));
        found = true;
      }
    }
  }
  ptx::fence_proxy_async_smem();
  return found;
}

// qdecode.cu: the kernel for units of up to QD_MOST rows.
constexpr int QD_MOST = 16;
cudaError_t launch_attend_few(int D, bool fp16, const QMaps &maps, const AttendArgs &a, int ctas, cudaStream_t s);

}  // namespace moe
