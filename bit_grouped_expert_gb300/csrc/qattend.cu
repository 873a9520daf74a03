// Attention over the 8-bit paged KV cache (qcache.h).
//
// The query heads of a KV head and the last rows of a sequence together make the
// rows of one matrix (row = token * G + head), so that a K or V tile read once
// serves all of them.  The codes are matrix operands as they lie in the pages:
// per tile of 128 positions
//   S[128 rows x 128] = (Qh + Ql) . K^T          tcgen05 (e4m3), K in shared memory
//   P = 2^(S scales + log2 V scales - u)         two threads a row, running maxima and sum
//   O[128 rows x D]  += (Ph + Pm + Pl) . V       tcgen05 (e5m2 x e4m3), P in tensor memory, V in shared memory
// An MMA over 8-bit values runs twice as fast as one over 16-bit ones, so that
// factors may be sums of 8-bit parts, each the nearest to what the ones before leave:
//   q times a power of two that takes its row's largest value to 224 .. 448 is two e4m3
//   parts of bf16, three of fp16: to 2^-9 (2^-14) of every value, which is to say whole, or
//   to 2^-10, 2^-18 of the row's largest;
//   the weights P are three e5m2 parts, to 2^-11 of each or 2^-23 of the one at the
//   running maximum.  (Two e4m3 parts keep 2^-9 of the large ones, but their range is
//   small: O had to be rescaled wherever a maximum grew by more than 2^1.75, most
//   tiles of 32 rows.)
// A page's K scale multiplies its columns of S, its V scale its columns of P, which are taken
// relative to the largest that the row sees (qattend.cuh), so that O stays one sum of one unit.
//
// A unit is (sequence, KV head, up to 128 rows); its tiles are the positions
// that its last row sees.  All units' tiles, in a row, are cut into one equal run
// per CTA, whatever the lengths: a unit that spans CTAs leaves partial results
// (m, l, O in fp32), which a second kernel joins (attn_join.cuh).
//
// Roles: eight warps own the rows, two load (TMA: pages by the table's numbers, K
// with the pages' scales and V, each into a ring of its own), two issue the MMAs
// of S (of the next tile during the softmax of this one) and of O.  The queries' parts
// are made beforehand, by a kernel of their own, so that they come as they are needed, by
// TMA.  (Four warps that cut the next unit's took 12 us for 128 rows.)  Who waits on a
// barrier's parity must know that the phase before has passed: the comments at the waits say from what.
//
// A tile of 128 rows, heads of 256, bf16, is 1,024 cycles of MMA for S and 1,536 for O; the rows
// take 3,100 to 3,600 and bound it, K and V are there in time.  4 sequences' 500 rows over 8,000
// positions, 16 heads on 2: 171 to 178 us with the cut (8.5) and the join (13.5), 1,020 TFLOP/s and more; 5 rows over
// 131,000 positions 45.5 us, 2.9 TB/s.  (Sixteen row warps of 96 registers: 220 and 53.7 us where these
// eight took 215 and 50.3.)
//
// Every wait is bounded: after one second the kernel records
// MOE_ERR_DEVICE_TIMEOUT, drains its copies and MMAs, frees tensor memory
// and exits.
#include <math.h>

#include "qattend.cuh"

namespace moe {
namespace {

// PARTS: e4m3 parts of a query, 2 for bf16, 3 for fp16.
template <int D, int PARTS>
struct QCfg {
  static constexpr int ROWB = D < 128 ? D : 128;    // bytes of a row in a column span
  static constexpr int CHUNKS = D / ROWB;           // column spans
  static constexpr int ROW_WARPS = 8, LOAD_K = 8, ISSUE_S = 9, ISSUE_O = 10, LOAD_V = 11;
  static constexpr int WARPS = 12, THREADS = WARPS * 32;  // (168 registers a thread at most)
  // What a unit costs besides its tiles, in tiles.  (4 prompts' 500 rows over 8,000 positions, heads of 256, with
  // 3, 4, 5, 6: 174, 171.5, 172.5, 173.5 us; 20 of 80 over 4,000, heads of 128: 66.0, 67.6, 67.1, 68.9.)
  static constexpr int OVERHEAD = D == 256 ? 4 : 3;
  static constexpr int SLOT = QT_TILE * D, SPAN = QT_TILE * ROWB;  // a tile of K or V, one column span of it
  static constexpr int Q_SPAN = QT_ROWS * ROWB, Q_PART = CHUNKS * Q_SPAN;
  static constexpr int NSK = D == 256 ? 2 : D == 128 ? 5 : 8, NSV = D == 256 ? 5 - PARTS : NSK;  // ring slots of K, of V
  // Slots of the scales' ring.  Those of tile x are asked for when K of tile x - NSK has been
  // used up, which was after all row warps had read the scores of the tile before: they are past
  // the scales of tile x - NSK - 2.
  static constexpr int SCALES = D == 256 ? 4 : D == 128 ? 8 : 16;
  static_assert(SCALES >= NSK + 2, "scales");
  static constexpr int OFF_RING = PARTS * Q_PART;
  static constexpr int OFF_V = OFF_RING + NSK * SLOT, OFF_MISC = OFF_V + NSV * SLOT;
  static constexpr int SMEM = OFF_MISC + (D == 256 ? 3 : 4) * 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  // Tensor memory columns: O, one S tile, one P tile of three parts, four weights a
  // column.  The rows take a whole S tile into registers first thing, so that the next one's
  // MMAs run during the softmax, and write P last thing, when the product with the one
  // before is done.  (Two tiles, each first S and then P, made the scores of a tile wait for the
  // product of two before: 2.2 us a tile of 128 rows where this took 1.75.)
  static constexpr uint32_t S_COL = D, P_COL = D + QT_TILE, P_PART = QT_TILE / 4, TMEM = 512;
  static_assert(P_COL + 3 * P_PART <= TMEM, "tensor memory");
};

template <typename C>
struct QMisc : QRing<C> {
  uint64_t q_free, s_full, s_free, p_ready, pv_done, pair_bar[4];
  int nonfinite[4];                // by the unit's number: that unit, if NaN was taken out of its V
  union {
    struct {
      long long wsum[C::WARPS];
      int2 wunits[C::WARPS];  // units, the longest
    };
    float row[2][2][QT_ROWS];      // later: what the two threads of a row exchange, [turn][half]
  };
};
static_assert(sizeof(QMisc<QCfg<256, 2>>) <= 3 * 1024 && sizeof(QMisc<QCfg<128, 2>>) <= 4 * 1024 &&
                  sizeof(QMisc<QCfg<64, 2>>) <= 4 * 1024,
              "misc area");

template <int D, bool FP16>
__global__ void __launch_bounds__(QCfg<D, 2>::THREADS, 1)
    qattend_kernel(const __grid_constant__ QMaps maps, const __grid_constant__ CUtensorMap q_map,
                   const __grid_constant__ AttendArgs a) {
  constexpr int PARTS = FP16 ? 3 : 2;
  using C = QCfg<D, PARTS>;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzled tiles want 1024
  QMisc<C> *m = reinterpret_cast<QMisc<C> *>(smem + C::OFF_MISC);
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
  if (warp == C::LOAD_V && lane == 0) {
    ptx::prefetch_tmap(&maps.v);
    ptx::prefetch_tmap(&q_map);
  }
  if (warp == C::ISSUE_S) {
    ptx::tmem_alloc(&m->tmem, C::TMEM);
    ptx::tmem_relinquish();
  }
  if (tid >= 32 && tid < 32 + C::SCALES) {
    ptx::mbar_init(&m->sc_full[tid - 32], 16);
    ptx::fence_mbar_init();
  } else if (tid >= 128 && tid < 128 + C::NSK) {
    ptx::mbar_init(&m->k_full[tid - 128], 1);
    ptx::mbar_init(&m->k_empty[tid - 128], 1);
    ptx::fence_mbar_init();
  } else if (tid >= 160 && tid < 160 + C::NSV) {
    ptx::mbar_init(&m->v_full[tid - 160], 1);
    ptx::mbar_init(&m->v_empty[tid - 160], 1);
    ptx::fence_mbar_init();
  } else if (tid == 64) {
    m->abort_flag = 0;
    for (int i = 0; i < 4; ++i) m->nonfinite[i] = -1;
    ptx::mbar_init(&m->q_full, 1);
    ptx::mbar_init(&m->q_free, 1);
    ptx::mbar_init(&m->final_bar, 2);
    ptx::fence_mbar_init();
  } else if (tid == 96) {
    ptx::mbar_init(&m->p_ready, C::ROW_WARPS);
    ptx::mbar_init(&m->pv_done, 1);
    ptx::mbar_init(&m->s_full, 1);
    ptx::mbar_init(&m->s_free, C::ROW_WARPS);
    ptx::mbar_init(&m->o_free, C::ROW_WARPS);
    for (int i = 0; i < 4; ++i) ptx::mbar_init(&m->pair_bar[i], 2);
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
  uint8_t *k_ring = smem + C::OFF_RING, *v_ring = smem + C::OFF_V;
  int32_t *status = c.status;

  if (warp == C::LOAD_K) {
    load_tiles<C, false>(&maps.k, a, m, w, k_ring, [](uint32_t) { return true; });
  } else if (warp == C::LOAD_V) {
    // a unit's queries, all parts, when the last unit's scores are done; then its V tiles
    uint32_t issued = 0;
    load_tiles<C, true>(&maps.v, a, m, w, v_ring, [&](uint32_t units) {
      if (units > 0 && !q_wait_warp(&m->q_free, (units - 1) & 1u, m, status)) return false;
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(&m->q_full, (uint32_t)(a.j.rows_cap * PARTS * D));
        for (int ch = 0; ch < PARTS * C::CHUNKS; ++ch)
          ptx::tma_load_4d(smem + ch * C::Q_SPAN, &q_map, &m->q_full, 0, w.g * a.G, w.s.lo + w.token0(), ch);
      }
      __syncwarp();
      ++issued;
      return true;
    });
    if (lane == 0 && issued > 0) q_drain(&m->q_full, (issued - 1) & 1u);  // none on its way when the CTA ends
  } else if (warp == C::ISSUE_S || warp == C::ISSUE_O) {
    // ----------------------------------------------------------------- MMAs
    const bool does_s = warp == C::ISSUE_S;
    const uint32_t id_s = ptx::idesc_f8(QT_TILE, false, false, false, false), id_o = ptx::idesc_f8(D, true, false, false, true);
    const uint64_t qd = ptx::sdesc_rows(ptx::smem_u32(smem), C::ROWB, 16);
    uint32_t units = 0, jj = 0;  // jj: running tile count
    bool ok = true;
    auto scores = [&](uint32_t t) {  // S of running tile t
      const uint32_t slot = t % C::NSK;
      if ((t >= 1 && !q_wait_warp(&m->s_free, (t - 1) & 1u, m, status)) ||
          !q_wait_warp(&m->k_full[slot], (t / C::NSK) & 1u, m, status))
        return false;
      ptx::tc_fence_after();
      const uint64_t kd = ptx::sdesc_rows(ptx::smem_u32(k_ring + slot * C::SLOT), C::ROWB, 16);
      if (ptx::elect_one()) {
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
          for (int ch = 0; ch < C::CHUNKS; ++ch)
#pragma unroll
            for (int i = 0; i < C::ROWB / 32; ++i)
              ptx::mma_ss_f8(tmem + C::S_COL, qd + (part * C::Q_PART + ch * C::Q_SPAN + i * 32) / 16,
                               kd + (ch * C::SPAN + i * 32) / 16, id_s, (part | ch | i) != 0);
        ptx::mma_commit(&m->k_empty[slot]);
        ptx::mma_commit(&m->s_full);
      }
      __syncwarp();
      return true;
    };
    auto values = [&](uint32_t t, bool first) {  // O += P V of running tile t
      const uint32_t slot = t % C::NSV;
      if (!q_wait_warp(&m->p_ready, t & 1u, m, status) ||
          (first && units > 0 && !q_wait_warp(&m->o_free, (units - 1) & 1u, m, status)) ||
          !q_wait_warp(&m->v_full[slot], (t / C::NSV) & 1u, m, status))
        return false;
      ptx::tc_fence_after();
      const uint32_t p_col = tmem + C::P_COL;
      const uint64_t vd = ptx::sdesc_rows(ptx::smem_u32(v_ring + slot * C::SLOT), C::ROWB, C::SPAN);
      if (ptx::elect_one()) {
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int i = 0; i < QT_TILE / 32; ++i)
            ptx::mma_ts_f8(tmem, p_col + part * C::P_PART + 8 * i, vd + i * 32 * C::ROWB / 16, id_o,
                             !first || part > 0 || i > 0);
        ptx::mma_commit(&m->v_empty[slot]);
        ptx::mma_commit(&m->pv_done);
      }
      __syncwarp();
      return true;
    };
    while (ok && w.next()) {
      if (does_s) ok = q_wait_warp(&m->q_full, units & 1u, m, status) && scores(jj);
      for (int j = 0; ok && j < w.n; ++j, ++jj) {
        if (does_s) {
          if (j + 1 < w.n) ok = scores(jj + 1);
          // the unit's last scores are under way
          if (ok && j + 1 == max(1, w.n - 1) && ptx::elect_one()) ptx::mma_commit(&m->q_free);
          __syncwarp();
        } else {
          ok = values(jj, j == 0);
        }
      }
      ++units;
    }
    __syncwarp();
    if (ptx::elect_one()) ptx::mma_commit(&m->final_bar);  // every MMA done before tensor memory is freed
    __syncwarp();
    q_drain(&m->final_bar, 0);
  } else {
    // ----------------------------------------------------------------- rows
    constexpr int COLS = QT_TILE / 2, OCOLS = D / 2;  // this thread's columns of S and of O
    const int r = tid & (QT_ROWS - 1), half = tid / QT_ROWS;
    const int my_token = r * a.g_mul >> 16, my_head = r - my_token * a.G;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t jj = 0, pairs = 0;
    int units = 0;
    bool ok = true;
    SplitDesc split{};
    // one arrival a warp, for all of its lanes
    auto arrive = [&](uint64_t *bar) {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar);
    };
    // the value of the row's other thread; the two warps meet here (two buffers
    // in turn: who writes one again has met the other's reader since)
    auto exchange = [&](float v, bool &got) {
      const uint32_t turn = pairs++ & 1u;
      m->row[turn][half][r] = v;
      arrive(&m->pair_bar[warp & 3]);
      got = q_wait_warp(&m->pair_bar[warp & 3], turn, m, status);
      return m->row[turn][half ^ 1][r];
    };
    // The unit whose tiles were the last: its result is taken out of tensor
    // memory while the next unit's first scores run.
    struct Unit {
      int slot, lo, token0, rows, g, t0, n, nt_all;
      int all_see, some_see;  // positions that all of its rows see, that its last one does
      long long done;         // where this CTA's part ends in the count of all
    } un{};
    // of this thread's half of the positions the largest score and the sum, of the row the largest score + log2 (V scale)
    float mx = -INFINITY, sum = 0.f, most = -INFINITY;
    bool in = false;
    int own = -1;  // the last position that this row sees
    auto finish = [&]() {
      if (!q_wait_warp(&m->pv_done, (jj - 1) & 1u, m, status)) return false;
      ptx::tc_fence_after();
      // the halves' maxima and sums to the row's (a half that saw nothing has the sum 0; NaN stays)
      bool got;
      const float row_mx = fmaxf(mx, exchange(mx, got));
      if (!got) return false;
      if (mx != row_mx) sum *= exp2f(mx - row_mx);
      sum += exchange(sum, got);
      if (!got) return false;
      const float o_unit = most == -INFINITY ? 0.f : exp2f(most - row_mx);  // what a one in O is
      const bool whole = un.n == un.nt_all, starts = un.t0 == 0;
      if (!whole && starts) {
        const long long u1 = un.done - un.n + un.nt_all;  // the unit's end in the count of all
        const int ends = (int)q_mul_div(u1 * run.runs + run.T - 1, 1, run.T);
        split = SplitDesc{ends - cta, 1, un.rows, un.lo + un.token0, un.g * a.G, {}};
      }
      // PV has ended, and with it every write of the flag
      const bool fix = *reinterpret_cast<volatile int *>(&m->nonfinite[(units - 1) & 3]) == units - 1;
      const size_t pslot = (size_t)2 * cta + (starts ? 1 : 0);
      const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      if (fix) {  // NaN into O, apart from the usual way out: codes that were taken out of the edge's tiles
        const int p0 = max(un.all_see, un.t0 * QT_TILE), p1 = min(un.some_see, (un.t0 + un.n) * QT_TILE);
        const int32_t *table = c.table + (size_t)un.slot * c.max_pages;
#pragma unroll 1
        for (int d = half * OCOLS; d < (half + 1) * OCOLS; d += 32) {
          uint32_t v[32];
          __syncwarp();
          ptx::tmem_ld_x32(lanes + d, v);
          ptx::tmem_wait_ld();
          for (int p = p0; p < p1; ++p) {
            const unsigned page = (unsigned)table[p >> c.page_shift];
            if (!in || p > own || page >= (unsigned)c.n_pages) continue;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(
                a.v_layer + ((((size_t)page << c.page_shift) + (p & ((1 << c.page_shift) - 1))) * a.Hkv + un.g) * D + d);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const uint32_t bad = nan_codes(src[q]);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (bad >> (8 * k + 7) & 1) v[4 * q + k] = 0x7FC00000u;
            }
          }
          __syncwarp();
          ptx::tmem_st_x32(lanes + d, v);
        }
        ptx::tmem_wait_st();
      }
      if ((warp & 3) * 32 < un.rows) {
        uint16_t *out = a.o + ((size_t)(un.lo + un.token0 + my_token) * a.Hq + un.g * a.G + my_head) * D;
        const float f = whole ? o_unit * inv : o_unit;
        auto put = [&](int d, uint32_t (&v)[32]) {  // columns d .. d + 31 of this row
          if (whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              float y[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = sum == 0.f ? 0.f : __uint_as_float(v[i + k]) * f;
              *reinterpret_cast<uint4 *>(out + d + i) = pack8<FP16>(y);
            }
          } else {
            float4 *part = reinterpret_cast<float4 *>(a.j.part) + (pslot * (D / 4) + d / 4) * a.j.rows_cap + r;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              part[i * a.j.rows_cap] =
                  make_float4(__uint_as_float(v[4 * i]) * f, __uint_as_float(v[4 * i + 1]) * f,
                              __uint_as_float(v[4 * i + 2]) * f, __uint_as_float(v[4 * i + 3]) * f);
          }
        };
#pragma unroll 1
        for (int d = half * OCOLS; d < (half + 1) * OCOLS; d += 32) {
          uint32_t v[32];
          __syncwarp();
          ptx::tmem_ld_x32(lanes + d, v);
          ptx::tmem_wait_ld();
          if (in) put(d, v);
        }
        if (in && !whole && half == 0)
          *reinterpret_cast<float2 *>(a.j.ml + (pslot * a.j.rows_cap + r) * 2) = make_float2(row_mx, sum);
      }
      ptx::tc_fence_before();
      arrive(&m->o_free);
      return true;
    };
    while (ok) {
      const bool more = w.next();
      if (un.n > 0) ok = finish();
      if (!more || !ok) break;
      un = Unit{w.s.slot, w.s.lo, w.token0(), w.tokens() * a.G, w.g, w.t0, w.n, w.nt_all, 0, 0, run.end - w.left};
      const int pos0 = w.s.L - w.s.n + un.token0;  // of the first token
      un.all_see = max(0, pos0 + 1);
      un.some_see = max(0, pos0 + w.tokens());
      in = r < un.rows;
      own = in ? pos0 + my_token : -1;
      const bool active = (warp & 3) * 32 < un.rows;  // the warp has rows
      mx = most = -INFINITY;
      sum = 0.f;
      const float q_scale =
          in ? a.q_factor[(size_t)(un.lo + un.token0 + my_token) * a.Hq + un.g * a.G + my_head] * a.scale_log2 : 0.f;
      for (int j = 0; j < un.n; ++j, ++jj) {
        const int t = un.t0 + j;
        const bool edge = (t + 1) * QT_TILE > un.all_see;
        // The scores are there, and the scales (this warp has waited for their slot's phase before, SCALES tiles ago).
        if (!(ok = q_wait_warp(&m->s_full, jj & 1u, &m->sc_full[jj % C::SCALES], (jj / C::SCALES) & 1u, &m->s_full, jj & 1u,
                               m, status)))
          break;
        ptx::tc_fence_after();
        if (edge) {
          // (codes NaN that are taken out: finish() puts them where they belong)
          const uint32_t slot = jj % C::NSV;
          // (the slot's last load, of tile jj - 2 or before, has been used up: this warp has waited for the product)
          static_assert(C::NSV >= 2, "V slots");
          if (!(ok = q_wait_warp(&m->v_full[slot], (jj / C::NSV) & 1u, m, status))) break;
          if (clear_edge<C, QT_ROWS * 2>(v_ring + slot * C::SLOT, t * QT_TILE, un.all_see, un.some_see))
            m->nonfinite[units & 3] = units;
          __syncwarp();
        }
        if (active) {
          uint32_t x[COLS / 32][32];
          const uint32_t s_col = lanes + C::S_COL;
#pragma unroll
          for (int h = 0; h < COLS / 32; ++h) ptx::tmem_ld_x32(s_col + half * COLS + 32 * h, x[h]);
          ptx::tmem_wait_ld();
          ptx::tc_fence_before();
          arrive(&m->s_free);
          if (edge) {
            const int left = own - t * QT_TILE - half * COLS + 1;  // of this thread's columns
#pragma unroll
            for (int i = 0; i < COLS; ++i)
              if (i >= left) x[i / 32][i % 32] = 0xFF800000u;  // -infinity
          }
          const float(*sc)[8] = m->scales[jj % C::SCALES];
          float kf[COLS / QT_GROUP], vl[COLS / QT_GROUP], tmax = -INFINITY, umax = -INFINITY;
#pragma unroll
          for (int g = 0; g < COLS / QT_GROUP; ++g) {
            // (not zero: it multiplies -infinity; and a scale of zero leaves scores of next to nothing)
            kf[g] = fmaxf(q_scale * sc[0][half * (COLS / QT_GROUP) + g], 1e-37f);
            float two[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < QT_GROUP; i += 2)
              two[i / 2 & 1] = largest_of(two[i / 2 & 1], __uint_as_float(x[g / 2][g % 2 * QT_GROUP + i]),
                                          __uint_as_float(x[g / 2][g % 2 * QT_GROUP + i + 1]));
            const float s = fmaxf(two[0], two[1]) * kf[g];
            vl[g] = v_log2(sc[1][half * (COLS / QT_GROUP) + g]);
            tmax = fmaxf(tmax, s);
            umax = fmaxf(umax, s + vl[g]);
          }
          umax = fmaxf(umax, exchange(umax, ok));
          if (!ok) break;
          // (also the first a row sees)
          const bool grows = in && tmax > mx + QT_SLACK, wider = in && umax > most + QT_SLACK;
          const bool rescales = __any_sync(0xffffffffu, wider);
          float o_f = 1.f;  // what O's earlier tiles are to be multiplied by
          if (grows) {
            sum *= mx == -INFINITY ? 0.f : exp2f(mx - tmax);
            mx = tmax;
          }
          if (wider) {
            o_f = most == -INFINITY ? 0.f : exp2f(most - umax);
            most = umax;
          }
          const float base = QT_TOP - (mx == -INFINITY ? 0.f : mx), apart = mx == -INFINITY ? 0.f : mx - most;
          uint32_t part[3][COLS / 4];
          float2 acc[2] = {};
#pragma unroll
          for (int i = 0; i < COLS; i += 4) {
            // (finite also for scales that this row does not see: it multiplies their weights, zeros)
            const float vf = ex2(fminf(vl[i / QT_GROUP] + apart, 127.f));
            float2 p[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              p[k] = fma_both(__uint_as_float(x[i / 32][i % 32 + 2 * k]), __uint_as_float(x[i / 32][i % 32 + 2 * k + 1]),
                              kf[i / QT_GROUP], base);
              p[k] = make_float2(ex2(p[k].x), ex2(p[k].y));
              acc[k] = add_both(acc[k], p[k]);
              p[k] = mul_both(p[k], vf);
            }
            uint32_t h0, m0, l0, h1, m1, l1;
            cut_weights(p[0].x, p[0].y, h0, m0, l0);
            cut_weights(p[1].x, p[1].y, h1, m1, l1);
            part[0][i / 4] = __byte_perm(h0, h1, 0x7531);
            part[1][i / 4] = __byte_perm(m0, m1, 0x7531);
            part[2][i / 4] = __byte_perm(l0, l1, 0x5410);
          }
          sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
          // the product with the tile before is done: its P has been used up, and O may be changed
          // (Here, not where the maximum is found, which is to wait for the product before the weights are made:
          // 181 us for 215 in the case above, whose heads of large scores rescale in most tiles.)
          if (jj >= 1 && !(ok = q_wait_warp(&m->pv_done, (jj - 1) & 1u, m, status))) break;
          ptx::tc_fence_after();
          if (rescales && j > 0) {
#pragma unroll 1
            for (int d = half * OCOLS; d < (half + 1) * OCOLS; d += 32) {
              uint32_t v[32];
              ptx::tmem_ld_x32(lanes + d, v);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * o_f);
              ptx::tmem_st_x32(lanes + d, v);
            }
          }
#pragma unroll
          for (int k = 0; k < 3; ++k) ptx::tmem_st_x16(lanes + C::P_COL + k * C::P_PART + half * (COLS / 4), part[k]);
          ptx::tmem_wait_st();
        } else {
          arrive(&m->s_free);
          // (as the others: who is ahead of the product by two would take a phase of p_ready for the one before)
          if (jj >= 1 && !(ok = q_wait_warp(&m->pv_done, (jj - 1) & 1u, m, status))) break;
        }
        ptx::tc_fence_before();
        arrive(&m->p_ready);
      }
      ++units;
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

// Parts and factors of all queries: [row][head][part][D], a few heads a warp.
template <int D, bool FP16>
__global__ void __launch_bounds__(256) cut_queries_kernel(const uint16_t *x, uint8_t *parts, float *factor, int n) {
  constexpr int LANES = D / 8, AT_ONCE = 32 / LANES, PARTS = FP16 ? 3 : 2;
  start_dependent();
  const int lane = threadIdx.x & 31, d = lane % LANES * 8;
  for (int r0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * AT_ONCE; r0 < n; r0 += gridDim.x * 8 * AT_ONCE) {
    const int r = r0 + lane / LANES;
    float f[8] = {};
    if (r < n) unpack8<FP16>(*reinterpret_cast<const uint4 *>(x + (size_t)r * D + d), f);
    uint2 part[PARTS];
    const int e = cut_row<LANES, PARTS>(f, part);
    if (r >= n) continue;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) *reinterpret_cast<uint2 *>(parts + ((size_t)r * PARTS + k) * D + d) = part[k];
    if (d == 0) factor[r] = exp2_int(e);
  }
}

// ---------------------------------------------------------------- host

// A unit's queries: boxes of G heads x nt tokens of one column span of a part.
bool parts_map(CUtensorMap *map, const void *p, int rows, int Hq, int D, int parts, int G, int nt) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const int rowb = D < 128 ? D : 128;
  cuuint64_t dims[4] = {(cuuint64_t)rowb, (cuuint64_t)Hq, (cuuint64_t)rows, (cuuint64_t)(parts * D / rowb)};
  cuuint64_t strides[3] = {(cuuint64_t)parts * D, (cuuint64_t)Hq * parts * D, (cuuint64_t)rowb};
  cuuint32_t box[4] = {(cuuint32_t)rowb, (cuuint32_t)G, (cuuint32_t)nt, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, rowb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool code_map(CUtensorMap *map, const void *p, int64_t rows, int heads, int D, int box_rows, int box_spans) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const int rowb = D < 128 ? D : 128;
  cuuint64_t dims[3] = {(cuuint64_t)rowb, (cuuint64_t)rows, (cuuint64_t)(heads * (D / rowb))};
  cuuint64_t strides[2] = {(cuuint64_t)heads * D, (cuuint64_t)rowb};
  cuuint32_t box[3] = {(cuuint32_t)rowb, (cuuint32_t)box_rows, (cuuint32_t)box_spans};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, rowb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             D == 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
             : D == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                        : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,  // no more than the row: the next head is another's
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int attend_ctas(int sms) { return sms < QT_MAX_SMS ? sms : QT_MAX_SMS; }

int unit_tokens(int G, int max_rows) {
  const int nt = QT_ROWS / G;
  return nt < max_rows ? nt : max_rows;
}

// Workspace: the split units, then maxima and sums, then partial outputs; for whole
// matrices also the queries' parts and factors.
struct AttendSpace {
  size_t ml, part, q_parts, q_factor, all;
};
AttendSpace attend_ws(int D, int ctas, int rows_cap, int64_t q_rows) {
  AttendSpace w;
  w.ml = (size_t)ctas * sizeof(SplitDesc);
  w.part = w.ml + ((size_t)2 * ctas * rows_cap * 8 + 255) / 256 * 256;
  w.q_parts = w.all = w.part + (size_t)2 * ctas * rows_cap * D * 4;
  w.q_factor = w.q_parts + (size_t)q_rows * 3 * D;  // (bf16 takes two parts)
  if (rows_cap > QD_MOST) w.all = w.q_factor + (size_t)q_rows * 4;
  return w;
}

template <int D, bool FP16>
cudaError_t launch_rows(const QMaps &maps, const AttendArgs &a, void *q_parts, float *q_factor, int ctas, cudaStream_t s) {
  constexpr int PARTS = FP16 ? 3 : 2;
  using C = QCfg<D, PARTS>;
  CUtensorMap q_map;
  if (!parts_map(&q_map, q_parts, a.n_rows, a.Hq, D, PARTS, a.G, a.nt)) return cudaErrorInvalidValue;
  // per device and cheap: set on every call rather than remembered
  cudaError_t e = cudaFuncSetAttribute(qattend_kernel<D, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const int n = a.n_rows * a.Hq, need = (n + 8 * (256 / D) - 1) / (8 * (256 / D));
  e = launch_dep(prof_chain(0), cut_queries_kernel<D, FP16>, dim3(need < 152 * 8 ? need : 152 * 8), dim3(256), 0, s, a.x,
                 static_cast<uint8_t *>(q_parts), q_factor, n);
  if (e != cudaSuccess) return e;
  const bool pdl = prof_quiet(MOE_KERNEL_ATTN_QCACHE);
  prof_before(MOE_KERNEL_ATTN_QCACHE, s);
  e = launch_dep(pdl, qattend_kernel<D, FP16>, dim3(ctas), dim3(C::THREADS), C::SMEM, s, maps, q_map, a);
  prof_after(MOE_KERNEL_ATTN_QCACHE, s);
  return e;
}

template <bool FP16>
cudaError_t launch_attend(int D, const QMaps &maps, const AttendArgs &a, void *q_parts, float *q_factor, int ctas,
                          cudaStream_t s) {
  const bool quiet = prof_quiet(MOE_KERNEL_ATTN_QCACHE);
  const cudaError_t e = a.j.rows_cap <= QD_MOST ? launch_attend_few(D, FP16, maps, a, ctas, s)
                        : D == 64               ? launch_rows<64, FP16>(maps, a, q_parts, q_factor, ctas, s)
                        : D == 128              ? launch_rows<128, FP16>(maps, a, q_parts, q_factor, ctas, s)
                                                : launch_rows<256, FP16>(maps, a, q_parts, q_factor, ctas, s);
  if (e != cudaSuccess) return e;
  auto join = D == 64 ? join_kernel<64, FP16> : D == 128 ? join_kernel<128, FP16> : join_kernel<256, FP16>;
  return launch_dep(quiet, join, dim3(ctas * 2), dim3(JOIN_THREADS), 0, s, a.j, ctas);
}

}  // namespace
}  // namespace moe

extern "C" size_t attn_qcache_attend_workspace_bytes(const attn_qcache *c, int32_t B, int32_t n_rows, int32_t max_rows,
                                                     int32_t Hq) {
  moe::QCacheView v;
  if (moe::qcache_view(c, &v) != MOE_OK || B < 1 || B > moe::CACHE_MAX_SEQS || n_rows < 1 || max_rows < 1 || Hq < 1 ||
      Hq % c->n_kv_heads || Hq / c->n_kv_heads > moe::QT_ROWS)
    return 0;
  const int G = Hq / c->n_kv_heads;
  return moe::attend_ws(c->head_dim, moe::attend_ctas(moe::QT_MAX_SMS), G * moe::unit_tokens(G, max_rows),
                        (int64_t)n_rows * Hq).all;
}

extern "C" moe_status attn_qcache_attend(const attn_qcache *c, int32_t layer, const void *q_d, int32_t dtype,
                                         const int32_t *slots_d, const int32_t *offsets_d, int32_t B, int32_t n_rows,
                                         int32_t max_rows, int32_t Hq, float scale, void *ws_d, size_t ws_bytes,
                                         void *o_d, void *stream) {
  using moe::aligned16;
  moe::AttendArgs a;
  const moe_status st = moe::qcache_view(c, &a.q);
  if (st != MOE_OK) return st;
  if (layer < 0 || layer >= c->n_layers || B < 0 || n_rows < 0 || max_rows < 1 || Hq < 1 || !(scale >= 0.f) ||
      isinf(scale))
    return MOE_ERR_INVALID_ARGUMENT;
  const int D = c->head_dim, G = Hq / c->n_kv_heads;
  if (Hq % c->n_kv_heads || G > moe::QT_ROWS || B > moe::CACHE_MAX_SEQS || (dtype != MOE_BF16 && dtype != MOE_FP16))
    return MOE_ERR_UNSUPPORTED;
  if (B == 0 || n_rows == 0) return MOE_OK;
  if (!q_d || !offsets_d || !ws_d || !o_d) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned16(q_d) || !aligned16(slots_d) || !aligned16(offsets_d) || !aligned16(ws_d) || !aligned16(o_d))
    return MOE_ERR_MISALIGNED;
  if ((int64_t)n_rows * Hq > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  const size_t no = (size_t)n_rows * Hq * D * 2;
  const int64_t pool_rows = (int64_t)c->n_pages * c->page_size;
  const size_t layer_bytes = (size_t)pool_rows * c->n_kv_heads * D, np = c->n_layers * layer_bytes;
  const size_t ns = (size_t)c->n_layers * c->n_pages * c->n_kv_heads * 4;
  if (moe::ranges_meet(o_d, no, q_d, no) || moe::ranges_meet(o_d, no, c->k_d, np) ||
      moe::ranges_meet(o_d, no, c->v_d, np) || moe::ranges_meet(o_d, no, c->k_scale_d, ns) ||
      moe::ranges_meet(o_d, no, c->v_scale_d, ns))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws_bytes < attn_qcache_attend_workspace_bytes(c, B, n_rows, max_rows, Hq)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return moe::note_cuda_error(e);
  if (scale == 0.f) scale = 1.f / sqrtf((float)D);
  const int ctas = moe::attend_ctas(sms);
  const size_t scales_at = (size_t)layer * c->n_pages * c->n_kv_heads;
  a.ks = a.q.ks + scales_at;
  a.vs = a.q.vs + scales_at;
  a.x = static_cast<const uint16_t *>(q_d);
  a.slots = slots_d;
  a.offsets = offsets_d;
  a.o = static_cast<uint16_t *>(o_d);
  a.B = B;
  a.n_rows = n_rows;
  a.max_rows = max_rows;
  a.Hq = Hq;
  a.Hkv = c->n_kv_heads;
  a.G = G;
  a.nt = moe::unit_tokens(G, max_rows);
  a.g_mul = 65536 / G + 1;
  a.page_box = c->page_size < moe::QT_TILE ? c->page_size : moe::QT_TILE;
  const uint8_t *k = static_cast<const uint8_t *>(c->k_d) + layer * layer_bytes;
  a.v_layer = static_cast<const uint8_t *>(c->v_d) + layer * layer_bytes;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.j.rows_cap = a.nt * G;
  const moe::AttendSpace w = moe::attend_ws(D, ctas, a.j.rows_cap, (int64_t)n_rows * Hq);
  a.j.desc = static_cast<moe::SplitDesc *>(ws_d);
  a.j.ml = moe::ws_ptr<float>(ws_d, w.ml);
  a.j.part = moe::ws_ptr<float>(ws_d, w.part);
  void *q_parts = moe::ws_ptr<uint8_t>(ws_d, w.q_parts);
  float *q_factor = moe::ws_ptr<float>(ws_d, w.q_factor);
  a.q_factor = q_factor;
  a.j.row_major = a.j.rows_cap <= moe::QD_MOST;
  a.j.most_groups = 32;
  a.j.o = a.o;
  a.j.Hq = Hq;
  a.j.G = G;
  const int spans = a.page_box == moe::QT_TILE && D == 256 ? 2 : 1;
  moe::QMaps maps;
  if (!moe::code_map(&maps.k, k, pool_rows, c->n_kv_heads, D, a.page_box, spans) ||
      !moe::code_map(&maps.v, a.v_layer, pool_rows, c->n_kv_heads, D, a.page_box, spans))
    return moe::note_cuda_error(cudaErrorInvalidValue);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = dtype == MOE_FP16 ? moe::launch_attend<true>(D, maps, a, q_parts, q_factor, ctas, s)
                        : moe::launch_attend<false>(D, maps, a, q_parts, q_factor, ctas, s);
  return moe::note_cuda_error(e);
}
