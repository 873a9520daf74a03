// Appending to the 8-bit paged KV cache (qcache.h); its forks and cuts are the
// 16-bit cache's (cache.cu), which move codes as they are.
//
// For a page's part x of some rows (one layer and head, K or V) with the scale s before,
//   s' = max(s, 2^e), e the least with max |x| <= 448 * 2^e;   code = e4m3(x / s');   old codes: e4m3(code s / s')
// (without earlier rows s' = 2^e).  After the plan (cache.cu) a CTA takes one part, the rows that
// the call adds to one page, of K or of V in some layers.  Its warps go over them twice, a few
// rows of one (layer, head) at a time: for the largest value of each (layer, head), and, with the
// scales settled, for the codes; the second time most rows come from L2, and nothing waits in
// registers, so that an SM has 24 warps to hide the loads behind (16: 158 us for 130 in the case
// below).  Then the page's earlier codes are rounded anew where their scale grew (or moved, where the page is
// a copy).  A lane has sixteen values of one row, the same of every (layer, head) that its warp goes
// over, so that their angles are made once for all of these.
//
// 9,318 rows for 24 prompts, 10 layers of 2 heads of 256, fp16, all of K turned: 130 us for 286 MB with the
// trim and the plan before it (17 of them), floor 42.  In copies that leave a part of the work out: V's
// maxima 26 us, its codes 35, K's 32 and 38: each is a stream through the SMs of 4.5 TB/s at most with
// half of the issue slots used.  Infinities and NaN, which do not count for the scale and become
// NaN, are looked for only where a maximum shows that there are any.
// (Rows backwards the second time, so that the last ones read are the first ones wanted, takes 54 MB of
// reads off DRAM and no time; places gone on to by adding instead of multiplying 133 us.)
#include "qcache.cuh"
#include "rotary.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int QA_THREADS = 256, QA_WARPS = QA_THREADS / 32;
constexpr int QA_CTAS = 152 * 3;  // that run at once
constexpr int QA_MOST = 256;      // (layer, head)s of a job
constexpr int QA_AHEAD = 4;       // places of a warp's ring: three loads on their way while one is worked on

struct QAppendArgs {
  AppendArgs a;
  QCacheView q;
  attn_rotary_table table;
  int turns;               // K rows are turned
  int k_groups, v_groups;  // parts of the layers, a job each
};

// The largest of sixteen values; CAREFUL: of those that are finite.  (NaN does not count either way.)
template <bool CAREFUL>
__device__ __forceinline__ float largest(const float (&x)[8], const float (&y)[8]) {
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (CAREFUL) {
      if (fabsf(x[i]) < INFINITY) most = fmaxf(most, fabsf(x[i]));
      if (fabsf(y[i]) < INFINITY) most = fmaxf(most, fabsf(y[i]));
    } else {
      most = fmaxf(most, fmaxf(fabsf(x[i]), fabsf(y[i])));
    }
  }
  return most;
}
// The largest of sixteen 16-bit values by their bits, which order magnitudes; infinite where one is not finite.
template <bool FP16>
__device__ __forceinline__ float largest_bits(uint4 p, uint4 q) {
  constexpr uint32_t SIZE = 0x7FFF7FFFu, LIMIT = FP16 ? 0x7C00u : 0x7F80u;
  uint32_t m = __vmaxu2(__vmaxu2(__vmaxu2(p.x & SIZE, p.y & SIZE), __vmaxu2(p.z & SIZE, p.w & SIZE)),
                        __vmaxu2(__vmaxu2(q.x & SIZE, q.y & SIZE), __vmaxu2(q.z & SIZE, q.w & SIZE)));
  m = max(m & 0xFFFFu, m >> 16);
  return m >= LIMIT ? INFINITY : half_value<FP16>(m);
}
// Codes of eight values times f.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = to_codes(x[2 * i] * f, x[2 * i + 1] * f);
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

template <bool FP16>
__global__ void __launch_bounds__(QA_THREADS, 3) qcache_append_kernel(const __grid_constant__ QAppendArgs g) {
  __shared__ int parts_s[CACHE_MAX_SEQS], wsum[QA_WARPS];
  __shared__ int job_s;
  __shared__ unsigned most_s[QA_MOST];
  __shared__ float inv_s[QA_MOST], grow_s[QA_MOST];
  __shared__ uint64_t rate_s[8][16];  // of pair 8 j + i, at [i][j]
  __shared__ uint4 ring_s[QA_WARPS][QA_AHEAD][2][32];  // a lane's two runs
  start_dependent();
  const AppendArgs &a = g.a;
  const CacheView &c = a.c;
  const int rows = *a.rows, shift = c.page_shift, in_page = (1 << shift) - 1;
  if (rows == 0) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto kept = [&](int b) {  // rows the call adds to sequence b
    return (b + 1 < a.B ? a.seg[b + 1].start : rows) - a.seg[b].start - a.seg[b].cow;
  };
  // the parts before each sequence's
  constexpr int PER = CACHE_MAX_SEQS / QA_THREADS;
  int mine[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    mine[i] = sum;
    if (b < a.B) {
      const int n = kept(b), len = a.seg[b].len;
      if (n > 0) sum += ((len + n - 1) >> shift) - (len >> shift) + 1;
    }
  }
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += t;
  }
  if (lane == 31) wsum[warp] = upto;
  __syncthreads();
  int before = upto - sum, total = 0;
  for (int w = 0; w < QA_WARPS; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (tid * PER + i < a.B) parts_s[tid * PER + i] = before + mine[i];

  const int H = g.q.heads, D = g.q.dim, items = D / 16, together = 32 / items;  // rows of a warp at a time
  const int k_jobs = total * g.k_groups, jobs = k_jobs + total * g.v_groups;
  const size_t row_bytes = (size_t)c.row * 2, layer_bytes = ((size_t)c.n_pages << shift) * row_bytes;
  const size_t new_row = (size_t)H * D, new_layer = (size_t)a.n_rows * new_row;  // values
  const int j = lane % items, row0 = lane / items;
  if (g.turns && tid < 128) rate_s[tid % 8][tid / 8] = g.table.turns[tid];
  // Jobs are handed out one by one (of unequal parts; K's, the longer ones, first).
#pragma unroll 1
  for (;;) {
    __syncthreads();  // the parts are there; the last job's readers are done
    if (tid == 0) job_s = atomicAdd(&a.rows[1], 1);
    __syncthreads();
    const int job = job_s;
    if (job >= jobs) break;
    const bool is_k = job < k_jobs;
    const int groups = is_k ? g.k_groups : g.v_groups, of_kind = is_k ? job : job - k_jobs;
    const int part = of_kind / groups, group = of_kind - part * groups;
    const int layer0 = group * c.n_layers / groups, layers = (group + 1) * c.n_layers / groups - layer0, VH = layers * H;
    // the last sequence whose parts begin at or before this one (those without parts begin where the next does)
    const int b = segment_of(parts_s, a.B, part);
    const AppendSeg seg = a.seg[b];
    const int n = kept(b), nth = part - parts_s[b];
    const int first = nth == 0 ? seg.len : ((seg.len >> shift) + nth) << shift;  // its first new position
    const int count = min(seg.len + n, ((first >> shift) + 1) << shift) - first;
    const int old = nth == 0 ? first & in_page : 0;  // the page's earlier rows
    const int page = c.table[(size_t)seg.slot * c.max_pages + (first >> shift)];
    const int from_page = nth == 0 && seg.cow ? seg.old_page : page;
    for (int i = tid; i < VH; i += QA_THREADS) most_s[i] = 0;
    __syncthreads();
    if ((unsigned)page >= (unsigned)c.n_pages) continue;  // (the same for all threads)
    const bool turns = is_k && g.turns && j < g.table.dim / 16, inter = !turns || g.table.interleaved;
    const int run_a = inter ? 16 * j : 8 * j, run_b = inter ? 16 * j + 8 : g.table.dim / 2 + 8 * j;
    uint8_t *pool = reinterpret_cast<uint8_t *>(is_k ? c.k : c.v) + layer0 * layer_bytes;
    uint8_t *to = pool + ((size_t)page << shift) * row_bytes;
    const uint8_t *from = pool + ((size_t)from_page << shift) * row_bytes;
    // a warp's share of all (rows, (layer, head))s, in a row
    const int steps = (count + together - 1) / together, shares = steps * VH, each = (shares + QA_WARPS - 1) / QA_WARPS;
    const int i0 = min(shares, warp * each), i1 = min(shares, i0 + each);
    RotaryPairs angle;
    // f(run a, run b, row, (layer, head), head's place in a row, layer) for each of them (rows that are not there
    // as the last one, at its position, so that they raise no maximum), their values coming through the warp's
    // ring; a lane reads what it has copied itself
    auto go = [&](auto f) {
      int row, vh, l, h;
      auto begin = [&]() {
        const int step = i0 / VH;
        vh = i0 - step * VH, l = vh / H, h = vh - l * H, row = step * together + row0;
      };
      auto next = [&]() {  // true with a new row
        ++vh;
        if (++h < H) return false;
        h = 0, ++l;
        if (vh < VH) return false;
        vh = l = 0, row += together;
        return true;
      };
      // what is copied runs ahead of what is worked on: both from one state, one after the other
      int c_row = 0, c_vh = 0, c_l = 0, c_h = 0;  // copied next
      const uint16_t *src = nullptr;
      auto source_of = [&](int r) {
        r = first - seg.len + min(r, count - 1);
        return (is_k ? a.k_new : a.v_new) + layer0 * new_layer +
               ((size_t)seg.src + (a.path ? a.path[(size_t)b * a.path_stride + r] : r)) * new_row;
      };
      auto copy = [&](int i) {
        if (i < i1) {
          const uint16_t *s = src + c_l * new_layer + c_h * D;
          ptx::cp_async_16(&ring_s[warp][i % QA_AHEAD][0][lane], s + run_a, 16);
          ptx::cp_async_16(&ring_s[warp][i % QA_AHEAD][1][lane], s + run_b, 16);
          ++c_vh;
          if (++c_h == H) {
            c_h = 0, ++c_l;
            if (c_vh == VH) {
              c_vh = c_l = 0, c_row += together;
              if (i + 1 < i1) src = source_of(c_row);
            }
          }
        }
        ptx::cp_async_commit();
      };
      begin();
      c_row = row, c_vh = vh, c_l = l, c_h = h;
      if (i0 < i1) src = source_of(row);
#pragma unroll
      for (int k = 0; k < QA_AHEAD - 1; ++k) copy(i0 + k);
      bool fresh = true;
#pragma unroll 1
      for (int i = i0; i < i1; ++i) {
        copy(i + QA_AHEAD - 1);  // to the place that was read last
        if (fresh && is_k && g.turns)
          angle.at(first + min(row, count - 1), [&](int k) { return rate_s[k][j]; }, g.table.factor);
        asm volatile("cp.async.wait_group %0;" ::"n"(QA_AHEAD - 1) : "memory");
        f(ring_s[warp][i % QA_AHEAD][0][lane], ring_s[warp][i % QA_AHEAD][1][lane], row, vh, h * D, l);
        fresh = next();
      }
      ptx::cp_async_wait_all();
    };
    auto turned = [&](uint4 p, uint4 q, float(&x)[8], float(&y)[8]) {
      unpack8<FP16>(p, x);
      unpack8<FP16>(q, y);
      if (turns) angle.turn(x, y, inter);
    };
    auto note = [&](float most, int vh) {  // of the warp, to the (layer, head)
      const unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
      if (lane == 0) atomicMax(&most_s[vh], bits);
      return bits >= 0x7F800000u;
    };
    bool infinite = false;
    if (is_k && g.turns)
      go([&](uint4 p, uint4 q, int, int vh, int, int) {
        float x[8], y[8];
        turned(p, q, x, y);
        infinite |= note(largest<false>(x, y), vh);
      });
    else
      go([&](uint4 p, uint4 q, int, int vh, int, int) { infinite |= note(largest_bits<FP16>(p, q), vh); });
    infinite = __syncthreads_or(infinite);
    if (infinite) {  // some do not count
      for (int i = tid; i < VH; i += QA_THREADS) most_s[i] = 0;
      __syncthreads();
      go([&](uint4 p, uint4 q, int, int vh, int, int) {
        float x[8], y[8];
        turned(p, q, x, y);
        note(largest<true>(x, y), vh);
      });
      __syncthreads();
    }
    for (int i = tid; i < VH; i += QA_THREADS) {
      const int l = i / H;
      float *scales = (is_k ? g.q.ks : g.q.vs) + (size_t)(layer0 + l) * c.n_pages * H + (i - l * H);
      float s = exp2_int(scale_exp(__uint_as_float(most_s[i])));
      const float was = old ? scales[(size_t)from_page * H] : s;
      s = fmaxf(s, was);
      scales[(size_t)page * H] = s;
      inv_s[i] = 1.f / s;
      grow_s[i] = was / s;
    }
    __syncthreads();
    go([&](uint4 p, uint4 q, int row, int vh, int head, int l) {
      float x[8], y[8];
      turned(p, q, x, y);
      if (infinite) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (fabsf(x[i]) == INFINITY) x[i] = NAN;
          if (fabsf(y[i]) == INFINITY) y[i] = NAN;
        }
      }
      uint8_t *at = to + l * layer_bytes + ((first & in_page) + row) * row_bytes + head;
      const float f = inv_s[vh];
      const uint2 u = codes8(x, f), v = codes8(y, f);
      if (row >= count) return;
      if (inter) {
        *reinterpret_cast<uint4 *>(at + run_a) = make_uint4(u.x, u.y, v.x, v.y);
      } else {
        *reinterpret_cast<uint2 *>(at + run_a) = u;
        *reinterpret_cast<uint2 *>(at + run_b) = v;
      }
    });
    if (!old) continue;
    // the page's earlier rows, to the new scale or (a copy) from the page before
    for (int i = 0; i < VH; ++i) {
      const int l = i / H;
      const float f = grow_s[i];
      if (f == 1.f && from_page == page) continue;
      const size_t head = l * layer_bytes + (size_t)(i - l * H) * D + tid % items * 16;
      constexpr int AHEAD = 4;
      const int step = QA_THREADS / items;
      for (int r0 = tid / items; r0 < old; r0 += step * AHEAD) {
        uint4 w[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
          if (r0 + k * step < old) w[k] = *reinterpret_cast<const uint4 *>(from + head + (r0 + k * step) * row_bytes);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
          if (r0 + k * step >= old) break;
          if (f != 1.f) {
            uint32_t *y = &w[k].x;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 lo = from_codes(y[q] & 0xFFFFu), hi = from_codes(y[q] >> 16);
              y[q] = to_codes(lo.x * f, lo.y * f) | to_codes(hi.x * f, hi.y * f) << 16;
            }
          }
          *reinterpret_cast<uint4 *>(to + head + (r0 + k * step) * row_bytes) = w[k];
        }
      }
    }
  }
}

}  // namespace

moe_status qcache_view(const attn_qcache *c, QCacheView *out) {
  if (!c || !c->k_scale_d || !c->v_scale_d) return MOE_ERR_INVALID_ARGUMENT;
  const moe_status st =
      cache_view_any(c->k_d, c->v_d, c->refs_d, c->table_d, c->lens_d, c->status_d, c->n_layers, c->n_pages,
                     c->page_size, c->n_kv_heads, c->head_dim, c->n_slots, c->max_pages,
                     c->n_kv_heads * c->head_dim / 2, &out->c);
  if (st != MOE_OK) return st;
  if (!aligned16(c->k_scale_d) || !aligned16(c->v_scale_d)) return MOE_ERR_MISALIGNED;
  out->ks = c->k_scale_d;
  out->vs = c->v_scale_d;
  out->heads = c->n_kv_heads;
  out->dim = c->head_dim;
  return MOE_OK;
}

}  // namespace moe

extern "C" size_t attn_qcache_append_workspace_bytes(const attn_qcache *c, int32_t B, int32_t n_rows) {
  moe::QCacheView v;
  if (moe::qcache_view(c, &v) != MOE_OK || B < 1 || B > moe::CACHE_MAX_SEQS || n_rows < 0) return 0;
  size_t at;
  return moe::append_ws(c->page_size, B, n_rows, &at);
}

extern "C" moe_status attn_qcache_append(const attn_qcache *c, const attn_rotary_table *table, const void *k_new_d,
                                         const void *v_new_d, int32_t dtype, const int32_t *slots_d,
                                         const int32_t *offsets_d, const int32_t *n_keep_d, const int32_t *path_d,
                                         int32_t path_stride, int32_t B, int32_t n_rows, void *ws_d, size_t ws_bytes,
                                         void *stream) {
  moe::QAppendArgs g;
  moe_status st = moe::qcache_view(c, &g.q);
  if (st == MOE_OK && table) st = moe::rotary_check(table, c->head_dim);
  if (st != MOE_OK) return st;
  if (dtype != MOE_BF16 && dtype != MOE_FP16) return MOE_ERR_UNSUPPORTED;
  st = moe::append_args(g.q.c, moe::AppendCall{k_new_d, v_new_d, slots_d, offsets_d, n_keep_d, path_d, path_stride, B,
                                               n_rows, ws_d, ws_bytes}, g.q.c.row * 2, &g.a);
  if (st != MOE_OK || g.a.B == 0) return st;
  g.turns = table != nullptr;
  if (table) g.table = *table;
  // Jobs of a part, of K and of V: one a layer, or as many as give the CTAs that run at once
  // one of each (K's rows then make their angles less often: 24 prompts' chunks of up to 500 rows 137 us, with twice
  // as many jobs 144), or one of both at most where a part has few rows (one row for each of 48 sequences: 17.3 us;
  // two jobs for some of the CTAs 19.0, for all 22.1); but each of QA_MOST (layer, head)s at most.
  const long long parts = (long long)n_rows / c->page_size + B;
  const int layers = c->n_layers, least = (layers * c->n_kv_heads + moe::QA_MOST - 1) / moe::QA_MOST;
  const int fewest = least > 1 ? layers / (moe::QA_MOST / c->n_kv_heads) + 1 : 1;
  const bool few = n_rows <= 8 * B;
  auto groups = [&](int ctas) {
    const long long want = few ? ctas / parts : (ctas + parts - 1) / parts, g = want < fewest ? fewest : want;
    return (int)(g < layers ? g : layers);
  };
  g.k_groups = g.v_groups = groups(few ? moe::QA_CTAS / 2 : moe::QA_CTAS);
  // Long V jobs, the last to be handed out, are halved, so that the CTAs end closer to one another (parts of
  // 128 rows, 5 (layer, head)s of 256 a job: 137 us whole, 130 halved; of 16 rows, 20 a job: 119 and 124).
  if (!few && (long long)c->page_size * layers * c->n_kv_heads * c->head_dim / g.v_groups >= 128 << 10)
    g.v_groups = 2 * g.v_groups < layers ? 2 * g.v_groups : layers;
  const long long jobs = (parts + B) * (g.k_groups + g.v_groups);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = moe::launch_append_plan(g.a, s);
  if (e != cudaSuccess) return moe::note_cuda_error(e);
  const dim3 grid((unsigned)(jobs < moe::QA_CTAS ? jobs : moe::QA_CTAS)), block(moe::QA_THREADS);
  const bool pdl = moe::prof_quiet(MOE_KERNEL_CACHE_COPY);
  moe::prof_before(MOE_KERNEL_CACHE_COPY, s);
  e = dtype == MOE_FP16 ? moe::launch_dep(pdl, moe::qcache_append_kernel<true>, grid, block, 0, s, g)
                        : moe::launch_dep(pdl, moe::qcache_append_kernel<false>, grid, block, 0, s, g);
  moe::prof_after(MOE_KERNEL_CACHE_COPY, s);
  return moe::note_cuda_error(e);
}

extern "C" size_t attn_qcache_fork_workspace_bytes(const attn_qcache *c, int32_t n) {
  moe::QCacheView v;
  return moe::qcache_view(c, &v) == MOE_OK ? moe::fork_ws(n) : 0;
}

extern "C" moe_status attn_qcache_fork(const attn_qcache *c, const int32_t *src_d, const int32_t *dst_d, int32_t n,
                                       void *ws_d, size_t ws_bytes, void *stream) {
  moe::QCacheView v;
  const moe_status st = moe::qcache_view(c, &v);
  return st != MOE_OK ? st
                      : moe::fork_call(v.c, src_d, dst_d, n, ws_d, ws_bytes, v.ks, v.vs, v.heads,
                                       static_cast<cudaStream_t>(stream));
}

extern "C" moe_status attn_qcache_trim(const attn_qcache *c, const int32_t *slots_d, const int32_t *new_lens_d,
                                       int32_t n, void *stream) {
  moe::QCacheView v;
  const moe_status st = moe::qcache_view(c, &v);
  return st != MOE_OK ? st : moe::trim_call(v.c, slots_d, new_lens_d, n, static_cast<cudaStream_t>(stream));
}
