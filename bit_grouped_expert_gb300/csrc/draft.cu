// Verification of drafted trees (tree.h).
//
// One CTA per tree walks its nodes in index order: parents come first, so a
// node whose parent is the current one is the next child to try.  The test of
// a first child needs two values, p and q at its token; only a child that is
// not taken costs a pass over the vocabulary, and so does the final draw.
// Sums and the residual run in fp64: the sampled token is a whole number that
// sums in another order must not change.
#include "common.cuh"
#include "kernels.h"
#include "tree.h"

namespace moe {
namespace {

constexpr int DV_THREADS = 1024;
constexpr int DV_MAXN = 1024;  // nodes of a tree

struct VerifyArgs {
  const float *p, *q;
  const int32_t *tokens, *parent, *offsets;
  const float *u_accept, *u_sample;
  int n_nodes, V;
  int32_t *path;
  int path_stride;
  int32_t *n_path, *next, *status;
};

// Sum over the CTA in a fixed order; every thread gets it.
__device__ double block_sum(double v, double *red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = red[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__global__ void __launch_bounds__(DV_THREADS) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ double red[32], mass_s[DV_MAXN];  // S before each of the current node's refused children
  __shared__ int drop_s[DV_MAXN];              // their tokens
  __shared__ double wsum[32];
  __shared__ int pick, last;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int lo = a.offsets[b], hi = a.offsets[b + 1], n = hi - lo;
  int32_t *path = a.path + (size_t)b * a.path_stride;
  bool ok = lo >= 0 && lo <= hi && hi <= a.n_nodes && n <= a.path_stride;
  if (ok)
    for (int i = tid; i < n; i += DV_THREADS) {
      const int par = a.parent[lo + i], x = a.tokens[lo + i];
      // node 0 is the root; the token of a node that is padding does not matter
      if (par >= i || par < -2 || (i == 0 && par != -1) || (i > 0 && par >= 0 && (x < 0 || x >= a.V))) ok = false;
    }
  ok = __syncthreads_and(ok);
  for (int i = tid; i < a.path_stride; i += DV_THREADS) path[i] = -1;
  if (!ok || n == 0) {
    if (tid == 0) {
      a.n_path[b] = 0;
      a.next[b] = -1;
      if (!ok) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    }
    return;
  }
  __syncthreads();
  int cur = 0, count = 1, ndrop = 0;
  double S = 1.0;
  const float *p = a.p + (size_t)lo * a.V, *q = a.q ? a.q + (size_t)lo * a.V : nullptr;
  // R of token t after the children refused so far
  auto residual = [&](int t) {
    double r = p[t];
    if (q) {
      const double qt = q[t];
      for (int i = 0; i < ndrop; ++i) r = fmax(r - mass_s[i] * qt, 0.0);
    } else {
      for (int i = 0; i < ndrop; ++i)
        if (drop_s[i] == t) r = 0.0;
    }
    return r;
  };
  if (tid == 0) path[0] = 0;
  for (int j = 1; j < n; ++j) {
    if (a.parent[lo + j] != cur) continue;
    const int x = a.tokens[lo + j];
    const double Rx = residual(x), qx = q ? (double)q[x] : 1.0;
    if ((double)a.u_accept[lo + j] * S * qx < Rx) {
      if (tid == 0) path[count] = j;
      ++count;
      cur = j;
      ndrop = 0;
      S = 1.0;
      p = a.p + (size_t)(lo + j) * a.V;
      if (q) q = a.q + (size_t)(lo + j) * a.V;
      continue;
    }
    __syncthreads();
    if (tid == 0) {
      mass_s[ndrop] = S;
      drop_s[ndrop] = x;
    }
    ++ndrop;
    __syncthreads();
    if (q) {
      double s = 0.0;
      for (int t = tid; t < a.V; t += DV_THREADS) s += residual(t);
      S = block_sum(s, red);
    } else {
      S -= Rx;
    }
  }
  // the draw: each thread sums a run of tokens, the runs in order
  const int run = (a.V + DV_THREADS - 1) / DV_THREADS, t0 = min(a.V, tid * run), t1 = min(a.V, t0 + run);
  for (int tries = 0; tries < 2; ++tries) {
    double s = 0.0;
    for (int t = t0; t < t1; ++t) s += residual(t);
    double inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double v = __shfl_up_sync(0xffffffffu, inc, o);
      if ((tid & 31) >= o) inc += v;
    }
    __syncthreads();
    if ((tid & 31) == 31) wsum[tid >> 5] = inc;
    if (tid == 0) {
      pick = a.V;
      last = -1;
    }
    __syncthreads();
    double before = 0.0, total = 0.0;
    for (int w = 0; w < DV_THREADS / 32; ++w) {
      if (w < (tid >> 5)) before += wsum[w];
      total += wsum[w];
    }
    before += inc - s;
    if (total > 0.0 && total < 1e300) {
      const double want = (double)a.u_sample[b] * total;
      double c = before;
      int mine = -1, first = a.V;
      for (int t = t0; t < t1; ++t) {
        const double r = residual(t);
        c += r;
        if (r > 0.0) mine = t;
        if (first == a.V && c > want && r > 0.0) first = t;
      }
      if (first < a.V) atomicMin(&pick, first);
      if (mine >= 0) atomicMax(&last, mine);
      __syncthreads();
      if (tid == 0) {
        a.next[b] = min(pick, last);
        a.n_path[b] = count;
      }
      return;
    }
    if (ndrop == 0) break;
    ndrop = 0;  // no residual mass: draw from p itself
    __syncthreads();
  }
  for (int i = tid; i < a.path_stride; i += DV_THREADS) path[i] = -1;
  if (tid == 0) {
    a.n_path[b] = 0;
    a.next[b] = -1;
    set_status(a.status, MOE_ERR_NONFINITE);
  }
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_draft_verify(const float *p_d, const float *q_d, const int32_t *tokens_d,
                                       const int32_t *parent_d, const int32_t *offsets_d, const float *u_accept_d,
                                       const float *u_sample_d, int32_t B, int32_t n_nodes, int32_t V,
                                       int32_t *path_d, int32_t path_stride, int32_t *n_path_d, int32_t *next_d,
                                       int32_t *status_d, void *stream) {
  using moe::aligned16;
  if (B < 0 || n_nodes < 0 || V < 1 || path_stride < 1) return MOE_ERR_INVALID_ARGUMENT;
  if (V > (1 << 20) || path_stride > moe::DV_MAXN || B > 65535) return MOE_ERR_UNSUPPORTED;
  if (B == 0) return MOE_OK;
  if (!offsets_d || !u_sample_d || !path_d || !n_path_d || !next_d || !status_d ||
      (n_nodes > 0 && (!p_d || !tokens_d || !parent_d || !u_accept_d)))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned16(p_d) || !aligned16(q_d) || !aligned16(tokens_d) || !aligned16(parent_d) || !aligned16(offsets_d) ||
      !aligned16(u_accept_d) || !aligned16(u_sample_d) || !aligned16(path_d) || !aligned16(n_path_d) ||
      !aligned16(next_d) || !aligned16(status_d))
    return MOE_ERR_MISALIGNED;
  moe::VerifyArgs a;
  a.p = p_d;
  a.q = q_d;
  a.tokens = tokens_d;
  a.parent = parent_d;
  a.offsets = offsets_d;
  a.u_accept = u_accept_d;
  a.u_sample = u_sample_d;
  a.n_nodes = n_nodes;
  a.V = V;
  a.path = path_d;
  a.path_stride = path_stride;
  a.n_path = n_path_d;
  a.next = next_d;
  a.status = status_d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  moe::prof_before(MOE_KERNEL_DRAFT_VERIFY, s);
  const cudaError_t e = moe::launch_dep(false, moe::verify_kernel, dim3(B), dim3(moe::DV_THREADS), 0, s, a);
  moe::prof_after(MOE_KERNEL_DRAFT_VERIFY, s);
  return moe::note_cuda_error(e);
}
