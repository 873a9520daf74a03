// Verification of drafted trees (tree.h).
//
// One cluster of up to 16 CTAs per tree.  The first warp of its first CTA
// walks the nodes in index order: parents come first, so a node whose parent is
// the current one is the next child to try, and every test needs two values, p
// and q at the node's token, which are all read at the start.  Only a child
// that is refused, and the final draw, need sums over the vocabulary: the
// walker then sends the cluster a command (through distributed shared memory),
// the CTAs go over their parts of the rows, and the walker adds up what they
// send back.  One CTA alone decides, so the cluster's barriers always meet.
//
// The sampled token is a whole number that sums in another order must not
// change, but an SM does two fp64 operations a cycle: residuals and sums are
// pairs of fp32 (value and error, some 45 bits; T. J. Dekker, "A floating-point
// technique for extending the available precision", 1971; the sum with its error
// without a comparison is D. E. Knuth's, "The Art of Computer Programming" 2, 4.2.2).  With fp64 for the
// sums of warps and CTAs and for the draw's prefixes alone, one tree over 32,000
// tokens took 37.6 us, most of it there.
//
// Bound by the row's bytes, and for few trees by latency: the start's two
// round trips, a pass and three cluster barriers.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "tree.h"

namespace moe {
namespace {

constexpr int DV_THREADS = 512, DV_WARPS = DV_THREADS / 32;
constexpr int DV_MAXN = 1024;     // nodes of a tree
constexpr int DV_MAX_CTAS = 16;   // CTAs of a cluster
constexpr int DV_MAX_CACHE = 80 * 1024;  // bytes of the residual kept by a CTA at most: two CTAs an SM

struct VerifyArgs {
  const float *p, *q;
  const int32_t *tokens, *parent, *offsets;
  const float *u_accept, *u_sample;
  int n_nodes, V;
  int32_t *path;
  int path_stride;
  int32_t *n_path, *next, *status;
};

// A value and its error.
struct Pair {
  float h, l;
};

__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.h, b.h);
  const float l = __fadd_rn(s.l, __fadd_rn(a.l, b.l)), h = __fadd_rn(s.h, l);
  return Pair{h, __fsub_rn(l, __fsub_rn(h, s.h))};
}
// The same without bringing the error back below the value's last bit (a few times in a row).
__device__ __forceinline__ Pair add_loose(Pair a, Pair b) {
  const Pair s = two_sum(a.h, b.h);
  return Pair{s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l))};
}
__device__ __forceinline__ Pair minus(Pair a) { return Pair{-a.h, -a.l}; }
__device__ __forceinline__ bool above(Pair a, Pair b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }
// s q, the pair times a float
__device__ __forceinline__ Pair scaled(Pair s, float q) {
  const float h = __fmul_rn(s.h, q), l = __fmaf_rn(s.l, q, __fmaf_rn(s.h, q, -h)), t = __fadd_rn(h, l);
  return Pair{t, __fsub_rn(l, __fsub_rn(t, h))};
}
__device__ __forceinline__ Pair shfl(Pair a, int from) {
  return Pair{__shfl_sync(0xffffffffu, a.h, from), __shfl_sync(0xffffffffu, a.l, from)};
}
// Sum over the lanes up to this one.
__device__ __forceinline__ Pair scan_lanes(Pair a) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair t{__shfl_up_sync(0xffffffffu, a.h, o), __shfl_up_sync(0xffffffffu, a.l, o)};
    if ((int)(threadIdx.x & 31) >= o) a = add(a, t);
  }
  return a;
}

// max(r - s q, 0).  NaN stays NaN, so that the sum shows it; an infinite q
// leaves 0 (the product's error is NaN then, and the difference with it).
__device__ __forceinline__ Pair drop(Pair r, Pair s, float q) {
  const float ph = __fmul_rn(s.h, q), pl = __fmaf_rn(s.l, q, __fmaf_rn(s.h, q, -ph));
  const Pair d = add(r, Pair{-ph, -pl});
  return d.h <= 0.f || ph == INFINITY ? Pair{0.f, 0.f} : d;
}

enum { CMD_END = 0, CMD_PASS = 1, CMD_DRAW = 2 };

struct Cmd {
  int op, node, rounds;  // PASS: sum the residual of `node` after `rounds` refused children
  Pair mass;             // S before the last of them
  int target;            // DRAW: the CTA that finds the token
  Pair threshold;        // whose sum passes this, counted from that CTA's first token
};

struct Shared {
  // the walker's
  float p_at[DV_MAXN], q_at[DV_MAXN], u[DV_MAXN];  // p and q of a node's parent at the node's token
  int token[DV_MAXN];
  int16_t parent[DV_MAXN];
  Pair cta_sum[DV_MAX_CTAS];
  // every CTA's
  Cmd cmd;
  Pair mass[DV_MAXN];     // S before each of the node's refused children
  int dropped[DV_MAXN];   // their tokens (drafts without probabilities)
  Pair warp_sum[DV_WARPS];
  Pair scan[DV_WARPS];
  int pick, last;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_barrier() {
  cluster_arrive();
  cluster_wait();
}
// Store into the same place of another CTA of the cluster.
template <typename T>
__device__ __forceinline__ void remote_store(T *p, uint32_t cta, const T &v) {
  static_assert(sizeof(T) % 4 == 0, "whole words");
  const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 4); ++i) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at)
                 : "r"((uint32_t)__cvta_generic_to_shared(p) + 4 * i), "r"(cta));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(w[i]) : "memory");
  }
}

// A row of p (and q) in aligned quads: quad k holds tokens 4 k - a .. 4 k - a + 3.
template <bool Q>
struct Row {
  const float *p, *q;
  int a, V, quads;
  __device__ Row(const VerifyArgs &args, int node) : V(args.V) {
    const size_t at = (size_t)node * V;
    a = (int)(at & 3);
    p = args.p + at;
    q = Q ? args.q + at : nullptr;
    quads = (a + V + 3) / 4;
  }
  __device__ __forceinline__ bool whole(int k) const { return 4 * k >= a && 4 * k - a + 4 <= V; }
  // a whole quad (zeros where !in)
  __device__ __forceinline__ void load(int k, bool in, float4 &pv, float4 &qv) const {
    const int t = 4 * k - a;
    pv = in ? *reinterpret_cast<const float4 *>(p + t) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (Q) qv = in ? *reinterpret_cast<const float4 *>(q + t) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // any quad, the row's ends among them (zeros outside the row)
  __device__ __forceinline__ void load_any(int k, float4 &pv, float4 &qv) const {
    if (whole(k)) return load(k, true, pv, qv);
    const int t = 4 * k - a;
    float x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = t + i >= 0 && t + i < V;
      x[i] = in ? p[t + i] : 0.f;
      y[i] = Q && in ? q[t + i] : 0.f;
    }
    pv = make_float4(x[0], x[1], x[2], x[3]);
    qv = make_float4(y[0], y[1], y[2], y[3]);
  }
};

// A CTA's part of the residual in shared memory, where it fits, so that every
// pass after a node's first is one step on instead of all steps again.
struct Cache {
  float4 *h, *l;
  bool on;
  __device__ void put(int i, const Pair (&r)[4]) const {
    h[i] = make_float4(r[0].h, r[1].h, r[2].h, r[3].h);
    l[i] = make_float4(r[0].l, r[1].l, r[2].l, r[3].l);
  }
  __device__ void get(int i, Pair (&r)[4]) const {
    const float4 x = h[i], y = l[i];
    r[0] = Pair{x.x, y.x}, r[1] = Pair{x.y, y.y}, r[2] = Pair{x.z, y.z}, r[3] = Pair{x.w, y.w};
  }
};

// R of a quad's tokens t .. t + 3 after `rounds` refused children: by their
// masses with q (S = 1 before the first), by their tokens without.
template <bool Q>
__device__ __forceinline__ void residual(const Shared &s, int rounds, int t, float4 pv, float4 qv, Pair (&r)[4]) {
  const float p[4] = {pv.x, pv.y, pv.z, pv.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = Pair{p[i], 0.f};
  if (Q) {
    const float q[4] = {qv.x, qv.y, qv.z, qv.w};
    if (rounds > 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[i] = two_sum(p[i], -q[i]);
        if (r[i].h <= 0.f) r[i] = Pair{0.f, 0.f};  // (NaN stays)
      }
    }
    for (int k = 1; k < rounds; ++k) {
      const Pair m = s.mass[k];
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = drop(r[i], m, q[i]);
    }
  } else {
    for (int k = 0; k < rounds; ++k) {
      const int d = s.dropped[k] - t;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (d == i) r[i].h = 0.f;
    }
  }
}

template <bool Q>
__global__ void __launch_bounds__(DV_THREADS, 2) verify_kernel(const __grid_constant__ VerifyArgs a, int ctas,
                                                             int cache_quads) {
  __shared__ Shared s;
  extern __shared__ float4 cache_mem[];
  const Cache cache{cache_mem, cache_mem + cache_quads, Q && cache_quads > 0};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int b = blockIdx.x / ctas;
  // A dependent of the kernel before, whose results are read by ordinary loads
  // only: a read-only one may look at what was there before.  (Its own dependents
  // wait for its end: let in early, they took the clusters' places, 24 us a call
  // of 96 trees over 100,003 tokens instead of 16.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  cluster_arrive();  // no CTA's memory is written to before all have started (waited for below)
  int lo = 0, n = 0;
  bool ok = true;
  if (rank == 0) {
    lo = a.offsets[b];
    const int hi = a.offsets[b + 1];
    n = hi - lo;
    ok = lo >= 0 && lo <= hi && hi <= a.n_nodes && n <= a.path_stride;
    if (ok)
      for (int i = tid; i < n; i += DV_THREADS) {
        const int par = a.parent[lo + i], x = a.tokens[lo + i];
        // node 0 is the root; the token of a node that is padding does not matter
        if (par >= i || par < -2 || (i == 0 && par != -1) || (i > 0 && par >= 0 && (x < 0 || x >= a.V)))
          ok = false;
        else if (par >= 0) {
          const size_t at = (size_t)(lo + par) * a.V + x;
          s.p_at[i] = a.p[at];
          s.q_at[i] = Q ? a.q[at] : 1.f;
          s.u[i] = a.u_accept[lo + i];
          s.token[i] = x;
        }
        s.parent[i] = (int16_t)par;
      }
    for (int i = tid; i < a.path_stride; i += DV_THREADS) a.path[(size_t)b * a.path_stride + i] = -1;
    ok = __syncthreads_and(ok);
  }

  cluster_wait();

  const float u_sample = rank == 0 ? a.u_sample[b] : 0.f;
  // the walker's state
  int32_t *path = a.path + (size_t)b * a.path_stride;
  int cur = 0, at = 0, count = 1, rounds = 0;  // at: the last node looked at
  const Pair zero{0.f, 0.f}, one{1.f, 0.f}, none{INFINITY, 0.f};  // none: a threshold that nothing passes
  Pair S = one;
  bool summed = false, started = false;        // summed: the last pass was over the current residual
  for (;;) {
    if (rank == 0 && warp == 0) {
      Cmd c{CMD_END, 0, 0, zero, 0, zero};
      if (!ok || n == 0) {
        if (lane == 0) {
          a.n_path[b] = 0;
          a.next[b] = -1;
          if (!ok) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
        }
      } else {
        if (!started && lane == 0) path[0] = 0;
        started = true;
        Pair upto = zero, total = zero;  // the CTAs' sums up to this lane's, and all of them
        if (summed) {
          upto = scan_lanes(lane < ctas ? s.cta_sum[lane] : zero);
          total = shfl(upto, 31);
          if (Q && rounds > 0) S = total;
        }
        bool pass = false;
        while (!pass) {
          // the next child of the current node
          unsigned found = 0;
          int base = (at + 1) & ~31;
          for (; base < n; base += 32) {
            const int i = base + lane;
            found = __ballot_sync(0xffffffffu, i > at && i < n && s.parent[i] == cur);
            if (found) break;
          }
          if (!found) {
            at = n;
            break;
          }
          at = base + __ffs(found) - 1;
          Pair R{s.p_at[at], 0.f};
          const float q = s.q_at[at];
          for (int i = 0; i < rounds; ++i) {
            if (Q)
              R = drop(R, s.mass[i], q);
            else if (s.dropped[i] == s.token[at])
              R = zero;
          }
          // u q is exact as a pair; with S = 1 the test is too
          const float uq = __fmul_rn(s.u[at], q);
          const Pair uqS = add(scaled(S, uq), scaled(S, __fmaf_rn(s.u[at], q, -uq)));
          if (above(R, uqS)) {
            if (lane == 0) path[count] = at;
            ++count;
            cur = at;
            rounds = 0;
            S = one;
            summed = false;
            continue;
          }
          c.mass = S;
          if (Q)
            pass = true;  // S comes from the pass
          else
            S = add(S, minus(R));
          if (!Q && lane < ctas) remote_store(&s.dropped[rounds], lane, s.token[at]);
          if (lane == 0) s.mass[rounds] = c.mass;
          __syncwarp();
          ++rounds;
          summed = false;
        }
        if (pass || !summed) {
          c.op = CMD_PASS;
          c.node = lo + cur;
          c.rounds = rounds;
          summed = true;
        } else if (total.h > 0.f && total.h < INFINITY && S.h == S.h) {  // (S: NaN among the refused tokens' R too)
          // draw: the first CTA whose sum takes the running sum past the
          // threshold; where rounding leaves none, the last with any mass.  (A CTA
          // without mass takes it nowhere, but the scan adds in another order for
          // each lane, and a threshold may lie between two roundings of one sum.)
          const Pair want = scaled(total, u_sample), mine = lane < ctas ? s.cta_sum[lane] : zero;
          const unsigned past = __ballot_sync(0xffffffffu, lane < ctas && mine.h > 0.f && above(upto, want));
          const unsigned some = __ballot_sync(0xffffffffu, mine.h > 0.f);
          c.op = CMD_DRAW;
          c.node = lo + cur;
          c.rounds = rounds;
          c.target = past ? __ffs(past) - 1 : 31 - __clz(some);
          const Pair before = shfl(upto, max(c.target - 1, 0));
          c.threshold = !past ? none : c.target ? add(want, minus(before)) : want;
          if (lane == 0) a.n_path[b] = count;
        } else if (rounds > 0 && total.h <= 0.f && S.h == S.h) {  // no residual mass: draw from p itself
          rounds = 0;
          c.op = CMD_PASS;
          c.node = lo + cur;
        } else {
          __syncwarp();
          for (int i = lane; i < a.path_stride; i += 32) path[i] = -1;
          if (lane == 0) {
            a.n_path[b] = 0;
            a.next[b] = -1;
            set_status(a.status, MOE_ERR_NONFINITE);
          }
        }
      }
      __syncwarp();
      if (lane < ctas) remote_store(&s.cmd, lane, c);
    }
    cluster_barrier();
    const Cmd c = s.cmd;
    if (c.op == CMD_END) break;
    const Row<Q> row(a, c.node);
    if (tid == 0 && c.op == CMD_PASS && c.rounds > 0) s.mass[c.rounds - 1] = c.mass;
    if (c.op == CMD_PASS) __syncthreads();
    // a warp's run of quads, the warps of all CTAs in the row's order
    const int each = (row.quads + ctas * DV_WARPS - 1) / (ctas * DV_WARPS);
    if (c.op == CMD_PASS) {
      const int k0 = min(row.quads, ((int)rank * DV_WARPS + warp) * each), k1 = min(row.quads, k0 + each);
      Pair sum{0.f, 0.f};
      const int c0 = (int)rank * DV_WARPS * each;  // the CTA's first quad
      if (cache.on && c.rounds > 1) {
        const Pair m = c.mass;
        for (int k = k0 + lane; k < k1; k += 64) {
          float4 pv, qv[2];
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (k + 32 * u < k1) row.load_any(k + 32 * u, pv, qv[u]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (k + 32 * u >= k1) break;
            Pair r[4];
            cache.get(k + 32 * u - c0, r);
            r[0] = drop(r[0], m, qv[u].x);
            r[1] = drop(r[1], m, qv[u].y);
            r[2] = drop(r[2], m, qv[u].z);
            r[3] = drop(r[3], m, qv[u].w);
            cache.put(k + 32 * u - c0, r);
            sum = add(sum, add_loose(add_loose(r[0], r[1]), add_loose(r[2], r[3])));
          }
        }
      } else {
        auto take = [&](int k, float4 pv, float4 qv) {
          Pair r[4];
          residual<Q>(s, c.rounds, 4 * k - row.a, pv, qv, r);
          if (cache.on) cache.put(k - c0, r);
          if (Q)
            sum = add(sum, add_loose(add_loose(r[0], r[1]), add_loose(r[2], r[3])));
          else  // no errors yet
            sum = add(sum, add_loose(two_sum(r[0].h, r[1].h), two_sum(r[2].h, r[3].h)));
        };
        constexpr int U = Q ? 2 : 4;  // quads of p (and q) in flight per thread
        for (int k = k0 + lane; k < k1; k += 32 * U) {
          float4 pv[U], qv[U];
          bool in[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            in[u] = k + 32 * u < k1 && row.whole(k + 32 * u);
            row.load(k + 32 * u, in[u], pv[u], qv[u]);
          }
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (in[u]) take(k + 32 * u, pv[u], qv[u]);
        }
        if (lane < 2 && k0 < k1) {  // the row's ends
          const int k = lane ? row.quads - 1 : 0;
          if (k >= k0 && k < k1 && !row.whole(k) && (lane == 0 || k > 0)) {
            float4 pv, qv;
            row.load_any(k, pv, qv);
            take(k, pv, qv);
          }
        }
      }
      __syncwarp();
      sum = scan_lanes(sum);
      if (lane == 31) s.warp_sum[warp] = sum;
      __syncthreads();
      if (warp == 0) {
        sum = scan_lanes(lane < DV_WARPS ? s.warp_sum[lane] : zero);
        if (lane == 31) remote_store(&s.cta_sum[rank], 0, sum);
      }
      cluster_barrier();
      continue;
    }
    if (rank == (uint32_t)c.target) {
      // the warp run (one with mass, as above), then the token: the first past
      // the threshold, or the last with any mass where rounding leaves none
      const Pair mine_w = lane < DV_WARPS ? s.warp_sum[lane] : zero, upto = scan_lanes(mine_w);
      const unsigned past = __ballot_sync(0xffffffffu, lane < DV_WARPS && mine_w.h > 0.f && above(upto, c.threshold));
      const unsigned some = __ballot_sync(0xffffffffu, mine_w.h > 0.f);
      const int w = past ? __ffs(past) - 1 : some ? 31 - __clz(some) : 0;
      const Pair want = past ? c.threshold : none;
      Pair from = shfl(upto, max(w - 1, 0));  // what comes before the run
      if (w == 0) from = zero;
      const int k0 = min(row.quads, ((int)rank * DV_WARPS + w) * each), k1 = min(row.quads, k0 + each);
      if (tid == 0) {
        s.pick = row.V;
        s.last = -1;
      }
      __syncthreads();
      for (int kb = k0; kb < k1; kb += DV_THREADS) {
        const int k = kb + tid, t0 = 4 * k - row.a;
        Pair r[4] = {zero, zero, zero, zero};
        if (k < k1) {
          if (cache.on) {
            cache.get(k - (int)rank * DV_WARPS * each, r);
          } else {
            float4 pv, qv;
            row.load_any(k, pv, qv);
            residual<Q>(s, c.rounds, t0, pv, qv, r);
          }
        }
        const Pair four = add(add_loose(r[0], r[1]), add_loose(r[2], r[3]));
        const Pair inc = scan_lanes(four);
        if (lane == 31) s.scan[warp] = inc;
        __syncthreads();
        const Pair warps = scan_lanes(lane < DV_WARPS ? s.scan[lane] : zero);
        const Pair ahead = shfl(warps, max(warp - 1, 0)), all = shfl(warps, 31);
        Pair run = add(warp ? add(from, ahead) : from, add(inc, minus(four)));
        from = add(from, all);
        int first = row.V, mine = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          run = add(run, r[i]);
          if (r[i].h > 0.f) {
            mine = t0 + i;
            if (first == row.V && above(run, want)) first = t0 + i;
          }
        }
        if (first < row.V) atomicMin(&s.pick, first);
        if (mine >= 0) atomicMax(&s.last, mine);
        __syncthreads();
        if (s.pick < row.V) break;
      }
      if (tid == 0) a.next[b] = min(s.pick, s.last);
    }
    break;
  }
}

// CTAs of a tree's cluster: as many as run at once for B trees, two an SM, up
// to 16 and down to 1024 tokens a CTA.  With at least 512, 1024, 2048 or 4096, us:
//   1 tree of 8,192 tokens, 7 refusals with q    31, 30, 29, 32
//   1 tree of 32,000                             31, 31, 33, 36
//   16 trees of 16,384                           63, 63, 35, 33
//   16 trees of 32,000                           63, 63, 68, 45
//   16 trees of 131,072 (16 CTAs in any case)    85, 84, 84, 84
// One tree, which waits for its passes, is served best by 1024.  Sixteen clusters
// of sixteen CTAs do not all run at once, it seems: there fewer would be better.
int cluster_ctas(int B, int V) {
  const int n = std::min({DV_MAX_CTAS, 2 * 152 / B, V / 1024});
  return n < 1 ? 1 : n;
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
  const int ctas = moe::cluster_ctas(B, V);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * ctas));
  cfg.blockDim = dim3(moe::DV_THREADS);
  cfg.stream = s;
  // the residual's cache: a CTA's quads (a row begins up to three tokens into
  // its first), if two CTAs an SM have room for it.  Seven refusals, with it and
  // without: 1 tree of 32,000 tokens 31 and 38 us, 48 trees 76 and 118, 20 trees of
  // 131,072 102 and 162; 24 of those have no room and take 187.
  int cache_quads = (V / 4 + 2 + ctas * moe::DV_WARPS - 1) / (ctas * moe::DV_WARPS) * moe::DV_WARPS;
  if (!q_d || cache_quads * 32 > moe::DV_MAX_CACHE) cache_quads = 0;
  cfg.dynamicSmemBytes = (size_t)cache_quads * 32;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = moe::prof_chain(MOE_KERNEL_DRAFT_VERIFY) ? 2 : 1;
  auto kernel = q_d ? moe::verify_kernel<true> : moe::verify_kernel<false>;
  // clusters above eight CTAs want leave, and so does much shared memory; per device
  // and cheap: asked on every call rather than remembered.  Both are the kernel's, not
  // the call's, so every call asks for the same: a thread with a smaller row
  // must not take back what another's launch is about to need.
  cudaError_t e = cudaSuccess;
  if (ctas > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && cache_quads)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, moe::DV_MAX_CACHE);
  if (e != cudaSuccess) return moe::note_cuda_error(e);
  moe::prof_before(MOE_KERNEL_DRAFT_VERIFY, s);
  e = cudaLaunchKernelEx(&cfg, kernel, a, ctas, cache_quads);
  moe::prof_after(MOE_KERNEL_DRAFT_VERIFY, s);
  return moe::note_cuda_error(e);
}
