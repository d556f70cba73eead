// Verification of a tree of drafted tokens against the target's probabilities,
// with the uniform numbers passed in.
//
// Sources: [CS336] "CS336 from scratch — pretraining" section 5 (softmax at a
// temperature, top-p), [LECTURE] top-k.  Accepting or rejecting drafted tokens
// has no counterpart on the pages; the rule is rejection sampling: a token
// drawn from q is kept with probability min(1, p/q) and otherwise replaced by a
// draw from max(0, p - q), which together gives a draw from p.
//
// Weights.  A row z of logits stands for the integers
//   w_i = rint(2^36 exp((z_i - max z) / temperature))      (64-bit exp)
// with the ids outside the top-k and top-p cuts set to 0 (ids ordered by logit,
// the smaller id first among equal ones).  Sums of integers do not depend on
// their order, so every decision below is exact and repeatable.  With S the sum
// of the target's weights, x the draft's weights and X their sum, at the node
// that the walk stands at, for its children c in id order:
//   accept  iff  u_c x_c S / X < w_c   (draft given)   or   u_c S < w_c
//   reject:  w <- max(0, w - rint(x S / X))   or   w_c <- 0
// (kept as they were if nothing would be left); after the last child the next
// token is the first id whose running weight exceeds u_0 S.
//
// One cluster of up to 8 CTAs per sequence, each with a slice of the vocabulary
// in shared memory; only the rows of nodes that the walk reaches are read (a
// tree of 64 with 3 accepted tokens: 4 of 64 rows).  A node costs one exchange
// over the cluster for the maximum, one for the sum, one for each rejected
// child; the children's own weights are fetched once and kept up to date by
// every CTA.  What bounds it is the latency of that chain, not bandwidth.

#include <cooperative_groups.h>

#include "kernels.h"
#include "tree_internal.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 256;
constexpr int kCand = 64;  // candidates of a cut per CTA before the bisection takes over
constexpr double kOne = 68719476736.0;  // 2^36

struct Shared {
  uint64_t warp_red[2][3][kWarps];
  uint64_t red[2][3];
  uint32_t hist_lo[2][kBins], hist_hi[2][kBins];
  uint64_t tot[kBins];
  uint64_t cand_key[kCand], cand_w[kCand];
  uint64_t all_key[kCand * kMaxCluster], all_w[kCand * kMaxCluster];
  uint32_t n_cand;
  int bin, found;
  uint64_t before;
  uint64_t tau;
  int tok[kTreeMaxNodes], par[kTreeMaxNodes], kid[kTreeMaxNodes];
  uint64_t kw[kTreeMaxNodes], kx[kTreeMaxNodes];
  int n_kids;
  int pick;
};

// Order of the ids of a row: by logit, the smaller id first among equal ones.
__device__ __forceinline__ uint64_t order_key(float z, int id) {
  const uint32_t b = __float_as_uint(z + 0.f);  // -0 counts as 0
  const uint32_t ord = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return (uint64_t(ord) << 32) | uint64_t(0xFFFFFFFFu - uint32_t(id));
}
__device__ __forceinline__ float key_logit(uint64_t key) {
  const uint32_t ord = uint32_t(key >> 32);
  return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7FFFFFFFu) : ~ord);
}
__device__ __forceinline__ float clean(float z) { return z != z ? -INFINITY : z; }

struct Max {
  __device__ uint64_t operator()(uint64_t a, uint64_t b) const { return a > b ? a : b; }
};
struct Add {
  __device__ uint64_t operator()(uint64_t a, uint64_t b) const { return a + b; }
};

struct Walk {
  Shared& sh;
  cg::cluster_group cl;
  int lane, warp, rank, cs;
  int lo, n;  // this CTA's ids [lo, lo + n)
  int turn;   // exchange buffer of the next reduction

  // Block-wide reductions of K values exchanged over the cluster: afterwards
  // lane c < cs of every warp holds CTA c's values (0 elsewhere).  Two buffers
  // in turn: the barrier of the next exchange orders this one's reads before
  // the buffer is written again.
  template <int K, typename Op>
  __device__ void exchange(uint64_t (&v)[K], Op op) {
    const int t = turn;
    turn ^= 1;
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[k] = op(v[k], __shfl_xor_sync(0xffffffffu, v[k], o));
      if (lane == 0) sh.warp_red[t][k][warp] = v[k];
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        uint64_t x = sh.warp_red[t][k][lane & (kWarps - 1)];
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
        if (lane == 0) sh.red[t][k] = x;
      }
    }
    cl.sync();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0;
      if (lane < cs) v[k] = *cl.map_shared_rank(&sh.red[t][k], lane);
    }
  }
  // over the (at most 8) lanes that hold the CTAs' values
  template <typename Op>
  __device__ uint64_t over(uint64_t v, Op op) {
#pragma unroll
    for (int o = kMaxCluster / 2; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    return __shfl_sync(0xffffffffu, v, 0);
  }

  // Distance of a logit below the row's maximum.
  static __device__ double below(float zmax, float z) {
    return z == zmax ? 0.0 : double(zmax) - double(z);
  }

  // Keeps the ids before the first at which the running count (by_weight
  // false, goal = k) or weight (goal = a weight) of the ordered ids has reached
  // the goal, that one included; the others' weights become 0.  Ids of weight
  // 0 do not matter either way.  Two levels of a 256-bin histogram over the
  // distance below the maximum narrow the place down to a few ids, which
  // every CTA then orders exactly; if there are many (equal logits), it bisects
  // over the ordering keys.
  __device__ void cut(const float* z, uint64_t* w, float zmax, double T, bool by_weight,
                      double goal) {
    const double scale = kBins / (26.0 * T);
    int bin[2];
    uint64_t before = 0;
    bool none = false;
    for (int level = 0; level < 2 && !none; ++level) {
      for (int i = threadIdx.x; i < kBins; i += kThreads)
        sh.hist_lo[level][i] = sh.hist_hi[level][i] = 0;
      if (threadIdx.x == 0) sh.found = -1;
      __syncthreads();
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t wi = w[i];
        if (wi == 0) continue;
        const double d = below(zmax, clean(z[lo + i])) * scale;
        int at = min(kBins - 1, int(d));
        if (level == 1) {
          if (at != bin[0]) continue;
          at = max(0, min(kBins - 1, int((d - bin[0]) * kBins)));
        }
        if (by_weight) {
          // sums of 18-bit halves over a slice of at most 2^14 ids fit 32 bits
          atomicAdd(&sh.hist_lo[level][at], uint32_t(wi & 0x3FFFF));
          atomicAdd(&sh.hist_hi[level][at], uint32_t(wi >> 18));
        } else {
          atomicAdd(&sh.hist_lo[level][at], 1u);
        }
      }
      cl.sync();
      if (threadIdx.x < kBins) {
        uint64_t t = 0;
        for (int c = 0; c < cs; ++c) {
          t += *cl.map_shared_rank(&sh.hist_lo[level][threadIdx.x], c);
          t += uint64_t(*cl.map_shared_rank(&sh.hist_hi[level][threadIdx.x], c)) << 18;
        }
        sh.tot[threadIdx.x] = t;
      }
      __syncthreads();
      if (warp == 0) {  // lane l scans bins [8 l, 8 l + 8)
        uint64_t mine[8], s = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          mine[j] = sh.tot[lane * 8 + j];
          s += mine[j];
        }
        uint64_t incl = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        uint64_t at = before + incl - s;
        const bool here = double(before + incl) >= goal && double(at) < goal;
        if (here) {
          for (int j = 0; j < 8; ++j) {
            if (double(at + mine[j]) >= goal) {
              sh.found = lane * 8 + j;
              sh.before = at;
              break;
            }
            at += mine[j];
          }
        }
      }
      __syncthreads();
      bin[level] = sh.found;
      if (bin[level] < 0)
        none = true;  // everything is kept
      else
        before = sh.before;
      __syncthreads();
    }
    if (none) {  // the same in every CTA
      cl.sync();   // the histograms are read no more
      return;
    }
    // the ids of the bin
    if (threadIdx.x == 0) {
      sh.n_cand = 0;
      sh.tau = ~uint64_t(0);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      if (w[i] == 0) continue;
      const float zi = clean(z[lo + i]);
      const double d = below(zmax, zi) * scale;
      if (min(kBins - 1, int(d)) != bin[0]) continue;
      if (max(0, min(kBins - 1, int((d - bin[0]) * kBins))) != bin[1]) continue;
      const uint32_t at = atomicAdd(&sh.n_cand, 1u);
      if (at < kCand) {
        sh.cand_key[at] = order_key(zi, lo + i);
        sh.cand_w[at] = w[i];
      }
    }
    cl.sync();
    uint32_t cnt = 0;
    if (lane < cs) cnt = *cl.map_shared_rank(&sh.n_cand, lane);
    const bool many = __any_sync(0xffffffffu, cnt > kCand);
    uint64_t tau;
    if (!many) {
      uint32_t incl = cnt;  // where each CTA's candidates go in the joint list
#pragma unroll
      for (int o = 1; o < kMaxCluster; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const int total = int(__shfl_sync(0xffffffffu, incl, kMaxCluster - 1));
      for (int c = warp; c < cs; c += kWarps) {
        const int nc = int(__shfl_sync(0xffffffffu, cnt, c));
        const int off = int(__shfl_sync(0xffffffffu, incl, c)) - nc;
        for (int j = lane; j < nc; j += 32) {
          sh.all_key[off + j] = *cl.map_shared_rank(&sh.cand_key[j], c);
          sh.all_w[off + j] = *cl.map_shared_rank(&sh.cand_w[j], c);
        }
      }
      __syncthreads();
      for (int j = threadIdx.x; j < total; j += kThreads) {
        const uint64_t key = sh.all_key[j];
        uint64_t excl = before;
        for (int i = 0; i < total; ++i)
          if (sh.all_key[i] > key) excl += by_weight ? sh.all_w[i] : 1;
        if (double(excl) < goal)
          atomicMin(reinterpret_cast<unsigned long long*>(&sh.tau), (unsigned long long)key);
      }
      __syncthreads();
      tau = sh.tau;
    } else {
      // largest t whose ids of key >= t reach the goal
      uint64_t a = 0;
      for (int bit = 63; bit >= 0; --bit) {
        const uint64_t t = a | (uint64_t(1) << bit);
        uint64_t v[1] = {0};
        for (int i = threadIdx.x; i < n; i += kThreads)
          if (w[i] && order_key(clean(z[lo + i]), lo + i) >= t) v[0] += by_weight ? w[i] : 1;
        exchange(v, Add());
        if (double(over(v[0], Add())) >= goal) a = t;
      }
      tau = a;
    }
    for (int i = threadIdx.x; i < n; i += kThreads)
      if (w[i] && order_key(clean(z[lo + i]), lo + i) < tau) w[i] = 0;
  }

  // Weights of a row from its logits (top: the ordering key of its maximum).
  __device__ void weights(const float* z, uint64_t* w, uint64_t top, double T, int top_k,
                          double top_p) {
    const float zmax = key_logit(top);
    const int arg = int(0xFFFFFFFFu - uint32_t(top));
    if (T == 0.0) {
      for (int i = threadIdx.x; i < n; i += kThreads) w[i] = lo + i == arg ? uint64_t(kOne) : 0;
      return;
    }
    const double far = 26.0 * T;  // 2^36 exp(-26) < 1/2
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const double d = below(zmax, __uint_as_float(uint32_t(w[i])));
      w[i] = d > far ? 0 : uint64_t(__double2ll_rn(exp(-d / T) * kOne));
    }
    if (top_k > 0) cut(z, w, zmax, T, false, double(top_k));
    if (top_p < 1.0) {
      uint64_t v[1] = {0};
      for (int i = threadIdx.x; i < n; i += kThreads) v[0] += w[i];
      exchange(v, Add());
      cut(z, w, zmax, T, true, top_p * double(over(v[0], Add())));
    }
  }
};

__global__ void __launch_bounds__(kThreads) tree_verify_kernel(TreeVerifyArgs a, int slice) {
  extern __shared__ uint64_t rows[];  // w[slice], then x[slice] when a draft is given
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x;
  const int cs = int(cl.num_blocks()), rank = int(cl.block_rank());
  const int b = blockIdx.x / cs;
  Walk wk{sh, cl, tid & 31, tid >> 5, rank, cs, 0, 0, 0};
  const int lane = wk.lane;
  wk.lo = min(a.V, rank * slice);
  wk.n = min(a.V, wk.lo + slice) - wk.lo;
  uint64_t* w = rows;
  uint64_t* x = a.draft ? rows + slice : nullptr;
  const double T = double(a.temperature), top_p = double(a.top_p);
  const int top_k = a.top_k < a.V ? a.top_k : 0;
  const float* u = a.uniform + int64_t(b) * a.N;
  int32_t* path = a.path + int64_t(b) * a.N;
  auto unit = [](float v) { return double(fminf(fmaxf(v, 0.f), 1.f)); };

  int N = a.counts ? a.counts[b] : a.N;
  bool bad = N < 0 || N > a.N;
  if (bad) N = 0;
  for (int i = tid; i < a.N; i += kThreads) {
    if (rank == 0) path[i] = i == 0 && N > 0 ? 0 : -1;
    sh.tok[i] = a.tokens[int64_t(b) * a.N + i];
    const int p = a.parent ? a.parent[int64_t(b) * a.N + i] : i - 1;
    if (i < N && (p < -1 || p >= i)) bad = true;
    sh.par[i] = p;
  }
  if (bad && rank == 0) atomicExch(a.err, kTreeBadInput);
  __syncthreads();
  if (N == 0) {  // the whole cluster
    if (rank == 0 && tid == 0) {
      a.n_path[b] = 0;
      a.next[b] = -1;
    }
    return;
  }

  int cur = 0, n_path = 1;
  while (true) {
    // children of cur, in id order
    if (wk.warp == 0) {
      int k = 0;
      for (int i0 = cur + 1; i0 < N; i0 += 32) {
        const int i = i0 + lane;
        const bool is = i < N && sh.par[i] == cur;
        const unsigned m = __ballot_sync(0xffffffffu, is);
        if (is) sh.kid[k + __popc(m & ((1u << lane) - 1))] = i;
        k += __popc(m);
      }
      if (lane == 0) sh.n_kids = k;
    }
    __syncthreads();
    const int n_kids = sh.n_kids;
    const bool use_x = x != nullptr && n_kids > 0;
    const int64_t row = int64_t(b) * a.N + cur;
    const float* z = a.logits + row * a.ld;
    const float* y = use_x ? a.draft + row * a.ld_draft : nullptr;
    // the rows, kept as logits until their maxima are known
    uint64_t top[2] = {0, 0};
#pragma unroll 4
    for (int i = tid; i < wk.n; i += kThreads) {
      const float v = clean(z[wk.lo + i]);
      w[i] = __float_as_uint(v);
      top[0] = Max()(top[0], order_key(v, wk.lo + i));
    }
    if (use_x) {
#pragma unroll 4
      for (int i = tid; i < wk.n; i += kThreads) {
        const float v = clean(y[wk.lo + i]);
        x[i] = __float_as_uint(v);
        top[1] = Max()(top[1], order_key(v, wk.lo + i));
      }
    }
    wk.exchange(top, Max());
    wk.weights(z, w, wk.over(top[0], Max()), T, top_k, top_p);
    if (use_x) wk.weights(y, x, wk.over(top[1], Max()), T, top_k, top_p);
    uint64_t sum[2] = {0, 0};
    for (int i = tid; i < wk.n; i += kThreads) {
      sum[0] += w[i];
      if (use_x) sum[1] += x[i];
    }
    wk.exchange(sum, Add());
    uint64_t part = sum[0];  // lane c: CTA c's share of S
    uint64_t S = wk.over(sum[0], Add());
    const uint64_t X = wk.over(sum[1], Add());
    // the children's weights, from the CTAs that hold them (ordered by the
    // exchange above)
    for (int j = tid; j < n_kids; j += kThreads) {
      const int t = sh.tok[sh.kid[j]];
      uint64_t tw = 0, tx = 0;
      if (t >= 0 && t < a.V) {
        tw = *cl.map_shared_rank(&w[t % slice], t / slice);
        if (use_x) tx = *cl.map_shared_rank(&x[t % slice], t / slice);
      }
      sh.kw[j] = tw;
      sh.kx[j] = tx;
    }
    // every CTA has its copies before any weight changes
    cl.sync();
    int go = -1;
    for (int j = 0; j < n_kids; ++j) {
      const int c = sh.kid[j];
      const double uc = unit(u[c]);
      const uint64_t wc = sh.kw[j];
      double f = 0.0, lhs;
      if (use_x) {
        f = double(S) / double(X);
        lhs = uc * (double(sh.kx[j]) * f);
      } else {
        lhs = uc * double(S);
      }
      if (lhs < double(wc)) {
        go = c;
        break;
      }
      if (use_x) {
        auto less = [f](uint64_t wi, uint64_t xi) {
          const int64_t r = int64_t(wi) - __double2ll_rn(double(xi) * f);
          return r > 0 ? uint64_t(r) : uint64_t(0);
        };
        uint64_t left[1] = {0};
        for (int i = tid; i < wk.n; i += kThreads) left[0] += less(w[i], x[i]);
        wk.exchange(left, Add());
        const uint64_t total = wk.over(left[0], Add());
        if (total) {
          S = total;
          part = left[0];
          for (int i = tid; i < wk.n; i += kThreads) w[i] = less(w[i], x[i]);
          for (int i = tid; i < n_kids; i += kThreads) sh.kw[i] = less(sh.kw[i], sh.kx[i]);
        }
      } else if (wc && S > wc) {
        const int t = sh.tok[c];
        S -= wc;
        if (lane == t / slice) part -= wc;
        if (rank == t / slice && tid == 0) w[t % slice] = 0;
        __syncthreads();  // every thread has read its child's weight
        for (int i = tid; i < n_kids; i += kThreads)
          if (sh.tok[sh.kid[i]] == t) sh.kw[i] = 0;
      }
      __syncthreads();
    }
    if (go >= 0) {
      if (rank == 0 && tid == 0) path[n_path] = go;
      ++n_path;
      cur = go;
      __syncthreads();  // the children's list is read no more
      continue;
    }
    // the draw from what is left
    const double target = unit(u[0]) * double(S);
    uint64_t incl = part;
#pragma unroll
    for (int o = 1; o < kMaxCluster; o <<= 1) {
      const uint64_t yv = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += yv;
    }
    const unsigned past = __ballot_sync(0xffffffffu, lane < cs && part && double(incl) > target);
    const unsigned some = __ballot_sync(0xffffffffu, lane < cs && part);
    const int owner = past ? __ffs(int(past)) - 1 : 31 - __clz(int(some));
    if (rank == owner) {
      const uint64_t base = __shfl_sync(0xffffffffu, incl - part, owner);
      // thread t: ids [t R, t R + R) of the slice
      const int R = (wk.n + kThreads - 1) / kThreads;
      const int i0 = min(wk.n, tid * R), i1 = min(wk.n, i0 + R);
      if (tid == 0) sh.pick = past ? 0x7FFFFFFF : -1;
      __syncthreads();  // also: the last changes of w
      uint64_t s = 0;
      int last = -1;
      for (int i = i0; i < i1; ++i)
        if (w[i]) {
          s += w[i];
          last = i;
        }
      uint64_t in = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t yv = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += yv;
      }
      if (lane == 31) sh.warp_red[0][0][wk.warp] = in;
      __syncthreads();
      uint64_t at = base + in - s;
      for (int k = 0; k < wk.warp; ++k) at += sh.warp_red[0][0][k];
      if (past) {
        for (int i = i0; i < i1; ++i) {
          at += w[i];
          if (w[i] && double(at) > target) {
            atomicMin(&sh.pick, i);
            break;
          }
        }
      } else if (last >= 0) {
        atomicMax(&sh.pick, last);
      }
      __syncthreads();
      if (tid == 0) {
        a.next[b] = wk.lo + sh.pick;
        a.n_path[b] = n_path;
      }
    }
    break;
  }
  cl.sync();  // no CTA leaves while another may read its shared memory
}

}  // namespace

int launch_tree_verify(const TreeVerifyArgs& a, cudaStream_t st) {
  const int cs = kMaxCluster;
  const int slice = cdiv(a.V, cs);
  const size_t smem = size_t(slice) * sizeof(uint64_t) * (a.draft ? 2 : 1);
  GPT2_CUDA_TRY(cudaFuncSetAttribute(tree_verify_kernel,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(cs);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(cs) * unsigned(a.B));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  GPT2_CUDA_TRY(cudaLaunchKernelEx(&cfg, tree_verify_kernel, a, slice));
  COUNT_LAUNCH(1);
  return GPT2_OK;
}
