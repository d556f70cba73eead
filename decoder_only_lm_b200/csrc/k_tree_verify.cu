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
//   w_i = 2^36 exp((z_i - max z) / temperature)      (64-bit exp, see Exp)
// as whole numbers, the ids outside the top-k and top-p cuts set to 0 (ids ordered
// by logit, the smaller id first among equal ones).  Sums of integers do not
// depend on their order, so every decision below is repeatable.  With S the sum
// of the target's weights, x the draft's weights and X their sum, at the node
// that the walk stands at, for its children c in id order:
//   accept  iff  u_c x_c S / X < w_c   (draft given)   or   u_c S < w_c
//   reject:  w <- max(0, w - rint(x S / X))   or   w_c <- 0
// (kept as they were if nothing would be left); after the last child the next
// token is the first id whose running weight exceeds u_0 S.
//
// One cluster of 8 CTAs per sequence, each with a slice of the vocabulary; only
// the rows of nodes that the walk reaches are read (a tree of 64 with 3 accepted
// tokens: 4 of 64 rows).  What bounds it is the latency of that chain, so a node
// costs as few exchanges over the cluster as it can: one for the maxima of both
// rows, one for their sums or two for their cuts (which give the sums too), and
// one for each rejected child of a drafted row.  Every exchange pushes a CTA's
// values into the others' shared memory before the cluster barrier, so that
// behind it reads are local, but for the fine bins of a cut, which are read from
// the others' memory; the work between two barriers that does not grow with the
// vocabulary is left to one warp.  A child's own weights need no exchange: every
// CTA computes them from the logits.  (B200, 50257 ids, a node of the walk: a
// temperature and guesses 3.8 us, with the draft's rows 6.5, top-p and guesses 8.5;
// a chain of 4 drafted tokens with the draft's rows, 2 nodes walked, 19 us.  15
// clusters run at a time: 16 trees of 64 guesses with top-p, up to 3 nodes walked,
// take two waves, 36 us.)

#include <cooperative_groups.h>

#include "kernels.h"
#include "tree_verify.cuh"

namespace cg = cooperative_groups;
using namespace tree;

namespace {

constexpr int kIlp = 8;              // weights of a thread computed together
constexpr int kCoarse = 37;          // bins by the exponent of a weight (1 .. 2^36)
constexpr int kBins = kCoarse * 32;  // ... and the 5 bits behind its leading one
constexpr int kCand = 48;            // ids of a cut's bin per CTA; more are bisected
// Weights below 2^kLow are counted in one bin (coarse bin kLow - 1) until a cut
// falls among them: they are most of a vocabulary and next to nothing of the
// probability, and a histogram's cost is its atomics (16 trees of 64, 50257 ids,
// top-p: 37.4 -> 35.9 us).
constexpr int kLow = 22;

// A row's cuts: this CTA's weights (in halves of 18 bits; a slice holds at most
// 2^13 ids, so 32 bits hold every sum) and ids by bin.
struct Cut {
  uint32_t lo[kBins], hi[kBins], count[kBins];
  // pushed by every CTA: weights and ids by coarse bin
  uint64_t in_w[kCluster][kCoarse];
  uint32_t in_n[kCluster][kCoarse];
  // the fine bins of the coarse bin that a cut falls into, of every CTA
  uint64_t fine_w[kCluster][32];
  uint32_t fine_n[kCluster][32];
  // pushed by every CTA: the ids of the cut's bin, for the top-k and top-p cut
  uint64_t key[2][kCluster][kCand], w[2][kCluster][kCand];
  uint32_t n_in[2][kCluster];
  uint32_t n_mine[2];
  uint16_t mine[kCand];  // this CTA's ids of the bin, before they are pushed
  bool fine_low;         // the low weights have been sorted into their bins
  int coarse, bin;  // where the cut falls, -1: nowhere
  uint64_t at_n, at_w;  // ids and weight of the bins above it
  double goal;
  uint64_t tau, kept;  // lowest ordering key that stays, weight that stays
};

struct Shared : Tree {
  uint64_t warp_red[2][2][kWarps];
  uint32_t warp_n[2][kWarps];
  uint64_t red[2][2][kCluster];  // pushed
};

// Bin of a weight >= 1 (as 2^52 + weight): its exponent and the 5 bits behind
// the leading one; the bin's weights are [bin_low(bin), bin_low(bin + 1)).
__device__ __forceinline__ int bin_of(double v) {
  return (__double2hiint(v - kOnes) >> 15) - (1023 << 5);
}
__device__ __forceinline__ uint64_t bin_low(int bin) {
  const uint64_t m = uint64_t(32 + (bin & 31)) << (bin >> 5);
  return (m + 31) >> 5;  // small exponents have fewer than 32 weights
}

struct Row {
  const float* z;  // logits
  uint64_t* w;     // weights of this CTA's ids
  Cut* cut;
  uint64_t top;    // ordering key of the maximum
  uint64_t sum;    // of all weights
  uint64_t tau;    // lowest ordering key that stays
  uint64_t low;    // weights below this went with the cuts, those of the cut's
  uint64_t high;   // bin, [low, high), by their ordering keys
};

struct Walk {
  Shared& sh;
  cg::cluster_group cl;
  int lane, warp, rank;
  int lo, n;   // this CTA's ids [lo, lo + n)
  int i0, i1;  // this warp's part of them, lane by lane
  int turn;    // exchange buffer of the next reduction

  template <typename T>
  __device__ T* remote(T* p, int r) {
    return cl.map_shared_rank(p, r);
  }

  // K sums (or maxima) over the cluster.  Two buffers in turn: a CTA pushes into
  // one again only behind the next exchange's barrier, which the others reach
  // after reading it.
  template <int K, bool kMax>
  __device__ void exchange(uint64_t (&v)[K]) {
    const int t = turn;
    turn ^= 1;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const uint64_t x = kMax ? warp_top(v[k]) : warp_add(v[k]);
      if (lane == 0) sh.warp_red[t][k][warp] = x;
    }
    __syncthreads();
    if (warp < K) {
      const uint64_t mine = lane < kWarps ? sh.warp_red[t][warp][lane] : 0;
      const uint64_t x = kMax ? warp_top(mine) : warp_add(mine);
      if (lane < kCluster) *remote(&sh.red[t][warp][rank], lane) = x;
    }
    cl.sync();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = sh.red[t][k][0];
#pragma unroll
      for (int r = 1; r < kCluster; ++r) {
        const uint64_t x = sh.red[t][k][r];
        v[k] = kMax ? (x > v[k] ? x : v[k]) : v[k] + x;
      }
    }
  }

  // One warp: the coarse bin at which the ids counted from the top (by_weight
  // false) or their weight reach the goal, with what lies above it.
  __device__ void find_coarse(Cut& c, bool by_weight, double share) {
    // lane l: coarse bins 36 - 2 l and 35 - 2 l, from the top
    uint64_t un[2] = {0, 0}, uw[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = kCoarse - 1 - 2 * lane - j;
      if (k >= (c.fine_low ? 0 : kLow - 1))
#pragma unroll
        for (int r = 0; r < kCluster; ++r) {
          un[j] += c.in_n[r][k];
          uw[j] += c.in_w[r][k];
        }
    }
    const uint64_t in = warp_scan(un[0] + un[1], lane), iw = warp_scan(uw[0] + uw[1], lane);
    const uint64_t total = __shfl_sync(kAll, iw, 31);
    // share: of the whole weight (no top-k cut before); else the goal stands
    const double goal = share > 0.0 ? share * double(total) : c.goal;
    const unsigned hit = __ballot_sync(kAll, double(by_weight ? iw : in) >= goal);
    if (!hit) {  // fewer ids of positive weight than the goal: all stay
      if (lane == 0) {
        c.coarse = c.bin = -1;
        c.kept = total;
      }
      return;
    }
    if (lane == __ffs(int(hit)) - 1) {
      uint64_t an = in - un[0] - un[1], aw = iw - uw[0] - uw[1];
      int k = kCoarse - 1 - 2 * lane;
      if (double(by_weight ? aw + uw[0] : an + un[0]) < goal) {
        an += un[0];
        aw += uw[0];
        --k;
      }
      c.coarse = k;
      c.at_n = an;
      c.at_w = aw;
      c.goal = goal;
    }
  }
  // One warp: the bin within it (lane 0 the topmost).
  __device__ void find_fine(Cut& c, bool by_weight) {
    uint64_t fn = 0, fw = 0;
#pragma unroll
    for (int r = 0; r < kCluster; ++r) {
      fn += c.fine_n[r][lane];
      fw += c.fine_w[r][lane];
    }
    const uint64_t an = c.at_n, aw = c.at_w;
    const uint64_t in = an + warp_scan(fn, lane), iw = aw + warp_scan(fw, lane);
    const unsigned hit = __ballot_sync(kAll, double(by_weight ? iw : in) >= c.goal);
    if (lane == __ffs(int(hit)) - 1) {
      c.bin = c.coarse * 32 + 31 - lane;
      c.at_n = in - fn;
      c.at_w = c.kept = iw - fw;
    }
  }

  // Sums of the coarse bins [k0, k1) of the histogram pushed to every CTA.
  __device__ void push_coarse(Cut& c, int k0, int k1) {
    for (int e = k0 + warp; e < k1; e += kWarps) {
      const int f = e * 32 + lane;
      const uint64_t w = warp_add(c.lo[f] + (uint64_t(c.hi[f]) << 18));
      const uint32_t m = __reduce_add_sync(kAll, c.count[f]);
      if (lane < kCluster) {
        *remote(&c.in_w[rank][e], lane) = w;
        *remote(&c.in_n[rank][e], lane) = m;
      }
    }
  }
  // The low weights sorted into their bins, of the rows whose cut is among them.
  template <int K>
  __device__ void refine(Row (&row)[K], int rows) {
    bool mine[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
      mine[k] = k < rows && !row[k].cut->fine_low && row[k].cut->coarse == kLow - 1;
    cl.sync();  // every CTA has read the bin that the others' sums replace
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (mine[k]) {
        Cut& c = *row[k].cut;
        for (int i = threadIdx.x; i < kLow * 32; i += kThreads) c.lo[i] = c.hi[i] = c.count[i] = 0;
        if (threadIdx.x == 0) c.fine_low = true;
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (mine[k]) {
        Cut& c = *row[k].cut;
        for (int i = i0 + lane; i < i1; i += 32) {
          const uint64_t w = row[k].w[i];
          if (w == 0 || w >> kLow) continue;
          const int bin = bin_of(double(w) + kOnes);
          atomicAdd(&c.lo[bin], uint32_t(w & 0x3FFFF));
          atomicAdd(&c.hi[bin], uint32_t(w >> 18));
          atomicAdd(&c.count[bin], 1u);
        }
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (mine[k]) push_coarse(*row[k].cut, 0, kLow);
    cl.sync();
  }

  // A cut of the rows: the ids before the first at which the running count
  // (by_weight false: to c.goal ids) or weight reaches the goal stay, that one
  // included.  The bin of the place comes from the histograms; its ids are
  // pushed to every CTA, which orders them.  Sets tau, sum, low and high.
  template <int K>
  __device__ void settle(Row (&row)[K], int rows, bool by_weight, double share) {
    const int phase = by_weight;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < rows && warp == k) find_coarse(*row[k].cut, by_weight, share);
    __syncthreads();
    bool again = false;
#pragma unroll
    for (int k = 0; k < K; ++k)
      again |= k < rows && !row[k].cut->fine_low && row[k].cut->coarse == kLow - 1;
    if (again) {  // the same in every CTA: a cut among the low weights
      refine(row, rows);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (k < rows && warp == k && row[k].cut->fine_low) find_coarse(*row[k].cut, by_weight, share);
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < K; ++k)  // warps 8 k .. 8 k + 7: one CTA's fine bins each
      if (k < rows && warp / kCluster == k && row[k].cut->coarse >= 0) {
        Cut& c = *row[k].cut;
        const int r = warp % kCluster, f = c.coarse * 32 + 31 - lane;
        const uint32_t a = *remote(&c.lo[f], r), h = *remote(&c.hi[f], r);
        const uint32_t m = *remote(&c.count[f], r);
        c.fine_w[r][lane] = a + (uint64_t(h) << 18);
        c.fine_n[r][lane] = m;
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < rows && warp == k && row[k].cut->coarse >= 0) {
        Cut& c = *row[k].cut;
        find_fine(c, by_weight);
        if (lane == 0) {
          c.tau = ~uint64_t(0);
          c.n_mine[phase] = 0;
        }
      }
    __syncthreads();
    // its ids: first a list of this CTA's, then eight threads an id push them
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < rows && row[k].cut->coarse >= 0) {
        Cut& c = *row[k].cut;
        row[k].low = bin_low(c.bin);
        row[k].high = bin_low(c.bin + 1);
#pragma unroll 4
        for (int i = i0 + lane; i < i1; i += 32) {
          const uint64_t w = row[k].w[i];
          if (w >= row[k].low && w < row[k].high) {
            const uint32_t at = atomicAdd(&c.n_mine[phase], 1u);
            if (at < kCand) c.mine[at] = uint16_t(i);
          }
        }
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < rows && row[k].cut->coarse >= 0) {
        Cut& c = *row[k].cut;
        const int count = min(int(c.n_mine[phase]), kCand);
        for (int q = threadIdx.x; q < count * kCluster; q += kThreads) {
          const int at = q / kCluster, r = q % kCluster, i = c.mine[at];
          const uint64_t key = order_key(clean(row[k].z[lo + i]), lo + i);
          // (an id that is cut away already counts nothing)
          *remote(&c.key[phase][rank][at], r) = key < row[k].tau ? 0 : key;
          *remote(&c.w[phase][rank][at], r) = row[k].w[i];
        }
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < rows && threadIdx.x < kCluster)
        *remote(&row[k].cut->n_in[phase][rank], threadIdx.x) = row[k].cut->n_mine[phase];
    cl.sync();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < rows && row[k].cut->coarse >= 0) {
        Cut& c = *row[k].cut;
        uint32_t most = 0;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) most = max(most, c.n_in[phase][r]);
        if (most > kCand) {  // the same choice in every CTA
          bisect(row[k], c, by_weight);
          continue;
        }
        // one warp per id, its lanes over the others
        const uint64_t above = by_weight ? c.at_w : c.at_n;
        const int grid = kCluster * int(most);
        for (int e = warp; e < grid; e += kWarps) {
          const int r0 = e % kCluster, j0 = e / kCluster;
          if (j0 >= int(c.n_in[phase][r0])) continue;
          const uint64_t key = c.key[phase][r0][j0];
          if (key == 0) continue;
          uint64_t ahead = 0;
          for (int q = lane; q < grid; q += 32) {
            const int r = q % kCluster, j = q / kCluster;
            if (j < int(c.n_in[phase][r]) && c.key[phase][r][j] > key)
              ahead += by_weight ? c.w[phase][r][j] : 1;
          }
          ahead = warp_add(ahead);
          if (lane == 0 && double(above + ahead) < c.goal) {
            atomicMin(reinterpret_cast<unsigned long long*>(&c.tau), (unsigned long long)key);
            atomicAdd(reinterpret_cast<unsigned long long*>(&c.kept),
                      (unsigned long long)c.w[phase][r0][j0]);
          }
        }
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < rows) {
        row[k].sum = row[k].cut->kept;
        if (row[k].cut->coarse >= 0) row[k].tau = row[k].cut->tau;
      }
  }
  // The same for a bin with many ids (equal logits): the largest key t such
  // that the ids of key >= t reach the goal, bit by bit.
  __device__ void bisect(const Row& row, Cut& c, bool by_weight) {
    const uint64_t above = by_weight ? c.at_w : c.at_n;
    uint64_t tau = 0, kept = 0;
    for (int bit = 63; bit >= -1; --bit) {  // the last round: the weight of what stays
      const uint64_t t = bit >= 0 ? tau | (uint64_t(1) << bit) : tau;
      uint64_t v[2] = {0, 0};
      for (int i = i0 + lane; i < i1; i += 32) {
        const uint64_t w = row.w[i];
        if (w < row.low || w >= row.high) continue;
        const uint64_t key = order_key(clean(row.z[lo + i]), lo + i);
        if (key < row.tau || key < t) continue;
        v[0] += by_weight ? w : 1;
        v[1] += w;
      }
      exchange<2, false>(v);
      kept = v[1];
      if (bit >= 0 && double(above + v[0]) >= c.goal) tau = t;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      c.tau = tau;
      c.kept = c.at_w + kept;
    }
    __syncthreads();
  }

  // Removes what the cuts removed from a row's weights (only the rows that are
  // drawn from or subtracted need it).
  __device__ void trim(const Row& row) {
    if (row.tau == 0) return;
#pragma unroll 4
    for (int i = i0 + lane; i < i1; i += 32) {
      const uint64_t w = row.w[i];
      if (w < row.low || (w < row.high && order_key(clean(row.z[lo + i]), lo + i) < row.tau))
        row.w[i] = 0;
    }
  }
};

template <bool kDraft, bool kCuts>
__global__ void __launch_bounds__(kThreads) tree_verify_kernel(const __grid_constant__ TreeVerifyArgs a, int slice) {
  constexpr int K = kDraft ? 2 : 1;
  extern __shared__ uint64_t dyn[];  // w[slice], x[slice] (draft), the rows' cuts
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x;
  const int rank = int(cl.block_rank()), b = blockIdx.x / kCluster;
  Walk wk{sh, cl, tid & 31, tid >> 5, rank, 0, 0, 0, 0, 0};
  const int lane = wk.lane;
  wk.lo = min(a.V, rank * slice);
  wk.n = min(a.V, wk.lo + slice) - wk.lo;
  const int per = (slice + kThreads - 1) / kThreads;  // ids of a lane
  wk.i0 = min(wk.n, wk.warp * per * 32);
  wk.i1 = min(wk.n, wk.i0 + per * 32);
  const double T = double(a.temperature), top_p = double(a.top_p);
  const int top_k = a.top_k < a.V ? a.top_k : 0;
  Cut* cut = reinterpret_cast<Cut*>(dyn + slice * K);
  int32_t* path = a.path + int64_t(b) * a.N;

  const int N = load_tree(a, sh, b, rank, tid);
  const Exp ex(sh.exp_table, a.temperature);
  if (N == 0) return;  // the whole cluster
  cl.sync();  // every CTA has started: the others may write into its shared memory

  int cur = 0, n_path = 1;
  while (true) {
    // the rows' logits, all in flight; leaves need no draft row
    const int64_t at = int64_t(b) * a.N + cur;
    Row row[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      row[k].z = k ? a.draft + at * a.ld_draft : a.logits + at * a.ld;
      row[k].w = dyn + slice * k;
      row[k].cut = cut + k;
      row[k].tau = row[k].low = row[k].high = 0;
    }
    float v[K][kPer];
    auto fetch = [&](int k) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = wk.i0 + 32 * j + lane;
        v[k][j] = j < per && i < wk.i1 ? __ldg(row[k].z + wk.lo + i) : -INFINITY;
      }
    };
    fetch(0);
    if (wk.warp == 0) find_children(sh, cur, N, lane);
    __syncthreads();
    const int n_kids = sh.n_kids;
    const int rows = K == 2 && n_kids > 0 ? 2 : 1;
    if (K == 2 && rows == 2) fetch(K - 1);
    // thread j: the logits of child j's token
    const int kid_tok = tid < n_kids ? sh.tok[sh.kid[tid]] : -1;
    const bool kid_real = kid_tok >= 0 && kid_tok < a.V;
    float kid_z[K];
#pragma unroll
    for (int k = 0; k < K; ++k) kid_z[k] = kid_real ? clean(row[k].z[kid_tok]) : 0.f;
    uint64_t top[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      top[k] = 0;
      if (k >= rows) continue;
      if (T > 0.0) {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < kPer; ++j) m = fmaxf(m, v[k][j]);  // (fmaxf passes over NaN)
        top[k] = uint64_t(order_of(m)) << 32;
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int i = wk.i0 + 32 * j + lane;
          const uint64_t key = order_key(clean(v[k][j]), wk.lo + i);
          if (j < per && i < wk.i1 && key > top[k]) top[k] = key;
        }
      }
    }
    wk.template exchange<K, true>(top);
    // the weights
    uint64_t sum[K], low_w[K];
    uint32_t low_n[K];
    if (kCuts) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        for (int i = kLow * 32 + tid; i < kBins; i += kThreads)
          cut[k].lo[i] = cut[k].hi[i] = cut[k].count[i] = 0;
      if (tid < K) {
        cut[tid].fine_low = false;
        cut[tid].goal = double(top_k);
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      row[k].top = top[k];
      row[k].sum = uint64_t(kOne);  // temperature 0: the highest logit alone
      sum[k] = low_w[k] = 0;
      low_n[k] = 0;
      if (k >= rows || T == 0.0) continue;
      float zmax = key_logit(top[k]);
      if (ex.lone(zmax)) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[k][j] = only(v[k][j], zmax);
        zmax = 0.f;
      }
      const float zmin = ex.lowest(zmax);
      // kIlp at a time with no branch between them: the chains of dependent fp64
      // operations overlap
#pragma unroll
      for (int j0 = 0; j0 < kPer; j0 += kIlp) {
        if (j0 >= per) break;
        double e[kIlp];
#pragma unroll
        for (int j = 0; j < kIlp; ++j) e[j] = ex(v[k][j0 + j], zmax, zmin);
#pragma unroll
        for (int j = 0; j < kIlp; ++j) {
          const int i = wk.i0 + 32 * (j0 + j) + lane;
          const uint64_t w = integer_of(e[j]);
          if (j0 + j < per && i < wk.i1) {
            row[k].w[i] = w;
            sum[k] += w;
            if (kCuts) {
              if (w >> kLow) {
                const int bin = bin_of(e[j]);
                atomicAdd(&cut[k].lo[bin], uint32_t(w & 0x3FFFF));
                atomicAdd(&cut[k].hi[bin], uint32_t(w >> 18));
                if (top_k > 0) atomicAdd(&cut[k].count[bin], 1u);
              } else {
                low_w[k] += w;
                low_n[k] += w != 0;
              }
            }
          }
        }
      }
    }
    if (!kCuts) {
      if (T > 0.0) {
        wk.template exchange<K, false>(sum);
#pragma unroll
        for (int k = 0; k < K; ++k) row[k].sum = sum[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint64_t lw = warp_add(low_w[k]);
        const uint32_t ln = __reduce_add_sync(kAll, low_n[k]);
        if (lane == 0) {
          sh.warp_red[0][k][wk.warp] = lw;
          sh.warp_n[k][wk.warp] = ln;
        }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (k >= rows) continue;
        wk.push_coarse(cut[k], kLow, kCoarse);
        if (wk.warp == kWarps - 1 - k) {
          const uint64_t lw = warp_add(lane < kWarps ? sh.warp_red[0][k][lane] : 0);
          const uint32_t ln = __reduce_add_sync(kAll, lane < kWarps ? sh.warp_n[k][lane] : 0u);
          if (lane < kCluster) {
            *wk.remote(&cut[k].in_w[rank][kLow - 1], lane) = lw;
            *wk.remote(&cut[k].in_n[rank][kLow - 1], lane) = ln;
          }
        }
      }
      cl.sync();
      if (top_k > 0) {
        wk.settle(row, rows, false, 0.0);
        if (top_p < 1.0) {
          if (tid < K) cut[tid].goal = top_p * double(cut[tid].kept);
          __syncthreads();
          wk.settle(row, rows, true, 0.0);
        }
      } else {
        wk.settle(row, rows, true, top_p);
      }
    }
    // the children's weights, by the same arithmetic as the rows'
    if (tid < n_kids) {
      uint64_t kid_w[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint64_t key = order_key(kid_z[k], kid_tok);
        if (!kid_real || k >= rows)
          kid_w[k] = 0;
        else if (T == 0.0)
          kid_w[k] = key == row[k].top ? uint64_t(kOne) : 0;
        else
          kid_w[k] = key < row[k].tau ? 0 : weight_of(ex, kid_z[k], key_logit(row[k].top));
      }
      sh.kw[tid] = kid_w[0];
      sh.kx[tid] = kid_w[K - 1];
    }
    __syncthreads();
    uint64_t S = row[0].sum;
    const uint64_t X = row[K - 1].sum;
    uint64_t* w = row[0].w;
    const uint64_t* x = row[K - 1].w;
    int go = -1;
    bool trimmed = !kCuts;
    for (int j = 0; j < n_kids; ++j) {
      const int c = sh.kid[j];
      const double uc = unit(sh.u[c]);
      const uint64_t wc = sh.kw[j];
      const double f = kDraft ? double(S) / double(X) : 0.0;
      const double lhs = kDraft ? uc * (double(sh.kx[j]) * f) : uc * double(S);
      if (lhs < double(wc)) {
        go = c;
        break;
      }
      if (T == 0.0) continue;  // the one weight stays: it is accepted or not proposed
      if (kDraft) {
        if (!trimmed) {
          wk.trim(row[0]);
          wk.trim(row[K - 1]);
          trimmed = true;
        }
        uint64_t left[1] = {0}, wi[kPer];
#pragma unroll
        for (int j1 = 0; j1 < kPer; j1 += 4) {
          if (j1 >= per) break;
#pragma unroll
          for (int q = j1; q < j1 + 4; ++q) {
            const int i = wk.i0 + 32 * q + lane;
            wi[q] = q < per && i < wk.i1 ? less(w[i], x[i], f) : 0;
            left[0] += wi[q];
          }
        }
        wk.template exchange<1, false>(left);
        if (left[0]) {
          S = left[0];
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            const int i = wk.i0 + 32 * q + lane;
            if (q < per && i < wk.i1) w[i] = wi[q];
          }
          for (int i = tid; i < n_kids; i += kThreads) sh.kw[i] = less(sh.kw[i], sh.kx[i], f);
        }
      } else if (wc && S > wc) {
        const int t = sh.tok[c];
        S -= wc;
        __syncthreads();  // every thread has read its child's weight
        const int mine = t - wk.lo;  // by the lane that reads it in every pass
        if (mine >= wk.i0 && mine < wk.i1 && (mine - wk.i0) % 32 == lane) w[mine] = 0;
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
    if (T == 0.0) {
      if (rank == 0 && tid == 0) {
        a.next[b] = int(0xFFFFFFFFu - uint32_t(row[0].top));
        a.n_path[b] = n_path;
      }
      break;
    }
    // the draw from what is left: the CTA, its warp, the id (a warp's ids are
    // consecutive)
    const double target = unit(sh.u[0]) * double(S);
    if (!trimmed) wk.trim(row[0]);
    uint64_t share[1] = {0};
#pragma unroll 4
    for (int i = wk.i0 + lane; i < wk.i1; i += 32) share[0] += w[i];
    const int turn = wk.turn;
    wk.template exchange<1, false>(share);
    uint64_t run = 0, before = 0;
    int owner = -1, last = -1;
#pragma unroll
    for (int r = 0; r < kCluster; ++r) {
      const uint64_t part = sh.red[turn][0][r];
      if (part) {
        if (owner < 0 && double(run + part) > target) {
          owner = r;
          before = run;
        }
        last = r;
      }
      run += part;
    }
    const bool past = owner >= 0;  // else the last id that is left
    if (!past) owner = last;
    if (rank != owner) break;
    const uint64_t mine = lane < kWarps ? sh.warp_red[turn][0][lane] : 0;
    const uint64_t in = warp_scan(mine, lane);
    const unsigned over = __ballot_sync(kAll, mine && double(before + in) > target);
    const unsigned any = __ballot_sync(kAll, mine != 0);
    const int ow = past ? __ffs(int(over)) - 1 : 31 - __clz(int(any));
    if (wk.warp != ow) break;
    run = before + __shfl_sync(kAll, in - mine, ow);
    int pick = -1;
    for (int base = wk.i0; base < wk.i1; base += 32) {
      const uint64_t wi = base + lane < wk.i1 ? w[base + lane] : 0;
      const uint64_t upto = warp_scan(wi, lane);
      const unsigned hit = __ballot_sync(kAll, wi && (!past || double(run + upto) > target));
      if (past && hit) {
        pick = base + __ffs(int(hit)) - 1;
        break;
      }
      if (hit) pick = base + 31 - __clz(int(hit));  // the last one so far
      run += __shfl_sync(kAll, upto, 31);
    }
    if (lane == 0) {
      a.next[b] = wk.lo + pick;
      a.n_path[b] = n_path;
    }
    break;
  }
  // (behind the last exchange nobody touches another CTA's shared memory)
}

template <bool kDraft, bool kCuts>
int launch(const TreeVerifyArgs& a, cudaStream_t st) {
  const int slice = cdiv(a.V, kCluster);
  const size_t smem = (size_t(slice) * sizeof(uint64_t) + (kCuts ? sizeof(Cut) : 0)) * (kDraft ? 2 : 1);
  constexpr size_t kMost =
      (kTreeMaxVocab / kCluster * sizeof(uint64_t) + (kCuts ? sizeof(Cut) : 0)) * (kDraft ? 2 : 1);
  static std::atomic<uint64_t> allowed{0};
  GPT2_CUDA_TRY(allow_smem(allowed, tree_verify_kernel<kDraft, kCuts>, kMost));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(kCluster) * unsigned(a.B));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  GPT2_CUDA_TRY(cudaLaunchKernelEx(&cfg, tree_verify_kernel<kDraft, kCuts>, a, slice));
  COUNT_LAUNCH(1);
  return GPT2_OK;
}

}  // namespace

int launch_tree_verify(const TreeVerifyArgs& a, cudaStream_t st) {
  const bool top = a.temperature > 0.f && a.top_k > 0 && a.top_k < a.V;
  // the kept ids as a list, as long as they fit (2.7 to 4.3 times as fast as the
  // histogram where both were measured: the figures stand with the list's kernel)
  if (top && a.top_k <= kTreeTop) return launch_tree_verify_top(a, st);
  const bool cuts = top || (a.temperature > 0.f && a.top_p < 1.f);
  if (a.draft) return cuts ? launch<true, true>(a, st) : launch<true, false>(a, st);
  return cuts ? launch<false, true>(a, st) : launch<false, false>(a, st);
}
