// Verification of a tree of drafted tokens where a top-k of up to 256 ids cuts
// the rows: the same rule, weights and results as without one, with the ids that
// stay held as a list.
//
// Sources: [CS336] "CS336 from scratch — pretraining" section 5 (softmax at a
// temperature, top-p), [LECTURE] top-k.
//
// Only the kept ids have a weight, so a row costs its maxima, one comparison an
// id, and an exponential for each of at most 256; no weight of the vocabulary is
// stored and no histogram kept.  The ids are found from a lower bound: with 512
// groups of ids, the k-th highest of the groups' maxima is at most the k-th highest
// logit, and with ids dealt out to the groups few others reach it (50257 normal
// logits: 56 do for k = 50, 253 for k = 200).
//
// One cluster of 8 CTAs per sequence (33 run at a time).  What bounds it is the
// latency of the walk; a node takes three exchanges over the cluster: of the groups' maxima, of the ids
// that reach the bound, and of each one's place among them, which the CTA that it
// came from counts.  Behind them every CTA holds the list in order, and accepting,
// rejecting, taking the draft's weights off and the draw need no other CTA.  A row's
// logits stay in registers: with 256 threads of 128 registers they fit for two rows
// with two CTAs on an SM (512 threads of 64: 112 us where this takes 79).
// B200, 50257 ids, drafted rows, against the kernel with a histogram of all ids:
// 64 sequences of 12 nodes with top-k 200 and top-p 343 -> 79 us, with top-k 256
// 342 -> 89; one with top-k 10 59 -> 14, with 256 68 -> 23 (1000 ids, 50: 27 -> 10).

#include <cooperative_groups.h>
#include <type_traits>

#include "kernels.h"
#include "tree_verify.cuh"

namespace cg = cooperative_groups;
using namespace tree;

namespace {

constexpr int kTopThreads = 256;
constexpr int kTopWarps = kTopThreads / 32;
constexpr int kIds = 32;      // ids of a thread at most, all in flight and in registers
constexpr int kGroups = 512;  // of ids
constexpr int kLanes = 4;     // lanes that count for a key or two
constexpr int kHalf = kTopThreads / 2;  // threads of a row of two
constexpr int kHalfWarps = kTopWarps / 2;
constexpr int kTrials = kHalfWarps;     // trial bounds at a time, a warp each
static_assert(kGroups >= kTreeTop, "a bound needs k groups");
static_assert(kTopThreads >= kTreeTop && kTopThreads >= kTreeMaxNodes, "one thread for each");

// A row's kept ids.
struct alignas(16) List {
  float group[kCluster][kGroups / kCluster];  // pushed by every CTA: its groups' maxima
  uint64_t in[kCluster][kTreeTop];            // ... ordering keys that reach the bound
  uint32_t n_in[kCluster];                    // ... their number (none if above kTreeTop)
  uint32_t counted[2][kCluster];              // ... ids that reach a trial key
  uint64_t key[kTreeTop], w[kTreeTop];        // ... the highest k, in order
  uint64_t mine[kTreeTop];                    // this CTA's share of in
  uint32_t reach[2][kTrials];                 // groups that reach a trial bound
  uint32_t n_mine;
  float from, zmax;  // the bound, the maximum
  uint64_t tau;      // lowest key that is gathered, then that stays
  uint64_t sum;      // weight that stays
  int kept;
};

struct Shared : Tree {
  uint64_t part[2][kTopWarps];
  uint32_t counted[2][kTopWarps];
  uint64_t kid_key[2][kTreeMaxNodes];
  uint32_t first, last;
};

template <bool kDraft>
__global__ void __launch_bounds__(kTopThreads, 2)
    tree_verify_top_kernel(const __grid_constant__ TreeVerifyArgs a) {
  constexpr int K = kDraft ? 2 : 1;
  extern __shared__ __align__(16) uint64_t dyn[];
  __shared__ Shared sh;
  List* list = reinterpret_cast<List*>(dyn);
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = int(cl.block_rank()), b = blockIdx.x / kCluster;
  const int top_k = a.top_k;
  // ids: a warp's 32, then the other warps', then the other CTAs'
  const int id0 = (warp * kCluster + rank) * 32 + lane;
  constexpr int kStep = kTopThreads * kCluster;
  static_assert(kStep * kIds >= kTreeMaxVocab, "a thread holds its ids");
  // what does not go over the vocabulary: half the threads for each of two rows
  const int half = tid / kHalf, slot = tid % kHalf;

  const int N = load_tree(a, sh, b, rank, tid);
  if (N == 0) return;  // the whole cluster
  const Exp ex(sh.exp_table, a.temperature);
  cl.sync();  // every CTA has started: the others may write into its shared memory

  int cur = 0, n_path = 1;
  while (true) {
    const int64_t at = int64_t(b) * a.N + cur;
    const float* z[K];
    z[0] = a.logits + at * a.ld;
    if (kDraft) z[K - 1] = a.draft + at * a.ld_draft;
    float v[K][kIds];
    auto fetch = [&](int k) {
#pragma unroll
      for (int j = 0; j < kIds; ++j) {
        const int id = id0 + j * kStep;
        v[k][j] = id < a.V ? __ldg(z[k] + id) : -INFINITY;
      }
    };
    fetch(0);
    if (warp == 0) find_children(sh, cur, N, lane);
    __syncthreads();
    const int n_kids = sh.n_kids;
    const int rows = K == 2 && n_kids > 0 ? 2 : 1;  // leaves need no draft row
    if (K == 2 && rows == 2) fetch(K - 1);

    // the groups' maxima, each of a group's lanes to one of the CTAs
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k >= rows) continue;
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < kIds; ++j) m = fmaxf(m, v[k][j]);  // (fmaxf passes over NaN)
      constexpr int kOf = kTopThreads * kCluster / kGroups;  // lanes of a group
#pragma unroll
      for (int o = 1; o < kOf; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
#pragma unroll
      for (int r = 0; r < kCluster; r += kOf)
        *cl.map_shared_rank(&list[k].group[rank][tid / kOf], r + lane % kOf) = m;
    }
    cl.sync();

    // A bound that the k highest ids reach: a value that at least k groups reach
    // (or below which no id has a weight), raised until few more than k do, each
    // of a row's warps counting for one of the values tried at a time.
    {
      const int k = K == 2 && half < rows ? half : 0;
      List& l = list[k];
      float g[kGroups / 32];
      const float4* in = reinterpret_cast<const float4*>(l.group[0]);
      float high = -INFINITY, low = INFINITY;
#pragma unroll
      for (int q = 0; q < kGroups / 128; ++q) {
        const float4 x = in[q * 32 + lane];
        g[4 * q] = x.x, g[4 * q + 1] = x.y, g[4 * q + 2] = x.z, g[4 * q + 3] = x.w;
      }
#pragma unroll
      for (int q = 0; q < kGroups / 32; ++q) {
        high = fmaxf(high, g[q]);
        low = fminf(low, g[q]);
      }
      const float best = key_logit(uint64_t(__reduce_max_sync(kAll, order_of(high))) << 32);
      float lo = key_logit(uint64_t(__reduce_min_sync(kAll, order_of(low))) << 32), hi = best;
      lo = isinf(best) ? best : fmaxf(lo, fmaxf(ex.lowest(best), -3.4028234e38f));
#pragma unroll
      for (int round = 0; round < 3; ++round) {
        const float step = hi * (1.f / (kTrials + 1)) - lo * (1.f / (kTrials + 1));
        const int trial = warp % kTrials;
        const float t = fmaf(float(trial + 1), step, lo);
        int n = 0;
#pragma unroll
        for (int q = 0; q < kGroups / 32; ++q) n += g[q] >= t;
        n = __reduce_add_sync(kAll, n);
        if (lane == 0 && half == k) l.reach[round & 1][trial] = uint32_t(n);
        __syncthreads();
        int m = 0;  // (the counts fall as the values rise)
#pragma unroll
        for (int q = 0; q < kTrials; ++q) m += l.reach[round & 1][q] >= uint32_t(top_k);
        if (m < kTrials) hi = fmaf(float(m + 1), step, lo);
        if (m > 0) lo = fmaf(float(m), step, lo);
      }
      if (slot == 0 && half == k) {
        l.from = lo;
        l.zmax = best;
        l.n_mine = best == -INFINITY ? kTreeTop + 1 : 0;  // (no bound: as too many)
      }
    }
    __syncthreads();
    // The keys that reach the bound, to every CTA.  (exact: with the order among
    // equal logits, and NaN as -inf.)
    auto gather = [&](auto of, auto exact) {
      constexpr bool kExact = decltype(exact)::value;
      uint32_t hits[K], place[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        hits[k] = 0;
        if (!of(k)) continue;
        if (kExact) fetch(k);
        const float from = list[k].from;
#pragma unroll
        for (int j = 0; j < kIds; ++j) {
          const int id = id0 + j * kStep;
          const bool hit = !kExact ? v[k][j] >= from
                                   : id < a.V && order_key(clean(v[k][j]), id) >= list[k].tau;
          hits[k] |= hit ? 1u << j : 0u;
        }
      }
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (hits[k]) place[k] = atomicAdd(&list[k].n_mine, uint32_t(__popc(hits[k])));
#pragma unroll
      for (int k = 0; k < K; ++k)
        while (hits[k]) {
          const int at = __ffs(int(hits[k])) - 1;
          float x = v[k][0];
#pragma unroll
          for (int j = 1; j < kIds; ++j) x = at == j ? v[k][j] : x;
          if (place[k] < kTreeTop) list[k].mine[place[k]] = order_key(clean(x), id0 + at * kStep);
          ++place[k];
          hits[k] &= hits[k] - 1;
        }
    };
    auto push = [&]() {
      if (half < rows) {
        List& l = list[half];
        const int n = int(l.n_mine);
        if (n <= kTreeTop)
          for (int e = slot; e < n * kCluster; e += kHalf)
            *cl.map_shared_rank(&l.in[rank][e / kCluster], e % kCluster) = l.mine[e / kCluster];
        if (slot < kCluster) *cl.map_shared_rank(&l.n_in[rank], slot) = uint32_t(n);
      }
    };
    gather([&](int k) { return k < rows; }, std::false_type());
    __syncthreads();
    push();
    cl.sync();
    bool over[K], any = false;  // more than a list holds: many equal or near ones
#pragma unroll
    for (int k = 0; k < K; ++k) {
      over[k] = false;
      if (k < rows)
        for (int r = 0; r < kCluster; ++r) over[k] |= list[k].n_in[r] > kTreeTop;
      any |= over[k];
    }
    if (any) {  // the same in every CTA: the k-th highest key itself, bit by bit
      int turn = 0;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!over[k]) continue;
        uint64_t tau = 0xFFFF0000u;  // ids are below 2^16
        for (int bit = 63; bit >= 0; bit -= bit == 32 ? 17 : 1) {
          const uint64_t t = tau | (uint64_t(1) << bit);
          int n = 0;
          for (int id = id0; id < a.V; id += kStep)
            n += order_key(clean(__ldg(z[k] + id)), id) >= t;
          n = __reduce_add_sync(kAll, n);
          if (lane == 0) sh.counted[turn][warp] = uint32_t(n);
          __syncthreads();
          if (warp == 0) {
            const uint32_t c = __reduce_add_sync(kAll, lane < kTopWarps ? sh.counted[turn][lane] : 0u);
            if (lane < kCluster) *cl.map_shared_rank(&list[k].counted[turn][rank], lane) = c;
          }
          cl.sync();
          uint32_t total = 0;
#pragma unroll
          for (int r = 0; r < kCluster; ++r) total += list[k].counted[turn][r];
          if (total >= uint32_t(top_k)) tau = t;
          turn ^= 1;
        }
        if (tid == 0) {
          list[k].tau = tau;
          list[k].n_mine = 0;
        }
      }
      __syncthreads();
      gather([&](int k) { return over[k]; }, std::true_type());
      __syncthreads();
      push();
      cl.sync();
    }

    // A key's place is the number of higher ones; each CTA counts for its own, four
    // lanes to two keys, and pushes them with their weights.
    if (half < rows) {
      List& l = list[half];
      const int part = slot % kLanes, own = int(l.n_mine);
      int n[kCluster], most = 0, total = 0;
#pragma unroll
      for (int r = 0; r < kCluster; ++r) {
        n[r] = int(l.n_in[r]);
        most = max(most, n[r]);
        total += n[r];
      }
      if (slot == 0) l.kept = min(total, top_k);
      constexpr int kPass = kHalf / kLanes;
      for (int i0 = warp % kHalfWarps * (32 / kLanes); i0 < own; i0 += 2 * kPass) {
        const int i = i0 + lane / kLanes;
        const uint64_t key0 = i < own ? l.mine[i] : 0;
        const uint64_t key1 = i + kPass < own ? l.mine[i + kPass] : 0;
        int place0 = 0, place1 = 0;
        for (int j = part; j < most; j += kLanes)
#pragma unroll
          for (int r = 0; r < kCluster; ++r) {
            const uint64_t x = j < n[r] ? l.in[r][j] : 0;
            place0 += x > key0;
            place1 += x > key1;
          }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) {
          place0 += __shfl_xor_sync(kAll, place0, o);
          place1 += __shfl_xor_sync(kAll, place1, o);
        }
        // half of the lanes push one of the keys, the others the other
        const bool second = part >= kLanes / 2;
        const uint64_t key = second ? key1 : key0;
        const int place = second ? place1 : place0;
        if (key && place < top_k) {
          const uint64_t w = weight_of(ex, key_logit(key), l.zmax);
#pragma unroll
          for (int r = part % (kLanes / 2); r < kCluster; r += kLanes / 2) {
            *cl.map_shared_rank(&l.key[place], r) = key;
            *cl.map_shared_rank(&l.w[place], r) = w;
          }
        }
      }
    }
    cl.sync();
    // top-p of what is left, and its weight; meanwhile the children's weights
    if (warp % kHalfWarps) {
      const int at = (warp - 1 - warp / kHalfWarps) * 32 + lane;
      for (int j = at; j < n_kids; j += (kTopWarps - 2) * 32) {
        const int t = sh.tok[sh.kid[j]];
        const bool real = t >= 0 && t < a.V;
        uint64_t w[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const float y = real ? clean(__ldg(z[k] + t)) : 0.f;
          w[k] = real ? weight_of(ex, y, list[k].zmax) : 0;
          sh.kid_key[k][j] = order_key(y, t);
        }
        sh.kw[j] = w[0];
        sh.kx[j] = w[K - 1];
      }
    }
    if (half < rows && warp % kHalfWarps == 0) {
      List& l = list[half];
      constexpr int kEach = kTreeTop / 32;
      const int kept = l.kept;
      uint64_t w[kEach], own = 0;
#pragma unroll
      for (int q = 0; q < kEach; ++q) {
        const int i = lane * kEach + q;
        w[q] = i < kept ? l.w[i] : 0;
        own += w[q];
      }
      uint64_t ahead = warp_scan(own, lane) - own;
      const uint64_t total = __shfl_sync(kAll, ahead + own, 31);
      const double goal = a.top_p < 1.f ? double(a.top_p) * double(total) : INFINITY;
      int m = 0;
      own = 0;
#pragma unroll
      for (int q = 0; q < kEach; ++q) {
        if (lane * kEach + q < kept && double(ahead) < goal) {
          ++m;
          own += w[q];
        }
        ahead += w[q];
      }
      m = __reduce_add_sync(kAll, m);
      const uint64_t sum = warp_add(own);
      if (lane == 0) {
        l.kept = m;
        l.sum = sum;
        l.tau = l.key[m - 1];
      }
    }
    __syncthreads();
    if (tid < n_kids) {
      if (sh.kid_key[0][tid] < list[0].tau) sh.kw[tid] = 0;
      if (kDraft && sh.kid_key[1][tid] < list[K - 1].tau) sh.kx[tid] = 0;
    }
    const int kept = list[0].kept;
    const bool mine = tid < kept;  // the kept id of this thread
    const int id = mine ? int(0xFFFFFFFFu - uint32_t(list[0].key[tid])) : -1;
    uint64_t w = mine ? list[0].w[tid] : 0, x = 0;
    uint64_t S = list[0].sum;
    const uint64_t X = list[K - 1].sum;
    __syncthreads();
    int go = -1;
    bool first = true;
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
      if (kDraft) {
        if (first && mine) {
          const float y = clean(__ldg(z[K - 1] + id));
          x = order_key(y, id) < list[K - 1].tau ? 0 : weight_of(ex, y, list[K - 1].zmax);
        }
        first = false;
        const uint64_t left = less(w, x, f);
        const uint64_t part = warp_add(left);
        if (lane == 0) sh.part[j & 1][warp] = part;
        __syncthreads();  // (also: every thread has read its child's weights)
        uint64_t total = 0;
#pragma unroll
        for (int q = 0; q < kTreeTop / 32; ++q) total += sh.part[j & 1][q];
        if (total) {
          S = total;
          w = left;
          if (tid < n_kids) sh.kw[tid] = less(sh.kw[tid], sh.kx[tid], f);
        }
      } else if (wc && S > wc) {
        const int t = sh.tok[c];
        S -= wc;
        __syncthreads();  // every thread has read its child's weight
        if (id == t) w = 0;
        if (tid < n_kids && sh.tok[sh.kid[tid]] == t) sh.kw[tid] = 0;
      }
      __syncthreads();
    }
    if (go >= 0) {
      if (rank == 0 && tid == 0) a.path[int64_t(b) * a.N + n_path] = go;
      ++n_path;
      cur = go;
      __syncthreads();  // the children's list is read no more
      continue;
    }
    // the draw from what is left: running weights in id order
    if (rank != 0) break;
    if (mine) list[0].w[tid] = w;
    if (tid == 0) {
      sh.first = ~0u;
      sh.last = 0;
    }
    __syncthreads();
    const double target = unit(sh.u[0]) * double(S);
    if (mine && w) {
      uint64_t run = 0;
      for (int j = 0; j < kept; ++j)
        run += int(0xFFFFFFFFu - uint32_t(list[0].key[j])) <= id ? list[0].w[j] : 0;
      if (double(run) > target) atomicMin(&sh.first, uint32_t(id));
      atomicMax(&sh.last, uint32_t(id));
    }
    __syncthreads();
    if (tid == 0) {
      a.next[b] = int(sh.first != ~0u ? sh.first : sh.last);  // else the last id that is left
      a.n_path[b] = n_path;
    }
    break;
  }
  // (behind the last exchange nobody touches another CTA's shared memory)
}

template <bool kDraft>
int launch(const TreeVerifyArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(List) * (kDraft ? 2 : 1);
  static std::atomic<uint64_t> allowed{0};
  GPT2_CUDA_TRY(allow_smem(allowed, tree_verify_top_kernel<kDraft>, smem));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(kCluster) * unsigned(a.B));
  cfg.blockDim = dim3(kTopThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  GPT2_CUDA_TRY(cudaLaunchKernelEx(&cfg, tree_verify_top_kernel<kDraft>, a));
  COUNT_LAUNCH(1);
  return GPT2_OK;
}

}  // namespace

int launch_tree_verify_top(const TreeVerifyArgs& a, cudaStream_t st) {
  return a.draft ? launch<true>(a, st) : launch<false>(a, st);
}
