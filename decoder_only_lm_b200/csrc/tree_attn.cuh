// Shared parts of the tree-attention kernels: the split of the work over the
// grid, the ancestor masks and the partial results.
//
// Work: sequence b has len cached positions and n drafted nodes.  Its queries
// are rows r = i * G + g (node i, query head g of the G heads that share a
// key/value head), cut into row tiles of MR rows; its keys are the cached
// positions followed by the nodes, each cut into key tiles of KT.  A segment is
// one (b, key/value head, row tile); the key tiles of all segments, in that
// order, form one list, and every CTA takes an equal run of consecutive tiles,
// whatever the lengths are: a long sequence is split over many CTAs, short ones
// share one.  Lengths are read on the device, so a recorded launch follows
// them.  A segment inside one CTA's run is finished there; the pieces of any
// other go to the workspace (unnormalised output, running maximum and sum in
// fp32) and tree_combine_kernel merges them in tile order, so the result does
// not depend on timing.
#pragma once

#include "kernels.h"
#include <type_traits>

#include "tree_internal.h"

namespace tree {

constexpr int kMaxNodes = 256;
constexpr int kMaskWords = kMaxNodes / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct SeqDims {
  int len, n;
};
// Lengths of sequence b; out-of-range values make the sequence empty.
__device__ __forceinline__ SeqDims seq_dims(const TreeAttnArgs& a, int b, bool* bad = nullptr) {
  SeqDims s;
  s.len = a.lens[b];
  s.n = a.counts ? a.counts[b] : a.N;
  if (s.len < 0 || s.len > a.Tc || s.n < 0 || s.n > a.N) {
    if (bad) *bad = true;
    s.len = s.n = 0;
  }
  return s;
}
__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

template <int MR, int KT>
struct Split {
  __device__ static int row_tiles(const TreeAttnArgs& a, SeqDims s) {
    return ceil_div(s.n * a.G, MR);
  }
  __device__ static int cache_tiles(SeqDims s) { return ceil_div(s.len, KT); }
  // key tiles of each segment of the sequence (0 when it has no node)
  __device__ static int key_tiles(SeqDims s) {
    return s.n ? ceil_div(s.len, KT) + ceil_div(s.n, KT) : 0;
  }
  __device__ static int64_t tiles(const TreeAttnArgs& a, SeqDims s) {
    return int64_t(a.Hkv) * row_tiles(a, s) * key_tiles(s);
  }
  // Tiles before sequence `upto`, and over all; by every warp on its own.
  __device__ static int64_t prefix(const TreeAttnArgs& a, int upto, int64_t* total, bool* bad) {
    const int lane = threadIdx.x & 31;
    int64_t before = 0, all = 0;
    for (int b = lane; b < a.B; b += 32) {
      const int64_t t = tiles(a, seq_dims(a, b, bad));
      all += t;
      if (b < upto) before += t;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    *total = all;
    return before;
  }
  // Sequence that holds tile `pos` (< total), and the tiles before it.
  __device__ static int find(const TreeAttnArgs& a, int64_t pos, int64_t* first) {
    const int lane = threadIdx.x & 31;
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      const int64_t t = b < a.B ? tiles(a, seq_dims(a, b)) : 0;
      int64_t incl = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + incl > pos);
      if (hit) {
        const int src = __ffs(int(hit)) - 1;
        *first = base + __shfl_sync(0xffffffffu, incl - t, src);
        return b0 + src;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    *first = base;
    return a.B;
  }
};

// Tiles of every CTA's run.
__device__ __forceinline__ int64_t run_length(int64_t total, int grid) {
  return total > 0 ? (total + grid - 1) / grid : 1;
}

// Partial slot of CTA c for a segment that starts at tile s0: 0 for a segment
// that began before the CTA's run, 1 for one that begins in it and goes on.
__device__ __forceinline__ int64_t slot_of(int64_t c, int64_t s0, int64_t run) {
  return 2 * c + (s0 >= c * run ? 1 : 0);
}

// Ancestor masks of the sequence's nodes, bit j of mask i: node j is on the
// path from node i to the root, i included.  Doubling: mask(i) |= mask(up(i)),
// up(i) = up(up(i)); ceil(log2 n) rounds for a chain of n.  All threads of the
// block.  A parent outside [-1, i) counts as -1 and is reported.
__device__ __forceinline__ void build_masks(const int32_t* parent, int n, uint32_t* mask, int* up,
                                            int* err) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    int p = parent ? parent[i] : i - 1;
    if (p < -1 || p >= i) {
      atomicExch(err, kTreeBadInput);
      p = -1;
    }
    up[i] = p;
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w) mask[i * kMaskWords + w] = (i >> 5) == w ? 1u << (i & 31) : 0;
  }
  __syncthreads();
  for (int reach = 1; reach < n; reach <<= 1) {
    // reads of this round, then its writes (n <= kMaxNodes <= 2 blockDim.x)
    uint32_t add[2][kMaskWords];
    int nu[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = threadIdx.x + k * blockDim.x;
      nu[k] = -1;
      if (i < n && up[i] >= 0) {
        nu[k] = up[up[i]];
#pragma unroll
        for (int w = 0; w < kMaskWords; ++w) add[k][w] = mask[up[i] * kMaskWords + w];
      } else {
#pragma unroll
        for (int w = 0; w < kMaskWords; ++w) add[k][w] = 0;
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = threadIdx.x + k * blockDim.x;
      if (i < n) {
        up[i] = nu[k];
#pragma unroll
        for (int w = 0; w < kMaskWords; ++w) mask[i * kMaskWords + w] |= add[k][w];
      }
    }
    __syncthreads();
  }
}

// Workspace: 2 slots per CTA, each MR x D fp32 outputs, then the rows' running
// maximum and sum (log2 domain), MR of each.
template <int MR>
__host__ __device__ inline int64_t slot_floats(int D) {
  return int64_t(MR) * (D + 2);
}

// One warp (WPR = 1) or one block of WPR warps per query row: the pieces of a
// split segment merged in order,
//   M = max m_c,  out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c.
template <typename T, int MR, int KT, int WPR>
__global__ void __launch_bounds__(128) tree_combine_kernel(TreeAttnArgs a, int grid) {
  using S = Split<MR, KT>;
  constexpr int RPB = 4 / WPR;  // rows of a block
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float sh_o[WPR > 1 ? 4 : 1][WPR > 1 ? 128 : 1];
  __shared__ float sh_l[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int R = a.N * a.G;  // rows of a (sequence, key/value head)
  const int64_t row = int64_t(blockIdx.x) * RPB + (WPR > 1 ? 0 : warp);
  if (row >= int64_t(a.B) * a.Hkv * R) return;  // WPR > 1: whole block
  const int r = int(row % R), hk = int(row / R % a.Hkv), b = int(row / R / a.Hkv);
  const SeqDims s = seq_dims(a, b);
  if (r >= s.n * a.G) return;
  int64_t total;
  const int64_t first = S::prefix(a, b, &total, nullptr);
  const int64_t run = run_length(total, grid);
  const int kt = S::key_tiles(s);
  const int64_t s0 = first + (int64_t(hk) * S::row_tiles(a, s) + r / MR) * kt, s1 = s0 + kt;
  const int64_t c0 = s0 / run, c1 = (s1 - 1) / run;
  if (c0 == c1) return;  // finished by its CTA
  const int rr = r % MR, D = a.D;
  const int64_t sf = slot_floats<MR>(D);
  float M = -INFINITY;
  for (int64_t c = c0 + lane; c <= c1; c += 32)
    M = fmaxf(M, a.ws[slot_of(c, s0, run) * sf + int64_t(MR) * D + rr]);
  M = warp_max(M);
  const int sub = WPR > 1 ? warp : 0;
  float o[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
  for (int64_t c = c0 + sub; c <= c1; c += WPR) {
    const float* p = a.ws + slot_of(c, s0, run) * sf;
    const float m = p[int64_t(MR) * D + rr];
    const float w = m == -INFINITY ? 0.f : exp2f(m - M);
    l = fmaf(w, p[int64_t(MR) * D + MR + rr], l);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = lane + 32 * k;
      if (d < D) o[k] = fmaf(w, p[int64_t(rr) * D + d], o[k]);
    }
  }
  if (WPR > 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (lane + 32 * k < D) sh_o[warp][lane + 32 * k] = o[k];
    if (lane == 0) sh_l[warp] = l;
    __syncthreads();
    if (warp) return;
    l = 0.f;
    for (int w = 0; w < WPR; ++w) l += sh_l[w];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[k] = 0.f;
      if (lane + 32 * k < D)
        for (int w = 0; w < WPR; ++w) o[k] += sh_o[w][lane + 32 * k];
    }
  }
  const int i = r / a.G, h = hk * a.G + r % a.G;
  T* out = static_cast<T*>(a.out) + (int64_t(b) * a.N + i) * a.ld_out + int64_t(h) * D;
  const float inv = 1.f / l;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (lane + 32 * k < D) out[lane + 32 * k] = from_f32<T>(o[k] * inv);
  if (a.lse && lane == 0)
    a.lse[(int64_t(b) * a.H + h) * a.N + i] = (M + log2f(l)) * kLn2;
}

// Launched with programmatic serialisation: its blocks may be resident before
// the attention kernel ends and wait for it on the device.
template <typename T, int MR, int KT>
int launch_combine(const TreeAttnArgs& a, int grid, cudaStream_t st) {
  const int64_t rows = int64_t(a.B) * a.N * a.H;
  // few rows: each has many pieces, four warps share them
  const bool wide = rows < 8 * int64_t(gpt2_internal::sm_count());
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned(wide ? rows : cdiv64(rows, 4)));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  GPT2_CUDA_TRY(wide ? cudaLaunchKernelEx(&cfg, tree_combine_kernel<T, MR, KT, 4>, a, grid)
                     : cudaLaunchKernelEx(&cfg, tree_combine_kernel<T, MR, KT, 1>, a, grid));
  COUNT_LAUNCH(1);
  return GPT2_OK;
}

}  // namespace tree
