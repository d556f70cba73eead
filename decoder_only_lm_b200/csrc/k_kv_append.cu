// The keys and values of accepted nodes stored into the caches of all layers.
//
// Source: [CS336] section 5 (the cache that reuses the history's keys and
// values).
//
// A copy: row r of sequence b goes from node path[b][r] of the layer's qkv
// block to cache row lens[b] + r.  One warp per (row, layer, sequence) copies
// the node's 2 Hkv D contiguous elements (keys, then values) in 16-byte
// vectors, D of them to each head's cache.  Bound by memory: a lane keeps four
// vectors in flight (B200, the accepted paths of 16 trees of 64, 24 layers of 16
// heads of 64: 6.8 us, 5.85 TB/s; one at a time with a division for the head:
// 7.7; all 64 nodes: 35 against 44 us, 5.74 TB/s).

#include "kernels.h"
#include "tree_internal.h"

namespace {

constexpr int kWarps = 8;
constexpr int kIlp = 4;  // vectors of a lane in flight

__global__ void __launch_bounds__(kWarps * 32) kv_append_kernel(KvAppendArgs a, int eb) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y, l = blockIdx.z;
  const int64_t len = a.lens[b], n = a.n_path ? a.n_path[b] : a.N;
  const bool lead = blockIdx.x == 0 && l == 0 && threadIdx.x == 0;
  if (len < 0 || n < 0 || n > a.N || len + n > a.Tc) {
    if (lead) {
      note_bad_input(a.err);
      if (a.new_lens) a.new_lens[b] = int32_t(len);
    }
    return;
  }
  if (lead && a.new_lens) a.new_lens[b] = int32_t(len + n);
  const int shift = __ffs(a.D * eb) - 5;  // 2^shift 16-byte vectors of one head's row
  const int vecs = a.Hkv << shift;        // ... of all heads
  const char* x = static_cast<const char*>(a.qkv) +
                  ((int64_t(l) * a.B + b) * a.N * a.ld_qkv + int64_t(a.H) * a.D) * eb;
  const int64_t cache = (int64_t(l) * a.B + b) * a.Hkv * a.Tc;  // rows before this sequence's
  for (int r = blockIdx.x * kWarps + (threadIdx.x >> 5); r < n; r += gridDim.x * kWarps) {
    const int node = a.path ? a.path[int64_t(b) * a.N + r] : r;
    if (node < 0 || node >= a.N) {
      if (lane == 0) note_bad_input(a.err);
      continue;
    }
    const uint4* src = reinterpret_cast<const uint4*>(x + int64_t(node) * a.ld_qkv * eb);
    for (int e0 = lane; e0 < 2 * vecs; e0 += 32 * kIlp) {
      uint4 v[kIlp];
#pragma unroll
      for (int i = 0; i < kIlp; ++i)
        if (e0 + 32 * i < 2 * vecs) v[i] = src[e0 + 32 * i];
#pragma unroll
      for (int i = 0; i < kIlp; ++i) {
        const int e = e0 + 32 * i;
        const bool is_v = e >= vecs;
        const int c = is_v ? e - vecs : e;
        if (e < 2 * vecs)
          (static_cast<uint4*>(is_v ? a.v : a.k) + ((cache + len + r) << shift))[
              ((int64_t(c >> shift) * a.Tc) << shift) + (c & ((1 << shift) - 1))] = v[i];
      }
    }
  }
}

}  // namespace

int launch_kv_append(const KvAppendArgs& a, int elem_bytes, cudaStream_t st) {
  const dim3 grid(cdiv(a.N, kWarps), a.B, a.L);
  kv_append_kernel<<<grid, kWarps * 32, 0, st>>>(a, elem_bytes);
  COUNT_LAUNCH(1);
  GPT2_LAUNCH_CHECK();
  return GPT2_OK;
}
