// The keys and values of accepted nodes stored into the caches of all layers.
//
// Source: [CS336] section 5 (the cache that reuses the history's keys and
// values).
//
// A copy: row r of sequence b goes from node path[b][r] of the layer's qkv
// block to cache row lens[b] + r.  One warp per (row, layer, sequence) copies
// the node's 2 Hkv D contiguous elements (keys, then values) in 16-byte
// vectors, D of them to each head's cache.

#include "kernels.h"
#include "tree_internal.h"

namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32) kv_append_kernel(KvAppendArgs a, int eb) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y, l = blockIdx.z;
  const int64_t len = a.lens[b], n = a.n_path ? a.n_path[b] : a.N;
  const bool lead = blockIdx.x == 0 && l == 0 && threadIdx.x == 0;
  if (len < 0 || n < 0 || n > a.N || len + n > a.Tc) {
    if (lead) {
      atomicExch(a.err, kTreeBadInput);
      if (a.new_lens) a.new_lens[b] = int32_t(len);
    }
    return;
  }
  if (lead && a.new_lens) a.new_lens[b] = int32_t(len + n);
  const int row_vec = a.D * eb / 16;     // 16-byte vectors of one head's row
  const int vecs = a.Hkv * row_vec;      // ... of all heads
  const char* x = static_cast<const char*>(a.qkv) +
                  ((int64_t(l) * a.B + b) * a.N * a.ld_qkv + int64_t(a.H) * a.D) * eb;
  const int64_t cache = (int64_t(l) * a.B + b) * a.Hkv * a.Tc;  // rows before this sequence's
  for (int r = blockIdx.x * kWarps + (threadIdx.x >> 5); r < n; r += gridDim.x * kWarps) {
    const int node = a.path ? a.path[int64_t(b) * a.N + r] : r;
    if (node < 0 || node >= a.N) {
      if (lane == 0) atomicExch(a.err, kTreeBadInput);
      continue;
    }
    const uint4* src = reinterpret_cast<const uint4*>(x + int64_t(node) * a.ld_qkv * eb);
    for (int e = lane; e < 2 * vecs; e += 32) {
      const bool is_v = e >= vecs;
      const int c = is_v ? e - vecs : e;
      const int hk = c / row_vec, k = c % row_vec;
      uint4* dst = static_cast<uint4*>(is_v ? a.v : a.k) +
                   (cache + int64_t(hk) * a.Tc + len + r) * row_vec + k;
      *dst = src[e];
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
