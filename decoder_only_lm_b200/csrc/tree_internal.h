// Decoding with drafted tokens (internal): attention of a tree of drafted
// tokens over a cache, verification, and the cache store.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

// A length, count, parent or path out of range, noted in its own word behind the
// error word (err): a timeout recorded there stays, and calls that look for one
// leave this alone.  Read back as GPT2_ERR_ARG.
__device__ __forceinline__ void note_bad_input(int* err) { atomicExch(err + 1, 1); }

// Allows a kernel its dynamic shared memory, once per device (`done`: the devices
// that have it; more than 64 are asked every time).
template <typename Kernel>
cudaError_t allow_smem(std::atomic<uint64_t>& done, Kernel kernel, size_t bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

struct TreeAttnArgs {
  const void* qkv;
  int64_t ld_qkv;
  const void *k, *v;
  const int32_t *lens, *parent, *counts;
  int B, N, H, Hkv, G, D, Tc;  // G = H / Hkv
  void* out;
  int64_t ld_out;
  float* lse;
  float* ws;
  int* err;
  int2* seg;  // in the workspace, set by the launchers
  bool zero;  // rows without a node become 0
};

size_t tree_attn_workspace(int B, int N, int H, int Hkv, int D, int bf16);
int launch_tree_attn(const TreeAttnArgs& a, int bf16, cudaStream_t st);

struct TreeVerifyArgs {
  const float* logits;
  int64_t ld;
  const float* draft;  // nullable
  int64_t ld_draft;
  const int32_t *tokens, *parent, *counts;
  const float* uniform;
  int B, N, V;
  float temperature;
  int top_k;
  float top_p;
  int32_t *path, *n_path, *next;
  int* err;
};
constexpr int kTreeMaxNodes = 256;
// Rows of a cache: tiles of 64 keys are counted and placed in 32 bits, the last one
// reaching up to 63 behind a length.
constexpr int64_t kTreeMaxRows = 0x7FFFFFFF - 64;
constexpr int kTreeMaxVocab = 65536;
int launch_tree_verify(const TreeVerifyArgs& a, cudaStream_t st);
// the same for a temperature above 0 and 1 <= top_k <= kTreeTop, top_k < V
constexpr int kTreeTop = 256;
int launch_tree_verify_top(const TreeVerifyArgs& a, cudaStream_t st);

struct KvAppendArgs {
  const void* qkv;
  int64_t ld_qkv;
  const int32_t *path, *n_path, *lens;
  int L, B, N, H, Hkv, D, Tc;
  void *k, *v;
  int32_t* new_lens;
  int* err;
};
int launch_kv_append(const KvAppendArgs& a, int elem_bytes, cudaStream_t st);
