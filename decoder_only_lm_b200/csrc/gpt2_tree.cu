// C ABI of decoding with drafted tokens: tree attention, verification and the
// cache store.  Argument checks on the host; the kernels check what lives on
// the device (lengths, counts, trees, paths).

#include <string>

#include "kernels.h"
#include "tree_internal.h"

using gpt2_internal::set_error;

namespace {

int refuse(const char* what) noexcept {
  try {
    set_error(what);
  } catch (...) {
  }
  return GPT2_ERR_ARG;
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// n elements of 4 bytes at p share memory with m at q
bool overlap(const void* p, uint64_t n, const void* q, uint64_t m) {
  const auto a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + m * 4 && b < a + n * 4;
}
// limits shared by the calls: grid sizes and 32-bit row counts
bool heads_ok(int B, int N, int H, int Hkv, int D) {
  return B >= 1 && B <= 65535 && N >= 1 && N <= kTreeMaxNodes && Hkv >= 1 && H >= Hkv &&
         H % Hkv == 0 && H <= 65535 && (D == 16 || D == 32 || D == 64 || D == 128) &&
         int64_t(B) * N * H <= int64_t(0x7FFFFFFF);
}
bool type_ok(int dtype) { return dtype == GPT2_F32 || dtype == GPT2_BF16; }
bool row_ok(int64_t ld, int dtype, int64_t width) {
  return ld >= width && ld % (dtype == GPT2_BF16 ? 8 : 4) == 0;
}

}  // namespace

extern "C" {

int gpt2_tree_attention_workspace(int B, int N, int H, int Hkv, int D, int dtype, size_t* bytes) {
  if (!bytes || !heads_ok(B, N, H, Hkv, D) || !type_ok(dtype))
    return refuse("tree_attention_workspace: bad arguments");
  *bytes = tree_attn_workspace(B, N, H, Hkv, D, dtype == GPT2_BF16);
  return GPT2_OK;
}

int gpt2_tree_attention(const void* qkv, int64_t ld_qkv, const void* k_cache, const void* v_cache,
                        const int32_t* lens, const int32_t* parent, const int32_t* counts,
                        int dtype, int B, int N, int H, int Hkv, int D, int Tc, void* out,
                        int64_t ld_out, float* lse, void* workspace, size_t workspace_bytes,
                        void* stream) {
  if (!qkv || !k_cache || !v_cache || !lens || !out)
    return refuse("tree_attention: null pointer");
  const bool zero = dtype & GPT2_ZERO_ROWS;
  dtype &= ~GPT2_ZERO_ROWS;
  if (!type_ok(dtype)) return refuse("tree_attention: bad dtype");
  if (!heads_ok(B, N, H, Hkv, D) || Tc < 1 || int64_t(B) * Hkv * Tc > kTreeMaxRows)
    return refuse("tree_attention: B, N (1..256), H, Hkv, D (16, 32, 64, 128) or Tc out of range");
  if (!row_ok(ld_qkv, dtype, (int64_t(H) + 2 * Hkv) * D) || !row_ok(ld_out, dtype, int64_t(H) * D))
    return refuse("tree_attention: ld_qkv or ld_out too small or not a multiple of 16 bytes");
  if (!aligned16(qkv) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned16(workspace))
    return refuse("tree_attention: pointers must be 16-byte aligned");
  if (!workspace ||
      workspace_bytes < tree_attn_workspace(B, N, H, Hkv, D, dtype == GPT2_BF16))
    return refuse("tree_attention: workspace too small");
  try {
    TreeAttnArgs a{qkv, ld_qkv, k_cache, v_cache, lens, parent, counts, B, N, H, Hkv, H / Hkv, D,
                   Tc, out, ld_out, lse, static_cast<float*>(workspace), device_error_word(), nullptr,
                   zero};
    if (!a.err) return GPT2_ERR_CUDA;
    return launch_tree_attn(a, dtype == GPT2_BF16, static_cast<cudaStream_t>(stream));
  } catch (...) {
    return GPT2_ERR_OOM;
  }
}

int gpt2_tree_verify(const float* logits, int64_t ld, const float* draft_logits, int64_t ld_draft,
                     const int32_t* tokens, const int32_t* parent, const int32_t* counts,
                     const float* uniform, int B, int N, int V, float temperature, int top_k,
                     float top_p, int32_t* path, int32_t* n_path, int32_t* next, void* stream) {
  if (!logits || !tokens || !uniform || !path || !n_path || !next)
    return refuse("tree_verify: null pointer");
  if (B < 1 || B > 65535 || N < 1 || N > kTreeMaxNodes || V < 1 || V > kTreeMaxVocab || ld < V ||
      (draft_logits && ld_draft < V))
    return refuse("tree_verify: B, N (1..256), V (1..65536) or a row stride out of range");
  if (!(temperature >= 0.f && temperature <= 1e20f) || top_k < 0 ||
      !(top_p > 0.f && top_p <= 1.f))
    return refuse("tree_verify: bad sampling settings");
  // (a sequence's CTAs read while one of them writes)
  const uint64_t nodes = uint64_t(B) * N, rows = nodes - 1;
  const struct { const void* p; uint64_t n; } bufs[] = {
      {path, nodes}, {n_path, uint64_t(B)}, {next, uint64_t(B)}, {logits, rows * uint64_t(ld) + V},
      {draft_logits, rows * uint64_t(ld_draft) + V}, {tokens, nodes}, {parent, nodes}, {counts, uint64_t(B)},
      {uniform, nodes}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 9; ++j)
      if (overlap(bufs[i].p, bufs[i].n, bufs[j].p, bufs[j].n))
        return refuse("tree_verify: path, n_path and next must not overlap anything");
  try {
    TreeVerifyArgs a{logits, ld, draft_logits, ld_draft, tokens, parent, counts, uniform, B, N, V,
                     temperature, top_k, top_p, path, n_path, next, device_error_word()};
    if (!a.err) return GPT2_ERR_CUDA;
    return launch_tree_verify(a, static_cast<cudaStream_t>(stream));
  } catch (...) {
    return GPT2_ERR_OOM;
  }
}

int gpt2_kv_append(const void* qkv, int64_t ld_qkv, const int32_t* lens, const int32_t* path,
                   const int32_t* n_path, int dtype, int n_layer, int B, int N, int H, int Hkv,
                   int D, int Tc, void* k_cache, void* v_cache, int32_t* new_lens, void* stream) {
  if (!qkv || !lens || !k_cache || !v_cache) return refuse("kv_append: null pointer");
  if (!type_ok(dtype)) return refuse("kv_append: bad dtype");
  if (!heads_ok(B, N, H, Hkv, D) || Tc < 1 || n_layer < 1 || n_layer > 65535)
    return refuse("kv_append: n_layer, B, N (1..256), H, Hkv, D (16, 32, 64, 128) or Tc out of range");
  if (!row_ok(ld_qkv, dtype, (int64_t(H) + 2 * Hkv) * D))
    return refuse("kv_append: ld_qkv too small or not a multiple of 16 bytes");
  if (!aligned16(qkv) || !aligned16(k_cache) || !aligned16(v_cache))
    return refuse("kv_append: pointers must be 16-byte aligned");
  // (one block writes them while others have yet to read)
  if (overlap(new_lens, B, lens, B) || overlap(new_lens, B, n_path, B) ||
      overlap(new_lens, B, path, uint64_t(B) * N))
    return refuse("kv_append: new_lens must not overlap lens, n_path or path");
  try {
    KvAppendArgs a{qkv, ld_qkv, path, n_path, lens, n_layer, B, N, H, Hkv, D, Tc, k_cache, v_cache,
                   new_lens, device_error_word()};
    if (!a.err) return GPT2_ERR_CUDA;
    return launch_kv_append(a, dtype == GPT2_BF16 ? 2 : 4, static_cast<cudaStream_t>(stream));
  } catch (...) {
    return GPT2_ERR_OOM;
  }
}

}  // extern "C"
