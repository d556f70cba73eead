// Attention of drafted tokens over a key/value cache, the fp32 mode's
// CUDA-core kernel, head sizes 16, 32, 64 and 128.
//
// Source: [ZERO] "GPT training", Attention (softmax(q k^T / sqrt(D)) v over the
// positions a query may see); [CS336] section 5 (the cache that reuses the
// history).  The tree form has no counterpart on the pages: node i sees the
// cached positions and the nodes on its own path to the root.
//
// One pass over the keys with the running maximum m and sum l of each row
// (log2 domain): for a tile of scores s, m' = max(m, max s), p = 2^(s - m'),
// l' = l 2^(m - m') + sum p, o' = o 2^(m - m') + p v.  All of it in fp32.

#include "tree_attn.cuh"

using namespace tree;

namespace {

constexpr int kThreads = 128;
constexpr int MR = 16;  // query rows of a tile
constexpr int KT = 64;  // keys of a tile

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}

template <int D>
struct Smem {
  static constexpr int LD = D + 4;   // row stride: 8 rows of float4 hit 32 banks
  static constexpr int LP = KT + 4;
  float q[MR * LD];
  float k[KT * LD];
  float v[KT * LD];
  float p[MR * LP];
  alignas(16) uint32_t mask[kMaxNodes * kMaskWords];
  int up[kMaxNodes];
  SeqDims table[kTable];
  uint32_t flag;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) tree_attn_simt_kernel(const __grid_constant__ TreeAttnArgs a) {
  using S = Split<MR, KT, 2>;
  constexpr int LD = Smem<D>::LD, LP = Smem<D>::LP;
  constexpr int V4 = D / 4;              // float4 of a row
  constexpr int NO = (V4 + 7) / 8;       // float4 of the output a thread holds
  extern __shared__ float4 smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int tid = threadIdx.x;
  const int r = tid >> 3, kk = tid & 7;  // row of the tile, lane of the row
  asm volatile("griddepcontrol.launch_dependents;");
  auto pieces = S::plan(a, sm.table, threadIdx.x < 32);
  __syncthreads();
  int mask_of = -1;  // sequence whose masks are in shared memory
  const float scale = rsqrtf(float(D)) * kLog2e;
  const T* qkv = static_cast<const T*>(a.qkv);

  Piece p;
  while (pieces.next(p)) {
    const SeqDims s{p.len, p.n};
    const int b = p.b, hk = p.hk, rt = p.rt, t0 = p.t0, t1 = p.t1, ct = p.ct, rows = p.rows;
    if (tid == 0 && t0 == 0) pieces.note(p);
    const T* xb = qkv + int64_t(b) * a.N * a.ld_qkv;  // this sequence's nodes
    __syncthreads();  // the previous piece is done with shared memory
    for (int e = tid; e < MR * V4; e += kThreads) {
      const int rr = e / V4, c = e % V4;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (rr < rows) {
        const int gr = rt * MR + rr, node = gr / a.G, h = hk * a.G + gr % a.G;
        f = load4(xb + int64_t(node) * a.ld_qkv + int64_t(h) * D + c * 4);
        f.x *= scale; f.y *= scale; f.z *= scale; f.w *= scale;
      }
      *reinterpret_cast<float4*>(&sm.q[rr * LD + c * 4]) = f;
    }
    if (a.parent && t1 > ct && mask_of != b) {
      Parents parents;
      parents.load(a.parent + int64_t(b) * a.N, s.n, tid, kThreads);
      build_masks(parents, s.n, sm.mask, sm.up, &sm.flag, a.err, tid, kThreads,
                  [] { __syncthreads(); });
      mask_of = b;
    }
    const int node = r < rows ? (rt * MR + r) / a.G : 0;
    float m = -INFINITY, l = 0.f;
    float4 o[NO];
#pragma unroll
    for (int j = 0; j < NO; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);

    for (int t = t0; t < t1; ++t) {
      const bool fresh = t >= ct;  // keys are nodes, not cache rows
      const int k0 = (fresh ? t - ct : t) * KT;
      const int nk = min(KT, (fresh ? s.n : s.len) - k0);
      const T *kp, *vp;
      int64_t ld;
      if (fresh) {
        kp = xb + int64_t(k0) * a.ld_qkv + int64_t(a.H + hk) * D;
        vp = kp + int64_t(a.Hkv) * D;
        ld = a.ld_qkv;
      } else {
        const int64_t base = ((int64_t(b) * a.Hkv + hk) * a.Tc + k0) * D;
        kp = static_cast<const T*>(a.k) + base;
        vp = static_cast<const T*>(a.v) + base;
        ld = D;
      }
      for (int e = tid; e < KT * V4; e += kThreads) {
        const int row = e / V4, c = e % V4;
        float4 fk = make_float4(0.f, 0.f, 0.f, 0.f), fv = fk;
        if (row < nk) {
          fk = load4(kp + row * ld + c * 4);
          fv = load4(vp + row * ld + c * 4);
        }
        *reinterpret_cast<float4*>(&sm.k[row * LD + c * 4]) = fk;
        *reinterpret_cast<float4*>(&sm.v[row * LD + c * 4]) = fv;
      }
      __syncthreads();
      if (rows > (r & ~3)) {  // some row of this warp is real
        float sc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sc[j] = 0.f;
#pragma unroll 4
        for (int c = 0; c < V4; ++c) {
          const float4 q4 = *reinterpret_cast<const float4*>(&sm.q[r * LD + c * 4]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 k4 = *reinterpret_cast<const float4*>(&sm.k[(kk + 8 * j) * LD + c * 4]);
            sc[j] = fmaf(q4.x, k4.x, sc[j]);
            sc[j] = fmaf(q4.y, k4.y, sc[j]);
            sc[j] = fmaf(q4.z, k4.z, sc[j]);
            sc[j] = fmaf(q4.w, k4.w, sc[j]);
          }
        }
        float mx = m;
        const uint64_t see = fresh ? sees(!a.parent, sm.mask, node, k0) : ~uint64_t(0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = kk + 8 * j;
          if (key >= nk || !((see >> key) & 1)) sc[j] = -INFINITY;
          mx = fmaxf(mx, sc[j]);
        }
#pragma unroll
        for (int x = 1; x < 8; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        // a row that has seen nothing yet: every p is 2^(-inf) = 0
        const float base = mx == -INFINITY ? 0.f : mx;
        const float alpha = exp2f(m - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float pj = exp2f(sc[j] - base);
          sum += pj;
          sm.p[r * LP + kk + 8 * j] = pj;
        }
#pragma unroll
        for (int x = 1; x < 8; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l = fmaf(l, alpha, sum);
        m = mx;
#pragma unroll
        for (int j = 0; j < NO; ++j) {
          o[j].x *= alpha; o[j].y *= alpha; o[j].z *= alpha; o[j].w *= alpha;
        }
        __syncwarp();  // a row's probabilities are written and read by one warp
        for (int key = 0; key < nk; ++key) {
          const float p = sm.p[r * LP + key];
          // a node outside the path may hold anything (0 * inf is not 0)
          if (fresh && p == 0.f) continue;
#pragma unroll
          for (int j = 0; j < NO; ++j) {
            if (kk + 8 * j < V4) {
              const float4 v4 =
                  *reinterpret_cast<const float4*>(&sm.v[key * LD + (kk + 8 * j) * 4]);
              o[j].x = fmaf(p, v4.x, o[j].x);
              o[j].y = fmaf(p, v4.y, o[j].y);
              o[j].z = fmaf(p, v4.z, o[j].z);
              o[j].w = fmaf(p, v4.w, o[j].w);
            }
          }
        }
      }
      __syncthreads();
    }

    if (p.whole()) {  // finished here
      if (r < rows) {
        const int gr = rt * MR + r, h = hk * a.G + gr % a.G;
        T* out = static_cast<T*>(a.out) + (int64_t(b) * a.N + node) * a.ld_out + int64_t(h) * D;
        const float inv = 1.f / l;
#pragma unroll
        for (int j = 0; j < NO; ++j) {
          const int c = (kk + 8 * j) * 4;
          if (c < D) {
            out[c] = from_f32<T>(o[j].x * inv);
            out[c + 1] = from_f32<T>(o[j].y * inv);
            out[c + 2] = from_f32<T>(o[j].z * inv);
            out[c + 3] = from_f32<T>(o[j].w * inv);
          }
        }
        if (a.lse && kk == 0)
          a.lse[(int64_t(b) * a.H + h) * a.N + node] = (m + log2f(l)) * kLn2;
      }
    } else {
      float* w = a.ws + pieces.slot(p) * slot_floats<MR>(D);
      if (r < rows) {
#pragma unroll
        for (int j = 0; j < NO; ++j)
          if (kk + 8 * j < V4) *reinterpret_cast<float4*>(&w[r * D + (kk + 8 * j) * 4]) = o[j];
        if (kk == 0) {
          w[MR * D + r] = m;
          w[MR * D + MR + r] = l;
        }
      }
    }
  }
}

int simt_grid() { return 4 * gpt2_internal::sm_count(); }

template <typename T, int D>
int launch_simt(const TreeAttnArgs& a, cudaStream_t st) {
  const int smem = int(sizeof(Smem<D>));
  GPT2_CUDA_TRY(cudaFuncSetAttribute(tree_attn_simt_kernel<T, D>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  const int grid = simt_grid();
  const TreeAttnArgs w = with_workspace<MR>(a, grid);
  tree_attn_simt_kernel<T, D><<<grid, kThreads, smem, st>>>(w);
  COUNT_LAUNCH(1);
  GPT2_LAUNCH_CHECK();
  return launch_combine<T, MR, D>(w, st);
}

template <typename T>
int launch_simt_d(const TreeAttnArgs& a, cudaStream_t st) {
  switch (a.D) {
    case 16: return launch_simt<T, 16>(a, st);
    case 32: return launch_simt<T, 32>(a, st);
    case 64: return launch_simt<T, 64>(a, st);
    default: return launch_simt<T, 128>(a, st);
  }
}

}  // namespace

size_t tree_attn_mma_workspace(int B, int N, int H, int Hkv, int D);
int launch_tree_attn_mma(const TreeAttnArgs& a, cudaStream_t st);
size_t tree_attn_tc_workspace(int B, int N, int H, int Hkv, int D);
int launch_tree_attn_tc(const TreeAttnArgs& a, cudaStream_t st);

// bf16 with head size 64 or 128 and more than 32 query rows per key/value head
// goes to the 5th-generation tensor cores: their tile of 128 rows costs the same
// however few are real, the warp-level instructions grow with the rows.  Measured
// (head size 64, us, warp level / 5th generation): 16 sequences of 500-1000, 16
// rows 18.5 / 21.6, 32 rows 22.3 / 23.5, 48 rows 26.4 / 23.8, 64 rows 27.7 / 24.8;
// 4 sequences of 8-16 thousand, 32 rows 36.4 / 35.1, 48 rows 49.1 / 40.0.
static bool on_tc(int N, int H, int Hkv, int D) { return D >= 64 && N * (H / Hkv) > 32; }

size_t tree_attn_workspace(int B, int N, int H, int Hkv, int D, int bf16_in) {
  if (!bf16_in) return workspace_bytes<MR>(simt_grid(), B, N, H, Hkv, D);
  return on_tc(N, H, Hkv, D) ? tree_attn_tc_workspace(B, N, H, Hkv, D)
                             : tree_attn_mma_workspace(B, N, H, Hkv, D);
}

int launch_tree_attn(const TreeAttnArgs& a, int bf16_in, cudaStream_t st) {
  if (!bf16_in) return launch_simt_d<float>(a, st);
  return on_tc(a.N, a.H, a.Hkv, a.D) ? launch_tree_attn_tc(a, st) : launch_tree_attn_mma(a, st);
}
