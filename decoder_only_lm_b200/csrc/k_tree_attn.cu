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
//
// Keys and values come by asynchronous copies, each while the other is used: the
// next tile's keys during a tile's product with V, its values during the next
// scores, so two buffers do for the overlap (B200, 16 single tokens over 500-2000
// positions, 12 heads of 64: 48 -> 35 us, 3.5 TB/s; trees of 13 over up to 1000,
// 4 sequences: 14 us; trees of up to 64 over 500-2000, 8 sequences: 83 us, 18
// TFLOP/s, bound by shared memory reads).

#include <type_traits>

#include "tree_attn.cuh"

using namespace tree;

namespace {

constexpr int kThreads = 128;
constexpr int KT = 64;  // keys of a tile

// A thread holds RQ x KQ scores of a tile (rows x keys) and RQ rows x NO vectors
// of 4 channels of its output: KL lanes share RQ rows.  What bounds the kernel is
// the shared memory's 128 bytes a clock: a step over 4 channels loads RQ + KQ
// vectors for 4 RQ KQ multiply-adds, so more rows a thread are better where there
// are rows.
template <int D, int MR_>
struct Cfg {
  static constexpr int MR = MR_;                   // query rows of a tile
  static constexpr int KQ = MR == 16 ? 4 : 8;
  static constexpr int KL = KT / KQ;
  static constexpr int RQ = MR * KL / kThreads;
  static constexpr int V4 = D / 4;                 // float4 of a row
  static constexpr int NO = (V4 + KL - 1) / KL;
  static constexpr int LD = D + 4;                 // row strides: 8 rows of float4 hit
  static constexpr int LP = KT + 4;                // 32 banks
  static constexpr int kLoads = KT * V4 / kThreads;  // float4 of K (and V) a thread
  static constexpr int kCtas = MR == 16 ? (D == 128 ? 2 : 4) : 2;  // per SM
  struct Smem {
    float q[MR * LD];
    float k[KT * LD];
    float v[KT * LD];
    float p[MR * LP];
    alignas(16) uint32_t mask[kMaxNodes * kMaskWords];
    int up[kMaxNodes];
    SeqDims table[kTable];
    uint32_t flag;
  };
};

__device__ __forceinline__ void cp_async16(float* dst, const float* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   uint32_t(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(real ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ void fma4(float4& o, float p, const float4& v) {
  o.x = fmaf(p, v.x, o.x);
  o.y = fmaf(p, v.y, o.y);
  o.z = fmaf(p, v.z, o.z);
  o.w = fmaf(p, v.w, o.w);
}

template <int D, int MR>
__global__ void __launch_bounds__(kThreads, Cfg<D, MR>::kCtas)
    tree_attn_simt_kernel(const __grid_constant__ TreeAttnArgs a) {
  using S = Split<MR, KT, 2>;
  using C = Cfg<D, MR>;
  constexpr int LD = C::LD, LP = C::LP, V4 = C::V4, NO = C::NO, KL = C::KL, KQ = C::KQ, RQ = C::RQ;
  extern __shared__ float4 smem_raw[];
  auto& sm = *reinterpret_cast<typename C::Smem*>(smem_raw);
  const int tid = threadIdx.x;
  const int r0 = tid / KL * RQ, kk = tid % KL;  // first row, lane of its rows
  const int warp_row = tid / 32 * (32 / KL) * RQ;
  asm volatile("griddepcontrol.launch_dependents;");
  auto pieces = S::plan(a, sm.table, threadIdx.x < 32);
  __syncthreads();
  int mask_of = -1;  // sequence whose masks are in shared memory
  const float scale = rsqrtf(float(D)) * kLog2e;
  const float* qkv = static_cast<const float*>(a.qkv);

  Piece p;
  while (pieces.next(p)) {
    const SeqDims s{p.len, p.n};
    const int b = p.b, hk = p.hk, rt = p.rt, t0 = p.t0, t1 = p.t1, ct = p.ct, rows = p.rows;
    if (tid == 0 && t0 == 0) pieces.note(p);
    const float* xb = qkv + int64_t(b) * a.N * a.ld_qkv;  // this sequence's nodes
    __syncthreads();  // the previous piece is done with shared memory
    // K (or V) of tile t on its way to shared memory, zeros behind the last key
    auto bring = [&](int t, bool is_v) {
      if (t < t1) {
        const bool fresh = t >= ct;  // keys are nodes, not cache rows
        const int k0 = (fresh ? t - ct : t) * KT;
        const int nk = min(KT, (fresh ? s.n : s.len) - k0);
        const float* src;
        int64_t ld;
        if (fresh) {
          src = xb + int64_t(k0) * a.ld_qkv + int64_t(a.H + hk + (is_v ? a.Hkv : 0)) * D;
          ld = a.ld_qkv;
        } else {
          src = static_cast<const float*>(is_v ? a.v : a.k) +
                ((int64_t(b) * a.Hkv + hk) * a.Tc + k0) * D;
          ld = D;
        }
        float* dst = is_v ? sm.v : sm.k;
#pragma unroll
        for (int i = 0; i < C::kLoads; ++i) {
          const int e = tid + i * kThreads, row = e / V4, c = e % V4;
          cp_async16(&dst[row * LD + c * 4], row < nk ? src + row * ld + c * 4 : src, row < nk);
        }
      }
      asm volatile("cp.async.commit_group;");
    };
    bring(t0, false);
    bring(t0, true);
    for (int e = tid; e < MR * V4; e += kThreads) {
      const int rr = e / V4, c = e % V4;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (rr < rows) {
        const int gr = rt * MR + rr, node = gr / a.G, h = hk * a.G + gr % a.G;
        f = *reinterpret_cast<const float4*>(xb + int64_t(node) * a.ld_qkv + int64_t(h) * D + c * 4);
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
    float m[RQ], l[RQ];
    float4 o[RQ][NO];
#pragma unroll
    for (int i = 0; i < RQ; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NO; ++j) o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }

    for (int t = t0; t < t1; ++t) {
      const bool fresh = t >= ct;
      const int k0 = (fresh ? t - ct : t) * KT;
      const int nk = min(KT, (fresh ? s.n : s.len) - k0);
      const bool busy = rows > warp_row;  // some row of this warp is real
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();  // K is there
      float sc[RQ][KQ];
      if (busy) {
#pragma unroll
        for (int i = 0; i < RQ; ++i)
#pragma unroll
          for (int j = 0; j < KQ; ++j) sc[i][j] = 0.f;
#pragma unroll 2
        for (int c = 0; c < V4; ++c) {
          float4 q4[RQ];
#pragma unroll
          for (int i = 0; i < RQ; ++i)
            q4[i] = *reinterpret_cast<const float4*>(&sm.q[(r0 + i) * LD + c * 4]);
#pragma unroll
          for (int j = 0; j < KQ; ++j) {
            const float4 k4 = *reinterpret_cast<const float4*>(&sm.k[(kk + KL * j) * LD + c * 4]);
#pragma unroll
            for (int i = 0; i < RQ; ++i) {
              sc[i][j] = fmaf(q4[i].x, k4.x, sc[i][j]);
              sc[i][j] = fmaf(q4[i].y, k4.y, sc[i][j]);
              sc[i][j] = fmaf(q4[i].z, k4.z, sc[i][j]);
              sc[i][j] = fmaf(q4[i].w, k4.w, sc[i][j]);
            }
          }
        }
      }
      __syncthreads();  // K is read: the next one may come while this tile's V is used
      bring(t + 1, false);
      if (busy) {
#pragma unroll
        for (int i = 0; i < RQ; ++i) {
          const int node = r0 + i < rows ? (rt * MR + r0 + i) / a.G : 0;
          float mx = m[i];
          const uint64_t see = fresh ? sees(!a.parent, sm.mask, node, k0) : ~uint64_t(0);
#pragma unroll
          for (int j = 0; j < KQ; ++j) {
            const int key = kk + KL * j;
            if (key >= nk || !((see >> key) & 1)) sc[i][j] = -INFINITY;
            mx = fmaxf(mx, sc[i][j]);
          }
#pragma unroll
          for (int x = 1; x < KL; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
          // a row that has seen nothing yet: every p is 2^(-inf) = 0
          const float base = mx == -INFINITY ? 0.f : mx;
          const float alpha = exp2f(m[i] - base);
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < KQ; ++j) {
            const float pj = exp2f(sc[i][j] - base);
            sum += pj;
            sm.p[(r0 + i) * LP + kk + KL * j] = pj;
          }
#pragma unroll
          for (int x = 1; x < KL; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          l[i] = fmaf(l[i], alpha, sum);
          m[i] = mx;
#pragma unroll
          for (int j = 0; j < NO; ++j) {
            o[i][j].x *= alpha; o[i][j].y *= alpha; o[i][j].z *= alpha; o[i][j].w *= alpha;
          }
        }
      }
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();  // V is there (and the probabilities)
      if (busy) {
        auto product = [&](auto is_fresh) {
#pragma unroll 1
          for (int key0 = 0; key0 < nk; key0 += 4) {  // (p and v are 0 from nk on)
            float pk[RQ][4];
#pragma unroll
            for (int i = 0; i < RQ; ++i) {
              const float4 p4 = *reinterpret_cast<const float4*>(&sm.p[(r0 + i) * LP + key0]);
              pk[i][0] = p4.x, pk[i][1] = p4.y, pk[i][2] = p4.z, pk[i][3] = p4.w;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int j = 0; j < NO; ++j) {
                if (NO * KL > V4 && kk + KL * j >= V4) continue;
                const float4 v4 =
                    *reinterpret_cast<const float4*>(&sm.v[(key0 + x) * LD + (kk + KL * j) * 4]);
#pragma unroll
                for (int i = 0; i < RQ; ++i)
                  // a node outside the path may hold anything (0 * inf is not 0)
                  if (!decltype(is_fresh)::value || pk[i][x] != 0.f) fma4(o[i][j], pk[i][x], v4);
              }
          }
        };
        if (fresh)
          product(std::true_type());
        else
          product(std::false_type());
      }
      __syncthreads();  // V is read
      bring(t + 1, true);
    }

    float* w = p.whole() ? nullptr : a.ws + pieces.slot(p) * slot_floats<MR>(D);
#pragma unroll
    for (int i = 0; i < RQ; ++i) {
      const int r = r0 + i;
      if (r >= rows) continue;
      if (!w) {  // finished here
        const int gr = rt * MR + r, node = gr / a.G, h = hk * a.G + gr % a.G;
        float* out = static_cast<float*>(a.out) + (int64_t(b) * a.N + node) * a.ld_out + int64_t(h) * D;
        const float inv = 1.f / l[i];
#pragma unroll
        for (int j = 0; j < NO; ++j)
          if (kk + KL * j < V4)
            *reinterpret_cast<float4*>(out + (kk + KL * j) * 4) =
                make_float4(o[i][j].x * inv, o[i][j].y * inv, o[i][j].z * inv, o[i][j].w * inv);
        if (a.lse && kk == 0)
          a.lse[(int64_t(b) * a.H + h) * a.N + node] = (m[i] + log2f(l[i])) * kLn2;
      } else {
#pragma unroll
        for (int j = 0; j < NO; ++j)
          if (kk + KL * j < V4) *reinterpret_cast<float4*>(&w[r * D + (kk + KL * j) * 4]) = o[i][j];
        if (kk == 0) {
          w[MR * D + r] = m[i];
          w[MR * D + MR + r] = l[i];
        }
      }
    }
  }
}

template <int D, int MR>
int simt_grid() { return Cfg<D, MR>::kCtas * gpt2_internal::sm_count(); }

template <int D, int MR>
int launch_simt(const TreeAttnArgs& a, cudaStream_t st) {
  const int smem = int(sizeof(typename Cfg<D, MR>::Smem));
  static std::atomic<uint64_t> allowed{0};
  GPT2_CUDA_TRY(allow_smem(allowed, tree_attn_simt_kernel<D, MR>, smem));
  const int grid = simt_grid<D, MR>();
  const TreeAttnArgs w = with_workspace<MR>(a, grid);
  tree_attn_simt_kernel<D, MR><<<grid, kThreads, smem, st>>>(w);
  COUNT_LAUNCH(1);
  GPT2_LAUNCH_CHECK();
  return launch_combine<float, MR, D>(w, st);
}

// Calls f with the fp32 kernel's head size and rows of a tile as constants.  Few
// query rows per key/value head take tiles of 16, more of them tiles that read a
// key once for 64 (head size 128: 32, two CTAs on an SM).  Measured (us, tiles of
// 16 / of more): head size 64, 16 sequences of 500-2000, 32 rows 99 / 144, 48 rows
// 137 / 150, 64 rows 168 / 156, 4 sequences to 1000, 48 rows 31 / 30, 64 rows
// 37 / 31; head size 128, 16 sequences, 16 rows 121 / 149, 24 rows 169 / 160, 4
// sequences, 16 rows 24 / 29, 24 rows 40 / 31.
template <typename F>
auto simt_variant(int N, int H, int Hkv, int D, F f) {
  const bool few = N * (H / Hkv) <= (D == 128 ? 16 : 48);
  using std::integral_constant;
  switch (D) {
    case 16:
      return few ? f(integral_constant<int, 16>(), integral_constant<int, 16>())
                 : f(integral_constant<int, 16>(), integral_constant<int, 64>());
    case 32:
      return few ? f(integral_constant<int, 32>(), integral_constant<int, 16>())
                 : f(integral_constant<int, 32>(), integral_constant<int, 64>());
    case 64:
      return few ? f(integral_constant<int, 64>(), integral_constant<int, 16>())
                 : f(integral_constant<int, 64>(), integral_constant<int, 64>());
    default:
      return few ? f(integral_constant<int, 128>(), integral_constant<int, 16>())
                 : f(integral_constant<int, 128>(), integral_constant<int, 32>());
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
  if (!bf16_in)
    return simt_variant(N, H, Hkv, D, [&](auto d, auto mr) {
      return workspace_bytes<mr()>(simt_grid<d(), mr()>(), B, N, H, Hkv, D);
    });
  return on_tc(N, H, Hkv, D) ? tree_attn_tc_workspace(B, N, H, Hkv, D)
                             : tree_attn_mma_workspace(B, N, H, Hkv, D);
}

int launch_tree_attn(const TreeAttnArgs& a, int bf16_in, cudaStream_t st) {
  if (!bf16_in)
    return simt_variant(a.N, a.H, a.Hkv, a.D,
                        [&](auto d, auto mr) { return launch_simt<d(), mr()>(a, st); });
  return on_tc(a.N, a.H, a.Hkv, a.D) ? launch_tree_attn_tc(a, st) : launch_tree_attn_mma(a, st);
}
