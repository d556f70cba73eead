// Attention of drafted tokens over a key/value cache for bf16: warp-level
// matrix instructions (m16n8k16, fp32 accumulation) over tiles of 64 keys.
//
// Source and split of the work: as the CUDA-core kernel and tree_attn.cuh.
//
// A step of decoding reads every cached key and value once and does little with
// them: with R = N G query rows per key/value head it is R FLOP a byte, so up
// to a few hundred rows the cache's bandwidth bounds it, and what matters is
// enough loads in flight.  A warp holds 16 query rows in registers (queries,
// running maximum and sum, output); WM warps cover the rows of a tile and WK
// warps share its keys (few rows: all warps split the keys and merge their
// results at the end of a piece; then no warp waits for another while it
// streams).  Key and value tiles come by 16-byte asynchronous copies into a
// ring of stages, with the 16-byte chunks of a row XOR-swizzled so that the
// matrix loads of 8 rows touch all banks.
//
// Scores and probabilities stay in registers: the accumulator layout of
// S = Q K^T is the operand layout of P for O += P V.  P is rounded to bf16 for
// that product (the tensor cores' operand type; the sums of p stay fp32), as
// in the training attention.

#include "tree_attn.cuh"

using namespace tree;

namespace {

constexpr int KT = 64;  // keys of a tile

template <int D, int WM, int WK>
struct Cfg {
  static constexpr int kThreads = 32 * WM * WK;
  static constexpr int MR = 16 * WM;
  static constexpr int KW = KT / WK;          // keys of a warp
  static constexpr int kTile = KT * D * 2;    // bytes of a K (or V) tile
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kRing = kStages * 2 * kTile;
  static constexpr int LO = D + 4;            // row stride of the merge buffer
  static constexpr int kMerge = WK > 1 ? WK * MR * (LO + 2) * 4 : 0;
  static constexpr int kBuf = kRing > kMerge ? kRing : kMerge;
  static constexpr int kSmem = kBuf + kMaxNodes * (kMaskWords + 1) * 4 + 16 + kTable * 8;
  static constexpr int kCtas = WM == 8 ? (D == 128 ? 1 : 2) : D == 128 ? 2 : 3;  // per SM
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes, or zeros where `real` is false
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
// Byte offset of 16-byte chunk c of row r in a tile of D bf16 a row: the chunk
// index is XORed with row bits so that 8 consecutive rows at one chunk fall
// into 8 different 16-byte bank groups.
template <int D>
__device__ __forceinline__ uint32_t at(int r, int c) {
  constexpr int C = D / 8;  // chunks of a row
  const int x = C >= 8 ? (r & 7) : C == 4 ? ((r >> 1) & 3) : ((r >> 2) & 1);
  return uint32_t(r * C + (c ^ x)) * 16;
}

template <int D, int WM, int WK>
__global__ void __launch_bounds__(Cfg<D, WM, WK>::kThreads, Cfg<D, WM, WK>::kCtas)
    tree_attn_mma_kernel(TreeAttnArgs a) {
  using F = Cfg<D, WM, WK>;
  using S = Split<F::MR, KT>;
  constexpr int MR = F::MR, KW = F::KW, ST = F::kStages;
  constexpr int NT = KW / 8;   // score tiles of 8 keys
  constexpr int DT = D / 8;    // output tiles of 8 channels
  constexpr int KS = D / 16;   // steps of the score product
  constexpr int C = D / 8;     // 16-byte chunks of a row
  // with all warps splitting the keys each streams its own rows of the tiles
  constexpr bool kOwn = WM == 1;
  extern __shared__ uint4 smem_raw[];
  char* buf = reinterpret_cast<char*>(smem_raw);
  const uint32_t ring = smem_addr(buf);
  uint32_t* mask = reinterpret_cast<uint32_t*>(buf + F::kBuf);
  int* up = reinterpret_cast<int*>(mask + kMaxNodes * kMaskWords);
  uint32_t* odd = reinterpret_cast<uint32_t*>(up + kMaxNodes);  // 64 bits: keys of non-finite V
  SeqDims* table = reinterpret_cast<SeqDims*>(odd + 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp % WM, wk = warp / WM;
  const int gr = lane >> 2, gc = lane & 3;  // fragment row and column pair
  asm volatile("griddepcontrol.launch_dependents;");
  auto pieces = S::plan(a, table);
  __syncthreads();
  int mask_of = -1;
  const float scale = rsqrtf(float(D)) * kLog2e;
  const bf16* qkv = static_cast<const bf16*>(a.qkv);

  Piece pc;
  while (pieces.next(pc)) {
    const SeqDims s{pc.len, pc.n};
    const int b = pc.b, hk = pc.hk, rt = pc.rt, t0 = pc.t0, t1 = pc.t1, ct = pc.ct, rows = pc.rows;
    if (tid == 0 && t0 == 0) pieces.note(pc);
    const bf16* xb = qkv + int64_t(b) * a.N * a.ld_qkv;
    const bf16* kc = static_cast<const bf16*>(a.k) + (int64_t(b) * a.Hkv + hk) * a.Tc * D;
    const bf16* vc = static_cast<const bf16*>(a.v) + (int64_t(b) * a.Hkv + hk) * a.Tc * D;
    const bf16* kn = xb + int64_t(a.H + hk) * D;
    const bf16* vn = kn + int64_t(a.Hkv) * D;
    __syncthreads();  // the previous piece is done with shared memory

    // one stage: the keys and values of tile t (zeros behind the last one)
    auto load = [&](int t) {
      if (t < t1) {
        const bool fresh = t >= ct;
        const int k0 = (fresh ? t - ct : t) * KT;
        const int nk = (fresh ? s.n : s.len) - k0;
        const bf16* kp = fresh ? kn + k0 * a.ld_qkv : kc + int64_t(k0) * D;
        const bf16* vp = fresh ? vn + k0 * a.ld_qkv : vc + int64_t(k0) * D;
        const int64_t ld = fresh ? a.ld_qkv : D;
        const uint32_t dk = ring + uint32_t((t - t0) % ST) * (2 * F::kTile), dv = dk + F::kTile;
        constexpr int kRows = kOwn ? KW : KT, kBy = kOwn ? 32 : F::kThreads;
        const int r0 = kOwn ? wk * KW : 0, me = kOwn ? lane : tid;
#pragma unroll
        for (int e0 = 0; e0 < kRows * C; e0 += kBy) {
          const int e = e0 + me;
          if (kRows * C % kBy == 0 || e < kRows * C) {
            const int r = r0 + e / C, c = e % C;
            const bool real = r < nk;
            const int64_t off = real ? r * ld + c * 8 : 0;
            copy16(dk + at<D>(r, c), kp + off, real);
            copy16(dv + at<D>(r, c), vp + off, real);
          }
        }
      }
      copy_commit();
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) load(t0 + i);

    // this warp's 16 query rows as matrix operands; zeros behind the last row
    uint32_t q[KS][4];
    int node[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = wm * 16 + gr + 8 * h;
      const bool real = r < rows;
      const int g = rt * MR + (real ? r : 0);
      node[h] = g / a.G;
      const bf16* p = xb + int64_t(node[h]) * a.ld_qkv + int64_t(hk * a.G + g % a.G) * D + 2 * gc;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        q[k][h] = real ? *reinterpret_cast<const uint32_t*>(p + 16 * k) : 0u;
        q[k][2 + h] = real ? *reinterpret_cast<const uint32_t*>(p + 16 * k + 8) : 0u;
      }
    }
    if (a.parent && t1 > ct && mask_of != b) {
      build_masks(a.parent + int64_t(b) * a.N, s.n, mask, up, odd + 2, a.err, tid, F::kThreads,
                  [] { __syncthreads(); });
      mask_of = b;
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[DT][4];
#pragma unroll
    for (int j = 0; j < DT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    const bool busy = wm * 16 < rows;  // some row of this warp is real

    for (int t = t0; t < t1; ++t) {
      const bool fresh = t >= ct;
      copy_wait<ST - 2>();
      // the tile has landed for every thread that reads it, and the stage
      // loaded next has been read by all
      if (kOwn && !fresh)
        __syncwarp();
      else
        __syncthreads();
      load(t + ST - 1);
      const int k0 = (fresh ? t - ct : t) * KT;
      const int nk = (fresh ? s.n : s.len) - k0 - wk * KW;  // keys of this warp
      const uint32_t sk = ring + uint32_t((t - t0) % ST) * (2 * F::kTile), sv = sk + F::kTile;
      uint64_t bad_v = 0;
      if (fresh) {
        // A node that a row may not see can hold anything, and 0 times a
        // non-finite value is not 0: such value rows become 0 for the product
        // and reach the rows that see them one by one below.
        if (tid < 2) odd[tid] = 0;
        __syncthreads();
        char* vt = buf + (sv - ring);
        for (int e = tid; e < KT * C; e += F::kThreads) {
          const uint4 u = *reinterpret_cast<const uint4*>(vt + at<D>(e / C, e % C));
          auto inf = [](uint32_t w) {
            return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
          };
          if (inf(u.x) || inf(u.y) || inf(u.z) || inf(u.w))
            atomicOr(&odd[(e / C) >> 5], 1u << ((e / C) & 31));
        }
        __syncthreads();
        bad_v = odd[0] | (uint64_t(odd[1]) << 32);
        if (bad_v) {
          for (int e = tid; e < KT * C; e += F::kThreads)
            if ((bad_v >> (e / C)) & 1)
              *reinterpret_cast<uint4*>(vt + at<D>(e / C, e % C)) = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
      }
      if (!busy || nk <= 0) continue;
      // scores
      float sc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
        const int r = wk * KW + j * 8 + (lane & 7);
        if (KS >= 2) {
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint32_t kb[4];
            ldm4(kb, sk + at<D>(r, 2 * k + (lane >> 3)));
            mma16816(sc[j], q[k], kb[0], kb[1]);
            mma16816(sc[j], q[(k + 1) % KS], kb[2], kb[3]);
          }
        }
      }
      if (KS == 1) {  // D = 16: one step, two key tiles a load
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          uint32_t kb[4];
          ldm4(kb, sk + at<D>(wk * KW + j * 8 + (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1));
          mma16816(sc[j], q[0], kb[0], kb[1]);
          mma16816(sc[j + 1], q[0], kb[2], kb[3]);
        }
      }
      if (fresh || nk < KW) {
        uint64_t see[2] = {~uint64_t(0), ~uint64_t(0)};
        if (fresh) {
          see[0] = sees(!a.parent, mask, node[0], k0) >> (wk * KW);
          see[1] = sees(!a.parent, mask, node[1], k0) >> (wk * KW);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = j * 8 + gc * 2 + (e & 1);
            if (key >= nk || !((see[e >> 1] >> key) & 1)) sc[j][e] = -INFINITY;
          }
      }
      // running maximum (log2 domain: s scale), probabilities, sums
      float base[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = m[h];
#pragma unroll
        for (int j = 0; j < NT; ++j)
          mx = fmaxf(mx, fmaxf(sc[j][2 * h], sc[j][2 * h + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // a row that has seen nothing yet: every p is 2^(-inf) = 0
        // (products rounded, not fused: an unchanged maximum gives alpha = 1)
        base[h] = mx == -INFINITY ? 0.f : __fmul_rn(mx, scale);
        const float alpha = ex2(__fmul_rn(m[h], scale) - base[h]);
        m[h] = mx;
        l[h] *= alpha;
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
          for (int j = 0; j < DT; ++j) {
            o[j][2 * h] *= alpha;
            o[j][2 * h + 1] *= alpha;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[j][e] = ex2(fmaf(sc[j][e], scale, -base[e >> 1]));
          l[e >> 1] += sc[j][e];
        }
      // O += P V
#pragma unroll
      for (int k = 0; k < NT / 2; ++k) {
        uint32_t p[4] = {pack2(sc[2 * k][0], sc[2 * k][1]), pack2(sc[2 * k][2], sc[2 * k][3]),
                         pack2(sc[2 * k + 1][0], sc[2 * k + 1][1]),
                         pack2(sc[2 * k + 1][2], sc[2 * k + 1][3])};
        const int r = wk * KW + k * 16 + (lane & 15);
#pragma unroll
        for (int j = 0; j < DT; j += 2) {
          uint32_t vb[4];
          ldm4_trans(vb, sv + at<D>(r, j + (lane >> 4)));
          mma16816(o[j], p, vb[0], vb[1]);
          mma16816(o[j + 1], p, vb[2], vb[3]);
        }
      }
      if (bad_v) {
        for (int key = 0; key < KW; ++key) {
          if (!((bad_v >> (wk * KW + key)) & 1)) continue;
          float p0 = 0.f, p1 = 0.f;  // from the lane of the row that holds this key
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (j * 8 + e == (key & ~7) + (key & 1)) {
                p0 = sc[j][e];
                p1 = sc[j][2 + e];
              }
          const int src = (lane & ~3) | ((key & 7) >> 1);
          p0 = __shfl_sync(0xffffffffu, p0, src);
          p1 = __shfl_sync(0xffffffffu, p1, src);
          const bf16* v = vn + (k0 + wk * KW + key) * a.ld_qkv;
#pragma unroll
          for (int j = 0; j < DT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float ve = __bfloat162float(v[j * 8 + gc * 2 + e]);
              if (p0 != 0.f) o[j][e] = fmaf(p0, ve, o[j][e]);
              if (p1 != 0.f) o[j][2 + e] = fmaf(p1, ve, o[j][2 + e]);
            }
        }
      }
    }
    copy_wait<0>();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      m[h] = __fmul_rn(m[h], scale);  // log2 domain, the base of the sums
    }
    const bool whole = pc.whole();
    float* w = a.ws + pieces.slot(pc) * slot_floats<MR>(D);
    bf16* out = static_cast<bf16*>(a.out) + int64_t(b) * a.N * a.ld_out;
    if (WK == 1) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = wm * 16 + gr + 8 * h;
        if (r >= rows) continue;
        if (whole) {
          const int hq = hk * a.G + (rt * MR + r) % a.G;
          bf16* p = out + int64_t(node[h]) * a.ld_out + int64_t(hq) * D + 2 * gc;
          const float inv = 1.f / l[h];
#pragma unroll
          for (int j = 0; j < DT; ++j)
            *reinterpret_cast<uint32_t*>(p + 8 * j) = pack2(o[j][2 * h] * inv, o[j][2 * h + 1] * inv);
          if (a.lse && gc == 0)
            a.lse[(int64_t(b) * a.H + hq) * a.N + node[h]] = (m[h] + log2f(l[h])) * kLn2;
        } else {
#pragma unroll
          for (int j = 0; j < DT; ++j)
            *reinterpret_cast<float2*>(w + r * D + 8 * j + 2 * gc) =
                make_float2(o[j][2 * h], o[j][2 * h + 1]);
          if (gc == 0) {
            w[MR * D + r] = m[h];
            w[MR * D + MR + r] = l[h];
          }
        }
      }
    } else {
      // the warps' results over the same rows, merged in warp order
      float* ex = reinterpret_cast<float*>(buf);
      float* ml = ex + WK * MR * F::LO;
      __syncthreads();  // the last tile has been read
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = wk * MR + wm * 16 + gr + 8 * h;
#pragma unroll
        for (int j = 0; j < DT; ++j)
          *reinterpret_cast<float2*>(ex + r * F::LO + 8 * j + 2 * gc) =
              make_float2(o[j][2 * h], o[j][2 * h + 1]);
        if (gc == 0) {
          ml[2 * r] = m[h];
          ml[2 * r + 1] = l[h];
        }
      }
      __syncthreads();
      for (int e = tid; e < rows * (D / 4); e += F::kThreads) {
        const int r = e / (D / 4), c = e % (D / 4);
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int k = 0; k < WK; ++k) M = fmaxf(M, ml[2 * (k * MR + r)]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < WK; ++k) {
          const float mk = ml[2 * (k * MR + r)];
          const float f = mk == -INFINITY ? 0.f : ex2(mk - M);
          const float4 x = *reinterpret_cast<const float4*>(ex + (k * MR + r) * F::LO + 4 * c);
          L = fmaf(f, ml[2 * (k * MR + r) + 1], L);
          acc.x = fmaf(f, x.x, acc.x);
          acc.y = fmaf(f, x.y, acc.y);
          acc.z = fmaf(f, x.z, acc.z);
          acc.w = fmaf(f, x.w, acc.w);
        }
        if (whole) {
          const int g = rt * MR + r, nd = g / a.G, hq = hk * a.G + g % a.G;
          const float inv = 1.f / L;
          *reinterpret_cast<uint2*>(out + int64_t(nd) * a.ld_out + int64_t(hq) * D + 4 * c) =
              make_uint2(pack2(acc.x * inv, acc.y * inv), pack2(acc.z * inv, acc.w * inv));
          if (a.lse && c == 0)
            a.lse[(int64_t(b) * a.H + hq) * a.N + nd] = (M + log2f(L)) * kLn2;
        } else {
          *reinterpret_cast<float4*>(w + r * D + 4 * c) = acc;
          if (c == 0) {
            w[MR * D + r] = M;
            w[MR * D + MR + r] = L;
          }
        }
      }
    }
  }
}

template <int D, int WM, int WK>
struct Variant {
  using F = Cfg<D, WM, WK>;
  static int grid() { return F::kCtas * gpt2_internal::sm_count(); }
  static int launch(const TreeAttnArgs& a, cudaStream_t st) {
    GPT2_CUDA_TRY(cudaFuncSetAttribute(tree_attn_mma_kernel<D, WM, WK>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem));
    const TreeAttnArgs w = with_workspace<F::MR>(a, grid());
    tree_attn_mma_kernel<D, WM, WK><<<grid(), F::kThreads, F::kSmem, st>>>(w);
    COUNT_LAUNCH(1);
    GPT2_LAUNCH_CHECK();
    return launch_combine<bf16, F::MR, D>(w, st);
  }
};

// Rows of a key/value head decide how many warps cover rows: up to 16 rows all
// four split the keys, up to 32 two, up to 64 none; beyond that eight warps
// cover 128 rows, so that a cache tile is read half as often.
template <typename Fn>
auto pick(int D, int rows, Fn fn) {
  auto by_rows = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    if (rows <= 16) return fn(Variant<kD, 1, 4>{});
    if (rows <= 32) return fn(Variant<kD, 2, 2>{});
    if (rows <= 64) return fn(Variant<kD, 4, 1>{});
    return fn(Variant<kD, 8, 1>{});
  };
  switch (D) {
    case 16: return by_rows(std::integral_constant<int, 16>{});
    case 32: return by_rows(std::integral_constant<int, 32>{});
    case 64: return by_rows(std::integral_constant<int, 64>{});
    default: return by_rows(std::integral_constant<int, 128>{});
  }
}

}  // namespace

size_t tree_attn_mma_workspace(int B, int N, int H, int Hkv, int D) {
  return pick(D, N * (H / Hkv), [&](auto v) {
    using V = decltype(v);
    return workspace_bytes<V::F::MR>(V::grid(), B, N, H, Hkv, D);
  });
}

int launch_tree_attn_mma(const TreeAttnArgs& a, cudaStream_t st) {
  return pick(a.D, a.N * a.G, [&](auto v) { return decltype(v)::launch(a, st); });
}
