// Attention of drafted tokens over a key/value cache for bf16: warp-level
// matrix instructions (m16n8k16, fp32 accumulation) over tiles of 64 keys.
//
// Source and split of the work: as the CUDA-core kernel and tree_attn.cuh.
//
// A step of decoding reads every cached key and value once and does little with
// them: with R = N G query rows per key/value head it is R FLOP a byte, so up
// to a few hundred rows the cache's bandwidth bounds it, and what matters is
// enough loads in flight and few instructions a tile.  One lane of an extra warp
// brings the tiles by TMA into a ring of stages, ahead across the pieces of its
// CTA's run; the other warps wait for a stage and hand it back on their own, with
// no barrier of the block between them.  A warp holds 16 query rows in registers
// (queries, running maximum and sum, output); WM warps cover the rows of a tile
// and WK warps share its keys (few rows: all of them split the keys and merge
// their results at a piece's end).  The tensor maps' swizzle lets the matrix
// loads of 8 rows touch all banks.
//
// Scores and probabilities stay in registers: the accumulator layout of
// S = Q K^T is the operand layout of P for O += P V.  P is rounded to bf16 for
// that product (the tensor cores' operand type; the sums of p stay fp32), as
// in the training attention.  (B200, single tokens, 12 heads of 64: one sequence
// over 700 positions 7.6 us, two launches' latency; 16 over 64-1023 12.4 us.)

#include "tc_common.cuh"
#include "tree_attn.cuh"

using namespace tc;
using namespace tree;

namespace {

constexpr int KT = 64;  // keys of a tile

template <int D, int WM, int WK>
struct Cfg {
  static constexpr int NW = WM * WK;          // warps that compute
  static constexpr int kThreads = 32 * (NW + 1);
  static constexpr int MR = 16 * WM;
  static constexpr int KW = KT / WK;          // keys of a warp
  static constexpr int kTile = KT * D * 2;    // bytes of a K (or V) tile
  static constexpr int NS = D == 128 ? 2 : 3; // stages of K + V
  static constexpr int kRing = NS * 2 * kTile;
  static constexpr int LO = D + 4;            // row stride of the merge buffer
  static constexpr int kMerge = (WK - 1) * MR * (LO + 2) * 4;
  static constexpr int kMasks = kMaxNodes * (kMaskWords + 1) * 4;
  static constexpr int kSmem = 1024 + kRing + kMerge + kMasks + 512 + kListed * int(sizeof(Listed));
  static constexpr int kCtas = WM == 8 ? 1 : D == 128 ? 2 : 3;  // per SM
};

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
// Byte offset of 16-byte chunk c of row r in a tile as TMA leaves it: boxes of
// up to 64 channels, the chunk index within a box's row XORed with row bits so
// that 8 consecutive rows at one chunk fall into 8 different bank groups (the
// 128-, 64- and 32-byte swizzles).
template <int D>
__device__ __forceinline__ uint32_t at(int r, int c) {
  constexpr int C = D < 64 ? D / 8 : 8;  // chunks of a box's row
  const int x = C >= 8 ? (r & 7) : C == 4 ? ((r >> 1) & 3) : ((r >> 2) & 1);
  return uint32_t((c / C) * (KT * 128) + (r * C + ((c % C) ^ x)) * 16);
}
// Tile t of a piece is wholly cached: no key of it is masked.
__device__ __forceinline__ bool plain(const Piece& p, int t) { return (t + 1) * KT <= p.len; }

template <int D, int WM, int WK>
__global__ void __launch_bounds__(Cfg<D, WM, WK>::kThreads, Cfg<D, WM, WK>::kCtas)
    tree_attn_mma_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                         const __grid_constant__ CUtensorMap mx, const __grid_constant__ TreeAttnArgs a) {
  using F = Cfg<D, WM, WK>;
  using S = Split<F::MR, KT, 4>;  // (0, 2, 4, 6: 16.1, 13.0, 12.5, 13.1 us for 16 single tokens)
  constexpr int MR = F::MR, KW = F::KW, NS = F::NS, NW = F::NW;
  constexpr int NT = KW / 8;   // score tiles of 8 keys
  constexpr int DT = D / 8;    // output tiles of 8 channels
  constexpr int KS = D / 16;   // steps of the score product
  constexpr int C = D / 8;     // 16-byte chunks of a row
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sring = smem_u32(ring);
  float* ex = reinterpret_cast<float*>(ring + F::kRing);  // outputs, maxima and sums to merge
  uint32_t* mask = reinterpret_cast<uint32_t*>(ring + F::kRing + F::kMerge);
  int* up = reinterpret_cast<int*>(mask + kMaxNodes * kMaskWords);
  // full[NS] | empty[NS] | listed[kListed] | rows
  uint64_t* bars = reinterpret_cast<uint64_t*>(up + kMaxNodes);
  const uint32_t b_rows = smem_u32(bars + 2 * NS + kListed);
  Listed* list = reinterpret_cast<Listed*>(bars + 2 * NS + kListed + 1);
  // nodes of non-finite values, 64 bits per node tile
  uint64_t* bad = reinterpret_cast<uint64_t*>(list + kListed);
  uint32_t* flag = reinterpret_cast<uint32_t*>(bad + kMaxNodes / 64);
  SeqDims* table = reinterpret_cast<SeqDims*>(flag + 2);
  auto b_full = [&](int s) { return smem_u32(bars + s); };
  auto b_empty = [&](int s) { return smem_u32(bars + NS + s); };
  auto b_listed = [&](int k) { return smem_u32(bars + 2 * NS + k % kListed); };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(b_full(s), 1);
      mbar_init(b_empty(s), NW);
    }
    for (int k = 0; k < kListed; ++k) mbar_init(b_listed(k), 1);
    mbar_init(b_rows, NW);
    fence_mbar_init();
    fence_proxy_async();
  }
  typename S::Pieces pieces{&a, table, 0, 0, 0, 0, 0, 0, 0};
  if (warp == NW) pieces = S::plan(a, table, true);
  __syncthreads();

  if (warp == NW) {
    // ------------------------------------------------ loads
    if (lane) return;
    int g = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Listed& p = list[k % kListed];
      Piece q;
      if (pieces.next(q)) {
        p.slot = pieces.slot(q);
        if (q.t0 == 0) pieces.note(q);
      } else {
        q.kt = 0;
      }
      static_cast<Piece&>(p) = q;
      mbar_arrive(b_listed(k));
      if (q.kt == 0) break;
      const int row0 = (q.b * a.Hkv + q.hk) * a.Tc;  // rows of the caches fit 31 bits
      for (int t = q.t0; t < q.t1; ++t, ++g) {
        const int s = g % NS;
        if (!mbar_wait(b_empty(s), ((g / NS) & 1) ^ 1, a.err, 31)) {
          ok = false;
          break;
        }
        const bool fresh = t >= q.ct;
        const uint32_t dk = sring + s * 2 * F::kTile, dv = dk + F::kTile;
        const int y = fresh ? q.b * a.N + (t - q.ct) * KT : row0 + t * KT;
        const int xk = fresh ? (a.H + q.hk) * D : 0, xv = fresh ? xk + a.Hkv * D : 0;
        mbar_expect_tx(b_full(s), 2 * F::kTile);
#pragma unroll
        for (int c = 0; c < D; c += 64) {
          tma_load_2d(dk + c * KT * 2, fresh ? &mx : &mk, b_full(s), xk + c, y);
          tma_load_2d(dv + c * KT * 2, fresh ? &mx : &mv, b_full(s), xv + c, y);
        }
      }
    }
    // every issued copy has landed before the CTA may exit
    for (int q = max(0, g - NS); q < g; ++q) mbar_wait(b_full(q % NS), (q / NS) & 1, a.err, 32);
    return;
  }

  // -------------------------------------------------- rows
  const int wm = warp % WM, wk = warp / WM;
  const int gr = lane >> 2, gc = lane & 3;  // fragment row and column pair
  int mask_of = -1, g = 0;
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t parity, int where) {
    const bool w = mbar_wait(bar, parity, a.err, where);
    if (!__all_sync(0xffffffffu, w)) ok = false;
  };
  // barrier of these warps with a bounded wait: a warp that gave up does not
  // leave the others waiting
  uint32_t syncs = 0;
  auto sync = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(b_rows);
    wait(b_rows, syncs++ & 1, 35);
  };
  const float scale = rsqrtf(float(D)) * kLog2e;
  const bf16* qkv = static_cast<const bf16*>(a.qkv);

  for (int k = 0;; ++k) {
    wait(b_listed(k), (k / kListed) & 1, 34);
    if (!ok) break;
    const Listed& p = list[k % kListed];
    if (p.kt == 0) break;
    const bf16* xb = qkv + int64_t(p.b) * a.N * a.ld_qkv;
    // this warp's 16 query rows as matrix operands; zeros behind the last row
    uint32_t q[KS][4];
    int node[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = wm * 16 + gr + 8 * h;
      const bool real = r < p.rows;
      const int gq = p.rt * MR + (real ? r : 0);
      node[h] = gq / a.G;
      const bf16* src = xb + int64_t(node[h]) * a.ld_qkv + int64_t(p.hk * a.G + gq % a.G) * D + 2 * gc;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        q[k][h] = real ? *reinterpret_cast<const uint32_t*>(src + 16 * k) : 0u;
        q[k][2 + h] = real ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8) : 0u;
      }
    }
    const bool new_masks = a.parent && p.t1 > p.ct && mask_of != p.b;
    Parents parents;  // in flight until the nodes' tiles are reached
    if (new_masks) parents.load(a.parent + int64_t(p.b) * a.N, p.n, tid, 32 * NW);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[DT][4];
#pragma unroll
    for (int j = 0; j < DT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    const bool busy = wm * 16 < p.rows;  // some row of this warp is real
    bool any_bad = false;

    for (int t = p.t0; t < p.t1; ++t, ++g) {
      const int s = g % NS;
      wait(b_full(s), (g / NS) & 1, 33);
      if (!ok) break;
      const bool fresh = t >= p.ct;
      const int k0 = (fresh ? t - p.ct : t) * KT;
      const int nk = (fresh ? p.n : p.len) - k0;  // keys of the tile
      const int nw = nk - wk * KW;                // ... from this warp's first on
      const uint32_t sk = sring + s * 2 * F::kTile, sv = sk + F::kTile;
      if (!plain(p, t)) {
        // Value rows behind the last key are foreign, and a node that a row may not
        // see can hold anything: the rows that are not this sequence's, and node
        // values that are not finite (see add_nonfinite), become 0 for the product.
        uint8_t* vt = ring + (sv - sring);
        uint64_t* word = bad + (k0 >> 6);
        if (fresh && t == max(p.t0, p.ct)) {  // the piece's first: no other tile's words count
          sync();                             // (the last piece's words and masks have been read)
          if (tid < kMaxNodes / 64) bad[tid] = 0;
          if (new_masks) {
            build_masks(parents, p.n, mask, up, flag, a.err, tid, 32 * NW, sync);
            mask_of = p.b;
          }
          sync();
        }
        for (int e = tid; e < KT * C; e += 32 * NW) {
          const int r = e / C;
          uint4* at_e = reinterpret_cast<uint4*>(vt + at<D>(r, e % C));
          if (r >= nk) {
            *at_e = make_uint4(0, 0, 0, 0);
          } else if (fresh) {
            uint4 u = *at_e;
            if (drop_nonfinite(u)) {
              *at_e = u;
              atomicOr(reinterpret_cast<unsigned long long*>(word), 1ull << r);
            }
          }
        }
        fence_proxy_async();  // before the stage is handed back
        sync();
        if (fresh && *word) any_bad = true;
        if (!ok) break;
      }
      if (busy && nw > 0) {
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
            const int r = wk * KW + j * 8 + (lane & 7) + ((lane >> 4) << 3);
            ldm4(kb, sk + at<D>(r, (lane >> 3) & 1));
            mma16816(sc[j], q[0], kb[0], kb[1]);
            mma16816(sc[j + 1], q[0], kb[2], kb[3]);
          }
        }
        if (fresh || nw < KW) {
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
              if (key >= nw || !((see[e >> 1] >> key) & 1)) sc[j][e] = -INFINITY;
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
          uint32_t pr[4] = {pack2(sc[2 * k][0], sc[2 * k][1]), pack2(sc[2 * k][2], sc[2 * k][3]),
                           pack2(sc[2 * k + 1][0], sc[2 * k + 1][1]),
                           pack2(sc[2 * k + 1][2], sc[2 * k + 1][3])};
          const int r = wk * KW + k * 16 + (lane & 15);
#pragma unroll
          for (int j = 0; j < DT; j += 2) {
            uint32_t vb[4];
            ldm4_trans(vb, sv + at<D>(r, j + (lane >> 4)));
            mma16816(o[j], pr, vb[0], vb[1]);
            mma16816(o[j + 1], pr, vb[2], vb[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b_empty(s));
    }
    if (!ok) break;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      m[h] = __fmul_rn(m[h], scale);  // log2 domain, the base of the sums
    }
    if constexpr (WK > 1) {
      // the warps' results over the same rows, merged in warp order by the first
      float* ml = ex + (WK - 1) * MR * F::LO;
      if (wk > 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = (wk - 1) * MR + wm * 16 + gr + 8 * h;
#pragma unroll
          for (int j = 0; j < DT; ++j)
            *reinterpret_cast<float2*>(ex + r * F::LO + 8 * j + 2 * gc) =
                make_float2(o[j][2 * h], o[j][2 * h + 1]);
          if (gc == 0) *reinterpret_cast<float2*>(ml + 2 * r) = make_float2(m[h], l[h]);
        }
      }
      sync();
      if (wk == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = wm * 16 + gr + 8 * h;
          float2 u[WK - 1];
          float M = m[h];
#pragma unroll
          for (int k = 0; k < WK - 1; ++k) {
            u[k] = *reinterpret_cast<const float2*>(ml + 2 * (k * MR + r));
            M = fmaxf(M, u[k].x);
          }
          const float f = m[h] == -INFINITY ? 0.f : ex2(m[h] - M);
          l[h] *= f;
#pragma unroll
          for (int j = 0; j < DT; ++j) {
            o[j][2 * h] *= f;
            o[j][2 * h + 1] *= f;
          }
#pragma unroll
          for (int k = 0; k < WK - 1; ++k) {
            const float fk = u[k].x == -INFINITY ? 0.f : ex2(u[k].x - M);
            l[h] = fmaf(fk, u[k].y, l[h]);
#pragma unroll
            for (int j = 0; j < DT; ++j) {
              const float2 x =
                  *reinterpret_cast<const float2*>(ex + (k * MR + r) * F::LO + 8 * j + 2 * gc);
              o[j][2 * h] = fmaf(fk, x.x, o[j][2 * h]);
              o[j][2 * h + 1] = fmaf(fk, x.y, o[j][2 * h + 1]);
            }
          }
          m[h] = M;
        }
      }
      sync();  // the buffer may take the next piece's results
    }
    if (wk == 0) {
      bf16* out = static_cast<bf16*>(a.out) + int64_t(p.b) * a.N * a.ld_out;
      float* w = a.ws + p.slot * slot_floats<MR>(D);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = wm * 16 + gr + 8 * h;
        if (r >= p.rows) continue;
        if (p.whole()) {
          const int hq = p.hk * a.G + (p.rt * MR + r) % a.G;
          bf16* dst = out + int64_t(node[h]) * a.ld_out + int64_t(hq) * D + 2 * gc;
          const float inv = 1.f / l[h];
#pragma unroll
          for (int j = 0; j < DT; ++j)
            *reinterpret_cast<uint32_t*>(dst + 8 * j) = pack2(o[j][2 * h] * inv, o[j][2 * h + 1] * inv);
          if (a.lse && gc == 0)
            a.lse[(int64_t(p.b) * a.H + hq) * a.N + node[h]] = (m[h] + log2f(l[h])) * kLn2;
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
        if (any_bad) {
          const int hq = p.hk * a.G + (p.rt * MR + r) % a.G;
          for (int j = 0; j < DT; ++j) {
            const int c = 8 * j + 2 * gc;
            if (p.whole())
              add_nonfinite<bf16, bf16>(a, p.b, p.hk, hq, node[h], p.n, bad, mask, m[h], 1.f / l[h],
                                        out + int64_t(node[h]) * a.ld_out + int64_t(hq) * D, c, c + 2);
            else
              add_nonfinite<bf16, float>(a, p.b, p.hk, hq, node[h], p.n, bad, mask, m[h], 1.f,
                                         w + r * D, c, c + 2);
          }
        }
      }
    }
  }
}

// Tensor map over row-major [outer, inner] bf16 with row stride ld (elements), box
// {box_inner, KT}, box_inner 64, 32 or 16 elements and the swizzle of its width
// (128, 64 or 32 bytes), zero fill out of range.
bool make_map_rows(CUtensorMap* map, const void* base, int64_t inner, int64_t outer, int64_t ld,
                   int box_inner) {
  static const auto encode = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(
        e == cudaSuccess && q == cudaDriverEntryPointSuccess ? p : nullptr);
  }();
  if (!encode) return false;
  const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(outer)};
  const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
  const cuuint32_t box[2] = {cuuint32_t(box_inner), cuuint32_t(KT)};
  const cuuint32_t step[2] = {1, 1};
  const CUtensorMapSwizzle swizzle = box_inner == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : box_inner == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                       : CU_TENSOR_MAP_SWIZZLE_32B;
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
                step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int WM, int WK>
struct Variant {
  using F = Cfg<D, WM, WK>;
  static int grid() { return F::kCtas * gpt2_internal::sm_count(); }
  static int launch(const TreeAttnArgs& a, cudaStream_t st) {
    CUtensorMap mk, mv, mx;
    const int64_t rows = int64_t(a.B) * a.Hkv * a.Tc;
    constexpr int box = D < 64 ? D : 64;
    if (!make_map_rows(&mk, a.k, D, rows, D, box) || !make_map_rows(&mv, a.v, D, rows, D, box) ||
        !make_map_rows(&mx, a.qkv, int64_t(a.H + 2 * a.Hkv) * D, int64_t(a.B) * a.N, a.ld_qkv, box)) {
      gpt2_internal::set_error("tree_attention: tensor map encoding failed");
      return GPT2_ERR_CUDA;
    }
    static std::atomic<uint64_t> allowed{0};
    GPT2_CUDA_TRY(allow_smem(allowed, tree_attn_mma_kernel<D, WM, WK>, F::kSmem));
    const TreeAttnArgs w = with_workspace<F::MR>(a, grid());
    tree_attn_mma_kernel<D, WM, WK><<<grid(), F::kThreads, F::kSmem, st>>>(mk, mv, mx, w);
    COUNT_LAUNCH(1);
    GPT2_LAUNCH_CHECK();
    return launch_combine<bf16, F::MR, D>(w, st);
  }
};

// Rows of a key/value head decide how many warps cover rows: up to 16 rows all
// four split the keys, up to 32 two do.  More rows come here only with head sizes
// 16 and 32: four warps for 64 rows, and eight for 128, so that a cache tile is
// read half as often.
template <typename Fn>
auto pick(int D, int rows, Fn fn) {
  auto by_rows = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    if (rows <= 16) return fn(Variant<kD, 1, 4>{});
    if constexpr (kD < 64) {
      if (rows > 64) return fn(Variant<kD, 8, 1>{});
      if (rows > 32) return fn(Variant<kD, 4, 1>{});
    }
    return fn(Variant<kD, 2, 2>{});
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
