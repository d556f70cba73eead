// Attention of drafted tokens over a key/value cache on the 5th-generation
// tensor cores: bf16, head sizes 64 and 128, up to 128 query rows a tile.
//
// Source and split of the work: as the CUDA-core kernel and tree_attn.cuh; the
// key/value tiles of 64 are streamed once for up to 128 rows (nodes x query
// heads of a key/value head).
//
// CTAs of 192 threads, two per SM, each with its run of key tiles:
//   warp 0, one lane  TMA loads of the tiles (cache, then nodes) into a ring of
//                     stages, ahead across the run's pieces;
//   warp 1            owns the TMEM allocation; one lane issues S = Q K^T
//                     (TMEM, double buffered) and O += P V (P in TMEM);
//   warps 2-5         thread = query row = TMEM lane: running maximum and sum,
//                     P (bf16) written over its own scores, O rescaled when a
//                     maximum grows by more than 2^8, results at a piece's end.
// What a tile holds behind the last key (or the last node) is not the
// sequence's: its scores are masked, and warps 2-5 clear its value rows before
// the product.  They also bring the query rows, the next piece's before they
// write a piece's results.  Warps without a real row only pass the barriers.
// 256 TMEM columns and about 100 KB of shared memory let two CTAs share an SM,
// so that one's softmax overlaps the other's MMAs.
//
// Every wait is bounded (2 s) and reports a timeout in the error word.

#include "tc_common.cuh"
#include "tree_attn.cuh"

using namespace tc;
using namespace tree;

namespace {

constexpr int kThreads = 192;
constexpr int MR = 128;  // query rows of a tile = TMEM lanes
constexpr int KT = 64;   // keys of a tile
constexpr int kTmemCols = 256;
constexpr float kRescale = 8.f;  // lazy-rescale threshold, log2 units

template <int D>
struct Cfg {
  static constexpr int KC = D / 64;              // 64-channel chunks of a row
  static constexpr int kChunkQ = MR * 128;       // 16 KB: 128 rows x 64 bf16
  static constexpr int kChunk = KT * 128;        // 8 KB: 64 rows x 64 bf16
  static constexpr int kQ = KC * kChunkQ;
  static constexpr int kTile = KC * kChunk;      // a K (or V) tile
  static constexpr int NS = D == 64 ? 5 : 2;     // stages of K + V
  static constexpr int kMasks = kMaxNodes * (kMaskWords + 1) * 4;
  static constexpr int kSmem = kQ + NS * 2 * kTile + kMasks + 512 + 1024;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Tile t of a piece is wholly cached: no key of it is masked.
__device__ __forceinline__ bool plain(const Piece& p, int t) { return (t + 1) * KT <= p.len; }

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    tree_attn_tc_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                        const __grid_constant__ CUtensorMap mx, const __grid_constant__ TreeAttnArgs a) {
  using F = Cfg<D>;
  constexpr int NS = F::NS, KC = F::KC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* ring = smem + F::kQ;
  const uint32_t sQ = smem_u32(smem), sKV = smem_u32(ring);
  uint32_t* mask = reinterpret_cast<uint32_t*>(ring + NS * 2 * F::kTile);
  int* up = reinterpret_cast<int*>(mask + kMaxNodes * kMaskWords);
  uint64_t* bars = reinterpret_cast<uint64_t*>(up + kMaxNodes);
  // q_full | kv_full[NS] | kv_empty[NS] | s_full[2] | s_free[2] | p_full[2] | o_done[2] | rows
  const uint32_t b_q = smem_u32(bars);
  auto b_kvf = [&](int s) { return smem_u32(bars + 1 + s); };
  auto b_kve = [&](int s) { return smem_u32(bars + 1 + NS + s); };
  auto b_sf = [&](int i) { return smem_u32(bars + 1 + 2 * NS + i); };
  auto b_sfr = [&](int i) { return smem_u32(bars + 3 + 2 * NS + i); };
  auto b_pf = [&](int i) { return smem_u32(bars + 5 + 2 * NS + i); };
  auto b_od = [&](int i) { return smem_u32(bars + 7 + 2 * NS + i); };
  const uint32_t b_rows = smem_u32(bars + 9 + 2 * NS);
  uint32_t* slot = reinterpret_cast<uint32_t*>(bars + 10 + 2 * NS);
  SeqDims* table = reinterpret_cast<SeqDims*>(slot + 6);
  uint32_t* odd = slot + 1;  // keys of a node tile whose values are not finite

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    mbar_init(b_q, 1);
    mbar_init(b_rows, 128);
    for (int s = 0; s < NS; ++s) {
      mbar_init(b_kvf(s), 1);
      mbar_init(b_kve(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_sf(i), 1);
      mbar_init(b_sfr(i), 128);
      mbar_init(b_pf(i), 128);
      mbar_init(b_od(i), 1);
    }
    fence_mbar_init();
    fence_proxy_async();
  }
  if (warp == 1) tmem_alloc(smem_u32(slot), kTmemCols);
  auto pieces = Split<MR, KT>::plan(a, table, threadIdx.x < 32);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const uint32_t tS = tmem, tO = tmem + 128;  // S buffers at +0 and +64, O at +128

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------ TMA
    int g = 0;
    bool ok = true;
    Piece p;
    while (ok && pieces.next(p)) {
      const int row0 = (p.b * a.Hkv + p.hk) * a.Tc;  // B Hkv Tc rows of >= 128 B fit 31 bits
      for (int t = p.t0; t < p.t1; ++t, ++g) {
        const int s = g % NS;
        if (!mbar_wait(b_kve(s), ((g / NS) & 1) ^ 1, a.err, 11)) {
          ok = false;
          break;
        }
        const bool fresh = t >= p.ct;
        const uint32_t dk = sKV + s * 2 * F::kTile, dv = dk + F::kTile;
        const int y = fresh ? p.b * a.N + (t - p.ct) * KT : row0 + t * KT;
        const int xk = fresh ? (a.H + p.hk) * D : 0, xv = fresh ? xk + a.Hkv * D : 0;
        mbar_expect_tx(b_kvf(s), 2 * F::kTile);
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          tma_load_2d(dk + c * F::kChunk, fresh ? &mx : &mk, b_kvf(s), xk + 64 * c, y);
          tma_load_2d(dv + c * F::kChunk, fresh ? &mx : &mv, b_kvf(s), xv + 64 * c, y);
        }
      }
    }
    // every issued copy has landed before the CTA may exit
    for (int q = max(0, g - NS); q < g; ++q) mbar_wait(b_kvf(q % NS), (q / NS) & 1, a.err, 15);
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------ MMA
    const uint32_t id_s = idesc_bf16(MR, KT, 0, 0), id_o = idesc_bf16(MR, D, 0, 1);
    const uint64_t dQ = desc_kmajor(sQ, 0), dK = desc_kmajor(sKV, 0);
    const uint64_t dV = desc_mnmajor(sKV + F::kTile, 0);
    int g = 0, k = 0;
    bool ok = true;
    auto issue_pv = [&](int gt, bool acc) -> bool {
      if (!mbar_wait(b_pf(gt & 1), (gt >> 1) & 1, a.err, 13)) return false;
      tc_fence_after();
      const uint64_t v = desc_offset(dV, (gt % NS) * 2 * F::kTile);
      const uint32_t pa = tS + (gt & 1) * KT;
      if (acc)
        umma_ts_i<1>(tO, pa, v, id_o);
      else
        umma_ts_i<0>(tO, pa, v, id_o);
#pragma unroll
      for (int i = 1; i < 4; ++i) umma_ts_i<1>(tO, pa + 8 * i, v + i * 128, id_o);
      umma_commit(b_od(gt & 1));
      umma_commit(b_kve(gt % NS));
      return true;
    };
    Piece p;
    for (; ok && pieces.next(p); ++k) {
      if (!mbar_wait(b_q, k & 1, a.err, 12)) break;
      for (int t = p.t0; t < p.t1; ++t, ++g) {
        const int s = g % NS;
        if (!mbar_wait(b_kvf(s), (g / NS) & 1, a.err, 12) ||
            !mbar_wait(b_sfr(g & 1), ((g >> 1) & 1) ^ 1, a.err, 12)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t kd = desc_offset(dK, s * 2 * F::kTile);
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t qa = desc_offset(dQ, c * F::kChunkQ) + 2 * i;
            const uint64_t kb = desc_offset(kd, c * F::kChunk) + 2 * i;
            if (c == 0 && i == 0)
              umma_i<0>(tS + (g & 1) * KT, qa, kb, id_s);
            else
              umma_i<1>(tS + (g & 1) * KT, qa, kb, id_s);
          }
        umma_commit(b_sf(g & 1));
        if (t > p.t0 && !issue_pv(g - 1, t - 1 > p.t0)) {
          ok = false;
          break;
        }
      }
      if (ok) ok = issue_pv(g - 1, p.t1 - 1 > p.t0);
    }
    // all issued MMAs complete before TMEM is released
    if (g > 0) mbar_wait(b_od((g - 1) & 1), ((g - 1) >> 1) & 1, a.err, 16);
  } else if (warp >= 2) {
    // ------------------------------------------------ rows
    const int e = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lo = uint32_t((warp & 3) * 32) << 16;
    const float scale = rsqrtf(float(D)) * kLog2e;
    const bf16* qkv = static_cast<const bf16*>(a.qkv);
    int g = 0, mask_of = -1;
    bool ok = true;
    uint32_t syncs = 0;
    // the 128 row threads, with a bounded wait (a warp that gave up does not
    // leave the others waiting)
    auto rows_sync = [&] {
      mbar_arrive(b_rows);
      const bool w = mbar_wait(b_rows, syncs++ & 1, a.err, 22);
      if (!__all_sync(0xffffffffu, w)) ok = false;
    };
    Piece p;
    // the query rows of a piece (every MMA that read the last piece's is
    // complete: its scores have been taken)
    auto load_q = [&](const Piece& q) {
      const bool real = e < q.rows;
      const int gr = q.rt * MR + (real ? e : 0), node = gr / a.G, h = q.hk * a.G + gr % a.G;
      const uint4* src = reinterpret_cast<const uint4*>(
          qkv + (int64_t(q.b) * a.N + node) * a.ld_qkv + int64_t(h) * D);
#pragma unroll
      for (int c0 = 0; c0 < D / 8; c0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = real ? src[c0 + c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(smem + (c0 >> 3) * F::kChunkQ + e * 128 + ((c ^ (e & 7)) << 4)) = v[c];
      }
      fence_proxy_async();  // visible to the MMAs
      rows_sync();
      if (e == 0) mbar_arrive(b_q);
    };
    // A tile with foreign rows, or with nodes that a row may not see: those can
    // hold anything, and 0 times a non-finite value is not 0.  Value rows behind
    // the last key become 0; so do rows with non-finite values among the nodes,
    // whose keys are returned (they reach the rows that see them one by one).
    auto clear = [&](const Piece& q, int t, int gt) -> uint64_t {
      const int s = gt % NS;
      const bool fresh = t >= q.ct;
      const int nk = fresh ? q.n - (t - q.ct) * KT : q.len - t * KT;
      const bool w = mbar_wait(b_kvf(s), (gt / NS) & 1, a.err, 21);  // complete: its scores are
      if (!__all_sync(0xffffffffu, w)) ok = false;
      uint8_t* v = ring + s * 2 * F::kTile + F::kTile;
      uint64_t drop = nk >= KT ? 0 : ~uint64_t(0) << nk;
      uint64_t bad_v = 0;
      if (fresh) {
        if (e < 2) odd[e] = 0;
        rows_sync();
#pragma unroll
        for (int x = e; x < KT * D / 8; x += 128) {  // 16-byte units, the swizzle left alone
          const int r = x / 8 % KT;
          const uint4 u = *reinterpret_cast<const uint4*>(v + x * 16);
          auto inf = [](uint32_t w2) {
            return (w2 & 0x7F80u) == 0x7F80u || (w2 & 0x7F800000u) == 0x7F800000u;
          };
          if (r < nk && (inf(u.x) || inf(u.y) || inf(u.z) || inf(u.w)))
            atomicOr(&odd[r >> 5], 1u << (r & 31));
        }
        rows_sync();
        bad_v = odd[0] | (uint64_t(odd[1]) << 32);
        drop |= bad_v;
      }
      if (drop) {
        for (int x = e; x < KT * D / 8; x += 128)
          if ((drop >> (x / 8 % KT)) & 1) *reinterpret_cast<uint4*>(v + x * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async();  // before this thread's arrival that the product waits for
      }
      return bad_v;
    };
    bool have = pieces.next(p);
    if (have) load_q(p);
    while (ok && have) {
      const bool real = e < p.rows;
      const bool busy = ((warp & 3) * 32) < p.rows;
      const int gr = p.rt * MR + (real ? e : 0), node = gr / a.G, hq = p.hk * a.G + gr % a.G;
      if (e == 0 && p.t0 == 0) pieces.note(p);
      if (a.parent && p.t1 > p.ct && mask_of != p.b) {
        build_masks(a.parent + int64_t(p.b) * a.N, p.n, mask, up, odd + 2, a.err, e, 128, rows_sync);
        mask_of = p.b;
      }
      float m = -INFINITY, l = 0.f;
      for (int t = p.t0; t < p.t1; ++t, ++g) {
        bool wt = mbar_wait(b_sf(g & 1), (g >> 1) & 1, a.err, 14);
        if (!__all_sync(0xffffffffu, wt)) {
          ok = false;
          break;
        }
        const uint64_t bad_v = plain(p, t) ? 0 : clear(p, t, g);
        if (!ok) break;
        if (!busy) {
          mbar_arrive(b_sfr(g & 1));
          mbar_arrive(b_pf(g & 1));
          continue;
        }
        tc_fence_after();
        uint32_t r0[32], r1[32];
        tmem_ld32_async(tS + lo + (g & 1) * KT, r0);
        tmem_ld32_async(tS + lo + (g & 1) * KT + 32, r1);
        tmem_wait_ld(r0);
        reg_after_wait(r1);
        tc_fence_before();
        mbar_arrive(b_sfr(g & 1));
        float x[64];  // raw scores; keys that the row may not see become -inf
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          x[i] = __uint_as_float(r0[i]);
          x[32 + i] = __uint_as_float(r1[i]);
        }
        if (!plain(p, t)) {
          const bool fresh = t >= p.ct;
          const int k0 = (fresh ? t - p.ct : t) * KT, nk = (fresh ? p.n : p.len) - k0;
          uint64_t see = nk >= KT ? ~uint64_t(0) : (uint64_t(1) << nk) - 1;
          if (fresh) see &= sees(!a.parent, mask, node, k0);
#pragma unroll
          for (int i = 0; i < 64; ++i) x[i] = (see >> i) & 1 ? x[i] : -INFINITY;
        }
        float c4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float* y = x + 16 * k;
          float mm = max3f(y[0], y[1], y[2]);
#pragma unroll
          for (int i = 3; i < 15; i += 2) mm = max3f(mm, y[i], y[i + 1]);
          c4[k] = fmaxf(mm, y[15]);
        }
        // log2 domain; the base of the probabilities follows the maximum only
        // when it grows by more than 2^8 (they stay <= 256); 0 while the row
        // has seen nothing (every p is then 2^(-inf) = 0)
        const float mn = fmaxf(m, __fmul_rn(max3f(c4[0], c4[1], fmaxf(c4[2], c4[3])), scale));
        const bool resc = mn > m + kRescale;
        const float mu = resc ? mn : m;
        const float corr = resc ? ex2(m - mn) : 1.f;
        const float base = mu == -INFINITY ? 0.f : mu;
        uint32_t pk[32];
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float u0, u1;
          fma2(u0, u1, x[i], x[i + 1], scale, scale, -base, -base);
          const float p0 = ex2(u0), p1 = ex2(u1);
          add2(sa[(i >> 1) & 3], sb[(i >> 1) & 3], p0, p1);
          pk[i >> 1] = pack2(p0, p1);
        }
        const float rs = ((sa[0] + sb[0]) + (sa[1] + sb[1])) + ((sa[2] + sb[2]) + (sa[3] + sb[3]));
        l = l * corr + rs;
        m = mu;
        if (t > p.t0 && __any_sync(0xffffffffu, resc)) {
          // O must hold the last tile's product before it is rescaled
          wt = mbar_wait(b_od((g - 1) & 1), ((g - 1) >> 1) & 1, a.err, 17);
          if (!__all_sync(0xffffffffu, wt)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            float f[32];
            tmem_ld32_async(tO + lo + c, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]) * corr;
            tmem_st32(tO + lo + c, f);
          }
        }
        // P (bf16) over the first 32 columns of its scores, the A operand of P V
        tmem_st32_async(tS + lo + (g & 1) * KT, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(b_pf(g & 1));
        if (bad_v) {
          // A node that a row may not see can hold anything, and 0 times a
          // non-finite value is not 0: such value rows are zeros in the tile
          // and reach the rows that see them here.
          wt = mbar_wait(b_od(g & 1), (g >> 1) & 1, a.err, 20);
          if (!__all_sync(0xffffffffu, wt)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int k0 = (t - p.ct) * KT;
          const bf16* v = qkv + (int64_t(p.b) * a.N + k0) * a.ld_qkv + int64_t(a.H + a.Hkv + p.hk) * D;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            float f[32];
            tmem_ld32_async(tO + lo + c, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]);
#pragma unroll 1
            for (int key = 0; key < KT; ++key) {
              if (!((bad_v >> key) & 1)) continue;
              float pj = 0.f;
#pragma unroll
              for (int i = 0; i < 64; i += 2) {
                const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&pk[i >> 1]);
                if (i == key) pj = __bfloat162float(h.x);
                if (i + 1 == key) pj = __bfloat162float(h.y);
              }
              if (pj != 0.f)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  f[i] = fmaf(pj, __bfloat162float(v[key * a.ld_qkv + c + i]), f[i]);
            }
            tmem_st32(tO + lo + c, f);
          }
          tc_fence_before();
        }
      }
      if (!ok) break;
      const Piece done = p;
      have = pieces.next(p);
      if (have) load_q(p);  // the next piece's scores overlap this one's results
      if (!ok) break;
      const int last = g - 1;
      bool wt = mbar_wait(b_od(last & 1), (last >> 1) & 1, a.err, 19);
      if (!__all_sync(0xffffffffu, wt)) break;
      if (!busy) continue;
      tc_fence_after();
      const bool whole = done.whole();
      const float inv = 1.f / l;
      bf16* out = static_cast<bf16*>(a.out) + (int64_t(done.b) * a.N + node) * a.ld_out + int64_t(hq) * D;
      float* w = a.ws + pieces.slot(done) * slot_floats<MR>(D);
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32_async(tO + lo + c, o);
        tmem_wait_ld(o);
        if (!real) continue;
        if (whole) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint4 v;
            v.x = pack2(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv);
            v.y = pack2(__uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
            v.z = pack2(__uint_as_float(o[i + 4]) * inv, __uint_as_float(o[i + 5]) * inv);
            v.w = pack2(__uint_as_float(o[i + 6]) * inv, __uint_as_float(o[i + 7]) * inv);
            *reinterpret_cast<uint4*>(out + c + i) = v;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(w + int64_t(e) * D + c + i) =
                make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
      }
      tc_fence_before();
      if (real) {
        if (whole) {
          if (a.lse) a.lse[(int64_t(done.b) * a.H + hq) * a.N + node] = (m + log2f(l)) * kLn2;
        } else {
          w[MR * D + e] = m;
          w[MR * D + MR + e] = l;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

int grid_size() { return 2 * gpt2_internal::sm_count(); }

template <int D>
int launch_tc(const TreeAttnArgs& a, cudaStream_t st) {
  using F = Cfg<D>;
  CUtensorMap mk, mv, mx;
  const int64_t rows = int64_t(a.B) * a.Hkv * a.Tc;
  if (!make_map_bf16(&mk, a.k, D, rows, D, KT) || !make_map_bf16(&mv, a.v, D, rows, D, KT) ||
      !make_map_bf16(&mx, a.qkv, int64_t(a.H + 2 * a.Hkv) * D, int64_t(a.B) * a.N, a.ld_qkv, KT)) {
    gpt2_internal::set_error("tree_attention: tensor map encoding failed");
    return GPT2_ERR_CUDA;
  }
  GPT2_CUDA_TRY(cudaFuncSetAttribute(tree_attn_tc_kernel<D>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem));
  const TreeAttnArgs w = with_workspace<MR>(a, grid_size());
  tree_attn_tc_kernel<D><<<grid_size(), kThreads, F::kSmem, st>>>(mk, mv, mx, w);
  COUNT_LAUNCH(1);
  GPT2_LAUNCH_CHECK();
  return launch_combine<bf16, MR, D>(w, st);
}

}  // namespace

size_t tree_attn_tc_workspace(int B, int N, int H, int Hkv, int D) {
  return workspace_bytes<MR>(grid_size(), B, N, H, Hkv, D);
}

int launch_tree_attn_tc(const TreeAttnArgs& a, cudaStream_t st) {
  return a.D == 64 ? launch_tc<64>(a, st) : launch_tc<128>(a, st);
}
