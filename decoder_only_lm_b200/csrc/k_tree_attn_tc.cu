// Attention of drafted tokens over a key/value cache on the 5th-generation
// tensor cores: bf16, head sizes 64 and 128, up to 128 query rows a tile.
//
// Source and split of the work: as the CUDA-core kernel and tree_attn.cuh; the
// key/value tiles of 64 are streamed once for up to 128 rows (nodes x query
// heads of a key/value head).
//
// Two CTAs of 192 threads per SM, each with its run of key tiles:
//   warp 0            plans the run; one lane publishes its pieces and brings the
//                     tiles (cache, then nodes) by TMA into a ring of stages,
//                     ahead across the pieces;
//   warp 1            owns the TMEM allocation; one lane issues S = Q K^T and
//                     O += P V (P in TMEM);
//   warps 2-5         thread = TMEM lane: running maximum and sum of a query
//                     row, P (bf16) written over its own scores, O rescaled
//                     when a maximum grows by more than 2^8, results at a
//                     piece's end.
// S has two buffers, so that the next tile's scores are there when a softmax
// ends.  A softmax is a chain of latencies (scores from TMEM, exponentials,
// probabilities to TMEM) that grows with the keys a thread takes, and with few
// rows most lanes would be idle: up to 64 rows are held P = 2 times, in lanes
// row + 64 i, and copy i takes its half of each tile's keys, with zeros for the
// other among its probabilities, so the products stay the same instructions
// (long trees of 48: 57.3 -> 53.9 us).  The copies' maxima, sums and outputs
// merge at a piece's end, where share_nonfinite looks after cached values that 0
// times is not 0.
// What a tile holds behind the last key (or the last node) is not the
// sequence's: its scores are masked, and the row threads clear its value rows
// before the product.  They also bring the query rows, the next piece's before
// they write a piece's results.  Warps without a real row only pass barriers.
// With two CTAs' shared memory little is left for the L1 cache, so nothing in
// the steps may live in local memory (a spilled register costs an L2 access).
//
// What bounds it: with few rows a head the cache's bytes (B200, 4 trees of 48 over
// 9-33 thousand positions, 12 heads of 64: 52 us, 4.9 TB/s), with full tiles the
// softmax and the wait for scores (8 trees of 64 over 1000-8191, 32 heads on 8 of
// 128: 62 us), and in short calls the start, a piece's end and the merge (16 trees
// of 64 over 100-1024, 16 heads of 64: 25 us).
//
// Every wait is bounded (2 s) and reports a timeout in the error word.

#include "tc_common.cuh"
#include "tree_attn.cuh"

using namespace tc;
using namespace tree;

namespace {

constexpr int kThreads = 192;
constexpr int kLanes = 128;  // TMEM lanes = row threads
constexpr int KT = 64;       // keys of a tile
constexpr int kTmemCols = 256;
constexpr float kRescale = 8.f;  // lazy-rescale threshold, log2 units

template <int D, int P>
struct Cfg {
  static constexpr int MR = kLanes / P;          // query rows of a tile
  static constexpr int KC = D / 64;              // 64-channel chunks of a row
  static constexpr int kChunkQ = kLanes * 128;   // 16 KB: 128 rows x 64 bf16
  static constexpr int kChunk = KT * 128;        // 8 KB: 64 rows x 64 bf16
  static constexpr int kQ = KC * kChunkQ;
  static constexpr int kTile = KC * kChunk;      // a K (or V) tile
  static constexpr int NS = D == 128 ? 2 : P > 1 ? 4 : 5;  // stages of K + V
  static constexpr int kNodes = P > 1 ? MR : kMaxNodes;   // a node has a row at least
  static constexpr int kMasks = kNodes * (kMaskWords + 1) * 4;
  static constexpr int LX = 20;                  // row stride of the copies' exchange
  static constexpr int kXch = D == 64 ? 2 : 1;   // ... and its buffers
  static constexpr int kExchange = P > 1 ? kLanes * (kXch * LX + 2) * 4 : 0;
  static constexpr int kSmem = kQ + NS * 2 * kTile + kMasks + kExchange + 1280 + 1024;
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
__device__ __forceinline__ void tmem_ld16_raw(uint32_t taddr, uint32_t (&r)[16]) {
  float v[16];
  tmem_ld16(taddr, v);
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
}
// 16 columns of this thread's TMEM lane from registers; complete after tmem_wait_st()
__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// 16 bytes to shared memory, zeros where the row is not real
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
template <typename T>
__device__ __forceinline__ T uniform(T v) {
  return __shfl_sync(0xffffffffu, v, 0);
}
// Values that are not finite, behind the stores of a piece's results (of row
// `node`, base m in the log2 domain, times inv_l; `mine`: this lane stored some, the
// columns from 16 copy on in every Pth group of 16).  By a whole warp.
//
// Where a row's copies multiply each other's keys by 0, a cached value that is not
// finite (0 times it is not 0) makes the row's sum NaN whatever its share is.  A
// column that came out not finite becomes the sum of such values' shares, beside
// which the finite ones do not count; without any it stays (an overflow).  Then the
// shares of the nodes in `bad`, if any_bad (see add_nonfinite).
template <int D, int P, typename Out>
__device__ void share_nonfinite(const TreeAttnArgs& a, const Piece& p, int hq, int node, bool mine,
                                bool any_bad, const uint64_t* bad, const uint32_t* mask, float m,
                                float inv_l, Out* dst, int copy) {
  if constexpr (P > 1) {
    constexpr int kCols = D / P;  // columns of a copy
    static_assert(kCols <= 64, "a bit for each column");
    auto column = [&](int i) { return 16 * (copy + P * (i / 16)) + i % 16; };
    const bf16* q = static_cast<const bf16*>(a.qkv) + (int64_t(p.b) * a.N + node) * a.ld_qkv +
                    int64_t(hq) * D;
    const int64_t row0 = (int64_t(p.b) * a.Hkv + p.hk) * a.Tc;
    const bf16* kc = static_cast<const bf16*>(a.k) + row0 * D;
    const bf16* vc = static_cast<const bf16*>(a.v) + row0 * D;
    const float scale = rsqrtf(float(D)) * kLog2e;
    uint64_t odd = 0, found = 0;
    if (mine)
      for (int i = 0; i < kCols; ++i)
        if (!finite(dst[column(i)])) odd |= uint64_t(1) << i;
    // the piece's cached keys, 32 at a time
    const int k1 = p.t1 <= p.ct ? min(p.len, p.t1 * KT) : p.len;
    for (int j0 = __any_sync(0xffffffffu, odd != 0) ? p.t0 * KT : k1; j0 < k1; j0 += 32) {
      bool hit = false;
      if (const int j = j0 + int(threadIdx.x) % 32; j < k1) {
#pragma unroll
        for (int i = 0; i < kCols; i += 8) {
          uint4 u = *reinterpret_cast<const uint4*>(vc + int64_t(j) * D + column(i));
          hit |= drop_nonfinite(u);
        }
      }
      for (unsigned which = __ballot_sync(0xffffffffu, hit); which; which &= which - 1) {
        const int64_t at = (j0 + int64_t(__ffs(int(which)) - 1)) * D;
        if (!odd) continue;
        float s = 0.f;
        for (int d = 0; d < D; ++d) s = fmaf(to_f32<bf16>(q[d]), to_f32<bf16>(kc[at + d]), s);
        const float pj = ex2(fmaf(s, scale, -m)) * inv_l;
        for (int i = 0; i < kCols; ++i) {
          const bf16 v = vc[at + column(i)];
          const uint64_t bit = uint64_t(1) << i;
          if (!(odd & bit) || finite(v)) continue;
          Out& x = dst[column(i)];
          x = from_f32<Out>(found & bit ? fmaf(pj, to_f32<bf16>(v), to_f32<Out>(x)) : pj * to_f32<bf16>(v));
          found |= bit;
        }
      }
    }
  }
  if (any_bad && mine)
    for (int c = 16 * copy; c < D; c += 16 * P)
      add_nonfinite<bf16, Out>(a, p.b, p.hk, hq, node, p.n, bad, mask, m, inv_l, dst, c, c + 16);
}
template <int D, int P>
__device__ __noinline__ void share_nonfinite(const TreeAttnArgs& a, const Listed& p, int row, int copy,
                                             bool any_bad, const uint64_t* bad, const uint32_t* mask,
                                             float m, float l) {
  constexpr int MR = Cfg<D, P>::MR;
  const bool mine = row < p.rows;
  const int gr = p.rt * MR + (mine ? row : 0), node = gr / a.G, hq = p.hk * a.G + gr % a.G;
  if (p.whole())
    share_nonfinite<D, P>(
        a, p, hq, node, mine, any_bad, bad, mask, m, 1.f / l,
        static_cast<bf16*>(a.out) + (int64_t(p.b) * a.N + node) * a.ld_out + int64_t(hq) * D, copy);
  else
    share_nonfinite<D, P>(a, p, hq, node, mine, any_bad, bad, mask, m, 1.f,
                          a.ws + p.slot * slot_floats<MR>(D) + int64_t(row) * D, copy);
}
template <int D, int P>
__global__ void __launch_bounds__(kThreads, 2)
    tree_attn_tc_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                        const __grid_constant__ CUtensorMap mx,
                        const __grid_constant__ TreeAttnArgs a) {
  using F = Cfg<D, P>;
  constexpr int NS = F::NS, KC = F::KC, MR = F::MR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* ring = smem + F::kQ;
  const uint32_t sQ = smem_u32(smem), sKV = smem_u32(ring);
  uint32_t* mask = reinterpret_cast<uint32_t*>(ring + NS * 2 * F::kTile);
  int* up = reinterpret_cast<int*>(mask + F::kNodes * kMaskWords);
  float* xch = reinterpret_cast<float*>(up + F::kNodes);  // 16 outputs a lane, for the other copies
  float2* ml = reinterpret_cast<float2*>(xch + kLanes * F::LX * F::kXch);  // ... maximum and sum
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(up + F::kNodes) + F::kExchange);
  // k_full[NS] | v_full[NS] | k_empty[NS] | v_empty[NS] | q_full | s_full[2] | p_full[2] |
  // o_done[2] | rows | listed[kListed] | go
  auto b_kf = [&](int s) { return smem_u32(bars + s); };
  auto b_vf = [&](int s) { return smem_u32(bars + NS + s); };
  auto b_ke = [&](int s) { return smem_u32(bars + 2 * NS + s); };
  auto b_ve = [&](int s) { return smem_u32(bars + 3 * NS + s); };
  const uint32_t b_q = smem_u32(bars + 4 * NS);
  auto b_sf = [&](int i) { return smem_u32(bars + 4 * NS + 1 + i); };
  auto b_pf = [&](int i) { return smem_u32(bars + 4 * NS + 3 + i); };
  auto b_od = [&](int i) { return smem_u32(bars + 4 * NS + 5 + i); };
  const uint32_t b_rows = smem_u32(bars + 4 * NS + 7);
  auto b_listed = [&](int k) { return smem_u32(bars + 4 * NS + 8 + k % kListed); };
  const uint32_t b_go = smem_u32(bars + 4 * NS + 8 + kListed);
  Listed* list = reinterpret_cast<Listed*>(bars + 4 * NS + 9 + kListed);
  uint64_t* bad = reinterpret_cast<uint64_t*>(list + kListed);  // nodes of non-finite values
  uint32_t* flag = reinterpret_cast<uint32_t*>(bad + kMaxNodes / 64);
  uint32_t* slot = flag + 1;
  SeqDims* table = reinterpret_cast<SeqDims*>(flag + 2);
  // tile g: buffer of its scores, and parity of the buffer's use
  auto buf_of = [](int g) { return g & 1; };
  auto par_of = [](int g) { return uint32_t((g >> 1) & 1); };

  const int warp = uniform(int(threadIdx.x / 32)), lane = threadIdx.x % 32;
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 32) {
    mbar_init(b_q, 1);
    mbar_init(b_rows, kLanes / 32);
    mbar_init(b_go, kLanes / 32);
    for (int s = 0; s < NS; ++s) {
      mbar_init(b_kf(s), 1);
      mbar_init(b_vf(s), 1);
      mbar_init(b_ke(s), 1);
      mbar_init(b_ve(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_sf(i), 1);
      mbar_init(b_pf(i), kLanes / 32);
      mbar_init(b_od(i), 1);
    }
    for (int k = 0; k < kListed; ++k) mbar_init(b_listed(k), 1);
    fence_mbar_init();
    fence_proxy_async();
  }
  __syncwarp();
  if (warp == 1) tmem_alloc(smem_u32(slot), kTmemCols);
  typename Split<MR, KT, 6>::Pieces pieces{&a, table, 0, 0, 0, 0, 0, 0, 0};
  if (warp == 0) pieces = Split<MR, KT, 6>::plan(a, table, true);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  // S buffers at +0 and +64, O at +128
  const uint32_t tS = tmem, tO = tmem + 128;

  if (warp == 0) {
    // ------------------------------------------------ plan, loads
    if (lane == 0) {
      int s = 0;          // stage, and how often the ring has come round
      uint32_t round = 0;
      int filled_k = 0, filled = 0;  // keys', values' fills
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
        // the first queries are asked for ahead of a ring of tiles, behind which
        // they would queue (from cold caches, 16 trees of 64 39 -> 37 us, 8 trees of
        // 64 with 4 query heads for a cache head 84 -> 80)
        if (k == 0 && !mbar_wait(b_go, 0, a.err, 27)) {
          ok = false;
          break;
        }
        const int row0 = (q.b * a.Hkv + q.hk) * a.Tc;  // rows of the caches fit 31 bits
        for (int t = q.t0; t < q.t1; ++t) {
          const bool fresh = t >= q.ct;
          const uint32_t dk = sKV + s * 2 * F::kTile, dv = dk + F::kTile;
          const int y = fresh ? q.b * a.N + (t - q.ct) * KT : row0 + t * KT;
          const int xk = fresh ? (a.H + q.hk) * D : 0, xv = fresh ? xk + a.Hkv * D : 0;
          // keys go when the tile's scores are done, values only after its product
          if (!mbar_wait(b_ke(s), (round & 1) ^ 1, a.err, 11)) {
            ok = false;
            break;
          }
          mbar_expect_tx(b_kf(s), F::kTile);
#pragma unroll
          for (int c = 0; c < KC; ++c)
            tma_load_2d(dk + c * F::kChunk, fresh ? &mx : &mk, b_kf(s), xk + 64 * c, y);
          ++filled_k;
          if (!mbar_wait(b_ve(s), (round & 1) ^ 1, a.err, 11)) {
            ok = false;
            break;
          }
          mbar_expect_tx(b_vf(s), F::kTile);
#pragma unroll
          for (int c = 0; c < KC; ++c)
            tma_load_2d(dv + c * F::kChunk, fresh ? &mx : &mv, b_vf(s), xv + 64 * c, y);
          ++filled;
          if (++s == NS) {
            s = 0;
            ++round;
          }
        }
      }
      // every issued copy has landed before the CTA may exit
      for (int q = max(0, filled_k - NS); q < filled_k; ++q) mbar_wait(b_kf(q % NS), (q / NS) & 1, a.err, 15);
      for (int q = max(0, filled - NS); q < filled; ++q) mbar_wait(b_vf(q % NS), (q / NS) & 1, a.err, 15);
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA
    // The whole warp runs the loop, so that its control and the descriptors are
    // warp-uniform (from one lane's branch every operand of an MMA has to be moved
    // to the uniform registers first), and one elected lane issues.
    const bool leader = elect_one();
    const uint32_t id_s = idesc_bf16(kLanes, KT, 0, 0), id_o = idesc_bf16(kLanes, D, 0, 1);
    const uint64_t dQ = desc_kmajor(sQ, 0), dK = desc_kmajor(sKV, 0);
    const uint64_t dV = desc_mnmajor(sKV + F::kTile, 0);
    const uint32_t uS = uniform(tS), uO = uniform(tO);
    int g = 0, s = 0, last = 0;  // tile, its stage, the stage of the tile before
    uint32_t round = 0, last_round = 0;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity, int where) {
      const bool w = mbar_wait(bar, parity, a.err, where);
      if (!__all_sync(0xffffffffu, w)) ok = false;
    };
    // O += P V of tile gt in stage st
    auto issue_pv = [&](int gt, int st, uint32_t rd, bool acc) {
      wait(b_vf(st), rd & 1, 13);
      wait(b_pf(buf_of(gt)), par_of(gt), 13);
      if (!ok) return;
      tc_fence_after();
      if (leader) {
        const uint64_t v = desc_offset(dV, st * 2 * F::kTile);
        const uint32_t pa = uS + buf_of(gt) * KT;
        if (acc)
          umma_ts_i<1>(uO, pa, v, id_o);
        else
          umma_ts_i<0>(uO, pa, v, id_o);
#pragma unroll
        for (int i = 1; i < 4; ++i) umma_ts_i<1>(uO, pa + 8 * i, v + i * 128, id_o);
        umma_commit(b_od(buf_of(gt)));
        umma_commit(b_ve(st));
      }
      __syncwarp();
    };
    for (int k = 0; ok; ++k) {
      wait(b_listed(k), (k / kListed) & 1, 25);
      const int kt = uniform(list[k % kListed].kt), t0 = uniform(list[k % kListed].t0);
      const int t1 = uniform(list[k % kListed].t1);
      if (!ok || kt == 0) break;
      wait(b_q, k & 1, 12);
      for (int t = t0; ok && t < t1; ++t, ++g) {
        // (the scores' buffer is free: it held the probabilities of tile g - 2,
        // whose product was issued before this)
        wait(b_kf(s), round & 1, 12);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint64_t kd = desc_offset(dK, s * 2 * F::kTile);
          const uint32_t ts = uS + buf_of(g) * KT;
#pragma unroll
          for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t qa = desc_offset(dQ, c * F::kChunkQ) + 2 * i;
              const uint64_t kb = desc_offset(kd, c * F::kChunk) + 2 * i;
              if (c == 0 && i == 0)
                umma_i<0>(ts, qa, kb, id_s);
              else
                umma_i<1>(ts, qa, kb, id_s);
            }
          umma_commit(b_sf(buf_of(g)));
          umma_commit(b_ke(s));
        }
        __syncwarp();
        if (t > t0) issue_pv(g - 1, last, last_round, t - 1 > t0);
        last = s;
        last_round = round;
        if (++s == NS) {
          s = 0;
          ++round;
        }
      }
      if (ok) issue_pv(g - 1, last, last_round, t1 - 1 > t0);
    }
    // all issued MMAs complete before TMEM is released
    if (g > 0) mbar_wait(b_od(buf_of(g - 1)), par_of(g - 1), a.err, 16);
  } else {
    // ------------------------------------------------ rows
    constexpr int NC = KT / P;               // keys of a tile that a copy takes
    const int e = (warp & 3) * 32 + lane;    // TMEM lane
    const int row = e % MR, copy = e / MR;   // of the tile
    const uint32_t lo = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tOw = tO + lo;            // this lane's output
    const float scale = rsqrtf(float(D)) * kLog2e;
    const bf16* qkv = static_cast<const bf16*>(a.qkv);
    int g = 0, mask_of = -1;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity, int where) {
      const bool w = mbar_wait(bar, parity, a.err, where);
      if (!__all_sync(0xffffffffu, w)) ok = false;
    };
    // barrier of the row threads with a bounded wait: a warp that gave up does
    // not leave the others waiting
    uint32_t syncs = 0;
    auto arrive = [&](uint32_t bar) {  // once a warp (128 arrivals take their time)
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto rows_sync = [&] {
      arrive(b_rows);
      wait(b_rows, syncs++ & 1, 22);
    };
    // The query rows of a piece, on their way as soon as the last piece's last
    // scores are there (every MMA that read its rows is complete then) ...
    auto start_q = [&](const Piece& q) {
      const bool real = row < q.rows;
      const int gr = q.rt * MR + (real ? row : 0), node = gr / a.G, h = q.hk * a.G + gr % a.G;
      const bf16* src = qkv + (int64_t(q.b) * a.N + node) * a.ld_qkv + int64_t(h) * D;
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        cp_async16(sQ + (c >> 3) * F::kChunkQ + e * 128 + (((c & 7) ^ (e & 7)) << 4), src + c * 8, real);
    };
    // ... and theirs to multiply.
    auto finish_q = [&] {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async();  // visible to the MMAs
      rows_sync();
      if (e == 0) mbar_arrive(b_q);
    };
    // A tile with foreign rows, or with nodes that a row may not see: value rows
    // behind the last key become 0, and so do node values that are not finite, whose
    // nodes are noted in `bad` (see add_nonfinite).
    auto clear = [&](const Piece& q, int t, int gt) -> bool {
      const int s = gt % NS;
      const bool fresh = t >= q.ct;
      const int nk = fresh ? q.n - (t - q.ct) * KT : q.len - t * KT;
      wait(b_vf(s), (gt / NS) & 1, 21);
      uint8_t* v = ring + s * 2 * F::kTile + F::kTile;
      uint64_t* word = bad + (fresh ? t - q.ct : 0);
      for (int x = e; x < KT * D / 8; x += kLanes) {  // 16-byte units, the swizzle left alone
        const int r = x / 8 % KT;
        uint4* at = reinterpret_cast<uint4*>(v + x * 16);
        if (r >= nk) {
          *at = make_uint4(0, 0, 0, 0);
        } else if (fresh) {
          uint4 u = *at;
          if (drop_nonfinite(u)) {
            *at = u;
            atomicOr(reinterpret_cast<unsigned long long*>(word), 1ull << r);
          }
        }
      }
      fence_proxy_async();  // before this thread's arrival that the product waits for
      if (!fresh) return false;
      rows_sync();
      return *word != 0;
    };
    wait(b_listed(0), 0, 26);
    if (ok && list[0].kt > 0) {
      start_q(list[0]);
      arrive(b_go);
      const Piece& q = list[0];
      if (a.parent && q.t1 > q.ct) {  // meanwhile its sequence's masks
        Parents parents;
        parents.load(a.parent + int64_t(q.b) * a.N, q.n, e, kLanes);
        build_masks(parents, q.n, mask, up, flag, a.err, e, kLanes, rows_sync);
        mask_of = q.b;
      }
      finish_q();
    }
    for (int k = 0; ok; ++k) {
      const Listed& p = list[k % kListed];
      if (p.kt == 0) break;
      const int rows = p.rows, t1 = p.t1, len = p.len, ct = p.ct, pn = p.n;
      const bool real = row < rows;
      const bool busy = (row & ~31) < rows;  // some row of this warp is real
      const int gr = p.rt * MR + (real ? row : 0), node = gr / a.G;
      const bool new_masks = a.parent && t1 > ct && mask_of != p.b;
      Parents parents;  // in flight until the nodes' tiles are reached
      if (new_masks) parents.load(a.parent + int64_t(p.b) * a.N, pn, e, kLanes);
      bool any_bad = false, first = true;
      float m = -INFINITY, l = 0.f;
      for (int t = p.t0; t < t1; ++t, ++g, first = false) {
        wait(b_sf(buf_of(g)), par_of(g), 14);
        if (t == t1 - 1) {  // (the plan does not wait for this tile)
          wait(b_listed(k + 1), ((k + 1) / kListed) & 1, 26);
          if (ok && list[(k + 1) % kListed].kt > 0) start_q(list[(k + 1) % kListed]);
        }
        if ((t + 1) * KT > len) {
          if (t == max(p.t0, ct)) {  // the piece's first node tile
            rows_sync();             // (the last piece's words and masks have been read)
            if (e < kMaxNodes / 64) bad[e] = 0;
            if (new_masks) {
              build_masks(parents, pn, mask, up, flag, a.err, e, kLanes, rows_sync);
              mask_of = p.b;
            }
            rows_sync();
          }
          any_bad |= clear(p, t, g);
        }
        if (!ok) break;
        if (!busy) {
          arrive(b_pf(buf_of(g)));
          continue;
        }
        tc_fence_after();
        const uint32_t tSw = tS + lo + buf_of(g) * KT;
        const bool open = (t + 1) * KT <= len;  // no key masked
        uint64_t see = ~uint64_t(0);
        if (!open) {
          const bool fresh = t >= ct;
          const int k0 = (fresh ? t - ct : t) * KT, nk = (fresh ? pn : len) - k0;
          if (nk < KT) see = (uint64_t(1) << nk) - 1;
          if (fresh) see &= sees(!a.parent, mask, node, k0);
        }
        // This copy's keys, up to 32 at a time: x = raw scores, keys that the row may
        // not see -inf.  The base m of the probabilities (log2 domain) follows the
        // maximum only when it grows by more than 2^8 (they stay <= 256); 0 is used
        // while the row has seen nothing (every p is then 2^(-inf) = 0).
#pragma unroll
        for (int h = 0; h < NC / 32; ++h) {
          const int key0 = copy * NC + h * 32;
          uint32_t r[32];
          tmem_ld32_async(tSw + key0, r);
          tmem_wait_ld(r);
          float x[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
          if (!open) {
            const uint32_t bits = uint32_t(see >> key0);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = (bits >> i) & 1 ? x[i] : -INFINITY;
          }
          float c2[2];
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            const float* y = x + 16 * k2;
            float mm = max3f(y[0], y[1], y[2]);
#pragma unroll
            for (int i = 3; i < 15; i += 2) mm = max3f(mm, y[i], y[i + 1]);
            c2[k2] = fmaxf(mm, y[15]);
          }
          const float mn = __fmul_rn(fmaxf(c2[0], c2[1]), scale);
          const bool resc = mn > m + kRescale;
          if (__any_sync(0xffffffffu, resc)) {
            // (between the halves by a whole number: the first half's probabilities are
            // in bf16 already, and scaled by a power of two they are not rounded again)
            const float by = h == 1 && m != -INFINITY ? ceilf(mn - m) : mn - m;
            const float corr = resc ? ex2(-by) : 1.f;
            if (resc) m = m != -INFINITY ? m + by : mn;
            l *= corr;
            if (h == 1) {  // the first half's probabilities had the old base
              uint32_t q[16];
              tmem_wait_st();
              tmem_ld16_raw(tSw, q);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&q[i]);
                q[i] = pack2(__low2float(v) * corr, __high2float(v) * corr);
              }
              tmem_st16_async(tSw, q);
            }
            if (!first) {  // O holds the last tile's product
              wait(b_od(buf_of(g - 1)), par_of(g - 1), 17);
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tmem_ld16_raw(tOw + c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
                tmem_st16_async(tOw + c, o);
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : m;
          uint32_t pk[16];
          float sa[2] = {0.f, 0.f}, sb[2] = {0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float u0, u1;
            fma2(u0, u1, x[i], x[i + 1], scale, scale, -base, -base);
            const float p0 = ex2(u0), p1 = ex2(u1);
            add2(sa[(i >> 1) & 1], sb[(i >> 1) & 1], p0, p1);
            pk[i >> 1] = pack2(p0, p1);
          }
          l += (sa[0] + sb[0]) + (sa[1] + sb[1]);
          // P (bf16) over the first 32 columns of its scores, the A operand of P V:
          // what it overwrites has been read; zeros for the other copies' keys
          if constexpr (P == 1) {
            tmem_st16_async(tSw + 16 * h, pk);
          } else {
            uint32_t zero[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) zero[i] = 0;
            tmem_st16_async(tSw + 16 * copy, pk);
            tmem_st16_async(tSw + 16 * (copy ^ 1), zero);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(b_pf(buf_of(g)));
      }
      if (!ok) break;
      if (list[(k + 1) % kListed].kt > 0) finish_q();  // its scores overlap this one's results
      wait(b_od(buf_of(g - 1)), par_of(g - 1), 19);
      if (!ok) break;
      tc_fence_after();
      const bool whole = p.whole();
      const int hq = p.hk * a.G + gr % a.G;
      bf16* out = static_cast<bf16*>(a.out) + (int64_t(p.b) * a.N + node) * a.ld_out + int64_t(hq) * D;
      float* w = a.ws + p.slot * slot_floats<MR>(D);
      float M = m, L = l, f = 1.f;
      if constexpr (P > 1) {  // over the row's copies
        ml[e] = make_float2(m, l);
        rows_sync();
        L = 0.f;
#pragma unroll
        for (int c = 0; c < P; ++c) M = fmaxf(M, ml[row + c * MR].x);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          const float2 u = ml[row + c * MR];
          L += u.x == -INFINITY ? 0.f : ex2(u.x - M) * u.y;
        }
        f = m == -INFINITY ? 0.f : ex2(m - M);
      }
      if (whole) f /= L;
      float odd = 0.f;  // NaN: the thread stored columns that are not finite (P > 1)
#pragma unroll
      for (int c = 0; c < D; c += 16) {
        float x[16];
        if (busy) {
          tmem_ld16(tOw + c, x);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= f;
        }
        if constexpr (P > 1) {
          // 16 columns at a time; the copies finish them in turn.  (With two buffers
          // the next exchange's barrier tells that this one has been read.)
          float* xc = xch + (c / 16) % F::kXch * (kLanes * F::LX);
          if (busy) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4*>(xc + e * F::LX + i) =
                  make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
          }
          rows_sync();
          if (busy && copy == (c / 16) % P) {
#pragma unroll
            for (int k2 = 1; k2 < P; ++k2) {
              const float* y = xc + (row + (copy + k2) % P * MR) * F::LX;
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(y + i);
                x[i] += v.x;
                x[i + 1] += v.y;
                x[i + 2] += v.z;
                x[i + 3] += v.w;
              }
            }
          }
          if (F::kXch == 1) rows_sync();
        }
        if (!real || copy != (c / 16) % P) continue;
        if constexpr (P > 1) {
          float y[4];  // (a sum with infinities or NaN is one)
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = (x[i] + x[i + 4]) + (x[i + 8] + x[i + 12]);
          odd = fmaf((y[0] + y[1]) + (y[2] + y[3]), 0.f, odd);
        }
        if (whole) {
#pragma unroll
          for (int i = 0; i < 16; i += 8)
            *reinterpret_cast<uint4*>(out + c + i) =
                make_uint4(pack2(x[i], x[i + 1]), pack2(x[i + 2], x[i + 3]), pack2(x[i + 4], x[i + 5]),
                           pack2(x[i + 6], x[i + 7]));
        } else {
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(w + int64_t(row) * D + c + i) =
                make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        }
      }
      if (!ok) break;
      tc_fence_before();
      if (real) {
        if (copy == 0) {
          if (whole) {
            if (a.lse) a.lse[(int64_t(p.b) * a.H + hq) * a.N + node] = (M + log2f(L)) * kLn2;
          } else {
            w[MR * D + row] = M;
            w[MR * D + MR + row] = L;
          }
        }
      }
      if (__any_sync(0xffffffffu, any_bad || odd != 0.f))
        share_nonfinite<D, P>(a, p, row, copy, any_bad, bad, mask, M, L);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

int grid_size() { return 2 * gpt2_internal::sm_count(); }

template <int D, int P>
int launch_tc(const TreeAttnArgs& a, cudaStream_t st) {
  using F = Cfg<D, P>;
  CUtensorMap mk, mv, mx;
  const int64_t rows = int64_t(a.B) * a.Hkv * a.Tc;
  if (!make_map_bf16(&mk, a.k, D, rows, D, KT) || !make_map_bf16(&mv, a.v, D, rows, D, KT) ||
      !make_map_bf16(&mx, a.qkv, int64_t(a.H + 2 * a.Hkv) * D, int64_t(a.B) * a.N, a.ld_qkv, KT)) {
    gpt2_internal::set_error("tree_attention: tensor map encoding failed");
    return GPT2_ERR_CUDA;
  }
  static std::atomic<uint64_t> allowed{0};
  GPT2_CUDA_TRY(allow_smem(allowed, tree_attn_tc_kernel<D, P>, F::kSmem));
  const TreeAttnArgs w = with_workspace<F::MR>(a, grid_size());
  tree_attn_tc_kernel<D, P><<<grid_size(), kThreads, F::kSmem, st>>>(mk, mv, mx, w);
  COUNT_LAUNCH(1);
  GPT2_LAUNCH_CHECK();
  return launch_combine<bf16, F::MR, D>(w, st);
}

int copies(int rows) { return rows <= 64 ? 2 : 1; }

}  // namespace

size_t tree_attn_tc_workspace(int B, int N, int H, int Hkv, int D) {
  return copies(N * (H / Hkv)) == 2 ? workspace_bytes<64>(grid_size(), B, N, H, Hkv, D)
                                    : workspace_bytes<128>(grid_size(), B, N, H, Hkv, D);
}

int launch_tree_attn_tc(const TreeAttnArgs& a, cudaStream_t st) {
  if (copies(a.N * a.G) == 2) return a.D == 128 ? launch_tc<128, 2>(a, st) : launch_tc<64, 2>(a, st);
  return a.D == 128 ? launch_tc<128, 1>(a, st) : launch_tc<64, 1>(a, st);
}
