// Shared parts of the tree-attention kernels: the split of the work over the
// grid, the ancestor masks and the partial results.
//
// Work: sequence b has len cached positions and n drafted nodes.  Its queries
// are rows r = i * G + g (node i, query head g of the G heads that share a
// key/value head), cut into row tiles of MR rows; its keys are the cached
// positions followed by the nodes, each cut into key tiles of KT.  A segment is
// one (b, key/value head, row tile); the key tiles of all segments, in that
// order, form one list, and every CTA takes an equal run of it, whatever the
// lengths are: a long sequence is split over many CTAs, short ones share one.
// Each segment counts kExtra tiles more than it has, for what a piece costs
// besides its tiles (queries, masks, results; each kernel has its own number).
// Lengths are read on the device, so a recorded launch follows them.  A segment
// inside one CTA's run is finished there; the pieces of any other go to the
// workspace (unnormalised output, running maximum and sum in fp32) and
// tree_combine_kernel merges them in tile order, so the result does not depend on
// timing.
#pragma once

#include "kernels.h"
#include <type_traits>

#include "tree_internal.h"

namespace tree {

constexpr int kMaxNodes = 256;
constexpr int kMaskWords = kMaxNodes / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct SeqDims {
  int len, n;
};
// Lengths of sequence b; out-of-range values make the sequence empty.
__device__ __forceinline__ SeqDims seq_dims(const TreeAttnArgs& a, int b, bool* bad = nullptr) {
  SeqDims s;
  s.len = a.lens[b];
  s.n = a.counts ? a.counts[b] : a.N;
  if (s.len < 0 || s.len > a.Tc || s.n < 0 || s.n > a.N) {
    if (bad) *bad = true;
    s.len = s.n = 0;
  }
  return s;
}
__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

constexpr int kTable = 32;  // sequences whose lengths a CTA keeps in shared memory

// One piece of a CTA's run: key tiles [t0, t1) of a segment.
struct Piece {
  int b, hk, rt, t0, t1;
  int len, n, rows;  // the sequence's lengths, real rows of the row tile
  int kt, ct;        // key tiles of the segment, of them cache tiles
  int64_t s0;        // the segment's first tile in the list
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == kt; }
};

template <int MR, int KT, int kExtra>
struct Split {
  __device__ __forceinline__ static int row_tiles(const TreeAttnArgs& a, SeqDims s) {
    return ceil_div(s.n * a.G, MR);
  }
  // key tiles of each segment of the sequence (0 when it has no node)
  __device__ __forceinline__ static int key_tiles(SeqDims s) {
    return s.n ? ceil_div(s.len, KT) + ceil_div(s.n, KT) : 0;
  }
  // places in the list
  __device__ __forceinline__ static int64_t tiles(const TreeAttnArgs& a, SeqDims s) {
    return s.n ? int64_t(a.Hkv) * row_tiles(a, s) * (key_tiles(s) + kExtra) : 0;
  }

  // The pieces of a CTA's run in order.
  struct Pieces {
    const TreeAttnArgs* args;
    const SeqDims* table;  // lengths of sequences b0 .. b0 + 31
    int64_t pos, end, total, first;
    int ctas;  // CTAs with a run: never more than places, so that none is empty
    int b0, b;
    // (false: the run is done, p holds nothing)
    __device__ __forceinline__ bool next(Piece& p) {
      const TreeAttnArgs& a = *args;
      while (pos < end) {
        const SeqDims s = b - b0 < kTable ? table[b - b0] : seq_dims(a, b);
        const int64_t n = tiles(a, s);
        if (pos >= first + n) {
          first += n;
          ++b;
          continue;
        }
        p.b = b;
        p.len = s.len;
        p.n = s.n;
        p.kt = key_tiles(s);
        p.ct = ceil_div(s.len, KT);
        const int rts = row_tiles(a, s), places = p.kt + kExtra;
        const int seg = n < (int64_t(1) << 31) ? int(uint32_t(pos - first) / uint32_t(places))
                                               : int((pos - first) / places);
        p.s0 = first + int64_t(seg) * places;
        p.t0 = int(pos - p.s0);
        p.t1 = int(min64(p.kt, end - p.s0));
        pos = min64(end, p.s0 + places);
        if (p.t0 >= p.kt) continue;  // only the places behind the tiles
        p.hk = seg / rts;
        p.rt = seg % rts;
        p.rows = min(MR, s.n * a.G - p.rt * MR);
        return true;
      }
      return false;
    }
    // Workspace slot of a piece that is not a whole segment: 2 per CTA, the first
    // for a segment that began before the run, the second for one that begins
    // in it and goes on.
    __device__ __forceinline__ int64_t slot(const Piece& p) const { return 2 * int64_t(blockIdx.x) + (p.t0 == 0); }
    __device__ __forceinline__ int last_cta(int64_t x1) const {  // of place x1 - 1
      return total <= (1 << 20) && ctas <= 2048
                 ? int((uint32_t(x1) * uint32_t(ctas) - 1) / uint32_t(total))
                 : int((x1 * ctas - 1) / total);
    }
    // By the CTA in whose run the segment begins: the first and last CTA that
    // hold a piece of it (place x is CTA ((x + 1) ctas - 1) / total's).
    __device__ __forceinline__ void note(const Piece& p) const {
      const TreeAttnArgs& a = *args;
      const int rts = ceil_div(a.N * a.G, MR);
      a.seg[(int64_t(p.b) * a.Hkv + p.hk) * rts + p.rt] =
          make_int2(int(blockIdx.x), p.whole() ? int(blockIdx.x) : last_cta(p.s0 + p.kt));
    }
  };

  // floor(total c / ctas), in 32 bits where they do (64-bit divisions take longer
  // than the rest of the plan)
  __device__ __forceinline__ static int64_t share(int64_t total, int c, int ctas) {
    return total <= (1 << 20) && ctas <= 2048 ? int64_t(uint32_t(total) * uint32_t(c) / uint32_t(ctas))
                                              : total * c / ctas;
  }

  // This CTA's run, found by a whole warp; with `fill` it also writes the table
  // (a barrier with the table's readers must follow).
  __device__ __forceinline__ static Pieces plan(const TreeAttnArgs& a, SeqDims* table, bool fill) {
    const int lane = threadIdx.x & 31;
    bool bad = false;
    int64_t total = 0, first = 0, base = 0;
    int b0 = a.B;
    Pieces q{&a, table, 0, 0, 1, 0, 0, 0, 0};
    auto scan = [&](int64_t v) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      return v;
    };
    SeqDims s{0, 0};
    int64_t t = 0, in = 0;
    for (int c = 0; c < a.B; c += 32) {
      s = c + lane < a.B ? seq_dims(a, c + lane, &bad) : SeqDims{0, 0};
      t = tiles(a, s);
      in = scan(t);
      total += __shfl_sync(0xffffffffu, in, 31);
    }
    if (bad && blockIdx.x == 0) note_bad_input(a.err);
    q.total = total;
    q.ctas = int(min64(total, gridDim.x));
    if (int(blockIdx.x) >= q.ctas) return q;  // an empty run
    q.pos = share(total, blockIdx.x, q.ctas);
    q.end = share(total, blockIdx.x + 1, q.ctas);
    for (int c = 0; c < a.B; c += 32) {
      if (a.B > 32) {  // (else the lane's values are those of the loop above)
        s = c + lane < a.B ? seq_dims(a, c + lane) : SeqDims{0, 0};
        t = tiles(a, s);
        in = scan(t);
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + in > q.pos);
      if (hit) {
        const int src = __ffs(int(hit)) - 1;
        first = base + __shfl_sync(0xffffffffu, in - t, src);
        b0 = c + src;
        if (fill) {
          if (lane >= src) table[lane - src] = s;
          // the rest of the table (b0 .. b0 + 31) when the batch goes on
          const int more = c + 32 + lane;
          if (lane < src && more < a.B) table[more - b0] = seq_dims(a, more);
        }
        break;
      }
      base += __shfl_sync(0xffffffffu, in, 31);
    }
    q.first = first;
    q.b0 = q.b = b0;
    return q;
  }
};

// A run's pieces as one lane finds them and the CTA's other roles read them: kept
// in shared memory (their state would cost every thread's registers), published
// one by one, an empty one (kt = 0) last.  The lane that publishes also fills the
// ring of NS <= 6 tile stages, at least one tile a piece, and waits for a stage's
// release before it fills it again: when it writes piece k + kListed, every
// reader has left piece k.
constexpr int kListed = 8;
struct Listed : Piece {
  int64_t slot;  // workspace slot of the piece's results
};

// Ancestor masks of the sequence's nodes, bit j of mask i: node j is on the
// path from node i to the root, i included.  Every thread walks its nodes' paths
// up to kWalk steps; what is left of deeper trees goes by doubling, mask(i) |=
// mask(up(i)), up(i) = up(up(i)).  By the `threads` threads that call it (>=
// kMaxNodes / 2; thread tid of them), with `sync` their barrier; flag is a word
// of shared memory.  The thread's parents come in registers (see Parents), loaded
// long before.  A parent outside [-1, i) counts as -1 and is reported.
constexpr int kWalk = 16;
struct Parents {
  int p[2];
  __device__ __forceinline__ void load(const int32_t* parent, int n, int tid, int threads) {
    p[0] = tid < n ? parent[tid] : -1;
    p[1] = tid + threads < n ? parent[tid + threads] : -1;
  }
};
template <typename Sync>
__device__ __forceinline__ void build_masks(const Parents& parents, int n, uint32_t* mask, int* up,
                                            uint32_t* flag, int* err, int tid, int threads,
                                            Sync sync) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = tid + k * threads;
    int p = parents.p[k];
    if (i < n) {
      if (p < -1 || p >= i) {
        note_bad_input(err);
        p = -1;
      }
      up[i] = p;
    }
  }
  if (tid == 0) *flag = 0;
  sync();
  int left[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = tid + k * threads;
    left[k] = -1;
    if (i >= n) continue;
    uint64_t m[4] = {0, 0, 0, 0};
    int p = i;
#pragma unroll 1
    for (int step = 0; step <= kWalk && p >= 0; ++step) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if ((p >> 6) == q) m[q] |= uint64_t(1) << (p & 63);
      p = up[p];
    }
    if (p >= 0) *flag = 1;
    left[k] = p;
    uint4* dst = reinterpret_cast<uint4*>(mask + i * kMaskWords);
    dst[0] = make_uint4(uint32_t(m[0]), uint32_t(m[0] >> 32), uint32_t(m[1]), uint32_t(m[1] >> 32));
    dst[1] = make_uint4(uint32_t(m[2]), uint32_t(m[2] >> 32), uint32_t(m[3]), uint32_t(m[3] >> 32));
  }
  sync();
  if (*flag == 0) return;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (tid + k * threads < n) up[tid + k * threads] = left[k];
  sync();
  for (int reach = kWalk + 1; reach < n; reach <<= 1) {
    // reads of this round, then its writes
    uint32_t add[2][kMaskWords];
    int nu[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = tid + k * threads;
      nu[k] = -1;
      if (i < n && up[i] >= 0) {
        nu[k] = up[up[i]];
#pragma unroll
        for (int w = 0; w < kMaskWords; ++w) add[k][w] = mask[up[i] * kMaskWords + w];
      } else {
#pragma unroll
        for (int w = 0; w < kMaskWords; ++w) add[k][w] = 0;
      }
    }
    sync();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = tid + k * threads;
      if (i < n) {
        up[i] = nu[k];
#pragma unroll
        for (int w = 0; w < kMaskWords; ++w) mask[i * kMaskWords + w] |= add[k][w];
      }
    }
    sync();
  }
}
// Which of the 64 nodes k0 .. k0 + 63 node i sees: by the masks, or, with no
// tree given (a chain), those up to i.
__device__ __forceinline__ uint64_t sees(bool chain, const uint32_t* mask, int i, int k0) {
  if (chain) {
    const int d = i - k0;
    return d < 0 ? 0 : d >= 63 ? ~uint64_t(0) : (uint64_t(2) << d) - 1;
  }
  const uint32_t* w = mask + i * kMaskWords + (k0 >> 5);
  return w[0] | (uint64_t(w[1]) << 32);
}

// Node values that are not finite: the products take zeros in their place (0
// times such a value is not 0, and most rows may not see the node); the rows that
// see one get its share here, after their results were stored by this thread:
// channels [c0, c1) of a row whose result has base m (log2 domain), times inv_l,
// the probability once more from the query and the key.  bad: the nodes that hold
// such values, 64 bits per 64 nodes.
template <typename T>
__device__ __forceinline__ bool finite(T x) {
  return fabsf(to_f32<T>(x)) <= 3.4028234e38f;
}
template <typename T, typename Out>
__device__ __noinline__ void add_nonfinite(const TreeAttnArgs& a, int b, int hk, int hq, int node,
                                           int n, const uint64_t* bad, const uint32_t* mask, float m,
                                           float inv_l, Out* dst, int c0, int c1) {
  const T* x = static_cast<const T*>(a.qkv) + int64_t(b) * a.N * a.ld_qkv;
  const T* q = x + int64_t(node) * a.ld_qkv + int64_t(hq) * a.D;
  const float scale = rsqrtf(float(a.D)) * kLog2e;
  for (int k0 = 0; k0 < n; k0 += 64) {
    const uint64_t keys = bad[k0 >> 6] & sees(!a.parent, mask, node, k0);
    for (int j = 0; j < 64; ++j) {
      if (!((keys >> j) & 1)) continue;
      const T* k = x + int64_t(k0 + j) * a.ld_qkv + int64_t(a.H + hk) * a.D;
      const T* v = k + int64_t(a.Hkv) * a.D;
      float s = 0.f;
      for (int d = 0; d < a.D; ++d) s = fmaf(to_f32<T>(q[d]), to_f32<T>(k[d]), s);
      const float p = exp2f(fmaf(s, scale, -m)) * inv_l;
      if (p != 0.f)
        for (int c = c0; c < c1; ++c)
          if (!finite(v[c])) dst[c] = from_f32<Out>(fmaf(p, to_f32<T>(v[c]), to_f32<Out>(dst[c])));
    }
  }
}
// 8 bf16 values with those that are not finite (exponent bits all ones: one more
// carries into the sign's place) replaced by 0; whether there are any.
__device__ __forceinline__ bool drop_nonfinite(uint4& u) {
  auto carry = [](uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; };
  if (((carry(u.x) | carry(u.y) | carry(u.z) | carry(u.w)) & 0x80008000u) == 0) return false;
  auto clean = [&](uint32_t& w) { w &= ~(((carry(w) >> 15) & 0x00010001u) * 0xFFFFu); };
  clean(u.x), clean(u.y), clean(u.z), clean(u.w);
  return true;
}

// Workspace: 2 slots per CTA, each MR x D fp32 outputs, then the rows' running
// maximum (log2 domain) and sum, MR of each; then the segments' first and last
// CTA.
template <int MR>
__host__ __device__ inline int64_t slot_floats(int D) {
  return int64_t(MR) * (D + 2);
}
template <int MR>
size_t workspace_bytes(int grid, int B, int N, int H, int Hkv, int D) {
  return size_t(2) * grid * slot_floats<MR>(D) * sizeof(float) +
         size_t(B) * Hkv * cdiv(N * (H / Hkv), MR) * sizeof(int2);
}
template <int MR>
TreeAttnArgs with_workspace(TreeAttnArgs a, int grid) {
  a.seg = reinterpret_cast<int2*>(a.ws + 2 * int64_t(grid) * slot_floats<MR>(a.D));
  return a;
}

// The pieces of a split segment merged in order,
//   M = max m_c,  out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c,
// by D / 4 lanes per query row (16-byte loads); kWide: a row's pieces shared by
// the groups of lanes of a whole block, whose results are merged once more.
// One pass, the running maximum kept: every load of a row is in flight at once,
// and latency is what a merge of few pieces costs.
template <typename T, int MR, int D, bool kWide>
__global__ void __launch_bounds__(128) tree_combine_kernel(const __grid_constant__ TreeAttnArgs a) {
  constexpr int LP = D / 4;                // lanes of a row
  constexpr int NG = 128 / LP;             // groups of a block
  constexpr int kAhead = 8;                // pieces in flight
  __shared__ float4 sh_o[kWide ? 128 : 1];
  __shared__ float2 sh_ml[kWide ? NG : 1];
  const int group = threadIdx.x / LP, lane = threadIdx.x % LP;
  const uint32_t R = uint32_t(a.N) * a.G;  // rows of a (sequence, key/value head)
  const uint32_t row = kWide ? blockIdx.x : blockIdx.x * NG + group;
  if (row >= uint32_t(a.B) * a.Hkv * R) return;  // kWide: whole block
  const int r = int(row % R), bh = int(row / R), b = bh / a.Hkv, hk = bh % a.Hkv;
  const bool there = r < seq_dims(a, b).n * a.G;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 seg = a.seg[int64_t(bh) * ceil_div(int(R), MR) + r / MR];
  const int i = r / a.G, h = hk * a.G + r % a.G;
  T* out = static_cast<T*>(a.out) + (int64_t(b) * a.N + i) * a.ld_out + int64_t(h) * D + lane * 4;
  float* lse = a.lse ? a.lse + (int64_t(b) * a.H + h) * a.N + i : nullptr;
  if (!there) {
    if (a.zero && (!kWide || group == 0)) {
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2*>(out) = make_uint2(0, 0);
      else
        *reinterpret_cast<float4*>(out) = make_float4(0.f, 0.f, 0.f, 0.f);
      if (lse && lane == 0) *lse = 0.f;
    }
    return;
  }
  const int np = seg.y - seg.x + 1;  // the first in its CTA's second slot
  if (np == 1) return;               // finished by its CTA
  const int64_t sf = slot_floats<MR>(D);
  const int rr = r % MR;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, l = 0.f;
  auto add = [&](float m1, float l1, float4 x) {
    const float mn = fmaxf(M, m1);
    const float f0 = M == -INFINITY ? 0.f : exp2f(M - mn), f1 = m1 == -INFINITY ? 0.f : exp2f(m1 - mn);
    M = mn;
    l = fmaf(l, f0, l1 * f1);
    o.x = fmaf(o.x, f0, x.x * f1);
    o.y = fmaf(o.y, f0, x.y * f1);
    o.z = fmaf(o.z, f0, x.z * f1);
    o.w = fmaf(o.w, f0, x.w * f1);
  };
  constexpr int step = kWide ? NG : 1;
  for (int i = kWide ? group : 0; i < np; i += kAhead * step) {
    float mi[kAhead], li[kAhead];
    float4 x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int c = i + j * step;
      const float* p = a.ws + (2 * int64_t(seg.x + c) + (c == 0)) * sf;
      mi[j] = c < np ? p[MR * D + rr] : -INFINITY;
      li[j] = c < np ? p[MR * D + MR + rr] : 0.f;
      if (c < np) x[j] = *reinterpret_cast<const float4*>(p + int64_t(rr) * D + lane * 4);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i + j * step < np) add(mi[j], li[j], x[j]);
  }
  if (kWide) {
    sh_o[threadIdx.x] = o;
    if (lane == 0) sh_ml[group] = make_float2(M, l);
    __syncthreads();
    if (group) return;
#pragma unroll
    for (int g = 1; g < NG; ++g) add(sh_ml[g].x, sh_ml[g].y, sh_o[g * LP + lane]);
  }
  const float inv = 1.f / l;
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    *reinterpret_cast<float4*>(out) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  }
  if (lse && lane == 0) *lse = (M + log2f(l)) * kLn2;
}

// Launched with programmatic serialisation: its blocks may be resident before
// the attention kernel ends and wait for it on the device.
template <typename T, int MR, int D>
int launch_combine(const TreeAttnArgs& a, cudaStream_t st) {
  const int64_t rows = int64_t(a.B) * a.N * a.H;
  // few rows: each has many pieces, a block shares them
  const bool wide = rows < 8 * int64_t(gpt2_internal::sm_count());
  constexpr int NG = 128 / (D / 4);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned(wide ? rows : cdiv64(rows, NG)));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  GPT2_CUDA_TRY(wide ? cudaLaunchKernelEx(&cfg, tree_combine_kernel<T, MR, D, true>, a)
                     : cudaLaunchKernelEx(&cfg, tree_combine_kernel<T, MR, D, false>, a));
  COUNT_LAUNCH(1);
  return GPT2_OK;
}

}  // namespace tree
