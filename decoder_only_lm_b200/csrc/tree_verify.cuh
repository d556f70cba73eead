// Shared by the kernels of tree verification: the tree, the order and the weights
// of a row's ids, and warp operations on 64-bit integers.
#pragma once

#include "tree_internal.h"

namespace tree {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;  // CTAs of a sequence
constexpr int kPer = kTreeMaxVocab / kCluster / kThreads;  // ids of a thread at most
constexpr double kOne = 68719476736.0;  // 2^36
constexpr unsigned kAll = 0xffffffffu;

// A uniform number as the walk uses it (NaN counts as 0).
__device__ __forceinline__ double unit(float v) { return double(fminf(fmaxf(v, 0.f), 1.f)); }

// Order of the ids of a row: by logit, the smaller id first among equal ones.
__device__ __forceinline__ uint32_t order_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);  // -0 counts as 0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(float z, int id) {
  return (uint64_t(order_of(z)) << 32) | uint64_t(0xFFFFFFFFu - uint32_t(id));
}
__device__ __forceinline__ float key_logit(uint64_t key) {
  const uint32_t ord = uint32_t(key >> 32);
  return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7FFFFFFFu) : ~ord);
}
__device__ __forceinline__ float clean(float z) { return z != z ? -INFINITY : z; }

// rint(2^36 exp(-d / T)) for d = zmax - z >= 0 by a table and a short polynomial
// (P. Tang's scheme, 1989).  With x = 64 d log2(e) / T = r - n, n the nearest
// integer (from the 1.5 * 2^52 shift): 2^36 exp(-d / T) = 2^(36 + n / 64) 2^(r / 64),
// the first factor from a table of 64 and an exponent, the second from its Taylor
// sum, |r ln2 / 64| < 0.0055: the first term left out is below 4e-17.  What is
// rounded is within 2^-14 of 2^36 exp(-d / T) (below 2^-16 in 40000 arguments
// computed in 60 digits), so a weight is the nearest whole number except, rarely,
// next to the middle of two.  Returned as 2^52 + weight, whose low 52 bits are the
// integer.
constexpr double kOnes = 4503599627370496.0;  // 2^52
struct Exp {
  const double* table;  // 2^(36 + i / 64)
  double per_unit;      // -64 log2(e) / T
  float most;           // 40 T: from this d on a weight is 0, 2^36 exp(-40) < 1/2
  __device__ Exp(const double* t, float T)
      : table(t), per_unit(-64.0 * 1.4426950408889634 / double(T)), most(40.f * T) {}
  __device__ static double entry(int i) { return exp2(36.0 + i / 64.0); }
  __device__ double of(double d) const {
    constexpr double kShift = 6755399441055744.0;  // 1.5 * 2^52
    constexpr double c = 0.010830424696249145;     // ln(2) / 64
    const double t = fma(d, per_unit, kShift);
    const double r = fma(d, per_unit, kShift - t);
    const int n = max(__double2loint(t), -64 * 64);  // (2^-28 at most: none)
    double p = fma(r, c * c * c * c * c / 120, c * c * c * c / 24);
    p = fma(r, p, c * c * c / 6);
    p = fma(r, p, c * c / 2);
    p = fma(r, p, c);
    p = fma(r, p, 1.0) * table[n & 63];
    return __hiloint2double(__double2hiint(p) + ((n & ~63) << 14), __double2loint(p)) + kOnes;
  }
  // z is limited from below in fp32 (NaN and -inf with it), at an fp32 step behind
  // zmax - 40 T.
  __device__ float lowest(float zmax) const { return __fsub_rd(zmax, most); }
  __device__ double operator()(float z, float zmax, float low) const {
    return of(double(zmax) - double(fmaxf(z, low)));
  }
  // Where that step is thousands of 40 T wide, or the maximum infinite, the ids at
  // the maximum have weight 2^36 and the others none (the steps are 2^-24 of the
  // maximum and T <= 1e20, so with a maximum so low that 40 T below it is no
  // number they are as wide): as with maximum 0 and the logits of only().
  __device__ bool lone(float zmax) const { return !(zmax - lowest(zmax) < 16384.f * most); }
};
__device__ __forceinline__ float only(float z, float zmax) {
  return clean(z) == zmax ? 0.f : -INFINITY;
}
__device__ __forceinline__ uint64_t integer_of(double v) {
  return uint64_t(__double_as_longlong(v)) & 0xFFFFFFFFFFFFFull;
}

__device__ __forceinline__ uint64_t weight_of(const Exp& ex, float z, float zmax) {
  if (ex.lone(zmax)) {
    z = only(z, zmax);
    zmax = 0.f;
  }
  return integer_of(ex(z, zmax, ex.lowest(zmax)));
}

// Sum over a warp of values below 2^53: three parts of 21 bits, 32 of which fit
// 32 bits.
__device__ __forceinline__ uint64_t warp_add(uint64_t v) {
  const uint64_t a = __reduce_add_sync(kAll, uint32_t(v) & 0x1FFFFFu);
  const uint64_t b = __reduce_add_sync(kAll, uint32_t(v >> 21) & 0x1FFFFFu);
  const uint64_t c = __reduce_add_sync(kAll, uint32_t(v >> 42));
  return a + (b << 21) + (c << 42);
}
__device__ __forceinline__ uint64_t warp_top(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(kAll, uint32_t(v >> 32));
  const uint32_t lo = __reduce_max_sync(kAll, uint32_t(v >> 32) == hi ? uint32_t(v) : 0u);
  return (uint64_t(hi) << 32) | lo;
}
// Inclusive running sum over a warp's lanes.
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(kAll, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// A sequence's tree in shared memory, and the children of the node at hand.
struct Tree {
  int tok[kTreeMaxNodes], par[kTreeMaxNodes], kid[kTreeMaxNodes];
  float u[kTreeMaxNodes];
  uint64_t kw[kTreeMaxNodes], kx[kTreeMaxNodes];  // the children's weights
  double exp_table[64];
  int n_kids;
};
// Loads it and starts the outputs; the number of nodes (0: the call is over).
__device__ __forceinline__ int load_tree(const TreeVerifyArgs& a, Tree& t, int b, int rank, int tid) {
  int N = a.counts ? a.counts[b] : a.N;
  bool bad = N < 0 || N > a.N;
  if (bad) N = 0;
  if (const int i = tid; i < a.N) {  // (no more nodes than threads)
    const int64_t at = int64_t(b) * a.N + i;
    if (rank == 0) a.path[at] = i == 0 && N > 0 ? 0 : -1;
    t.tok[i] = a.tokens[at];
    t.u[i] = a.uniform[at];
    const int p = a.parent ? a.parent[at] : i - 1;
    if (i < N && (p < -1 || p >= i)) bad = true;
    t.par[i] = p;
  }
  if (bad && rank == 0) note_bad_input(a.err);
  if (tid < 64) t.exp_table[tid] = Exp::entry(tid);
  if (N == 0 && rank == 0 && tid == 0) {
    a.n_path[b] = 0;
    a.next[b] = -1;
  }
  return N;
}
// One warp: the children of cur, in id order.
__device__ __forceinline__ void find_children(Tree& t, int cur, int N, int lane) {
  int m = 0;
  for (int j0 = cur + 1; j0 < N; j0 += 32) {
    const int j = j0 + lane;
    const bool is = j < N && t.par[j] == cur;
    const unsigned which = __ballot_sync(kAll, is);
    if (is) t.kid[m + __popc(which & ((1u << lane) - 1))] = j;
    m += __popc(which);
  }
  if (lane == 0) t.n_kids = m;
}

// x S / X taken from a weight, not below 0.
__device__ __forceinline__ uint64_t less(uint64_t w, uint64_t x, double f) {
  const int64_t r = int64_t(w) - __double2ll_rn(double(x) * f);
  return r > 0 ? uint64_t(r) : uint64_t(0);
}

}  // namespace tree
