// Decode attention of groups with a common prefix: what its kernels share. A row's keys are cut
// into parts: Sp of the prefix ([s Lp, (s + 1) Lp) of the group's tokens) and Ss of its own
// tokens (from the first it sees, cut down to a 16-token tile, every Ls). Each part leaves the state
// of a softmax (m, l, acc[D]) for each (row, query head) that sees a key of it; the joining
// kernel adds them up: out = sum 2^(m - M) acc / sum 2^(m - M) l, M = max m.
#pragma once
#include "hyb_internal.cuh"

namespace hyb {

struct PrefixPlan {
  int Lp, Sp;          // keys of a prefix part; parts of the longest prefix
  int Ls, Ss;          // keys of a part of a row's own tokens; parts of the longest
  size_t ws_bytes;
};

// What the kernels take of the call.
struct PrefixArgs {
  const int32_t *bt, *lens, *cu, *pre;
  int B, G, Hq, Hk, NB, MB, rsh, window;   // rsh: log2(block size / 16)
  int max_group, max_prefix, max_suffix;
  float scale_log2;
  int Lp, Sp, Ls, Ss;
  float* ws_acc;                           // [B][Hq][Sp + Ss][D]
  float2* ws_ml;                           // [B][Hq][Sp + Ss]
  unsigned* status;
};

bool prefix_mma_supported(int dtype, int D);
// prefix: the prefixes' parts too, not only those of the rows' own tokens
cudaError_t launch_prefix_mma(int D, const void* q, const void* kc, const void* vc, const PrefixArgs& a,
                              bool prefix, cudaStream_t s);

#ifdef __CUDACC__
// Rows [b0, b1) and prefix of a group; false where the call has to leave the group out.
__device__ __forceinline__ bool group_ok(const PrefixArgs& a, int g, int& b0, int& b1, int& P) {
  b0 = a.cu[g];
  b1 = a.cu[g + 1];
  P = a.pre[g];
  return b0 >= 0 && b1 >= b0 && b1 <= a.B && b1 - b0 <= a.max_group && P >= 0 &&
         P <= a.max_prefix && P <= (a.MB << a.rsh) * kBlockSize;
}

// Keys of row b: [lo, min(P, n)) of the prefix, [max(P, lo), n) of its own. n < 0: left out.
struct RowSpan {
  int first, P, n, lo;
  __device__ __forceinline__ int own_lo() const { return max(P, lo); }
  // tokens of its own are cut from here
  __device__ __forceinline__ int own_base() const { return own_lo() & ~(kBlockSize - 1); }
  __device__ __forceinline__ bool prefix_part(int s, int Lp) const {
    return max(s * Lp, lo) < min(min(P, n), (s + 1) * Lp);
  }
  __device__ __forceinline__ int own_parts(int Ls) const {
    return n > own_lo() ? (n - own_base() + Ls - 1) / Ls : 0;
  }
};
__device__ __forceinline__ RowSpan row_span(const PrefixArgs& a, int b, int first, int P) {
  RowSpan r;
  r.first = first;
  r.P = P;
  const int n = a.lens[b];
  r.n = max(n, 0);
  r.lo = (a.window > 0 && n > a.window) ? n - a.window : 0;
  // (n and P are at most 2^31 - 1 and 2^24: the difference cannot overflow)
  if (n - P > a.max_suffix || n > (a.MB << a.rsh) * kBlockSize) r.n = -1;
  return r;
}

// Whole warp: the group of row b (-1: none).
__device__ __forceinline__ int group_of(const PrefixArgs& a, int b) {
  const int lane = threadIdx.x & 31;
  for (int g0 = 0; g0 < a.G; g0 += 32) {
    const int g = g0 + lane;
    const bool mine = g < a.G && a.cu[g] <= b && b < a.cu[g + 1];
    const unsigned m = __ballot_sync(0xffffffffu, mine);
    if (m) return g0 + __ffs(m) - 1;
  }
  return -1;
}
// Whole warp: row b's keys (n < 0: left out)
__device__ __forceinline__ RowSpan find_row(const PrefixArgs& a, int b) {
  const int g = group_of(a, b);
  RowSpan r;
  r.first = r.P = r.lo = 0;
  r.n = -1;
  int b0, b1, P;
  if (g < 0 || !group_ok(a, g, b0, b1, P)) return r;
  return row_span(a, b, b0, P);
}
#endif

}  // namespace hyb
