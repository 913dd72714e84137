// Decode attention of groups with a common prefix: what its kernels share. A row's keys are cut
// into parts: Sp of the prefix ([s Lp, (s + 1) Lp) of the group's tokens) and Ss of its own
// tokens (from the first it sees, cut down to a 16-token tile, every Ls). Each part leaves the state
// of a softmax (m, l, acc[D]) for each (row, query head) that sees a key of it; the joining
// kernel adds them up: out = sum 2^(m - M) acc / sum 2^(m - M) l, M = max m.
#pragma once
#include "hyb_internal.cuh"

namespace hyb {

struct PrefixPlan {
  bool tc;             // the prefixes on the tensor cores
  int Lp, Sp;          // keys of a prefix part; parts of the longest prefix
  int Ls, Ss;          // keys of a part of a row's own tokens; parts of the longest
  size_t ws_bytes;
};

// What the kernels take of the call.
struct PrefixArgs {
  const int32_t *bt, *lens, *cu, *pre;
  int B, G, Hq, Hk, NB, MB, rsh, window;   // rsh: log2(block size / 16)
  int max_group, max_prefix, max_suffix;
  int cap;                                 // tokens that a table row holds (2^31 - 1 at most)
  float scale_log2;                        // log2(e) |scale|, not 0 (which is the same as a tiny one)
  uint32_t q_sign;                         // a pair's bf16 sign bits where the scale is negative
  int Lp, Sp, Ls, Ss;
  float* ws_acc;                           // [B][Hq][Sp + Ss][D]
  float2* ws_ml;                           // [B][Hq][Sp + Ss]
  unsigned* status;
};

constexpr int kMmaMaxPart = 1536;          // keys of a prefix part on warp matrix instructions, at most
bool prefix_mma_supported(int dtype, int D);
// prefix: the prefixes' parts too, not only those of the rows' own tokens; early: behind launch_prefix_tc of
// the same call
cudaError_t launch_prefix_mma(int D, const void* q, const void* kc, const void* vc, const PrefixArgs& a,
                              bool prefix, bool early, cudaStream_t s);

// the prefixes' parts on the tensor cores (bf16, D = 128, scale > 0, at most 128 query heads a key head)
int prefix_tc_tile_rows(int rep);          // rows of one of its row tiles; a CTA takes two
cudaError_t launch_prefix_tc(const void* q, const void* kc, const void* vc, const PrefixArgs& a, cudaStream_t s);

#ifdef __CUDACC__
// Rows [b0, b1) and prefix of a group; false where the call has to leave the group out.
__device__ __forceinline__ bool group_ok(const PrefixArgs& a, int g, int& b0, int& b1, int& P) {
  b0 = a.cu[g];
  b1 = a.cu[g + 1];
  P = a.pre[g];
  return b0 >= 0 && b1 >= b0 && b1 <= a.B && b1 - b0 <= a.max_group && P >= 0 &&
         P <= a.max_prefix && P <= a.cap;
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
__device__ __forceinline__ RowSpan row_span(const PrefixArgs& a, int n, int first, int P) {
  RowSpan r;
  n = max(n, 0);
  r.first = first;
  r.P = P;
  r.n = n;
  r.lo = (a.window > 0 && n > a.window) ? n - a.window : 0;
  if (n - P > a.max_suffix || n > a.cap) r.n = -1;
  return r;
}

// The keys of a prefix that some requests see: [lo, hi) from the first to the last of them. With a window, one request
// that ends early in the prefix and one that goes on behind it leave keys between that neither sees (gaps): then
// any_sees tells. What none sees is neither fetched nor looked at, whatever its table entries hold.
struct Hull {
  int lo = INT32_MAX, hi = 0;
  bool gaps = false;
  __device__ __forceinline__ void add(const PrefixArgs& a, int len, int P) {
    const RowSpan x = row_span(a, len, 0, P);
    const int end = min(P, x.n);
    if (end <= x.lo) return;
    lo = min(lo, x.lo);
    hi = max(hi, end);
    gaps |= end < P && a.window > 0;
  }
  __device__ __forceinline__ void join() {                     // the whole warp's
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    gaps = __any_sync(0xffffffffu, gaps);
  }
};
// Whether one of requests [b0, b1) sees one of the prefix's keys [k0, k1)
__device__ __forceinline__ bool any_sees(const PrefixArgs& a, int b0, int b1, int P, int k0, int k1) {
  for (int b = b0; b < b1; ++b) {
    const RowSpan x = row_span(a, a.lens[b], 0, P);
    if (max(x.lo, k0) < min(min(P, x.n), k1)) return true;
  }
  return false;
}

// Whole warp: row b's keys (n < 0: left out); bad: whether that is for its length. Group bounds, prefixes
// and the row's length are loaded side by side, so that a CTA with nothing to do leaves after one round trip.
__device__ __forceinline__ RowSpan find_row(const PrefixArgs& a, int b, bool* bad = nullptr) {
  const int lane = threadIdx.x & 31, n = a.lens[b];
  RowSpan r;
  r.first = r.P = r.lo = 0;
  r.n = -1;
  if (bad) *bad = false;
  // the last group that begins at b or before, 32 probes a step (cu does not decrease), down to 32 of them
  int g0 = 0, g1 = a.G;
  while (g1 - g0 > 32) {
    const int step = (g1 - g0 + 31) / 32, g = g0 + lane * step;
    const int k = __popc(__ballot_sync(0xffffffffu, g < g1 && a.cu[g] <= b));
    if (k == 0) return r;
    g0 += (k - 1) * step;
    g1 = min(g1, g0 + step);
  }
  {
    const int g = g0 + lane;
    int b0 = 0, b1 = 0, P = 0;
    const bool ok = g < g1 && group_ok(a, g, b0, b1, P);
    const unsigned m = __ballot_sync(0xffffffffu, g < g1 && b0 <= b && b < b1);
    if (!m) return r;
    const int src = __ffs(m) - 1;
    const bool good = __shfl_sync(0xffffffffu, ok, src);
    b0 = __shfl_sync(0xffffffffu, b0, src);
    P = __shfl_sync(0xffffffffu, P, src);
    if (good) {
      r = row_span(a, n, b0, P);
      if (bad) *bad = r.n < 0;
    }
  }
  return r;
}
#endif

}  // namespace hyb
