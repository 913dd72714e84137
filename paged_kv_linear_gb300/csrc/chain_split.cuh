// Work split of the chunked prefill kernels: (request, head) chains shared out evenly over the
// CTAs of a cooperative launch, chains cut between two CTAs included.
//
// Units are the (request, head) chains, in order u = b * H + h; unit u has chunks_of(b) chunks.
// Laid end to end they occupy G chunk positions. CTA p takes positions [p*L, (p+1)*L) with
// L = max(longest chain, ceil(G / P)) (McNaughton's wrap-around rule for preemptive
// scheduling on P machines), so no chain crosses more than one CTA boundary. A chain cut
// at the boundary (p+1)*L is run in two parts, its first chunks by CTA p+1 FIRST and the
// rest by CTA p LAST: the first part is no longer than the work CTA p does before its last
// part, so the state it hands over (through the state pool) is ready when it is needed.
// A handoff is announced by a flag that names the call: the call's epoch (a counter that a
// one-thread kernel bumps right before every launch, in stream order, so graph replays get
// fresh epochs too) and the launch's grid id (distinct for launches that run at the same
// time). A waiting CTA accepts only its own call's value, never one left by an earlier call.
// Epoch and flags live in the caller's workspace: hs[0] is the epoch, hs[1 + p] holds the tag
// of the call whose CTA p has written the state of the chain it cut (at its first boundary)
// to the pool. The library itself holds no handoff state, so calls with distinct workspaces
// never see each other's flags.
#pragma once
#include "hyb_internal.cuh"

#ifdef __CUDACC__
namespace hyb {

struct Plan {
  int head_u, head_end;      // chain run first, chunks [0, head_end); -1: none
  int full_u0, full_u1;      // chains run whole, in order
  int tail_u, tail_begin;    // chain run last, chunks [tail_begin, nch); -1: none
};

__device__ __forceinline__ int warp_incl_scan(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Run by one whole warp; every lane returns the same plan for CTA p of P. chunks_of(b): the
// chunks of request b's chains. kCost: what a chain costs beside its chunks (its state's way in and
// out), in chunks; it lies before the chain's first chunk, and a chain of whose chunks none would
// come before the cut is not cut.
template <int kCost = 0, typename F>
__device__ Plan make_plan(const F& chunks_of, int B, int H, int P, int p, int lane) {
  auto span = [&](int b) {
    const int nc = chunks_of(b);
    return nc > 0 ? nc + kCost : 0;
  };
  long long total = 0;
  int longest = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int nc = b0 + lane < B ? span(b0 + lane) : 0;
    total += __reduce_add_sync(0xffffffffu, (unsigned)nc);
    longest = max(longest, (int)__reduce_max_sync(0xffffffffu, (unsigned)nc));
  }
  const long long G = total * H;
  const long long L = max((long long)longest, (G + P - 1) / P);
  const long long s = (long long)p * L, e = min(s + L, G);
  Plan pl{-1, 0, 0, 0, -1, 0};
  if (s >= G) return pl;
  // locate positions s and e: request b holds [base + H*excl, base + H*incl)
  int us = -1, offs = 0, ue = -1, offe = 0;
  long long base = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int b = b0 + lane;
    const int nc = b < B ? span(b) : 0;
    const int incl = warp_incl_scan(nc, lane);
    const long long lo = base + (long long)H * (incl - nc), hi = base + (long long)H * incl;
    const bool in_s = nc > 0 && s >= lo && s < hi, in_e = nc > 0 && e >= lo && e < hi;
    const unsigned ms = __ballot_sync(0xffffffffu, in_s), me = __ballot_sync(0xffffffffu, in_e);
    const int u_s = in_s ? b * H + (int)((s - lo) / nc) : 0, o_s = in_s ? (int)((s - lo) % nc) : 0;
    const int u_e = in_e ? b * H + (int)((e - lo) / nc) : 0, o_e = in_e ? (int)((e - lo) % nc) : 0;
    if (ms) {
      const int l = __ffs(ms) - 1;
      us = __shfl_sync(0xffffffffu, u_s, l);
      offs = __shfl_sync(0xffffffffu, o_s, l);
    }
    if (me) {
      const int l = __ffs(me) - 1;
      ue = __shfl_sync(0xffffffffu, u_e, l);
      offe = __shfl_sync(0xffffffffu, o_e, l);
    }
    base += (long long)H * __shfl_sync(0xffffffffu, incl, 31);
  }
  if (offs > 0) {
    const int end = span(us / H) - offs - kCost;
    if (end > 0) {
      pl.head_u = us;
      pl.head_end = end;
    }
    pl.full_u0 = us + 1;
  } else {
    pl.full_u0 = us;
  }
  if (e >= G) {
    pl.full_u1 = B * H;
  } else if (offe > 0) {
    pl.tail_u = ue;
    pl.tail_begin = max(0, span(ue / H) - offe - kCost);
    pl.full_u1 = ue;
  } else {
    pl.full_u1 = ue;
  }
  return pl;
}

__device__ __forceinline__ unsigned long long grid_id() {
  unsigned long long g;
  asm volatile("mov.u64 %0, %%gridid;" : "=l"(g));
  return g;
}
__device__ __forceinline__ void st_release_u64(unsigned long long* p, unsigned long long v) {
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long ld_acquire_u64(const unsigned long long* p) {
  unsigned long long v;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
// Waits, as a whole warp, until the CTA that ran a chain's start has handed its state over in this
// call, and brings the warp together again. False when limit_ns is up: the state may then still be
// written there, so the caller reads and writes none of it and ends its part of the kernel.
__device__ __forceinline__ bool take_handoff(const unsigned long long* fl, unsigned long long tag,
                                             uint64_t limit_ns = 2000000000ull) {
  const uint64_t t0 = global_ns();
  bool ok = ld_acquire_u64(fl) == tag;
#pragma unroll 1
  while (!ok && global_ns() - t0 <= limit_ns) {
    __nanosleep(100);
    ok = ld_acquire_u64(fl) == tag;
  }
  ok = __all_sync(0xffffffffu, ok);
  __syncwarp();
  return ok;
}

}  // namespace hyb
#endif
