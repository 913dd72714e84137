// Beam selection (hyb_beam_select): for each request the best continuations over its beams and
// the vocabulary.
//
// The first kernel reads the logits once. A CTA takes a slice of a live row in batches of 8192 (fp32: 4096)
// and keeps its maximum, its sum of exponentials and its N best, as keys (logit as an ordered integer, token
// complemented), which no two tokens share: equal logits go by the lower token without further ado. From the first
// batch's 256 thread maxima comes a bound that N logits reach (of each of the 8 warps the ceil(N / 8)-th largest,
// of these the least); what reaches it is collected in shared memory. From then on only logits above the bound are
// collected, few of a batch; whenever more than kKeep are there, they are thinned out and the bound rises. A
// batch fits behind kKeep entries whatever its logits, so rising, constant or tied rows need no other path. The order
// in which threads collect changes nothing: keys are unique. Which token is summed where depends on the token alone,
// not on where its row lies, so equal rows have equal sums and their candidates tie.
//
// The second kernel, one CTA a request, joins the slices' sums in 64 bits and picks among W S N candidates the
// same way, by totals in 64 bits.
//
// Bytes would bound it, each logit read once; instructions do. 64 x 8 beams over 131072 tokens, bf16 (134 MB): 43 us a
// call, 20 at the copy rate; the first kernel 38 us, 3.5 TB/s, 27 million warp instructions, issue slots 57 % busy: some
// 140 of a warp's 400 a batch are the exponentials and their sum, 110 the loads, maxima and loop, the rest the
// candidates. Four CTAs an SM with the next batch's loads in flight, and a slice of 8 batches where there are rows enough
// (while the whole took 48 us: five CTAs without loads ahead 54; slices of 4 batches 50, 2 61, 1 75, since each starts
// its bound anew). Warps that put down their own best without a barrier a batch: 47 us, and rising rows 0.8 ms or more.
// The same shape with 8 choices and every row constant takes 56 us, falling 43, rising, where each batch raises the
// bound, 170. More choices collect more: 16 / 24 / 32 / 64 / 128 take 52 / 58 / 60 / 84 / 123 us (random), 66 / 70 / 64 / 78
// / 84 (constant), 52 / 57 / 53 / 68 / 93 (falling), 180 / 187 / 206 / 241 / 277 (rising). One request of 4 beams over
// 32768 tokens, fp32: 10 us, two kernels of some 4 us.
#include <cuda_bf16.h>

#include <cmath>
#include <type_traits>

#include "tc.cuh"

namespace hyb {
namespace {

constexpr int kThreads = 256;
constexpr int kSpan = 65536;              // tokens of a slice, at most
constexpr int kKeep = 512;               // candidates kept between batches, at most
constexpr unsigned kNone = 0xffffffffu;

// What the first kernel leaves of (row, slice): (max, sum of e^(x - max)), then N (logit, token).
struct SelectArgs {
  const float* scores;
  const uint8_t* finished;
  int R, W, N, V, S, slice;              // slices of a row, elements of a slice (whole batches)
  int64_t stride;
  int eos;
  float2* ml;                            // [R W][S]
  float2* best;                          // [R W][S][N]: logit, token as bits
  unsigned* status;
};

// Keys whose order as integers is (value descending, index ascending): -0 counts as +0.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}
struct Key {                             // of a total and its position w V + v, complemented
  uint64_t hi;
  uint32_t lo;
  __device__ __forceinline__ bool operator>(const Key& o) const { return hi != o.hi ? hi > o.hi : lo > o.lo; }
};

// a key's upper 32 bits: in the keys' order, equal for keys that are nearly so; 0 is below all
__device__ __forceinline__ uint32_t coarse(uint32_t k) { return k; }
__device__ __forceinline__ uint32_t coarse(uint64_t k) { return (uint32_t)(k >> 32); }
__device__ __forceinline__ uint32_t coarse(const Key& k) { return (uint32_t)(k.hi >> 32); }

// Whole warp: a key that at least r >= 1 of the lanes' reach, the r-th largest; 0 where fewer have one.
__device__ __forceinline__ uint32_t rth_largest(uint32_t mine, int r) {
  if (r > 10) {
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < 32; ++j) above += __shfl_sync(0xffffffffu, mine, j) > mine;
    // lanes with fewer than r above them hold the r largest; the least of those is the r-th
    const int most = __reduce_max_sync(0xffffffffu, above < r ? above : -1);
    return __shfl_sync(0xffffffffu, mine, __ffs(__ballot_sync(0xffffffffu, above == most)) - 1);
  }
  uint32_t top = __reduce_max_sync(0xffffffffu, mine);
  for (; r > 1; --r) {
    const unsigned at = __ballot_sync(0xffffffffu, mine == top);
    if ((threadIdx.x & 31) == __ffs(at) - 1) mine = 0;
    top = __reduce_max_sync(0xffffffffu, mine);
  }
  return top;
}
// A bound that N of the CTA's 256 keys (and so of what they are the largest of) reach, in two steps with a barrier
// between: each warp puts down some of its largest, and every warp reads the bound off them (0: none). Up to N = 24
// each puts down its ceil(N / 8) + 1 largest, and the N-th largest of all of these is the bound: it is nearly the
// N-th largest of the 256. Beyond, the ceil(N / 8)-th of each warp, and the least of those.
constexpr int kLow = 32;
__device__ __forceinline__ void put_low(uint32_t* low, uint32_t mine, int N) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (N > 24) {
    const uint32_t b = rth_largest(mine, (N + 7) / 8);
    if (lane == 0) low[warp] = b;
    return;
  }
  const int t = (N + 7) / 8 + 1;
  for (int k = 0; k < t; ++k) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, mine);
    if (lane == 0) low[warp * t + k] = top;
    const unsigned at = __ballot_sync(0xffffffffu, mine == top);
    if (lane == __ffs(at) - 1) mine = 0;
  }
}
__device__ __forceinline__ uint32_t read_low(const uint32_t* low, int N) {
  const int lane = threadIdx.x & 31;
  if (N > 24) return __reduce_min_sync(0xffffffffu, low[lane & 7]);
  return rth_largest(lane < 8 * ((N + 7) / 8 + 1) ? low[lane] : 0u, N);
}

// Whole CTA: thins list[0, count) to at most kThreads entries that hold its N <= 128 best; returns how many.
// A round finds a bound among the threads' own largest and drops what does not reach it. First the quick
// bound (see the top), which mostly suffices; then the N-th largest of the 256, which N ceil(count / 256) <=
// 128 ceil(count / 256) entries reach at most: from 4608 entries (fp32) 2304, 1152, 640, 384, 256, from 8704 (bf16) 4352,
// 2176, 1152 and so on.
template <typename K>
__device__ __forceinline__ int thin_out(K* list, int count, int N, K* scratch, uint32_t* low, int* left) {
  const int tid = threadIdx.x;
  for (bool quick = true; count > kThreads; quick = false) {
    __syncthreads();
    K top = K();
    for (int i = tid; i < count; i += kThreads)
      if (list[i] > top) top = list[i];
    if (tid == 0) *left = 0;
    if (quick) {
      put_low(low, coarse(top), N);
    } else {
      scratch[tid] = top;
    }
    __syncthreads();
    if (!quick) {                        // (all threads have entries, and no two keys are equal)
      int above = 0;
#pragma unroll 8
      for (int i = 0; i < kThreads; ++i) above += scratch[i] > top;
      __syncthreads();
      if (above == N - 1) scratch[0] = top;
      __syncthreads();
    }
    const K bound = quick ? K() : scratch[0];
    const uint32_t about = quick ? read_low(low, N) : 0u;
    // in rounds, so that an entry is read before its place may be written: places written lie below those read
    for (int i0 = 0; i0 < count; i0 += kThreads) {
      const int i = i0 + tid;
      K k = K();
      if (i < count) k = list[i];
      const bool keep = i < count && coarse(k) >= about && !(bound > k);
      __syncthreads();
      if (keep) list[atomicAdd(left, 1)] = k;
      __syncthreads();
    }
    count = *left;
  }
  return count;
}

// Whole CTA, at the end: the N best of list[0, count) in order, give(rank, key) for each; returns how many there
// are (N at most). More than 64 are first held against a bound as of a batch's maxima: it leaves some 3 N.
template <typename K, typename F>
__device__ __forceinline__ int in_order(K* list, int count, int N, K* scratch, uint32_t* low, int* left, F&& give) {
  const int tid = threadIdx.x;
  count = thin_out(list, count, N, scratch, low, left);
  __syncthreads();
  if (count > 64) {
    const K mine = tid < count ? list[tid] : K();
    put_low(low, coarse(mine), N);
    if (tid == 0) *left = 0;
    __syncthreads();
    const uint32_t b = read_low(low, N);
    if (tid < count && coarse(mine) >= b) list[atomicAdd(left, 1)] = mine;   // (all were read before the barrier)
    __syncthreads();
    count = *left;
  }
  if (tid < count) {
    const K k = list[tid];
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < count; ++i) rank += list[i] > k;
    if (rank < N) give(rank, k);
  }
  return min(count, N);
}

// 16 bytes of logits, kept raw until their batch's turn. Key: unique in a slice, greater for a greater logit or
// the same at a lower token (t: the token's number in the slice, below kSpan); 0 is below all.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4, VECS = 4;  // vectors of a thread in a batch: 64 bytes
  using Key = uint64_t;
  __device__ static Key key(float x, int t) { return (uint64_t)ordered(x) << 32 | (uint32_t)(kSpan - t); }
  __device__ static float logit(Key k) { return unordered((uint32_t)(k >> 32)); }
  __device__ static int token(Key k) { return kSpan - (int)(uint32_t)k; }
  __device__ static void unpack(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  __device__ static float max_of(const uint4& u) {             // (NaN is passed over)
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  __device__ static float at(const uint4& u, int e) {
    return __uint_as_float(e & 2 ? (e & 1 ? u.w : u.z) : (e & 1 ? u.y : u.x));
  }
  // bit e: element e is above b, or equal to it where `equal`
  __device__ static unsigned reach(const uint4& u, float b, bool equal) {
    float f[4];
    unpack(u, f);
    unsigned m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) m |= (unsigned)(equal ? f[e] >= b : f[e] > b) << e;
    return m;
  }
  __device__ static uint4 edge(const float* x, int i, int lo, int hi) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(i + e >= lo && i + e < hi ? x[i + e] : -INFINITY);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8, VECS = 4;
  using Key = uint32_t;
  // (the 16 bits of a bf16 and the token's number, 65535 - t)
  __device__ static Key key(float x, int t) { return (ordered(x) & 0xffff0000u) | (uint32_t)(kSpan - 1 - t); }
  __device__ static float logit(Key k) {
    const uint32_t o = k & 0xffff0000u;
    return __uint_as_float((o & 0x80000000u) ? o & 0x7fff0000u : ~o & 0xffff0000u);
  }
  __device__ static int token(Key k) { return kSpan - 1 - (int)(k & 0xffffu); }
  __device__ static void unpack(const uint4& u, float* f) {
    f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x); f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
    f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z); f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
  }
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ static float max_of(const uint4& u) {
    const uint32_t m = max2(max2(u.x, u.y), max2(u.z, u.w));
    return fmaxf(bf16_lo(m), bf16_hi(m));
  }
  __device__ static float at(const uint4& u, int e) {
    const uint32_t w = e & 4 ? (e & 2 ? u.w : u.z) : (e & 2 ? u.y : u.x);
    return e & 1 ? bf16_hi(w) : bf16_lo(w);
  }
  __device__ static unsigned reach(const uint4& u, float b, bool equal) {
    const uint32_t b2 = (__float_as_uint(b) >> 16) * 0x10001u, w[4] = {u.x, u.y, u.z, u.w};   // (b is a bf16)
    unsigned m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t y;
      if (equal) asm("set.ge.u32.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(w[e]), "r"(b2));
      else asm("set.gt.u32.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(w[e]), "r"(b2));
      m |= (y & 1u) << (2 * e) | (y >> 31) << (2 * e + 1);
    }
    return m;
  }
  __device__ static uint4 edge(const __nv_bfloat16* x, int i, int lo, int hi) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = i + 2 * e;
      const uint32_t a = k >= lo && k < hi ? __bfloat16_as_ushort(x[k]) : 0xff80u;
      const uint32_t b = k + 1 >= lo && k + 1 < hi ? __bfloat16_as_ushort(x[k + 1]) : 0xff80u;
      w[e] = a | b << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <typename T>
constexpr int batch_of() { return kThreads * Vec<T>::VECS * Vec<T>::N; }

// Elements i, i + 1, ... of a row that starts `off` bytes behind a 16-byte boundary; those outside [lo, hi) count as
// -infinity. An unaligned vector is cut out of the two that it lies in.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* x, int off, int i, int lo, int hi) {
  constexpr int N = Vec<T>::N;
  if (i < lo || i + (off ? 2 * N : N) > hi) return Vec<T>::edge(x, i, lo, hi);
  const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(x + i) - off);
  const uint4 u = __ldcs(p);
  if (off == 0) return u;
  const uint4 v = __ldg(p + 1);          // (its neighbour's first: from L1)
  uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  if (off & 8)
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
  if (off & 4)
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  const int sh = (off & 2) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh), __funnelshift_r(w[2], w[3], sh),
                    __funnelshift_r(w[3], w[4], sh));
}

// A thread's vectors of the batch at base
template <typename T>
__device__ __forceinline__ void load_batch(uint4* u, const T* x, int off, int base, int lo, int hi) {
  constexpr int VEC = Vec<T>::N, NV = Vec<T>::VECS;
  const T* p = x + base + threadIdx.x * VEC;
  if (off == 0 && base + batch_of<T>() <= hi) {
#pragma unroll
    for (int v = 0; v < NV; ++v) u[v] = __ldcs(reinterpret_cast<const uint4*>(p + v * kThreads * VEC));
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) u[v] = load_vec(x, off, base + (v * kThreads + threadIdx.x) * VEC, lo, hi);
  }
}

// e^d as 2^(d log2 e). The constant's own rounding, 1.3e-8 of log2 e, makes a row's log sum some 1e-7 too small, all
// rows' nearly alike: what counts between beams is the difference.
constexpr float kLog2e = 1.44269502f;
__device__ __forceinline__ float exp_of(float d) { return fast_exp2(d * kLog2e); }

__device__ __forceinline__ float bound_of(uint32_t b) { return b ? unordered(b) : -INFINITY; }

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) beam_slice_kernel(const T* __restrict__ logits, const SelectArgs a) {
  using X = Vec<T>;
  using K = typename X::Key;
  constexpr int VEC = X::N, NV = X::VECS, kBatch = batch_of<T>();
  __shared__ K list[kKeep + kBatch];
  __shared__ K scratch[kThreads];
  __shared__ int count, left;
  __shared__ volatile int full;          // the last batch that filled the list beyond kKeep
  __shared__ float red[kThreads / 32];
  __shared__ uint32_t low[kLow];
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x / a.S, s = blockIdx.x - row * a.S;
  const float score = a.scores[row];
  if (!(fabsf(score) < INFINITY) || (a.finished && a.finished[row])) return;
  const T* x = logits + row * a.stride;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int off = (int)(reinterpret_cast<uintptr_t>(x) & 15);
  const int lo = s * a.slice, hi = min(a.V, lo + a.slice);   // this slice's tokens
  const int64_t o = (int64_t)row * a.S + s;
  if (tid == 0) count = full = 0;
  float bound_x = -INFINITY;             // logits that do not reach it are not among the N best
  float lm = -INFINITY;                  // the thread's maximum
  float m = -INFINITY, l = 0.f;          // the warp's maximum, and the thread's sum of e^(x - m)
  uint4 next[NV];                        // the next batch is on its way while one is worked on
  load_batch(next, x, off, lo, lo, hi);

  for (int base = lo, batch = 1; base < hi; base += kBatch, ++batch) {
    // vector v of a thread: tokens base + (v 256 + tid) VEC on
    uint4 cur[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) cur[v] = next[v];
    if (base + kBatch < hi) load_batch(next, x, off, base + kBatch, lo, hi);
    float vm[NV], bm = -INFINITY;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      vm[v] = X::max_of(cur[v]);
      bm = fmaxf(bm, vm[v]);
    }
    lm = fmaxf(lm, bm);
    const uint32_t wm = __reduce_max_sync(0xffffffffu, ordered(bm));
    if (wm > ordered(m)) {               // (the same in the warp; less and less often)
      const float to = unordered(wm);
      l = m == -INFINITY ? l : l * exp_of(m - to);
      m = to;
    }
    // the batch's sum in four chains; NaN and +infinity make it NaN
    const float c = m == -INFINITY ? 0.f : -m;
    const f32x2 c2 = pair(c, c), e2 = pair(kLog2e, kLog2e);
    f32x2 sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float f[VEC];
      X::unpack(cur[v], f);
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) {
        float y0, y1;
        unpair(mul2(add2(pair(f[2 * e], f[2 * e + 1]), c2), e2), y0, y1);
        sum[e & 1] = add2(sum[e & 1], pair(fast_exp2(y0), fast_exp2(y1)));
      }
    }
    float s0, s1;
    unpair(add2(sum[0], sum[1]), s0, s1);
    l += s0 + s1;

    // The bound, from the first batch and again whenever their number has doubled: N of the logits so far reach
    // it. The first batch's own are held against it with >=; a later one equal to it comes behind those N.
    const bool first = batch == 1, again = (batch & (batch - 1)) == 0;
    if (again) put_low(low, lm > -INFINITY ? ordered(lm) : 0u, a.N);
    if (first) {
      __syncthreads();
      bound_x = bound_of(read_low(low, a.N));
    }
    const bool equal = first && bound_x > -INFINITY;
    if (equal ? bm >= bound_x : bm > bound_x)
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (equal ? vm[v] >= bound_x : vm[v] > bound_x) {
          unsigned mask = X::reach(cur[v], bound_x, equal);
          int at = atomicAdd(&count, __popc(mask));
          for (; mask; mask &= mask - 1) {
            const int e = __ffs(mask) - 1;
            list[at++] = X::key(X::at(cur[v], e), base - lo + (v * kThreads + tid) * VEC + e);
          }
          if (at > kKeep) full = batch;
        }
    __syncthreads();
    // Whether this batch filled the list beyond kKeep, the same in all threads: a fast warp may be at the next batch
    // already when a late one looks here, and what it writes (to count, or the next batch's number to full) then says
    // "not this one" as well; where it is this one, no warp leaves before all have looked.
    if (full == batch) {
      const int kept = thin_out(list, count, a.N, scratch, low, &left);
      __syncthreads();
      // what is left are N at least, and they bound those to come
      const uint32_t mine = tid < kept ? ordered(X::logit(list[tid])) : ~0u;
      const uint32_t least = __reduce_min_sync(0xffffffffu, mine);
      if (lane == 0) low[warp] = least;
      if (tid == 0) count = kept;
      __syncthreads();
      bound_x = fmaxf(bound_x, bound_of(__reduce_min_sync(0xffffffffu, low[lane & 7])));
      __syncthreads();
    } else if (again && !first) {
      bound_x = fmaxf(bound_x, bound_of(read_low(low, a.N)));
      __syncthreads();                   // (before low or count is written again)
    }
  }

  // the slice's maximum and sum
  if (lane == 0) red[warp] = m;
  __syncthreads();
  float M = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) M = fmaxf(M, red[w]);
  const float c = M == -INFINITY ? 0.f : M;
  l = m == -INFINITY ? l : l * exp_of(m - c);
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  __syncthreads();
  if (lane == 0) red[warp] = l;
  __syncthreads();
  if (tid == 0) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += red[w];
    a.ml[o] = make_float2(c, t);
  }
  const int n = in_order(list, count, a.N, scratch, low, &left, [&](int rank, K k) {
    a.best[o * a.N + rank] = make_float2(X::logit(k), __uint_as_float((uint32_t)(lo + X::token(k))));
  });
  for (int i = n + tid; i < a.N; i += kThreads) a.best[o * a.N + i] = make_float2(0.f, __uint_as_float(kNone));
}

__global__ void __launch_bounds__(kThreads)
beam_pick_kernel(float* __restrict__ scores_out, int32_t* __restrict__ parents, int32_t* __restrict__ tokens,
                 uint8_t* __restrict__ finished_out, const SelectArgs a) {
  // total = (x - top) + base with base = score - log sum e^(x - top) (NaN: no candidates of logits);
  // a logit of any size then keeps its distance from the largest
  __shared__ double base[128], terms[kThreads];
  __shared__ float top[128];
  __shared__ float score[128];
  __shared__ uint8_t done[128];
  __shared__ Key list[kKeep + kThreads];
  __shared__ Key scratch[kThreads];
  __shared__ int count, left;
  __shared__ uint32_t low[kLow];
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = a.S * a.N, C = a.W * per;
  // a thread's first candidates are on their way while the sums are joined
  const float2* best = a.best + (int64_t)r * C;
  float2 early[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) early[k] = tid + k * kThreads < C ? best[tid + k * kThreads] : make_float2(0.f, 0.f);
  if (tid == 0) count = 0;
  // Each row's maximum (and whether it has one), a row a warp
  for (int w = warp; w < a.W; w += kThreads / 32) {
    const int row = r * a.W + w;
    const float2* ml = a.ml + (int64_t)row * a.S;
    const float2 v0 = lane < a.S ? ml[lane] : make_float2(0.f, 0.f);      // (not used where the row is not live)
    const float s = a.scores[row];
    const bool fin = a.finished && a.finished[row], live = fabsf(s) < INFINITY && !fin;
    float M = -INFINITY;
    if (live)
      for (int i = lane; i < a.S; i += 32) {
        const float2 v = i == lane ? v0 : ml[i];
        if (v.y > 0.f) M = fmaxf(M, v.x);
      }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) {
      base[w] = live ? 0.0 : (double)NAN;
      top[w] = M;
      score[w] = s;
      done[w] = fin;
      if (!(s < INFINITY)) flag(a.status, HYB_DEVERR_BAD_VALUE);
    }
  }
  __syncthreads();
  // and its sum in 64 bits, a (row, slice) a thread and then a row a thread: the 64-bit unit is narrow, so what
  // fits into one warp goes through it once (a row a warp: 4 us more for 8 beams).
  const int group = max(1, kThreads / a.S);      // rows at a time
  for (int w0 = 0; w0 < a.W; w0 += group) {
    const int rows = min(group, a.W - w0);
    double part = 0.0;
    for (int i = tid; i < rows * a.S; i += kThreads) {           // (more than one a thread only for one row)
      const int w = w0 + i / a.S;
      if (base[w] != base[w]) continue;
      const float2 v = a.ml[((int64_t)r * a.W + w) * a.S + i % a.S];
      if (v.y != 0.f) part += v.x == top[w] ? (double)v.y : (double)v.y * exp((double)v.x - (double)top[w]);
    }
    terms[tid] = part;
    __syncthreads();
    if (tid < rows && base[w0 + tid] == base[w0 + tid]) {
      const int n = min(a.S, kThreads);
      double l = 0.0;
      for (int i = 0; i < n; ++i) l += terms[tid * n + i];
      if (l != l) flag(a.status, HYB_DEVERR_BAD_VALUE);
      base[w0 + tid] = l > 0.0 ? (double)score[w0 + tid] - log(l) : (double)NAN;
    }
    __syncthreads();
  }
  // Candidates 256 at a time, behind those kept; more than kKeep of them are thinned to 256 at most. Whether there are
  // more is what the barrier says of the places that were given out: the counter itself may already be on its way to the
  // next 256 when a late warp looks at it.
  for (int i0 = 0; i0 < C + a.W; i0 += kThreads) {
    const int i = i0 + tid;
    int at = -1;                         // this thread's place
    if (i < C) {
      const int w = i / per;
      const float2 c = i0 == 0 ? early[0] : i0 == kThreads ? early[1] : best[i];
      if (base[w] == base[w] && __float_as_uint(c.y) != kNone) {
        Key y;
        y.hi = ordered(base[w] + ((double)c.x - (double)top[w]));
        y.lo = kNone - ((uint32_t)w * (uint32_t)a.V + __float_as_uint(c.y));
        list[at = atomicAdd(&count, 1)] = y;
      }
    } else if (i < C + a.W) {
      const int w = i - C;
      if (done[w] && fabsf(score[w]) < INFINITY) {
        Key y;
        y.hi = ordered((double)score[w]);
        y.lo = kNone - ((uint32_t)w * (uint32_t)a.V + (uint32_t)a.eos);
        list[at = atomicAdd(&count, 1)] = y;
      }
    }
    if (__syncthreads_or(at >= kKeep)) {
      const int kept = thin_out(list, count, a.N, scratch, low, &left);
      __syncthreads();
      if (tid == 0) count = kept;
      __syncthreads();
    }
  }
  const int n = in_order(list, count, a.N, scratch, low, &left, [&](int rank, Key k) {
    const int64_t o = (int64_t)r * a.N + rank;
    const uint32_t at = kNone - k.lo;
    const int w = (int)(at / (uint32_t)a.V), v = (int)(at % (uint32_t)a.V);
    scores_out[o] = (float)unordered(k.hi);
    parents[o] = w;
    tokens[o] = v;
    if (finished_out) finished_out[o] = done[w] || v == a.eos;
  });
  for (int i = n + tid; i < a.N; i += kThreads) {
    const int64_t o = (int64_t)r * a.N + i;
    scores_out[o] = -INFINITY;
    parents[o] = tokens[o] = -1;
    if (finished_out) finished_out[o] = 0;
  }
}

struct SelectPlan {
  int S, slice;
  size_t ws_bytes;
};
SelectPlan plan_select(int R, const hyb_beam_dims_t* d) {
  SelectPlan p;
  const int batch = d->dtype == HYB_BF16 ? batch_of<__nv_bfloat16>() : batch_of<float>();
  const int64_t batches = (d->vocab + batch - 1) / batch;
  const int64_t rows = (int64_t)R * d->num_beams, slots = (int64_t)num_sms() * 4;
  const int64_t nb = std::max<int64_t>(1, std::min<int64_t>(kSpan / batch, batches * rows / slots));
  p.S = (int)((batches + nb - 1) / nb);
  p.slice = (int)((batches + p.S - 1) / p.S) * batch;
  p.ws_bytes = (size_t)rows * p.S * (1 + d->num_out) * 8;
  return p;
}

bool al(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

hyb_status_t check_beam_dims(int R, const hyb_beam_dims_t* d) {
  if (!d || R < 0 || d->num_beams <= 0 || d->num_out <= 0 || d->vocab <= 0) return HYB_ERR_INVALID_ARG;
  if (d->dtype != HYB_BF16 && d->dtype != HYB_F32) return HYB_ERR_INVALID_ARG;
  if (d->eos_token < -1 || d->eos_token >= d->vocab) return HYB_ERR_INVALID_ARG;
  if (d->row_stride != 0 && d->row_stride < d->vocab) return HYB_ERR_INVALID_ARG;
  const int64_t all = (int64_t)d->num_beams * d->vocab;
  if (d->num_out > all) return HYB_ERR_INVALID_ARG;
  if (d->num_beams > 128 || d->num_out > 128 || d->vocab > (1 << 30) || all > INT32_MAX || d->row_stride > ((int64_t)1 << 40) ||
      (int64_t)R * d->num_beams > (1 << 20))
    return HYB_ERR_UNSUPPORTED;
  return HYB_OK;
}

}  // namespace
}  // namespace hyb

using namespace hyb;

extern "C" {

size_t hyb_beam_select_workspace_size(int32_t R, const hyb_beam_dims_t* d) {
  if (R <= 0 || check_beam_dims(R, d) != HYB_OK) return 0;
  return plan_select(R, d).ws_bytes;
}

hyb_status_t hyb_beam_select(float* scores_out, int32_t* parents, int32_t* tokens,
                             uint8_t* finished_out, const void* logits, const float* scores,
                             const uint8_t* finished, int32_t R, const hyb_beam_dims_t* d,
                             void* workspace, size_t ws_bytes, void* stream) {
  const hyb_status_t st = check_beam_dims(R, d);
  if (st != HYB_OK) return st;
  if (finished && d->eos_token < 0) return HYB_ERR_INVALID_ARG;
  if (R == 0) return HYB_OK;
  if (!scores_out || !parents || !tokens || !logits || !scores || !workspace) return HYB_ERR_INVALID_ARG;
  if (!al(scores_out, 4) || !al(parents, 4) || !al(tokens, 4) || !al(scores, 4) || !al(logits, 16) ||
      !al(workspace, 16))
    return HYB_ERR_INVALID_ARG;
  if (d->num_out != d->num_beams && (scores_out == scores || (finished && finished_out == finished)))
    return HYB_ERR_INVALID_ARG;
  const SelectPlan p = plan_select(R, d);
  if (ws_bytes < p.ws_bytes) return HYB_ERR_INVALID_ARG;
  const int64_t ctas = (int64_t)R * d->num_beams * p.S;
  if (ctas > INT32_MAX) return HYB_ERR_UNSUPPORTED;
  unsigned* sw = status_word();
  if (!sw) return HYB_ERR_CUDA;
  SelectArgs a;
  a.scores = scores;
  a.finished = finished;
  a.R = R;
  a.W = d->num_beams;
  a.N = d->num_out;
  a.V = d->vocab;
  a.S = p.S;
  a.slice = p.slice;
  a.stride = d->row_stride ? d->row_stride : d->vocab;
  a.eos = d->eos_token;
  a.ml = static_cast<float2*>(workspace);
  a.best = a.ml + (size_t)R * a.W * a.S;
  a.status = sw;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = d->dtype == HYB_BF16
                      ? launch_pdl(beam_slice_kernel<__nv_bfloat16>, dim3((unsigned)ctas), dim3(kThreads), 0, s,
                                   (const __nv_bfloat16*)logits, a)
                      : launch_pdl(beam_slice_kernel<float>, dim3((unsigned)ctas), dim3(kThreads), 0, s,
                                   (const float*)logits, a);
  count_launch();
  if (e != cudaSuccess) return cuda_status(e);
  e = launch_pdl(beam_pick_kernel, dim3(R), dim3(kThreads), 0, s, scores_out, parents, tokens, finished_out, a);
  count_launch();
  return cuda_status(e);
}

}  // extern "C"
