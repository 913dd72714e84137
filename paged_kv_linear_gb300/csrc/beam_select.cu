// Beam selection (hyb_beam_select): for each request the best continuations over its beams and
// the vocabulary. First kernel: slices of the live rows, each leaves its maximum, its sum of
// exponentials and its best logits. Second: one CTA a request joins the sums and picks among what the
// slices left.
#include <cuda_bf16.h>

#include <cmath>

#include "hyb_internal.cuh"

namespace hyb {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kNone = 0xffffffffu;

// What the first kernel leaves of (row, slice): (max, sum of e^(x - max)), then N (logit, token).
struct SelectArgs {
  const float* scores;
  const uint8_t* finished;
  int R, W, N, V, S, slice;              // slices of a row, elements of a slice
  int64_t stride;
  int eos;
  float2* ml;                            // [R W][S]
  float2* best;                          // [R W][S][N]: logit, token as bits
  unsigned* status;
};

__device__ __forceinline__ float logit(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float logit(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }

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
struct Key {                             // of a total and its position w V + v
  uint64_t hi;
  uint32_t lo;
  __device__ __forceinline__ bool operator>(const Key& o) const { return hi != o.hi ? hi > o.hi : lo > o.lo; }
};

__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) k = max(k, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)k, o));
  return k;
}
__device__ __forceinline__ Key warp_max(Key k) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    Key y;
    y.hi = __shfl_xor_sync(0xffffffffu, (unsigned long long)k.hi, o);
    y.lo = __shfl_xor_sync(0xffffffffu, k.lo, o);
    if (y > k) k = y;
  }
  return k;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_slice_kernel(const T* __restrict__ logits, const SelectArgs a) {
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x / a.S, s = blockIdx.x - row * a.S;
  const float score = a.scores[row];
  if (!(fabsf(score) < INFINITY) || (a.finished && a.finished[row])) return;
  const T* x = logits + row * a.stride;
  const int i0 = s * a.slice, i1 = min(a.V, i0 + a.slice);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ float red[8];
  __shared__ uint64_t redk[8];
  float m = -INFINITY;
  for (int i = i0 + tid; i < i1; i += kThreads) m = fmaxf(m, logit(x, i));
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = red[0];
  for (int w = 1; w < 8; ++w) m = fmaxf(m, red[w]);
  const float mm = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int i = i0 + tid; i < i1; i += kThreads) l += expf(logit(x, i) - mm);   // NaN, infinity: NaN
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  __syncthreads();
  if (lane == 0) red[warp] = l;
  __syncthreads();
  const int64_t o = (int64_t)row * a.S + s;
  if (tid == 0) {
    float t = 0.f;
    for (int w = 0; w < 8; ++w) t += red[w];
    a.ml[o] = make_float2(mm, t);
  }
  uint64_t last = ~0ull;
  for (int n = 0; n < a.N; ++n) {
    uint64_t k = 0;
    for (int i = i0 + tid; i < i1; i += kThreads) {
      const float v = logit(x, i);
      const uint64_t y = (uint64_t)ordered(v) << 32 | (kNone - (uint32_t)i);
      if (v > -INFINITY && y < last) k = max(k, y);
    }
    k = warp_max(k);
    __syncthreads();
    if (lane == 0) redk[warp] = k;
    __syncthreads();
    for (int w = 0; w < 8; ++w) k = max(k, redk[w]);
    if (tid == 0)
      a.best[o * a.N + n] = make_float2(unordered((uint32_t)(k >> 32)), __uint_as_float(k ? kNone - (uint32_t)k : kNone));
    if (!k) {
      for (int r = n + 1 + tid; r < a.N; r += kThreads) a.best[o * a.N + r] = make_float2(0.f, __uint_as_float(kNone));
      break;
    }
    last = k;
  }
}

__global__ void __launch_bounds__(kThreads)
beam_pick_kernel(float* __restrict__ scores_out, int32_t* __restrict__ parents, int32_t* __restrict__ tokens,
                 uint8_t* __restrict__ finished_out, const SelectArgs a) {
  // total = (x - top) + base with base = score - log sum e^(x - top) (NaN: no candidates of logits);
  // a logit of any size then keeps its distance from the largest
  __shared__ double base[128];
  __shared__ float top[128];
  __shared__ float score[128];
  __shared__ uint8_t done[128];
  __shared__ Key redk[8];
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int w = warp; w < a.W; w += 8) {
    const int row = r * a.W + w;
    const float s = a.scores[row];
    const bool fin = a.finished && a.finished[row];
    double b = NAN;
    float M = -INFINITY;
    if (fabsf(s) < INFINITY && !fin) {
      for (int i = lane; i < a.S; i += 32) {
        const float2 v = a.ml[(int64_t)row * a.S + i];
        if (v.y > 0.f) M = fmaxf(M, v.x);
      }
      for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      double l = 0.0;
      for (int i = lane; i < a.S; i += 32) {
        const float2 v = a.ml[(int64_t)row * a.S + i];
        if (v.y != 0.f) l += (double)v.y * exp((double)v.x - (double)M);
      }
      for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (l > 0.0) b = (double)s - log(l);
      else if (l != l && lane == 0) flag(a.status, HYB_DEVERR_BAD_VALUE);
    } else if (!(s < INFINITY) && lane == 0) {
      flag(a.status, HYB_DEVERR_BAD_VALUE);
    }
    if (lane == 0) {
      base[w] = b;
      top[w] = M;
      score[w] = s;
      done[w] = fin;
    }
  }
  __syncthreads();
  const int per = a.S * a.N, C = a.W * per;
  Key last;
  last.hi = ~0ull;
  last.lo = ~0u;
  for (int n = 0; n < a.N; ++n) {
    Key k;
    k.hi = 0;
    k.lo = 0;
    auto offer = [&](double total, int w, uint32_t v) {
      Key y;
      y.hi = ordered(total);
      y.lo = kNone - ((uint32_t)w * (uint32_t)a.V + v);
      if (last > y && y > k) k = y;
    };
    for (int i = tid; i < C; i += kThreads) {
      const int w = i / per;
      const float2 c = a.best[(int64_t)r * C + i];
      if (base[w] == base[w] && __float_as_uint(c.y) != kNone) offer(base[w] + ((double)c.x - (double)top[w]), w, __float_as_uint(c.y));
    }
    for (int w = tid; w < a.W; w += kThreads)
      if (done[w] && fabsf(score[w]) < INFINITY) offer((double)score[w], w, (uint32_t)a.eos);
    k = warp_max(k);
    __syncthreads();
    if (lane == 0) redk[warp] = k;
    __syncthreads();
    for (int w = 0; w < 8; ++w)
      if (redk[w] > k) k = redk[w];
    last = k;
    if (tid == 0) {
      const int64_t o = (int64_t)r * a.N + n;
      const bool any = k.hi != 0;
      const uint32_t at = kNone - k.lo;
      const int w = any ? (int)(at / (uint32_t)a.V) : -1, v = any ? (int)(at % (uint32_t)a.V) : -1;
      scores_out[o] = any ? (float)unordered(k.hi) : -INFINITY;
      parents[o] = w;
      tokens[o] = v;
      if (finished_out) finished_out[o] = any && (done[w] || v == a.eos);
    }
  }
}

struct SelectPlan {
  int S, slice;
  size_t ws_bytes;
};
SelectPlan plan_select(int R, const hyb_beam_dims_t* d) {
  SelectPlan p;
  p.slice = 4096;
  p.S = (d->vocab + p.slice - 1) / p.slice;
  p.ws_bytes = (size_t)R * d->num_beams * p.S * (1 + d->num_out) * 8;
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
  if (d->num_beams > 128 || d->num_out > 128 || all > INT32_MAX || d->row_stride > ((int64_t)1 << 40) ||
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
