// The gated delta rule: its one-token step, its prefill on the CUDA cores, and the entry points
// of both calls (the tensor-core prefill is in delta_tc.cu).
//
// Per token and value head, with S the fp32 state (row i: key dim, column j: value dim):
//     S <- e^g S,   u = beta (v - S^T k),   S <- S + k u^T,   out = scale S^T q.
// Both kernels read the state once for k and q together: with S the state before the token,
//     u = beta (v - e^g S^T k),   out = scale (e^g S^T q + (q.k) u),
// so the two sums over i share their pass and their reduction, and the new state needs no second
// one. q and k brought to unit length are q / |q| and k / |k|: factors of the sums, never
// rounded rows. Where the decay is slow, the state decays as S + (e^g - 1) S: e^g rounded to
// fp32 would be off by the same 2^-25 at every token of a constant gate, and the state by the sum of
// that over the tokens it keeps. (Where it is fast, that form would lose what is left of S.)
#include <cuda_bf16.h>

#include <cmath>
#include <type_traits>

#include "tc.cuh"

namespace hyb {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
// 1 / |x| from the sum of squares; 1 where the rows are taken as they are
__device__ __forceinline__ float inv_len(float ss, float eps) {
  return eps > 0.f ? 1.f / sqrtf(ss + eps) : 1.f;
}

// ------------------------------------------------------------------ one token
// Bound by HBM: each state is read and written once (2 x 64 KiB at D = 128), against 7 flops an
// element. A CTA owns 32 columns of one state, 8 threads x float4 to a row and 32 rows a pass; all
// loads of a thread (PASSES x 16 bytes) are in flight before the first use, and columns do not
// depend on one another, so no CTA waits for another. k and q go through shared memory, and so
// do the sums over the 128 rows after a shuffle over the 4 rows of a warp: registers stay few (48, two of
// them spilled at D = 128, which costs less than a CTA), and five CTAs per SM keep the loads of some while others store (three, at 69 registers: 55.8 us where
// it takes 46.4; the exact form of slow decays brought it to 47.5; of that form, six CTAs take 48.1
// and four 52.0). States pass the caches as streams: plain stores 54.7, plain loads 48.2.
// bf16, D = 128: 64 requests x 32 heads 47.5 us, 5.7 TB/s, 0.84 of the copy rate; 256 x 32 heads 193 us,
// 0.82 (178 in passes over one pool, of which a part stays in L2); one request 6.7 us a call, 2.7 on
// the GPU.
template <int D>
struct DeltaStep {
  static constexpr int COLS = D < 32 ? D : 32;
  static constexpr int TPR = COLS / 4;                      // threads per row (float4 each)
  static constexpr int THREADS = D * TPR < 256 ? D * TPR : 256;
  static constexpr int RPP = THREADS / TPR;                 // rows per pass
  static constexpr int PASSES = D / RPP;
  static constexpr int NW = THREADS / 32;
  static constexpr int CTAS = PASSES > 4 ? 3 : 5;           // per SM
  static_assert(PASSES * RPP == D && NW * 32 == THREADS, "shape");
};

template <typename T, int D>
__global__ void __launch_bounds__(DeltaStep<D>::THREADS, DeltaStep<D>::CTAS)
delta_step_kernel(T* __restrict__ out, const T* __restrict__ q, const T* __restrict__ k,
                  const T* __restrict__ v, const float* __restrict__ g,
                  const float* __restrict__ beta, float* __restrict__ pool, int NS,
                  const int32_t* __restrict__ slots, int Hv, int rep, int64_t qs, int64_t ks,
                  int64_t vs, float scale, float eps, unsigned* status) {
  using Sh = DeltaStep<D>;
  constexpr int COLS = Sh::COLS, TPR = Sh::TPR, RPP = Sh::RPP, PASSES = Sh::PASSES, NW = Sh::NW;
  __shared__ __align__(16) float sh_k[D], sh_q[D];
  __shared__ __align__(16) float red_k[NW][COLS], red_q[NW][COLS], sums[4];

  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z;
  const int slot = slots[b];
  if (slot < 0 || slot >= NS) {
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) flag(status, HYB_DEVERR_BAD_STATE);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tc = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  const int col = blockIdx.x * COLS + tc * 4;
  float* S = pool + ((int64_t)slot * Hv + h) * D * D + rg * D + col;

  float4 st[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) st[p] = __ldcs(reinterpret_cast<const float4*>(S + p * RPP * D));
  pdl_trigger();                           // the next kernel may launch (it waits for this one)
  for (int i = threadIdx.x; i < D; i += Sh::THREADS) {
    sh_k[i] = to_f(k[b * ks + (int64_t)(h / rep) * D + i]);
    sh_q[i] = to_f(q[b * qs + (int64_t)(h / rep) * D + i]);
  }
  const T* vr = v + b * vs + (int64_t)h * D + col;
  const float gate = g[(int64_t)b * Hv + h], be = beta[(int64_t)b * Hv + h];
  const float eg = expf(gate), em1 = expm1f(gate);
  float vv[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) vv[e] = to_f(vr[e]);
  __syncthreads();

  float a[8] = {};                         // S^T k and S^T q, 4 columns each
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const float s[4] = {st[p].x, st[p].y, st[p].z, st[p].w};
    const float ki = sh_k[rg + p * RPP], qi = sh_q[rg + p * RPP];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = fmaf(ki, s[e], a[e]);
      a[4 + e] = fmaf(qi, s[e], a[4 + e]);
    }
  }
#pragma unroll
  for (int o = TPR; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] += __shfl_xor_sync(0xffffffffu, a[e], o);
  if (lane < TPR) {
    *reinterpret_cast<float4*>(&red_k[warp][lane * 4]) = make_float4(a[0], a[1], a[2], a[3]);
    *reinterpret_cast<float4*>(&red_q[warp][lane * 4]) = make_float4(a[4], a[5], a[6], a[7]);
  }
  if (warp == NW - 1) {                    // k.k, q.q, q.k
    float kk = 0.f, qq = 0.f, qk = 0.f;
    for (int i = lane; i < D; i += 32) {
      kk = fmaf(sh_k[i], sh_k[i], kk);
      qq = fmaf(sh_q[i], sh_q[i], qq);
      qk = fmaf(sh_q[i], sh_k[i], qk);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      kk += __shfl_xor_sync(0xffffffffu, kk, o);
      qq += __shfl_xor_sync(0xffffffffu, qq, o);
      qk += __shfl_xor_sync(0xffffffffu, qk, o);
    }
    if (lane == 0) *reinterpret_cast<float4*>(sums) = make_float4(kk, qq, qk, 0.f);
  }
  __syncthreads();
  const float rk = inv_len(sums[0], eps);
  float u[4] = {};                         // S^T k, then the correction, times rk for the state's k
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const float4 x = *reinterpret_cast<const float4*>(&red_k[w][tc * 4]);
    u[0] += x.x; u[1] += x.y; u[2] += x.z; u[3] += x.w;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = be * (vv[e] - eg * (rk * u[e])) * rk;
  const bool slow = em1 >= -0.5f;
  const float fade = slow ? em1 : eg;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const float ki = sh_k[rg + p * RPP];
    float4 x = st[p];
    x.x = fmaf(ki, u[0], fmaf(fade, x.x, slow ? x.x : 0.f));
    x.y = fmaf(ki, u[1], fmaf(fade, x.y, slow ? x.y : 0.f));
    x.z = fmaf(ki, u[2], fmaf(fade, x.z, slow ? x.z : 0.f));
    x.w = fmaf(ki, u[3], fmaf(fade, x.w, slow ? x.w : 0.f));
    __stcs(reinterpret_cast<float4*>(S + p * RPP * D), x);
  }
  if (rg == 0) {
    const float rq = scale * inv_len(sums[1], eps), qk = sums[2];
    float o[4] = {};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(&red_q[w][tc * 4]);
      o[0] += y.x; o[1] += y.y; o[2] += y.z; o[3] += y.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      put(out + ((int64_t)b * Hv + h) * D + col + e, rq * fmaf(qk, u[e], eg * o[e]));
  }
}

// ------------------------------------------------------------------ prefill on the CUDA cores
// The recurrence itself, for the shapes without a tensor-core kernel (fp32 rows, other head
// sizes): fp32 throughout. Columns of a state do not depend on one another, so a CTA carries 32
// columns of one (request, head) in registers for the whole prompt, and D / 32 CTAs share a
// state. A column's D rows lie with RG lanes of one warp (see scan_pick), so a token takes two sums over
// registers and a few shuffles, and no barrier. Tokens come in batches of kTB, whose rows and scalars
// are staged in shared memory; the next batch's rows are on their way to registers meanwhile. Bound
// by the latency of that chain when there are few chains (0.18 us a token at D = 64; 24 chains of up to
// 700 rows: 127 us, with 32 rows a lane 176, and 461 without the next batch's rows on their way), by
// fp32 arithmetic (4 D^2 fma per token and head, in packed pairs) when there are many (2048 chains of
// 512 tokens at D = 64: 0.97 ms).
template <int D, int RG_>
struct DeltaScan {
  static constexpr int COLS = D < 32 ? D : 32;              // columns per CTA
  static constexpr int RG = RG_;                            // lanes per column
  static constexpr int R = D / RG;                          // rows per lane
  static constexpr int NT = COLS * RG;                      // threads
  static constexpr int CW = 32 / RG;                        // columns per warp
  static constexpr int TB = 16;                             // tokens per batch
  static constexpr int LQ = TB * D / 4 / NT;                // 4-element loads of q (and of k) per thread
  static constexpr int LV = (TB * COLS / 4 + NT - 1) / NT;  // of v (D = 256: half of the threads)
  static constexpr int LT = NT / TB < 8 ? NT / TB : 8;      // lanes that work out a token's lengths
  static_assert(R % 4 == 0 && NT % 32 == 0 && LQ * 4 * NT == TB * D, "shape");
};

// Whether the recurrence takes a call that the tensor-core kernel could take. That one needs a chunk's
// time (14 us, and 4.5 us a chunk and a state for every SM's further ones) for a few rows too; the
// recurrence 4 us and some 0.25 to 0.35 us a row of the longest request as long as its CTAs, four a chain,
// find SMs of their own, and 0.04 us a chain and 0.003 us a row and head beyond that. So it takes
//   * up to 8 rows a request, in any batch;
//   * few rows in all, T x heads <= 1536, none of them in a long request;
//   * more chains than SMs whose requests have few rows in the mean (decode steps beside a prompt), as
//     long as the longest is over before the others' states have passed.
// Recurrence / tensor cores in us, heads of 128:
//     equal requests, chains 32: 32 rows 11.2 / 14.1, 40 rows 14.3 / 14.2    192: 8 rows 14.4 / 22.2
//                            64: 24 rows 12.7 / 14.0, 32 rows 14.8 / 14.2    512: 8 rows 32 / 36, 12 rows 38 / 36
//                           128: 12 rows 13.3 / 13.9, 16 rows 15.2 / 14.0   2048: 8 rows 122 / 128, 12 rows 144 / 128
//     one request of m rows beside others of one row, 32 heads:
//          3 others: m = 16 11.6 / 14.1, 32 17.6 / 14.3      31 others: m = 32 51 / 57, 64 67 / 59
//          7 others: m = 16 16.4 / 22.6, 32 22.3 / 22.9     255 others: m = 64 359 / 489, 128 388 / 489
inline bool short_call(int max_len, int T, int B, int heads) {
  const int64_t chains = (int64_t)B * heads;
  return max_len <= 8 || (max_len <= 32 && T * (int64_t)heads <= 1536) ||
         (chains > num_sms() && T <= 10 * (int64_t)B && max_len <= 16 + chains / 16);
}

struct Quad {
  float x[4];
};
__device__ __forceinline__ Quad load4(const float* p) {
  const float4 u = *reinterpret_cast<const float4*>(p);
  return {u.x, u.y, u.z, u.w};
}
__device__ __forceinline__ Quad load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)};
}

template <typename T, int D, int RG_>
__global__ void __launch_bounds__(DeltaScan<D, RG_>::NT)
delta_scan_kernel(T* __restrict__ out, const T* __restrict__ q, const T* __restrict__ k,
                  const T* __restrict__ v, const float* __restrict__ g,
                  const float* __restrict__ beta, const int32_t* __restrict__ cu,
                  float* __restrict__ pool, int NS, const int32_t* __restrict__ slots,
                  const uint8_t* __restrict__ reset, int rows_total, int max_len, int Hv, int rep,
                  int64_t qs, int64_t ks, int64_t vs, float scale, float eps, unsigned* status) {
  using Sh = DeltaScan<D, RG_>;
  constexpr int COLS = Sh::COLS, RG = Sh::RG, R = Sh::R, CW = Sh::CW, NT = Sh::NT, TB = Sh::TB;
  constexpr int LQ = Sh::LQ, LV = Sh::LV, LT = Sh::LT;
  constexpr int LD = D + 4;                // rows of different tokens start at different banks
  __shared__ __align__(16) float sq[TB][LD], sk[TB][LD];    // unit (or given) rows; q times scale
  __shared__ __align__(16) float sv[TB][COLS];
  __shared__ __align__(16) float4 s_f[TB];                  // e^g, beta, q.k, e^g - 1

  const int c0 = blockIdx.x * COLS, h = blockIdx.y, b = blockIdx.z;
  const bool first = blockIdx.x == 0 && h == 0 && threadIdx.x == 0;
  const int slot = slots[b], t0 = cu[b], t1 = cu[b + 1];
  if (slot < 0 || slot >= NS) {
    if (first) flag(status, HYB_DEVERR_BAD_STATE);
    return;
  }
  if (!delta_rows_ok(t0, t1, rows_total, max_len)) {
    if (first) flag(status, HYB_DEVERR_BAD_LENGTH);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = lane / CW, c = warp * CW + lane % CW;      // row group, column of this CTA
  float* S = pool + ((int64_t)slot * Hv + h) * D * D + c0 + c;
  const bool zero = reset && reset[b];
  if (t0 == t1 && !zero) return;
  q += (int64_t)(h / rep) * D;
  k += (int64_t)(h / rep) * D;
  v += (int64_t)h * D + c0;

  // rows of the batch at tb, zeros behind the last; token and scalars of this thread
  Quad nq[LQ], nk[LQ], nv[LV];
  float ng = 0.f, nb = 0.f;
  const int lt = threadIdx.x / LT;         // this thread's token in the lengths (if < TB)
  auto fetch = [&](int tb) {
    const Quad none = {};
#pragma unroll
    for (int e = 0; e < LQ; ++e) {
      const int i = (threadIdx.x + e * NT) * 4, t = tb + i / D;
      nq[e] = t < t1 ? load4(q + t * qs + i % D) : none;
      nk[e] = t < t1 ? load4(k + t * ks + i % D) : none;
    }
#pragma unroll
    for (int e = 0; e < LV; ++e) {
      const int i = (threadIdx.x + e * NT) * 4, t = tb + i / COLS;
      nv[e] = i < TB * COLS && t < t1 ? load4(v + t * vs + i % COLS) : none;
    }
    const bool in = lt < TB && tb + lt < t1;
    ng = in ? g[(int64_t)(tb + lt) * Hv + h] : 0.f;
    nb = in ? beta[(int64_t)(tb + lt) * Hv + h] : 0.f;
  };
  fetch(t0);
  // rows 4 (m RG + rg) + e: the RG lanes' 16-byte reads of a staged row lie side by side
  f32x2 s[R / 2];
#pragma unroll
  for (int m = 0; m < R; m += 2) {
    const int i = 4 * ((m / 4) * RG + rg) + m % 4;
    s[m / 2] = zero ? pair(0.f, 0.f) : pair(S[(int64_t)i * D], S[(int64_t)(i + 1) * D]);
  }
#pragma unroll 1
  for (int tb = t0; tb < t1; tb += TB) {
    __syncthreads();                       // the last batch is used up
#pragma unroll
    for (int e = 0; e < LQ; ++e) {
      const int i = (threadIdx.x + e * NT) * 4;
      *reinterpret_cast<float4*>(&sq[i / D][i % D]) = make_float4(nq[e].x[0], nq[e].x[1], nq[e].x[2], nq[e].x[3]);
      *reinterpret_cast<float4*>(&sk[i / D][i % D]) = make_float4(nk[e].x[0], nk[e].x[1], nk[e].x[2], nk[e].x[3]);
    }
#pragma unroll
    for (int e = 0; e < LV; ++e) {
      const int i = (threadIdx.x + e * NT) * 4;
      if (i < TB * COLS)
        *reinterpret_cast<float4*>(&sv[0][0] + i) = make_float4(nv[e].x[0], nv[e].x[1], nv[e].x[2], nv[e].x[3]);
    }
    const float fg = ng, fb = nb;
    __syncthreads();
    bool slow = true;
    if (lt < TB) {                         // lengths and q.k: LT lanes a token
      const int l = threadIdx.x % LT;
      float kk = 0.f, qq = 0.f, qk = 0.f;
#pragma unroll 4
      for (int i = l; i < D; i += LT) {
        const float x = sk[lt][i], y = sq[lt][i];
        kk = fmaf(x, x, kk);
        qq = fmaf(y, y, qq);
        qk = fmaf(x, y, qk);
      }
      const unsigned mask = __activemask();
#pragma unroll
      for (int o = LT / 2; o >= 1; o >>= 1) {
        kk += __shfl_xor_sync(mask, kk, o);
        qq += __shfl_xor_sync(mask, qq, o);
        qk += __shfl_xor_sync(mask, qk, o);
      }
      const float rk = inv_len(kk, eps), rq = scale * inv_len(qq, eps);
#pragma unroll 4
      for (int i = l; i < D; i += LT) {
        sk[lt][i] *= rk;
        sq[lt][i] *= rq;
      }
      const float em1 = expm1f(fg);
      slow = em1 >= -0.5f;
      if (l == 0) s_f[lt] = make_float4(expf(fg), fb, qk * rk * rq, em1);
    }
    slow = __syncthreads_and(slow);        // of the whole batch: within a faster one less than half is kept
    if (tb + TB < t1) fetch(tb + TB);
    const int nt = min(TB, t1 - tb);
    T* o_row = out + ((int64_t)tb * Hv + h) * D + c0 + c;
    auto tokens = [&](auto is_slow) {
#pragma unroll 2
    for (int t = 0; t < nt; ++t) {
      const float4 f = s_f[t];
      const float vt = sv[t][c];
      f32x2 x[R / 2], pk[2], pq[2];        // two sums of pairs each: a shorter chain
#pragma unroll
      for (int e = 0; e < 2; ++e) pk[e] = pq[e] = pair(0.f, 0.f);
#pragma unroll
      for (int m = 0; m < R / 2; m += 2) {
        const int i = 4 * ((m / 2) * RG + rg);
        const float4 y = *reinterpret_cast<const float4*>(&sq[t][i]);
        const float4 z = *reinterpret_cast<const float4*>(&sk[t][i]);
        x[m] = pair(z.x, z.y);
        x[m + 1] = pair(z.z, z.w);
        pk[0] = fma2(x[m], s[m], pk[0]);
        pk[1] = fma2(x[m + 1], s[m + 1], pk[1]);
        pq[0] = fma2(pair(y.x, y.y), s[m], pq[0]);
        pq[1] = fma2(pair(y.z, y.w), s[m + 1], pq[1]);
      }
      float dk, dk1, dq, dq1;
      unpair(add2(pk[0], pk[1]), dk, dk1);
      unpair(add2(pq[0], pq[1]), dq, dq1);
      dk += dk1;
      dq += dq1;
#pragma unroll
      for (int o = CW; o < 32; o <<= 1) {
        dk += __shfl_xor_sync(0xffffffffu, dk, o);
        dq += __shfl_xor_sync(0xffffffffu, dq, o);
      }
      const float u = f.y * (vt - f.x * dk);
      if (rg == 0) put(o_row + (int64_t)t * Hv * D, fmaf(f.z, u, f.x * dq));
      const float fade = is_slow ? f.w : f.x;
      const f32x2 u2 = pair(u, u), f2 = pair(fade, fade);
#pragma unroll
      for (int m = 0; m < R / 2; ++m)
        s[m] = fma2(x[m], u2, is_slow ? fma2(s[m], f2, s[m]) : mul2(s[m], f2));
    }
    };
    if (slow) tokens(std::true_type());
    else tokens(std::false_type());
  }
#pragma unroll
  for (int m = 0; m < R; m += 2) {
    const int i = 4 * ((m / 4) * RG + rg) + m % 4;
    float a, b;
    unpair(s[m / 2], a, b);
    S[(int64_t)i * D] = a;
    S[(int64_t)(i + 1) * D] = b;
  }
}

// ------------------------------------------------------------------ launches
struct Strides {
  int64_t q, k, v;
};
Strides strides_of(const hyb_delta_dims_t* d) {
  const int64_t qk = (int64_t)d->num_qk_heads * d->head_dim, vv = (int64_t)d->num_v_heads * d->head_dim;
  return {d->q_stride ? d->q_stride : qk, d->k_stride ? d->k_stride : qk,
          d->v_stride ? d->v_stride : vv};
}

template <typename T, int D>
cudaError_t step_typed(void* out, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, float* pool, int NS, const int32_t* slots, int B,
                       const hyb_delta_dims_t* d, unsigned* status, cudaStream_t s) {
  using Sh = DeltaStep<D>;
  const Strides st = strides_of(d);
  const dim3 grid(D / Sh::COLS, d->num_v_heads, B);
  const cudaError_t e = launch_pdl(
      delta_step_kernel<T, D>, grid, dim3(Sh::THREADS), 0, s, (T*)out, (const T*)q, (const T*)k,
      (const T*)v, g, beta, pool, NS, slots, d->num_v_heads, d->num_v_heads / d->num_qk_heads, st.q,
      st.k, st.v, d->scale, d->qk_norm_eps, status);
  count_launch();
  return e;
}

template <typename T, int D, int RG>
cudaError_t scan_typed(void* out, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, const int32_t* cu, float* pool, int NS,
                       const int32_t* slots, const uint8_t* reset, int B, int rows, int max_len,
                       const hyb_delta_dims_t* d, unsigned* status, cudaStream_t s) {
  using Sh = DeltaScan<D, RG>;
  const Strides st = strides_of(d);
  const dim3 grid(D / Sh::COLS, d->num_v_heads, B);
  delta_scan_kernel<T, D, RG><<<grid, Sh::NT, 0, s>>>(
      (T*)out, (const T*)q, (const T*)k, (const T*)v, g, beta, cu, pool, NS, slots, reset, rows,
      max_len, d->num_v_heads, d->num_v_heads / d->num_qk_heads, st.q, st.k, st.v, d->scale,
      d->qk_norm_eps, status);
  count_launch();
  return cudaGetLastError();
}

// Lanes to a column: 32 of its rows each, or 16 for small heads while a token's latency counts, not the
// arithmetic: as long as two CTAs per SM hold all chains. 16 rows / 32 rows, 256 tokens, us: D = 64, fp32:
// 72 chains 49 / 66, 152 chains 62 / 68, 304 chains 94 / 93, 1024 chains 310 / 275; D = 32: 72 chains
// 49 / 60, 304 chains 49 / 62, 1024 chains 88 / 81. At D = 128 the third round of shuffles takes what the
// shorter sums give (24 chains 72 / 70); 8 rows at D = 64: 62.
template <typename T, int D, typename... Args>
cudaError_t scan_pick(int64_t chains, Args... args) {
  constexpr int RG = D < 32 ? 2 : D / 32;
  if constexpr (D == 32 || D == 64) {
    if (chains * (D / 32) <= 2 * num_sms()) return scan_typed<T, D, 2 * RG>(args...);
  }
  return scan_typed<T, D, RG>(args...);
}

#define HYB_DELTA_EACH(CALL)                                                            \
  switch (d->head_dim) {                                                                \
    case 16: return d->dtype == HYB_BF16 ? CALL(__nv_bfloat16, 16) : CALL(float, 16);    \
    case 32: return d->dtype == HYB_BF16 ? CALL(__nv_bfloat16, 32) : CALL(float, 32);    \
    case 64: return d->dtype == HYB_BF16 ? CALL(__nv_bfloat16, 64) : CALL(float, 64);    \
    case 128: return d->dtype == HYB_BF16 ? CALL(__nv_bfloat16, 128) : CALL(float, 128); \
    case 256: return d->dtype == HYB_BF16 ? CALL(__nv_bfloat16, 256) : CALL(float, 256); \
  }                                                                                     \
  return cudaErrorInvalidValue;

cudaError_t launch_step(void* out, const void* q, const void* k, const void* v, const float* g,
                        const float* beta, float* pool, int NS, const int32_t* slots, int B,
                        const hyb_delta_dims_t* d, unsigned* status, cudaStream_t s) {
#define HYB_CALL(T, DD) step_typed<T, DD>(out, q, k, v, g, beta, pool, NS, slots, B, d, status, s)
  HYB_DELTA_EACH(HYB_CALL)
#undef HYB_CALL
}

cudaError_t launch_scan(void* out, const void* q, const void* k, const void* v, const float* g,
                        const float* beta, const int32_t* cu, float* pool, int NS,
                        const int32_t* slots, const uint8_t* reset, int B, int rows, int max_len,
                        const hyb_delta_dims_t* d, unsigned* status, cudaStream_t s) {
#define HYB_CALL(T, DD)                                                                             \
  scan_pick<T, DD>((int64_t)B * d->num_v_heads, out, q, k, v, g, beta, cu, pool, NS, slots, reset, B, rows, max_len, d, status, s)
  HYB_DELTA_EACH(HYB_CALL)
#undef HYB_CALL
}
#undef HYB_DELTA_EACH

// ------------------------------------------------------------------ argument checks
bool al(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

hyb_status_t check_delta_dims(const hyb_delta_dims_t* d) {
  if (!d || d->num_qk_heads <= 0 || d->num_v_heads <= 0 || d->head_dim <= 0) return HYB_ERR_INVALID_ARG;
  if (d->num_v_heads % d->num_qk_heads != 0) return HYB_ERR_INVALID_ARG;
  if (d->dtype != HYB_BF16 && d->dtype != HYB_F32) return HYB_ERR_INVALID_ARG;
  if (!std::isfinite(d->scale) || !(d->qk_norm_eps >= 0.f) || !std::isfinite(d->qk_norm_eps))
    return HYB_ERR_INVALID_ARG;
  const int D = d->head_dim;
  if (d->num_v_heads > 65535 || (D != 16 && D != 32 && D != 64 && D != 128 && D != 256))
    return HYB_ERR_UNSUPPORTED;
  const int64_t qk = (int64_t)d->num_qk_heads * D, vv = (int64_t)d->num_v_heads * D;
  const int64_t unit = d->dtype == HYB_BF16 ? 8 : 4;       // 16 bytes
  const int64_t given[3] = {d->q_stride, d->k_stride, d->v_stride}, least[3] = {qk, qk, vv};
  for (int i = 0; i < 3; ++i)
    if (given[i] != 0 && (given[i] < least[i] || given[i] % unit != 0 || given[i] > ((int64_t)1 << 32)))
      return HYB_ERR_INVALID_ARG;
  return HYB_OK;
}

// rows: whether the call has any (their pointers may be null otherwise)
hyb_status_t check_delta(const void* out, const void* q, const void* k, const void* v,
                         const float* g, const float* beta, const float* pool, int NS,
                         const int32_t* slots, int B, bool rows, const hyb_delta_dims_t* d) {
  const hyb_status_t st = check_delta_dims(d);
  if (st != HYB_OK) return st;
  if (B < 0 || NS <= 0) return HYB_ERR_INVALID_ARG;
  if (B > 65535 || (int64_t)B * d->num_v_heads > INT32_MAX) return HYB_ERR_UNSUPPORTED;   // grid.z; chains
  if ((int64_t)NS * d->num_v_heads * d->head_dim * d->head_dim > ((int64_t)1 << 40))
    return HYB_ERR_UNSUPPORTED;
  if (B == 0) return HYB_OK;
  if (!pool || !slots || (rows && (!out || !q || !k || !v || !g || !beta))) return HYB_ERR_INVALID_ARG;
  if (!al(out, 16) || !al(q, 16) || !al(k, 16) || !al(v, 16) || !al(pool, 16) || !al(g, 4) ||
      !al(beta, 4) || !al(slots, 4))
    return HYB_ERR_INVALID_ARG;
  return HYB_OK;
}

}  // namespace
}  // namespace hyb

using namespace hyb;

extern "C" {

hyb_status_t hyb_gated_delta_step(void* out, const void* q, const void* k, const void* v,
                                  const float* g, const float* beta, float* state_pool,
                                  int32_t num_state_slots, const int32_t* state_slots, int32_t B,
                                  const hyb_delta_dims_t* d, void* stream) {
  const hyb_status_t st =
      check_delta(out, q, k, v, g, beta, state_pool, num_state_slots, state_slots, B, true, d);
  if (st != HYB_OK || B == 0) return st;
  unsigned* sw = status_word();
  if (!sw) return HYB_ERR_CUDA;
  return cuda_status(launch_step(out, q, k, v, g, beta, state_pool, num_state_slots, state_slots, B,
                                 d, sw, (cudaStream_t)stream));
}

size_t hyb_gated_delta_chunked_prefill_workspace_size(int32_t B, int32_t T,
                                                      const hyb_delta_dims_t* d) {
  if (B <= 0 || T < 0 || check_delta_dims(d) != HYB_OK) return 0;
  return kLinPrefillWsBytes;
}

hyb_status_t hyb_gated_delta_chunked_prefill(void* out, const void* q, const void* k,
                                             const void* v, const float* g, const float* beta,
                                             const int32_t* cu_seqlens, float* state_pool,
                                             int32_t num_state_slots, const int32_t* state_slots,
                                             const uint8_t* reset, int32_t B, int32_t T,
                                             int32_t max_len, const hyb_delta_dims_t* d,
                                             void* workspace, size_t ws_bytes, void* stream) {
  const hyb_status_t st =
      check_delta(out, q, k, v, g, beta, state_pool, num_state_slots, state_slots, B, T > 0, d);
  if (st != HYB_OK) return st;
  if (T < 0 || max_len < 0 || max_len > T) return HYB_ERR_INVALID_ARG;
  if (T > INT32_MAX - 64) return HYB_ERR_UNSUPPORTED;      // rows are counted on by up to a chunk
  if (B == 0) return HYB_OK;
  if (!cu_seqlens || !al(cu_seqlens, 4)) return HYB_ERR_INVALID_ARG;
  if (!workspace || !al(workspace, 8) || ws_bytes < kLinPrefillWsBytes) return HYB_ERR_INVALID_ARG;
  unsigned* sw = status_word();
  if (!sw) return HYB_ERR_CUDA;
  if (delta_prefill_tc_supported(d) && !short_call(max_len, T, B, d->num_v_heads)) {
    const Strides x = strides_of(d);
    return cuda_status(launch_delta_prefill_tc(out, q, k, v, g, beta, cu_seqlens, state_pool,
                                               num_state_slots, state_slots, reset, B, T, max_len,
                                               d, x.q, x.k, x.v, workspace, sw,
                                               (cudaStream_t)stream));
  }
  return cuda_status(launch_scan(out, q, k, v, g, beta, cu_seqlens, state_pool, num_state_slots,
                                 state_slots, reset, B, T, max_len, d, sw, (cudaStream_t)stream));
}

}  // extern "C"
