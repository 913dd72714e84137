// A Full layer's q, k and v rows from the projection to attention in one pass: RMS norm of each
// q and k head, rotation to the token's position, q to its own rows, k and v into the paged cache.
//
// Bound by the bytes: every row is read once and written once, 2 (Hq + 2 Hk) D elements a token.
// A warp takes one token and a share of its head rows. D / 8 lanes cover a row, 8 elements a lane,
// as two groups of 4 that hold both elements of each pair: 4 at x[e] and 4 at x[e + rot/2] in the
// half layout, so that neither layout needs a shuffle to rotate; the part behind rot_dim is cut
// in two the same way. The token's rot_dim / 2 cosines and sines are computed once per warp, by
// all lanes, and kept in registers for all of its rows; the loads of kU rounds of rows are in
// flight together.
//
// Angles. p f loses its fraction in fp32 once p f passes some thousand turns, so the
// frequency is kept in turns, f / 2 pi = hi + lo (two fp32, from one fp64 product per warp), and
// p hi is split into its rounded product and that product's exact error: the whole turns drop
// out without loss, and sincospi gets the fraction to about 2^-24 of a turn, for p <= 2^24.
#include <cuda_bf16.h>

#include <cmath>

#include "hyb_internal.cuh"

namespace hyb {
namespace {

constexpr int kWarps = 8;                  // warps per CTA
constexpr int kU = 4;                      // rounds of rows in flight
constexpr int kMaxPos = 1 << 24;           // positions are exact in fp32

// Four elements: the raw bits as loaded, their values, and the way back.
template <typename T>
struct Four;
template <>
struct Four<__nv_bfloat16> {
  using Raw = uint2;
  __device__ static void get(const Raw& r, float* x) {
    x[0] = bf16_lo(r.x); x[1] = bf16_hi(r.x); x[2] = bf16_lo(r.y); x[3] = bf16_hi(r.y);
  }
  __device__ static Raw pack(const float* x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};
template <>
struct Four<float> {
  using Raw = float4;
  __device__ static void get(const Raw& r, float* x) { x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w; }
  __device__ static Raw pack(const float* x) { return make_float4(x[0], x[1], x[2], x[3]); }
};

template <typename T>
struct RopeArgs {
  T *q_out, *k_out, *kc, *vc;
  const T *q, *k, *v;
  const int32_t* positions;
  const int64_t* slot;
  const float *inv_freq, *qw, *kw;
  int64_t qs, ks, vs;                      // elements between tokens
  int64_t n_slots;
  int T_, Hq, Hk, bs, rot, parts, rounds;  // parts: warps per token; rounds: row rounds of a part
  float eps, w_off, m;
  unsigned* status;
};

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kWarps * 32)
norm_rope_kernel(const __grid_constant__ RopeArgs<T> a) {
  using F = Four<T>;
  using Raw = typename F::Raw;
  constexpr int LPR = D / 8;               // lanes per row
  constexpr int RPR = 32 / LPR;            // rows per round
  constexpr int NF = (D / 2 + 31) / 32;    // frequencies per lane
  __shared__ float2 cs_sh[kWarps][D / 2];

  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = lane % LPR, rr = lane / LPR;
  float2* cs = cs_sh[warp];
  // this lane's two groups of 4 elements, and where the group's pairs find their angle
  const int nrot = a.rot / 8;              // lanes of a row with turning elements
  const bool turns = c < nrot;
  const int e0 = INTER ? 8 * c : turns ? 4 * c : a.rot + 4 * (c - nrot);
  const int e1 = INTER ? e0 + 4 : e0 + (turns ? a.rot / 2 : (D - a.rot) / 2);
  float wq[8], wk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int at = (e < 4 ? e0 : e1 - 4) + e;
    wq[e] = a.qw ? a.qw[at] + a.w_off : 1.f;
    wk[e] = a.kw ? a.kw[at] + a.w_off : 1.f;
  }
  float fhi[NF], flo[NF];                  // frequencies in turns per position
#pragma unroll
  for (int n = 0; n < NF; ++n) {
    const int i = lane + 32 * n;
    const double f = i < a.rot / 2 ? (double)a.inv_freq[i] * 0.15915494309189533577 : 0.0;
    fhi[n] = (float)f;
    flo[n] = (float)(f - (double)fhi[n]);
  }
  const int rows = a.Hq + 2 * a.Hk;        // a token's rows: q, k, v
  const int64_t items = (int64_t)a.T_ * a.parts;
  for (int64_t it = (int64_t)blockIdx.x * kWarps + warp; it < items; it += (int64_t)gridDim.x * kWarps) {
    const int t = (int)(it / a.parts), part = (int)(it - (int64_t)t * a.parts);
    const int p = a.positions[t];
    if (p < 0) continue;
    if (p > kMaxPos) {
      if (lane == 0) flag(a.status, HYB_DEVERR_BAD_LENGTH);
      continue;
    }
    int64_t slot = a.slot ? a.slot[t] : -1;
    if (slot >= a.n_slots) {
      if (lane == 0) flag(a.status, HYB_DEVERR_BAD_SLOT);
      slot = -1;
    }
    const int64_t blk = slot >= 0 ? slot / a.bs : 0, off = slot - blk * a.bs;
    const int row_end = min(rows, (part + 1) * a.rounds * RPR);
    float2 ang[4];                         // (cos, sin) of this lane's pairs
    bool first = true;
    for (int row0 = part * a.rounds * RPR; row0 < row_end; row0 += kU * RPR) {
      Raw raw[kU][2];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int row = row0 + u * RPR + rr;
        if (row >= row_end) continue;
        const T* src = row < a.Hq ? a.q + t * a.qs + (int64_t)row * D
                       : row < a.Hq + a.Hk ? a.k + t * a.ks + (int64_t)(row - a.Hq) * D
                                           : a.v + t * a.vs + (int64_t)(row - a.Hq - a.Hk) * D;
        if (row >= a.Hq + a.Hk && slot < 0) continue;        // v goes nowhere
        raw[u][0] = *reinterpret_cast<const Raw*>(src + e0);
        raw[u][1] = *reinterpret_cast<const Raw*>(src + e1);
      }
      if (first) {                         // the token's angles, while the first rows arrive
        first = false;
        const float pf = (float)p;
        __syncwarp();
#pragma unroll
        for (int n = 0; n < NF; ++n) {
          const float x = pf * fhi[n];
          const float r = (x - rintf(x)) + (fmaf(pf, fhi[n], -x) + pf * flo[n]);
          float sn, cn;
          sincospif(2.f * r, &sn, &cn);
          if (lane + 32 * n < a.rot / 2) cs[lane + 32 * n] = make_float2(a.m * cn, a.m * sn);
        }
        __syncwarp();
        if (turns) {
#pragma unroll
          for (int e = 0; e < 4; ++e) ang[e] = cs[4 * c + e];
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int row = row0 + u * RPR + rr;
        float x[8], ss = 0.f;
        const bool is_q = row < a.Hq, is_v = row >= a.Hq + a.Hk;
        if (row < row_end && !is_v) {
          F::get(raw[u][0], x);
          F::get(raw[u][1], x + 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
        }
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (row >= row_end) continue;
        if (is_v) {
          if (slot >= 0) {
            T* dst = a.vc + ((blk * a.Hk + (row - a.Hq - a.Hk)) * a.bs + off) * D;
            *reinterpret_cast<Raw*>(dst + e0) = raw[u][0];
            *reinterpret_cast<Raw*>(dst + e1) = raw[u][1];
          }
          continue;
        }
        if (is_q ? a.qw != nullptr : a.kw != nullptr) {
          const float inv = 1.f / sqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= inv * (is_q ? wq[e] : wk[e]);
        }
        if (turns) {
          if (INTER) {                     // pairs (0, 1), (2, 3), ...
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float u0 = x[2 * e], u1 = x[2 * e + 1];
              x[2 * e] = u0 * ang[e].x - u1 * ang[e].y;
              x[2 * e + 1] = u1 * ang[e].x + u0 * ang[e].y;
            }
          } else {                         // pairs (0, 4), (1, 5), ...: the two groups
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float u0 = x[e], u1 = x[e + 4];
              x[e] = u0 * ang[e].x - u1 * ang[e].y;
              x[e + 4] = u1 * ang[e].x + u0 * ang[e].y;
            }
          }
        }
        const Raw y0 = F::pack(x), y1 = F::pack(x + 4);
        if (is_q) {
          T* dst = a.q_out + ((int64_t)t * a.Hq + row) * D;
          *reinterpret_cast<Raw*>(dst + e0) = y0;
          *reinterpret_cast<Raw*>(dst + e1) = y1;
        } else {
          const int h = row - a.Hq;
          if (a.k_out) {
            T* dst = a.k_out + ((int64_t)t * a.Hk + h) * D;
            *reinterpret_cast<Raw*>(dst + e0) = y0;
            *reinterpret_cast<Raw*>(dst + e1) = y1;
          }
          if (slot >= 0) {
            T* dst = a.kc + ((blk * a.Hk + h) * a.bs + off) * D;
            *reinterpret_cast<Raw*>(dst + e0) = y0;
            *reinterpret_cast<Raw*>(dst + e1) = y1;
          }
        }
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_typed(RopeArgs<T> a, bool inter, cudaStream_t s) {
  constexpr int RPR = 32 / (D / 8);
  const int total = (a.Hq + 2 * a.Hk + RPR - 1) / RPR;     // rounds of rows per token
  // A warp's share of a token: the whole token (its angles computed once) when there are
  // tokens enough to fill the GPU's warps, down to kU rounds when there are few.
  const int64_t warps = (int64_t)num_sms() * 4 * kWarps;
  const int64_t want = std::max<int64_t>(1, warps / std::max(1, a.T_));
  a.rounds = std::max(kU, (int)((total + want - 1) / want));
  a.rounds = (a.rounds + kU - 1) / kU * kU;
  a.parts = (total + a.rounds - 1) / a.rounds;
  const int64_t items = (int64_t)a.T_ * a.parts;
  const int64_t blocks = std::min<int64_t>((items + kWarps - 1) / kWarps, (int64_t)num_sms() * 8);
  const cudaError_t e = launch_pdl(inter ? norm_rope_kernel<T, D, true> : norm_rope_kernel<T, D, false>,
                                   dim3((unsigned)blocks), dim3(kWarps * 32), 0, s, a);
  count_launch();
  return e;
}

template <typename T>
cudaError_t launch(void* q_out, void* k_out, const void* q, const void* k, const void* v,
                   const int32_t* positions, const int64_t* slot, const float* inv_freq,
                   const float* qw, const float* kw, int T_, void* kc, void* vc,
                   const hyb_rope_dims_t* r, const hyb_attn_dims_t* d, unsigned* status,
                   cudaStream_t s) {
  const int Hq = r->num_q_heads, Hk = d->num_heads, D = d->head_dim;
  RopeArgs<T> a;
  a.q_out = (T*)q_out; a.k_out = (T*)k_out; a.kc = (T*)kc; a.vc = (T*)vc;
  a.q = (const T*)q; a.k = (const T*)k; a.v = (const T*)v;
  a.positions = positions; a.slot = slot; a.inv_freq = inv_freq; a.qw = qw; a.kw = kw;
  a.qs = r->q_stride ? r->q_stride : (int64_t)Hq * D;
  a.ks = r->k_stride ? r->k_stride : (int64_t)Hk * D;
  a.vs = r->v_stride ? r->v_stride : (int64_t)Hk * D;
  a.n_slots = (int64_t)d->num_blocks * d->block_size;
  a.T_ = T_; a.Hq = Hq; a.Hk = Hk; a.bs = d->block_size; a.rot = r->rot_dim;
  a.eps = r->eps; a.w_off = r->weight_offset; a.m = r->attn_factor;
  a.status = status;
  switch (D) {
    case 16: return launch_typed<T, 16>(a, r->interleaved != 0, s);
    case 32: return launch_typed<T, 32>(a, r->interleaved != 0, s);
    case 64: return launch_typed<T, 64>(a, r->interleaved != 0, s);
    case 128: return launch_typed<T, 128>(a, r->interleaved != 0, s);
    case 256: return launch_typed<T, 256>(a, r->interleaved != 0, s);
  }
  return cudaErrorInvalidValue;
}

bool al(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace hyb

using namespace hyb;

extern "C" hyb_status_t hyb_qk_norm_rope_append(void* q_out, void* k_out, const void* q,
                                                const void* k, const void* v,
                                                const int32_t* positions,
                                                const int64_t* slot_mapping, const float* inv_freq,
                                                const float* q_weight, const float* k_weight,
                                                int32_t T, void* k_cache, void* v_cache,
                                                const hyb_rope_dims_t* r, const hyb_attn_dims_t* d,
                                                void* stream) {
  const hyb_status_t st = check_dims(d);
  if (st != HYB_OK) return st;
  if (!r || T < 0) return HYB_ERR_INVALID_ARG;
  const int D = d->head_dim;
  if (D != 16 && D != 32 && D != 64 && D != 128 && D != 256) return HYB_ERR_UNSUPPORTED;
  if (r->num_q_heads < 0 || r->num_q_heads > 65535 || d->num_heads > 65535) return HYB_ERR_INVALID_ARG;
  if (r->rot_dim < 0 || r->rot_dim > D) return HYB_ERR_INVALID_ARG;
  if (r->rot_dim % 8 != 0) return HYB_ERR_UNSUPPORTED;     // a lane's pairs are all turned or none
  if (!std::isfinite(r->eps) || !(r->eps > 0.f) || !std::isfinite(r->weight_offset) ||
      !std::isfinite(r->attn_factor))
    return HYB_ERR_INVALID_ARG;
  const int64_t unit = d->dtype == HYB_BF16 ? 8 : 4;       // 16 bytes
  const int64_t given[3] = {r->q_stride, r->k_stride, r->v_stride};
  const int64_t packed[3] = {(int64_t)r->num_q_heads * D, (int64_t)d->num_heads * D,
                             (int64_t)d->num_heads * D};
  for (int i = 0; i < 3; ++i)
    if (given[i] != 0 && (given[i] < packed[i] || given[i] % unit != 0 || given[i] > ((int64_t)1 << 32)))
      return HYB_ERR_INVALID_ARG;
  if (T == 0) return HYB_OK;
  const bool append = k_cache != nullptr;
  if (!k || !positions || (r->rot_dim > 0 && !inv_freq)) return HYB_ERR_INVALID_ARG;
  if ((r->num_q_heads > 0) != (q_out != nullptr) || (r->num_q_heads > 0 && !q)) return HYB_ERR_INVALID_ARG;
  if (append != (v_cache != nullptr) || append != (slot_mapping != nullptr) || (append && !v))
    return HYB_ERR_INVALID_ARG;
  if (!append && !k_out) return HYB_ERR_INVALID_ARG;       // k would go nowhere
  if (append && k_cache == v_cache) return HYB_ERR_INVALID_ARG;
  const void* const rows[] = {q_out, k_out, q, k, v, k_cache, v_cache};
  for (const void* p : rows)
    if (!al(p, 16)) return HYB_ERR_INVALID_ARG;
  if (!al(positions, 4) || !al(slot_mapping, 8) || !al(inv_freq, 4) || !al(q_weight, 4) ||
      !al(k_weight, 4))
    return HYB_ERR_INVALID_ARG;
  // in place only where each row comes back to its own place
  if ((q_out && q_out == q && r->q_stride != 0 && r->q_stride != packed[0]) ||
      (k_out && k_out == k && r->k_stride != 0 && r->k_stride != packed[1]))
    return HYB_ERR_INVALID_ARG;
  unsigned* sw = status_word();
  if (!sw) return HYB_ERR_CUDA;
  const cudaStream_t s = (cudaStream_t)stream;
  return cuda_status(d->dtype == HYB_BF16
                         ? launch<__nv_bfloat16>(q_out, k_out, q, k, v, positions, slot_mapping,
                                                 inv_freq, q_weight, k_weight, T, k_cache, v_cache, r,
                                                 d, sw, s)
                         : launch<float>(q_out, k_out, q, k, v, positions, slot_mapping, inv_freq,
                                         q_weight, k_weight, T, k_cache, v_cache, r, d, sw, s));
}
