// A Full layer's q, k and v rows from the projection to attention in one pass: RMS norm of each
// q and k head, rotation to the token's position, q to its own rows, k and v into the paged cache.
//
// Bound by the bytes: every row is read once and written once, 2 (Hq + 2 Hk) D elements a token.
// A warp takes one token and a share of its head rows. D / 8 lanes cover a row, 8 elements a lane,
// as two groups of 4 that hold both elements of each pair: 4 at x[e] and 4 at x[e + rot/2] in the
// half layout, so that neither layout needs a shuffle to rotate; the part behind rot_dim is cut
// in two the same way. The token's rot_dim / 2 cosines and sines are computed once per warp, by
// all lanes; a lane folds those of its pairs and the weights into 16 factors, so that a row's
// element takes two products and the norm's one. The loads of kU rounds of rows are in flight
// together, and the next kU rounds' while these are worked on: 110 registers, two CTAs per SM.
//
// 65536 tokens of 32 + 2 x 8 heads of 128, bf16, from rows of a fused projection: 270 us, 6.0 TB/s, 0.88
// of the copy rate (issue slots 57 % busy; 422 us with one batch in flight, 305 with separate code for q
// and k). 64 tokens of 32 + 2 x 32 heads: 7.5 us a call, 4.1 on the GPU.
//
// Angles. p f loses its fraction in fp32 once p f passes some thousand turns, so the
// frequency is kept in turns, f / 2 pi = hi + lo (two fp32, from one fp64 product per warp), and
// p hi is split into its rounded product and that product's exact error: the whole turns drop
// out without loss, and sincospi gets the fraction to about 2^-24 of a turn, for p <= 2^24.
#include <cuda_bf16.h>

#include <cmath>

#include "tc.cuh"

namespace hyb {
namespace {

constexpr int kWarps = 8;                  // warps per CTA
constexpr int kU = 4;                      // rounds of rows in a batch; two batches in flight
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
  int T_, Hq, Hk, bs_log2, rot, parts, rounds;  // parts: warps per token; rounds: row rounds of a part
  float eps, w_off, m;
  unsigned* status;
};

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, 2)
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
  // this lane's two groups of 4 elements: 4 pairs (x[i], x[i + 4]), or (x[2i], x[2i + 1])
  const int nrot = a.rot / 8;              // lanes of a row with turning elements
  const bool turns = c < nrot;
  const int e0 = INTER ? 8 * c : turns ? 4 * c : a.rot + 4 * (c - nrot);
  const int e1 = INTER ? e0 + 4 : e0 + (turns ? a.rot / 2 : (D - a.rot) / 2);
  float fhi[NF], flo[NF];                  // frequencies in turns per position
#pragma unroll
  for (int n = 0; n < NF; ++n) {
    const int i = lane + 32 * n;
    const double f = i < a.rot / 2 ? (double)a.inv_freq[i] * 0.15915494309189533577 : 0.0;
    fhi[n] = (float)f;
    flo[n] = (float)(f - (double)fhi[n]);
  }
  // a token's rounds: those of q, of k, of v
  const int nq = (a.Hq + RPR - 1) / RPR, nk = (a.Hk + RPR - 1) / RPR;
  // items of one warp: (token, part) from here on in steps of the grid's warps
  const int step = gridDim.x * kWarps, step_t = step / a.parts, step_p = step - step_t * a.parts;
  const int it0 = blockIdx.x * kWarps + warp;
  int t_next = it0 / a.parts, part_next = it0 - t_next * a.parts;
  int p_next = t_next < a.T_ ? a.positions[t_next] : -1;
  int64_t slot_next = t_next < a.T_ && a.slot ? a.slot[t_next] : -1;
#pragma unroll 1
  while (t_next < a.T_) {
    const int64_t t = t_next;
    const int part = part_next, p = p_next;
    int64_t slot = slot_next;
    part_next += step_p;
    const bool over = part_next >= a.parts;
    part_next -= over ? a.parts : 0;
    t_next = a.T_ - t_next > step_t + over ? t_next + step_t + over : a.T_;
    if (t_next < a.T_) {
      p_next = a.positions[t_next];
      if (a.slot) slot_next = a.slot[t_next];
    }
    if (p < 0) continue;
    if (p > kMaxPos) {
      if (lane == 0) flag(a.status, HYB_DEVERR_BAD_LENGTH);
      continue;
    }
    if (slot >= a.n_slots) {
      if (lane == 0) flag(a.status, HYB_DEVERR_BAD_SLOT);
      slot = -1;
    }
    // where the token's first head lies in the caches, and from head to head
    const int64_t blk = slot >> a.bs_log2;   // (no slot: not used)
    const int64_t cache0 = (((blk * a.Hk) << a.bs_log2) + (slot - (blk << a.bs_log2))) * D;
    const int cache_h = D << a.bs_log2;
    const int begin = part * a.rounds, end = min(nq + 2 * nk, begin + a.rounds);

    // Batches of kU rounds of q's, then k's, then v's rows (section 0, 1, 2; 3: none left). The next
    // batch is on its way while one is worked on.
    int sec = -1, r = 0, r1 = 0;
    Raw next[kU][2];
    auto load_next = [&] {
      r += kU;
#pragma unroll 1
      while (r >= r1 && sec < 3) {
        ++sec;
        const int off = sec == 0 ? 0 : sec == 1 ? nq : nq + nk;
        r = max(begin - off, 0);
        r1 = sec == 3 || (sec == 2 && slot < 0) ? r : min(end - off, sec == 0 ? nq : nk);
      }
      if (sec == 3) return;
      const int heads = sec == 0 ? a.Hq : a.Hk, h0 = r * RPR + rr;
      const T* src = (sec == 0 ? a.q + t * a.qs : sec == 1 ? a.k + t * a.ks : a.v + t * a.vs) + h0 * D;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (h0 + u * RPR < min(heads, r1 * RPR)) {
          next[u][0] = *reinterpret_cast<const Raw*>(src + e0 + u * RPR * D);
          next[u][1] = *reinterpret_cast<const Raw*>(src + e1 + u * RPR * D);
        }
    };
    load_next();
    {                                      // the token's angles
      const float pf = (float)p;
      __syncwarp();
#pragma unroll
      for (int n = 0; n < NF; ++n) {
        const float x = pf * fhi[n];
        const float y = (x - rintf(x)) + (fmaf(pf, fhi[n], -x) + pf * flo[n]);
        float sn, cn;
        sincospif(2.f * y, &sn, &cn);
        if (lane + 32 * n < a.rot / 2) cs[lane + 32 * n] = make_float2(a.m * cn, a.m * sn);
      }
      __syncwarp();
    }
    // pair i: (u, v) -> (u c0 - v s1, v c1 + u s0), c and s times the weights of u (0) and v (1)
    f32x2 c0[2], s0[2], c1[2], s1[2];
    int have = -1;                         // the section that these are for
#pragma unroll 1
    while (sec < 3) {
      const int now = sec, h0 = r * RPR + rr, most = min(now == 0 ? a.Hq : a.Hk, r1 * RPR);
      Raw raw[kU][2];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        raw[u][0] = next[u][0];
        raw[u][1] = next[u][1];
      }
      load_next();
      const float* w = now == 0 ? a.qw : a.kw;
      if (now < 2 && have != now) {
        have = now;
        float x[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = turns ? cs[4 * c + i] : make_float2(1.f, 0.f);
          const int iu = INTER ? e0 + 2 * i : e0 + i, iv = INTER ? e0 + 2 * i + 1 : e1 + i;
          const float wu = w ? w[iu] + a.w_off : 1.f, wv = w ? w[iv] + a.w_off : 1.f;
          x[0][i] = wu * f.x; x[1][i] = wu * f.y; x[2][i] = wv * f.x; x[3][i] = -wv * f.y;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          c0[i] = pair(x[0][2 * i], x[0][2 * i + 1]);
          s0[i] = pair(x[1][2 * i], x[1][2 * i + 1]);
          c1[i] = pair(x[2][2 * i], x[2][2 * i + 1]);
          s1[i] = pair(x[3][2 * i], x[3][2 * i + 1]);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + u * RPR;
        const bool in = h < most;
        Raw y0 = raw[u][0], y1 = raw[u][1];
        if (now < 2) {
          float x[8];
          F::get(y0, x);
          F::get(y1, x + 4);
          f32x2 xu[2], xv[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            xu[i] = INTER ? pair(x[4 * i], x[4 * i + 2]) : pair(x[2 * i], x[2 * i + 1]);
            xv[i] = INTER ? pair(x[4 * i + 1], x[4 * i + 3]) : pair(x[4 + 2 * i], x[5 + 2 * i]);
          }
          float inv = 1.f;
          if (w) {
            float ss, s2;
            unpair(fma2(xv[1], xv[1], fma2(xv[0], xv[0], fma2(xu[1], xu[1], mul2(xu[0], xu[0])))), ss, s2);
            ss += s2;
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            inv = rsqrtf(ss * (1.f / D) + a.eps);
          }
          const f32x2 inv2 = pair(inv, inv);
          float y[8];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const f32x2 yu = mul2(inv2, fma2(xv[i], s1[i], mul2(xu[i], c0[i])));
            const f32x2 yv = mul2(inv2, fma2(xu[i], s0[i], mul2(xv[i], c1[i])));
            if (INTER) {
              unpair(yu, y[4 * i], y[4 * i + 2]);
              unpair(yv, y[4 * i + 1], y[4 * i + 3]);
            } else {
              unpair(yu, y[2 * i], y[2 * i + 1]);
              unpair(yv, y[4 + 2 * i], y[5 + 2 * i]);
            }
          }
          y0 = F::pack(y);
          y1 = F::pack(y + 4);
        }
        if (!in) continue;
        T* d0 = now == 0 ? a.q_out + (t * a.Hq + h) * D
                : now == 1 && a.k_out ? a.k_out + (t * a.Hk + h) * D : nullptr;
        if (d0) {
          *reinterpret_cast<Raw*>(d0 + e0) = y0;
          *reinterpret_cast<Raw*>(d0 + e1) = y1;
        }
        if (now > 0 && slot >= 0) {
          T* d1 = (now == 1 ? a.kc : a.vc) + cache0 + (int64_t)h * cache_h;
          *reinterpret_cast<Raw*>(d1 + e0) = y0;
          *reinterpret_cast<Raw*>(d1 + e1) = y1;
        }
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_typed(RopeArgs<T> a, bool inter, cudaStream_t s) {
  constexpr int RPR = 32 / (D / 8);
  const int total = (a.Hq + RPR - 1) / RPR + 2 * ((a.Hk + RPR - 1) / RPR);   // rounds of rows per token
  // A warp's share of a token: the whole token (its angles computed once) when there are
  // tokens enough to fill the GPU's warps, down to kU rounds when there are few. 64 tokens of 96
  // head rows take 7.7 us in shares, 16.2 whole; 65536 of 48 rows 428 us in shares of kU, 270 whole.
  const int64_t warps = (int64_t)num_sms() * 4 * kWarps;
  const int64_t want = std::max<int64_t>(1, warps / std::max(1, a.T_));
  a.rounds = std::max(kU, (int)((total + want - 1) / want));
  a.rounds = (a.rounds + kU - 1) / kU * kU;
  a.parts = (total + a.rounds - 1) / a.rounds;
  const int64_t items = (int64_t)a.T_ * a.parts;
  const int64_t blocks = std::min<int64_t>((items + kWarps - 1) / kWarps, (int64_t)num_sms() * 2);
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
  a.T_ = T_; a.Hq = Hq; a.Hk = Hk; a.bs_log2 = log2_int(d->block_size); a.rot = r->rot_dim;
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
