// Chunked prefill of the gated delta rule on the tensor cores (tcgen05 + TMEM + TMA): bf16
// q/k/v, D = 128, fp32 state.
//
// Mathematics. Chunks of C = 64 rows; within one, G_t is the running sum of g, S the state at
// its start, k_t and q_t the (unit) rows. Eliminating the state between the rows of the chunk
// leaves one triangular system for the corrections x_t (the u_t of the recurrence):
//     A_ts = beta_t e^(G_t - G_s) k_t.k_s  (s < t),      (1 + A) X = beta (V - e^G K S)
//     O    = scale (e^G Q S + P X),   P_ts = e^(G_t - G_s) q_t.k_s  (s <= t)
//     S    <- e^(G_C) S + sum_t e^(G_C - G_t) k_t x_t^T
// (1 + A)^-1 = W depends on K, beta and g alone, so it is made ahead of the state's chain:
// by forward substitution, which stays exact where keys repeat (the entries of the powers of A do
// not). What remains on the chain is four steps: K S, W R, the state's sum, and the next
// state's operand; O hangs off its side.
//
// Precision. The state is fp32 and what reads or changes it is computed to fp32's accuracy on
// bf16 tensor cores: K and Q are bf16 as given (their lengths, decays, beta and scale go into
// fp32 factors of rows and columns, never into rounded operands), and S, W, the right-hand side R
// and the corrections are each cut into three bf16 terms, h + m + l, which hold an fp32 number
// without loss. K S and the state's sum then are exact products; of W R the terms beyond 2^-24 are
// left out (six of nine products). The outputs, rounded to bf16 in the end, take two terms of S, X
// and P (about 2^-16). With two terms throughout, states were off by some 3e-6 instead of 3e-7.
//
// Layout. Everything on the chain is kept transposed: TMEM lane j is the state's value column j, so
// each thread owns a column (half of its columns' range), nothing on the chain crosses threads, and
// the results (accumulators in TMEM) become the next product's A operand by the same thread
// writing them back as bf16 terms; shared memory holds only what TMA brings (K, Q, V) and W and P.
//   (k) D1K[j][t] = S^T K^T     A = S (TMEM, 3 terms),  B = K rows     24 MMAs 128 x 64 x 16
//   (q) D1Q[j][t] = S^T Q^T     A = S (TMEM, 2 terms),  B = Q rows     16
//   (0) [K; Q] K^T of the next chunk (128 x 64)                         8
//   (w) X^T       = R^T W^T     A = R (TMEM),  B = W rows (6 pairs)    24
//   (s) S^T      += X'^T K      A = X e^(G_C - G) (TMEM), B = K^T       12 MMAs 128 x 128 x 16
//   (o) D1Q       = X^T P^T     A = X (TMEM, 2 terms), B = P (3 pairs) 12
// The state's fp32 accumulator stays in TMEM; whoever reads a chunk's final state to cut it into
// terms writes it back times the next chunk's decay.
//
// Warps: 0-3 prepare a chunk (lengths, gates, W, P), one chunk ahead of 4-11, which carry the
// chain (two warps to 32 lanes, each half of the columns); 12-15 write outputs; 16 issues TMA
// loads (two stages), 17 the MMAs. Chains are shared out over the CTAs as in chain_split.cuh: the
// 256 chains of 8 requests x 32 heads would leave the second wave of 152 CTAs a third full.
#include <cuda_bf16.h>

#include "chain_split.cuh"
#include "tc.cuh"

namespace hyb {
namespace {

constexpr int kC = 64, kD = 128;
constexpr int kSubKQ = 128 * 128;              // [64 K rows; 64 Q rows][64 cols], SW128
constexpr int kStageKQ = 2 * kSubKQ;
constexpr int kSubV = 64 * 128;
constexpr int kStageV = 2 * kSubV;
constexpr int kTile64 = 64 * 128;              // [64][64] bf16
constexpr int kOffKQ = 0;
constexpr int kOffV = kOffKQ + 2 * kStageKQ;
constexpr int kOffW = kOffV + 2 * kStageV;     // [buffer][term]
constexpr int kOffP = kOffW + 2 * 3 * kTile64;
constexpr int kOffA = kOffP + 2 * 2 * kTile64; // the system, fp32, then its inverse
constexpr int kLdA = 68;                       // floats per row (16-byte rows, banks spread)
constexpr int kOffG = kOffA + kC * kLdA * 4;

struct Gates {                                 // factors of a chunk's rows
  float hi[kC], lo[kC];                        // G in units of log 2, as a sum of two
  float aR[kC], bt[kC], wX[kC], oq[kC];        // R = bt V - aR (K S); wX: X to the state; oq: Q S to O
  float cA[kC], rk[kC], pq[kC];                // beta / |k|, 1 / |k|, scale / |q|
  float dec, pad[3];                           // e^(G_C)
};
// What the warps need to know of a chunk. Warp 16 walks the CTA's runs and writes these, four
// chunks deep; n = 0 ends them.
struct Chunk {
  float* S;                                    // the chain's state in the pool
  int row, n, h, flags;                        // first row, rows, value head
  int pad[2];
};
constexpr int kFirst = 1, kLast = 2, kZero = 4, kTake = 8, kHand = 16;   // of a run; its state: zero
                                               // at first, taken over first, handed over at last
constexpr int kOffChunk = kOffG + 2 * (int)sizeof(Gates);
constexpr int kOffBar = kOffChunk + 4 * (int)sizeof(Chunk);

struct Bars {
  uint64_t full_kq[2], full_v[2], free_kq[2], free_v[2];
  uint64_t info[2], gates[2], w_ready[2], o_free[2];   // two: their readers may lag a chunk
  uint64_t d0_ready, d0_free, sa_ready, d1k_ready, d1q_ready, ra_ready, x_ready, xa_ready, s_ready;
  uint64_t q_read, o_ready, published, drain;
};
constexpr int kSmem = kOffBar + 512 + 1024;    // + slack for 1024-byte alignment
static_assert(sizeof(Bars) <= 512 && kOffG % 16 == 0 && kOffBar % 8 == 0 && kSmem <= 227 * 1024, "smem");

constexpr int kWarpMain = 4, kWarpOut = 12, kWarpFeed = 16, kWarpMma = 17;
constexpr int kThreads = 18 * 32;
constexpr uint32_t kTmemCols = 512;
// D0 | D1K | D1Q | S fp32 | operand terms of S. Once (k) and (q) have read the terms, R, X and X'
// take their places: R's h and m over S's l, R's l inside D1K (each thread over columns that only
// it reads); X over S's h; X' over S's m and R's h; X's two terms for (o) over D1K.
constexpr uint32_t kCol0 = 0, kCol1K = 64, kCol1Q = 128, kColS = 192, kColSA = 320;
constexpr uint32_t kColRh = kColSA + 128, kColRm = kColSA + 160, kColRl = kCol1K + 16;
constexpr uint32_t kColX = kColSA;
constexpr uint32_t kColXh = kColSA + 64, kColXm = kColSA + 96, kColXl = kColSA + 128;
constexpr uint32_t kColOh = kCol1K, kColOm = kCol1K + 32;

constexpr uint32_t kIdesc64 = idesc_bf16(128, 64, 0, 0);
constexpr uint32_t kIdescS = idesc_bf16(128, 128, 0, 1);   // B = K rows as K^T: N (key dim) major

constexpr float kGateMax = 1e4f;               // e^-g is 0 and e^g infinite in fp32 far below
constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.92596303e-8f;   // their sum is 1 / ln 2

// ------------------------------------------------------------------ runs
struct In {
  const int32_t *cu, *slots;
  const uint8_t* reset;
  float* pool;
  int NS, T, max_len, H;
};
// rows of request b, 0 where they are not within the call's
__device__ __forceinline__ int rows_of(const In& in, int b) {
  const int t0 = in.cu[b], t1 = in.cu[b + 1];
  return delta_rows_ok(t0, t1, in.T, in.max_len) ? t1 - t0 : 0;
}
__device__ __forceinline__ int chunks_of(const In& in, int b) { return (rows_of(in, b) + kC - 1) / kC; }

// A contiguous run of one chain's chunks, [c0, c1).
struct Seg {
  int h, t0, n, c0, c1;
  float* S;                  // the chain's state in the pool
  bool zero_start;           // c0 == 0 and the request is reset
  bool wait_handoff;         // c0 > 0: the state comes from the CTA that ran chunks [0, c0)
  bool publish;              // c1 < the chain's chunks: hand the state over at the end
};
__device__ __forceinline__ bool make_run(const In& in, int unit, int c0, int c1, Seg& s) {
  const int b = unit / in.H, n = rows_of(in, b), slot = in.slots[b];
  if (n == 0 || slot < 0 || slot >= in.NS) return false;
  const int nc = (n + kC - 1) / kC;
  s.h = unit - b * in.H;
  s.t0 = in.cu[b];
  s.n = n;
  s.c0 = c0;
  s.c1 = c1 < 0 ? nc : c1;
  s.S = in.pool + ((int64_t)slot * in.H + s.h) * kD * kD;
  s.zero_start = c0 == 0 && in.reset && in.reset[b];
  s.wait_handoff = c0 > 0;
  s.publish = s.c1 < nc;
  return true;
}
// This CTA's chunks one after another: the first chain's part, the whole chains, the last
// chain's part.
struct Walk {
  Seg sg;
  int ci;
  int stage, u;
};
__device__ __forceinline__ bool next_run(const In& in, const Plan& pl, Walk& w) {
  while (w.stage < 3) {
    bool ok = false;
    if (w.stage == 0) {
      w.stage = 1;
      w.u = pl.full_u0;
      ok = pl.head_u >= 0 && make_run(in, pl.head_u, 0, pl.head_end, w.sg);
    } else if (w.stage == 1) {
      if (w.u < pl.full_u1) ok = make_run(in, w.u++, 0, -1, w.sg);
      else w.stage = 2;
    } else {
      w.stage = 3;
      ok = pl.tail_u >= 0 && make_run(in, pl.tail_u, pl.tail_begin, -1, w.sg);
    }
    if (ok) {
      w.ci = w.sg.c0;
      return true;
    }
  }
  return false;
}
__device__ __forceinline__ bool first_chunk(const In& in, const Plan& pl, Walk& w) {
  w.stage = 0;
  return next_run(in, pl, w);
}
__device__ __forceinline__ bool next_chunk(const In& in, const Plan& pl, Walk& w) {
  return ++w.ci < w.sg.c1 || next_run(in, pl, w);
}

// ------------------------------------------------------------------ three-term splits
// x = h + m + l by cutting off 8 bits of significand at a time: each remainder is exact, the
// last has at most 8 bits left. Pairs are packed as the tensor core reads them.
__device__ __forceinline__ uint32_t pack_hi(float a, float b) {        // upper halves of a, b
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float cut(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
__device__ __forceinline__ void rest(float& a, float& b) {             // x - cut(x) for both
  unpair(fma2(pair(cut(a), cut(b)), pair(-1.f, -1.f), pair(a, b)), a, b);
}
__device__ __forceinline__ void split3(float a, float b, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = pack_hi(a, b);
  rest(a, b);
  m = pack_hi(a, b);
  rest(a, b);
  l = pack_hi(a, b);
}
// two terms, the second rounded: off by at most 2^-16
__device__ __forceinline__ void split2(float a, float b, uint32_t& h, uint32_t& m) {
  h = pack_hi(a, b);
  rest(a, b);
  m = pack_bf16(a, b);
}

// a gate in units of log 2 and steps of 2^-36 (a NaN is carried beside it)
__device__ __forceinline__ long long to_fixed(float g) {
  const float x = fminf(fmaxf(g, -kGateMax), kGateMax);
  const float h = x * kLog2eHi, l = fmaf(x, kLog2eHi, -h) + x * kLog2eLo;
  return __float2ll_rn(h * 0x1p36f) + __float2ll_rn(l * 0x1p36f);
}
__device__ __forceinline__ void from_fixed(long long x, bool nan, float& hi, float& lo) {
  const float h = __ll2float_rn(x);
  hi = nan ? __int_as_float(0x7fffffff) : h * 0x1p-36f;
  lo = __ll2float_rn(x - __float2ll_rn(h)) * 0x1p-36f;
}
// As mbar_wait, timed by the SM's own clock (some 2 s), which is cheaper to read.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > 4000000000ll) return false;
  return true;
}

__device__ __forceinline__ void bar_prep() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// the same, and whether ok holds for all of the preparing warps: they stop together
__device__ __forceinline__ bool bar_prep_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

// 16 values as operand terms: 8 columns at each of h, m and l
__device__ __forceinline__ void put_terms(uint32_t h_at, uint32_t m_at, uint32_t l_at, const float* v) {
  uint32_t h[8], m[8], l[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) split3(v[2 * e], v[2 * e + 1], h[e], m[e], l[e]);
  tmem_st8u(h_at, h);
  tmem_st8u(m_at, m);
  tmem_st8u(l_at, l);
}
// 16 values of this lane's state (key dims i0 ..): operand terms, and the accumulator times the
// coming chunk's decay
__device__ __forceinline__ void put_state(uint32_t tl, int i0, float* v, float dec) {
  put_terms(tl + kColSA + i0 / 2, tl + kColSA + 64 + i0 / 2, tl + kColSA + 128 + i0 / 2, v);
  const f32x2 d2 = pair(dec, dec);
#pragma unroll
  for (int e = 0; e < 16; e += 2) unpair(mul2(pair(v[e], v[e + 1]), d2), v[e], v[e + 1]);
  tmem_st16(tl + kColS + i0, v);
}

__global__ void __launch_bounds__(kThreads, 1)
delta_prefill_tc_kernel(const __grid_constant__ CUtensorMap tq,
                        const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, __nv_bfloat16* __restrict__ out,
                        const float* __restrict__ g, const float* __restrict__ beta, const __grid_constant__ In in,
                        int B, int rep, float scale, float eps,
                        unsigned long long* __restrict__ hs, int cut_chains, unsigned* status) {
  const int p = blockIdx.x, P = gridDim.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ Plan plan_sh;
  __shared__ uint32_t tmem_base;

  // prologue: invalid requests are reported; a reset request without rows gets a zero state
  for (int b = p; b < B; b += P) {
    const int slot = in.slots[b];
    const bool bad_rows = !delta_rows_ok(in.cu[b], in.cu[b + 1], in.T, in.max_len);
    if (slot < 0 || slot >= in.NS) {
      if (tid == 0) flag(status, HYB_DEVERR_BAD_STATE);
    } else if (bad_rows) {
      if (tid == 0) flag(status, HYB_DEVERR_BAD_LENGTH);
    } else if (in.cu[b + 1] == in.cu[b] && in.reset && in.reset[b]) {
      float4* S = reinterpret_cast<float4*>(in.pool + (int64_t)slot * in.H * kD * kD);
      for (int e = tid; e < in.H * kD * kD / 4; e += kThreads) S[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  if (warp == 0) {
    Plan pl{-1, 0, p, p + 1, -1, 0};      // chain p
    if (cut_chains) pl = make_plan([&](int b) { return chunks_of(in, b); }, B, in.H, P, p, lane);
    if (lane == 0) plan_sh = pl;
  }
  __syncthreads();
  {
    Walk any;
    if (!first_chunk(in, plan_sh, any)) return;
  }
  unsigned long long tag = 0;
  if (cut_chains)
    tag = (*reinterpret_cast<volatile unsigned long long*>(hs) << 32) | (grid_id() & 0xffffffffull);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  Bars* bars = reinterpret_cast<Bars*>(sm + kOffBar);
  Gates* gates = reinterpret_cast<Gates*>(sm + kOffG);
  Chunk* chunks = reinterpret_cast<Chunk*>(sm + kOffChunk);

  for (int e = tid; e < (kOffA - kOffW) / 16; e += kThreads)   // W and P: zero above the diagonal
    reinterpret_cast<uint4*>(sm + kOffW)[e] = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  if (warp == kWarpMma) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars->full_kq[i], 1);
        mbar_init(&bars->full_v[i], 1);
        mbar_init(&bars->free_kq[i], 1);
        mbar_init(&bars->free_v[i], 256);
        mbar_init(&bars->info[i], 32);
        mbar_init(&bars->gates[i], 128);
        mbar_init(&bars->w_ready[i], 128);
        mbar_init(&bars->o_free[i], 128);
      }
      mbar_init(&bars->d0_ready, 1);
      mbar_init(&bars->d0_free, 128);
      mbar_init(&bars->sa_ready, 256);
      mbar_init(&bars->d1k_ready, 1);
      mbar_init(&bars->d1q_ready, 1);
      mbar_init(&bars->ra_ready, 256);
      mbar_init(&bars->x_ready, 1);
      mbar_init(&bars->xa_ready, 256);
      mbar_init(&bars->s_ready, 1);
      mbar_init(&bars->q_read, 128);
      mbar_init(&bars->o_ready, 1);
      mbar_init(&bars->published, 256);
      mbar_init(&bars->drain, 1);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(&tmem_base, kTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);   // this warp's TMEM lanes

#define HYB_WAIT(bar, parity) __all_sync(0xffffffffu, wait(&(bar), (parity)))
  bool ok = true;
  if (warp < kWarpMain) {
    // ------------------------------------------------------------ preparation
    float* A = reinterpret_cast<float*>(sm + kOffA);
    for (int c = 0;; ++c) {
      const int st = c & 1;
      Gates& G = gates[st];
      ok = bar_prep_all(HYB_WAIT(bars->info[st], (c >> 1) & 1));
      if (!ok) break;
      const int n = chunks[c & 3].n;
      if (n == 0) break;
      ok = HYB_WAIT(bars->full_kq[st], (c >> 1) & 1);
      {                                      // lengths: thread r, row r of the stacked [K; Q]
        const uint8_t* kq = sm + kOffKQ + st * kStageKQ + tid * 128;
        float ss = 0.f;
#pragma unroll
        for (int ch = 0; ch < 16; ++ch) {
          const uint4 u = *reinterpret_cast<const uint4*>(kq + (ch >> 3) * kSubKQ + (((ch & 7) ^ (tid & 7)) << 4));
          const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ss = fmaf(bf16_lo(x[e]), bf16_lo(x[e]), ss);
            ss = fmaf(bf16_hi(x[e]), bf16_hi(x[e]), ss);
          }
        }
        const float inv = eps > 0.f ? 1.f / sqrtf(ss + eps) : 1.f;
        const int t = tid & 63;
        if (tid < 64) G.rk[t] = t < n ? inv : 0.f;
        else G.pq[t] = t < n ? scale * inv : 0.f;
      }
      ok = bar_prep_all(ok);
      if (!ok) break;
      if (tid < 64) {
        const float e = exp2f(G.hi[tid]);    // G.lo is below half an ulp of G.hi
        G.cA[tid] = G.bt[tid] * G.rk[tid];
        G.aR[tid] = G.cA[tid] * e;
        G.oq[tid] = G.pq[tid] * e;
        G.wX[tid] = G.rk[tid] * exp2f((G.hi[63] - G.hi[tid]) + (G.lo[63] - G.lo[tid]));
        if (tid == 63) G.dec = e;
      }
      bar_prep();
      mbar_arrive(&bars->gates[st]);
      ok = HYB_WAIT(bars->d0_ready, c & 1);
      tc_fence_after();
      {
        // warps 0, 1: row t of K K^T -> column t of A^T; warps 2, 3: row t of Q K^T -> row t of P.
        // Rows below 32 have nothing in the columns from 32 on.
        const int t = tid & 63;
        const bool is_p = tid >= 64;
        const float ghi = G.hi[t], glo = G.lo[t], f = is_p ? G.pq[t] : G.cA[t];
        const f32x2 neg = pair(-1.f, -1.f), gh2 = pair(ghi, ghi), gl2 = pair(glo, glo), f2 = pair(f, f);
#pragma unroll 1
        for (int part = 0; part <= (t >> 5); ++part) {
          float v[32];
          tmem_ld32(tl + kCol0 + part * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 h4 = *reinterpret_cast<const float4*>(&G.hi[part * 32 + e]);
            const float4 l4 = *reinterpret_cast<const float4*>(&G.lo[part * 32 + e]);
            const float4 r4 = *reinterpret_cast<const float4*>(&G.rk[part * 32 + e]);
            float d[4];
            unpair(add2(fma2(pair(h4.x, h4.y), neg, gh2), fma2(pair(l4.x, l4.y), neg, gl2)), d[0], d[1]);
            unpair(add2(fma2(pair(h4.z, h4.w), neg, gh2), fma2(pair(l4.z, l4.w), neg, gl2)), d[2], d[3]);
            unpair(mul2(mul2(pair(fast_exp2(d[0]), fast_exp2(d[1])), pair(v[e], v[e + 1])),
                        mul2(pair(r4.x, r4.y), f2)), v[e], v[e + 1]);
            unpair(mul2(mul2(pair(fast_exp2(d[2]), fast_exp2(d[3])), pair(v[e + 2], v[e + 3])),
                        mul2(pair(r4.z, r4.w), f2)), v[e + 2], v[e + 3]);
          }
          if (part == (t >> 5)) {            // at the diagonal: s < t, or s <= t for P
            const int most = lane + (is_p ? 1 : 0);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = e < most ? v[e] : 0.f;
          }
          if (!is_p) {
#pragma unroll
            for (int e = 0; e < 32; ++e) A[(part * 32 + e) * kLdA + t] = v[e];
          } else {
            uint8_t* dst = sm + kOffP + st * 2 * kTile64 + t * 128;
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              uint32_t h[4], m[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) split2(v[ch * 8 + 2 * e], v[ch * 8 + 2 * e + 1], h[e], m[e]);
              const int off = ((part * 4 + ch) ^ (t & 7)) << 4;
              *reinterpret_cast<uint4*>(dst + off) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(dst + kTile64 + off) = make_uint4(m[0], m[1], m[2], m[3]);
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bars->d0_free);
      ok = bar_prep_all(ok);
      if (!ok) break;
      // W = (1 + A)^-1 by blocks, 16, 32, 64; A is held transposed, A^T[s][t] at A[s * kLdA + t], W
      // row-major in its place. Two blocks W00, W11 on the diagonal and A10 below give
      // W10 = -W11 (A10 W00): the first product goes where W10 will be, A10^T lies in the (zero)
      // block above it.
      // 16 x 16, a warp each, a lane a column (lanes 16-31 do the same): once w_m is final it is
      // taken from every later row (independent fma, one 16-byte broadcast read for four).
      {
        float* D = A + warp * 16 * (kLdA + 1);
        const int col = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < 15; ++m) {
#pragma unroll
          for (int i4 = (m + 1) / 4; i4 < 4; ++i4) {
            const float4 a = *reinterpret_cast<const float4*>(&D[m * kLdA + i4 * 4]);
            const float y[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (i4 * 4 + e > m) x[i4 * 4 + e] = fmaf(-y[e], x[m], x[i4 * 4 + e]);
          }
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
          for (int i = 0; i < 16; ++i) D[i * kLdA + col] = x[i];
        }
      }
      bar_prep();
      {                                      // 32 x 32: two warps each, a lane 4 rows of a column
        float* D = A + (warp >> 1) * 32 * (kLdA + 1);
        const int col = lane & 15, r0 = 8 * (warp & 1) + 4 * (lane >> 4);
        f32x2 x0 = pair(0.f, 0.f), x1 = x0;
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          const float b = D[m * kLdA + col];
          const float4 a = *reinterpret_cast<const float4*>(&D[m * kLdA + 16 + r0]);
          x0 = fma2(pair(a.x, a.y), pair(b, b), x0);
          x1 = fma2(pair(a.z, a.w), pair(b, b), x1);
        }
        float y[4];
        unpair(x0, y[0], y[1]);
        unpair(x1, y[2], y[3]);
#pragma unroll
        for (int r = 0; r < 4; ++r) D[(16 + r0 + r) * kLdA + col] = y[r];
        bar_prep();
        f32x2 z[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) z[r] = pair(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < 16; m += 4) {
          const f32x2 b0 = pair(D[(16 + m) * kLdA + col], D[(17 + m) * kLdA + col]);
          const f32x2 b1 = pair(D[(18 + m) * kLdA + col], D[(19 + m) * kLdA + col]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float4 a = *reinterpret_cast<const float4*>(&D[(16 + r0 + r) * kLdA + 16 + m]);
            z[r] = fma2(pair(a.x, a.y), b0, z[r]);
            z[r] = fma2(pair(a.z, a.w), b1, z[r]);
          }
        }
        bar_prep();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float a, b;
          unpair(z[r], a, b);
          D[(16 + r0 + r) * kLdA + col] = -(a + b);
          D[(r0 + r) * kLdA + 16 + col] = 0.f;
        }
      }
      bar_prep();
      {                                      // 64 x 64: each warp 8 rows, a lane a column
        f32x2 x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = pair(0.f, 0.f);
#pragma unroll 8
        for (int m = 0; m < 32; ++m) {
          const float b = A[m * kLdA + lane];
          const float4 a0 = *reinterpret_cast<const float4*>(&A[m * kLdA + 32 + 8 * warp]);
          const float4 a1 = *reinterpret_cast<const float4*>(&A[m * kLdA + 36 + 8 * warp]);
          const f32x2 b2 = pair(b, b);
          x[0] = fma2(pair(a0.x, a0.y), b2, x[0]);
          x[1] = fma2(pair(a0.z, a0.w), b2, x[1]);
          x[2] = fma2(pair(a1.x, a1.y), b2, x[2]);
          x[3] = fma2(pair(a1.z, a1.w), b2, x[3]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float a, b;
          unpair(x[r], a, b);
          A[(32 + 8 * warp + 2 * r) * kLdA + lane] = a;
          A[(33 + 8 * warp + 2 * r) * kLdA + lane] = b;
        }
        bar_prep();
        f32x2 z[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) z[r] = pair(0.f, 0.f);
#pragma unroll 4
        for (int m = 0; m < 32; m += 4) {
          const f32x2 b0 = pair(A[(32 + m) * kLdA + lane], A[(33 + m) * kLdA + lane]);
          const f32x2 b1 = pair(A[(34 + m) * kLdA + lane], A[(35 + m) * kLdA + lane]);
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const float4 a = *reinterpret_cast<const float4*>(&A[(32 + 8 * warp + r) * kLdA + 32 + m]);
            z[r] = fma2(pair(a.x, a.y), b0, z[r]);
            z[r] = fma2(pair(a.z, a.w), b1, z[r]);
          }
        }
        // not back into its place, where others still read: over A10^T (rows r, columns 32-63)
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          float a, b;
          unpair(z[r], a, b);
          A[(8 * warp + r) * kLdA + 32 + lane] = -(a + b);
        }
      }
      bar_prep();
      // W as three bf16 terms: row t, half of its columns (the upper right block is zero from the start)
      if (tid >= 64 || (tid & 1) == 0) {
        const int t = tid >> 1, half = tid & 1;
        const float* src = t < 32 ? A + t * kLdA : A + (half ? t * kLdA + 32 : (t - 32) * kLdA + 32);
        uint8_t* dst = sm + kOffW + st * 3 * kTile64 + t * 128;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const float4 u = *reinterpret_cast<const float4*>(src + ch * 8 + e);
            v[e] = u.x; v[e + 1] = u.y; v[e + 2] = u.z; v[e + 3] = u.w;
          }
          uint32_t h[4], m[4], l[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split3(v[2 * e], v[2 * e + 1], h[e], m[e], l[e]);
          const int off = ((half * 4 + ch) ^ (t & 7)) << 4;
          *reinterpret_cast<uint4*>(dst + off) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + kTile64 + off) = make_uint4(m[0], m[1], m[2], m[3]);
          *reinterpret_cast<uint4*>(dst + 2 * kTile64 + off) = make_uint4(l[0], l[1], l[2], l[3]);
        }
      }
      fence_async_smem();
      mbar_arrive(&bars->w_ready[st]);
    }
    if (!ok && lane == 0) flag(status, HYB_DEVERR_TIMEOUT);
  } else if (warp < kWarpOut) {
    // ------------------------------------------------------------ the state's chain
    const int half = (warp - kWarpMain) >> 2;
    const int j = (warp & 3) * 32 + lane;    // value column: TMEM lane of this thread
    const int x0 = half * 32, i0 = half * 64;
    for (int c = 0;; ++c) {
      const int st = c & 1;
      const Gates& G = gates[st];
      ok = HYB_WAIT(bars->info[st], (c >> 1) & 1);
      if (!ok) break;
      const Chunk& ch = chunks[c & 3];
      const int n = ch.n, flags = ch.flags;
      if (n == 0) break;
      ok = HYB_WAIT(bars->gates[st], (c >> 1) & 1);
      if (!ok) break;
      // this chunk's first state: the run's from the pool, or what the last chunk left in TMEM
      if (flags & kFirst) {
        if (flags & kTake) {
          const unsigned long long* fl = hs + 1 + (p + 1);
          const uint64_t t0 = global_ns();
          while (ld_acquire_u64(fl) != tag) {
            if (global_ns() - t0 > 2000000000ull) {
              flag(status, HYB_DEVERR_TIMEOUT);
              break;
            }
            __nanosleep(100);
          }
        }
        const float* S = ch.S;
#pragma unroll 1
        for (int i = i0; i < i0 + 64; i += 16) {
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            v[e] = flags & kZero ? 0.f : __ldcg(S + (i + e) * kD + j);
          put_state(tl, i, v, G.dec);
        }
      } else {
        const float dec = G.dec;
#pragma unroll 2
        for (int i = i0; i < i0 + 64; i += 16) {
          float s[16];
          tmem_ld16(tl + kColS + i, s);
          tmem_ld_wait();
          put_state(tl, i, s, dec);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars->sa_ready);
      // V of this column while (k) runs; rows past the request may hold anything
      ok = HYB_WAIT(bars->full_v[st], (c >> 1) & 1);
      if (!ok) break;
      float v[32];
      {
        const uint8_t* vs = sm + kOffV + st * kStageV + (j >> 6) * kSubV + (j & 7) * 2;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int t = x0 + e;
          const uint16_t b = *reinterpret_cast<const uint16_t*>(vs + t * 128 + ((((j & 63) >> 3) ^ (t & 7)) << 4));
          v[e] = t < n ? __uint_as_float((uint32_t)b << 16) : 0.f;
        }
      }
      mbar_arrive(&bars->free_v[st]);
      // R = beta (V - e^G K S)
      ok = HYB_WAIT(bars->d1k_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
      {
        float d[32];                         // all read before R's l goes into the same columns
        tmem_ld32(tl + kCol1K + x0, d);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 b = *reinterpret_cast<const float4*>(&G.bt[x0 + e]);
          const float4 a = *reinterpret_cast<const float4*>(&G.aR[x0 + e]);
          d[e] = fmaf(-a.x, d[e], b.x * v[e]);
          d[e + 1] = fmaf(-a.y, d[e + 1], b.y * v[e + 1]);
          d[e + 2] = fmaf(-a.z, d[e + 2], b.z * v[e + 2]);
          d[e + 3] = fmaf(-a.w, d[e + 3], b.w * v[e + 3]);
        }
#pragma unroll
        for (int x = 0; x < 32; x += 16) {
          const int at = (x0 + x) / 2;
          put_terms(tl + kColRh + at, tl + kColRm + at, tl + kColRl + at, d + x);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars->ra_ready);
      // X: times its way to the chunk's end for the state, and as it is for the outputs
      ok = HYB_WAIT(bars->x_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int x = 0; x < 32; x += 16) {
        float d[16];
        tmem_ld16(tl + kColX + x0 + x, d);
        tmem_ld_wait();
        const int at = (x0 + x) / 2;
        uint32_t h[8], m[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split2(d[2 * e], d[2 * e + 1], h[e], m[e]);
        tmem_st8u(tl + kColOh + at, h);
        tmem_st8u(tl + kColOm + at, m);
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 a = *reinterpret_cast<const float4*>(&G.wX[x0 + x + e]);
          d[e] *= a.x;
          d[e + 1] *= a.y;
          d[e + 2] *= a.z;
          d[e + 3] *= a.w;
        }
        put_terms(tl + kColXh + at, tl + kColXm + at, tl + kColXl + at, d);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars->xa_ready);
      // the chunk's last state
      ok = HYB_WAIT(bars->s_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
      if (flags & kLast) {                   // end of a run: to the pool, and handed over if cut
        float* S = ch.S;
#pragma unroll 1
        for (int i = i0; i < i0 + 64; i += 16) {
          float s[16];
          tmem_ld16(tl + kColS + i, s);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) S[(i + e) * kD + j] = s[e];
        }
        if (flags & kHand) {                 // at most once per CTA (its first run)
          __threadfence();
          mbar_arrive(&bars->published);
          if (tid == kWarpMain * 32) {
            if (mbar_wait(&bars->published, 0)) st_release_u64(hs + 1 + p, tag);
            else flag(status, HYB_DEVERR_TIMEOUT);
          }
        }
      }
    }
    if (!ok && lane == 0) flag(status, HYB_DEVERR_TIMEOUT);
  } else if (warp < kWarpFeed) {
    // ------------------------------------------------------------ outputs
    const int j = (warp & 3) * 32 + lane;
    for (int c = 0;; ++c) {
      const int st = c & 1;
      const Gates& G = gates[st];
      ok = HYB_WAIT(bars->info[st], (c >> 1) & 1);
      if (!ok) break;
      const int n = chunks[c & 3].n;
      if (n == 0) break;
      __nv_bfloat16* dst = out + ((int64_t)chunks[c & 3].row * in.H + chunks[c & 3].h) * kD + j;
      ok = HYB_WAIT(bars->gates[st], (c >> 1) & 1);
      if (!ok) break;
      ok = HYB_WAIT(bars->d1q_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
      float o[64];
#pragma unroll
      for (int x = 0; x < 64; x += 16) tmem_ld16(tl + kCol1Q + x, o + x);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(&bars->q_read);
#pragma unroll
      for (int t = 0; t < 64; ++t) o[t] *= G.oq[t];
      ok = HYB_WAIT(bars->o_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int x = 0; x < 64; x += 16) {
        float d[16];
        tmem_ld16(tl + kCol1Q + x, d);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[x + e] += d[e];
      }
      tc_fence_before();
      mbar_arrive(&bars->o_free[st]);
#pragma unroll
      for (int t = 0; t < 64; ++t)
        if (t < n) dst[(int64_t)t * in.H * kD] = __float2bfloat16_rn(o[t]);
    }
    if (!ok && lane == 0) flag(status, HYB_DEVERR_TIMEOUT);
  } else if (warp == kWarpFeed) {
    // ------------------------------------------------------------ chunks, loads, gates
    if (lane == 0) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
    }
    Walk w;
    bool more = first_chunk(in, plan_sh, w);
    int ckq = 0, cv = 0;                     // chunks requested
    for (int c = 0;; ++c) {
      const int st = c & 1, row = w.sg.t0 + w.ci * kC;
      const int n = more ? min(kC, w.sg.n - w.ci * kC) : 0;
      // gates and betas of rows lane and lane + 32
      const int64_t at = (int64_t)row * in.H + w.sg.h + (int64_t)lane * in.H, at2 = at + 32ll * in.H;
      const float ga = lane < n ? g[at] : 0.f, gb = lane + 32 < n ? g[at2] : 0.f;
      const float ba = lane < n ? beta[at] : 0.f, bb = lane + 32 < n ? beta[at2] : 0.f;
      if (n > 0) {
        if (c >= 2) ok = HYB_WAIT(bars->free_kq[st], ((c - 2) >> 1) & 1);
        if (!ok) break;
        const int hk = w.sg.h / rep;
        if (lane == 0) {
          uint8_t* kq = sm + kOffKQ + st * kStageKQ;
          mbar_expect_tx(&bars->full_kq[st], kStageKQ);
          for (int sb = 0; sb < 2; ++sb) {
            tma_load_3d(kq + sb * kSubKQ, &tk, sb * 64, hk, row, &bars->full_kq[st]);
            tma_load_3d(kq + sb * kSubKQ + 64 * 128, &tq, sb * 64, hk, row, &bars->full_kq[st]);
          }
        }
        ckq = c + 1;
        if (c >= 2) ok = HYB_WAIT(bars->free_v[st], ((c - 2) >> 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          uint8_t* vs = sm + kOffV + st * kStageV;
          mbar_expect_tx(&bars->full_v[st], kStageV);
          for (int sb = 0; sb < 2; ++sb)
            tma_load_3d(vs + sb * kSubV, &tv, sb * 64, w.sg.h, row, &bars->full_v[st]);
        }
        cv = c + 1;
      }
      // the buffers' last users are done (a slot of `chunks` is used two chunks longer)
      if (c >= 2) ok = HYB_WAIT(bars->o_free[st], ((c - 2) >> 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        const int flags = (w.ci == w.sg.c0 ? kFirst | (w.sg.zero_start ? kZero : 0) | (w.sg.wait_handoff ? kTake : 0) : 0) |
                          (w.ci == w.sg.c1 - 1 ? kLast | (w.sg.publish ? kHand : 0) : 0);
        chunks[c & 3] = Chunk{w.sg.S, row, n, w.sg.h, flags, {0, 0}};
      }
      // running sum in units of log 2, exact in integer steps of 2^-36 (fp32 would lose the
      // small gates behind large ones, and fp64 is slow on this GPU)
      Gates& G = gates[st];
      long long a = to_fixed(ga), b = to_fixed(gb);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        a += lane >= o ? x : 0;
        b += lane >= o ? y : 0;
      }
      b += __shfl_sync(0xffffffffu, a, 31);
      const unsigned na = __ballot_sync(0xffffffffu, ga != ga), nb = __ballot_sync(0xffffffffu, gb != gb);
      const unsigned upto = 0xffffffffu >> (31 - lane);
      from_fixed(a, (na & upto) != 0, G.hi[lane], G.lo[lane]);
      from_fixed(b, na != 0 || (nb & upto) != 0, G.hi[lane + 32], G.lo[lane + 32]);
      G.bt[lane] = ba;
      G.bt[lane + 32] = bb;
      mbar_arrive(&bars->info[st]);
      if (n == 0) break;
      more = next_chunk(in, plan_sh, w);
    }
    if (!ok && lane == 0) {                  // let the loads in flight land before exiting
      flag(status, HYB_DEVERR_TIMEOUT);
      for (int i = max(0, ckq - 2); i < ckq; ++i) mbar_wait(&bars->full_kq[i & 1], (i >> 1) & 1, 100000000ull);
      for (int i = max(0, cv - 2); i < cv; ++i) mbar_wait(&bars->full_v[i & 1], (i >> 1) & 1, 100000000ull);
    }
  } else {
    // ------------------------------------------------------------ MMAs
    const uint32_t sm0 = smem_u32(sm);
    const uint64_t km0 = sw128_desc(sm0, 16, 1024);            // K-major operands
    const uint64_t mn0 = sw128_desc(sm0, kSubKQ, 1024);        // K as [t][i], i-major: two 64-wide blocks
    bool more = true;
    // (0) of chunk cn, if there is one: rows past the request become zero rows of K first
    auto issue0 = [&](int cn) {
      const int st = cn & 1;
      if (!HYB_WAIT(bars->info[st], (cn >> 1) & 1)) return false;
      const int n = chunks[cn & 3].n;
      more = n > 0;
      if (!more) return true;
      if (!HYB_WAIT(bars->full_kq[st], (cn >> 1) & 1)) return false;
      if (n < kC) {
        uint8_t* ks = sm + kOffKQ + st * kStageKQ;
        for (int e = lane; e < (kC - n) * 16; e += 32)
          *reinterpret_cast<uint4*>(ks + ((e >> 3) & 1) * kSubKQ + (n + (e >> 4)) * 128 + (e & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        fence_async_smem();
      }
      if (cn >= 1 && !HYB_WAIT(bars->d0_free, (cn - 1) & 1)) return false;
      __syncwarp();
      if (elect_one()) {
        tc_fence_after();
        const uint32_t kq = kOffKQ + st * kStageKQ;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t d = desc_add(km0, kq + (k >> 2) * kSubKQ + (k & 3) * 32);
          tc_mma(tmem + kCol0, d, d, kIdesc64, k > 0);
        }
        tc_commit(&bars->d0_ready);
      }
      __syncwarp();
      return true;
    };
    ok = issue0(0);
    for (int c = 0; ok && more; ++c) {
      const int st = c & 1;
      const uint32_t kq = kOffKQ + st * kStageKQ;
      ok = HYB_WAIT(bars->sa_ready, c & 1);
      if (!ok) break;
      if (elect_one()) {
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 24; ++x) {       // (k)
          const int k = x & 7;
          tc_mma_ta(tmem + kCol1K, tmem + kColSA + x * 8, desc_add(km0, kq + (k >> 2) * kSubKQ + (k & 3) * 32), kIdesc64, x > 0);
        }
        tc_commit(&bars->d1k_ready);
      }
      __syncwarp();
      if (c >= 1) ok = HYB_WAIT(bars->o_free[st ^ 1], ((c - 1) >> 1) & 1);
      if (!ok) break;
      if (elect_one()) {
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 16; ++x) {       // (q)
          const int k = x & 7;
          tc_mma_ta(tmem + kCol1Q, tmem + kColSA + x * 8, desc_add(km0, kq + 64 * 128 + (k >> 2) * kSubKQ + (k & 3) * 32), kIdesc64, x > 0);
        }
        tc_commit(&bars->d1q_ready);
      }
      __syncwarp();
      ok = issue0(c + 1);
      if (!ok) break;
      ok = HYB_WAIT(bars->w_ready[st], (c >> 1) & 1) && HYB_WAIT(bars->ra_ready, c & 1);
      if (!ok) break;
      if (elect_one()) {
        tc_fence_after();
        const uint64_t wd = desc_add(km0, kOffW + st * 3 * kTile64);
#pragma unroll
        for (int x = 0; x < 6; ++x) {        // (w): R h W h, h m, m h, h l, m m, l h
          const int r = x == 2 || x == 4 ? 1 : x == 5 ? 2 : 0, t = x == 1 || x == 4 ? 1 : x == 3 ? 2 : 0;
          const uint32_t ra = r == 0 ? kColRh : r == 1 ? kColRm : kColRl;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_ta(tmem + kColX, tmem + ra + k * 8, desc_add(wd, t * kTile64 + k * 32), kIdesc64, x + k > 0);
        }
        tc_commit(&bars->x_ready);
      }
      __syncwarp();
      ok = HYB_WAIT(bars->xa_ready, c & 1);
      if (!ok) break;
      if (elect_one()) {
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 3; ++x) {        // (s)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_ta(tmem + kColS, tmem + kColXh + x * 32 + k * 8, desc_add(mn0, kq + k * 2048), kIdescS, 1);
        }
        tc_commit(&bars->s_ready);
        tc_commit(&bars->free_kq[st]);       // the last use of K and Q
      }
      __syncwarp();
      ok = HYB_WAIT(bars->q_read, c & 1);
      if (!ok) break;
      if (elect_one()) {
        tc_fence_after();
        const uint64_t pd = desc_add(km0, kOffP + st * 2 * kTile64);
#pragma unroll
        for (int x = 0; x < 3; ++x) {        // (o): X h P h, h m, m h
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_ta(tmem + kCol1Q, tmem + (x == 2 ? kColOm : kColOh) + k * 8, desc_add(pd, (x == 1 ? kTile64 : 0) + k * 32), kIdesc64, x + k > 0);
        }
        tc_commit(&bars->o_ready);
      }
      __syncwarp();
    }
    if (elect_one()) {
      if (!ok) {                             // let every issued MMA finish before exiting
        flag(status, HYB_DEVERR_TIMEOUT);
        tc_commit(&bars->drain);
        mbar_wait(&bars->drain, 0, 100000000ull);
      }
    }
  }
#undef HYB_WAIT
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

bool delta_prefill_tc_supported(const hyb_delta_dims_t* d) {
  return d->dtype == HYB_BF16 && d->head_dim == kD;
}

cudaError_t launch_delta_prefill_tc(void* out, const void* q, const void* k, const void* v,
                                    const float* g, const float* beta, const int32_t* cu,
                                    float* pool, int NS, const int32_t* slots,
                                    const uint8_t* reset, int B, int T, int max_len,
                                    const hyb_delta_dims_t* d, int64_t qs, int64_t ks, int64_t vs,
                                    void* ws, unsigned* status, cudaStream_t s) {
  const int Hv = d->num_v_heads, Hk = d->num_qk_heads;
  CUtensorMap mq, mk, mv;
  const uint32_t box[3] = {64, 1, 64};
  const uint64_t rows = T > 0 ? T : 1;
  auto encode = [&](CUtensorMap* m, const void* base, int heads, int64_t stride) {
    const uint64_t dims[3] = {(uint64_t)kD, (uint64_t)heads, rows};
    const uint64_t strides[2] = {(uint64_t)kD * 2, (uint64_t)stride * 2};
    return encode_tmap_bf16(m, base, 3, dims, strides, box);
  };
  if (!encode(&mq, q, Hk, qs) || !encode(&mk, k, Hk, ks) || !encode(&mv, v, Hv, vs))
    return cudaErrorInvalidValue;
  cudaError_t e = set_smem((const void*)delta_prefill_tc_kernel, kSmem);
  if (e != cudaSuccess) return e;
  // One CTA per SM at most. A CTA for each chain when the GPU has SMs enough: no chain is cut then.
  // With more chains than SMs they are cut, and a CTA may wait for the state another one hands
  // over: all must be resident at once, so that launch is cooperative.
  const int64_t units = (int64_t)B * Hv;
  const int sms = std::min(num_sms(), kLinMaxCtas);
  const int cut_chains = units > sms;
  if (cut_chains) {
    e = launch_handoff_epoch(ws, s);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(sms, units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = cut_chains;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const In in{cu, slots, reset, pool, NS, T, max_len, Hv};
  e = cudaLaunchKernelEx(&cfg, delta_prefill_tc_kernel, mq, mk, mv, static_cast<__nv_bfloat16*>(out),
                         g, beta, in, B, Hv / Hk, d->scale, d->qk_norm_eps,
                         static_cast<unsigned long long*>(ws), cut_chains, status);
  count_launch();
  return e;
}

}  // namespace hyb
