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
// and the corrections are each split into three bf16 terms, h + m + l, which hold an fp32 number
// without loss. K S and the state's change then are exact products; of W R the terms beyond 2^-24
// are left out (six of nine products). The tensor core's fp32 sums are cut, not rounded, at 24
// bits: products go in with the smallest terms first (within each half of a sum, for the halves are
// issued as their operands come: of K S 16 cuts, of X 14, of the state's change 8 are of a sum of full
// size), and the state's change is summed by itself and then added to the decayed state, rounded to
// nearest. (Summed up in the state's own accumulator, 12 cuts towards zero in 64 rows, 8192 rows of
// small changes put it off by 3.0e-5; now 3.2e-7, the fp32 recurrence 2.3e-6.) Slow decays are applied
// as S + (e^G - 1) S: see get_state.
// The outputs, rounded to bf16 in the end, take two terms of S, X and P, 2^-18.5 of each in the mean of
// squares: TMEM and shared memory have no room for the third. 0.35 % of them come out as the bf16 next to
// the one that the exact value rounds to (of the fp32 recurrence's 0.03 %). With two terms throughout,
// states were off by some 3e-6; now by 1.6e-7 after 77 rows, 2e-7 after 1024.
//
// Layout. Everything on the chain is kept transposed: TMEM lane j is the state's value column j, so
// each thread owns a column (half of its columns' range), nothing on the chain crosses threads, and
// the results (accumulators in TMEM) become the next product's A operand by the same thread
// writing them back as bf16 terms; shared memory holds only what TMA brings (K, Q, V), W and P, and
// X's second term, for which TMEM has no columns left.
//   (k) D1K[j][t] = S^T K^T     A = S (TMEM, 3 terms),  B = K rows     24 MMAs 128 x 64 x 16
//   (q) D1Q[j][t] = S^T Q^T     A = S (TMEM, 2 terms),  B = Q rows     16
//   (0) [K; Q] K^T, two chunks ahead (128 x 64)                         8
//   (w) X^T       = R^T W^T     A = R (TMEM),  B = W rows (6 pairs)    24
//   (s) dS^T      = X'^T K      A = X e^(G_C - G) (TMEM), B = K^T      12 MMAs 128 x 128 x 16
//   (o) D1Q       = X^T P^T     A = X (2 terms), B = P (3 pairs)       12
// MMAs of N = 64 take 34 cycles of the tensor core, N = 128 67: 3.7K cycles a chunk; with W's warp MMAs
// the pipe is busy for 3.9K.
//
// W = (1 + A)^-1 in fp32 on the warps' own MMAs (tf32, two terms each) by blocks of 8, 16, 32 and 64. What
// it is off by adds up over a chunk's rows where keys repeat: see tf32_terms. States against fp64 after
// 1024 rows, no decay, beta 1: one key 4.4e-7 (fp32 recurrence 8.1e-7), keys of 2 dimensions 4.0e-7.
//
// Warps: 0-7 prepare chunks (lengths, factors, W, P), two groups of four with a chunk each, so a
// chunk's preparation may take two chunks' time; 8-15 carry the chain (two warps to 32 lanes, each
// half of the columns); 16-19 scale and write outputs; 20 walks the CTA's chunks, sums the gates
// and issues TMA loads (three stages of K and Q, one of V, which the chain keeps in registers); 21
// issues the MMAs. Chains are shared out over the CTAs as in chain_split.cuh: the 256 chains of 8
// requests x 32 heads would leave the second wave of 152 CTAs a third full.
//
// What bounds it: a chunk's way round its three loops (chain, preparation, outputs), each about 10K
// cycles of waits for one another; leaving any one piece of work out changes the time by 0-3 %.
// 8 requests of 8192 rows, 32 heads: 1.20 ms (tensor pipe 37 % busy, issue slots 51 %, 1.8 TB/s;
// 0.27 of the copy rate); one request of 4096 rows: 326 us, 5.1 us a chunk; one of 77: 20 us. On the way,
// 8 x 8192: 13.5 ms token by token -> 2.54 (this design) -> 1.94 (elected MMA issue, integer gate
// sums, chunk descriptors instead of local arrays) -> 1.56 (two preparing groups) -> 1.42 (warp MMAs
// in W) -> 1.19 (rolled loops: less of the code falls out of the instruction cache) -> 1.12 (one site
// for a run's setup) -> 1.19 (the state rounded to nearest) -> 1.17 (fewer instructions for W, waits on
// the SM's clock) -> 1.20 (slow decays without a drift, one prompt 318 -> 322 us; W's first terms and the
// three-term splits rounded to nearest, one prompt 311 -> 318 and 322 -> 326 us).
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
constexpr int kNKQ = 3;                        // stages of K and Q; one of V
constexpr int kOffV = kOffKQ + kNKQ * kStageKQ;
constexpr int kOffW = kOffV + kStageV;         // [term]
constexpr int kOffP = kOffW + 3 * kTile64;     // [buffer][term]
constexpr int kOffA = kOffP + 2 * 2 * kTile64; // [group] the system, fp32, then its inverse
constexpr int kLdA = 72;                       // floats per row: fragments of 4 x 8 hit 32 banks
constexpr int kOffG = kOffA + 2 * kC * kLdA * 4;

struct Gates {                                 // factors of a chunk's rows
  float hi[kC], lo[kC];                        // G in units of log 2, as a sum of two
  float bt[kC];                                // beta
  float eR[kC], cA[kC], wB[kC];                // e^G / |k|, beta / |k|^2, beta / |k|
  float wX[kC], pq[kC], oq[kC];                // e^(G_C - G), scale / |q|, scale e^G / |q|
  float dec, keep, pad[2];                     // of the state, S <- dec S + keep S: e^(G_C) and 0, or,
                                               // where the decay is slow, e^(G_C) - 1 and 1
};
// What the warps need to know of a chunk. The feeding warp walks the CTA's runs and writes these,
// four chunks deep as the gates: chunk c's place is free once (s) of chunk c - 3 is done, which
// implies that everybody has left chunk c - 4. n = 0 ends them.
struct Chunk {
  float* S;                                    // the chain's state in the pool
  int row, n, h, flags;                        // first row, rows, value head
  int pad[2];
};
constexpr int kFirst = 1, kLast = 2, kZero = 4, kTake = 8, kHand = 16;   // of a run; its state: zero
                                               // at first, taken over first, handed over at last
constexpr int kOffChunk = kOffG + 4 * (int)sizeof(Gates);
constexpr int kOffBar = kOffChunk + 4 * (int)sizeof(Chunk);

struct Bars {
  uint64_t full_kq[kNKQ], free_kq[kNKQ], full_v, free_v;
  uint64_t info[4], gates[4];                  // their readers may lag by more than a chunk
  uint64_t w_ready[2], o_free[2];
  uint64_t sa_ready[2], ra_ready[2], xa_ready[2];   // an operand's first and second half
  uint64_t d0_ready[2], d0_free, d1k_ready, d1q_ready, x_ready, s_ready;
  uint64_t om_ready, q_scaled, o_ready, d1q_free, published, drain;
};
constexpr int kSmem = kOffBar + 512 + 1024;    // + slack for 1024-byte alignment
static_assert(sizeof(Bars) <= 512 && kOffG % 16 == 0 && kOffBar % 8 == 0 && kSmem <= 227 * 1024, "smem");

constexpr int kWarpMain = 8, kWarpOut = 16, kWarpFeed = 20, kWarpMma = 21;
constexpr int kThreads = 22 * 32;
// Chunks that a chain's state (a read and a write of 64 KB, nothing under way meanwhile) counts as in
// the work split: 24 ragged requests of up to 5000 rows take 632 us with 0, 480 with 1, 477 with 2,
// 8 x 8192 1.21, 1.19 and 1.19 ms.
constexpr int kChainCost = 1;
constexpr uint32_t kTmemCols = 512;
// D0 | D1K | D1Q | S fp32 | operand terms of S (per 16 key dims 8 columns of h and 8 of m; then l).
// Once (k) and (q) have read the terms, others take their places: R's h and m over S's l, R's l
// inside D1K (each thread over columns that only it reads); X over the first half of S's h and m.
// After (w), X' goes over R's h and m and over D1K's second half, X's h for (o) over its first; the
// state's change over all of S's h and m, each 16 columns of it where the same thread's next
// terms will be. X's m lies in V's buffer, once every thread has V in its registers: the next V
// is loaded when (o) is done.
constexpr uint32_t kCol0 = 0, kCol1K = 64, kCol1Q = 128, kColS = 192, kColSA = 320;
constexpr uint32_t kColRh = kColSA + 128, kColRm = kColSA + 160, kColRl = kCol1K + 16;
constexpr uint32_t kColX = kColSA, kColDS = kColSA;
constexpr uint32_t kColXh = kColSA + 128, kColXm = kColSA + 160, kColXl = kCol1K + 32;
constexpr uint32_t kColOh = kCol1K;

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
  int ci = 0, stage = 0, u = 0;
};
__device__ __forceinline__ bool next_chunk(const In& in, const Plan& pl, Walk& w) {
  if (w.stage > 0 && ++w.ci < w.sg.c1) return true;
#pragma unroll 1
  while (true) {
    int unit = -1, c0 = 0, c1 = -1;
    if (w.stage == 0) {
      w.stage = 1;
      w.u = pl.full_u0;
      unit = pl.head_u;
      c1 = pl.head_end;
    } else if (w.stage == 1 && w.u < pl.full_u1) {
      unit = w.u++;
    } else if (w.stage == 1) {
      w.stage = 2;
      unit = pl.tail_u;
      c0 = pl.tail_begin;
    } else {
      return false;
    }
    if (unit >= 0 && make_run(in, unit, c0, c1, w.sg)) {
      w.ci = w.sg.c0;
      return true;
    }
  }
}

// ------------------------------------------------------------------ three-term splits
// x = h + m + l, h and m rounded to nearest: each remainder is exact, the last has at most 8 bits
// left. (Cut instead of rounded, remainders are twice as large and have one sign: outputs, which take h
// and m only, then come out on the other side of a bf16 rounding twice as often, 0.8 % of them for 0.35 %;
// one prompt takes 322 us for 326, batches the same.) Pairs are packed as the tensor core reads them.
__device__ __forceinline__ uint32_t pack_hi(float a, float b) {        // upper halves of a, b
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ void rest(float& a, float& b, uint32_t t) { // less their terms t
  unpair(fma2(pair(bf16_lo(t), bf16_hi(t)), pair(-1.f, -1.f), pair(a, b)), a, b);
}
__device__ __forceinline__ void split3(float a, float b, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = pack_bf16(a, b);
  rest(a, b, h);
  m = pack_bf16(a, b);
  rest(a, b, m);
  l = pack_hi(a, b);
}
// two terms: off by at most 2^-16, 2^-18.5 in the mean of squares
__device__ __forceinline__ void split2(float a, float b, uint32_t& h, uint32_t& m) {
  h = pack_bf16(a, b);
  rest(a, b, h);
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

// Operands of a warp's 16 x 8 x 8 product in two tf32 terms, the first rounded to nearest, the second
// cut: h + l is off by at most one ulp of x, and what the products leave out (l l) has either sign.
// (The first term cut as well loses two bits and all of it towards zero, which adds up over a chunk
// where keys repeat.) The low 13 bits of each word are zero. A NaN stays one in l.
__device__ __forceinline__ uint32_t cut_tf32(uint32_t x) { return x & 0xffffe000u; }
__device__ __forceinline__ void tf32_terms(float x, uint32_t& h, uint32_t& l) {
  h = cut_tf32(__float_as_uint(x) + 0x1000u);
  l = cut_tf32(__float_as_uint(x - __uint_as_float(h)));
}
struct FragA {                                 // 16 x 8, element (r, k) at p[r * RS + k * KS]
  uint32_t h[4], l[4];
  // top, bottom: rows 0-7, 8-15 are read; else they are zero
  template <int RS, int KS>
  __device__ __forceinline__ void load(const float* p, int lane, bool top = true, bool bottom = true) {
    const float* q = p + (lane >> 2) * RS + (lane & 3) * KS;
    tf32_terms(top ? q[0] : 0.f, h[0], l[0]);
    tf32_terms(bottom ? q[8 * RS] : 0.f, h[1], l[1]);
    tf32_terms(top ? q[4 * KS] : 0.f, h[2], l[2]);
    tf32_terms(bottom ? q[8 * RS + 4 * KS] : 0.f, h[3], l[3]);
  }
};
struct FragB {                                 // 8 x 8, element (k, n) at p[k * kLdA + n]
  uint32_t h[2], l[2];
  __device__ __forceinline__ void load(const float* p, int lane) {
    const float* q = p + (lane & 3) * kLdA + (lane >> 2);
    tf32_terms(q[0], h[0], l[0]);
    tf32_terms(q[4 * kLdA], h[1], l[1]);
  }
};
__device__ __forceinline__ void mma_tf32(float* c, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void mma_tf32(float* c, const FragA& a, const FragB& b) {
  mma_tf32(c, a.l, b.h);
  mma_tf32(c, a.h, b.l);
  mma_tf32(c, a.h, b.h);
}
// a result of such products, times sign, to p[r * kLdA + n]
__device__ __forceinline__ void store_c(float* p, const float* c, float sign, int lane, bool bottom = true) {
  float* q = p + (lane >> 2) * kLdA + 2 * (lane & 3);
  *reinterpret_cast<float2*>(q) = make_float2(sign * c[0], sign * c[1]);
  if (bottom) *reinterpret_cast<float2*>(q + 8 * kLdA) = make_float2(sign * c[2], sign * c[3]);
}

// Barrier of a group of four warps.
__device__ __forceinline__ void bar_group(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
// The same, and whether ok holds for the whole group: where a wait runs out, its warps stop together.
__device__ __forceinline__ bool bar_group_all(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.and.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}
// A row of 256 bytes from shared to global memory by the copy engine.
__device__ __forceinline__ void bulk_row(void* dst, const void* src) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], 256;" ::"l"(dst), "r"(smem_u32(src))
               : "memory");
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
// 16 values of this lane's state (key dims i0 ..) as (s) left them: the old ones times the chunk's
// decay plus their change, rounded to nearest. Where the decay is slow it is applied as S + (e^G - 1) S:
// e^G rounded to fp32 would be off alike in every chunk of a constant gate (8192 rows of gate -3e-4
// put a state off by 8.7e-6).
__device__ __forceinline__ void get_state(uint32_t tl, int i0, const Gates& G, float* v) {
  float x[16];
  tmem_ld16(tl + kColS + i0, v);
  tmem_ld16(tl + kColDS + i0, x);
  tmem_ld_wait();
  const float2 f = *reinterpret_cast<const float2*>(&G.dec);
  const f32x2 d2 = pair(f.x, f.x), k2 = pair(f.y, f.y);
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const f32x2 s = pair(v[e], v[e + 1]);
    unpair(fma2(s, k2, fma2(s, d2, pair(x[e], x[e + 1]))), v[e], v[e + 1]);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
delta_prefill_tc_kernel(const __grid_constant__ CUtensorMap tq,
                        const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv,
                        const __grid_constant__ CUtensorMap to, __nv_bfloat16* __restrict__ out,
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
    if (cut_chains) pl = make_plan<kChainCost>([&](int b) { return chunks_of(in, b); }, B, in.H, P, p, lane);
    if (lane == 0) plan_sh = pl;
  }
  __syncthreads();
  if (plan_sh.head_u < 0 && plan_sh.tail_u < 0 && plan_sh.full_u0 >= plan_sh.full_u1) return;
  unsigned long long tag = 0;
  if (cut_chains)
    tag = (*reinterpret_cast<volatile unsigned long long*>(hs) << 32) | (grid_id() & 0xffffffffull);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  Bars* bars = reinterpret_cast<Bars*>(sm + kOffBar);
  Gates* gates = reinterpret_cast<Gates*>(sm + kOffG);
  Chunk* chunks = reinterpret_cast<Chunk*>(sm + kOffChunk);

  for (int e = tid; e < (kOffP - kOffW) / 16; e += kThreads)   // W: zero above the diagonal
    reinterpret_cast<uint4*>(sm + kOffW)[e] = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  if (warp == kWarpMma) {
    if (lane == 0) {
      for (int i = 0; i < kNKQ; ++i) {
        mbar_init(&bars->full_kq[i], 1);
        mbar_init(&bars->free_kq[i], 1);
      }
      mbar_init(&bars->full_v, 1);
      mbar_init(&bars->free_v, 256);
      for (int i = 0; i < 4; ++i) {
        mbar_init(&bars->info[i], 32);
        mbar_init(&bars->gates[i], 128);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars->w_ready[i], 128);
        mbar_init(&bars->o_free[i], 128);
        mbar_init(&bars->sa_ready[i], 256);
        mbar_init(&bars->ra_ready[i], 256);
        mbar_init(&bars->xa_ready[i], 256);
        mbar_init(&bars->d0_ready[i], 1);
      }
      mbar_init(&bars->d0_free, 128);
      mbar_init(&bars->d1k_ready, 1);
      mbar_init(&bars->d1q_ready, 1);
      mbar_init(&bars->x_ready, 1);
      mbar_init(&bars->s_ready, 1);
      mbar_init(&bars->q_scaled, 128);
      mbar_init(&bars->d1q_free, 128);
      mbar_init(&bars->o_ready, 1);
      mbar_init(&bars->om_ready, 256);
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

#define HYB_WAIT(bar, parity) __all_sync(0xffffffffu, mbar_wait_cycles(&(bar), (parity)))
  bool ok = true;
  if (warp < kWarpMain) {
    // ------------------------------------------------------------ preparation
    // two groups of four warps, each for every second chunk
    const int grp = warp >> 2, gw = warp & 3, gt = tid & 127, bar = 1 + grp;
    const int st = grp;
    float* A = reinterpret_cast<float*>(sm + kOffA) + grp * kC * kLdA;
    for (int c = grp;; c += 2) {
      Gates& G = gates[c & 3];
      ok = bar_group_all(bar, HYB_WAIT(bars->info[c & 3], (c >> 2) & 1));
      if (!ok) break;
      const int n = chunks[c & 3].n;
      if (n == 0) break;
      ok = HYB_WAIT(bars->full_kq[c % kNKQ], (c / kNKQ) & 1);
      {                                      // lengths: thread r, row r of the stacked [K; Q]
        const uint8_t* kq = sm + kOffKQ + (c % kNKQ) * kStageKQ + gt * 128;
        f32x2 s2 = pair(0.f, 0.f);
#pragma unroll 4
        for (int ch = 0; ch < 16; ++ch) {
          const uint4 u = *reinterpret_cast<const uint4*>(kq + (ch >> 3) * kSubKQ + (((ch & 7) ^ (gt & 7)) << 4));
          const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f32x2 y = pair(bf16_lo(x[e]), bf16_hi(x[e]));
            s2 = fma2(y, y, s2);
          }
        }
        float ss, s1;
        unpair(s2, ss, s1);
        ss += s1;
        const float inv = eps > 0.f ? 1.f / sqrtf(ss + eps) : 1.f;
        const int t = gt & 63;
        if (gt < 64) {
          const float rk = t < n ? inv : 0.f;
          G.wB[t] = G.bt[t] * rk;
          G.cA[t] = G.bt[t] * rk * rk;
          G.eR[t] = rk * exp2f(G.hi[t]);     // G.lo is below half an ulp of G.hi
          G.wX[t] = exp2f((G.hi[63] - G.hi[t]) + (G.lo[63] - G.lo[t]));
          if (t == 63) {
            constexpr float kLn2 = 0.693147181f;
            const float em1 = expm1f(fmaf(G.hi[63], kLn2, G.lo[63] * kLn2));
            const bool slow = em1 >= -0.5f;
            G.dec = slow ? em1 : exp2f(G.hi[63]);
            G.keep = slow ? 1.f : 0.f;
          }
        } else {
          const float f = t < n ? scale * inv : 0.f;
          G.pq[t] = f;
          G.oq[t] = f * exp2f(G.hi[t]);
        }
      }
      ok = bar_group_all(bar, ok);
      if (!ok) break;
      mbar_arrive(&bars->gates[c & 3]);
      ok = HYB_WAIT(bars->d0_ready[st], (c >> 1) & 1);
      if (c >= 2) ok = HYB_WAIT(bars->o_free[st], ((c - 2) >> 1) & 1) && ok;   // P's buffer
      tc_fence_after();
      {
        // warps 0, 1: row t of K K^T -> column t of A^T; warps 2, 3: row t of Q K^T -> row t of P.
        // Rows below 32 have nothing in the columns from 32 on.
        const int t = gt & 63;
        const bool is_p = gt >= 64;
        if (is_p && t < 32) {
          uint8_t* dst = sm + kOffP + st * 2 * kTile64 + t * 128;
#pragma unroll
          for (int ch = 4; ch < 8; ++ch) {
            *reinterpret_cast<uint4*>(dst + ((ch ^ (t & 7)) << 4)) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(dst + kTile64 + ((ch ^ (t & 7)) << 4)) = make_uint4(0, 0, 0, 0);
          }
        }
        const float ghi = G.hi[t], glo = G.lo[t], f = is_p ? G.pq[t] : G.cA[t];
        const f32x2 neg = pair(-1.f, -1.f), gh2 = pair(ghi, ghi), gl2 = pair(glo, glo), f2 = pair(f, f);
#pragma unroll 1
        for (int s0 = 0; s0 <= (t & 32) + 16; s0 += 16) {
          float v[16];
          tmem_ld16(tl + kCol0 + s0, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 h4 = *reinterpret_cast<const float4*>(&G.hi[s0 + e]);
            const float4 l4 = *reinterpret_cast<const float4*>(&G.lo[s0 + e]);
            float d[4];
            unpair(add2(fma2(pair(h4.x, h4.y), neg, gh2), fma2(pair(l4.x, l4.y), neg, gl2)), d[0], d[1]);
            unpair(add2(fma2(pair(h4.z, h4.w), neg, gh2), fma2(pair(l4.z, l4.w), neg, gl2)), d[2], d[3]);
            unpair(mul2(mul2(pair(fast_exp2(d[0]), fast_exp2(d[1])), f2), pair(v[e], v[e + 1])), v[e], v[e + 1]);
            unpair(mul2(mul2(pair(fast_exp2(d[2]), fast_exp2(d[3])), f2), pair(v[e + 2], v[e + 3])), v[e + 2], v[e + 3]);
          }
          if (s0 >= (t & 32)) {              // at the diagonal: s < t, or s <= t for P
            const int most = t - s0 + (is_p ? 1 : 0);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = e < most ? v[e] : 0.f;
          }
          if (!is_p) {
#pragma unroll
            for (int e = 0; e < 16; ++e) A[(s0 + e) * kLdA + t] = v[e];
          } else {
            uint8_t* dst = sm + kOffP + st * 2 * kTile64 + t * 128;
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
              uint32_t h[4], m[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) split2(v[ch * 8 + 2 * e], v[ch * 8 + 2 * e + 1], h[e], m[e]);
              const int off = ((s0 / 8 + ch) ^ (t & 7)) << 4;
              *reinterpret_cast<uint4*>(dst + off) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(dst + kTile64 + off) = make_uint4(m[0], m[1], m[2], m[3]);
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bars->d0_free);
      ok = bar_group_all(bar, ok);
      if (!ok) break;
      // W = (1 + A)^-1 by blocks of 8, 16, 32, 64. A is held transposed, A^T[s][t] at A[s * kLdA + t], W
      // row-major in its place. Two blocks W00, W11 on the diagonal and A10 below give
      // W10 = -W11 (A10 W00); the first product goes where W10 will be. What is left of A^T above the
      // diagonal blocks is never read as W: those products are skipped. The products are warp
      // MMAs of 16 x 8 x 8 on two tf32 terms (three products; the fourth, up to 2^-22, has either
      // sign): on the CUDA cores their
      // operands, broadcast from shared memory, took two thirds of its bandwidth.
      {
        // 8 x 8: a warp two blocks, a lane a column (lanes 16-31 do the same). Once w_m is final it is
        // taken from every later row.
        float* D = A + gw * 16 * (kLdA + 1);
        float* E = D + ((lane >> 3) & 1) * 8 * (kLdA + 1);
        const int col = lane & 7;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i == col ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < 7; ++m) {
#pragma unroll
          for (int i4 = (m + 1) / 4; i4 < 2; ++i4) {
            const float4 a = *reinterpret_cast<const float4*>(&E[m * kLdA + i4 * 4]);
            const float y[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (i4 * 4 + e > m) x[i4 * 4 + e] = fmaf(-y[e], x[m], x[i4 * 4 + e]);
          }
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
          for (int i = 0; i < 8; ++i) E[i * kLdA + col] = x[i];
        }
        __syncwarp();
        // 16 x 16, this warp's two blocks (rows 8-15 of the products are idle)
        FragA fa;
        FragB fb;
        float y[4] = {}, z[4] = {};
        fa.load<1, kLdA>(D + 8, lane, true, false);
        fb.load(D, lane);
        mma_tf32(y, fa, fb);
        store_c(D + 8 * kLdA, y, 1.f, lane, false);
        __syncwarp();
        fa.load<kLdA, 1>(D + 8 * (kLdA + 1), lane, true, false);
        fb.load(D + 8 * kLdA, lane);
        mma_tf32(z, fa, fb);
        __syncwarp();
        store_c(D + 8 * kLdA, z, -1.f, lane, false);
      }
      bar_group(bar);
      {                                      // 32 x 32: two warps each, 8 columns a warp
        float* D = A + (gw >> 1) * 32 * (kLdA + 1);
        const int j0 = 8 * (gw & 1);
        FragA fa;
        FragB fb;
        float y[4] = {}, z[4] = {};
        if (j0 == 0) {
          fa.load<1, kLdA>(D + 16, lane);
          fb.load(D, lane);
          mma_tf32(y, fa, fb);
        }
        fa.load<1, kLdA>(D + 8 * kLdA + 16, lane);
        fb.load(D + 8 * kLdA + j0, lane);
        mma_tf32(y, fa, fb);
        store_c(D + 16 * kLdA + j0, y, 1.f, lane);
        bar_group(bar);
        fa.load<kLdA, 1>(D + 16 * (kLdA + 1), lane);
        fb.load(D + 16 * kLdA + j0, lane);
        mma_tf32(z, fa, fb);
        fa.load<kLdA, 1>(D + 16 * (kLdA + 1) + 8, lane, false);   // rows 0-7 end before column 8
        fb.load(D + 24 * kLdA + j0, lane);
        mma_tf32(z, fa, fb);
        bar_group(bar);
        store_c(D + 16 * kLdA + j0, z, -1.f, lane);
      }
      bar_group(bar);
      {                                      // 64 x 64: each warp 16 rows by 16 columns
        const int r0 = 16 * (gw >> 1), j0 = 16 * (gw & 1);
        FragA fa;
        FragB fb;
        float y[2][4] = {}, z[2][4] = {};
#pragma unroll 1
        for (int m = j0; m < 32; m += 8) {
          fa.load<1, kLdA>(A + m * kLdA + 32 + r0, lane);
          fb.load(A + m * kLdA + j0, lane);
          mma_tf32(y[0], fa, fb);
          if (m > j0) {
            fb.load(A + m * kLdA + j0 + 8, lane);
            mma_tf32(y[1], fa, fb);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) store_c(A + (32 + r0) * kLdA + j0 + 8 * i, y[i], 1.f, lane);
        bar_group(bar);
#pragma unroll 1
        for (int m = 0; m <= r0 + 8; m += 8) {
          fa.load<kLdA, 1>(A + (32 + r0) * kLdA + 32 + m, lane, m <= r0);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            fb.load(A + (32 + m) * kLdA + j0 + 8 * i, lane);
            mma_tf32(z[i], fa, fb);
          }
        }
        // not back into its place, where others still read: over A21^T (rows r, columns 32-63)
#pragma unroll
        for (int i = 0; i < 2; ++i) store_c(A + r0 * kLdA + 32 + j0 + 8 * i, z[i], -1.f, lane);
      }
      // W has one buffer: (w) of the last chunk must have read it
      ok = bar_group_all(bar, c == 0 || HYB_WAIT(bars->x_ready, (c - 1) & 1));
      if (!ok) break;
      // W's columns times beta / |k|, as three bf16 terms: a warp 32 rows of one half of the columns
      // (the upper right block is zero from the start)
      if (gw != 1) {
        const int half = gw & 1, t = 32 * (gw >> 1) + lane;
        const float* src = A + (half == (gw >> 1) ? t * kLdA + 32 * half : lane * kLdA + 32);
        const bool diag = half == (gw >> 1);
        uint8_t* dst = sm + kOffW + t * 128;
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const float4 u = *reinterpret_cast<const float4*>(src + ch * 8 + e);
            const float4 f = *reinterpret_cast<const float4*>(&G.wB[half * 32 + ch * 8 + e]);
            v[e] = u.x * f.x; v[e + 1] = u.y * f.y; v[e + 2] = u.z * f.z; v[e + 3] = u.w * f.w;
          }
          if (diag && ch > (lane >> 3)) {    // above the diagonal blocks
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
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
    // Rows in two pieces of 16 (the lower half of the rows starts with its second, see R below).
    const int xa = x0 + (half ? 0 : 16), xb = x0 + (half ? 16 : 0);
    int n = 0, flags = 0;
    uint32_t v[16];                          // pairs of rows of V, this column
    // Chunk c's description and V: fetched while the chunk before is under way.
    auto fetch = [&](int c) -> bool {
      if (!HYB_WAIT(bars->info[c & 3], (c >> 2) & 1)) return false;
      n = chunks[c & 3].n;
      flags = chunks[c & 3].flags;
      if (n == 0) return true;
      if (!HYB_WAIT(bars->full_v, c & 1)) return false;
      const uint8_t* vs = sm + kOffV + (j >> 6) * kSubV + (j & 7) * 2;
      const int cj = (j & 63) >> 3;
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const uint8_t* r = vs + ((e < 16 ? xa : xb - 16) + e) * 128;   // pieces start at rows of 8
        const uint32_t lo = *reinterpret_cast<const uint16_t*>(r + ((cj ^ (e & 7)) << 4));
        const uint32_t hi = *reinterpret_cast<const uint16_t*>(r + 128 + ((cj ^ ((e + 1) & 7)) << 4));
        v[e / 2] = __byte_perm(lo, hi, 0x5410);
      }
      if (n < kC) {                          // rows past the request may hold anything
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const int t = (e < 16 ? xa : xb - 16) + e;
          if (t >= n) v[e / 2] = 0;
          else if (t + 1 >= n) v[e / 2] &= 0xffffu;
        }
      }
      mbar_arrive(&bars->free_v);
      return true;
    };
    ok = fetch(0);
    for (int c = 0; ok && n > 0; ++c) {
      const Gates& G = gates[c & 3];
      float* const S = chunks[c & 3].S;
      const bool last = flags & kLast, hand = flags & kHand;
      // this chunk's first state: the run's from the pool, or what the last chunk left in TMEM
      if ((flags & (kFirst | kTake)) == (kFirst | kTake)) {
        ok = take_handoff(hs + 1 + (p + 1), tag);
        if (!ok) break;
      }
      {
        const bool from_tmem = !(flags & kFirst), from_pool = !(flags & kZero);
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {        // pieces of 16 key dims; (k) starts with the first two
          const int i = i0 + 16 * x;
          float s[16];
          if (from_tmem) {
            get_state(tl, i, gates[(c - 1) & 3], s);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = from_pool ? __ldcg(S + (i + e) * kD + j) : 0.f;
          }
          put_terms(tl + kColSA + i, tl + kColSA + i + 8, tl + kColSA + 128 + i / 2, s);
          tmem_st16(tl + kColS + i, s);
          if (x & 1) {
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bars->sa_ready[x >> 1]);
          }
        }
      }
      // R = V - e^G K S (beta is in W)
      ok = HYB_WAIT(bars->gates[c & 3], (c >> 2) & 1) && HYB_WAIT(bars->d1k_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
      // R's l goes to columns 16-47 of D1K: the thread's own 16 first rows of d may lie there, so the
      // piece that lies apart from them is read second
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int t0 = x ? xb : xa;
        float d[16];
        tmem_ld16(tl + kCol1K + t0, d);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 a = *reinterpret_cast<const float4*>(&G.eR[t0 + e]);
          const uint32_t v0 = v[x * 8 + e / 2], v1 = v[x * 8 + e / 2 + 1];
          unpair(fma2(pair(-a.x, -a.y), pair(d[e], d[e + 1]), pair(bf16_lo(v0), bf16_hi(v0))), d[e], d[e + 1]);
          unpair(fma2(pair(-a.z, -a.w), pair(d[e + 2], d[e + 3]), pair(bf16_lo(v1), bf16_hi(v1))), d[e + 2], d[e + 3]);
        }
        put_terms(tl + kColRh + t0 / 2, tl + kColRm + t0 / 2, tl + kColRl + t0 / 2, d);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars->ra_ready[x]);
      }
      ok = fetch(c + 1);
      if (!ok) break;
      // X: times its way to the chunk's end for the state, and as it is for the outputs. All of it is
      // read before the first half is announced: the state's change goes over it. V's buffer is
      // free for X's second term once all have fetched from it.
      ok = HYB_WAIT(bars->x_ready, c & 1) && HYB_WAIT(bars->free_v, (c + (n > 0)) & 1);
      if (!ok) break;
      tc_fence_after();
      {
        float d[16];
        tmem_ld16(tl + kColX + x0, d);
        tmem_ld_wait();
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          const int at = x0 / 2 + 8 * x;
          uint32_t h[8], m[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) split2(d[2 * e], d[2 * e + 1], h[e], m[e]);
          tmem_st8u(tl + kColOh + at, h);
          uint8_t* om = sm + kOffV + j * 128;
          *reinterpret_cast<uint4*>(om + (((at >> 2) ^ (j & 7)) << 4)) = make_uint4(m[0], m[1], m[2], m[3]);
          *reinterpret_cast<uint4*>(om + ((((at >> 2) + 1) ^ (j & 7)) << 4)) = make_uint4(m[4], m[5], m[6], m[7]);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 a = *reinterpret_cast<const float4*>(&G.wX[x0 + 16 * x + e]);
            unpair(mul2(pair(a.x, a.y), pair(d[e], d[e + 1])), d[e], d[e + 1]);
            unpair(mul2(pair(a.z, a.w), pair(d[e + 2], d[e + 3])), d[e + 2], d[e + 3]);
          }
          put_terms(tl + kColXh + at, tl + kColXm + at, tl + kColXl + at, d);
          if (x == 0) {
            tmem_ld16(tl + kColX + x0 + 16, d);
            tmem_ld_wait();
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&bars->xa_ready[x]);
        }
      }
      fence_async_smem();
      mbar_arrive(&bars->om_ready);
      // the chunk's last state
      ok = HYB_WAIT(bars->s_ready, c & 1);
      if (!ok) break;
      tc_fence_after();
      if (last) {                            // end of a run: to the pool, and handed over if cut
#pragma unroll 1
        for (int i = i0; i < i0 + 64; i += 16) {
          float s[16];
          get_state(tl, i, G, s);
#pragma unroll
          for (int e = 0; e < 16; ++e) S[(i + e) * kD + j] = s[e];
        }
        if (hand) {                          // at most once per CTA (its first run)
          __threadfence();
          mbar_arrive(&bars->published);
          if (tid == kWarpMain * 32) {
            if (mbar_wait(&bars->published, 0)) st_release_u64(hs + 1 + p, tag);
            else flag(status, HYB_DEVERR_TIMEOUT);
          }
          __syncwarp();
        }
      }
    }
    if (!ok && lane == 0) flag(status, HYB_DEVERR_TIMEOUT);
  } else if (warp < kWarpFeed) {
    // ------------------------------------------------------------ outputs
    const int j = (warp & 3) * 32 + lane, ot = tid - kWarpOut * 32;
    for (int c = 0;; ++c) {
      const int st = c & 1;
      const Gates& G = gates[c & 3];
      ok = bar_group_all(3, HYB_WAIT(bars->info[c & 3], (c >> 2) & 1));
      if (!ok) break;
      const int n = chunks[c & 3].n;
      if (n == 0) break;
      const int row = chunks[c & 3].row, h = chunks[c & 3].h;
      ok = HYB_WAIT(bars->gates[c & 3], (c >> 2) & 1) && HYB_WAIT(bars->d1q_ready, c & 1);
      tc_fence_after();
      // Q S times scale e^G / |q|, in place; (o) adds to it
#pragma unroll 1
      for (int x = 0; x < 64; x += 16) {
        float d[16];
        tmem_ld16(tl + kCol1Q + x, d);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&G.oq[x + e]);
          unpair(mul2(pair(f.x, f.y), pair(d[e], d[e + 1])), d[e], d[e + 1]);
          unpair(mul2(pair(f.z, f.w), pair(d[e + 2], d[e + 3])), d[e + 2], d[e + 3]);
        }
        tmem_st16(tl + kCol1Q + x, d);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars->q_scaled);
      ok = bar_group_all(3, ok && HYB_WAIT(bars->o_ready, c & 1));
      if (!ok) break;
      tc_fence_after();
      // rows of 256 bytes in the place of P, which (o) has used up, and from there to global memory
      uint8_t* rows = sm + kOffP + st * 2 * kTile64;
#pragma unroll 1
      for (int x = 0; x < 64; x += 16) {
        float d[16];
        tmem_ld16(tl + kCol1Q + x, d);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const uint32_t y = pack_bf16(d[e], d[e + 1]);
          *reinterpret_cast<uint16_t*>(rows + (x + e) * 256 + j * 2) = (uint16_t)y;
          *reinterpret_cast<uint16_t*>(rows + (x + e + 1) * 256 + j * 2) = (uint16_t)(y >> 16);
        }
      }
      tc_fence_before();
      mbar_arrive(&bars->d1q_free);
      fence_async_smem();
      bar_group(3);
      // a whole chunk in one store; of the last, partial one only the request's rows, one by one
      if (n == kC ? ot == 0 : ot < n) {
        if (n == kC) tma_store_3d(&to, rows, 0, h, row);
        else bulk_row(out + ((int64_t)(row + ot) * in.H + h) * kD, rows + ot * 256);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      }
      mbar_arrive(&bars->o_free[st]);
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok && lane == 0) flag(status, HYB_DEVERR_TIMEOUT);
  } else if (warp == kWarpFeed) {
    // ------------------------------------------------------------ chunks, loads, gates
    if (lane == 0) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
    }
    Walk w;
    bool more = true, ended = false;
    int ckq = 0, cv = 0;                     // chunks requested
    for (int c = 0;; ++c) {
      if (more) more = next_chunk(in, plan_sh, w);
      const int st = c % kNKQ, row = more ? w.sg.t0 + w.ci * kC : 0;
      const int n = more ? min(kC, w.sg.n - w.ci * kC) : 0;
      // gates and betas of rows lane and lane + 32
      const int head = more ? w.sg.h : 0;
      const int64_t at = (int64_t)row * in.H + head + (int64_t)lane * in.H, at2 = at + 32ll * in.H;
      const float ga = lane < n ? g[at] : 0.f, gb = lane + 32 < n ? g[at2] : 0.f;
      const float ba = lane < n ? beta[at] : 0.f, bb = lane + 32 < n ? beta[at2] : 0.f;
      // running sum in units of log 2, exact in integer steps of 2^-36 (fp32 would lose the
      // small gates behind large ones, and fp64 is slow on this GPU)
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
      float h0, l0, h1, l1;
      from_fixed(a, (na & upto) != 0, h0, l0);
      from_fixed(b, na != 0 || (nb & upto) != 0, h1, l1);
      if (c >= kNKQ) ok = HYB_WAIT(bars->free_kq[c % kNKQ], (c / kNKQ - 1) & 1);
      if (!ok) break;
      Gates& G = gates[c & 3];
      G.hi[lane] = h0;
      G.lo[lane] = l0;
      G.hi[lane + 32] = h1;
      G.lo[lane + 32] = l1;
      G.bt[lane] = ba;
      G.bt[lane + 32] = bb;
      if (lane == 0) {
        const int flags = !more ? 0 : (w.ci == w.sg.c0 ? kFirst | (w.sg.zero_start ? kZero : 0) | (w.sg.wait_handoff ? kTake : 0) : 0) |
                          (w.ci == w.sg.c1 - 1 ? kLast | (w.sg.publish ? kHand : 0) : 0);
        chunks[c & 3] = Chunk{more ? w.sg.S : nullptr, row, n, head, flags, {0, 0}};
      }
      if (n > 0) {
        const int hk = head / rep;
        if (lane == 0) {
          uint8_t* kq = sm + kOffKQ + st * kStageKQ;
          mbar_expect_tx(&bars->full_kq[st], kStageKQ);
          for (int sb = 0; sb < 2; ++sb) {
            tma_load_3d(kq + sb * kSubKQ, &tk, sb * 64, hk, row, &bars->full_kq[st]);
            tma_load_3d(kq + sb * kSubKQ + 64 * 128, &tq, sb * 64, hk, row, &bars->full_kq[st]);
          }
        }
        ckq = c + 1;
      }
      mbar_arrive(&bars->info[c & 3]);
      if (n > 0) {
        if (c == 1) ok = HYB_WAIT(bars->free_v, 0);
        if (c >= 2) ok = HYB_WAIT(bars->o_ready, c & 1);   // (o) of chunk c - 2 has read X's terms
        if (!ok) break;
        if (lane == 0) {
          uint8_t* vs = sm + kOffV;
          mbar_expect_tx(&bars->full_v, kStageV);
          for (int sb = 0; sb < 2; ++sb)
            tma_load_3d(vs + sb * kSubV, &tv, sb * 64, head, row, &bars->full_v);
        }
        cv = c + 1;
      }
      if (ended) break;                      // two end marks: each preparing group gets one
      ended = n == 0;
    }
    if (!ok && lane == 0) {                  // let the loads in flight land before exiting
      flag(status, HYB_DEVERR_TIMEOUT);
      for (int i = max(0, ckq - kNKQ); i < ckq; ++i)
        mbar_wait(&bars->full_kq[i % kNKQ], (i / kNKQ) & 1, 100000000ull);
      if (cv > 0) mbar_wait(&bars->full_v, (cv - 1) & 1, 100000000ull);
    }
  } else {
    // ------------------------------------------------------------ MMAs
    const uint32_t sm0 = smem_u32(sm);
    const uint64_t km0 = sw128_desc(sm0, 16, 1024);            // K-major operands
    const uint64_t mn0 = sw128_desc(sm0, kSubKQ, 1024);        // K as [t][i], i-major: two 64-wide blocks
    int end = 0x7fffffff;                    // number of chunks, once it is known
    // (0) of chunk cn, if there is one: rows past the request become zero rows of K first
    auto issue0 = [&](int cn) -> bool {
      if (cn >= end) return true;
      if (!HYB_WAIT(bars->info[cn & 3], (cn >> 2) & 1)) return false;
      const int n = chunks[cn & 3].n, st = cn % kNKQ;
      if (n == 0) {
        end = cn;
        return true;
      }
      if (!HYB_WAIT(bars->full_kq[st], (cn / kNKQ) & 1)) return false;
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
        tc_commit(&bars->d0_ready[cn & 1]);
      }
      __syncwarp();
      return true;
    };
    ok = issue0(0) && issue0(1);             // two chunks ahead
    for (int c = 0; ok && c < end; ++c) {
      const uint32_t kq = kOffKQ + (c % kNKQ) * kStageKQ;
      for (int x = 0; x < 2; ++x) {          // (k): key dims 0-31 and 64-95, then the others
        ok = HYB_WAIT(bars->sa_ready[x], c & 1);
        if (!ok) break;
        if (elect_one()) {
          tc_fence_after();
#pragma unroll
          for (int y = 0; y < 12; ++y) {
            const int k = (y & 1) + ((y & 2) << 1) + 2 * x, term = 2 - (y >> 2);
            tc_mma_ta(tmem + kCol1K, tmem + kColSA + (term == 2 ? 128 + k * 8 : k * 16 + term * 8), desc_add(km0, kq + (k >> 2) * kSubKQ + (k & 3) * 32), kIdesc64, x + y > 0);
          }
          if (x == 1) tc_commit(&bars->d1k_ready);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (c >= 1) ok = HYB_WAIT(bars->d1q_free, (c - 1) & 1);
      if (!ok) break;
      if (elect_one()) {
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 16; ++x) {       // (q)
          const int k = x & 7;
          tc_mma_ta(tmem + kCol1Q, tmem + kColSA + k * 16 + (x >> 3) * 8, desc_add(km0, kq + 64 * 128 + (k >> 2) * kSubKQ + (k & 3) * 32), kIdesc64, x > 0);
        }
        tc_commit(&bars->d1q_ready);
      }
      __syncwarp();
      ok = HYB_WAIT(bars->w_ready[c & 1], (c >> 1) & 1);
      if (!ok) break;
      for (int x = 0; x < 2; ++x) {          // (w): rows 16-47, then the others
        ok = HYB_WAIT(bars->ra_ready[x], c & 1);
        if (!ok) break;
        if (elect_one()) {
          tc_fence_after();
          const uint64_t wd = desc_add(km0, kOffW);
#pragma unroll
          for (int y = 0; y < 6; ++y) {      // R l W h, m m, h l, m h, h m, h h
            const int r = y == 3 || y == 1 ? 1 : y == 0 ? 2 : 0, t = y == 4 || y == 1 ? 1 : y == 2 ? 2 : 0;
            const uint32_t ra = r == 0 ? kColRh : r == 1 ? kColRm : kColRl;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int k = x == 0 ? 1 + z : 3 * z;
              tc_mma_ta(tmem + kColX, tmem + ra + k * 8, desc_add(wd, t * kTile64 + k * 32), kIdesc64, x + y + z > 0);
            }
          }
          if (x == 1) tc_commit(&bars->x_ready);
        }
        __syncwarp();
      }
      ok = ok && issue0(c + 2);
      if (!ok) break;
      for (int x = 0; x < 2; ++x) {          // (s): rows 0-15 and 32-47, then the others
        ok = HYB_WAIT(bars->xa_ready[x], c & 1);
        if (!ok) break;
        if (elect_one()) {
          tc_fence_after();
#pragma unroll
          for (int y = 0; y < 6; ++y) {
            const int k = x + 2 * (y & 1);
            const uint32_t xt = y < 2 ? kColXl : y < 4 ? kColXm : kColXh;
            tc_mma_ta(tmem + kColDS, tmem + xt + k * 8, desc_add(mn0, kq + k * 2048), kIdescS, x + y > 0);
          }
          if (x == 1) {
            tc_commit(&bars->s_ready);
            tc_commit(&bars->free_kq[c % kNKQ]);   // the last use of K and Q
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      ok = HYB_WAIT(bars->q_scaled, c & 1) && HYB_WAIT(bars->om_ready, c & 1);
      if (!ok) break;
      if (elect_one()) {
        tc_fence_after();
        const uint64_t pd = desc_add(km0, kOffP + (c & 1) * 2 * kTile64);
#pragma unroll
        for (int x = 0; x < 3; ++x) {        // (o): X h P h, h m, m h
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (x == 2) tc_mma(tmem + kCol1Q, desc_add(km0, kOffV + k * 32), desc_add(pd, k * 32), kIdesc64, 1);
            else tc_mma_ta(tmem + kCol1Q, tmem + kColOh + k * 8, desc_add(pd, x * kTile64 + k * 32), kIdesc64, 1);
          }
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
  CUtensorMap mq, mk, mv, mo;
  const uint64_t rows = T > 0 ? T : 1;
  auto encode = [&](CUtensorMap* m, const void* base, int heads, int64_t stride, bool store = false) {
    const uint64_t dims[3] = {(uint64_t)kD, (uint64_t)heads, rows};
    const uint64_t strides[2] = {(uint64_t)kD * 2, (uint64_t)stride * 2};
    const uint32_t box[3] = {store ? 128u : 64u, 1, kC};
    return encode_tmap_bf16(m, base, 3, dims, strides, box, !store);
  };
  if (!encode(&mq, q, Hk, qs) || !encode(&mk, k, Hk, ks) || !encode(&mv, v, Hv, vs) ||
      !encode(&mo, out, Hv, (int64_t)Hv * kD, true))
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
  e = cudaLaunchKernelEx(&cfg, delta_prefill_tc_kernel, mq, mk, mv, mo, static_cast<__nv_bfloat16*>(out),
                         g, beta, in, B, Hv / Hk, d->scale, d->qk_norm_eps,
                         static_cast<unsigned long long*>(ws), cut_chains, status);
  count_launch();
  return e;
}

}  // namespace hyb
