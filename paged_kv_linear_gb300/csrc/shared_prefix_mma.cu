// Parts of shared-prefix decode attention, bf16, D = 64, 128 or 256, on warp matrix instructions:
// a part's keys are streamed once for 16 NT query rows (the rows of a group times the query heads
// of one key head), or for one request's query heads, its own tokens.
//
// Per 16-token piece of the cache, with Q the rows as A fragments in registers:
//   S = Q K^T (16 x 16 a warp), p = 2^(scale S - m), O += P V
// all in registers: S's accumulators are the A fragment of P V. K and V come by TMA, one box a piece of all D
// columns, 128-byte swizzled, so that ldmatrix meets no bank twice. The base m moves only when a row's maximum
// outgrows it by 2^8. P is rounded to bf16 for the product, half a step of each weight, as in the causal prefill; its
// sum is not. (P in two bf16 terms, 2^-17: 63 -> 68 us for 16 prompts of 8, 46 -> 59 us for 64 rows on 8192 tokens.)
//
// NT row tiles, one a warp, read a stage together; the other 4 / NT warps take other stages (key groups) through
// rings of their own, and join at the end. Each ring is filled by a warp that reads it. 64 KiB of rings let three CTAs
// share an SM (96 KiB and two: 64 rows 48 -> 64 us, 16 prompts of 8 63 -> 78 us), 168 registers do too. Stages of 64
// tokens for four row tiles, whose warps are bound by a step's own latency (32: 48 -> 46.5 us), of 32 for two (16: 62.7
// -> 63.9 us), of 16 for one, which waits for memory in any case.
//
// 16 prompts of 8, 32 query and 8 key heads, up to 8192 tokens: 60 us, 5.5 TB/s, 0.81 of the copy rate (issue slots
// 20 % busy, tensor pipe 22 %): it waits for memory, and for the start of its CTAs (group, then lengths and the part's
// block ids, then queries and keys: three round trips, 4 us). 32 groups of 4 rows, 8 key heads
// of 8192 tokens (1.08 GB) run at 0.96.
#include <cuda_bf16.h>

#include <type_traits>

#include "shared_prefix.cuh"
#include "tc.cuh"

namespace hyb {
namespace {

constexpr int kWarps = 4;
constexpr float kRescale = 8.f;                // log2: the largest p before the base moves
constexpr float kNoBase = -3.3e38f;            // the base of a row that has seen no key

constexpr int kPieces = kMmaMaxPart / kBlockSize;
static_assert(kPieces % 32 == 0, "a part's pieces are looked up by whole warps, in stages of up to four");

template <int D, int NT>
struct MmaShape {
  static constexpr int KG = kWarps / NT;       // key groups: rings of stages, each read by NT warps
  static constexpr int KP = NT == 1 ? 1 : NT == 4 && D <= 128 ? 4 : 2;   // pieces of a stage
  static constexpr int TILE = 16 * D * 2;      // K or V of a piece
  static constexpr int FIT = 65536 / (KG * KP * 2 * TILE);
  static constexpr int NST = FIT > 2 ? FIT : 2;
  static constexpr int LAG = NT == 1 || NST < 4 ? 0 : 1;
  static constexpr int RING = KG * NST * KP * 2 * TILE;
  static constexpr int PITCH = D + 8;          // floats of a row where key groups are joined
  static constexpr int JOIN = kWarps * 16 * PITCH * 4;
  static constexpr int BODY = KG > 1 && JOIN > RING ? JOIN : RING;
  static constexpr int BARS = BODY;            // full, empty: u64 [KG][NST]; have: int [KG][NST]
  static constexpr int ROWS = (BARS + KG * NST * 20 + 15) / 16 * 16;   // float2 ml[64]
  static constexpr int PIECES = ROWS + 64 * 8; // int [kPieces]
  static constexpr int UNIT = PIECES + kPieces * 4;              // Unit
  static constexpr int SMEM = UNIT + 64 + 1024;                 // 1 KiB of alignment slack
};

template <int D>
struct OwnShape {
  static constexpr int TILE = 16 * D * 2;
  static constexpr int NST = 16384 / (2 * TILE) > 2 ? 16384 / (2 * TILE) : 2;
  static constexpr int RING = kWarps * NST * 2 * TILE;
  static constexpr int SMEM = RING + kWarps * NST * 8 + 1024;
};

// What a CTA (of a request's own tokens: a warp) works on: rows row0 .. row0 + rows - 1 of those of key head hk
// from request first on (row i: request first + i / rep, query head hk rep + i % rep), keys [k0, k1) through `table`.
struct Unit {
  const int32_t* table;
  int first, hk, row0, rows, part, k0, k1;
};
static_assert(sizeof(Unit) <= 64, "what MmaShape sets aside");

// four 8 x 8 matrices at addr + OFF (an immediate), as they are or transposed
template <int OFF>
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF));
}
template <int OFF>
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF));
}
// f(0), f(1), ... with the number as a constant
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<N, I + 1>(f);
  }
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A warp's 16 query rows against pieces of 16 keys: rows lane / 4 and lane / 4 + 8, key or column pairs
// lane % 4 of every 8.
template <int D>
struct WarpTile {
  static constexpr int TILE = 16 * D * 2;
  uint32_t qa[D / 16][4];
  float o[D / 8][4], m[2], l[2];
  int lo0, hi0, lo1, hi1;              // keys that the two rows see

  // sign: turns q's sign bits where the scale is negative
  __device__ __forceinline__ void start(const __nv_bfloat16* q0, const __nv_bfloat16* q1, uint32_t sign) {
    const int quad = threadIdx.x & 3;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const int c = k * 16 + quad * 2;
      qa[k][0] = q0 ? *reinterpret_cast<const uint32_t*>(q0 + c) ^ sign : 0u;
      qa[k][1] = q1 ? *reinterpret_cast<const uint32_t*>(q1 + c) ^ sign : 0u;
      qa[k][2] = q0 ? *reinterpret_cast<const uint32_t*>(q0 + c + 8) ^ sign : 0u;
      qa[k][3] = q1 ? *reinterpret_cast<const uint32_t*>(q1 + c + 8) ^ sign : 0u;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
    m[0] = m[1] = kNoBase;
    l[0] = l[1] = 0.f;
    lo0 = hi0 = lo1 = hi1 = 0;
  }

  // KP pieces (16 KP tokens from tok on) at kt, each K, then V. Only keys [k0, k1) are there, and of the
  // pieces only those of the mask `have`; keys in [max_lo, min_hi) are seen by every row.
  template <int KP>
  __device__ __forceinline__ void step(int tok, uint8_t* kt, unsigned have, int k0, int k1, int min_hi, int max_lo,
                                       float scale_log2) {
    const int lane = threadIdx.x & 31, quad = lane & 3;
    // a lane's row and 16-byte chunk in the four 8 x 8 matrices of a load
    const int krow = (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;
    const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vch = lane >> 4;
    constexpr int kKeys = KP * kBlockSize, NC = KP == 1 ? 2 : 1;     // chains of sums per 8 keys
    // Chunk 2 k + kch of row krow lies at ((2 k + kch) ^ (krow & 7)) * 16 of its 128 bytes. The stage lies on
    // 1 KiB, so the k-th address is the first with bits 5 and 6 turned by k % 4, and the
    // rest an immediate.
    const uint32_t ks = smem_u32(kt) + sw128_off(krow, kch), vs = smem_u32(kt) + TILE + sw128_off(vrow, vch);
    const uint32_t ka[4] = {ks, ks ^ 32u, ks ^ 64u, ks ^ 96u}, va[4] = {vs, vs ^ 32u, vs ^ 64u, vs ^ 96u};
    float s[NC][2 * KP][4];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[n][i][c] = 0.f;
    each<D / 16 * KP>([&](auto n) {
      constexpr int k = n / KP, j = n % KP;
      uint32_t b[4];
      ldsm4<j * 2 * TILE + (k / 4) * 2048>(ka[k % 4], b);
      mma16816(s[k % NC][2 * j], qa[k], b[0], b[1]);
      mma16816(s[k % NC][2 * j + 1], qa[k], b[2], b[3]);
    });
    float x[2 * KP][4];
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[i][c] = NC == 2 ? s[0][i][c] + s[NC - 1][i][c] : s[0][i][c];
    const bool edge = tok < k0 || tok + kKeys > k1 || have != (1u << KP) - 1;
    if (edge || tok < max_lo || tok + kKeys > min_hi) {
#pragma unroll
      for (int i = 0; i < 2 * KP; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int key = tok + i * 8 + quad * 2 + (c & 1);
          const bool see = ((have >> (i / 2)) & 1) && key >= k0 && key < k1 &&
                           (c < 2 ? key >= lo0 && key < hi0 : key >= lo1 && key < hi1);
          if (!see) x[i][c] = -INFINITY;
        }
      if (edge) {
        // rows that hold no key of the part may hold NaN, and 0 x NaN is NaN (every warp that
        // reads the stage writes the same zeros first)
        for (int e = lane; e < kKeys * D / 8; e += 32) {
          const int r = e / (D / 8), ch = e % (D / 8);
          if (tok + r < k0 || tok + r >= k1 || !((have >> (r / kBlockSize)) & 1))
            *reinterpret_cast<uint4*>(kt + (r / kBlockSize) * 2 * TILE + TILE + (ch >> 3) * 2048 +
                                      (r % kBlockSize) * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();                // the ring's next copy comes after these writes
        __syncwarp();
      }
    }
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i) {
      mx0 = fmaxf(mx0, fmaxf(x[i][0], x[i][1]));
      mx1 = fmaxf(mx1, fmaxf(x[i][2], x[i][3]));
    }
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
    }
    mx0 *= scale_log2;                     // (scale > 0 keeps the order)
    mx1 *= scale_log2;
    // the base moves only where a row's maximum outgrows it: p stays below 2^8
    const bool g0 = mx0 > m[0] + kRescale, g1 = mx1 > m[1] + kRescale;
    if (__any_sync(0xffffffffu, g0 || g1)) {
      const float a0 = g0 ? fast_exp2(m[0] - mx0) : 1.f, a1 = g1 ? fast_exp2(m[1] - mx1) : 1.f;
      if (g0) m[0] = mx0;
      if (g1) m[1] = mx1;
      l[0] *= a0;
      l[1] *= a1;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= a0;
        o[i][1] *= a0;
        o[i][2] *= a1;
        o[i][3] *= a1;
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * KP; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[i][c] = fast_exp2(fmaf(x[i][c], scale_log2, -m[c / 2]));
      l[0] += x[i][0] + x[i][1];
      l[1] += x[i][2] + x[i][3];
    }
#pragma unroll
    for (int j = 0; j < KP; ++j) {
      // P as bf16: half a step of each weight
      const uint32_t pa[4] = {pack_bf16(x[2 * j][0], x[2 * j][1]), pack_bf16(x[2 * j][2], x[2 * j][3]),
                              pack_bf16(x[2 * j + 1][0], x[2 * j + 1][1]), pack_bf16(x[2 * j + 1][2], x[2 * j + 1][3])};
      each<D / 16>([&](auto kk) {
        constexpr int k = kk;
        uint32_t b[4];
        ldsm4_t<(k / 4) * 2048>(va[k % 4] + j * 2 * TILE, b);
        mma16816(o[2 * k], pa, b[0], b[1]);
        mma16816(o[2 * k + 1], pa, b[2], b[3]);
      });
    }
  }

  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
    }
    if (m[0] == kNoBase) m[0] = -INFINITY;
    if (m[1] == kNoBase) m[1] = -INFINITY;
  }
};

// The pool row of 16-token piece `sub` of a sequence, block id pb; -1, and flagged, for a bad block
__device__ __forceinline__ int pool_row(const PrefixArgs& a, int pb, int hk, int sub) {
  if (pb < 0 || pb >= a.NB) {
    flag(a.status, HYB_DEVERR_BAD_BLOCK);
    return -1;
  }
  return ((pb * a.Hk + hk) << (4 + a.rsh)) + ((sub & ((1 << a.rsh) - 1)) << 4);
}

// Fills a ring of NST pieces with pieces [sub0, sub0 + subs) of a sequence, by a whole warp.
template <int D, int NST>
struct Fetch {
  static constexpr int TILE = 16 * D * 2;
  const int32_t* table;
  uint8_t* ring;
  uint64_t* full;
  int hk, sub0, subs;
  int y, next;                               // pool rows of 32 pieces, one a lane; the piece to ask for next

  // asks for the next piece; returned: whether there is one (a bad block's is left out)
  __device__ __forceinline__ bool issue(const PrefixArgs& a, const CUtensorMap* tk, const CUtensorMap* tv) {
    const int lane = threadIdx.x & 31;
    if (next % 32 == 0) {
      y = -1;
      const int sub = sub0 + next + lane;
      if (next + lane < subs) y = pool_row(a, table[sub >> a.rsh], hk, sub);
    }
    const int st = next % NST, row = __shfl_sync(0xffffffffu, y, next % 32);
    if (row >= 0 && lane == 0) {
      uint8_t* dst = ring + st * 2 * TILE;
      mbar_expect_tx(&full[st], 2 * TILE);
      tma_load_3d(dst, tk, 0, row, 0, &full[st]);
      tma_load_3d(dst + TILE, tv, 0, row, 0, &full[st]);
    } else if (lane == 0) {
      mbar_arrive(&full[st]);
    }
    ++next;
    return row >= 0;
  }
};

// One warp's part of a request's own tokens: its ring of pieces is its own, filled by its lane 0. A key head a warp:
// 64 requests of 512 tokens, 32 heads 34 us (the plain decode's 35); two or four heads one after the other in a warp
// were slower (38, 61), and a CTA's four warps on one head, which have to join, too (64 requests of up to 2048: 153 -> 111 us).
template <int D>
__device__ __forceinline__ void attend_own(const CUtensorMap* tk, const CUtensorMap* tv,
                                           const __nv_bfloat16* __restrict__ q, const PrefixArgs& a, const Unit& u,
                                           int own_lo, uint8_t* sm) {
  constexpr int TILE = 16 * D * 2, NST = OwnShape<D>::NST;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rep = a.Hq / a.Hk;
  uint8_t* ring = sm + warp * NST * 2 * TILE;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + OwnShape<D>::RING) + warp * NST;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < NST; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  const int k0 = max(u.k0, own_lo), k1 = u.k1, np = (k1 - u.k0 + kBlockSize - 1) / kBlockSize;
  WarpTile<D> w;
  const int r0 = lane >> 2, r1 = r0 + 8, quad = lane & 3;
  const int64_t row = (int64_t)u.first * a.Hq + u.hk * rep + u.row0;
  w.start(r0 < u.rows ? q + (row + r0) * D : nullptr, r1 < u.rows ? q + (row + r1) * D : nullptr, a.q_sign);
  w.lo0 = w.lo1 = k0;
  w.hi0 = w.hi1 = k1;
  Fetch<D, NST> f{u.table, ring, full, u.hk, u.k0 / kBlockSize, np, -1, 0};
  unsigned have = 0;                     // of the pieces in the ring, by stage
  auto issue = [&]() {
    const int st = f.next % NST;
    have = (have & ~(1u << st)) | (unsigned)f.issue(a, tk, tv) << st;
  };
  while (f.next < NST && f.next < np) issue();
  for (int i = 0; i < np; ++i) {
    const int st = i % NST;
    if (!__all_sync(0xffffffffu, mbar_wait_cycles(&full[st], (i / NST) & 1))) {
      if (lane == 0) {                   // report, and let the copies in flight land
        flag(a.status, HYB_DEVERR_TIMEOUT);
        for (int j = i; j < f.next; ++j) mbar_wait_cycles(&full[j % NST], (j / NST) & 1, 200000000u);
      }
      break;
    }
    if ((have >> st) & 1)
      w.template step<1>(u.k0 + i * kBlockSize, ring + st * 2 * TILE, 1u, k0, k1, k1, k0, a.scale_log2);
    __syncwarp();
    if (f.next < np) issue();
  }
  w.finish();
  const int parts = a.Sp + a.Ss;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = half ? r1 : r0;
    if (r >= u.rows) continue;
    const int64_t at = (row + r) * parts + u.part;
    if (quad == 0) a.ws_ml[at] = make_float2(w.m[half], w.l[half]);
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      *reinterpret_cast<float2*>(a.ws_acc + at * D + i * 8 + quad * 2) = make_float2(w.o[i][2 * half], w.o[i][2 * half + 1]);
  }
}

template <int D, int NT>
__device__ __forceinline__ void attend(const CUtensorMap* tk, const CUtensorMap* tv,
                                       const __nv_bfloat16* __restrict__ q, const PrefixArgs& a, const Unit& u,
                                       int P, uint8_t* sm) {
  using S = MmaShape<D, NT>;
  constexpr int KG = S::KG, NST = S::NST, KP = S::KP, TILE = S::TILE;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::BARS);
  uint64_t* empty = full + KG * NST;
  int* have_s = reinterpret_cast<int*>(empty + KG * NST);
  float2* red_ml = reinterpret_cast<float2*>(sm + S::ROWS);
  int* pieces = reinterpret_cast<int*>(sm + S::PIECES);         // pool rows of the part's pieces; -1: left out
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rep = a.Hq / a.Hk;
  // with four row tiles registers are short in the loop: the end reads the unit here (64 requests 85.7 -> 85.0 us; with
  // one row tile it costs 0.5 of 18)
  Unit* const us = reinterpret_cast<Unit*>(sm + S::UNIT);
  if (tid == 96) {
    if (NT == 4) *us = u;
    for (int i = 0; i < KG * NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], NT);
    }
    fence_mbar_init();
  }
  int k0 = u.k0, k1 = u.k1;
  const int b0 = u.first + u.row0 / rep, b1 = u.first + (u.row0 + u.rows - 1) / rep + 1;
  Hull seen;                                   // only keys that one of the rows sees
  auto see = [&]() {
    for (int b = b0 + lane; b < b1; b += 32) seen.add(a, a.lens[b], P);
    seen.join();
    k0 = max(k0, seen.lo);
    k1 = min(k1, seen.hi);
    return k0 < k1;                            // (the same in every warp)
  };
  if (a.window > 0 && !see()) return;
  __syncthreads();
  const int kb = k0 & ~(kBlockSize - 1);

  // warp t = 0 of a key group fills its ring: stage n + NST - LAG once all have done with stage n - LAG
  const int t = warp % NT, kg = warp / NT;     // row tile, key group
  uint8_t* ring = sm + kg * NST * KP * 2 * TILE;
  full += kg * NST;
  empty += kg * NST;
  have_s += kg * NST;
  const int r0 = t * 16 + (lane >> 2), r1 = r0 + 8, quad = lane & 3;
  const __nv_bfloat16 *q0 = nullptr, *q1 = nullptr;
  if (r0 < u.rows) {
    const int i = u.row0 + r0;
    q0 = q + ((int64_t)(u.first + i / rep) * a.Hq + u.hk * rep + i % rep) * D;
  }
  if (r1 < u.rows) {
    const int i = u.row0 + r1;
    q1 = q + ((int64_t)(u.first + i / rep) * a.Hq + u.hk * rep + i % rep) * D;
  }
  // The requests' lengths and the block ids: one round trip, so both are asked for first; the queries come while the
  // first keys do. (Without a window the rows see all keys, or all up to the longest one's last, which cuts the part
  // short only then.)
  int ids[kPieces / 32];
#pragma unroll
  for (int i = 0; i < kPieces / 32; ++i) {
    const int p = kb + (i * 32 + lane) * kBlockSize;
    ids[i] = t == 0 && p < k1 ? u.table[p / kBlockSize >> a.rsh] : -1;
  }
  if (a.window == 0 && !see()) return;
  const int ns = (k1 - kb + KP * kBlockSize - 1) / (KP * kBlockSize), mine = ns > kg ? (ns - kg + KG - 1) / KG : 0;   // stages, this ring's
  if (t == 0) {
#pragma unroll
    for (int i = 0; i < kPieces / 32; ++i) {                   // (the same of every ring)
      const int p = kb + (i * 32 + lane) * kBlockSize;
      const bool want = p < k1 && (!seen.gaps || any_sees(a, b0, b1, P, p, p + kBlockSize));
      pieces[i * 32 + lane] = want ? pool_row(a, ids[i], u.hk, p / kBlockSize) : -1;
    }
    __syncwarp();
  }
  // lane 0 of the warp that fills the ring: asks for the ring's stage n; which of its pieces there are goes to
  // have_s, before the arrival that the readers wait for
  auto issue = [&](int n) {
    const int st = n % NST, *p = pieces + (kg + n * KG) * KP;
    unsigned have = 0;
#pragma unroll
    for (int j = 0; j < KP; ++j) have |= (unsigned)(p[j] >= 0) << j;
    have_s[st] = have;
    if (have) mbar_expect_tx(&full[st], __popc(have) * 2 * TILE);
    else mbar_arrive(&full[st]);
#pragma unroll
    for (int j = 0; j < KP; ++j)
      if (p[j] >= 0) {
        uint8_t* dst = ring + (st * KP + j) * 2 * TILE;
        tma_load_3d(dst, tk, 0, p[j], 0, &full[st]);
        tma_load_3d(dst + TILE, tv, 0, p[j], 0, &full[st]);
      }
  };
  if (t == 0 && lane == 0)
    for (int n = 0; n < min(NST, mine); ++n) issue(n);
  const int len0 = q0 ? a.lens[u.first + (u.row0 + r0) / rep] : 0, len1 = q1 ? a.lens[u.first + (u.row0 + r1) / rep] : 0;
  WarpTile<D> w;
  w.start(q0, q1, a.q_sign);
  // keys that the lane's rows see, and those that all of the warp's rows do
  if (q0) {
    const RowSpan x = row_span(a, len0, 0, P);
    w.lo0 = x.lo;
    w.hi0 = min(P, x.n);
  }
  if (q1) {
    const RowSpan x = row_span(a, len1, 0, P);
    w.lo1 = x.lo;
    w.hi1 = min(P, x.n);
  }
  const int min_hi = __reduce_min_sync(0xffffffffu, min(q0 ? w.hi0 : INT32_MAX, q1 ? w.hi1 : INT32_MAX));
  const int max_lo = __reduce_max_sync(0xffffffffu, max(w.lo0, w.lo1));
  for (int n = 0; n < mine; ++n) {
    const int st = n % NST;
    bool ok = __all_sync(0xffffffffu, mbar_wait_cycles(&full[st], (n / NST) & 1));
    const unsigned have = ok ? have_s[st] : 0;
    if (have && t * 16 < u.rows)
      w.template step<KP>(kb + (kg + n * KG) * KP * kBlockSize, ring + st * KP * 2 * TILE, have, k0, k1, min_hi, max_lo,
                          a.scale_log2);
    __syncwarp();
    if (NT > 1 && lane == 0) mbar_arrive(&empty[st]);
    if (ok && t == 0 && n >= S::LAG && n - S::LAG + NST < mine) {
      const int m = n - S::LAG;
      if (NT > 1) ok = __all_sync(0xffffffffu, mbar_wait_cycles(&empty[m % NST], (m / NST) & 1));
      if (ok && lane == 0) issue(m + NST);
      __syncwarp();
    }
    if (!ok) {                                 // report, and let the copies in flight land
      if (lane == 0) {
        flag(a.status, HYB_DEVERR_TIMEOUT);
        if (t == 0)
          // asked for so far: up to the stage NST behind the last that was done with
          for (int j = max(0, n - S::LAG); j < min(mine, max(0, n - S::LAG) + NST); ++j)
            mbar_wait_cycles(&full[j % NST], (j / NST) & 1, 200000000u);
      }
      break;
    }
  }
  w.finish();

  // -------------------------------------------------------------------- the part's state
  const int parts = a.Sp + a.Ss;
  const Unit& end = NT == 4 ? *us : u;
  auto slot = [&](int r) {                     // of tile row r
    const int i = end.row0 + r, n = a.Hq / a.Hk;
    return ((int64_t)(end.first + i / n) * a.Hq + end.hk * n + i % n) * parts + end.part;
  };
  if (KG == 1) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = half ? r1 : r0;
      if (r >= end.rows) continue;
      const int64_t at = slot(r);
      if (quad == 0) a.ws_ml[at] = make_float2(w.m[half], w.l[half]);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(a.ws_acc + at * D + i * 8 + quad * 2) = make_float2(w.o[i][2 * half], w.o[i][2 * half + 1]);
    }
    return;
  }
  __syncthreads();                             // all pieces are read: the rings hold the sums now
  float* red = reinterpret_cast<float*>(sm);
  {
    const int base = (kg * NT + t) * 16 + (lane >> 2);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      *reinterpret_cast<float2*>(red + base * S::PITCH + i * 8 + quad * 2) = make_float2(w.o[i][0], w.o[i][1]);
      *reinterpret_cast<float2*>(red + (base + 8) * S::PITCH + i * 8 + quad * 2) = make_float2(w.o[i][2], w.o[i][3]);
    }
    if (quad == 0) {
      red_ml[base] = make_float2(w.m[0], w.l[0]);
      red_ml[base + 8] = make_float2(w.m[1], w.l[1]);
    }
  }
  __syncthreads();
  {
    for (int r = warp; r < end.rows; r += kWarps) {
      float M = -INFINITY, L = 0.f, x[KG];
#pragma unroll
      for (int k = 0; k < KG; ++k) M = fmaxf(M, red_ml[k * NT * 16 + r].x);
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        const float2 v = red_ml[k * NT * 16 + r];
        x[k] = v.x == -INFINITY ? 0.f : fast_exp2(v.x - M);
        L += x[k] * v.y;
      }
      const int64_t at = slot(r);
      if (lane == 0) a.ws_ml[at] = make_float2(M, L);
      for (int e = lane * 2; e < D; e += 64) {
        float2 A = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < KG; ++k) {
          const float2 v = *reinterpret_cast<const float2*>(red + (k * NT * 16 + r) * S::PITCH + e);
          A.x = fmaf(x[k], v.x, A.x);
          A.y = fmaf(x[k], v.y, A.y);
        }
        *reinterpret_cast<float2*>(a.ws_acc + at * D + e) = A;
      }
    }
  }
}

// CTAs [0, pre_ctas): ((group Hk + key head) tiles + row tile) Sp + part of the prefixes; the others:
// request own_ctas + four of its (part, key head, row tile), one a warp.
template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, D == 256 ? 2 : 3)
prefix_mma_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                  const __nv_bfloat16* __restrict__ q, const PrefixArgs a, int pre_ctas, int pre_tiles,
                  int own_ctas, int own_tiles, int early) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  // early: launched behind the tensor-core kernel of the same call, which began when everything before it had
  // ended and writes nothing that this one reads or writes. So this one runs beside it, on the SMs that it leaves, and
  // its last CTA alone waits for it: the joining kernel waits for this one, which then ends after both. (With every
  // CTA waiting, the first ones kept the others off those SMs: 256 requests on 32768 tokens 135 us against 122.)
  if (!early) pdl_wait();
  pdl_trigger();
  const int rep = a.Hq / a.Hk;
  Unit u;
  int i = blockIdx.x;
  if (i < pre_ctas) {
    u.part = i % a.Sp;
    i /= a.Sp;
    const int tile = i % pre_tiles;
    i /= pre_tiles;
    u.hk = i % a.Hk;
    int b1, P;
    if (!group_ok(a, i / a.Hk, u.first, b1, P)) return;
    u.row0 = tile * 16 * NT;
    u.rows = min(16 * NT, (b1 - u.first) * rep - u.row0);
    u.k0 = u.part * a.Lp;
    u.k1 = min(P, u.k0 + a.Lp);
    u.table = a.bt + (int64_t)u.first * a.MB;
    if (u.rows <= 0 || u.k0 >= u.k1) return;
    attend<D, NT>(&tk, &tv, q, a, u, P, sm);
  } else {
    // every warp takes one of the request's (part, key head, row tile)
    i -= pre_ctas;
    u.first = i / own_ctas;
    const RowSpan r = find_row(a, u.first);
    i = (i % own_ctas) * kWarps + (threadIdx.x >> 5);
    const int tile = i % own_tiles;
    i /= own_tiles;
    u.hk = i % a.Hk;
    u.part = i / a.Hk;
    if (r.n >= 0 && u.part < r.own_parts(a.Ls)) {
      u.row0 = tile * 16;
      u.rows = min(16, rep - u.row0);
      u.k0 = r.own_base() + u.part * a.Ls;
      u.k1 = min(r.n, u.k0 + a.Ls);
      u.part += a.Sp;
      u.table = a.bt + (int64_t)u.first * a.MB;
      attend_own<D>(&tk, &tv, q, a, u, r.own_lo(), sm);
    }
    if (early && blockIdx.x == gridDim.x - 1) pdl_wait();
  }
}

template <int D, int NT>
cudaError_t launch_typed(const CUtensorMap& tk, const CUtensorMap& tv, const __nv_bfloat16* q, const PrefixArgs& a,
                         bool prefix, bool early, cudaStream_t s) {
  const int rep = a.Hq / a.Hk;
  const int64_t pre_tiles = ((int64_t)a.max_group * rep + 16 * NT - 1) / (16 * NT), own_tiles = (rep + 15) / 16;
  const int64_t pre = prefix ? (int64_t)a.G * a.Hk * pre_tiles * a.Sp : 0;
  const int64_t own_ctas = ((int64_t)a.Ss * a.Hk * own_tiles + kWarps - 1) / kWarps, own = a.B * own_ctas;
  if (pre + own == 0) return cudaSuccess;
  if (pre + own > INT32_MAX) return cudaErrorInvalidConfiguration;   // its workspace would be above 1 TB
  constexpr int smem = MmaShape<D, NT>::SMEM > OwnShape<D>::SMEM ? MmaShape<D, NT>::SMEM : OwnShape<D>::SMEM;
  cudaError_t e = set_smem((const void*)prefix_mma_kernel<D, NT>, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(prefix_mma_kernel<D, NT>, dim3((unsigned)(pre + own)), dim3(kWarps * 32), smem, s, tk, tv, q, a,
                 (int)pre, (int)pre_tiles, (int)own_ctas, (int)own_tiles, early ? 1 : 0);
  count_launch();
  return e;
}

}  // namespace

bool prefix_mma_supported(int dtype, int D) {
  return dtype == HYB_BF16 && (D == 64 || D == 128 || D == 256);
}

cudaError_t launch_prefix_mma(int D, const void* q, const void* kc, const void* vc, const PrefixArgs& a, bool prefix,
                              bool early, cudaStream_t s) {
  CUtensorMap tk, tv;
  // {64 columns, rows, column blocks}: one box is a piece of all columns, [D / 64][16 rows][64], swizzled
  const uint64_t dims[3] = {64, (uint64_t)a.NB * a.Hk * (kBlockSize << a.rsh), (uint64_t)D / 64};
  const uint64_t str[2] = {(uint64_t)D * 2, 128};
  const uint32_t box[3] = {64, kBlockSize, (uint32_t)D / 64};
  if (!encode_tmap_bf16(&tk, kc, 3, dims, str, box) || !encode_tmap_bf16(&tv, vc, 3, dims, str, box))
    return cudaErrorInvalidValue;
  const int64_t rows = (int64_t)a.max_group * (a.Hq / a.Hk);
  const int nt = !prefix || rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
#define HYB_MMA(DD, N) \
  if (D == DD && nt == N) return launch_typed<DD, N>(tk, tv, (const __nv_bfloat16*)q, a, prefix, early, s);
  HYB_MMA(64, 1)
  HYB_MMA(64, 2)
  HYB_MMA(64, 4)
  HYB_MMA(128, 1)
  HYB_MMA(128, 2)
  HYB_MMA(128, 4)
  HYB_MMA(256, 1)
  HYB_MMA(256, 2)
  HYB_MMA(256, 4)
#undef HYB_MMA
  return cudaErrorInvalidValue;
}

}  // namespace hyb
