// Parts of shared-prefix decode attention, bf16, D = 64, 128 or 256, on warp matrix instructions:
// a part's keys are streamed once for 16 NT query rows (the rows of a group times the query heads
// of one key head, or one request's query heads for its own tokens).
//
// Per 16-token piece of the cache, with Q the rows as A fragments in registers:
//   S = Q K^T (16 x 16 a warp), p = 2^(scale S - m), O += P V
// all in registers: S's accumulators are the A fragment of P V.
#include <cuda_bf16.h>

#include "shared_prefix.cuh"
#include "tc.cuh"

namespace hyb {
namespace {

constexpr int kWarps = 4;                      // computing warps; one more fetches
constexpr float kRescale = 8.f;                // log2: the largest p before the base moves

template <int D, int NT>
struct MmaShape {
  static constexpr int KG = kWarps / NT;       // key groups: rings of pieces, each read by NT warps
  static constexpr int TILE = 16 * D * 2;      // K or V of a piece
  static constexpr int NST = 65536 / (KG * 2 * TILE) > 2 ? 65536 / (KG * 2 * TILE) : 2;
  static constexpr int RING = KG * NST * 2 * TILE;
  static constexpr int PITCH = D + 8;          // floats of a row where key groups are joined
  static constexpr int JOIN = kWarps * 16 * PITCH * 4;
  static constexpr int BODY = KG > 1 && JOIN > RING ? JOIN : RING;
  static constexpr int BARS = BODY;            // full, empty: u64 [KG][NST]; ok: int [KG][NST]
  static constexpr int ROWS = BARS + KG * NST * 20 + 16;         // int lo[64], hi[64]; float2 ml[64]
  static constexpr int SMEM = ROWS + 64 * 16 + 1024;             // 1 KiB of alignment slack
};

// What a CTA works on: rows row0 .. row0 + rows - 1 of those of key head hk from request first on
// (row i: request first + i / rep, query head hk rep + i % rep), keys [k0, k1) through `table`.
struct Unit {
  const int32_t* table;
  int first, hk, row0, rows, part, k0, k1;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int NT>
__device__ __forceinline__ void attend(const CUtensorMap* tk, const CUtensorMap* tv,
                                       const __nv_bfloat16* __restrict__ q, const PrefixArgs& a, const Unit& u,
                                       int P, bool shared, uint8_t* sm) {
  using S = MmaShape<D, NT>;
  constexpr int KG = S::KG, NST = S::NST, TILE = S::TILE, NB64 = D / 64;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::BARS);
  uint64_t* empty = full + KG * NST;
  int* okp = reinterpret_cast<int*>(empty + KG * NST);
  int* row_lo = reinterpret_cast<int*>(sm + S::ROWS);
  int* row_hi = row_lo + 64;
  float2* red_ml = reinterpret_cast<float2*>(row_hi + 64);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rep = a.Hq / a.Hk;

  if (tid < 16 * NT) {                         // keys that a row sees; hi 0: a row that is not there
    int lo = 0, hi = 0;
    if (tid < u.rows) {
      const RowSpan r = row_span(a, u.first + (u.row0 + tid) / rep, 0, P);
      lo = shared ? r.lo : r.own_lo();
      hi = shared ? min(P, r.n) : r.n;
    }
    row_lo[tid] = lo;
    row_hi[tid] = hi;
  }
  if (tid == kWarps * 32) {
    for (int i = 0; i < KG * NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], NT);
    }
    fence_mbar_init();
  }
  __syncthreads();
  // the tile's bounds over its rows (rows that see nothing do not count for the lower ones)
  int max_hi = 0, min_lo = INT32_MAX, min_hi = INT32_MAX, max_lo = 0;
#pragma unroll
  for (int i = 0; i < (16 * NT + 31) / 32; ++i) {
    const int r = i * 32 + lane;
    if (r < 16 * NT && row_hi[r] > row_lo[r]) {
      max_hi = max(max_hi, row_hi[r]);
      min_lo = min(min_lo, row_lo[r]);
    }
    if (r < u.rows) {
      min_hi = min(min_hi, row_hi[r]);
      max_lo = max(max_lo, row_lo[r]);
    }
  }
  max_hi = __reduce_max_sync(0xffffffffu, max_hi);
  min_lo = __reduce_min_sync(0xffffffffu, min_lo);
  min_hi = __reduce_min_sync(0xffffffffu, min_hi);
  max_lo = __reduce_max_sync(0xffffffffu, max_lo);
  const int k0 = max(u.k0, min_lo), k1 = min(u.k1, max_hi);
  if (k0 >= k1) return;                        // nothing that a row sees (min_lo may be INT32_MAX)
  const int kb = k0 & ~(kBlockSize - 1), np = (k1 - kb + kBlockSize - 1) / kBlockSize;

  bool ok = true;
  if (warp == kWarps) {
    // ------------------------------------------------------------------ fetching
    int issued = 0;
    for (int i0 = 0; i0 < np && ok; i0 += 32) {
      int y = -1;                              // pool row of piece i0 + lane
      if (i0 + lane < np) {
        const int sub = kb / kBlockSize + i0 + lane;
        const int pb = u.table[sub >> a.rsh];
        if (pb < 0 || pb >= a.NB) flag(a.status, HYB_DEVERR_BAD_BLOCK);
        else y = ((pb * a.Hk + u.hk) << (4 + a.rsh)) + ((sub & ((1 << a.rsh) - 1)) << 4);
      }
      const int cnt = min(32, np - i0);
      for (int j = 0; j < cnt; ++j) {
        const int i = i0 + j, n = i / KG, st = (i % KG) * NST + n % NST;
        const int row = __shfl_sync(0xffffffffu, y, j);
        if (n >= NST) {
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], (n / NST - 1) & 1));
          if (!ok) break;
        }
        if (lane == 0) {
          okp[st] = row >= 0;
          if (row >= 0) {
            uint8_t* dst = sm + st * 2 * TILE;
            mbar_expect_tx(&full[st], 2 * TILE);
#pragma unroll
            for (int c = 0; c < NB64; ++c) tma_load_2d(dst + c * 2048, tk, c * 64, row, &full[st]);
#pragma unroll
            for (int c = 0; c < NB64; ++c) tma_load_2d(dst + TILE + c * 2048, tv, c * 64, row, &full[st]);
          } else {
            mbar_arrive(&full[st]);
          }
        }
        __syncwarp();
        issued = i + 1;
      }
    }
    if (!ok && lane == 0) {                    // report, and let the copies in flight land
      flag(a.status, HYB_DEVERR_TIMEOUT);
      for (int i = max(0, issued - KG * NST); i < issued; ++i)
        mbar_wait(&full[(i % KG) * NST + (i / KG) % NST], (i / KG / NST) & 1, 100000000ull);
    }
  }

  // -------------------------------------------------------------------- computing
  const int t = warp % NT, kg = warp / NT;     // row tile, key group
  const int r0 = t * 16 + (lane >> 2), r1 = r0 + 8, quad = lane & 3;
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  if (warp < kWarps) {
    uint32_t qa[D / 16][4];
    const __nv_bfloat16 *q0 = nullptr, *q1 = nullptr;
    if (r0 < u.rows) {
      const int i = u.row0 + r0;
      q0 = q + ((int64_t)(u.first + i / rep) * a.Hq + u.hk * rep + i % rep) * D;
    }
    if (r1 < u.rows) {
      const int i = u.row0 + r1;
      q1 = q + ((int64_t)(u.first + i / rep) * a.Hq + u.hk * rep + i % rep) * D;
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const int c = k * 16 + quad * 2;
      qa[k][0] = q0 ? *reinterpret_cast<const uint32_t*>(q0 + c) : 0u;
      qa[k][1] = q1 ? *reinterpret_cast<const uint32_t*>(q1 + c) : 0u;
      qa[k][2] = q0 ? *reinterpret_cast<const uint32_t*>(q0 + c + 8) : 0u;
      qa[k][3] = q1 ? *reinterpret_cast<const uint32_t*>(q1 + c + 8) : 0u;
    }
    const int lo0 = row_lo[r0], hi0 = row_hi[r0], lo1 = row_lo[r1], hi1 = row_hi[r1];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
    // a lane's row and 16-byte chunk in the four 8 x 8 matrices of a load
    const int krow = (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;
    const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vch = lane >> 4;

    for (int n = 0; kg + n * KG < np; ++n) {
      const int st = kg * NST + n % NST;
      ok = __all_sync(0xffffffffu, mbar_wait(&full[st], (n / NST) & 1));
      if (!ok) {
        if (lane == 0) flag(a.status, HYB_DEVERR_TIMEOUT);
        break;
      }
      if (okp[st]) {
        const int tok = kb + (kg + n * KG) * kBlockSize;
        uint8_t* kt = sm + st * 2 * TILE;
        const uint32_t ks = smem_u32(kt), vs = ks + TILE;
        float s[2][2][4];                      // [half of the head][8 keys][.]: two chains each
#pragma unroll
        for (int i = 0; i < 16; ++i) (&s[0][0][0])[i] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t b[4];
          const int ch = k * 2 + kch;
          ldsm4(ks + (ch >> 3) * 2048 + sw128_off(krow, ch & 7), b);
          mma16816(s[k & 1][0], qa[k], b[0], b[1]);
          mma16816(s[k & 1][1], qa[k], b[2], b[3]);
        }
        float x[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[i][c] = (s[0][i][c] + s[1][i][c]) * a.scale_log2;
        if (tok < max_lo || tok + kBlockSize > min_hi || tok < k0 || tok + kBlockSize > k1) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int key = tok + i * 8 + quad * 2 + (c & 1);
              const bool see = key >= k0 && key < k1 && (c < 2 ? key >= lo0 && key < hi0 : key >= lo1 && key < hi1);
              if (!see) x[i][c] = -INFINITY;
            }
          if (tok < k0 || tok + kBlockSize > k1) {
            // rows that hold no key of the part may hold NaN, and 0 x NaN is NaN (every warp that
            // reads the piece writes the same zeros first)
            for (int e = lane; e < kBlockSize * D / 8; e += 32) {
              const int r = e / (D / 8), ch = e % (D / 8);
              if (tok + r < k0 || tok + r >= k1)
                *reinterpret_cast<uint4*>(kt + TILE + (ch >> 3) * 2048 + r * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();                // the ring's next copy comes after these writes
            __syncwarp();
          }
        }
        float mx0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
        float mx1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
#pragma unroll
        for (int d = 1; d <= 2; d <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
        }
        // the base moves only where a row's maximum outgrows it: p stays below 2^8
        const bool g0 = mx0 > m[0] + kRescale || (m[0] == -INFINITY && mx0 != -INFINITY);
        const bool g1 = mx1 > m[1] + kRescale || (m[1] == -INFINITY && mx1 != -INFINITY);
        if (__any_sync(0xffffffffu, g0 || g1)) {
          const float a0 = g0 ? (m[0] == -INFINITY ? 0.f : fast_exp2(m[0] - mx0)) : 1.f;
          const float a1 = g1 ? (m[1] == -INFINITY ? 0.f : fast_exp2(m[1] - mx1)) : 1.f;
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
        const float b0 = m[0] == -INFINITY ? 0.f : m[0], b1 = m[1] == -INFINITY ? 0.f : m[1];
        float p[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) p[i][c] = fast_exp2(x[i][c] - (c < 2 ? b0 : b1));
        l[0] += (p[0][0] + p[0][1]) + (p[1][0] + p[1][1]);
        l[1] += (p[0][2] + p[0][3]) + (p[1][2] + p[1][3]);
        // P as bf16: half a step of a weight, 2^-9 of it on average less, of bf16 outputs
        const uint32_t pa[4] = {pack_bf16(p[0][0], p[0][1]), pack_bf16(p[0][2], p[0][3]),
                                pack_bf16(p[1][0], p[1][1]), pack_bf16(p[1][2], p[1][3])};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t b[4];
          const int ch = k * 2 + vch;
          ldsm4_t(vs + (ch >> 3) * 2048 + sw128_off(vrow, ch & 7), b);
          mma16816(o[2 * k], pa, b[0], b[1]);
          mma16816(o[2 * k + 1], pa, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
      l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
    }
  }

  // -------------------------------------------------------------------- the part's state
  const int parts = a.Sp + a.Ss;
  auto slot = [&](int r) {                     // of tile row r
    const int i = u.row0 + r;
    return ((int64_t)(u.first + i / rep) * a.Hq + u.hk * rep + i % rep) * parts + u.part;
  };
  if (KG == 1) {
    if (warp < kWarps)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = half ? r1 : r0;
        if (r >= u.rows) continue;
        const int64_t at = slot(r);
        if (quad == 0) a.ws_ml[at] = make_float2(m[half], l[half]);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(a.ws_acc + at * D + i * 8 + quad * 2) = make_float2(o[i][2 * half], o[i][2 * half + 1]);
      }
    return;
  }
  __syncthreads();                             // all pieces are read: the rings hold the sums now
  float* red = reinterpret_cast<float*>(sm);
  if (warp < kWarps) {
    const int base = (kg * NT + t) * 16 + (lane >> 2);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      *reinterpret_cast<float2*>(red + base * S::PITCH + i * 8 + quad * 2) = make_float2(o[i][0], o[i][1]);
      *reinterpret_cast<float2*>(red + (base + 8) * S::PITCH + i * 8 + quad * 2) = make_float2(o[i][2], o[i][3]);
    }
    if (quad == 0) {
      red_ml[base] = make_float2(m[0], l[0]);
      red_ml[base + 8] = make_float2(m[1], l[1]);
    }
  }
  __syncthreads();
  if (warp < kWarps) {
    for (int r = warp; r < u.rows; r += kWarps) {
      float M = -INFINITY, L = 0.f, w[KG];
#pragma unroll
      for (int k = 0; k < KG; ++k) M = fmaxf(M, red_ml[k * NT * 16 + r].x);
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        const float2 v = red_ml[k * NT * 16 + r];
        w[k] = v.x == -INFINITY ? 0.f : fast_exp2(v.x - M);
        L += w[k] * v.y;
      }
      const int64_t at = slot(r);
      if (lane == 0) a.ws_ml[at] = make_float2(M, L);
      for (int e = lane * 2; e < D; e += 64) {
        float2 A = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < KG; ++k) {
          const float2 v = *reinterpret_cast<const float2*>(red + (k * NT * 16 + r) * S::PITCH + e);
          A.x = fmaf(w[k], v.x, A.x);
          A.y = fmaf(w[k], v.y, A.y);
        }
        *reinterpret_cast<float2*>(a.ws_acc + at * D + e) = A;
      }
    }
  }
}

// CTAs [0, pre_ctas): ((group Hk + key head) tiles + row tile) Sp + part of the prefixes; the others:
// ((request Hk + key head) tiles + row tile) Ss + part of the requests' own tokens.
template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32 + 32)
prefix_mma_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                  const __nv_bfloat16* __restrict__ q, const PrefixArgs a, int pre_ctas, int pre_tiles,
                  int own_tiles) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  pdl_wait();
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
    attend<D, NT>(&tk, &tv, q, a, u, P, true, sm);
  } else {
    i -= pre_ctas;
    u.part = i % a.Ss;
    i /= a.Ss;
    const int tile = i % own_tiles;
    i /= own_tiles;
    u.hk = i % a.Hk;
    u.first = i / a.Hk;
    const RowSpan r = find_row(a, u.first);
    if (r.n < 0 || u.part >= r.own_parts(a.Ls)) return;
    u.row0 = tile * 16;
    u.rows = min(16, rep - u.row0);
    u.k0 = r.own_base() + u.part * a.Ls;
    u.k1 = min(r.n, u.k0 + a.Ls);
    u.part += a.Sp;
    u.table = a.bt + (int64_t)u.first * a.MB;
    attend<D, 1>(&tk, &tv, q, a, u, r.P, false, sm);
  }
}

template <int D, int NT>
cudaError_t launch_typed(const CUtensorMap& tk, const CUtensorMap& tv, const __nv_bfloat16* q, const PrefixArgs& a,
                         bool prefix, cudaStream_t s) {
  const int rep = a.Hq / a.Hk;
  const int64_t pre_tiles = ((int64_t)a.max_group * rep + 16 * NT - 1) / (16 * NT), own_tiles = (rep + 15) / 16;
  const int64_t pre = prefix ? (int64_t)a.G * a.Hk * pre_tiles * a.Sp : 0;
  const int64_t own = (int64_t)a.B * a.Hk * own_tiles * a.Ss;
  if (pre + own == 0) return cudaSuccess;
  if (pre + own > INT32_MAX) return cudaErrorInvalidConfiguration;   // its workspace would be above 1 TB
  constexpr int smem = MmaShape<D, NT>::SMEM > MmaShape<D, 1>::SMEM ? MmaShape<D, NT>::SMEM : MmaShape<D, 1>::SMEM;
  cudaError_t e = set_smem((const void*)prefix_mma_kernel<D, NT>, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(prefix_mma_kernel<D, NT>, dim3((unsigned)(pre + own)), dim3(kWarps * 32 + 32), smem, s, tk, tv, q, a,
                 (int)pre, (int)pre_tiles, (int)own_tiles);
  count_launch();
  return e;
}

}  // namespace

bool prefix_mma_supported(int dtype, int D) {
  return dtype == HYB_BF16 && (D == 64 || D == 128 || D == 256);
}

cudaError_t launch_prefix_mma(int D, const void* q, const void* kc, const void* vc, const PrefixArgs& a, bool prefix,
                              cudaStream_t s) {
  CUtensorMap tk, tv;
  const uint64_t dims[2] = {(uint64_t)D, (uint64_t)a.NB * a.Hk * (kBlockSize << a.rsh)};
  const uint64_t str[1] = {(uint64_t)D * 2};
  const uint32_t box[2] = {64, kBlockSize};
  if (!encode_tmap_bf16(&tk, kc, 2, dims, str, box) || !encode_tmap_bf16(&tv, vc, 2, dims, str, box))
    return cudaErrorInvalidValue;
  const int64_t rows = (int64_t)a.max_group * (a.Hq / a.Hk);
  const int nt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
#define HYB_MMA(DD, N) \
  if (D == DD && nt == N) return launch_typed<DD, N>(tk, tv, (const __nv_bfloat16*)q, a, prefix, s);
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
