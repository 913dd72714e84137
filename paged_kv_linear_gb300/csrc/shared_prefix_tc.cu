// The prefixes' parts of shared-prefix decode attention for large groups, bf16, D = 128, on the tensor cores
// (tcgen05 + TMEM + TMA).
//
// A group's requests times the query heads of one key head are the rows of a product against the same
// keys, as a prompt's rows are in the causal prefill, and this kernel is built like that one (its reasons
// stand there): one CTA per (pair of row tiles, part, key head, group); two TMA warps (K ring, V ring),
// one MMA-issuing thread, a landing warp, and two softmax warpgroups, one per row tile with one thread per row.
// S_t = Q_t K_j^T and O_t += P_t V_j live in TMEM, P_t over S_t. What differs: every row sees every key of the
// part but for rows that end inside it and windows, so both row tiles walk the same key tiles; rows come
// through a tensor map {D, query heads, requests} whose box of rep x (128 / rep) rows is a tile (rep: query
// heads of a key head; 126 rows where it is 3); and a CTA leaves its softmax's state instead of dividing.
//
// 256 requests of 4 query heads a key head on 32768 tokens, 8 key heads: 128 CTAs of 64 key tiles, 108 us, 1.28 PFLOP/s,
// 0.67 of the bf16 rate (tensor pipe 53 % busy over 152 SMs): a key tile takes 1.43 us, as in the causal prefill, the
// start 4 us and the end 3, and 24 SMs have no CTA (they run the requests' own tokens). Parts of half the length
// fill them but start and end twice (128 us). Not kept: the two softmax warpgroups on every other key tile of one row
// tile (no change at 64 to 128 rows, and its registers cost the large case 13 us).
#include <cuda_bf16.h>

#include "shared_prefix.cuh"
#include "tc.cuh"

namespace hyb {
namespace {

constexpr int kBM = 128, kBN = 128, kD = 128;
constexpr int kSubQ = 128 * 128;             // [128 rows][64 cols] bf16 sub-tile = 16 KiB
constexpr int kTile = 2 * kSubQ;             // [128][128] bf16 = 32 KiB
constexpr int kNK = 2, kNV = 3;              // K and V ring depths
constexpr int kOffQ = 0;                     // two row tiles
constexpr int kOffK = kOffQ + 2 * kTile;
constexpr int kOffV = kOffK + kNK * kTile;
constexpr int kOffBar = kOffV + kNV * kTile;
constexpr int kSmem = kOffBar + 1024 + 1024;  // barriers + 1 KiB alignment slack
constexpr int kNSW = 8;                      // softmax warps: 4 per row tile
constexpr int kWarpTmaK = kNSW, kWarpTmaV = kNSW + 1, kWarpMma = kNSW + 2, kWarpLand = kNSW + 3;
constexpr int kNSF = 4;                      // "step done" ring
constexpr int kThreads = (kNSW + 4) * 32;
// (200 + 200 + 104) x 128 = 64 512 registers: the launch's 384 x 168
constexpr uint32_t kRegsSoftmax = 200, kRegsProducer = 104;
constexpr uint32_t kTmemCols = 512;          // S_0/P_0 | S_1/P_1 | O_0 | O_1
constexpr uint32_t kColO = 256;
constexpr float kRescaleLog2 = 8.f;

constexpr uint32_t kIdescQK = idesc_bf16(128, 128, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16(128, 128, 0, 1);   // A = P from TMEM

struct Bars {
  uint64_t qfull, kfull[kNK], vfull[kNV], stepf[kNSF];
  uint64_t sfull[2], pfull[2], odone[2], drain;    // per row tile
};

// asks L2 for a box of a tensor map
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Whole warp: rows [r0, r1) of a [128 keys][128] bf16 V tile (two SW128 sub-tiles) := 0.
__device__ __forceinline__ void zero_v_rows(uint8_t* tile, int r0, int r1, int lane) {
  for (int e = lane; e < (r1 - r0) * 16; e += 32) {
    const int r = r0 + e / 16, sb = (e >> 3) & 1, ch = e & 7;
    *reinterpret_cast<uint4*>(tile + sb * kSubQ + r * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
  }
}

// grid: (((group Hk + key head) Sp + part) pairs + pair of row tiles); tile_rows: rep x (128 / rep)
// kWindow: with a window, the requests' keys may begin inside a piece and leave gaps (Hull). Without one they cannot, and
// the code for it stays out: it costs 256 requests on 32768 tokens 3 to 5 us of 120 though it never runs.
template <bool kWindow>
__global__ void __launch_bounds__(kThreads, 1)
prefix_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const __grid_constant__ CUtensorMap tv, const PrefixArgs a, int pairs, int tile_rows) {
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rep = a.Hq / a.Hk;
  int i = blockIdx.x;
  const int duo = i % pairs;
  i /= pairs;
  const int part = i % a.Sp;
  i /= a.Sp;
  const int hk = i % a.Hk;
  int b0, b1, P;
  if (!group_ok(a, i / a.Hk, b0, b1, P)) return;
  const int cnt = (b1 - b0) * rep, row0 = duo * 2 * tile_rows;   // rows of the group; the pair's first
  int k0 = part * a.Lp, k1 = min(P, k0 + a.Lp);
  if (row0 >= cnt || k0 >= k1) return;
  const int duos = (cnt + 2 * tile_rows - 1) / (2 * tile_rows);   // CTAs that read the same keys
  const bool two = row0 + tile_rows < cnt;             // second row tile present
  if (a.window > 0) {                                  // only keys that one of the rows sees
    int max_hi = 0, min_lo = INT32_MAX;
    for (int r = row0 / rep + lane; r <= (min(row0 + 2 * tile_rows, cnt) - 1) / rep; r += 32) {
      const RowSpan x = row_span(a, a.lens[b0 + r], 0, P);
      if (min(P, x.n) > x.lo) {
        max_hi = max(max_hi, min(P, x.n));
        min_lo = min(min_lo, x.lo);
      }
    }
    k0 = max(k0, __reduce_min_sync(0xffffffffu, min_lo));
    k1 = min(k1, __reduce_max_sync(0xffffffffu, max_hi));
    if (k0 >= k1) return;                              // (the same in every warp)
  }
  const int kb = k0 & ~(kBlockSize - 1), nloc = (k1 - kb + kBN - 1) / kBN;   // key tiles [kb + 128 j, ..)
  const int32_t* btrow = a.bt + (int64_t)b0 * a.MB;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  Bars* bars = reinterpret_cast<Bars*>(sm + kOffBar);
  __shared__ uint32_t tmem_base;
  // what the softmax threads need rarely waits here: their registers are all spoken for
  __shared__ struct {
    const int32_t* btrow;
    int b0, row0, cnt, part, head0, two;             // head0: the first query head of hk
    int vend;                                        // behind the last key that a row sees
  } info;
  if (tid == 0) {
    info.btrow = btrow;
    info.b0 = b0;
    info.row0 = row0;
    info.cnt = cnt;
    info.part = part;
    info.head0 = hk * rep;
    info.two = two;
  }

  // What none of the rows' requests [q0, q1) sees is not loaded, whatever the table holds there; looked up while the
  // barriers and TMEM are set up.
  const int q0 = b0 + row0 / rep, q1 = b0 + (min(row0 + 2 * tile_rows, cnt) - 1) / rep + 1;
  Hull seen;
  if (warp == kWarpTmaK || warp == kWarpTmaV) {
    for (int b = q0 + lane; b < q1; b += 32) seen.add(a, a.lens[b], P);
    seen.join();
    if (lane == 0) info.vend = min(k1, seen.hi);
  }

  if (warp == kWarpMma) {
    if (lane == 0) {
      mbar_init(&bars->qfull, 1);
      for (int n = 0; n < kNK; ++n) mbar_init(&bars->kfull[n], 1);
      for (int n = 0; n < kNV; ++n) mbar_init(&bars->vfull[n], 1);
      for (int n = 0; n < kNSF; ++n) mbar_init(&bars->stepf[n], 1);
      for (int t = 0; t < 2; ++t) {
        mbar_init(&bars->sfull[t], 1);
        mbar_init(&bars->pfull[t], 128 + 1);          // softmax threads + landing warp
        mbar_init(&bars->odone[t], 1);
      }
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
  uint8_t* const q_s = sm + kOffQ;

  if (warp >= kNSW) {                               // producer warpgroup
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsProducer));
    if (warp == kWarpTmaK || warp == kWarpTmaV) {
      // ------------------------------------------------------------ TMA warps (K ring, V ring)
      const bool isk = warp == kWarpTmaK;
      const CUtensorMap* map = isk ? &tk : &tv;
      const int depth = isk ? kNK : kNV;
      uint8_t* const ring = sm + (isk ? kOffK : kOffV);
      uint64_t* const fullb = isk ? bars->kfull : bars->vfull;
      bool ok = true;
      int issued = 0;
      if (lane == 0 && isk) {                            // the row tiles (requests past B read 0)
        const int per = tile_rows / rep;                 // requests of a tile
        mbar_expect_tx(&bars->qfull, (two ? 2 : 1) * tile_rows * 256);
        for (int t = 0; t < (two ? 2 : 1); ++t) {
          tma_load_3d(q_s + t * kTile, &tq, 0, hk * rep, b0 + (duo * 2 + t) * per, &bars->qfull);
          tma_load_3d(q_s + t * kTile + kSubQ, &tq, 64, hk * rep, b0 + (duo * 2 + t) * per, &bars->qfull);
        }
      }
      // pool rows of 4 tiles' pieces, one per lane, looked up 4 tiles ahead; L2 is asked for the pieces then, each
      // by one of the CTAs that read the same keys: the rings are too short for memory's latency
      const int kend = min(k1, seen.hi);
      auto rows_of = [&](int j) {
        const int s = kb / kBlockSize + j * 8 + lane;
        if (s * kBlockSize >= kend) return -1;
        if (kWindow && seen.gaps && !any_sees(a, q0, q1, P, s * kBlockSize, (s + 1) * kBlockSize)) return -1;
        const int pb = btrow[s >> a.rsh];
        const bool there = pb >= 0 && pb < a.NB;
        if (isk && !there) flag(a.status, HYB_DEVERR_BAD_BLOCK);
        return there ? ((pb * a.Hk + hk) << (4 + a.rsh)) + ((s & ((1 << a.rsh) - 1)) << 4) : -1;
      };
      int ids = -1, ahead = rows_of(0);
      for (int jj = 0; jj < nloc; ++jj) {
        if ((jj & 3) == 0) {
          ids = ahead;
          ahead = rows_of(jj + 4);
          if (ahead >= 0 && lane % duos == duo % 32) {
            tma_prefetch_2d(map, 0, ahead);
            tma_prefetch_2d(map, 64, ahead);
          }
        }
        int blk[8];
        int nbox = 0;
#pragma unroll
        for (int bi = 0; bi < 8; ++bi) {
          blk[bi] = __shfl_sync(0xffffffffu, ids, (jj & 3) * 8 + bi);
          nbox += blk[bi] >= 0 ? 2 : 0;
        }
        const int slot = jj % depth;
        if (jj >= depth) {
          // the slot held K_{jj-kNK} (read by the Q K^T of the step before key tile jj-kNK)
          // or V_{jj-kNV} (read by the P V of its own step): free once that step is done
          const int m = isk ? jj - kNK : jj - kNV + 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->stepf[m % kNSF], (m / kNSF) & 1));
          if (!ok) break;
        }
        // V rows that hold no key of the part must be finite (P is 0 there, but 0 x NaN is NaN): pieces that
        // are not loaded are zeroed here, rows before the first and past the last key inside their pieces by the landing warp
        if (!isk && nbox < 16) {
#pragma unroll
          for (int bi = 0; bi < 8; ++bi)
            if (blk[bi] < 0) zero_v_rows(ring + slot * kTile, bi * 16, bi * 16 + 16, lane);
          fence_async_smem();
          __syncwarp();
        }
        if (lane == 0) {
          uint8_t* dst = ring + slot * kTile;
          if (nbox) mbar_expect_tx(&fullb[slot], nbox * 2048);
          else mbar_arrive(&fullb[slot]);
#pragma unroll
          for (int bi = 0; bi < 8; ++bi)
            if (blk[bi] >= 0) {
              tma_load_2d(dst + bi * 2048, map, 0, blk[bi], &fullb[slot]);
              tma_load_2d(dst + kSubQ + bi * 2048, map, 64, blk[bi], &fullb[slot]);
            }
        }
        issued = jj + 1;
      }
      if (!ok && lane == 0) {                            // let the loads in flight land
        flag(a.status, HYB_DEVERR_TIMEOUT);
        for (int j = max(0, issued - depth); j < issued; ++j)
          mbar_wait(&fullb[j % depth], (j / depth) & 1, 100000000ull);
      }
    } else if (warp == kWarpLand) {
      // ------------------------------------------------------------ landing warp
      // Per key tile j: (1) the step before it is done -> stepf; (2) once V_j and K_{j+1} have
      // landed, one arrival on pfull[t] per row tile. Every phase of each barrier is observed in order.
      const int vend = info.vend;
      bool ok = __all_sync(0xffffffffu, mbar_wait(&bars->kfull[0], 0));
      for (int jj = 0; jj < nloc && ok; ++jj) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->sfull[two ? 1 : 0], jj & 1));
        if (!ok) break;
        if (lane == 0) mbar_arrive(&bars->stepf[jj % kNSF]);
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->vfull[jj % kNV], (jj / kNV) & 1));
        if (!ok) break;
        const int vtail = vend - (kb + jj * kBN);
        if ((vtail & 15) != 0 && vtail < kBN && vtail > 0) {   // rows past the last key in its piece
          zero_v_rows(sm + kOffV + (jj % kNV) * kTile, vtail, (vtail + 15) & ~15, lane);
          fence_async_smem();
          __syncwarp();
        }
        if (kWindow && jj == 0 && kb < k0) {             // and before the first key in its piece
          zero_v_rows(sm + kOffV, 0, k0 - kb, lane);
          fence_async_smem();
          __syncwarp();
        }
        if (jj + 1 < nloc) {
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->kfull[(jj + 1) % kNK], ((jj + 1) / kNK) & 1));
          if (!ok) break;
        }
        if (lane == 0) {
          mbar_arrive(&bars->pfull[0]);
          if (two) mbar_arrive(&bars->pfull[1]);
        }
        __syncwarp();
      }
      if (!ok && lane == 0) flag(a.status, HYB_DEVERR_TIMEOUT);
    } else if (warp == kWarpMma && lane == 0) {
      // ------------------------------------------------------------ MMA issue (one thread)
      // Per key tile j: wait for P_0 (which also means V_j and K_{j+1} have landed), P_0 V_j,
      // Q_0 K_{j+1}^T + commit; the same for tile 1. Nothing else.
      bool ok = true;
      const uint64_t qdesc = sw128_desc(smem_u32(q_s), 16, 1024);
      const uint64_t kdesc = sw128_desc(smem_u32(sm + kOffK), 16, 1024);
      const uint64_t vdesc = sw128_desc(smem_u32(sm + kOffV), kSubQ, 1024);
      auto issue_qk = [&](int t, int ks) {               // S_t = Q_t K^T, K from ring slot ks
        tc_fence_after();
        const uint64_t qd = desc_add(qdesc, t * kTile);
        const uint64_t kd = desc_add(kdesc, ks * kTile);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = (k >> 2) * kSubQ + (k & 3) * 32;
          tc_mma(tmem + t * 128, desc_add(qd, off), desc_add(kd, off), kIdescQK, k > 0);
        }
        tc_commit(&bars->sfull[t]);
      };
      auto issue_pv = [&](int t, int vs, bool first) {   // O_t += P_t V_j
        tc_fence_after();
        const uint64_t vd = desc_add(vdesc, vs * kTile);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc_mma_ta(tmem + kColO + t * 128, tmem + t * 128 + k * 8, desc_add(vd, k * 2048), kIdescPV,
                    (!first || k > 0) ? 1u : 0u);
      };
      ok = mbar_wait(&bars->qfull, 0) && mbar_wait(&bars->kfull[0], 0);
      if (ok) {
        issue_qk(0, 0);
        if (two) issue_qk(1, 0);
      }
      for (int jj = 0; jj < nloc && ok; ++jj) {
        const int vs = jj % kNV, ks1 = (jj + 1) % kNK;
        const bool next = jj + 1 < nloc;
        ok = mbar_wait(&bars->pfull[0], jj & 1);
        if (!ok) break;
        issue_pv(0, vs, jj == 0);
        if (next) issue_qk(0, ks1);
        else tc_commit(&bars->odone[0]);                 // O_0 complete
        if (two) {
          ok = mbar_wait(&bars->pfull[1], jj & 1);
          if (!ok) break;
          issue_pv(1, vs, jj == 0);
          if (next) issue_qk(1, ks1);
          else tc_commit(&bars->odone[1]);
        }
      }
      if (!ok) {
        flag(a.status, HYB_DEVERR_TIMEOUT);
        tc_commit(&bars->drain);
        mbar_wait(&bars->drain, 0, 100000000ull);
      }
    }
  } else {                                           // softmax warpgroups
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, quarter = warp & 3;       // row tile, TMEM lane quarter
    const int r = quarter * 32 + lane;                 // row of the tile = TMEM lane
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_col = tl + t * 128, o_col = tl + kColO + t * 128;
    // keys that the row sees, of the part's; a row that is not there: none, and it does not count below
    int lo = 0, hi = 0, max_lo = 0, min_hi = INT32_MAX;
    {
      const int f = row0 + t * tile_rows + r;          // row of the group
      if ((t == 0 || two) && r < tile_rows && f < cnt) {
        const RowSpan x = row_span(a, a.lens[b0 + f / rep], 0, P);
        lo = max_lo = max(x.lo, k0);
        hi = min_hi = min(min(P, x.n), k1);
      }
    }
    const bool any = __any_sync(0xffffffffu, min_hi != INT32_MAX);   // a warp without rows only keeps the pace
    bool good = true;                                  // no bad block in the part
#pragma unroll 8
    for (int s = kb / kBlockSize + lane; s < (k1 + kBlockSize - 1) / kBlockSize; s += 32) {
      const int pb = btrow[s >> a.rsh];                // (all asked for at once)
      good = good & (pb >= 0) & (pb < a.NB);
    }
    if (!good) min_hi = 0;                             // one: every tile takes the masking path
    max_lo = __reduce_max_sync(0xffffffffu, max_lo);
    min_hi = __reduce_min_sync(0xffffffffu, min_hi);
    const float scale_log2 = a.scale_log2;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    const int steps = (t == 0 || two) ? nloc : 0;
    for (int it = 0; !any && it < steps && ok; ++it) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->sfull[t], it & 1));
      tc_fence_before();
      if (ok) mbar_arrive(&bars->pfull[t]);
    }
    for (int it = 0; any && it < steps && ok; ++it) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->sfull[t], it & 1));
      if (!ok) break;
      tc_fence_after();
      float x[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(s_col + c * 32, x + c * 32);
      tmem_ld_wait();
      const int kbase = kb + it * kBN;
      if (kbase < max_lo || kbase + kBN > min_hi) {
        int pb = -1;                                 // pieces that are there
        if (lane < 8 && kbase + lane * kBlockSize < a.max_prefix) pb = info.btrow[(kbase / kBlockSize + lane) >> a.rsh];
        const unsigned have = __ballot_sync(0xffffffffu, pb >= 0 && pb < a.NB);
#pragma unroll
        for (int c = 0; c < 128; ++c) {
          const int kp = kbase + c;
          x[c] = (kp >= lo && kp < hi && ((have >> (c / 16)) & 1)) ? x[c] : -INFINITY;
        }
      }
      // row max of the raw scores (scale > 0 keeps the order)
      float mp[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) mp[n] = x[n];
#pragma unroll
      for (int c = 8; c + 16 <= 128; c += 16)
#pragma unroll
        for (int n = 0; n < 8; ++n) mp[n] = max3f(mp[n], x[c + n], x[c + 8 + n]);
#pragma unroll
      for (int n = 0; n < 8; ++n) mp[n] = fmaxf(mp[n], x[120 + n]);
      const float mx = max3f(max3f(mp[0], mp[1], mp[2]), max3f(mp[3], mp[4], mp[5]),
                             fmaxf(mp[6], mp[7])) * scale_log2;
      const float m_new = fmaxf(m_used, mx);
      const bool grow = m_new > m_used + kRescaleLog2 || (m_used == -INFINITY && m_new != -INFINITY);
      const float m_tgt = grow ? m_new : m_used;
      const float m_sub = m_tgt == -INFINITY ? 0.f : m_tgt;   // no key seen yet: P = 0
      uint32_t w[64];
      f32x2 sp[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) sp[n] = pair(0.f, 0.f);
      const f32x2 sc2 = pair(scale_log2, scale_log2), nm2 = pair(-m_sub, -m_sub);
#pragma unroll
      for (int c = 0; c < 64; ++c) {
        float y0, y1;
        unpair(fma2(pair(x[2 * c], x[2 * c + 1]), sc2, nm2), y0, y1);
        const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
        sp[c & 3] = add2(sp[c & 3], pair(p0, p1));
        w[c] = pack_bf16(p0, p1);                    // P as bf16: half a step of each weight
      }
      float s0, s1;
      unpair(add2(add2(sp[0], sp[1]), add2(sp[2], sp[3])), s0, s1);
      const float ls = s0 + s1;
      if (it >= 1 && __any_sync(0xffffffffu, grow)) {
        const float alpha = (grow && m_used != -INFINITY) ? fast_exp2(m_used - m_new) : 1.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {                // warp-wide TMEM access, per-row factor
          float o[32];
          tmem_ld32(o_col + c * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= alpha;
          tmem_st32(o_col + c * 32, o);
        }
        if (grow) l *= alpha;
      }
      m_used = m_tgt;
      l += ls;
      tmem_st32u(s_col, w);                          // P_t: keys 0..127 as bf16 pairs
      tmem_st32u(s_col + 32, w + 32);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars->pfull[t]);
    }
    if (ok && steps) ok = __all_sync(0xffffffffu, mbar_wait(&bars->odone[t], 0));
    // The state of the warp's 32 rows through shared memory (the rings', once no product reads them any more), so
    // that a row is written by 32 lanes side by side (a row a thread: 5.3 us at the end of each CTA).
    if (ok && info.two) ok = __all_sync(0xffffffffu, mbar_wait(&bars->odone[t ^ 1], 0));
    if (ok && steps && any) {
      tc_fence_after();
      constexpr int kPitch = kD + 4;
      static_assert(kNSW * 32 * kPitch * 4 <= (kNK + kNV) * kTile, "the rings hold all rows' sums");
      float* const stage = reinterpret_cast<float*>(sm + kOffK) + (size_t)warp * 32 * kPitch;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float o[32];
        tmem_ld32(o_col + c * 32, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4*>(stage + lane * kPitch + c * 32 + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      }
      __syncwarp();
      const int of = a.Hq / a.Hk;
      auto slot = [&](int row) {                       // of a row of the tile; -1: none there
        const int f = info.row0 + t * tile_rows + row;
        return row < tile_rows && f < info.cnt
                   ? ((int64_t)(info.b0 + f / of) * a.Hq + info.head0 + f % of) * (a.Sp + a.Ss) + info.part
                   : (int64_t)-1;
      };
      const int64_t mine = slot(quarter * 32 + lane);
      if (mine >= 0) a.ws_ml[mine] = make_float2(m_used, l);
#pragma unroll 8
      for (int n = 0; n < 32; ++n) {
        const int64_t at = __shfl_sync(0xffffffffu, mine, n);
        if (at >= 0)
          *reinterpret_cast<float4*>(a.ws_acc + at * kD + lane * 4) =
              *reinterpret_cast<const float4*>(stage + n * kPitch + lane * 4);
      }
    } else if (!ok && lane == 0) {
      flag(a.status, HYB_DEVERR_TIMEOUT);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

int prefix_tc_tile_rows(int rep) { return rep * (kBM / rep); }

cudaError_t launch_prefix_tc(const void* q, const void* kc, const void* vc, const PrefixArgs& a, cudaStream_t s) {
  const int rep = a.Hq / a.Hk, tile_rows = prefix_tc_tile_rows(rep);
  const int64_t pairs = ((int64_t)a.max_group * rep + 2 * tile_rows - 1) / (2 * tile_rows);
  const int64_t ctas = (int64_t)a.G * a.Hk * a.Sp * pairs;
  if (ctas == 0) return cudaSuccess;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  CUtensorMap mq, mk, mv;
  const uint64_t qdims[3] = {(uint64_t)kD, (uint64_t)a.Hq, (uint64_t)a.B};
  const uint64_t qstr[2] = {(uint64_t)kD * 2, (uint64_t)a.Hq * kD * 2};
  const uint32_t qbox[3] = {64, (uint32_t)rep, (uint32_t)(tile_rows / rep)};
  const uint64_t cdims[2] = {(uint64_t)kD, (uint64_t)a.NB * a.Hk * (kBlockSize << a.rsh)};
  const uint64_t cstr[1] = {(uint64_t)kD * 2};
  const uint32_t cbox[2] = {64, kBlockSize};
  if (!encode_tmap_bf16(&mq, q, 3, qdims, qstr, qbox) || !encode_tmap_bf16(&mk, kc, 2, cdims, cstr, cbox) ||
      !encode_tmap_bf16(&mv, vc, 2, cdims, cstr, cbox))
    return cudaErrorInvalidValue;
  const auto kernel = a.window > 0 ? prefix_tc_kernel<true> : prefix_tc_kernel<false>;
  cudaError_t e = set_smem((const void*)kernel, kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3((unsigned)ctas), dim3(kThreads), kSmem, s, mq, mk, mv, a, (int)pairs, tile_rows);
  count_launch();
  return e;
}

}  // namespace hyb
