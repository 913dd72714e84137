// Decode attention of groups of requests with a common prefix (hyb_paged_attn_decode_shared_prefix): the entry point,
// how the keys are cut into parts, the kernels without matrix instructions, and the one that joins the parts.
//
// Bytes bound it: a group's common keys and values once, each request's own, and for large groups the tensor
// core (4 D flop a row and key). A part's kernel reads its keys for as many rows as there are:
//   bf16, D = 64, 128, 256: shared_prefix_mma.cu, up to 64 rows a CTA, and every row's own tokens
//   bf16, D = 128, more than 64 rows of a key head: shared_prefix_tc.cu (96 rows on 8192 tokens, 4 groups of 8 key
//   heads: 45 us against 73 on warp matrix instructions; at 64 rows both take 46)
//   the others: prefix_tile_kernel and prefix_part_kernel below, in fp32
// Then prefix_join_kernel adds the parts' states up. Time of a call in a stream of calls (inputs larger than L2): 4 beams
// on 4096 tokens, 32 heads 17.8 us (10.0 at the copy rate); 64 requests behind 2048 tokens, 80 % short and 20 % long
// answers up to 2048 85 us (68); 16 prompts of up to 8192 tokens, 8 beams, 32 query and 8 key heads 61 us (48); 256
// requests on 32768 tokens, 32 and 8 heads 122 us (72 at the tensor rate); the same of hyb_paged_attn_decode, which reads
// the prefix for each request (32 key heads): 4 beams on 4096 tokens 38 us.
#include <cuda_bf16.h>

#include <cmath>

#include "shared_prefix.cuh"

namespace hyb {
namespace {

template <typename T>
struct Row;
template <>
struct Row<__nv_bfloat16> {
  static constexpr int VEC = 8;
  __device__ static void unpack(const uint4& u, float* f) {
    f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x); f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
    f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z); f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
  }
  __device__ static float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
};
template <>
struct Row<float> {
  static constexpr int VEC = 4;
  __device__ static void unpack(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  __device__ static float one(const float* p) { return *p; }
  __device__ static void store(float* p, float x) { *p = x; }
};

constexpr int kU = 4;                    // keys of a lane group in flight

// One part of one (row, query head): 4 warps take every fourth group of keys, D / VEC lanes a key. For types and heads
// without matrix instructions (fp32, heads of 16 and 32); the group's rows meet its keys in L2.
template <typename T, int D>
__global__ void __launch_bounds__(128)
prefix_part_kernel(const T* __restrict__ q, const T* __restrict__ kc, const T* __restrict__ vc,
                   const PrefixArgs a, int part0) {
  constexpr int VEC = Row<T>::VEC, LPR = D / VEC, KPW = 32 / LPR;   // keys of a warp's load
  __shared__ float red[4][D];
  __shared__ float2 red_ml[4];
  pdl_wait();
  pdl_trigger();
  const int part = part0 + blockIdx.x, b = blockIdx.y, h = blockIdx.z, hk = h / (a.Hq / a.Hk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LPR, rr = lane / LPR;
  const RowSpan r = find_row(a, b);
  if (r.n < 0) return;
  const bool shared = part < a.Sp;
  if (shared ? !r.prefix_part(part, a.Lp) : part - a.Sp >= r.own_parts(a.Ls)) return;
  int lo, hi;
  if (shared) {
    lo = max(part * a.Lp, r.lo);
    hi = min((part + 1) * a.Lp, min(r.P, r.n));
  } else {
    const int base = r.own_base() + (part - a.Sp) * a.Ls;
    lo = max(base, r.own_lo());
    hi = min(base + a.Ls, r.n);
  }
  const int bs = kBlockSize << a.rsh;
  const int32_t* table = a.bt + (int64_t)(shared ? r.first : b) * a.MB;
  float qf[VEC], acc[VEC] = {}, m = -INFINITY, l = 0.f;
  Row<T>::unpack(*reinterpret_cast<const uint4*>(q + ((int64_t)b * a.Hq + h) * D + c * VEC), qf);
#pragma unroll
  for (int e = 0; e < VEC; ++e) qf[e] *= a.q_sign ? -a.scale_log2 : a.scale_log2;
  for (int p0 = lo + warp * KPW; p0 < hi; p0 += kU * 4 * KPW) {
    // kU keys of a lane group at once: block ids, then rows, then their scores
    uint4 kr[kU], vr[kU];
    bool ok[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int p = p0 + u * 4 * KPW + rr;
      const int pb = p < hi ? table[p / bs] : 0;
      ok[u] = p < hi && pb >= 0 && pb < a.NB;
      if (p < hi && !ok[u] && c == 0) flag(a.status, HYB_DEVERR_BAD_BLOCK);
      const int64_t at = (((int64_t)pb * a.Hk + hk) * bs + p % bs) * D + c * VEC;
      if (ok[u]) {
        kr[u] = *reinterpret_cast<const uint4*>(kc + at);
        vr[u] = *reinterpret_cast<const uint4*>(vc + at);
      }
    }
    float s[kU], mn = m;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float kf[VEC];
      s[u] = 0.f;
      if (ok[u]) {
        Row<T>::unpack(kr[u], kf);
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[u] = fmaf(qf[e], kf[e], s[u]);
      }
#pragma unroll
      for (int o = LPR / 2; o >= 1; o >>= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
      if (ok[u]) mn = fmaxf(mn, s[u]);
    }
    const float al = m == -INFINITY ? 0.f : fast_exp2(m - mn);
    l *= al;
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] *= al;
    m = mn;
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (ok[u]) {
        float vf[VEC];
        Row<T>::unpack(vr[u], vf);
        const float w = s[u] == -INFINITY ? 0.f : fast_exp2(s[u] - mn);
        l += w;
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = fmaf(w, vf[e], acc[e]);
      }
  }
  // the warp's key groups, then the warps
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
    const float M = fmaxf(m, m2);
    const float x = m == -INFINITY ? 0.f : fast_exp2(m - M), y = m2 == -INFINITY ? 0.f : fast_exp2(m2 - M);
    l = l * x + l2 * y;
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = acc[e] * x + __shfl_xor_sync(0xffffffffu, acc[e], o) * y;
    m = M;
  }
  if (rr == 0)
#pragma unroll
    for (int e = 0; e < VEC; ++e) red[warp][c * VEC + e] = acc[e];
  if (lane == 0) red_ml[warp] = make_float2(m, l);
  __syncthreads();
  const int64_t o = ((int64_t)b * a.Hq + h) * (a.Sp + a.Ss) + part;
  const float M = fmaxf(fmaxf(red_ml[0].x, red_ml[1].x), fmaxf(red_ml[2].x, red_ml[3].x));
  for (int t = threadIdx.x; t < D; t += 128) {
    float A = 0.f, Lsum = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float x = red_ml[w].x == -INFINITY ? 0.f : fast_exp2(red_ml[w].x - M);
      A += x * red[w][t];
      Lsum += x * red_ml[w].y;
    }
    a.ws_acc[o * D + t] = A;
    if (t == 0) a.ws_ml[o] = make_float2(M, Lsum);
  }
}

// ---- a group's rows against its keys without matrix instructions
constexpr int kTileRows = 16, kTileKeys = 32;  // rows of a CTA, four a warp; keys of a stage, one a lane

template <typename T, int D>
struct TileShape {
  static constexpr int VEC = Row<T>::VEC, VPR = D / VEC;         // 16-byte vectors of a row
  static constexpr int KP = D + VEC;                             // pitch of K: a lane reads its key's row
  static constexpr int K = kTileKeys * KP * (int)sizeof(T), V = kTileKeys * D * (int)sizeof(T);
  static constexpr int Q = kTileRows * D * 4, P = kTileKeys * kTileRows * 4;
  static constexpr int SMEM = 2 * (K + V) + Q + P + 2 * kTileKeys * 4;
};

__device__ __forceinline__ void cp16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}

// grid (((group Hk + key head) tiles + row tile) Sp + part): 16 rows of the group (request, query head of the key
// head) against the part's keys, 32 at a time through two stages in shared memory. A lane scores one key for
// its warp's four rows, the weights go through shared memory, and a lane sums D / 32 columns. Bound by shared memory's
// reads (8 cycles of them to 16 of products for the scores), not by L2, as with a row a CTA: 64 requests of 8 heads
// of 128, fp32, on 4096 common tokens: 257 us so, 92 here.
template <typename T, int D>
__global__ void __launch_bounds__(128)
prefix_tile_kernel(const T* __restrict__ q, const T* __restrict__ kc, const T* __restrict__ vc, const PrefixArgs a,
                   int tiles) {
  using S = TileShape<T, D>;
  constexpr int VEC = S::VEC, E = D / 32 > 0 ? D / 32 : 1, RW = kTileRows / 4;
  extern __shared__ __align__(16) uint8_t smem[];
  float* qs = reinterpret_cast<float*>(smem + 2 * (S::K + S::V));                // [16][D], times the scale
  float* ps = qs + kTileRows * D;                                               // [4 warps][32 keys][4 rows]
  int* there = reinterpret_cast<int*>(ps + kTileKeys * kTileRows);              // [2 stages][32 keys]
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rep = a.Hq / a.Hk;
  int i = blockIdx.x;
  const int part = i % a.Sp;
  i /= a.Sp;
  const int row0 = i % tiles * kTileRows;
  i /= tiles;
  const int hk = i % a.Hk;
  int b0, b1, P;
  if (!group_ok(a, i / a.Hk, b0, b1, P)) return;
  const int rows = min(kTileRows, (b1 - b0) * rep - row0);
  int k0 = part * a.Lp, k1 = min(P, k0 + a.Lp);
  if (rows <= 0 || k0 >= k1) return;
  // keys that the warp's rows see, and those of the tile's requests
  int lo[RW], hi[RW];
  const int q0 = b0 + row0 / rep, q1 = b0 + (row0 + rows - 1) / rep + 1;
  Hull seen;
  for (int b = q0 + lane; b < q1; b += 32) seen.add(a, a.lens[b], P);
  seen.join();
  k0 = max(k0, seen.lo);
  k1 = min(k1, seen.hi);
  if (k0 >= k1) return;                        // (the same in every warp)
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    const int f = warp * RW + r;
    lo[r] = hi[r] = 0;
    if (f < rows) {
      const RowSpan x = row_span(a, a.lens[b0 + (row0 + f) / rep], 0, P);
      lo[r] = x.lo;
      hi[r] = min(P, x.n);
    }
  }
  const float scale = a.q_sign ? -a.scale_log2 : a.scale_log2;
  for (int e = tid; e < kTileRows * S::VPR; e += 128) {
    const int r = e / S::VPR, c = e % S::VPR, f = row0 + r;
    float x[VEC] = {};
    if (r < rows)
      Row<T>::unpack(*reinterpret_cast<const uint4*>(q + ((int64_t)(b0 + f / rep) * a.Hq + hk * rep + f % rep) * D + c * VEC), x);
#pragma unroll
    for (int v = 0; v < VEC; ++v) qs[r * D + c * VEC + v] = x[v] * scale;
  }
  const int bs = kBlockSize << a.rsh;
  const int32_t* table = a.bt + (int64_t)b0 * a.MB;
  auto fetch = [&](int t, int st) {            // keys k0 + 32 t on into stage st; those that are not there as zeros
    T* ks = reinterpret_cast<T*>(smem + st * (S::K + S::V));
    T* vs = ks + kTileKeys * S::KP;
    constexpr int N = (kTileKeys * S::VPR + 127) / 128;
    int pb[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int e = tid + n * 128, p = k0 + t * kTileKeys + e / S::VPR;
      pb[n] = e < kTileKeys * S::VPR && p < k1 ? table[p / bs] : -1;
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int e = tid + n * 128, k = e / S::VPR, c = e % S::VPR, p = k0 + t * kTileKeys + k;
      if (e >= kTileKeys * S::VPR) break;
      const bool want = p < k1 && (!seen.gaps || any_sees(a, q0, q1, P, p, p + 1));
      const bool ok = want && pb[n] >= 0 && pb[n] < a.NB;
      if (want && !ok && c == 0) flag(a.status, HYB_DEVERR_BAD_BLOCK);
      const int64_t at = ok ? (((int64_t)pb[n] * a.Hk + hk) * bs + p % bs) * D + c * VEC : 0;
      cp16(ks + k * S::KP + c * VEC, kc + at, ok);
      cp16(vs + k * D + c * VEC, vc + at, ok);
      if (c == 0) there[st * kTileKeys + k] = ok;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float m[RW], l[RW], acc[RW][E];
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[r][e] = 0.f;
  }
  const int nt = (k1 - k0 + kTileKeys - 1) / kTileKeys;
  fetch(0, 0);
  for (int t = 0; t < nt; ++t) {
    const int st = t & 1;
    if (t + 1 < nt) {
      fetch(t + 1, st ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const T* ks = reinterpret_cast<const T*>(smem + st * (S::K + S::V));
    const T* vs = ks + kTileKeys * S::KP;
    const int p = k0 + t * kTileKeys + lane;
    float s[RW] = {};
#pragma unroll 4
    for (int c = 0; c < S::VPR; ++c) {
      float kf[VEC];
      Row<T>::unpack(*reinterpret_cast<const uint4*>(ks + lane * S::KP + c * VEC), kf);
#pragma unroll
      for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int v = 0; v < VEC; v += 4) {
          const float4 x = *reinterpret_cast<const float4*>(qs + (warp * RW + r) * D + c * VEC + v);
          s[r] = fmaf(x.x, kf[v], s[r]);
          s[r] = fmaf(x.y, kf[v + 1], s[r]);
          s[r] = fmaf(x.z, kf[v + 2], s[r]);
          s[r] = fmaf(x.w, kf[v + 3], s[r]);
        }
    }
    const bool ok = there[st * kTileKeys + lane];
    float w[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const bool see = ok && p >= lo[r] && p < hi[r];
      float mx = see ? s[r] : -INFINITY;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[r], mx), al = m[r] == -INFINITY ? 0.f : fast_exp2(m[r] - mn);
      w[r] = !see || s[r] == -INFINITY ? 0.f : fast_exp2(s[r] - mn);     // (NaN comes through)
      m[r] = mn;
      l[r] = fmaf(l[r], al, w[r]);             // of this lane's keys
#pragma unroll
      for (int e = 0; e < E; ++e) acc[r][e] *= al;
    }
    *reinterpret_cast<float4*>(ps + (warp * kTileKeys + lane) * RW) = make_float4(w[0], w[1], w[2], w[3]);
    __syncwarp();
    if (lane * E < D) {
#pragma unroll 8
      for (int k = 0; k < kTileKeys; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(ps + (warp * kTileKeys + k) * RW);
        float vf[E];
#pragma unroll
        for (int e = 0; e < E; ++e) vf[e] = Row<T>::one(vs + k * D + lane * E + e);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          acc[0][e] = fmaf(x.x, vf[e], acc[0][e]);
          acc[1][e] = fmaf(x.y, vf[e], acc[1][e]);
          acc[2][e] = fmaf(x.z, vf[e], acc[2][e]);
          acc[3][e] = fmaf(x.w, vf[e], acc[3][e]);
        }
      }
    }
    __syncthreads();                           // the stage is free for the next copies
  }
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    float ls = l[r];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
    const int f = row0 + warp * RW + r;
    if (warp * RW + r >= rows) continue;
    const int64_t at = ((int64_t)(b0 + f / rep) * a.Hq + hk * rep + f % rep) * (a.Sp + a.Ss) + part;
    if (lane == 0) a.ws_ml[at] = make_float2(m[r], ls);
    if (lane * E < D)
#pragma unroll
      for (int e = 0; e < E; ++e) a.ws_acc[at * D + lane * E + e] = acc[r][e];
  }
}

constexpr int kJoinWarps = 4;

// Joins the parts of a (row, query head), one a warp, D / 32 columns a lane. early: behind a parts' kernel of the same
// call; what says which parts a row has was there before that one began, so it is read before that one
// ends. The first CTA also reports bad groups.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
prefix_join_kernel(T* __restrict__ out, const PrefixArgs a, int early) {
  constexpr int E = D / 32 > 0 ? D / 32 : 1, kBatch = E <= 4 ? 12 : 6;   // parts whose loads are in flight together
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x, h = blockIdx.y * kJoinWarps + warp;
  if (!early) pdl_wait();
  pdl_trigger();
  if (b == 0 && blockIdx.y == 0)
    for (int g = threadIdx.x; g < a.G; g += kJoinWarps * 32) {
      int b0, b1, P;
      if (!group_ok(a, g, b0, b1, P)) flag(a.status, HYB_DEVERR_BAD_LENGTH);
    }
  bool bad;
  const RowSpan r = find_row(a, b, &bad);
  if (early) pdl_wait();
  if (r.n < 0) {
    if (bad && h == 0 && lane == 0) flag(a.status, HYB_DEVERR_BAD_LENGTH);
    return;
  }
  if (h >= a.Hq) return;
  const int64_t bh = (int64_t)b * a.Hq + h, S = a.Sp + a.Ss;
  // the used parts: [s0, s0 + np) of the prefix, then the row's own
  const int p1 = min(r.P, r.n), s0 = r.lo / a.Lp, np = p1 > r.lo ? (p1 - 1) / a.Lp - s0 + 1 : 0;
  const int used = np + r.own_parts(a.Ls);
  const float2* ml = a.ws_ml + bh * S;
  const float* acc = a.ws_acc + bh * S * D + lane * E;
  float M = -INFINITY, L = 0.f, A[E] = {};
  for (int u0 = 0; u0 < used; u0 += kBatch) {  // (the sums keep the parts' order)
    float2 v[kBatch];
    float y[kBatch][E];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int u = u0 + i, part = u < np ? s0 + u : a.Sp + u - np;
      v[i] = u < used ? ml[part] : make_float2(-INFINITY, 0.f);
      const float* p = acc + (int64_t)part * D;
#pragma unroll
      for (int e = 0; e < E; ++e) y[i][e] = 0.f;
      if (u >= used) continue;
      if (E >= 4) {
#pragma unroll
        for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(y[i] + e) = *reinterpret_cast<const float4*>(p + e);
      } else if (E == 2) {
        *reinterpret_cast<float2*>(y[i]) = *reinterpret_cast<const float2*>(p);
      } else if (lane < D) {
        y[i][0] = p[0];
      }
    }
    float m = M;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) m = fmaxf(m, v[i].x);
    const float old = M == -INFINITY ? 0.f : fast_exp2(M - m);
    L *= old;
#pragma unroll
    for (int e = 0; e < E; ++e) A[e] *= old;
    M = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float x = v[i].x == -INFINITY ? 0.f : fast_exp2(v[i].x - m);
      L = fmaf(x, v[i].y, L);                  // (NaN comes through, also where no maximum is)
#pragma unroll
      for (int e = 0; e < E; ++e) A[e] = fmaf(x, y[i][e], A[e]);
    }
  }
  if (lane * E < D)
#pragma unroll
    for (int e = 0; e < E; ++e) Row<T>::store(out + bh * D + lane * E + e, L == 0.f ? 0.f : A[e] / L);
}

// Without matrix instructions a group's rows meet its keys in tiles of 16 from 8 rows on; below, a row a CTA is
// quicker (fp32, 8 heads of 128, 4096 common tokens: 4 rows 30 us against 39 in tiles, 8 rows 50 against 39).
bool use_tiles(int64_t rows) { return rows >= 8; }

int round16(int64_t x) { return (int)((x + 15) / 16 * 16); }

PrefixPlan plan_prefix(int B, const hyb_prefix_dims_t* p, const hyb_attn_dims_t* d) {
  PrefixPlan r;
  const int rep = p->num_q_heads / d->num_heads, D = d->head_dim, P = p->max_prefix_len;
  const int64_t rows = (int64_t)p->max_group * rep, heads = (int64_t)p->num_groups * d->num_heads;
  const int sms = num_sms();
  const bool mma = prefix_mma_supported(d->dtype, D);
  r.tc = mma && D == 128 && rep <= 128 && d->scale > 0.f && rows > 64;
  if (r.tc) {
    // one CTA an SM; a key tile of 128 counts as 1.6 us, setup and drain as 8 us, a part's state, written and read once,
    // at 6 TB/s. (The kernel now takes 1.43 and 7 us. With these, 2 % of 20000 random shapes would be cut otherwise, for
    // a gain of 2.6 % at most by this very sum.)
    const int64_t tr = 2 * prefix_tc_tile_rows(rep), units = std::max<int64_t>(1, heads * ((rows + tr - 1) / tr));
    const int tiles = std::max(1, (P + 127) / 128);
    const double state_us = (double)B * p->num_q_heads * (D * 4 + 8) * 2 / 6e6;
    double best = 1e30;
    r.Lp = 128;
    for (int n = 1; n <= std::min(tiles, 64); ++n) {
      const int64_t per = (tiles + n - 1) / n, used = (tiles + per - 1) / per, waves = (units * used + sms - 1) / sms;
      const double t = waves * (1.6 * per + 8.0) + used * state_us;
      if (t < best) {
        best = t;
        r.Lp = (int)per * 128;
      }
    }
  } else if (mma) {
    const int64_t nt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4, units = std::max<int64_t>(1, heads * ((rows + 16 * nt - 1) / (16 * nt)));
    const int64_t slots = (int64_t)sms * (D == 256 ? 1 : 3);   // (D = 256: rings of 128 KiB but for four row tiles)
    r.Lp = round16(std::min<int64_t>(kMmaMaxPart, std::max<int64_t>(nt == 1 ? 512 : 256, P * units / slots)));
  } else if (use_tiles(rows)) {
    // one wave of the CTAs that shared memory holds, if that leaves parts of 128 to 512 keys
    const int es = d->dtype == HYB_BF16 ? 2 : 4, smem = kTileKeys * (4 * D * es + 32) + kTileRows * (D + kTileKeys) * 4 + 256;
    const int64_t units = std::max<int64_t>(1, heads * ((rows + kTileRows - 1) / kTileRows));
    const int64_t n = std::max<int64_t>(1, std::min(227 * 1024 / (smem + 1024), 5) * sms / units);
    r.Lp = (int)std::min<int64_t>(512, std::max<int64_t>(128, (P / n + 32) / 32 * 32));
  } else {
    r.Lp = round16(std::min<int64_t>(256, std::max<int64_t>(64, (int64_t)P * B * p->num_q_heads / (8 * sms))));
  }
  // A row's own tokens: on matrix instructions a warp takes a part of a key head. Parts of 128 where that leaves warps
  // without work (8 requests of 2048 tokens, 8 heads: 14.3 us against 17.5 with 256), else of 256 (64 requests of up
  // to 2048, 32 heads: 87 us against 91 with 128 and 91 with 512).
  const int64_t S = p->max_suffix_len, own_tiles = (rep + 15) / 16;
  if (mma)
    r.Ls = B * (int64_t)d->num_heads * own_tiles * ((S + 255) / 256) < 12 * sms ? 128 : 256;
  else
    r.Ls = round16(std::min<int64_t>(256, std::max<int64_t>(64, S * B * p->num_q_heads / (8 * sms))));
  r.Sp = (P + r.Lp - 1) / r.Lp;
  int own = p->max_suffix_len;
  if (d->window > 0) own = std::min(own, d->window);
  r.Ss = own > 0 ? (own + kBlockSize - 1 + r.Ls - 1) / r.Ls : 0;
  r.ws_bytes = (size_t)B * p->num_q_heads * (r.Sp + r.Ss) * ((size_t)D * 4 + 8);
  return r;
}

template <typename T, int D>
cudaError_t launch_typed(void* out, const void* q, const void* kc, const void* vc, const PrefixArgs& a,
                         bool tc, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if constexpr (sizeof(T) == 2 && (D == 64 || D == 128 || D == 256)) {
    const bool behind = tc && a.Sp > 0;
    if (behind) e = launch_prefix_tc(q, kc, vc, a, s);
    if (e == cudaSuccess) e = launch_prefix_mma(D, q, kc, vc, a, !tc, behind, s);
    if (e != cudaSuccess) return e;
  } else {
    const int rep = a.Hq / a.Hk;
    const int64_t rows = (int64_t)a.max_group * rep, tiles = (rows + kTileRows - 1) / kTileRows;
    const bool tiled = use_tiles(rows) && a.Sp > 0;
    if (tiled && a.G > 0) {
      const int64_t ctas = (int64_t)a.G * a.Hk * tiles * a.Sp;
      if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
      constexpr int smem = TileShape<T, D>::SMEM;
      e = set_smem((const void*)prefix_tile_kernel<T, D>, smem);
      if (e != cudaSuccess) return e;
      e = launch_pdl(prefix_tile_kernel<T, D>, dim3((unsigned)ctas), dim3(128), smem, s, (const T*)q, (const T*)kc,
                     (const T*)vc, a, (int)tiles);
      count_launch();
      if (e != cudaSuccess) return e;
    }
    const int part0 = tiled ? a.Sp : 0, parts = a.Sp + a.Ss - part0;
    if (parts > 0) {
      e = launch_pdl(prefix_part_kernel<T, D>, dim3(parts, a.B, a.Hq), dim3(128), 0, s, (const T*)q, (const T*)kc,
                     (const T*)vc, a, part0);
      count_launch();
      if (e != cudaSuccess) return e;
    }
  }
  e = launch_pdl(prefix_join_kernel<T, D>, dim3(a.B, (a.Hq + kJoinWarps - 1) / kJoinWarps),
                 dim3(kJoinWarps * 32), 0, s, (T*)out, a, (a.Ss > 0 || (a.Sp > 0 && a.max_group > 0)) ? 1 : 0);
  count_launch();
  return e;
}

cudaError_t launch_prefix(int dtype, int D, void* out, const void* q, const void* kc, const void* vc,
                          const PrefixArgs& a, bool tc, cudaStream_t s) {
#define HYB_PRE(T, DD) \
  if (D == DD) return launch_typed<T, DD>(out, q, kc, vc, a, tc, s);
  if (dtype == HYB_BF16) {
    HYB_PRE(__nv_bfloat16, 16)
    HYB_PRE(__nv_bfloat16, 32)
    HYB_PRE(__nv_bfloat16, 64)
    HYB_PRE(__nv_bfloat16, 128)
    HYB_PRE(__nv_bfloat16, 256)
  } else {
    HYB_PRE(float, 16)
    HYB_PRE(float, 32)
    HYB_PRE(float, 64)
    HYB_PRE(float, 128)
  }
#undef HYB_PRE
  return cudaErrorInvalidValue;
}

bool al(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

hyb_status_t check_prefix_dims(int B, const hyb_prefix_dims_t* p, const hyb_attn_dims_t* d) {
  const hyb_status_t st = check_dims(d);
  if (st != HYB_OK) return st;
  if (!p || B < 0 || p->num_q_heads <= 0 || p->num_groups < 0 || p->max_group < 0 ||
      p->max_prefix_len < 0 || p->max_suffix_len < 0)
    return HYB_ERR_INVALID_ARG;
  if (p->num_q_heads % d->num_heads != 0) return HYB_ERR_INVALID_ARG;
  if (!decode_supported(d->dtype, d->head_dim)) return HYB_ERR_UNSUPPORTED;
  if (B > 65535 || p->num_q_heads > 65535 || (int64_t)B * p->num_q_heads >= ((int64_t)1 << 23) ||
      p->num_groups > B + 65535)
    return HYB_ERR_UNSUPPORTED;
  const int64_t cap = (int64_t)d->max_blocks_per_seq * d->block_size;
  if (p->max_prefix_len > cap || p->max_suffix_len > cap || p->max_group > B) return HYB_ERR_INVALID_ARG;
  if (p->max_prefix_len > (1 << 24) || p->max_suffix_len > (1 << 24)) return HYB_ERR_UNSUPPORTED;
  return HYB_OK;
}

}  // namespace
}  // namespace hyb

using namespace hyb;

extern "C" {

size_t hyb_paged_attn_decode_shared_prefix_workspace_size(int32_t B, const hyb_prefix_dims_t* p,
                                                          const hyb_attn_dims_t* d) {
  if (B <= 0 || check_prefix_dims(B, p, d) != HYB_OK) return 0;
  return plan_prefix(B, p, d).ws_bytes;
}

hyb_status_t hyb_paged_attn_decode_shared_prefix(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* seq_lens, const int32_t* cu_groups,
    const int32_t* prefix_lens, int32_t B, const hyb_prefix_dims_t* p, const hyb_attn_dims_t* d,
    void* workspace, size_t ws_bytes, void* stream) {
  const hyb_status_t st = check_prefix_dims(B, p, d);
  if (st != HYB_OK) return st;
  if (B == 0 || p->num_groups == 0) return HYB_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !cu_groups || !prefix_lens)
    return HYB_ERR_INVALID_ARG;
  if (!al(out, 16) || !al(q, 16) || !al(k_cache, 16) || !al(v_cache, 16) || !al(block_tables, 4) ||
      !al(seq_lens, 4) || !al(cu_groups, 4) || !al(prefix_lens, 4))
    return HYB_ERR_INVALID_ARG;
  const PrefixPlan plan = plan_prefix(B, p, d);
  if (plan.ws_bytes > 0 && (!workspace || !al(workspace, 16) || ws_bytes < plan.ws_bytes))
    return HYB_ERR_INVALID_ARG;
  unsigned* sw = status_word();
  if (!sw) return HYB_ERR_CUDA;
  PrefixArgs a;
  a.bt = block_tables;
  a.lens = seq_lens;
  a.cu = cu_groups;
  a.pre = prefix_lens;
  a.B = B;
  a.G = p->num_groups;
  a.Hq = p->num_q_heads;
  a.Hk = d->num_heads;
  a.NB = d->num_blocks;
  a.MB = d->max_blocks_per_seq;
  a.rsh = log2_int(d->block_size / kBlockSize);
  a.window = d->window;
  a.max_group = p->max_group;
  a.max_prefix = p->max_prefix_len;
  a.max_suffix = p->max_suffix_len;
  a.cap = (int)std::min<int64_t>(INT32_MAX, (int64_t)d->max_blocks_per_seq * d->block_size);
  a.scale_log2 = std::max(std::fabs(d->scale) * 1.4426950408889634f, 1e-37f);
  a.q_sign = d->scale < 0.f ? 0x80008000u : 0u;
  a.Lp = plan.Lp;
  a.Sp = plan.Sp;
  a.Ls = plan.Ls;
  a.Ss = plan.Ss;
  a.ws_acc = static_cast<float*>(workspace);
  a.ws_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) +
                                      (size_t)B * a.Hq * (plan.Sp + plan.Ss) * d->head_dim * 4);
  a.status = sw;
  return cuda_status(launch_prefix(d->dtype, d->head_dim, out, q, k_cache, v_cache, a, plan.tc,
                                   (cudaStream_t)stream));
}

}  // extern "C"
