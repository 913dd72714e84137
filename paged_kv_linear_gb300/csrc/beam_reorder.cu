// Reordering of beams (hyb_beam_reorder): tables, lengths and state slots move by permutation,
// cached tokens and states are copied only for a beam's second and later children.
//
// Two kernels, the copies first: they go by the old tables and slots, and each CTA works out for itself from
// its request's W parents what its row gets from where (a load and some votes). The permutation follows in
// place; it reads and sorts while the copies run, and writes once they have ended (the other way round, with a list of
// the copies in memory: 16.5 us against 7.2 for one request of 4 beams in 4 layers).
//
// Bound by the bytes that are copied, each read once and written once: 16 x 4 beams in 8 layers, up to 1024 tokens, 828
// MB 127 us, 0.96 of the copy rate; 32 x 8 beams in two Linear layers, 755 MB 107 us, 1.04. Eight vectors of 16 bytes a
// thread in flight (one: 150 us for the former). Streaming loads and stores: the next step reads other layers first.
#include <vector>

#include "hyb_internal.cuh"

namespace hyb {
namespace {

constexpr int kMaxBeams = 128, kMaxLayers = 96;
constexpr int kCols = 32;                // table columns of a CTA

// What the request's next beam i gets: the row of old beam `seat`, and a copy of old beam `from`'s data there
// (-1: none, the row's own data go on or there is no parent).
struct Move {
  int seat, from;
};

// Whole CTA (a multiple of 32 threads, W <= kMaxBeams): beam i's move, the same in all threads, or with i < 0
// that of beam threadIdx.x (of those below W). Bits over the beams: `first`, the first children of their
// parents; `child`, the beams that have some. The k-th beam that is not a first child gets the k-th
// beam's row that has none.
__device__ __forceinline__ Move moves(const int32_t* __restrict__ parents, int W, int i, int* par, unsigned* bits,
                                      unsigned* status) {
  const int tid = threadIdx.x;
  unsigned *rest = bits, *child = bits + kMaxBeams / 32;
  if (tid < 2 * kMaxBeams / 32) bits[tid] = 0;
  for (int j = tid; j < W; j += blockDim.x) {
    int p = parents[j];
    if (p < -1 || p >= W) {
      flag(status, HYB_DEVERR_BAD_VALUE);
      p = -1;
    }
    par[j] = p;
  }
  __syncthreads();
  for (int j = tid; j < W; j += blockDim.x) {
    const int p = par[j];
    bool first = p >= 0;
    for (int k = 0; k < j && first; ++k) first = par[k] != p;
    if (!first) atomicOr(&rest[j / 32], 1u << (j % 32));
    if (p >= 0) atomicOr(&child[p / 32], 1u << (p % 32));
  }
  __syncthreads();
  const int me = i < 0 ? min(tid, W - 1) : i;
  Move mv{par[me], -1};
  if ((rest[me / 32] >> (me % 32)) & 1) {
    int k = __popc(rest[me / 32] & ((1u << (me % 32)) - 1));
    for (int w = 0; w < me / 32; ++w) k += __popc(rest[w]);
    int w = 0;                             // the k-th beam without children (there are as many as in `rest`)
    unsigned none = ~child[0];
    while (k >= __popc(none)) {
      k -= __popc(none);
      none = ~child[++w];
    }
    for (; k > 0; --k) none &= none - 1;
    mv.from = mv.seat;
    mv.seat = w * 32 + __ffs(none) - 1;
  }
  return mv;
}

// grid (table columns / 32, at least 1; R). early: behind this call's copies, which write nothing that is read here
__global__ void __launch_bounds__(kMaxBeams)
beam_seat_kernel(const int32_t* __restrict__ parents, int32_t* __restrict__ bt, int32_t* __restrict__ lens,
                 const int32_t* __restrict__ pre, int32_t* __restrict__ slots, int W, int MB, int bs, int early,
                 unsigned* status) {
  __shared__ int par[kMaxBeams], seat[kMaxBeams];
  __shared__ unsigned bits[2 * kMaxBeams / 32];
  __shared__ int32_t strip[kMaxBeams][kCols];
  if (!early) pdl_wait();
  const int r = blockIdx.y, tid = threadIdx.x, row0 = r * W;
  const Move mv = moves(parents + row0, W, -1, par, bits, blockIdx.x == 0 ? status : nullptr);
  seat[tid] = mv.seat;
  int n = 0, sl = 0;
  if (blockIdx.x == 0 && tid < W) {
    if (lens) n = lens[row0 + (par[tid] >= 0 ? par[tid] : mv.seat)];
    if (slots) sl = slots[row0 + mv.seat];
  }
  const int c0 = max((int)blockIdx.x * kCols, pre ? max(pre[r], 0) / bs : 0);
  const int c1 = bt ? min(MB, (int)(blockIdx.x + 1) * kCols) : 0, col = c0 + (tid & 31);
  for (int w = tid >> 5; w < W; w += kMaxBeams / 32)
    if (col < c1) strip[w][tid & 31] = bt[(int64_t)(row0 + w) * MB + col];
  __syncthreads();
  if (early) pdl_wait();                   // the copies go by the old tables, lengths and slots
  pdl_trigger();
  if (blockIdx.x == 0 && tid < W) {
    if (lens) lens[row0 + tid] = n;
    if (slots) slots[row0 + tid] = sl;
  }
  for (int w = tid >> 5; w < W; w += kMaxBeams / 32)
    if (col < c1) bt[(int64_t)(row0 + w) * MB + col] = strip[seat[w]][tid & 31];
}

struct Layer {
  void *a, *b;                           // K and V cache, or the state pool and null
  int slots, window;
};
struct Layers {
  Layer l[kMaxLayers];
};

constexpr int kCopyThreads = 256, kU = 8;   // vectors of a thread in flight

// grid (pieces, rows, layers): what row blockIdx.y's beam gets of its parent's state or tokens. A CTA takes every
// gridDim.x-th piece: of the tokens 16 of all heads, of a state 32 KiB.
__global__ void __launch_bounds__(kCopyThreads)
beam_copy_kernel(const __grid_constant__ Layers layers, const int32_t* __restrict__ parents,
                 const int32_t* __restrict__ bt, const int32_t* __restrict__ lens, const int32_t* __restrict__ pre,
                 const int32_t* __restrict__ slots, int W, int64_t state_vecs, int max_suffix, int H, int vpr, int NB,
                 int MB, int bs, unsigned* status) {
  __shared__ int par[kMaxBeams];
  __shared__ unsigned bits[2 * kMaxBeams / 32];
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.y / W, tid = threadIdx.x;
  const Move mv = moves(parents + (int64_t)r * W, W, blockIdx.y - r * W, par, bits, nullptr);
  if (mv.from < 0) return;
  const int src = r * W + mv.from, dst = r * W + mv.seat;
  const Layer ly = layers.l[blockIdx.z];
  const bool says = blockIdx.x == 0 && tid == 0;
  if (!ly.b) {
    const int s0 = slots[src], s1 = slots[dst];
    if (s0 < 0 || s0 >= ly.slots || s1 < 0 || s1 >= ly.slots) {
      if (says) flag(status, HYB_DEVERR_BAD_STATE);
      return;
    }
    const uint4* x = static_cast<const uint4*>(ly.a) + s0 * state_vecs;
    uint4* y = static_cast<uint4*>(ly.a) + s1 * state_vecs;
    constexpr int kPiece = kCopyThreads * kU;
    for (int64_t i0 = (int64_t)blockIdx.x * kPiece + tid; i0 < state_vecs; i0 += (int64_t)gridDim.x * kPiece) {
      uint4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (i0 + u * kCopyThreads < state_vecs) v[u] = __ldcs(x + i0 + u * kCopyThreads);
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (i0 + u * kCopyThreads < state_vecs) __stcs(y + i0 + u * kCopyThreads, v[u]);
    }
    return;
  }
  const int P = pre ? max(pre[r], 0) : 0, n = lens[src];
  if ((int64_t)n - P > max_suffix || n > min((int64_t)MB * bs, (int64_t)1 << 30)) {
    if (says) flag(status, HYB_DEVERR_BAD_LENGTH);
    return;
  }
  // the next token is number n: a window of W ending there starts at n + 1 - W
  const int lo = ly.window > 0 ? max(P, n + 1 - ly.window) : P;
  const int64_t head = (int64_t)bs * vpr;
  for (int t = (lo & ~15) + blockIdx.x * 16; t < n; t += gridDim.x * 16) {
    const int p0 = bt[(int64_t)src * MB + t / bs], p1 = bt[(int64_t)dst * MB + t / bs];
    if (p0 < 0 || p0 >= NB || p1 < 0 || p1 >= NB) {
      if (tid == 0) flag(status, HYB_DEVERR_BAD_BLOCK);
      continue;
    }
    const int a = max(lo, t), vecs = (min(n, t + 16) - a) * vpr;
    const int64_t x0 = p0 * H * head + (int64_t)(a % bs) * vpr, y0 = p1 * H * head + (int64_t)(a % bs) * vpr;
    for (int e = tid; e < vecs; e += kCopyThreads)
      for (int h0 = 0; h0 < H; h0 += kU / 2) {
        uint4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (h0 + u / 2 < H) v[u] = __ldcs(static_cast<const uint4*>(u & 1 ? ly.b : ly.a) + x0 + (h0 + u / 2) * head + e);
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (h0 + u / 2 < H) __stcs(static_cast<uint4*>(u & 1 ? ly.b : ly.a) + y0 + (h0 + u / 2) * head + e, v[u]);
      }
  }
}

bool al(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace hyb

using namespace hyb;

extern "C" {

size_t hyb_beam_reorder_workspace_size(int32_t, int32_t) { return 0; }

hyb_status_t hyb_beam_reorder(const int32_t* parents, int32_t* block_tables, int32_t* seq_lens,
                              const int32_t* prefix_lens, int32_t* state_slots,
                              const int32_t* layer_types, int32_t L, const hyb_layer_io_t* layers,
                              int32_t R, int32_t W, int32_t max_suffix_len, int64_t state_size,
                              const hyb_attn_dims_t* d, void* workspace, size_t ws_bytes,
                              void* stream) {
  const hyb_status_t st = check_dims(d);
  if (st != HYB_OK) return st;
  if (R < 0 || W <= 0 || L < 0 || max_suffix_len < 0 || (L > 0 && (!layer_types || !layers)))
    return HYB_ERR_INVALID_ARG;
  if (d->window != 0) return HYB_ERR_INVALID_ARG;          // windows come from the layer types
  if (W > kMaxBeams || (int64_t)R * W > 65535 || L > 65535) return HYB_ERR_UNSUPPORTED;
  bool full = false, linear = false;
  std::vector<const void*> pools;                          // each layer owns its own
  pools.reserve(2 * (size_t)L);
  for (int l = 0; l < L; ++l) {
    const hyb_layer_io_t& io = layers[l];
    const int lt = layer_types[l];
    if (lt == HYB_SLIDING ? io.window <= 0 : io.window != 0) return HYB_ERR_INVALID_ARG;
    if (lt == HYB_FULL || lt == HYB_SLIDING) {
      if (!io.k_cache || !io.v_cache || !al(io.k_cache, 16) || !al(io.v_cache, 16)) return HYB_ERR_INVALID_ARG;
      pools.push_back(io.k_cache);
      pools.push_back(io.v_cache);
      full = true;
    } else if (lt == HYB_LINEAR) {
      if (!io.state_pool || !al(io.state_pool, 16) ||
          io.num_state_slots <= 0 || state_size <= 0 || state_size % 4 != 0)
        return HYB_ERR_INVALID_ARG;
      if (state_size > ((int64_t)1 << 40) / io.num_state_slots) return HYB_ERR_UNSUPPORTED;
      pools.push_back(io.state_pool);
      linear = true;
    } else {
      return HYB_ERR_INVALID_ARG;
    }
  }
  std::sort(pools.begin(), pools.end());
  if (std::adjacent_find(pools.begin(), pools.end()) != pools.end()) return HYB_ERR_INVALID_ARG;
  if (R == 0) return HYB_OK;
  if (!parents || !al(parents, 4) || !al(block_tables, 4) || !al(seq_lens, 4) || !al(prefix_lens, 4) ||
      !al(state_slots, 4))
    return HYB_ERR_INVALID_ARG;
  if ((full && (!block_tables || !seq_lens)) || (linear && !state_slots)) return HYB_ERR_INVALID_ARG;
  (void)workspace;
  (void)ws_bytes;
  unsigned* sw = status_word();
  if (!sw) return HYB_ERR_CUDA;
  const cudaStream_t s = (cudaStream_t)stream;
  const int MB = d->max_blocks_per_seq, bs = d->block_size, esize = d->dtype == HYB_BF16 ? 2 : 4;
  // Pieces of a row and layer, each a CTA's: 16 of them fill the GPU from a handful of copies on, and a long
  // state or answer has more work for each.
  const int pieces = 16;
  cudaError_t e = cudaSuccess;
  for (int l0 = 0; l0 < L && e == cudaSuccess; l0 += kMaxLayers) {
    Layers ls = {};
    const int n = std::min(kMaxLayers, L - l0);
    for (int l = 0; l < n; ++l) {
      const hyb_layer_io_t& io = layers[l0 + l];
      ls.l[l] = layer_types[l0 + l] == HYB_LINEAR ? Layer{io.state_pool, nullptr, io.num_state_slots, 0}
                                                  : Layer{io.k_cache, io.v_cache, 0, io.window};
    }
    e = launch_pdl(beam_copy_kernel, dim3(pieces, R * W, n), dim3(kCopyThreads), 0, s, ls, parents,
                   (const int32_t*)block_tables, (const int32_t*)seq_lens, prefix_lens, (const int32_t*)state_slots, W,
                   state_size / 4, max_suffix_len, d->num_heads, d->head_dim * esize / 16, d->num_blocks, MB, bs, sw);
    count_launch();
  }
  if (e != cudaSuccess) return cuda_status(e);
  e = launch_pdl(beam_seat_kernel, dim3(block_tables ? (MB + kCols - 1) / kCols : 1, R), dim3(kMaxBeams), 0, s, parents,
                 block_tables, seq_lens, prefix_lens, state_slots, W, MB, bs, L > 0 ? 1 : 0, sw);
  count_launch();
  return cuda_status(e);
}

}  // extern "C"
