// Reordering of beams (hyb_beam_reorder): tables, lengths and state slots move by permutation,
// cached tokens and states are copied only for a beam's second and later children.
#include <set>

#include "hyb_internal.cuh"

namespace hyb {
namespace {

constexpr int kMaxBeams = 128, kMaxLayers = 96;
constexpr int kCols = 32;                // table columns of a CTA

// Rows of request r's next beams, by all threads: seat[i] (the old row, 0 .. W - 1, whose table
// and slot beam i gets) and from[i] (the beam whose row holds the data to copy there, -1: none).
__device__ __forceinline__ void seats(const int32_t* __restrict__ parents, int W, int* par, int* seat, int* from,
                                      unsigned* status) {
  const int tid = threadIdx.x;
  for (int i = tid; i < W; i += blockDim.x) {
    int p = parents[i];
    if (p < -1 || p >= W) {
      flag(status, HYB_DEVERR_BAD_VALUE);
      p = -1;
    }
    par[i] = p;
  }
  __syncthreads();
  for (int i = tid; i < W; i += blockDim.x) {
    // first child of its parent? and how many before it are not
    int heir = -1, later = 0;
    const int p = par[i];
    for (int j = 0; j < i; ++j) {
      if (par[j] == p && heir < 0) heir = j;
      bool first = par[j] >= 0;
      for (int k = 0; k < j && first; ++k) first = par[k] != par[j];
      later += !first;
    }
    if (p >= 0 && heir < 0) {
      seat[i] = p;
      from[i] = -1;
    } else {
      int c = -1, left = later;          // the beam without children of that number
      for (int w = 0; w < W && c < 0; ++w) {
        bool child = false;
        for (int k = 0; k < W && !child; ++k) child = par[k] == w;
        if (!child && left-- == 0) c = w;
      }
      seat[i] = c;
      from[i] = p >= 0 ? heir : -1;
    }
  }
  __syncthreads();
}

// grid (table columns / 32, at least 1; R)
__global__ void __launch_bounds__(128)
beam_seat_kernel(const int32_t* __restrict__ parents, int32_t* __restrict__ bt, int32_t* __restrict__ lens,
                 const int32_t* __restrict__ pre, int32_t* __restrict__ slots, int32_t* __restrict__ copy, int W,
                 int MB, int bs, unsigned* status) {
  __shared__ int par[kMaxBeams], seat[kMaxBeams], from[kMaxBeams];
  __shared__ int32_t strip[kMaxBeams][kCols];
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.y, tid = threadIdx.x, row0 = r * W;
  seats(parents + row0, W, par, seat, from, blockIdx.x == 0 ? status : nullptr);
  if (blockIdx.x == 0) {
    int n = 0, sl = 0;
    if (tid < W) {
      if (lens) n = lens[row0 + (par[tid] >= 0 ? par[tid] : seat[tid])];
      if (slots) sl = slots[row0 + seat[tid]];
    }
    __syncthreads();
    if (tid < W) {
      if (lens) lens[row0 + tid] = n;
      if (slots) slots[row0 + tid] = sl;
      copy[row0 + tid] = from[tid] < 0 ? -1 : row0 + from[tid];
    }
  }
  if (!bt) return;
  const int c0 = max((int)blockIdx.x * kCols, pre ? max(pre[r], 0) / bs : 0), c1 = min(MB, (int)(blockIdx.x + 1) * kCols);
  if (c0 >= c1) return;
  const int col = c0 + (tid & 31);
  for (int w = tid >> 5; w < W; w += 4)
    if (col < c1) strip[w][tid & 31] = bt[(int64_t)(row0 + w) * MB + col];
  __syncthreads();
  for (int w = tid >> 5; w < W; w += 4)
    if (col < c1) bt[(int64_t)(row0 + w) * MB + col] = strip[seat[w]][tid & 31];
}

struct Layer {
  void *a, *b;                           // K and V cache, or the state pool and null
  int slots, window;
};
struct Layers {
  Layer l[kMaxLayers];
};

// grid (pieces, rows, layers): row blockIdx.y's copy of its parent's state (pieces of 1024 vectors) or
// tokens (a piece is 16 tokens of all heads)
__global__ void __launch_bounds__(256)
beam_copy_kernel(const __grid_constant__ Layers layers, const int32_t* __restrict__ copy,
                 const int32_t* __restrict__ bt, const int32_t* __restrict__ lens, const int32_t* __restrict__ pre,
                 const int32_t* __restrict__ slots, int W, int64_t state_vecs, int max_suffix, int H, int vpr, int NB,
                 int MB, int bs, unsigned* status) {
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.y, src = copy[row];
  if (src < 0) return;
  const Layer ly = layers.l[blockIdx.z];
  const int tid = threadIdx.x;
  if (!ly.b) {
    const int s0 = slots[src], s1 = slots[row];
    if (s0 < 0 || s0 >= ly.slots || s1 < 0 || s1 >= ly.slots) {
      if (blockIdx.x == 0 && tid == 0) flag(status, HYB_DEVERR_BAD_STATE);
      return;
    }
    const uint4* x = static_cast<const uint4*>(ly.a) + s0 * state_vecs;
    uint4* y = static_cast<uint4*>(ly.a) + s1 * state_vecs;
    for (int64_t i = (int64_t)blockIdx.x * 256 + tid; i < state_vecs; i += (int64_t)gridDim.x * 256) y[i] = x[i];
    return;
  }
  const int P = pre ? max(pre[row / W], 0) : 0, n = lens[src];
  if (n - P > max_suffix || n > (int64_t)MB * bs) {
    if (blockIdx.x == 0 && blockIdx.z == 0 && tid == 0) flag(status, HYB_DEVERR_BAD_LENGTH);
    return;
  }
  // the next token is number n: a window of W ending there starts at n + 1 - W
  const int lo = ly.window > 0 ? max(P, n + 1 - ly.window) : P;
  for (int t = (lo & ~15) + blockIdx.x * 16; t < n; t += gridDim.x * 16) {
    const int p0 = bt[(int64_t)src * MB + t / bs], p1 = bt[(int64_t)row * MB + t / bs];
    if (p0 < 0 || p0 >= NB || p1 < 0 || p1 >= NB) {
      if (tid == 0) flag(status, HYB_DEVERR_BAD_BLOCK);
      continue;
    }
    const int a = max(lo, t), rows = min(n, t + 16) - a, vecs = rows * vpr;
    for (int i = tid; i < 2 * H * vecs; i += 256) {
      const int kv = i / (H * vecs), h = (i - kv * H * vecs) / vecs, e = i % vecs;
      uint4* c = static_cast<uint4*>(kv ? ly.b : ly.a);
      const int64_t off = (int64_t)(a % bs) * vpr + e;
      c[((int64_t)p1 * H + h) * bs * vpr + off] = c[((int64_t)p0 * H + h) * bs * vpr + off];
    }
  }
}

bool al(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace hyb

using namespace hyb;

extern "C" {

size_t hyb_beam_reorder_workspace_size(int32_t R, int32_t W) {
  if (R <= 0 || W <= 0 || W > kMaxBeams || (int64_t)R * W > 65535) return 0;
  return (size_t)R * W * 4;
}

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
  std::set<const void*> seen;                              // each layer owns its pools
  for (int l = 0; l < L; ++l) {
    const hyb_layer_io_t& io = layers[l];
    const int lt = layer_types[l];
    if (lt == HYB_SLIDING ? io.window <= 0 : io.window != 0) return HYB_ERR_INVALID_ARG;
    if (lt == HYB_FULL || lt == HYB_SLIDING) {
      if (!io.k_cache || !io.v_cache || !al(io.k_cache, 16) || !al(io.v_cache, 16) ||
          !seen.insert(io.k_cache).second || !seen.insert(io.v_cache).second)
        return HYB_ERR_INVALID_ARG;
      full = true;
    } else if (lt == HYB_LINEAR) {
      if (!io.state_pool || !al(io.state_pool, 16) || !seen.insert(io.state_pool).second ||
          io.num_state_slots <= 0 || state_size <= 0 || state_size % 4 != 0)
        return HYB_ERR_INVALID_ARG;
      if (state_size > ((int64_t)1 << 40) / io.num_state_slots) return HYB_ERR_UNSUPPORTED;
      linear = true;
    } else {
      return HYB_ERR_INVALID_ARG;
    }
  }
  if (R == 0) return HYB_OK;
  if (!parents || !al(parents, 4) || !al(block_tables, 4) || !al(seq_lens, 4) || !al(prefix_lens, 4) ||
      !al(state_slots, 4))
    return HYB_ERR_INVALID_ARG;
  if ((full && (!block_tables || !seq_lens)) || (linear && !state_slots)) return HYB_ERR_INVALID_ARG;
  if (!workspace || !al(workspace, 4) || ws_bytes < hyb_beam_reorder_workspace_size(R, W))
    return HYB_ERR_INVALID_ARG;
  if (R > 65535) return HYB_ERR_UNSUPPORTED;
  unsigned* sw = status_word();
  if (!sw) return HYB_ERR_CUDA;
  const cudaStream_t s = (cudaStream_t)stream;
  int32_t* copy = static_cast<int32_t*>(workspace);
  const int MB = d->max_blocks_per_seq, bs = d->block_size;
  cudaError_t e = launch_pdl(beam_seat_kernel, dim3(block_tables ? (MB + kCols - 1) / kCols : 1, R), dim3(128), 0, s,
                             parents, block_tables, seq_lens, prefix_lens, state_slots, copy, W, MB, bs, sw);
  count_launch();
  const int esize = d->dtype == HYB_BF16 ? 2 : 4;
  for (int l0 = 0; l0 < L && e == cudaSuccess; l0 += kMaxLayers) {
    Layers ls = {};
    const int n = std::min(kMaxLayers, L - l0);
    for (int l = 0; l < n; ++l) {
      const hyb_layer_io_t& io = layers[l0 + l];
      ls.l[l] = layer_types[l0 + l] == HYB_LINEAR ? Layer{io.state_pool, nullptr, io.num_state_slots, 0}
                                                  : Layer{io.k_cache, io.v_cache, 0, io.window};
    }
    e = launch_pdl(beam_copy_kernel, dim3(16, R * W, n), dim3(256), 0, s, ls, (const int32_t*)copy,
                   (const int32_t*)block_tables, (const int32_t*)seq_lens, prefix_lens, (const int32_t*)state_slots, W,
                   state_size / 4, max_suffix_len, d->num_heads, d->head_dim * esize / 16, d->num_blocks, MB, bs, sw);
    count_launch();
  }
  return cuda_status(e);
}

}  // extern "C"
