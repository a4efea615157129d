// cache_moves.cu -- rows and pages that move within the paged cache: the rows of
// accepted draft nodes up behind the prefix, and whole pages to pages of a forked
// request. Bit-exact copies, in the pools of all layers in one launch (a call per
// layer would cost a launch each for a few kilobytes).
#include <cuda_runtime.h>

#include "pkv_device.cuh"
#include "pkv_fp8.cuh"
#include "pkv_kernels.h"

namespace pkv {
namespace {

// ---------------------------------------------------------------------------- pages
// A page of one pool is contiguous: num_kv_heads * 16 rows. A warp copies a span of 2 KiB of it, four 16-byte loads a
// lane before the first store; the page's scale bytes go with the first span of the K pool.
constexpr int kCopyThreads = 256;
constexpr int kSpanBytes = 4 * 32 * 16;

struct CopyArgs {
  MovePools pools;
  const int* src;
  const int* dst;
  int* status;
  int n, spans, num_pages, page_bytes, scale_bytes;
};

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  grid_dependency_wait();
  allow_dependents();
  const int lane = threadIdx.x & 31;
  const long long units = static_cast<long long>(a.n) * a.spans;
  const int layer = blockIdx.y >> 1, kv = blockIdx.y & 1;
  unsigned char* pool = static_cast<unsigned char*>(kv ? a.pools.v[layer] : a.pools.k[layer]);
  const long long stride = static_cast<long long>(gridDim.x) * (kCopyThreads / 32);
  for (long long u = static_cast<long long>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5); u < units; u += stride) {
    const int pair = static_cast<int>(u / a.spans), span = static_cast<int>(u - static_cast<long long>(pair) * a.spans);
    const int src = __ldg(a.src + pair), dst = __ldg(a.dst + pair);
    if (src < 0 || dst < 0) continue;
    if (src >= a.num_pages || dst >= a.num_pages) {
      if (lane == 0) set_status(a.status, PKV_ERR_OUT_OF_BOUNDS);
      continue;
    }
    const unsigned char* from = pool + static_cast<size_t>(src) * a.page_bytes;
    unsigned char* to = pool + static_cast<size_t>(dst) * a.page_bytes;
    const int at = span * kSpanBytes + lane * 16;
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i * 512 < a.page_bytes) x[i] = __ldcs(reinterpret_cast<const uint4*>(from + at + i * 512));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i * 512 < a.page_bytes) __stcs(reinterpret_cast<uint4*>(to + at + i * 512), x[i]);
    if (span == 0 && kv == 0 && a.scale_bytes > 0) {
      unsigned char* sc = static_cast<unsigned char*>(a.pools.scales[layer]);
      for (int b = lane * 16; b < a.scale_bytes; b += 512)
        *reinterpret_cast<uint4*>(sc + static_cast<size_t>(dst) * a.scale_bytes + b) =
            *reinterpret_cast<const uint4*>(sc + static_cast<size_t>(src) * a.scale_bytes + b);
    }
  }
}

// ---------------------------------------------------------------------------- rows
// A thread takes one 16-byte column of one KV head's rows in one pool and walks the path in order, eight rows at a time,
// loads before stores. A path's numbers rise, so row i of it moves down or stays (path[i] >= i) and the rows that a thread
// has yet to read lie behind all that it has written: no thread needs another's, and nothing is read after it is
// overwritten. A CTA takes 256 columns of a request, across heads, K and V and layers: where the rows lie is worked out
// once for them.
constexpr int kKeepThreads = 256;
constexpr int kMaxPath = 64;
constexpr int kBatch = 8;

struct KeepArgs {
  MovePools pools;
  const int* path;
  const int* path_lens;
  const int* prefix_lens;
  const int* block_table;
  int* status;
  int max_path, max_pages, num_pages, hkv, cols;  // cols: 16-byte columns of a row
  int blocks;                                     // CTAs of a request
  long long columns;                              // of a request: layers * 2 * hkv * cols
};

template <bool kFp8>
__global__ void __launch_bounds__(kKeepThreads) keep_nodes_kernel(const __grid_constant__ KeepArgs a) {
  // the rows to move, in order: (page, slot) in 32 bits each of where from and where to
  __shared__ int from_page[kMaxPath], to_page[kMaxPath], slots[kMaxPath], count;
  grid_dependency_wait();
  allow_dependents();
  const int s = blockIdx.x / a.blocks, part = blockIdx.x - s * a.blocks;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int prefix = __ldg(a.prefix_lens + s), given = __ldg(a.path_lens + s);
    // (entries of the path are read before its length is known: the row is max_path long)
    int node[kMaxPath / 32];
#pragma unroll
    for (int b = 0; b < kMaxPath / 32; ++b)
      node[b] = 32 * b + lane < a.max_path ? __ldg(a.path + static_cast<size_t>(s) * a.max_path + 32 * b + lane) : -1;
    int n = given;
    if (n < 0 || n > a.max_path || prefix < 0) {
      if (lane == 0) set_status(a.status, PKV_ERR_OUT_OF_BOUNDS);
      n = n < 0 || prefix < 0 ? 0 : a.max_path;
    }
    int moves = 0, before = -1;
#pragma unroll
    for (int b = 0; b < kMaxPath / 32; ++b) {
      const int i = 32 * b + lane, x = node[b];
      const int up = __shfl_up_sync(0xffffffffu, x, 1);
      const int prev = lane == 0 ? before : up;
      before = __shfl_sync(0xffffffffu, x, 31);
      bool move = false;
      int p = 0, q = 0;
      const long long at = static_cast<long long>(prefix) + x, put = static_cast<long long>(prefix) + i;
      if (i < n) {
        bool fine = x > prev && x >= i && at < static_cast<long long>(a.max_pages) * kPageSize;
        if (fine) {
          const int* row = a.block_table + static_cast<size_t>(s) * a.max_pages;
          p = __ldg(row + at / kPageSize);
          q = __ldg(row + put / kPageSize);
          fine = p >= 0 && p < a.num_pages && q >= 0 && q < a.num_pages;
          move = fine && x != i;
        }
        if (!fine) set_status(a.status, PKV_ERR_OUT_OF_BOUNDS);
      }
      const unsigned vote = __ballot_sync(0xffffffffu, move);
      if (move) {
        const int m = moves + __popc(vote & ((1u << lane) - 1));
        from_page[m] = p;
        to_page[m] = q;
        slots[m] = static_cast<int>(at % kPageSize) | static_cast<int>(put % kPageSize) << 8;
      }
      moves += __popc(vote);
    }
    if (lane == 0) count = moves;
  }
  __syncthreads();
  const int n = count;
  const long long column = static_cast<long long>(part) * kKeepThreads + threadIdx.x;
  if (column >= a.columns) return;
  const int per = a.hkv * a.cols;  // columns of a pool's row
  const int pool_i = static_cast<int>(column / per), c = static_cast<int>(column - static_cast<long long>(pool_i) * per);
  const int layer = pool_i >> 1, kv = pool_i & 1, h = c / a.cols, col = c - h * a.cols;
  uint4* pool =
      static_cast<uint4*>(kv ? a.pools.v[layer] : a.pools.k[layer]) + static_cast<size_t>(h) * kPageSize * a.cols + col;
  const size_t page_cols = static_cast<size_t>(a.hkv) * kPageSize * a.cols;
  uint8_t* sc = nullptr;
  if (kFp8 && col == 0)
    sc = static_cast<uint8_t*>(a.pools.scales[layer]) + static_cast<size_t>(h) * kScaleBytes + kv * kPageSize;
  const size_t page_scales = static_cast<size_t>(a.hkv) * kScaleBytes;
  for (int b = 0; b < n; b += kBatch) {
    uint4 x[kBatch];
    uint8_t y[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (b + j < n) {
        const int slot = slots[b + j] & 0xff;
        x[j] = pool[from_page[b + j] * page_cols + slot * a.cols];
        if (sc != nullptr) y[j] = sc[from_page[b + j] * page_scales + slot];
      }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (b + j < n) {
        const int slot = slots[b + j] >> 8;
        pool[to_page[b + j] * page_cols + slot * a.cols] = x[j];
        if (sc != nullptr) sc[to_page[b + j] * page_scales + slot] = y[j];
      }
  }
}

}  // namespace

int launch_copy_pages(const MovePools& pools, int layers, bool fp8, const int32_t* src, const int32_t* dst, int n,
                      int num_kv_heads, int head_dim, int32_t num_pages, int* status, cudaStream_t stream) {
  CopyArgs a = {};
  a.pools = pools;
  a.src = src;
  a.dst = dst;
  a.status = status;
  a.n = n;
  a.num_pages = num_pages;
  a.page_bytes = num_kv_heads * kPageSize * head_dim * (fp8 ? 1 : 2);
  a.scale_bytes = fp8 ? num_kv_heads * kScaleBytes : 0;
  a.spans = (a.page_bytes + kSpanBytes - 1) / kSpanBytes;
  const long long units = static_cast<long long>(n) * a.spans;
  long long blocks = (units + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  if (blocks > 65536) blocks = 65536;
  const cudaError_t e = launch_pdl(copy_pages_kernel, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(2 * layers)),
                                   dim3(kCopyThreads), 0, stream, a);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int launch_keep_nodes(const MovePools& pools, int layers, bool fp8, const int32_t* path, const int32_t* path_lens,
                      const int32_t* prefix_lens, const int32_t* block_table, int num_seqs, int max_path, int max_pages,
                      int num_kv_heads, int head_dim, int32_t num_pages, int* status, cudaStream_t stream) {
  KeepArgs a = {};
  a.pools = pools;
  a.path = path;
  a.path_lens = path_lens;
  a.prefix_lens = prefix_lens;
  a.block_table = block_table;
  a.status = status;
  a.max_path = max_path;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.hkv = num_kv_heads;
  a.cols = head_dim * (fp8 ? 1 : 2) / 16;
  a.columns = static_cast<long long>(layers) * 2 * num_kv_heads * a.cols;
  a.blocks = static_cast<int>((a.columns + kKeepThreads - 1) / kKeepThreads);
  const long long grid = static_cast<long long>(num_seqs) * a.blocks;
  if (grid > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  const dim3 g(static_cast<unsigned>(grid)), b(kKeepThreads);
  const cudaError_t e = fp8 ? launch_pdl(keep_nodes_kernel<true>, g, b, 0, stream, a)
                            : launch_pdl(keep_nodes_kernel<false>, g, b, 0, stream, a);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
