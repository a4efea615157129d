// expand_fp8.cu -- pages of the 8-bit cache, by block table, as bf16 pages.
//
// Chunked prefill multiplies bf16 tiles on the tensor cores, so a prompt whose
// prefix is cached in 8 bits has that prefix expanded into a staging pool
// before each of its chunks. A value is 2^e v with v in e4m3 (4 significant
// bits): exact in bf16 for every e of the format, so the staged pages stand for
// the cache bit for bit and prefill and decode see the same keys and values.
//
// A copy: (D + 1) bytes read and 2 D written per row of K and of V, bound by
// memory. One warp takes the K and V tiles of a (page, KV head); lane i holds
// scale byte i of the tile's 32 (16 K rows, 16 V rows). A lane turns 8 bytes
// into 16, so that a warp's loads and its stores are both contiguous, and all
// of a tile pair's loads are issued before the first store.
#include <cuda_runtime.h>

#include "pkv_device.cuh"
#include "pkv_fp8.cuh"
#include "pkv_kernels.h"

namespace pkv {
namespace {

constexpr int kExpandThreads = 256;

template <int D>
__global__ void __launch_bounds__(kExpandThreads) expand_fp8_kernel(const ExpandArgs a) {
  constexpr int kChunks = kPageSize * D / 8 / 32;  // 8-byte chunks per lane of a tile
  grid_dependency_wait();
  allow_dependents();
  const int lane = threadIdx.x & 31;
  const long long units = static_cast<long long>(a.num_seqs) * a.max_pages * a.hkv;
  const long long stride = static_cast<long long>(gridDim.x) * (kExpandThreads / 32);
  for (long long u = static_cast<long long>(blockIdx.x) * (kExpandThreads / 32) + (threadIdx.x >> 5); u < units;
       u += stride) {
    const long long sp = u / a.hkv;  // (request, page)
    const int h = static_cast<int>(u - sp * a.hkv);
    const int s = static_cast<int>(sp / a.max_pages);
    const int p = static_cast<int>(sp - static_cast<long long>(s) * a.max_pages);
    int len = __ldg(a.seq_lens + s);
    if (len < 0 || len > a.max_pages * kPageSize) {
      if (lane == 0) set_status(a.status, PKV_ERR_OUT_OF_BOUNDS);
      len = len < 0 ? 0 : a.max_pages * kPageSize;
    }
    const int rows = min(len - p * kPageSize, kPageSize);  // of this page (max_pages is below 2^27 - 1: host check)
    if (rows <= 0) continue;
    const int src = __ldg(a.block_table + sp), dst = __ldg(a.out_block_table + sp);
    if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.out_pages) {
      if (lane == 0) set_status(a.status, PKV_ERR_OUT_OF_BOUNDS);
      continue;
    }
    const size_t from = static_cast<size_t>(src) * a.hkv + h, to = static_cast<size_t>(dst) * a.hkv + h;
    const uint2* k = reinterpret_cast<const uint2*>(a.k_pages + from * (kPageSize * D));
    const uint2* v = reinterpret_cast<const uint2*>(a.v_pages + from * (kPageSize * D));
    const int sc = __ldg(a.scales + from * kScaleBytes + lane);
    uint2 x[2][kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      x[0][i] = __ldg(k + i * 32 + lane);
      x[1][i] = __ldg(v + i * 32 + lane);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint4* out = reinterpret_cast<uint4*>((w ? a.v_out : a.k_out) + to * (kPageSize * D));
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int row = (i * 32 + lane) / (D / 8);
        const float f = __uint_as_float(static_cast<uint32_t>(__shfl_sync(0xffffffffu, sc, w * kPageSize + row)) << 23);
        uint32_t y[4];
        e4m3x4_to_f16x4(x[w][i].x, y[0], y[1]);
        e4m3x4_to_f16x4(x[w][i].y, y[2], y[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&y[j]));
          y[j] = pack_bf16x2(g.x * f, g.y * f);
        }
        if (row < rows) out[i * 32 + lane] = make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
  }
}

}  // namespace

int launch_expand_fp8(const ExpandArgs& a, int head_dim, int num_sms, cudaStream_t stream) {
  const long long units = static_cast<long long>(a.num_seqs) * a.max_pages * a.hkv;
  long long blocks = (units + kExpandThreads / 32 - 1) / (kExpandThreads / 32);
  const long long cap = static_cast<long long>(num_sms) * 32;
  if (blocks > cap) blocks = cap;
  const dim3 grid(static_cast<unsigned>(blocks)), block(kExpandThreads);
  cudaError_t e;
  if (head_dim == 64)
    e = launch_pdl(expand_fp8_kernel<64>, grid, block, 0, stream, a);
  else if (head_dim == 128)
    e = launch_pdl(expand_fp8_kernel<128>, grid, block, 0, stream, a);
  else
    return PKV_ERR_UNSUPPORTED;
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
