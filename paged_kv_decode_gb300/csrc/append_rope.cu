// append_rope.cu -- KV append with the rotary embedding (and per-head RMS norm)
// on the way, into the bf16 pools or into the 8-bit ones.
//
// A decoder step hands over the q, k and v rows of its new tokens as the fused
// projection wrote them (a token's rows side by side). Per token at position p
// and head row x of D values, all in fp32:
//   u = x * w                                  (with norm weights w; else u = x)
//   y_i       = u_i c_i - u_{i + D/2} s_i      (with a table; c, s of row p)
//   y_{i+D/2} = u_{i+D/2} c_i + u_i s_i
//   y *= 1 / sqrt(mean(x^2) + eps)             (with norm weights)
// The norm's factor is one number per row, so it is applied after the rotation;
// x * w of two bf16 values is exact in fp32. Without weights y is the fused
// decode call's rotation, bit for bit (each product rounded, then one fma).
// Query rows go to q_out in bf16. Key rows go to their slot in bf16, or
// quantised from the fp32 y as pkv_fp8.cuh says (one rounding, no bf16 in
// between); value rows are copied or quantised, never rotated.
//
// The op reads and writes every row once and is bound by memory. D / 16 lanes
// take a row, lane l dims 8l .. 8l + 7 and D/2 + 8l .. D/2 + 8l + 7: both halves
// of a pair are in one lane (no exchange for the rotation), every access is 16
// bytes, and the row's sum of squares and largest magnitude are 2 or 3 shuffles
// away. A group of lanes takes up to kRows rows of one kind of one token, so
// that the table row and the weights are loaded once for them and the loads of
// all rows are in flight together.
#include <cuda_runtime.h>
#include <math_constants.h>

#include "pkv_device.cuh"
#include "pkv_fp8.cuh"
#include "pkv_kernels.h"

namespace pkv {
namespace {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ void unpack8(const uint4& x, float* y) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf2_to_f2(w[i]);
    y[2 * i] = f.x;
    y[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float* y) {
  return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                    pack_bf16x2(y[6], y[7]));
}
__device__ __forceinline__ uint2 quant8(const float* y, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = static_cast<uint32_t>(to_e4m3x2(y[4 * i] * inv, y[4 * i + 1] * inv)) |
           static_cast<uint32_t>(to_e4m3x2(y[4 * i + 2] * inv, y[4 * i + 3] * inv)) << 16;
  return make_uint2(w[0], w[1]);
}

template <int D, bool kFp8, int kRows>
__global__ void __launch_bounds__(kAppendThreads) append_rope_kernel(const AppendRopeArgs a) {
  constexpr int L = D / 16;  // lanes per row
  grid_dependency_wait();
  allow_dependents();
  const int lane = threadIdx.x & 31;
  const int l = lane % L;
  const unsigned cq = (a.hq + kRows - 1) / kRows, ck = (a.hkv + kRows - 1) / kRows;  // units per token
  const unsigned per_token = cq + 2 * ck;
  const unsigned units = static_cast<unsigned>(a.n_tokens) * per_token;  // below 2^31 (host check)
  const unsigned stride = gridDim.x * (kAppendThreads / L);
  // (warp-uniform bound: the row reductions shuffle over the whole warp)
  for (unsigned base = blockIdx.x * (kAppendThreads / L) + (threadIdx.x >> 5) * (32 / L); base < units;
       base += stride) {
    const unsigned u = base + lane / L;
    const bool live = u < units;
    const unsigned uu = live ? u : units - 1;
    const unsigned t = uu / per_token;
    unsigned c = uu - t * per_token;
    const int kind = c < cq ? 0 : c < cq + ck ? 1 : 2;  // q, k, v
    c -= kind == 0 ? 0 : kind == 1 ? cq : cq + ck;
    const int heads = kind == 0 ? a.hq : a.hkv;
    const int h0 = static_cast<int>(c) * kRows;
    const __nv_bfloat16* src = kind == 0   ? a.q + t * a.q_stride
                               : kind == 1 ? a.k_new + t * a.k_stride
                                           : a.v_new + t * a.v_stride;
    uint4 xl[kRows], xh[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int h = h0 + j < heads ? h0 + j : heads - 1;
      const uint4* row = reinterpret_cast<const uint4*>(src + static_cast<size_t>(h) * D);
      xl[j] = row[l];
      xh[j] = row[L + l];
    }
    int slot = -1;
    if (kind != 0) {
      slot = __ldg(a.slot_mapping + t);
      if (slot >= 0 && slot / kPageSize >= a.num_pages) {
        if (live) set_status(a.status, PKV_ERR_OUT_OF_BOUNDS);
        slot = -1;
      }
    }
    const bool turn = a.cos_sin != nullptr && kind != 2;
    float cs[8], sn[8];
    if (turn) {
      int p = __ldg(a.positions + t);
      if (p < 0 || p >= a.rope_max_pos) {
        if (live && (kind == 0 || slot >= 0)) set_status(a.status, PKV_ERR_OUT_OF_BOUNDS);
        p = p < 0 ? 0 : a.rope_max_pos - 1;
      }
      const float4* row = reinterpret_cast<const float4*>(a.cos_sin + static_cast<size_t>(p) * D);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<float4*>(cs + 4 * i) = __ldg(row + 2 * l + i);
        *reinterpret_cast<float4*>(sn + 4 * i) = __ldg(row + D / 8 + 2 * l + i);
      }
    }
    const __nv_bfloat16* w = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
    float wl[8], wh[8];
    if (w != nullptr) {
      unpack8(__ldg(reinterpret_cast<const uint4*>(w) + l), wl);
      unpack8(__ldg(reinterpret_cast<const uint4*>(w) + L + l), wh);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      float y[16];  // dims 8l .., then D/2 + 8l ..
      unpack8(xl[j], y);
      unpack8(xh[j], y + 8);
      float norm = 1.f;
      float sq = 0.f;
      if (w != nullptr) {
#pragma unroll
        for (int i = 0; i < 16; ++i) sq = fmaf(y[i], y[i], sq);
      }
#pragma unroll
      for (int m = 1; m < L; m <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
      if (w != nullptr) {
        norm = __frsqrt_rn(sq * (1.f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] *= wl[i];
          y[8 + i] *= wh[i];
        }
      }
      if (turn) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x1 = y[i], x2 = y[8 + i];
          y[i] = __fmaf_rn(x1, cs[i], -__fmul_rn(x2, sn[i]));
          y[8 + i] = __fmaf_rn(x2, cs[i], __fmul_rn(x1, sn[i]));
        }
      }
      if (w != nullptr) {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] *= norm;
      }
      const bool mine = live && h0 + j < heads;
      const int h = h0 + j;
      if (kind == 0) {
        if (mine) {
          uint4* dst = reinterpret_cast<uint4*>(a.q_out + (static_cast<size_t>(t) * a.hq + h) * D);
          dst[l] = pack8(y);
          dst[L + l] = pack8(y + 8);
        }
      }
      if constexpr (kFp8) {
        float most = 0.f;  // over the finite values
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float m = fabsf(y[i]);
          most = fmaxf(most, m < CUDART_INF_F ? m : 0.f);
        }
#pragma unroll
        for (int m = 1; m < L; m <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
        if (kind != 0 && mine && slot >= 0) {
          const int e = row_exponent(most);
          const float inv = pow2i(-e);
          const size_t tile = static_cast<size_t>(slot / kPageSize) * a.hkv + h;
          uint8_t* pool = static_cast<uint8_t*>(kind == 1 ? a.k_pages : a.v_pages);
          uint2* dst = reinterpret_cast<uint2*>(pool + (tile * kPageSize + slot % kPageSize) * D);
          dst[l] = quant8(y, inv);
          dst[L + l] = quant8(y + 8, inv);
          if (l == 0)
            a.scales[tile * kScaleBytes + (kind - 1) * kPageSize + slot % kPageSize] = static_cast<uint8_t>(e + 127);
        }
      } else if (kind != 0 && mine && slot >= 0) {
        const size_t tile = static_cast<size_t>(slot / kPageSize) * a.hkv + h;
        __nv_bfloat16* pool = static_cast<__nv_bfloat16*>(kind == 1 ? a.k_pages : a.v_pages);
        uint4* dst = reinterpret_cast<uint4*>(pool + (tile * kPageSize + slot % kPageSize) * D);
        // (value rows and plain key rows keep their bits, NaN payloads included)
        const bool as_is = kind == 2 || (!turn && w == nullptr);
        dst[l] = as_is ? xl[j] : pack8(y);
        dst[L + l] = as_is ? xh[j] : pack8(y + 8);
      }
    }
  }
}

template <int D, bool kFp8, int kRows>
int launch_rows(const AppendRopeArgs& a, int num_sms, cudaStream_t stream) {
  const long long units =
      static_cast<long long>(a.n_tokens) * ((a.hq + kRows - 1) / kRows + 2 * ((a.hkv + kRows - 1) / kRows));
  const long long per_block = kAppendThreads / (D / 16);
  long long blocks = (units + per_block - 1) / per_block;
  const long long cap = static_cast<long long>(num_sms) * 16;
  if (blocks > cap) blocks = cap;
  return launch_pdl(append_rope_kernel<D, kFp8, kRows>, dim3(static_cast<unsigned>(blocks)), dim3(kAppendThreads), 0,
                    stream, a) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

}  // namespace

int launch_append_rope(const AppendRopeArgs& a, int head_dim, int num_sms, cudaStream_t stream) {
  const bool fp8 = a.scales != nullptr;
  if (head_dim == 64)
    return fp8 ? launch_rows<64, true, 2>(a, num_sms, stream) : launch_rows<64, false, 2>(a, num_sms, stream);
  if (head_dim == 128)
    return fp8 ? launch_rows<128, true, 2>(a, num_sms, stream) : launch_rows<128, false, 2>(a, num_sms, stream);
  return PKV_ERR_UNSUPPORTED;
}

}  // namespace pkv
