// pkv_rows.cuh -- one row of head_dim values (a query, key or value row of one
// head) spread over D / 16 lanes: norm, rotation and quantisation, as used by
// the append (append_rope.cu) and by the fused decode step of the 8-bit cache
// (decode_kernel.cuh). Both run the same instructions in the same order, so a
// row comes out with the same bits from either.
//
// Lane l of a row holds dims 8l .. 8l + 7 and D/2 + 8l .. D/2 + 8l + 7: both
// halves of a rotated pair are in one lane, and memory is touched 16 bytes (or
// 8 quantised ones) at a time. Sums and maxima over a row shuffle among its
// lanes, with the whole warp taking part.
#pragma once

#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "pkv_device.cuh"
#include "pkv_fp8.cuh"

namespace pkv {

// A lane's 16 values: pairs 0 .. 3 are dims 8l .. 8l + 7, pairs 4 .. 7 dims D/2 + 8l .. D/2 + 8l + 7.
struct Row {
  float2 y[8];
};
__device__ __forceinline__ Row unpack(const uint4& lo, const uint4& hi) {
  return {{bf2_to_f2(lo.x), bf2_to_f2(lo.y), bf2_to_f2(lo.z), bf2_to_f2(lo.w), bf2_to_f2(hi.x), bf2_to_f2(hi.y),
           bf2_to_f2(hi.z), bf2_to_f2(hi.w)}};
}
__device__ __forceinline__ uint4 pack4(const float2* y) {
  return make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y), pack_bf16x2(y[2].x, y[2].y),
                    pack_bf16x2(y[3].x, y[3].y));
}
__device__ __forceinline__ uint32_t quant4(const float2& a, const float2& b, float f) {
  const float2 f2 = make_float2(f, f);
  const float2 x = __fmul2_rn(a, f2), y = __fmul2_rn(b, f2);
  return static_cast<uint32_t>(to_e4m3x2(x.x, x.y)) | static_cast<uint32_t>(to_e4m3x2(y.x, y.y)) << 16;
}

// Largest finite magnitude of the row's values (over its lanes).
template <int L>
__device__ __forceinline__ float row_max(const Row& x) {
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = fmaxf(most, fmaxf(fabsf(x.y[i].x), fabsf(x.y[i].y)));  // (drops NaN)
#pragma unroll
  for (int m = 1; m < L; m <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
  if (__any_sync(0xffffffffu, most == CUDART_INF_F)) {  // rare: again without the infinities
    float fin = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(x.y[i].x), b = fabsf(x.y[i].y);
      fin = fmaxf(fin, fmaxf(a < CUDART_INF_F ? a : 0.f, b < CUDART_INF_F ? b : 0.f));
    }
#pragma unroll
    for (int m = 1; m < L; m <<= 1) fin = fmaxf(fin, __shfl_xor_sync(0xffffffffu, fin, m));
    most = fin;
  }
  return most;
}

// A position's table row: c, s and -s of the lane's 8 pairs.
struct Turn {
  float2 c[4], s[4], n[4];
};
// ... read from a row of D floats (cos, then sin) in shared memory
template <int D>
__device__ __forceinline__ void load_turn(const float* row, int l, Turn& t) {
  const float4* r = reinterpret_cast<const float4*>(row) + 2 * l;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float4 c = r[j], s = r[D / 8 + j];
    t.c[2 * j] = make_float2(c.x, c.y);
    t.c[2 * j + 1] = make_float2(c.z, c.w);
    t.s[2 * j] = make_float2(s.x, s.y);
    t.s[2 * j + 1] = make_float2(s.z, s.w);
    t.n[2 * j] = make_float2(-s.x, -s.y);
    t.n[2 * j + 1] = make_float2(-s.z, -s.w);
  }
}

// x becomes x * w rotated by t (each where asked for); returns the norm's factor 1 / sqrt(mean(x^2) + eps), or 1,
// which is still to be applied.
template <int D>
__device__ __forceinline__ float turn_row(Row& x, bool norms, const Row& w, float eps, bool turns, const Turn& t) {
  float norm = 1.f;
  if (norms) {
    float2 sq = __fmul2_rn(x.y[0], x.y[0]), sr = __fmul2_rn(x.y[1], x.y[1]);
#pragma unroll
    for (int j = 2; j < 8; j += 2) {
      sq = __ffma2_rn(x.y[j], x.y[j], sq);
      sr = __ffma2_rn(x.y[j + 1], x.y[j + 1], sr);
    }
    float sum = (sq.x + sq.y) + (sr.x + sr.y);
#pragma unroll
    for (int m = 1; m < D / 16; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    norm = __frsqrt_rn(sum * (1.f / D) + eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x.y[j] = __fmul2_rn(x.y[j], w.y[j]);
  }
  if (turns) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x1 = x.y[j], x2 = x.y[4 + j];
      x.y[j] = __ffma2_rn(x1, t.c[j], __fmul2_rn(x2, t.n[j]));
      x.y[4 + j] = __ffma2_rn(x2, t.c[j], __fmul2_rn(x1, t.s[j]));
    }
  }
  return norm;
}

__device__ __forceinline__ void scale_row(Row& x, float f) {
  const float2 f2 = make_float2(f, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) x.y[j] = __fmul2_rn(x.y[j], f2);
}

// The row times `norm`, quantised: 8 codes of each half, and the row's scale byte.
template <int D>
__device__ __forceinline__ int quantise_row(const Row& x, float norm, uint2& lo, uint2& hi) {
  // rounding is monotonic: the largest of the rounded products by norm is the largest value's
  const int e = row_exponent(row_max<D / 16>(x) * norm);
  const float f = norm * pow2i(-e);
  lo = make_uint2(quant4(x.y[0], x.y[1], f), quant4(x.y[2], x.y[3], f));
  hi = make_uint2(quant4(x.y[4], x.y[5], f), quant4(x.y[6], x.y[7], f));
  return e + 127;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, const uint2& v) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ void sts8(uint32_t addr, int v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

}  // namespace pkv
