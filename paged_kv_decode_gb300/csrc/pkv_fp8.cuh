// pkv_fp8.cuh -- the 8-bit paged KV cache: its number format and the
// tensor-core MMA step of one of its pages.
//
// A cached row x of D values (one token of one KV head, K or V) is stored as D
// e4m3 values (4 exponent bits, 3 mantissa bits, largest 448, no infinities)
// and one power of two 2^e, kept as the byte e + 127 (e8m0): x_i = 2^e v_i with
// e the least integer such that max |x_i| <= 448 * 2^e, and v_i = x_i 2^-e
// rounded to nearest even. A power of two is enough because e4m3 is itself a
// floating-point format: against a free scale it costs at most one of the
// row's 18 binades of range and no precision. In return a value is rounded
// once, e is found without a division, 2^e v is exact in bf16 and in fp32, and
// a page's 32 scales per KV head fill one 32-byte memory sector.
// e is clamped to [kExpMin, kExpMax]: a row below 448 * 2^kExpMin rounds on a
// fixed grid of 2^(kExpMin - 9), values above 448 * 2^kExpMax saturate (as
// infinities do), NaN stays NaN and takes no part in the maximum. The clamp
// keeps the scales normal floats and the weighted sums of values inside fp32's
// range.
//
// Pools: e4m3 [num_pages][num_kv_heads][16][D] for K and for V, scales
// [num_pages][num_kv_heads][2][16] bytes (16 K rows, then 16 V rows).
// PTX forms as in the PTX ISA (cvt e4m3x2, ldmatrix, movmatrix, mma.sync).
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include "pkv_device.cuh"
#include "pkv_mma.cuh"

namespace pkv {

constexpr int kExpMin = -80;
constexpr int kExpMax = 100;
constexpr int kScaleBytes = 2 * kPageSize;  // scales of one (page, KV head): 16 K rows, 16 V rows

// Tensor maps of the 8-bit pools, [page * hkv + KV head][16 rows][head_dim] bytes; one box is a whole
// (page, KV head) tile of K or V, swizzled over its rows' head_dim bytes (128-byte swizzle at head_dim
// 128, 64-byte at 64: the layouts swz8() reads). PKV_ERR_UNSUPPORTED past 2^31 tiles.
int encode_page_maps_fp8(const void* k_pages, const void* v_pages, int head_dim, int num_pages, int hkv,
                         CUtensorMap* kmap, CUtensorMap* vmap);

// e (clamped) of a row whose largest finite magnitude is `a`. 448 = 1.75 * 2^8: the mantissa decides
// between floor(log2 a) - 8 and the next; exact for every float, 0 and subnormals land on kExpMin.
__device__ __forceinline__ int row_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kExpMin), kExpMax);
}
// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// lo and hi (already scaled) as two e4m3 values, lo in the low byte; to nearest even, saturating
__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// four e4m3 values (32 bits) -> two pairs of fp16 values, exactly
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// c += a * b, m16n8k16, fp16 operands, fp32 accumulators
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Untiled bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes) with an L2 policy.
__device__ __forceinline__ void bulk_load_hint(void* smem_dst, const void* gmem_src, uint32_t bytes, uint64_t* bar,
                                               uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(smem_dst)),
      "l"(gmem_src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// Byte offset of 16-byte chunk c (16 dims) of token row t in a swizzled tile of D-byte rows.
template <int D>
__device__ __forceinline__ uint32_t swz8(int t, int c) {
  static_assert(D == 64 || D == 128, "head_dim 64 or 128");
  return static_cast<uint32_t>(t * D + ((D == 128 ? c ^ (t & 7) : c ^ ((t >> 1) & 3)) << 4));
}

// This lane's ldmatrix row address inside a tile, per pair of 16-dim chunks i: matrices (tokens 0-7, chunk
// 2i), (tokens 8-15, 2i), (tokens 0-7, 2i + 1), (tokens 8-15, 2i + 1); the same for K and (transposed) V.
template <int D>
__device__ __forceinline__ void fp8_offsets(uint32_t (&off)[D / 32]) {
  const int lane = threadIdx.x & 31, mi = lane >> 3, mr = lane & 7;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) off[i] = swz8<D>(mr + ((mi & 1) << 3), 2 * i + (mi >> 1));
}

// The query rows as the B operand of the score product: lane (r, c) holds head r's dims 16 ks + 4c .. 4c + 3
// (staged at `row`, bf16), as fp16 scaled by the power of two that brings the row's largest value into
// [2^14, 2^15), the top of fp16's range: bf16's 8 significant bits are exact down to 2^-31 of the row's largest
// value, below that they are held to 2^-39 of it. (With [1, 2) a row with one value 2^26 above the others lost
// the others.) qs0, qs1: qscale times the powers taken out of heads 2c and 2c + 1.
template <int KS>
__device__ __forceinline__ void fp8_query(uint32_t row, bool live, float qscale, uint32_t (&qf)[KS][2], float& qs0,
                                          float& qs1) {
  const int lane = threadIdx.x & 31, c = lane & 3;
  uint32_t x[KS][2];
  uint32_t most = 0;  // magnitude bits of the largest value (bf16 magnitudes order as integers)
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      x[ks][e] = live ? lds32(row + (16 * ks + 4 * c + 2 * e) * 2) : 0u;
      most = max(most, max(x[ks][e] & 0x7fffu, (x[ks][e] >> 16) & 0x7fffu));
    }
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
  // field E of the largest value; the factor 2^(127 + 14 - E) and its inverse stay normal floats
  const uint32_t E = min(max(most >> 7, 15u), 254u);
  const float down = __uint_as_float((268u - E) << 23), up = __uint_as_float((E - 14u) << 23);
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 f = bf2_to_f2(x[ks][e]);
      qf[ks][e] = pack_f16x2(f.x * down, f.y * down);
    }
  qs0 = qscale * __shfl_sync(0xffffffffu, up, 8 * c);      // lane (2c, 0)
  qs1 = qscale * __shfl_sync(0xffffffffu, up, 8 * c + 4);  // lane (2c + 1, 0)
}

// Weights enter the value product 2^kWeightShift above their own size, so that fp16 holds them to 2^-39 of
// the largest (half its subnormals' step, 2^-25) while the largest, 2^14, stays below fp16's 65504.
constexpr float kWeightShift = 14.f;

// log2 of the scale that byte b stands for, b - 127, without a conversion (2^23 + b from its bits)
__device__ __forceinline__ float scale_log2(uint32_t b) { return __uint_as_float(0x4b000000u | b) - 8388735.f; }

// What takes w (below) out of a warp's o at the end; a warp without units has w = -inf and o = 0.
__device__ __forceinline__ float value_power(float w) { return ex2(w - kWeightShift); }

// One unit of NP pages: the scores of its 16 NP tokens for the 8 head columns, the online-softmax update of
// this lane's heads (2c, 2c + 1), and the value product. kt, vt: shared addresses of the pages' swizzled
// tiles, one behind the other; st: of their 32 scale bytes each; nv: the unit's tokens before seq_len (what
// lies behind them may be anything).
//
// With k_j = 2^(ek_j) k8_j and v_j = 2^(ev_j) v8_j, s_j = qscale 2^(ek_j) <q, k8_j> (log2 domain), the sums
// are l = sum_j 2^(s_j - m) in fp32, m the running maximum of s, and
//   o = sum_j [2^(s_j - m + ev_j - w + kWeightShift)] v8_j
// on the tensor cores, w the running maximum of s - m + ev, a token's contribution (value_power() takes it out
// at the end). The key's power multiplies the fp32 score; the value's joins the exponent, which is held against
// m first (s + ev would lose ev where scores are large; the sum's rounding costs the weights that count 2^-17 at
// most). The e4m3 operands become fp16 in registers (exact), so K and V enter the products unrounded; the
// bracket is rounded to fp16 (2^-11 of it), tighter than the bf16 output's own rounding. Its largest value
// belongs to the token that contributes most, so a value row of any size that the softmax gives nothing takes
// no precision from the others. With the maximum of ev alone in w's place (one power for both heads, no second
// exponential), such a row 2^39 above the rest left nothing of them (16 requests at 16/8/128 14.55 us that way,
// 14.78 this, 32 requests 30.4 and 30.7; finding w from s + ev beside m, where scores are small, saved nothing).
//
// ldmatrix moves 16-byte rows of 8 x 16-bit units. For K a lane's 32 bits are dims 4c .. 4c + 3 of token r:
// as the pairs (k slots 2c, 2c + 1) and (8 + 2c, 9 + 2c) of the A operand, with the query's slots permuted
// alike. For V, transposed, they are dims 2r, 2r + 1 of tokens 2c and 2c + 1: a byte permute gives the two
// token pairs, dim 2r as row r of the A operand and dim 2r + 1 as row r + 8, so o[ks] holds dims
// 16 ks + 2r (elements 0, 1) and 16 ks + 2r + 1 (elements 2, 3).
template <int KS, int NP>
__device__ __forceinline__ void mma_unit_fp8(uint32_t kt, uint32_t vt, uint32_t st, const uint32_t (&off)[KS / 2],
                                             const uint32_t (&qf)[KS][2], int nv, float qs0, float qs1,
                                             float (&o)[KS][4], float& m0, float& m1, float& l0, float& l1,
                                             float& w0, float& w1) {
  constexpr int kTile = kPageSize * KS * 16;  // bytes of a page's K or V
  const int lane = threadIdx.x & 31, r = lane >> 2;
  if (nv < kPageSize * NP) {
    // the request's last unit: value rows behind it become zeros (0 times a stale NaN would be NaN)
    for (int i = nv * KS + lane; i < kPageSize * NP * KS; i += 32)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vt + i * 16), "r"(0) : "memory");
    fence_proxy_async_smem();  // before the stage's next tensor copy
    __syncwarp();
  }
  float s[NP][4];  // tokens r and r + 8 of each page x heads 2c, 2c + 1
  float ev[NP][2];
  float x0 = -CUDART_INF_F, x1 = -CUDART_INF_F;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const uint32_t sp = st + p * kScaleBytes;
    const bool v0 = r < nv - p * kPageSize, v1 = r + 8 < nv - p * kPageSize;
    const uint32_t ek0 = lds8(sp + r), ek1 = lds8(sp + r + 8);
    ev[p][0] = scale_log2(lds8(sp + kPageSize + r));
    ev[p][1] = scale_log2(lds8(sp + kPageSize + r + 8));
    float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KS / 2; ++i) {
      uint32_t x[4], a0, a1, a2, a3;
      ldsm4(kt + p * kTile + off[i], x);
      e4m3x4_to_f16x4(x[0], a0, a2);
      e4m3x4_to_f16x4(x[1], a1, a3);
      mma_f16(sa, a0, a1, a2, a3, qf[2 * i][0], qf[2 * i][1]);
      e4m3x4_to_f16x4(x[2], a0, a2);
      e4m3x4_to_f16x4(x[3], a1, a3);
      mma_f16(sb, a0, a1, a2, a3, qf[2 * i + 1][0], qf[2 * i + 1][1]);
    }
    const float k0 = __uint_as_float(ek0 << 23), k1 = __uint_as_float(ek1 << 23);  // 2^ek
    s[p][0] = v0 ? (sa[0] + sb[0]) * (k0 * qs0) : -CUDART_INF_F;
    s[p][1] = v0 ? (sa[1] + sb[1]) * (k0 * qs1) : -CUDART_INF_F;
    s[p][2] = v1 ? (sa[2] + sb[2]) * (k1 * qs0) : -CUDART_INF_F;
    s[p][3] = v1 ? (sa[3] + sb[3]) * (k1 * qs1) : -CUDART_INF_F;
    x0 = fmaxf(x0, fmaxf(s[p][0], s[p][2]));
    x1 = fmaxf(x1, fmaxf(s[p][1], s[p][3]));
  }
#pragma unroll
  for (int m = 4; m < 32; m <<= 1) {
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, m));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, m));
  }
  const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
  float y0 = -CUDART_INF_F, y1 = -CUDART_INF_F;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    s[p][0] -= n0;
    s[p][1] -= n1;
    s[p][2] -= n0;
    s[p][3] -= n1;
    y0 = fmaxf(y0, fmaxf(s[p][0] + ev[p][0], s[p][2] + ev[p][1]));
    y1 = fmaxf(y1, fmaxf(s[p][1] + ev[p][0], s[p][3] + ev[p][1]));
  }
#pragma unroll
  for (int m = 4; m < 32; m <<= 1) {
    y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, m));
    y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, m));
  }
  const float g0 = m0 - n0, g1 = m1 - n1;  // -inf on the first unit
  const float u0 = fmaxf(w0 + g0, y0), u1 = fmaxf(w1 + g1, y1);
  if (__any_sync(0xffffffffu, g0 != 0.f || g1 != 0.f || u0 != w0 || u1 != w1)) {
    l0 *= ex2(g0);
    l1 *= ex2(g1);
    const float o0 = ex2(w0 + g0 - u0), o1 = ex2(w1 + g1 - u1);  // 0 on the first unit
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      o[ks][0] *= o0;
      o[ks][1] *= o1;
      o[ks][2] *= o0;
      o[ks][3] *= o1;
    }
    m0 = n0;
    m1 = n1;
    w0 = u0;
    w1 = u1;
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    l0 += ex2(s[p][0]) + ex2(s[p][2]);  // tokens r and r + 8
    l1 += ex2(s[p][1]) + ex2(s[p][3]);
    const float c0 = kWeightShift - u0, c1 = kWeightShift - u1;
    const uint32_t pb0 = movm_t(pack_f16x2(ex2(s[p][0] + ev[p][0] + c0), ex2(s[p][1] + ev[p][0] + c1)));
    const uint32_t pb1 = movm_t(pack_f16x2(ex2(s[p][2] + ev[p][1] + c0), ex2(s[p][3] + ev[p][1] + c1)));
#pragma unroll
    for (int i = 0; i < KS / 2; ++i) {
      uint32_t y[4], a0, a1, a2, a3;
      ldsm4_t(vt + p * kTile + off[i], y);
      e4m3x4_to_f16x4(__byte_perm(y[0], 0, 0x3120), a0, a1);
      e4m3x4_to_f16x4(__byte_perm(y[1], 0, 0x3120), a2, a3);
      mma_f16(o[2 * i], a0, a1, a2, a3, pb0, pb1);
      e4m3x4_to_f16x4(__byte_perm(y[2], 0, 0x3120), a0, a1);
      e4m3x4_to_f16x4(__byte_perm(y[3], 0, 0x3120), a2, a3);
      mma_f16(o[2 * i + 1], a0, a1, a2, a3, pb0, pb1);
    }
  }
}

}  // namespace pkv
