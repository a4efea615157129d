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
// The op reads and writes every row once and is bound by memory; what stands in
// the way is the arithmetic between, so it is kept down: 225 warp instructions
// per 4 rows at D = 128, copies and bookkeeping included (a plain copy takes 118),
// 253 in the 8-bit form. D / 16 lanes take a row, lane l dims 8l .. 8l + 7 and
// D/2 + 8l .. D/2 + 8l + 7: both halves of a pair are in one lane (no exchange
// for the rotation), every access is 16 bytes, and the row's sum of squares and
// largest magnitude are 2 or 3 shuffles away. The rows that a warp's lanes hold
// at once (a batch: 4 rows at D = 128, 8 at 64) are all q, all k or all v, so
// that each kind runs its own straight code, in packed pairs of fp32.
// The batches of all tokens form one list that the warps split evenly. Each
// warp keeps the next kDepth of its batches on the way in a shared-memory ring
// of its own (cp.async; a lane reads back what it copied), with the table rows
// of their tokens beside them: the bytes in flight do not depend on registers
// or occupancy, and a token's positions and slots are loaded 32 at a time, so
// that no batch waits for a chain of loads.
#include <cuda_runtime.h>
#include <math_constants.h>

#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_fp8.cuh"
#include "pkv_kernels.h"
#include "pkv_rows.cuh"

namespace pkv {
namespace {

// Launch shape: on 4096 tokens of 16/8/128 into bf16 (8-bit)
// pools, rings of 4 / 6 / 8 batches measured 13.6 / 14.0 / 14.5 (13.7 / 14.6 / 15.3) us, and 2 / 3 / 4 / 5 blocks
// per SM 19.3 / 16.8 / 14.0 / 14.2 us.
constexpr int kWarps = 4;                // per block
constexpr int kBlocksPerSm = 4;
constexpr int kDepth = 4;                // batches on the way per warp
constexpr int kTables = kDepth / 2 + 2;  // tokens that kDepth + 1 batches touch (a token has at least 2)
constexpr int kBatchBytes = 1024;        // 32 lanes x 16 values

template <int D, bool kFp8>
__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSm) append_rope_kernel(const AppendRopeArgs a) {
  constexpr int L = D / 16;  // lanes per row
  constexpr int R = 32 / L;  // rows per batch
  __shared__ __align__(16) unsigned char ring_s[kWarps][kDepth * kBatchBytes];
  __shared__ __align__(16) unsigned char table_s[kWarps][kTables * D * 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % L, g = lane / L;
  const unsigned bq = (a.hq + R - 1) / R, bk = (a.hkv + R - 1) / R;  // batches of a token: bq of q, bk of k, bk of v
  const unsigned per_token = bq + 2 * bk;
  const unsigned long long total = static_cast<unsigned long long>(a.n_tokens) * per_token;  // below 2^31 (host check)
  const unsigned warps = gridDim.x * kWarps, me = blockIdx.x * kWarps + warp;
  const unsigned lo = static_cast<unsigned>(total * me / warps), hi = static_cast<unsigned>(total * (me + 1) / warps);
  const uint32_t ring = smem_u32(ring_s[warp]) + lane * 16, ring_end = ring + kDepth * kBatchBytes;
  const uint32_t table = smem_u32(table_s[warp]);
  const bool turn = a.cos_sin != nullptr;
  const unsigned last_token = static_cast<unsigned>(a.n_tokens) - 1;
  grid_dependency_wait();
  allow_dependents();
  if (lo >= hi) return;

  // Batch i of a token: its kind (0 q, 1 k, 2 v) and how many batches lie before it in that kind.
  auto place = [&](unsigned i, int& kind, unsigned& before) {
    kind = i < bq ? 0 : i < bq + bk ? 1 : 2;
    before = i - (kind == 0 ? 0 : kind == 1 ? bq : bq + bk);
  };
  auto batches_of = [&](int kind) { return kind == 0 ? bq : bk; };

  // ---- what is on the way: batch `next`, of kind nkind of token nt, the lane's row nh, goes to ring address nring
  unsigned next = lo, nt = lo / per_token, nleft;
  int nkind, nh, ntable = 0;
  uint32_t nring = ring;
  const char* nsrc;  // the lane's chunk of row 0 of that kind
  unsigned pos_base = nt;
  int pos = 0;  // of token pos_base + lane
  if (turn) pos = __ldg(a.positions + min(pos_base + lane, last_token));
  bool fresh = true;  // token nt's table row is still to be copied
  auto source = [&]() {
    nsrc = reinterpret_cast<const char*>(nkind == 0   ? a.q + nt * a.q_stride
                                         : nkind == 1 ? a.k_new + nt * a.k_stride
                                                      : a.v_new + nt * a.v_stride) +
           l * 16;
  };
  {
    unsigned before;
    place(lo - nt * per_token, nkind, before);
    nleft = batches_of(nkind) - before;
    nh = before * R + g;
    source();
  }
  auto fetch = [&]() {
    if (next < hi) {
      const char* row = nsrc + static_cast<unsigned>(min(nh, (nkind == 0 ? a.hq : a.hkv) - 1) * (D * 2));
      cp_async16(nring, row);
      cp_async16(nring + kBatchBytes / 2, row + D);
      if (fresh && turn) {
        if (nt - pos_base >= 32) {
          pos_base = nt;
          pos = __ldg(a.positions + min(pos_base + lane, last_token));
        }
        const int p = min(max(__shfl_sync(0xffffffffu, pos, nt - pos_base), 0), a.rope_max_pos - 1);
        if (lane < D / 4)
          cp_async16(table + (ntable * D + lane * 4) * 4, a.cos_sin + static_cast<size_t>(p) * D + lane * 4);
      }
      fresh = false;
      nring += kBatchBytes;
      if (nring == ring_end) nring = ring;
      ++next;
      nh += R;
      if (--nleft == 0) {
        nh = g;
        if (++nkind == 3) {
          nkind = bq > 0 ? 0 : 1;
          ++nt;
          fresh = true;
          ntable = ntable + 1 == kTables ? 0 : ntable + 1;
        }
        nleft = batches_of(nkind);
        source();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int j = 0; j < kDepth; ++j) fetch();
  auto landed = [&]() {  // the oldest batch on the way, and with a token's first batch its table row
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    __syncwarp();
  };

  // ---- the batches in order
  unsigned t = lo / per_token, info_base = t;
  int slots = 0, poss = 0;  // of token info_base + lane
  auto load_info = [&]() {
    const unsigned x = min(info_base + lane, last_token);
    slots = __ldg(a.slot_mapping + x);
    if (turn) poss = __ldg(a.positions + x);
  };
  load_info();
  uint32_t rring = ring;
  int rtable = 0;
  bool enter = true;  // token t's slot and table row are still to be read
  int in_page = -1;   // slot in its page, -1: k and v are not written
  size_t tile0 = 0;
  Turn cs;
  int weights_of = -1;  // kind whose weights w holds
  Row w;
  int kind;
  unsigned before;
  place(lo - t * per_token, kind, before);

  // n batches of kind K from the lane's row h on
  auto batches = [&](auto kind_c, unsigned n, int h) {
    constexpr int K = decltype(kind_c)::value;
    constexpr bool kQuant = kFp8 && K != 0;
    const int heads = K == 0 ? a.hq : a.hkv;
    const bool norms = K == 0 ? a.q_weight != nullptr : K == 1 ? a.k_weight != nullptr : false;
    const bool turns = K != 2 && turn;
    if (norms && weights_of != K) {
      const uint4* wp = reinterpret_cast<const uint4*>(K == 0 ? a.q_weight : a.k_weight) + l;
      w = unpack(__ldg(wp), __ldg(wp + L));
      weights_of = K;
    }
    // the lane's chunk of row 0 of that kind of this token; rows of heads are D (q_out) or 16 D (a page) apart
    constexpr int kElem = kQuant ? 1 : 2;
    char* out = K == 0 ? reinterpret_cast<char*>(a.q_out + static_cast<size_t>(t) * (a.hq * D))
                       : static_cast<char*>(K == 1 ? a.k_pages : a.v_pages) +
                             (tile0 * kPageSize + max(in_page, 0)) * (D * kElem);
    out += l * 8 * kElem;
    constexpr int kHeadStep = (K == 0 ? D : kPageSize * D) * kElem;
#pragma unroll 1
    for (; n > 0; --n, h += R) {
      landed();
      const uint4 xl = lds128(rring), xh = lds128(rring + kBatchBytes / 2);
      rring += kBatchBytes;
      if (rring == ring_end) rring = ring;
      const bool writes = h < heads && (K == 0 || in_page >= 0);
      char* to = out + static_cast<size_t>(static_cast<unsigned>(h)) * kHeadStep;
      if (!kQuant && !norms && !turns) {  // copied bit for bit
        if (writes) {
          reinterpret_cast<uint4*>(to)[0] = xl;
          reinterpret_cast<uint4*>(to)[L] = xh;
        }
      } else {
        Row x = unpack(xl, xh);
        const float norm = turn_row<D>(x, norms, w, a.eps, turns, cs);
        if constexpr (kQuant) {
          uint2 q0, q1;
          const int e = quantise_row<D>(x, norm, q0, q1);
          if (writes) {
            reinterpret_cast<uint2*>(to)[0] = q0;
            reinterpret_cast<uint2*>(to)[L] = q1;
            if (l == 0) a.scales[(tile0 + h) * kScaleBytes + (K - 1) * kPageSize + in_page] = static_cast<uint8_t>(e);
          }
        } else {
          if (norms) scale_row(x, norm);
          if (writes) {
            reinterpret_cast<uint4*>(to)[0] = pack4(x.y);
            reinterpret_cast<uint4*>(to)[L] = pack4(x.y + 4);
          }
        }
      }
      fetch();
    }
  };
#pragma unroll 1
  for (unsigned f = lo; f < hi;) {
    if (enter) {
      landed();
      if (t - info_base >= 32) {
        info_base = t;
        load_info();
      }
      const int slot = __shfl_sync(0xffffffffu, slots, t - info_base);
      const int p = __shfl_sync(0xffffffffu, poss, t - info_base);
      const bool inside = slot >= 0 && slot / kPageSize < a.num_pages;
      if (slot >= 0 && !inside) set_status(a.status, PKV_ERR_OUT_OF_BOUNDS);
      if (turn && (p < 0 || p >= a.rope_max_pos) && (a.hq > 0 || inside)) set_status(a.status, PKV_ERR_OUT_OF_BOUNDS);
      in_page = inside ? slot % kPageSize : -1;
      tile0 = static_cast<size_t>(inside ? slot / kPageSize : 0) * a.hkv;
      if (turn) load_turn<D>(reinterpret_cast<const float*>(table_s[warp]) + rtable * D, l, cs);
      enter = false;
    }
    const unsigned n = min(batches_of(kind) - before, hi - f);
    const int h = static_cast<int>(before) * R + g;
    if (kind == 0)
      batches(std::integral_constant<int, 0>(), n, h);
    else if (kind == 1)
      batches(std::integral_constant<int, 1>(), n, h);
    else
      batches(std::integral_constant<int, 2>(), n, h);
    f += n;
    before = 0;
    if (++kind == 3) {
      kind = bq > 0 ? 0 : 1;
      ++t;
      enter = true;
      rtable = rtable + 1 == kTables ? 0 : rtable + 1;
    }
  }
}

template <int D, bool kFp8>
int launch(const AppendRopeArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int R = 512 / D;
  const long long batches = static_cast<long long>(a.n_tokens) * ((a.hq + R - 1) / R + 2 * ((a.hkv + R - 1) / R));
  long long blocks = (batches + kWarps - 1) / kWarps;  // a batch per warp, until every SM is full
  const long long cap = static_cast<long long>(num_sms) * kBlocksPerSm;
  if (blocks > cap) blocks = cap;
  return launch_pdl(append_rope_kernel<D, kFp8>, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), 0, stream,
                    a) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

}  // namespace

int launch_append_rope(const AppendRopeArgs& a, int head_dim, int num_sms, cudaStream_t stream) {
  const bool fp8 = a.scales != nullptr;
  if (head_dim == 64) return fp8 ? launch<64, true>(a, num_sms, stream) : launch<64, false>(a, num_sms, stream);
  if (head_dim == 128) return fp8 ? launch<128, true>(a, num_sms, stream) : launch<128, false>(a, num_sms, stream);
  return PKV_ERR_UNSUPPORTED;
}

}  // namespace pkv
