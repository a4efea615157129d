// tree_attn.cu -- attention of drafted tokens (the nodes of a tree) over the
// paged cache, bf16 or 8-bit.
//
// Row t of request b (node t of T) sees the P cached positions of the request
// and, of the nodes behind them, those whose bit is set in its mask (or, without
// masks, nodes 0 .. t):
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale <q, k_j> - m),
// in one pass over the keys with the running maximum m and sum of each row.
//
// A (request, KV head) has T * G query rows (G query heads per KV head) that
// share every key: T * G flops per byte of the cache, so that a tree of 16 to 64
// nodes is bound by the cache's bytes as long as the two products run on the
// tensor cores at their rate (tcgen05; the row counts are too large for the
// decode kernel's warp-level products of 8 columns). The kernel is therefore a
// decode kernel in its schedule and a prefill kernel in its products:
//
//  * An item is (request, KV head, tile of up to 128 / G nodes): its rows are
//    the M = 128 rows of the products, node-major, heads of a node side by side
//    (one 3-D TMA box). Items cost kItemCost + ceil((P + T) / 128) units; every
//    CTA (one per SM) takes an equal contiguous share of the units, cutting
//    items; a cut item's partial results go to records, and the CTA that
//    completes an item merges them in CTA order (the same bits every time).
//  * Warp 9 loads Q and the K and V tiles of 128 keys through the block table
//    into rings. Warp 8 issues S = Q K^T into TMEM and O += P V with P as the
//    tensor-memory operand. Key tiles alternate between two groups of four
//    softmax warps, each with its own S, P, O, maximum and sum: one group's
//    exponentials run beside the other's products. The two halves of a row are
//    joined in the epilogue, straight from TMEM. Warps whose 32 rows are all
//    past the item's last one do no arithmetic.
//  * 8-bit cache: a value 2^e v is exact in bf16, so four warps for K and four
//    for V expand each tile into the bf16 ring and everything behind that is
//    the bf16 kernel: the outputs are those of pkv_expand_fp8 followed by the
//    bf16 call, bit for bit.
//  * P is rounded to bf16 before it multiplies V, the operand type of the product (at
//    most 2^-9 of a weight; the sum l keeps the unrounded weights in fp32).
//  * Value rows behind the last node are zeroed in shared memory (they may hold
//    anything, and 0 * NaN = NaN). A node's value row that holds infinities or
//    NaN would reach rows that do not see the node the same way: such elements
//    are zeroed too, and added back, in the epilogue, to the rows that see them.
#include <cuda.h>
#include <math_constants.h>

#include "pkv_device.cuh"
#include "pkv_fp8.cuh"
#include "pkv_kernels.h"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kTrRows = 128;  // rows of an item (TMEM lanes)
constexpr int kTrKeys = 128;  // keys of a tile
constexpr int kTrTilePages = kTrKeys / kPageSize;
constexpr int kTrMaxNodes = 64;
constexpr int kTrMaxSeqs = 1024;
constexpr int kTrMmaWarp = 8, kTrTmaWarp = 9;  // bf16: warp 10 mends the value tiles, 8-bit: the others expand tiles
constexpr int kTrHalfBytes = kTrKeys * 128;                     // 64 columns of a 128-row bf16 tile
constexpr uint32_t kTrColS = 0, kTrColO = 256, kTrTmemCols = 512;  // S_w, O_w at + 128 w

// Fixed work of an item (query load, pipeline fill and drain, epilogue) in key tiles, and the least share of a
// CTA: below it another CTA would cost more in merging than it takes over.
#ifndef PKV_TREE_ITEM_COST
#define PKV_TREE_ITEM_COST 2
#endif
#ifndef PKV_TREE_MIN_SHARE
#define PKV_TREE_MIN_SHARE 4
#endif
constexpr long long kDrainCycles = 20000000LL;  // 10 ms: far more than a copy in flight takes
constexpr int kItemCost = PKV_TREE_ITEM_COST;
constexpr int kMinShare = PKV_TREE_MIN_SHARE;

template <int D, bool kFp8>
struct TrDim {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * kTrHalfBytes;  // K or V tile (bf16)
  static constexpr int kPage = kPageSize * D * 2;       // a page of it
  static constexpr int kSlots = kFp8 ? (D == 128 ? 2 : 3) : (D == 128 ? 3 : 6);
  static constexpr int kRawTile = kTrKeys * D;  // 8-bit tile
  static constexpr int kRawSlots = kFp8 ? (D == 128 ? 2 : 5) : 0;
  static constexpr int kRawAlloc = kFp8 ? kRawSlots : 1;  // array sizes may not be 0
  static constexpr int kConvWarps = 4;                    // each for K and for V
  static constexpr int kMenders = kFp8 ? kConvWarps : 1;  // warps that look for infinities and NaN in value rows
  // pieces whose masks of such rows are kept: a warp that works on a tile kSlots tiles ahead of the products is at most
  // kSlots pieces ahead of the one whose epilogue may be reading
  static constexpr int kBadRing = kSlots + 2;
  static constexpr int kThreads = (kFp8 ? 10 + 2 * kConvWarps : 11) * 32;
  // shared memory, from a 1024-byte aligned base
  static constexpr int kOffQ = 0;  // one buffer of up to 128 rows, or two of up to 64
  static constexpr int kOffK = kOffQ + kTile;
  static constexpr int kOffV = kOffK + kSlots * kTile;
  static constexpr int kOffRawK = kOffV + kSlots * kTile;
  static constexpr int kOffRawV = kOffRawK + kRawSlots * kRawTile;
  static constexpr int kOffScales = kOffRawV + kRawSlots * kRawTile;  // [raw slot][K, V][128] bytes
  static constexpr int kOffCtl = kOffScales + kRawSlots * 2 * kTrKeys;
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(kTrRows, kTrKeys, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(kTrRows, D, true);  // V is MN-major
};

template <int D, bool kFp8>
struct TrCtl {
  using Dm = TrDim<D, kFp8>;
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[Dm::kSlots], k_empty[Dm::kSlots], v_full[Dm::kSlots], v_empty[Dm::kSlots];
  uint64_t s_full[2], p_full[2];
  uint64_t v_fixed[Dm::kSlots];
  uint64_t o_done, o_free, drain;
  uint64_t raw_k_full[Dm::kRawAlloc], raw_k_empty[Dm::kRawAlloc], raw_v_full[Dm::kRawAlloc], raw_v_empty[Dm::kRawAlloc];
  long long lo, hi, units, base;  // the CTA's share, all units, units before request `first`
  int first, ctas;
  uint32_t tmem;
  int fail, merge;
  uint32_t bad[Dm::kBadRing][Dm::kMenders][2];  // nodes whose value rows hold infinities or NaN, of the last pieces
  float stat[2][2][kTrRows];  // [group][m, l][row]
};

template <int D, bool kFp8>
constexpr int tr_smem_bytes() {
  return TrDim<D, kFp8>::kOffCtl + static_cast<int>(sizeof(TrCtl<D, kFp8>));
}
static_assert(tr_smem_bytes<128, false>() <= 232448 && tr_smem_bytes<128, true>() <= 232448, "shared memory of an SM");
static_assert(tr_smem_bytes<64, false>() > 120 * 1024 && tr_smem_bytes<64, true>() > 120 * 1024,
              "one CTA per SM: each holds all TMEM columns");
static_assert(tr_smem_bytes<64, false>() <= 232448 && tr_smem_bytes<64, true>() <= 232448, "shared memory of an SM");

// A record: O (unnormalised) [D / 4][128 rows] float4, then m and l of the rows. Room of head_dim 128's at any.
constexpr size_t kTrRecBytes = static_cast<size_t>(kTrRows) * (128 + 2) * 4;

struct TrArgs {
  const int* block_table;
  const int* prefix_lens;
  const int* cu_nodes;
  const unsigned long long* masks;  // [total], or nullptr: a chain
  const uint8_t* k_raw;             // 8-bit pools
  const uint8_t* v_raw;
  const uint8_t* scales;
  const __nv_bfloat16* v_pages;     // bf16 pool (rows added back)
  __nv_bfloat16* out;
  int* status;
  int* counters;  // [SMs], zero between calls
  float* records; // [2 * SMs][kTrRecBytes / 4]
  int num_seqs, total, max_pages, num_pages, max_nodes;
  int hq, hkv, grp;
  int tile_nodes;  // nodes of an item: 128 / grp
  int box_rows;    // rows of the query box: grp * min(tile_nodes, max_nodes)
  int q_rows;      // ... rounded up to whole swizzle atoms of 8 rows
  int q_bufs;      // query buffers: 2 where two fit
  int ctas;        // CTAs of the grid
  float scale_log2;
};

struct TrPiece {
  int n, h, rt;          // request, KV head, tile of nodes
  int P, T, q0;          // prefix, nodes, first row of the request
  int nt, k0, k1;        // key tiles of the item; [k0, k1) of them here
  long long fseg, fend;  // the item's units start at fseg; this piece ends at fend
};

// Prefix and nodes of request n (0 nodes where the lengths are out of bounds).
__device__ __forceinline__ void tr_request(const TrArgs& a, int n, int& P, int& T, int& q0) {
  P = __ldg(a.prefix_lens + n);
  q0 = __ldg(a.cu_nodes + n);
  const long long t = static_cast<long long>(__ldg(a.cu_nodes + n + 1)) - q0;
  if (P < 0 || q0 < 0 || t < 0 || t > a.max_nodes || q0 + t > a.total ||
      P + t > static_cast<long long>(a.max_pages) * kPageSize) {
    set_status(a.status, PKV_ERR_OUT_OF_BOUNDS);
    T = 0;
  } else {
    T = static_cast<int>(t);
  }
}
__device__ __forceinline__ int tr_key_tiles(int P, int T) { return (P + T + kTrKeys - 1) / kTrKeys; }
__device__ __forceinline__ long long tr_units(const TrArgs& a, int P, int T) {
  return T == 0 ? 0
                : static_cast<long long>(a.hkv) * ((T + a.tile_nodes - 1) / a.tile_nodes) *
                      (kItemCost + tr_key_tiles(P, T));
}
__device__ __forceinline__ long long tr_share(long long c, long long units, int ctas) { return c * units / ctas; }
__device__ __forceinline__ int tr_cta_of(long long f, long long units, int ctas) {
  return static_cast<int>(((f + 1) * ctas + units - 1) / units - 1);
}

// The first piece at or behind unit f of the share that ends at hi. (n, base): a request at or before f's and the
// units before it; both move on.
__device__ __forceinline__ bool tr_next(const TrArgs& a, long long f, long long hi, int& n, long long& base, TrPiece& pc) {
  for (; f < hi; f = pc.fend) {
    int P, T, q0;
    long long units;
    for (;; ++n) {
      if (n >= a.num_seqs) return false;
      tr_request(a, n, P, T, q0);
      units = tr_units(a, P, T);
      if (f < base + units) break;
      base += units;
    }
    pc.n = n;
    pc.P = P;
    pc.T = T;
    pc.q0 = q0;
    pc.nt = tr_key_tiles(P, T);
    const int rts = (T + a.tile_nodes - 1) / a.tile_nodes;
    const int cost = kItemCost + pc.nt;
    const long long item = (f - base) / cost;
    pc.h = static_cast<int>(item / rts);
    pc.rt = static_cast<int>(item - static_cast<long long>(pc.h) * rts);
    pc.fseg = base + item * cost;
    const long long p0 = f - pc.fseg;
    const long long p1 = p0 + (hi - f) < cost ? p0 + (hi - f) : cost;
    pc.k0 = static_cast<int>(p0 > kItemCost ? p0 - kItemCost : 0);
    pc.k1 = static_cast<int>(p1 > kItemCost ? p1 - kItemCost : 0);
    pc.fend = f + (p1 - p0);
    if (pc.k1 > pc.k0) return true;
  }
  return false;
}

template <typename Ctl>
__device__ __forceinline__ bool tr_wait(uint64_t* bar, uint32_t use, Ctl* ctl, int* status) {
  const uint32_t parity = use & 1u;
  if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity))) return true;
  bool ok = *reinterpret_cast<volatile int*>(&ctl->fail) == 0;
  if (ok && !mbar_wait_bounded(bar, parity)) {
    *reinterpret_cast<volatile int*>(&ctl->fail) = 1;
    set_status(status, PKV_ERR_DEVICE_TIMEOUT);
    ok = false;
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void tr_group_sync(int id) {  // the eight softmax warps
  asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool tr_group_all(int id, bool ok) {  // ... and whether all of them say ok
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.and.pred q, %1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(ok ? 1u : 0u)
      : "memory");
  return all != 0;
}
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* gmem_src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(smem_dst)),
               "l"(gmem_src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ bool nonfinite_bf16x2(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t x) {  // infinities and NaN become 0
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0x0000ffffu;
  return x;
}

// Byte offset of 16-byte chunk c (8 dims) of token row t: in a K tile ([half][128 rows], 128-byte swizzle), in a V
// tile ([page][half][16 rows], so that a page is one TMA box and one step of the value product).
__device__ __forceinline__ uint32_t tr_k_off(int t, int c) {
  return static_cast<uint32_t>((c >> 3) * kTrHalfBytes + t * 128 + (((c & 7) ^ (t & 7)) << 4));
}
template <int D>
__device__ __forceinline__ uint32_t tr_v_off(int t, int c) {
  return static_cast<uint32_t>((t >> 4) * (kPageSize * D * 2) + (c >> 3) * 2048 + (t & 15) * 128 + (((c & 7) ^ (t & 7)) << 4));
}

// n values times inv, rounded to bf16
template <int N>
__device__ __forceinline__ void tr_store(__nv_bfloat16* dst, const float (&o)[N], float inv) {
#pragma unroll
  for (int q = 0; q < N / 8; ++q) {
    uint4 x;
    x.x = pack_bf16x2(o[8 * q] * inv, o[8 * q + 1] * inv);
    x.y = pack_bf16x2(o[8 * q + 2] * inv, o[8 * q + 3] * inv);
    x.z = pack_bf16x2(o[8 * q + 4] * inv, o[8 * q + 5] * inv);
    x.w = pack_bf16x2(o[8 * q + 6] * inv, o[8 * q + 7] * inv);
    reinterpret_cast<uint4*>(dst)[q] = x;
  }
}

// Columns col .. col + 31 of a row: the infinities and NaN of the nodes' value rows in `bad` that this piece holds.
template <int D, bool kFp8>
__device__ __noinline__ void tr_add_nonfinite(const TrArgs& a, const TrPiece& pc, unsigned long long bad, int col,
                                              float (&o)[32]) {
  for (int j = 0; j < kTrMaxNodes; ++j) {
    const int pos = pc.P + j;
    if (!(bad >> j & 1ull) || pos < pc.k0 * kTrKeys || pos >= pc.k1 * kTrKeys) continue;
    const int id = __ldg(a.block_table + static_cast<size_t>(pc.n) * a.max_pages + pos / kPageSize);
    if (id < 0 || id >= a.num_pages) continue;
    const size_t at = ((static_cast<size_t>(id) * a.hkv + pc.h) * kPageSize + pos % kPageSize) * D + col;
    for (int e = 0; e < 32; ++e) {
      float x;
      if constexpr (kFp8)
        x = (a.v_raw[at + e] & 0x7f) == 0x7f ? CUDART_NAN_F : 0.f;
      else
        x = __bfloat162float(a.v_pages[at + e]);
      if (!(fabsf(x) < CUDART_INF_F)) o[e] += x;
    }
  }
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(TrDim<D, kFp8>::kThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const TrArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  using Dm = TrDim<D, kFp8>;
  using Ctl = TrCtl<D, kFp8>;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + Dm::kOffCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  grid_dependency_wait();
  allow_dependents();
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzle atoms need it; no shared memory precedes the array
    if (tid == 0) set_status(a.status, PKV_ERR_MISALIGNED);
    return;
  }

  if (warp == 0) {
    // all units, this CTA's share and the request that it starts in
    long long units = 0;
    for (int b0 = 0; b0 < a.num_seqs; b0 += 32) {
      int P = 0, T = 0, q0;
      if (b0 + lane < a.num_seqs) tr_request(a, b0 + lane, P, T, q0);
      units += tr_units(a, P, T);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
    const long long want = (units + kMinShare - 1) / kMinShare;
    const int ctas = static_cast<int>(want < a.ctas ? want : a.ctas);
    const int me = blockIdx.x;
    const long long lo = me < ctas ? tr_share(me, units, ctas) : 0, hi = me < ctas ? tr_share(me + 1, units, ctas) : 0;
    int first = 0;
    long long base = 0;
    if (lo < hi) {
      long long carry = 0;
      bool found = false;
      for (int b0 = 0; b0 < a.num_seqs && !found; b0 += 32) {
        int P = 0, T = 0, q0;
        if (b0 + lane < a.num_seqs) tr_request(a, b0 + lane, P, T, q0);
        const long long u = tr_units(a, P, T);
        long long x = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, carry + x > lo);
        if (hit != 0) {
          const int src = __ffs(hit) - 1;
          first = b0 + src;
          base = carry + __shfl_sync(0xffffffffu, x - u, src);
          found = true;
        }
        carry += __shfl_sync(0xffffffffu, x, 31);
      }
    }
    if (lane == 0) {
      ctl->lo = lo;
      ctl->hi = hi;
      ctl->units = units;
      ctl->base = base;
      ctl->first = first;
      ctl->ctas = ctas;
    }
  } else if (warp == 1 && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], 1);
      mbar_init(&ctl->q_empty[i], 1);
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], 4);
    }
    for (int i = 0; i < Dm::kSlots; ++i) {
      mbar_init(&ctl->k_full[i], kFp8 ? Dm::kConvWarps : 1);
      mbar_init(&ctl->v_full[i], kFp8 ? Dm::kConvWarps : 1);
      mbar_init(&ctl->k_empty[i], 1);
      mbar_init(&ctl->v_empty[i], 1);
      mbar_init(&ctl->v_fixed[i], 1);
    }
    for (int i = 0; i < Dm::kRawAlloc; ++i) {
      mbar_init(&ctl->raw_k_full[i], 1);
      mbar_init(&ctl->raw_v_full[i], 1);
      mbar_init(&ctl->raw_k_empty[i], Dm::kConvWarps);
      mbar_init(&ctl->raw_v_empty[i], Dm::kConvWarps);
    }
    mbar_init(&ctl->o_done, 1);
    mbar_init(&ctl->o_free, 8);
    mbar_init(&ctl->drain, 1);
    ctl->fail = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const long long lo = ctl->lo, hi = ctl->hi;
  if (lo >= hi) return;
  if (warp == kTrMmaWarp) {
    tmem_alloc(&ctl->tmem, kTrTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  int n = ctl->first;  // every role walks the share's pieces by itself
  long long base = ctl->base;
  TrPiece pc;

  if (warp == kTrTmaWarp) {
    // ---------------------------------------------------------------- loads
    uint32_t g = 0, pi = 0;
    bool run = true;
    for (long long f = lo; run && tr_next(a, f, hi, n, base, pc); f = pc.fend, ++pi) {
      const uint32_t qb = pi % a.q_bufs, quse = pi / a.q_bufs;
      if (quse > 0 && !tr_wait(&ctl->q_empty[qb], quse - 1, ctl, a.status)) break;
      if (lane == 0) {
        unsigned char* dst = smem + Dm::kOffQ + qb * Dm::kHalves * a.q_rows * 128;
        mbar_arrive_expect_tx(&ctl->q_full[qb], static_cast<uint32_t>(Dm::kHalves * a.box_rows * 128));
#pragma unroll
        for (int half = 0; half < Dm::kHalves; ++half)
          tma_load_3d(dst + half * a.q_rows * 128, &qmap, 64 * half, pc.h * a.grp, pc.q0 + pc.rt * a.tile_nodes,
                      &ctl->q_full[qb]);
      }
      const int n_pages = (pc.P + pc.T + kPageSize - 1) / kPageSize;
      const int* row = a.block_table + static_cast<size_t>(pc.n) * a.max_pages;
      int id_next = lane < kTrTilePages && pc.k0 * kTrTilePages + lane < n_pages ? __ldg(row + pc.k0 * kTrTilePages + lane) : 0;
      for (int k = pc.k0; k < pc.k1; ++k, ++g) {
        const int pg = k * kTrTilePages + lane;
        const int id = id_next;
        if (k + 1 < pc.k1 && lane < kTrTilePages && pg + kTrTilePages < n_pages) id_next = __ldg(row + pg + kTrTilePages);
        bool valid = lane < kTrTilePages && pg < n_pages;
        if (valid && (id < 0 || id >= a.num_pages)) {
          set_status(a.status, PKV_ERR_OUT_OF_BOUNDS);
          valid = false;
        }
        const uint32_t pages = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, valid)));
        const long long tile = static_cast<long long>(id) * a.hkv + pc.h;
        if constexpr (kFp8) {
          const uint32_t rs = g % Dm::kRawAlloc, use = g / Dm::kRawAlloc;
          const uint32_t bytes = pages * static_cast<uint32_t>(kPageSize * D + kPageSize);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            uint64_t* full = kv ? &ctl->raw_v_full[rs] : &ctl->raw_k_full[rs];
            uint64_t* empty = kv ? &ctl->raw_v_empty[rs] : &ctl->raw_k_empty[rs];
            if (use > 0 && !tr_wait(empty, use - 1, ctl, a.status)) {
              run = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(full, bytes);
            __syncwarp();
            if (valid) {
              bulk_load(smem + (kv ? Dm::kOffRawV : Dm::kOffRawK) + rs * Dm::kRawTile + lane * (kPageSize * D),
                        (kv ? a.v_raw : a.k_raw) + tile * (kPageSize * D), kPageSize * D, full);
              bulk_load(smem + Dm::kOffScales + (rs * 2 + kv) * kTrKeys + lane * kPageSize,
                        a.scales + tile * kScaleBytes + kv * kPageSize, kPageSize, full);
            }
          }
          if (!run) break;
        } else {
          const uint32_t st = g % Dm::kSlots, use = g / Dm::kSlots;
          const uint32_t bytes = pages * static_cast<uint32_t>(Dm::kPage);
          if (use > 0 && !tr_wait(&ctl->k_empty[st], use - 1, ctl, a.status)) {
            run = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&ctl->k_full[st], bytes);
          __syncwarp();
          if (valid) {
            unsigned char* kd = smem + Dm::kOffK + st * Dm::kTile + lane * (kPageSize * 128);
#pragma unroll
            for (int half = 0; half < Dm::kHalves; ++half)
              tma_load_4d(kd + half * kTrHalfBytes, &kmap, 0, 0, half, static_cast<int>(tile), &ctl->k_full[st]);
          }
          if (use > 0 && !tr_wait(&ctl->v_empty[st], use - 1, ctl, a.status)) {
            run = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&ctl->v_full[st], bytes);
          __syncwarp();
          if (valid)
            tma_load_4d(smem + Dm::kOffV + st * Dm::kTile + lane * Dm::kPage, &vmap, 0, 0, 0, static_cast<int>(tile),
                        &ctl->v_full[st]);
        }
      }
    }
    if (*reinterpret_cast<volatile int*>(&ctl->fail) != 0) {
      // the CTA gave up: its copies in flight land before it ends (a wait for one that was never issued runs out)
      constexpr uint32_t kRing = kFp8 ? Dm::kRawAlloc : Dm::kSlots;
      for (uint32_t i = g > kRing ? g - kRing : 0; i <= g; ++i) {
        uint64_t* kf = kFp8 ? &ctl->raw_k_full[i % Dm::kRawAlloc] : &ctl->k_full[i % Dm::kSlots];
        uint64_t* vf = kFp8 ? &ctl->raw_v_full[i % Dm::kRawAlloc] : &ctl->v_full[i % Dm::kSlots];
        mbar_wait_bounded(kf, (i / kRing) & 1u, kDrainCycles);
        mbar_wait_bounded(vf, (i / kRing) & 1u, kDrainCycles);
      }
      for (uint32_t i = pi > 1 ? pi - 1 : 0; i <= pi; ++i)
        mbar_wait_bounded(&ctl->q_full[i % a.q_bufs], (i / a.q_bufs) & 1u, kDrainCycles);
    }
  } else if (warp == kTrMmaWarp) {
    // ---------------------------------------------------------------- products
    // S of tile g + 2 follows the values of tile g (same group, S and P share their columns); tiles run across pieces
    struct Tile {
      TrPiece pc;
      int n, k;
      long long base;
      uint32_t pi, g;
      bool ok;
    };
    auto start = [&](Tile& t) {
      t.n = n;
      t.base = base;
      t.pi = t.g = 0;
      t.ok = tr_next(a, lo, hi, t.n, t.base, t.pc);
      t.k = t.pc.k0;
    };
    auto step = [&](Tile& t) {
      ++t.g;
      if (++t.k < t.pc.k1) return;
      ++t.pi;
      t.ok = tr_next(a, t.pc.fend, hi, t.n, t.base, t.pc);
      t.k = t.pc.k0;
    };
    Tile s, v;
    start(s);
    start(v);
    auto scores = [&]() {
      const uint32_t st = s.g % Dm::kSlots, w = s.g & 1u, qb = s.pi % a.q_bufs;
      if (s.k == s.pc.k0 && !tr_wait(&ctl->q_full[qb], s.pi / a.q_bufs, ctl, a.status)) return false;
      if (!tr_wait(&ctl->k_full[st], s.g / Dm::kSlots, ctl, a.status)) return false;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t qa = smem_u32(smem + Dm::kOffQ + qb * Dm::kHalves * a.q_rows * 128);
        const uint32_t kb = smem_u32(smem + Dm::kOffK + st * Dm::kTile);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_ss(tmem + kTrColS + 128 * w, sdesc_sw128(qa + (i >> 2) * a.q_rows * 128 + (i & 3) * 32, 16, 1024),
                 sdesc_sw128(kb + (i >> 2) * kTrHalfBytes + (i & 3) * 32, 16, 1024), Dm::kIdescQK, i > 0 ? 1u : 0u);
        mma_commit(&ctl->s_full[w]);
        mma_commit(&ctl->k_empty[st]);
        if (s.k == s.pc.k1 - 1) mma_commit(&ctl->q_empty[qb]);
      }
      __syncwarp();
      step(s);
      return true;
    };
    bool ok = true;
    for (int i = 0; i < 2; ++i)
      if (ok && s.ok) ok = scores();
    while (ok && v.ok) {
      const uint32_t st = v.g % Dm::kSlots, w = v.g & 1u;
      const bool first = v.k == v.pc.k0, last = v.k == v.pc.k1 - 1;
      // the previous piece's O is read
      if (first && v.pi > 0 && !(ok = tr_wait(&ctl->o_free, v.pi - 1, ctl, a.status))) break;
      if (!(ok = tr_wait(&ctl->v_full[st], v.g / Dm::kSlots, ctl, a.status))) break;
      if (!kFp8 && !(ok = tr_wait(&ctl->v_fixed[st], v.g / Dm::kSlots, ctl, a.status))) break;
      if (!(ok = tr_wait(&ctl->p_full[w], v.g >> 1, ctl, a.status))) break;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t vb = smem_u32(smem + Dm::kOffV + st * Dm::kTile);
        const bool fresh = v.k - v.pc.k0 < 2;  // the group's first tile of the piece
#pragma unroll
        for (int i = 0; i < kTrTilePages; ++i)
          mma_ts(tmem + kTrColO + 128 * w, tmem + kTrColS + 128 * w + 8 * i, sdesc_sw128(vb + i * Dm::kPage, 2048, 1024),
                 Dm::kIdescPV, (!fresh || i > 0) ? 1u : 0u);
        mma_commit(&ctl->v_empty[st]);
        if (last) mma_commit(&ctl->o_done);
      }
      __syncwarp();
      step(v);
      if (s.ok) ok = scores();
    }
    if (!ok) {  // the CTA gave up: the products in flight end before it frees their memory
      if (lane == 0) {
        mma_commit(&ctl->drain);
        mbar_wait_bounded(&ctl->drain, 0, kDrainCycles);
      }
      __syncwarp();
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax and epilogue
    const int w = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lanes + kTrColS + 128 * w, t_o = tmem + lanes + kTrColO;
    uint32_t g = 0, pi = 0;
    bool ok = true;
    for (long long f = lo; ok && tr_next(a, f, hi, n, base, pc); f = pc.fend, ++pi) {
      const int nodes = min(a.tile_nodes, pc.T - pc.rt * a.tile_nodes);
      const int rows = nodes * a.grp;
      const bool work = quarter * 32 < rows;
      const int node = pc.rt * a.tile_nodes + r / a.grp;
      unsigned long long mask = 0;
      if (r < rows) {
        mask = a.masks != nullptr ? __ldg(a.masks + pc.q0 + node) : (2ull << node) - 1;
        mask &= pc.T < 64 ? (1ull << pc.T) - 1 : ~0ull;
      }
      float m = -CUDART_INF_F, l = 0.f;
      int mine = 0;  // this group's tiles so far
      for (int k = pc.k0; k < pc.k1; ++k, ++g) {
        if ((g & 1u) != static_cast<uint32_t>(w)) continue;
        if (!(ok = tr_wait(&ctl->s_full[w], g >> 1, ctl, a.status))) break;
        if (work) {
          tc_fence_after();
          const bool tail = (k + 1) * kTrKeys > pc.P;  // nodes, or keys past the end, among the tile's
          uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
          if (tail) {
            const int sh = pc.P - k * kTrKeys;  // keys of the prefix in this tile
            unsigned long long v0, v1;
            if (sh <= 0) {
              v0 = sh > -64 ? mask >> -sh : 0;
              v1 = 0;
            } else if (sh < 64) {
              v0 = (mask << sh) | ((1ull << sh) - 1);
              v1 = mask >> (64 - sh);
            } else {
              v0 = ~0ull;
              v1 = sh == 64 ? mask : (mask << (sh - 64)) | ((1ull << (sh - 64)) - 1);
            }
            vis[0] = static_cast<uint32_t>(v0);
            vis[1] = static_cast<uint32_t>(v0 >> 32);
            vis[2] = static_cast<uint32_t>(v1);
            vis[3] = static_cast<uint32_t>(v1 >> 32);
          }
          const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
          float mx = -CUDART_INF_F;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t sr[32];
            tmem_ld32(t_s + 32 * c, sr);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float2 x = __fmul2_rn(make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), sc2);
              if (tail) {
                if (!(vis[c] >> e & 1u)) x.x = -CUDART_INF_F;
                if (!(vis[c] >> (e + 1) & 1u)) x.y = -CUDART_INF_F;
              }
              mx = fmaxf(mx, fmaxf(x.x, x.y));
            }
          }
          // the maximum moves, and O with it, only when it grows by more than 2^8 (weights up to 2^8 are fine)
          const float m_new = fmaxf(m, mx);
          const bool grow = m == -CUDART_INF_F ? m_new != -CUDART_INF_F : m_new - m > 8.f;
          if (__any_sync(0xffffffffu, grow)) {
            const float alpha = !grow ? 1.f : m == -CUDART_INF_F ? 0.f : ex2(m - m_new);
            if (mine > 0) {
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(t_o + 128 * w + 32 * c, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st32(t_o + 128 * w + 32 * c, o);
              }
            }
            if (grow) {
              l *= alpha;
              m = m_new;
            }
          }
          const float base_m = m == -CUDART_INF_F ? 0.f : -m;
          const float2 nm2 = make_float2(base_m, base_m);
          float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t sr[32], pk[16];
            tmem_ld32(t_s + 32 * c, sr);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 t =
                  __ffma2_rn(make_float2(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), sc2, nm2);
              float2 p = make_float2(ex2(t.x), ex2(t.y));
              if (tail) {
                if (!(vis[c] >> e & 1u)) p.x = 0.f;
                if (!(vis[c] >> (e + 1) & 1u)) p.y = 0.f;
              }
              l2 = __fadd2_rn(l2, p);
              pk[e >> 1] = pack_bf16x2(p.x, p.y);
            }
            tmem_st16(t_s + 16 * c, pk);  // columns that are read: 16 c + 16 <= 32 c + 32
          }
          l += l2.x + l2.y;
          tmem_st_wait();
          tc_fence_before();
        }
        ++mine;
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&ctl->p_full[w]);
      }
      // ---- the two groups' halves of the row, and its output or record; each group takes half of the columns
      ctl->stat[w][0][r] = m;
      ctl->stat[w][1][r] = l;
      ok = ok && tr_wait(&ctl->o_done, pi, ctl, a.status);
      tc_fence_after();
      if (!(ok = tr_group_all(1, ok))) break;  // all eight warps go on, or none
      const float m0 = ctl->stat[0][0][r], l0 = ctl->stat[0][1][r], m1 = ctl->stat[1][0][r], l1 = ctl->stat[1][1][r];
      const float M = fmaxf(m0, m1);
      // (a half that saw nothing has sum 0, or NaN where every score was NaN)
      const float a0 = m0 == -CUDART_INF_F ? 0.f : ex2(m0 - M), a1 = m1 == -CUDART_INF_F ? 0.f : ex2(m1 - M);
      const float L = (m0 == -CUDART_INF_F ? l0 : l0 * a0) + (m1 == -CUDART_INF_F ? l1 : l1 * a1);
      const bool both = pc.k1 - pc.k0 > 1;
      const uint32_t w0 = (g - static_cast<uint32_t>(pc.k1 - pc.k0)) & 1u;  // the group of the first tile
      const bool have0 = both || w0 == 0, have1 = both || w0 == 1;
      unsigned long long bad = 0;
      if (pc.k1 * kTrKeys > pc.P) {
#pragma unroll
        for (int i = 0; i < Dm::kMenders; ++i) {
          const volatile uint32_t* b = ctl->bad[pi % Dm::kBadRing][i];
          bad |= static_cast<unsigned long long>(b[1]) << 32 | b[0];
        }
        bad &= mask;
      }
      const bool whole = pc.k0 == 0 && pc.k1 == pc.nt;
      const float inv = L == 0.f ? 0.f : 1.f / L;
      __nv_bfloat16* orow = a.out + (static_cast<size_t>(pc.q0 + node) * a.hq + pc.h * a.grp + r % a.grp) * D + w * (D / 2);
      // record: slot 1 of the CTA where the item's first key tile is, slot 0 of the others
      float* rec = a.records + (static_cast<size_t>(blockIdx.x) * 2 + (pc.k0 == 0 ? 1 : 0)) * (kTrRecBytes / 4);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t x[32], y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = y[e] = 0u;
        __syncwarp();
        if (work) {
          const uint32_t at = t_o + w * (D / 2) + 32 * c;
          if (have0) tmem_ld32(at, x);
          if (have1) tmem_ld32(at + 128, y);
          tmem_ld_wait();
        }
        if (c == D / 64 - 1) {  // O is read: the next piece's products may overwrite it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&ctl->o_free);
        }
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = a0 * __uint_as_float(x[e]) + a1 * __uint_as_float(y[e]);
        if (bad != 0) tr_add_nonfinite<D, kFp8>(a, pc, bad, w * (D / 2) + 32 * c, o);
        if (r < rows) {
          if (whole) {
            tr_store<32>(orow + 32 * c, o, inv);
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              reinterpret_cast<float4*>(rec)[(w * (D / 8) + c * 8 + q) * kTrRows + r] =
                  make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          }
        }
      }
      if (!whole) {
        if (r < rows && w == 0) {
          rec[128 * kTrRows + r] = M;
          rec[129 * kTrRows + r] = L;
        }
        __threadfence();
      }
      tr_group_sync(2);  // the rows' maxima and sums are read, the record is written
      if (!whole) {
        const long long units = ctl->units;
        const int ctas = ctl->ctas;
        const int c0 = tr_cta_of(pc.fseg + kItemCost, units, ctas);
        const int c1 = tr_cta_of(pc.fseg + kItemCost + pc.nt - 1, units, ctas);
        if (tid == 0) {
          const int done = atomicAdd(a.counters + c0, 1) == c1 - c0;
          if (done) a.counters[c0] = 0;
          __threadfence();
          *reinterpret_cast<volatile int*>(&ctl->merge) = done;
        }
        tr_group_sync(1);
        if (*reinterpret_cast<volatile int*>(&ctl->merge) != 0 && r < rows) {
          // all pieces are there: joined in CTA order
          auto record = [&](int c) { return a.records + (static_cast<size_t>(c) * 2 + (c == c0 ? 1 : 0)) * (kTrRecBytes / 4); };
          float top = -CUDART_INF_F;
          for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(record(c) + 128 * kTrRows + r));
#pragma unroll
          for (int ch = 0; ch < D / 64; ++ch) {
            float o[32], sum = 0.f;
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
            for (int c = c0; c <= c1; ++c) {
              const float* x = record(c);
              const float mc = __ldcg(x + 128 * kTrRows + r), lc = __ldcg(x + 129 * kTrRows + r);
              const float wc = mc == -CUDART_INF_F ? 0.f : ex2(mc - top);
              sum += mc == -CUDART_INF_F ? lc : lc * wc;
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const float4 y = __ldcg(reinterpret_cast<const float4*>(x) + (w * (D / 8) + ch * 8 + q) * kTrRows + r);
                o[4 * q] += wc * y.x;
                o[4 * q + 1] += wc * y.y;
                o[4 * q + 2] += wc * y.z;
                o[4 * q + 3] += wc * y.w;
              }
            }
            tr_store<32>(orow + 32 * ch, o, sum == 0.f ? 0.f : 1.f / sum);
          }
        }
      }
    }
  } else if constexpr (!kFp8) {
    // ---------------------------------------------------------------- value tiles with nodes or an end in them
    uint32_t g = 0, pi = 0;
    bool ok = true;
    for (long long f = lo; ok && tr_next(a, f, hi, n, base, pc); f = pc.fend, ++pi) {
      unsigned long long bad = 0;
      for (int k = pc.k0; k < pc.k1; ++k, ++g) {
        const uint32_t st = g % Dm::kSlots;
        if (!(ok = tr_wait(&ctl->v_full[st], g / Dm::kSlots, ctl, a.status))) break;
        if ((k + 1) * kTrKeys <= pc.P) {
          if (lane == 0) mbar_arrive_cta(&ctl->v_fixed[st]);
          continue;
        }
        const int len = pc.P + pc.T - k * kTrKeys;          // rows of the tile before the end
        const int t0 = max(pc.P - k * kTrKeys, 0);          // its first row behind the prefix
        unsigned char* vt = smem + Dm::kOffV + st * Dm::kTile;
        constexpr int kChunks = D / 8;
        for (int i = t0 * kChunks + lane; i < kTrKeys * kChunks; i += 32) {
          const int t = i / kChunks;
          uint4* at = reinterpret_cast<uint4*>(vt + tr_v_off<D>(t, i % kChunks));
          if (t >= len) {
            *at = make_uint4(0, 0, 0, 0);
            continue;
          }
          uint4 x = *at;
          if (nonfinite_bf16x2(x.x) || nonfinite_bf16x2(x.y) || nonfinite_bf16x2(x.z) || nonfinite_bf16x2(x.w)) {
            *at = make_uint4(finite_bf16x2(x.x), finite_bf16x2(x.y), finite_bf16x2(x.z), finite_bf16x2(x.w));
            bad |= 1ull << (k * kTrKeys + t - pc.P);
          }
        }
        // (the nodes' bits are complete before the products of the piece's last tile)
        const uint32_t b0 = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(bad));
        const uint32_t b1 = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(bad >> 32));
        if (lane == 0) {
          ctl->bad[pi % Dm::kBadRing][0][0] = b0;
          ctl->bad[pi % Dm::kBadRing][0][1] = b1;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&ctl->v_fixed[st]);
      }
    }
  } else {
    // ---------------------------------------------------------------- 8-bit tiles as bf16 tiles
    const int kv = (warp - 10) / Dm::kConvWarps;                  // 0: K, 1: V
    const int sub = ((warp - 10) % Dm::kConvWarps);               // this warp's rows: 32 sub ..
    uint64_t* full = kv ? ctl->v_full : ctl->k_full;
    uint64_t* empty = kv ? ctl->v_empty : ctl->k_empty;
    uint64_t* raw_full = kv ? ctl->raw_v_full : ctl->raw_k_full;
    uint64_t* raw_empty = kv ? ctl->raw_v_empty : ctl->raw_k_empty;
    uint32_t g = 0, pi = 0;
    bool ok = true;
    for (long long f = lo; ok && tr_next(a, f, hi, n, base, pc); f = pc.fend, ++pi) {
      unsigned long long bad = 0;
      for (int k = pc.k0; k < pc.k1; ++k, ++g) {
        const uint32_t st = g % Dm::kSlots, use = g / Dm::kSlots, rs = g % Dm::kRawAlloc;
        if (!(ok = tr_wait(&raw_full[rs], g / Dm::kRawAlloc, ctl, a.status))) break;
        if (use > 0 && !(ok = tr_wait(&empty[st], use - 1, ctl, a.status))) break;
        const unsigned char* src = smem + (kv ? Dm::kOffRawV : Dm::kOffRawK) + rs * Dm::kRawTile;
        const unsigned char* sc = smem + Dm::kOffScales + (rs * 2 + kv) * kTrKeys;
        unsigned char* dst = smem + (kv ? Dm::kOffV : Dm::kOffK) + st * Dm::kTile;
        const bool tail = kv && (k + 1) * kTrKeys > pc.P;
        const int len = pc.P + pc.T - k * kTrKeys;
        // 16 values a lane at a time. Of 8 lanes four take one half of a row, four the other half of the next, so
        // that the reads (128-byte rows) and the writes (swizzled) both hit every bank once.
        constexpr int kC = D / 16;  // 16-value chunks of a row
#pragma unroll 4
        for (int i = 0; i < 32 * kC / 32; ++i) {
          int t, c;
          if constexpr (D == 128) {
            const int pair = lane >> 3, bit = (lane >> 2) & 1;
            t = 32 * sub + (i >> 1) * 8 + pair * 2 + bit;
            c = (lane & 3) + 4 * (bit ^ (i & 1));
          } else {
            t = 32 * sub + i * 8 + (lane >> 2);
            c = lane & 3;
          }
          const uint4 x = *reinterpret_cast<const uint4*>(src + t * D + c * 16);
          const float s = __uint_as_float(static_cast<uint32_t>(sc[t]) << 23);
          uint32_t y[8];
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t lo2, hi2;
            e4m3x4_to_f16x4(xs[q], lo2, hi2);
            const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&lo2));
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hi2));
            y[2 * q] = pack_bf16x2(u.x * s, u.y * s);
            y[2 * q + 1] = pack_bf16x2(v.x * s, v.y * s);
          }
          if (tail && k * kTrKeys + t >= pc.P) {
            bool odd = false;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              if (t >= len) y[q] = 0u;
              if (nonfinite_bf16x2(y[q])) {
                odd = true;
                y[q] = finite_bf16x2(y[q]);
              }
            }
            if (odd) bad |= 1ull << (k * kTrKeys + t - pc.P);
          }
          const uint32_t o0 = kv ? tr_v_off<D>(t, 2 * c) : tr_k_off(t, 2 * c);
          const uint32_t o1 = kv ? tr_v_off<D>(t, 2 * c + 1) : tr_k_off(t, 2 * c + 1);
          *reinterpret_cast<uint4*>(dst + o0) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(dst + o1) = make_uint4(y[4], y[5], y[6], y[7]);
        }
        if (tail) {  // (the nodes' bits are complete before the products of the piece's last tile)
          const uint32_t b0 = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(bad));
          const uint32_t b1 = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(bad >> 32));
          if (lane == 0) {
            ctl->bad[pi % Dm::kBadRing][sub][0] = b0;
            ctl->bad[pi % Dm::kBadRing][sub][1] = b1;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cta(&raw_empty[rs]);
          mbar_arrive_cta(&full[st]);
        }
      }
    }
  }

  // ---------------------------------------------------------------- end
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kTrMmaWarp) tmem_dealloc(tmem, kTrTmemCols);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
  static EncodeTiledFn fn = nullptr;
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// Counters (one per CTA: the CTA that holds an item's first key tile, where that item is cut) in a block of fixed
// size, then the records: what a call leaves in the records never lies where another one looks for zeros.
size_t counter_bytes(int num_sms) { return (static_cast<size_t>(num_sms) * 4 + 255) / 256 * 256; }

template <int D, bool kFp8>
int launch(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap, const TrArgs& a, cudaStream_t stream) {
  static bool attr_set[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  if (dev >= 64 || !attr_set[dev]) {
    if (cudaFuncSetAttribute(tree_attn_kernel<D, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             tr_smem_bytes<D, kFp8>()) != cudaSuccess)
      return PKV_ERR_CUDA;
    if (dev < 64) attr_set[dev] = true;
  }
  return launch_pdl(tree_attn_kernel<D, kFp8>, dim3(static_cast<unsigned>(a.ctas)), dim3(TrDim<D, kFp8>::kThreads),
                    tr_smem_bytes<D, kFp8>(), stream, qmap, kmap, vmap, a) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

}  // namespace

int tree_max_nodes() { return kTrMaxNodes; }
int tree_max_seqs() { return kTrMaxSeqs; }

size_t tree_workspace_bytes(int num_sms) { return PKV_STATUS_BYTES + counter_bytes(num_sms) + 2 * num_sms * kTrRecBytes; }

int launch_tree_attn(const TreeAttn& t, int num_q_heads, int num_kv_heads, int head_dim, int32_t num_pages, void* workspace,
                     int num_sms, cudaStream_t stream) {
  if (!decode_supported(num_q_heads, num_kv_heads, head_dim, kPageSize)) return PKV_ERR_UNSUPPORTED;
  const bool fp8 = t.kv_scales != nullptr;
  EncodeTiledFn enc = encoder();
  if (enc == nullptr) return PKV_ERR_CUDA;
  TrArgs a = {};
  a.block_table = t.block_table;
  a.prefix_lens = t.prefix_lens;
  a.cu_nodes = t.cu_nodes;
  a.masks = reinterpret_cast<const unsigned long long*>(t.tree_mask);
  a.k_raw = static_cast<const uint8_t*>(t.k_pages);
  a.v_raw = static_cast<const uint8_t*>(t.v_pages);
  a.scales = static_cast<const uint8_t*>(t.kv_scales);
  a.v_pages = static_cast<const __nv_bfloat16*>(t.v_pages);
  a.out = static_cast<__nv_bfloat16*>(t.out);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.status = reinterpret_cast<int*>(ws);
  a.counters = reinterpret_cast<int*>(ws + PKV_STATUS_BYTES);
  a.records = reinterpret_cast<float*>(ws + PKV_STATUS_BYTES + counter_bytes(num_sms));
  a.num_seqs = t.num_seqs;
  a.total = t.total_nodes;
  a.max_pages = t.max_pages;
  a.num_pages = num_pages;
  a.max_nodes = t.max_nodes;
  a.hq = num_q_heads;
  a.hkv = num_kv_heads;
  a.grp = num_q_heads / num_kv_heads;
  a.tile_nodes = kTrRows / a.grp;
  a.box_rows = a.grp * (t.max_nodes < a.tile_nodes ? t.max_nodes : a.tile_nodes);
  a.q_rows = (a.box_rows + 7) / 8 * 8;
  a.q_bufs = a.q_rows <= kTrRows / 2 ? 2 : 1;
  a.ctas = num_sms;
  a.scale_log2 = t.scale * kLog2e;

  const cuuint64_t hd = static_cast<cuuint64_t>(head_dim);
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  CUtensorMap qmap, kmap, vmap;
  {
    const cuuint64_t dims[3] = {hd, static_cast<cuuint64_t>(num_q_heads), static_cast<cuuint64_t>(t.total_nodes)};
    const cuuint64_t strides[2] = {hd * 2, static_cast<cuuint64_t>(num_q_heads) * hd * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.grp), static_cast<cuuint32_t>(a.box_rows / a.grp)};
    if (enc(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(t.q), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return PKV_ERR_CUDA;
  }
  if (fp8) {  // read through plain bulk copies
    kmap = qmap;
    vmap = qmap;
    return head_dim == 64 ? launch<64, true>(qmap, kmap, vmap, a, stream) : launch<128, true>(qmap, kmap, vmap, a, stream);
  }
  const int rc = encode_page_maps(t.k_pages, t.v_pages, head_dim, num_pages, num_kv_heads, &kmap, &vmap);
  if (rc != PKV_OK) return rc;
  {
    // K in boxes of one 64-dim half of a page: the halves of a tile's 128 rows lie apart in shared memory
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(kPageSize), hd / 64, static_cast<cuuint64_t>(num_pages) * num_kv_heads};
    const cuuint64_t strides[3] = {hd * 2, 128, hd * 2 * kPageSize};
    const cuuint32_t box[4] = {64, kPageSize, 1, 1};
    if (enc(&kmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(t.k_pages), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return PKV_ERR_CUDA;
  }
  return head_dim == 64 ? launch<64, false>(qmap, kmap, vmap, a, stream) : launch<128, false>(qmap, kmap, vmap, a, stream);
}

}  // namespace pkv
