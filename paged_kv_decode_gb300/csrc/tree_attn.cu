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
//    (a 3-D TMA box for each 64 dims). Items cost kItemCost + ceil((P + T) / 128) units; every
//    CTA (one per SM) takes an equal contiguous share of the units, cutting
//    items; a cut item's partial results go to records, and a second small
//    kernel joins them in CTA order (the same bits every time). Where all items
//    are small, or whole items balance as well, none is cut.
//  * Warp 9 plans the CTA's pieces, publishes them to the other warps and loads
//    Q and the K and V tiles of 128 keys through the block table into rings.
//    Warp 8 issues S = Q K^T into TMEM, warp 11 O += P V with P as the
//    tensor-memory operand. Key tiles alternate between two groups of four
//    softmax warps, each with its own S, P, O, maximum and sum: one group's
//    exponentials run beside the other's products. The two halves of a row are
//    joined in the epilogue, straight from TMEM. Warps whose 32 rows are all
//    past the item's last one do no arithmetic.
//  * 8-bit cache: a value 2^e v is exact in bf16, so four warps for K and four
//    for V expand each tile into the bf16 ring and everything behind that is
//    the bf16 kernel: the outputs are those of pkv_expand_fp8 followed by the
//    bf16 call, bit for bit.
//  * P is rounded to bf16 before it multiplies V, the operand type of the product
//    (off by at most 2^-8 of a weight); the sum l keeps the unrounded weights in
//    fp32. Against 64 bits outputs are off by 0.0022 (relative, in the square mean)
//    where the bf16 output's own rounding gives 0.0017. The 8-bit decode kernel's
//    weights are fp16, three bits more: its operands are.
//  * Value rows behind the last node are zeroed in shared memory (they may hold
//    anything, and 0 * NaN = NaN). A node's value row that holds infinities or
//    NaN would reach rows that do not see the node the same way: such elements
//    are zeroed too, and added back, in the epilogue, to the rows that see them.
//
// Measured on one GB300 (us in a graph, inputs resident, of 16 / 8 / 128 where not
// said otherwise; in brackets the cache's bytes at 6682 GB/s): 16 requests of 300
// to 3000 tokens with 16 nodes 31.8 (20.0), one of 40k tokens with 32 nodes 35.5
// (24.6), 27 ragged requests of 32 / 8 / 128 119 (65), two of 37 and 200 tokens
// 7.4; 8-bit cache: the 16 requests 32.0 (10.2), the one 33.3 (12.4), about the
// times of the bf16 cache. What is left: long batches run at 92 % of the memory's
// rate (16 requests of 6600 tokens: 70.7 of 65.2, in 8 bits 74.7 of 33.0); shorter
// ones pay 4 us from the launch to the first tile
// (the lengths, the table and the tile are three dependent reads), 2 us an item and
// 3.5 us for the join and its launch. Where a request has more than 128 rows each
// tile of rows reads the keys for itself, at the copies' rate (1.3 us a tile).
// Neither the products nor the softmax bound the bf16 form (the ragged requests
// took 119.8 us, 119.9 without the softmax, 120.4 without the value product). The
// 8-bit form is bound by the instructions that expand its tiles, then by the
// softmax (of 36.0 us at one stage 27.0 were left without the expansion's steps,
// 33.4 without the softmax; 34 with twice as many expanding warps).
#include <cuda.h>
#include <float.h>
#include <math_constants.h>

#include <type_traits>

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
constexpr int kTrQkWarp = 8, kTrTmaWarp = 9, kTrMendWarp = 10, kTrPvWarp = 11;
constexpr uint32_t kTrColS = 0, kTrColO = 256, kTrTmemCols = 512;  // S_w, O_w at + 128 w
constexpr long long kDrainCycles = 20000000LL;                     // 10 ms: far more than a copy in flight takes

// Fixed work of an item (query load, pipeline fill and drain, epilogue) in key tiles: 27 ragged requests of 32 / 8 / 128 take
// 119 us with 3, 126 with 2. And the largest item, in the same units, that is never cut where all items are that small: with
// 7 two requests of 37 and 200 tokens take 9.1 us and 16 of 50 to 490 12.3, cut into shares 10.5 and 14.4 (as nothing can be
// cut at up to 32 pages, the join is not launched there either: 7.4 and 10.8). Many such requests would rather be cut: 64 of
// them take 34.1 us whole, 30.0 in shares.
#ifndef PKV_TREE_ITEM_COST
#define PKV_TREE_ITEM_COST 3
#endif
#ifndef PKV_TREE_SMALL_ITEM
#define PKV_TREE_SMALL_ITEM 7
#endif
constexpr int kItemCost = PKV_TREE_ITEM_COST;
constexpr int kSmallItem = PKV_TREE_SMALL_ITEM;

template <int D, bool kFp8>
struct TrDim {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kTrKeys * D * 2;  // K or V tile (bf16)
  static constexpr int kPage = kPageSize * D * 2;       // a page of it
  static constexpr int kSlots = kFp8 ? (D == 128 ? 2 : 3) : (D == 128 ? 3 : 6);
  static constexpr int kPieces = kSlots + 1;  // descriptors of pieces in flight
  static constexpr int kRawTile = kTrKeys * D;  // 8-bit tile
  static constexpr int kRawSlots = kFp8 ? (D == 128 ? 2 : 5) : 0;
  static constexpr int kRawAlloc = kFp8 ? kRawSlots : 1;  // array sizes may not be 0
  static constexpr int kConvWarps = 4;                    // each for K (warps 12 ..) and for V (16 ..)
  // bf16: 12 warps. 8-bit: 20 warps, 10 idle; the launch gives each thread 96 registers, the two softmax warpgroups rise
  // to 152, the other three drop to 56.
  static constexpr int kThreads = (kFp8 ? 12 + 2 * kConvWarps : 12) * 32;
  static constexpr int kRegsSoftmax = 152, kRegsOther = 56;
  static_assert(!kFp8 || 256 * kRegsSoftmax + (kThreads - 256) * kRegsOther <= kThreads * 96, "register split");
  static constexpr int kReaders = 10 + (kFp8 ? 2 * kConvWarps : 1);  // warps that read a piece's descriptor
  // shared memory, from a 1024-byte aligned base
  static constexpr int kOffQ = 0;  // one buffer of up to 128 rows, or two of up to 64
  static constexpr int kOffK = kOffQ + kTile;
  static constexpr int kOffV = kOffK + kSlots * kTile;
  static constexpr int kOffRawK = kOffV + kSlots * kTile;
  static constexpr int kOffRawV = kOffRawK + kRawSlots * kRawTile;
  static constexpr int kOffScales = kOffRawV + kRawSlots * kRawTile;  // [raw slot][K, V][128] bytes
  static constexpr int kOffCtl = kOffScales + kRawSlots * 2 * kTrKeys;
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(kTrRows, D, true);  // V is MN-major
};

// The part of an item that a CTA computes.
struct TrPiece {
  int k0, k1;         // key tiles [k0, k1); k1 = 0: the end of the share
  int P, T;           // prefix and nodes of the request
  int row0;           // q / out row (node) of the item's first node
  int node0, rows;    // that node's number in the request; rows of the item
  int h, n;           // KV head, request
  int slot;           // record of a cut item's piece: 0 or 1, or -1: the item is whole
  unsigned long long bad;  // nodes whose value rows in these tiles hold infinities or NaN
};

template <int D, bool kFp8>
struct TrCtl {
  using Dm = TrDim<D, kFp8>;
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[Dm::kSlots], k_empty[Dm::kSlots], v_full[Dm::kSlots], v_empty[Dm::kSlots];
  uint64_t s_full[2], p_full[2];
  uint64_t v_fixed[kFp8 ? 1 : Dm::kSlots];
  uint64_t o_done, o_free, drain, pv_done[2];
  uint64_t raw_k_full[Dm::kRawAlloc], raw_k_empty[Dm::kRawAlloc], raw_v_full[Dm::kRawAlloc], raw_v_empty[Dm::kRawAlloc];
  uint64_t piece_full[Dm::kPieces], piece_empty[Dm::kPieces];
  TrPiece piece[Dm::kPieces];
  uint32_t tmem;
  int fail;
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

// A record: float4 [D / 4 + 1][128 rows]: (m, l, 0, 0) of the rows, then O (unnormalised). Room of head_dim 128's at any.
constexpr size_t kTrRecFloats = static_cast<size_t>(kTrRows) * (128 + 4);
constexpr size_t kTrRecBytes = kTrRecFloats * 4;
// A cut item: what the joining kernel reads (rows 0: none).
struct TrCut {
  int rows, row0, h;
  uint32_t span;  // the CTAs with its first and (in the high half) its last piece
};

struct TrArgs {
  const int* block_table;
  const int* prefix_lens;
  const int* cu_nodes;
  const unsigned long long* masks;  // [total], or nullptr: a chain
  const uint8_t* k_raw;             // 8-bit pools
  const uint8_t* v_raw;
  const uint8_t* scales;
  const __nv_bfloat16* v_pages;  // bf16 pool (rows added back)
  __nv_bfloat16* out;
  int* status;
  TrCut* cuts;     // [ctas], written by every call: of item (n * hkv + h) * node_tiles + rt where by_item, else of the item
                   // whose first key tile CTA i has
  int by_item;     // num_seqs * hkv * node_tiles where that is at most ctas, else 0
  int node_tiles;  // items of a (request, KV head), at most
  float* records;  // [2 * ctas][kTrRecFloats]
  int num_seqs, total, max_pages, num_pages, max_nodes;
  int hq, hkv, grp;
  int tile_nodes;  // nodes of an item: 128 / grp
  uint32_t node_magic;  // 2^32 / tile_nodes, rounded up: x * node_magic >> 32 = x / tile_nodes for the x < 2^15 here
  int box_rows;    // rows of the query box: grp * min(tile_nodes, max_nodes)
  int q_rows;      // ... rounded up to whole swizzle atoms of 8 rows
  int q_bufs;      // query buffers: 2 where two fit
  int ctas;        // CTAs of the grid
  float scale_log2;      // |scale| / ln 2
  uint32_t idesc_qk;     // S = Q K^T, with -Q where the scale is negative
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
__device__ __forceinline__ uint32_t tr_key_tiles(int P, int T) {
  return (static_cast<uint32_t>(P) + T + kTrKeys - 1) / kTrKeys;
}
// Items of a request and KV head, and units of one of them (whole: items are not cut, each counts 1). All units of a call
// fit 32 bits: 4 items of each of up to 1024 * 65535 (request, head) pairs, each of 4 units and one more for 8 pages,
// which are fewer than 2^31: at most 2^30 + 2^30 units.
__device__ __forceinline__ uint32_t tr_node_tiles(const TrArgs& a, int T) {  // T / tile_nodes, rounded up
  return __umulhi(static_cast<uint32_t>(T) + a.tile_nodes - 1, a.node_magic);
}
__device__ __forceinline__ uint32_t tr_cost(int P, int T, bool whole) { return whole ? 1 : kItemCost + tr_key_tiles(P, T); }

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

// A barrier of the eight softmax warps, and whether all of them say ok.
__device__ __forceinline__ bool tr_group_all(int id, bool ok) {
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
// A whole page of one KV head: all of a box's dims but the tile number start at 0.
__device__ __forceinline__ void tma_load_5d(void* smem_dst, const CUtensorMap* map, int tile, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %2, %3}], "
      "[%4];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(tile), "r"(smem_u32(bar))
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

// Byte offset of 16-byte chunk c (8 dims) of token row t in a K or V tile: [8 rows][64-dim half][row of 128 bytes], each
// such block of 1 KiB an atom of the 128-byte swizzle. A page is one TMA box of 4 KiB, and the blocks of a half lie at one
// stride through the whole tile, which is what a descriptor can say of K (8-row groups of a K-major operand) and of V
// (8-key groups of an MN-major one).
template <int D>
__device__ __forceinline__ uint32_t tr_off(int t, int c) {
  return static_cast<uint32_t>((t >> 3) * (8 * D * 2) + (c >> 3) * 1024 + (t & 7) * 128 + (((c & 7) ^ (t & 7)) << 4));
}

// The infinities and NaN in column col of the nodes' value rows in `bad` that this piece holds (0 if there are none).
template <int D, bool kFp8>
__device__ __noinline__ float tr_nonfinite(const TrArgs& a, const TrPiece* pc, unsigned long long bad, int col) {
  float sum = 0.f;
  for (int j = 0; j < kTrMaxNodes; ++j) {
    const int pos = pc->P + j;
    if (!(bad >> j & 1ull) || pos < pc->k0 * kTrKeys || pos >= pc->k1 * kTrKeys) continue;
    const int id = __ldg(a.block_table + static_cast<size_t>(pc->n) * a.max_pages + pos / kPageSize);
    if (id < 0 || id >= a.num_pages) continue;
    const size_t tile = static_cast<size_t>(id) * a.hkv + pc->h;
    const size_t at = (tile * kPageSize + pos % kPageSize) * D + col;
    float x;
    if constexpr (kFp8) {  // the expansion's arithmetic: the scale byte, too, can make infinities and NaN
      const uint32_t e = a.scales[tile * kScaleBytes + kPageSize + pos % kPageSize];
      uint32_t lo, hi;
      e4m3x4_to_f16x4(a.v_raw[at], lo, hi);
      const float v = __half2float(__ushort_as_half(static_cast<unsigned short>(lo)));
      x = __bfloat162float(__float2bfloat16_rn(v * __uint_as_float(e << 23)));
    } else {
      x = __bfloat162float(a.v_pages[at]);
    }
    if (!(fabsf(x) < CUDART_INF_F)) sum += x;
  }
  return sum;
}

// 64 columns of S: two loads, one wait
__device__ __forceinline__ void tr_load64(uint32_t taddr, uint32_t (&x)[2][32]) {
  tmem_ld32(taddr, x[0]);
  tmem_ld32(taddr + 32, x[1]);
  tmem_ld_wait();
}
__device__ __forceinline__ float tr_max64(const uint32_t (&x)[2][32]) {
  float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      m0 = fmaxf(m0, __uint_as_float(x[c][e]));
      m1 = fmaxf(m1, __uint_as_float(x[c][e + 1]));
    }
  return fmaxf(m0, m1);
}
// the weight of a score or of a part whose maximum lies d <= 0 below the row's
__device__ __forceinline__ float tr_weight(float d, float scale_log2) { return ex2(d * scale_log2); }
// P = 2^((s - m) * scale) of 64 columns, as bf16 over 32 columns; their sum joins l2. The difference comes first: the
// largest score's weight is 2^0 whatever its size, where s * scale - m * scale as one multiply-add leaves the rounding of
// m * scale, which for scores past 2^30 is a weight of infinity or 0.
__device__ __forceinline__ void tr_exp64(uint32_t taddr, const uint32_t (&x)[2][32], float2 sc2, float2 nm2, float2& l2) {
  uint32_t pk[32];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float2 t =
          __fmul2_rn(__fadd2_rn(make_float2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])), nm2), sc2);
      const float2 p = make_float2(ex2(t.x), ex2(t.y));
      l2 = __fadd2_rn(l2, p);
      pk[c * 16 + (e >> 1)] = pack_bf16x2(p.x, p.y);
    }
  tmem_st32(taddr, pk);
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

  // ---- before the wait for the kernel in front: nothing here touches an argument buffer
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzle atoms need it; no shared memory precedes the array
    grid_dependency_wait();
    if (tid == 0) set_status(a.status, PKV_ERR_MISALIGNED);
    return;
  }
  if (warp == kTrQkWarp) {
    tmem_alloc(&ctl->tmem, kTrTmemCols);
    tmem_relinquish();
  } else if (warp == kTrTmaWarp && lane == 0) {
    prefetch_tensormap(&qmap);
    if constexpr (!kFp8) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
    }
  } else if (warp == 0 && lane == 0) {
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
      if (!kFp8) mbar_init(&ctl->v_fixed[kFp8 ? 0 : i], 1);
    }
    for (int i = 0; i < Dm::kRawAlloc; ++i) {
      mbar_init(&ctl->raw_k_full[i], 33);  // the copies' bytes, and each lane's scales
      mbar_init(&ctl->raw_v_full[i], 33);
      mbar_init(&ctl->raw_k_empty[i], Dm::kConvWarps);
      mbar_init(&ctl->raw_v_empty[i], Dm::kConvWarps);
    }
    for (int i = 0; i < Dm::kPieces; ++i) {
      mbar_init(&ctl->piece_full[i], 1);
      mbar_init(&ctl->piece_empty[i], Dm::kReaders);
    }
    mbar_init(&ctl->o_done, 1);
    mbar_init(&ctl->o_free, 8);
    mbar_init(&ctl->drain, 2);
    mbar_init(&ctl->pv_done[0], 1);
    mbar_init(&ctl->pv_done[1], 1);
    ctl->fail = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  grid_dependency_wait();
  allow_dependents();

  // A role walks the pieces that the loading warp publishes: piece pi in entry pi % kPieces, until one with k1 = 0.
  auto piece_at = [&](uint32_t pi) -> const TrPiece* {
    if (!tr_wait(&ctl->piece_full[pi % Dm::kPieces], pi / Dm::kPieces, ctl, a.status)) return nullptr;
    const TrPiece* pc = &ctl->piece[pi % Dm::kPieces];
    return *reinterpret_cast<const volatile int*>(&pc->k1) == 0 ? nullptr : pc;
  };
  auto piece_done = [&](uint32_t pi) {
    __syncwarp();
    if (lane == 0) mbar_arrive_cta(&ctl->piece_empty[pi % Dm::kPieces]);
  };

  if (warp == kTrTmaWarp) {
    if constexpr (kFp8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Dm::kRegsOther));
    // ---------------------------------------------------------------- schedule and loads
    // (this is on the way to the first load: few divisions, some 130 cycles each, and the lengths are read once)
    // lane i holds request 32 blk + i
    int blk = -1, lane_P = 0, lane_T = 0, lane_q0 = 0;
    auto load_block = [&](int b) {
      if (b == blk) return;
      blk = b;
      lane_T = 0;
      if (32 * b + lane < a.num_seqs) tr_request(a, 32 * b + lane, lane_P, lane_T, lane_q0);
    };
    // all units, cut or whole, the largest item
    uint32_t units = 0, items = 0, largest = 0;
    for (int b = (a.num_seqs - 1) / 32; b >= 0; --b) {  // (the first block last: the search below begins there)
      load_block(b);
      if (lane_T > 0) {
        const uint32_t cost = tr_cost(lane_P, lane_T, false), mine = a.hkv * tr_node_tiles(a, lane_T);
        items += mine;
        units += mine * cost;
        largest = max(largest, cost);
      }
    }
    units = __reduce_add_sync(0xffffffffu, units);
    items = __reduce_add_sync(0xffffffffu, items);
    largest = __reduce_max_sync(0xffffffffu, largest);
    // whole items where all are small, or where the CTAs' largest number of them is as good a balance as shares would be
    // (within a quarter; every CTA computes the same floats): 16 requests of 4000 tokens 46.9 us, in shares 51.1; 36 of 3000
    // 73.5 and 77.3; 16 of 1500 24.1 and 26.0 (a bound of a tenth leaves the first and the last in shares, one of a half changes
    // nothing)
    const float rounds = ceilf(static_cast<float>(items) / static_cast<float>(a.ctas));
    const float longest = static_cast<float>(largest) * rounds * static_cast<float>(a.ctas);
    const bool whole = largest <= kSmallItem || 4.f * longest <= 5.f * static_cast<float>(units);
    if (whole) units = items;
    // CTA c's share: units / ctas of them, one more for the first units % ctas
    const uint32_t ctas = min(units, static_cast<uint32_t>(a.ctas)), me = blockIdx.x;
    const uint32_t quota = ctas > 0 ? units / ctas : 0, more = units - quota * ctas;
    uint32_t f = me < ctas ? me * quota + min(me, more) : 0;
    const uint32_t hi = me < ctas ? f + quota + (me < more ? 1 : 0) : 0;
    auto cta_of = [&](uint32_t u) {  // the CTA whose share has unit u
      const uint32_t split = more * (quota + 1);
      return static_cast<int>(u < split ? u / (quota + 1) : more + (u - split) / quota);
    };
    // the request that unit f lies in, and the units before it
    int n = 0;
    uint32_t base = 0;
    for (int b = 0; f < hi && 32 * b < a.num_seqs; ++b) {
      load_block(b);
      const uint32_t u = lane_T > 0 ? a.hkv * tr_node_tiles(a, lane_T) * tr_cost(lane_P, lane_T, whole) : 0;
      uint32_t x = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + x > f);
      if (hit != 0) {
        const int src = __ffs(hit) - 1;
        n = 32 * b + src;
        base += __shfl_sync(0xffffffffu, x - u, src);
        break;
      }
      base += __shfl_sync(0xffffffffu, x, 31);
    }
    constexpr uint32_t kRing = kFp8 ? Dm::kRawAlloc : Dm::kSlots;  // tiles that the loads may be ahead
    // This lane's page of a tile of K or of V (kv = 1), < 0: none; eight lanes have a tile's. `full` completes with them.
    // (One copy a page: a copy costs the TMA unit 27 ns and 13.5 ns a KiB, so that boxes of 2 KiB held it to 1.5 us for a
    // tile of K and V, no faster than the memory; scales, 16 bytes a page, go by the load units instead.)
    auto load = [&](int kv, uint32_t i, long long tile) {
      const uint32_t st = i % kRing, use = i / kRing;
      uint64_t* full = kFp8 ? (kv ? &ctl->raw_v_full[kFp8 ? st : 0] : &ctl->raw_k_full[kFp8 ? st : 0])
                            : (kv ? &ctl->v_full[kFp8 ? 0 : st] : &ctl->k_full[kFp8 ? 0 : st]);
      uint64_t* empty = kFp8 ? (kv ? &ctl->raw_v_empty[kFp8 ? st : 0] : &ctl->raw_k_empty[kFp8 ? st : 0])
                             : (kv ? &ctl->v_empty[kFp8 ? 0 : st] : &ctl->k_empty[kFp8 ? 0 : st]);
      const uint32_t pages = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, tile >= 0)));
      if (use > 0 && !tr_wait(empty, use - 1, ctl, a.status)) return false;
      if (lane == 0) mbar_arrive_expect_tx(full, pages * static_cast<uint32_t>(kFp8 ? kPageSize * D : Dm::kPage));
      __syncwarp();
      if constexpr (kFp8) {
        if (tile >= 0) {
          bulk_load(smem + (kv ? Dm::kOffRawV : Dm::kOffRawK) + st * Dm::kRawTile + lane * (kPageSize * D),
                    (kv ? a.v_raw : a.k_raw) + tile * (kPageSize * D), kPageSize * D, full);
          cp_async16(smem_u32(smem + Dm::kOffScales + (st * 2 + kv) * kTrKeys + lane * kPageSize),
                     a.scales + tile * kScaleBytes + kv * kPageSize);
        }
        // (every lane: its arrival comes when its own copies have landed)
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full)) : "memory");
      } else if (tile >= 0) {
        tma_load_5d(smem + (kv ? Dm::kOffV : Dm::kOffK) + st * Dm::kTile + lane * Dm::kPage, kv ? &vmap : &kmap,
                    static_cast<int>(tile), full);
      }
      __syncwarp();
      return true;
    };
    uint32_t g = 0, pi = 0;
    bool run = true;
    TrCut cut = {0, 0, 0, 0};
    while (run && f < hi) {
      int P = 0, T = 0, q0 = 0;
      uint32_t cost = 1, rts = 1;
      for (; n < a.num_seqs; ++n) {  // requests without nodes are passed over
        load_block(n / 32);
        P = __shfl_sync(0xffffffffu, lane_P, n % 32);
        T = __shfl_sync(0xffffffffu, lane_T, n % 32);
        q0 = __shfl_sync(0xffffffffu, lane_q0, n % 32);
        rts = tr_node_tiles(a, T);
        cost = tr_cost(P, T, whole);
        const uint32_t u = a.hkv * rts * cost;
        if (f - base < u) break;
        base += u;
      }
      if (n >= a.num_seqs) break;  // (lengths that changed under the call)
      const uint32_t item = whole ? f - base : (f - base) / cost, p0 = f - base - item * cost, p1 = min(p0 + (hi - f), cost);
      const int nt = static_cast<int>(tr_key_tiles(P, T));
      f += p1 - p0;
      const int k0 = whole ? 0 : static_cast<int>(p0 > kItemCost ? p0 - kItemCost : 0);
      const int k1 = whole ? nt : static_cast<int>(p1 > kItemCost ? p1 - kItemCost : 0);
      if (k1 <= k0) continue;  // a share's end inside an item's fixed units
      const int n_pages = (P + T + kPageSize - 1) / kPageSize;
      const int* row = a.block_table + static_cast<size_t>(n) * a.max_pages;
      // this lane's page of the first tile; then of each next tile while the one before waits for its place
      int id_next = lane < kTrTilePages && k0 * kTrTilePages + lane < n_pages ? __ldg(row + k0 * kTrTilePages + lane) : 0;
      const int h = static_cast<int>(rts == 1 ? item : item / rts), rt = static_cast<int>(item - h * rts);
      const int node0 = rt * a.tile_nodes, nodes = min(a.tile_nodes, T - node0);
      const uint32_t qb = pi % a.q_bufs, quse = pi / a.q_bufs;
      if (quse > 0 && !tr_wait(&ctl->q_empty[qb], quse - 1, ctl, a.status)) break;
      const uint32_t e = pi % Dm::kPieces;
      if (pi >= Dm::kPieces && !tr_wait(&ctl->piece_empty[e], pi / Dm::kPieces - 1, ctl, a.status)) break;
      if (lane == 0) {
        unsigned char* dst = smem + Dm::kOffQ + qb * Dm::kHalves * a.q_rows * 128;
        mbar_arrive_expect_tx(&ctl->q_full[qb], static_cast<uint32_t>(Dm::kHalves * a.box_rows * 128));
#pragma unroll
        for (int half = 0; half < Dm::kHalves; ++half)
          tma_load_3d(dst + half * a.q_rows * 128, &qmap, 64 * half, h * a.grp, q0 + node0, &ctl->q_full[qb]);
        TrPiece& pc = ctl->piece[e];
        pc.k0 = k0;
        pc.k1 = k1;
        pc.P = P;
        pc.T = T;
        pc.row0 = q0 + node0;
        pc.node0 = node0;
        pc.rows = nodes * a.grp;
        pc.h = h;
        pc.n = n;
        pc.bad = 0;
        pc.slot = k0 == 0 ? (k1 == nt ? -1 : 1) : 0;
        mbar_arrive_cta(&ctl->piece_full[e]);
      }
      __syncwarp();
      for (int k = k0; k < k1; ++k, ++g) {
        const int pg = k * kTrTilePages + lane, id = id_next;
        if (k + 1 < k1 && lane < kTrTilePages && pg + kTrTilePages < n_pages) id_next = __ldg(row + pg + kTrTilePages);
        bool valid = lane < kTrTilePages && pg < n_pages;
        if (valid && (id < 0 || id >= a.num_pages)) {
          set_status(a.status, PKV_ERR_OUT_OF_BOUNDS);
          valid = false;
        }
        const long long tile = valid ? static_cast<long long>(id) * a.hkv + h : -1;
        if (!(run = load(0, g, tile) && load(1, g, tile))) break;
      }
      if (k0 == 0 && k1 < nt)  // the item goes on in later CTAs, to the one that has its last unit
        cut = {nodes * a.grp, q0 + node0, h, me | static_cast<uint32_t>(cta_of(base + (item + 1) * cost - 1)) << 16};
      if (a.by_item && k0 == 0 && lane == 0)
        a.cuts[(n * a.hkv + h) * a.node_tiles + rt] = k1 < nt ? cut : TrCut{0, 0, 0, 0};
      ++pi;
    }
    if (lane == 0 && a.by_item == 0) a.cuts[me] = cut;
    if (lane == 0 && static_cast<int>(me) < a.by_item) {  // an item that there could be and is not
      int P, T, q0;
      tr_request(a, static_cast<int>(me) / (a.hkv * a.node_tiles), P, T, q0);
      if (me % a.node_tiles >= tr_node_tiles(a, T)) a.cuts[me].rows = 0;
    }
    const uint32_t e = pi % Dm::kPieces;
    if (pi < Dm::kPieces || tr_wait(&ctl->piece_empty[e], pi / Dm::kPieces - 1, ctl, a.status)) {
      if (lane == 0) {
        ctl->piece[e].k1 = 0;
        mbar_arrive_cta(&ctl->piece_full[e]);
      }
    }
    __syncwarp();
    if (*reinterpret_cast<volatile int*>(&ctl->fail) != 0) {
      // the CTA gave up: its copies in flight land before it ends (a wait for one that was never issued runs out)
      for (uint32_t i = g > kRing ? g - kRing : 0; i <= g; ++i) {
        const uint32_t st = i % kRing;
        uint64_t* kf = kFp8 ? &ctl->raw_k_full[kFp8 ? st : 0] : &ctl->k_full[kFp8 ? 0 : st];
        uint64_t* vf = kFp8 ? &ctl->raw_v_full[kFp8 ? st : 0] : &ctl->v_full[kFp8 ? 0 : st];
        mbar_wait_bounded(kf, (i / kRing) & 1u, kDrainCycles);
        mbar_wait_bounded(vf, (i / kRing) & 1u, kDrainCycles);
      }
      for (uint32_t i = pi > 1 ? pi - 1 : 0; i <= pi; ++i)
        mbar_wait_bounded(&ctl->q_full[i % a.q_bufs], (i / a.q_bufs) & 1u, kDrainCycles);
    }
  } else if (warp == kTrQkWarp) {
    if constexpr (kFp8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Dm::kRegsOther));
    // ---------------------------------------------------------------- S = Q K^T
    const uint64_t q_desc = sdesc_sw128(smem_u32(smem + Dm::kOffQ), 16, 1024);
    const uint64_t k_desc = sdesc_sw128(smem_u32(smem + Dm::kOffK), 16, 8 * D * 2);
    const uint32_t q_half = (a.q_rows * 128) >> 4;
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t pi = 0; ok; ++pi) {
      const TrPiece* pc = piece_at(pi);
      if (pc == nullptr) break;
      const int tiles = pc->k1 - pc->k0;
      piece_done(pi);
      const uint32_t qb = pi % a.q_bufs;
      if (!(ok = tr_wait(&ctl->q_full[qb], pi / a.q_bufs, ctl, a.status))) break;
      const uint64_t qa = q_desc + ((qb * Dm::kHalves * a.q_rows * 128) >> 4);
      for (int k = 0; k < tiles; ++k, ++g) {
        const uint32_t st = g % Dm::kSlots, w = g & 1u;
        // S and P share their columns: the values of the group's tile before are done
        if (g >= 2 && !(ok = tr_wait(&ctl->pv_done[w], (g >> 1) - 1, ctl, a.status))) break;
        if (!(ok = tr_wait(&ctl->k_full[st], g / Dm::kSlots, ctl, a.status))) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t kb = k_desc + ((st * Dm::kTile) >> 4);
#pragma unroll
          for (int half = 0; half < Dm::kHalves; ++half)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_ss(tmem + kTrColS + 128 * w, qa + half * q_half + 2 * i, kb + half * (1024 >> 4) + 2 * i, a.idesc_qk,
                     half + i > 0 ? 1u : 0u);
          mma_commit(&ctl->s_full[w]);
          mma_commit(&ctl->k_empty[st]);
          if (k == tiles - 1) mma_commit(&ctl->q_empty[qb]);
        }
        __syncwarp();
      }
    }
    if (*reinterpret_cast<volatile int*>(&ctl->fail) != 0) {
      if (lane == 0) {
        mma_commit(&ctl->drain);
        mbar_wait_bounded(&ctl->drain, 0, kDrainCycles);
      }
      __syncwarp();
    }
  } else if (warp == kTrPvWarp) {
    if constexpr (kFp8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Dm::kRegsOther));
    // ---------------------------------------------------------------- O += P V
    const uint64_t v_desc = sdesc_sw128(smem_u32(smem + Dm::kOffV), 1024, 8 * D * 2);
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t pi = 0; ok; ++pi) {
      const TrPiece* pc = piece_at(pi);
      if (pc == nullptr) break;
      const int tiles = pc->k1 - pc->k0;
      piece_done(pi);
      if (pi > 0 && !(ok = tr_wait(&ctl->o_free, pi - 1, ctl, a.status))) break;
      for (int k = 0; k < tiles; ++k, ++g) {
        const uint32_t st = g % Dm::kSlots, w = g & 1u;
        if (!(ok = tr_wait(&ctl->v_full[st], g / Dm::kSlots, ctl, a.status))) break;
        if (!kFp8 && !(ok = tr_wait(&ctl->v_fixed[kFp8 ? 0 : st], g / Dm::kSlots, ctl, a.status))) break;
        if (!(ok = tr_wait(&ctl->p_full[w], g >> 1, ctl, a.status))) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t vb = v_desc + ((st * Dm::kTile) >> 4);
#pragma unroll
          for (int i = 0; i < kTrTilePages; ++i)
            mma_ts(tmem + kTrColO + 128 * w, tmem + kTrColS + 128 * w + 8 * i, vb + ((i * Dm::kPage) >> 4), Dm::kIdescPV,
                   (k >= 2 || i > 0) ? 1u : 0u);
          mma_commit(&ctl->pv_done[w]);
          mma_commit(&ctl->v_empty[st]);
          if (k == tiles - 1) mma_commit(&ctl->o_done);
        }
        __syncwarp();
      }
    }
    if (*reinterpret_cast<volatile int*>(&ctl->fail) != 0) {  // the CTA gave up: the products in flight end first
      if (lane == 0) {
        mma_commit(&ctl->drain);
        mbar_wait_bounded(&ctl->drain, 0, kDrainCycles);
      }
      __syncwarp();
    }
  } else if (warp < 8) {
    if constexpr (kFp8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Dm::kRegsSoftmax));
    // ---------------------------------------------------------------- softmax and epilogue
    const int w = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const int own_node = r / a.grp, own_head = r - own_node * a.grp;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lanes + kTrColS + 128 * w, t_o = tmem + lanes + kTrColO;
    const uint32_t masked = __float_as_uint(-CUDART_INF_F);
    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
    uint32_t g = 0, pi = 0;
    for (;; ++pi) {
      const TrPiece* pc = piece_at(pi);
      // (a warp that gives up in this wait leaves alone: the others' next barrier wants to hear of it, so all agree here)
      if (!tr_group_all(1, pc != nullptr)) break;
      const int k0 = pc->k0, k1 = pc->k1, P = pc->P, row0 = pc->row0;
      const bool live = r < pc->rows, work = quarter * 32 < pc->rows;
      unsigned long long mask = 0;
      if (live) {
        const int node = pc->node0 + own_node, T = pc->T;
        mask = a.masks != nullptr ? __ldg(a.masks + row0 + own_node) : (2ull << node) - 1;
        mask &= T < 64 ? (1ull << T) - 1 : ~0ull;
      }
      float m = -CUDART_INF_F, l = 0.f;
      bool fresh = true, ok = true;  // fresh: this group's first tile of the piece
      const uint32_t g0 = g;
      for (int k = k0; k < k1; ++k, ++g) {
        if ((g & 1u) != static_cast<uint32_t>(w) || !ok) continue;
        if (!(ok = tr_wait(&ctl->s_full[w], g >> 1, ctl, a.status))) continue;
        if (work) {
          tc_fence_after();
          uint32_t x[2][32];  // half of the row's 128 scores
          if ((k + 1) * kTrKeys > P) {
            // nodes, or keys past the end, among the tile's: 128 bits of what the row sees
            const int sh = P - k * kTrKeys;  // keys of the prefix in this tile
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
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t vis = static_cast<uint32_t>((c < 2 ? v0 : v1) >> (32 * (c & 1)));
              tmem_ld32(t_s + 32 * c, x[0]);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(vis >> e & 1u)) x[0][e] = masked;
              tmem_st32(t_s + 32 * c, x[0]);
            }
            tmem_st_wait();
          }
          // the second half for its maximum, the first half, which then stays in registers; the weights of the first
          // half overwrite its own columns alone (loops: half the code in the instruction caches, 1 % in 8 bits)
          float mx = -CUDART_INF_F;
#pragma unroll 1
          for (int c = 1; c >= 0; --c) {
            tr_load64(t_s + 64 * c, x);
            mx = fmaxf(mx, tr_max64(x));
          }
          // the maximum moves, and O with it, only when it grows by more than 2^8 (weights up to 2^8 are fine)
          const float m_new = fmaxf(m, mx);
          const bool grow = m == -CUDART_INF_F ? m_new != -CUDART_INF_F : (m_new - m) * a.scale_log2 > 8.f;
          if (__any_sync(0xffffffffu, grow)) {
            const float alpha = !grow ? 1.f : m == -CUDART_INF_F ? 0.f : tr_weight(m - m_new, a.scale_log2);
            if (!fresh) {
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(t_o + 128 * w + 16 * c, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st16(t_o + 128 * w + 16 * c, o);
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
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            if (c > 0) tr_load64(t_s + 64, x);
            tr_exp64(t_s + 32 * c, x, sc2, nm2, l2);
          }
          l += l2.x + l2.y;
          tmem_st_wait();
          tc_fence_before();
        }
        fresh = false;
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&ctl->p_full[w]);
      }
      // ---- the two groups' halves of the row, and its output or record; each group takes half of the columns
      ctl->stat[w][0][r] = m;
      ctl->stat[w][1][r] = l;
      ok = ok && tr_wait(&ctl->o_done, pi, ctl, a.status);
      tc_fence_after();
      if (!tr_group_all(2, ok)) break;  // all eight warps go on, or none
      const float m0 = ctl->stat[0][0][r], l0 = ctl->stat[0][1][r], m1 = ctl->stat[1][0][r], l1 = ctl->stat[1][1][r];
      const float M = fmaxf(m0, m1);
      // (a half that saw nothing has sum 0, or NaN where every score was NaN)
      const float a0 = m0 == -CUDART_INF_F ? 0.f : tr_weight(m0 - M, a.scale_log2);
      const float a1 = m1 == -CUDART_INF_F ? 0.f : tr_weight(m1 - M, a.scale_log2);
      const float L = (m0 == -CUDART_INF_F ? l0 : l0 * a0) + (m1 == -CUDART_INF_F ? l1 : l1 * a1);
      const bool have0 = k1 - k0 > 1 || (g0 & 1u) == 0, have1 = k1 - k0 > 1 || (g0 & 1u) == 1;
      const int slot = pc->slot;
      unsigned long long bad = 0;  // nodes that this row sees whose value rows hold a NaN or an infinity
      if (k1 * kTrKeys > P) bad = mask & *reinterpret_cast<const volatile unsigned long long*>(&pc->bad);
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const int col0 = w * (D / 2);
      __nv_bfloat16* orow =
          a.out + (static_cast<size_t>(row0 + own_node) * a.hq + pc->h * a.grp + own_head) * D + col0;
      float4* rec = reinterpret_cast<float4*>(a.records + (static_cast<size_t>(blockIdx.x) * 2 + max(slot, 0)) * kTrRecFloats);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {  // 16 columns at a time (with 32, which spilled, batches took 3 us longer)
        float o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0.f;
        __syncwarp();
        if (work) {
          uint32_t x[16], y[16];
          const uint32_t at = t_o + col0 + 16 * c;
          tmem_ld16(at, x);
          tmem_ld16(at + 128, y);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) {  // (a group without a tile: what its columns hold is not a number of this piece)
            if (have0) o[e] = a0 * __uint_as_float(x[e]);
            if (have1) o[e] = fmaf(a1, __uint_as_float(y[e]), o[e]);
          }
        }
        if (bad != 0) {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] += tr_nonfinite<D, kFp8>(a, pc, bad, col0 + 16 * c + e);
        }
        if (live) {
          if (slot < 0) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint4 y;
              y.x = pack_bf16x2(o[8 * q] * inv, o[8 * q + 1] * inv);
              y.y = pack_bf16x2(o[8 * q + 2] * inv, o[8 * q + 3] * inv);
              y.z = pack_bf16x2(o[8 * q + 4] * inv, o[8 * q + 5] * inv);
              y.w = pack_bf16x2(o[8 * q + 6] * inv, o[8 * q + 7] * inv);
              reinterpret_cast<uint4*>(orow + 16 * c)[q] = y;
            }
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              rec[(col0 / 4 + 4 * c + q + 1) * kTrRows + r] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          }
        }
      }
      if (slot >= 0 && live && w == 0) rec[r] = make_float4(M, L, 0.f, 0.f);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&ctl->o_free);  // O is read: the next piece's products may overwrite it
      piece_done(pi);
    }
  } else if (warp == kTrMendWarp && !kFp8) {
    // ---------------------------------------------------------------- value tiles with nodes or an end in them
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t pi = 0; ok; ++pi) {
      const TrPiece* pc = piece_at(pi);
      if (pc == nullptr) break;
      const int k0 = pc->k0, k1 = pc->k1, P = pc->P, T = pc->T;
      unsigned long long bad = 0;
      for (int k = k0; k < k1 && ok; ++k, ++g) {
        const uint32_t st = g % Dm::kSlots;
        if (!(ok = tr_wait(&ctl->v_full[st], g / Dm::kSlots, ctl, a.status))) break;
        if ((k + 1) * kTrKeys > P) {
          const int len = P + T - k * kTrKeys;     // rows of the tile before the end
          const int t0 = max(P - k * kTrKeys, 0);  // its first row behind the prefix
          unsigned char* vt = smem + Dm::kOffV + st * Dm::kTile;
          constexpr int kChunks = D / 8;
          for (int i = t0 * kChunks + lane; i < kTrKeys * kChunks; i += 32) {
            const int t = i / kChunks;
            uint4* at = reinterpret_cast<uint4*>(vt + tr_off<D>(t, i % kChunks));
            if (t >= len) {
              *at = make_uint4(0, 0, 0, 0);
              continue;
            }
            const uint4 x = *at;
            if (nonfinite_bf16x2(x.x) || nonfinite_bf16x2(x.y) || nonfinite_bf16x2(x.z) || nonfinite_bf16x2(x.w)) {
              *at = make_uint4(finite_bf16x2(x.x), finite_bf16x2(x.y), finite_bf16x2(x.z), finite_bf16x2(x.w));
              bad |= 1ull << (k * kTrKeys + t - P);
            }
          }
          if (bad != 0) atomicOr(&ctl->piece[pi % Dm::kPieces].bad, bad);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_cta(&ctl->v_fixed[kFp8 ? 0 : st]);
      }
      piece_done(pi);
    }
  } else if (kFp8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Dm::kRegsOther));
    if (warp >= 12) {
      // ---------------------------------------------------------------- 8-bit tiles as bf16 tiles
      const int kv = (warp - 12) / Dm::kConvWarps;   // 0: K, 1: V
      const int sub = (warp - 12) % Dm::kConvWarps;  // this warp's rows: 32 sub ..
      uint64_t* full = kv ? ctl->v_full : ctl->k_full;
      uint64_t* empty = kv ? ctl->v_empty : ctl->k_empty;
      uint64_t* raw_full = kv ? ctl->raw_v_full : ctl->raw_k_full;
      uint64_t* raw_empty = kv ? ctl->raw_v_empty : ctl->raw_k_empty;
      // this lane's row and its places in the first 8 rows of the raw and of the expanded tile
      const int bit = D == 128 ? (lane >> 2) & 1 : 0;
      const int t0 = 32 * sub + (D == 128 ? (lane >> 3) * 2 + bit : lane >> 2);
      const int c0 = (lane & 3) + 4 * bit;
      const uint32_t src0 = t0 * D + c0 * 16, dst0 = tr_off<D>(t0, 2 * c0);
      uint32_t g = 0;
      bool ok = true;
      for (uint32_t pi = 0; ok; ++pi) {
        const TrPiece* pc = piece_at(pi);
        if (pc == nullptr) break;
        const int k0 = pc->k0, k1 = pc->k1, P = pc->P, T = pc->T;
        for (int k = k0; k < k1 && ok; ++k, ++g) {
          const uint32_t st = g % Dm::kSlots, use = g / Dm::kSlots, rs = g % Dm::kRawAlloc;
          if (!(ok = tr_wait(&raw_full[rs], g / Dm::kRawAlloc, ctl, a.status))) break;
          if (use > 0 && !(ok = tr_wait(&empty[st], use - 1, ctl, a.status))) break;
          const unsigned char* src = smem + (kv ? Dm::kOffRawV : Dm::kOffRawK) + rs * Dm::kRawTile;
          const unsigned char* sc = smem + Dm::kOffScales + (rs * 2 + kv) * kTrKeys;
          unsigned char* dst = smem + (kv ? Dm::kOffV : Dm::kOffK) + st * Dm::kTile;
          const bool tail = kv && (k + 1) * kTrKeys > P;
          const int len = P + T - k * kTrKeys;
          // 16 values a lane at a time. Of 8 lanes four take one half of a row, four the other half of the next, so
          // that the reads (128-byte rows) and the writes (swizzled) both hit every bank once. The expansion is bound
          // by its instructions: tiles with rows to mend take a loop of their own and addresses differ by constants
          // (16 requests 36.0 -> 32.0 us); two steps unrolled, as the roles share the SM's instruction caches (four
          // 35.3, eight 39.6).
          constexpr int kSteps = D / 16;
          auto expand = [&](auto mend) {
#pragma unroll 2
            for (int i = 0; i < kSteps; ++i) {
              const int rows8 = D == 128 ? i >> 1 : i;  // groups of 8 rows ahead
              const int odd = D == 128 ? i & 1 : 0;
              const uint4 x = *reinterpret_cast<const uint4*>(src + (src0 ^ odd << 6) + rows8 * (8 * D));
              const float s = __uint_as_float(static_cast<uint32_t>(sc[t0 + rows8 * 8]) << 23);
              const float2 s2 = make_float2(s, s);
              uint32_t y[8];
              const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t lo2, hi2;
                e4m3x4_to_f16x4(xs[q], lo2, hi2);
                const float2 u = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&lo2)), s2);
                const float2 v = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&hi2)), s2);
                y[2 * q] = pack_bf16x2(u.x, u.y);
                y[2 * q + 1] = pack_bf16x2(v.x, v.y);
              }
              if constexpr (decltype(mend)::value) {
                const int t = t0 + rows8 * 8;
                if (k * kTrKeys + t >= P) {
                  bool bad = false;
#pragma unroll
                  for (int q = 0; q < 8; ++q) {
                    if (t >= len) y[q] = 0u;
                    if (nonfinite_bf16x2(y[q])) {
                      bad = true;
                      y[q] = finite_bf16x2(y[q]);
                    }
                  }
                  if (bad) atomicOr(&ctl->piece[pi % Dm::kPieces].bad, 1ull << (k * kTrKeys + t - P));
                }
              }
              *reinterpret_cast<uint4*>(dst + (dst0 ^ odd << 10) + rows8 * (8 * D * 2)) = make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4*>(dst + (dst0 ^ (odd << 10 | 16)) + rows8 * (8 * D * 2)) = make_uint4(y[4], y[5], y[6], y[7]);
            }
          };
          if (tail)
            expand(std::true_type{});
          else
            expand(std::false_type{});
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_cta(&raw_empty[rs]);
            mbar_arrive_cta(&full[st]);
          }
        }
        piece_done(pi);
      }
    }
  }

  // ---------------------------------------------------------------- end
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kTrQkWarp) tmem_dealloc(tmem, kTrTmemCols);
}

// The records of cut items, joined: o = sum_c o_c 2^(m_c - M) / sum_c l_c 2^(m_c - M), each warp over every eighth
// record, then over the warps, in order: the same bits every time. CTA (i, part, quarter) takes 4 N columns and 32 rows (a
// thread to a row) of cut item i. N = 8 keeps the grid within one wave of CTAs for batches (152 x 4 for 32 rows); few items
// are spread over more CTAs with N = 2 (one request of 40k tokens 1.7 us less). A kernel of its own: joined by the last CTA
// of an item instead, the 20 records of a long request's item took that one SM 17 us; shared out between the item's CTAs
// by atomics, each of which takes 0.8 us, 5 us.
constexpr int kJoinWarps = 8;
template <int D, int N>
__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(const TrArgs a) {
  __shared__ float4 part_o[kJoinWarps][N][32];
  __shared__ float part_m[kJoinWarps][32], part_l[kJoinWarps][32];
  grid_dependency_wait();
  allow_dependents();
  const int q0 = blockIdx.y * N;
  const int4 cut = __ldcg(reinterpret_cast<const int4*>(a.cuts + blockIdx.x));
  const int rows = cut.x, row0 = cut.y, h = cut.z, c0 = cut.w & 0xffff, c1 = static_cast<uint32_t>(cut.w) >> 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.z * 32 + lane;
  if (static_cast<int>(blockIdx.z) * 32 >= rows) return;
  // (a call that gave up may leave another call's descriptors: nothing of them reaches past this call's buffers)
  if (rows > kTrRows || row0 < 0 || row0 + (rows + a.grp - 1) / a.grp > a.total || h < 0 || h >= a.hkv || c1 >= a.ctas) return;
  float M = -CUDART_INF_F, L = 0.f;
  float4 o[N];
#pragma unroll
  for (int q = 0; q < N; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll(N == 8 ? 1 : 3)
  for (int c = c0 + warp; c <= c1 && r < rows; c += kJoinWarps) {
    // the first piece is in slot 1 of its CTA, the others in slot 0 of theirs
    const float4* x =
        reinterpret_cast<const float4*>(a.records + (static_cast<size_t>(c) * 2 + (c == c0 ? 1 : 0)) * kTrRecFloats) + r;
    const float4 ml = __ldcg(x);
    float4 y[N];
#pragma unroll
    for (int q = 0; q < N; ++q) y[q] = __ldcg(x + (q0 + q + 1) * kTrRows);
    const float top = fmaxf(M, ml.x);
    const float old = M == -CUDART_INF_F ? 0.f : tr_weight(M - top, a.scale_log2);
    const float now = ml.x == -CUDART_INF_F ? 0.f : tr_weight(ml.x - top, a.scale_log2);
    L = (M == -CUDART_INF_F ? L : L * old) + (ml.x == -CUDART_INF_F ? ml.y : ml.y * now);
#pragma unroll
    for (int q = 0; q < N; ++q) {
      o[q].x = o[q].x * old + y[q].x * now;
      o[q].y = o[q].y * old + y[q].y * now;
      o[q].z = o[q].z * old + y[q].z * now;
      o[q].w = o[q].w * old + y[q].w * now;
    }
    M = top;
  }
#pragma unroll
  for (int q = 0; q < N; ++q) part_o[warp][q][lane] = o[q];
  part_m[warp][lane] = M;
  part_l[warp][lane] = L;
  __syncthreads();
  if (r >= rows || warp >= N) return;
  // thread (row, 4 columns): the warps' parts
  float top = -CUDART_INF_F, sum = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, part_m[w][lane]);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float m = part_m[w][lane], l = part_l[w][lane];
    const float now = m == -CUDART_INF_F ? 0.f : tr_weight(m - top, a.scale_log2);
    const float4 y = part_o[w][warp][lane];
    sum += m == -CUDART_INF_F ? l : l * now;
    s.x += y.x * now;
    s.y += y.y * now;
    s.z += y.z * now;
    s.w += y.w * now;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int node = r / a.grp;
  __nv_bfloat16* dst = a.out + (static_cast<size_t>(row0 + node) * a.hq + h * a.grp + r - node * a.grp) * D + 4 * (q0 + warp);
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(s.x * inv, s.y * inv), pack_bf16x2(s.z * inv, s.w * inv));
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

// The cut items' descriptors, one per CTA, in front of the records. Every call writes what it reads of both.
size_t cut_bytes(int num_sms) { return (static_cast<size_t>(num_sms) * sizeof(TrCut) + 255) / 256 * 256; }

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
  if (launch_pdl(tree_attn_kernel<D, kFp8>, dim3(static_cast<unsigned>(a.ctas)), dim3(TrDim<D, kFp8>::kThreads),
                 tr_smem_bytes<D, kFp8>(), stream, qmap, kmap, vmap, a) != cudaSuccess)
    return PKV_ERR_CUDA;
  // a table so narrow that no item can be cut needs no joining (a join that finds nothing to do takes 1.6 us)
  if (kItemCost + (static_cast<long long>(a.max_pages) + kTrTilePages - 1) / kTrTilePages <= kSmallItem) return PKV_OK;
  const unsigned items = static_cast<unsigned>(a.by_item > 0 ? a.by_item : a.ctas);
  const unsigned quarters = static_cast<unsigned>((a.box_rows + 31) / 32);
  const cudaError_t e =
      items * quarters * (D / 8) <= 4u * a.ctas
          ? launch_pdl(tree_join_kernel<D, 2>, dim3(items, D / 8, quarters), dim3(kJoinWarps * 32), 0, stream, a)
          : launch_pdl(tree_join_kernel<D, 8>, dim3(items, D / 32, quarters), dim3(kJoinWarps * 32), 0, stream, a);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

int tree_max_nodes() { return kTrMaxNodes; }
int tree_max_seqs() { return kTrMaxSeqs; }

size_t tree_workspace_bytes(int num_sms) { return PKV_STATUS_BYTES + cut_bytes(num_sms) + 2 * num_sms * kTrRecBytes; }

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
  a.cuts = reinterpret_cast<TrCut*>(ws + PKV_STATUS_BYTES);
  a.records = reinterpret_cast<float*>(ws + PKV_STATUS_BYTES + cut_bytes(num_sms));
  a.num_seqs = t.num_seqs;
  a.total = t.total_nodes;
  a.max_pages = t.max_pages;
  a.num_pages = num_pages;
  a.max_nodes = t.max_nodes;
  a.hq = num_q_heads;
  a.hkv = num_kv_heads;
  a.grp = num_q_heads / num_kv_heads;
  a.tile_nodes = kTrRows / a.grp;
  a.node_magic = static_cast<uint32_t>(((1ull << 32) + a.tile_nodes - 1) / a.tile_nodes);
  a.box_rows = a.grp * (t.max_nodes < a.tile_nodes ? t.max_nodes : a.tile_nodes);
  a.q_rows = (a.box_rows + 7) / 8 * 8;
  a.q_bufs = a.q_rows <= kTrRows / 2 ? 2 : 1;
  a.ctas = num_sms;
  a.node_tiles = (t.max_nodes + a.tile_nodes - 1) / a.tile_nodes;
  const long long items = static_cast<long long>(t.num_seqs) * num_kv_heads * a.node_tiles;
  a.by_item = items <= num_sms ? static_cast<int>(items) : 0;
  a.scale_log2 = fabsf(t.scale) * kLog2e;
  a.idesc_qk = idesc_bf16_f32(kTrRows, kTrKeys, false) | (t.scale < 0.f ? 1u << 13 : 0u);  // bit 13 negates A
  // a masked score, infinity, times 0 would be NaN; times this, differences of up to 2^128 have weights of 2^(-2^-21) (with
  // FLT_MIN scores of 2^119 and more were told apart)
  if (a.scale_log2 == 0.f) a.scale_log2 = FLT_TRUE_MIN;

  const cuuint64_t hd = static_cast<cuuint64_t>(head_dim);
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
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
  {
    // (dim of a half, row of 8, half, 8-row group, tile): a box is a page, laid out as tr_off says
    const long long tiles = static_cast<long long>(num_pages) * num_kv_heads;
    if (tiles > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;  // tile coordinates are 32-bit
    const cuuint32_t halves = static_cast<cuuint32_t>(head_dim / 64);
    const cuuint64_t dims[5] = {64, 8, halves, 2, static_cast<cuuint64_t>(tiles)};
    const cuuint64_t strides[4] = {hd * 2, 128, hd * 2 * 8, hd * 2 * kPageSize};
    const cuuint32_t box[5] = {64, 8, halves, 2, 1};
    const void* pools[2] = {t.k_pages, t.v_pages};
    CUtensorMap* maps[2] = {&kmap, &vmap};
    for (int i = 0; i < 2; ++i)
      if (enc(maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(pools[i]), dims, strides, box, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return PKV_ERR_CUDA;
  }
  return head_dim == 64 ? launch<64, false>(qmap, kmap, vmap, a, stream) : launch<128, false>(qmap, kmap, vmap, a, stream);
}

}  // namespace pkv
