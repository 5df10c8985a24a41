// Ragged attention over a paged cache: sequence b brings its own number n_b of
// query rows, the newest n_b of its seq_lens[b] cached tokens, packed row after
// row into one [T, Hq, d] tensor. Chunks of prompts, drafted tokens to verify
// and single decoded tokens share one launch.
//
//   O = softmax(scale * Q K^T + M) V per query head, with key j visible to the
//   query at position i iff j <= i, and with a window W and n_sink kept
//   positions iff also i - j < W or j < n_sink; every key without a mask. A
//   learned sink logit of the head adds exp(sink) to the softmax's sum.
//
// Rows. A K/V head's group of query heads shares its keys, so a tile's 128 rows
// are (token, head of the group) pairs, tpt = 128 / group tokens of them: one
// decoded token of 4 heads fills 4 rows, a chunk fills whole tiles, and K and V
// are read once for the whole group. An item is the two tiles (256 rows) of one
// (sequence, K/V head, stretch of 2 tpt tokens). It streams 128-key tiles.
//   wide item (more than tpt tokens): both tiles take every key tile;
//   narrow item: there is one tile of rows, and the two softmax teams take the
//   even and the odd key tiles with an accumulator each, joined at the end.
//
// Split. What the items cost is known only on the GPU and differs by four
// orders of magnitude within a batch, so the work is dealt by the tile: the
// items stand in one line, an item as long as its key tiles cost, and CTA c of
// G takes [W c / G, W (c + 1) / G) of the line's length W. Every CTA finds its
// stretch by scanning the batch for itself. An item cut by a boundary leaves
// partial outputs (fp32, unnormalised, with each row's maximum and sum), which
// a second, small grid joins in a fixed order: nothing depends on timing. A CTA
// has at most two partials, one per end, so the workspace does not depend on
// the batch. The line counts n_sink's tiles and one more for every item under a
// window, also where the window still reaches position 0: with sinks longer than some
// of the sequences the dealing gets uneven (a batch half of short sequences, window
// 128: the busiest CTA 14 % above the mean at n_sink = 200, 34 % at 1,000, else 4-9 %).
//
// What bounds it. Narrow items: HBM (64 KB of K and V a tile at d = 128, 1.45 us of
// an SM's share of HBM, against 0.55 us of MMAs); at d = 64 the chain scores ->
// softmax -> P V -> scores of the two teams. Wide items: that chain, the softmax's
// exponentials and the tensor cores in turn, as in the prefill kernel. Short items
// (a window of 128): the latency of an item's steps, 13,000 cycles for two tiles.
// Measured, in passes one after another for a second, at the power cap, and in runs of
// a few passes: 64 sequences of 1K-32K tokens with 1-8 rows each, 32 / 8 heads, d = 128
// 703 and 645 us (6,020 and 6,560 GB/s); one of 131,072 tokens 109 and 104 us (4,920
// and 5,180 GB/s); 4 chunks of 2,048 rows on 16,384 tokens 2,177 and 1,867 us (947 and
// 1,104 TFLOP/s); 4 chunks of 1K-2K rows beside 32 single rows 1,360 and 1,155 us; 48
// chunks of up to 512 rows and 16 single ones, window 128, 64 / 8 heads, d = 64 216 us.
//
// Roles, pipeline and the lazily moved maximum are those of the prefill kernel
// (prefill_sm100.cu): 8 softmax warps, an MMA warp, here two TMA warps (K and V),
// and a warp that works out the items ahead of their use. (An MMA warp for each
// team was slower: their products wait for one another in the tensor cores' queue,
// 4,400 cycles a wide tile instead of 3,450.) Probabilities go to the second
// product as bf16 (the tensor cores take nothing wider at this
// rate; at most 2^-8 of each p, averaged over the row), sums and outputs stay in fp32.

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kBM = 128;  // query rows per tile (= TMEM lanes)
constexpr int kBN = 128;  // keys per tile

// Instruction descriptor for kind::f16: fp32 accumulate, bf16 A and B, A
// K-major, B K-major (0) or MN-major (1), N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(b_mn_major) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void raise_abort(volatile int* abort_flag, int32_t* status) {
  *abort_flag = 1;
  if (status != nullptr) atomicOr(status, ATTN_STATUS_BIT_TIMEOUT);
}

// Warp-collective forms: every lane of a converged warp executes them and the
// lane that elect.sync picks issues four steps at a time. A branch on one lane
// leaves the compiler to find the lane for every instruction: a step then took
// about 100 cycles to issue, more than it takes to run at d = 64.
// d (+)= A B over four steps of 16 along the head dimension, operands from their bases.
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ss4_w(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred e, p, t;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
      " setp.ne.b32 p, %3, 0;\n setp.eq.b32 t, 0, 0;\n"
      " add.s64 a1, %1, 2;\n add.s64 a2, %1, 4;\n add.s64 a3, %1, 6;\n"
      " add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
      " elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %4, t;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(accumulate), "n"(IDESC)
      : "memory");
}
// The same with A in TMEM, 8 columns a step, and B 2 KB a step (16 keys of V).
template <uint32_t IDESC>
__device__ __forceinline__ void mma_ts4_w(uint32_t d_tmem, uint32_t a, uint64_t b, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred e, p, t;\n .reg .b32 a1, a2, a3;\n .reg .b64 b1, b2, b3;\n"
      " setp.ne.b32 p, %3, 0;\n setp.eq.b32 t, 0, 0;\n"
      " add.u32 a1, %1, 8;\n add.u32 a2, %1, 16;\n add.u32 a3, %1, 24;\n"
      " add.s64 b1, %2, 128;\n add.s64 b2, %2, 256;\n add.s64 b3, %2, 384;\n"
      " elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %4, t;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %4, t;\n}\n" ::"r"(d_tmem),
      "r"(a), "l"(b), "r"(accumulate), "n"(IDESC)
      : "memory");
}
template <int D>
__device__ __forceinline__ void mma_scores_w(uint32_t d_tmem, uint64_t dq, uint64_t dk) {
  mma_ss4_w<idesc_bf16(kBM, kBN, 0)>(d_tmem, dq, dk, 0u);
  if constexpr (D == 128) mma_ss4_w<idesc_bf16(kBM, kBN, 0)>(d_tmem, dq + 1024, dk + 1024, 1u);
}
// Half of one P V: keys 0-63 (half 0) or 64-127 of a tile.
template <int D>
__device__ __forceinline__ void mma_pv_w(uint32_t d_tmem, uint32_t p_tmem, uint64_t dv, int half, bool first) {
  mma_ts4_w<idesc_bf16(kBM, D, 1)>(d_tmem, p_tmem + 32u * half, dv + 512ull * half, first && half == 0 ? 0u : 1u);
}

// Multiply this thread's TMEM output row by f (warp-collective).
template <int D>
__device__ __forceinline__ void rescale_row_t(uint32_t colO, float f) {
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    uint32_t ov[16];
    tmem_ld_32x32b_x16(colO + c * 16, ov);
    tc_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
    tmem_st_32x32b_x16(colO + c * 16, ov);
  }
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The paged pool [num_blocks][block_size][Hkv][d] bf16 as a rank-4 tensor
// (d, Hkv, slot, block); box = 64 columns x 1 head x box_slots slots x 1
// block, 128-byte swizzle: box_slots = block_size loads one block of one head,
// box_slots = 1 one token row.
bool encode_pool(CUtensorMap* map, const void* base, int d, int hkv, int block_size, int num_blocks,
                 int box_slots) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(hkv),
                              static_cast<cuuint64_t>(block_size), static_cast<cuuint64_t>(num_blocks)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(hkv) * d * 2,
                                 static_cast<cuuint64_t>(block_size) * hkv * d * 2};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(box_slots), 1};
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
                         estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

constexpr int kVlThreads = 384;
constexpr int kVlWarps = kVlThreads / 32;
constexpr int kVlTmaWarp = 8;
constexpr int kVlMmaWarp = 9;
constexpr int kVlPlanWarp = 10;
constexpr int kVlTmaVWarp = 11;
constexpr int kVlRows = 2 * kBM;  // rows of an item
// the register split of the prefill kernel: 256 x 224 + 128 x 56 = 384 x 168
constexpr uint32_t kVlRegsSoftmax = 224;
constexpr uint32_t kVlRegsControl = 56;
static_assert(256 * kVlRegsSoftmax + 128 * kVlRegsControl == kVlThreads * 168, "register split");
constexpr float kVlRescale = 8.0f;  // base 2: the maximum moves only past this (p <= 2^8)
// What a key costs on the line, and what an item costs besides, in proportion to
// the cycles measured (a fit over the SMs of batches of each kind): a wide tile of
// 128 keys 3,400, a narrow one 1,900 (d = 128) and 1,400 (d = 64) beside wide ones,
// an item's ends 8,000-13,000. (With 4,800 and 8,200 for a wide and a narrow item's
// ends the busiest SM of 64 short chunks and 64 short decodes had 25 % more than the
// mean: 309 us, so 293.)
constexpr int kCostWide = 20, kCostItem = 60 * kBN, kCostItemNarrow = 74 * kBN;
template <int D>
constexpr int kCostNarrow = D == 128 ? 11 : 8;
// A CTA's stretch holds a tile at least (a piece of every item it passes through).
constexpr int kMinStretch = kCostWide * kBN;

template <int D>
struct VlCfg {
  static constexpr int kHalf = 128 * 128;  // bytes of one 64-column box of 128 rows
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * kHalf;
  static constexpr int kStages = (D == 128) ? 2 : 4;  // K ring and V ring, each
  // A narrow item's V ring has one slot more, in the place of the second Q tile:
  // a V tile waits for its softmax, 1 us after its K tile was used.
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + 2 * kTile;
  static constexpr int kVOff = kKOff + kStages * kTile;
  static constexpr int kStageOff = kVOff + kStages * kTile;  // 4 KB per softmax warp
  static constexpr int kBarOff = kStageOff + 8 * 4096;
  static constexpr int kBytes = kBarOff + 384;
  static constexpr int kAlloc = kBytes + 1024;  // slack to align the base to 1024 bytes
  static_assert(kAlloc <= 232448 - 1024, "shared memory per CTA (under 1 KB is static)");
  // TMEM columns: scores of both teams (128 each; the probabilities overwrite the
  // first 64), then outputs. (At d = 64 there is room for the probabilities beside
  // the scores, so that a team's next scores need not wait for P V; measured, the
  // wide tile stayed at 3,300 cycles and the narrow one at 1,900.)
  __host__ __device__ static constexpr uint32_t col_s(int x) { return x ? 128u : 0u; }
  __host__ __device__ static constexpr uint32_t col_o(int x) { return 256u + static_cast<uint32_t>(x * D); }
};

enum : int {
  kVbQFull = 0,
  kVbKFull = 1,    // + stage (up to 4)
  kVbVFull = 5,    // + slot (up to 5)
  kVbKEmpty = 10,  // + stage
  kVbVEmpty = 14,  // + slot
  kVbSFull = 19,   // + team
  kVbPLo = 21,     // + team: probabilities of keys 0-63 written
  kVbPHi = 23,     // + team: probabilities of keys 64-127 written
  kVbOFinal = 25,  // + team
  kVbDrain = 27,
  // + item (mod 2): the V warp may look for an item's phase when the next item's is
  // over too, and the parity of one barrier's phases would not tell them apart
  kVbQEmpty = 28,
  kVbPiece = 30,      // + entry of the piece ring (4)
  kVbPieceDone = 34,  // + entry
  kVbPair = 38,       // + pair of warps that join rows (4, and 2 where team 1 is shifted)
};
constexpr int kVbTmemSlot = 352, kVbAbort = 356;  // bytes behind the barriers
constexpr int kPieces = 4;                        // pieces worked out ahead

// An item whose first piece is CTA c's last: what the joining grid needs of it.
struct VarlenSplit {
  int pieces;  // 0: CTA c's stretch ends with a whole item
  int row0, ntok, head0, nheads, wide, pad0, pad1;
};

struct VarlenParams {
  __nv_bfloat16* o;
  float* lse;
  int32_t* status;
  const float* sinks;
  const int32_t* block_table;
  const int32_t* cu_q;
  const int32_t* seq_lens;
  float4* part_o;      // [2 G][d / 4][256]
  float2* part_ml;     // [2 G][256]
  VarlenSplit* splits;  // [G]
  int B, T, Hq, group, gsz, hchunks, tpt, units;  // gsz heads a tile, hchunks tiles a group, units = Hkv * hchunks
  int tph;             // tokens of 64 rows
  int tma_out;         // a warp's 32 rows are whole tokens: they leave as one box
  int row_magic;       // ceil(2^16 / gsz): row * magic >> 16 = row / gsz for rows below 128
  int mask_kind, window, n_sink, max_blocks, block_size, num_blocks, max_seq_len;
  float scale_log2;
  long long budget;
};

// A sequence's rows and context. bad: lengths that do not fit; it has no items.
struct VlSeq {
  int row0, n, nk;
  bool bad;
};
__device__ __forceinline__ VlSeq seq_at(const VarlenParams& p, int b) {
  const int r0 = __ldg(p.cu_q + b), r1 = __ldg(p.cu_q + b + 1), nk = __ldg(p.seq_lens + b);
  const bool order = r0 >= 0 && r0 <= r1 && r1 <= p.T;
  const bool bad = !order || (r1 > r0 && (nk < r1 - r0 || nk > p.max_seq_len));
  return VlSeq{r0, bad ? 0 : r1 - r0, nk, bad};
}

// One stretch of rows of a sequence: its tokens, the keys some row sees (the
// sink positions [0, sink_end) and [key_lo, key_end)), and the T key tiles that
// hold them: nst tiles from position 0, the others from `base` on, the block
// with key_lo (a tile may start at any block).
struct VlGeom {
  int tok0, ntok, pos_lo, key_lo, key_end, sink_end, nst, base, T;
  bool wide;
  __device__ __forceinline__ int tile_key(int j) const { return j < nst ? j * kBN : base + (j - nst) * kBN; }
};
__device__ __forceinline__ VlGeom geom_at(const VarlenParams& p, int n, int nk, int rt) {
  VlGeom g;
  g.tok0 = rt * 2 * p.tpt;
  g.ntok = min(n - g.tok0, 2 * p.tpt);
  g.wide = g.ntok > p.tpt;
  g.pos_lo = nk - n + g.tok0;
  g.key_end = p.mask_kind == ATTN_MASK_FULL ? nk : g.pos_lo + g.ntok;
  g.key_lo = p.mask_kind == ATTN_MASK_SLIDING_WINDOW ? max(0, g.pos_lo - p.window + 1) : 0;
  g.sink_end = min(p.n_sink, g.key_lo);
  g.nst = (g.sink_end + kBN - 1) / kBN;
  g.base = max(g.key_lo & ~(p.block_size - 1), g.nst * kBN);
  g.T = g.nst + max(0, (g.key_end - g.base + kBN - 1) / kBN);
  return g;
}
__device__ __forceinline__ int row_tiles(const VarlenParams& p, int n) { return (n + 2 * p.tpt - 1) / (2 * p.tpt); }

// Length on the line of the first R row tiles of a sequence of one K/V head, in
// closed form: kCostItem an item, and its keys (with a window at most so many:
// whole blocks and tiles of sinks; every key tile must start inside its item's
// length). All R tiles are wide but a sequence's last.
template <int D>
__device__ __forceinline__ long long line_of(const VarlenParams& p, int n, int nk, int R) {
  const int nrt = row_tiles(p, n), S = 2 * p.tpt;
  const long long pos0 = nk - n;
  const bool last = R == nrt;  // the last one may be shorter, and narrow
  const long long F = last ? R - 1 : R;
  const int tail = n - (nrt - 1) * S;
  long long keys, tail_keys;
  if (p.mask_kind == ATTN_MASK_FULL) {
    keys = F * nk;
    tail_keys = nk;
  } else if (p.mask_kind == ATTN_MASK_CAUSAL) {
    keys = F * pos0 + S * (F * (F + 1) / 2);
    tail_keys = nk;
  } else {
    const int W = p.window, extra = ((p.n_sink + kBN - 1) / kBN) * kBN + kBN;
    // the first F0 row tiles start at a position that sees position 0
    const int reach = W - 1 - static_cast<int>(pos0);
    const long long F0 = reach < 0 ? 0 : min(static_cast<long long>(reach / S + 1), F);
    keys = F0 * pos0 + S * (F0 * (F0 + 1) / 2) + (F - F0) * (S + W - 1) + F * extra;
    tail_keys = min(nk, tail + W - 1) + extra;
  }
  long long c = F * static_cast<long long>(kCostItem) + keys * kCostWide;
  if (last) c += tail > p.tpt ? kCostItem + tail_keys * kCostWide : kCostItemNarrow + tail_keys * kCostNarrow<D>;
  return c;
}

// CTA c's stretch of the line and where it starts in the batch.
struct VlPlan {
  long long start, end, total;
  int G;
  int b, u, rt;      // the item that holds `start`
  long long s;       // where that item starts
};

// A place in the CTA's stretch.
struct VlWalk {
  int b, u, rt, nrt;
  long long s;
  VlSeq sq;
};
// A piece of an item: key tiles [j0, j0 + nt) of its list, nt = 0 behind the last piece.
struct VlPiece {
  VlGeom g;
  int j0, nt, b, nk, row0, kvh, head0, nheads;
  bool half;   // a narrow item of at most 64 rows: team 1 has them in its lanes 64 and up
  bool whole;
  int slot;    // of its partial output
  int pieces;  // of the item, when this is the first of several
};
// The first tile that starts at or after `x` (keys' cost from the item's first tile).
template <int D>
__device__ __forceinline__ int tile_from(long long x, const VlGeom& g) {
  constexpr unsigned long long kWide = kCostWide * kBN, kNarrow = kCostNarrow<D> * kBN;
  if (x <= 0) return 0;
  const unsigned long long v = x, t = g.wide ? (v + kWide - 1) / kWide : (v + kNarrow - 1) / kNarrow;
  return t < static_cast<unsigned long long>(g.T) ? static_cast<int>(t) : g.T;
}
// The next piece of the stretch that has any key tile; nt = 0 at its end.
template <int D>
__device__ __forceinline__ void next_piece(const VarlenParams& p, const VlPlan& pl, int cta, VlWalk& w, VlPiece& out) {
  while (w.s < pl.end) {
    const VlGeom g = geom_at(p, w.sq.n, w.sq.nk, w.rt);
    const long long x0 = w.s + (g.wide ? kCostItem : kCostItemNarrow);  // where the item's first tile stands
    const int j0 = tile_from<D>(pl.start - x0, g), j1 = tile_from<D>(pl.end - x0, g);
    const int kvh = w.u / p.hchunks, hc = w.u - kvh * p.hchunks;
    out.g = g;
    out.j0 = j0;
    out.nt = j1 - j0;
    out.half = g.ntok <= p.tph;
    out.b = w.b;
    out.nk = w.sq.nk;
    out.row0 = w.sq.row0 + g.tok0;
    out.kvh = kvh;
    out.head0 = kvh * p.group + hc * p.gsz;
    out.nheads = min(p.gsz, p.group - hc * p.gsz);
    out.whole = j0 == 0 && j1 == g.T;
    out.slot = cta * 2 + (j0 == 0 ? 1 : 0);
    out.pieces = 0;
    if (j0 == 0 && j1 < g.T) {
      // up to the CTA that holds the item's last tile, by the line's arithmetic
      const long long last = x0 + static_cast<long long>(g.T - 1) * (g.wide ? kCostWide : kCostNarrow<D>) * kBN;
      out.pieces = static_cast<int>(((last + 1) * pl.G - 1) / pl.total) - cta + 1;
    }
    int keys = g.key_end - g.key_lo;
    if (p.mask_kind == ATTN_MASK_SLIDING_WINDOW) keys += ((p.n_sink + kBN - 1) / kBN) * kBN + kBN;
    w.s = x0 + static_cast<long long>(keys) * (g.wide ? kCostWide : kCostNarrow<D>);
    if (++w.rt == w.nrt) {
      w.rt = 0;
      if (++w.u == p.units) {
        w.u = 0;
        if (w.s < pl.end) {  // so a sequence with items follows
          do w.sq = seq_at(p, ++w.b);
          while (w.sq.n == 0);
          w.nrt = row_tiles(p, w.sq.n);
        }
      }
    }
    if (j0 < j1) return;
  }
  out.nt = 0;
}
__device__ __forceinline__ VarlenSplit split_of(const VlPiece& pc) {
  return VarlenSplit{pc.pieces, pc.row0, pc.g.ntok, pc.head0, pc.nheads, pc.g.wide ? 1 : 0, 0, 0};
}
// The V ring: slots are taken in turn, a wide item's without the last one. Both
// ends step through it alike; bit s is the parity of slot s's next use.
template <int STAGES>
struct VRing {
  int next = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void enter(bool wide) {
    if (wide && next == STAGES) next = 0;
  }
  __device__ __forceinline__ uint32_t phase(int s) const { return (parity >> s) & 1u; }
  __device__ __forceinline__ int take(bool wide) {
    const int s = next;
    parity ^= 1u << s;
    next = s + 1 < STAGES + (wide ? 0 : 1) ? s + 1 : 0;
    return s;
  }
};

// Whether this lane's row, at position `pos`, sees a key of the piece in a block whose
// table entry is outside the pool (warp-collective: a lane looks at every 32nd block,
// then all rows at each bad one). Only pieces with such an entry ask, so the key loop
// pays nothing for it.
__device__ __forceinline__ bool sees_bad_entry(const VarlenParams& p, const VlPiece& pc, int pos, int lane) {
  const bool win = p.mask_kind == ATTN_MASK_SLIDING_WINDOW;
  const int hi = p.mask_kind == ATTN_MASK_FULL ? pc.nk - 1 : pos, lo = win ? pos - p.window + 1 : 0;
  const int sink = win ? p.n_sink : 0;
  const int bs = p.block_size, per = kBN / bs, blocks = pc.nt * per;
  const int32_t* row = p.block_table + static_cast<size_t>(pc.b) * p.max_blocks;
  bool sees = false;
#pragma unroll 1
  for (int i0 = 0; i0 < blocks; i0 += 32) {
    const int i = i0 + lane, key = pc.g.tile_key(pc.j0 + i / per) + i % per * bs;
    bool bad = false;
    if (i < blocks && key < pc.g.key_end && (key + bs > pc.g.key_lo || key < pc.g.sink_end)) {  // as the copies ask
      const int ent = __ldg(row + key / bs);
      bad = ent < 0 || ent >= p.num_blocks;
    }
    for (unsigned who = __ballot_sync(0xffffffffu, bad); who != 0; who &= who - 1) {
      const int k = __shfl_sync(0xffffffffu, key, __ffs(who) - 1);
      sees |= k <= hi && (k + bs > lo || k < sink);
    }
  }
  return sees;
}

// Every (row, key) pair of a tile is visible: rows at positions [qa, qb], keys [k0, k0 + 128).
__device__ __forceinline__ bool vl_tile_is_full(const VarlenParams& p, int qa, int qb, int k0, int nk) {
  if (p.mask_kind == ATTN_MASK_FULL) return k0 + kBN <= nk;
  bool full = k0 + kBN - 1 <= qa;
  if (p.mask_kind == ATTN_MASK_SLIDING_WINDOW) full = full && (qb - k0 < p.window || k0 + kBN <= p.n_sink);
  return full;
}

// The running maximum of a row takes in a tile's: the sum and, where the maximum
// moved (lazily, see kVlRescale), the output row in TMEM are rescaled.
template <int D>
__device__ __forceinline__ void move_max(float tile_max, uint32_t colO, float& m_used, float& l_sum) {
  const float m_new = fmaxf(m_used, tile_max);
  bool rescale_o = false;
  float factor = 1.f;
  if (m_new > m_used + kVlRescale) {  // also true for the first visible key (m_used = -inf)
    const bool prev_finite = (m_used != -INFINITY);
    factor = prev_finite ? fast_exp2(m_used - m_new) : 0.f;
    l_sum *= factor;
    rescale_o = prev_finite;
    m_used = m_new;
  }
  // The score barrier was committed after this team's previous P V: O is stable.
  if (__any_sync(0xffffffffu, rescale_o)) rescale_row_t<D>(colO, rescale_o ? factor : 1.f);
}

// 32 scores to probabilities: p = 2^(s * scale * log2 e - m), their sum into acc.
__device__ __forceinline__ void exp_32(const float* sv, float sl2, float neg_m, float2 (&acc)[4], uint32_t (&pk)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float2 xv = ffma2(make_float2(sv[2 * e], sv[2 * e + 1]), make_float2(sl2, sl2), make_float2(neg_m, neg_m));
    float2 pv;
    pv.x = fast_exp2(xv.x);
    pv.y = fast_exp2(xv.y);
    acc[e & 3] = fadd2(acc[e & 3], pv);
    pk[e] = pack_bf16x2(pv.x, pv.y);
  }
}
__device__ __forceinline__ float sum_8(const float2 (&a)[4]) {
  return ((a[0].x + a[0].y) + (a[1].x + a[1].y)) + ((a[2].x + a[2].y) + (a[3].x + a[3].y));
}
__device__ __forceinline__ float max_32(const float* v, float m) {
  float mx0 = m, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
  for (int c = 0; c < 32; c += 8) {
    mx0 = max3f(mx0, v[c], v[c + 1]);
    mx1 = max3f(mx1, v[c + 2], v[c + 3]);
    mx2 = max3f(mx2, v[c + 4], v[c + 5]);
    mx3 = max3f(mx3, v[c + 6], v[c + 7]);
  }
  return max3f(mx0, mx1, fmaxf(mx2, mx3));
}

// One key tile of a team's rows that every row sees: scores from TMEM (colS), the
// running maximum and sum of this thread's row, and the probabilities back over
// the scores, in two halves that are announced as they land.
template <int D>
__device__ __forceinline__ void softmax_tile(float sl2, uint32_t colS, uint32_t colO, uint32_t bar_lo, uint32_t bar_hi,
                                             float& m_used, float& l_sum) {
  uint32_t raw[kBN];
#pragma unroll
  for (int cc = 0; cc < kBN / 32; ++cc)
    tmem_ld_32x32b_x32(colS + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&raw[cc * 32]));
  tc_wait_ld();
  float sv[kBN];
#pragma unroll
  for (int c = 0; c < kBN; ++c) sv[c] = __uint_as_float(raw[c]);
  float mx = -INFINITY;
#pragma unroll
  for (int cc = 0; cc < kBN / 32; ++cc) mx = max_32(&sv[cc * 32], mx);
  move_max<D>(mx * sl2, colO, m_used, l_sum);
  const float neg_m = (m_used == -INFINITY) ? 0.f : -m_used;  // scores of -inf alone
  float2 acc[4] = {};
#pragma unroll
  for (int cc = 0; cc < kBN / 32; ++cc) {
    uint32_t pk[16];
    exp_32(&sv[cc * 32], sl2, neg_m, acc, pk);
    tmem_st_32x32b_x16(colS + cc * 16, pk);  // over score columns already consumed
    if (cc == 1 || cc == 3) {
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(cc == 1 ? bar_lo : bar_hi);
    }
  }
  l_sum += sum_8(acc);
}

// The same at the mask's edge: visible to this row are the columns [cmin, cmax]
// and those before csink. Groups of 32 columns that no row of the warp sees are
// not computed (with a window most are not), so the groups go one by one, twice:
// maximum, then exponentials, each from TMEM. Both halves are announced at the end
// (one store wait less: 1-3 % of batches of short items).
template <int D>
__device__ __forceinline__ void softmax_edge_tile(float sl2, uint32_t colS, uint32_t colO, uint32_t bar_lo,
                                                  uint32_t bar_hi, int cmin, int cmax, int csink, bool row_valid,
                                                  float& m_used, float& l_sum) {
  auto visible = [&](int cc) -> uint32_t {
    const int lo = cmin - 32 * cc, hi = cmax - 32 * cc, sk = csink - 32 * cc;
    const uint32_t from = lo <= 0 ? ~0u : (lo > 31 ? 0u : ~0u << lo);
    const uint32_t to = hi < 0 ? 0u : (hi > 30 ? ~0u : (2u << hi) - 1u);
    const uint32_t sink = sk <= 0 ? 0u : (sk > 31 ? ~0u : (1u << sk) - 1u);
    return row_valid ? (from | sink) & to : 0u;
  };
  // some: not all rows see the whole group (else nothing is left to mask)
  auto load = [&](int cc, uint32_t vis, bool some, float (&sv)[32]) {
    uint32_t raw[32];
    tmem_ld_32x32b_x32(colS + cc * 32, raw);
    tc_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) sv[e] = __uint_as_float(raw[e]);
    if (some) {
#pragma unroll
      for (int e = 0; e < 32; ++e) sv[e] = vis & (1u << e) ? sv[e] : -INFINITY;
    }
  };
  float mx = -INFINITY;
  unsigned seen = 0, part = 0;
#pragma unroll 1
  for (int cc = 0; cc < kBN / 32; ++cc) {
    const uint32_t vis = visible(cc);
    if (!__any_sync(0xffffffffu, vis != 0u)) continue;
    const bool some = !__all_sync(0xffffffffu, vis == ~0u || !row_valid);
    seen |= 1u << cc;
    part |= static_cast<unsigned>(some) << cc;
    float sv[32];
    load(cc, vis, some, sv);
    mx = max_32(sv, mx);
  }
  move_max<D>(mx * sl2, colO, m_used, l_sum);
  const float neg_m = (m_used == -INFINITY) ? 0.f : -m_used;  // a row with nothing visible yet uses m = 0
  float2 acc[4] = {};
#pragma unroll 1
  for (int cc = 0; cc < kBN / 32; ++cc) {
    uint32_t pk[16];
    if (seen >> cc & 1u) {
      float sv[32];
      load(cc, visible(cc), part >> cc & 1u, sv);
      exp_32(sv, sl2, neg_m, acc, pk);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) pk[e] = 0u;
    }
    tmem_st_32x32b_x16(colS + cc * 16, pk);  // group cc / 2 of the scores has been read
  }
  tc_wait_st();
  tc_fence_before();
  mbar_arrive(bar_lo);
  mbar_arrive(bar_hi);
  l_sum += sum_8(acc);
}

template <int D>
__global__ void __launch_bounds__(kVlThreads, 1)
    prefill_varlen_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qh,
                          const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const __grid_constant__ CUtensorMap tm_vr, const __grid_constant__ CUtensorMap tm_o,
                          const VarlenParams p) {
  using C = VlCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long sums_s[kVlWarps];
  __shared__ VlPlan plan_s;
  __shared__ VlPiece pieces_s[kPieces];
  __shared__ volatile int bad_s[kPieces];  // the piece's blocks have an entry outside the pool
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t sbase = (raw_u32 + 1023u) & ~1023u;  // swizzled tiles need 1024-byte alignment
  uint8_t* smem = smem_raw + (sbase - raw_u32);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  // the joining grid may be set up now; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  const uint32_t bars = sbase + C::kBarOff;
  auto bar = [&](int i) -> uint32_t { return bars + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + kVbTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBarOff + kVbAbort);

  if (threadIdx.x == 0) {
    mbar_init(bar(kVbQFull), 1);
    mbar_init(bar(kVbQEmpty), 1);
    mbar_init(bar(kVbQEmpty + 1), 1);
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(kVbKFull + s), 1);
      mbar_init(bar(kVbKEmpty + s), 1);
    }
    for (int s = 0; s < 5; ++s) {
      mbar_init(bar(kVbVFull + s), 1);
      mbar_init(bar(kVbVEmpty + s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(kVbSFull + x), 1);
      mbar_init(bar(kVbPLo + x), kBM);
      mbar_init(bar(kVbPHi + x), kBM);
      mbar_init(bar(kVbOFinal + x), 1);
    }
    for (int s = 0; s < kPieces; ++s) {
      mbar_init(bar(kVbPiece + s), 1);
      mbar_init(bar(kVbPieceDone + s), 11);  // both TMA warps, the MMA warp, 8 softmax warps
    }
    for (int s = 0; s < 6; ++s) mbar_init(bar(kVbPair + s), 2);
    mbar_init(bar(kVbDrain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    p.splits[cta].pieces = 0;
  }
  for (int i = threadIdx.x; i < C::kTile / 16; i += kVlThreads)
    reinterpret_cast<uint4*>(smem + C::kQOff)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == kVlMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }

  // ---- the line: total length, then the item at this CTA's start. Warp w takes
  // sequences [32 (12 r + w), + 32) in round r; costs of one round stay in registers.
  {
    const int rounds = (p.B + kVlThreads - 1) / kVlThreads;
    VlSeq sq{0, 0, 0, false};
    long long uc = 0, sum = 0;
    for (int r = 0; r < rounds; ++r) {
      const int b = r * kVlThreads + static_cast<int>(threadIdx.x);
      sq = b < p.B ? seq_at(p, b) : VlSeq{0, 0, 0, false};
      uc = sq.n > 0 ? line_of<D>(p, sq.n, sq.nk, row_tiles(p, sq.n)) : 0;
      sum += uc * p.units;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) sums_s[warp] = sum;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kVlWarps; ++w) total += sums_s[w];
    const long long most = total / kMinStretch;
    const int G = most < 1 ? 1 : (most < gridDim.x ? static_cast<int>(most) : static_cast<int>(gridDim.x));
    const long long start = cta < G ? total * cta / G : 0, end = cta < G ? total * (cta + 1) / G : 0;
    long long before = 0;  // of all earlier rounds
    for (int r = 0; r < rounds; ++r) {
      const int b = r * kVlThreads + static_cast<int>(threadIdx.x);
      if (rounds > 1) {
        sq = b < p.B ? seq_at(p, b) : VlSeq{0, 0, 0, false};
        uc = sq.n > 0 ? line_of<D>(p, sq.n, sq.nk, row_tiles(p, sq.n)) : 0;
      }
      const long long c = uc * p.units;
      long long inc = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      __syncthreads();  // sums_s has been read
      if (lane == 31) sums_s[warp] = inc;
      __syncthreads();
      long long mine = before;
      for (int w = 0; w < kVlWarps; ++w) {
        if (w < warp) mine += sums_s[w];
        before += sums_s[w];
      }
      mine += inc - c;
      if (c > 0 && start < end && mine <= start && start < mine + c) {
        long long off = start - mine;
        const int u = static_cast<int>(off / uc);
        off -= u * uc;
        int rt = 0;  // the last row tile that starts at or before it
        for (int hi = row_tiles(p, sq.n); hi - rt > 1;) {
          const int mid = (rt + hi) >> 1;
          if (line_of<D>(p, sq.n, sq.nk, mid) <= off) rt = mid;
          else hi = mid;
        }
        const long long at = rt > 0 ? line_of<D>(p, sq.n, sq.nk, rt) : 0;
        plan_s.b = b;
        plan_s.u = u;
        plan_s.rt = rt;
        plan_s.s = start - (off - at);
      }
    }
    if (threadIdx.x == 0) {
      plan_s.start = start;
      plan_s.end = end;
      plan_s.total = total;
      plan_s.G = G;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long budget = p.budget;
  const VlPlan& pl = plan_s;
  auto first_walk = [&]() -> VlWalk {
    VlWalk w;
    w.s = pl.start < pl.end ? pl.s : pl.end;
    w.b = w.u = w.rt = w.nrt = 0;
    w.sq = VlSeq{0, 0, 0, false};
    if (pl.start < pl.end) {
      w.b = pl.b;
      w.u = pl.u;
      w.rt = pl.rt;
      w.sq = seq_at(p, w.b);
      w.nrt = row_tiles(p, w.sq.n);
    }
    return w;
  };
  // piece `it`, worked out ahead by the plan warp; the reader gives the entry back
  auto piece_wait = [&](int it) -> bool {
    return mbar_wait_bounded(bar(kVbPiece + it % kPieces), (it / kPieces) & 1, budget, abort_flag);
  };
  auto piece_done = [&](int it) { mbar_arrive(bar(kVbPieceDone + it % kPieces)); };

  if (warp >= kVlTmaWarp) {
    regs_dec<kVlRegsControl>();
    if (warp == kVlTmaWarp || warp == kVlTmaVWarp) {
      // ---------------------------------------------------------- TMA producers: Q and K by one warp, V by the other
      // (a box of a block of 16 tokens takes about as long to issue as to move:
      // one warp for both held 64 sequences of 1K-32K tokens at 4,800 GB/s, two reach 6,180).
      // Lane 0 waits on the ring and arms the barriers, lane e copies block e of a
      // key tile, its table entry read one tile ahead. A block that no row of the
      // item sees, that lies past the sequence or whose entry is outside the pool is
      // asked for at block num_blocks, which TMA fills with zeros: nothing is read of
      // it, its keys are masked, and its probabilities of 0 meet zeros in V. In the
      // block where the sequence ends, V goes row by row (all lanes), zeros behind
      // the end, for the same reason: 0 times what a pool holds there could be NaN.
      // K's rows there are masked.
      const bool k_warp = warp == kVlTmaWarp;
      if (lane == 0) {
        prefetch_tmap(k_warp ? &tm_k : &tm_v);
        if (k_warp) prefetch_tmap(&tm_q);
      }
      const int bs = p.block_size, boxes = kBN / bs;
      int g = 0, it = 0;  // K tiles and items so far
      VRing<C::kStages> vr;
      bool ok = true;
      for (;; ++it) {
        ok = __all_sync(0xffffffffu, piece_wait(it));
        if (!ok) break;
        const int flag = it % kPieces;
        const VlPiece pc = pieces_s[flag];
        const VlGeom& gm = pc.g;
        const int nt = pc.nt;
        if (nt == 0) break;
        if (k_warp && lane == 0) bad_s[flag] = 0;
        __syncwarp();
        // this lane's block of key tile j: whether it is asked for, and its raw entry,
        // which nothing looks at before the next tile's turn
        bool asked = false;
        int raw = 0;
        auto fetch = [&](int j) {
          const int key = gm.tile_key(pc.j0 + j) + lane * bs;
          asked = j < nt && lane < boxes && key < gm.key_end && (key + bs > gm.key_lo || key < gm.sink_end);
          if (asked) raw = __ldg(p.block_table + static_cast<size_t>(pc.b) * p.max_blocks + key / bs);
        };
        fetch(0);
        // The second Q tile's place is a V slot of narrow items: the item before has
        // read its Q, and a wide item's Q waits for the slot's last V tile.
        bool armed = true;
        if (lane == 0) {
          armed = (it == 0) ||
                  mbar_wait_bounded(bar(kVbQEmpty + ((it - 1) & 1)), ((it - 1) >> 1) & 1, budget, abort_flag);
          if (k_warp) {
            if (armed && gm.wide)
              armed = mbar_wait_bounded(bar(kVbVEmpty + C::kStages), vr.phase(C::kStages) ^ 1u, budget, abort_flag);
            if (armed) {
              const int tiles = gm.wide ? 2 : 1;
              const int rows = pc.half ? 2 * gm.ntok * p.gsz : tiles * p.tpt * p.gsz;
              mbar_arrive_expect_tx(bar(kVbQFull), rows * C::kHalves * 128);
              if (!pc.half)
                for (int x = 0; x < tiles; ++x)
                  for (int hh = 0; hh < C::kHalves; ++hh)
                    tma_load_3d(sbase + C::kQOff + x * C::kTile + hh * C::kHalf, &tm_q, bar(kVbQFull), hh * 64,
                                pc.head0, pc.row0 + x * p.tpt);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, armed, 0);
        if (!ok) break;
        if (k_warp && pc.half) {
          // the same rows for both teams, token by token: the tile's other rows stay as
          // they were, zeros unless a larger item came before (zeros cost less power)
          __syncwarp();
          for (int t = lane; t < 2 * C::kHalves * gm.ntok; t += 32) {
            const int tk = t / (2 * C::kHalves), x = t & 1, hh = (t >> 1) & (C::kHalves - 1);
            tma_load_3d(sbase + C::kQOff + x * 64 * 128 + hh * C::kHalf + tk * p.gsz * 128, &tm_qh, bar(kVbQFull),
                        hh * 64, pc.head0, pc.row0 + tk);
          }
        }
        vr.enter(gm.wide);
        for (int i = 0; i < nt; ++i) {
          int ent = p.num_blocks;
          if (asked) {
            if (raw >= 0 && raw < p.num_blocks) ent = raw;
            else if (k_warp) bad_s[flag] = 1;
          }
          fetch(i + 1);
          __syncwarp();
          if (k_warp) {
            const int gi = g + i, s = gi % C::kStages, rnd = gi / C::kStages;
            if (lane == 0) {
              armed = (rnd == 0) || mbar_wait_bounded(bar(kVbKEmpty + s), (rnd - 1) & 1, budget, abort_flag);
              if (armed) mbar_arrive_expect_tx(bar(kVbKFull + s), C::kTile);
            }
            ok = __shfl_sync(0xffffffffu, armed, 0);
            if (!ok) {
              g += i;
              break;
            }
            vr.take(gm.wide);
            const uint32_t dst = sbase + C::kKOff + s * C::kTile + lane * bs * 128;
            if (lane < boxes)
              for (int hh = 0; hh < C::kHalves; ++hh)
                tma_load_4d(dst + hh * C::kHalf, &tm_k, bar(kVbKFull + s), hh * 64, pc.kvh, 0, ent);
          } else {
            const int s = vr.next;
            if (lane == 0) {
              armed = mbar_wait_bounded(bar(kVbVEmpty + s), vr.phase(s) ^ 1u, budget, abort_flag);
              if (armed) mbar_arrive_expect_tx(bar(kVbVFull + s), C::kTile);
            }
            ok = __shfl_sync(0xffffffffu, armed, 0);
            if (!ok) break;
            vr.take(gm.wide);
            const uint32_t dst = sbase + (s < C::kStages ? C::kVOff + s * C::kTile : C::kQOff + C::kTile);
            const uint32_t full = bar(kVbVFull + s);
            const int key = gm.tile_key(pc.j0 + i) + lane * bs;
            const bool part = lane < boxes && key < pc.nk && key + bs > pc.nk && ent != p.num_blocks;
            if (lane < boxes && !part)
              for (int hh = 0; hh < C::kHalves; ++hh)
                tma_load_4d(dst + lane * bs * 128 + hh * C::kHalf, &tm_v, full, hh * 64, pc.kvh, 0, ent);
            const unsigned who = __ballot_sync(0xffffffffu, part);
            if (who != 0) {
              const int src = __ffs(who) - 1;
              const int phys = __shfl_sync(0xffffffffu, ent, src);
              const int valid = pc.nk - __shfl_sync(0xffffffffu, key, src);  // 1 .. bs - 1 rows hold tokens
              for (int r = lane; r < bs * C::kHalves; r += 32) {
                const int slot = r / C::kHalves, hh = r - slot * C::kHalves;
                tma_load_4d(dst + (src * bs + slot) * 128 + hh * C::kHalf, &tm_vr, full, hh * 64, pc.kvh, slot,
                            slot < valid ? phys : p.num_blocks);
              }
            }
          }
        }
        if (!ok) {
          ++it;  // this item's Q is in flight
          break;
        }
        g += nt;
        __syncwarp();
        if (lane == 0) piece_done(it);
      }
      if (lane == 0) {
        if (!ok) raise_abort(abort_flag, p.status);
        // Drain: this warp's newest copy of every stage has landed before the CTA may exit.
        volatile int never = 0;
        if (k_warp) {
          if (it > 0) mbar_wait_bounded(bar(kVbQFull), (it - 1) & 1, kDrainBudgetCycles, &never);
          for (int j = (g > C::kStages ? g - C::kStages : 0); j < g; ++j)
            mbar_wait_bounded(bar(kVbKFull + j % C::kStages), (j / C::kStages) & 1, kDrainBudgetCycles, &never);
        } else {
          for (int s = 0; s <= C::kStages; ++s)
            mbar_wait_bounded(bar(kVbVFull + s), vr.phase(s) ^ 1u, kDrainBudgetCycles, &never);
        }
      }
    } else if (warp == kVlMmaWarp) {
      // ---------------------------------------------------------- MMA issuer (the warp stays converged)
      auto wait = [&](int i, uint32_t parity) -> bool {
        const bool r = __all_sync(0xffffffffu, mbar_wait_bounded(bar(i), parity, budget, abort_flag));
        tc_fence_after();
        return r;
      };
      const uint64_t dq0 = desc_sw128(sbase + C::kQOff, 16, 1024);
      const uint64_t dk0 = desc_sw128(sbase + C::kKOff, 16, 1024);
      const uint64_t dv0 = desc_sw128(sbase + C::kVOff, C::kHalf, 1024);
      const uint64_t dvq = desc_sw128(sbase + C::kQOff + C::kTile, C::kHalf, 1024);  // the V ring's last slot
      constexpr uint64_t kTileUnits = C::kTile >> 4;
      auto wait_k = [&](int g) -> bool {
        return wait(kVbKFull + g % C::kStages, (g / C::kStages) & 1);
      };
      // team x's scores of key tile g (counted over the CTA's stretch) with Q tile qx
      uint32_t p_par = 0;  // bit x: parity of team x's next probabilities
      auto issue_s = [&](int x, int qx, int g) {
        mma_scores_w<D>(tmem + C::col_s(x), dq0 + static_cast<uint64_t>(qx) * kTileUnits,
                      dk0 + static_cast<uint64_t>(g % C::kStages) * kTileUnits);
        tc_commit_w(bar(kVbSFull + x));
      };
      // O_x (+)= P_x V, each half of P as it lands
      auto pv = [&](int x, int s, bool first) -> bool {
        const uint64_t dv = s < C::kStages ? dv0 + static_cast<uint64_t>(s) * kTileUnits : dvq;
        const uint32_t parity = (p_par >> x) & 1u;
        if (!wait(kVbPLo + x, parity)) return false;
        mma_pv_w<D>(tmem + C::col_o(x), tmem + C::col_s(x), dv, 0, first);
        if (!wait(kVbPHi + x, parity)) return false;
        mma_pv_w<D>(tmem + C::col_o(x), tmem + C::col_s(x), dv, 1, first);
        p_par ^= 1u << x;
        return true;
      };
      int g = 0, it = 0;
      VRing<C::kStages> vr;
      bool ok = true;
      for (; ok; ++it) {
        ok = wait(kVbPiece + it % kPieces, (it / kPieces) & 1);
        if (!ok) break;
        const int nt = pieces_s[it % kPieces].nt;
        const bool wide = pieces_s[it % kPieces].g.wide;
        __syncwarp();
        if (lane == 0) piece_done(it);
        if (nt == 0) break;
        vr.enter(wide);
        const int teams = wide ? 2 : 1, ahead = wide ? 1 : 2;  // key tiles a score runs ahead of its P V
        ok = wait(kVbQFull, it & 1);
        if (!ok) break;
        // the first scores of both teams
        for (int j = 0; j < min(ahead, nt) && ok; ++j) {
          ok = wait_k(g + j);
          if (!ok) break;
          issue_s(wide ? 0 : j, 0, g + j);
          if (wide) issue_s(1, 1, g);
          tc_commit_w(bar(kVbKEmpty + (g + j) % C::kStages));
          if (j == nt - 1) tc_commit_w(bar(kVbQEmpty + (it & 1)));
        }
        for (int j = 0; j < nt && ok; ++j) {
          const int jn = j + ahead;
          const uint32_t parity = vr.phase(vr.next);
          const int s = vr.take(wide);
          ok = wait(kVbVFull + s, parity);
          for (int t = 0; t < teams && ok; ++t) {
            const int x = wide ? t : (j & 1);
            const bool last_team = t == teams - 1;
            // P V of key tile j, then (in issue order, so they overwrite P only after it is
            // read) this team's next scores
            ok = pv(x, s, wide ? j == 0 : j < 2);
            if (!ok) break;
            if (jn >= nt) tc_commit_w(bar(kVbOFinal + x));
            if (last_team) tc_commit_w(bar(kVbVEmpty + s));
            if (jn < nt) {
              if (t == 0) ok = wait_k(g + jn);
              if (!ok) break;
              issue_s(x, wide ? t : 0, g + jn);
              if (last_team) {
                tc_commit_w(bar(kVbKEmpty + (g + jn) % C::kStages));
                if (jn == nt - 1) tc_commit_w(bar(kVbQEmpty + (it & 1)));  // that was the item's last read of Q
              }
            }
          }
        }
        g += nt;
      }
      if (!ok && lane == 0) raise_abort(abort_flag, p.status);
      __syncwarp();
      // Drain: every MMA this warp issued has completed before TMEM is freed.
      tc_commit_w(bar(kVbDrain));
      volatile int never = 0;
      mbar_wait_bounded(bar(kVbDrain), 0, kDrainBudgetCycles, &never);
    } else if (warp == kVlPlanWarp) {
      // ---------------------------------------------------------- the pieces of the stretch, a few ahead of their use
      if (lane == 0) {
        VlWalk w = first_walk();
        for (int it = 0;; ++it) {
          const int e = it % kPieces;
          // The piece that holds the entry (pieces_s[e] until it is given back) may take as
          // long as its tiles do, each a chain of at most 8 waits: so many budgets, where
          // every other wait is for one step of the pipeline.
          if (it >= kPieces && !mbar_wait_bounded(bar(kVbPieceDone + e), (it / kPieces - 1) & 1,
                                                  min(budget, 1LL << 35) * 8 * (pieces_s[e].nt + 2), abort_flag)) {
            raise_abort(abort_flag, p.status);
            break;
          }
          VlPiece pc;
          next_piece<D>(p, pl, cta, w, pc);
          pieces_s[e] = pc;
          if (pc.nt > 0 && pc.pieces > 0) p.splits[cta] = split_of(pc);
          mbar_arrive(bar(kVbPiece + e));
          if (pc.nt == 0) break;
        }
      }
      __syncwarp();
      // then the rows of sequences whose lengths do not fit
      for (int base = cta * 32; base < p.B; base += gridDim.x * 32) {
        const bool mine = base + lane < p.B && seq_at(p, base + lane).bad;
        for (unsigned bad = __ballot_sync(0xffffffffu, mine); bad != 0; bad &= bad - 1) {
          const int b = base + __ffs(bad) - 1;
          if (lane == 0 && p.status != nullptr) atomicOr(p.status, ATTN_STATUS_BIT_DEVICE_CHECK);
          const int r0 = max(0, __ldg(p.cu_q + b)), r1 = min(p.T, __ldg(p.cu_q + b + 1));
          for (int r = r0; r < r1; ++r) {
            __nv_bfloat16* row = p.o + static_cast<size_t>(r) * p.Hq * D;
            for (int i = lane; i < p.Hq * D / 8; i += 32)
              reinterpret_cast<uint4*>(row)[i] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
            if (p.lse != nullptr)
              for (int i = lane; i < p.Hq; i += 32) p.lse[static_cast<size_t>(r) * p.Hq + i] = NAN;
          }
        }
      }
    }
  } else {
    regs_inc<kVlRegsSoftmax>();
    // ------------------------------------------------------------ softmax teams (warps 0-3, 4-7)
    const int x = warp >> 2;
    const int r = threadIdx.x & (kBM - 1);  // row of the tile = TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t colS = lane_base + C::col_s(x);
    const uint32_t colO = lane_base + C::col_o(x);
    int cnt = 0, fin = 0, it = 0;  // this team's score tiles, finished outputs; items
    bool ok = true;
    // Both warps of pair `id` have come here. Bounded like every wait: after an expired
    // wait elsewhere the other warp may have left.
    uint32_t pair_par = 0;
    auto pair_sync = [&](int id) -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kVbPair + id));
      const bool r =
          __all_sync(0xffffffffu, mbar_wait_bounded(bar(kVbPair + id), (pair_par >> id) & 1u, budget, abort_flag));
      pair_par ^= 1u << id;
      return r;
    };
    for (; ok; ++it) {
      ok = __all_sync(0xffffffffu, piece_wait(it));
      if (!ok) break;
      const VlPiece& pc = pieces_s[it % kPieces];
      const VlGeom& gm = pc.g;
      const int nt = pc.nt;
      if (nt == 0) break;
      const bool wide = gm.wide;
      const int nheads = pc.nheads, head0 = pc.head0;
      const int t0 = wide ? x * p.tpt : 0;                 // the tile's first token in the item
      const int ntok = min(gm.ntok - t0, p.tpt);           // and its tokens (a wide item's second tile has some)
      const int qa = gm.pos_lo + t0;
      // This thread's row of the item's tile, its token and head. A narrow item of at
      // most 64 rows stands in the lanes 64 and up for team 1: its warps then run on
      // the SM partitions that team 0's leave idle (warps 0 and 4 share one). Sustained,
      // 4 chunks beside 32 single rows take 1,382 us so and 1,397 with both teams on
      // the same lanes; batches of narrow items alone the same either way.
      const int shift = pc.half && x == 1 ? 2 : 0;  // in warps
      const int wr = (warp & 3) - shift, row = wr * 32 + lane;
      const int rtok = (row * p.row_magic) >> 16, rhead = row - rtok * p.gsz;
      const bool active = wr >= 0 && wr * 32 < ntok * p.gsz;  // the warp has rows of the item
      const bool row_valid = active && rtok < ntok && rhead < nheads;
      const float sink2 = p.sinks != nullptr && row_valid ? __ldg(p.sinks + head0 + rhead) * kLog2e : -INFINITY;
      // Max the exponentials are taken against (base 2). Rows that are none: +inf, so
      // that their probabilities are 0 (no output is made of them; zeros cost less power).
      float m_used = row_valid ? -INFINITY : INFINITY;
      float l_sum = 0.f;         // running sum of 2^(s - m_used)
      for (int j = wide ? 0 : x; j < nt && ok; j += wide ? 1 : 2, ++cnt) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kVbSFull + x), cnt & 1, budget, abort_flag));
        if (!ok) break;
        if (!active) {  // rows nobody reads: whatever P holds there is fine
          mbar_arrive(bar(kVbPLo + x));
          mbar_arrive(bar(kVbPHi + x));
          continue;
        }
        const int k0 = gm.tile_key(pc.j0 + j);
        tc_fence_after();
        if (vl_tile_is_full(p, qa, qa + ntok - 1, k0, pc.nk))
          softmax_tile<D>(p.scale_log2, colS, colO, bar(kVbPLo + x), bar(kVbPHi + x), m_used, l_sum);
        else
          softmax_edge_tile<D>(p.scale_log2, colS, colO, bar(kVbPLo + x), bar(kVbPHi + x),
                               p.mask_kind == ATTN_MASK_SLIDING_WINDOW ? qa + rtok - k0 - p.window + 1 : 0,
                               (p.mask_kind == ATTN_MASK_FULL ? pc.nk - 1 : qa + rtok) - k0, p.n_sink - k0, row_valid,
                               m_used, l_sum);
      }
      const bool took_part = wide || nt > x;
      if (ok && took_part)
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kVbOFinal + x), fin & 1, budget, abort_flag));
      if (took_part) ++fin;
      if (!ok) raise_abort(abort_flag, p.status);
      tc_fence_after();
      if (!active || !took_part) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) piece_done(it);
        continue;
      }

      // After an expired wait the accumulators are read all the same and come out as NaN.
      const uint32_t stage = sbase + C::kStageOff + warp * 4096;
      if (lane == 0) bulk_wait_read_all();  // the last output has left the staging box
      __syncwarp();

      // ---- the two teams of a narrow item are joined: both know both sums, team 1
      // hands its output over in 32-column pieces through its staging box
      const bool join = !wide && nt > 1;
      const int other_warp = x == 0 ? warp + 4 + (pc.half ? 2 : 0) : wr, pair = wr + (pc.half ? 4 : 0);
      float f = 1.f;
      if (join) {
        float2* mine = reinterpret_cast<float2*>(smem + C::kStageOff + warp * 4096);
        mine[lane] = make_float2(m_used, ok ? l_sum : NAN);
        if (!pair_sync(pair)) ok = false;
        const float2 other = reinterpret_cast<float2*>(smem + C::kStageOff + other_warp * 4096)[lane];
        if (!pair_sync(pair)) ok = false;  // read before the boxes are written again
        const float m = fmaxf(m_used, other.x);
        f = m_used == -INFINITY ? 0.f : exp2f(m_used - m);
        l_sum = l_sum * f + (other.x == -INFINITY ? 0.f * other.y : other.y * exp2f(other.x - m));
        m_used = m;
      }
      if (join && x == 1) {
        float* box = reinterpret_cast<float*>(smem + C::kStageOff + warp * 4096);
#pragma unroll
        for (int c32 = 0; c32 < D / 32; ++c32) {
          uint32_t ov[32];
          tmem_ld_32x32b_x32(colO + c32 * 32, ov);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) box[e * 32 + lane] = f == 0.f ? 0.f : __uint_as_float(ov[e]) * f;
          if (!pair_sync(pair)) ok = false;
          if (!pair_sync(pair)) ok = false;
        }
        if (!ok) raise_abort(abort_flag, p.status);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) piece_done(it);
        continue;
      }

      const bool whole = pc.whole;
      const bool bad = __any_sync(0xffffffffu, bad_s[it % kPieces] != 0);
      if (bad && lane == 0 && p.status != nullptr) atomicOr(p.status, ATTN_STATUS_BIT_DEVICE_CHECK);
      float l = !ok || (bad && sees_bad_entry(p, pc, qa + rtok, lane)) ? NAN : l_sum, norm = 1.f;
      if (whole) {
        float m = m_used, ff = 1.f;
        if (p.sinks != nullptr) {  // one more column with no value
          m = fmaxf(m_used, sink2);
          ff = exp2f(m_used - m);
          l = l * ff + exp2f(sink2 - m);
          if (row_valid && !(sink2 < INFINITY)) {  // NaN or +inf
            l = NAN;
            if (p.status != nullptr) atomicOr(p.status, ATTN_STATUS_BIT_DEVICE_CHECK);
          }
        }
        norm = ff / l;
        if (row_valid && p.lse != nullptr)
          p.lse[static_cast<size_t>(pc.row0 + t0 + rtok) * p.Hq + head0 + rhead] = (m + log2f(l)) * kLn2;
      } else {
        p.part_ml[static_cast<size_t>(pc.slot) * kVlRows + x * kBM + r] = make_float2(m_used, l);
      }
      const float* box = reinterpret_cast<const float*>(smem + C::kStageOff + other_warp * 4096);
      // a warp's rows are whole tokens of the sequence: they leave as a box
      const int wtok = p.tma_out ? 32 / p.gsz : 0;
      const bool as_box = p.tma_out && (wr + 1) * wtok <= ntok;
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh) {
        if (hh > 0 && whole && as_box) {
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
        }
#pragma unroll
        for (int q32 = 0; q32 < 2; ++q32) {
          uint32_t ov[32];
          tmem_ld_32x32b_x32(colO + hh * 64 + q32 * 32, ov);
          tc_wait_ld();
          if (join) {
            if (!pair_sync(pair)) ok = false;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              ov[e] = __float_as_uint((f == 0.f ? 0.f : __uint_as_float(ov[e]) * f) + box[e * 32 + lane]);
            if (!pair_sync(pair)) ok = false;
            if (!ok) norm = NAN;
          }
          if (whole) {
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) {
              uint32_t w4[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w4[e] = pack_bf16x2(__uint_as_float(ov[c4 * 8 + 2 * e]) * norm,
                                    __uint_as_float(ov[c4 * 8 + 2 * e + 1]) * norm);
              const uint32_t dst = stage + lane * 128 + (((q32 * 4 + c4) ^ (lane & 7)) << 4);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(dst), "r"(w4[0]), "r"(w4[1]), "r"(w4[2]),
                           "r"(w4[3])
                           : "memory");
            }
          } else {
#pragma unroll
            for (int c4 = 0; c4 < 8; ++c4)
              p.part_o[(static_cast<size_t>(pc.slot) * (D / 4) + hh * 16 + q32 * 8 + c4) * kVlRows + x * kBM + r] =
                  make_float4(__uint_as_float(ov[4 * c4]), __uint_as_float(ov[4 * c4 + 1]),
                              __uint_as_float(ov[4 * c4 + 2]), __uint_as_float(ov[4 * c4 + 3]));
          }
        }
        if (whole && as_box) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tm_o, stage, hh * 64, head0, pc.row0 + t0 + wr * wtok);
            bulk_commit();
          }
        } else if (whole) {  // 8 lanes a row, 16 bytes each; only rows of this sequence and these heads
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int sr = i * 4 + (lane >> 3), c = lane & 7;
            const int tk = ((wr * 32 + sr) * p.row_magic) >> 16, hd = wr * 32 + sr - tk * p.gsz;
            if (tk < ntok && hd < nheads) {
              uint4 v;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                           : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                           : "r"(stage + sr * 128 + ((c ^ (sr & 7)) << 4)));
              __nv_bfloat16* dst =
                  p.o + (static_cast<size_t>(pc.row0 + t0 + tk) * p.Hq + head0 + hd) * D + hh * 64;
              reinterpret_cast<uint4*>(dst)[c] = v;
            }
          }
          __syncwarp();
        }
      }
      if (join && !ok) {
        raise_abort(abort_flag, p.status);
        if (!whole) p.part_ml[static_cast<size_t>(pc.slot) * kVlRows + x * kBM + r] = make_float2(m_used, NAN);
      }
      // The next item's first P V overwrites O: its P is announced only after
      // these loads completed (tcgen05.wait::ld above, fence before the arrive).
      tc_fence_before();
      __syncwarp();
      if (lane == 0) piece_done(it);
    }
    if (lane == 0) bulk_wait_all();  // output stores complete before the CTA exits
    if (!ok) {
      // a wait expired: every row of the pieces not reached becomes NaN
      raise_abort(abort_flag, p.status);
      VlWalk w = first_walk();
      VlPiece pc;
      for (int i = 0;; ++i) {
        next_piece<D>(p, pl, cta, w, pc);
        if (pc.nt == 0) break;
        if (i < it) continue;
        if (pc.pieces > 0 && threadIdx.x == 0) p.splits[cta] = split_of(pc);
        const int rtok = (r * p.row_magic) >> 16, rhead = r - rtok * p.gsz, tok = x * p.tpt + rtok;
        if (rtok >= p.tpt || tok >= pc.g.ntok || rhead >= pc.nheads) continue;
        if (!pc.whole) {
          p.part_ml[static_cast<size_t>(pc.slot) * kVlRows + x * kBM + r] = make_float2(0.f, NAN);
          continue;
        }
        const size_t row = static_cast<size_t>(pc.row0 + tok) * p.Hq + pc.head0 + rhead;
        for (int i8 = 0; i8 < D / 8; ++i8)
          reinterpret_cast<uint4*>(p.o + row * D)[i8] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        if (p.lse != nullptr) p.lse[row] = NAN;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kVlMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the item that CTA blockIdx.x of the grid above started
// and did not finish: out = sum_i O_i 2^(m_i - m) / sum_i l_i 2^(m_i - m), in
// the order of the pieces, kJoinBatch of them loaded at a time. A thread takes 4
// columns of a row.
constexpr int kJoinThreads = 256, kJoinParts = 8, kJoinBatch = 8;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) prefill_varlen_join_kernel(const VarlenParams p) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the other grid has finished and its stores are visible
  const int c = blockIdx.x;
  const VarlenSplit sp = p.splits[c];
  if (sp.pieces == 0) return;
  // rows in use, in whole warps: the first tile's, or both tiles
  const int nr = sp.wide ? kVlRows : (min(sp.ntok, p.tpt) * p.gsz + 31) & ~31;
  for (int i = blockIdx.y * kJoinThreads + threadIdx.x; i < nr * (D / 4); i += kJoinParts * kJoinThreads) {
    const int c4 = i / nr, row = i - c4 * nr;
    const int r = row & (kBM - 1);
    const int tk = (r * p.row_magic) >> 16, hd = r - tk * p.gsz;
    const int tok = (row >> 7) * p.tpt + tk;
    if (tk >= p.tpt || tok >= sp.ntok || hd >= sp.nheads) continue;
    const float sk = p.sinks != nullptr ? __ldg(p.sinks + sp.head0 + hd) * kLog2e : -INFINITY;
    float m = sk, l = p.sinks != nullptr ? 1.f : 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < sp.pieces; k0 += kJoinBatch) {  // loads of kJoinBatch pieces in flight
      float2 ml[kJoinBatch];
      float4 v[kJoinBatch];
#pragma unroll
      for (int j = 0; j < kJoinBatch; ++j) {
        const int k = min(k0 + j, sp.pieces - 1);
        const size_t slot = 2 * (c + k) + (k == 0);
        ml[j] = p.part_ml[slot * kVlRows + row];
        v[j] = p.part_o[(slot * (D / 4) + c4) * kVlRows + row];
      }
      float m_new = m;
#pragma unroll
      for (int j = 0; j < kJoinBatch; ++j) m_new = fmaxf(m_new, ml[j].x);
      // what has seen nothing yet has the maximum -inf, the sum 0 and the output 0
      const float f0 = m == -INFINITY ? 0.f : exp2f(m - m_new);
      l *= f0;
      acc = make_float4(acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0);
      m = m_new;
#pragma unroll
      for (int j = 0; j < kJoinBatch; ++j) {
        if (k0 + j >= sp.pieces) break;
        const float f = ml[j].x == -INFINITY ? 0.f : exp2f(ml[j].x - m);
        l += ml[j].y * f;
        acc.x += v[j].x * f;
        acc.y += v[j].y * f;
        acc.z += v[j].z * f;
        acc.w += v[j].w * f;
      }
    }
    if (p.sinks != nullptr && !(sk < INFINITY)) {  // NaN or +inf
      l = NAN;
      if (p.status != nullptr) atomicOr(p.status, ATTN_STATUS_BIT_DEVICE_CHECK);
    }
    const float inv = 1.f / l;
    const size_t out = static_cast<size_t>(sp.row0 + tok) * p.Hq + sp.head0 + hd;
    *reinterpret_cast<uint2*>(p.o + out * D + 4 * c4) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (c4 == 0 && p.lse != nullptr) p.lse[out] = (m + log2f(l)) * kLn2;
  }
}

// Packed rows [T, Hq, d] as a rank-3 tensor; box = 64 columns x heads x tokens.
bool encode_packed(CUtensorMap* map, const void* base, int d, int hq, int tokens, int box_heads, int box_tokens) {
  const auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(hq),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(hq) * d * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
  const cuuint32_t estride[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
                         estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

template <int D>
int launch_varlen_t(const VarlenArgs& a, cudaStream_t stream) {
  VarlenParams p{};
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.status = a.status;
  p.sinks = a.sinks;
  p.block_table = a.block_table;
  p.cu_q = a.cu_q;
  p.seq_lens = a.seq_lens;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.part_o = reinterpret_cast<float4*>(ws);
  ws += static_cast<size_t>(2 * a.sms) * kVlRows * D * sizeof(float);
  p.part_ml = reinterpret_cast<float2*>(ws);
  ws += static_cast<size_t>(2 * a.sms) * kVlRows * sizeof(float2);
  p.splits = reinterpret_cast<VarlenSplit*>(ws);
  p.B = a.B;
  p.T = a.T;
  p.Hq = a.Hq;
  p.group = a.Hq / a.Hkv;
  p.gsz = p.group < kBM ? p.group : kBM;
  p.hchunks = (p.group + p.gsz - 1) / p.gsz;
  p.tpt = kBM / p.gsz;
  p.units = a.Hkv * p.hchunks;
  p.tph = 64 / p.gsz;
  p.tma_out = 32 % p.gsz == 0;
  p.row_magic = (65536 + p.gsz - 1) / p.gsz;
  p.mask_kind = a.mask_kind;
  p.window = a.window;
  p.n_sink = a.n_sink;
  p.max_blocks = a.max_blocks_per_seq;
  p.block_size = a.block_size;
  p.num_blocks = a.num_blocks;
  p.max_seq_len = a.max_seq_len;
  p.scale_log2 = a.scale * kLog2e;
  p.budget = wait_budget_cycles();
  CUtensorMap tq, tqh, tk, tv, tvr, to;
  if (!encode_packed(&tq, a.q, D, a.Hq, a.T, p.gsz, p.tpt) ||
      !encode_packed(&tqh, a.q, D, a.Hq, a.T, p.gsz, 1) ||
      !encode_packed(&to, a.o, D, a.Hq, a.T, p.gsz, p.tma_out ? 32 / p.gsz : 1) ||
      !encode_pool(&tk, a.k_cache, D, a.Hkv, a.block_size, a.num_blocks, a.block_size) ||
      !encode_pool(&tv, a.v_cache, D, a.Hkv, a.block_size, a.num_blocks, a.block_size) ||
      !encode_pool(&tvr, a.v_cache, D, a.Hkv, a.block_size, a.num_blocks, 1))
    return ATTN_ERR_CUDA;
  constexpr int smem = VlCfg<D>::kAlloc;
  if (cudaFuncSetAttribute(prefill_varlen_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return ATTN_ERR_CUDA;
  prefill_varlen_kernel<D><<<a.sms, kVlThreads, smem, stream>>>(tq, tqh, tk, tv, tvr, to, p);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.sms, kJoinParts);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_varlen_join_kernel<D>, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

size_t varlen_workspace_bytes(int d, int sms) {
  return static_cast<size_t>(2 * sms) * kVlRows * (d * sizeof(float) + sizeof(float2)) + sms * sizeof(VarlenSplit);
}

int launch_prefill_varlen(const VarlenArgs& a, cudaStream_t stream) {
  return a.d == 128 ? launch_varlen_t<128>(a, stream) : launch_varlen_t<64>(a, stream);
}

}  // namespace attn
