// A key-value cache held in 4 bits: its layout, and how the kernels find a row's place.
//
// The pool is a sequence of pages of `page` tokens.  A page holds its heads one after the other, a head its
// tiles of 16 tokens, a tile
//   K codes   16 rows of D / 2 bytes, two codes a byte, the even feature in the low nibble
//   V codes   for each 4 tokens 16 pieces of 4 x D / 32 bytes: piece r holds D / 16 features of the 4 tokens, token
//             by token.  MXFP4, NVFP4: features r D / 16 ..; INT4: 64 g + 4 r .. + 3 of every 64-group g in turn
//   K scales  MXFP4, NVFP4: 16 rows of D / group bytes; INT4: for each group 16 fp16
//   V scales  for each group 16 bytes (INT4: 16 fp16)
// INT4 codes are stored as q + 8.  Scales are E8M0 bytes (MXFP4), fp16 (INT4), E4M3 bytes (NVFP4, tensor scale 1).
//
// Why so: with the tokens as rows of a 16x16x32 MFMA's A operand, lane (r, c) of a wave holds token r's features
// c D / 4 .. + D / 4 (INT4: 16 of each group), 8 or 16 bytes of a K row.  The scores then lie in registers as lane
// (query r, tokens 4 c .. 4 c + 3), which is the B operand of V^T P^T over 32 tokens if its k order is tokens 4 c .. of
// one tile and of the next; the A operand's lane (feature piece r, c) needs the same 4 tokens' piece r: 8 or 16
// bytes that lie together.  So a tile is four loads a lane, all of them whole lines, and neither K, V nor the
// probabilities pass through LDS.
#pragma once
#include "common.h"

namespace svdq {

constexpr int kKvTile = 16;
constexpr int64_t kKvMaxRows = int64_t(1) << 22;    // rows, batch x heads: workgroups of 256 in one grid dimension
constexpr int kKvMaxBatch = 16384;
constexpr int kKvMaxHeads = 256;
constexpr int kKvMaxPlanes = 4096;
constexpr int kKvMaxQHeads = 4096;
constexpr int64_t kKvMaxRowHeads = int64_t(1) << 27;   // rows x query heads of an attention call
constexpr int kKvMaxPage = 1024;
constexpr int kKvMaxAxes = 16;
constexpr int64_t kKvMaxPages = int64_t(1) << 30;
constexpr int64_t kKvMaxTokens = int64_t(1) << 30;  // of one sequence's table

__host__ __device__ constexpr int kv_group(int fmt) { return fmt == kFmtMXFP4 ? 32 : fmt == kFmtINT4 ? 64 : 16; }
// Scale bytes of one token's K or V.
__host__ __device__ constexpr int kv_scales(int fmt, int D) { return D / kv_group(fmt) * (fmt == kFmtINT4 ? 2 : 1); }
__host__ __device__ constexpr int kv_tile_bytes(int fmt, int D) { return kKvTile * (D + 2 * kv_scales(fmt, D)); }

// svdq_kv_compact in place.  Up to kKvCompactFew tokens a wave walks a sequence's tiles.  More are walked by a workgroup
// where the batch's heads and layers are workgroups enough or the walk is short, else they go through a workspace, `slab`
// heads at a time (0: none).  Half of L tokens kept, 8 heads of 128 in 4 layers, NVFP4, walk / workspace (us):
//   128 walks (4 sequences) L 500 13.1 / 20.3, L 5000 91.0 / 46.3    32 walks L 20000 341 / 47.6    1 walk L 100000 1702 / 19.2
//   256 walks L 500 12.4 / 22.6, L 5000 93.4 / 91.2                  512 walks L 5000 143 / 180
constexpr int kKvCompactFew = 64;
constexpr int kKvCompactShort = 384;
constexpr int64_t kKvCompactWalks = 256;
constexpr int64_t kKvCompactSpace = int64_t(64) << 20;     // bytes, unless one head's tokens are more
inline int64_t kv_compact_tiles(int64_t most) { return most / 16 + 2; }
inline int kv_compact_slab(int fmt, int D, int batch, int64_t all, int64_t most) {
  if (most <= kKvCompactShort || batch * all >= kKvCompactWalks) return 0;
  const int64_t slab = kKvCompactSpace / (batch * kv_compact_tiles(most) * kv_tile_bytes(fmt, D));
  return int(slab < 1 ? 1 : slab < all ? slab : all);
}

// How a call of svdq_kv_attention is cut: `rows` query rows of a K/V head (a sequence's tokens x the heads that share
// it) a workgroup, `jobs` such tiles at most; split: `ranges` workgroups a head share the units of all jobs.
//
// Rows by what a sequence has on average, and 128 where that fills them and there are 384 such tiles (then a wave's 32
// rows see all tokens, 4 waves side by side; with fewer, a tile's tokens are shared out).  us in a graph, MXFP4, 8 heads
// x 4 queries of 128, 16 sequences of 2000 tokens, new tokens each: 16 rows / 32 / 128
//   q 2 21.0 / 21.3 / 61    q 12 29.1 / 28.7 / 64    q 32 - / 41.5 / 66
// and 32 rows / 128 (rows a sequence, 128-row tiles in all):
//   128 sequences to 2000 tokens, 32 rows, 256 tiles 59.0 / 98.8     128 to 2000, 64 rows, 512 tiles 94.3 / 116
//   64 to 2000, 128 rows, 512 tiles 91.8 / 72.6                      32 to 4000, 128 rows, 256 tiles 90.1 / 111
//   48 to 2000, 132 rows, 392 tiles 82.5 / 89.9                      4 to 4000, 1536 rows, 384 tiles 126 / 134
//   4 of 4000, 1536 rows, 384 tiles 165 / 148
//   1 of 8192, 4096 rows, 256 tiles 220 / 215                        1 of 8192, 8192 rows, 512 tiles 372 / 265
// (INT4 alike: 512 tiles 141 / 108, 256 tiles 263 / 277.)
// That is by the average: the sweeps have sequences of alike rows.  A call that holds a prompt and single tokens has
// one form for both, and one of 128 rows is not split.  2048 rows on 8192 tokens beside n single ones, 8 heads x 4
// queries, MXFP4, in one call / in two (us): n 16, 63, 127 of 8192 tokens 411 / 284, 465 / 360, 657 / 458; of 65536
// 1638 / 475, 1832 / 1002, 2278 / 1793.
// Split where a table's tokens are many for the tiles there are: more than 16 a tile, at least 1024 (32 rows: 12 and
// 512), at most 4096, since a few long sequences among many short ones are not to be a workgroup's each.  Whole / split,
// 8 heads, ragged lengths (and all of one):
//   16 rows    8 tiles  512 8.0 / 10.0    1024 10.4 / 10.2    2048 15.1 / 10.5
//             64        1024 10.4 / 11.1 (10.6 / 11.2)        2048 15.3 / 13.0 (15.5 / 13.3)
//            128        2048 15.5 / 14.8 (15.9 / 17.8)        4096 24.7 / 18.4 (25.5 / 24.1)
//            256        4096 25.9 / 25.7 (26.9 / 34.9)        8192 44.2 / 36.2 (46.3 / 55.1)
//           2048        4096 122 / 125 (204 / 221)
//   32 rows    8        512 13.1 / 13.0    1024 17.9 / 13.2
//            128        1024 16.6 / 17.9 (17.1 / 19.4)        1536 21.3 / 20.1 (21.8 / 21.7)    2048 25.5 / 22.0
//            256        2048 26.5 / 27.7 (27.4 / 30.3)        4096 43.8 / 41.3 (45.1 / 44.0)    8192 76.3 / 56.2
//           1024        4096 95.5 / 94.6 (136 / 145)          8192 174 / 164 (280 / 286)
// INT4 alike.  The table's width counts, not the lengths, which are on the device: tables of the longest sequence /
// of 131072 tokens, 1 of 700 9.4 / 11.6, 64 to 300 8.8 / 14.6, 1024 to 300 56.6 / 75.2, 16 to 4000 16.6 / 16.3.
// Ranges: three workgroups a CU (1, 2, 3, 4 a CU: 64 x 8192 MXFP4 76.9 63.7 59.7 63.4, 3 x 131072 38.7 35.0 35.7
// 38.2, INT4 64 x 8192 89.3 75.7 69.0 72.7), two where a wave has 32 rows and registers for two.
constexpr int64_t kKvWhole = 1024;           // tokens up to which a job is one workgroup's, at least (32 rows: half)
constexpr int64_t kKvWholeMany = 4096;       // and at most
constexpr int64_t kKvWholeTile = 16;         // between them, for each tile (32 rows: 12)
struct KvPlan {
  int rows, jobs, ranges;
  bool split;
  size_t bytes;
};
inline KvPlan kv_plan(int D, int batch, int64_t M, int q_heads, int heads, int64_t places) {
  KvPlan p;
  const int64_t group = q_heads / heads, each = (M * group + batch - 1) / (batch > 0 ? batch : 1);
  auto tiles = [&](int rows) { return (M * group + rows - 1) / rows + batch; };
  p.rows = each <= 16 ? 16 : each >= 128 && M * q_heads >= 384 * 128 ? 128 : 32;
  const int64_t jobs = tiles(p.rows);
  p.jobs = int(jobs);
  const int64_t least = p.rows == 16 ? kKvWhole : kKvWhole / 2, each_tile = p.rows == 16 ? kKvWholeTile : 12;
  const int64_t whole = each_tile * heads * (jobs - batch > batch ? jobs - batch : batch);
  p.split = p.rows < 128 && places > (whole < least ? least : whole > kKvWholeMany ? kKvWholeMany : whole) &&
            jobs * (places / 128 + 1) <= INT32_MAX - 4096;     // units are counted in 32 bits
  p.ranges = p.split ? (256 * (p.rows == 16 ? 3 : 2) + heads - 1) / heads : 0;
  p.bytes = p.split ? align256(size_t(p.ranges) * heads * 2 * p.rows * (D + 2) * 4) : 0;
  return p;
}

// A cache and its sequences, as the kernels take them.  Places beyond a sequence's table or with a page outside
// [0, pages) hold no token: writes to them are dropped, reads find nothing.
struct KvCache {
  uint8_t* pool;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;               // rows of sequence b: cu[b] .. cu[b + 1]; NULL: one row each
  int64_t page_bytes, ldt;
  int32_t pages, cols, batch, M, heads, page_shift;   // a page has 1 << page_shift tiles

  __host__ __device__ __forceinline__ int capacity() const { return cols << (page_shift + 4); }
  // Tokens, first row and rows of sequence b.
  __device__ __forceinline__ void sequence(int b, int& len, int& row, int& rows) const {
    len = max(lens[b], 0);
    if (cu == nullptr) {
      row = b;
      rows = 1;
    } else {
      row = min(max(cu[b], 0), M);
      rows = max(min(cu[b + 1], M) - row, 0);
    }
  }
  // The page of a place (tile) of sequence b, -1 if there is none.
  __device__ __forceinline__ int page_of(int b, int tile) const {
    const int at = tile >> page_shift;
    if (tile < 0 || at >= cols) return -1;
    const int p = table[b * ldt + at];
    return p >= 0 && p < pages ? p : -1;
  }
};

// The sequence of row m, by the whole wave: the last b with cu[b] <= m; -1 behind the last row.
__device__ __forceinline__ int kv_sequence_of(const int32_t* cu, int batch, int m, int lane) {
  if (cu[batch] <= m || cu[0] > m) return -1;
  int lo = 0, n = batch;                                    // the answer is in lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 63) / 64, i = lane * step;
    const uint64_t le = __ballot(i < n && cu[lo + i] <= m);
    const int k = 63 - __builtin_clzll(le | 1);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// ---- 4-bit codes of K and V (tensor scale 1) ----

// Finite bf16 of x: NaN becomes 0, infinities (and what rounds to them) the largest of their sign.
__device__ __forceinline__ float kv_finite_bf16(float x) {
  const float b = bf_lo(f2bf(x));
  return x != x ? 0.f : fminf(fmaxf(b, -3.38953138925e38f), 3.38953138925e38f);
}

// Scale of a group whose largest magnitude is amax: its bits in the pool, and the number that x is divided by.
template <int FMT>
__device__ __forceinline__ uint32_t kv_scale(float amax, float& div) {
  if constexpr (FMT == kFmtMXFP4) {
    const uint32_t b = e8m0_of_amax(amax);
    div = scale_operand(b);
    return b;
  } else if constexpr (FMT == kFmtINT4) {
    const _Float16 s = static_cast<_Float16>(fminf(amax / 7.0f, 65504.0f));
    div = float(s);
    return __builtin_bit_cast(uint16_t, s);
  } else {
    const uint32_t b = e4m3_rne(amax / 6.0f);
    div = e4m3_value(b);
    return b;
  }
}
// The two values of a byte, given the scale's bits.
template <int FMT>
__device__ __forceinline__ v2f kv_decode(uint32_t byte, uint32_t scale) {
  if constexpr (FMT == kFmtMXFP4) {
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(byte, scale_operand(scale), 0);
  } else if constexpr (FMT == kFmtINT4) {
    const float s = float(__builtin_bit_cast(_Float16, uint16_t(scale)));
    return v2f{(int(byte & 15) - 8) * s, (int(byte >> 4) - 8) * s};
  } else {
    const v2f v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(byte, 1.0f, 0);
    const float s = e4m3_value(scale);
    return v2f{v.x * s, v.y * s};
  }
}

// Where, in a tile, the byte of features d, d + 1 (d even) of token t lies, and the scale of d's group.
template <int FMT, int D>
__device__ __forceinline__ int kv_k_code(int t, int d) { return t * (D / 2) + d / 2; }
template <int FMT, int D>
__device__ __forceinline__ int kv_v_code(int t, int d) {
  const int r = FMT == kFmtINT4 ? (d & 63) >> 2 : d / (D / 16);
  const int byte = FMT == kFmtINT4 ? (d >> 6) * 2 + ((d & 3) >> 1) : (d % (D / 16)) / 2;
  return 8 * D + ((t >> 2) * 16 + r) * (D / 8) + (t & 3) * (D / 32) + byte;
}
template <int FMT, int D>
__device__ __forceinline__ int kv_k_scale(int t, int g) {
  return 16 * D + (FMT == kFmtINT4 ? (g * 16 + t) * 2 : t * (D / kv_group(FMT)) + g);
}
template <int FMT, int D>
__device__ __forceinline__ int kv_v_scale(int t, int g) {
  return 16 * (D + kv_scales(FMT, D)) + (FMT == kFmtINT4 ? (g * 16 + t) * 2 : g * 16 + t);
}

}  // namespace svdq
