// Physical layouts of the packed weight blob and the activation workspace.
//
// Everything the GEMM reads is stored in the order one MFMA operand fragment is
// consumed, so each fragment is one fully coalesced 1 KiB load (64 lanes x 16 B)
// and no shuffling happens in the hot loop.
//
// Scaled FP4 MFMA (v_mfma_scale_f32_16x16x128_f8f6f4), per 16-row x 128-K tile:
//   lane L holds row (L % 16) and the 32-element K block (L / 16): 16 bytes,
//   element t of the block in byte t/2 (low nibble for even t).  The E8M0 scale
//   of that (row, block) is one byte of a per-lane 32-bit scale register.
//   Scale "superfragment" per 16 rows x 512 K: lane L's dword holds, in byte j,
//   the scale of row L%16, block L/16 of the 128-K step j.
// INT8 MFMA (v_mfma_i32_16x16x64_i8) for INT4: per 16-row x 128-K tile, lane L
//   holds row L%16 and, for both 64-element groups g of the tile, the 16 codes
//   at group offset (L/16)*16: bytes [8g, 8g+8) = 16 nibbles, two dwords of 8
//   codes each.  Inside a dword, code e (0..7) is in byte e%4, low nibble for
//   e < 4: masking the low (high) nibbles gives codes 0-3 (4-7) one per byte, in
//   order, which is what both the int8 expansion and the bf16 conversion of the
//   W4A16 kernel want.  Scales: per 128-K step and row, two fp16 (groups 0 and
//   1) in 4 bytes, rows contiguous.
// NVFP4-style (E2M1 codes, an E4M3 scale per 16): the codes use the MXFP4
//   fragment layout (lane L: row L%16, 32-element block L/16, 16 B).  Scales:
//   per 16-row tile and 128-K step, lane L's two E4M3 bytes (its block's halves
//   0 and 1) at 2 L, 128 B per tile-step.  The weight blob also holds the
//   residual's max |R| (fp32 bits), from which the tensor scale is derived.
// bf16 MFMA (v_mfma_f32_16x16x32_bf16) fragments for the low-rank branch: lane
//   L holds row/column L%16 and 8 consecutive K (rank) elements at (L/16)*8.
//
// Both operands use the same in-lane element order, so the product is the dot
// product over each K block regardless of that order.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace svdq {

constexpr int kTileRows = 256;     // rows of N (weights) and M (activations) are padded to this
constexpr int kFusedTileCols = 128; // narrowest output tile of a GEMM that quantizes its output
constexpr int kKStep = 128;        // K per MFMA step
constexpr int kKSuper = 512;       // K per scale superfragment; K must be a multiple
constexpr int kRankAlign = 32;     // rank padded to the bf16 MFMA K
constexpr int kFmtMXFP4 = 1;
constexpr int kFmtINT4 = 2;
constexpr int kFmtNVFP4 = 3;
constexpr float kNvfp4GlobalDiv = 2688.0f;   // E2M1 max 6 times E4M3 max 448

// svdq_moe: experts, choices per token, and (token, choice) pairs per pair of launches
// (longer calls run in parts).
constexpr int kMoeMaxE = 512;
constexpr int kMoeMaxTopK = 32;
constexpr int kMoeMaxPairs = 2048;
// The plan: 16 words for each unit of the down product, of which there are at most min(E, P) + P / 5
// < 922, and 32 that end it; from 64 KiB on 32 words for each of at most min(E, P) + P / 16 = 640
// blocks of the gate/up product.
constexpr size_t kMoePlanBytes = 65536 + 640 * 128;

// svdq_moe_route: one kernel, a workgroup per token, while one CU forms all of a token's logits about as
// fast as a second launch costs and each token has a CU; otherwise the logits are formed in tiles of
// 16 experts x 16 tokens, K split over route_splits workgroups while there are CUs for them, and a
// second kernel chooses.  The one kernel's time goes by the rounds of 64 experts that its waves take,
// K features each; up to 16 experts some waves have none, and K x E counts.  One kernel against two
// (us a call in a graph; at 1, 64 and 250 tokens):
//   E 64 (and 16, 32 within 10%)  K 1536  6.3 / 7.0   6.7 / 8.3   6.9 / 8.6
//                                 K 2560  8.3 / 7.8   8.7 / 9.3   9.0 / 11.1
//                                 K 3584 10.3 / 7.8  10.7 / 9.6  11.0 / 11.1
//   E 128                         K 1024  8.4 / 7.4   8.9 / 8.6   9.3 / 8.6
//                                 K 2048 12.5 / 8.2  12.9 / 9.1  13.4 / 10.6
//   E 8                           K 4096  6.8 / 7.5   7.3 / 8.5   7.7 / 8.7
//                                 K 8192 11.8 / 9.0  12.7 / 10.2 12.7 / 10.9
// and at 300 tokens (a second round of workgroups) E 64 K 1024 9.8 / 9.2, K 2560 15.4 / 12.1.
constexpr int64_t kRouteOneFeatures = 2560;
constexpr int64_t kRouteOneMacs = 32768;
constexpr int64_t kRouteOneTokens = 256;
__host__ __device__ inline bool route_one(int64_t M, int K, int E) {
  return M <= kRouteOneTokens && (int64_t((E + 63) / 64) * K <= kRouteOneFeatures || int64_t(E) * K <= kRouteOneMacs);
}
__host__ __device__ inline int route_splits(int64_t M, int K, int E) {
  const int64_t tiles = ((M + 15) / 16) * ((E + 15) / 16), z = 256 / (tiles > 0 ? tiles : 1);
  const int64_t most = (K + 511) / 512 < 8 ? (K + 511) / 512 : 8;      // a wave keeps four 32-K steps
  return int(z < 1 ? 1 : z < most ? z : most);
}

// Scale bytes per row: K/32 (E8M0 per 32, or fp16 per 64), K/16 for NVFP4 (E4M3 per 16).
__host__ __device__ inline size_t scale_row_bytes(int fmt, int K) { return fmt == kFmtNVFP4 ? K / 16 : K / 32; }
constexpr uint32_t kLamRangeBit = 1;   // weight flags: a lambda outside [2^-32, 2^32]
constexpr uint32_t kDivSlowBit = 2;    // weight flags: the two-operation division is not exact for some lambda

__host__ __device__ inline int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }
__host__ __device__ inline size_t align256(size_t a) { return (a + 255) & ~size_t(255); }

// svdq_moe's down product.  One kernel whose workgroups each take 16 rows of all tokens and add a
// token's pairs in LDS, or (moe_by_pairs) pairs' products to memory and a kernel that adds them: the
// first takes a CU about 170 cycles for each block of pairs (16 / planes of one expert) and 128 of F, in
// N / 16 workgroups over 256 CUs; the second shares a block's columns between two row tiles and fills
// the GPU whatever N is, for a launch more and the products' way through memory.  One kernel against two,
// whole calls (us, in a graph), by a CU's blocks x steps of 128:
//   80 (50 tokens, 2 of 8, 512 -> 2048) MXFP4 24.6 / 22.8, NVFP4 27.7 / 27.1; float32 112: 28.3 / 26.0, 29.5 / 30.3
//   112 (24, 4 of 16, 512 -> 4096)     MXFP4 25.0 / 23.7, NVFP4 27.4 / 28.5, INT4 26.6 / 27.2
//   160 (8, 2 of 8, 2048 -> 4096)      MXFP4 22.4 / 20.9, NVFP4 27.8 / 24.9, INT4 25.3 / 23.8
//   264 (6, 5 of 40, 1024 -> 2048)     MXFP4 26.1 / 24.7, NVFP4 32.5 / 29.5, INT4 31.9 / 30.6
//   320 (8, 4 of 16, 2048 -> 2048)     MXFP4 32.8 / 23.4, NVFP4 34.4 / 27.5, INT4 35.8 / 25.9
//   864 (400, 2 of 8, 1024 -> 4096)    MXFP4 134 / 78, NVFP4 144 / 100, INT4 142 / 97
constexpr int64_t kMoeDownSteps = 140;     // steps a CU from which the second is taken
__host__ __device__ inline bool moe_by_pairs(int64_t experts, int64_t pairs, int F, int N, int planes) {
  return (experts + pairs / (16 / planes)) * (F / kKStep) * ((N / 16 + 255) / 256) > kMoeDownSteps;
}
__host__ __device__ inline int64_t moe_part_pairs(int64_t M, int top_k) {
  const int64_t pairs = M * top_k;
  return pairs < 1 ? 1 : pairs < kMoeMaxPairs ? pairs : kMoeMaxPairs;
}
__host__ __device__ inline size_t moe_h_bytes(int64_t M, int top_k, int F) {
  return align256(size_t(moe_part_pairs(M, top_k)) * F * 6);
}
// The plan, h's planes and, where any number of experts up to the pairs' and either output may need them,
// the products.
__host__ __device__ inline size_t moe_workspace(int64_t M, int top_k, int F, int N) {
  const int64_t pairs = moe_part_pairs(M, top_k);
  const bool by_pairs = moe_by_pairs(pairs < kMoeMaxE ? pairs : kMoeMaxE, pairs, F, N, 3);
  return kMoePlanBytes + moe_h_bytes(M, top_k, F) + (by_pairs ? align256(size_t(pairs) * N * 4) : 0);
}

// svdq_linear_w4a16: which form a call takes.  Few tokens (`few`): one kernel that holds
// x_hat's S planes of all tokens in LDS beside the down projection's sums, when the columns of
// one 16-column MFMA hold them and they fit; it forms the down projection itself (`own_d`) for
// up to four tiles of 16 ranks, which a wave's registers hold beside its pipeline, and a small
// K x rank, since every workgroup then reads all of L1.  A prepare launch against an own down
// projection (us a call in a graph, one token, N 512 / 2048 / 4096 / 8192 / 16384, NVFP4):
//   L1 256 KB (K 2048 r 64)  10.8 11.1 12.5 14.0 17.6  /   8.3  8.4  9.2 12.1 15.0
//   L1 448 KB (K 3584 r 64)  12.3 14.2 14.9 16.5 21.9  /  10.9 11.3 13.8 16.0 20.8
//   L1 512 KB (K 8192 r 32)  15.4 17.5 18.2 22.1 30.5  /  13.1 16.1 16.8 20.8 29.6
//   L1 576 KB (K 4608 r 64)  13.2 15.3 15.8 18.1 24.4  /  12.6 14.9 16.0 18.6 23.8
//   L1 768 KB (K 6144 r 64)  14.5 16.7 17.1 20.3 27.2  /  14.8 18.1 18.7 21.7 27.9
// (MXFP4, INT4, 5 tokens with float32 output and 8 tokens alike.)
constexpr int kFewWaves = 8;
constexpr int kFewMaxRank = 64;
constexpr int kFewMaxL1Bytes = 524288;
constexpr int64_t kFewLds = 155648;    // of 160 KiB
// Workgroups at most: one a CU where each forms the down projection or only one fits a CU's LDS, else two.
// 256 against 512 (us a call in a graph): own down projection, one token, 2048 -> 8192 rank 32, MXFP4
// 9.1 / 10.1, INT4 9.5 / 13.3, NVFP4 9.9 / 10.7, -> 24576 13.8 / 14.2, 14.8 / 19.0, 15.5 / 15.8; 5
// tokens float32, 2560 -> 16384, 115 KB of LDS, prepared, MXFP4 21.0 / 26.6; rank 0, one token, 2048 ->
// 8208 MXFP4 6.7 / 6.1, -> 10240 6.8 / 7.4, -> 24576 10.2 / 9.2; prepared, 2048 -> 16384 15.7 / 13.9.
constexpr int kFewGroups = 256;
__host__ __device__ inline int few_row_bytes(int K) { return K * 2 + 16; }   // 16 skews the banks

struct W4A16Plan {
  bool few, own_d;
  int groups;
  int64_t lds;
};
__host__ __device__ inline W4A16Plan w4a16_plan(int K, int64_t r_pad, int64_t M, int S) {
  W4A16Plan p;
  p.own_d = r_pad <= kFewMaxRank && K * r_pad * 2 <= kFewMaxL1Bytes;
  // x_hat, the down projection, and one space for its waves' sums and then for the tiles' (two buffers)
  const int64_t sums = p.own_d && r_pad > 32 ? kFewWaves * r_pad / 16 * 1024 : 2 * kFewWaves * 1024;
  p.lds = S * M * few_row_bytes(K) + M * r_pad * 4 + sums;
  p.few = M <= 16 / S && p.lds <= kFewLds;
  p.groups = (p.own_d && r_pad) || p.lds > 81920 ? kFewGroups : 2 * kFewGroups;
  return p;
}

// More tokens: x_hat's planes go to memory in the order of the MFMA's B operands, groups of `Mg`
// tokens in NB blocks of 16 columns (column p Mg + t: plane p of token t), and each workgroup takes
// T row tiles, reading a group's columns once for them.  When that leaves CUs without a workgroup,
// T is halved if the columns read altogether stay within kWideTraffic; otherwise K is split over Z
// workgroups, whose sums a last kernel adds, while a wave keeps two 128-K steps.
constexpr int kWideWaves = 8;
constexpr int kWideBlocks = 6;         // at most
constexpr int kWideGroups = 256;       // one workgroup a CU
constexpr int64_t kWideTraffic = 450000000;   // sweep at M 16..48: 1e8 25.3, 2e8 20.1, 4.5e8 18.6 us at 48 x 4096 -> 4096;
                                               // 1e9 slower where the columns are many (33 x 12288 -> 4096: 26.9 -> 31.2)

struct W4A16Wide {
  int64_t groups, Mg;
  int NB, T, Z;
};
__host__ __device__ inline W4A16Wide w4a16_wide(int fmt, int K, int N, int64_t M, int S) {
  W4A16Wide p;
  const int64_t most = kWideBlocks * 16 / S, tiles = N / 16;
  p.groups = (M + most - 1) / most;
  p.Mg = (M + p.groups - 1) / p.groups;
  const int nb = int((S * p.Mg + 15) / 16);
  p.NB = nb <= 2 ? 2 : nb;
  p.T = fmt == kFmtINT4 && p.NB > 3 ? 2 : 4;       // registers: INT4 holds a group's sums beside the accumulators
  const int64_t slab = int64_t(p.NB) * K * 32;     // a group's columns
  while (p.T > 1 && (tiles + p.T - 1) / p.T * p.groups < kWideGroups &&
         (tiles + p.T / 2 - 1) / (p.T / 2) * p.groups * slab <= kWideTraffic)
    p.T /= 2;
  const int64_t wgs = (tiles + p.T - 1) / p.T * p.groups;
  const int zmax = K / kKStep / (2 * kWideWaves);
  const int64_t z = wgs * 2 <= kWideGroups ? kWideGroups / wgs : 1;
  p.Z = int(z < 1 || zmax < 1 ? 1 : z < zmax ? z : zmax);
  return p;
}

// Its workspace: x_hat's planes, the down projection's partial sums (one per 512 of K) and the
// sums of the Z parts; nothing where the one kernel does all, whatever the output type.
struct W4A16Layout {
  size_t planes, part, zsum, total;
};
__host__ __device__ inline W4A16Layout w4a16_layout(int fmt, int K, int N, int rank, int64_t M) {
  const int64_t rows = M > 0 ? M : 1, r_pad = round_up(rank, kRankAlign);
  W4A16Layout l{0, 0, 0, 0};
  size_t part = 0;
  for (int S = 2; S <= 3; ++S) {
    const W4A16Plan few = w4a16_plan(K, r_pad, rows, S);
    const W4A16Wide w = w4a16_wide(fmt, K, N, rows, S);
    const size_t planes = few.few ? 0 : align256(size_t(w.groups) * w.NB * K * 32);
    const size_t zsum = few.few || w.Z == 1 ? 0 : align256(size_t(w.Z) * rows * N * 4);
    if (!few.few || !few.own_d) part = align256(size_t(K / kKSuper) * rows * r_pad * 4);
    if (planes > l.part) l.part = planes;
    if (zsum > l.total) l.total = zsum;
  }
  l.zsum = l.part + part;
  l.total += l.zsum;
  return l;
}

struct WeightLayout {
  int64_t N_pad, r_pad;
  size_t codes, scales, L1, L2, lam, rlam, rlo, bias, flags, amax, total;
};

struct ActLayout {
  int64_t M_pad, r_pad;
  int kr, splits;                  // activation kernel: K per workgroup, K splits (K / kr)
  size_t codes, scales, D, part, total;
};

// Codes: N_pad x K/2 bytes.  Scales: N_pad x scale_row_bytes(fmt, K) bytes.
// L1: K x r_pad bf16 (B fragments of the down projection).  L2: N_pad x r_pad bf16
// (A fragments of the up projection).  lambda, r = RN(1/lambda) and the correction
// rl = RN((1 - r lambda) r): fp32[K] each.  bias: bf16[N_pad].  flags: uint32
// (kLamRangeBit, kDivSlowBit).  amax: the NVFP4 residual's max |R| as fp32 bits.
__host__ __device__ inline WeightLayout weight_layout(int fmt, int K, int N, int rank) {
  WeightLayout w;
  w.N_pad = round_up(N, kTileRows);
  w.r_pad = round_up(rank, kRankAlign);
  size_t o = 0;
  w.codes = o;  o = align256(o + size_t(w.N_pad) * K / 2);
  w.scales = o; o = align256(o + size_t(w.N_pad) * scale_row_bytes(fmt, K));
  w.L1 = o;     o = align256(o + size_t(K) * w.r_pad * 2);
  w.L2 = o;     o = align256(o + size_t(w.N_pad) * w.r_pad * 2);
  w.lam = o;    o = align256(o + size_t(K) * 4);
  w.rlam = o;   o = align256(o + size_t(K) * 4);
  w.rlo = o;    o = align256(o + size_t(K) * 4);
  w.bias = o;   o = align256(o + size_t(w.N_pad) * 2);
  w.flags = o;  o = align256(o + 4);
  w.amax = o;   o = align256(o + 4);
  w.total = o;
  return w;
}

constexpr int kActRowTiles = 8;        // 16-row tiles (one per wave) per activation workgroup
constexpr int kActLdsBytes = 81920;    // LDS for one workgroup's lambda, r, rl and L1 fragments (two fit a CU)
constexpr int kActMinWorkgroups = 384; // fewer leave CUs idle

// Work split of the activation kernel: a workgroup takes kActRowTiles 16-row
// tiles and one K range of kr (its lambda, r, rl and L1 fragments staged in
// LDS, kr * (12 + 2 r_pad) bytes).  kr is the largest power of two dividing K
// within the LDS budget, halved (down to 128) while the grid has fewer than
// kActMinWorkgroups workgroups.  With more than one split, each workgroup
// writes an fp32 partial of the down projection, summed in split order by a
// second small kernel.
__host__ __device__ inline void act_split(int K, int r_pad, int64_t M_pad, int* kr_out, int* splits) {
  const int64_t groups = M_pad / (16 * kActRowTiles);
  int kr = 64;
  for (int c = 4096; c >= 64; c /= 2)
    if (K % c == 0 && int64_t(c) * (12 + 2 * r_pad) <= kActLdsBytes) {
      kr = c;
      break;
    }
  while (kr > 128 && groups * (K / kr) < kActMinWorkgroups) kr /= 2;
  *kr_out = kr;
  *splits = K / kr;
}

// Codes: M_pad x K/2.  Scales: M_pad x scale_row_bytes(fmt, K).  D: M_pad x r_pad x {hi, lo} bf16.
// part: fp32 partial down projections, P x M_pad x r_pad, for the larger of the two
// producers: the activation kernel's K splits (when it splits K), and the GEMM of a
// previous layer that quantizes its output for this layer (one partial per tile
// column of that output: K / 128 of them with 128-wide tiles, K / 256 with 256-wide).
__host__ __device__ inline ActLayout act_layout(int fmt, int K, int rank, int64_t M) {
  ActLayout a;
  a.M_pad = round_up(M > 0 ? M : 1, kTileRows);
  a.r_pad = round_up(rank, kRankAlign);
  act_split(K, int(a.r_pad), a.M_pad, &a.kr, &a.splits);
  size_t o = 0;
  a.codes = o;  o = align256(o + size_t(a.M_pad) * K / 2);
  a.scales = o; o = align256(o + size_t(a.M_pad) * scale_row_bytes(fmt, K));
  a.D = o;      o = align256(o + size_t(a.M_pad) * a.r_pad * 4);
  const int nparts = (a.splits > 1 && a.splits > K / kFusedTileCols) ? a.splits : K / kFusedTileCols;
  a.part = o;   o = align256(o + size_t(nparts) * a.M_pad * a.r_pad * 4);
  a.total = o;
  return a;
}

// Bytes of the workspace that the two launches of one layer touch: codes,
// scales, D and the activation kernel's K-split partials (without the room a
// fused producer's partials take).
__host__ __device__ inline size_t act_linear_bytes(const ActLayout& a) {
  return a.part + (a.splits > 1 ? size_t(a.splits) * a.M_pad * a.r_pad * 4 : 0);
}

// ---- codes: byte offset of the 16-byte lane chunk of tile (rt, ks), lane L ----
__host__ __device__ inline size_t code_chunk(int64_t rt, int ks, int K, int L) {
  return (size_t(rt) * (K / kKStep) + ks) * 1024 + size_t(L) * 16;
}

// Canonical (row, k) -> (byte offset, high-nibble?) in the code section.
__host__ __device__ inline size_t code_byte(int fmt, int64_t row, int k, int K, int* hi) {
  const int64_t rt = row / 16;
  const int r = int(row % 16);
  const int ks = k / kKStep;
  const int kk = k % kKStep;
  if (fmt != kFmtINT4) {                         // MXFP4 and NVFP4
    const int blk = kk / 32, t = kk % 32;
    *hi = t & 1;
    return code_chunk(rt, ks, K, blk * 16 + r) + t / 2;
  }
  const int g = kk / 64, o = kk % 64, c = o / 16, t = o % 16, e = t % 8;
  *hi = e >> 2;
  return code_chunk(rt, ks, K, c * 16 + r) + g * 8 + (t / 8) * 4 + (e & 3);
}

// ---- scales ----
// MXFP4: byte offset of the scale of (row, 32-block index kb) (kb = k / 32).
__host__ __device__ inline size_t mx_scale_byte(int64_t row, int kb, int K) {
  const int64_t rt = row / 16;
  const int r = int(row % 16);
  const int ks = kb / 4, blk = kb % 4;          // 128-K step and block within it
  const int sup = ks / 4, j = ks % 4;           // superfragment and byte within the dword
  return ((size_t(rt) * (K / kKSuper) + sup) * 64 + (blk * 16 + r)) * 4 + j;
}
// NVFP4: byte offset of the E4M3 scale of (row, 16-group index kg) (kg = k / 16).
__host__ __device__ inline size_t nv_scale_byte(int64_t row, int kg, int K) {
  const int64_t rt = row / 16;
  const int r = int(row % 16);
  const int ks = kg / 8, blk = (kg / 2) % 4, half = kg % 2;
  return ((size_t(rt) * (K / kKStep) + ks) * 64 + (blk * 16 + r)) * 2 + half;
}
// INT4: byte offset of the fp16 scale of (row, 64-group index g) with rows padded to rows_pad.
__host__ __device__ inline size_t i4_scale_byte(int64_t row, int g, int64_t rows_pad) {
  const int ks = g / 2, h = g % 2;
  return ((size_t(ks) * rows_pad + row) * 2 + h) * 2;
}

// ---- low-rank fragments (bf16 element offsets) ----
// L1 (K x r_pad): B fragment of the down projection, tile (k32, i16), lane L, element e:
//   k = k32*32 + (L/16)*8 + e, i = i16*16 + L%16.
__host__ __device__ inline size_t l1_elem(int k, int i, int r_pad) {
  const int k32 = k / 32, kk = k % 32, i16 = i / 16, L = (kk / 8) * 16 + (i % 16), e = kk % 8;
  return ((size_t(k32) * (r_pad / 16) + i16) * 64 + L) * 8 + e;
}
// L2 (N_pad x r_pad): A fragment of the up projection, tile (n16, r32), lane L, element e:
//   n = n16*16 + L%16, rank = r32*32 + (L/16)*8 + e.
__host__ __device__ inline size_t l2_elem(int64_t n, int rk, int r_pad) {
  const int64_t n16 = n / 16;
  const int r32 = rk / 32, kk = rk % 32, L = (kk / 8) * 16 + int(n % 16), e = kk % 8;
  return ((size_t(n16) * (r_pad / 32) + r32) * 64 + L) * 8 + e;
}
// D (M_pad x r_pad, hi/lo bf16): B fragment of the up projection, tile (m16, r32), part h.
__host__ __device__ inline size_t d_elem(int64_t m, int rk, int h, int r_pad) {
  const int64_t m16 = m / 16;
  const int r32 = rk / 32, kk = rk % 32, L = (kk / 8) * 16 + int(m % 16), e = kk % 8;
  return (((size_t(m16) * (r_pad / 32) + r32) * 2 + h) * 64 + L) * 8 + e;
}

}  // namespace svdq
