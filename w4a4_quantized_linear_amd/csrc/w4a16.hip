// A packed layer applied to 16-bit activations (few tokens):
//
//   Y[m, n] = act( sum_k deQ(R)[n, k] x_hat[m, k] + sum_i L2[i, n] D[m, i] + b[n] ),
//   x_hat = fp32(X / lambda),  D = X_hat L1.
//
// What is to be read is the weights, so few tokens are bound by bytes in principle and by
// latency in practice: 4096 x 4096 INT4 is 9 MB, 1.5 us at the rate of large reads, and a launch that
// only reads 10 MB takes 6.0 us, one of 25 MB 7.8.  Two forms (layout.h, w4a16_plan):
//   w4a16_few_kernel   all tokens' planes are columns of one MFMA: one launch.
//   w4a16_wide_kernel  more: w4a16_prepare_kernel divides by lambda, splits x_hat into bf16
//                      planes (w4frag.h) in the order of the B operands and forms D's partial
//                      sums, one per 512 of K; the product; w4a16_join_kernel adds parts of K.
#include <hip/hip_runtime.h>

#include "svdq.h"
#include "w4frag.h"

namespace svdq {

struct W4A16LinearArgs {
  const uint8_t* wblob;
  size_t w_codes, w_scales, w_L1, w_L2, w_lam, w_bias, w_amax;
  const uint16_t* X;
  uint4* planes;           // groups x K / 128 x 4 x NB x 64 B operands (null: not wanted)
  float* part;             // K / 512 x M x r_pad
  float* zsum;             // Z x M x N
  void* Y;
  int64_t ldx, ldy, M, N_pad;
  int K, r_pad;            // r_pad 0: no low-rank branch
  uint32_t epi;
  int N, NB, Z, int4;
  int64_t Mg, groups;
};

constexpr int kPrepWaves = 8;          // 64 K each
constexpr int kPrepTiles = 4;          // 16-rank tiles whose sums meet in LDS at a time

// One workgroup: 16 tokens, 512 of K.  4.8 us for 8 tokens of 4096, 6.1 us for 33 of 12288: the
// latency of one dependent chain (X and lambda, the division, the MFMAs, the exchange), not bytes.
template <int S>
__global__ void __launch_bounds__(512) w4a16_prepare_kernel(W4A16LinearArgs a) {
  __shared__ v4f red[kPrepWaves][kPrepTiles][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tl = lane & 15, c = lane >> 4;
  const int RT = a.r_pad / 16;
  const int k0 = blockIdx.x * kKSuper + w * 64;
  const float* lam = reinterpret_cast<const float*>(a.wblob + a.w_lam);
  const uint4* L1f = reinterpret_cast<const uint4*>(a.wblob + a.w_L1);
  for (int64_t m0 = int64_t(blockIdx.y) * 16; m0 < a.M; m0 += int64_t(gridDim.y) * 16) {
    const int64_t m = m0 + tl < a.M ? m0 + tl : a.M - 1;
    uint4 p[2][S], l1f[2][2];                              // the first two rank tiles' L1 fragments, ahead
    if (RT) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) l1f[s][i] = L1f[(size_t(k0 / 32 + s) * RT + i) * 64 + lane];
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = k0 + s * 32 + c * 8;
      float v[8];
      unpack_bf8(*reinterpret_cast<const uint4*>(a.X + m * a.ldx + k), v);
      const float4 l0 = *reinterpret_cast<const float4*>(lam + k), l1 = *reinterpret_cast<const float4*>(lam + k + 4);
      const float l[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] / l[e];       // IEEE: x_hat is this quotient by definition
      split_planes<S>(v, p[s]);
      if (a.planes && m0 + tl < a.M) {
        // lane group and MFMA that these 8 K elements belong to (k_of)
        const int kk = k & 127, kc = a.int4 ? (kk & 63) >> 4 : kk >> 5;
        const int u = a.int4 ? ((kk >> 6) << 1) + ((kk >> 3) & 1) : (kk >> 3) & 3;
        uint4* const at = a.planes + (((m / a.Mg) * (a.K / kKStep) + k / kKStep) * 4 + u) * a.NB * 64 + kc * 16;
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const int col = int(i * a.Mg + m % a.Mg);
          at[(col >> 4) * 64 + (col & 15)] = p[s][i];
        }
      }
    }
    for (int i0 = 0; i0 < RT; i0 += kPrepTiles) {
      const int tiles = RT - i0 < kPrepTiles ? RT - i0 : kPrepTiles;
#pragma unroll
      for (int i = 0; i < kPrepTiles; ++i) {
        if (i >= tiles) break;
        v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint4 l1 = i < 2 && i0 == 0 ? l1f[s][i & 1] : L1f[(size_t(k0 / 32 + s) * RT + i0 + i) * 64 + lane];
#pragma unroll
          for (int q = 0; q < S; ++q) acc = mfma_bf16(p[s][q], l1, acc);
        }
        red[w][i][lane] = acc;
      }
      __syncthreads();
      // lane: rank tl of tile i, tokens 4 c .. 4 c + 3; the waves' sums in order
      if (w < tiles) {
        v4f d = red[0][w][lane];
#pragma unroll
        for (int v = 1; v < kPrepWaves; ++v) d += red[v][w][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t t = m0 + c * 4 + e;
          if (t < a.M) a.part[(int64_t(blockIdx.x) * a.M + t) * a.r_pad + (i0 + w) * 16 + tl] = d[e];
        }
      }
      __syncthreads();
    }
  }
}

// Y[m, row .. row + 3] = act(y + b)
__device__ __forceinline__ void w4a16_store(const W4A16LinearArgs& a, int64_t m, int64_t row, v4f y, bool f32) {
  if (a.epi & SVDQ_EPI_BIAS) {
    const uint2 b = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(a.wblob + a.w_bias) + row);
    y += v4f{bf_lo(b.x), bf_hi(b.x), bf_lo(b.y), bf_hi(b.y)};
  }
  if (a.epi & SVDQ_EPI_GELU) {
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = gelu_erf(y[e]);
  }
  if (f32)
    *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.Y) + m * a.ldy + row) = y;
  else
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.Y) + m * a.ldy + row) =
        make_uint2(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]));
}

// Few tokens, one launch: all S planes of the M tokens are columns of one MFMA.
//
// A workgroup of eight waves computes x_hat of all tokens once into LDS (planes x tokens rows of
// K bf16), forms D = X_hat L1 from it where the rank allows (OWN_D; otherwise it sums
// w4a16_prepare_kernel's partial sums), and then takes row tiles blockIdx.x, + gridDim.x, ...:
// wave w the 128-K steps w, w + 8, ..., kFewDepth steps of codes in flight, the pipeline running
// on from tile to tile.  The waves' sums meet in LDS (two buffers, so one barrier a tile); one
// wave, another each tile, adds them and the up projection and writes the tile.
//
// Bound by start-up and latency (6.2 us for 1 x 1024 -> 1024 MXFP4 rank 16) and by the down projection,
// whose L1 every workgroup reads: 9.5 us for 1 x 4096 -> 4096 INT4 rank 32 (9.9 MB of weights; 88 MB of
// L2 reads, 67 of them L1's; in a graph 11.1 us, without the branch 6.5), 13.2 us for 5 x 2048 -> 8208
// NVFP4 rank 64 (11 MB; 64 MB).  The two launches that this replaces (x_hat and D prepared, then
// streamed) took 12.7 us at 1 x 4096 -> 4096.
constexpr int kFewDepth = 4;

// RT: 16-rank tiles of OWN_D (0: no low-rank branch, or its sums are given)
template <int FMT, int S, int RT>
__global__ void __launch_bounds__(512) w4a16_few_kernel(W4A16LinearArgs a, int tiles) {
  constexpr int TPB = tokens_per_block(S);
  constexpr int W = kFewWaves;
  extern __shared__ uint4 lds[];
  const int tid = threadIdx.x;
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tl = lane & 15, c = lane >> 4;
  const int M = int(a.M), KS = a.K / kKStep, row_b = few_row_bytes(a.K);
  const int n = KS > w ? (KS - w + W - 1) / W : 0;         // this wave's steps of each tile
  uint8_t* const xl = reinterpret_cast<uint8_t*>(lds);
  float* const dsum = reinterpret_cast<float*>(xl + S * M * row_b);              // M x r_pad
  v4f* const red = reinterpret_cast<v4f*>(dsum + M * a.r_pad);                   // 2 x W x 64; first W x RT x 64

  const W4Rows<FMT> rows(a.wblob + a.w_codes, a.wblob + a.w_scales, a.K, a.N_pad);
  int lt = blockIdx.x, li = 0;                             // the next step to load
  W4Stage<FMT> st[kFewDepth];
  auto load = [&](W4Stage<FMT>& s) {
    rows.load(uint32_t(lt), uint32_t(w + li * W), lt < tiles, lane, s);
    if (++li >= n) {
      li = 0;
      lt += gridDim.x;
    }
  };
  if (n > 0) {
#pragma unroll
    for (int j = 0; j < kFewDepth; ++j) {
      load(st[j]);
      keep_order();
    }
  }
  const float gs = w4_tensor_scale<FMT>(a.wblob + a.w_amax);
  // L1 fragments in batches of U 32-K steps (the wave's: w, w + 8, ...), two batches in flight
  constexpr int NF = 8, U = RT ? NF / RT : 1;
  const int batches = (a.K / (32 * W) + U - 1) / U;
  uint4 f[2][NF];
  auto load_l1 = [&](int b, uint4 (&q)[NF]) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int it = b * U + j;
      const bool there = it < a.K / (32 * W);
      const __amdgpu_buffer_rsrc_t r = make_rsrc(a.wblob + a.w_L1, there ? uint32_t(a.K) * a.r_pad * 2 : 0);
#pragma unroll
      for (int i = 0; i < RT; ++i) q[j * RT + i] = buffer_load16(r, uint32_t(lane) * 16, ((it * W + w) * RT + i) * 1024);
    }
  };
  if (RT) load_l1(0, f[0]);

  // x_hat: IEEE division, as it is defined.  Narrow K: the threads take several tokens at a time.
  const float* lam = reinterpret_cast<const float*>(a.wblob + a.w_lam);
  const int kp = a.K / 8, G = kp < 512 ? 512 / kp : 1;
  const int mg = kp < 512 ? tid / kp : 0;
  for (int q = kp < 512 ? tid % kp : tid; q < kp && mg < G; q += kp < 512 ? kp : 512) {
    const int k = q * 8;
    const float4 l0 = *reinterpret_cast<const float4*>(lam + k), l1 = *reinterpret_cast<const float4*>(lam + k + 4);
    const float l[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w};
    for (int m0 = mg; m0 < M; m0 += 4 * G) {
      uint4 xr[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + j * G < M ? m0 + j * G : m0;
        xr[j] = *reinterpret_cast<const uint4*>(a.X + m * a.ldx + k);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + j * G;
        if (m < M) {
          float v[8];
          unpack_bf8(xr[j], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = v[e] / l[e];
          uint4 p[S];
          split_planes<S>(v, p);
#pragma unroll
          for (int i = 0; i < S; ++i) *reinterpret_cast<uint4*>(xl + (i * M + m) * row_b + k * 2) = p[i];
        }
      }
    }
  }
  lds_barrier();
  // this lane's column: plane pl of token t (columns past the last repeat it; they are independent)
  const int t = tl % TPB < M ? tl % TPB : M - 1, pl = tl / TPB < S ? tl / TPB : S - 1;
  const uint8_t* const xp = xl + (pl * M + t) * row_b;

  if constexpr (RT != 0) {
    // rows of the MFMA: the columns above
    v4f d[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) d[i] = v4f{0.f, 0.f, 0.f, 0.f};
    auto add_l1 = [&](int b, const uint4 (&q)[NF]) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int it = b * U + j, k32 = it < a.K / (32 * W) ? it * W + w : w;      // beyond K: zero fragments
        const uint4 x = *reinterpret_cast<const uint4*>(xp + (k32 * 32 + c * 8) * 2);
#pragma unroll
        for (int i = 0; i < RT; ++i) d[i] = mfma_bf16(x, q[j * RT + i], d[i]);
      }
    };
    for (int b = 0; b < batches; b += 2) {
      load_l1(b + 1, f[1]);
      add_l1(b, f[0]);
      load_l1(b + 2, f[0]);
      add_l1(b + 1, f[1]);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) red[(w * RT + i) * 64 + lane] = d[i];
    lds_barrier();
    const float* dp = reinterpret_cast<const float*>(red);
    for (int i = tid; i < M * RT * 16; i += 512) {
      const int m = i / (RT * 16), r = i % (RT * 16);
      float v = 0.f;
#pragma unroll
      for (int p = 0; p < S; ++p) {
        const int row = p * TPB + m, at = ((r >> 4) * 64 + (row >> 2) * 16 + (r & 15)) * 4 + (row & 3);
#pragma unroll
        for (int q = 0; q < W; ++q) v += dp[q * RT * 256 + at];
      }
      dsum[i] = v;
    }
    lds_barrier();                                         // red is the tiles' from here
  } else {
    for (int i = tid; i < M * a.r_pad; i += 512) {
      float v = 0.f;
      for (int q = 0; q < a.K / kKSuper; ++q) v += a.part[int64_t(q) * M * a.r_pad + i];
      dsum[i] = v;
    }
  }

  // tile rt: the waves' sums `acc` to LDS; wave turn % 8 finishes it, its L2 fragments and bias
  // loaded one tile ahead (by the other waves through buffers of no bytes, see W4Rows)
  int turn = 0;
  uint4 l2f[RT ? RT / 2 : 1];
  uint2 bias = make_uint2(0u, 0u);
  auto load_end = [&](int rt, int turn) {
    const bool mine = w == (turn & (W - 1)) && rt < tiles;
    const __amdgpu_buffer_rsrc_t rl = make_rsrc(a.wblob + a.w_L2, mine ? uint32_t(a.N_pad) * a.r_pad * 2 : 0);
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.wblob + a.w_bias, mine && (a.epi & SVDQ_EPI_BIAS) ? uint32_t(a.N_pad) * 2 : 0);
#pragma unroll
    for (int i = 0; i < RT / 2; ++i) l2f[i] = buffer_load16(rl, uint32_t(lane) * 16, (rt * (RT / 2) + i) * 1024);
    bias = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rb, uint32_t(c) * 8, rt * 32, 0));
  };
  load_end(blockIdx.x, 0);
  auto finish = [&](int rt, v4f acc) {
    red[((turn & 1) * W + w) * 64 + lane] = acc;
    lds_barrier();
    if (w == (turn & (W - 1))) {
      v4f y = {0.f, 0.f, 0.f, 0.f};
      const int64_t row = int64_t(rt) * 16 + c * 4;
      // up projection of token tl (the MFMA's columns), after NVFP4's tensor scale
      v4f z = {0.f, 0.f, 0.f, 0.f};
      auto add_l2 = [&](int r32, const uint4& l2) {
        float dv[8];
        const float4* dq = reinterpret_cast<const float4*>(dsum + (tl < M ? tl : M - 1) * a.r_pad + r32 * 32 + c * 8);
        const float4 d0 = dq[0], d1 = dq[1];
        dv[0] = d0.x; dv[1] = d0.y; dv[2] = d0.z; dv[3] = d0.w; dv[4] = d1.x; dv[5] = d1.y; dv[6] = d1.z; dv[7] = d1.w;
        uint4 p[3];                                        // D to fp32's rounding for any number of tokens
        split_planes<3>(dv, p);
#pragma unroll
        for (int i = 0; i < 3; ++i) z = mfma_bf16(l2, p[i], z);
      };
      if constexpr (RT != 0) {
#pragma unroll
        for (int i = 0; i < RT / 2; ++i) add_l2(i, l2f[i]);
      } else {
        const uint4* L2f = reinterpret_cast<const uint4*>(a.wblob + a.w_L2) + size_t(rt) * (a.r_pad / 32) * 64 + lane;
        for (int r32 = 0; r32 < a.r_pad / 32; ++r32) add_l2(r32, L2f[r32 * 64]);
      }
      if (tl < M) {
#pragma unroll
        for (int v = 0; v < W; ++v)
#pragma unroll
          for (int i = 0; i < S; ++i) y += red[((turn & 1) * W + v) * 64 + lane + i * TPB];
        if (FMT == kFmtNVFP4) y *= gs;
        y += z;
        y += v4f{bf_lo(bias.x), bf_hi(bias.x), bf_lo(bias.y), bf_hi(bias.y)};
        if (a.epi & SVDQ_EPI_GELU) {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = gelu_erf(y[e]);
        }
        const int64_t o = tl * a.ldy + row;
        if (S == 3)                                        // three planes: float32 output
          *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.Y) + o) = y;
        else
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.Y) + o) =
              make_uint2(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]));
      }
    }
    ++turn;
    load_end(rt + gridDim.x, turn);
  };

  const v4f zero = {0.f, 0.f, 0.f, 0.f};
  if (n == 0) {
    for (int rt = blockIdx.x; rt < tiles; rt += gridDim.x) finish(rt, zero);
    return;
  }
  int rt = blockIdx.x, i = 0;
  v4f acc = zero;
  for (;;) {
#pragma unroll
    for (int j = 0; j < kFewDepth; ++j) {
      const int ks = w + i * W;
      uint4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const uint4*>(xp + (ks * kKStep + k_of<FMT>(c, u)) * 2);
      w4_step<FMT>(st[j], ks, x, acc);
      load(st[j]);
      keep_order();
      if (++i == n) {
        finish(rt, acc);
        acc = zero;
        i = 0;
        rt += gridDim.x;
        if (rt >= tiles) return;
      }
    }
  }
}

// More tokens.  A workgroup takes T row tiles, one group of tokens and one of Z parts of K; its
// eight waves take every eighth 128-K step of the part with all NB column blocks, so a step's codes
// are converted once and its columns are read once for T tiles, straight from L2 in whole 1 KiB
// operands (two halves of a step in flight; no wave shares another's).  The waves' sums meet in LDS.
//
// Bound by the columns through L1 and L2, which T tiles share, and by latency: 8 x 4096 -> 16384 INT4
// float32 13.8 us (36 MB of weights; 106 MB of L2 reads, 38 MB past it), 33 x 12288 -> 4096 MXFP4 18.6 us
// (26.7 MB; 295 MB, 45 MB past it).  A kernel that reads 16 columns a pass for each tile on its own took
// 44.7 and 69.2 us with its preparation (now 17.1 and 26.0 us a call).
template <int FMT, int NB, int T>
__global__ void __launch_bounds__(512) w4a16_wide_kernel(W4A16LinearArgs a, int S) {
  constexpr int W = kWideWaves;
  extern __shared__ uint4 lds[];
  v4f* const slot = reinterpret_cast<v4f*>(lds);           // W / 2 x T x NB x 64
  float* const dsum = reinterpret_cast<float*>(slot + W / 2 * T * NB * 64);      // Mg x r_pad
  const int tid = threadIdx.x;
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tl = lane & 15, c = lane >> 4;
  const int KS = a.K / kKStep, tiles = a.N / 16, rt0 = blockIdx.x * T, Mg = int(a.Mg);
  const int ks0 = int(blockIdx.z) * KS / a.Z, ks1 = int(blockIdx.z + 1) * KS / a.Z;
  const int n = ks1 - ks0 > w ? (ks1 - ks0 - w + W - 1) / W : 0;
  const W4Rows<FMT> rows(a.wblob + a.w_codes, a.wblob + a.w_scales, a.K, a.N_pad);
  const float gs = w4_tensor_scale<FMT>(a.wblob + a.w_amax);
  const uint32_t slab = uint32_t(KS) * 4 * NB * 1024;      // a group's columns
  const int rp = blockIdx.z == 0 ? a.r_pad : 0;
  for (int64_t g = blockIdx.y; g < a.groups; g += gridDim.y) {
    const uint8_t* const xg = reinterpret_cast<const uint8_t*>(a.planes) + g * slab;
    auto load_w = [&](int i, W4Stage<FMT> (&st)[T]) {
      // a tile past the last is one of the packed weight's padding rows
      rows.template load<T>(uint32_t(rt0), uint32_t(ks0 + w + i * W), i < n, lane, st);
    };
    auto load_x = [&](int i, int u, uint4 (&x)[NB]) {
      const __amdgpu_buffer_rsrc_t r = make_rsrc(xg, i < n ? slab : 0);
#pragma unroll
      for (int b = 0; b < NB; ++b)
        x[b] = buffer_load16(r, uint32_t(lane) * 16 + b * 1024, ((ks0 + w + i * W) * 4 + u) * NB * 1024);
    };
    v4f acc[T][NB];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[t][b] = v4f{0.f, 0.f, 0.f, 0.f};
    // XD operand sets in flight; past the last step codes and columns are zeros
    constexpr int XD = FMT == kFmtINT4 || NB <= 3 ? 4 : 2;
    W4Stage<FMT> st[2][T];
    uint4 x[XD / 2][2][NB];
    load_w(0, st[0]);
#pragma unroll
    for (int q = 0; q < XD; ++q) {
      keep_order();
      load_x(0, q, x[q / 2][q % 2]);
    }
    keep_order();
    load_w(1, st[1]);
    keep_order();
    // the down projection of the group's tokens (the first part of K adds the low-rank branch);
    // the rows of a group lie one after the other in each partial sum
    const int64_t left = a.M - g * Mg < Mg ? a.M - g * Mg : Mg;
    for (int i = tid * 4; i < int(left) * rp; i += 512 * 4) {
      const float* const pp = a.part + g * Mg * rp + i;
      v4f v = {0.f, 0.f, 0.f, 0.f};
      for (int q0 = 0; q0 < a.K / kKSuper; q0 += 8) {
        v4f d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int q = q0 + j < a.K / kKSuper ? q0 + j : q0;
          d[j] = *reinterpret_cast<const v4f*>(pp + q * a.M * rp);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (q0 + j < a.K / kKSuper) v += d[j];
      }
      *reinterpret_cast<v4f*>(dsum + i) = v;
    }
    for (int i0 = 0; i0 < n; i0 += 2) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (FMT == kFmtINT4) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            w4_half<T, NB>(st[j], half, x[half], acc);
            load_x(i0 + j + 1, half * 2, x[half][0]);
            load_x(i0 + j + 1, half * 2 + 1, x[half][1]);
            keep_order();
          }
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint4 (&xs)[NB] = x[u % XD / 2][u % 2];
            w4_mfma<FMT, T, NB>(st[j], ks0 + w + (i0 + j) * W, u, xs, acc);
            load_x(i0 + j + (u + XD) / 4, (u + XD) % 4, xs);
            keep_order();
          }
        }
        load_w(i0 + j + 2, st[j]);
        keep_order();
      }
    }
    if (FMT == kFmtNVFP4) {
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[t][b] *= gs;
    }
    // the waves' sums: 4 .. 7 onto 0 .. 3, then all eight waves add four
    auto at = [&](int q, int t, int b) -> v4f& { return slot[((q * T + t) * NB + b) * 64 + lane]; };
    if (w >= W / 2) {
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b) at(w - W / 2, t, b) = acc[t][b];
    }
    lds_barrier();
    if (w < W / 2) {
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b) at(w, t, b) += acc[t][b];
    }
    lds_barrier();
    const int TB = (Mg + 15) / 16;
    for (int u = w; u < T * TB; u += W) {
      const int t = u / TB, tok = (u % TB) * 16 + tl;
      const int64_t m = g * Mg + tok;
      if (rt0 + t >= tiles) continue;
      v4f y = {0.f, 0.f, 0.f, 0.f};
      for (int r32 = 0; r32 < rp / 32; ++r32) {
        const uint4 l2 = reinterpret_cast<const uint4*>(a.wblob + a.w_L2)[(size_t(rt0 + t) * (rp / 32) + r32) * 64 + lane];
        const float4* dq = reinterpret_cast<const float4*>(dsum + (tok < Mg ? tok : Mg - 1) * rp + r32 * 32 + c * 8);
        const float4 d0 = dq[0], d1 = dq[1];
        float dv[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
        uint4 pl[3];
        split_planes<3>(dv, pl);
#pragma unroll
        for (int i = 0; i < 3; ++i) y = mfma_bf16(l2, pl[i], y);
      }
      if (tok >= Mg || m >= a.M) continue;
#pragma unroll
      for (int q = 0; q < W / 2; ++q)
        for (int p = 0; p < S; ++p) {
          const int col = p * Mg + tok;
          y += slot[((q * T + t) * NB + (col >> 4)) * 64 + c * 16 + (col & 15)];
        }
      const int64_t row = int64_t(rt0 + t) * 16 + c * 4;
      if (a.Z > 1) {
        *reinterpret_cast<v4f*>(a.zsum + (int64_t(blockIdx.z) * a.M + m) * a.N + row) = y;
        continue;
      }
      w4a16_store(a, m, row, y, S == 3);
    }
    lds_barrier();
  }
}

// The Z parts' sums in order.
__global__ void __launch_bounds__(256) w4a16_join_kernel(W4A16LinearArgs a, int S) {
  const int64_t per = a.N / 4, total = a.M * per;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    const int64_t m = i / per, row = i % per * 4;
    v4f y = {0.f, 0.f, 0.f, 0.f};
    for (int z = 0; z < a.Z; ++z) y += *reinterpret_cast<const v4f*>(a.zsum + (z * a.M + m) * a.N + row);
    w4a16_store(a, m, row, y, S == 3);
  }
}

// Requires K % 512 == 0, N % 16 == 0, X and Y rows 16-byte aligned, M >= 1.
hipError_t launch_linear_w4a16(int fmt, const uint8_t* wblob, const WeightLayout& wl, int K, int N, const uint16_t* X,
                               int64_t ldx, int64_t M, void* Y, int64_t ldy, uint32_t epi, void* planes, float* part,
                               float* zsum, hipStream_t s) {
  W4A16LinearArgs a{};
  a.wblob = wblob;
  a.w_codes = wl.codes; a.w_scales = wl.scales; a.w_L1 = wl.L1; a.w_L2 = wl.L2; a.w_lam = wl.lam;
  a.w_bias = wl.bias; a.w_amax = wl.amax;
  a.X = X; a.planes = static_cast<uint4*>(planes); a.part = part; a.zsum = zsum; a.Y = Y;
  a.ldx = ldx; a.ldy = ldy; a.M = M; a.N_pad = wl.N_pad;
  a.K = K; a.r_pad = (epi & SVDQ_EPI_LOWRANK) ? int(wl.r_pad) : 0; a.epi = epi;
  const bool f32 = (epi & SVDQ_EPI_OUT_F32) != 0;
  const int S = f32 ? 3 : 2;                       // planes: see w4frag.h
  const auto blocks = [](int64_t v) { return unsigned(v < 65535 ? v : 65535); };
  const W4A16Plan plan = w4a16_plan(K, a.r_pad, M, S);
  const W4A16Wide wide = w4a16_wide(fmt, K, N, M, S);
  a.N = N; a.NB = wide.NB; a.Z = wide.Z; a.Mg = wide.Mg; a.groups = wide.groups; a.int4 = fmt == kFmtINT4;
  if (!plan.few || !plan.own_d) {
    if (plan.few) a.planes = nullptr;
    const dim3 pgrid(unsigned(K / kKSuper), blocks((M + 15) / 16));
    if (f32)
      hipLaunchKernelGGL((w4a16_prepare_kernel<3>), pgrid, dim3(512), 0, s, a);
    else
      hipLaunchKernelGGL((w4a16_prepare_kernel<2>), pgrid, dim3(512), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (plan.few) {
    const int tiles = N / 16, per = (tiles + plan.groups - 1) / plan.groups;
    const dim3 fgrid(unsigned((tiles + per - 1) / per));
    const int rt = plan.own_d ? a.r_pad / 16 : 0;   // 0, 2 or 4
#define SVDQ_FEW_S(FMT_, S_)                                                                                \
  do {                                                                                                      \
    if (rt == 0)                                                                                            \
      hipLaunchKernelGGL((w4a16_few_kernel<FMT_, S_, 0>), fgrid, dim3(512), plan.lds, s, a, tiles);         \
    else if (rt == 2)                                                                                       \
      hipLaunchKernelGGL((w4a16_few_kernel<FMT_, S_, 2>), fgrid, dim3(512), plan.lds, s, a, tiles);         \
    else                                                                                                    \
      hipLaunchKernelGGL((w4a16_few_kernel<FMT_, S_, 4>), fgrid, dim3(512), plan.lds, s, a, tiles);         \
  } while (0)
#define SVDQ_FEW(FMT_)              \
  do {                              \
    if (f32) SVDQ_FEW_S(FMT_, 3);   \
    else SVDQ_FEW_S(FMT_, 2);       \
  } while (0)
    if (fmt == kFmtMXFP4) SVDQ_FEW(kFmtMXFP4);
    else if (fmt == kFmtINT4) SVDQ_FEW(kFmtINT4);
    else SVDQ_FEW(kFmtNVFP4);
#undef SVDQ_FEW
#undef SVDQ_FEW_S
    return hipGetLastError();
  }
  const dim3 grid(unsigned((N / 16 + wide.T - 1) / wide.T), blocks(wide.groups), unsigned(wide.Z));
  const size_t lds = size_t(kWideWaves / 2) * wide.T * wide.NB * 1024 + size_t(wide.Mg) * a.r_pad * 4;
#define SVDQ_WIDE(FMT_, NB_, T_) \
  hipLaunchKernelGGL((w4a16_wide_kernel<FMT_, NB_, T_>), grid, dim3(512), lds, s, a, S)
#define SVDQ_WIDE_T(FMT_, NB_)                                                   \
  do {                                                                           \
    constexpr int kT = FMT_ == kFmtINT4 && NB_ > 3 ? 2 : 4;                      \
    if (wide.T == 1) SVDQ_WIDE(FMT_, NB_, 1);                                    \
    else if (wide.T == 2) SVDQ_WIDE(FMT_, NB_, 2);                               \
    else SVDQ_WIDE(FMT_, NB_, kT);                                               \
  } while (0)
#define SVDQ_WIDE_FMT(FMT_)                                       \
  do {                                                            \
    if (wide.NB == 2) SVDQ_WIDE_T(FMT_, 2);                       \
    else if (wide.NB == 3) SVDQ_WIDE_T(FMT_, 3);                  \
    else if (wide.NB == 4) SVDQ_WIDE_T(FMT_, 4);                  \
    else if (wide.NB == 5) SVDQ_WIDE_T(FMT_, 5);                  \
    else SVDQ_WIDE_T(FMT_, 6);                                    \
  } while (0)
  if (fmt == kFmtMXFP4) SVDQ_WIDE_FMT(kFmtMXFP4);
  else if (fmt == kFmtINT4) SVDQ_WIDE_FMT(kFmtINT4);
  else SVDQ_WIDE_FMT(kFmtNVFP4);
#undef SVDQ_WIDE_FMT
#undef SVDQ_WIDE_T
#undef SVDQ_WIDE
  if (wide.Z > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(w4a16_join_kernel, dim3(blocks((M * N / 4 + 255) / 256)), dim3(256), 0, s, a, S);
  }
  return hipGetLastError();
}

}  // namespace svdq
