// A packed layer applied to 16-bit activations (few tokens):
//
//   Y[m, n] = act( sum_k deQ(R)[n, k] x_hat[m, k] + sum_i L2[i, n] D[m, i] + b[n] ),
//   x_hat = fp32(X / lambda),  D = X_hat L1.
//
// Two launches.  w4a16_prepare_kernel divides by lambda, splits x_hat into bf16
// planes (w4frag.h) and forms D's partial sums, one per 512 of K;
// w4a16_kernel streams the codes once per 16 columns.
#include <hip/hip_runtime.h>

#include "svdq.h"
#include "w4frag.h"

namespace svdq {

struct W4A16LinearArgs {
  const uint8_t* wblob;
  size_t w_codes, w_scales, w_L1, w_L2, w_lam, w_bias, w_amax;
  const uint16_t* X;
  uint16_t* planes;        // S x M x K bf16
  float* part;             // K / 512 x M x r_pad
  void* Y;
  int64_t ldx, ldy, M, N_pad;
  int K, r_pad;            // r_pad 0: no low-rank branch
  uint32_t epi;
};

constexpr int kPrepWaves = 8;          // 64 K each
constexpr int kPrepTiles = 4;          // 16-rank tiles whose sums meet in LDS at a time

// One workgroup: 16 tokens, 512 of K.
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
    uint4 p[2][S];
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
#pragma unroll
        for (int i = 0; i < S; ++i) *reinterpret_cast<uint4*>(a.planes + (i * a.M + m) * a.K + k) = p[s][i];
      }
    }
    for (int i0 = 0; i0 < RT; i0 += kPrepTiles) {
      const int tiles = RT - i0 < kPrepTiles ? RT - i0 : kPrepTiles;
      for (int i = 0; i < tiles; ++i) {
        v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint4 l1 = L1f[(size_t(k0 / 32 + s) * RT + i0 + i) * 64 + lane];
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

// Few tokens, one launch: all S planes of the M tokens are columns of one MFMA.
//
// A workgroup of eight waves computes x_hat of all tokens once into LDS (planes x tokens rows of
// K bf16), forms D = X_hat L1 from it where the rank allows (OWN_D; otherwise it sums
// w4a16_prepare_kernel's partial sums), and then takes row tiles blockIdx.x, + gridDim.x, ...:
// wave w the 128-K steps w, w + 8, ..., kFewDepth steps of codes in flight, the pipeline running
// on from tile to tile.  The waves' sums meet in LDS (two buffers, so one barrier a tile); one
// wave, another each tile, adds them and the up projection and writes the tile.
constexpr int kFewDepth = 4;
constexpr int kFewGroups = 512;        // workgroups at most

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
    for (int j = 0; j < kFewDepth; ++j) load(st[j]);
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
        uint4 p[S];
        split_planes<S>(dv, p);
#pragma unroll
        for (int i = 0; i < S; ++i) z = mfma_bf16(l2, p[i], z);
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
  v4f acc[1] = {zero};
  for (;;) {
#pragma unroll
    for (int j = 0; j < kFewDepth; ++j) {
      const int ks = w + i * W;
      uint4 x[1][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[0][u] = *reinterpret_cast<const uint4*>(xp + (ks * kKStep + k_of<FMT>(c, u)) * 2);
      w4_step<FMT, 1>(st[j], ks, x, acc);
      load(st[j]);
      if (++i == n) {
        finish(rt, acc[0]);
        acc[0] = zero;
        i = 0;
        rt += gridDim.x;
        if (rt >= tiles) return;
      }
    }
  }
}

constexpr int kLinWaves = 8;

// One workgroup: one 16-row tile, its waves taking every eighth 128-K step.
// PACKED: all planes of the (at most 16 / S) tokens are columns of one MFMA.
// Otherwise blocks of 16 tokens, one MFMA per plane.
template <int FMT, int S, bool PACKED, bool OUT_F32>
__global__ void __launch_bounds__(512) w4a16_kernel(W4A16LinearArgs a) {
  constexpr int NB = PACKED ? 1 : S;               // B operands per step and MFMA
  constexpr int TPB = PACKED ? tokens_per_block(S) : 16;
  constexpr int DEPTH = PACKED ? 3 : 2;            // steps in flight
  __shared__ v4f red[kLinWaves][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tl = lane & 15, c = lane >> 4;
  const int KS = a.K / kKStep;
  const int64_t rt = blockIdx.x;
  const W4Rows<FMT> rows(a.wblob + a.w_codes, a.wblob + a.w_scales, a.K, a.N_pad);
  const int n = KS > w ? (KS - w + kLinWaves - 1) / kLinWaves : 0;
  const float gs = w4_tensor_scale<FMT>(a.wblob + a.w_amax);
  for (int64_t m0 = int64_t(blockIdx.y) * TPB; m0 < a.M; m0 += int64_t(gridDim.y) * TPB) {
    const int64_t left = a.M - m0;
    // this lane's column(s): past the last they repeat it (columns are independent)
    const int t_raw = PACKED ? tl % TPB : tl;
    const int64_t t = m0 + (t_raw < left ? t_raw : left - 1);
    const int pl = PACKED ? (tl / TPB < S ? tl / TPB : S - 1) : 0;
    const uint16_t* xp = a.planes + (pl * a.M + t) * a.K;
    struct Stage { W4Stage<FMT> w; uint4 x[NB][4]; };
    auto load = [&](int i, Stage& st) {
      const int ks = w + (i < n ? i : n - 1) * kLinWaves;
      rows.load(uint32_t(rt), ks, i < n, lane, st.w);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          st.x[b][u] = *reinterpret_cast<const uint4*>(xp + b * a.M * a.K + ks * kKStep + k_of<FMT>(c, u));
    };
    v4f acc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = v4f{0.f, 0.f, 0.f, 0.f};
    if (n > 0) {
      Stage st[DEPTH];
#pragma unroll
      for (int j = 0; j < DEPTH; ++j) load(j, st[j]);
      for (int i0 = 0; i0 < n; i0 += DEPTH) {
#pragma unroll
        for (int j = 0; j < DEPTH; ++j) {
          if (i0 + j < n) w4_step<FMT, NB>(st[j].w, w + (i0 + j) * kLinWaves, st[j].x, acc);
          load(i0 + j + DEPTH, st[j]);
        }
      }
    }
    v4f sum = acc[0];
#pragma unroll
    for (int b = 1; b < NB; ++b) sum += acc[b];
    if (FMT == kFmtNVFP4) sum *= gs;
    // up projection: wave w takes ranks 32 w .. 32 w + 31
    if (w * 32 < a.r_pad) {
      const uint4 l2 = reinterpret_cast<const uint4*>(a.wblob + a.w_L2)[(size_t(rt) * (a.r_pad / 32) + w) * 64 + lane];
      float d[8] = {};
      const float* dp = a.part + t * a.r_pad + w * 32 + c * 8;
      for (int s = 0; s < a.K / kKSuper; ++s) {
        const float4 d0 = *reinterpret_cast<const float4*>(dp + int64_t(s) * a.M * a.r_pad);
        const float4 d1 = *reinterpret_cast<const float4*>(dp + int64_t(s) * a.M * a.r_pad + 4);
        d[0] += d0.x; d[1] += d0.y; d[2] += d0.z; d[3] += d0.w;
        d[4] += d1.x; d[5] += d1.y; d[6] += d1.z; d[7] += d1.w;
      }
      uint4 p[S];
      split_planes<S>(d, p);
      if constexpr (PACKED) {
        uint4 x = p[0];
#pragma unroll
        for (int i = 1; i < S; ++i) x = pl == i ? p[i] : x;
        sum = mfma_bf16(l2, x, sum);
      } else {
#pragma unroll
        for (int i = 0; i < S; ++i) sum = mfma_bf16(l2, p[i], sum);
      }
    }
    red[w][lane] = sum;
    __syncthreads();
    if (w == 0 && tl < (left < TPB ? left : TPB)) {
      v4f y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < kLinWaves; ++v)
#pragma unroll
        for (int i = 0; i < (PACKED ? S : 1); ++i) y += red[v][lane + i * TPB];
      const int64_t row = rt * 16 + c * 4;
      if (a.epi & SVDQ_EPI_BIAS) {
        const uint2 b = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(a.wblob + a.w_bias) + row);
        y += v4f{bf_lo(b.x), bf_hi(b.x), bf_lo(b.y), bf_hi(b.y)};
      }
      if (a.epi & SVDQ_EPI_GELU) {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = gelu_erf(y[e]);
      }
      const int64_t o = (m0 + tl) * a.ldy + row;
      if (OUT_F32)
        *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.Y) + o) = y;
      else
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.Y) + o) =
            make_uint2(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]));
    }
    __syncthreads();
  }
}

// Requires K % 512 == 0, N % 16 == 0, X and Y rows 16-byte aligned, M >= 1.
hipError_t launch_linear_w4a16(int fmt, const uint8_t* wblob, const WeightLayout& wl, int K, int N, const uint16_t* X,
                               int64_t ldx, int64_t M, void* Y, int64_t ldy, uint32_t epi, void* planes, float* part,
                               hipStream_t s) {
  W4A16LinearArgs a{};
  a.wblob = wblob;
  a.w_codes = wl.codes; a.w_scales = wl.scales; a.w_L1 = wl.L1; a.w_L2 = wl.L2; a.w_lam = wl.lam;
  a.w_bias = wl.bias; a.w_amax = wl.amax;
  a.X = X; a.planes = static_cast<uint16_t*>(planes); a.part = part; a.Y = Y;
  a.ldx = ldx; a.ldy = ldy; a.M = M; a.N_pad = wl.N_pad;
  a.K = K; a.r_pad = (epi & SVDQ_EPI_LOWRANK) ? int(wl.r_pad) : 0; a.epi = epi;
  const bool f32 = (epi & SVDQ_EPI_OUT_F32) != 0;
  const int S = f32 ? 3 : 2;                       // planes: see w4frag.h
  const auto blocks = [](int64_t v) { return unsigned(v < 65535 ? v : 65535); };
  const W4A16Plan plan = w4a16_plan(K, a.r_pad, M, S);
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
    const int tiles = N / 16, per = (tiles + kFewGroups - 1) / kFewGroups;
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
  const bool packed = M <= tokens_per_block(S);
  const dim3 grid(unsigned(N / 16), packed ? 1 : blocks((M + 15) / 16));
#define SVDQ_LIN(FMT_, P_)                                                                            \
  do {                                                                                                \
    if (f32)                                                                                          \
      hipLaunchKernelGGL((w4a16_kernel<FMT_, 3, P_, true>), grid, dim3(512), 0, s, a);                \
    else                                                                                              \
      hipLaunchKernelGGL((w4a16_kernel<FMT_, 2, P_, false>), grid, dim3(512), 0, s, a);               \
  } while (0)
#define SVDQ_LIN_FMT(FMT_)                                                                            \
  do {                                                                                                \
    if (packed) SVDQ_LIN(FMT_, true);                                                                 \
    else SVDQ_LIN(FMT_, false);                                                                       \
  } while (0)
  if (fmt == kFmtMXFP4) SVDQ_LIN_FMT(kFmtMXFP4);
  else if (fmt == kFmtINT4) SVDQ_LIN_FMT(kFmtINT4);
  else SVDQ_LIN_FMT(kFmtNVFP4);
#undef SVDQ_LIN_FMT
#undef SVDQ_LIN
  return hipGetLastError();
}

}  // namespace svdq
