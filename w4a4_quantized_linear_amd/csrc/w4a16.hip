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
      if (m0 + tl < a.M) {
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
  const W4Tile<FMT> tile(a.wblob + a.w_codes, a.wblob + a.w_scales, rt, a.K, a.N_pad, lane);
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
      tile.load(ks, st.w);
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
  const dim3 pgrid(unsigned(K / kKSuper), blocks((M + 15) / 16));
  if (f32)
    hipLaunchKernelGGL((w4a16_prepare_kernel<3>), pgrid, dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((w4a16_prepare_kernel<2>), pgrid, dim3(512), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
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
