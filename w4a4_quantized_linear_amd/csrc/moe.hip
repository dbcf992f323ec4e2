// Mixture of experts for few tokens: the router and the experts' products.
//
//   logits[m, e] = sum_k X[m, k] Wr[e, k];  ids, weights: the top experts of each token
//   h[m, j]  = act(X[m] Wg_e^T + bg_e) * (X[m] Wu_e^T + bu_e),     e = ids[m, j]
//   Y[m]     = sum_j weights[m, j] (h[m, j] Wd_e^T + bd_e)
//
// The experts are 4-bit weights (w4frag.h).  A pair is one (token, j); P = M top_k pairs.
#include <hip/hip_runtime.h>

#include "svdq.h"
#include "w4frag.h"

namespace svdq {

// ------------------------------------------------------------------ router

struct RouteArgs {
  const uint16_t* X;
  const uint16_t* Wr;
  const float* bias;       // added to the scores for the choice only; may be null
  double* logits;          // M x E
  int32_t* ids;
  float* weights;
  int64_t ldx, M;
  int K, E, top_k;
  uint32_t flags;
  float scale;
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Logits in fp64: products of two bf16 are exact in fp32, and the sums keep 53 bits, so
// which expert is chosen does not depend on the order of summation.  A wave takes TE experts
// and TM tokens, its lanes 8 consecutive K each.
template <int TE, int TM>
__global__ void __launch_bounds__(256) route_logits_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e0 = (blockIdx.x * 4 + w) * TE;
  if (e0 >= a.E) return;
  for (int64_t m0 = int64_t(blockIdx.y) * TM; m0 < a.M; m0 += int64_t(gridDim.y) * TM) {
    const uint16_t* wp[TE];
    const uint16_t* xp[TM];
#pragma unroll
    for (int i = 0; i < TE; ++i) wp[i] = a.Wr + int64_t(e0 + i < a.E ? e0 + i : a.E - 1) * a.K;
#pragma unroll
    for (int j = 0; j < TM; ++j) xp[j] = a.X + (m0 + j < a.M ? m0 + j : a.M - 1) * a.ldx;
    double acc[TE][TM] = {};
    for (int k = lane * 8; k < a.K; k += 512) {
      uint4 wq[TE], xq[TM];
#pragma unroll
      for (int i = 0; i < TE; ++i) wq[i] = *reinterpret_cast<const uint4*>(wp[i] + k);
#pragma unroll
      for (int j = 0; j < TM; ++j) xq[j] = *reinterpret_cast<const uint4*>(xp[j] + k);
      float xf[TM][8];
#pragma unroll
      for (int j = 0; j < TM; ++j) unpack_bf8(xq[j], xf[j]);
#pragma unroll
      for (int i = 0; i < TE; ++i) {
        float wf[8];
        unpack_bf8(wq[i], wf);
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[i][j] = fma(double(wf[q]), double(xf[j][q]), acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < TE; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const double v = wave_sum(acc[i][j]);
        if (lane == 0 && e0 + i < a.E && m0 + j < a.M) a.logits[(m0 + j) * a.E + e0 + i] = v;
      }
  }
}

// Scores, the choice and the weights of one token whose logits lie in `l` (LDS); every thread
// of the workgroup takes part.  An expert's place is the number of experts that come before it:
// a larger key, or the same and a lower index; a NaN key counts as -infinity.
__device__ __forceinline__ void choose_experts(const RouteArgs& a, int64_t m, const double* l, double* key, double* red,
                                               double* chosen) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 63, w = tid >> 6, nw = nt >> 6;
  const bool sig = (a.flags & SVDQ_ROUTE_SIGMOID) != 0;
  double top = -__builtin_huge_val(), sum = 0.0;
  if (!sig) {
    for (int e = tid; e < a.E; e += nt) top = fmax(top, l[e]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmax(top, __shfl_xor(top, o));
    if (lane == 0) red[w] = top;
    __syncthreads();
    for (int v = 0; v < nw; ++v) top = fmax(top, red[v]);
    __syncthreads();
    for (int e = tid; e < a.E; e += nt) sum += exp(l[e] - top);
    sum = wave_sum(sum);
    if (lane == 0) red[w] = sum;
    __syncthreads();
    sum = 0.0;
    for (int v = 0; v < nw; ++v) sum += red[v];
  }
  auto score = [&](int e) { return sig ? 1.0 / (1.0 + exp(-l[e])) : exp(l[e] - top) / sum; };
  for (int e = tid; e < a.E; e += nt) {
    const double k = a.bias ? score(e) + double(a.bias[e]) : l[e];   // without a bias the logits order the scores
    key[e] = k == k ? k : -__builtin_huge_val();
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += nt) {
    const double k = key[e];
    int place = 0;
    for (int f = 0; f < a.E; ++f) place += (key[f] > k || (key[f] == k && f < e)) ? 1 : 0;
    if (place < a.top_k) {
      a.ids[m * a.top_k + place] = e;
      chosen[place] = score(e);
    }
  }
  __syncthreads();
  if (tid < a.top_k) {
    double v = chosen[tid];
    if (a.flags & SVDQ_ROUTE_RENORM) {
      double s = 0.0;
      for (int j = 0; j < a.top_k; ++j) s += chosen[j];
      v = s == 0.0 ? 0.0 : v / s;
    }
    a.weights[m * a.top_k + tid] = float(v * double(a.scale));
  }
  __syncthreads();
}

__global__ void __launch_bounds__(256) route_choose_kernel(RouteArgs a) {
  __shared__ double l[kMoeMaxE], key[kMoeMaxE], red[4], chosen[kMoeMaxTopK];
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    for (int e = threadIdx.x; e < a.E; e += 256) l[e] = a.logits[m * a.E + e];
    __syncthreads();
    choose_experts(a, m, l, key, red, chosen);
  }
}

hipError_t launch_moe_route(const uint16_t* X, int64_t M, int64_t ldx, int K, const uint16_t* Wr, const float* bias,
                            int E, int top_k, uint32_t flags, float scale, int32_t* ids, float* weights, double* logits,
                            hipStream_t s) {
  RouteArgs a{};
  a.X = X; a.Wr = Wr; a.bias = bias; a.logits = logits; a.ids = ids; a.weights = weights;
  a.ldx = ldx; a.M = M; a.K = K; a.E = E; a.top_k = top_k; a.flags = flags; a.scale = scale;
  const auto cap = [](int64_t v) { return unsigned(v < 65535 ? v : 65535); };
  if (M < 4)
    hipLaunchKernelGGL((route_logits_kernel<1, 1>), dim3((E + 3) / 4, cap(M)), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((route_logits_kernel<2, 4>), dim3((E + 7) / 8, cap((M + 3) / 4)), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(route_choose_kernel, dim3(cap(M)), dim3(256), 0, s, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------ experts

struct MoeArgs {
  const uint8_t* wg;                   // E packed [gate | up] weights, blob_g bytes each
  const uint8_t* wd;                   // E packed down weights
  size_t blob_g, g_codes, g_scales, g_bias, g_amax;
  size_t blob_d, d_codes, d_scales, d_bias, d_amax;
  const uint16_t* X;
  const int32_t* ids;
  const float* weights;
  uint16_t* h;                         // S x P x F bf16 planes
  void* Y;
  int64_t ldx, ldy, Ng_pad, Nd_pad;
  int H, F, N, E, top_k, P;            // gate/up: H -> 2 F, down: F -> N
  uint32_t epi;
};

constexpr int kGateWaves = 8;

// One workgroup: 16 gate and 16 up rows of the blockIdx.y-th expert that some pair asks for.
template <int FMT, int S, int NB>
__global__ void __launch_bounds__(512) moe_gate_up_kernel(MoeArgs a) {
  constexpr int DEPTH = 2;
  __shared__ int list[kMoeMaxPairs];
  __shared__ int asked[kMoeMaxE];
  __shared__ int count;
  __shared__ v4f red[kGateWaves][2][NB][64];
  const int tid = threadIdx.x;
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tl = lane & 15, c = lane >> 4;
  for (int e = tid; e < a.E; e += 512) asked[e] = 0;
  if (tid == 0) count = 0;
  __syncthreads();
  for (int p = tid; p < a.P; p += 512) {
    const int id = a.ids[p];
    if (id >= 0 && id < a.E) asked[id] = 1;
  }
  __syncthreads();
  int ex = -1, before = 0;
  for (int e0 = 0; e0 < a.E && ex < 0; e0 += 64) {
    const uint64_t b = __ballot(e0 + lane < a.E && asked[e0 + lane] != 0);
    const int here = __popcll(b), want = int(blockIdx.y) - before;
    if (want < here) {
      uint64_t m = b;
      for (int i = 0; i < want; ++i) m &= m - 1;
      ex = e0 + __ffsll((unsigned long long)m) - 1;
    }
    before += here;
  }
  if (ex < 0) return;                                       // fewer experts are asked for
  ex = __builtin_amdgcn_readfirstlane(ex);
  // the expert's pairs, in any order: a pair is a column of its own
  for (int p = tid; p < a.P; p += 512)
    if (a.ids[p] == ex) list[atomicAdd(&count, 1)] = p;
  __syncthreads();
  const int T = count;

  const uint8_t* blob = a.wg + size_t(ex) * a.blob_g;
  const int KS = a.H / kKStep, FT = a.F / 16;
  const int ft = blockIdx.x;
  const W4Rows<FMT> rows(blob + a.g_codes, blob + a.g_scales, a.H, a.Ng_pad);
  const float gs = w4_tensor_scale<FMT>(blob + a.g_amax);
  const int n = KS > w ? (KS - w + kGateWaves - 1) / kGateWaves : 0;
  struct Stage { W4Stage<FMT> g, u; uint4 x[NB][4]; };
  for (int t0 = 0; t0 < T; t0 += 16 * NB) {
    const uint16_t* xp[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int i = t0 + b * 16 + tl;
      xp[b] = a.X + int64_t(list[i < T ? i : T - 1] / a.top_k) * a.ldx;
    }
    auto load = [&](int i, Stage& st) {
      const int ks = w + (i < n ? i : n - 1) * kGateWaves;
      rows.load(ft, ks, i < n, lane, st.g);
      rows.load(FT + ft, ks, i < n, lane, st.u);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int u = 0; u < 4; ++u) st.x[b][u] = *reinterpret_cast<const uint4*>(xp[b] + ks * kKStep + k_of<FMT>(c, u));
    };
    v4f ag[NB], au[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) ag[b] = au[b] = v4f{0.f, 0.f, 0.f, 0.f};
    if (n > 0) {
      Stage st[DEPTH];
#pragma unroll
      for (int j = 0; j < DEPTH; ++j) load(j, st[j]);
      for (int i0 = 0; i0 < n; i0 += DEPTH) {
#pragma unroll
        for (int j = 0; j < DEPTH; ++j) {
          if (i0 + j < n) {
            const int ks = w + (i0 + j) * kGateWaves;
            w4_step<FMT, NB>(st[j].g, ks, st[j].x, ag);
            w4_step<FMT, NB>(st[j].u, ks, st[j].x, au);
          }
          load(i0 + j + DEPTH, st[j]);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      red[w][0][b][lane] = ag[b];
      red[w][1][b][lane] = au[b];
    }
    __syncthreads();
    // wave b finishes block b: rows 4 c .. 4 c + 3 of pair tl
    for (int b = w; b < NB; b += kGateWaves) {
      const int i = t0 + b * 16 + tl;
      if (i < T) {
        v4f g = red[0][0][b][lane], u = red[0][1][b][lane];
#pragma unroll
        for (int v = 1; v < kGateWaves; ++v) {
          g += red[v][0][b][lane];
          u += red[v][1][b][lane];
        }
        if (FMT == kFmtNVFP4) { g *= gs; u *= gs; }
        const int row = ft * 16 + c * 4;
        if (a.epi & SVDQ_EPI_BIAS) {
          const uint16_t* bias = reinterpret_cast<const uint16_t*>(blob + a.g_bias);
          const uint2 bg = *reinterpret_cast<const uint2*>(bias + row), bu = *reinterpret_cast<const uint2*>(bias + a.F + row);
          g += v4f{bf_lo(bg.x), bf_hi(bg.x), bf_lo(bg.y), bf_hi(bg.y)};
          u += v4f{bf_lo(bu.x), bf_hi(bu.x), bf_lo(bu.y), bf_hi(bu.y)};
        }
        float hv[8] = {};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          hv[e] = ((a.epi & SVDQ_EPI_GELU) ? gelu_erf(g[e]) : g[e] / (1.0f + expf(-g[e]))) * u[e];
        uint4 p[S];
        split_planes<S>(hv, p);
#pragma unroll
        for (int s = 0; s < S; ++s)
          *reinterpret_cast<uint2*>(a.h + (int64_t(s) * a.P + list[i]) * a.F + row) = make_uint2(p[s].x, p[s].y);
      }
    }
    __syncthreads();
  }
}

constexpr int kDownWaves = 16;
constexpr int kDownMinSlots = 256;     // pairs x K chunks that the LDS sums have room for at least
constexpr int kDownMaxBlocks = 1024;   // column blocks: at most min(E, P) + P / 5

// One workgroup: 16 output rows of all tokens.  A unit is one block of an expert's pairs (all S
// planes of up to 16 / S pairs are columns) and one chunk of K; waves take units in turn and
// leave each pair's sums in a place of its own, so the final sums have one order.
template <int FMT, int S, bool OUT_F32>
__global__ void __launch_bounds__(1024) moe_down_kernel(MoeArgs a) {
  constexpr int TPB = tokens_per_block(S);
  constexpr int DEPTH = 3;
  extern __shared__ v4f slot[];                    // [chunk][pair][4]: 16 rows of a pair
  __shared__ int list[kMoeMaxPairs];
  __shared__ int first[kMoeMaxE + 1], cursor[kMoeMaxE];
  __shared__ int blk_e[kDownMaxBlocks], blk_t[kDownMaxBlocks];
  __shared__ int nblocks;
  const int tid = threadIdx.x;
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tl = lane & 15, c = lane >> 4;
  // pairs sorted by expert, and the column blocks
  for (int e = tid; e < a.E; e += 1024) cursor[e] = 0;
  __syncthreads();
  for (int p = tid; p < a.P; p += 1024) {
    const int id = a.ids[p];
    if (id >= 0 && id < a.E) atomicAdd(&cursor[id], 1);
  }
  __syncthreads();
  if (w == 0) {
    int pairs = 0, blocks = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + lane, cnt = e < a.E ? cursor[e] : 0, nb = (cnt + TPB - 1) / TPB;
      int sp = cnt, sb = nb;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int vp = __shfl_up(sp, o), vb = __shfl_up(sb, o);
        if (lane >= o) { sp += vp; sb += vb; }
      }
      if (e < a.E) {
        first[e] = pairs + sp - cnt;
        cursor[e] = first[e];
        for (int b = 0; b < nb; ++b) {
          blk_e[blocks + sb - nb + b] = e;
          blk_t[blocks + sb - nb + b] = b * TPB;
        }
      }
      pairs += __shfl(sp, 63);
      blocks += __shfl(sb, 63);
    }
    if (lane == 0) { first[a.E] = pairs; nblocks = blocks; }
  }
  __syncthreads();
  for (int p = tid; p < a.P; p += 1024) {
    const int id = a.ids[p];
    if (id >= 0 && id < a.E) list[atomicAdd(&cursor[id], 1)] = p;
  }
  __syncthreads();

  const int KS = a.F / kKStep;
  const int slots = a.P > kDownMinSlots ? a.P : kDownMinSlots;
  // as many chunks of K as it takes to give every wave a unit, where the LDS has room
  int KC = 1;
  while (nblocks * KC < kDownWaves && KC * 2 <= KS && KC * 2 * a.P <= slots) KC *= 2;
  const int64_t rt = blockIdx.x;
  for (int u = w; u < nblocks * KC; u += kDownWaves) {
    const int b = u / KC, kc = u % KC;
    const int ex = __builtin_amdgcn_readfirstlane(blk_e[b]), t0 = blk_t[b];
    const int f0 = first[ex] + t0, cnt = first[ex + 1] - f0 < TPB ? first[ex + 1] - f0 : TPB;
    const int ks0 = kc * KS / KC, n = (kc + 1) * KS / KC - ks0;
    const uint8_t* blob = a.wd + size_t(ex) * a.blob_d;
    const W4Rows<FMT> rows(blob + a.d_codes, blob + a.d_scales, a.F, a.Nd_pad);
    const int t = tl % TPB < cnt ? tl % TPB : cnt - 1, pl = tl / TPB < S ? tl / TPB : S - 1;
    const int pair = list[f0 + t];
    const uint16_t* xp = a.h + (int64_t(pl) * a.P + pair) * a.F;
    struct Stage { W4Stage<FMT> w; uint4 x[1][4]; };
    auto load = [&](int i, Stage& st) {
      const int ks = ks0 + (i < n ? i : n - 1);
      rows.load(uint32_t(rt), ks, i < n, lane, st.w);
#pragma unroll
      for (int q = 0; q < 4; ++q) st.x[0][q] = *reinterpret_cast<const uint4*>(xp + ks * kKStep + k_of<FMT>(c, q));
    };
    v4f acc[1] = {v4f{0.f, 0.f, 0.f, 0.f}};
    Stage st[DEPTH];
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) load(j, st[j]);
    for (int i0 = 0; i0 < n; i0 += DEPTH) {
#pragma unroll
      for (int j = 0; j < DEPTH; ++j) {
        if (i0 + j < n) w4_step<FMT, 1>(st[j].w, ks0 + i0 + j, st[j].x, acc);
        load(i0 + j + DEPTH, st[j]);
      }
    }
    v4f y = acc[0];
    if (FMT == kFmtNVFP4) y *= w4_tensor_scale<FMT>(blob + a.d_amax);
    // the planes' columns of a pair
    v4f sum = y;
#pragma unroll
    for (int i = 1; i < S; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += __shfl(y[e], lane + i * TPB);
    if (kc == 0 && (a.epi & SVDQ_EPI_BIAS)) {
      const uint2 bb = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(blob + a.d_bias) + rt * 16 + c * 4);
      sum += v4f{bf_lo(bb.x), bf_hi(bb.x), bf_lo(bb.y), bf_hi(bb.y)};
    }
    if (tl < cnt) slot[(kc * a.P + pair) * 4 + c] = sum;
  }
  __syncthreads();
  // Y[m] = sum_j w_j (sum over chunks), j and chunks in order; pairs without an expert add nothing
  const int M = a.P / a.top_k;
  for (int i = tid; i < M * 4; i += 1024) {
    const int m = i >> 2, q = i & 3;
    v4f y = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < a.top_k; ++j) {
      const int p = m * a.top_k + j, id = a.ids[p];
      if (id < 0 || id >= a.E) continue;
      v4f v = slot[p * 4 + q];
      for (int k = 1; k < KC; ++k) v += slot[(k * a.P + p) * 4 + q];
      const float wt = a.weights[p];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = fmaf(wt, v[e], y[e]);
    }
    const int64_t o = int64_t(m) * a.ldy + rt * 16 + q * 4;
    if (OUT_F32)
      *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.Y) + o) = y;
    else
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.Y) + o) =
          make_uint2(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]));
  }
}

template <int FMT, int S>
static void gate_up(const MoeArgs& a, hipStream_t s) {
  const int slots = a.E < a.P ? a.E : a.P;
  const dim3 grid(unsigned(a.F / 16), unsigned(slots));
  const int avg = (a.P + slots - 1) / slots;
  if (avg <= 8)
    hipLaunchKernelGGL((moe_gate_up_kernel<FMT, S, 1>), grid, dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((moe_gate_up_kernel<FMT, S, 2>), grid, dim3(512), 0, s, a);
}

template <int FMT>
static void down(const MoeArgs& a, bool f32, hipStream_t s) {
  const size_t lds = size_t(a.P > kDownMinSlots ? a.P : kDownMinSlots) * 64;
  const dim3 grid(unsigned(a.N / 16));
  if (f32)
    hipLaunchKernelGGL((moe_down_kernel<FMT, 3, true>), grid, dim3(1024), lds, s, a);
  else
    hipLaunchKernelGGL((moe_down_kernel<FMT, 2, false>), grid, dim3(1024), lds, s, a);
}

// Requires 1 <= top_k <= kMoeMaxTopK, 1 <= E <= kMoeMaxE, H % 512 == 0, F % 512 == 0, N % 16 == 0, M >= 1.  h has room for
// 3 planes of F values for each pair of one part (at most kMoeMaxPairs).
hipError_t launch_moe(int fmt_g, const uint8_t* wg, const WeightLayout& lg, int fmt_d, const uint8_t* wd,
                      const WeightLayout& ld, int H, int F, int N, int E, const uint16_t* X, int64_t M, int64_t ldx,
                      const int32_t* ids, const float* weights, int top_k, void* Y, int64_t ldy, uint32_t epi,
                      void* h, hipStream_t s) {
  MoeArgs a{};
  a.wg = wg; a.blob_g = lg.total; a.g_codes = lg.codes; a.g_scales = lg.scales; a.g_bias = lg.bias; a.g_amax = lg.amax;
  a.wd = wd; a.blob_d = ld.total; a.d_codes = ld.codes; a.d_scales = ld.scales; a.d_bias = ld.bias; a.d_amax = ld.amax;
  a.h = static_cast<uint16_t*>(h);
  a.ldx = ldx; a.ldy = ldy; a.Ng_pad = lg.N_pad; a.Nd_pad = ld.N_pad;
  a.H = H; a.F = F; a.N = N; a.E = E; a.top_k = top_k; a.epi = epi;
  const bool f32 = (epi & SVDQ_EPI_OUT_F32) != 0;
  const int64_t part = kMoeMaxPairs / top_k;
  for (int64_t m0 = 0; m0 < M; m0 += part) {
    const int64_t mc = M - m0 < part ? M - m0 : part;
    a.P = int(mc * top_k);
    a.X = X + m0 * ldx;
    a.ids = ids + m0 * top_k;
    a.weights = weights + m0 * top_k;
    a.Y = static_cast<uint8_t*>(Y) + m0 * ldy * (f32 ? 4 : 2);
#define SVDQ_GATE(FMT_)                       \
  do {                                        \
    if (f32) gate_up<FMT_, 3>(a, s);          \
    else gate_up<FMT_, 2>(a, s);              \
  } while (0)
    if (fmt_g == kFmtMXFP4) SVDQ_GATE(kFmtMXFP4);
    else if (fmt_g == kFmtINT4) SVDQ_GATE(kFmtINT4);
    else SVDQ_GATE(kFmtNVFP4);
#undef SVDQ_GATE
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (fmt_d == kFmtMXFP4) down<kFmtMXFP4>(a, f32, s);
    else if (fmt_d == kFmtINT4) down<kFmtINT4>(a, f32, s);
    else down<kFmtNVFP4>(a, f32, s);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace svdq
