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
  double* logits;          // Z x M x E
  int32_t* ids;
  float* weights;
  int64_t ldx, M;
  int K, E, top_k, Z;
  uint32_t flags;
  float scale;
};

// Lane 63's combination of a wave's values over the row shifts and broadcasts of DPP: sums of
// doubles, maxima of unsigned words.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xF, false));   // 0 where no lane is read
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, uint64_t(dpp<CTRL, ROWS>(uint32_t(u))) | uint64_t(dpp<CTRL, ROWS>(uint32_t(u >> 32))) << 32);
}
constexpr int kShr1 = 0x111, kShr2 = 0x112, kShr4 = 0x114, kShr8 = 0x118, kBcast15 = 0x142, kBcast31 = 0x143;
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto up = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  v = up(v, dpp<kShr1, 0xF>(v));
  v = up(v, dpp<kShr2, 0xF>(v));
  v = up(v, dpp<kShr4, 0xF>(v));
  v = up(v, dpp<kShr8, 0xF>(v));
  v = up(v, dpp<kBcast15, 0xA>(v));
  v = up(v, dpp<kBcast31, 0xC>(v));
  return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, uint64_t(uint32_t(__builtin_amdgcn_readlane(int(u), lane))) |
                                        uint64_t(uint32_t(__builtin_amdgcn_readlane(int(u >> 32), lane))) << 32);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp<kShr1, 0xF>(v);
  v += dpp<kShr2, 0xF>(v);
  v += dpp<kShr4, 0xF>(v);
  v += dpp<kShr8, 0xF>(v);
  v += dpp<kBcast15, 0xA>(v);
  v += dpp<kBcast31, 0xC>(v);
  return lane_value(v, 63);
}

// A double's place among doubles as an unsigned number above 0: NaN 1, below -infinity; -0 as 0.
__device__ __forceinline__ uint64_t order_of(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  return !(v == v) ? 1 : u >> 63 ? ~u : u | (uint64_t(1) << 63);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = wave_max(uint32_t(v >> 32));
  return uint64_t(hi) << 32 | wave_max(uint32_t(v >> 32) == hi ? uint32_t(v) : 0u);
}

template <int PER>
__device__ __forceinline__ void load_bias(const RouteArgs& a, int lane, float (&bias)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) bias[i] = a.bias && i * 64 + lane < a.E ? a.bias[i * 64 + lane] : 0.f;
}

// One wave chooses one token's experts and writes their weights; l[i] and bias[i] are those of expert
// 64 i + lane.  Each round takes the largest score + bias left, the lowest index among equals (scores
// of other logits may be equal: a sigmoid of 40 and of 50 are both 1); lane t keeps the t-th choice.
template <int PER>
__device__ __forceinline__ void choose_experts(const RouteArgs& a, int64_t m, const double (&l)[PER], const float (&bias)[PER],
                                               int lane) {
  const bool sig = (a.flags & SVDQ_ROUTE_SIGMOID) != 0;
  double top = 0.0, sum = 1.0;
  if (!sig) {
    uint64_t t = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint64_t o = i * 64 + lane < a.E ? order_of(l[i]) : 0;
      t = o > t ? o : t;
    }
    t = wave_max(t);
    top = __builtin_bit_cast(double, t >> 63 ? t & ~(uint64_t(1) << 63) : ~t);
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * 64 + lane < a.E) sum += exp(l[i] - top);
    sum = wave_sum(sum);
  }
  double p[PER];
  uint64_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    p[i] = sig ? 1.0 / (1.0 + exp(-l[i])) : exp(l[i] - top) / sum;
    key[i] = i * 64 + lane < a.E ? order_of(p[i] + double(bias[i])) : 0;
  }
  int id = 0;
  double mine = 0.0;
  for (int t = 0; t < a.top_k; ++t) {
    uint64_t best = 0;
    int at = 0;
    double v = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] > best) { best = key[i]; at = i; v = p[i]; }
    const uint64_t most = wave_max(best);
    const uint64_t tied = __ballot(best == most);
    int from = __ffsll((unsigned long long)tied) - 1;
    if (tied & (tied - 1)) {                               // equal keys: the lowest index
      const uint32_t low = ~wave_max(best == most ? ~uint32_t(at * 64 + lane) : 0u);
      from = int(low & 63u);
    }
    const int e = __builtin_amdgcn_readlane(at, from) * 64 + from;
    const double won = lane_value(v, from);
    if (lane == t) { id = e; mine = won; }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane == from && at == i) key[i] = 0;
  }
  if (a.flags & SVDQ_ROUTE_RENORM) {
    const double s = wave_sum(mine);                       // 0 in lanes without a choice
    mine = s == 0.0 ? 0.0 : mine / s;
  }
  if (lane < a.top_k) {
    a.ids[m * a.top_k + lane] = id;
    a.weights[m * a.top_k + lane] = float(mine * double(a.scale));
  }
}

// Logits in fp64: products of two bf16 are exact there and the sums keep 53 bits, so which expert
// is chosen does not hang on the order of summation.
//
// One workgroup: a token.  Wave w takes experts w, w + 16, ..., four at a time, its lanes 8
// consecutive K each; wave 0 then chooses.  Bound by the CU's fp64 conversions and FMAs: 1 x 2048 ->
// 64, 7.5 us (10.4 us a call).
constexpr int kRouteOneWaves = 16;
template <int PER>
__global__ void __launch_bounds__(1024) route_one_kernel(RouteArgs a) {
  __shared__ double logit[kMoeMaxE];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m = blockIdx.x;
  const uint16_t* const x = a.X + m * a.ldx;
  for (int e0 = w; e0 < a.E; e0 += 4 * kRouteOneWaves) {
    double acc[4] = {};
    for (int k = lane * 8; k < a.K; k += 512) {
      uint4 q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = e0 + i * kRouteOneWaves;
        q[i] = *reinterpret_cast<const uint4*>(a.Wr + int64_t(e < a.E ? e : e0) * a.K + k);
      }
      float xf[8];
      unpack_bf8(*reinterpret_cast<const uint4*>(x + k), xf);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float wf[8];
        unpack_bf8(q[i], wf);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i] = fma(double(wf[j]), double(xf[j]), acc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double v = wave_sum(acc[i]);
      if (lane == 0 && e0 + i * kRouteOneWaves < a.E) logit[e0 + i * kRouteOneWaves] = v;
    }
  }
  float bias[PER];
  load_bias<PER>(a, lane, bias);
  __syncthreads();
  if (w) return;
  double l[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) l[i] = i * 64 + lane < a.E ? logit[i * 64 + lane] : 0.0;
  choose_experts<PER>(a, m, l, bias, lane);
}

// A tile of 16 experts x 16 tokens and one of Z parts of K on the fp64 MFMA (16x16x4): lane (r, c)
// holds 8 consecutive K of expert and token r, so element e of both operands is one MFMA's K.  The
// waves take every fourth 32 of K; their sums meet in LDS, the parts' in the next kernel.  Bound by
// the fp64 units (1000 x 2888 -> 128: 23.4 us, the MFMA busy 49% of a SIMD's time beside the conversions
// of its operands; tiles of 32 x 32, half the conversions an MFMA: 26 us).
typedef double v4d __attribute__((ext_vector_type(4)));
__global__ void __launch_bounds__(256) route_logits_kernel(RouteArgs a) {
  constexpr int AHEAD = 4;                                 // steps of one batch of loads
  __shared__ v4d part[4][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int e0 = blockIdx.x * 16, steps = (a.K + 31) / 32;
  const int s0 = int(int64_t(blockIdx.z) * steps / a.Z), s1 = int(int64_t(blockIdx.z + 1) * steps / a.Z);
  const uint16_t* const wp = a.Wr + int64_t(e0 + r < a.E ? e0 + r : a.E - 1) * a.K;
  for (int64_t m0 = int64_t(blockIdx.y) * 16; m0 < a.M; m0 += int64_t(gridDim.y) * 16) {
    const uint16_t* const xp = a.X + (m0 + r < a.M ? m0 + r : a.M - 1) * a.ldx;
    v4d acc = {0.0, 0.0, 0.0, 0.0};
    // two batches in flight; past the part's end and K's (a multiple of 8) zeros
    uint4 q[2][AHEAD], x[2][AHEAD];
    auto load = [&](int s, uint4 (&qs)[AHEAD], uint4 (&xs)[AHEAD]) {
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int k = (s + 4 * j) * 32 + c * 8;
        const bool there = s + 4 * j < s1 && k < a.K;
        qs[j] = *reinterpret_cast<const uint4*>(wp + (there ? k : 0));
        xs[j] = *reinterpret_cast<const uint4*>(xp + (there ? k : 0));
        if (!there) qs[j] = xs[j] = make_uint4(0u, 0u, 0u, 0u);
      }
    };
    auto add = [&](const uint4 (&qs)[AHEAD], const uint4 (&xs)[AHEAD]) {
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        float wf[8], xf[8];
        unpack_bf8(qs[j], wf);
        unpack_bf8(xs[j], xf);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          acc = __builtin_amdgcn_mfma_f64_16x16x4f64(double(wf[e]), double(xf[e]), acc, 0, 0, 0);
      }
    };
    load(s0 + w, q[0], x[0]);
    for (int s = s0 + w; s < s1; s += 8 * AHEAD) {
      load(s + 4 * AHEAD, q[1], x[1]);
      add(q[0], x[0]);
      if (s + 4 * AHEAD >= s1) break;
      load(s + 8 * AHEAD, q[0], x[0]);
      add(q[1], x[1]);
    }
    part[w][lane] = acc;
    __syncthreads();
    if (w == 0) {
      acc = part[0][lane] + part[1][lane] + part[2][lane] + part[3][lane];
      // column (token) r, rows (experts) c, c + 4, c + 8, c + 12
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (m0 + r < a.M && e0 + i * 4 + c < a.E)
          a.logits[(blockIdx.z * a.M + m0 + r) * a.E + e0 + i * 4 + c] = acc[i];
    }
    __syncthreads();
  }
}

// One wave a token.
template <int PER>
__global__ void __launch_bounds__(256) route_choose_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float bias[PER];
  load_bias<PER>(a, lane, bias);
  for (int64_t m = int64_t(blockIdx.x) * 4 + w; m < a.M; m += int64_t(gridDim.x) * 4) {
    double l[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = 0.0;
    for (int z0 = 0; z0 < a.Z; z0 += 4) {                  // four parts' loads at once
      double v[4][PER];
#pragma unroll
      for (int z = 0; z < 4; ++z)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int e = i * 64 + lane;
          v[z][i] = a.logits[((z0 + z < a.Z ? z0 + z : z0) * a.M + m) * a.E + (e < a.E ? e : 0)];
        }
#pragma unroll
      for (int z = 0; z < 4; ++z)
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (z0 + z < a.Z) l[i] += v[z][i];
    }
    choose_experts<PER>(a, m, l, bias, lane);
  }
}

hipError_t launch_moe_route(const uint16_t* X, int64_t M, int64_t ldx, int K, const uint16_t* Wr, const float* bias,
                            int E, int top_k, uint32_t flags, float scale, int32_t* ids, float* weights, double* logits,
                            hipStream_t s) {
  RouteArgs a{};
  a.X = X; a.Wr = Wr; a.bias = bias; a.logits = logits; a.ids = ids; a.weights = weights;
  a.ldx = ldx; a.M = M; a.K = K; a.E = E; a.top_k = top_k; a.flags = flags; a.scale = scale;
  const auto cap = [](int64_t v) { return unsigned(v < 65535 ? v : 65535); };
#define SVDQ_ROUTE(KERNEL_, GRID_, BLOCK_)                                                   \
  do {                                                                                       \
    if (E <= 64) hipLaunchKernelGGL((KERNEL_<1>), GRID_, BLOCK_, 0, s, a);                   \
    else if (E <= 128) hipLaunchKernelGGL((KERNEL_<2>), GRID_, BLOCK_, 0, s, a);             \
    else if (E <= 256) hipLaunchKernelGGL((KERNEL_<4>), GRID_, BLOCK_, 0, s, a);             \
    else hipLaunchKernelGGL((KERNEL_<8>), GRID_, BLOCK_, 0, s, a);                           \
  } while (0)
  if (route_one(M, K, E)) {
    SVDQ_ROUTE(route_one_kernel, dim3(unsigned(M)), dim3(64 * kRouteOneWaves));
    return hipGetLastError();
  }
  a.Z = route_splits(M, K, E);
  hipLaunchKernelGGL(route_logits_kernel, dim3(unsigned((E + 15) / 16), cap((M + 15) / 16), unsigned(a.Z)), dim3(256), 0,
                     s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  SVDQ_ROUTE(route_choose_kernel, dim3(cap((M + 3) / 4)), dim3(256));
#undef SVDQ_ROUTE
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
  uint16_t* h;                         // S x P x F bf16 planes, each 128 of F in operand order (stored_at)
  int32_t* plan;                       // the down kernel's column blocks (moe_plan)
  float* o;                            // P x N: the pairs' down products (long calls)
  void* Y;
  int64_t ldx, ldy, Ng_pad, Nd_pad;
  int H, F, N, E, top_k, P;            // gate/up: H -> 2 F, down: F -> N
  int d_int4;
  int slots, down_slots, KW;           // blocks of pairs at most; waves that share a tile's K
  int planes;                          // of h
  int cols, cols_inv;                  // unplanned gate/up: pairs a block, 65536 / cols rounded up
  uint32_t epi, inv_h, inv_f;          // segment_inverse of H and F
};

// i / (K / 512) as i * segment_inverse(K) >> 20, for i up to 16 rows of at most 128 segments.
__host__ __device__ inline uint32_t segment_inverse(int K) { return ((1u << 20) + K / 512 - 1) / (K / 512); }

// A column of an MFMA that no pair has: beyond every buffer, so its loads read nothing (zeros).
constexpr uint32_t kNoColumn = 0x80000000u;

// The plan of moe_down_kernel: its units, kPlanWords words each: expert, pairs, K chunk, K chunks,
// and the pairs (at most 16 / S of one expert, all their planes being columns of one MFMA); units
// without pairs end every wave's sequence.  An expert's pairs stand in the order of their numbers, so
// which of them share a block does not change from call to call: a full block and a shorter one may
// form their sums differently (rows that do not fit the LDS whole come in parts).
constexpr int kPlanWords = 16;
constexpr int kDownWaves = 16;
constexpr int kDownMinSlots = 256;     // pairs x K chunks that the LDS sums have room for at least
__device__ __forceinline__ int down_slots(int P) { return P > kDownMinSlots ? P : kDownMinSlots; }

// With GATE it also holds, from kGatePlan on, the gate/up product's blocks: expert, pairs and up to 16
// pairs of kGatePlanWords words each, ended by blocks without pairs up to the grid's `slots`.
constexpr int kGatePlan = 16384;       // in words
constexpr int kGatePlanWords = 32;
constexpr int kPlanWaves = 8;
constexpr int kPlanRounds = kMoeMaxPairs / (64 * kPlanWaves);
constexpr int kPlanLdsWords = (kPlanWaves + 3) * kMoeMaxE + 2;
template <bool GATE>
__device__ __forceinline__ void moe_plan(const MoeArgs& a, int* lds) {
  constexpr int THREADS = 64 * kPlanWaves;
  const int TPB = a.planes == 3 ? tokens_per_block(3) : tokens_per_block(2);
  // before[w]: an expert's pairs that wave w has met, then those of the waves before it
  int *const before = lds, *const count = lds + kPlanWaves * kMoeMaxE, *const base = count + kMoeMaxE, *const gbase = base + kMoeMaxE;
  int &total = gbase[kMoeMaxE], &gtotal = gbase[kMoeMaxE + 1];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  int* const met = before + w * kMoeMaxE;
  for (int e = lane; e < a.E; e += 64) met[e] = 0;
  // a wave takes consecutive pairs, 64 a round; a pair's place among its expert's in the wave
  const int rounds = (a.P + THREADS - 1) / THREADS, p0 = w * rounds * 64 + lane;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  int ex[kPlanRounds], at[kPlanRounds];
#pragma unroll
  for (int r = 0; r < kPlanRounds; ++r) {
    const int p = p0 + r * 64, id = r < rounds && p < a.P ? a.ids[p] : -1;
    ex[r] = id < a.E ? id : -1;
  }
#pragma unroll
  for (int r = 0; r < kPlanRounds; ++r) {
    if (r >= rounds) break;
    const bool valid = ex[r] >= 0;
    uint64_t same = __ballot(valid);                       // lanes with this one's expert
#pragma unroll
    for (int b = 1; b < kMoeMaxE; b <<= 1) {
      const uint64_t set = __ballot((ex[r] & b) != 0);
      same &= ex[r] & b ? set : ~set;
    }
    keep_order();                                          // one wave's LDS operations are in order
    const int met_before = valid ? met[ex[r]] : 0;
    at[r] = met_before + __popcll(same & below);
    keep_order();
    if (valid && !(same & below)) met[ex[r]] = met_before + __popcll(same);
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += THREADS) {
    int n = 0;
#pragma unroll
    for (int v = 0; v < kPlanWaves; ++v) {
      const int m = before[v * kMoeMaxE + e];
      before[v * kMoeMaxE + e] = n;
      n += m;
    }
    count[e] = n;
  }
  __syncthreads();
  if (tid < (GATE ? 128 : 64)) {                           // one wave for each kind of block
    const int size = tid < 64 ? TPB : 16;
    int blocks = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + lane, nb = e < a.E ? (count[e] + size - 1) / size : 0;
      int sb = nb;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(sb, o);
        if (lane >= o) sb += v;
      }
      if (e < a.E) (tid < 64 ? base : gbase)[e] = blocks + sb - nb;   // the expert's first block
      blocks += __shfl(sb, 63);
    }
    if (lane == 0) (tid < 64 ? total : gtotal) = blocks;
  }
  __syncthreads();
  // as many chunks of K as it takes to give every wave a unit, where the LDS has room
  const int KS = a.F / kKStep, slots = down_slots(a.P);
  int KC = 1;
  while (!a.o && total * KC < kDownWaves && KC * 2 <= KS && KC * 2 * a.P <= slots) KC *= 2;
  int32_t* const gate = a.plan + kGatePlan;
  for (int e = tid; e < a.E; e += THREADS) {
    const int cnt = count[e];
    if (GATE)
      for (int b = 0; b * 16 < cnt; ++b)
        *reinterpret_cast<int2*>(gate + kGatePlanWords * (gbase[e] + b)) = make_int2(e, cnt - b * 16 < 16 ? cnt - b * 16 : 16);
    for (int b = 0; b * TPB < cnt; ++b)
      for (int k = 0; k < KC; ++k)
        *reinterpret_cast<int4*>(a.plan + kPlanWords * ((base[e] + b) * KC + k)) =
            make_int4(e, cnt - b * TPB < TPB ? cnt - b * TPB : TPB, k, KC);
  }
  // (the down product by pairs has a grid of its own, which may reach further)
  const int ends = a.o ? a.down_slots - total : 2 * kDownWaves;
  for (int i = tid; i < ends; i += THREADS)
    *reinterpret_cast<int4*>(a.plan + kPlanWords * (total * KC + i)) = make_int4(0, 0, 0, KC);
  if (GATE)
    for (int i = gtotal + tid; i < a.slots; i += THREADS)
      *reinterpret_cast<int2*>(gate + kGatePlanWords * i) = make_int2(0, 0);
#pragma unroll
  for (int r = 0; r < kPlanRounds; ++r) {
    if (ex[r] < 0) continue;
    const int p = p0 + r * 64, i = met[ex[r]] + at[r];
    const int b = a.planes == 3 ? i / tokens_per_block(3) : i / tokens_per_block(2);
    for (int k = 0; k < KC; ++k) a.plan[kPlanWords * ((base[ex[r]] + b) * KC + k) + 4 + i - b * TPB] = p;
    if (GATE) gate[kGatePlanWords * (gbase[ex[r]] + i / 16) + 2 + i % 16] = p;
  }
}

__global__ void __launch_bounds__(512) moe_plan_kernel(MoeArgs a) {
  __shared__ int lds[kPlanLdsWords];
  moe_plan<true>(a, lds);
}

// Rows in LDS (S planes x n rows of K bf16, row_b bytes apart) to fp16, in place, scaled by
// 2^f16_row_power of each row's largest magnitude, whose bits go to top[0 .. n): the planes' sum becomes
// fp16 hi (+ lo).  One wave takes a row.  The rows are written before; the caller's barrier follows.
template <int S, int WAVES>
__device__ __forceinline__ void rows_to_f16(uint8_t* xl, int row_b, int K, int n, uint32_t* top) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  lds_barrier();
  for (int r = w; r < n; r += WAVES) {
    uint32_t m = 0;
    for (int k = lane * 8; k < K; k += 512) {
      const uint4 q = *reinterpret_cast<const uint4*>(xl + r * row_b + k * 2);
      const uint32_t d[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t hi = d[i] & 0x7FFF0000u, lo = (d[i] << 16) & 0x7FFF0000u;
        m = hi > m ? hi : m;
        m = lo > m ? lo : m;
      }
    }
    m = wave_max(m);
    if (lane == 0) top[r] = m;
    const int s = f16_row_power(__uint_as_float(m));
    for (int k = lane * 8; k < K; k += 512) {
      float v[8];
      unpack_bf8(*reinterpret_cast<const uint4*>(xl + r * row_b + k * 2), v);
#pragma unroll
      for (int p = 1; p < S; ++p) {
        float l[8];
        unpack_bf8(*reinterpret_cast<const uint4*>(xl + (p * n + r) * row_b + k * 2), l);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += l[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = ldexpf(v[e], s);
#pragma unroll
      for (int p = 0; p < S; ++p) {
        const uint4 h = to_f16(v);
        *reinterpret_cast<uint4*>(xl + (p * n + r) * row_b + k * 2) = h;
        float b[8];
        unpack_h8(h, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] -= b[e];
      }
    }
  }
}

// Rows of one expert for a block of its pairs: the gate and up rows (a tile is 16 gate and the same
// 16 up rows), or, DOWN, down rows of long calls (a tile is 32 rows, and a pair's sums go to memory,
// where moe_join_kernel adds a token's pairs).
// The workgroup takes 8 / KW tiles and the blockIdx.y-th block: up to 16 pairs (DOWN: 16 / S, all
// their planes being columns).  KW waves share a tile's K (every KW-th 128-K step each); KW is the
// smallest that fills the GPU, since with few there is little exchange and a wave streams long runs
// of codes.  (Blocks of 32 pairs, which halve the reads of an expert with many, left one workgroup
// a CU and were 4% slower at 48 tokens, 8 of 24 experts, 3584 -> 1536.)
// PLANNED: the blocks are in the plan.  Otherwise (gate/up of at most 64 pairs, a wave's lanes) every
// wave finds its block of up to a.cols pairs by ballots, which saves the plan's launch, and the grid's
// last row (blockIdx.y == slots) holds one workgroup that writes the plan for the down product.  Whole
// calls by ballots and with a plan: 2 pairs 13.6 / 17.4 us, 16 22.9 / 26.2, 64 (16 tokens, 4 of 32, 2048
// -> 2 x 1024 MXFP4) 37.0 / 39.8; INT4 and NVFP4 2 to 4 us likewise, but 16 tokens, 4 of 64, 4096 INT4 80.3 / 78.5.
//
// Bound by the weights' bytes where experts have few pairs: MXFP4, 64 tokens, 6 of 64 experts, 4096 ->
// 2 x 2048, gate/up 100 us for 571 MB (5.7 TB/s; a kernel that only reads reaches 6.1), down 57 us for
// 285 MB (5.0 TB/s).  By L1 and LDS reads of the columns where they have many: 128 tokens, 4 of 16,
// 2048 -> 2 x 1024, 19 and 19 us (experts of 32 pairs are read two and four times, from L2).  By
// latency at one token: 4 of 32, 2048 -> 2 x 2048, 8.5 us for 18 MB.
constexpr int kGateWaves = 8;
constexpr int kGateFill = 2048;
constexpr int kGateXLds = 81664;       // two workgroups a CU
template <int FMT, int S, bool PLANNED>
__global__ void __launch_bounds__(512, 4) moe_rows_kernel(MoeArgs a) {
  constexpr bool DOWN = S > 1;
  constexpr int TPB = tokens_per_block(S);
  static_assert(PLANNED || !DOWN, "down blocks are planned");
  extern __shared__ uint4 xlds[];                          // kGateXLds bytes
  v4f (*const red)[2][64] = reinterpret_cast<v4f(*)[2][64]>(xlds);   // after the rows of X
  constexpr bool F16 = FMT == kFmtNVFP4;                   // rows in LDS become fp16
  __shared__ uint32_t top[TPB];
  const int tid = threadIdx.x;
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tl = lane & 15, c = lane >> 4;
  const int slot = blockIdx.y;
  int ex = -1, T = 0, mine = 0;        // the expert, the block's pairs; lane i holds the i-th
  if constexpr (PLANNED) {
    const int words = DOWN ? a.plan[kPlanWords * slot + tl] : a.plan[kGatePlan + kGatePlanWords * slot + (lane & 31)];
    ex = __builtin_amdgcn_readlane(words, 0);
    T = __builtin_amdgcn_readlane(words, 1);
    if (T == 0) return;
    mine = __shfl(words, (lane & 15) + (DOWN ? 4 : 2));
  } else {
    if (slot == a.slots) {
      if (blockIdx.x == 0) moe_plan<false>(a, reinterpret_cast<int*>(xlds));
      return;
    }
    const uint64_t below = (uint64_t(1) << lane) - 1;
    const int id = lane < a.P ? a.ids[lane] : -1;
    uint64_t left = __ballot(id >= 0 && id < a.E), eq = 0;
    int t0 = slot;                                         // the block among the expert's
    while (left) {
      ex = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
      eq = __ballot(id == ex);
      const int blocks = (__popcll(eq) + a.cols - 1) * a.cols_inv >> 16;
      if (t0 < blocks) break;
      t0 -= blocks;
      left &= ~eq;
    }
    if (!left) return;
    T = __popcll(eq);
    t0 *= a.cols;                                          // its first pair
    const int to = eq >> lane & 1 ? __popcll(eq & below) : T + __popcll(~eq & below);
    mine = __shfl(__builtin_amdgcn_ds_permute(to * 4, lane), (lane + t0) & 63);
    T = T - t0 < a.cols ? T - t0 : a.cols;
  }
  ex = __builtin_amdgcn_readfirstlane(ex);
  auto pair_of = [&](int i) { return __shfl(mine, i); };

  const uint8_t* const blob = DOWN ? a.wd + size_t(ex) * a.blob_d : a.wg + size_t(ex) * a.blob_g;
  const int K = DOWN ? a.F : a.H, KS = K / kKStep, KW = a.KW, kq = w % KW;
  const int ft = blockIdx.x * (kGateWaves / KW) + w / KW;
  const bool there = !DOWN || ft * 32 < a.N;               // the last workgroup may have tiles too many
  const int rt0 = DOWN ? ft * 2 : ft, rt1 = DOWN ? ft * 2 + 1 : a.F / 16 + ft;
  const int n = there && KS > kq ? (KS - kq + KW - 1) / KW : 0;
  const W4Rows<FMT> rows(blob + (DOWN ? a.d_codes : a.g_codes), blob + (DOWN ? a.d_scales : a.g_scales), K,
                         DOWN ? a.Nd_pad : a.Ng_pad);
  const uint16_t* const xbase = DOWN ? a.h : a.X;
  const float gs = w4_tensor_scale<FMT>(blob + (DOWN ? a.d_amax : a.g_amax));
  const uint32_t xbytes = uint32_t((DOWN ? int64_t(S) * a.P * a.F : int64_t(a.P / a.top_k - 1) * a.ldx + a.H) * 2);
  // element offset of a pair's row of X (of h)
  auto row_of = [&](int p, int plane) -> int64_t { return DOWN ? (int64_t(plane) * a.P + p) * a.F : int64_t(p / a.top_k) * a.ldx; };
  {
    v4f ag = {0.f, 0.f, 0.f, 0.f}, au = ag;
    auto load_w = [&](int i, W4Stage<FMT>& g, W4Stage<FMT>& u) {
      const uint32_t ks = uint32_t(kq + i * KW);
      rows.load(rt0, ks, i < n, lane, g);
      rows.load(rt1, ks, i < n, lane, u);
    };
    // The block's rows of X (of h) go through LDS: a load of a step's columns from memory costs the L1
    // as many cycles as sixteen, however many there are, for every wave.  Rows too long for it
    // come in parts.
    const int xrows = S * T;
    uint8_t* const xl = reinterpret_cast<uint8_t*>(xlds);
    // kc of K from k0 on; a wave's copies of 64 lanes x 16 bytes, `batch` in flight (an absent one,
    // through a buffer of no bytes, still costs the L1 a load)
    auto fill_by = [&](auto batch, int k0, int segs, int row_b, uint32_t inv) {
      constexpr int N = decltype(batch)::value;
      for (int g0 = w; g0 < xrows * segs; g0 += N * kGateWaves) {
        uint4 v[N];
        int at[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int g = g0 + j * kGateWaves;
          const int r = int(uint32_t(g) * inv >> 20), seg = g - r * segs, plane = (S > 1 && r >= T) + (S > 2 && r >= 2 * T);
          const int p = __builtin_amdgcn_readlane(mine, (r - plane * T) & 15);
          v[j] = buffer_load16(make_rsrc(xbase, g < xrows * segs ? xbytes : 0), uint32_t(lane) * 16,
                               uint32_t(row_of(p, plane) + k0 + seg * 512) * 2);
          at[j] = r * row_b + seg * 1024;
        }
        keep_order();                                      // all loads before the first store
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (g0 + j * kGateWaves < xrows * segs) *reinterpret_cast<uint4*>(xl + at[j] + lane * 16) = v[j];
      }
    };
    auto fill = [&](int k0, int kc, int row_b, uint32_t inv) {
      if (xrows * kc <= 2 * kGateWaves * 512)
        fill_by(std::integral_constant<int, 1>(), k0, kc / 512, row_b, inv);
      else
        fill_by(std::integral_constant<int, 8>(), k0, kc / 512, row_b, inv);
    };
    const int t = tl % TPB, pl = tl / TPB;
    const int row = pl < S && t < T ? pl * T + t : 0;        // any where there is no column
    auto operands = [&](const uint8_t* xp, int k, uint4 (&x)[4]) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        x[u] = *reinterpret_cast<const uint4*>(xp + (k + (DOWN ? u * 32 + c * 8 : k_of<FMT>(c, u))) * 2);
    };
    if (!PLANNED || xrows * few_row_bytes(K) <= kGateXLds) {
      const int row_b = few_row_bytes(K);
      constexpr int AHEAD = FMT == kFmtINT4 ? 3 : 4;
      W4Stage<FMT> sg[AHEAD], su[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        load_w(j, sg[j], su[j]);
        keep_order();
      }
      fill(0, K, row_b, DOWN ? a.inv_f : a.inv_h);
      if constexpr (F16) rows_to_f16<S, kGateWaves>(xl, row_b, K, T, top);
      lds_barrier();
      const uint8_t* const xp = xl + row * row_b;
      for (int i0 = 0; i0 < n; i0 += AHEAD) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          const int ks = kq + (i0 + j < n ? i0 + j : n - 1) * KW;   // past the last step: codes are zeros
          uint4 x[4];
          operands(xp, ks * kKStep, x);
          w4_step<FMT, F16>(sg[j], ks, x, ag);
          w4_step<FMT, F16>(su[j], ks, x, au);
          load_w(i0 + j + AHEAD, sg[j], su[j]);
          keep_order();
        }
      }
      if constexpr (F16) {
        const int back = -f16_row_power(__uint_as_float(top[t < T ? t : 0]));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ag[e] = ldexpf(ag[e], back);
          au[e] = ldexpf(au[e], back);
        }
      }
    } else {
      // a part is a multiple of 2048 of K, so each wave has an even number of its steps
      constexpr int AHEAD = 2;
      const int KC = (kGateXLds / xrows - 16) / 2 & ~2047, row_b = few_row_bytes(KC), per = KC / kKStep / KW;
      const uint8_t* const xp = xl + row * row_b;
      W4Stage<FMT> sg[AHEAD], su[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        load_w(j, sg[j], su[j]);
        keep_order();
      }
      for (int k0 = 0, i = 0; k0 < K; k0 += KC) {
        if (k0) lds_barrier();                             // the part before is read
        const int kc = K - k0 < KC ? K - k0 : KC;
        fill_by(std::integral_constant<int, 8>(), k0, kc / 512, row_b, segment_inverse(kc));
        lds_barrier();
        for (const int end = i + per < n ? i + per : n; i < end; i += AHEAD) {
#pragma unroll
          for (int j = 0; j < AHEAD; ++j) {
            const int ks = kq + (i + j < n ? i + j : n - 1) * KW;   // past the last step: codes are zeros
            uint4 x[4];
            operands(xp, ks * kKStep - k0, x);
            w4_step<FMT>(sg[j], ks, x, ag);
            w4_step<FMT>(su[j], ks, x, au);
            load_w(i + j + AHEAD, sg[j], su[j]);
            keep_order();
          }
        }
      }
    }
    if (KW > 1) {
      lds_barrier();
      red[w][0][lane] = ag;
      red[w][1][lane] = au;
      lds_barrier();
    }
    if constexpr (DOWN) {
      if (kq == 0) {
        v4f y[2] = {ag, au};
#pragma unroll
        for (int v = 1; v < kGateWaves; ++v)
          if (v < KW) {
            y[0] += red[w + v][0][lane];
            y[1] += red[w + v][1][lane];
          }
        const int p = pair_of(tl < T ? tl : 0);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          v4f sum = y[q];                                  // the planes' columns of a pair
#pragma unroll
          for (int i = 1; i < S; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += __shfl(y[q][e], lane + i * TPB);
          const int row = ft * 32 + q * 16 + c * 4;
          if (tl >= T || row >= a.N) continue;
          if (FMT == kFmtNVFP4) sum *= gs;
          if (a.epi & SVDQ_EPI_BIAS) {
            const uint2 bd = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(blob + a.d_bias) + row);
            sum += v4f{bf_lo(bd.x), bf_hi(bd.x), bf_lo(bd.y), bf_hi(bd.y)};
          }
          *reinterpret_cast<v4f*>(a.o + int64_t(p) * a.N + row) = sum;
        }
      }
    } else if (kq == 0) {
      const int p = pair_of(tl < T ? tl : 0);
      if (tl < T) {
        v4f g = ag, u = au;                                // rows 4 c .. 4 c + 3 of pair p
        for (int v = 1; v < KW; ++v) {
          g += red[w + v][0][lane];
          u += red[w + v][1][lane];
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
        uint4 hp[3];
        split_planes<3>(hv, hp);
        // in the order of the down product's operands
        const int kk = row & (kKStep - 1), at = row - kk + (a.d_int4 ? stored_at<kFmtINT4>(kk) : stored_at<kFmtMXFP4>(kk));
#pragma unroll
        for (int s = 0; s < 3; ++s)
          if (s < a.planes) *reinterpret_cast<uint2*>(a.h + (int64_t(s) * a.P + p) * a.F + at) = make_uint2(hp[s].x, hp[s].y);
      }
    }
  }
}

// Y[m] = sum_j w_j o[m, j], j in order; a pair without an expert adds nothing.  5.3 us for 64 tokens of
// 6 x 4096 (6.3 MB from L2): a launch's start and one round of loads.
template <bool OUT_F32>
__global__ void __launch_bounds__(256) moe_join_kernel(MoeArgs a) {
  const int per = a.N / 4, total = a.P / a.top_k * per;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    const int m = i / per, row = i % per * 4;
    v4f y = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < a.top_k; j0 += 4) {              // four pairs' loads at once
      int id[4];
      float wt[4];
      v4f v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = m * a.top_k + (j0 + j < a.top_k ? j0 + j : j0);
        id[j] = a.ids[p];
        wt[j] = a.weights[p];
        v[j] = *reinterpret_cast<const v4f*>(a.o + int64_t(p) * a.N + row);
      }
      keep_order();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j0 + j >= a.top_k || id[j] < 0 || id[j] >= a.E) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = fmaf(wt[j], v[j][e], y[e]);
      }
    }
    const int64_t at = int64_t(m) * a.ldy + row;
    if (OUT_F32)
      *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.Y) + at) = y;
    else
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.Y) + at) =
          make_uint2(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]));
  }
}

// Down rows.  One workgroup: 16 output rows of all tokens, 16 waves.  A unit is one column block of
// the plan and one of KC chunks of K; waves take every sixteenth unit, one pipeline running on from
// unit to unit, and leave each pair's sums in a place of its own, so the sum over a token's experts
// has one order.  Bound by the latency of the first loads and by one CU's L1: 8.4 us at one token, 4 of
// 32 experts, 2048 -> 2048 MXFP4 (9 MB).  Calls with more steps go through memory (moe_by_pairs): 7
// tokens, 5 of 60, 1024 -> 2560 NVFP4 takes 19.2 us here (160 workgroups for 256 CUs) and 11.6 + 3.8 there.
constexpr int64_t kDownLds = 163840;   // HL: all of h in LDS where it fits (one workgroup a CU)

template <int FMT, int S, bool HL>
__global__ void __launch_bounds__(1024) moe_down_kernel(MoeArgs a) {
  constexpr int TPB = tokens_per_block(S);
  constexpr int DEPTH = HL ? 5 : 3;
  extern __shared__ v4f slot[];                    // [chunk][pair][4]: 16 rows of a pair; the pairs' weights; HL: h
  const int tid = threadIdx.x;
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tl = lane & 15, c = lane >> 4;
  float* const wt = reinterpret_cast<float*>(slot + down_slots(a.P) * 4);
  const int KS = a.F / kKStep;
  const int rt = blockIdx.x;
  const int t = tl % TPB, pl = tl / TPB;

  // a unit as its wave sees it; the plan's words are loaded one unit ahead
  struct Unit { const uint8_t* blob; int cnt, pair, kc, ks0, n, row; uint32_t xoff; };
  auto fetch = [&](int u) -> int { return a.plan[kPlanWords * u + tl]; };
  auto open = [&](int words, Unit& d) {
    d.cnt = __builtin_amdgcn_readlane(words, 1);
    d.kc = __builtin_amdgcn_readlane(words, 2);
    const int KC = __builtin_amdgcn_readlane(words, 3);
    d.blob = a.wd + size_t(__builtin_amdgcn_readlane(words, 0)) * a.blob_d;
    const bool column = pl < S && t < d.cnt;
    d.pair = __shfl(words, 4 + (t < d.cnt ? t : 0));
    d.row = column ? pl * a.P + d.pair : 0;                // HL: any row where there is no column
    d.ks0 = d.kc * KS / KC;
    d.n = d.cnt ? (d.kc + 1) * KS / KC - d.ks0 : 0;
    d.xoff = column ? uint32_t(((pl * a.P + d.pair) * int64_t(a.F) + c * 8) * 2) : kNoColumn;
  };
  const uint32_t h_bytes = uint32_t(int64_t(S) * a.P * a.F * 2);
  struct Stage { W4Stage<FMT> w; uint4 x[4]; };                    // x unused with HL
  Stage st[DEPTH];
  constexpr bool F16 = HL && FMT == kFmtNVFP4;             // h becomes fp16
  uint32_t* const top = reinterpret_cast<uint32_t*>(wt + (a.P + 3) / 4 * 4);
  uint8_t* const hl = reinterpret_cast<uint8_t*>(top + (a.P + 3) / 4 * 4);
  const int row_b = few_row_bytes(a.F);
  int lu = w, li = 0, words = fetch(w);
  Unit ld, cu;                                             // the unit being loaded, the one being computed
  auto enter = [&]() {                                     // the load side's next unit
    open(words, ld);
    if (ld.n) words = fetch(lu + kDownWaves);
  };
  auto load = [&](Stage& s) {
    const bool valid = li < ld.n;
    const uint32_t ks = uint32_t(ld.ks0 + li);
    const W4Rows<FMT> rows(ld.blob + a.d_codes, ld.blob + a.d_scales, a.F, a.Nd_pad);
    rows.load(rt, ks, valid, lane, s.w);
    if constexpr (!HL) {
      const __amdgpu_buffer_rsrc_t r = make_rsrc(a.h, valid ? h_bytes : 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) s.x[q] = buffer_load16(r, ld.xoff + q * 64, ks * kKStep * 2);
    }
    if (++li >= ld.n && ld.n) {
      li = 0;
      lu += kDownWaves;
      enter();
    }
  };
  int u = w;
  const int first_words = words, KC = __builtin_amdgcn_readlane(words, 3);
  enter();
#pragma unroll
  for (int j = 0; j < DEPTH; ++j) {
    load(st[j]);
    keep_order();
  }
  // the compute side: the words one unit ahead too, the unit's tensor scale and bias when it opens
  int cwords = first_words;
  float gs = 1.0f;
  uint2 bias = make_uint2(0u, 0u);
  auto begin = [&]() {
    open(cwords, cu);
    if (cu.n) cwords = fetch(u + kDownWaves);
    gs = w4_tensor_scale<FMT>(cu.blob + a.d_amax);
    if (cu.kc == 0 && (a.epi & SVDQ_EPI_BIAS))
      bias = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(cu.blob + a.d_bias) + rt * 16 + c * 4);
    else
      bias = make_uint2(0u, 0u);
  };
  begin();
  if constexpr (HL) {
    // a wave's copies of 64 lanes x 16 bytes, one after the other: together, the absent ones of few
    // pairs cost more (9.0 against 8.6 us at one token, 4 of 32 experts, 2048 -> 2048)
    const int segs = a.F / 512;
    for (int g = w; g < S * a.P * segs; g += kDownWaves)
      *reinterpret_cast<uint4*>(hl + g / segs * row_b + g % segs * 1024 + lane * 16) =
          reinterpret_cast<const uint4*>(a.h)[g * 64 + lane];
  }
  // the pairs' weights; a pair without an expert adds zero
  for (int p = tid; p < a.P; p += 1024) {
    const int id = a.ids[p];
    const bool there = id >= 0 && id < a.E;
    wt[p] = there ? a.weights[p] : 0.0f;
    if (!there)
      for (int k = 0; k < KC; ++k)
        for (int q = 0; q < 4; ++q) slot[(k * a.P + p) * 4 + q] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  if constexpr (F16) rows_to_f16<S, kDownWaves>(hl, row_b, a.F, a.P, top);
  if (HL) lds_barrier();
  int i = 0;
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  while (cu.n) {
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) {
      if constexpr (HL) {
        uint4 x[4];
        const int at = cu.ks0 + i < KS ? cu.ks0 + i : 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          x[q] = *reinterpret_cast<const uint4*>(hl + cu.row * row_b + (at * kKStep + q * 32 + c * 8) * 2);
        w4_step<FMT, F16>(st[j].w, cu.ks0 + i, x, acc);
      } else {
        w4_step<FMT>(st[j].w, cu.ks0 + i, st[j].x, acc);
      }
      load(st[j]);
      keep_order();
      if (cu.n && ++i == cu.n) {
        v4f y = acc;
        if constexpr (F16) {
          const int back = -f16_row_power(__uint_as_float(top[cu.pair]));
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = ldexpf(y[e], back);
        }
        if (FMT == kFmtNVFP4) y *= gs;
        v4f sum = y;                                       // the planes' columns of a pair
#pragma unroll
        for (int p = 1; p < S; ++p)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] += __shfl(y[e], lane + p * TPB);
        sum += v4f{bf_lo(bias.x), bf_hi(bias.x), bf_lo(bias.y), bf_hi(bias.y)};
        if (tl < cu.cnt) slot[(cu.kc * a.P + cu.pair) * 4 + c] = sum;
        acc = v4f{0.f, 0.f, 0.f, 0.f};
        i = 0;
        u += kDownWaves;
        begin();
      }
    }
  }
  lds_barrier();
  // Y[m] = sum_j w_j (sum over chunks), j and chunks in order
  const int M = a.P / a.top_k;
  for (int o = tid; o < M * 4; o += 1024) {
    const int m = o >> 2, q = o & 3;
    v4f y = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < a.top_k; ++j) {
      const int p = m * a.top_k + j;
      v4f v = slot[p * 4 + q];
      for (int k = 1; k < KC; ++k) v += slot[(k * a.P + p) * 4 + q];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = fmaf(wt[p], v[e], y[e]);
    }
    const int64_t at = int64_t(m) * a.ldy + rt * 16 + q * 4;
    if (S == 3)                                            // three planes: float32 output
      *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.Y) + at) = y;
    else
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.Y) + at) =
          make_uint2(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]));
  }
}

template <int FMT>
static void gate_up(const MoeArgs& a, hipStream_t s) {
  const unsigned tiles = unsigned(a.F / 16 * a.KW / kGateWaves);
  if (a.cols) {
    hipLaunchKernelGGL((moe_rows_kernel<FMT, 1, false>), dim3(tiles, unsigned(a.slots + 1)), dim3(512), kGateXLds, s, a);
  } else {
    hipLaunchKernelGGL(moe_plan_kernel, dim3(1), dim3(512), 0, s, a);
    hipLaunchKernelGGL((moe_rows_kernel<FMT, 1, true>), dim3(tiles, unsigned(a.slots)), dim3(512), kGateXLds, s, a);
  }
}

// Waves that share a tile's K: the fewest that make kGateFill waves (eight a CU) of the tiles that there
// are at least.  Whole call (us, in a graph) with 1, 2, 4 and 8 of them for gate/up, 1 to 16 tokens, 4 or
// 8 of 16 to 64 experts, 2048 -> 2 x 1024 MXFP4: 256 tiles 17.6 15.6 14.5 14.7, 512 19.9 17.9 16.6 17.5,
// 1024 23.7 22.0 22.4 26.9, 2048 27.7 28.6 31.3 40.9, 4096 40.7 43.2 54.7 81.6; INT4 and NVFP4 alike,
// and the down product by pairs (512 19.5 18.2 18.0 19.8, 1024 22.0 21.6 22.5 26.9, 2048 26.0 27.1 29.2
// 34.9).
static int waves_per_tile(int64_t tiles) {
  int kw = 1;
  while (kw < kGateWaves && tiles * kw < kGateFill) kw *= 2;
  return kw;
}

template <int FMT, int S>
static void down(MoeArgs a, hipStream_t s) {
  if (a.o) {
    const int experts = a.E < a.P ? a.E : a.P, tiles = (a.N + 31) / 32;
    a.KW = waves_per_tile(int64_t(experts) * tiles);
    const int per = kGateWaves / a.KW;
    const dim3 grid(unsigned((tiles + per - 1) / per), unsigned(a.down_slots));
    hipLaunchKernelGGL((moe_rows_kernel<FMT, S, true>), grid, dim3(512), kGateXLds, s, a);
    const int64_t quads = int64_t(a.P) / a.top_k * (a.N / 4);
    hipLaunchKernelGGL((moe_join_kernel<S == 3>), dim3(unsigned((quads + 255) / 256)), dim3(256), 0, s, a);
    return;
  }
  const int64_t sums = (a.P > kDownMinSlots ? a.P : kDownMinSlots) * 64 + int64_t(a.P + 3) / 4 * 32;
  const int64_t all = sums + int64_t(S) * a.P * few_row_bytes(a.F);
  const dim3 grid(unsigned(a.N / 16));
  if (all <= kDownLds)
    hipLaunchKernelGGL((moe_down_kernel<FMT, S, true>), grid, dim3(1024), size_t(all), s, a);
  else
    hipLaunchKernelGGL((moe_down_kernel<FMT, S, false>), grid, dim3(1024), size_t(sums), s, a);
}

// Requires 1 <= top_k <= kMoeMaxTopK, 1 <= E <= kMoeMaxE, H % 512 == 0, F % 512 == 0, N % 16 == 0, M >= 1.  ws has room for
// the plan and 3 planes of F values for each pair of one part (at most kMoeMaxPairs).
hipError_t launch_moe(int fmt_g, const uint8_t* wg, const WeightLayout& lg, int fmt_d, const uint8_t* wd,
                      const WeightLayout& ld, int H, int F, int N, int E, const uint16_t* X, int64_t M, int64_t ldx,
                      const int32_t* ids, const float* weights, int top_k, void* Y, int64_t ldy, uint32_t epi,
                      void* ws, hipStream_t s) {
  MoeArgs a{};
  a.wg = wg; a.blob_g = lg.total; a.g_codes = lg.codes; a.g_scales = lg.scales; a.g_bias = lg.bias; a.g_amax = lg.amax;
  a.wd = wd; a.blob_d = ld.total; a.d_codes = ld.codes; a.d_scales = ld.scales; a.d_bias = ld.bias; a.d_amax = ld.amax;
  a.plan = static_cast<int32_t*>(ws);
  a.h = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + kMoePlanBytes);
  float* const o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMoePlanBytes + moe_h_bytes(M, top_k, F));
  a.ldx = ldx; a.ldy = ldy; a.Ng_pad = lg.N_pad; a.Nd_pad = ld.N_pad;
  a.H = H; a.F = F; a.N = N; a.E = E; a.top_k = top_k; a.epi = epi; a.d_int4 = fmt_d == kFmtINT4;
  a.inv_h = segment_inverse(H); a.inv_f = segment_inverse(F);
  const bool f32 = (epi & SVDQ_EPI_OUT_F32) != 0;
  a.planes = f32 ? 3 : 2;
  // a part's pairs fit the kernels' LDS and its rows of X one buffer
  const int64_t span = (int64_t(1) << 31) / (2 * ldx), most = kMoeMaxPairs / top_k, part = span < most ? span : most;
  for (int64_t m0 = 0; m0 < M; m0 += part) {
    const int64_t mc = M - m0 < part ? M - m0 : part;
    a.P = int(mc * top_k);
    a.X = X + m0 * ldx;
    a.ids = ids + m0 * top_k;
    a.weights = weights + m0 * top_k;
    a.Y = static_cast<uint8_t*>(Y) + m0 * ldy * (f32 ? 4 : 2);
    const int experts = E < a.P ? E : a.P; // that may be asked for
    // at most 64 pairs: no plan, if at least four rows of X fit the LDS whole
    a.cols = kGateXLds / few_row_bytes(H) < 16 ? kGateXLds / few_row_bytes(H) : 16;
    if (a.P > 64 || a.cols < 4) a.cols = 0;
    a.cols_inv = a.cols ? (65535 + a.cols) / a.cols : 0;
    a.slots = experts + a.P / (a.cols ? a.cols : 16);
    a.down_slots = experts + a.P / tokens_per_block(a.planes);
    a.KW = waves_per_tile(int64_t(experts) * (F / 16));
    a.o = moe_by_pairs(experts, a.P, F, N, a.planes) ? o : nullptr;
    if (fmt_g == kFmtMXFP4) gate_up<kFmtMXFP4>(a, s);
    else if (fmt_g == kFmtINT4) gate_up<kFmtINT4>(a, s);
    else gate_up<kFmtNVFP4>(a, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
#define SVDQ_DOWN(FMT_)             \
  do {                              \
    if (f32) down<FMT_, 3>(a, s);   \
    else down<FMT_, 2>(a, s);       \
  } while (0)
    if (fmt_d == kFmtMXFP4) SVDQ_DOWN(kFmtMXFP4);
    else if (fmt_d == kFmtINT4) SVDQ_DOWN(kFmtINT4);
    else SVDQ_DOWN(kFmtNVFP4);
#undef SVDQ_DOWN
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace svdq
