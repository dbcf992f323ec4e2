// svdq_kv_attention: softmax(scale Q K^T) V over a paged 4-bit key-value cache (layout: kv.h).
//
// A wave holds 16 NQ query rows (a row is a query token and one of the heads that share a K/V head) as columns and
// walks the tokens in steps of 32, two tiles.  Per step
//     S^T = K Q^T     A operand: K's codes, made 16-bit in registers; B operand: Q, loaded once
//     P = exp2(S k - m)
//     O^T += V^T P^T  A operand: V's codes; B operand: P as it lies in the score registers
// so nothing passes through LDS or a shuffle but the rare new maximum.  m is the running maximum of a column, moved
// only when a score exceeds it by kGrow (powers of two that then stand in P, l and O alike cancel), l the running
// sum in fp32 of the probabilities before they are rounded.
//
// The 16-bit operands, exact but for P:
//   MXFP4  bf16: E2M1 times its power of two; P bf16
//   INT4   bf16: q + 8 out of E4M3 subnormals and smallest normals, n 2^-9 for a byte n < 16, scaled by 2^9.  K: -8
//          times the group's sum of Q starts the scores' sums; the fp16 scale multiplies a group's sum.  V:
//          the scale of (token, group) multiplies P, and -8 times the sum of those, formed by one more MFMA
//          against -8, is added at the end
//   NVFP4  fp16: E2M1 times E4M3 (2^-10 .. 2688); Q's rows scaled by a power of two; P fp16, times 2^11 so that
//          probabilities down to 2^-25 of the largest keep all bits
// P is rounded to half a unit in its last place (2^-8 of it in bf16, 2^-11 in fp16); with PLANES = 2 what bf16
// leaves is a second operand (2^-16).
#include "kv.h"
#include "w4frag.h"

namespace svdq {

namespace {

constexpr float kGrow = 4.0f;            // powers of two that a score may exceed the running maximum by
constexpr float kLowest = -3.0e38f;      // the running maximum before the first score

struct KvAttn {
  const uint16_t* Q;
  uint16_t* Y;
  float* lse;
  float* part;                     // partial results of split jobs
  int64_t ldq, ldy;
  int32_t group, q_heads;          // query heads for each K/V head, and in all
  int32_t window, causal, ranges;
  float scale2;                    // scale log2(e)
};

template <int FMT, int D>
struct KvStage {
  static constexpr int W = D / 32;                       // dwords of K or V a lane has of a tile
  uint32_t k[W], v[W];
  uint32_t ks[FMT == kFmtINT4 ? D / 32 : 1], vs[FMT == kFmtINT4 ? D / 32 : 1];
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&d)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    d[0] = v.x; d[1] = v.y;
  }
}

// One tile's data of a lane; `tile` is the same for the whole wave.
template <int FMT, int D>
__device__ __forceinline__ void load_tile(const uint8_t* tile, int r, int c, KvStage<FMT, D>& st) {
  constexpr int KS = 16 * D, VS = 16 * (D + kv_scales(FMT, D));
  if constexpr (FMT == kFmtINT4) {
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
      const uint2 v = *reinterpret_cast<const uint2*>(tile + r * (D / 2) + g * 32 + c * 8);
      st.k[2 * g] = v.x;
      st.k[2 * g + 1] = v.y;
      const uint2 s = *reinterpret_cast<const uint2*>(tile + KS + (g * 16 + 4 * c) * 2);
      st.ks[2 * g] = s.x;
      st.ks[2 * g + 1] = s.y;
      const uint2 z = *reinterpret_cast<const uint2*>(tile + VS + (g * 16 + 4 * c) * 2);
      st.vs[2 * g] = z.x;
      st.vs[2 * g + 1] = z.y;
    }
  } else {
    load_words(tile + r * (D / 2) + c * (D / 8), st.k);
    if constexpr (FMT == kFmtMXFP4) {
      st.ks[0] = tile[KS + r * (D / 32) + c * (D / 4) / 32];
      st.vs[0] = *reinterpret_cast<const uint32_t*>(tile + VS + r * (D / 16) / 32 * 16 + 4 * c);
    } else {
      if constexpr (D == 128)
        st.ks[0] = *reinterpret_cast<const uint16_t*>(tile + KS + r * 8 + 2 * c);
      else
        st.ks[0] = tile[KS + r * 4 + c];
      st.vs[0] = *reinterpret_cast<const uint32_t*>(tile + VS + r * (D / 16) / 16 * 16 + 4 * c);
    }
  }
  load_words(tile + 8 * D + (c * 16 + r) * (D / 8), st.v);
}

// Tokens of a tile outside [first, behind): their V scales are made 0 (what lies in the pool there may be
// anything, and a probability of 0 times an infinity or a NaN would not be 0).
template <int FMT, int D>
__device__ __forceinline__ void clear_outside(int first, int behind, int c, KvStage<FMT, D>& st) {
  uint32_t keep[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) keep[i] = 4 * c + i >= first && 4 * c + i < behind ? 0xFFFFFFFFu : 0u;
  if constexpr (FMT == kFmtINT4) {
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
      st.vs[2 * g] &= (keep[0] & 0xFFFFu) | (keep[1] & 0xFFFF0000u);
      st.vs[2 * g + 1] &= (keep[2] & 0xFFFFu) | (keep[3] & 0xFFFF0000u);
    }
  } else {
    st.vs[0] &= (keep[0] & 0xFFu) | (keep[1] & 0xFF00u) | (keep[2] & 0xFF0000u) | (keep[3] & 0xFF000000u);
  }
}

__device__ __forceinline__ uint32_t fp8_pair(uint32_t d, bool high) {       // bytes n < 16 -> bf16 n
  return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 512.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 512.0f, false));
}

template <int FMT>
__device__ __forceinline__ v4f mfma16(const uint4& a, const uint4& b, v4f c) {
  return FMT == kFmtNVFP4 ? mfma_f16(a, b, c) : mfma_bf16(a, b, c);
}

// A operand of K's MFMA j.
template <int FMT, int D>
__device__ __forceinline__ uint4 k_operand(const KvStage<FMT, D>& st, int j) {
  if constexpr (FMT == kFmtMXFP4) {
    return mx_to_bf16(st.k[j], scale_operand(st.ks[0]));
  } else if constexpr (FMT == kFmtNVFP4) {
    const _Float16 s = static_cast<_Float16>(e4m3_value(D == 128 ? (st.ks[0] >> ((j >> 1) * 8)) & 0xFFu : st.ks[0]));
    return nv_to_f16(st.k[j], v2h{s, s});
  } else {
    const uint32_t lo = st.k[j] & 0x0F0F0F0Fu, hi = (st.k[j] >> 4) & 0x0F0F0F0Fu;
    return make_uint4(fp8_pair(lo, false), fp8_pair(lo, true), fp8_pair(hi, false), fp8_pair(hi, true));
  }
}

// The 8 features of a query row that MFMA j takes from lane group c, in the order of k_operand.
template <int FMT, int D>
__device__ __forceinline__ uint4 q_operand(const uint16_t* row, int c, int j) {
  if constexpr (FMT == kFmtINT4) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + (j >> 1) * 64 + c * 16 + (j & 1) * 8);
    return make_uint4(__builtin_amdgcn_perm(v.y, v.x, 0x05040100u), __builtin_amdgcn_perm(v.w, v.z, 0x05040100u),
                      __builtin_amdgcn_perm(v.y, v.x, 0x07060302u), __builtin_amdgcn_perm(v.w, v.z, 0x07060302u));
  } else {
    return *reinterpret_cast<const uint4*>(row + c * (D / 4) + j * 8);
  }
}

// E2M1 byte b of token t's piece -> the pair of features (2 b, 2 b + 1) in 16 bits.
template <int FMT, int D, int T, int B>
__device__ __forceinline__ uint32_t v_pair(const KvStage<FMT, D>& st, const v2h (&nv)[2]) {
  constexpr int at = T * (D / 32) + B;
  if constexpr (FMT == kFmtMXFP4) {
    // the convert takes the exponent field of its scale operand alone, so the bits around the byte may stay
    const uint32_t s = T == 0 ? st.vs[0] << 23 : T == 1 ? st.vs[0] << 15 : T == 2 ? st.vs[0] << 7 : st.vs[0] >> 1;
    return __builtin_bit_cast(uint32_t,
                              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(st.v[at / 4], __uint_as_float(s), at % 4));
  } else {
    const _Float16 s = T & 1 ? nv[T / 2].y : nv[T / 2].x;
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(st.v[at / 4], 1.0f, at % 4) * v2h{s, s});
  }
}
constexpr uint32_t kLowHalves = 0x05040100u, kHighHalves = 0x07060302u;

// O^T += V^T P^T over a step for every feature tile; p[n][x] is the B operand of column tile n, plane x, and with
// INT4 of group g in p[n][g PL + x].
template <int FMT, int D, int NQ, int PL, int NP>
__device__ __forceinline__ void add_values(const KvStage<FMT, D> (&st)[2], const uint4 (&p)[NQ][NP],
                                           v4f (&o)[NQ][D / 16]) {
  if constexpr (FMT == kFmtINT4) {
    // token pairs: low and high nibbles of their pieces, then bytes of the two tokens side by side
    uint32_t w[2][2][D / 16][2];                            // tile, tokens 0 1 / 2 3, two features' bytes, nibble
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t lo[2], hi[2];
        if constexpr (D == 128) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            lo[i] = st[t].v[2 * h + i] & 0x0F0F0F0Fu;
            hi[i] = (st[t].v[2 * h + i] >> 4) & 0x0F0F0F0Fu;
          }
          w[t][h][0][0] = __builtin_amdgcn_perm(lo[1], lo[0], 0x05010400u);
          w[t][h][0][1] = __builtin_amdgcn_perm(hi[1], hi[0], 0x05010400u);
          w[t][h][1][0] = __builtin_amdgcn_perm(lo[1], lo[0], 0x07030602u);
          w[t][h][1][1] = __builtin_amdgcn_perm(hi[1], hi[0], 0x07030602u);
        } else {
          lo[0] = st[t].v[h] & 0x0F0F0F0Fu;
          hi[0] = (st[t].v[h] >> 4) & 0x0F0F0F0Fu;
          w[t][h][0][0] = __builtin_amdgcn_perm(lo[0], lo[0], 0x03010200u);
          w[t][h][0][1] = __builtin_amdgcn_perm(hi[0], hi[0], 0x03010200u);
        }
      }
#pragma unroll
    for (int g = 0; g < D / 64; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) {                         // feature 64 g + 4 r + e: byte e / 2, nibble e % 2
        const uint4 a = make_uint4(fp8_pair(w[0][0][g][e & 1], e >> 1), fp8_pair(w[0][1][g][e & 1], e >> 1),
                                   fp8_pair(w[1][0][g][e & 1], e >> 1), fp8_pair(w[1][1][g][e & 1], e >> 1));
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int x = 0; x < PL; ++x) o[n][4 * g + e] = mfma16<FMT>(a, p[n][g * PL + x], o[n][4 * g + e]);
      }
  } else {
    v2h nv[2][2];
    if constexpr (FMT == kFmtNVFP4) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        nv[t][0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(st[t].vs[0], 1.0f, false);
        nv[t][1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(st[t].vs[0], 1.0f, true);
      }
    }
    auto one = [&](auto byte) {
      constexpr int B = decltype(byte)::value;
      const uint32_t x[8] = {v_pair<FMT, D, 0, B>(st[0], nv[0]), v_pair<FMT, D, 1, B>(st[0], nv[0]),
                             v_pair<FMT, D, 2, B>(st[0], nv[0]), v_pair<FMT, D, 3, B>(st[0], nv[0]),
                             v_pair<FMT, D, 0, B>(st[1], nv[1]), v_pair<FMT, D, 1, B>(st[1], nv[1]),
                             v_pair<FMT, D, 2, B>(st[1], nv[1]), v_pair<FMT, D, 3, B>(st[1], nv[1])};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t sel = i ? kHighHalves : kLowHalves;
        const uint4 a = make_uint4(__builtin_amdgcn_perm(x[1], x[0], sel), __builtin_amdgcn_perm(x[3], x[2], sel),
                                   __builtin_amdgcn_perm(x[5], x[4], sel), __builtin_amdgcn_perm(x[7], x[6], sel));
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int y = 0; y < PL; ++y) o[n][2 * B + i] = mfma16<FMT>(a, p[n][y], o[n][2 * B + i]);
      }
    };
    one(std::integral_constant<int, 0>{});
    one(std::integral_constant<int, 1>{});
    if constexpr (D == 128) {
      one(std::integral_constant<int, 2>{});
      one(std::integral_constant<int, 3>{});
    }
  }
}

// First feature of the four (i = 0 .. 3 at stride `step`) that lane group c holds in o[..][dt].
template <int FMT, int D>
__device__ __forceinline__ constexpr int o_feature(int c, int dt, int i) {
  return FMT == kFmtINT4 ? (dt >> 2) * 64 + (4 * c + i) * 4 + (dt & 3) : (4 * c + i) * (D / 16) + dt;
}

// N features from d on of one query row: O / l in bf16 (0 where nothing is seen), and the logarithm of the row's sum.
template <int N>
__device__ __forceinline__ void kv_store(const KvAttn& a, int64_t token, int head, int D, int d, const float (&v)[N],
                                         float m, float l) {
  const float x = l == 0.f ? 0.f : 1.0f / l;
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w[i] = cvt_bf2(v[2 * i] * x, v[2 * i + 1] * x);
  uint16_t* y = a.Y + token * a.ldy + int64_t(head) * D + d;
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(y) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (N == 4)
    *reinterpret_cast<uint2*>(y) = make_uint2(w[0], w[1]);
  else
#pragma unroll
    for (int i = 0; i < N / 2; ++i) reinterpret_cast<uint32_t*>(y)[i] = w[i];
  if (a.lse != nullptr && d == 0)
    a.lse[token * a.q_heads + head] =
        l == 0.f ? -__builtin_huge_valf() : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
}

// A job is a tile of R query rows of one sequence on one K/V head; its tokens are cut into units of U.
template <int NQ, int WQ, int WK>
struct KvTiles {
  static constexpr int R = 16 * NQ * WQ, U = 32 * WK;
};

struct KvSeq {
  int len, row, rows, tiles, lo, units;       // lo: first token that any row sees, a multiple of 32
};
template <int R, int U, bool SPLIT>
__device__ __forceinline__ KvSeq kv_seq(const KvCache& kc, const KvAttn& a, int b) {
  KvSeq s;
  kc.sequence(b, s.len, s.row, s.rows);
  s.tiles = (int64_t(s.rows) * a.group + R - 1) / R;
  const int64_t first = a.window > 0 ? int64_t(s.len) - s.rows + 1 - a.window : 0;
  s.lo = int(first > 0 ? first : 0) & ~31;
  const int seen = max(min(s.len, kc.capacity()) - s.lo, 0);
  s.units = SPLIT ? max((seen + U - 1) / U, 1) : 1;
  return s;
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int x = 1; x < 64; x *= 2) {
    const int u = __shfl_up(v, x);
    if (lane >= x) v += u;
  }
  return v;
}

// Over the batch, by a workgroup of NT threads: the units of all jobs (SPLIT; else jobs).  With at >= 0 also the
// sequence that unit `at` falls into (-1: none) and the units before it; at may depend on the total.
struct KvFound {
  int b, before;
};
template <int R, int U, bool SPLIT, int NT>
__device__ __forceinline__ int kv_total(const KvCache& kc, const KvAttn& a, int* sh, int& mine) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int total = 0;
  for (int base = 0; base < kc.batch; base += NT) {
    const int b = base + threadIdx.x;
    int v = 0;
    if (b < kc.batch) {
      const KvSeq s = kv_seq<R, U, SPLIT>(kc, a, b);
      v = s.tiles * s.units;
    }
    v = wave_scan(v, lane);
    if (NT > 64) {
      if (base) __syncthreads();
      if (lane == 63) sh[wave] = v;
      __syncthreads();
      int before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < NT / 64; ++w) {
        before += w < wave ? sh[w] : 0;
        all += sh[w];
      }
      mine = total + before + v;
      total += all;
    } else {
      mine = total + v;
      total += __shfl(v, 63);
    }
  }
  return total;
}
// mine: this thread's inclusive sum of the last (for a batch of up to NT, the only) chunk.
template <int R, int U, bool SPLIT, int NT>
__device__ __forceinline__ KvFound kv_find(const KvCache& kc, const KvAttn& a, int at, int* sh, int mine) {
  if (threadIdx.x == 0) sh[8] = -1;
  __syncthreads();
  int total = 0;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int base = 0; base < kc.batch; base += NT) {
    const int b = base + threadIdx.x;
    int v = 0;
    if (b < kc.batch) {
      const KvSeq s = kv_seq<R, U, SPLIT>(kc, a, b);
      v = s.tiles * s.units;
    }
    int end = mine;
    if (kc.batch > NT) {
      const int scan = wave_scan(v, lane);
      __syncthreads();
      if (lane == 63) sh[wave] = scan;
      __syncthreads();
      int before = 0, all = 0;
      for (int w = 0; w < NT / 64; ++w) {
        before += w < wave ? sh[w] : 0;
        all += sh[w];
      }
      end = total + before + scan;
      total += all;
    }
    if (at >= end - v && at < end) {
      sh[8] = b;
      sh[9] = end - v;
    }
  }
  __syncthreads();
  return {__builtin_amdgcn_readfirstlane(sh[8]), __builtin_amdgcn_readfirstlane(sh[9])};
}

// Units that a range takes: the total over the ranges, and no fewer than `least`.
__device__ __forceinline__ int units_a_range(int total, int ranges, int least) {
  return max((total + ranges - 1) / ranges, least);
}
constexpr int kLeastUnits = 2;

template <int FMT, int D, int NQ, int WQ, int WK, int PLANES, bool SPLIT>
__global__ void __launch_bounds__(64 * WQ * WK) kv_attention_kernel(KvCache kc, KvAttn a) {
  using TL = KvTiles<NQ, WQ, WK>;
  constexpr int R = TL::R, U = TL::U, NT = 64 * WQ * WK, DT = D / 16, NG = FMT == kFmtINT4 ? D / 64 : 1;
  constexpr int PL = FMT == kFmtNVFP4 ? 1 : PLANES;            // fp16 needs no second plane
  constexpr int TB = kv_tile_bytes(FMT, D), OS = D + 4;        // floats of a row of O in LDS
  __shared__ int sh[16];
  __shared__ float merge_o[WK > 1 ? WK * 16 * OS : 4];
  __shared__ float merge_m[WK > 1 ? WK : 1][16], merge_l[WK > 1 ? WK : 1][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4, wq = wave / WK, wk = wave % WK;
  const int h = blockIdx.x % kc.heads, range = blockIdx.x / kc.heads;

  int mine = 0;
  const int total = kv_total<R, U, SPLIT, NT>(kc, a, sh, mine);
  const int per = SPLIT ? units_a_range(total, a.ranges, kLeastUnits) : 1;
  const int64_t first = int64_t(range) * per;
  if (first >= total) return;
  const KvFound f = kv_find<R, U, SPLIT, NT>(kc, a, int(first), sh, mine);
  int left = min(per, total - int(first)), b = f.b;
  if (b < 0) return;
  KvSeq s = kv_seq<R, U, SPLIT>(kc, a, b);
  int job = (int(first) - f.before) / s.units, unit = (int(first) - f.before) % s.units;

  while (left > 0) {
    while (job >= s.tiles) {                                  // the next sequence with rows
      if (++b >= kc.batch) return;
      s = kv_seq<R, U, SPLIT>(kc, a, b);
      job = 0;
      unit = 0;
    }
    const int n_units = min(left, s.units - unit);
    const int tile_rows = SPLIT ? job : s.tiles - 1 - job;    // long causal tiles first
    const int64_t row0 = int64_t(tile_rows) * R + wq * 16 * NQ;
    const int64_t rows = int64_t(s.rows) * a.group;
    const int capacity = kc.capacity();

    // Query rows, and the tokens [lo, hi) that each sees.
    uint4 q[NQ][D / 32];
    float k2[NQ];
    int lo[NQ], hi[NQ];
    v4f s0[FMT == kFmtINT4 ? NQ : 1][FMT == kFmtINT4 ? NG : 1];
    int first_all = INT32_MAX, last_all = 0, first_max = 0, last_min = INT32_MAX;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int64_t i = row0 + n * 16 + r;
      const bool there = i < rows;
      const int token = there ? int(i / a.group) : 0, head = there ? int(i % a.group) : 0;
      const uint16_t* row = a.Q + int64_t(s.row + token) * a.ldq + int64_t(h * a.group + head) * D;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) q[n][j] = there ? q_operand<FMT, D>(row, c, j) : make_uint4(0, 0, 0, 0);
      const int at = s.len - s.rows + token;                  // the query's place
      hi[n] = !there ? 0 : a.causal ? min(max(at + 1, 0), min(s.len, capacity)) : min(s.len, capacity);
      lo[n] = a.window > 0 ? max(at - a.window + 1, 0) : 0;
      if (!there) lo[n] = 0;
      first_all = min(first_all, hi[n] > 0 ? lo[n] : INT32_MAX);
      last_all = max(last_all, hi[n]);
      first_max = max(first_max, lo[n]);
      last_min = min(last_min, there ? hi[n] : INT32_MAX);
      k2[n] = a.scale2;
      if constexpr (FMT == kFmtNVFP4) {
        float v[D / 32][8], top = 0.f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          unpack_bf8(q[n][j], v[j]);
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[j][e]));
        }
        const int e2 = f16_row_power(rowgroup_max(top));
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] = ldexpf(v[j][e], e2);
          q[n][j] = to_f16(v[j]);
        }
        k2[n] = ldexpf(k2[n], -e2);
      }
      if constexpr (FMT == kFmtINT4) {
        const uint4 m8 = make_uint4(0xC100C100u, 0xC100C100u, 0xC100C100u, 0xC100C100u);      // bf16 -8
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          v4f z = {0.f, 0.f, 0.f, 0.f};
          z = mfma_bf16(m8, q[n][2 * g], z);
          s0[n][g] = mfma_bf16(m8, q[n][2 * g + 1], z);
        }
      }
    }
    // Over the 16 rows of a column tile (lanes c hold the same).
#pragma unroll
    for (int x = 1; x < 16; x *= 2) {
      first_all = min(first_all, __shfl_xor(first_all, x));
      last_all = max(last_all, __shfl_xor(last_all, x));
      first_max = max(first_max, __shfl_xor(first_max, x));
      last_min = min(last_min, __shfl_xor(last_min, x));
    }
    first_all = __builtin_amdgcn_readfirstlane(first_all);
    last_all = __builtin_amdgcn_readfirstlane(last_all);
    first_max = __builtin_amdgcn_readfirstlane(first_max);
    last_min = __builtin_amdgcn_readfirstlane(last_min);

    v4f o[NQ][DT], off[FMT == kFmtINT4 ? NQ : 1][NG];
    float m[NQ], l[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      m[n] = kLowest;
      l[n] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[n][d] = v4f{0.f, 0.f, 0.f, 0.f};
      if constexpr (FMT == kFmtINT4)
#pragma unroll
        for (int g = 0; g < NG; ++g) off[n][g] = v4f{0.f, 0.f, 0.f, 0.f};
    }

    // This wave's steps: 32 tokens from s.lo + 32 (unit WK + wk) on, every WK-th; those before every row's window
    // are left out.
    constexpr int STRIDE = 32 * WK;
    int t0 = s.lo + unit * U + 32 * wk;
    const int end = min(SPLIT ? s.lo + (unit + n_units) * U : INT32_MAX, last_all);
    if (first_all > t0 && end > t0) t0 += (min(first_all, end) - t0) / STRIDE * STRIDE;
    const int steps = end > t0 ? (end - t0 + STRIDE - 1) / STRIDE : 0;
    const uint8_t* base = kc.pool + (int64_t(TB) << kc.page_shift) * h;
    const int mask = (1 << kc.page_shift) - 1;

    // Pages of 32 steps, one a lane (a step's two tiles in lanes 2 i, 2 i + 1), loaded 32 steps ahead.
    auto pages_from = [&](int i) {
      const int64_t tile = (int64_t(t0) + int64_t(i + (lane >> 1)) * STRIDE) / 16 + (lane & 1);
      return tile * 16 < end ? kc.page_of(b, int(tile)) : -1;
    };
    int pages = -1, next_pages = steps > 0 ? pages_from(0) : -1;
    auto fetch = [&](int i, KvStage<FMT, D> (&st)[2], int (&ok)[2]) {
      if ((i & 31) == 0) {
        pages = next_pages;
        next_pages = pages_from(i + 32);
      }
      const int tile = (t0 >> 4) + i * (STRIDE / 16);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int p = __builtin_amdgcn_readlane(pages, (i & 31) * 2 + x);
        ok[x] = p >= 0;
        load_tile<FMT, D>(base + int64_t(p >= 0 ? p : 0) * kc.page_bytes + int64_t((tile + x) & mask) * TB, r, c, st[x]);
      }
    };

    auto step = [&](int t, KvStage<FMT, D> (&st)[2], const int (&ok)[2]) {
      // Scores: lane (query r, tokens t + 16 i + 4 c + e).
      float z[NQ][2][4];
      const bool whole = t + 32 <= last_min && t >= first_max && ok[0] && ok[1];
      if (t + 32 > last_all || t < first_all || !ok[0] || !ok[1]) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          clear_outside<FMT, D>(first_all - t - 16 * i, ok[i] ? last_all - t - 16 * i : 0, c, st[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (FMT == kFmtINT4) {
          uint4 ka[D / 32];
#pragma unroll
          for (int j = 0; j < D / 32; ++j) ka[j] = k_operand<FMT, D>(st[i], j);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) z[n][i][e] = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              v4f x = mfma_bf16(ka[2 * g], q[n][2 * g], s0[n][g]);
              x = mfma_bf16(ka[2 * g + 1], q[n][2 * g + 1], x);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                z[n][i][e] = fmaf(x[e], f16_value(st[i].ks[2 * g + (e >> 1)] >> (16 * (e & 1))), z[n][i][e]);
            }
          }
        } else {
          v4f x[NQ];
#pragma unroll
          for (int n = 0; n < NQ; ++n) x[n] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint4 ka = k_operand<FMT, D>(st[i], j);
#pragma unroll
            for (int n = 0; n < NQ; ++n) x[n] = mfma16<FMT>(ka, q[n][j], x[n]);
          }
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[n][i][e] = x[n][e];
        }
      }
      if (!whole) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = t + 16 * i + 4 * c + e;
              if (!(ok[i] && at < hi[n] && at >= lo[n])) z[n][i][e] = -__builtin_huge_valf();
            }
      }
      // New maxima.
      bool grow = false;
      float top[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        top[n] = fmaxf(fmaxf(fmaxf(z[n][0][0], z[n][0][1]), fmaxf(z[n][0][2], z[n][0][3])),
                       fmaxf(fmaxf(z[n][1][0], z[n][1][1]), fmaxf(z[n][1][2], z[n][1][3]))) * k2[n];
        grow |= top[n] > m[n] + kGrow;
      }
      if (__any(grow)) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const float now = fmaxf(m[n], rowgroup_max(top[n]));
          const float x = __builtin_amdgcn_exp2f(m[n] - now);
          m[n] = now;
          l[n] *= x;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[n][d] *= x;
          if constexpr (FMT == kFmtINT4)
#pragma unroll
            for (int g = 0; g < NG; ++g) off[n][g] *= x;
        }
      }
      // Probabilities, and their operands.
      uint4 p[NQ][NG * PL];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float e[8];
        const float base2 = FMT == kFmtNVFP4 ? m[n] - 11.0f : m[n];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[i] = __builtin_amdgcn_exp2f(fmaf(z[n][i >> 2][i & 3], k2[n], -base2));
          l[n] += e[i];
        }
        if constexpr (FMT == kFmtNVFP4) {
          p[n][0] = to_f16(e);
        } else if constexpr (FMT == kFmtINT4) {
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = e[i] * f16_value(st[i >> 2].vs[2 * g + ((i & 3) >> 1)] >> (16 * (i & 1)));
            uint4 planes[PL];
            split_planes<PL>(x, planes);
#pragma unroll
            for (int y = 0; y < PL; ++y) p[n][g * PL + y] = planes[y];
          }
        } else {
          uint4 planes[PL];
          split_planes<PL>(e, planes);
#pragma unroll
          for (int y = 0; y < PL; ++y) p[n][y] = planes[y];
        }
      }
      add_values<FMT, D, NQ, PL>(st, p, o);
      if constexpr (FMT == kFmtINT4) {
        const uint4 m8 = make_uint4(0xC100C100u, 0xC100C100u, 0xC100C100u, 0xC100C100u);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int y = 0; y < PL; ++y) off[n][g] = mfma_bf16(m8, p[n][g * PL + y], off[n][g]);
      }
    };

    if (steps > 0) {
      KvStage<FMT, D> st[2][2];
      int ok[2][2];
      fetch(0, st[0], ok[0]);
      for (int i = 0; i < steps; i += 2) {
        if (i + 1 < steps) fetch(i + 1, st[1], ok[1]);
        step(t0 + i * STRIDE, st[0], ok[0]);
        if (i + 1 >= steps) break;
        if (i + 2 < steps) fetch(i + 2, st[0], ok[0]);
        step(t0 + (i + 1) * STRIDE, st[1], ok[1]);
      }
    }

    // Results of the segment: a whole job's rows are written, a part's go to the workspace.
    const bool all = !SPLIT || (unit == 0 && n_units == s.units);
    float* part = SPLIT ? a.part + ((int64_t(range) * kc.heads + h) * 2 + (unit > 0 ? 0 : 1)) * (R * (D + 2)) : nullptr;
    auto emit = [&](int in_tile, int d, auto& v, float mm, float ll) {        // features d .. of row in_tile
      constexpr int N = sizeof(v) / sizeof(float);
      const int64_t i = int64_t(tile_rows) * R + in_tile;
      if (i >= rows) return;
      if (!all) {
        if (d == 0) {
          part[in_tile] = mm;
          part[R + in_tile] = ll;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) part[2 * R + in_tile * D + d + e] = v[e];
        return;
      }
      const int token = s.row + int(i / a.group), head = h * a.group + int(i % a.group);
      kv_store<N>(a, token, head, D, d, v, mm, ll);
    };
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      l[n] = rowgroup_sum(l[n]);
      if constexpr (FMT == kFmtINT4)
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] += off[n][d >> 2];
      const float mm = FMT == kFmtNVFP4 ? m[n] - 11.0f : m[n];
      if constexpr (WK == 1) {
#pragma unroll
        for (int d = 0; d < DT; d += 4)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float v[4] = {o[n][d][i], o[n][d + 1][i], o[n][d + 2][i], o[n][d + 3][i]};
            emit(wq * 16 * NQ + n * 16 + r, o_feature<FMT, D>(c, d, i), v, mm, l[n]);
          }
      } else {
        __syncthreads();                                      // the rows before are read
        float* mine_o = merge_o + (wk * 16 + r) * OS;
#pragma unroll
        for (int d = 0; d < DT; d += 4)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(mine_o + o_feature<FMT, D>(c, d, i)) =
                make_float4(o[n][d][i], o[n][d + 1][i], o[n][d + 2][i], o[n][d + 3][i]);
        if (c == 0) {
          merge_m[wk][r] = mm;
          merge_l[wk][r] = l[n];
        }
        __syncthreads();
        constexpr int TPR = NT / 16, FPT = D / TPR;           // threads a row, features a thread
        const int row = threadIdx.x / TPR, d = threadIdx.x % TPR * FPT;
        float mx = merge_m[0][row], ll = 0.f, v[FPT] = {};
#pragma unroll
        for (int w = 1; w < WK; ++w) mx = fmaxf(mx, merge_m[w][row]);
#pragma unroll
        for (int w = 0; w < WK; ++w) {
          const float x = __builtin_amdgcn_exp2f(merge_m[w][row] - mx);
          ll += merge_l[w][row] * x;
#pragma unroll
          for (int e = 0; e < FPT; ++e) v[e] += merge_o[(w * 16 + row) * OS + d + e] * x;
        }
        emit(n * 16 + row, d, v, mx, ll);
      }
    }
    left -= n_units;
    unit += n_units;
    if (unit == s.units) {
      unit = 0;
      ++job;
    }
  }
}

// Joins the parts of split jobs: a workgroup takes the first range border inside a job (and only that), 4 of its
// rows; wave w adds parts w, w + 4, ...
template <int D, int R, int U>
__global__ void __launch_bounds__(256) kv_join_kernel(KvCache kc, KvAttn a) {
  constexpr int F = D / 16;
  __shared__ int sh[16];
  __shared__ float sm[4][4], sl[4][4], so[4][4][D];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int h = blockIdx.x % kc.heads, border = blockIdx.x / kc.heads + 1;
  int mine = 0;
  const int total = kv_total<R, U, true, 256>(kc, a, sh, mine);
  const int per = units_a_range(total, a.ranges, kLeastUnits);
  const int64_t at = int64_t(border) * per;
  if (at >= total) return;
  const KvFound f = kv_find<R, U, true, 256>(kc, a, int(at), sh, mine);
  if (f.b < 0) return;
  const KvSeq s = kv_seq<R, U, true>(kc, a, f.b);
  const int job = (int(at) - f.before) / s.units, start = f.before + job * s.units;
  if (start == at || start < at - per) return;
  const int last = (start + s.units - 1) / per;              // ranges border - 1 .. last hold parts
  const int row = blockIdx.y * 4 + (lane >> 4), d = (lane & 15) * F;
  const int64_t i = int64_t(job) * R + row;
  const bool there = i < int64_t(s.rows) * a.group;
  float m = kLowest, l = 0.f, v[F] = {};
  if (there)
    for (int g = border - 1 + wave; g <= last; g += 4) {
      const float* part = a.part + ((int64_t(g) * kc.heads + h) * 2 + (g == border - 1 ? 1 : 0)) * (R * (D + 2));
      const float pm = part[row], pl = part[R + row], now = fmaxf(m, pm);
      const float x = __builtin_amdgcn_exp2f(m - now), y = __builtin_amdgcn_exp2f(pm - now);
      const float* o = part + 2 * R + row * D + d;
#pragma unroll
      for (int e = 0; e < F; ++e) v[e] = v[e] * x + o[e] * y;
      l = l * x + pl * y;
      m = now;
    }
  sm[wave][lane >> 4] = m;
  sl[wave][lane >> 4] = l;
#pragma unroll
  for (int e = 0; e < F; ++e) so[wave][lane >> 4][d + e] = v[e];
  __syncthreads();
  if (wave != 0 || !there) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    const float pm = sm[w][lane >> 4], now = fmaxf(m, pm);
    const float x = __builtin_amdgcn_exp2f(m - now), y = __builtin_amdgcn_exp2f(pm - now);
#pragma unroll
    for (int e = 0; e < F; ++e) v[e] = v[e] * x + so[w][lane >> 4][d + e] * y;
    l = l * x + sl[w][lane >> 4] * y;
    m = now;
  }
  kv_store<F>(a, s.row + i / a.group, h * a.group + int(i % a.group), D, d, v, m, l);
}

template <int FMT, int D, int NQ, int WQ, int WK, int PL>
void attend(const KvCache& kc, const KvAttn& a, bool split, int jobs, hipStream_t s) {
  constexpr int NT = 64 * WQ * WK, R = KvTiles<NQ, WQ, WK>::R, U = KvTiles<NQ, WQ, WK>::U;
  if (!split) {
    kv_attention_kernel<FMT, D, NQ, WQ, WK, PL, false><<<dim3(unsigned(jobs) * kc.heads), NT, 0, s>>>(kc, a);
    return;
  }
  kv_attention_kernel<FMT, D, NQ, WQ, WK, PL, true><<<dim3(a.ranges * kc.heads), NT, 0, s>>>(kc, a);
  if (a.ranges > 1) kv_join_kernel<D, R, U><<<dim3((a.ranges - 1) * kc.heads, R / 4), 256, 0, s>>>(kc, a);
}

template <int FMT, int D>
void attend_plan(const KvPlan& p, const KvCache& kc, const KvAttn& a, hipStream_t s) {
  if (p.rows == 16)
    attend<FMT, D, 1, 1, 4, 2>(kc, a, p.split, p.jobs, s);
  else if (p.rows == 32)
    attend<FMT, D, 2, 1, 4, 2>(kc, a, p.split, p.jobs, s);
  else
    attend<FMT, D, 2, 4, 1, 1>(kc, a, p.split, p.jobs, s);
}

}  // namespace

hipError_t launch_kv_attention(int fmt, int D, const KvCache& kc, const uint16_t* Q, int64_t ldq, int q_heads,
                               float scale, int window, bool causal, uint16_t* Y, int64_t ldy, float* lse, float* part,
                               hipStream_t s) {
  const KvPlan p = kv_plan(D, kc.batch, kc.M, q_heads, kc.heads);
  const KvAttn a = {Q, Y, lse, part, ldq, ldy, q_heads / kc.heads, q_heads, window, causal ? 1 : 0, p.ranges,
                    scale * 1.44269504088896341f};
  if (fmt == kFmtMXFP4)
    D == 64 ? attend_plan<kFmtMXFP4, 64>(p, kc, a, s) : attend_plan<kFmtMXFP4, 128>(p, kc, a, s);
  else if (fmt == kFmtINT4)
    D == 64 ? attend_plan<kFmtINT4, 64>(p, kc, a, s) : attend_plan<kFmtINT4, 128>(p, kc, a, s);
  else
    D == 64 ? attend_plan<kFmtNVFP4, 64>(p, kc, a, s) : attend_plan<kFmtNVFP4, 128>(p, kc, a, s);
  return hipGetLastError();
}

}  // namespace svdq
