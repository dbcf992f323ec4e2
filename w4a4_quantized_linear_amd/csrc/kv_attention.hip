// svdq_kv_attention: softmax(scale Q K^T) V over a paged 4-bit key-value cache (layout: kv.h).
//
// A wave holds 16 NQ query rows (a row is a query token and one of the heads that share a K/V head) as columns and
// walks the tokens in steps of 32, two tiles.  Per step
//     S^T = K Q^T     A operand: K's codes, made 16-bit in registers; B operand: Q, loaded once
//     P = exp2(S k - m)
//     O^T += V^T P^T  A operand: V's codes; B operand: P as it lies in the score registers
// so nothing passes through LDS or a shuffle but the rare new maximum.  m is the running maximum of a column, moved
// only when a score of its own exceeds it by kGrow (powers of two that then stand in P, l and O alike cancel), l the
// running sum in fp32 of the probabilities before they are rounded.
//
// The 16-bit operands, exact but for P:
//   MXFP4  bf16: E2M1 times its power of two; P bf16
//   INT4   bf16: q + 8 out of E4M3 subnormals and smallest normals, n 2^-9 for a byte n < 16, scaled by 2^9.  K: -8
//          times the group's sum of Q starts the scores' sums; the fp16 scale multiplies a group's sum.  V:
//          the scale of (token, group) multiplies P, and -8 times the sum of those, formed by one more MFMA
//          against -8, is added at the end
//   NVFP4  fp16: E2M1 times E4M3 (2^-10 .. 2688); Q's rows scaled by a power of two; P fp16, times 2^11 so that
//          probabilities down to 2^-25 of the largest keep all bits
// P is rounded to half a unit in its last place (2^-8 of it in bf16, 2^-11 in fp16); what bf16 leaves is a second
// operand (2^-16), but in kv_prompt_kernel, where that would be half again the matrix work.
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
  uint32_t ks[1], vs[FMT == kFmtINT4 ? 2 : 1];           // scales (INT4: all in vs, see kv_scales4)
};

template <int N>
__device__ __forceinline__ void load_words(__amdgpu_buffer_rsrc_t t, uint32_t off, uint32_t more, uint32_t (&d)[N]) {
  if constexpr (N == 4) {
    const uint4 v = buffer_load16(t, off, more);
    d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
  } else {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(t, off, more, 0);
    d[0] = uint32_t(v[0]); d[1] = uint32_t(v[1]);
  }
}

// A lane's offsets in a tile.
template <int FMT, int D>
struct KvLane {
  uint32_t k, ks, v, vs;
  __device__ __forceinline__ KvLane(uint32_t r, uint32_t c) {
    constexpr int G = kv_group(FMT);
    v = (c * 16 + r) * (D / 8);
    k = r * (D / 2) + c * (D / 8);
    ks = r * (D / G) + c * (D / 4) / G;
    vs = FMT == kFmtINT4 ? r % (D / 32) * 32 + c * 8 : r * (D / 16) / G * 16 + 4 * c;
  }
};

// One tile's data of a lane.  The tile is the whole wave's, as a buffer of its bytes (of none where its page is not
// there: zeros), so a load is scalar registers, one of four lane offsets and a constant.
template <int FMT, int D>
__device__ __forceinline__ void load_tile(__amdgpu_buffer_rsrc_t t, const KvLane<FMT, D>& at, KvStage<FMT, D>& st) {
  constexpr uint32_t KS = 16 * D, VS = 16 * (D + kv_scales(FMT, D));
  load_words(t, at.k, 0, st.k);
  if constexpr (FMT == kFmtINT4) {
    load_words(t, at.vs, KS, st.vs);
  } else {
    if constexpr (FMT == kFmtNVFP4 && D == 128)
      st.ks[0] = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(t, at.ks, KS, 0));
    else
      st.ks[0] = uint8_t(__builtin_amdgcn_raw_buffer_load_b8(t, at.ks, KS, 0));
    st.vs[0] = uint32_t(__builtin_amdgcn_raw_buffer_load_b32(t, at.vs, VS, 0));
  }
  load_words(t, at.v, 8 * D, st.v);
}

// INT4: the scales of tokens 4 c .. 4 c + 3, kind K of group 0, of group 1, V of group 0, of group 1 (a head of 64
// features: K, V), lie in lanes r % 4 (% 2) of the quads; every lane gets a word of piece `kind`.
template <int D>
__device__ __forceinline__ uint32_t kv_scales4(uint32_t x, int kind) {
  constexpr int Q0 = 0x00, Q1 = 0x55, Q2 = 0xAA, Q3 = 0xFF;            // quad_perm: lane 0, 1, 2, 3 of the quad
  switch (kind) {
    case 0: return uint32_t(__builtin_amdgcn_mov_dpp(int(x), Q0, 0xF, 0xF, true));
    case 1: return uint32_t(__builtin_amdgcn_mov_dpp(int(x), Q1, 0xF, 0xF, true));
    case 2: return uint32_t(__builtin_amdgcn_mov_dpp(int(x), Q2, 0xF, 0xF, true));
    default: return uint32_t(__builtin_amdgcn_mov_dpp(int(x), Q3, 0xF, 0xF, true));
  }
}

__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Tokens of a tile outside [first, behind): their V scales are made 0 (what lies in the pool there may be
// anything, and a probability of 0 times an infinity or a NaN would not be 0).
template <int FMT, int D>
__device__ __forceinline__ void clear_outside(int first, int behind, int c, KvStage<FMT, D>& st) {
  uint32_t keep[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) keep[i] = 4 * c + i >= first && 4 * c + i < behind ? 0xFFFFFFFFu : 0u;
  if constexpr (FMT == kFmtINT4) {
    st.vs[0] &= (keep[0] & 0xFFFFu) | (keep[1] & 0xFFFF0000u);
    st.vs[1] &= (keep[2] & 0xFFFFu) | (keep[3] & 0xFFFF0000u);
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

// INT4 heads of 128 features: a lane loads 32 features that lie together, all of one group, but a group's MFMAs
// need every lane.  Lanes c and c + 2 trade halves: afterwards words 0, 1 are of group 0 and 2, 3 of group 1.
template <int FMT, int D>
__device__ __forceinline__ void trade_groups(KvStage<FMT, D>& st) {
  if constexpr (FMT == kFmtINT4 && D == 128) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const auto x = __builtin_amdgcn_permlane32_swap(st.k[i], st.k[2 + i], false, false);
      st.k[i] = x[0];
      st.k[2 + i] = x[1];
    }
  }
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
    const int piece = D == 64 ? c : (c & 1) * 2 + (c >> 1);                // of the group's four
    const uint4 v = *reinterpret_cast<const uint4*>(row + (j >> 1) * 64 + piece * 16 + (j & 1) * 8);
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

// INT4: bytes of group g's features of tokens 2 t and 2 t + 1, one beside the other.
template <int D>
__device__ __forceinline__ uint32_t value_pair(const KvStage<kFmtINT4, D>& st, int t, int g) {
  if constexpr (D == 128)
    return __builtin_amdgcn_perm(st.v[2 * t + 1], st.v[2 * t], g ? 0x07030602u : 0x05010400u);
  else
    return __builtin_amdgcn_perm(st.v[t], st.v[t], 0x03010200u);
}

// O^T += V^T P^T over a step for every feature tile, e the probabilities of a lane's 8 tokens.  INT4: a group's scales
// multiply its probabilities, so they are rounded once, and off is -8 times their sums.
template <int FMT, int D, int NQ, int PL>
__device__ __forceinline__ void add_values(const KvStage<FMT, D> (&st)[2], const float (&e)[NQ][8], v4f (&o)[NQ][D / 16],
                                           v4f (&off)[NQ][D / 64]) {
  if constexpr (FMT == kFmtINT4) {
    const uint4 m8 = make_uint4(0xC100C100u, 0xC100C100u, 0xC100C100u, 0xC100C100u);          // bf16 -8
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
      uint4 p[NQ][PL];
      uint32_t sv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sv[i] = kv_scales4<D>(st[i >> 1].vs[i & 1], D / 64 + g);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = e[n][i] * f16_value(sv[i >> 1] >> (16 * (i & 1)));
        split_planes<PL>(x, p[n]);
#pragma unroll
        for (int y = 0; y < PL; ++y) off[n][g] = mfma_bf16(m8, p[n][y], off[n][g]);
      }
      uint32_t w[4][2];                                     // token pairs: two features' bytes of both, by nibble
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t x = value_pair<D>(st[t >> 1], t & 1, g);
        w[t][0] = x & 0x0F0F0F0Fu;
        w[t][1] = (x >> 4) & 0x0F0F0F0Fu;
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) {                         // feature 64 g + 4 r + f: byte f / 2, nibble f % 2
        const uint4 a = make_uint4(fp8_pair(w[0][f & 1], f >> 1), fp8_pair(w[1][f & 1], f >> 1),
                                   fp8_pair(w[2][f & 1], f >> 1), fp8_pair(w[3][f & 1], f >> 1));
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int y = 0; y < PL; ++y) o[n][4 * g + f] = mfma_bf16(a, p[n][y], o[n][4 * g + f]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
    uint4 p[NQ][PL];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      if constexpr (FMT == kFmtNVFP4) {
        p[n][0] = to_f16(e[n]);
      } else {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = e[n][i];
        split_planes<PL>(x, p[n]);
      }
    }
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
      __builtin_amdgcn_sched_barrier(0);
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
template <int NQ, int WK>
struct KvTiles {
  static constexpr int R = 16 * NQ, U = 32 * WK;
};

struct KvSeq {
  int len, row, rows, tiles, lo, units;       // lo: first token that any row sees, a multiple of 32
};
template <int R, int U, bool SPLIT>
__device__ __forceinline__ KvSeq kv_seq(const KvCache& kc, const KvAttn& a, int len, int row, int rows) {
  KvSeq s;
  s.len = len;
  s.row = row;
  s.rows = rows;
  s.tiles = (rows * a.group + R - 1) / R;
  const int first = a.window > 0 ? len - rows + 1 - a.window : 0;
  s.lo = (first > 0 ? first : 0) & ~31;
  const int seen = max(min(len, kc.capacity()) - s.lo, 0);
  s.units = SPLIT ? max((seen + U - 1) / U, 1) : 1;
  return s;
}
// The same of sequence b, which all lanes ask for: scalar loads.
template <int R, int U, bool SPLIT>
__device__ __forceinline__ KvSeq kv_seq_of(const KvCache& kc, const KvAttn& a, int b) {
  typedef const __attribute__((address_space(4))) int32_t* Words;
  const Words lens = (Words)(uintptr_t)kc.lens, cu = (Words)(uintptr_t)kc.cu;
  b = uni(b);
  const int len = max(lens[b], 0);
  if (kc.cu == nullptr) return kv_seq<R, U, SPLIT>(kc, a, len, b, 1);
  const int row = min(max(cu[b], 0), kc.M);
  return kv_seq<R, U, SPLIT>(kc, a, len, row, max(min(cu[b + 1], kc.M) - row, 0));
}

// The query rows of a sequence on one K/V head, and the tokens [first, behind) that they see.
struct KvSpan {
  int first, behind, first_most, behind_least;                // outermost and innermost of a run of rows
};
struct KvRows {
  int rows, place0, there, window, causal, group;             // place0: the first row's place in its sequence
  __device__ __forceinline__ KvRows(const KvCache& kc, const KvAttn& a, const KvSeq& s)
      : rows(s.rows * a.group), place0(s.len - s.rows), there(min(s.len, kc.capacity())), window(a.window),
        causal(a.causal), group(a.group) {}
  __device__ __forceinline__ int first(int token) const { return window > 0 ? max(place0 + token - window + 1, 0) : 0; }
  __device__ __forceinline__ int behind(int token) const {
    return causal ? min(max(place0 + token + 1, 0), there) : there;
  }
  __device__ __forceinline__ KvSpan span(int row, int n) const {
    if (row >= rows) return {0, 0, 0, 0};
    const int a = row / group, z = (min(row + n, rows) - 1) / group;
    return {first(a), behind(z), first(z), behind(a)};
  }
};

// A wave's 16 NQ query rows from row0 on, as they lie, and what each sees; rows that are not there are zeros that see nothing.
template <int FMT, int D, int NQ>
__device__ __forceinline__ void load_queries(const KvAttn& a, const KvSeq& s, const KvRows& rows, int row0, int h, int r,
                                             int c, uint4 (&q)[NQ][D / 32], int (&lo)[NQ], int (&hi)[NQ]) {
  asm volatile("" : "+v"(r), "+v"(c));                        // opaque: its addresses are not kept in registers
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int i = row0 + n * 16 + r;
    const bool there = i < rows.rows;
    const int token = there ? int(unsigned(i) / unsigned(a.group)) : 0, head = there ? i - token * a.group : 0;
    const uint16_t* row = a.Q + int64_t(s.row + token) * a.ldq + (h * a.group + head) * D;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) q[n][j] = there ? q_operand<FMT, D>(row, c, j) : make_uint4(0, 0, 0, 0);
    hi[n] = there ? rows.behind(token) : 0;
    lo[n] = there ? rows.first(token) : 0;
  }
}

// The rows as operands (NVFP4: fp16, scaled by a power of two), the factor of their scores, and what INT4's sums start at.
template <int FMT, int D, int NQ, int NG>
__device__ __forceinline__ void finish_queries(const KvAttn& a, uint4 (&q)[NQ][D / 32], float (&k2)[NQ],
                                               v4f (&s0)[NQ][NG]) {
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    k2[n] = a.scale2;
    if constexpr (FMT == kFmtNVFP4) {
      u16x2 top = {0, 0};                                     // the largest magnitude's bits
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (uint32_t x : {q[n][j].x, q[n][j].y, q[n][j].z, q[n][j].w})
          top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, x & 0x7FFF7FFFu));
      const int e2 = f16_row_power(rowgroup_max(__uint_as_float(uint32_t(top.x > top.y ? top.x : top.y) << 16)));
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        float v[8];
        unpack_bf8(q[n][j], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = ldexpf(v[e], e2);
        q[n][j] = to_f16(v);
        __builtin_amdgcn_sched_barrier(0);
      }
      k2[n] = ldexpf(k2[n], -e2);
    }
    if constexpr (FMT == kFmtINT4) {
      const uint4 m8 = make_uint4(0xC100C100u, 0xC100C100u, 0xC100C100u, 0xC100C100u);        // bf16 -8
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        v4f z = {0.f, 0.f, 0.f, 0.f};
        z = mfma_bf16(m8, q[n][2 * g], z);
        s0[n][g] = mfma_bf16(m8, q[n][2 * g + 1], z);
      }
    }
  }
}

// Scores z[n][tile][token] of tokens t + 16 tile + 4 c + token, T tiles; those that a row does not see become -infinity.
template <int NQ, int T>
__device__ __forceinline__ void mask_scores(float (&z)[NQ][T][4], int t, int c, const bool (&ok)[T], const int (&lo)[NQ],
                                            const int (&hi)[NQ]) {
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = t + 16 * i + 4 * c + e;
        if (!(ok[i] && at < hi[n] && at >= lo[n])) z[n][i][e] = -__builtin_huge_valf();
      }
}

template <int N>
__device__ __forceinline__ float largest(const float (&x)[N]) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
  return top;
}

// Probabilities e of the scores z, relative to the running maxima, which move where a score exceeds one by kGrow; l, O
// and off with them.  A column's maximum moves by its own scores alone, so no row's bits hang on what stands beside it
// (a row of infinities, say).  The scores are brought to the exponent first and their largest sought there: what a matrix
// instruction gives would cost one more operation each on its way into a maximum.
template <int FMT, int D, int NQ, int T>
__device__ __forceinline__ void probabilities(const float (&z)[NQ][T][4], const float (&k2)[NQ], float (&m)[NQ],
                                              float (&l)[NQ], v4f (&o)[NQ][D / 16], v4f (&off)[NQ][D / 64],
                                              float (&e)[NQ][4 * T]) {
  constexpr float kUp = FMT == kFmtNVFP4 ? 11.0f : 0.0f;      // powers of two that probabilities are kept larger by
  bool grow = false;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const float base = m[n] - kUp;
#pragma unroll
    for (int i = 0; i < 4 * T; ++i) e[n][i] = fmaf(z[n][i >> 2][i & 3], k2[n], -base);
    grow |= largest(e[n]) > kGrow + kUp;
  }
  if (__any(grow)) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float top = z[n][0][0];
#pragma unroll
      for (int i = 1; i < 4 * T; ++i) top = fmaxf(top, z[n][i >> 2][i & 3]);
      top = rowgroup_max(top);
      const bool up = fmaf(top, k2[n], kUp - m[n]) > kGrow + kUp;
      const float now = up ? top * k2[n] : m[n], x = __builtin_amdgcn_exp2f(m[n] - now);
      m[n] = now;
      l[n] *= x;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[n][d] *= x;
      if constexpr (FMT == kFmtINT4)
#pragma unroll
        for (int g = 0; g < D / 64; ++g) off[n][g] *= x;
      const float base = now - kUp;
#pragma unroll
      for (int i = 0; i < 4 * T; ++i) e[n][i] = fmaf(z[n][i >> 2][i & 3], k2[n], -base);
    }
  }
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int i = 0; i < 4 * T; ++i) {
      e[n][i] = __builtin_amdgcn_exp2f(e[n][i]);
      l[n] += e[n][i];
    }
}

// Inclusive sum over the wave's lanes: within rows of 16 by shifts, then the rows' last lanes on to those after.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);     // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);    // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);    // row_bcast:31 into rows 2 and 3
  return v;
}

// A job of a call that is not split, by its workgroup's number; a number that no tile has does nothing.  One query a
// sequence: a division.  Up to 64 sequences: counted by a wave's scan, without a gap.  More: the first `batch` numbers
// are one tile of each; sequence b's others have the numbers from cu[b] group / R (rounded down) on, which are enough
// for its x = rows group rows: x / R, rounded down, at least.  Where gaps come in turn with tiles, as with x = 2 R,
// every 8 numbers are put in another order, so that they fall on all XCDs.  Counting all lengths in every workgroup,
// as ranges do, grew with the square of the batch: 16384 sequences to 300 tokens, 2 heads, 3291 us (561 so), drafts of
// 4 tokens, 16 query heads, 4740 (570).  Gaps cost little among many tiles, but one prompt's 512 tiles, two for every
// CU, took 379 us with one gap among them, 265 without.
struct KvJob {
  int b, tile;
};
template <int R>
int kv_numbers(const KvCache& kc, const KvAttn& a) {
  if (kc.cu == nullptr) return kc.batch * ((a.group + R - 1) / R);
  return kc.batch + (int(unsigned(kc.M) * unsigned(a.group) / R) + 7) / 8 * 8;
}
template <int R>
__device__ __forceinline__ KvJob kv_job(const KvCache& kc, const KvAttn& a, int index, int lane) {
  if (kc.cu == nullptr) {
    const int each = (a.group + R - 1) / R, b = int(unsigned(index) / unsigned(each));   // tiles of one token
    return {b, index - b * each};
  }
  auto row = [&](int b) { return min(max(kc.cu[b], 0), kc.M); };
  if (kc.batch <= 64) {
    const int n = lane < kc.batch ? (max(row(lane + 1) - row(lane), 0) * a.group + R - 1) / R : 0, end = wave_scan(n);
    const uint64_t in = __ballot(index < end);
    if (in == 0) return {0, -1};
    const int b = __builtin_ctzll(in);
    return {b, index - __builtin_amdgcn_readlane(end - n, b)};
  }
  if (index < kc.batch) return {index, 0};
  index -= kc.batch;
  index ^= (index >> 3) & 7;
  auto from = [&](int b) { return int(unsigned(row(b)) * unsigned(a.group) / R); };
  int lo = 0, n = kc.batch;                                   // the last b with from(b) <= index is in lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 63) / 64, i = lane * step;
    const uint64_t le = __ballot(i < n && from(lo + i) <= index);
    const int k = 63 - __builtin_clzll(le | 1);
    lo += k * step;
    n = min(step, n - k * step);
  }
  const int at = index - uni(from(lo));                        // below 0: rows in front of the first sequence
  return {lo, at < 0 ? -1 : 1 + at};
}

// The work of all sequences in units (of jobs x tokens), and the sequence that unit `at` falls into with the units
// before it (b = -1: none).  A batch of up to 64 is one wave's scan, which each
// wave does for itself; a larger one goes through the workgroup in chunks of NT.
struct KvFound {
  int b, before;
};
constexpr int kLeastUnits = 2;           // of a range
constexpr int kShortUnits = 8;           // of a range, up to which a range is part of one job

template <int R, int U, int NT>
struct KvScan {
  const KvCache& kc;
  const KvAttn& a;
  int* sh;                                     // 16 words of LDS
  int v = 0, end = 0, total = 0, tiles = 0, units = 1;
  int per = 1;                                 // units of a range
  bool short_ranges = false;                   // a range is part of one job; then v and end count ranges

  __device__ __forceinline__ KvSeq seq(int b) const {
    int len, row, rows;
    kc.sequence(b, len, row, rows);
    return kv_seq<R, U, true>(kc, a, len, row, rows);
  }
  __device__ __forceinline__ int units_of(int b) const {
    if (b >= kc.batch) return 0;
    const KvSeq s = seq(b);
    return s.tiles * s.units;
  }
  // This thread's inclusive sum in the chunk at `base`, the chunks before it being `before`; adds the chunk to it.
  __device__ __forceinline__ int chunk(int base, int& before) {
    v = units_of(base + int(threadIdx.x));
    const int sum = wave_scan(v), wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 63) sh[wave] = sum;
    __syncthreads();
    int lower = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      lower += w < wave ? sh[w] : 0;
      all += sh[w];
    }
    const int e = before + lower + sum;
    before += all;
    return e;
  }
  __device__ __forceinline__ int count() {
    if (kc.batch <= 64) {
      const int b = threadIdx.x & 63;
      if (b < kc.batch) {
        const KvSeq s = seq(b);
        tiles = s.tiles;
        units = s.units;
      }
      v = tiles * units;
      end = wave_scan(v);
      return total = __builtin_amdgcn_readlane(end, 63);
    }
    for (int base = 0; base < kc.batch; base += NT) end = chunk(base, total);
    return total = __builtin_amdgcn_readfirstlane(total);
  }
  // Cuts the units into ranges.  Evenly, so that a range may end one job and begin others; but where ranges are
  // short, what a second job costs (its rows, pages and first tokens one after the other, some 5 us) is more than an
  // uneven cut: then a job is cut into as many ranges as it has `per` units, if all of them are no more than the
  // workgroups there are (16 sequences of 400 .. 4000 tokens, 8 heads: 17.0 us evenly, 14.9 so).
  __device__ __forceinline__ void cut(int ranges) {
    per = max((total + ranges - 1) / ranges, kLeastUnits);
    if (kc.batch == 1 || kc.batch > 64 || per > kShortUnits) return;
    for (int p = per; p <= 2 * per; ++p) {
      const int n = tiles * int(unsigned(units + p - 1) / unsigned(p)), sum = wave_scan(n);
      if (__builtin_amdgcn_readlane(sum, 63) <= ranges) {
        v = n;
        end = sum;
        per = p;
        short_ranges = true;
        return;
      }
    }
  }
  // Units (short ranges: ranges) before sequence b.
  __device__ __forceinline__ int before(int b) {
    if (kc.batch <= 64) return __builtin_amdgcn_readlane(end - v, b);
    int sum = 0;
    for (int base = 0; base <= b; base += NT) {
      const int e = kc.batch <= NT ? end : chunk(base, sum);
      __syncthreads();
      if (base + int(threadIdx.x) == b) sh[9] = e - v;
    }
    __syncthreads();
    return uni(sh[9]);
  }
  __device__ __forceinline__ KvFound find(int at) {
    if (kc.batch <= 64) {
      const uint64_t in = __ballot(at < end);
      if (in == 0) return {-1, 0};
      const int lane = __builtin_ctzll(in);
      return {lane, __builtin_amdgcn_readlane(end - v, lane)};
    }
    __syncthreads();
    if (threadIdx.x == 0) sh[8] = -1;
    int before = 0;
    for (int base = 0; base < kc.batch; base += NT) {
      const int e = kc.batch <= NT ? end : chunk(base, before);
      __syncthreads();
      if (at >= e - v && at < e) {
        sh[8] = base + int(threadIdx.x);
        sh[9] = e - v;
      }
    }
    __syncthreads();
    return {__builtin_amdgcn_readfirstlane(sh[8]), __builtin_amdgcn_readfirstlane(sh[9])};
  }
};

// WK waves take the steps of the same 16 NQ rows in turn.
template <int FMT, int D, int NQ, int WK, bool SPLIT>
__global__ void __launch_bounds__(64 * WK, NQ == 1 ? 3 : 2) kv_attention_kernel(KvCache kc, KvAttn a) {
  using TL = KvTiles<NQ, WK>;
  constexpr int R = TL::R, U = TL::U, NT = 64 * WK, DT = D / 16, NG = FMT == kFmtINT4 ? D / 64 : 1;
  constexpr int PL = FMT == kFmtNVFP4 ? 1 : 2;                 // fp16 needs no second plane
  constexpr int TB = kv_tile_bytes(FMT, D), OS = D + 4;        // floats of a row of O in LDS
  __shared__ int sh[16];
  __shared__ float merge_o[WK * 16 * OS];
  __shared__ float merge_m[WK][16], merge_l[WK][16];
  const int lane = threadIdx.x & 63, wk = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int h = blockIdx.x % kc.heads, range = blockIdx.x / kc.heads;

  int b, job, unit = 0, left = 1;
  KvSeq s;
  if constexpr (SPLIT) {
    KvScan<R, U, NT> scan{kc, a, sh};
    const int total = scan.count();
    scan.cut(a.ranges);
    const int per = scan.per;
    const int64_t first64 = scan.short_ranges ? range : int64_t(range) * per;
    if (!scan.short_ranges && first64 >= total) return;
    const int first = int(first64);
    const KvFound f = scan.find(first);
    left = min(per, total - first);
    b = f.b;
    if (b < 0) return;
    s = kv_seq_of<R, U, SPLIT>(kc, a, b);
    if (scan.short_ranges) {
      const int each = (s.units + per - 1) / per;             // ranges of a job
      job = (first - f.before) / each;
      unit = ((first - f.before) % each) * per;
      left = min(per, s.units - unit);
    } else {
      job = (first - f.before) / s.units;
      unit = (first - f.before) % s.units;
    }
  } else {
    const KvJob f = kv_job<R>(kc, a, range, lane);
    b = f.b;
    job = f.tile;
    s = kv_seq_of<R, U, SPLIT>(kc, a, b);
    if (job < 0 || job >= s.tiles) return;
  }

  while (left > 0) {
    while (job >= s.tiles) {                                  // the next sequence with rows
      if (++b >= kc.batch) return;
      s = kv_seq_of<R, U, SPLIT>(kc, a, b);
      job = 0;
      unit = 0;
    }
    const int n_units = min(left, s.units - unit);
    const int tile_rows = SPLIT ? job : s.tiles - 1 - job;    // long causal tiles first
    const int row0 = tile_rows * R;
    const KvRows rows(kc, a, s);
    const KvSpan span = rows.span(row0, R);
    uint4 q[NQ][D / 32];
    float k2[NQ];
    int lo[NQ], hi[NQ];
    v4f s0[NQ][NG];
    load_queries<FMT, D, NQ>(a, s, rows, row0, h, r, c, q, lo, hi);

    // This wave's steps: 32 tokens from s.lo + 32 (unit WK + wk) on, every WK-th; those before every row's window
    // are left out.
    constexpr int STRIDE = 32 * WK;
    int t0 = s.lo + unit * U + 32 * wk;
    const int end = min(SPLIT ? s.lo + (unit + n_units) * U : INT32_MAX, span.behind);
    if (span.first > t0 && end > t0) t0 += (min(span.first, end) - t0) / STRIDE * STRIDE;
    const int steps = end > t0 ? (end - t0 + STRIDE - 1) / STRIDE : 0;
    const uint8_t* base = kc.pool + (int64_t(TB) << kc.page_shift) * h;
    const int mask = (1 << kc.page_shift) - 1;
    const KvLane<FMT, D> at(r, c);

    // Pages of 32 steps, one a lane (a step's two tiles in lanes 2 i, 2 i + 1), loaded 32 steps ahead.
    auto pages_from = [&](int i) {
      const int tile = (t0 >> 4) + (i + (lane >> 1)) * (STRIDE / 16) + (lane & 1);
      return tile * 16 < end ? kc.page_of(b, tile) : -1;
    };
    int pages = -1, next_pages = pages_from(0);
    auto fetch = [&](int i, KvStage<FMT, D> (&st)[2], bool (&ok)[2]) {
      if ((i & 31) == 0) {
        pages = next_pages;
        next_pages = pages_from(i + 32);
      }
      const int tile = (t0 >> 4) + i * (STRIDE / 16);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int p = __builtin_amdgcn_readlane(pages, (i & 31) * 2 + x);
        ok[x] = p >= 0;
        const uint8_t* from = base + int64_t(p >= 0 ? p : 0) * kc.page_bytes + uint32_t((tile + x) & mask) * uint32_t(TB);
        load_tile<FMT, D>(make_rsrc(from, p >= 0 ? TB : 0), at, st[x]);
      }
    };
    KvStage<FMT, D> now[2], next[2];
    bool now_ok[2], next_ok[2];
    fetch(0, now, now_ok);                                    // without a step: of no pages, so no bytes
    __builtin_amdgcn_sched_barrier(0);                        // these loads are on their way before Q is waited for

    finish_queries<FMT, D, NQ>(a, q, k2, s0);
    v4f o[NQ][DT], off[NQ][D / 64];
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

    auto step = [&](int t, KvStage<FMT, D> (&st)[2], const bool (&ok)[2]) {
      // Scores: lane (query r, tokens t + 16 i + 4 c + e).
      float z[NQ][2][4];
      if (t + 32 > span.behind || t < span.first) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          clear_outside<FMT, D>(span.first - t - 16 * i, span.behind - t - 16 * i, c, st[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (FMT == kFmtINT4) {
          uint4 ka[D / 32];
          uint32_t sk[NG][2];
          trade_groups<FMT, D>(st[i]);
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int w = 0; w < 2; ++w) sk[g][w] = kv_scales4<D>(st[i].vs[w], g);
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
                z[n][i][e] = fmaf(x[e], f16_value(sk[g][e >> 1] >> (16 * (e & 1))), z[n][i][e]);
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
      __builtin_amdgcn_sched_barrier(0);
      if (!(t + 32 <= span.behind_least && t >= span.first_most && ok[0] && ok[1])) mask_scores<NQ, 2>(z, t, c, ok, lo, hi);
      float e[NQ][8];
      probabilities<FMT, D, NQ, 2>(z, k2, m, l, o, off, e);
      __builtin_amdgcn_sched_barrier(0);
      add_values<FMT, D, NQ, PL>(st, e, o, off);
    };

    for (int i = 0; i < steps; ++i) {
      fetch(i + 1, next, next_ok);                            // behind the last step: no bytes
      step(t0 + i * STRIDE, now, now_ok);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        now[x] = next[x];
        now_ok[x] = next_ok[x];
      }
    }

    // Results of the segment: a whole job's rows are written, a part's go to the workspace.
    const bool all = !SPLIT || (unit == 0 && n_units == s.units);
    int tid = threadIdx.x;                                    // opaque: what follows from it is not kept in registers
    asm volatile("" : "+v"(tid));                             // over the steps
    const int er = tid & 15, ec = (tid >> 4) & 3;
    float* part = SPLIT ? a.part + ((int64_t(range) * kc.heads + h) * 2 + (unit > 0 ? 0 : 1)) * (R * (D + 2)) : nullptr;
    auto emit = [&](int in_tile, int d, auto& v, float mm, float ll) {        // features d .. of row in_tile
      constexpr int N = sizeof(v) / sizeof(float);
      const int i = tile_rows * R + in_tile;
      if (i >= rows.rows) return;
      if (!all) {
        if (d == 0) {
          part[in_tile] = mm;
          part[R + in_tile] = ll;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) part[2 * R + in_tile * D + d + e] = v[e];
        return;
      }
      const int token = int(unsigned(i) / unsigned(a.group));
      kv_store<N>(a, s.row + token, h * a.group + i - token * a.group, D, d, v, mm, ll);
    };
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      l[n] = rowgroup_sum(l[n]);
      if constexpr (FMT == kFmtINT4)
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] += off[n][d >> 2];
      const float mm = FMT == kFmtNVFP4 ? m[n] - 11.0f : m[n];
      __syncthreads();                                      // the rows before are read
      float* mine_o = merge_o + (wk * 16 + er) * OS;
#pragma unroll
      for (int d = 0; d < DT; d += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(mine_o + o_feature<FMT, D>(ec, d, i)) =
              make_float4(o[n][d][i], o[n][d + 1][i], o[n][d + 2][i], o[n][d + 3][i]);
      if (ec == 0) {
        merge_m[wk][er] = mm;
        merge_l[wk][er] = l[n];
      }
      __syncthreads();
      constexpr int TPR = NT / 16, FPT = D / TPR;           // threads a row, features a thread
      const int row = tid / TPR, d = tid % TPR * FPT;
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
    left -= n_units;
    unit += n_units;
    if (unit == s.units) {
      unit = 0;
      ++job;
    }
  }
}

// Prompts: the same with what the waves of a workgroup share done once.  Four waves of 32 rows walk the tokens in chunks
// of 64; of a chunk each wave makes one tile's operands 16-bit and puts them in LDS in operand order (K's of a
// tile, its half of V's of a step of 32 tokens), the next chunk's while this one is worked on, with a barrier a chunk.
// Then a wave's vector instructions are the softmax's and a quarter of the conversions.  2048 queries x 32 heads on
// 8192 tokens, 8 heads of 128, MXFP4 (241 GFLOP): a wave converting for itself 312 us, so 249 (967 TFLOP/s); NVFP4 261,
// INT4, whose scales multiply scores and probabilities, 343.
template <int FMT, int D>
struct KvShared {
  uint4 k[2][4][D / 32][64];
  uint2 v[2][2][D / 16][64][2];
  uint2 s[2][4][FMT == kFmtINT4 ? D / 4 / 2 : 1];              // INT4: a tile's scales, as in the pool
};

template <int FMT, int D>
__device__ __forceinline__ void share_tile(KvStage<FMT, D>& st, int tile, int lane, KvShared<FMT, D>& sh, int half) {
  trade_groups<FMT, D>(st);
#pragma unroll
  for (int j = 0; j < D / 32; ++j) sh.k[half][tile][j][lane] = k_operand<FMT, D>(st, j);
  auto put = [&](int dt, uint32_t lo, uint32_t hi) { sh.v[half][tile >> 1][dt][lane][tile & 1] = make_uint2(lo, hi); };
  if constexpr (FMT == kFmtINT4) {
    if ((lane & 15) < D / 32) sh.s[half][tile][(lane & 15) * 4 + (lane >> 4)] = make_uint2(st.vs[0], st.vs[1]);
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
      uint32_t w[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t x = value_pair<D>(st, t, g);
        w[t][0] = x & 0x0F0F0F0Fu;
        w[t][1] = (x >> 4) & 0x0F0F0F0Fu;
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) put(4 * g + f, fp8_pair(w[0][f & 1], f >> 1), fp8_pair(w[1][f & 1], f >> 1));
    }
  } else {
    v2h nv[2] = {};
    if constexpr (FMT == kFmtNVFP4) {
      nv[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(st.vs[0], 1.0f, false);
      nv[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(st.vs[0], 1.0f, true);
    }
    auto one = [&](auto byte) {
      constexpr int B = decltype(byte)::value;
      const uint32_t x[4] = {v_pair<FMT, D, 0, B>(st, nv), v_pair<FMT, D, 1, B>(st, nv), v_pair<FMT, D, 2, B>(st, nv),
                             v_pair<FMT, D, 3, B>(st, nv)};
      put(2 * B, __builtin_amdgcn_perm(x[1], x[0], kLowHalves), __builtin_amdgcn_perm(x[3], x[2], kLowHalves));
      put(2 * B + 1, __builtin_amdgcn_perm(x[1], x[0], kHighHalves), __builtin_amdgcn_perm(x[3], x[2], kHighHalves));
    };
    one(std::integral_constant<int, 0>{});
    one(std::integral_constant<int, 1>{});
    if constexpr (D == 128) {
      one(std::integral_constant<int, 2>{});
      one(std::integral_constant<int, 3>{});
    }
  }
}

template <int FMT, int D>
__global__ void __launch_bounds__(256, 2) kv_prompt_kernel(KvCache kc, KvAttn a) {
  constexpr int NQ = 2, R = 128, DT = D / 16, NG = FMT == kFmtINT4 ? D / 64 : 1, TB = kv_tile_bytes(FMT, D);
  __shared__ KvShared<FMT, D> shared;
  __shared__ int marks[2][4];                                  // of a half's tiles: whether they are there
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int h = blockIdx.x % kc.heads, index = blockIdx.x / kc.heads;
  const KvJob f = kv_job<R>(kc, a, index, lane);
  const KvSeq s = kv_seq_of<R, 32, false>(kc, a, f.b);
  if (f.tile < 0 || f.tile >= s.tiles) return;
  const int tile_rows = s.tiles - 1 - f.tile;                  // long causal tiles first
  const KvRows rows(kc, a, s);
  const int wg0 = tile_rows * R, row0 = wg0 + wave * 32;

  uint4 q[NQ][D / 32];
  float k2[NQ];
  int lo[NQ], hi[NQ];
  v4f s0[NQ][NG];
  load_queries<FMT, D, NQ>(a, s, rows, row0, h, r, c, q, lo, hi);
  const KvSpan span = rows.span(row0, 32), wg = rows.span(wg0, R);
  const int t0 = wg.first & ~63, chunks = wg.behind > t0 ? (wg.behind - t0 + 63) / 64 : 0;
  const uint8_t* base = kc.pool + (int64_t(TB) << kc.page_shift) * h;
  const int mask = (1 << kc.page_shift) - 1;
  const KvLane<FMT, D> at(r, c);

  // This wave's tile of every chunk: pages of 64 chunks, one a lane.
  auto pages_from = [&](int i) {
    const int tile = (t0 >> 4) + (i + lane) * 4 + wave;
    return tile * 16 < wg.behind ? kc.page_of(f.b, tile) : -1;
  };
  int pages = -1, next_pages = pages_from(0);
  KvStage<FMT, D> st;
  auto fetch = [&](int i) {
    if ((i & 63) == 0) {
      pages = next_pages;
      next_pages = pages_from(i + 64);
    }
    const int p = __builtin_amdgcn_readlane(pages, i & 63), tile = (t0 >> 4) + i * 4 + wave;
    const uint8_t* from = base + int64_t(p >= 0 ? p : 0) * kc.page_bytes + uint32_t(tile & mask) * uint32_t(TB);
    load_tile<FMT, D>(make_rsrc(from, p >= 0 ? TB : 0), at, st);
    return p >= 0;
  };
  // The fetched tile of chunk i to LDS; a tile that is not there leaves a mark.
  auto share = [&](int i, bool there) {
    const int t = t0 + i * 64 + wave * 16;
    if (t + 16 > wg.behind || t < wg.first) clear_outside<FMT, D>(wg.first - t, wg.behind - t, c, st);
    share_tile<FMT, D>(st, wave, lane, shared, i & 1);
    if (lane == 0) marks[i & 1][wave] = there;
  };

  bool there = fetch(0);
  finish_queries<FMT, D, NQ>(a, q, k2, s0);
  v4f o[NQ][DT], off[NQ][D / 64];
  float m[NQ], l[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = kLowest;
    l[n] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[n][d] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < D / 64; ++g) off[n][g] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  if (chunks > 0) share(0, there);
  if (chunks > 1) there = fetch(1);
  for (int i = 0; i < chunks; ++i) {
    __syncthreads();                                           // chunk i is there, and the other half is read
    const int half = i & 1, t = t0 + i * 64;
    if (t + 64 > span.first && t < span.behind) {
      bool ok[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) ok[y] = uni(marks[half][y]) != 0;
      float z[NQ][4][4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        v4f acc[NQ][NG];
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int g = 0; g < NG; ++g) acc[n][g] = FMT == kFmtINT4 ? s0[n][g] : v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 ka = shared.k[half][y][j][lane];
#pragma unroll
          for (int n = 0; n < NQ; ++n)
            acc[n][FMT == kFmtINT4 ? j / 2 : 0] = mfma16<FMT>(ka, q[n][j], acc[n][FMT == kFmtINT4 ? j / 2 : 0]);
        }
        if constexpr (FMT == kFmtINT4) {
          uint2 sk[NG];
#pragma unroll
          for (int g = 0; g < NG; ++g) sk[g] = shared.s[half][y][g * 4 + c];
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              z[n][y][e] = 0.f;
#pragma unroll
              for (int g = 0; g < NG; ++g)
                z[n][y][e] = fmaf(acc[n][g][e], f16_value((e < 2 ? sk[g].x : sk[g].y) >> (16 * (e & 1))), z[n][y][e]);
            }
        } else {
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[n][y][e] = acc[n][0][e];
        }
      }
      if (!(t + 64 <= span.behind_least && t >= span.first_most && ok[0] && ok[1] && ok[2] && ok[3]))
        mask_scores<NQ, 4>(z, t, c, ok, lo, hi);
      float e[NQ][16];
      probabilities<FMT, D, NQ, 4>(z, k2, m, l, o, off, e);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          uint4 p[NQ];
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            float w[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) w[y] = e[n][8 * x + y];
            if constexpr (FMT == kFmtINT4) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint2 sv = shared.s[half][2 * x + y][(NG + g) * 4 + c];
#pragma unroll
                for (int b = 0; b < 4; ++b) w[4 * y + b] *= f16_value((b < 2 ? sv.x : sv.y) >> (16 * (b & 1)));
              }
            }
            if constexpr (FMT == kFmtNVFP4) {
              p[n] = to_f16(w);
            } else {
              uint4 one[1];
              split_planes<1>(w, one);
              p[n] = one[0];
            }
            if constexpr (FMT == kFmtINT4)
              off[n][g] = mfma_bf16(make_uint4(0xC100C100u, 0xC100C100u, 0xC100C100u, 0xC100C100u), p[n], off[n][g]);
          }
#pragma unroll
          for (int d = 0; d < DT / NG; ++d) {
            const uint4 va = *reinterpret_cast<const uint4*>(&shared.v[half][x][g * (DT / NG) + d][lane][0]);
#pragma unroll
            for (int n = 0; n < NQ; ++n) o[n][g * (DT / NG) + d] = mfma16<FMT>(va, p[n], o[n][g * (DT / NG) + d]);
          }
        }
    }
    if (i + 1 < chunks) {
      share(i + 1, there);
      if (i + 2 < chunks) there = fetch(i + 2);
    }
  }
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    l[n] = rowgroup_sum(l[n]);
    const int i = row0 + n * 16 + r;
    if (i >= rows.rows) continue;
    const int token = int(unsigned(i) / unsigned(a.group));
#pragma unroll
    for (int d = 0; d < DT; d += 4)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) v[y] = o[n][d + y][e] + (FMT == kFmtINT4 ? off[n][d >> 2][e] : 0.f);
        kv_store<4>(a, s.row + token, h * a.group + i - token * a.group, D, o_feature<FMT, D>(c, d, e), v,
                    FMT == kFmtNVFP4 ? m[n] - 11.0f : m[n], l[n]);
      }
  }
}

constexpr int kJoinGroups = 2048;        // workgroups of a join at most, if jobs x heads are not more

// Joins the parts of split jobs.  A workgroup takes a job and its rows: D / 8 threads take a row's features, and of the
// 2048 / D such groups as many share a row as the parts keep busy.  How it finds its job: by number, in a batch whose
// scan is one wave's; by sequence, where each is one job and they are not many; else as the one inside which a range
// border is the first (by sequence / border, 2 heads to 2000 tokens: 256 sequences 31.4 / 32.1 us with the attention,
// 1024 73.5 / 72.6, 4096 316 / 279).
constexpr int kJoinSeqs = 512;
enum { kByJob = 0, kBySeq = 1, kByBorder = 2 };
template <int D, int R, int U, int HOW>
__global__ void __launch_bounds__(256) kv_join_kernel(KvCache kc, KvAttn a) {
  constexpr int F = 8, TPR = D / F, NP = 256 / TPR;
  __shared__ int sh[16];
  __shared__ float sm[NP], sl[NP], so[NP][D];
  const int h = blockIdx.x % kc.heads, index = blockIdx.x / kc.heads;
  KvScan<R, U, 256> scan{kc, a, sh};
  const int total = scan.count();
  scan.cut(a.ranges);
  const int per = scan.per;
  int b, job, start;
  KvSeq s;
  if constexpr (HOW == kByJob) {
    const int sum = wave_scan(scan.tiles);
    const uint64_t in = __ballot(index < sum);
    if (in == 0) return;
    b = __builtin_ctzll(in);
    job = index - __builtin_amdgcn_readlane(sum - scan.tiles, b);
    s = kv_seq_of<R, U, true>(kc, a, b);
    start = scan.before(b);
    if (!scan.short_ranges) start += job * s.units;
  } else if constexpr (HOW == kBySeq) {
    b = index;
    job = 0;
    start = scan.before(b);
    s = kv_seq_of<R, U, true>(kc, a, b);
  } else {
    const int64_t at = int64_t(index + 1) * per;
    if (at >= total) return;
    const KvFound f = scan.find(int(at));
    if (f.b < 0) return;
    b = f.b;
    s = kv_seq_of<R, U, true>(kc, a, b);
    job = (int(at) - f.before) / s.units;
    start = f.before + job * s.units;
    if (start == at || start < at - per) return;
  }
  int first = start / per, last = (start + s.units - 1) / per;          // ranges that hold parts
  if (scan.short_ranges) {
    const int each = (s.units + per - 1) / per;
    first = start + job * each;
    last = first + each - 1;
  }
  if (first == last) return;
  const int d = threadIdx.x % TPR * F, slot = threadIdx.x / TPR;
  const int rows = min(s.rows * a.group - job * R, R);
  int shift = 0;                                             // 1 << shift slots share a row, parts / 2 or as many as there are
  while ((2 << shift) < last - first + 1 && (1 << shift) < NP) ++shift;
  const int x = slot & ((1 << shift) - 1), at_once = NP >> shift;
  for (int base = int(blockIdx.y) * at_once; base < rows; base += int(gridDim.y) * at_once) {
    const int row = base + (slot >> shift);
    float m = kLowest, l = 0.f, v[F] = {};
    if (row < rows)
      for (int g = first + x; g <= last; g += 1 << shift) {
        // the first range begins the job (a part of kind 1), the others go on with it
        const float* part = a.part + ((int64_t(g) * kc.heads + h) * 2 + (g == first ? 1 : 0)) * (R * (D + 2));
        const float4* o = reinterpret_cast<const float4*>(part + 2 * R + row * D + d);
        const float4 o0 = o[0], o1 = o[1];
        const float pm = part[row], pl = part[R + row], now = fmaxf(m, pm);
        const float y = __builtin_amdgcn_exp2f(m - now), z = __builtin_amdgcn_exp2f(pm - now);
        const float w[F] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
#pragma unroll
        for (int e = 0; e < F; ++e) v[e] = v[e] * y + w[e] * z;
        l = l * y + pl * z;
        m = now;
      }
    if (shift > 0) {
      __syncthreads();                                       // the rows before are read
      if (d == 0) {
        sm[slot] = m;
        sl[slot] = l;
      }
#pragma unroll
      for (int e = 0; e < F; ++e) so[slot][d + e] = v[e];
      __syncthreads();
      if (x == 0)
        for (int w = 1; w < 1 << shift; ++w) {
          const float pm = sm[slot + w], now = fmaxf(m, pm);
          const float y = __builtin_amdgcn_exp2f(m - now), z = __builtin_amdgcn_exp2f(pm - now);
#pragma unroll
          for (int e = 0; e < F; ++e) v[e] = v[e] * y + so[slot + w][d + e] * z;
          l = l * y + sl[slot + w] * z;
          m = now;
        }
    }
    if (x == 0 && row < rows) {
      const int i = job * R + row, token = int(unsigned(i) / unsigned(a.group));
      kv_store<F>(a, s.row + token, h * a.group + i - token * a.group, D, d, v, m, l);
    }
  }
}

template <int FMT, int D, int NQ, int WK>
void attend_whole(const KvCache& kc, const KvAttn& a, hipStream_t s) {
  const unsigned n = kv_numbers<KvTiles<NQ, WK>::R>(kc, a);
  kv_attention_kernel<FMT, D, NQ, WK, false><<<dim3(n * kc.heads), 64 * WK, 0, s>>>(kc, a);
}
template <int FMT, int D, int NQ, int WK>
void attend_split(const KvCache& kc, const KvAttn& a, int jobs, hipStream_t s) {
  constexpr int R = KvTiles<NQ, WK>::R, U = KvTiles<NQ, WK>::U;
  kv_attention_kernel<FMT, D, NQ, WK, true><<<dim3(a.ranges * kc.heads), 64 * WK, 0, s>>>(kc, a);   // two ranges at least
  const int64_t most = kc.cu == nullptr ? a.group : int64_t(kc.M) * a.group, rows = most < R ? most : R;
  const int how = kc.batch <= 64 ? kByJob : kc.cu == nullptr && a.group <= R && kc.batch <= kJoinSeqs ? kBySeq : kByBorder;
  const int x = (how == kByJob ? jobs : how == kBySeq ? kc.batch : a.ranges - 1) * kc.heads;
  const int fill = kJoinGroups / x;
  const dim3 grid(x, unsigned(fill < 1 ? 1 : fill < rows ? fill : rows));
  if (how == kByJob)
    kv_join_kernel<D, R, U, kByJob><<<grid, 256, 0, s>>>(kc, a);
  else if (how == kBySeq)
    kv_join_kernel<D, R, U, kBySeq><<<grid, 256, 0, s>>>(kc, a);
  else
    kv_join_kernel<D, R, U, kByBorder><<<grid, 256, 0, s>>>(kc, a);
}

template <int FMT, int D>
void attend_plan(const KvPlan& p, const KvCache& kc, const KvAttn& a, hipStream_t s) {
  // 8 waves are a CU's at a time, 4 three times: 8 heads, to 700 tokens, 8 waves / 4 (us): 32 sequences 9.8 / 10.2, 64
  // 16.3 / 12.7, 1024 176 / 98.8; to 300 7.5 / 7.7, 11.5 / 8.8, 125 / 59.3; INT4 8.4 / 8.6, 13.0 / 9.9.
  if (p.rows == 16 && p.split)
    attend_split<FMT, D, 1, 4>(kc, a, p.jobs, s);
  else if (p.rows == 16)
    kv_numbers<16>(kc, a) * kc.heads > 256 ? attend_whole<FMT, D, 1, 4>(kc, a, s)
                                           : attend_whole<FMT, D, 1, 8>(kc, a, s);
  else if (p.rows == 32)
    p.split ? attend_split<FMT, D, 2, 4>(kc, a, p.jobs, s) : attend_whole<FMT, D, 2, 4>(kc, a, s);
  else
    kv_prompt_kernel<FMT, D><<<dim3(unsigned(kv_numbers<128>(kc, a)) * kc.heads), 256, 0, s>>>(kc, a);
}

}  // namespace

hipError_t launch_kv_attention(int fmt, int D, const KvCache& kc, const uint16_t* Q, int64_t ldq, int q_heads,
                               float scale, int window, bool causal, uint16_t* Y, int64_t ldy, float* lse, float* part,
                               hipStream_t s) {
  KvPlan p = kv_plan(D, kc.batch, kc.M, q_heads, kc.heads, kc.capacity());
  // A window is all that a row sees of a long table: where its tokens would not be split, they are not (8 heads to 8192
  // tokens, split / whole: window 512, 4 sequences 10.9 / 8.5 us, 64 17.5 / 12.5; 1024, 1 10.2 / 10.2, 64 24.2 / 18.2).
  if (p.split && window > 0 && causal && window < kc.capacity()) {
    const KvPlan w = kv_plan(D, kc.batch, kc.M, q_heads, kc.heads, window);
    if (!w.split) p = w;
  }
  if (window > INT32_MAX - int(kKvMaxRows) - 1) window = INT32_MAX - int(kKvMaxRows) - 1;   // a row's place minus it fits
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
