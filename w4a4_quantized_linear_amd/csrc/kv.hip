// svdq_kv_append, svdq_kv_read, svdq_kv_copy and svdq_kv_compact: what fills a 4-bit key-value cache, reads it
// back and moves its pages and tokens.  Layout: kv.h.
#include <type_traits>

#include "kv.h"

namespace svdq {

namespace {

// v of the lane that differs in bit log2(X) of its number (X = 1, 2) or, X = 4, 8, of its mirror in 8, 16 lanes,
// which serves a reduction in rising order of X as well; X = -8: of the lane 8 further on of 16.
template <int X>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
  constexpr int ctrl = X == 1 ? 0xB1 : X == 2 ? 0x4E : X == 4 ? 0x141 : X == 8 ? 0x140 : 0x128;
  return uint32_t(__builtin_amdgcn_mov_dpp(int(v), ctrl, 0xF, 0xF, true));
}
template <int X>
__device__ __forceinline__ float partner_of(float v) {
  const uint32_t u = __float_as_uint(v);
  return __uint_as_float(partner<X>(u));
}
template <int X>
__device__ __forceinline__ double partner_of(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __float_as_uint(partner_of<X>(__uint_as_float(uint32_t(u))));
  const uint32_t hi = __float_as_uint(partner_of<X>(__uint_as_float(uint32_t(u >> 32))));
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

// max and sum of v over the W lanes of an aligned group
template <int W>
__device__ __forceinline__ float group_max(float v) {
  if constexpr (W > 1) v = fmaxf(v, partner_of<1>(v));
  if constexpr (W > 2) v = fmaxf(v, partner_of<2>(v));
  if constexpr (W > 4) v = fmaxf(v, partner_of<4>(v));
  return v;
}
template <int W, typename T>
__device__ __forceinline__ T group_sum(T v) {
  v += partner_of<1>(v);
  v += partner_of<2>(v);
  v += partner_of<4>(v);
  if constexpr (W > 8) v += partner_of<8>(v);
  return v;
}

struct KvRope {
  const float* freq;
  const int32_t* axis;
  const int32_t* pos;
  int32_t pairs, axes, halves;
};

struct KvAppend {
  const uint16_t *K, *V, *Q;
  uint16_t* Q_out;
  int64_t ldk, ldv, ldq, ldqo;
  const uint16_t *norm_q, *norm_k;
  float eps;
  int32_t q_heads;
  KvRope rope;
};

// A row's sines as a lane needs them: of pairs 4 l .. + 3 (neighbours) or of features 8 l .. + 7 (halves).
template <typename T>
struct KvSines {
  T c[8], s[8];
};

// A lane's 8 features turned.  Neighbours: they are 4 pairs.  Halves: feature d pairs with d + pairs, which lane
// l + pairs / 8 of the head holds.
template <int L, typename T>
__device__ __forceinline__ void turn(T (&x)[8], const KvRope& r, int l, const KvSines<T>& t) {
  if (!r.halves) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (4 * l + j >= r.pairs) continue;
      const T u = x[2 * j] * t.c[j] - x[2 * j + 1] * t.s[j];
      x[2 * j + 1] = x[2 * j] * t.s[j] + x[2 * j + 1] * t.c[j];
      x[2 * j] = u;
    }
    return;
  }
  const int step = r.pairs / 8, from = l < step ? l + step : l < 2 * step ? l - step : l;
  const T sign = l < step ? T(-1) : T(1);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const T other = L == 16 && step == 8 ? partner_of<-8>(x[j]) : __shfl(x[j], from, L);
    const T u = x[j] * t.c[j] + sign * (other * t.s[j]);     // (a c - b s, b c + a s)
    x[j] = l < 2 * step ? u : x[j];
  }
}

// a / b for the codes, b > 0: div_refined on the group's one correctly rounded reciprocal, with a's sign, which
// -0 would lose.  Where that is not the correctly rounded quotient (it is below 2^-40), the code is 0.
__device__ __forceinline__ float kv_div(float a, float b, float rb) { return copysignf(div_refined(a, b, rb), a); }

// 8 codes of a lane's 8 finite bf16 values, given the number they are divided by: a dword, in order.
template <int FMT>
__device__ __forceinline__ uint32_t kv_encode8(const float (&x)[8], float div) {
  uint32_t d = 0;
  if constexpr (FMT == kFmtMXFP4) {
    d = cvt_fp4x2_div<0>(d, x[0], x[1], div);
    d = cvt_fp4x2_div<1>(d, x[2], x[3], div);
    d = cvt_fp4x2_div<2>(d, x[4], x[5], div);
    d = cvt_fp4x2_div<3>(d, x[6], x[7], div);
  } else {
    const float rd = div == 0.f ? 0.f : 1.0f / div;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = kv_div(x[i], div, rd);     // 0 with x's sign where div is 0
    if constexpr (FMT == kFmtINT4) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        d |= uint32_t(int(fminf(fmaxf(__builtin_rintf(v[i]), -8.f), 7.f)) + 8) << (4 * i);
    } else {
      d = cvt_fp4x2<0>(d, v[0], v[1]);
      d = cvt_fp4x2<1>(d, v[2], v[3]);
      d = cvt_fp4x2<2>(d, v[4], v[5]);
      d = cvt_fp4x2<3>(d, v[6], v[7]);
    }
  }
  return d;
}

// 1 / sqrt(x) to about 2^-52, x > 0: the hardware's estimate (at least 2^-20) by two of Newton's steps.
__device__ __forceinline__ double rsqrt64(double x) {
  double y = __builtin_amdgcn_rsq(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = fma(0.5 * y, fma(-x * y, y, 1.0), y);
  return y;
}

// A head's 8 features of a lane, normalized in 64 bits.
template <int D>
__device__ __forceinline__ void norm64(double (&z)[8], const float (&w)[8], float eps) {
  double sum = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum = fma(z[j], z[j], sum);
  const double mean = group_sum<D / 8>(sum) * (1.0 / D) + double(eps);
  // a row of zeros with eps 0, or of infinities: as the definition has it
  const double k = mean > 0 && mean < __builtin_huge_val() ? rsqrt64(mean) : 1 / sqrt(mean);
#pragma unroll
  for (int j = 0; j < 8; ++j) z[j] = z[j] * k * w[j];
}

// A wave takes units of one row: 8 features a lane, so D / 8 lanes a head, and 4 heads (of 64 features: 8) of K, V
// or Q at once; all units of a row, or every `parts`-th where few rows would leave CUs idle.  The inputs of the next
// units are on their way while one is worked on.  A row's sines are computed once by its wave, pair p in lane p.
// K's norm and rotation are in 64 bits, so that its codes, which are choices, do not hang on an order of summation
// or on a sine's last bit; the angle pos x freq is a 64-bit product, which holds far positions.  Q's are
// in 32 bits with the same sines, but for the norm of a head whose squares are not in their range.
// 9165 rows, 32 + 2 x 8 heads of 128, NVFP4, norm and three axes (198 MB): with a feature pair a lane, IEEE divisions
// and 64-bit quotients it was bound by its instructions, 98 us; so 57.9 (3.4 TB/s), the vector units busy 67% of the
// time.  Without the norm 53.7, without the rotation 50.9, without both, so without 64-bit arithmetic, 49.5 (4.0 TB/s,
// busy 48%).  At the four waves a SIMD that the loads want, INT4 heads of 128 spill 11 registers, NVFP4's one.
template <int FMT, int D>
__global__ void __launch_bounds__(256, 4) kv_append_kernel(KvCache kc, KvAppend a, int parts) {
  constexpr int L = D / 8, HPW = 64 / L, G = kv_group(FMT), AHEAD = 2;
  const int lane = threadIdx.x & 63, l = lane % L;
  const int wave = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = wave / parts, part = wave - m * parts;
  if (m >= kc.M) return;
  const int kv_units = (kc.heads + HPW - 1) / HPW, units = 2 * kv_units + (a.q_heads + HPW - 1) / HPW;

  auto load = [&](int u) -> uint4 {
    const bool is_k = u < kv_units, is_q = u >= 2 * kv_units;
    const int h = (is_q ? u - 2 * kv_units : is_k ? u : u - kv_units) * HPW + lane / L;
    const uint16_t* src = is_q ? a.Q + int64_t(m) * a.ldq : is_k ? a.K + int64_t(m) * a.ldk : a.V + int64_t(m) * a.ldv;
    if (u >= units || h >= (is_q ? a.q_heads : kc.heads)) return make_uint4(0, 0, 0, 0);
    return *reinterpret_cast<const uint4*>(src + h * D + 8 * l);
  };
  const int b = kc.cu == nullptr ? m : kv_sequence_of(kc.cu, kc.batch, m, lane);
  if (b < 0) return;
  uint4 in[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) in[i] = load(part + i * parts);
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (a.norm_q) wq = *reinterpret_cast<const uint4*>(a.norm_q + 8 * l);
  if (a.norm_k) wk = *reinterpret_cast<const uint4*>(a.norm_k + 8 * l);
  int len, row, rows;
  kc.sequence(b, len, row, rows);
  const int t = len - rows + (m - row);                        // the row's place
  const int page = t < 0 ? -1 : kc.page_of(b, t >> 4);
  uint8_t* tile = nullptr;
  if (page >= 0)
    tile = kc.pool + int64_t(page) * kc.page_bytes +
           int64_t((t >> 4) & ((1 << kc.page_shift) - 1)) * kv_tile_bytes(FMT, D);
  const int64_t head_bytes = int64_t(kv_tile_bytes(FMT, D)) << kc.page_shift;

  KvSines<double> sines;
  const KvRope& r = a.rope;
  if (r.pairs > 0) {
    double s = 0, c = 1;
    if (lane < r.pairs) {
#pragma clang fp contract(off)
      const int ax = r.axis == nullptr ? 0 : r.axis[lane];
      int pos = t;
      if (r.pos != nullptr) pos = ax >= 0 && ax < r.axes ? r.pos[int64_t(ax) * kc.M + m] : 0;
      const double angle = double(pos) * double(r.freq[lane]);
      sincos(angle, &s, &c);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!r.halves && j >= 4) {
        sines.c[j] = 1;
        sines.s[j] = 0;
        continue;
      }
      const int p = r.halves ? 8 * l + j : 4 * l + j, from = p >= r.pairs ? p - r.pairs : p;
      sines.c[j] = __shfl(c, from & 63);
      sines.s[j] = __shfl(s, from & 63);
    }
  }
  // K's units, V's, Q's, in loops of their own: the 64-bit sines are K's alone.
  int u = part;
  auto next = [&]() -> uint4 {
    const uint4 now = in[0];
#pragma unroll
    for (int i = 0; i + 1 < AHEAD; ++i) in[i] = in[i + 1];
    in[AHEAD - 1] = load(u + AHEAD * parts);
    return now;
  };
  auto keep = [&](auto kind, float (&x)[8], int h) {             // kind 0: K, 1: V
    constexpr bool is_k = decltype(kind)::value == 0;
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = kv_finite_bf16(x[j]);
      top = fmaxf(top, fabsf(x[j]));
    }
    float div;
    const uint32_t s = kv_scale<FMT>(group_max<G / 8>(top), div);
    const uint32_t codes = kv_encode8<FMT>(x, div);
    if (h >= kc.heads || page < 0) return;
    uint8_t* to = tile + h * head_bytes;
    const int ti = t & 15, g = 8 * l / G;
    if constexpr (is_k) {
      *reinterpret_cast<uint32_t*>(to + kv_k_code<FMT, D>(ti, 8 * l)) = codes;
    } else if constexpr (FMT != kFmtINT4 && D == 128) {
      *reinterpret_cast<uint32_t*>(to + kv_v_code<FMT, D>(ti, 8 * l)) = codes;
    } else {                                                     // two pieces of 4 features
      *reinterpret_cast<uint16_t*>(to + kv_v_code<FMT, D>(ti, 8 * l)) = uint16_t(codes);
      *reinterpret_cast<uint16_t*>(to + kv_v_code<FMT, D>(ti, 8 * l + 4)) = uint16_t(codes >> 16);
    }
    if (l % (G / 8) == 0) {
      uint8_t* at = to + (is_k ? kv_k_scale<FMT, D>(ti, g) : kv_v_scale<FMT, D>(ti, g));
      if constexpr (FMT == kFmtINT4)
        *reinterpret_cast<uint16_t*>(at) = uint16_t(s);
      else
        *at = uint8_t(s);
    }
  };

  for (; u < kv_units; u += parts) {
    float x[8];
    unpack_bf8(next(), x);
    if (a.norm_k != nullptr || r.pairs > 0) {
      double z[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = x[j];
      if (a.norm_k != nullptr) {
        float w[8];
        unpack_bf8(wk, w);
        norm64<D>(z, w, a.eps);
      }
      if (r.pairs > 0) turn<L, double>(z, r, l, sines);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = float(z[j]);
    }
    keep(std::integral_constant<int, 0>{}, x, u * HPW + lane / L);
  }
  for (; u < 2 * kv_units; u += parts) {
    float x[8];
    unpack_bf8(next(), x);
    keep(std::integral_constant<int, 1>{}, x, (u - kv_units) * HPW + lane / L);
  }
  KvSines<float> sines32;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sines32.c[j] = float(sines.c[j]);
    sines32.s[j] = float(sines.s[j]);
  }
  for (; u < units; u += parts) {
    const int h = (u - 2 * kv_units) * HPW + lane / L;
    float x[8];
    unpack_bf8(next(), x);
    if (a.norm_q != nullptr) {
      float sum = 0.f, w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
      sum = group_sum<L>(sum);
      const float k = __builtin_amdgcn_rsqf(sum * (1.0f / D) + a.eps);
      unpack_bf8(wq, w);
      // Squares that leave 32 bits, above or (with an eps no larger) below: the head in 64 bits.  From 2^-80 on the
      // squares that underflow are no part of the sum's 24 bits.
      const bool in32 = h >= a.q_heads || (sum >= 0x1p-80f && sum <= 0x1p127f);
      if (__any(!in32)) {
        double z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = x[j];
        norm64<D>(z, w, a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = in32 ? x[j] * k * w[j] : float(z[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * k * w[j];
      }
    }
    if (r.pairs > 0) turn<L, float>(x, r, l, sines32);
    if (h < a.q_heads)
      *reinterpret_cast<uint4*>(a.Q_out + int64_t(m) * a.ldqo + h * D + 8 * l) =
          make_uint4(cvt_bf2(x[0], x[1]), cvt_bf2(x[2], x[3]), cvt_bf2(x[4], x[5]), cvt_bf2(x[6], x[7]));
  }
}

// A workgroup takes a row, a wave heads of K or V of it; a row without a place reads as zeros.  The append's 9165 rows
// to fp32 (85.6 MB) take 24.4 us (3.5 TB/s): two features a lane, the vector units busy 19% of the time, the rest waits.
template <int FMT, int D>
__global__ void __launch_bounds__(256) kv_read_kernel(KvCache kc, void* K, int64_t ldk, void* V, int64_t ldv, int f32) {
  constexpr int LPH = D / 2, HPW = 64 / LPH, G = kv_group(FMT);
  const int lane = threadIdx.x & 63, sub = lane % LPH;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + blockIdx.y * 4, waves = gridDim.y * 4;
  const int m = blockIdx.x;
  const int b = kc.cu == nullptr ? m : kv_sequence_of(kc.cu, kc.batch, m, lane);
  if (b < 0) return;
  int len, row, rows;
  kc.sequence(b, len, row, rows);
  const int t = len - rows + (m - row);
  const int page = t < 0 ? -1 : kc.page_of(b, t >> 4);
  const uint8_t* tile = kc.pool;
  if (page >= 0)
    tile += int64_t(page) * kc.page_bytes + int64_t((t >> 4) & ((1 << kc.page_shift) - 1)) * kv_tile_bytes(FMT, D);
  const int64_t head_bytes = int64_t(kv_tile_bytes(FMT, D)) << kc.page_shift;
  const int units = (kc.heads + HPW - 1) / HPW;
  for (int u = wave; u < 2 * units; u += waves) {
    const bool is_k = u < units;
    const int h = (is_k ? u : u - units) * HPW + lane / LPH;
    if (h >= kc.heads) continue;
    v2f x = {0.f, 0.f};
    if (page >= 0) {
      const uint8_t* from = tile + h * head_bytes;
      const int ti = t & 15, g = 2 * sub / G;
      const uint32_t code = from[is_k ? kv_k_code<FMT, D>(ti, 2 * sub) : kv_v_code<FMT, D>(ti, 2 * sub)];
      const uint8_t* at = from + (is_k ? kv_k_scale<FMT, D>(ti, g) : kv_v_scale<FMT, D>(ti, g));
      x = kv_decode<FMT>(code, FMT == kFmtINT4 ? *reinterpret_cast<const uint16_t*>(at) : *at);
    }
    const int64_t at = int64_t(m) * (is_k ? ldk : ldv) + h * D + 2 * sub;
    if (f32)
      *reinterpret_cast<float2*>(static_cast<float*>(is_k ? K : V) + at) = make_float2(x.x, x.y);
    else
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(is_k ? K : V) + at) = cvt_bf2(x.x, x.y);
  }
}

// Pairs of pages, by value: the host's list is the caller's again when the call returns, and no copy of it has to
// reach the GPU first.
constexpr int kCopyPairs = 480;              // 3840 of a kernel's 4096 bytes of arguments
struct KvPairs {
  int32_t src[kCopyPairs], dst[kCopyPairs];
};

// A workgroup copies an even share, up to 16 KiB, of one page of one layer: four 16-byte loads a lane in flight.
constexpr int kCopyChunk = 16384;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__global__ void __launch_bounds__(256) kv_copy_kernel(uint8_t* pool, int64_t plane_bytes, int64_t page_bytes, KvPairs p) {
  uint8_t* plane = pool + blockIdx.z * plane_bytes;
  const u32x4* src = reinterpret_cast<const u32x4*>(plane + p.src[blockIdx.y] * page_bytes);
  u32x4* dst = reinterpret_cast<u32x4*>(plane + p.dst[blockIdx.y] * page_bytes);
  const int n = int(page_bytes / 16), share = (n + gridDim.x - 1) / gridDim.x;
  const int at = blockIdx.x * share + threadIdx.x, end = min(n, int(blockIdx.x + 1) * share);
  u32x4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (at + i * 256 < end) v[i] = __builtin_nontemporal_load(src + at + i * 256);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (at + i * 256 < end) __builtin_nontemporal_store(v[i], dst + at + i * 256);
}

struct KvCompact {
  const int32_t* to;
  const int32_t* start;
  const int32_t* keep;
  const int32_t* n_keep;
  int64_t ldto, ldkeep, plane_bytes;
  int32_t cols_to, most, parts;
  uint8_t* space;                  // of kThrough and kBack: tiles of the heads x0 .. x1 - 1 (of all layers), batch x tiles each
  int32_t x0, x1, tiles;
};

// What a wave moves of one tile: lane (token lane / 4, quarter lane % 4) of K, lane (4 tokens lane / 16, piece lane % 16)
// of V, lane (token lane % 16, groups lane / 16 + 4 j) of the scales.
template <int FMT, int D>
struct KvMoved {
  static constexpr int DW = D / 32, NG = D / kv_group(FMT), NS = (NG + 3) / 4;
  uint32_t k[DW], v[4], sk[NS], sv[NS];
};

// A wave fills a tile of the new places of one sequence: it finds where the tile's 16 tokens come from once, then
// gathers and writes the tile of every head and layer (of a part of them where there are few tiles), the next one's
// loads on their way before the stores.  With a tile of one head a wave the four dependent loads in front (count,
// index, page, bytes) cost as much as the bytes: 32 sequences' 20 tokens, 24 layers of 8 heads took 11.0 us, so 6.4.  18000
// of 60000 tokens, 8 heads, 4 layers, NVFP4 (179 MB) take 73 us: a kept token's lines hold others' bytes too, and twice
// the tokens' own are read.  In place a
// workgroup walks a sequence's tiles in order, four at a time, all loads of a head before its stores: the tokens that
// are kept come in rising order, so those of later tiles lie behind every place written so far.
enum { kApart = 0, kInPlace = 1, kInPlaceByWave = 2, kThrough = 3, kBack = 4 };
template <int FMT, int D, int HOW>
__global__ void __launch_bounds__(256) kv_compact_kernel(KvCache kc, KvCompact a) {
  using Moved = KvMoved<FMT, D>;
  constexpr int TB = kv_tile_bytes(FMT, D), DW = Moved::DW, NG = Moved::NG, NS = Moved::NS;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int TILES = HOW == kInPlaceByWave ? 1 : 4;        // of a sequence at once
  const int b = blockIdx.x / a.parts, part = (blockIdx.x % a.parts) * (4 / TILES) + (TILES == 1 ? wave : 0);
  const int step = a.parts * (4 / TILES);
  const int64_t head_bytes = int64_t(TB) << kc.page_shift;
  const int start = a.start == nullptr ? 0 : max(a.start[b], 0);
  const int n = min(max(a.n_keep[b], 0), a.most);
  if (n == 0) return;
  const int64_t end = int64_t(start) + n;
  const int mask = (1 << kc.page_shift) - 1, all = a.x1;
  for (int64_t at = int64_t(start / 16) + blockIdx.y * TILES; at * 16 < end; at += gridDim.y * TILES) {
    const int64_t tile = at + (TILES == 1 ? 0 : wave);
    // Token lane % 16 of the tile: where it comes from, as a tile's offset in the pool and a place in it.
    int64_t from = -1;
    int place = 0;
    const int64_t i = tile * 16 + (lane & 15) - start;
    if (i >= 0 && i < n) {
      const int old = a.keep[b * a.ldkeep + i];
      const int p = old < 0 ? -1 : kc.page_of(b, old >> 4);
      if (p >= 0) from = int64_t(p) * kc.page_bytes + int64_t((old >> 4) & mask) * TB;
      place = old & 15;
    }
    int64_t to = -1;
    if (tile * 16 < end && (tile >> kc.page_shift) < a.cols_to) {
      const int p = a.to[b * a.ldto + (tile >> kc.page_shift)];
      if (p >= 0 && p < kc.pages) to = int64_t(p) * kc.page_bytes + (tile & mask) * TB;
    }
    if (to < 0) from = -1;
    const int64_t spare = (int64_t(b) * a.tiles + (tile - start / 16)) * TB;
    if constexpr (HOW == kThrough) to = spare;
    if constexpr (HOW == kBack) {
      if (from >= 0) from = spare;
      place = lane & 15;
    }
    auto pool_of = [&](int x) { return kc.pool + (x / kc.heads) * a.plane_bytes + (x % kc.heads) * head_bytes; };
    auto space_of = [&](int x) { return a.space + int64_t(x - a.x0) * (int64_t(a.tiles) * TB) * (gridDim.x / a.parts); };
    // Offsets of the lane's pieces; -1: not moved.
    const int kt = lane >> 2;
    const int64_t kf = __shfl(from, kt);
    int64_t vf[4];
    const int kp = __shfl(place, kt) * (D / 2) + (lane & 3) * (D / 8);
    int vp[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      vf[j] = __shfl(from, (lane >> 4) * 4 + j);
      const int p = __shfl(place, (lane >> 4) * 4 + j);
      vp[j] = 8 * D + ((p >> 2) * 16 + (lane & 15)) * (D / 8) + (p & 3) * DW;
    }
    auto load = [&](int x, Moved& m) {
      if (x >= all) return;
      const uint8_t* base = HOW == kBack ? space_of(x) : pool_of(x);
      if (kf >= 0) {
        const uint32_t* s = reinterpret_cast<const uint32_t*>(base + kf + kp);
#pragma unroll
        for (int j = 0; j < DW; ++j) m.k[j] = s[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (vf[j] >= 0) {
          const uint8_t* s = base + vf[j] + vp[j];
          m.v[j] = DW >= 4 ? *reinterpret_cast<const uint32_t*>(s) : *reinterpret_cast<const uint16_t*>(s);
        }
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const int g = (lane >> 4) + 4 * j;
        if (from >= 0 && g < NG) {
          const uint8_t *y = base + from + kv_k_scale<FMT, D>(place, g), *z = base + from + kv_v_scale<FMT, D>(place, g);
          m.sk[j] = FMT == kFmtINT4 ? *reinterpret_cast<const uint16_t*>(y) : *y;
          m.sv[j] = FMT == kFmtINT4 ? *reinterpret_cast<const uint16_t*>(z) : *z;
        }
      }
    };
    auto store = [&](int x, const Moved& m) {
      uint8_t* base = (HOW == kThrough ? space_of(x) : pool_of(x)) + to;
      if (kf >= 0) {
        uint32_t* d = reinterpret_cast<uint32_t*>(base + kt * (D / 2) + (lane & 3) * (D / 8));
#pragma unroll
        for (int j = 0; j < DW; ++j) d[j] = m.k[j];
      }
      uint8_t* dv = base + 8 * D + lane * (D / 8);
      if (vf[0] >= 0 && vf[1] >= 0 && vf[2] >= 0 && vf[3] >= 0) {
        if constexpr (DW >= 4)
          *reinterpret_cast<uint4*>(dv) = make_uint4(m.v[0], m.v[1], m.v[2], m.v[3]);
        else
          *reinterpret_cast<uint2*>(dv) = make_uint2(m.v[0] | m.v[1] << 16, m.v[2] | m.v[3] << 16);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (vf[j] >= 0) {
            if constexpr (DW >= 4)
              *reinterpret_cast<uint32_t*>(dv + j * DW) = m.v[j];
            else
              *reinterpret_cast<uint16_t*>(dv + j * DW) = uint16_t(m.v[j]);
          }
      }
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const int g = (lane >> 4) + 4 * j;
        if (from >= 0 && g < NG) {
          uint8_t *y = base + kv_k_scale<FMT, D>(lane & 15, g), *z = base + kv_v_scale<FMT, D>(lane & 15, g);
          if constexpr (FMT == kFmtINT4) {
            *reinterpret_cast<uint16_t*>(y) = uint16_t(m.sk[j]);
            *reinterpret_cast<uint16_t*>(z) = uint16_t(m.sv[j]);
          } else {
            *y = uint8_t(m.sk[j]);
            *z = uint8_t(m.sv[j]);
          }
        }
      }
    };
    Moved now, next;
    load(a.x0 + part, now);
    for (int x = a.x0 + part; x < all; x += step) {
      load(x + step, next);
      if constexpr (HOW == kInPlace) __syncthreads();          // every wave has what it reads of x
      store(x, now);
      now = next;
    }
  }
}

template <template <int, int> class F, typename... A>
void by_format(int fmt, int D, A&&... args) {
  if (fmt == kFmtMXFP4)
    D == 64 ? F<kFmtMXFP4, 64>::run(args...) : F<kFmtMXFP4, 128>::run(args...);
  else if (fmt == kFmtINT4)
    D == 64 ? F<kFmtINT4, 64>::run(args...) : F<kFmtINT4, 128>::run(args...);
  else
    D == 64 ? F<kFmtNVFP4, 64>::run(args...) : F<kFmtNVFP4, 128>::run(args...);
}

constexpr int64_t kAppendWaves = 4096;       // waves of an append, if it has units for them

// Workgroups a row: one, or more where few rows leave CUs idle, each wave then taking fewer heads.
int row_parts(int64_t M, int units) {
  const int64_t want = 512 / (M > 0 ? M : 1), most = (units + 3) / 4;
  return int(want < 1 ? 1 : want < most ? want : most);
}

template <int FMT, int D>
struct Append {
  static void run(const KvCache& kc, const KvAppend& a, hipStream_t s) {
    const int hpw = 512 / D, units = 2 * ((kc.heads + hpw - 1) / hpw) + (a.q_heads + hpw - 1) / hpw;
    const int64_t fill = kAppendWaves / kc.M, parts = fill < 1 ? 1 : fill < units ? fill : units;
    kv_append_kernel<FMT, D><<<unsigned((kc.M * parts + 3) / 4), 256, 0, s>>>(kc, a, int(parts));
  }
};
template <int FMT, int D>
struct Read {
  static void run(const KvCache& kc, void* K, int64_t ldk, void* V, int64_t ldv, int f32, hipStream_t s) {
    const int hpw = 128 / D, units = 2 * ((kc.heads + hpw - 1) / hpw);
    kv_read_kernel<FMT, D><<<dim3(kc.M, row_parts(kc.M, units)), 256, 0, s>>>(kc, K, ldk, V, ldv, f32);
  }
};
constexpr int64_t kCompactGroups = 2048;    // workgroups of a compaction, if it has heads and layers for them

template <int FMT, int D, int HOW>
void compact(const KvCache& kc, KvCompact a, int64_t y, hipStream_t s) {
  const int64_t all = a.x1 - a.x0, most = HOW == kInPlaceByWave ? (all + 3) / 4 : all;
  const int64_t fill = kCompactGroups / (kc.batch * y);
  a.parts = int(fill < 1 ? 1 : fill < most ? fill : most);
  kv_compact_kernel<FMT, D, HOW><<<dim3(unsigned(kc.batch) * a.parts, unsigned(y)), 256, 0, s>>>(kc, a);
}
template <int FMT, int D>
struct Compact {
  static void run(const KvCache& kc, KvCompact a, bool in_place, hipStream_t s) {
    const int64_t tiles = kv_compact_tiles(a.most), y = tiles < 4 * 65535 ? (tiles + 3) / 4 : 65535;
    if (!in_place) return compact<FMT, D, kApart>(kc, a, y, s);
    if (a.most <= kKvCompactFew) return compact<FMT, D, kInPlaceByWave>(kc, a, 1, s);
    const int all = a.x1, slab = kv_compact_slab(FMT, D, kc.batch, all, a.most);
    if (slab == 0) return compact<FMT, D, kInPlace>(kc, a, 1, s);
    a.tiles = int(tiles);
    for (a.x0 = 0; a.x0 < all; a.x0 += slab) {
      a.x1 = a.x0 + slab < all ? a.x0 + slab : all;
      compact<FMT, D, kThrough>(kc, a, y, s);
      compact<FMT, D, kBack>(kc, a, y, s);
    }
  }
};

}  // namespace

hipError_t launch_kv_append(int fmt, int D, const KvCache& kc, const uint16_t* K, int64_t ldk, const uint16_t* V,
                            int64_t ldv, const uint16_t* Q, int64_t ldq, int q_heads, uint16_t* Q_out, int64_t ldqo,
                            const uint16_t* norm_q, const uint16_t* norm_k, float eps, const float* freq,
                            const int32_t* axis, int pairs, const int32_t* pos, int axes, bool halves, hipStream_t s) {
  const KvAppend a = {K, V, Q, Q_out, ldk, ldv, ldq, ldqo, norm_q, norm_k, eps, Q == nullptr ? 0 : q_heads,
                      {freq, axis, pos, pairs, axes, halves ? 1 : 0}};
  by_format<Append>(fmt, D, kc, a, s);
  return hipGetLastError();
}

hipError_t launch_kv_read(int fmt, int D, const KvCache& kc, void* K, int64_t ldk, void* V, int64_t ldv, bool f32,
                          hipStream_t s) {
  by_format<Read>(fmt, D, kc, K, ldk, V, ldv, f32 ? 1 : 0, s);
  return hipGetLastError();
}

hipError_t launch_kv_copy(uint8_t* pool, int planes, int64_t plane_bytes, int64_t page_bytes, const int32_t* src,
                          const int32_t* dst, int64_t n, hipStream_t s) {
  const unsigned x = unsigned((page_bytes + kCopyChunk - 1) / kCopyChunk);
  for (int64_t at = 0; at < n; at += kCopyPairs) {
    KvPairs p;
    const int k = int(n - at < kCopyPairs ? n - at : kCopyPairs);
    for (int i = 0; i < k; ++i) {
      p.src[i] = src[at + i];
      p.dst[i] = dst[at + i];
    }
    kv_copy_kernel<<<dim3(x, k, planes), 256, 0, s>>>(pool, plane_bytes, page_bytes, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_kv_compact(int fmt, int D, const KvCache& kc, int planes, int64_t plane_bytes, const int32_t* to,
                             int64_t ldto, int cols_to, const int32_t* start, const int32_t* keep, int64_t ldkeep,
                             const int32_t* n_keep, int most, bool in_place, void* space, hipStream_t s) {
  const KvCompact a = {to, start, keep, n_keep, ldto, ldkeep, plane_bytes, cols_to, most, 1, static_cast<uint8_t*>(space),
                       0, planes * kc.heads, 0};
  by_format<Compact>(fmt, D, kc, a, in_place, s);
  return hipGetLastError();
}

}  // namespace svdq
