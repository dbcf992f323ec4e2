// svdq_kv_append, svdq_kv_read, svdq_kv_copy and svdq_kv_compact: what fills a 4-bit key-value cache, reads it
// back and moves its pages and tokens.  Layout: kv.h.
#include "kv.h"

namespace svdq {

namespace {

// max of v over the W (8, 16, 32) lanes of an aligned group
template <int W>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int x = 1; x < W; x *= 2) v = fmaxf(v, __shfl_xor(v, x));
  return v;
}
template <int W, typename T>
__device__ __forceinline__ T group_sum(T v) {
#pragma unroll
  for (int x = 1; x < W; x *= 2) v += __shfl_xor(v, x);
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

// A lane's two neighbouring features turned.  Neighbours: they are a pair.  Halves: feature d pairs with d + pairs,
// which the lane pairs / 2 further on holds.
template <int LPH, typename T>
__device__ __forceinline__ void turn(T& a, T& b, const KvRope& r, int sub, bool turned, T c0, T s0, T c1, T s1) {
  if (!r.halves) {
    if (turned) {
      const T u = a * c0 - b * s0;
      b = a * s0 + b * c0;
      a = u;
    }
    return;
  }
  const bool second = 2 * sub >= r.pairs;
  const int from = second ? sub - r.pairs / 2 : sub + r.pairs / 2;
  const T a2 = __shfl(a, from, LPH), b2 = __shfl(b, from, LPH);
  if (turned) {
    a = second ? a2 * s0 + a * c0 : a * c0 - a2 * s0;
    b = second ? b2 * s1 + b * c1 : b * c1 - b2 * s1;
  }
}

// A workgroup takes a row m, its waves the row's heads in turn: K's, V's, Q's.  A lane holds two neighbouring
// features, so D / 2 lanes a head.  K's norm and rotation are in 64 bits, so that its codes, which are
// choices, do not hang on an order of summation or on a sine's last bit; the angle pos x freq is a 64-bit
// product, which holds far positions.  Q's are in 32 bits with the same sines.  Bound by memory for prompts
// (Q in and out is most of it), by the chain lengths -> table -> row -> store for single tokens.
template <int FMT, int D>
__global__ void __launch_bounds__(256) kv_append_kernel(KvCache kc, KvAppend a) {
  constexpr int LPH = D / 2, HPW = 64 / LPH, G = kv_group(FMT);
  const int lane = threadIdx.x & 63, sub = lane % LPH;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + blockIdx.y * 4, waves = gridDim.y * 4;
  const int m = blockIdx.x;
  const int b = kc.cu == nullptr ? m : kv_sequence_of(kc.cu, kc.batch, m, lane);
  if (b < 0) return;
  int len, row, rows;
  kc.sequence(b, len, row, rows);
  const int t = len - rows + (m - row);                        // the row's place
  const int page = t < 0 ? -1 : kc.page_of(b, t >> 4);
  uint8_t* tile = nullptr;
  if (page >= 0)
    tile = kc.pool + int64_t(page) * kc.page_bytes +
           int64_t((t >> 4) & ((1 << kc.page_shift) - 1)) * kv_tile_bytes(FMT, D);
  const int64_t head_bytes = int64_t(kv_tile_bytes(FMT, D)) << kc.page_shift;

  double c0 = 1, s0 = 0, c1 = 1, s1 = 0;
  bool turned = false;
  const KvRope& r = a.rope;
  if (r.pairs > 0) {
    const int p0 = r.halves ? (2 * sub) % r.pairs : sub, p1 = r.halves ? (2 * sub + 1) % r.pairs : sub;
    turned = 2 * sub < 2 * r.pairs;
    if (turned) {
      auto angle = [&](int p) {
#pragma clang fp contract(off)
        const int ax = r.axis == nullptr ? 0 : r.axis[p];
        int pos = t;
        if (r.pos != nullptr) pos = ax >= 0 && ax < r.axes ? r.pos[int64_t(ax) * kc.M + m] : 0;
        return double(pos) * double(r.freq[p]);
      };
      sincos(angle(p0), &s0, &c0);
      if (r.halves) sincos(angle(p1), &s1, &c1);
    }
  }

  const int kv_units = (kc.heads + HPW - 1) / HPW, q_units = (a.q_heads + HPW - 1) / HPW;
  for (int u = wave; u < 2 * kv_units + q_units; u += waves) {
    const bool is_k = u < kv_units, is_q = u >= 2 * kv_units;
    const int heads = is_q ? a.q_heads : kc.heads;
    const int h = (is_q ? u - 2 * kv_units : is_k ? u : u - kv_units) * HPW + lane / LPH;
    const bool there = h < heads;
    const uint16_t* src = is_q ? a.Q + int64_t(m) * a.ldq : is_k ? a.K + int64_t(m) * a.ldk : a.V + int64_t(m) * a.ldv;
    const uint32_t in = there ? *reinterpret_cast<const uint32_t*>(src + h * D + 2 * sub) : 0;
    if (is_q) {
      float x = bf_lo(in), y = bf_hi(in);
      if (a.norm_q != nullptr) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(a.norm_q + 2 * sub);
        const float k = 1.0f / sqrtf(group_sum<LPH>(x * x + y * y) / D + a.eps);
        x = x * k * bf_lo(w);
        y = y * k * bf_hi(w);
      }
      turn<LPH, float>(x, y, r, sub, turned, float(c0), float(s0), float(c1), float(s1));
      if (there) *reinterpret_cast<uint32_t*>(a.Q_out + int64_t(m) * a.ldqo + h * D + 2 * sub) = cvt_bf2(x, y);
      continue;
    }
    float x = bf_lo(in), y = bf_hi(in);
    if (is_k) {
      double z = x, v = y;
      if (a.norm_k != nullptr) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(a.norm_k + 2 * sub);
        const double k = sqrt(group_sum<LPH>(z * z + v * v) / D + double(a.eps));
        z = z / k * bf_lo(w);
        v = v / k * bf_hi(w);
      }
      turn<LPH, double>(z, v, r, sub, turned, c0, s0, c1, s1);
      x = float(z);
      y = float(v);
    }
    x = kv_finite_bf16(x);
    y = kv_finite_bf16(y);
    float div;
    const uint32_t s = kv_scale<FMT>(group_max<G / 2>(fmaxf(fabsf(x), fabsf(y))), div);
    const uint32_t code = kv_encode<FMT>(x, y, div);
    if (!there || page < 0) continue;
    uint8_t* to = tile + h * head_bytes;
    const int ti = t & 15, g = 2 * sub / G;
    to[is_k ? kv_k_code<FMT, D>(ti, 2 * sub) : kv_v_code<FMT, D>(ti, 2 * sub)] = uint8_t(code);
    if (sub % (G / 2) == 0) {
      uint8_t* at = to + (is_k ? kv_k_scale<FMT, D>(ti, g) : kv_v_scale<FMT, D>(ti, g));
      if constexpr (FMT == kFmtINT4)
        *reinterpret_cast<uint16_t*>(at) = uint16_t(s);
      else
        *at = uint8_t(s);
    }
  }
}

// A workgroup takes a row, a wave heads of K or V of it; a row without a place reads as zeros.
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
constexpr int kCopyPairs = 256;
struct KvPairs {
  int32_t src[kCopyPairs], dst[kCopyPairs];
};

// A workgroup copies 16 KiB of one page of one layer: four 16-byte loads a lane in flight.
constexpr int kCopyChunk = 16384;
__global__ void __launch_bounds__(256) kv_copy_kernel(uint8_t* pool, int64_t plane_bytes, int64_t page_bytes, KvPairs p) {
  uint8_t* plane = pool + blockIdx.z * plane_bytes;
  const uint4* src = reinterpret_cast<const uint4*>(plane + p.src[blockIdx.y] * page_bytes);
  uint4* dst = reinterpret_cast<uint4*>(plane + p.dst[blockIdx.y] * page_bytes);
  const int64_t n = page_bytes / 16, at = int64_t(blockIdx.x) * (kCopyChunk / 16) + threadIdx.x;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (at + i * 256 < n) v[i] = src[at + i * 256];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (at + i * 256 < n) dst[at + i * 256] = v[i];
}

struct KvCompact {
  const int32_t* to;
  const int32_t* start;
  const int32_t* keep;
  const int32_t* n_keep;
  int64_t ldto, ldkeep, plane_bytes;
  int32_t cols_to, most;
};

// A wave fills a tile of the new places of one sequence, head and layer: it gathers the tile's 16 tokens and
// writes whole pieces.  In place a workgroup walks a sequence's tiles in order, four at a time, all loads
// before the stores: the tokens that are kept come in rising order, so those of later tiles lie behind
// every place written so far.
template <int FMT, int D, bool IN_PLACE>
__global__ void __launch_bounds__(256) kv_compact_kernel(KvCache kc, KvCompact a) {
  constexpr int TB = kv_tile_bytes(FMT, D), DW = D / 32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x / kc.heads, h = blockIdx.x % kc.heads;
  uint8_t* pool = kc.pool + blockIdx.z * a.plane_bytes + (int64_t(TB) << kc.page_shift) * h;
  const int start = a.start == nullptr ? 0 : max(a.start[b], 0);
  const int n = min(max(a.n_keep[b], 0), a.most);
  if (n == 0) return;
  const int64_t end = int64_t(start) + n;
  const int mask = (1 << kc.page_shift) - 1;
  for (int64_t at = int64_t(start / 16) + blockIdx.y * 4; at * 16 < end; at += gridDim.y * 4) {
    const int64_t tile = at + wave;
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
    uint8_t* to = nullptr;
    if (tile * 16 < end && (tile >> kc.page_shift) < a.cols_to) {
      const int p = a.to[b * a.ldto + (tile >> kc.page_shift)];
      if (p >= 0 && p < kc.pages) to = pool + int64_t(p) * kc.page_bytes + (tile & mask) * TB;
    }
    if (to == nullptr) from = -1;
    // K: lane (token lane / 4, quarter lane % 4).  V: lane (4 tokens lane / 16, piece lane % 16).  Scales one by
    // one: lane (token lane % 16, groups lane / 16 + 4 j).
    uint32_t k[DW], v[4];
    const int kt = lane >> 2;
    const int64_t kf = __shfl(from, kt);
    const int kp = __shfl(place, kt);
    if (kf >= 0) {
      const uint32_t* s = reinterpret_cast<const uint32_t*>(pool + kf + kp * (D / 2) + (lane & 3) * (D / 8));
#pragma unroll
      for (int j = 0; j < DW; ++j) k[j] = s[j];
    }
    int64_t vf[4];
    int vp[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      vf[j] = __shfl(from, (lane >> 4) * 4 + j);
      vp[j] = __shfl(place, (lane >> 4) * 4 + j);
      if (vf[j] >= 0) {
        const uint8_t* s = pool + vf[j] + 8 * D + ((vp[j] >> 2) * 16 + (lane & 15)) * (D / 8) + (vp[j] & 3) * DW;
        if constexpr (DW >= 4)
          v[j] = *reinterpret_cast<const uint32_t*>(s);
        else
          v[j] = *reinterpret_cast<const uint16_t*>(s);
      }
    }
    constexpr int NG = D / kv_group(FMT);
    uint32_t sk[(NG + 3) / 4], sv[(NG + 3) / 4];
    const int64_t sf = from;                                  // of token lane % 16
#pragma unroll
    for (int j = 0; j < (NG + 3) / 4; ++j) {
      const int g = (lane >> 4) + 4 * j;
      if (sf >= 0 && g < NG) {
        const uint8_t *x = pool + sf + kv_k_scale<FMT, D>(place, g), *y = pool + sf + kv_v_scale<FMT, D>(place, g);
        sk[j] = FMT == kFmtINT4 ? *reinterpret_cast<const uint16_t*>(x) : *x;
        sv[j] = FMT == kFmtINT4 ? *reinterpret_cast<const uint16_t*>(y) : *y;
      }
    }
    if constexpr (IN_PLACE) __syncthreads();
    if (kf >= 0) {
      uint32_t* d = reinterpret_cast<uint32_t*>(to + kt * (D / 2) + (lane & 3) * (D / 8));
#pragma unroll
      for (int j = 0; j < DW; ++j) d[j] = k[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (vf[j] >= 0) {
        uint8_t* d = to + 8 * D + lane * (D / 8) + j * DW;
        if constexpr (DW >= 4)
          *reinterpret_cast<uint32_t*>(d) = v[j];
        else
          *reinterpret_cast<uint16_t*>(d) = uint16_t(v[j]);
      }
#pragma unroll
    for (int j = 0; j < (NG + 3) / 4; ++j) {
      const int g = (lane >> 4) + 4 * j;
      if (sf >= 0 && g < NG) {
        uint8_t *x = to + kv_k_scale<FMT, D>(lane & 15, g), *y = to + kv_v_scale<FMT, D>(lane & 15, g);
        if constexpr (FMT == kFmtINT4) {
          *reinterpret_cast<uint16_t*>(x) = uint16_t(sk[j]);
          *reinterpret_cast<uint16_t*>(y) = uint16_t(sv[j]);
        } else {
          *x = uint8_t(sk[j]);
          *y = uint8_t(sv[j]);
        }
      }
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

// Workgroups a row: one, or more where few rows leave CUs idle, each wave then taking fewer heads.
int row_parts(int64_t M, int units) {
  const int64_t want = 512 / (M > 0 ? M : 1), most = (units + 3) / 4;
  return int(want < 1 ? 1 : want < most ? want : most);
}

template <int FMT, int D>
struct Append {
  static void run(const KvCache& kc, const KvAppend& a, hipStream_t s) {
    const int hpw = 128 / D, units = 2 * ((kc.heads + hpw - 1) / hpw) + (a.q_heads + hpw - 1) / hpw;
    kv_append_kernel<FMT, D><<<dim3(kc.M, row_parts(kc.M, units)), 256, 0, s>>>(kc, a);
  }
};
template <int FMT, int D>
struct Read {
  static void run(const KvCache& kc, void* K, int64_t ldk, void* V, int64_t ldv, int f32, hipStream_t s) {
    const int hpw = 128 / D, units = 2 * ((kc.heads + hpw - 1) / hpw);
    kv_read_kernel<FMT, D><<<dim3(kc.M, row_parts(kc.M, units)), 256, 0, s>>>(kc, K, ldk, V, ldv, f32);
  }
};
template <int FMT, int D>
struct Compact {
  static void run(const KvCache& kc, const KvCompact& a, int planes, bool in_place, hipStream_t s) {
    const int x = kc.batch * kc.heads;
    if (in_place) {
      kv_compact_kernel<FMT, D, true><<<dim3(x, 1, planes), 256, 0, s>>>(kc, a);
    } else {
      const int64_t tiles = a.most / 16 + 2, y = (tiles + 3) / 4;
      kv_compact_kernel<FMT, D, false><<<dim3(x, unsigned(y < 65535 ? y : 65535), planes), 256, 0, s>>>(kc, a);
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
                             const int32_t* n_keep, int most, bool in_place, hipStream_t s) {
  const KvCompact a = {to, start, keep, n_keep, ldto, ldkeep, plane_bytes, cols_to, most};
  by_format<Compact>(fmt, D, kc, a, planes, in_place, s);
  return hipGetLastError();
}

}  // namespace svdq
