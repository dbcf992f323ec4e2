// 4-bit weight fragments against 16-bit activations on the bf16 MFMA, shared by
// the few-token kernels (w4a16.hip, moe.hip).
//
// A lane holds 16 bytes of codes of one weight row per 16-row tile and 128-K step
// (layout.h).  Dword u of them is 8 codes, the A operand of one 16x16x32 MFMA;
// lane group c = lane / 16 then covers the K elements k_of(c, u) .. + 7 of the
// step, so the B operand holds the same elements of an activation row.
//
// Every code becomes a bf16 exactly, so a product of a code and a bf16 is exact in
// fp32 and only the sums round:
//   MXFP4  E2M1 times its power of two (the gfx950 convert applies the scale);
//   NVFP4  E2M1 times E4M3: 2 + 4 significant bits, in bf16's 8; the tensor scale
//          multiplies the sum;
//   INT4   24 + q (q + 8 in mantissa bits 3..6 of 16), with 24 times the group's sum
//          of the activations taken off by the same MFMA against -24; the fp16 scale
//          multiplies each 64-group's sum.  (16 is the smallest power of two whose
//          bf16 mantissa has room for the nibble; against 128 + q + 8 the sums that
//          cancel are 136 / 24 times smaller, and so is their rounding.)
// An fp32 activation is the sum of S bf16 planes, each the nearest bf16 of what the
// ones before leave: S = 2 leaves at most 2^-18 of it, S = 3 at most 2^-27 (the
// planes' exponents permitting), below fp32's own rounding.
#pragma once
#include <type_traits>

#include "common.h"

namespace svdq {

// First of the 8 consecutive K elements, within a 128-K step, that lane group c
// multiplies in the step's MFMA u.
template <int FMT>
__device__ __forceinline__ int k_of(int c, int u) {
  return FMT == kFmtINT4 ? (u >> 1) * 64 + c * 16 + (u & 1) * 8 : c * 32 + u * 8;
}

// Where those elements lie in a step stored in the order of the operands: MFMA u's four lane
// groups one after the other, so that a row's piece of one operand is 64 bytes at a stretch.  (At
// k_of it is four pieces of 16 bytes, and the address unit takes a cycle for each.)
template <int FMT>
__device__ __forceinline__ int stored_at(int kk) {           // kk: an element of the step; 8 go together
  const int c = FMT == kFmtINT4 ? (kk & 63) >> 4 : kk >> 5;
  const int u = FMT == kFmtINT4 ? ((kk >> 6) << 1) + ((kk >> 3) & 1) : (kk >> 3) & 3;
  return u * 32 + c * 8 + (kk & 7);
}

// Codes and scales of one 16-row tile and 128-K step, as one lane holds them.
template <int FMT>
struct W4Stage {
  uint4 q;
  typename std::conditional<FMT == kFmtINT4, uint4, uint32_t>::type s;
};

__device__ __forceinline__ uint4 buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  const v4i v = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
  return make_uint4(uint32_t(v[0]), uint32_t(v[1]), uint32_t(v[2]), uint32_t(v[3]));
}

// A packed weight's codes and scales as buffers.  A step that is not there (valid false) loads
// zeros through a buffer of no bytes: the load is issued all the same, so that the wait counts
// of a software pipeline stay exact, and reads no memory.
template <int FMT>
struct W4Rows {
  const uint8_t* codes;
  const uint8_t* scales;
  uint32_t code_bytes, scale_bytes, KS, s_step;
  __device__ __forceinline__ W4Rows(const uint8_t* c, const uint8_t* s, int K, int64_t N_pad)
      : codes(c), scales(s), code_bytes(uint32_t(N_pad * K / 2)),
        scale_bytes(uint32_t(N_pad * K / (FMT == kFmtNVFP4 ? 16 : 32))), KS(uint32_t(K / kKStep)),
        s_step(uint32_t(N_pad) * 4) {}
  // T tiles from rt on.  A tile's distance is in the lane's offset, so all share scalar operands.
  template <int T>
  __device__ __forceinline__ void load(uint32_t rt, uint32_t ks, bool valid, int lane, W4Stage<FMT> (&st)[T]) const {
    const __amdgpu_buffer_rsrc_t rc = make_rsrc(codes, valid ? code_bytes : 0);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(scales, valid ? scale_bytes : 0);
#pragma unroll
    for (uint32_t t = 0; t < T; ++t) {
      st[t].q = buffer_load16(rc, uint32_t(lane) * 16 + t * KS * 1024, (rt * KS + ks) * 1024);
      if constexpr (FMT == kFmtMXFP4)
        st[t].s = uint32_t(__builtin_amdgcn_raw_buffer_load_b32(rs, uint32_t(lane) * 4 + t * KS * 64,
                                                                (rt * KS + (ks & ~3u)) * 64, 0));
      if constexpr (FMT == kFmtNVFP4)
        st[t].s = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(rs, uint32_t(lane) * 2 + t * KS * 128,
                                                                (rt * KS + ks) * 128, 0));
      if constexpr (FMT == kFmtINT4)               // rows 4 c .. 4 c + 3 of the tile
        st[t].s = buffer_load16(rs, uint32_t(lane >> 4) * 16 + t * 64, ks * s_step + rt * 64);
    }
  }
  __device__ __forceinline__ void load(uint32_t rt, uint32_t ks, bool valid, int lane, W4Stage<FMT>& st) const {
    W4Stage<FMT> one[1];
    load<1>(rt, ks, valid, lane, one);
    st = one[0];
  }
};

// Keeps the loads before it ahead of those after it: a wait for the oldest of a pipeline's loads
// must not become a wait for all of them.
__device__ __forceinline__ void keep_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Workgroup barrier for data in LDS: waits for this wave's LDS operations and not, as a fence
// would, for its global loads in flight; the empty asm keeps memory accesses from moving across.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0); vmcnt and expcnt at their maxima
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ float f16_value(uint32_t bits) {
  return float(__builtin_bit_cast(_Float16, uint16_t(bits)));
}

// 8 E2M1 codes times a power of two -> 8 bf16.
__device__ __forceinline__ uint4 mx_to_bf16(uint32_t d, float scale) {
  return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3)));
}

// 8 E2M1 codes times an E4M3 value -> 8 bf16.
__device__ __forceinline__ uint4 nv_to_bf16(uint32_t d, float s) {
  const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 0);
  const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 1);
  const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 2);
  const v2f e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 3);
  return make_uint4(cvt_bf2(a.x * s, a.y * s), cvt_bf2(b.x * s, b.y * s), cvt_bf2(c.x * s, c.y * s),
                    cvt_bf2(e.x * s, e.y * s));
}

// The same in fp16, where it is exact too (2^-10 .. 2688) and a product is one packed multiply: half
// the operations, for activations that are fp16.  s holds the value twice.
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint4 nv_to_f16(uint32_t d, v2h s) {
  return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 0) * s),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 1) * s),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 2) * s),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 3) * s));
}

// fp16 activations of a row: the row times the power of two 2^f16_row_power that brings its largest
// magnitude `top` into [2^14, 2^15) (1 for zero, infinity and NaN).  A bf16 is then exact in fp16 down
// to 2^-28 of the row's largest, and off by at most 2^-39 of it below; hi + lo hold an fp32 to 2^-22.
// The power (-113 .. 147) is applied by ldexp: as a factor it would not fit fp32 for the smallest rows.
__device__ __forceinline__ int f16_row_power(float top) {
  return top > 0.f && top < __builtin_huge_valf() ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
}
__device__ __forceinline__ uint4 to_f16(const float (&v)[8]) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __builtin_bit_cast(uint32_t, v2h{static_cast<_Float16>(v[2 * i]), static_cast<_Float16>(v[2 * i + 1])});
  return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void unpack_h8(const uint4& r, float (&a)[8]) {
  const uint32_t d[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const v2h h = __builtin_bit_cast(v2h, d[i]);
    a[2 * i] = float(h.x);
    a[2 * i + 1] = float(h.y);
  }
}

// 8 INT4 codes in the packed dword order -> 8 bf16 24 + q.  k41 holds 0x41 in every byte
// (the high byte of bf16 16 .. 31).
__device__ __forceinline__ uint4 i4_to_bf16(uint32_t d, uint32_t k41) {
  d ^= 0x88888888u;                                         // nibbles q + 8
  const uint32_t lo = ((d << 3) & 0x78787878u) | 0x80808080u;   // codes 0..3: low bytes of 16 + (q + 8)
  const uint32_t hi = ((d >> 1) & 0x78787878u) | 0x80808080u;   // codes 4..7
  return make_uint4(__builtin_amdgcn_perm(k41, lo, 0x04010400u), __builtin_amdgcn_perm(k41, lo, 0x04030402u),
                    __builtin_amdgcn_perm(k41, hi, 0x04010400u), __builtin_amdgcn_perm(k41, hi, 0x04030402u));
}

// acc[t][b] += (rows of tile t) x (16 columns of block b) over MFMA u of a 128-K step (MXFP4,
// NVFP4); x[b] is the B operand.
template <int FMT, int T, int NB, bool F16 = false>
__device__ __forceinline__ void w4_mfma(const W4Stage<FMT> (&st)[T], int ks, int u, const uint4 (&x)[NB],
                                        v4f (&acc)[T][NB]) {
  static_assert(FMT != kFmtINT4, "INT4 takes half a step");
  static_assert(!F16 || FMT == kFmtNVFP4, "fp16 activations: NVFP4 weights");
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const uint32_t d[4] = {st[t].q.x, st[t].q.y, st[t].q.z, st[t].q.w};
    uint4 a;
    if constexpr (FMT == kFmtMXFP4)
      a = mx_to_bf16(d[u], __uint_as_float(((st[t].s >> ((ks & 3) * 8)) & 0xFFu) << 23));
    else if constexpr (F16) {
      const _Float16 s = static_cast<_Float16>(e4m3_value((st[t].s >> ((u >> 1) * 8)) & 0xFFu));
      a = nv_to_f16(d[u], v2h{s, s});
    } else
      a = nv_to_bf16(d[u], e4m3_value((st[t].s >> ((u >> 1) * 8)) & 0xFFu));
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[t][b] = F16 ? mfma_f16(a, x[b], acc[t][b]) : mfma_bf16(a, x[b], acc[t][b]);
  }
}

// The same over half `half` of a step (MFMAs 2 half and 2 half + 1) for INT4, a scale group;
// x[u][b] is the B operand of MFMA 2 half + u.
template <int T, int NB>
__device__ __forceinline__ void w4_half(const W4Stage<kFmtINT4> (&st)[T], int half, const uint4 (&x)[2][NB],
                                        v4f (&acc)[T][NB]) {
  const uint4 m24 = make_uint4(0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u);   // bf16 -24
  uint32_t k41 = 0x41414141u;
  asm volatile("" : "+v"(k41));                             // kept in a register for the byte permutes
  uint4 a[T][2];
  float s[T][4];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const uint32_t d[4] = {st[t].q.x, st[t].q.y, st[t].q.z, st[t].q.w};
    const uint32_t sd[4] = {st[t].s.x, st[t].s.y, st[t].s.z, st[t].s.w};
#pragma unroll
    for (int u = 0; u < 2; ++u) a[t][u] = i4_to_bf16(d[2 * half + u], k41);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[t][e] = f16_value(half == 0 ? sd[e] : sd[e] >> 16);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    v4f off = {0.f, 0.f, 0.f, 0.f};                         // -24 times the group's sum, for all tiles
    off = mfma_bf16(m24, x[0][b], off);
    off = mfma_bf16(m24, x[1][b], off);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      v4f p = mfma_bf16(a[t][0], x[0][b], off);
      p = mfma_bf16(a[t][1], x[1][b], p);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][b][e] = fmaf(s[t][e], p[e], acc[t][b][e]);
    }
  }
}

// A whole 128-K step of one tile; x[u] is the B operand of MFMA u.
template <int FMT, bool F16 = false>
__device__ __forceinline__ void w4_step(const W4Stage<FMT>& st, int ks, const uint4 (&x)[4], v4f& acc) {
  const W4Stage<FMT> one[1] = {st};
  v4f a[1][1] = {{acc}};
  if constexpr (FMT == kFmtINT4) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint4 h[2][1] = {{x[2 * half]}, {x[2 * half + 1]}};
      w4_half<1, 1>(one, half, h, a);
    }
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint4 h[1] = {x[u]};
      w4_mfma<FMT, 1, 1, F16>(one, ks, u, h, a);
    }
  }
  acc = a[0][0];
}

// The factor that the sums of a packed weight still lack: NVFP4's tensor scale
// fp32(max|R| / 2688), else 1.
template <int FMT>
__device__ __forceinline__ float w4_tensor_scale(const uint8_t* amax) {
  return FMT == kFmtNVFP4 ? *reinterpret_cast<const float*>(amax) / kNvfp4GlobalDiv : 1.0f;
}

// 8 fp32 -> S bf16 planes (each one MFMA operand of 8 elements).
template <int S>
__device__ __forceinline__ void split_planes(float (&v)[8], uint4 (&p)[S]) {
#pragma unroll
  for (int i = 0; i < S; ++i) {
    p[i] = make_uint4(cvt_bf2(v[0], v[1]), cvt_bf2(v[2], v[3]), cvt_bf2(v[4], v[5]), cvt_bf2(v[6], v[7]));
    if (i + 1 < S) {
      float h[8];
      unpack_bf8(p[i], h);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] -= h[e];             // exact
    }
  }
}

// Columns of one MFMA for tokens with S planes: plane p of token t is column p (16 / S) + t.
constexpr int tokens_per_block(int S) { return 16 / S; }

}  // namespace svdq
