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
  __device__ __forceinline__ void load(uint32_t rt, uint32_t ks, bool valid, int lane, W4Stage<FMT>& st) const {
    const __amdgpu_buffer_rsrc_t rc = make_rsrc(codes, valid ? code_bytes : 0);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(scales, valid ? scale_bytes : 0);
    st.q = buffer_load16(rc, uint32_t(lane) * 16, (rt * KS + ks) * 1024);
    if constexpr (FMT == kFmtMXFP4)
      st.s = uint32_t(__builtin_amdgcn_raw_buffer_load_b32(rs, uint32_t(lane) * 4, (rt * (KS / 4) + ks / 4) * 256, 0));
    if constexpr (FMT == kFmtNVFP4)
      st.s = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(rs, uint32_t(lane) * 2, (rt * KS + ks) * 128, 0));
    if constexpr (FMT == kFmtINT4) st.s = buffer_load16(rs, uint32_t(lane >> 4) * 16, ks * s_step + rt * 64);  // rows 4 c ..
  }
};

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

// 8 INT4 codes in the packed dword order -> 8 bf16 24 + q.  k41 holds 0x41 in every byte
// (the high byte of bf16 16 .. 31).
__device__ __forceinline__ uint4 i4_to_bf16(uint32_t d, uint32_t k41) {
  d ^= 0x88888888u;                                         // nibbles q + 8
  const uint32_t lo = ((d << 3) & 0x78787878u) | 0x80808080u;   // codes 0..3: low bytes of 16 + (q + 8)
  const uint32_t hi = ((d >> 1) & 0x78787878u) | 0x80808080u;   // codes 4..7
  return make_uint4(__builtin_amdgcn_perm(k41, lo, 0x04010400u), __builtin_amdgcn_perm(k41, lo, 0x04030402u),
                    __builtin_amdgcn_perm(k41, hi, 0x04010400u), __builtin_amdgcn_perm(k41, hi, 0x04030402u));
}

// acc[b] += (tile's 16 rows) x (16 columns of x[b]) over one 128-K step, for NB blocks
// of columns; x[b][u] is the B operand of MFMA u.
template <int FMT, int NB>
__device__ __forceinline__ void w4_step(const W4Stage<FMT>& st, int ks, const uint4 (&x)[NB][4], v4f (&acc)[NB]) {
  const uint32_t d[4] = {st.q.x, st.q.y, st.q.z, st.q.w};
  if constexpr (FMT == kFmtMXFP4) {
    const float sc = __uint_as_float(((st.s >> ((ks & 3) * 8)) & 0xFFu) << 23);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint4 a = mx_to_bf16(d[u], sc);
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[b] = mfma_bf16(a, x[b][u], acc[b]);
    }
  } else if constexpr (FMT == kFmtNVFP4) {
    const float sc[2] = {e4m3_value(st.s & 0xFFu), e4m3_value((st.s >> 8) & 0xFFu)};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint4 a = nv_to_bf16(d[u], sc[u >> 1]);
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[b] = mfma_bf16(a, x[b][u], acc[b]);
    }
  } else {
    const uint4 m24 = make_uint4(0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u);   // bf16 -24
    uint32_t k41 = 0x41414141u;
    asm volatile("" : "+v"(k41));                           // kept in a register for the byte permutes
    const uint32_t sd[4] = {st.s.x, st.s.y, st.s.z, st.s.w};
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint4 a0 = i4_to_bf16(d[2 * g], k41), a1 = i4_to_bf16(d[2 * g + 1], k41);
      float s[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = f16_value(g == 0 ? sd[e] : sd[e] >> 16);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        v4f p = {0.f, 0.f, 0.f, 0.f};
        p = mfma_bf16(a0, x[b][2 * g], p);
        p = mfma_bf16(a1, x[b][2 * g + 1], p);
        p = mfma_bf16(m24, x[b][2 * g], p);
        p = mfma_bf16(m24, x[b][2 * g + 1], p);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[b][e] = fmaf(s[e], p[e], acc[b][e]);
      }
    }
  }
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
