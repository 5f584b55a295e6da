// hqq_codes.h -- device decode of the stored code bitstream to binary16 weights, shared by
// the product kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hqq_internal.h"

namespace hqq {
namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float h2f(uint32_t h) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

// Code j (0-based, compile-time after unrolling) of an LSB-first string held in words w.
template <int NB, int NW>
__device__ __forceinline__ uint32_t code_at(const uint32_t (&w)[NW], int j) {
  const int bit = NB * j;
  const int wi = bit >> 5, sh = bit & 31;
  constexpr uint32_t mask = (1u << NB) - 1u;
  if (sh + NB <= 32) return (w[wi] >> sh) & mask;
  return __builtin_amdgcn_alignbit(w[wi + 1], w[wi], sh) & mask;
}

// The 32 codes (32*NB bits, NB words) starting at p (4*NB-byte aligned).
template <int NB>
__device__ __forceinline__ void load_codes32(const uint8_t* p, uint32_t (&w)[NB]) {
  if constexpr (NB == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else if constexpr (NB == 3) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
    w[0] = q[0]; w[1] = q[1]; w[2] = q[2];
  } else if constexpr (NB == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0];
    const uint4 b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}

// Packed-binary16 form of the codes for the dot products: every 32-bit word is a
// pair of consecutive codes as exact binary16 integers.  A byte of codes is placed
// beside the binary16 exponent byte 0x64 (1024 + mantissa) with one byte permute, the
// other code fields of the byte are masked off, and one packed FMA scales and shifts
// each half to the code itself (1024 + 16 c -> c: exact in binary16).
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ half2_t as_h2(uint32_t u) { return __builtin_bit_cast(half2_t, u); }

template <int NB>
struct CodePairs {  // the 16 codes of one 16-code block as 8 pairs
  static constexpr int kWords = 16 * NB / 32;
  half2_t q[8];
  __device__ __forceinline__ void from(const uint32_t (&w)[kWords]) {
    constexpr uint32_t kMagic = 0x64646464u;
    if constexpr (NB == 8) {  // one code per byte: bytes 2i, 2i+1
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t sel = 0x04000400u | (uint32_t)((2 * i) & 3) | ((uint32_t)((2 * i + 1) & 3) << 16);
        const uint32_t t = __builtin_amdgcn_perm(kMagic, w[i / 2], sel);
        q[i] = as_h2(t) - (half2_t){(_Float16)1024.f, (_Float16)1024.f};
      }
    } else if constexpr (NB == 4) {  // two codes per byte
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = (uint32_t)(i & 3);
        const uint32_t t = __builtin_amdgcn_perm(kMagic, w[i / 4], 0x04000400u | b | (b << 16)) &
                           0xFFF0FF0Fu;
        q[i] = __builtin_elementwise_fma(as_h2(t), (half2_t){(_Float16)1.f, (_Float16)0.0625f},
                                         (half2_t){(_Float16)-1024.f, (_Float16)-64.f});
      }
    } else {  // NB == 2: four codes per byte
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = (uint32_t)i;
        const uint32_t t = __builtin_amdgcn_perm(kMagic, w[0], 0x04000400u | b | (b << 16));
        q[2 * i] = __builtin_elementwise_fma(as_h2(t & 0xFF0CFF03u),
                                             (half2_t){(_Float16)1.f, (_Float16)0.25f},
                                             (half2_t){(_Float16)-1024.f, (_Float16)-256.f});
        q[2 * i + 1] = __builtin_elementwise_fma(as_h2(t & 0xFFC0FF30u),
                                                 (half2_t){(_Float16)0.0625f, (_Float16)0.015625f},
                                                 (half2_t){(_Float16)-64.f, (_Float16)-16.f});
      }
    }
  }
};

typedef float float2_t __attribute__((ext_vector_type(2)));

// Dequantize 32 codes of one weight row to binary16: w = s*q - s*z in fp32 (s*z exact,
// one rounding) rounded to binary16 (v_cvt_pk_f16_f32, nearest even).  s0, sz0 for
// codes 0..15 and s1, sz1 for 16..31 (different groups only when g = 16).
template <int NB>
__device__ __forceinline__ void dequant32(const uint32_t (&w)[NB], float s0, float sz0, float s1,
                                          float sz1, uint4 (&out)[4]) {
  uint32_t h[16];
  if constexpr (NB == 3) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float s = j < 8 ? s0 : s1;
      const float sz = j < 8 ? sz0 : sz1;
      const float w0 = __builtin_fmaf(s, (float)code_at<NB>(w, 2 * j), -sz);
      const float w1 = __builtin_fmaf(s, (float)code_at<NB>(w, 2 * j + 1), -sz);
      h[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t){w0, w1}, half2_t));
    }
  } else {  // the codes as exact binary16 pairs, converted inside the fp32 FMA (v_fma_mix_f32)
    constexpr int HW = NB / 2;  // words per 16 codes
    CodePairs<NB> cp[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      uint32_t ws[HW];
#pragma unroll
      for (int i = 0; i < HW; ++i) ws[i] = w[hh * HW + i];
      cp[hh].from(ws);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float s = j < 8 ? s0 : s1;
      const float sz = j < 8 ? sz0 : sz1;
      const half2_t qq = cp[j >> 3].q[j & 7];
      const float w0 = __builtin_fmaf(s, (float)qq[0], -sz);
      const float w1 = __builtin_fmaf(s, (float)qq[1], -sz);
      h[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t){w0, w1}, half2_t));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
}

// The 16 codes (16*NB bits) starting at p (2*NB-byte aligned), LSB first in words.
template <int NB>
struct Codes16 {
  static constexpr int kWords = (16 * NB + 31) / 32;
};
template <int NB>
__device__ __forceinline__ void load_codes16(const uint8_t* p, uint32_t (&w)[Codes16<NB>::kWords]) {
  if constexpr (NB == 2) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (NB == 3) {  // 6 bytes, 2-byte aligned
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    w[0] = (uint32_t)q[0] | ((uint32_t)q[1] << 16);
    w[1] = q[2];
  } else if constexpr (NB == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
}

// Dequantize 16 codes of one group to binary16, as dequant32 (w = s*q - s*z in fp32, one
// rounding, then binary16).
template <int NB>
__device__ __forceinline__ void dequant16(const uint32_t (&w)[Codes16<NB>::kWords], float s, float sz,
                                          uint4 (&out)[2]) {
  uint32_t h[8];
  if constexpr (NB == 3) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float w0 = __builtin_fmaf(s, (float)code_at<NB>(w, 2 * j), -sz);
      const float w1 = __builtin_fmaf(s, (float)code_at<NB>(w, 2 * j + 1), -sz);
      h[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t){w0, w1}, half2_t));
    }
  } else {
    CodePairs<NB> cp;
    cp.from(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float w0 = __builtin_fmaf(s, (float)cp.q[j][0], -sz);
      const float w1 = __builtin_fmaf(s, (float)cp.q[j][1], -sz);
      h[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t){w0, w1}, half2_t));
    }
  }
  out[0] = make_uint4(h[0], h[1], h[2], h[3]);
  out[1] = make_uint4(h[4], h[5], h[6], h[7]);
}

constexpr float kSub = 16777216.f;  // 2^24: a binary16 subnormal's unit is 2^-24

// s*q - s*z of two codes as binary16: fma in fp32 (s z exact, one rounding), rounded to binary16.
// The codes come as the halves of t, each shifted left inside an otherwise empty half: read as
// binary16 that is a subnormal, q 2^(shift - 24) exactly, and the scales carry the power back.  Two
// instructions a pair, where conversion in fp32 and a packing conversion take three (and
// exponents put in front of the codes one more).
// A matrix instruction must not read d within two wait states of its write, and the compiler, which
// keeps that distance for its own instructions, does not for these: callers put the result
// into LDS, or separate it by mfma_distance().
__device__ __forceinline__ uint32_t weight_pair(uint32_t t, float s_lo, float s_hi, float minus_sz) {
  uint32_t d;
  asm("v_fma_mixlo_f16 %0, %1, %2, %4 op_sel_hi:[1,0,0]\n\t"
      "v_fma_mixhi_f16 %0, %1, %3, %4 op_sel:[1,0,0] op_sel_hi:[1,0,0]"
      : "=&v"(d) : "v"(t), "v"(s_lo), "v"(s_hi), "v"(minus_sz));
  return d;
}

__device__ __forceinline__ void mfma_distance() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 1");
  __builtin_amdgcn_sched_barrier(0);
}

// A group's scales as decode_pair takes them: s 2^24 and -s z; the other shifts' powers of s.
struct PairScale {
  float a, c;
};

// Codes 8 step + 2 e and + 1 of a lane's 16 or 32 (LSB first in w) as two binary16 weights.
template <int NB, int W>
__device__ __forceinline__ uint32_t decode_pair(const uint32_t (&w)[W], int step, int e, PairScale p) {
  if constexpr (NB == 3) {         // codes straddle bytes: one by one
    const float sv = p.a * (1.f / kSub);
    const float w0 = __builtin_fmaf(sv, (float)code_at<NB>(w, 8 * step + 2 * e), p.c);
    const float w1 = __builtin_fmaf(sv, (float)code_at<NB>(w, 8 * step + 2 * e + 1), p.c);
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t){w0, w1}, half2_t));
  } else if constexpr (NB == 8) {  // bytes 2 e, 2 e + 1 of two words
    const uint32_t t = __builtin_amdgcn_perm(0u, w[2 * step + (e >> 1)], (e & 1) ? 0x0C030C02u : 0x0C010C00u);
    return weight_pair(t, p.a, p.a, p.c);
  } else if constexpr (NB == 4) {  // byte e of a word, in both halves
    const uint32_t t = __builtin_amdgcn_perm(0u, w[step], 0x0C000C00u | (uint32_t)e | ((uint32_t)e << 16));
    return weight_pair(t & 0x00F0000Fu, p.a, p.a * (1.f / 16.f), p.c);
  } else {                         // byte 2 (step % 2) + e / 2 of a word, two of its four codes
    const uint32_t at = (uint32_t)(2 * (step & 1) + (e >> 1));
    const uint32_t t = __builtin_amdgcn_perm(0u, w[step >> 1], 0x0C000C00u | at | (at << 16));
    return e & 1 ? weight_pair(t & 0x00C00030u, p.a * (1.f / 16.f), p.a * (1.f / 64.f), p.c)
                 : weight_pair(t & 0x000C0003u, p.a, p.a * (1.f / 4.f), p.c);
  }
}

// Block barrier that orders LDS accesses only: __syncthreads() also makes every wavefront
// wait for its outstanding global loads (vmcnt(0)), which would end each prefetch at
// the barrier.  The workgroup fences here are restricted to the LDS address space.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace
}  // namespace hqq
