// ff_ops.cuh -- what the feed-forward kernels share: the 16-bit float and
// 8-bit integer tcgen05 MMAs, the activations with their slopes, and the
// rounding of fp32 results to either 16-bit type.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace tg {

// Operand kinds of the feed-forward kernels.  Both move 128 bytes of K per
// k-block and 32 bytes of K per MMA, so they share every byte offset.
enum { kFfF16 = 0, kFfI8 = 1 };

// Activations of the gated block (the values of TG_ACT_*).
enum { kActRelu = 0, kActSilu = 1, kActGelu = 2 };

// Whether the phase with parity `parity` has completed, without waiting at all.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar_addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar_addr), "r"(parity)
      : "memory");
  return ok != 0u;
}

// D[tmem] (+)= A[smem desc] * B[smem desc] on a CTA pair: 16-bit floats into
// fp32, or signed 8-bit integers into 32-bit integers.
template <int KIND>
__device__ __forceinline__ void umma_ff_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  if (KIND == kFfF16) {
    umma_f16_ss_pair(d_tmem, a_desc, b_desc, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// The same on one CTA.
template <int KIND>
__device__ __forceinline__ void umma_ff(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  if (KIND == kFfF16) {
    umma_f16_ss(d_tmem, a_desc, b_desc, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// Instruction descriptor: bits 4-5 D format (1 = f32, 2 = s32); bits 7-9 /
// 10-12 A / B format (kind::f16: 0 = f16, 1 = bf16, the same for both;
// kind::i8: 1 = signed); bit 15 / 16 A / B major-ness (0 = K-major, 1 =
// MN-major, 16-bit operands only); bits 17-22 N >> 3; bits 24-28 M >> 4.
inline uint32_t make_idesc_ff(int kind, bool bf16, int M, int N, bool a_mn_major, bool b_mn_major) {
  const uint32_t d = kind == kFfI8 ? 2u : 1u;
  const uint32_t f = kind == kFfI8 ? 1u : (bf16 ? 1u : 0u);
  return (d << 4) | (f << 7) | (f << 10) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// ----------------------------------------------------------------------------
// Activations, in fp32
// ----------------------------------------------------------------------------
// Both smooth activations are g * s(z) with the logistic function s: z = g
// for silu, and for gelu (tanh form) z = 2 sqrt(2/pi) (g + 0.044715 g^3),
// since (1 + tanh(y)) / 2 = s(2y).  s(z) = 2^-8 / (2^-8 + 2^(-8 - z log2 e)), with
// -log2 e folded into the constants: one exponential and one reciprocal
// instruction, each good to about 2^-22.  (Far from 0 the exponent's own rounding
// adds up to 2^-15.)  Both are far below half a step of a 16-bit result.  The
// reciprocal instruction gives subnormal results as 0; the factors of 2^-8 keep
// it out of them down to s = 2^-134, a subnormal with 15 bits (in bf16, a far
// gate times a large U is not 0).  Below that (z < -92.9) s is 0.
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kGeluC1 = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kGeluC3 = 0.07135481282553557f;  // 2 sqrt(2/pi) 0.044715

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations per instruction (sm_100's packed pairs; each half
// rounds as the single operation does).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 same2(float a) { return make_float2(a, a); }

// s(z) of the activation's z, for two values.
template <int ACT>
__device__ __forceinline__ float2 act_logistic2(float2 g) {
  float2 t;  // -8 - z log2 e
  if (ACT == kActSilu)
    t = fma2(g, same2(-kLog2E), same2(-8.0f));
  else
    t = fma2(g, fma2(mul2(g, g), same2(-kLog2E * kGeluC3), same2(-kLog2E * kGeluC1)), same2(-8.0f));
  const float2 d = add2(make_float2(exp2_approx(t.x), exp2_approx(t.y)), same2(0.00390625f));
  return mul2(make_float2(rcp_approx(d.x), rcp_approx(d.y)), same2(0.00390625f));
}

template <int ACT>
__device__ __forceinline__ float2 act_value2(float2 g) {
  if (ACT == kActRelu) return make_float2(g.x > 0.0f ? g.x : 0.0f, g.y > 0.0f ? g.y : 0.0f);
  return mul2(g, act_logistic2<ACT>(g));
}

// act(g) and its derivative: with p = s(z), act = g p and act' = p + g p (1 - p) z'.
template <int ACT>
__device__ __forceinline__ void act_value_slope2(float2 g, float2& value, float2& slope) {
  if (ACT == kActRelu) {
    value = act_value2<ACT>(g);
    slope = make_float2(g.x > 0.0f ? 1.0f : 0.0f, g.y > 0.0f ? 1.0f : 0.0f);
    return;
  }
  const float2 p = act_logistic2<ACT>(g);
  value = mul2(g, p);
  const float2 q = fma2(p, same2(-1.0f), same2(1.0f));
  const float2 r = mul2(value, q);
  slope = ACT == kActSilu ? add2(p, r) : fma2(r, fma2(mul2(g, g), same2(3.0f * kGeluC3), same2(kGeluC1)), p);
  // Far gates: where p is 0 so is everything, and where it is 1 the slope is,
  // though g (an infinity, when the stored value overflowed) or z' is not finite.
  if (p.x == 0.0f) value.x = slope.x = 0.0f;
  if (p.y == 0.0f) value.y = slope.y = 0.0f;
  if (q.x == 0.0f) slope.x = 1.0f;
  if (q.y == 0.0f) slope.y = 1.0f;
}

// ----------------------------------------------------------------------------
// 16-bit results
// ----------------------------------------------------------------------------
// Two fp32 values rounded (nearest even) to fp16 or bf16 and packed, the
// first in the low half.
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two packed 16-bit values as fp32.
__device__ __forceinline__ float2 unpack_16(uint32_t w, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float load_16(const unsigned short* p, bool bf16) {
  const unsigned short v = __ldg(p);
  return bf16 ? __uint_as_float(static_cast<uint32_t>(v) << 16) : __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ unsigned short round_16(float x, bool bf16) {
  return static_cast<unsigned short>((bf16 ? pack_bf16(x, 0.0f) : pack_f16(x, 0.0f)) & 0xffffu);
}

// N fp32 values of one row as packed 16-bit pairs.
template <int N>
__device__ __forceinline__ void pack_row(const float (&v)[N], uint32_t* h, bool bf16) {
  if (bf16) {
#pragma unroll
    for (int e = 0; e < N / 2; ++e) h[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
  } else {
#pragma unroll
    for (int e = 0; e < N / 2; ++e) h[e] = pack_f16(v[2 * e], v[2 * e + 1]);
  }
}

}  // namespace tg
