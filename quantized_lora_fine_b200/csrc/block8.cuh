// The e4m3 block quantizer's arithmetic, shared by the row and weight quantizers and
// the RMS norm's 8-bit output.
//
//   a = max(max |x|, 2^-100) over a block,  scale = fp32(a / 448),
//   q = e4m3_rne(448 x / a) of the real quotient.
//
// The quotient is decided in fp32: with p = 2^-exponent(a), a' = a p is in [1, 2) and
// u = 448 p x, t = u y with y near 1 / a', and t is corrected once by its remainder,
// t + (u - t a') y (Markstein's quotient step; the remainder is exact, so y needs no more than
// a few last places).
//   bf16 x: u is exact (8 + 3 significant bits) and t is the real quotient wherever that is
// representable, so a quotient on the midpoint of two e4m3 values is seen as the midpoint and
// rounds to even; no other quotient of two bf16 values is within fp32 rounding of one.
//   fp32 weights: u is rounded too, t is up to two last places from the real quotient, and that may lie
// so near to a midpoint m on either side (4 weights in 10^7 of a normal distribution came out a code
// off): where t is within 8 places of an m, the sign of 448 p x - m a' decides (block8_decide).
//   The norm's y: quantized by t. y is itself a rounded product, and real quotients on a midpoint are
// common there (6 values in 10^4: h and w have 8 bits each); t's rounding returns most of them to
// the midpoint that y's rounding left. Deciding by the exact quotient of the rounded y gave half as many
// codes again that differ from those of the unrounded one (326 for 215 of 400 x 4096), and at 8192 x
// 4096 took 50 us for 40.
//   The scale is the same step with 448 (equal to the division for all 2^23 significands). A block that
// holds a NaN or an infinity gets NaN codes: its p is infinite.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/qlora_b200.h"

namespace qlb {

constexpr uint32_t kBlock8Floor = 0x0D800000u;   // 2^-100, as fp32 bits

struct Block8 {
  float scale;   // a / 448
  float c;       // 448 * 2^-exponent(a)
  float a;       // a', in [1, 2)
  float inv;     // near 1 / a'
};

// `bits`: the largest |x| of the block as fp32 bits (as integers, so that NaN > Inf >
// every number).
__device__ __forceinline__ Block8 block8_of(uint32_t bits) {
  bits = max(bits, kBlock8Floor);
  Block8 b;
  const float a = __uint_as_float(bits);
  constexpr float r448 = 1.f / 448.f;
  const float t = __fmul_rn(a, r448);
  b.scale = bits < 0x7F800000u ? __fmaf_rn(__fmaf_rn(-t, 448.f, a), r448, t) : a;
  // 2^-exponent(a): the exponent's complement; 2^-127, subnormal, for the largest; a NaN's or
  // infinity's (e = 255) comes out as -infinity.
  const uint32_t e = bits >> 23;                          // 27 .. 255
  b.c = 448.f * __uint_as_float(max((254u - e) << 23, 0x00400000u));
  b.a = __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b.inv) : "f"(b.a));
  return b;
}

__device__ __forceinline__ float block8_quotient(float x, const Block8& b) {
  const float u = __fmul_rn(x, b.c);
  const float t = __fmul_rn(u, b.inv);
  return __fmaf_rn(__fmaf_rn(-t, b.a, u), b.inv, t);
}

// Four quotients to four e4m3 bytes (nearest even; |q| <= 448 by construction, NaN to NaN).
__device__ __forceinline__ uint32_t e4m3x4(float q0, float q1, float q2, float q3) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(q1), "f"(q0));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(q3), "f"(q2));
  return uint32_t(lo) | (uint32_t(hi) << 16);
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t max_abs8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}

// The same of 8 bf16 values: magnitudes as 16-bit integers, two at a time.
__device__ __forceinline__ uint32_t max_abs8(const uint4& v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                              __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  return max(m << 16, m & 0xFFFF0000u);
}

// Over 16 consecutive lanes (one 128-value block at 8 values a lane).
__device__ __forceinline__ uint32_t max16(uint32_t m) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

// The quotient of an fp32 x, or where it is within 8 places of a value m of 5 significant bits (as
// midpoints are, all 2^-10 or more): m, if the real quotient is m, else m's neighbour on its side.
// u + lo is 448 p x; u - m a' is exact, for the two agree in all but their last places; its sum with lo
// has the real difference's sign.
__device__ __forceinline__ float block8_decide(float x, const Block8& b) {
  const float t = block8_quotient(x, b);
  const uint32_t bits = __float_as_uint(t) & 0x7FFFFFFFu;
  if (((bits + 8u) & 0x7FFFFu) >= 16u || bits - 0x3A000000u >= 0x0A000000u) return t;   // (2^-11 .. 2^9)
  const uint32_t m = (bits + 8u) & ~0x7FFFFu, sign = __float_as_uint(x) & 0x80000000u;
  const float u = __fmul_rn(x, b.c), lo = __fmaf_rn(x, b.c, -u);
  const float d = __fadd_rn(__fmaf_rn(-__uint_as_float(m | sign), b.a, u), lo);
  const bool in = (__float_as_uint(d) & 0x80000000u) != sign;      // towards zero
  return __uint_as_float((d == 0.f ? m : in ? m - 1u : m + 1u) | sign);
}

// EXACT: codes of the real quotients of fp32 values. (Few threads meet a value that needs it.)
template <bool EXACT = false>
__device__ __forceinline__ uint2 quantize8(const float (&f)[8], const Block8& b) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = block8_quotient(f[i], b);
  if constexpr (EXACT) {
    uint32_t off = 0x7FFFFu;
#pragma unroll
    for (int i = 0; i < 8; ++i) off = min(off, (__float_as_uint(q[i]) + 8u) & 0x7FFFFu);
    if (off < 16u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = block8_decide(f[i], b);
    }
  }
  return make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
}

// ---- launches (block8.cu, norm.cu)
qlora_status launch_quantize_rows8(const uint16_t* X, int64_t M, int64_t in, uint8_t* codes, float* scale,
                                   cudaStream_t s);
qlora_status launch_quantize_weight8(const void* W, bool f32, int64_t E, int64_t out, int64_t in, uint8_t* codes,
                                     float* scale, int* status, cudaStream_t s);
struct NormFwd {
  const uint16_t* x;
  const uint16_t* residual;   // may be null
  const void* w;
  bool w_f32;
  int64_t M, H;
  float eps;
  uint16_t* h;                // may be null without a residual
  uint16_t* y;                // bf16 output, or null
  uint8_t* y8;                // 8-bit output with y_scale, or null
  float* y_scale;
  float* rstd;
};
qlora_status launch_rms_norm_fwd(const NormFwd& a, cudaStream_t s);
struct NormBwd {
  const uint16_t* dy;
  const uint16_t* dh;         // may be null
  const uint16_t* h;
  const float* rstd;
  const void* w;
  bool w_f32;
  int64_t M, H;
  uint16_t* dx;
  float* dw;                  // may be null
  float* part;                // norm_bwd_parts(M, H) rows of H values (with dw)
};
int norm_bwd_parts(int64_t M, int64_t H);
qlora_status launch_rms_norm_bwd(const NormBwd& a, cudaStream_t s);
constexpr int64_t kMaxNormHidden = 32768;   // 512 threads of 8 vectors

}  // namespace qlb
