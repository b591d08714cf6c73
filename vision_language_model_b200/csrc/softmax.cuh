// Row softmax pieces of the attention kernels on the tensor cores: packed fp32
// arithmetic, row maxima, exponentials on two kinds of pipe, wide TMEM loads.
#pragma once

#include "common.cuh"
#include "exp2_poly.cuh"

namespace vlm {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Packed pairs of fp32 (first value in the low word) for the f32x2 instructions.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair_f32(float v) { return pack2(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Row maximum of N values with four independent chains of 3-input max.
template <int N>
__device__ __forceinline__ float row_max(const uint32_t (&u)[N]) {
  constexpr int NC = 4;
  float m[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) m[i] = -INFINITY;
#pragma unroll
  for (int c = 0; c < N; c += 2 * NC) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const float x = __uint_as_float(u[c + 2 * i]), y = __uint_as_float(u[c + 2 * i + 1]);
      m[i] = max3f(m[i], x, y);
    }
  }
#pragma unroll
  for (int w = NC / 2; w > 0; w /= 2)
#pragma unroll
    for (int i = 0; i < w; ++i) m[i] = fmaxf(m[i], m[i + w]);
  return m[0];
}

// 32 lanes x 64 columns of 32-bit TMEM words into registers (one lane per
// thread), waiting for completion inside the same asm block.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}

// One pair of scores in kPolyPairEvery takes its two exponentials from
// exp2_poly (FMA and ALU pipes) instead of ex2.approx (MUFU), so the two kinds
// of pipe share the softmax's exponentials. MUFU is the softmax's bottleneck;
// one pair in eight measured fastest: one in four fits the 96 registers a
// thread has at 2 CTAs of 320 threads per SM but is no faster, one in three
// spills.
#ifndef VLM_ATTN_POLY_PAIR_EVERY
#define VLM_ATTN_POLY_PAIR_EVERY 8
#endif
constexpr int kPolyPairEvery = VLM_ATTN_POLY_PAIR_EVERY;

// 2^x without MUFU: k = round(x) by adding 1.5 * 2^23, f = x - k in
// [-1/2, 1/2], 2^f from the degree-3 minimax polynomial of exp2_poly.cuh
// (relative error < 7.5e-5, fitted by fit_exp2_poly.py with the Remez
// algorithm), then k added to the exponent field. Scalar arithmetic with
// immediate constants (no register pairs). x is clamped to -126 so the
// exponent cannot wrap; the result is then ~1e-38 instead of 0, so keys that
// must weigh exactly 0 never take this path.
__device__ __forceinline__ float exp2_poly(float x) {
  x = fmaxf(x, -126.0f);
  const float j = x + 12582912.0f;
  const float f = x - (j - 12582912.0f);
  const float p = fmaf(fmaf(fmaf(kExp2C3, f, kExp2C2), f, kExp2C1), f, kExp2C0);
  return __int_as_float(__float_as_int(p) + (__float_as_int(j) << 23));
}

// Log2 units that fp16 weights are larger by, and their sums with them: they stay
// below 2^8 of their maximum, so this fills fp16's largest powers of two and takes
// the weights that it holds in 11 bits down from 2^-14 to 2^-21 of the maximum, the
// smallest that it tells from 0 from 2^-25 to 2^-32.
constexpr float kHalfLift = 7.0f;

// p_c = 2^(s_c * sl2 - m) for the thread's N scores of the row, packed as pairs (bf16,
// or fp16 with kHalf) into pk; returns sum_c p_c (fp32, before rounding). The elements are independent.
// With kHalf the caller takes kHalfLift from m.
// kRaw: m is in the scores' own units and p_c = 2^((s_c - m) * sl2) (with kHalf
// lifted here), one more operation per pair, for scores of any size: a product rounded before it is
// subtracted would be off by 2^-24 of itself, which counts from some 10^8 on.
// kPoly: let exp2_poly take one pair in kPolyPairEvery (never on a tile with
// masked keys, whose weights must be exactly 0).
template <bool kPoly, bool kHalf = false, bool kRaw = false, int N>
__device__ __forceinline__ float row_exp(const uint32_t (&u)[N], uint64_t sl2x2, float m, uint32_t (&pk)[N / 2]) {
  const uint64_t negm2 = pair_f32(-m);
  uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    float x0, x1, p0, p1;
    if (kRaw) {
      const uint64_t d = add2(pack2(u[c], u[c + 1]), negm2);
      unpack2(kHalf ? fma2(d, sl2x2, pair_f32(kHalfLift)) : mul2(d, sl2x2), x0, x1);
    } else {
      unpack2(fma2(pack2(u[c], u[c + 1]), sl2x2, negm2), x0, x1);
    }
    if (kPoly && kPolyPairEvery > 0 && (c >> 1) % (kPolyPairEvery > 0 ? kPolyPairEvery : 1) == kPolyPairEvery - 1) {
      p0 = exp2_poly(x0);
      p1 = exp2_poly(x1);
    } else {
      p0 = ex2(x0);
      p1 = ex2(x1);
    }
    const int i = (c >> 1) & 3;
    acc[i] = add2(acc[i], pack2(__float_as_uint(p0), __float_as_uint(p1)));
    pk[c >> 1] = kHalf ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
  }
  float s0, s1, s2, s3, s4, s5, s6, s7;
  unpack2(acc[0], s0, s1);
  unpack2(acc[1], s2, s3);
  unpack2(acc[2], s4, s5);
  unpack2(acc[3], s6, s7);
  return ((s0 + s1) + (s2 + s3)) + ((s4 + s5) + (s6 + s7));
}

}  // namespace vlm
