// act8.cuh -- device arithmetic shared by the channel-wise operators: 16-bit
// conversions, the activations and their derivatives, and the 8-bit
// checkpoint code.
//
// Checkpoint code.  32 consecutive channels of a row share one exponent byte
// b = max(7, biased exponent of the block's largest magnitude), and a value v
// is kept as the integer k = clamp(rint(v * 2^(133-b)), -127, 127), which
// stands for k * 2^(b-133): seven bits and a sign under a shared power of two
// (the layout of the open MX formats' 8-bit integers).  A power-of-two step
// makes the scaling exact, so one rounding (half a step, at most 1/128 of the
// block's largest magnitude) is all that is lost, the same code comes out of
// any precision that holds v, and every code is exactly representable in
// bf16.  Against e4m3 with the same exponent byte (3 fraction bits: up to 1/16
// of each value) the error of a block of normal deviates is about four times
// smaller.  b = 255 marks a block with an infinity or NaN; all of it reads
// back as NaN, so a diverged activation cannot pass as a finite one.  b >= 7
// keeps 2^(133-b) and the step normal numbers; smaller values lose at most
// 2^-127.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace conv3d {

constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2;   // conv3d_act_t

template <bool kBF16>
struct Val16 {
  static __device__ __forceinline__ float lo(uint32_t w) {
    if constexpr (kBF16) return __uint_as_float(w << 16);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(w & 0xFFFFu)));
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    if constexpr (kBF16) return __uint_as_float(w & 0xFFFF0000u);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16)));
  }
  // two values rounded to nearest even, the first in the low half
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    if constexpr (kBF16) {
      __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      return *reinterpret_cast<uint32_t*>(&h);
    }
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  // eight values as four pairs
  static __device__ __forceinline__ float2 pair(uint32_t w) {
    if constexpr (kBF16) return make_float2(lo(w), hi(w));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ void unpack8(const uint4& q, float2 (&f)[4]) {
    f[0] = pair(q.x); f[1] = pair(q.y); f[2] = pair(q.z); f[3] = pair(q.w);
  }
  static __device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
    return make_uint4(pack(f[0].x, f[0].y), pack(f[1].x, f[1].y), pack(f[2].x, f[2].y), pack(f[3].x, f[3].y));
  }
};

// ------------------------------------------------------------------ pairs

// Two fp32 values per instruction (sm_100's packed fp32 operations, each lane
// rounded as the scalar operation is): the channel-wise kernels are bound by
// instruction issue, and their sums and products come in pairs.
__device__ __forceinline__ unsigned long long f2_bits(float2 a) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 f2_from(unsigned long long b) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(b));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
  return f2_from(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_from(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_from(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// ------------------------------------------------------------------ activations

// silu(v) = v s(v), gelu(v) = v s(2 u(v)) with s(x) = 1 / (1 + e^-x) and u = sqrt(2/pi)
// (v + 0.044715 v^3): two special-function operations, 2^w and a reciprocal, w =
// -log2(e) times the argument of s.  Both are relative approximations, and w is off by
// a few 2^-24 of itself, so the relative error stays below 2^-15 out to the smallest
// results (h + h tanh(h), h = v/2, needs one operation, but the hardware tanh's error
// of 2^-11 is relative to v and not to the result: silu(-8) = -0.0027 could be off by
// 0.0020).  s below 2^-126 is 0, in both places that can find it so: 2^w is infinite
// from w = 128 on, and the reciprocal flushes what lies below the normal numbers.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }
__device__ __forceinline__ float2 rcp(float2 x) { return make_float2(rcp(x.x), rcp(x.y)); }

constexpr double kLog2e = 1.4426950408889634, kGeluA = 0.7978845608028654;   // sqrt(2 / pi)
constexpr float kSiluW = static_cast<float>(-kLog2e);
constexpr float kGeluW1 = static_cast<float>(-2.0 * kGeluA * kLog2e);
constexpr float kGeluW3 = static_cast<float>(-2.0 * kGeluA * kLog2e * 0.044715);
// 2 u'(v) = kGeluD0 + kGeluD2 v^2
constexpr float kGeluD0 = static_cast<float>(2.0 * kGeluA), kGeluD2 = static_cast<float>(6.0 * kGeluA * 0.044715);

// w of v, and of v = 2 h: the same bits (the constants differ by powers of two).
template <int kAct>
__device__ __forceinline__ float2 act_exponent(float2 v) {
  if constexpr (kAct == kActSilu) return mul2(v, both(kSiluW));
  return mul2(v, fma2(both(kGeluW3), mul2(v, v), both(kGeluW1)));
}
template <int kAct>
__device__ __forceinline__ float2 act_exponent_of_half(float2 h, float2 h2) {
  if constexpr (kAct == kActSilu) return mul2(h, both(2.0f * kSiluW));
  return mul2(h, fma2(both(8.0f * kGeluW3), h2, both(2.0f * kGeluW1)));
}

template <int kAct>
__device__ __forceinline__ float2 act_value(float2 v) {
  if constexpr (kAct == kActNone) return v;
  return mul2(v, rcp(add2(ex2(act_exponent<kAct>(v)), both(1.0f))));
}
template <int kAct>
__device__ __forceinline__ float act_value(float v) {
  return act_value<kAct>(both(v)).x;
}

// Both derivatives are s + c s (1 - s) = s (1 + c (1 - s)), 1 - s = 2^w s, with c = v
// (silu) or 2 v u'(v) (gelu).  Beyond |v| = 88 and 10.03, where w passes +-126.9, s is
// 0 or 1 exactly (and 2^w still finite); v^3 may overflow there, which would leave
// infinity times zero: such arguments are brought back to these bounds.
template <int kAct>
__host__ __device__ constexpr float act_half_bound() {
  return kAct == kActSilu ? 44.0f : 5.015f;
}

// The derivative at v = 2 h (the checkpoint's values are decoded to their halves), and
// the value there from the same s; `whole` is h before it was brought within the bound,
// which the value goes on growing with.
template <int kAct>
__device__ __forceinline__ float2 act_slope_and_value(float2 whole, float2 h, float2& value) {
  const float2 h2 = kAct == kActGelu ? mul2(h, h) : h;
  const float2 e = ex2(act_exponent_of_half<kAct>(h, h2));
  const float2 s = rcp(add2(e, both(1.0f)));
  value = mul2(add2(whole, whole), s);
  const float2 c = kAct == kActGelu ? mul2(h, fma2(both(8.0f * kGeluD2), h2, both(2.0f * kGeluD0))) : add2(h, h);
  return mul2(s, fma2(c, mul2(e, s), both(1.0f)));
}
template <int kAct>
__device__ __forceinline__ float2 act_slope_of_half(float2 h) {
  if constexpr (kAct == kActNone) return both(1.0f);
  float2 value;
  return act_slope_and_value<kAct>(h, h, value);
}

// The same at any v.  (NaN stays: fminf and fmaxf would drop it.)
template <int kAct>
__device__ __forceinline__ float act_slope_safe(float v) {
  if constexpr (kAct == kActNone) return 1.0f;
  constexpr float kBound = act_half_bound<kAct>();
  const float s = act_slope_of_half<kAct>(both(fminf(fmaxf(0.5f * v, -kBound), kBound))).x;
  return v == v ? s : v;
}

// ------------------------------------------------------------------ checkpoint code

// Magnitude as an unsigned integer: ordered like the magnitudes, with
// infinities and NaN above every finite one.
__device__ __forceinline__ uint32_t a8_mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The largest of a magnitude m, |v.x| and |v.y|, NaN if any is.
__device__ __forceinline__ float a8_max(float m, float2 v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(v.x)), "f"(fabsf(v.y)));
  return r;
}

// The largest magnitude of 8 values, as bits.
__device__ __forceinline__ uint32_t a8_mag8(const float2 (&f)[4]) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) m = a8_max(m, f[e]);
  return __float_as_uint(m);
}

// Exponent byte of a block whose largest magnitude has the bits `mag`.
__device__ __forceinline__ uint32_t a8_exponent(uint32_t mag) {
  const uint32_t b = mag >> 23;
  return b < 7u ? 7u : b;
}

// 2^(133-b); 0 for a block marked as not finite.
__device__ __forceinline__ float a8_inv_step(uint32_t b) {
  return b == 255u ? 0.0f : __uint_as_float((260u - b) << 23);
}

// 2^(b-133); NaN for a block marked as not finite.
__device__ __forceinline__ float a8_step(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7FFFFFFFu : (b - 6u) << 23);
}

// v * inv + 1.5 * 2^23 rounds v * inv (exact: inv is a power of two) to the
// nearest integer, ties to even, and leaves it in the low bits of the sum in
// two's complement.
constexpr float kA8Magic = 12582912.0f;
__device__ __forceinline__ float2 a8_round(float2 v, float inv) { return fma2(v, both(inv), both(kA8Magic)); }

// Only a block whose largest magnitude is 127.5 steps and more (its fraction
// bits are 0x7F0000 and up) rounds to 128 and has to be clamped.
__device__ __forceinline__ bool a8_clamps(uint32_t mag) { return (mag & 0x7FFFFFu) >= 0x7F0000u; }
__device__ __forceinline__ float2 a8_clamp(float2 r) {
  return make_float2(fminf(fmaxf(r.x, kA8Magic - 127.0f), kA8Magic + 127.0f),
                     fminf(fmaxf(r.y, kA8Magic - 127.0f), kA8Magic + 127.0f));
}

// The low bytes of four rounded values, the first lowest.
__device__ __forceinline__ uint32_t a8_bytes(float2 a, float2 b) {
  return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                     __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t a8_code4(float2 a, float2 b, float inv) {
  return a8_bytes(a8_clamp(a8_round(a, inv)), a8_clamp(a8_round(b, inv)));
}

// Values of four codes: the byte k + 128 under the exponent of 2^23 is the
// float 2^23 + 128 + k, from which the subtraction leaves k exactly.
__device__ __forceinline__ void a8_decode4(uint32_t w, float step, float2* v) {
  w ^= 0x80808080u;
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u + i));
  v[0] = mul2(add2(make_float2(f[0], f[1]), both(-8388736.0f)), both(step));
  v[1] = mul2(add2(make_float2(f[2], f[3]), both(-8388736.0f)), both(step));
}

// Whether halves of values (at most 127 half steps) can lie outside act_half_bound: with
// a step above 1/2 (silu) or 1/16 (gelu), and not in a block marked as not finite (NaN
// step).
template <int kAct>
__device__ __forceinline__ bool a8_wide(float half) {
  constexpr float kMost = kAct == kActSilu ? 0.25f : 0.03125f;
  static_assert(127.0f * kMost <= act_half_bound<kAct>(), "blocks of smaller steps need no narrowing");
  return half > kMost;
}
template <int kAct>
__device__ __forceinline__ float2 a8_narrow(float2 h) {
  constexpr float kBound = act_half_bound<kAct>();
  return make_float2(fminf(fmaxf(h.x, -kBound), kBound), fminf(fmaxf(h.y, -kBound), kBound));
}

// Halves of the values of 4 N codes, `half` the half step, brought back to the bound
// (see act_half_bound) if kNarrow.  Where the step is small the subtraction and the
// product are one exact fused operation; NaN steps go the same way and stay NaN.
template <int kAct, bool kNarrow, int N>
__device__ __forceinline__ void a8_decode_halves(const uint32_t (&w)[N], float half, float2 (&h)[2 * N]) {
  if (a8_wide<kAct>(half)) {
#pragma unroll
    for (int i = 0; i < N; ++i) a8_decode4(w[i], half, h + 2 * i);
    if constexpr (kNarrow)
#pragma unroll
      for (int e = 0; e < 2 * N; ++e) h[e] = a8_narrow<kAct>(h[e]);
    return;
  }
  const float off = -8388736.0f * half;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t x = w[i] ^ 0x80808080u;
    h[2 * i] = fma2(make_float2(__uint_as_float(__byte_perm(x, 0x4B000000u, 0x7440u)),
                                __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7441u))), both(half), both(off));
    h[2 * i + 1] = fma2(make_float2(__uint_as_float(__byte_perm(x, 0x4B000000u, 0x7442u)),
                                    __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7443u))), both(half), both(off));
  }
}

}  // namespace conv3d
