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

// One special-function operation per activation: the hardware tanh, whose
// error is about 2^-11 of a result of magnitude at most 1.  silu(v) = h + h
// tanh(h), h = v/2; gelu(v) = h + h tanh(u(v)), u = sqrt(2/pi) (v + 0.044715
// v^3).  The absolute error is at most |v| 2^-12, under half a bf16 step of v.
__device__ __forceinline__ float tanh_hw(float x) {
  float t;
  asm("tanh.approx.f32 %0, %1;" : "=f"(t) : "f"(x));
  return t;
}

constexpr float kGeluA = 0.7978845608028654f;             // sqrt(2 / pi)
constexpr float kGeluC = 0.7978845608028654f * 0.044715f;

template <int kAct>
__device__ __forceinline__ float act_value(float v) {
  if constexpr (kAct == kActSilu) {
    const float h = 0.5f * v;
    return fmaf(h, tanh_hw(h), h);
  } else if constexpr (kAct == kActGelu) {
    const float u = v * fmaf(kGeluC, v * v, kGeluA);
    const float h = 0.5f * v;
    return fmaf(h, tanh_hw(u), h);
  } else {
    return v;
  }
}

// silu'(v) = s + v s (1 - s) with s = (1 + t)/2, t = tanh(v/2):
//   = (1 + t)/2 + (v/4) (1 - t^2).
// gelu'(v) = (1 + t)/2 + (v/2) (1 - t^2) u'(v), t = tanh(u(v)).
template <int kAct>
__device__ __forceinline__ float act_slope(float v) {
  if constexpr (kAct == kActSilu) {
    const float t = tanh_hw(0.5f * v);
    const float c = 0.25f * v;
    return fmaf(c, fmaf(-t, t, 1.0f), fmaf(0.5f, t, 0.5f));
  } else if constexpr (kAct == kActGelu) {
    const float v2 = v * v;
    const float t = tanh_hw(v * fmaf(kGeluC, v2, kGeluA));
    const float c = 0.5f * v * fmaf(3.0f * kGeluC, v2, kGeluA);
    return fmaf(c, fmaf(-t, t, 1.0f), fmaf(0.5f, t, 0.5f));
  } else {
    return 1.0f;
  }
}

// The same for a pair: all but the two tanh in packed operations.
__device__ __forceinline__ float2 tanh_hw2(float2 x) { return make_float2(tanh_hw(x.x), tanh_hw(x.y)); }

template <int kAct>
__device__ __forceinline__ float2 act_value(float2 v) {
  if constexpr (kAct == kActSilu) {
    const float2 h = mul2(both(0.5f), v);
    return fma2(h, tanh_hw2(h), h);
  } else if constexpr (kAct == kActGelu) {
    const float2 u = mul2(v, fma2(both(kGeluC), mul2(v, v), both(kGeluA)));
    const float2 h = mul2(both(0.5f), v);
    return fma2(h, tanh_hw2(u), h);
  } else {
    return v;
  }
}

// The derivative in terms of h = v/2, which the checkpoint's values are decoded
// to (half the step): with q = t^2 - 1,
//   silu'(v) = (1 + t)/2 - (h/2) q,                      t = tanh(h)
//   gelu'(v) = (1 + t)/2 - h (a + 12 c h^2) q,           t = tanh(h (2a + 8 c h^2)),
// a = sqrt(2/pi), c = 0.044715 a.
template <int kAct>
__device__ __forceinline__ float2 act_slope_of_half(float2 h) {
  if constexpr (kAct == kActSilu) {
    const float2 t = tanh_hw2(h);
    return fma2(mul2(h, both(-0.5f)), fma2(t, t, both(-1.0f)), fma2(both(0.5f), t, both(0.5f)));
  } else if constexpr (kAct == kActGelu) {
    const float2 h2 = mul2(h, h);
    const float2 t = tanh_hw2(mul2(h, fma2(both(8.0f * kGeluC), h2, both(2.0f * kGeluA))));
    const float2 c = mul2(h, fma2(both(-12.0f * kGeluC), h2, both(-kGeluA)));
    return fma2(c, fma2(t, t, both(-1.0f)), fma2(both(0.5f), t, both(0.5f)));
  } else {
    return both(1.0f);
  }
}

// The derivative and the value, h + h t, from one tanh.  `hc` is h brought back
// to +-32 (the same h where the block's step keeps it there).
template <int kAct>
__device__ __forceinline__ float2 act_slope_and_value(float2 h, float2 hc, float2& value) {
  if constexpr (kAct == kActSilu) {
    const float2 t = tanh_hw2(hc);
    value = fma2(h, t, h);
    return fma2(mul2(hc, both(-0.5f)), fma2(t, t, both(-1.0f)), fma2(both(0.5f), t, both(0.5f)));
  } else {
    const float2 h2 = mul2(hc, hc);
    const float2 t = tanh_hw2(mul2(hc, fma2(both(8.0f * kGeluC), h2, both(2.0f * kGeluA))));
    value = fma2(h, t, h);
    const float2 c = mul2(hc, fma2(both(-12.0f * kGeluC), h2, both(-kGeluA)));
    return fma2(c, fma2(t, t, both(-1.0f)), fma2(both(0.5f), t, both(0.5f)));
  }
}

// Beyond |v| = 64 both derivatives are 0 or 1, t has long been -1 or 1 exactly,
// and v^3 may overflow, which would leave infinity times zero: such arguments
// are brought back to +-64.  (NaN stays: fminf and fmaxf would drop it.)
template <int kAct>
__device__ __forceinline__ float act_slope_safe(float v) {
  if constexpr (kAct == kActNone) return 1.0f;
  const float s = act_slope<kAct>(fminf(fmaxf(v, -64.0f), 64.0f));
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

// Whether halves of values under exponent byte b can lie outside +-32: not with a
// step of at most 1/2, nor in a block marked as not finite (NaN step).
__device__ __forceinline__ bool a8_wide(float half) { return half > 0.25f; }
__device__ __forceinline__ float2 a8_narrow(float2 h) {
  return make_float2(fminf(fmaxf(h.x, -32.0f), 32.0f), fminf(fmaxf(h.y, -32.0f), 32.0f));
}

// Halves of the values of 4 N codes, `half` the half step, brought back to +-32
// (see act_slope_safe) if kNarrow.  Where the step is at most 1/2 the subtraction and
// the product are one exact fused operation; NaN steps go the same way and stay NaN.
template <bool kNarrow, int N>
__device__ __forceinline__ void a8_decode_halves(const uint32_t (&w)[N], float half, float2 (&h)[2 * N]) {
  if (a8_wide(half)) {
#pragma unroll
    for (int i = 0; i < N; ++i) a8_decode4(w[i], half, h + 2 * i);
    if constexpr (kNarrow)
#pragma unroll
      for (int e = 0; e < 2 * N; ++e) h[e] = a8_narrow(h[e]);
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
