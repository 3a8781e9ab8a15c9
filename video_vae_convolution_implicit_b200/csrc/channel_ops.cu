// channel_ops.cu -- layer norm over the channels of each pixel (forward and
// backward) and the 8-bit activation checkpoints (written, read back through an
// affine map and an activation, and multiplied into a gradient).
//
// Every operator here reads and writes each element once with a handful of
// operations between, so HBM bounds all of them: the layouts below keep whole
// rows in registers (statistics in two passes over registers, one over memory)
// and several 16-byte loads in flight per thread.
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>

#include "act8.cuh"
#include "conv3d.h"
#include "internal.h"
#include "ptx.cuh"

namespace conv3d_channel {

using namespace conv3d;
using namespace conv3d_internal;

constexpr int kThreads = 256;

// ------------------------------------------------------------------ row groups

// A row belongs to a group of G threads: G = 8, 16 or 32 neighbouring lanes of
// a warp, or the whole block.  Thread `l` of the group holds the 8-channel
// vectors l, l + G, ..., V of them.  A walker (a warp, or a block-wide group's
// block) takes kPerWarp * R consecutive rows a step.
//
// Rows stream through a shared-memory ring by cp.async, D steps deep, each
// thread filling and reading its own slots only, so no barrier is needed: the
// bytes in flight are bounded by shared memory and not by registers (measured
// on B200 with the loads in registers: the backward pass of 104448 x 512 from
// 8 bits at 2.5 TB/s).

// Sums of N values over the threads of a group, in every thread.  Block-wide
// groups pass through `red` ([2][T/32][N] floats), whose halves alternate
// (`flip`) so that one barrier per sum is enough: a thread writes a half again
// only after the barrier of the sum in between, which every reader of the half
// has passed.
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red, int& flip) {
#pragma unroll
  for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xFFFFFFFFu, v[n], o);
  if constexpr (G > 32) {
    constexpr int kWarps = G / 32;
    float* r = red + flip * (kWarps * N);
    flip ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) r[(threadIdx.x >> 5) * N + n] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += r[w * N + n];
      v[n] = s;
    }
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// The first `bytes` of a 4-byte word; the rest of it is filled with zeros.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes = 4) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void st_global_v4(void* p, const uint4& v) { *reinterpret_cast<uint4*>(p) = v; }

// The rows of one walker.  Row r of step k is first + k * stride + r *
// kPerWarp; it exists while k < live(r), so that a step needs a 32-bit
// comparison and an addition to the running offsets.
template <int G, int R, int T>
struct Walk {
  static constexpr int kPerWarp = G < 32 ? 32 / G : 1;
  static constexpr int kStep = kPerWarp * R;
  long long first, stride;
  int steps;            // of the walker: the same in all of its threads
  int live_steps[R];
  __device__ __forceinline__ explicit Walk(long long rows) {
    const long long walker = G > 32 ? blockIdx.x : blockIdx.x * static_cast<long long>(T / 32) + threadIdx.x / 32;
    const long long walkers = static_cast<long long>(gridDim.x) * (G > 32 ? 1 : T / 32);
    const int sub = G < 32 ? (threadIdx.x % 32) / G : 0;
    first = walker * kStep + sub;
    stride = walkers * kStep;
    steps = count(rows - walker * kStep);
#pragma unroll
    for (int r = 0; r < R; ++r) live_steps[r] = count(rows - first - r * kPerWarp);
  }
  __device__ __forceinline__ int count(long long left) const {
    return left > 0 ? static_cast<int>((left + stride - 1) / stride) : 0;
  }
};

// ------------------------------------------------------------------ layer norm, forward

struct LnFwdParams {
  const uint16_t* x;
  const uint16_t* gamma;   // [C] or null (1)
  const uint16_t* beta;    // [C] or null (0)
  uint16_t* y;
  float* mean;             // [rows] or null
  float* rstd;             // [rows] or null
  uint8_t* q;              // checkpoint of (x - mean) * rstd (kCkpt)
  uint8_t* scales;
  long long rows;
  int C;
  float eps;
};

// y = xh * gamma + beta, xh = (x - mean) / sqrt(var + eps): the mean first, then
// the squared deviations from it, both from registers: no cancellation however
// far the row is off centre.  The checkpoint's 32-channel blocks are four
// neighbouring threads' vectors.  T threads a block, `kOcc` blocks an SM.
//
// Measured on B200 (bf16, graph replays): 147456 x 256 28.3 us (5.3 TB/s), 104448 x
// 512 40.5 us, with the checkpoint 50.1 (5.4), 12000 x 4096 33.8 us (5.8), 1 x 512
// 1.6 us.  Bound by HBM, with 64% of the issue slots taken under the checkpoint; odd
// channel counts leave lanes idle (16381 x 520, 65 vectors on 96: 9.4 us, 3.6 TB/s).
template <bool kBF16, int G, int V, int R, int T, int D, int kOcc, bool kCkpt>
__global__ void __launch_bounds__(T, kOcc) layernorm_fwd_kernel(const LnFwdParams p) {
  using H = Val16<kBF16>;
  constexpr uint32_t kSlot = R * V * T * 16;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ float red[G > 32 ? 2 * (T / 32) * R : 1];
  int flip = 0;
  const int l = threadIdx.x % G;
  const int vecs = p.C / 8;
  const int nb = (p.C + 31) / 32;
  const float inv_c = 1.0f / static_cast<float>(p.C);
  const Walk<G, R, T> walk(p.rows);
  const uint32_t ring = smem_addr(ring_mem) + threadIdx.x * 16u;
  bool in[V];
#pragma unroll
  for (int i = 0; i < V; ++i) in[i] = l + i * G < vecs;
  griddep_wait();
  griddep_launch_dependents();
  // byte offsets of this thread's first vector in x and y, now and of the next fetch
  const long long first = (walk.first * p.C + l * 8) * 2, advance = walk.stride * p.C * 2;
  const int per_row = Walk<G, R, T>::kPerWarp * p.C * 2;
  const char* next = reinterpret_cast<const char*>(p.x) + first;
  auto fetch = [&](int k, int slot) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (k < walk.live_steps[r])
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (in[i]) cp_async16(ring + slot * kSlot + (r * V + i) * (T * 16), next + r * per_row + i * (G * 16));
    next += advance;
    cp_async_commit();   // one group per step, empty ones included, so the count stays fixed
  };
#pragma unroll
  for (int k = 0; k < D - 1; ++k) fetch(k, k);
  float2 gm[V][4], bt[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gm[i][e] = both(1.0f);
      bt[i][e] = both(0.0f);
    }
    if (p.gamma && in[i]) H::unpack8(__ldg(reinterpret_cast<const uint4*>(p.gamma) + l + i * G), gm[i]);
    if (p.beta && in[i]) H::unpack8(__ldg(reinterpret_cast<const uint4*>(p.beta) + l + i * G), bt[i]);
  }
  char* out = reinterpret_cast<char*>(p.y) + first;
  long long row0 = walk.first;
  int slot = 0;
  for (int k = 0; k < walk.steps; ++k) {
    // the slot of the step before this one was read into registers then: refill it
    fetch(k + D - 1, slot == 0 ? D - 1 : slot - 1);
    cp_async_wait<D - 1>();
    float2 d[R][V][4];
    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 a = both(0.0f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (in[i] && k < walk.live_steps[r]) raw = ld_shared_v4(ring + slot * kSlot + (r * V + i) * (T * 16));
        H::unpack8(raw, d[r][i]);
        a = add2(a, add2(add2(d[r][i][0], d[r][i][1]), add2(d[r][i][2], d[r][i][3])));
      }
      s[r] = a.x + a.y;
    }
    slot = slot == D - 1 ? 0 : slot + 1;
    group_sum<G, R>(s, red, flip);
    float mean[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = s[r] * inv_c;
      float2 a = both(0.0f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float2 sq = both(0.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          d[r][i][e] = add2(d[r][i][e], both(-mean[r]));
          sq = fma2(d[r][i][e], d[r][i][e], sq);
        }
        if (in[i]) a = add2(a, sq);
      }
      s[r] = a.x + a.y;
    }
    group_sum<G, R>(s, red, flip);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool live = k < walk.live_steps[r];
      const long long row = row0 + r * Walk<G, R, T>::kPerWarp;
      const float rstd = rsqrtf(fmaf(s[r], inv_c, p.eps));
      if (l == 0 && live) {
        if (p.mean) p.mean[row] = mean[r];
        if (p.rstd) p.rstd[row] = rstd;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float2(&f)[4] = d[r][i];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = mul2(f[e], both(rstd));
        if constexpr (kCkpt) {
          const int c = l + i * G;
          uint32_t mag = a8_mag8(f);
          if (!in[i]) mag = 0u;
          mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 1));
          mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 2));
          const uint32_t b = a8_exponent(mag);
          const float inv = a8_inv_step(b);
          if (c < nb * 4 && live) {
            uint2 q = make_uint2(0, 0);   // zero codes behind the last channel
            if (in[i]) q = make_uint2(a8_code4(f[0], f[1], inv), a8_code4(f[2], f[3], inv));
            *reinterpret_cast<uint2*>(p.q + (row * nb * 4 + c) * 8) = q;
            if ((c & 3) == 0) p.scales[row * nb + (c >> 2)] = static_cast<uint8_t>(b);
          }
        }
        if (in[i] && live) {
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = fma2(f[e], gm[i][e], bt[i][e]);
          st_global_v4(out + r * per_row + i * (G * 16), H::pack8(f));
        }
      }
    }
    out += advance;
    row0 += walk.stride;
  }
  cp_async_wait<0>();
}

// ------------------------------------------------------------------ layer norm, backward

struct LnBwdParams {
  const uint16_t* dy;
  const uint16_t* x;        // with mean, or
  const uint8_t* q;         // the checkpoint of xh
  const uint8_t* scales;
  const float* mean;
  const float* rstd;
  const uint16_t* gamma;    // [C] or null (1)
  const uint16_t* dres;     // added to dx, or null
  uint16_t* dx;
  float* part;              // [blocks][2][C] partial {dgamma, dbeta}, or null
  long long rows;
  int C;
};

// Shared bytes per thread of one ring step: dy, then x or the codes, then dres
// (when there is one), then rstd, then the mean or the words that hold the
// vectors' exponent bytes.
__host__ __device__ constexpr int ln_bwd_src_bytes(bool ckpt) { return ckpt ? 8 : 16; }
__host__ __device__ constexpr int ln_bwd_step_bytes(int V, int R, bool ckpt, bool dres) {
  return R * (V * (16 + ln_bwd_src_bytes(ckpt) + (dres ? 16 : 0)) + 4 + (ckpt ? 4 * V : 4));
}

// dx = rstd * (g - mean(g) - xh * mean(g * xh)) + dres, g = dy * gamma, and
// each thread's share of dgamma = sum dy * xh and dbeta = sum dy for its own
// channels, kept in fp32 registers over all of its rows; at the end the
// block's groups are added in a fixed tree and the block writes one partial,
// which layernorm_param_kernel adds up in block order: no atomics, so the
// result does not depend on timing.
//
// Measured on B200, both kernels: 104448 x 512 from x 61.0 us (5.3 TB/s), from 8
// bits with dres 69.2 us (5.4), 147456 x 256 39.4 and 47.6 us (5.8 and 5.6), 50000 x
// 1024 51.8 us (5.9), 16381 x 520 fp16 19.3 us (2.6): there the second kernel and
// the start and the end of the first are 8 us of it.  Bound by HBM; rows of 4096
// and more, one or two blocks an SM, reach 4.2 to 4.8 TB/s.
template <bool kBF16, int G, int V, int R, int T, int D, int kOcc, bool kCkpt>
__global__ void __launch_bounds__(T, kOcc) layernorm_bwd_kernel(const LnBwdParams p) {
  using H = Val16<kBF16>;
  constexpr int kWarps = T / 32;
  constexpr int kPerWarp = Walk<G, R, T>::kPerWarp;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ float red[G > 32 ? 2 * (T / 32) * 2 * R : 1];
  int flip = 0;
  const int l = threadIdx.x % G;
  const int vecs = p.C / 8;
  const int nb = (p.C + 31) / 32;
  const float inv_c = 1.0f / static_cast<float>(p.C);
  const bool has_res = p.dres != nullptr;
  const Walk<G, R, T> walk(p.rows);
  // the parts of a ring step
  constexpr uint32_t kSrc = ln_bwd_src_bytes(kCkpt);
  const uint32_t base = smem_addr(ring_mem);
  const uint32_t step_bytes = has_res ? ln_bwd_step_bytes(V, R, kCkpt, true) * T : ln_bwd_step_bytes(V, R, kCkpt, false) * T;
  constexpr uint32_t kDyEnd = R * V * T * 16;
  constexpr uint32_t kSrcEnd = kDyEnd + R * V * T * kSrc;
  const uint32_t res_end = kSrcEnd + (has_res ? kDyEnd : 0u);
  bool in[V];
#pragma unroll
  for (int i = 0; i < V; ++i) in[i] = l + i * G < vecs;
  float2 dg[V][4], db[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) dg[i][e] = db[i][e] = both(0.0f);
  griddep_wait();
  griddep_launch_dependents();
  const long long scale_bytes = p.rows * nb;
  // running byte offsets: the 16-bit tensors share one, the codes' is its own
  const long long first = (walk.first * p.C + l * 8) * 2, advance = walk.stride * p.C * 2;
  const int per_row = kPerWarp * p.C * 2;
  long long ahead = first;
  const uint8_t* codes = kCkpt ? p.q + walk.first * nb * 32 + l * 8 : nullptr;
  long long row_ahead = walk.first;
  auto fetch = [&](int k, int slot) {
    const uint32_t s = base + slot * step_bytes;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (k < walk.live_steps[r]) {
        const long long row = row_ahead + r * kPerWarp;
        cp_async4(s + res_end + (r * T + threadIdx.x) * 4u, p.rstd + row);
        if constexpr (!kCkpt) cp_async4(s + res_end + ((R + r) * T + threadIdx.x) * 4u, p.mean + row);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (in[i]) {
            const uint32_t at = (r * V + i) * T + threadIdx.x;
            const long long off = ahead + r * per_row + i * (G * 16);
            cp_async16(s + at * 16u, reinterpret_cast<const char*>(p.dy) + off);
            if (has_res) cp_async16(s + kSrcEnd + at * 16u, reinterpret_cast<const char*>(p.dres) + off);
            if constexpr (kCkpt) {
              cp_async8(s + kDyEnd + at * 8u, codes + r * (kPerWarp * nb * 32) + i * (G * 8));
              // the aligned word that holds the exponent byte, short of the buffer's end
              const long long e = (row * nb + ((l + i * G) >> 2)) & ~3LL;
              const long long left = scale_bytes - e;
              cp_async4(s + res_end + (R * T + at) * 4u, p.scales + e, left < 4 ? static_cast<uint32_t>(left) : 4u);
            } else {
              cp_async16(s + kDyEnd + at * 16u, reinterpret_cast<const char*>(p.x) + off);
            }
          }
        }
      }
    }
    ahead += advance;
    if constexpr (kCkpt) codes += walk.stride * nb * 32;
    row_ahead += walk.stride;
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < D - 1; ++k) fetch(k, k);
  float2 gm[V][4];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) gm[i][e] = both(1.0f);
    if (p.gamma && in[i]) H::unpack8(__ldg(reinterpret_cast<const uint4*>(p.gamma) + l + i * G), gm[i]);
  }
  char* out_dx = reinterpret_cast<char*>(p.dx) + first;
  uint32_t row_nb = static_cast<uint32_t>(walk.first * nb);   // low bits of row * nb: the exponent byte's place
  int slot = 0;
  for (int k = 0; k < walk.steps; ++k) {
    fetch(k + D - 1, slot == 0 ? D - 1 : slot - 1);
    cp_async_wait<D - 1>();
    const uint32_t s = base + slot * step_bytes;
    float2 g[R][V][4], xh[R][V][4];
    float rstd[R], c12[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool live = k < walk.live_steps[r];
      rstd[r] = live ? __uint_as_float(ld_shared_u32(s + res_end + (r * T + threadIdx.x) * 4u)) : 0.0f;
      float mean = 0.0f;
      if constexpr (!kCkpt)
        mean = live ? __uint_as_float(ld_shared_u32(s + res_end + ((R + r) * T + threadIdx.x) * 4u)) : 0.0f;
      float2 a = both(0.0f), b = both(0.0f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t at = (r * V + i) * T + threadIdx.x;
        if (live && in[i]) {
          H::unpack8(ld_shared_v4(s + at * 16u), g[r][i]);
          if constexpr (kCkpt) {
            const uint32_t word = ld_shared_u32(s + res_end + (R * T + at) * 4u);
            const uint32_t byte = (row_nb + static_cast<uint32_t>(r * kPerWarp * nb + ((l + i * G) >> 2))) & 3u;
            const float step = a8_step((word >> (8u * byte)) & 0xFFu);
            const uint2 q = ld_shared_v2(s + kDyEnd + at * 8u);
            a8_decode4(q.x, step, xh[r][i]);
            a8_decode4(q.y, step, xh[r][i] + 2);
          } else {
            H::unpack8(ld_shared_v4(s + kDyEnd + at * 16u), xh[r][i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) xh[r][i][e] = mul2(add2(xh[r][i][e], both(-mean)), both(rstd[r]));
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 dy = g[r][i][e];
            db[i][e] = add2(db[i][e], dy);
            dg[i][e] = fma2(dy, xh[r][i][e], dg[i][e]);
            g[r][i][e] = mul2(dy, gm[i][e]);
            a = add2(a, g[r][i][e]);
            b = fma2(g[r][i][e], xh[r][i][e], b);
          }
        }
      }
      c12[2 * r] = a.x + a.y;
      c12[2 * r + 1] = b.x + b.y;
    }
    group_sum<G, 2 * R>(c12, red, flip);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // dx = rstd * g - rstd * c1 - xh * (rstd * c2)
      const float2 k1 = both(-rstd[r] * (c12[2 * r] * inv_c)), k2 = both(-rstd[r] * (c12[2 * r + 1] * inv_c));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (k < walk.live_steps[r] && in[i]) {
          float2 o[4];
          if (has_res) {
            H::unpack8(ld_shared_v4(s + kSrcEnd + ((r * V + i) * T + threadIdx.x) * 16u), o);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[e] = add2(o[e], fma2(g[r][i][e], both(rstd[r]), fma2(xh[r][i][e], k2, k1)));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fma2(g[r][i][e], both(rstd[r]), fma2(xh[r][i][e], k2, k1));
          }
          st_global_v4(out_dx + r * per_row + i * (G * 16), H::pack8(o));
        }
      }
    }
    out_dx += advance;
    row_nb += static_cast<uint32_t>(walk.stride * nb);
    slot = slot == D - 1 ? 0 : slot + 1;
  }
  cp_async_wait<0>();
  if (p.part == nullptr) return;
  float* out = p.part + static_cast<size_t>(blockIdx.x) * 2 * p.C;
  if constexpr (G <= 32) {
    // lanes that hold the same channels, then the warps by halves through the
    // ring's memory ([kWarps / 2][2][C] floats), which nobody fills any more
    float* fold = reinterpret_cast<float*>(ring_mem);
    __syncthreads();
#pragma unroll
    for (int o = G; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dg[i][e].x += __shfl_xor_sync(0xFFFFFFFFu, dg[i][e].x, o);
          dg[i][e].y += __shfl_xor_sync(0xFFFFFFFFu, dg[i][e].y, o);
          db[i][e].x += __shfl_xor_sync(0xFFFFFFFFu, db[i][e].x, o);
          db[i][e].y += __shfl_xor_sync(0xFFFFFFFFu, db[i][e].y, o);
        }
    const int warp = threadIdx.x / 32;
    const bool holds = threadIdx.x % 32 < G;
    for (int half = kWarps / 2; half > 0; half >>= 1) {
      if (holds && warp >= half && warp < 2 * half)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (l + i * G < vecs) {
            float4* f = reinterpret_cast<float4*>(fold + (static_cast<size_t>(warp - half) * 2) * p.C + (l + i * G) * 8);
            f[0] = make_float4(dg[i][0].x, dg[i][0].y, dg[i][1].x, dg[i][1].y);
            f[1] = make_float4(dg[i][2].x, dg[i][2].y, dg[i][3].x, dg[i][3].y);
            f += p.C / 4;
            f[0] = make_float4(db[i][0].x, db[i][0].y, db[i][1].x, db[i][1].y);
            f[1] = make_float4(db[i][2].x, db[i][2].y, db[i][3].x, db[i][3].y);
          }
      __syncthreads();
      if (holds && warp < half)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (l + i * G < vecs) {
            const float2* f = reinterpret_cast<const float2*>(fold + (static_cast<size_t>(warp) * 2) * p.C + (l + i * G) * 8);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              dg[i][e] = add2(dg[i][e], f[e]);
              db[i][e] = add2(db[i][e], f[p.C / 2 + e]);
            }
          }
      __syncthreads();
    }
    if (warp != 0 || !holds) return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = l + i * G;
    if (c < vecs) {
      float4* o = reinterpret_cast<float4*>(out + c * 8);
      o[0] = make_float4(dg[i][0].x, dg[i][0].y, dg[i][1].x, dg[i][1].y);
      o[1] = make_float4(dg[i][2].x, dg[i][2].y, dg[i][3].x, dg[i][3].y);
      o = reinterpret_cast<float4*>(out + p.C + c * 8);
      o[0] = make_float4(db[i][0].x, db[i][0].y, db[i][1].x, db[i][1].y);
      o[1] = make_float4(db[i][2].x, db[i][2].y, db[i][3].x, db[i][3].y);
    }
  }
}

// Adds the blocks' partials of 32 of the 2C sums per block: warp w takes the
// partials w, w + 32, ... in order, then the 32 warps' sums are added in order.
// (Measured with 8, 16 and 32 warps and 7 to 28 loads of a thread in flight: 16381 x
// 520, both kernels, 18.5 us with these, 18.9 with 32 x 10, 20 with 8 x 28.)
constexpr int kParamWarps = 32, kParamBatch = 7;
template <bool kBF16>
__global__ void __launch_bounds__(32 * kParamWarps) layernorm_param_kernel(const float* __restrict__ part, int blocks,
                                                               int C, uint16_t* dgamma, uint16_t* dbeta) {
  __shared__ float s[kParamWarps][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31);
  const int w = threadIdx.x >> 5;
  griddep_wait();
  griddep_launch_dependents();
  float a = 0.0f;
  if (col < 2 * C)
    for (int b = w; b < blocks; b += kParamWarps * kParamBatch) {
      float v[kParamBatch];
#pragma unroll
      for (int k = 0; k < kParamBatch; ++k)
        v[k] = b + kParamWarps * k < blocks ? __ldcg(part + static_cast<size_t>(b + kParamWarps * k) * 2 * C + col) : 0.0f;
#pragma unroll
      for (int k = 0; k < kParamBatch; ++k) a += v[k];
    }
  s[w][threadIdx.x & 31] = a;
  __syncthreads();
  if (w == 0 && col < 2 * C) {
    a = 0.0f;
#pragma unroll
    for (int k = 0; k < kParamWarps; ++k) a += s[k][threadIdx.x];
    const uint16_t v = static_cast<uint16_t>(Val16<kBF16>::pack(a, 0.0f) & 0xFFFFu);
    if (col < C) {
      if (dgamma) dgamma[col] = v;
    } else if (dbeta) {
      dbeta[col - C] = v;
    }
  }
}

// ------------------------------------------------------------------ 8-bit checkpoints

// The streaming kernels walk units of 16 channels (two neighbouring threads a
// 32-channel block) or 8: unit u of the flat index is row u / units, and unit
// u % units of the row's padded channels.  A thread's first unit is found by
// division and the next ones by adding the grid stride's quotient and remainder.
struct UnitWalk {
  long long row, drow;
  int v, dv, units;
  __device__ __forceinline__ UnitWalk(long long u, long long stride, int units_) : units(units_) {
    row = u / units;
    v = static_cast<int>(u - row * units);
    drow = stride / units;
    dv = static_cast<int>(stride - drow * units);
  }
  __device__ __forceinline__ void next() {
    row += drow;
    v += dv;
    if (v >= units) {
      v -= units;
      ++row;
    }
  }
};

constexpr int kUnroll = 4;   // units in flight per thread

// Measured on B200 (bf16, graph replays): 36864 x 2048 written 36 us (6.3 TB/s), read
// 39 (5.9), read through SiLU 48 (4.8), through GELU 50 (4.6), through gamma, beta and
// SiLU 54 (4.2), dy times GELU' 72 (5.3); 1000 x 136 2 us.  Bound by HBM, under an
// activation also by its two special functions a value (34 us of that unit's time here)
// and by issue.

template <bool kBF16>
__global__ void __launch_bounds__(kThreads) act8_pack_kernel(const uint16_t* __restrict__ x, uint8_t* __restrict__ q,
                                                             uint8_t* __restrict__ scales, long long total,
                                                             int units, int C) {
  using T = Val16<kBF16>;
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  long long u = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x;
  UnitWalk w(u, stride, units);
  griddep_wait();
  griddep_launch_dependents();
  // a warp's units end together (total is even and its lanes are consecutive), so the
  // exchange below always has both threads of a block
  for (long long u0 = u - (threadIdx.x & 31); u0 < total; u0 += kUnroll * stride) {
    uint4 a[kUnroll], b[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k, w.next()) {
      const long long uk = u0 + (threadIdx.x & 31) + k * stride;
      const uint16_t* src = x + w.row * C + w.v * 16;
      a[k] = b[k] = make_uint4(0, 0, 0, 0);
      if (uk < total && w.v * 16 < C) a[k] = *reinterpret_cast<const uint4*>(src);
      if (uk < total && w.v * 16 + 8 < C) b[k] = *reinterpret_cast<const uint4*>(src + 8);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const long long uk = u0 + (threadIdx.x & 31) + k * stride;
      float2 f[4], g[4];
      T::unpack8(a[k], f);
      T::unpack8(b[k], g);
      uint32_t mag = max(a8_mag8(f), a8_mag8(g));
      mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 1));
      const uint32_t eb = a8_exponent(mag);
      const float inv = a8_inv_step(eb);
      if (uk < total) {
        *reinterpret_cast<uint4*>(q + uk * 16) =
            make_uint4(a8_code4(f[0], f[1], inv), a8_code4(f[2], f[3], inv), a8_code4(g[0], g[1], inv),
                       a8_code4(g[2], g[3], inv));
        if ((uk & 1) == 0) scales[uk >> 1] = static_cast<uint8_t>(eb);
      }
    }
  }
}

struct ReadParams {
  const uint8_t* q;
  const uint8_t* scales;
  const uint16_t* gamma;   // unpack: [C] or null
  const uint16_t* beta;
  const uint16_t* dy;      // gradient: out = dy * act'(v); unpack: null
  uint16_t* out;
  long long total;
  int units, C;
};

// kPlain: out = act(v); kAffine: out = act(v * gamma + beta); kGrad: out = dy * act'(v).
// Units of 8 channels here: the 16-bit side, two thirds and more of the bytes,
// is then one contiguous 512-byte access a warp.
enum class Read { kPlain, kAffine, kGrad };

template <bool kBF16, int kAct, Read kMode>
__global__ void __launch_bounds__(kThreads, kMode == Read::kGrad ? 3 : 4) act8_read_kernel(const ReadParams p) {
  using T = Val16<kBF16>;
  constexpr bool kGrad = kMode == Read::kGrad;
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  long long u = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x;
  UnitWalk w(u, stride, p.units);
  griddep_wait();
  griddep_launch_dependents();
  // gamma and beta of this thread's channels; the host makes the stride a
  // multiple of a row where it can, and then they stay the same
  float2 g[4], b[4];
  int of = -1;
  for (; u < p.total; u += kUnroll * stride) {
    uint2 k[kUnroll];
    uint4 d[kUnroll];
    uint32_t eb[kUnroll];
    long long row[kUnroll];
    int c[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j, w.next()) {
      const long long uj = u + j * stride;
      row[j] = w.row;
      c[j] = uj < p.total ? w.v * 8 : p.C;                    // p.C: nothing to do
      if (c[j] < p.C) {
        k[j] = __ldg(reinterpret_cast<const uint2*>(p.q) + uj);
        eb[j] = __ldg(p.scales + (uj >> 2));
        if constexpr (kGrad) d[j] = *reinterpret_cast<const uint4*>(p.dy + row[j] * p.C + c[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      if (c[j] >= p.C) continue;
      float2 v[4];
      if constexpr (kGrad) {
        float2 dy[4];
        T::unpack8(d[j], dy);
        if constexpr (kAct != kActNone) {
          const uint32_t w[2] = {k[j].x, k[j].y};
          a8_decode_halves<kAct, true>(w, 0.5f * a8_step(eb[j]), v);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = mul2(dy[e], act_slope_of_half<kAct>(v[e]));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = dy[e];
        }
      } else {
        const float step = a8_step(eb[j]);
        a8_decode4(k[j].x, step, v);
        a8_decode4(k[j].y, step, v + 2);
        if constexpr (kMode == Read::kAffine) {
          if (c[j] != of) {
            of = c[j];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              g[e] = both(1.0f);
              b[e] = both(0.0f);
            }
            if (p.gamma) T::unpack8(__ldg(reinterpret_cast<const uint4*>(p.gamma + of)), g);
            if (p.beta) T::unpack8(__ldg(reinterpret_cast<const uint4*>(p.beta + of)), b);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = fma2(v[e], g[e], b[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = act_value<kAct>(v[e]);
      }
      *reinterpret_cast<uint4*>(p.out + row[j] * p.C + c[j]) = T::pack8(v);
    }
  }
}

// ------------------------------------------------------------------ host

constexpr int kMaxLnChannels = 8192;
// Blocks of the backward kernel: two per SM of a 148-SM part; each leaves one
// partial of 2C floats.
constexpr int kLnBwdBlocks = 296;

conv3d_status_t check_sizes(long long rows, int C, conv3d_dtype_t dtype, int max_c) {
  if (rows < 1 || C < 1) {
    set_error("sizes must be >= 1");
    return CONV3D_ERR_INVALID_ARG;
  }
  if (dtype != CONV3D_F16 && dtype != CONV3D_BF16) {
    set_error("unknown dtype %d", static_cast<int>(dtype));
    return CONV3D_ERR_INVALID_ARG;
  }
  if (C % 8 != 0 || C > max_c) {
    set_error("channels must be a multiple of 8 and at most %d (got %d)", max_c, C);
    return CONV3D_ERR_UNSUPPORTED;
  }
  if (rows > LLONG_MAX / 4 / C) {
    set_error("problem too large");
    return CONV3D_ERR_UNSUPPORTED;
  }
  return CONV3D_OK;
}

conv3d_status_t misaligned() {
  set_error("tensor pointers must be 16-byte aligned, and mean and rstd 4-byte aligned");
  return CONV3D_ERR_ALIGNMENT;
}

conv3d_status_t overlapping(const char* what) {
  set_error("%s", what);
  return CONV3D_ERR_INVALID_ARG;
}

unsigned blocks_for(long long work, long long per_block, long long cap) {
  long long b = (work + per_block - 1) / per_block;
  if (b > cap) b = cap;
  return static_cast<unsigned>(b < 1 ? 1 : b);
}

// Rows per step of a block.
constexpr int rows_per_step(int G, int R, int T) { return G > 32 ? R : (T / 32) * (32 / G) * R; }

template <typename K>
cudaError_t allow_smem(K kern, std::atomic<unsigned long long>& done, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

template <bool kBF16, int G, int V, int R, int T, int D, int kOcc, bool kCkpt>
cudaError_t run_fwd(const LnFwdParams& p, int sms, cudaStream_t stream) {
  static std::atomic<unsigned long long> ready{0};
  auto kern = layernorm_fwd_kernel<kBF16, G, V, R, T, D, kOcc, kCkpt>;
  const unsigned blocks = blocks_for(p.rows, rows_per_step(G, R, T), static_cast<long long>(sms) * kOcc);
  const size_t smem = static_cast<size_t>(D) * R * V * T * 16;
  const cudaError_t e = allow_smem(kern, ready, smem);
  if (e != cudaSuccess) return e;
  return launch(kern, blocks, T, smem, 1, stream, p);
}

// The narrowest group and vector count that hold a row.
template <bool kBF16, bool kCkpt>
cudaError_t dispatch_fwd(const LnFwdParams& p, int sms, cudaStream_t stream) {
  const int vecs = p.C / 8;
  if (vecs <= 8) return run_fwd<kBF16, 8, 1, 2, 256, 8, 3, kCkpt>(p, sms, stream);
  if (vecs <= 16) return run_fwd<kBF16, 8, 2, 1, 256, 8, 3, kCkpt>(p, sms, stream);
  if (vecs <= 32) return run_fwd<kBF16, 16, 2, 1, 256, 8, 3, kCkpt>(p, sms, stream);
  if (vecs <= 64) return run_fwd<kBF16, 32, 2, 1, 256, 8, 3, kCkpt>(p, sms, stream);
  if (vecs <= 96) return run_fwd<kBF16, 32, 3, 1, 256, 5, 2, kCkpt>(p, sms, stream);
  if (vecs <= 128) return run_fwd<kBF16, 128, 1, 4, 128, 4, 5, kCkpt>(p, sms, stream);
  if (vecs <= 256) return run_fwd<kBF16, 256, 1, 4, 256, 4, 2, kCkpt>(p, sms, stream);
  if (vecs <= 512) return run_fwd<kBF16, 256, 2, 1, 256, 8, 3, kCkpt>(p, sms, stream);
  return run_fwd<kBF16, 512, 2, 1, 512, 8, 1, kCkpt>(p, sms, stream);
}

// The ring is as deep as shared memory allows kOcc blocks an SM, which differs
// with and without dres.
template <bool kBF16, int G, int V, int R, int T, int D, int kOcc, bool kCkpt>
cudaError_t run_bwd_depth(const LnBwdParams& p, unsigned blocks, cudaStream_t stream) {
  static std::atomic<unsigned long long> ready{0};
  auto kern = layernorm_bwd_kernel<kBF16, G, V, R, T, D, kOcc, kCkpt>;
  size_t smem = static_cast<size_t>(D) * ln_bwd_step_bytes(V, R, kCkpt, p.dres != nullptr) * T;
  if constexpr (G <= 32) {   // the block's fold of its groups
    const size_t fold = static_cast<size_t>(T / 64) * 2 * p.C * sizeof(float);
    if (smem < fold) smem = fold;
  }
  const cudaError_t e = allow_smem(kern, ready, smem);
  if (e != cudaSuccess) return e;
  return launch(kern, blocks, T, smem, 1, stream, p);
}

template <bool kBF16, int G, int V, int R, int T, int D, int DRes, int kOcc, bool kCkpt>
cudaError_t run_bwd(const LnBwdParams& p, unsigned blocks, cudaStream_t stream) {
  static_assert(static_cast<size_t>(D) * ln_bwd_step_bytes(V, R, false, false) * T * kOcc <= 224 * 1024 &&
                    static_cast<size_t>(DRes) * ln_bwd_step_bytes(V, R, false, true) * T * kOcc <= 224 * 1024,
                "the ring of every block of an SM fits its shared memory");
  return p.dres ? run_bwd_depth<kBF16, G, V, R, T, DRes, kOcc, kCkpt>(p, blocks, stream)
                : run_bwd_depth<kBF16, G, V, R, T, D, kOcc, kCkpt>(p, blocks, stream);
}

unsigned bwd_blocks(long long rows, int C) {
  const int vecs = C / 8;
  const int per = vecs <= 8    ? rows_per_step(8, 2, 256)
                  : vecs <= 16 ? rows_per_step(8, 1, 256)
                  : vecs <= 32 ? rows_per_step(16, 1, 256)
                  : vecs <= 64 ? rows_per_step(32, 1, 256)
                  : vecs <= 128 ? rows_per_step(32, 1, 128)
                                : rows_per_step(256, 1, 256);
  // blocks of 128 threads: more of them fit an SM
  const int blocks = vecs > 128 && vecs <= 256 ? 2 * kLnBwdBlocks : vecs > 64 && vecs <= 96 ? 3 * kLnBwdBlocks / 2 : kLnBwdBlocks;
  return blocks_for(rows, per, blocks);
}

template <bool kBF16, bool kCkpt>
cudaError_t dispatch_bwd(const LnBwdParams& p, unsigned blocks, cudaStream_t stream) {
  const int vecs = p.C / 8;
  if (vecs <= 8) return run_bwd<kBF16, 8, 1, 2, 256, 5, 3, 2, kCkpt>(p, blocks, stream);
  if (vecs <= 16) return run_bwd<kBF16, 8, 2, 1, 256, 6, 4, 2, kCkpt>(p, blocks, stream);
  if (vecs <= 32) return run_bwd<kBF16, 16, 2, 1, 256, 6, 4, 2, kCkpt>(p, blocks, stream);
  if (vecs <= 64) return run_bwd<kBF16, 32, 2, 1, 256, 6, 4, 2, kCkpt>(p, blocks, stream);
  if (vecs <= 96) return run_bwd<kBF16, 32, 3, 1, 128, 5, 3, 3, kCkpt>(p, blocks, stream);
  if (vecs <= 128) return run_bwd<kBF16, 32, 4, 1, 128, 6, 4, 2, kCkpt>(p, blocks, stream);
  if (vecs <= 256) return run_bwd<kBF16, 128, 2, 1, 128, 6, 4, 4, kCkpt>(p, blocks, stream);
  if (vecs <= 512) return run_bwd<kBF16, 256, 2, 1, 256, 6, 4, 2, kCkpt>(p, blocks, stream);
  return run_bwd<kBF16, 256, 4, 1, 256, 6, 4, 1, kCkpt>(p, blocks, stream);
}

template <bool kBF16, Read kMode>
cudaError_t dispatch_read(int act, unsigned blocks, cudaStream_t stream, const ReadParams& p) {
  if (act == kActSilu) return launch(act8_read_kernel<kBF16, kActSilu, kMode>, blocks, kThreads, 0, 1, stream, p);
  if (act == kActGelu) return launch(act8_read_kernel<kBF16, kActGelu, kMode>, blocks, kThreads, 0, 1, stream, p);
  return launch(act8_read_kernel<kBF16, kActNone, kMode>, blocks, kThreads, 0, 1, stream, p);
}

template <bool kBF16>
cudaError_t dispatch_read(Read mode, int act, unsigned blocks, cudaStream_t stream, const ReadParams& p) {
  if (mode == Read::kGrad) return dispatch_read<kBF16, Read::kGrad>(act, blocks, stream, p);
  if (mode == Read::kAffine) return dispatch_read<kBF16, Read::kAffine>(act, blocks, stream, p);
  return dispatch_read<kBF16, Read::kPlain>(act, blocks, stream, p);
}

constexpr int kMaxAct8Channels = 1 << 24;

// Units of `channels` channels per row, whose last block is padded.
int units_per_row(int C, int channels) { return (32 / channels) * ((C + 31) / 32); }

}  // namespace conv3d_channel

using namespace conv3d_channel;

extern "C" {

conv3d_status_t conv3d_layernorm_fwd(const void* x, const void* gamma, const void* beta, void* y,
                                     float* mean, float* rstd, void* codes, void* exponents,
                                     long long rows, int C, float eps, conv3d_dtype_t dtype,
                                     struct CUstream_st* stream) {
  conv3d_status_t st = check_sizes(rows, C, dtype, kMaxLnChannels);
  if (st != CONV3D_OK) return st;
  if (!x || !y || !(eps >= 0.0f) || (codes == nullptr) != (exponents == nullptr)) {
    set_error("x and y must be non-null, eps >= 0, and codes and exponents given together");
    return CONV3D_ERR_INVALID_ARG;
  }
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(gamma, 16) || !aligned(beta, 16) ||
      !aligned(codes, 16) || !aligned(exponents, 16) || !aligned(mean, 4) || !aligned(rstd, 4))
    return misaligned();
  const size_t n = static_cast<size_t>(rows) * C * 2, cb = act8_code_bytes(rows, C),
               sb = act8_scale_bytes(rows, C), rb = static_cast<size_t>(rows) * 4, pb = C * 2ull;
  const struct { const void* p; size_t n; } outs[] = {{y, n}, {codes, cb}, {exponents, sb}, {mean, rb}, {rstd, rb}},
                                            ins[] = {{x, n}, {gamma, pb}, {beta, pb}};
  bool clash = false;
  for (const auto& o : outs) {
    for (const auto& i : ins) clash = clash || (overlaps(o.p, o.n, i.p, i.n) && !(o.p == y && i.p == x && x == y));
    for (const auto& q : outs) clash = clash || (&o != &q && overlaps(o.p, o.n, q.p, q.n));
  }
  if (clash)
    return overlapping("y must be exactly x or not overlap it; the other outputs must overlap nothing");
  Device dev;
  if ((st = current_device(dev)) != CONV3D_OK) return st;
  LnFwdParams p{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(gamma),
                static_cast<const uint16_t*>(beta), static_cast<uint16_t*>(y), mean, rstd,
                static_cast<uint8_t*>(codes), static_cast<uint8_t*>(exponents), rows, C, eps};
  const bool bf16 = dtype == CONV3D_BF16;
  const cudaError_t e = codes ? (bf16 ? dispatch_fwd<true, true>(p, dev.num_sms, stream)
                                      : dispatch_fwd<false, true>(p, dev.num_sms, stream))
                              : (bf16 ? dispatch_fwd<true, false>(p, dev.num_sms, stream)
                                      : dispatch_fwd<false, false>(p, dev.num_sms, stream));
  return e == cudaSuccess ? CONV3D_OK : cuda_fail(e, "layer norm launch");
}

size_t conv3d_layernorm_bwd_workspace_bytes(long long rows, int C) {
  if (rows < 1 || C < 8 || C > kMaxLnChannels) return 0;
  const size_t b = static_cast<size_t>(bwd_blocks(rows, C)) * 2 * C * sizeof(float);
  return (b + 255) & ~static_cast<size_t>(255);
}

conv3d_status_t conv3d_layernorm_bwd(const void* dy, const void* x, const float* mean,
                                     const void* codes, const void* exponents, const float* rstd,
                                     const void* gamma, const void* dres, void* dx, void* dgamma,
                                     void* dbeta, long long rows, int C, conv3d_dtype_t dtype,
                                     void* workspace, size_t ws_bytes, struct CUstream_st* stream) {
  conv3d_status_t st = check_sizes(rows, C, dtype, kMaxLnChannels);
  if (st != CONV3D_OK) return st;
  if (!dy || !dx || !rstd) {
    set_error("dy, dx and rstd must be non-null");
    return CONV3D_ERR_INVALID_ARG;
  }
  const bool from_x = x != nullptr && mean != nullptr, from_codes = codes != nullptr && exponents != nullptr;
  if (from_x == from_codes || (x != nullptr) != (mean != nullptr) ||
      (codes != nullptr) != (exponents != nullptr)) {
    set_error("either x and mean or codes and exponents must be given");
    return CONV3D_ERR_INVALID_ARG;
  }
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(codes, 16) || !aligned(exponents, 16) ||
      !aligned(gamma, 16) || !aligned(dres, 16) || !aligned(dx, 16) || !aligned(dgamma, 16) ||
      !aligned(dbeta, 16) || !aligned(mean, 4) || !aligned(rstd, 4))
    return misaligned();
  const bool params = dgamma != nullptr || dbeta != nullptr;
  const size_t need = params ? conv3d_layernorm_bwd_workspace_bytes(rows, C) : 0;
  if (params && (workspace == nullptr || ws_bytes < need)) {
    set_error("workspace of %zu bytes required", need);
    return CONV3D_ERR_WORKSPACE;
  }
  if (params && !aligned(workspace, 256)) {
    set_error("workspace must be 256-byte aligned");
    return CONV3D_ERR_ALIGNMENT;
  }
  const size_t n = static_cast<size_t>(rows) * C * 2, cb = act8_code_bytes(rows, C),
               sb = act8_scale_bytes(rows, C), rb = static_cast<size_t>(rows) * 4, pb = C * 2ull;
  const struct { const void* p; size_t n; } outs[] = {{dx, n}, {dgamma, pb}, {dbeta, pb}, {params ? workspace : nullptr, need}},
                                            ins[] = {{dy, n}, {x, n}, {codes, cb}, {exponents, sb}, {mean, rb},
                                                     {rstd, rb}, {gamma, pb}, {dres, n}};
  for (const auto& o : outs) {
    for (const auto& i : ins)
      if (overlaps(o.p, o.n, i.p, i.n) && !(o.p == dx && (i.p == dy || i.p == dres || i.p == x) && o.p == i.p))
        return overlapping("dx must be exactly dy, x or dres or overlap none of them; the other outputs must overlap nothing");
    for (const auto& q : outs)
      if (&o != &q && overlaps(o.p, o.n, q.p, q.n))
        return overlapping("dx, dgamma, dbeta and the workspace must not overlap");
  }
  Device dev;
  if ((st = current_device(dev)) != CONV3D_OK) return st;
  const unsigned blocks = bwd_blocks(rows, C);
  LnBwdParams p{static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(x),
                static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(exponents), mean, rstd,
                static_cast<const uint16_t*>(gamma), static_cast<const uint16_t*>(dres),
                static_cast<uint16_t*>(dx), params ? static_cast<float*>(workspace) : nullptr, rows, C};
  const bool bf16 = dtype == CONV3D_BF16;
  cudaError_t e = from_codes ? (bf16 ? dispatch_bwd<true, true>(p, blocks, stream) : dispatch_bwd<false, true>(p, blocks, stream))
                             : (bf16 ? dispatch_bwd<true, false>(p, blocks, stream) : dispatch_bwd<false, false>(p, blocks, stream));
  if (e != cudaSuccess) return cuda_fail(e, "layer norm gradient launch");
  if (!params) return CONV3D_OK;
  const unsigned cols = static_cast<unsigned>((2 * C + 31) / 32);
  uint16_t* g16 = static_cast<uint16_t*>(dgamma);
  uint16_t* b16 = static_cast<uint16_t*>(dbeta);
  e = dtype == CONV3D_BF16 ? launch(layernorm_param_kernel<true>, cols, 32 * kParamWarps, 0, 1, stream, p.part, static_cast<int>(blocks), C, g16, b16)
                           : launch(layernorm_param_kernel<false>, cols, 32 * kParamWarps, 0, 1, stream, p.part, static_cast<int>(blocks), C, g16, b16);
  return e == cudaSuccess ? CONV3D_OK : cuda_fail(e, "layer norm parameter gradient launch");
}

conv3d_status_t conv3d_act8_pack(const void* x, void* codes, void* exponents, long long rows, int C,
                                 conv3d_dtype_t dtype, struct CUstream_st* stream) {
  conv3d_status_t st = check_sizes(rows, C, dtype, kMaxAct8Channels);
  if (st != CONV3D_OK) return st;
  if (!x || !codes || !exponents) {
    set_error("x, codes and exponents must be non-null");
    return CONV3D_ERR_INVALID_ARG;
  }
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(exponents, 16)) return misaligned();
  const size_t n = static_cast<size_t>(rows) * C * 2, cb = act8_code_bytes(rows, C), sb = act8_scale_bytes(rows, C);
  if (overlaps(codes, cb, x, n) || overlaps(exponents, sb, x, n) || overlaps(codes, cb, exponents, sb))
    return overlapping("x, codes and exponents must not overlap");
  Device dev;
  if ((st = current_device(dev)) != CONV3D_OK) return st;
  const int units = units_per_row(C, 16);
  const long long total = rows * units;
  const unsigned blocks = blocks_for(total, kThreads * kUnroll, dev.num_sms * 6LL);
  const uint16_t* x16 = static_cast<const uint16_t*>(x);
  uint8_t* q = static_cast<uint8_t*>(codes);
  uint8_t* s = static_cast<uint8_t*>(exponents);
  const cudaError_t e = dtype == CONV3D_BF16
                            ? launch(act8_pack_kernel<true>, blocks, kThreads, 0, 1, stream, x16, q, s, total, units, C)
                            : launch(act8_pack_kernel<false>, blocks, kThreads, 0, 1, stream, x16, q, s, total, units, C);
  return e == cudaSuccess ? CONV3D_OK : cuda_fail(e, "checkpoint launch");
}

static conv3d_status_t act8_read(const void* codes, const void* exponents, const void* gamma, const void* beta,
                                 const void* dy, bool grad, conv3d_act_t act, void* out, long long rows, int C,
                                 conv3d_dtype_t dtype, cudaStream_t stream) {
  conv3d_status_t st = check_sizes(rows, C, dtype, kMaxAct8Channels);
  if (st != CONV3D_OK) return st;
  if (!codes || !exponents || !out || (grad && !dy) || static_cast<int>(act) > CONV3D_ACT_GELU || static_cast<int>(act) < 0) {
    set_error("a tensor pointer is null or the activation %d unknown", static_cast<int>(act));
    return CONV3D_ERR_INVALID_ARG;
  }
  if (!aligned(codes, 16) || !aligned(exponents, 16) || !aligned(gamma, 16) || !aligned(beta, 16) ||
      !aligned(dy, 16) || !aligned(out, 16))
    return misaligned();
  const size_t n = static_cast<size_t>(rows) * C * 2, cb = act8_code_bytes(rows, C), sb = act8_scale_bytes(rows, C),
               pb = static_cast<size_t>(C) * 2;
  if (overlaps(out, n, codes, cb) || overlaps(out, n, exponents, sb) || overlaps(out, n, gamma, pb) ||
      overlaps(out, n, beta, pb) || (dy != out && overlaps(out, n, dy, n)))
    return overlapping("the output must not overlap the inputs (the gradient's may be exactly dy)");
  Device dev;
  if ((st = current_device(dev)) != CONV3D_OK) return st;
  ReadParams p{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(exponents),
               static_cast<const uint16_t*>(gamma), static_cast<const uint16_t*>(beta),
               static_cast<const uint16_t*>(dy), static_cast<uint16_t*>(out), rows * units_per_row(C, 8),
               units_per_row(C, 8), C};
  unsigned blocks = blocks_for(p.total, kThreads * kUnroll, dev.num_sms * 8LL);
  if (gamma || beta) {   // whole rows per grid stride, so that a thread keeps its channels
    unsigned a = kThreads, b = static_cast<unsigned>(p.units);
    while (b != 0) {
      const unsigned r = a % b;
      a = b;
      b = r;
    }
    const unsigned m = static_cast<unsigned>(p.units) / a;   // blocks that hold a whole number of rows
    if (blocks > m) blocks -= blocks % m;
  }
  const bool bf16 = dtype == CONV3D_BF16;
  const Read mode = grad ? Read::kGrad : gamma || beta ? Read::kAffine : Read::kPlain;
  const cudaError_t e = bf16 ? dispatch_read<true>(mode, act, blocks, stream, p) : dispatch_read<false>(mode, act, blocks, stream, p);
  return e == cudaSuccess ? CONV3D_OK : cuda_fail(e, "checkpoint read launch");
}

conv3d_status_t conv3d_act8_unpack(const void* codes, const void* exponents, const void* gamma,
                                   const void* beta, conv3d_act_t act, void* y, long long rows, int C,
                                   conv3d_dtype_t dtype, struct CUstream_st* stream) {
  return act8_read(codes, exponents, gamma, beta, nullptr, false, act, y, rows, C, dtype, stream);
}

conv3d_status_t conv3d_act8_bwd(const void* dy, const void* codes, const void* exponents,
                                conv3d_act_t act, void* dx, long long rows, int C,
                                conv3d_dtype_t dtype, struct CUstream_st* stream) {
  return act8_read(codes, exponents, nullptr, nullptr, dy, true, act, dx, rows, C, dtype, stream);
}

}  // extern "C"
