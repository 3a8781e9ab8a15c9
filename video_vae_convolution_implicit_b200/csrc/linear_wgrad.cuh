// linear_wgrad.cuh -- the weight and bias gradients of the channel product:
//   dw[n, k] = sum_m dy[m, n] x[m, k],   dbias[n] = sum_m dy[m, n].
//
// The contraction runs over the rows, which neither tensor stores innermost, so
// both tcgen05 operands are MN-major as they lie in memory: A = dy^T (256 of its
// columns per CTA pair), B = x (256 of its columns), 128 rows a pipeline stage.
// The 1x1x1 convolution's weight-gradient kernel computes the same sums one CTA at
// a time and adds its parts by fp32 atomics; here a pair shares each operand
// (128 KB of loads for 16.8 MFLOP instead of 192 KB), the row ranges' parts go to
// the workspace and are added in their order -- the same bits every time -- and a
// call that needs one range only writes the result itself, in one launch.
//
// dbias rides along in the tiles of the first 256 columns of x: one more MMA of
// 32 columns per step, whose B operand is a tile of ones, leaves the row sums of
// A beside the accumulator, so dy is not read again.
//
// Units are (row range, tile), tiles fastest, so that the pairs at work share the
// rows they read: x and dy come from HBM about once.
//
// Measured (bf16 with dbias; the 1x1x1 convolution's kernel in brackets): 104448
// rows, 512 -> 2048 187 us (263) and 2048 -> 512 180 us (218), 1170 and 1220
// TFLOP/s (in bursts; replayed for a second, at the chip's power limit and 1.3 GHz, 231
// us each): the tensor cores are busy 65 to 68% of the cycles; stages of 64 rows, twice as many, took 235 and 208.  540672 rows of 512 ->
// 256 135 us (195), 6.1 TB/s: the rows' reads.  10000 rows of 128 x 128 12 us (13),
// 61 rows of 1000 x 1024 9 us (20): launches and latency.
#pragma once

#include "linear_kernel.cuh"

namespace conv3d {

constexpr int kWgRows = 128;                             // rows per stage
constexpr uint32_t kWgBoxBytes = kWgRows * 128;          // 128 rows of 64 columns
constexpr uint32_t kWgStageBytes = 4 * kWgBoxBytes;      // one CTA: two boxes of dy, two of x
constexpr int kWgStages = 3;
constexpr uint32_t kWgOnesBytes = 16 * 128;              // 16 rows (one MMA step) of ones
constexpr int kWgEpiWarps = 8;
constexpr int kWgThreads = 64 + 32 * kWgEpiWarps;
constexpr int kWgTile = 256;
constexpr int kWgSlotFloats = kWgTile * kWgTile;         // one unit's part

struct LinearWgradParams {
  int M, N, K;
  int chunks;               // ceil(M / 128)
  int tiles_n, tiles;       // tiles_n * tiles_k, n fastest
  int splits;               // row ranges
  int kw;                   // columns of x in a product: 256, or 128 where K has no more
  // 64-column boxes of dy and of x that CTA r of a pair loads (2 and kw / 128, or
  // fewer where the only tile along n or k ends before them: what shared memory
  // holds in their place reaches only products that nobody reads)
  int boxes_n[2], boxes_k[2];
  float* part;              // [splits][tiles][kWgSlotFloats] (splits > 1)
  float* bias_part;         // [splits][tiles_n * 256] (splits > 1, with dbias)
  uint16_t* dw;             // [N][K]
  uint16_t* dbias;          // [N] or null
  uint32_t idesc, idesc_bias;
  int* status;
  unsigned long long timeout_ns;
  int test_stall;
};

// Where the part of (CTA rank, 32-column chunk j, group q of four columns, row r of
// the CTA's 128) lies in a slot, in float4: a warp's accesses are contiguous.
__device__ __forceinline__ int wg_part_index(int rank, int j, int q, int r) {
  return ((rank * 8 + j) * 8 + q) * BM + r;
}

// kDirect: one row range, whose tiles are written to dw in 16 bits.
template <bool kBF16, bool kDirect>
__global__ void __launch_bounds__(kWgThreads, 1)
    linear_wgrad_kernel(const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ CUtensorMap map_x,
                        const LinearWgradParams p) {
  using T = Val16<kBF16>;
  extern __shared__ uint8_t lin_smem[];
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  __shared__ uint64_t s_peer_bar;
  __shared__ unsigned long long s_peer_count;
  const uint32_t warp = threadIdx.x / 32;
  const uint32_t lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x / 2;
  const int num_pairs = gridDim.x / 2;
  const int units = p.tiles * p.splits;

  const uint32_t ring = (smem_addr(lin_smem) + 1023u) & ~1023u;
  const uint32_t ones = ring + kWgStages * kWgStageBytes;
  const uint32_t bars = ones + kWgOnesBytes;
  const uint32_t full_bar = bars;
  const uint32_t empty_bar = full_bar + 8 * kWgStages;
  const uint32_t tfull_bar = empty_bar + 8 * kWgStages;
  const uint32_t tempty_bar = tfull_bar + 8;
  const uint32_t drain_bar = tempty_bar + 8;
  SharedCtl ctl{&s_abort, p.status, p.timeout_ns, mapa_shared(smem_addr(const_cast<int*>(&s_abort)), rank ^ 1u)};
  const uint32_t peer_bar = smem_addr(&s_peer_bar);
  const uint32_t peer_count = smem_addr(&s_peer_count);

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < kWgStages; ++s) {
      mbar_init(full_bar + 8 * s, 1);
      mbar_init(empty_bar + 8 * s, 1);
    }
    mbar_init(tfull_bar, 1);
    mbar_init(tempty_bar, kWgEpiWarps * 2);
    mbar_init(drain_bar, 1);
    mbar_init(peer_bar, 1);
    fence_mbar_init();
    prefetch_tensormap(&map_dy);
    prefetch_tensormap(&map_x);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(&s_tmem_base), 512);   // 256 columns of products, 32 of row sums
    tmem_relinquish_pair();
  }
  if (warp >= 2) {
    const uint32_t one2 = kBF16 ? 0x3F803F80u : 0x3C003C00u;
    for (uint32_t i = threadIdx.x - 64; i < kWgOnesBytes / 16; i += 32 * kWgEpiWarps)
      st_shared_v4(ones + i * 16, one2, one2, one2, one2);
    fence_proxy_async_shared();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the peer's barriers are initialised, and its ones written
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  griddep_wait();
  griddep_launch_dependents();

  // unit u: row chunks [lo, hi), tile columns n0 of dy and k0 of x
  struct Unit {
    int lo, hi, tile, n0, k0, split;
  };
  auto unit_of = [&](int u) {
    Unit r;
    r.split = u / p.tiles;
    r.tile = u - r.split * p.tiles;
    const int kt = r.tile / p.tiles_n;
    r.n0 = (r.tile - kt * p.tiles_n) * kWgTile;
    r.k0 = kt * kWgTile;
    r.lo = static_cast<int>(static_cast<long long>(r.split) * p.chunks / p.splits);
    r.hi = static_cast<int>(static_cast<long long>(r.split + 1) * p.chunks / p.splits);
    return r;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const bool stall = p.test_stall != 0;
      uint32_t stage = 0, phase = 0;
      long long issued = 0;
      bool ok = true;
      const int an = p.boxes_n[rank], bk = p.boxes_k[rank];
      const uint32_t peer_bytes = (p.boxes_n[rank ^ 1u] + p.boxes_k[rank ^ 1u]) * kWgBoxBytes;
      const uint32_t tx_bytes = (an + bk) * kWgBoxBytes + peer_bytes;
      for (int u = pair; ok && u < units; u += num_pairs) {
        const Unit w = unit_of(u);
        const int n = w.n0 + static_cast<int>(rank) * BM, k = w.k0 + static_cast<int>(rank) * (p.kw / 2);
        for (int c = w.lo; c < w.hi; ++c) {
          if (!wait_bounded(empty_bar + 8 * stage, phase ^ 1, ctl, true)) {
            ok = false;
            break;
          }
          const uint32_t fb = full_bar + 8 * stage;
          if (!(stall && issued == 0)) {
            // rows past M and columns past N or K read as zero
            if (leader) mbar_arrive_expect_tx(fb, tx_bytes);
            const uint32_t fb_leader = mapa_shared(fb, 0);
            const uint32_t at = ring + stage * kWgStageBytes;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (i < an) tma_load_2d_pair(at + i * kWgBoxBytes, &map_dy, fb_leader, n + 64 * i, c * kWgRows);
              if (i < bk) tma_load_2d_pair(at + (2 + i) * kWgBoxBytes, &map_x, fb_leader, k + 64 * i, c * kWgRows);
            }
          }
          ++issued;
          if (++stage == kWgStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      producer_finish<true>(!ok, issued, stall, kWgStages, full_bar, peer_bytes, peer_count, peer_bar, ctl, leader);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && leader) {
      uint32_t stage = 0, phase = 0, drained = 0;
      bool ok = true;
      const uint64_t d_ones = lin_desc_mn(ones, kWgOnesBytes);
      for (int u = pair; ok && u < units; u += num_pairs, ++drained) {
        const Unit w = unit_of(u);
        const bool sums = p.dbias != nullptr && w.k0 == 0;
        if (!wait_bounded(tempty_bar, (drained & 1) ^ 1, ctl, true)) break;
        tc_fence_after();
        for (int c = w.lo; c < w.hi; ++c) {
          if (!wait_bounded(full_bar + 8 * stage, phase, ctl, true)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = lin_desc_mn(ring + stage * kWgStageBytes, kWgBoxBytes);
          const uint64_t db = lin_desc_mn(ring + stage * kWgStageBytes + 2 * kWgBoxBytes, kWgBoxBytes);
#pragma unroll
          for (int k = 0; k < kWgRows / 16; ++k) {
            const uint32_t accumulate = c != w.lo || k != 0;
            mma_f16_ss_pair(tmem_base, da + k * (2048 >> 4), db + k * (2048 >> 4), p.idesc, accumulate);
            if (sums) mma_f16_ss_pair(tmem_base + kWgTile, da + k * (2048 >> 4), d_ones, p.idesc_bias, accumulate);
          }
          mma_commit_both(empty_bar + 8 * stage);
          if (++stage == kWgStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        mma_commit_both(tfull_bar);
      }
      mma_commit_pair(drain_bar);
      wait_bounded(drain_bar, 0, ctl, false);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // One row (a column of dy) per thread; two warps share a lane quarter and
    // take half of the 256 columns each.
    const uint32_t quarter = warp & 3;
    const int half = static_cast<int>(warp - 2) / 4;
    const int r = static_cast<int>(quarter * 32u + lane);
    const uint32_t t_row = tmem_base + ((quarter * 32u) << 16);
    uint32_t phase = 0;
    for (int u = pair; u < units; u += num_pairs, phase ^= 1) {
      const Unit w = unit_of(u);
      const int n = w.n0 + static_cast<int>(rank) * BM + r;
      const bool rows_live = n - static_cast<int>(lane) < p.N;   // some row of this warp is a channel of dy
      if (!__all_sync(0xFFFFFFFFu, wait_bounded(tfull_bar, phase, ctl, true))) break;   // the warp leaves as one
      tc_fence_after();
      if (p.dbias != nullptr && w.k0 == 0 && half == 0 && rows_live) {
        uint32_t sum;
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(sum) : "r"(t_row + kWgTile) : "memory");
        tmem_ld_wait();
        if (n < p.N) {
          if constexpr (kDirect)
            p.dbias[n] = static_cast<uint16_t>(T::pack(__uint_as_float(sum), 0.0f) & 0xFFFFu);
          else
            p.bias_part[static_cast<size_t>(w.split) * p.tiles_n * kWgTile + n] = __uint_as_float(sum);
        }
      }
      float4* slot = kDirect ? nullptr
                             : reinterpret_cast<float4*>(p.part + (static_cast<size_t>(w.split) * p.tiles + w.tile) * kWgSlotFloats);
      for (int j = half * 4; rows_live && j < half * 4 + 4; ++j) {
        const int k = w.k0 + 32 * j;
        if (k >= p.K) break;
        uint32_t v[32];
        tmem_ld_32x32b_x32(t_row + 32 * j, v);
        tmem_ld_wait();
        if constexpr (kDirect) {
          if (n < p.N) {
            uint16_t* dst = p.dw + static_cast<size_t>(n) * p.K + k;
#pragma unroll
            for (int g = 0; g < 4; ++g)
              if (k + 8 * g < p.K) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  o[e] = T::pack(__uint_as_float(v[8 * g + 2 * e]), __uint_as_float(v[8 * g + 2 * e + 1]));
                *reinterpret_cast<uint4*>(dst + 8 * g) = make_uint4(o[0], o[1], o[2], o[3]);
              }
          }
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            slot[wg_part_index(static_cast<int>(rank), j, q, r)] =
                make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                            __uint_as_float(v[4 * q + 3]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(tempty_bar, 0));
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // no CTA leaves while its peer may touch it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// Adds the row ranges' parts in a fixed order and rounds: block (tile, rank, chunk
// j, quarter h) takes 128 rows x 8 columns, one float4 of it per thread, with 16
// ranges' loads in flight (four float4 per thread and six ranges: 74 ranges of a
// 64 x 64 gradient took 13 trips to memory in two blocks), and writes 16-byte row
// pieces through shared memory.  The blocks after those add the bias gradient's
// parts, 32 columns each: group g of eight takes the ranges g, g + 8, ... , then
// the groups' sums are added in order.  Ranges are read in batches there too: one
// at a time, 66 of them took 67 us of load latency.
template <bool kBF16>
__global__ void __launch_bounds__(256) linear_wgrad_sum_kernel(const LinearWgradParams p) {
  using T = Val16<kBF16>;
  __shared__ uint2 rows[BM];
  griddep_wait();
  griddep_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= p.tiles * 64) {
    __shared__ float sums[8][32];
    const int n = (static_cast<int>(blockIdx.x) - p.tiles * 64) * 32 + static_cast<int>(threadIdx.x % 32);
    const int g = threadIdx.x / 32;
    float a = 0.0f;
    constexpr int kLoads = 8;
    if (n < p.N)
      for (int s0 = g; s0 < p.splits; s0 += 8 * kLoads) {
        float v[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          v[i] = s0 + 8 * i < p.splits ? __ldcg(p.bias_part + static_cast<size_t>(s0 + 8 * i) * p.tiles_n * kWgTile + n) : 0.0f;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) a += v[i];
      }
    sums[g][threadIdx.x % 32] = a;
    __syncthreads();
    if (g == 0 && n < p.N) {
      a = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) a += sums[i][threadIdx.x];
      p.dbias[n] = static_cast<uint16_t>(T::pack(a, 0.0f) & 0xFFFFu);
    }
    return;
  }
  const int h = blockIdx.x % 4, j = blockIdx.x / 4 % 8, rank = blockIdx.x / 32 % 2, tile = blockIdx.x / 64;
  const int kt = tile / p.tiles_n;
  const int n0 = (tile - kt * p.tiles_n) * kWgTile + rank * BM, k = kt * kWgTile + 32 * j + 8 * h;
  if (n0 >= p.N || k >= p.K) return;
  // warps whose 32 rows lie past N have no parts to read (none were written)
  const int r = threadIdx.x % BM;
  const bool live = n0 + (r & ~31) < p.N;
  const float4* part = reinterpret_cast<const float4*>(p.part) + static_cast<size_t>(tile) * (kWgSlotFloats / 4) +
                       wg_part_index(rank, j, 2 * h + threadIdx.x / BM, r);
  const size_t step = static_cast<size_t>(p.tiles) * (kWgSlotFloats / 4);
  float2 a[2] = {both(0.0f), both(0.0f)};
  constexpr int kBatch = 16;
  if (live)
    for (int s0 = 0; s0 < p.splits; s0 += kBatch) {
      float4 v[kBatch];
#pragma unroll
      for (int s = 0; s < kBatch; ++s)
        v[s] = s0 + s < p.splits ? __ldcg(part + (s0 + s) * step) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int s = 0; s < kBatch; ++s) {
        a[0] = add2(a[0], make_float2(v[s].x, v[s].y));
        a[1] = add2(a[1], make_float2(v[s].z, v[s].w));
      }
    }
  const uint2 mine = make_uint2(T::pack(a[0].x, a[0].y), T::pack(a[1].x, a[1].y));
  if (threadIdx.x >= BM) rows[r] = mine;
  __syncthreads();
  if (threadIdx.x < BM && n0 + r < p.N)
    *reinterpret_cast<uint4*>(p.dw + static_cast<size_t>(n0 + r) * p.K + k) = make_uint4(mine.x, mine.y, rows[r].x, rows[r].y);
}

}  // namespace conv3d
