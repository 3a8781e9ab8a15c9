// linear_kernel.cuh -- the product of channel rows with a weight matrix, with
// its bias, activation, residual and 8-bit checkpoint in the epilogue, and the
// product of a gradient with the same matrix, with the activation's derivative
// (from the checkpoint) in the epilogue:
//
//   forward   y[m, n]  = act(pre[m, n]) + residual[m, n],
//             pre[m, n] = bias[n] + sum_k x[m, k] w[n, k]       (pre -> checkpoint)
//   gradient  dx[m, k] = (sum_n dy[m, n] w[n, k]) * act'(pre[m, k])
//
// Both are C = A B^T with A row-major along the contraction; the gradient's B is
// w as it lies in memory, its output channels innermost (an MN-major operand),
// so no transposed copy of w is made.
//
// linear_pair_kernel (many rows): persistent CTA pairs over tiles of 256 rows x
// BN columns, warp-specialised as the convolution is -- TMA producer, one
// tcgen05.mma issuer (cta_group::2), and 8 epilogue warps over two TMEM
// accumulators -- since at 8 k-blocks a tile the epilogue has about as many
// issue slots to spend as the tensor cores take for the tile.  Columns are the
// fast tile index, so the tiles in flight share rows of A and A is read from
// HBM about once; w stays in L2.
//
// linear_rows_kernel (few rows): one 128-channel x up-to-128-row tile per
// cluster, transposed (w is the 128-row operand, the rows of x are the N side),
// with the contraction split over the cluster's CTAs, whose partial sums meet
// in shared memory: w, the bulk of the bytes, streams through as many SMs as
// there are pieces, in one launch and without a workspace, and the sum runs in
// rank order whatever the timing.
#pragma once

#include "act8.cuh"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace conv3d {

constexpr int kLinEpiWarps = 8;
constexpr int kLinThreads = 64 + 32 * kLinEpiWarps;   // producer, issuer, epilogue
constexpr int kLinRowsThreads = 64 + 32 * 4;
constexpr uint32_t kLinABytes = BM * BK * 2;           // one CTA's A rows of a k-block
constexpr uint32_t kLinOutBytes = 32 * 32 * 2;         // a 32 x 32 chunk of 16-bit values
constexpr uint32_t kLinCodeBytes = 32 * 32;            // the same chunk's codes

struct LinearParams {
  int M, N;                 // rows and columns of the result
  int kblocks;              // ceil(contraction / 64)
  int BN;                   // columns per tile (pair) / rows per tile (rows kernel)
  int tiles_n, num_tiles;
  int split;                // CTAs per cluster along the contraction (rows kernel)
  int stages;
  uint32_t tmem_cols;
  uint32_t idesc;
  const uint16_t* bias;     // [N] or null
  const uint16_t* residual; // rows kernel; the pair kernel reads it through map_aux
  uint16_t* out;            // rows kernel
  uint8_t* codes;           // rows kernel: written (forward) or read (gradient)
  uint8_t* exponents;       // written or read, [M][blocks]
  int blocks;               // ceil(N / 32)
  int has_aux;              // forward: a residual is added
  int* status;
  unsigned long long timeout_ns;
  int test_stall;           // failure-detection test: the first stage's copies are skipped
};

// 2D tiled TMA: {column, row} of a row-major matrix.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c, int r) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c), "r"(r)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int c,
                                                 int r) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(c),
      "r"(r)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int c, int r) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c), "r"(r)
               : "memory");
}

// MN-major operand in 64-element x 8-row atoms with the 128-byte swizzle:
// 64-element blocks `block_bytes` apart along M/N, 8-row groups 1 KB apart
// along the contraction.
__device__ __forceinline__ uint64_t lin_desc_mn(uint32_t saddr, uint32_t block_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>((block_bytes >> 4) & 0x3FFF) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
constexpr uint32_t kMnBlockBytes = 64 * 128;           // 64 contraction rows of 64 elements

// Byte offset of 16-byte half h of row r in a 32 x 32-byte buffer with the
// 32-byte swizzle (the half index XOR bit 7 of the row offset).
__device__ __forceinline__ uint32_t swz32(uint32_t r, uint32_t h) { return r * 32u + ((h ^ ((r >> 2) & 1u)) << 4); }

// ------------------------------------------------------------------ many rows

// kBwd: the gradient (B MN-major, no bias; the chunk is multiplied by
// act'(checkpoint) when kQ).  Forward: kQ writes the checkpoint.  Shared
// memory: A ring, B ring, then per epilogue warp two output buffers, two
// residual buffers (forward with a residual) and two code buffers (kQ), then
// the barriers.
template <bool kBF16, bool kBwd, int kAct, bool kQ>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                       const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_aux,
                       const __grid_constant__ CUtensorMap map_codes, const LinearParams p) {
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
  const int unit = blockIdx.x / 2;
  const int num_units = gridDim.x / 2;

  const uint32_t base = (smem_addr(lin_smem) + 1023u) & ~1023u;
  const uint32_t b_rows = static_cast<uint32_t>(p.BN) / 2;      // this CTA's half of B
  const uint32_t b_bytes = b_rows * BK * 2;
  const uint32_t a_ring = base;
  const uint32_t b_ring = a_ring + p.stages * kLinABytes;
  const uint32_t out_buf = b_ring + p.stages * b_bytes;
  const uint32_t aux_buf = out_buf + kLinEpiWarps * 2 * kLinOutBytes;
  const bool has_res = !kBwd && p.has_aux != 0;
  const uint32_t code_buf = aux_buf + (has_res ? kLinEpiWarps * 2 * kLinOutBytes : 0);
  const uint32_t bars = code_buf + (kQ ? kLinEpiWarps * 2 * kLinCodeBytes : 0);
  const uint32_t full_bar = bars;
  const uint32_t empty_bar = full_bar + 8 * p.stages;
  const uint32_t tfull_bar = empty_bar + 8 * p.stages;
  const uint32_t tempty_bar = tfull_bar + 16;
  const uint32_t drain_bar = tempty_bar + 16;
  const uint32_t lfull_bar = drain_bar + 8;                     // [epilogue warp][2]: loads of the epilogue

  SharedCtl ctl{&s_abort, p.status, p.timeout_ns, mapa_shared(smem_addr(const_cast<int*>(&s_abort)), rank ^ 1u)};
  const uint32_t peer_bar = smem_addr(&s_peer_bar);
  const uint32_t peer_count = smem_addr(&s_peer_count);

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar + 8 * s, 1);
      mbar_init(empty_bar + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar + 8 * a, 1);
      mbar_init(tempty_bar + 8 * a, kLinEpiWarps * 2);
    }
    mbar_init(drain_bar, 1);
    mbar_init(peer_bar, 1);
    for (int e = 0; e < 2 * kLinEpiWarps; ++e) mbar_init(lfull_bar + 8 * e, 1);
    fence_mbar_init();
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_b);
    prefetch_tensormap(&map_out);
    if (has_res) prefetch_tensormap(&map_aux);
    if (kQ) prefetch_tensormap(&map_codes);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(&s_tmem_base), p.tmem_cols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  griddep_wait();   // no global memory is touched before the previous kernel has finished

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t tx_bytes = 2 * (kLinABytes + b_bytes);
      const bool stall = p.test_stall != 0;
      uint32_t stage = 0, phase = 0;
      long long issued = 0;
      bool ok = true;
      for (int t = unit; ok && t < p.num_tiles; t += num_units) {
        const int mt = t / p.tiles_n;
        const int row0 = mt * 2 * BM + static_cast<int>(rank) * BM;
        const int col0 = (t - mt * p.tiles_n) * p.BN + static_cast<int>(rank * b_rows);
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (!wait_bounded(empty_bar + 8 * stage, phase ^ 1, ctl, true)) {
            ok = false;
            break;
          }
          const uint32_t fb = full_bar + 8 * stage;
          if (!(stall && issued == 0)) {
            // rows past M, columns past N and the contraction's end read as zero
            if (leader) mbar_arrive_expect_tx(fb, tx_bytes);
            const uint32_t fb_leader = mapa_shared(fb, 0);
            tma_load_2d_pair(a_ring + stage * kLinABytes, &map_a, fb_leader, kb * BK, row0);
            if constexpr (kBwd) {
              for (uint32_t i = 0; i < b_rows / 64; ++i)
                tma_load_2d_pair(b_ring + stage * b_bytes + i * kMnBlockBytes, &map_b, fb_leader,
                                 col0 + static_cast<int>(i) * 64, kb * BK);
            } else {
              tma_load_2d_pair(b_ring + stage * b_bytes, &map_b, fb_leader, kb * BK, col0);
            }
          }
          ++issued;
          if (++stage == static_cast<uint32_t>(p.stages)) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      producer_finish<true>(!ok, issued, stall, p.stages, full_bar, kLinABytes + b_bytes, peer_count, peer_bar, ctl,
                            leader);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && leader) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      int local = 0;
      for (int t = unit; ok && t < p.num_tiles; t += num_units, ++local) {
        const uint32_t acc = local & 1;
        if (!wait_bounded(tempty_bar + 8 * acc, ((local >> 1) & 1) ^ 1, ctl, true)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * static_cast<uint32_t>(p.BN);
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (!wait_bounded(full_bar + 8 * stage, phase, ctl, true)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = smem_desc_k_sw128(a_ring + stage * kLinABytes);
          const uint64_t db = kBwd ? lin_desc_mn(b_ring + stage * b_bytes, kMnBlockBytes)
                                   : smem_desc_k_sw128(b_ring + stage * b_bytes);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)   // 16 values along the contraction: 32 bytes of a K-major row, 16 rows of an MN-major block
            mma_f16_ss_pair(d_tmem, da + 2 * k, db + (kBwd ? (2048 >> 4) : 2) * k, p.idesc, (kb | k) != 0);
          mma_commit_pair(empty_bar + 8 * stage);
          mma_commit_pair(mapa_shared(empty_bar + 8 * stage, 1));
          if (++stage == static_cast<uint32_t>(p.stages)) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        mma_commit_pair(tfull_bar + 8 * acc);
        mma_commit_pair(mapa_shared(tfull_bar + 8 * acc, 1));
      }
      mma_commit_pair(drain_bar);
      wait_bounded(drain_bar, 0, ctl, false);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // Two warps share each quarter of the TMEM lanes (32 rows of the tile) and
    // take half of its columns each, 32 at a time: one row and one checkpoint
    // block per thread, so the block's exponent needs no exchange.
    const uint32_t quarter = warp & 3;
    const uint32_t ew = warp - 2;
    const int half = static_cast<int>(ew) / 4;
    const int nj = p.BN / 64;                                  // chunks per warp and tile
    const uint32_t obuf = out_buf + ew * 2 * kLinOutBytes;
    const uint32_t abuf = aux_buf + ew * 2 * kLinOutBytes;
    const uint32_t cbuf = code_buf + ew * 2 * kLinCodeBytes;
    const uint32_t lbar = lfull_bar + ew * 16;
    constexpr bool kLoadCodes = kBwd && kQ;
    const bool loads = has_res || kLoadCodes;
    const uint4* bias4 = reinterpret_cast<const uint4*>(p.bias);
    uint32_t out_no = 0;          // chunks stored so far: buffer out_no & 1
    uint32_t load_no = 0;         // chunks whose load was waited for: buffer load_no & 1
    uint32_t asked_no = 0;        // chunks whose load was issued
    bool ok = true;
    int local = 0;
    for (int t = unit; ok && t < p.num_tiles; t += num_units, ++local) {
      const uint32_t acc = local & 1;
      const int mt = t / p.tiles_n;
      const int row0 = mt * 2 * BM + static_cast<int>(rank) * BM + static_cast<int>(quarter) * 32;
      const int col0 = (t - mt * p.tiles_n) * p.BN + half * nj * 32;
      const int row = row0 + static_cast<int>(lane);
      int live = (p.N - col0 + 31) / 32;                        // chunks with a column of the result
      live = live < 0 ? 0 : live > nj ? nj : live;
      if (row0 >= p.M) live = 0;
      auto ask = [&](int j) {                                   // lane 0: load chunk j's residual or codes
        const uint32_t b = asked_no & 1;
        if constexpr (kLoadCodes) {
          mbar_arrive_expect_tx(lbar + 8 * b, kLinCodeBytes);
          tma_load_2d(cbuf + b * kLinCodeBytes, &map_codes, lbar + 8 * b, col0 + 32 * j, row0);
        } else {
          mbar_arrive_expect_tx(lbar + 8 * b, kLinOutBytes);
          tma_load_2d(abuf + b * kLinOutBytes, &map_aux, lbar + 8 * b, col0 + 32 * j, row0);
        }
      };
      if (loads)
        for (int j = 0; j < 2 && j < live; ++j) {
          if (lane == 0) ask(j);
          ++asked_no;
        }
      // gradient: this row's exponent bytes; forward: collected here, stored at the end
      uint32_t eb4 = 0;
      uint8_t* erow = p.exponents + static_cast<size_t>(row) * p.blocks + col0 / 32;
      const bool word = nj == 4 && (p.blocks & 3) == 0;         // col0 / 32 is a multiple of 4 then
      if (kLoadCodes && live > 0 && row < p.M) {
        if (word) {
          eb4 = __ldg(reinterpret_cast<const uint32_t*>(erow));
        } else {
          for (int j = 0; j < live; ++j) eb4 |= static_cast<uint32_t>(__ldg(erow + j)) << (8 * j);
        }
      }
      if (!wait_bounded(tfull_bar + 8 * acc, (local >> 1) & 1, ctl, true)) {
        ok = false;
      } else {
        tc_fence_after();
        const uint32_t t_row =
            tmem_base + ((quarter * 32u) << 16) + acc * static_cast<uint32_t>(p.BN) + half * nj * 32;
        for (int j = 0; j < live; ++j) {
          const int col = col0 + 32 * j;
          uint32_t raw[32];
          tmem_ld_32x32b_x32(t_row + j * 32, raw);
          float2 v[16];
          if constexpr (kLoadCodes) {
            const uint32_t b = load_no & 1;
            if (!wait_bounded(lbar + 8 * b, (load_no >> 1) & 1, ctl, true)) {
              ok = false;
              tmem_ld_wait();
              break;
            }
            ++load_no;
            const float step = a8_step((eb4 >> (8 * j)) & 0xFFu);
            const uint4 k0 = ld_shared_v4(cbuf + b * kLinCodeBytes + swz32(lane, 0));
            const uint4 k1 = ld_shared_v4(cbuf + b * kLinCodeBytes + swz32(lane, 1));
            a8_decode4(k0.x, step, v); a8_decode4(k0.y, step, v + 2);
            a8_decode4(k0.z, step, v + 4); a8_decode4(k0.w, step, v + 6);
            a8_decode4(k1.x, step, v + 8); a8_decode4(k1.y, step, v + 10);
            a8_decode4(k1.z, step, v + 12); a8_decode4(k1.w, step, v + 14);
            act_limit(v, step);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = act_slope<kAct>(v[e]);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e)
              v[e] = mul2(v[e], make_float2(__uint_as_float(raw[2 * e]), __uint_as_float(raw[2 * e + 1])));
          } else {
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = make_float2(__uint_as_float(raw[2 * e]), __uint_as_float(raw[2 * e + 1]));
          }
          if (!kBwd && bias4 != nullptr) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
              if (col + 8 * g < p.N) {
                float2 f[4];
                T::unpack8(__ldg(bias4 + col / 8 + g), f);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * g + e] = add2(v[4 * g + e], f[e]);
              }
          }
          const uint32_t ob = obuf + (out_no & 1) * kLinOutBytes;
          const uint32_t cb = cbuf + (out_no & 1) * kLinCodeBytes;
          // the stores issued from these buffers two chunks ago must have read them
          if (lane == 0) bulk_wait_group_read<1>();
          __syncwarp();
          if constexpr (!kBwd && kQ) {
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) m = a8_max(a8_max(m, v[e].x), v[e].y);
            const uint32_t eb = a8_exponent(__float_as_uint(m));
            const float inv = a8_inv_step(eb);
            eb4 |= eb << (8 * j);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              st_shared_v4(cb + swz32(lane, h), a8_code4(v[8 * h], v[8 * h + 1], inv),
                           a8_code4(v[8 * h + 2], v[8 * h + 3], inv), a8_code4(v[8 * h + 4], v[8 * h + 5], inv),
                           a8_code4(v[8 * h + 6], v[8 * h + 7], inv));
          }
          if constexpr (!kBwd && kAct != kActNone) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = act_value<kAct>(v[e]);
          }
          if (has_res) {
            const uint32_t b = load_no & 1;
            if (!wait_bounded(lbar + 8 * b, (load_no >> 1) & 1, ctl, true)) {
              ok = false;
              break;
            }
            ++load_no;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              float2 f[4];
              T::unpack8(ld_shared_v4(abuf + b * kLinOutBytes + swz64(lane, g)), f);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[4 * g + e] = add2(v[4 * g + e], f[e]);
            }
          }
#pragma unroll
          for (int g = 0; g < 4; ++g)
            st_shared_v4(ob + swz64(lane, g), T::pack(v[4 * g].x, v[4 * g].y), T::pack(v[4 * g + 1].x, v[4 * g + 1].y),
                         T::pack(v[4 * g + 2].x, v[4 * g + 2].y), T::pack(v[4 * g + 3].x, v[4 * g + 3].y));
          fence_proxy_async_shared();
          __syncwarp();   // the chunk is staged, and every lane has read its load buffer
          if (lane == 0) {
            tma_store_2d(&map_out, ob, col, row0);              // clips rows past M and columns past N
            if constexpr (!kBwd && kQ) tma_store_2d(&map_codes, cb, col, row0);
            bulk_commit_group();
            if (loads && j + 2 < live) ask(j + 2);
          }
          if (loads && j + 2 < live) ++asked_no;
          ++out_no;
        }
        if (!kBwd && kQ && ok && live > 0 && row < p.M) {
          if (word) {
            *reinterpret_cast<uint32_t*>(erow) = eb4;
          } else {
            for (int j = 0; j < live; ++j) erow[j] = static_cast<uint8_t>(eb4 >> (8 * j));
          }
        }
      }
      if (!ok) {
        // loads still in flight must land before exit
        if (lane == 0)
          for (; load_no != asked_no; ++load_no)
            wait_bounded(lbar + 8 * (load_no & 1), (load_no >> 1) & 1, ctl, false);
        break;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(tempty_bar + 8 * acc, 0));
    }
    if (lane == 0) bulk_wait_group_all();
    __syncwarp();
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // no CTA leaves while its peer may touch it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, p.tmem_cols);
  }
}

// ------------------------------------------------------------------ few rows

// Cluster rank r of tile t sums k-blocks [r * kblocks / split, (r+1) * kblocks /
// split) of 128 channels x BN rows, leaves them in its shared memory as
// [row][128 channels] fp32, and finishes the rows r, r + split, ...: the sum of
// the ranks' partials in rank order, then the epilogue with one channel per
// thread (a warp is one checkpoint block of the row, and its stores are
// contiguous).  The partials take the place of the operand ring, which nothing
// reads any more once the accumulator is complete.
template <bool kBF16, bool kBwd, int kAct, bool kQ>
__global__ void __launch_bounds__(kLinRowsThreads)
    linear_rows_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                       const LinearParams p) {
  using T = Val16<kBF16>;
  extern __shared__ uint8_t lin_smem[];
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  const uint32_t warp = threadIdx.x / 32;
  const uint32_t lane = threadIdx.x % 32;
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / p.split;
  const int ch0 = (tile % p.tiles_n) * BM;
  const int row0 = (tile / p.tiles_n) * p.BN;
  const int kb_lo = rank * p.kblocks / p.split, kb_hi = (rank + 1) * p.kblocks / p.split;

  const uint32_t base = (smem_addr(lin_smem) + 1023u) & ~1023u;
  const uint32_t x_bytes = static_cast<uint32_t>(p.BN) * BK * 2;
  const uint32_t w_ring = base;
  const uint32_t x_ring = w_ring + p.stages * kLinABytes;
  const uint32_t ring_end = x_ring + p.stages * x_bytes;
  const uint32_t part_end = base + static_cast<uint32_t>(p.BN) * BM * 4;
  const uint32_t bars = ring_end > part_end ? ring_end : part_end;
  const uint32_t full_bar = bars;
  const uint32_t empty_bar = full_bar + 8 * p.stages;
  const uint32_t tfull_bar = empty_bar + 8 * p.stages;
  SharedCtl ctl{&s_abort, p.status, p.timeout_ns, 0u};

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar + 8 * s, 1);
      mbar_init(empty_bar + 8 * s, 1);
    }
    mbar_init(tfull_bar, 1);
    fence_mbar_init();
    prefetch_tensormap(&map_w);
    prefetch_tensormap(&map_x);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&s_tmem_base), p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem_base;
  griddep_wait();

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      long long issued = 0;
      bool ok = true;
      const bool stall = p.test_stall != 0;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        if (!wait_bounded(empty_bar + 8 * stage, phase ^ 1, ctl, true)) {
          ok = false;
          break;
        }
        const uint32_t fb = full_bar + 8 * stage;
        if (!(stall && issued == 0)) {
          mbar_arrive_expect_tx(fb, kLinABytes + x_bytes);
          if constexpr (kBwd) {
            for (int i = 0; i < BM / 64; ++i)
              tma_load_2d(w_ring + stage * kLinABytes + i * kMnBlockBytes, &map_w, fb, ch0 + 64 * i, kb * BK);
          } else {
            tma_load_2d(w_ring + stage * kLinABytes, &map_w, fb, kb * BK, ch0);
          }
          tma_load_2d(x_ring + stage * x_bytes, &map_x, fb, kb * BK, row0);
        }
        ++issued;
        if (++stage == static_cast<uint32_t>(p.stages)) {
          stage = 0;
          phase ^= 1;
        }
      }
      producer_finish<false>(!ok, issued, stall, p.stages, full_bar, kLinABytes + x_bytes, 0, 0, ctl, true);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        if (!wait_bounded(full_bar + 8 * stage, phase, ctl, true)) break;
        tc_fence_after();
        const uint64_t da = kBwd ? lin_desc_mn(w_ring + stage * kLinABytes, kMnBlockBytes)
                                 : smem_desc_k_sw128(w_ring + stage * kLinABytes);
        const uint64_t db = smem_desc_k_sw128(x_ring + stage * x_bytes);
#pragma unroll
        for (int k = 0; k < BK / 16; ++k)
          mma_f16_ss(tmem_base, da + (kBwd ? (2048 >> 4) : 2) * k, db + 2 * k, p.idesc, (kb != kb_lo) || k != 0);
        mma_commit(empty_bar + 8 * stage);
        if (++stage == static_cast<uint32_t>(p.stages)) {
          stage = 0;
          phase ^= 1;
        }
      }
      // completes when every product above has (also after an abort)
      mma_commit(tfull_bar);
      wait_bounded(tfull_bar, 0, ctl, false);
    }
  } else {
    const uint32_t quarter = warp & 3;
    // (not watching the abort flag: the commit above always arrives)
    if (wait_bounded(tfull_bar, 0, ctl, false) && !s_abort) {
      tc_fence_after();
      const uint32_t t_row = tmem_base + ((quarter * 32u) << 16);
      for (int j = 0; j < p.BN; j += 16) {
        uint32_t raw[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(raw[0]), "=r"(raw[1]), "=r"(raw[2]), "=r"(raw[3]), "=r"(raw[4]), "=r"(raw[5]), "=r"(raw[6]),
              "=r"(raw[7]), "=r"(raw[8]), "=r"(raw[9]), "=r"(raw[10]), "=r"(raw[11]), "=r"(raw[12]), "=r"(raw[13]),
              "=r"(raw[14]), "=r"(raw[15])
            : "r"(t_row + j)
            : "memory");
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + ((j + e) * BM + quarter * 32u + lane) * 4u), "r"(raw[e])
                       : "memory");
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_sync();   // every rank's partials are in its shared memory
  if (warp >= 2) {
    const uint32_t quarter = warp & 3;
    const int ch = ch0 + static_cast<int>(quarter * 32u + lane);
    const bool live = ch < p.N;
    const int block = (ch0 + static_cast<int>(quarter) * 32) / 32;
    float bv = 0.0f;
    if (!kBwd && p.bias != nullptr && live) bv = T::lo(p.bias[ch]);
    const uint32_t mine = base + (quarter * 32u + lane) * 4u;
    int rows = p.M - row0;
    if (rows > p.BN) rows = p.BN;
    if (block >= p.blocks) rows = 0;
    for (int m = rank; m < rows; m += p.split) {
      float v = 0.0f;
      if (p.split == 1) {
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(mine + m * (BM * 4u)) : "memory");
      } else {
        float part[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < p.split)
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(part[r])
                         : "r"(mapa_shared(mine + m * (BM * 4u), r))
                         : "memory");
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < p.split) v += part[r];
      }
      const size_t row = static_cast<size_t>(row0 + m);
      if constexpr (kBwd && kQ) {
        const uint32_t b = __ldg(p.exponents + row * p.blocks + block);
        const int k = static_cast<int8_t>(__ldg(p.codes + row * p.blocks * 32 + ch));
        v *= act_slope_safe<kAct>(static_cast<float>(k) * a8_step(b));
      } else if constexpr (!kBwd) {
        v += bv;
        if constexpr (kQ) {
          const uint32_t b = a8_exponent(__reduce_max_sync(0xFFFFFFFFu, a8_mag(v)));
          p.codes[row * p.blocks * 32 + ch] = static_cast<uint8_t>(a8_code4(make_float2(v, 0.0f), both(0.0f), a8_inv_step(b)) & 0xFFu);
          if (lane == 0) p.exponents[row * p.blocks + block] = static_cast<uint8_t>(b);
        }
        v = act_value<kAct>(v);
        if (p.has_aux && live) v += T::lo(p.residual[row * p.N + ch]);
      }
      if (live) p.out[row * p.N + ch] = static_cast<uint16_t>(T::pack(v, 0.0f) & 0xFFFFu);
    }
  }
  if (p.split > 1) cluster_sync();   // no CTA leaves while its peers may read its partials
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

}  // namespace conv3d
