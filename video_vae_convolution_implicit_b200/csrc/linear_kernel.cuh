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
// tcgen05.mma issuer (cta_group::2), and epilogue warps over two TMEM
// accumulators.  At 8 k-blocks a tile the epilogue has about as many issue slots
// to spend as the tensor cores take for the tile (17 instructions a value with the
// GELU derivative, two of them special functions), and a chunk is a long chain of
// dependent steps (TMEM load, arithmetic, staging, store): 16 warps, four to a
// scheduler, hide it where 8 left two thirds of the slots empty.  The chunks go out by
// plain 16-byte stores through a swizzled buffer of the warp's own, and the residual and
// the codes come in by cp.async, 16 bytes a thread, one chunk ahead.  A warp hands its
// part of the accumulator back as soon as it is in registers, by an arrival that waits
// for no global store.  Columns are the fast tile index, so the tiles in flight share
// rows of A and A is read from HBM about once; w stays in L2.
//
// Measured on B200 (bf16, 36864 rows, 512 -> 2048, 77 GFLOP, graph replays, us: a
// burst of eight after a rest / replayed for a second, at the power limit, which takes
// the clock from 1.97 to between 1.3 and 1.5 GHz): plain 73 / 85 (a plain library
// product 72 / 80), SiLU 81 / 90, GELU 81 / 94, GELU and checkpoint 96 / 112, residual
// 85 / 105, gradient 71 / 83, with GELU' from the checkpoint 92 / 108, and the
// recomputed activation 118 / 139.  104448 rows: 2048 -> 512 175 / 210 (157 / 198),
// 512 -> 2048 197 / 236 (186 / 222).  Whether the operands lie in L2 or come from HBM
// changes none of these by more than 1%; the clock does.  What bounds it: under the
// plain product the tensor cores are busy 56% of the cycles, with an activation and its
// checkpoint 43 to 46%, issue slots 50%, the special functions' unit 46%, the
// shared-memory data path 42 to 50%, HBM 30%; no unit is full, each tile's 256 KB of
// operand copies, their reads by the tensor cores and the 130 to 200 KB of staging meet
// in one shared memory, and the chip runs at its power limit.
//
// linear_rows_kernel (few rows): one 128-channel x up-to-128-row tile per
// cluster, transposed (w is the 128-row operand, the rows of x are the N side),
// with the contraction split over the cluster's CTAs, whose partial sums meet
// in shared memory: w, the bulk of the bytes, streams through as many SMs as
// there are pieces, in one launch and without a workspace, and the sum runs in
// rank order whatever the timing.  Measured (bf16, GELU, weights from HBM, graph
// replays): 8 x 512 -> 2048 3.6 us, 61 x 1024 -> 1000 5.2, 64 x 2048 -> 2048 7.1; the
// gradient with GELU' of the same sizes 4.4, 5.1 and 7.2, of 1 x 512 -> 2048 4.1:
// latencies one after the other (a first copy 0.6 us, the following k-blocks 0.3 us
// each, the meeting of the ranks 0.5 to 1.2 us).
//
// linear_dot_kernel (forward, one to four rows): dot products on the ordinary
// units, for the latency of a token.
#pragma once

#include "act8.cuh"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace conv3d {

constexpr int kLinEpiWarps = 16;
constexpr int kLinThreads = 64 + 32 * kLinEpiWarps;   // producer, issuer, epilogue
// rows kernel: producer, issuer and 16 finishing warps, or 4 where a tile has few rows
constexpr int kLinRowsThreads = 64 + 32 * 16, kLinFewThreads = 64 + 32 * 4;
constexpr uint32_t kLinABytes = BM * BK * 2;           // one CTA's A rows of a k-block
constexpr uint32_t kLinOutBytes = 32 * 32 * 2;         // a 32 x 32 chunk of 16-bit values
// Chunks in an epilogue warp's output buffer: two where it writes twice, the codes
// or the recomputed activation beside the values (104448 rows, 512 -> 2048: GELU' and
// the activation 301 us, 345 with one; 36864 rows, GELU and checkpoint 90.6, 91.8; both
// measured with a cheaper activation);
// elsewhere a pipeline stage is worth more (36864 rows, plain: 71 us with one, 76 with
// two).
__host__ __device__ constexpr int lin_out_chunks(bool bwd, bool q, bool value) { return value || (q && !bwd) ? 2 : 1; }
constexpr uint32_t kLinCodeBytes = 32 * 32;            // the same chunk's codes
constexpr uint32_t kLinBiasBytes = 64 * 4;             // the biases of a warp's (at most two) chunks

struct LinearParams {
  int M, N;                 // rows and columns of the result
  int kblocks;              // ceil(contraction / 64)
  int BN;                   // columns per tile (pair) / rows per tile (rows kernel)
  int tiles_n, num_tiles;
  int split;                // CTAs per cluster along the contraction (rows kernel)
  uint32_t part_bytes;      // rows kernel: shared memory of the partials
  int resident;             // pair kernel: the CTA keeps its half of B's column tile in shared memory
  int stages;
  uint32_t tmem_cols;
  uint32_t idesc;
  const uint16_t* bias;     // [N] or null
  const uint16_t* residual; // [M][N] or null
  uint16_t* out;            // [M][N]
  uint16_t* value;          // gradient: act(checkpoint), [M][N], or null (pair kernel: kValue says which)
  uint8_t* codes;           // written (forward) or read (gradient), [M][32 * blocks], or null
  uint8_t* exponents;       // the same, [M][blocks]
  int blocks;               // ceil(N / 32)
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
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int c, int r) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(c), "r"(r)
               : "memory");
}
// Asynchronous 16-byte copy global -> shared and its group bookkeeping.
__device__ __forceinline__ void lin_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void lin_copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void lin_copy_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Arrive once on the mbarrier at this address in both CTAs of the pair when all
// prior tcgen05 operations of this thread complete.
__device__ __forceinline__ void mma_commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Arrive on an mbarrier of either CTA of the pair without ordering this
// thread's memory operations: a release at cluster scope waits until its global
// stores have been performed, a microsecond and more at every tile.  What it
// signals, that tensor memory has been read, is complete by tcgen05.wait::ld.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void st_cluster_v4(uint32_t cluster_addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// The cluster barrier in two halves; the arrival orders no memory operations (one
// with release semantics waits for this thread's global stores).
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

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
// act'(checkpoint) when kQ, and kValue writes act(checkpoint) too).  Forward: kQ
// writes the checkpoint.  Shared
// memory: A ring, B ring (or the whole column tile of B), then per epilogue warp
// an output buffer, a code buffer (kQ, where it cannot share) and 64 fp32
// biases, then the barriers.
//
// Resident B: with a short contraction (K <= 512 at BN = 256) a CTA's half of the
// column tile fits beside the A ring.  A pair then stays with its columns and
// loads only A, which halves what each tile draws from L2 and writes into shared
// memory.
template <bool kBF16, bool kBwd, int kAct, bool kQ, bool kValue = false>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                       const LinearParams p) {
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
  const uint32_t b_ring = a_ring + p.stages * kLinABytes;      // or the whole half tile, by k-block
  const uint32_t out_buf = b_ring + (p.resident ? p.kblocks : p.stages) * b_bytes;
  const bool has_res = !kBwd && p.residual != nullptr;
  constexpr uint32_t kOutBytes = lin_out_chunks(kBwd, kQ, kValue) * kLinOutBytes;
  // codes: a buffer of their own, or the second chunk's place before its values come
  const bool own_codes = kQ && (kBwd || has_res);
  const uint32_t code_buf = out_buf + (own_codes ? kLinEpiWarps * kOutBytes : kLinOutBytes);
  const uint32_t code_step = own_codes ? kLinCodeBytes : kOutBytes;
  const uint32_t bias_buf = out_buf + kLinEpiWarps * (kOutBytes + (own_codes ? kLinCodeBytes : 0));
  const uint32_t bars = bias_buf + (kBwd ? 0 : kLinEpiWarps * kLinBiasBytes);
  const uint32_t full_bar = bars;
  const uint32_t empty_bar = full_bar + 8 * p.stages;
  const uint32_t tfull_bar = empty_bar + 8 * p.stages;
  const uint32_t tempty_bar = tfull_bar + 16;
  const uint32_t drain_bar = tempty_bar + 16;
  const uint32_t bfull_bar = drain_bar + 8;                     // the resident tile of B has landed

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
    mbar_init(bfull_bar, 1);
    mbar_init(peer_bar, 1);
    fence_mbar_init();
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_b);
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
  griddep_launch_dependents();   // a dependent's set-up may overlap this kernel; it waits in the same place

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t half_bytes = kLinABytes + (p.resident ? 0u : b_bytes);   // this CTA's share of a stage
      const bool stall = p.test_stall != 0;
      uint32_t stage = 0, phase = 0;
      long long issued = 0;
      bool ok = true;
      auto load_b = [&](uint32_t dst, uint32_t bar, int kb, int col0) {
        if constexpr (kBwd) {
          for (uint32_t i = 0; i < b_rows / 64; ++i)
            tma_load_2d_pair(dst + i * kMnBlockBytes, &map_b, bar, col0 + static_cast<int>(i) * 64, kb * BK);
        } else {
          tma_load_2d_pair(dst, &map_b, bar, kb * BK, col0);
        }
      };
      if (p.resident) {
        // every tile of this pair has the same columns (the number of pairs is
        // a multiple of the column tiles): their B is loaded once
        const int col0 = (unit % p.tiles_n) * p.BN + static_cast<int>(rank * b_rows);
        if (leader) mbar_arrive_expect_tx(bfull_bar, 2 * p.kblocks * b_bytes);
        for (int kb = 0; kb < p.kblocks; ++kb) load_b(b_ring + kb * b_bytes, mapa_shared(bfull_bar, 0), kb, col0);
      }
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
            if (leader) mbar_arrive_expect_tx(fb, 2 * half_bytes);
            const uint32_t fb_leader = mapa_shared(fb, 0);
            tma_load_2d_pair(a_ring + stage * kLinABytes, &map_a, fb_leader, kb * BK, row0);
            if (!p.resident) load_b(b_ring + stage * b_bytes, fb_leader, kb, col0);
          }
          ++issued;
          if (++stage == static_cast<uint32_t>(p.stages)) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      producer_finish<true>(!ok, issued, stall, p.stages, full_bar, half_bytes, peer_count, peer_bar, ctl, leader);
      // after an abort: B's copies, both CTAs', complete on the leader's barrier
      if (!ok && p.resident && leader) wait_bounded(bfull_bar, 0, ctl, false);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && leader) {
      uint32_t stage = 0, phase = 0;
      bool ok = !p.resident || wait_bounded(bfull_bar, 0, ctl, true);
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
          const uint32_t b_at = b_ring + (p.resident ? static_cast<uint32_t>(kb) : stage) * b_bytes;
          const uint64_t db = kBwd ? lin_desc_mn(b_at, kMnBlockBytes) : smem_desc_k_sw128(b_at);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)   // 16 values along the contraction: 32 bytes of a K-major row, 16 rows of an MN-major block
            mma_f16_ss_pair(d_tmem, da + 2 * k, db + (kBwd ? (2048 >> 4) : 2) * k, p.idesc, (kb | k) != 0);
          mma_commit_both(empty_bar + 8 * stage);
          if (++stage == static_cast<uint32_t>(p.stages)) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        mma_commit_both(tfull_bar + 8 * acc);
      }
      mma_commit_pair(drain_bar);
      wait_bounded(drain_bar, 0, ctl, false);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // Four warps share each quarter of the TMEM lanes (32 rows of the tile) and
    // take a quarter of its columns each, 32 at a time: one row and one
    // checkpoint block per thread, so the block's exponent needs no exchange.
    const uint32_t quarter = warp & 3;
    const uint32_t ew = warp - 2;
    const int share = static_cast<int>(ew) / 4;
    const int nj = p.BN / 128;                                 // chunks per warp and tile
    const uint32_t ob = out_buf + ew * kOutBytes;
    const uint32_t cb = code_buf + ew * code_step;
    const uint32_t bb = bias_buf + ew * kLinBiasBytes;
    // this lane's 16 bytes of a chunk's rows in the row-contiguous order of
    // global memory: four lanes a 64-byte row of values, two a 32-byte row of codes
    const int vrow = static_cast<int>(lane >> 2), vpart = static_cast<int>(lane & 3);
    const int crow = static_cast<int>(lane >> 1), cpart = static_cast<int>(lane & 1);
    constexpr bool kLoadCodes = kBwd && kQ;
    const bool loads = has_res || kLoadCodes;
    // A tile and where this warp's rows and columns of it begin; the next one is
    // num_units further, found by addition.
    struct Place {
      int t, nt, row0, col0;
    };
    const int step_m = num_units / p.tiles_n, step_n = num_units - step_m * p.tiles_n;
    auto advance = [&](Place& a) {
      a.t += num_units;
      a.nt += step_n;
      a.row0 += step_m * 2 * BM;
      a.col0 += step_n * p.BN;
      if (a.nt >= p.tiles_n) {
        a.nt -= p.tiles_n;
        a.row0 += 2 * BM;
        a.col0 -= p.tiles_n * p.BN;
      }
    };
    // how many of the warp's chunks hold part of the result
    auto live_chunks = [&](const Place& a) {
      const int live = (p.N - a.col0 + 31) >> 5;
      return a.row0 >= p.M || live < 0 ? 0 : live > nj ? nj : live;
    };
    Place here;
    here.t = unit;
    here.nt = unit % p.tiles_n;
    here.row0 = (unit / p.tiles_n) * 2 * BM + static_cast<int>(rank) * BM + static_cast<int>(quarter) * 32;
    here.col0 = here.nt * p.BN + share * nj * 32;
    constexpr bool kTwo = lin_out_chunks(kBwd, kQ, kValue) == 2;
    // Place of 16-byte piece c of row r of the warp's chunk j.  (Two chunks' pieces of a
    // row lie in different banks.)
    auto slot = [&](int j, int r, int c) {
      const uint32_t at = swz64(static_cast<uint32_t>(r), static_cast<uint32_t>(c));
      return ob + (!kTwo || j == 0 ? at : kLinOutBytes + (at ^ 64u));
    };
    // What the warp's next live chunk reads, of this tile or a later one, is always
    // under way: its codes, and its exponent byte with them, as soon as the chunk
    // before it has been decoded; its residual (in a buffer of two chunks, the next
    // tile's) as soon as the output buffer is free, in which the sum replaces it.
    Place next = here;
    int next_j = 0;
    uint32_t next_eb = 0;
    auto ask = [&]() {
      while (next.t < p.num_tiles && next_j >= live_chunks(next)) {
        advance(next);
        next_j = 0;
      }
      if (next.t >= p.num_tiles) return;
      const int row0 = next.row0;
      if constexpr (kLoadCodes) {
        const int col = next.col0 + 32 * next_j;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = crow + 16 * i;
          if (row0 + r < p.M)
            lin_copy16(cb + swz32(r, cpart),
                       p.codes + (static_cast<size_t>(row0 + r) * p.blocks + col / 32) * 32 + cpart * 16);
        }
        const int row = row0 + static_cast<int>(lane);
        next_eb = row < p.M ? __ldg(p.exponents + static_cast<size_t>(row) * p.blocks + col / 32) : 0u;
        ++next_j;
      } else {
        do {
          const int col = next.col0 + 32 * next_j;
          if (col + vpart * 8 < p.N) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = vrow + 8 * i;
              if (row0 + r < p.M)
                lin_copy16(slot(next_j, r, vpart), p.residual + static_cast<size_t>(row0 + r) * p.N + col + vpart * 8);
            }
          }
        } while (++next_j < live_chunks(next) && kTwo);
      }
      lin_copy_commit();
    };
    if (loads) ask();
    int local = 0;
    int bias_col = -1;
    for (; here.t < p.num_tiles; advance(here), ++local) {
      const uint32_t acc = local & 1;
      const int row0 = here.row0, col0 = here.col0;
      const int live = live_chunks(here);
      const int row = row0 + static_cast<int>(lane);
      if (!kBwd && bias_col != col0 && live > 0) {              // this warp's biases, as fp32
        bias_col = col0;
        for (int c = static_cast<int>(lane); c < nj * 32; c += 32) {
          const float v = p.bias != nullptr && col0 + c < p.N ? T::lo(__ldg(p.bias + col0 + c)) : 0.0f;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(bb + c * 4u), "f"(v) : "memory");
        }
        __syncwarp();
      }
      if (!__all_sync(0xFFFFFFFFu, wait_bounded(tfull_bar + 8 * acc, (local >> 1) & 1, ctl, true))) break;   // the warp leaves as one
      tc_fence_after();
      const uint32_t t_row =
          tmem_base + ((quarter * 32u) << 16) + acc * static_cast<uint32_t>(p.BN) + share * nj * 32;
      // this warp has read its part of the accumulator: the next products may have it
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(tempty_bar + 8 * acc, 0));
      };
      if (live == 0) release();
      uint32_t first_eb = 0;
      for (int j = 0; j < live; ++j) {
        const int col = col0 + 32 * j;
        uint32_t raw[32];
        tmem_ld_32x32b_x32(t_row + j * 32, raw);
        uint32_t packed[16], packed_value[kValue ? 16 : 1];
        if constexpr (kLoadCodes) {
          lin_copy_wait();
          __syncwarp();
          const uint32_t eb = next_eb;
          const uint4 k0 = ld_shared_v4(cb + swz32(lane, 0));
          const uint4 k1 = ld_shared_v4(cb + swz32(lane, 1));
          __syncwarp();
          ask();
          const uint32_t ka[4] = {k0.x, k0.y, k0.z, k0.w}, kb[4] = {k1.x, k1.y, k1.z, k1.w};
          tmem_ld_wait();
          if (j + 1 == live) release();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float2 v[8];
            const float half = 0.5f * a8_step(eb);
            a8_decode_halves<kAct, !kValue>(h ? kb : ka, half, v);
            auto multiply = [&](int e, float2 slope) {
              const float2 d = mul2(slope, make_float2(__uint_as_float(raw[16 * h + 2 * e]),
                                                       __uint_as_float(raw[16 * h + 2 * e + 1])));
              packed[8 * h + e] = T::pack(d.x, d.y);
            };
            if constexpr (kValue) {
              auto both_of = [&](int e, float2 narrowed) {
                float2 value;
                multiply(e, act_slope_and_value<kAct>(v[e], narrowed, value));
                packed_value[8 * h + e] = T::pack(value.x, value.y);
              };
              if (a8_wide<kAct>(half)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) both_of(e, a8_narrow<kAct>(v[e]));
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) both_of(e, v[e]);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) multiply(e, act_slope_of_half<kAct>(v[e]));
            }
          }
        } else {
          tmem_ld_wait();
          if (j + 1 == live) release();
          float2 v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = make_float2(__uint_as_float(raw[2 * e]), __uint_as_float(raw[2 * e + 1]));
          if constexpr (!kBwd) {
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const uint4 b = ld_shared_v4(bb + (j * 32 + g * 4) * 4u);
              v[2 * g] = add2(v[2 * g], make_float2(__uint_as_float(b.x), __uint_as_float(b.y)));
              v[2 * g + 1] = add2(v[2 * g + 1], make_float2(__uint_as_float(b.z), __uint_as_float(b.w)));
            }
          }
          if constexpr (!kBwd && kQ) {
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) m = a8_max(m, v[e]);
            const uint32_t mag = __float_as_uint(m);
            const uint32_t eb = a8_exponent(mag);
            const float inv = a8_inv_step(eb);
            uint32_t q[8];
            if (a8_clamps(mag)) {
#pragma unroll
              for (int e = 0; e < 8; ++e) q[e] = a8_code4(v[2 * e], v[2 * e + 1], inv);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) q[e] = a8_bytes(a8_round(v[2 * e], inv), a8_round(v[2 * e + 1], inv));
            }
            st_shared_v4(cb + swz32(lane, 0), q[0], q[1], q[2], q[3]);
            st_shared_v4(cb + swz32(lane, 1), q[4], q[5], q[6], q[7]);
            __syncwarp();
            uint8_t* dst = p.codes + (static_cast<size_t>(row0 + crow) * p.blocks + col / 32) * 32 + cpart * 16;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (row0 + crow + 16 * i < p.M)
                *reinterpret_cast<uint4*>(dst + static_cast<size_t>(16 * i) * p.blocks * 32) =
                    ld_shared_v4(cb + swz32(crow + 16 * i, cpart));
            __syncwarp();
            // two chunks' bytes in one store where a row's blocks are even in number
            // (col0 / 32 is even then, and the second chunk holds a block too)
            uint8_t* e8 = p.exponents + static_cast<size_t>(row) * p.blocks + col / 32;
            if (nj == 2 && (p.blocks & 1) == 0) {
              if (j == 0) first_eb = eb;
              else if (row < p.M) *reinterpret_cast<uint16_t*>(e8 - 1) = static_cast<uint16_t>(first_eb | eb << 8);
            } else if (row < p.M) {
              *e8 = static_cast<uint8_t>(eb);
            }
          }
          if constexpr (!kBwd && kAct != kActNone) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = act_value<kAct>(v[e]);
          }
          if (has_res) {
            lin_copy_wait();
            __syncwarp();
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              float2 f[4];
              T::unpack8(ld_shared_v4(slot(j, lane, g)), f);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[4 * g + e] = add2(v[4 * g + e], f[e]);
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) packed[e] = T::pack(v[e].x, v[e].y);
        }
        // Into the output buffer, and out of it in whole rows: 64 bytes of each, or 128
        // of two chunks together (four lines a store instead of eight: the stores share
        // the data path of shared memory)
        auto stage = [&](int place, const uint32_t* w) {
#pragma unroll
          for (int g = 0; g < 4; ++g) st_shared_v4(slot(place, lane, g), w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
        };
        auto put = [&](int place, uint16_t* to) {
          if (col + vpart * 8 >= p.N) return;
          uint16_t* dst = to + static_cast<size_t>(row0 + vrow) * p.N + col + vpart * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (row0 + vrow + 8 * i < p.M)
              *reinterpret_cast<uint4*>(dst + static_cast<size_t>(8 * i) * p.N) = ld_shared_v4(slot(place, vrow + 8 * i, vpart));
        };
        if constexpr (kValue) {
          stage(0, packed);
          stage(1, packed_value);
          __syncwarp();
          put(0, p.out);
          put(1, p.value);
          __syncwarp();   // the buffer is free again
        } else {
          stage(j, packed);
          if (!kTwo || j + 1 == live) {
            __syncwarp();
            if (!kTwo || live == 1) {
              put(0, p.out);
            } else {
              const int wrow = static_cast<int>(lane >> 3), wpart = static_cast<int>(lane & 7);
              if (col0 + wpart * 8 < p.N) {
                uint16_t* dst = p.out + static_cast<size_t>(row0 + wrow) * p.N + col0 + wpart * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (row0 + wrow + 4 * i < p.M)
                    *reinterpret_cast<uint4*>(dst + static_cast<size_t>(4 * i) * p.N) =
                        ld_shared_v4(slot(wpart >> 2, wrow + 4 * i, wpart & 3));
              }
            }
            __syncwarp();   // the buffer is free again
            if (has_res) ask();
          }
        }
      }
    }
    lin_copy_wait();
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
// split) of 128 channels x BN rows and hands each rank an equal share of the rows
// of its fp32 sums; that rank adds the partials of its rows in rank order and
// finishes them with one channel per thread (a warp is one checkpoint block of the
// row, and its stores are contiguous), four rows of a warp at a time, which are
// one 16-byte access of a partial.  These calls last a
// few microseconds, most of it one latency after the other, so: the first copies
// are issued by the thread that initialises the barriers, before the other warps
// have met; what the epilogue reads is asked for before the products; partials
// are written into their owner's shared memory (beside its operand ring, which it
// may still be reading) and not fetched from the ranks after a barrier, a round
// trip more; and nothing waits for global stores but the end of the grid.
template <bool kBF16, bool kBwd, int kAct, bool kQ>
__global__ void __launch_bounds__(kLinRowsThreads, 1)
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
  // a rank's share of the tile's rows, whole fours; its partials as [rank][fours][128 channels][4]
  const int tile_rows = p.M - row0 < p.BN ? p.M - row0 : p.BN;
  const int share = (tile_rows + 4 * p.split - 1) / (4 * p.split) * 4;
  const uint32_t parts = ring_end;
  const uint32_t full_bar = parts + p.part_bytes;
  const uint32_t empty_bar = full_bar + 8 * p.stages;
  const uint32_t tfull_bar = empty_bar + 8 * p.stages;
  SharedCtl ctl{&s_abort, p.status, p.timeout_ns, 0u};

  uint32_t stage = 0, phase = 0;   // producer and issuer
  long long issued = 0;
  auto load = [&](int kb) {
    const uint32_t fb = full_bar + 8 * stage;
    if (!(p.test_stall != 0 && issued == 0)) {
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
  };
  int first = kb_lo;               // producer: the next k-block to load
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar + 8 * s, 1);
      mbar_init(empty_bar + 8 * s, 1);
    }
    mbar_init(tfull_bar, 1);
    fence_mbar_init();
    // With a token or a few, the way of the weight's first stages from HBM to L2 may
    // overlap the previous kernel (L2 stays coherent should that write them): 1 x 512
    // -> 2048 3.25 us, 3.43 without, 1 x 4096 -> 4096 9.2 and 9.7; 3.22 and 3.14 where
    // the weight is in L2 already.  All of a long contraction would pass this SM's copy
    // engine twice (1 x 8192 -> 8192 32.8 us, 26.2 with the first stages only).
    for (int kb = kb_lo; p.BN <= 32 && kb < kb_hi && kb < kb_lo + p.stages; ++kb) {
      if constexpr (kBwd) {
        for (int i = 0; i < BM / 64; ++i) tma_prefetch_2d(&map_w, ch0 + 64 * i, kb * BK);
      } else {
        tma_prefetch_2d(&map_w, kb * BK, ch0);
      }
    }
    griddep_wait();                // no global memory is touched before the previous kernel has finished
    for (; first < kb_hi && first < kb_lo + p.stages; ++first) load(first);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&s_tmem_base), p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.split > 1) cluster_arrive_relaxed();   // this CTA runs: its shared memory may be written
  const uint32_t tmem_base = s_tmem_base;
  griddep_wait();
  griddep_launch_dependents();

  // The finishing warps' part: channel `ch` of every `groups`-th four of the rank's
  // rows.  What they read beside the sums is asked for now.
  constexpr int kBatch = 4;
  const uint32_t quarter = warp & 3;
  const int ch = ch0 + static_cast<int>(quarter * 32u + lane);
  const bool live = ch < p.N;
  const int block = (ch0 + static_cast<int>(quarter) * 32) / 32;
  int rows = (rank + 1) * share;   // the end of this warp's rows
  if (rows > tile_rows) rows = tile_rows;
  if (block >= p.blocks || warp < 2) rows = 0;
  const int group = (static_cast<int>(warp) - 2) / 4, groups = (static_cast<int>(blockDim.x) / 32 - 2) / 4;
  const int m_first = rank * share + kBatch * group;
  float bv = 0.0f, aux[kBatch];
  uint32_t eb[kBatch];
  if (!kBwd && p.bias != nullptr && live) bv = T::lo(p.bias[ch]);
  auto ask = [&](int m0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int m = m0 + i;
      aux[i] = 0.0f;
      eb[i] = 7u;
      if (m < rows) {
        const size_t row = static_cast<size_t>(row0 + m);
        if constexpr (kBwd && kQ) {
          eb[i] = __ldg(p.exponents + row * p.blocks + block);
          aux[i] = static_cast<float>(static_cast<int8_t>(__ldg(p.codes + row * p.blocks * 32 + ch)));
        } else if (!kBwd && p.residual != nullptr && live) {
          aux[i] = T::lo(p.residual[row * p.N + ch]);
        }
      }
    }
  };
  ask(m_first);

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      for (int kb = first; ok && kb < kb_hi; ++kb) {
        ok = wait_bounded(empty_bar + 8 * stage, phase ^ 1, ctl, true);
        if (ok) load(kb);
      }
      producer_finish<false>(!ok, issued, p.test_stall != 0, p.stages, full_bar, kLinABytes + x_bytes, 0, 0, ctl, true);
    }
  } else if (warp == 1) {
    if (lane == 0) {
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
  }
  if (p.split > 1) {
    __syncwarp();
    cluster_wait();
  }
  if (warp >= 2) {
    // (not watching the abort flag: the commit above always arrives)
    if (__all_sync(0xFFFFFFFFu, wait_bounded(tfull_bar, 0, ctl, false) && !s_abort)) {   // the warp as one
      tc_fence_after();
      const uint32_t t_row = tmem_base + ((quarter * 32u) << 16);
      const uint32_t at = parts + (static_cast<uint32_t>(rank * share / 4) * BM + quarter * 32u + lane) * 16u;
      for (int j = 16 * group; j < tile_rows; j += 16 * groups) {
        uint32_t raw[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(raw[0]), "=r"(raw[1]), "=r"(raw[2]), "=r"(raw[3]), "=r"(raw[4]), "=r"(raw[5]), "=r"(raw[6]),
              "=r"(raw[7]), "=r"(raw[8]), "=r"(raw[9]), "=r"(raw[10]), "=r"(raw[11]), "=r"(raw[12]), "=r"(raw[13]),
              "=r"(raw[14]), "=r"(raw[15])
            : "r"(t_row + j)
            : "memory");
        int owner = j / share, four = (j - owner * share) / 4;
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          if (j + e < tile_rows) {
            const uint32_t to = at + static_cast<uint32_t>(four) * (BM * 16u);
            if (p.split == 1)
              st_shared_v4(to, raw[e], raw[e + 1], raw[e + 2], raw[e + 3]);
            else
              st_cluster_v4(mapa_shared(to, static_cast<uint32_t>(owner)), raw[e], raw[e + 1], raw[e + 2], raw[e + 3]);
          }
          if (4 * ++four == share) {
            four = 0;
            ++owner;
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if (p.split > 1) cluster_sync();   // every rank's partials of this rank's rows are here
  else __syncthreads();
  if (warp >= 2) {
    uint32_t mine = parts + (static_cast<uint32_t>(group) * BM + quarter * 32u + lane) * 16u;
    for (int m0 = m_first; m0 < rows; m0 += kBatch * groups, mine += groups * (BM * 16u)) {
      if (m0 != m_first) ask(m0);
      float v[kBatch] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int r = 0; r < p.split; ++r) {
        const uint4 part = ld_shared_v4(mine + static_cast<uint32_t>(r * share / 4) * (BM * 16u));
        v[0] += __uint_as_float(part.x);
        v[1] += __uint_as_float(part.y);
        v[2] += __uint_as_float(part.z);
        v[3] += __uint_as_float(part.w);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int m = m0 + i;
        if (m >= rows) break;
        const size_t row = static_cast<size_t>(row0 + m);
        float y = v[i];
        if constexpr (kBwd && kQ) {
          const float pre = aux[i] * a8_step(eb[i]);
          y *= act_slope_safe<kAct>(pre);
          if (p.value != nullptr && live)
            p.value[row * p.N + ch] = static_cast<uint16_t>(T::pack(act_value<kAct>(pre), 0.0f) & 0xFFFFu);
        } else if constexpr (!kBwd) {
          y += bv;
          if constexpr (kQ) {
            const uint32_t b = a8_exponent(__reduce_max_sync(0xFFFFFFFFu, a8_mag(y)));
            p.codes[row * p.blocks * 32 + ch] =
                static_cast<uint8_t>(a8_code4(make_float2(y, 0.0f), both(0.0f), a8_inv_step(b)) & 0xFFu);
            if (lane == 0) p.exponents[row * p.blocks + block] = static_cast<uint8_t>(b);
          }
          y = act_value<kAct>(y) + aux[i];
        }
        if (live) p.out[row * p.N + ch] = static_cast<uint16_t>(T::pack(y, 0.0f) & 0xFFFFu);
      }
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

// ------------------------------------------------------------------ one to four rows

// Forward with M <= R rows: dot products.  A matrix instruction would have 124 of
// its 128 rows idle, and what a call of a token costs is latency: here there is no
// tensor map to fetch, no tensor memory and no cluster to meet.  A block takes 32
// channels (one checkpoint block), a warp two of them, its lanes their contraction,
// 16 bytes a load and kUnroll loads of each channel in flight; twice the warps share
// a contraction of more than 1024.  x lies in shared memory as it came.  fp32 sums
// per lane, then over the lanes in a fixed tree, then the shares.  Measured (graph
// replays): 1 x 512 -> 2048 2.1 us (1.9 with the weight in L2; a layer norm of the
// row takes 1.6), 1 x 4096 -> 4096 8.1 us (4.1 TB/s): loads' latency, in one batch up
// to a contraction of 2048 and one after the other beyond.
constexpr int kDotThreads = 512;                       // per share of the contraction
constexpr int kDotShares = 2;                          // at most, each with its own warps
constexpr int kDotMaxRows = 4;
constexpr int kDotMaxBytes = 32 * 1024;                // of x in shared memory

template <bool kBF16, int kAct, bool kQ, int R>
__global__ void __launch_bounds__(kDotThreads * kDotShares, 1)
    linear_dot_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ w, const int K, const LinearParams p) {
  using T = Val16<kBF16>;
  constexpr int kUnroll = 4;
  extern __shared__ __align__(16) uint8_t dot_x[];
  __shared__ float sums[kDotShares][R][32];
  const int share = threadIdx.x / kDotThreads, shares = blockDim.x / kDotThreads;
  const int warp = threadIdx.x % kDotThreads / 32, lane = threadIdx.x % 32;
  const int ch0 = blockIdx.x * 32;
  const int vecs = K / 8;
  const int c0 = ch0 + 2 * warp;
  const bool live = c0 < p.N;                          // N is even: both channels or none
  const int lo = share * vecs / shares, hi = (share + 1) * vecs / shares;   // this share's vectors
  const uint4* wa = reinterpret_cast<const uint4*>(w + static_cast<size_t>(live ? c0 : 0) * K);
  const uint4* wb = wa + vecs;
  const uint32_t xs = smem_addr(dot_x);
  // into L2 while the previous kernel ends (L2 stays coherent should that write it)
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int v = lo + lane + 32 * i;
    if (live && v < hi && (lane & 7) == 0) {
      asm volatile("prefetch.global.L2 [%0];" ::"l"(wa + v) : "memory");
      asm volatile("prefetch.global.L2 [%0];" ::"l"(wb + v) : "memory");
    }
  }
  griddep_wait();
  griddep_launch_dependents();
  uint4 a[kUnroll], b[kUnroll];
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int v = base + lane + 32 * i;
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (live && v < hi) {
        a[i] = __ldg(wa + v);
        b[i] = __ldg(wb + v);
      }
    }
  };
  load(lo);
  for (int i = threadIdx.x; i < p.M * vecs; i += blockDim.x) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(x) + i);
    st_shared_v4(xs + i * 16u, q.x, q.y, q.z, q.w);
  }
  __syncthreads();
  float2 acc[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r][0] = acc[r][1] = both(0.0f);
  for (int base = lo; live && base < hi; base += 32 * kUnroll) {
    if (base != lo) load(base);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int v = base + lane + 32 * i;
      if (v < hi) {
        float2 fa[4], fb[4];
        T::unpack8(a[i], fa);
        T::unpack8(b[i], fb);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (r < p.M) {
            float2 fx[4];
            T::unpack8(ld_shared_v4(xs + (r * vecs + v) * 16u), fx);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[r][0] = fma2(fa[e], fx[e], acc[r][0]);
              acc[r][1] = fma2(fb[e], fx[e], acc[r][1]);
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float v = acc[r][c].x + acc[r][c].y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      if (lane == 0) sums[share][r][2 * warp + c] = v;
    }
  __syncthreads();
  if (share != 0 || warp >= p.M) return;               // a warp finishes a row, a lane a channel
  const int ch = ch0 + lane;
  const size_t row = warp;
  float y = sums[0][warp][lane];
  for (int s = 1; s < shares; ++s) y += sums[s][warp][lane];
  if (p.bias != nullptr && ch < p.N) y += T::lo(__ldg(p.bias + ch));
  if constexpr (kQ) {
    const uint32_t eb = a8_exponent(__reduce_max_sync(0xFFFFFFFFu, a8_mag(y)));
    p.codes[row * p.blocks * 32 + ch] =
        static_cast<uint8_t>(a8_code4(make_float2(y, 0.0f), both(0.0f), a8_inv_step(eb)) & 0xFFu);
    if (lane == 0) p.exponents[row * p.blocks + blockIdx.x] = static_cast<uint8_t>(eb);
  }
  y = act_value<kAct>(y);
  if (ch < p.N) {
    y += p.residual != nullptr ? T::lo(p.residual[row * p.N + ch]) : 0.0f;
    p.out[row * p.N + ch] = static_cast<uint16_t>(T::pack(y, 0.0f) & 0xFFFFu);
  }
}

}  // namespace conv3d
