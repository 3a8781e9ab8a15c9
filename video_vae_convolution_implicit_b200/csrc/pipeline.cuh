// pipeline.cuh -- what the warp-specialised tcgen05 kernels share: tile
// constants, the staging swizzle, bounded waits and the end of a producer's
// loop.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace conv3d {

constexpr int BM = 128;             // output pixels per tile (TMEM lanes)
constexpr int BK = 64;              // channels per k-block (128 bytes of fp16/bf16)
constexpr int A_STAGE_BYTES = BM * BK * 2;
constexpr int MAX_STAGES = 8;

constexpr int STATUS_TIMEOUT = 5;   // mirrors CONV3D_ERR_TIMEOUT

// Byte offset of 16-byte chunk c of row r in a 32 x 64-byte buffer written or
// read by TMA with the 64-byte swizzle (chunk index XOR bits 7-8 of the row
// offset).
__device__ __forceinline__ uint32_t swz64(uint32_t r, uint32_t c) {
  return r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
}

struct SharedCtl {
  volatile int* abort_flag;
  int* status;
  unsigned long long timeout_ns;
  uint32_t peer_abort;   // shared::cluster address of the peer CTA's abort flag (pairs), or 0
};

// Every role of this CTA (and of its peer, for a pair) leaves its loop.
__device__ __forceinline__ void raise_abort(const SharedCtl& c, int code) {
  *c.abort_flag = 1;
  if (c.peer_abort != 0) st_cluster_u32(c.peer_abort, 1);
  atomicCAS(c.status, 0, code);
}

// Wait for the phase of `bar` with the given parity.  Returns false when the
// wait ran out of time (and then raises the abort) or, if `watch_abort`, when
// another role already aborted.
static __device__ __noinline__ bool wait_bounded(uint32_t bar, uint32_t parity, const SharedCtl& c,
                                          bool watch_abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 15) == 0) {
      if (watch_abort && *c.abort_flag) return false;
      if (globaltimer_ns() - t0 > c.timeout_ns) {
        raise_abort(c, STATUS_TIMEOUT);
        return false;
      }
    }
  }
}

// The same for a barrier that the peer CTA of a pair arrives on with release
// semantics at cluster scope (what it stored before arriving is then visible).
static __device__ __noinline__ bool wait_bounded_cluster(uint32_t bar, uint32_t parity,
                                                  const SharedCtl& c) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 0;; ++i) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((i & 15) == 15 && globaltimer_ns() - t0 > c.timeout_ns) {
      raise_abort(c, STATUS_TIMEOUT);
      return false;
    }
  }
}

// End of a producer's loop.  After an abort no copy may still be writing into
// shared memory when the CTA exits, so the producer waits until every stage
// instance it (and, for a CTA pair, its peer) announced has landed:
//   issued      stage instances this producer counted; with `skip_first`
//               (the failure-detection test) instance 0 was counted but
//               neither announced nor copied;
//   half_bytes  one CTA's share of a stage's bytes (pairs).
// The copies of both CTAs of a pair complete on the even CTA's barriers, so
// the odd CTA publishes its own count in the even CTA (`peer_count`, a
// release-arrive on `peer_bar`) at the end of every run, and the even CTA
// settles each instance that only one of the two issued before waiting on it:
// an instance it announced whose odd half will never come has that half
// cancelled (complete_tx); one whose odd half is in flight but which it never
// announced is announced now for that half alone.  Both producers are paced
// by the same empty barriers and the MMAs need both halves, so the counts
// differ by at most `stages` and every instance before max - stages has been
// consumed.
template <bool kPair>
__device__ void producer_finish(bool aborted, long long issued, bool skip_first, int stages,
                                uint32_t full_bar, uint32_t half_bytes, uint32_t peer_count,
                                uint32_t peer_bar, const SharedCtl& c, bool leader) {
  if constexpr (kPair) {
    if (!leader) {
      st_cluster_u64(mapa_shared(peer_count, 0), static_cast<unsigned long long>(issued));
      mbar_arrive_cluster(mapa_shared(peer_bar, 0));
      return;
    }
  }
  if (!aborted) return;
  long long peer = issued;
  if constexpr (kPair) {
    if (!wait_bounded_cluster(peer_bar, 0, c)) return;   // the peer never reported
    unsigned long long v;
    asm volatile("ld.shared.u64 %0, [%1];" : "=l"(v) : "r"(peer_count) : "memory");
    peer = static_cast<long long>(v);
  }
  const long long top = issued > peer ? issued : peer;
  const long long first = top > stages ? top - stages : 0;
  for (long long i = first; i < top; ++i) {
    if (skip_first && i == 0) continue;
    const uint32_t fb = full_bar + 8 * static_cast<uint32_t>(i % stages);
    if constexpr (kPair) {
      if (i < issued && i >= peer) mbar_complete_tx(fb, half_bytes);
      else if (i >= issued && i < peer) mbar_arrive_expect_tx(fb, half_bytes);
    }
    wait_bounded(fb, static_cast<uint32_t>((i / stages) & 1), c, false);
  }
}

}  // namespace conv3d
