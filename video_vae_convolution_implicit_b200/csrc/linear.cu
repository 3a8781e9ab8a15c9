// linear.cu -- host side of the channel product (linear_kernel.cuh): argument
// checks, the choice between the kernels, tensor maps and launches.
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "conv3d.h"
#include "internal.h"
#include "linear_kernel.cuh"
#include "linear_wgrad.cuh"

namespace conv3d_linear {

using namespace conv3d;
using namespace conv3d_internal;

constexpr int kReserve = 1024 + 8 * (2 * MAX_STAGES + 2 + 2 + 1 + 1);   // alignment, barriers

// One product: C [M, N] = A [M, K] B^T, B = w [N, K] (forward) or w^T with w [K, N] (gradient).
struct Product {
  const void* a;
  const void* w;
  const void* bias;
  const void* residual;
  void* out;
  void* codes;
  void* exponents;
  void* value;        // gradient: act(checkpoint), also written
  int M, K, N;
  bool bwd;
  int act;
  conv3d_dtype_t dtype;
};

struct Plan {
  bool pair;
  int BN, split, stages;
  bool resident;      // pair kernel: B's column tile stays in shared memory
  int units;          // pair kernel: CTA pairs
  size_t smem;
  unsigned part;      // rows kernel: bytes of the partials
};

int env_int(const char* name) {
  const char* v = getenv(name);
  return v ? atoi(v) : 0;
}

uint32_t pow2(int v) {
  uint32_t p = 32;
  while (p < static_cast<uint32_t>(v)) p <<= 1;
  return p;
}

// Pair tiles of 256 rows x 256 or 128 columns when there are enough to keep
// about half of the SM pairs busy, otherwise the rows kernel.  Measured on B200
// (bf16, GELU, us; pair / rows kernel): 512 x 512 -> 2048 7.7 / 8.1, 256 rows of
// it 7.6 / 6.0, 1024 x 2048 -> 512 15.8 / 10.7, 1000 x 1024 -> 1024 10.3 / 11.1.
// A round of 128-column tiles takes about 0.65 of a round of 256-column ones
// (4096 x 512 -> 2048: 18.5 / 12.9; 1024 rows of it: 8.7 / 9.0).
Plan choose(const Product& P, const Device& dev) {
  Plan L{};
  const long long mt = (P.M + 255) / 256;
  const int kblocks = (P.K + BK - 1) / BK;
  const int pairs = dev.num_sms / 2;
  const long long tiles256 = mt * ((P.N + 255) / 256), tiles128 = mt * ((P.N + 127) / 128);
  const int forced = env_int("CONV3D_LINEAR");   // tuning and tests: 1 rows kernel, 128 or 256 pair tiles
  L.pair = P.M > 128 && tiles128 * 7 >= pairs * 3;
  const long long rounds256 = (tiles256 + pairs - 1) / pairs, rounds128 = (tiles128 + pairs - 1) / pairs;
  L.BN = P.N > 128 && rounds256 * 20 <= rounds128 * 13 ? 256 : 128;
  if (forced == 1) L.pair = false;
  if (forced == 128 || forced == 256) {
    L.pair = true;
    L.BN = forced;
  }
  if (L.pair) {
    L.split = 1;
    const bool q = P.codes != nullptr;
    const size_t epi = kLinEpiWarps * (lin_out_chunks(P.bwd, q, P.value != nullptr) * kLinOutBytes + (q && (P.bwd || P.residual) ? kLinCodeBytes : 0) +
                                       (P.bwd ? 0 : kLinBiasBytes));
    const size_t room = dev.max_smem_optin - 64 - kReserve - epi;
    const size_t b_bytes = static_cast<size_t>(L.BN / 2) * BK * 2;
    const int tiles_n = (P.N + L.BN - 1) / L.BN;
    const long long tiles = mt * tiles_n;
    // B resident where it leaves at least five stages for A (256 -> 1024 on
    // 36864 rows: 23.9 us, streamed 25.7; with three stages, 512 -> 2048, 81 against 74)
    // and the pairs, a multiple of the column tiles then, need at most a tenth
    // more rounds
    const long long units = pairs / tiles_n * tiles_n;
    L.resident = false;
    L.units = static_cast<int>(tiles < pairs ? tiles : pairs);
    const char* env = getenv("CONV3D_LINEAR_RESIDENT");   // tuning and tests: 0 never, 1 wherever it fits
    if (units > 0 && kblocks * b_bytes + 5 * kLinABytes <= room && (env == nullptr || env[0] != '0')) {
      const long long rounds = (tiles + pairs - 1) / pairs, rounds_r = (tiles + units - 1) / units;
      if (rounds_r * 10 <= rounds * 11 || (env != nullptr && env[0] == '1')) {
        L.resident = true;
        L.units = static_cast<int>(tiles < units ? tiles : units);
      }
    }
    const size_t stage = kLinABytes + (L.resident ? 0 : b_bytes);
    const size_t fixed = L.resident ? kblocks * b_bytes : 0;
    const size_t fit = (room - fixed) / stage;
    L.stages = static_cast<int>(fit < MAX_STAGES ? fit : MAX_STAGES);
    L.smem = kReserve + epi + fixed + L.stages * stage;
    return L;
  }
  // Rows per tile: those there are, up to 64, or 128 where 64 make more tiles
  // than SMs.  Pieces: while they fill idle SMs and keep two k-blocks each (61 x
  // 512 -> 2048: 5.3 us in two pieces, 4.4 in four).  Eight CTAs of a cluster need
  // room in one GPC, so eight pieces only for a few tiles, or where two CTAs fit an
  // SM (64 x 2048 -> 2048: 6.7 us in four pieces, 11.3 in eight; 16 rows of it 5.9
  // and 5.1; 1 x 2048 -> 512: 5.4 and 4.1).
  const long long nt = (P.N + 127) / 128;
  L.BN = P.M <= 16 ? 16 : P.M <= 32 ? 32 : nt * ((P.M + 63) / 64) <= dev.num_sms ? 64 : 128;
  const int forced_rows = env_int("CONV3D_LINEAR_ROWS");   // tuning and tests: rows per tile
  if (forced_rows == 16 || forced_rows == 32 || forced_rows == 64 || forced_rows == 128) L.BN = forced_rows;
  const long long tiles = nt * ((P.M + L.BN - 1) / L.BN);
  const int most8 = L.BN == 16 ? dev.num_sms : dev.num_sms * 2 / 3;
  L.split = 1;
  while (L.split < 8 && tiles * L.split * 2 <= (L.split < 4 ? dev.num_sms : most8) && L.split * 4 <= kblocks)
    L.split *= 2;
  const int forced_split = env_int("CONV3D_LINEAR_SPLIT");   // tuning and tests
  if (forced_split >= 1 && forced_split <= 8) L.split = forced_split <= kblocks ? forced_split : kblocks;
  const int per = (kblocks + L.split - 1) / L.split;
  const size_t stage = kLinABytes + static_cast<size_t>(L.BN) * BK * 2;
  const size_t part = static_cast<size_t>(L.split) * ((L.BN + 4 * L.split - 1) / (4 * L.split)) * BM * 16;
  L.part = static_cast<unsigned>(part);
  const size_t fit = (dev.max_smem_optin - 64 - kReserve - part) / stage;
  L.stages = per < 6 ? per : 6;
  if (static_cast<size_t>(L.stages) > fit) L.stages = static_cast<int>(fit);
  L.smem = kReserve + L.stages * stage + part;
  return L;
}

// Sets a kernel's dynamic shared memory limit once per device.
template <typename K>
conv3d_status_t allow_smem(K kern, std::atomic<unsigned long long>& done, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return CONV3D_OK;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  done.fetch_or(bit, std::memory_order_release);
  return CONV3D_OK;
}

// Dot products for one to four rows (forward), where their arithmetic and the
// blocks' waves cost less than the few-row kernel's latencies.  Measured on B200
// (bf16, GELU, weights from HBM, us; dot / few rows): 1 x 512 -> 2048 2.1 / 3.3, 1 x
// 2048 -> 512 3.2 / 4.1, 1 x 4096 -> 4096 8.1 / 9.4, 1 x 8192 -> 1024 8.7 / 8.7, 2 x
// 2048 -> 2048 4.6 / 5.0, 3 x 1024 -> 1000 3.8 / 3.9, 4 x 512 -> 2048 3.2 / 3.4; but 2 x
// 4096 -> 4096 9.8 / 9.6, 4 x 1024 -> 1000 4.2 / 3.9 and, in several waves of blocks,
// 1 x 4096 -> 14336 28.7 / 25.0, 3 x 512 of it 7.6 / 6.1 (1 x 512 of it 5.0 / 6.0).
bool choose_dot(const Product& P, const Device& dev) {
  if (P.bwd || P.M > kDotMaxRows || static_cast<long long>(P.M) * P.K * 2 > kDotMaxBytes) return false;
  const int forced = env_int("CONV3D_LINEAR");   // tuning and tests: 2 wherever it can, 1, 128 and 256 not
  if (forced != 0) return forced == 2;
  return (P.M - 1) * P.K <= 2048 && ((P.N + 31) / 32 <= dev.num_sms || (P.K <= 1024 && P.M <= 2));
}

template <bool kBF16, int kAct, bool kQ>
conv3d_status_t run_dot(const Product& P, const LinearParams& p, cudaStream_t stream) {
  const uint16_t* x = static_cast<const uint16_t*>(P.a);
  const uint16_t* w = static_cast<const uint16_t*>(P.w);
  const unsigned blocks = static_cast<unsigned>(p.blocks);
  const size_t smem = static_cast<size_t>(P.M) * P.K * 2;
  const unsigned threads = P.K > 1024 ? kDotThreads * kDotShares : kDotThreads;
  if (plan_log())
    fprintf(stderr, "libconv3d: channel product forward dot products, %d x %d x %d, %u blocks\n", P.M, P.N, P.K, blocks);
  const cudaError_t e = P.M == 1   ? launch(linear_dot_kernel<kBF16, kAct, kQ, 1>, blocks, threads, smem, 1, stream, x, w, P.K, p)
                        : P.M == 2 ? launch(linear_dot_kernel<kBF16, kAct, kQ, 2>, blocks, threads, smem, 1, stream, x, w, P.K, p)
                                   : launch(linear_dot_kernel<kBF16, kAct, kQ, 4>, blocks, threads, smem, 1, stream, x, w, P.K, p);
  return e == cudaSuccess ? CONV3D_OK : cuda_fail(e, "channel product launch");
}

template <bool kBF16, bool kBwd, int kAct, bool kQ, bool kValue = false>
conv3d_status_t run(const Product& P, cudaStream_t stream) {
  Device dev;
  conv3d_status_t st = current_device(dev);
  if (st != CONV3D_OK) return st;
  const Plan L = choose(P, dev);
  const CUtensorMapDataType dt = kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const unsigned long long K = P.K, N = P.N, M = P.M;
  LinearParams p{};
  p.M = P.M;
  p.N = P.N;
  p.kblocks = (P.K + BK - 1) / BK;
  p.BN = L.BN;
  p.split = L.split;
  p.resident = L.resident ? 1 : 0;
  p.stages = L.stages;
  p.part_bytes = L.part;
  p.bias = static_cast<const uint16_t*>(P.bias);
  p.residual = static_cast<const uint16_t*>(P.residual);
  p.out = static_cast<uint16_t*>(P.out);
  p.codes = static_cast<uint8_t*>(P.codes);
  p.exponents = static_cast<uint8_t*>(P.exponents);
  p.value = static_cast<uint16_t*>(P.value);
  p.blocks = (P.N + 31) / 32;
  p.status = dev.status;
  p.timeout_ns = wait_limit_ns();
  if constexpr (!kBwd)
    if (choose_dot(P, dev)) return run_dot<kBF16, kAct, kQ>(P, p, stream);
  p.test_stall = take_stall(p.timeout_ns) ? 1 : 0;
  CUtensorMap map_a, map_w;
  if (plan_log())
    fprintf(stderr, "libconv3d: channel product %s %s, %d x %d x %d, tiles of %d, %d pieces, %d stages, %zu B shared\n",
            kBwd ? "gradient" : "forward", L.resident ? "CTA pair, resident weight" : L.pair ? "CTA pair" : "few rows", P.M, P.N, P.K, L.BN, L.split, L.stages,
            L.smem);
  if (L.pair) {
    if ((st = encode_matrix(map_a, dt, P.a, K, M, K * 2, BK, BM, sw, "rows")) != CONV3D_OK) return st;
    st = kBwd ? encode_matrix(map_w, dt, P.w, N, K, N * 2, 64, BK, sw, "weight")
              : encode_matrix(map_w, dt, P.w, K, N, K * 2, BK, L.BN / 2, sw, "weight");
    if (st != CONV3D_OK) return st;
    p.tiles_n = (P.N + L.BN - 1) / L.BN;
    const long long tiles = static_cast<long long>(p.tiles_n) * ((P.M + 2 * BM - 1) / (2 * BM));
    if (tiles > INT_MAX / 2) {
      set_error("problem too large for 32-bit tile indexing");
      return CONV3D_ERR_UNSUPPORTED;
    }
    p.num_tiles = static_cast<int>(tiles);
    p.tmem_cols = pow2(2 * L.BN);
    p.idesc = idesc_f16(kBF16, 2 * BM, L.BN) | (kBwd ? 1u << 16 : 0u);   // bit 16: B is MN-major
    static std::atomic<unsigned long long> ready{0};
    auto kern = linear_pair_kernel<kBF16, kBwd, kAct, kQ, kValue>;
    if ((st = allow_smem(kern, ready, dev.max_smem_optin - 64)) != CONV3D_OK) return st;
    const unsigned grid = 2u * static_cast<unsigned>(L.units);
    const cudaError_t e = launch(kern, grid, kLinThreads, L.smem, 2, stream, map_a, map_w, p);
    return e == cudaSuccess ? CONV3D_OK : cuda_fail(e, "channel product launch");
  }
  st = kBwd ? encode_matrix(map_w, dt, P.w, N, K, N * 2, 64, BK, sw, "weight")
            : encode_matrix(map_w, dt, P.w, K, N, K * 2, BK, BM, sw, "weight");
  if (st != CONV3D_OK) return st;
  if ((st = encode_matrix(map_a, dt, P.a, K, M, K * 2, BK, L.BN, sw, "rows")) != CONV3D_OK) return st;
  p.tiles_n = (P.N + BM - 1) / BM;
  const long long ctas = static_cast<long long>(p.tiles_n) * ((P.M + L.BN - 1) / L.BN) * L.split;
  if (ctas > INT_MAX / 2) {
    set_error("problem too large for 32-bit tile indexing");
    return CONV3D_ERR_UNSUPPORTED;
  }
  p.tmem_cols = pow2(L.BN);
  p.idesc = idesc_f16(kBF16, BM, L.BN) | (kBwd ? 1u << 15 : 0u);   // bit 15: A (here w) is MN-major
  static std::atomic<unsigned long long> ready{0};
  auto kern = linear_rows_kernel<kBF16, kBwd, kAct, kQ>;
  if ((st = allow_smem(kern, ready, dev.max_smem_optin - 64)) != CONV3D_OK) return st;
  const cudaError_t e = launch(kern, static_cast<unsigned>(ctas), L.BN > 32 ? kLinRowsThreads : kLinFewThreads, L.smem, static_cast<unsigned>(L.split),
                               stream, map_w, map_a, p);
  return e == cudaSuccess ? CONV3D_OK : cuda_fail(e, "channel product launch");
}

template <bool kBF16>
conv3d_status_t dispatch(const Product& P, cudaStream_t stream) {
  const bool q = P.codes != nullptr;
  if (P.bwd) {
    if (!q) return run<kBF16, true, kActNone, false>(P, stream);
    if (P.value)
      return P.act == kActSilu ? run<kBF16, true, kActSilu, true, true>(P, stream) : run<kBF16, true, kActGelu, true, true>(P, stream);
    return P.act == kActSilu ? run<kBF16, true, kActSilu, true>(P, stream) : run<kBF16, true, kActGelu, true>(P, stream);
  }
  switch (P.act) {
    case kActSilu:
      return q ? run<kBF16, false, kActSilu, true>(P, stream) : run<kBF16, false, kActSilu, false>(P, stream);
    case kActGelu:
      return q ? run<kBF16, false, kActGelu, true>(P, stream) : run<kBF16, false, kActGelu, false>(P, stream);
    default:
      return q ? run<kBF16, false, kActNone, true>(P, stream) : run<kBF16, false, kActNone, false>(P, stream);
  }
}

// A persistent pair's next tile may lie this many rows behind the last one.
constexpr long long kMaxRows = INT_MAX - 65536;

// ------------------------------------------------------------------ weight gradient

constexpr int kWgPairs = 74;   // CTA pairs the row ranges are planned for (148 SMs)

// Row ranges: the fewest rounds of units times a range's stages, plus what a
// unit's epilogue costs (about three stages), a second launch (eight) and the
// parts' way through memory (a sixth of a stage each).  By sizes alone, so that
// the workspace and the order of the sums depend on nothing else.
int wgrad_splits(long long rows, int K, int N) {
  const long long chunks = (rows + kWgRows - 1) / kWgRows;
  const long long tiles = static_cast<long long>((N + kWgTile - 1) / kWgTile) * ((K + kWgTile - 1) / kWgTile);
  long long best = 1, best_cost = -1;
  for (long long s = 1; s <= chunks && s <= 148; ++s) {
    const long long rounds = (tiles * s + kWgPairs - 1) / kWgPairs;
    const long long cost = 6 * (rounds * ((chunks + s - 1) / s + 3) + (s > 1 ? 8 : 0)) + (s > 1 ? tiles * s : 0);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = s;
    }
    if (rounds > 8) break;
  }
  const int forced = env_int("CONV3D_LINEAR_WGRAD_SPLITS");   // tuning and tests
  if (forced >= 1 && forced <= chunks && forced <= best) return forced;
  return static_cast<int>(best);
}

size_t wgrad_part_bytes(long long rows, int K, int N) {
  const int s = wgrad_splits(rows, K, N);
  if (s == 1) return 0;
  const size_t tiles_n = (N + kWgTile - 1) / kWgTile, tiles_k = (K + kWgTile - 1) / kWgTile;
  return s * tiles_n * tiles_k * kWgSlotFloats * sizeof(float);
}
size_t wgrad_bias_bytes(long long rows, int K, int N) {
  const int s = wgrad_splits(rows, K, N);
  return s == 1 ? 0 : static_cast<size_t>(s) * ((N + kWgTile - 1) / kWgTile) * kWgTile * sizeof(float);
}

template <bool kBF16>
conv3d_status_t run_wgrad(const void* x, const void* dy, LinearWgradParams p, cudaStream_t stream) {
  Device dev;
  conv3d_status_t st = current_device(dev);
  if (st != CONV3D_OK) return st;
  const CUtensorMapDataType dt = kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap map_dy, map_x;
  const unsigned long long M = p.M, N = p.N, K = p.K;
  if ((st = encode_matrix(map_dy, dt, dy, N, M, N * 2, 64, kWgRows, CU_TENSOR_MAP_SWIZZLE_128B, "dy")) != CONV3D_OK) return st;
  if ((st = encode_matrix(map_x, dt, x, K, M, K * 2, 64, kWgRows, CU_TENSOR_MAP_SWIZZLE_128B, "x")) != CONV3D_OK) return st;
  p.idesc = idesc_f16(kBF16, 2 * BM, p.kw) | (1u << 15) | (1u << 16);   // both operands MN-major
  p.idesc_bias = idesc_f16(kBF16, 2 * BM, 32) | (1u << 15) | (1u << 16);
  p.status = dev.status;
  p.timeout_ns = wait_limit_ns();
  p.test_stall = take_stall(p.timeout_ns) ? 1 : 0;
  const long long units = static_cast<long long>(p.tiles) * p.splits;
  const int pairs = dev.num_sms / 2;
  const unsigned grid = 2u * static_cast<unsigned>(units < pairs ? units : pairs);
  const size_t smem = 1024 + kWgStages * kWgStageBytes + kWgOnesBytes + 8 * (2 * kWgStages + 3);
  if (plan_log())
    fprintf(stderr, "libconv3d: channel product weight gradient %d x %d x %d, %d tiles, %d row ranges of %d chunks\n", p.N,
            p.K, p.M, p.tiles, p.splits, p.chunks);
  cudaError_t e;
  if (p.splits == 1) {
    static std::atomic<unsigned long long> ready{0};
    auto kern = linear_wgrad_kernel<kBF16, true>;
    if ((st = allow_smem(kern, ready, dev.max_smem_optin - 64)) != CONV3D_OK) return st;
    e = launch(kern, grid, kWgThreads, smem, 2, stream, map_dy, map_x, p);
    return e == cudaSuccess ? CONV3D_OK : cuda_fail(e, "weight gradient launch");
  }
  static std::atomic<unsigned long long> ready{0};
  auto kern = linear_wgrad_kernel<kBF16, false>;
  if ((st = allow_smem(kern, ready, dev.max_smem_optin - 64)) != CONV3D_OK) return st;
  e = launch(kern, grid, kWgThreads, smem, 2, stream, map_dy, map_x, p);
  if (e != cudaSuccess) return cuda_fail(e, "weight gradient launch");
  const unsigned sum_blocks = static_cast<unsigned>(p.tiles) * 64 + (p.dbias ? static_cast<unsigned>((p.N + 31) / 32) : 0u);
  e = launch(linear_wgrad_sum_kernel<kBF16>, sum_blocks, 256, 0, 1, stream, p);
  return e == cudaSuccess ? CONV3D_OK : cuda_fail(e, "weight gradient sum launch");
}

conv3d_status_t check(long long rows, int K, int N, conv3d_act_t act, conv3d_dtype_t dtype) {
  if (rows < 1 || K < 1 || N < 1) {
    set_error("sizes must be >= 1");
    return CONV3D_ERR_INVALID_ARG;
  }
  if (dtype != CONV3D_F16 && dtype != CONV3D_BF16) {
    set_error("unknown dtype %d", static_cast<int>(dtype));
    return CONV3D_ERR_INVALID_ARG;
  }
  if (act < CONV3D_ACT_NONE || act > CONV3D_ACT_GELU) {
    set_error("unknown activation %d", static_cast<int>(act));
    return CONV3D_ERR_INVALID_ARG;
  }
  if (K % 8 != 0 || N % 8 != 0) {
    set_error("K and N must be multiples of 8 (got %d, %d)", K, N);
    return CONV3D_ERR_UNSUPPORTED;
  }
  if (rows > kMaxRows || K > INT_MAX - 512 || N > INT_MAX - 512) {
    set_error("problem too large for 32-bit tile indexing");
    return CONV3D_ERR_UNSUPPORTED;
  }
  return CONV3D_OK;
}

conv3d_status_t misaligned() {
  set_error("tensor pointers must be 16-byte aligned");
  return CONV3D_ERR_ALIGNMENT;
}

}  // namespace conv3d_linear

using namespace conv3d_linear;

extern "C" {

conv3d_status_t conv3d_linear_fwd(const void* x, const void* w, const void* bias, const void* residual,
                                  void* y, void* codes, void* exponents, long long rows, int K, int N,
                                  conv3d_act_t act, conv3d_dtype_t dtype, struct CUstream_st* stream) {
  conv3d_status_t st = check(rows, K, N, act, dtype);
  if (st != CONV3D_OK) return st;
  if (!x || !w || !y || (codes == nullptr) != (exponents == nullptr)) {
    set_error("x, w and y must be non-null, and codes and exponents given together");
    return CONV3D_ERR_INVALID_ARG;
  }
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(residual, 16) || !aligned(y, 16) ||
      !aligned(codes, 16) || !aligned(exponents, 16))
    return misaligned();
  const size_t xb = static_cast<size_t>(rows) * K * 2, wb = static_cast<size_t>(N) * K * 2,
               yb = static_cast<size_t>(rows) * N * 2, cb = act8_code_bytes(rows, N), sb = act8_scale_bytes(rows, N),
               bb = static_cast<size_t>(N) * 2;
  const struct { const void* p; size_t n; } outs[] = {{y, yb}, {codes, cb}, {exponents, sb}},
                                            ins[] = {{x, xb}, {w, wb}, {bias, bb}, {residual, yb}};
  for (const auto& o : outs) {
    for (const auto& i : ins)
      if (overlaps(o.p, o.n, i.p, i.n) && !(o.p == y && i.p == residual && y == residual)) {
        set_error("the outputs must not overlap the inputs (y may be exactly the residual)");
        return CONV3D_ERR_INVALID_ARG;
      }
    for (const auto& q : outs)
      if (&o != &q && overlaps(o.p, o.n, q.p, q.n)) {
        set_error("y, codes and exponents must not overlap");
        return CONV3D_ERR_INVALID_ARG;
      }
  }
  const Product P{x, w, bias, residual, y, codes, exponents, nullptr, static_cast<int>(rows), K, N, false, act, dtype};
  return dtype == CONV3D_BF16 ? dispatch<true>(P, stream) : dispatch<false>(P, stream);
}

conv3d_status_t conv3d_linear_bwd_data(const void* dy, const void* w, const void* codes,
                                       const void* exponents, conv3d_act_t act, void* dx, void* x,
                                       long long rows, int K, int N, conv3d_dtype_t dtype, struct CUstream_st* stream) {
  conv3d_status_t st = check(rows, K, N, act, dtype);
  if (st != CONV3D_OK) return st;
  if (!dy || !w || !dx || (codes == nullptr) != (exponents == nullptr)) {
    set_error("dy, w and dx must be non-null, and codes and exponents given together");
    return CONV3D_ERR_INVALID_ARG;
  }
  if (act != CONV3D_ACT_NONE && !codes) {
    set_error("the derivative of an activation needs the checkpoint of its argument");
    return CONV3D_ERR_INVALID_ARG;
  }
  if (act == CONV3D_ACT_NONE && x) {
    set_error("x is recomputed where an activation made it (CONV3D_ACT_NONE: conv3d_act8_unpack)");
    return CONV3D_ERR_INVALID_ARG;
  }
  if (!aligned(dy, 16) || !aligned(w, 16) || !aligned(codes, 16) || !aligned(exponents, 16) || !aligned(dx, 16) ||
      !aligned(x, 16))
    return misaligned();
  const size_t n = static_cast<size_t>(rows) * K * 2;
  bool clash = overlaps(dx, n, x, n);
  for (const void* o : {static_cast<const void*>(dx), static_cast<const void*>(x)})
    clash = clash || overlaps(o, n, dy, static_cast<size_t>(rows) * N * 2) ||
            overlaps(o, n, w, static_cast<size_t>(N) * K * 2) || overlaps(o, n, codes, act8_code_bytes(rows, K)) ||
            overlaps(o, n, exponents, act8_scale_bytes(rows, K));
  if (clash) {
    set_error("dx and x must not overlap the inputs or each other");
    return CONV3D_ERR_INVALID_ARG;
  }
  const bool q = act != CONV3D_ACT_NONE;   // without an activation the derivative is 1
  const Product P{dy, w, nullptr, nullptr, dx, q ? const_cast<void*>(codes) : nullptr,
                  q ? const_cast<void*>(exponents) : nullptr, x, static_cast<int>(rows), N, K, true, act, dtype};
  return dtype == CONV3D_BF16 ? dispatch<true>(P, stream) : dispatch<false>(P, stream);
}

size_t conv3d_linear_bwd_weight_workspace_bytes(long long rows, int K, int N) {
  if (rows < 1 || rows > kMaxRows || K < 1 || N < 1 || K > INT_MAX - 512 || N > INT_MAX - 512) return 0;
  const size_t b = wgrad_part_bytes(rows, K, N) + wgrad_bias_bytes(rows, K, N);
  return (b + 255) & ~static_cast<size_t>(255);
}

conv3d_status_t conv3d_linear_bwd_weight(const void* x, const void* dy, void* dw, void* dbias, long long rows,
                                         int K, int N, conv3d_dtype_t dtype, void* workspace, size_t ws_bytes,
                                         struct CUstream_st* stream) {
  conv3d_status_t st = check(rows, K, N, CONV3D_ACT_NONE, dtype);
  if (st != CONV3D_OK) return st;
  if (!x || !dy || !dw) {
    set_error("x, dy and dw must be non-null");
    return CONV3D_ERR_INVALID_ARG;
  }
  if (!aligned(x, 16) || !aligned(dy, 16) || !aligned(dw, 16) || !aligned(dbias, 16)) return misaligned();
  const size_t need = conv3d_linear_bwd_weight_workspace_bytes(rows, K, N);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) {
    set_error("workspace of %zu bytes required", need);
    return CONV3D_ERR_WORKSPACE;
  }
  if (need > 0 && !aligned(workspace, 256)) {
    set_error("workspace must be 256-byte aligned");
    return CONV3D_ERR_ALIGNMENT;
  }
  const size_t xb = static_cast<size_t>(rows) * K * 2, yb = static_cast<size_t>(rows) * N * 2,
               wb = static_cast<size_t>(N) * K * 2, bb = static_cast<size_t>(N) * 2;
  const void* ws = need > 0 ? workspace : nullptr;
  if (overlaps(dw, wb, x, xb) || overlaps(dw, wb, dy, yb) || overlaps(dbias, bb, x, xb) || overlaps(dbias, bb, dy, yb) ||
      overlaps(dw, wb, dbias, bb) || overlaps(ws, need, x, xb) || overlaps(ws, need, dy, yb) ||
      overlaps(ws, need, dw, wb) || overlaps(ws, need, dbias, bb)) {
    set_error("x, dy, dw, dbias and the workspace must not overlap");
    return CONV3D_ERR_INVALID_ARG;
  }
  LinearWgradParams p{};
  p.M = static_cast<int>(rows);
  p.N = N;
  p.K = K;
  p.chunks = static_cast<int>((rows + kWgRows - 1) / kWgRows);
  p.tiles_n = (N + kWgTile - 1) / kWgTile;
  const long long tiles = static_cast<long long>(p.tiles_n) * ((K + kWgTile - 1) / kWgTile);
  p.splits = wgrad_splits(rows, K, N);
  if (tiles * p.splits > INT_MAX / 128) {
    set_error("problem too large for 32-bit tile indexing");
    return CONV3D_ERR_UNSUPPORTED;
  }
  p.tiles = static_cast<int>(tiles);
  p.kw = K <= BM ? BM : kWgTile;
  const int most_k = p.kw / 128;
  for (int r = 0; r < 2; ++r) {
    const int n = (N - r * BM + 63) / 64, k = (K - r * p.kw / 2 + 63) / 64;
    p.boxes_n[r] = p.tiles_n > 1 || n > 2 ? 2 : n < 0 ? 0 : n;
    p.boxes_k[r] = K > kWgTile || k > most_k ? most_k : k < 0 ? 0 : k;
  }
  p.part = static_cast<float*>(workspace);
  p.bias_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + wgrad_part_bytes(rows, K, N));
  p.dw = static_cast<uint16_t*>(dw);
  p.dbias = static_cast<uint16_t*>(dbias);
  return dtype == CONV3D_BF16 ? run_wgrad<true>(x, dy, p, stream) : run_wgrad<false>(x, dy, p, stream);
}

}  // extern "C"
