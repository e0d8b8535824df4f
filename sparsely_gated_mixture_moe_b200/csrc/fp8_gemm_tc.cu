// Products of e4m3 operands with a scale for each block of 128, dense or grouped by expert,
// on the 5th-generation tensor cores:
//
//   out[m, n] = sum_kb sA[kb, m] sB[g, n / 128, kb] (sum_{k in block kb} A[m, k] B[g, n, k])
//
// for the rows m of each group g.  The tensor cores sum one 128-deep block of the contraction
// (four K = 32 MMAs) into a TMEM accumulator; the epilogue warps take each finished block
// out of TMEM and add it, times its two scales, to fp32 sums in registers, so the scales may
// be any fp32 numbers and every sum over blocks is an fp32 multiply-add.
//
// One CTA per SM, persistent over tiles of 128 rows x BN columns (BN = 256 or 128):
//   warp 0      TMA producer: A [128 x 128 B] in boxes of 32 rows (only as many as the tile's
//               rows need) and B [BN x 128 B] per block into a ring of 128-byte-swizzled
//               stages.
//   warp 1      TMEM owner and MMA issuer: each block into the next of 512 / BN accumulators.
//   others      four epilogue warps per 128 columns: a thread owns a row and 128 columns, that
//               is one scale of A and one of B per block, and the whole scale block of an
//               e4m3 output, whose maximum it takes in registers.
// A row past the tile's last may hold anything (another group's row, an earlier stage's
// bytes): it only reaches its own output row, which is not stored.  Columns past K and rows
// past the last group read as zero.
// No cross-CTA waits; every mbarrier wait is bounded and an expired wait sets kErrTimeout,
// drains this CTA's in-flight copies and MMAs and frees TMEM.
#include "fp8.cuh"
#include "internal.h"

namespace moe {
namespace f8 {

constexpr int BM = 128;
constexpr int BK = 128;  // bytes of a k-block's rows: one scale block of the contraction
constexpr int A_BOX = 32;
constexpr int A_BYTES = BM * BK;
constexpr int RING_BYTES = 192 * 1024;
constexpr int MAX_GROUPS = 1024;
constexpr int TMEM_COLS = 512;
constexpr int SMEM_BYTES = 1024 /*align slack*/ + RING_BYTES + 256 /*barriers, flags*/ +
                           4 * (MAX_GROUPS + 1 + 40);

template <int BN>
struct Cfg {
  static constexpr int STAGE_BYTES = A_BYTES + BN * BK;
  static constexpr int STAGES = RING_BYTES / STAGE_BYTES;  // 4 (BN = 256) or 6
  static constexpr int BUFS = TMEM_COLS / BN;              // 2 or 4
  static constexpr int EPI_WARPS = BN / 32;                // 8 or 4
  static constexpr int THREADS = 64 + EPI_WARPS * 32;
  static_assert(2 * STAGES + 2 * BUFS + 2 <= 32, "barriers and flags fit 256 bytes");
};

struct Args {
  const int32_t* offsets;
  int groups, N, kblocks, n_tiles, nblocks;
  int64_t rows;
  const float* a_scale;
  const float* b_scale;
  void* out;
  float* out_scale;
  int act;
  int vec32;  // output rows start on 32-byte boundaries
  int* err;
};

struct Tile {
  int g, nt;
  int64_t row0;
  int valid;
};

__device__ __forceinline__ Tile decode_tile(int L, const int* tp, const Args& a) {
  Tile t;
  if (a.offsets == nullptr) {
    t.g = 0;
    const int mt = L / a.n_tiles;
    t.nt = L - mt * a.n_tiles;
    t.row0 = static_cast<int64_t>(mt) * BM;
    t.valid = static_cast<int>(min(static_cast<int64_t>(BM), a.rows - t.row0));
    return t;
  }
  int lo = 0, hi = a.groups - 1;  // the largest g with tp[g] * n_tiles <= L
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(tp[mid]) * a.n_tiles <= L) lo = mid; else hi = mid - 1;
  }
  t.g = lo;
  const int local = L - tp[lo] * a.n_tiles;
  const int mt = local / a.n_tiles;
  t.nt = local - mt * a.n_tiles;
  const int r0 = __ldg(a.offsets + lo), r1 = __ldg(a.offsets + lo + 1);
  t.row0 = r0 + mt * BM;
  t.valid = min(BM, r1 - static_cast<int>(t.row0));
  return t;
}

// Stores of one row's finished sums: `n` columns (a multiple of 8, at most 128) from dst on.
__device__ __forceinline__ void store_bf16(void* out, int64_t at, const uint64_t (&acc)[64], int n,
                                           int vec32) {
  uint16_t* dst = static_cast<uint16_t*>(out) + at;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    if (c * 16 >= n) break;
    uint32_t p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float lo, hi;
      f2_unpack(acc[c * 8 + j], lo, hi);
      p[j] = pack_bf16x2(lo, hi);
    }
    if (vec32 && c * 16 + 16 <= n) {
      st_global_v8(dst + c * 16, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7]);
    } else {
      *reinterpret_cast<uint4*>(dst + c * 16) = make_uint4(p[0], p[1], p[2], p[3]);
      if (c * 16 + 8 < n) *reinterpret_cast<uint4*>(dst + c * 16 + 8) = make_uint4(p[4], p[5], p[6], p[7]);
    }
  }
}

__device__ __forceinline__ void store_f32(void* out, int64_t at, const uint64_t (&acc)[64], int n,
                                          int vec32) {
  float* dst = static_cast<float*>(out) + at;
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    if (c * 8 >= n) break;
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) f2_unpack(acc[c * 4 + j], v[2 * j], v[2 * j + 1]);
    if (vec32) {
      uint32_t u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(v[j]);
      st_global_v8(dst + c * 8, u[0], u[1], u[2], u[3], u[4], u[5], u[6], u[7]);
    } else {
      store8(dst + c * 8, v);
    }
  }
}

// Activation, then the row's scale block as e4m3 and its scale.  n is a multiple of 16.  The
// values are fp32 sums: a product with the rounded reciprocal of the scale errs by at most
// 2^-23 of the quotient, against e4m3's half step of 2^-4.
template <int ACT>
__device__ __forceinline__ void store_e4m3(void* out, int64_t at, float* scale,
                                           uint64_t (&acc)[64], int n) {
  float m = kAmaxFloor;
#pragma unroll
  for (int j = 0; j < 64; ++j) {
    float lo, hi;
    f2_unpack(acc[j], lo, hi);
    if (2 * j >= n) {
      lo = hi = 0.0f;
    } else if (ACT == 1) {
      // fmaxf would turn a NaN into 0
      lo = lo < 0.0f ? 0.0f : lo;
      hi = hi < 0.0f ? 0.0f : hi;
    } else if (ACT == 2) {
      gelu2_as7126(lo, hi, lo, hi);
    }
    m = max_nan(m, max_nan(fabsf(lo), fabsf(hi)));
    acc[j] = f2_pack(lo, hi);
  }
  const uint64_t inv = f2_splat(kE4m3Max / m);
  uint8_t* dst = static_cast<uint8_t*>(out) + at;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    if (c * 16 >= n) break;
    uint32_t p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v0, v1, v2, v3;
      f2_unpack(f2_mul(acc[c * 8 + 2 * j], inv), v0, v1);
      f2_unpack(f2_mul(acc[c * 8 + 2 * j + 1], inv), v2, v3);
      p[j] = pack_e4m3x4(v0, v1, v2, v3);
    }
    *reinterpret_cast<uint4*>(dst + c * 16) = make_uint4(p[0], p[1], p[2], p[3]);
  }
  *scale = block_scale(m);
}

template <int BN, int OUT>
__global__ void __launch_bounds__(Cfg<BN>::THREADS, 1)
    fp8_gemm_tc_kernel(const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmB, const Args a) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + RING_BYTES);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = smem_u32(bars + C::STAGES);
  const uint32_t tfull0 = smem_u32(bars + 2 * C::STAGES);
  const uint32_t tempty0 = smem_u32(bars + 2 * C::STAGES + C::BUFS);
  const uint32_t drain = smem_u32(bars + 2 * C::STAGES + 2 * C::BUFS);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * C::STAGES + 2 * C::BUFS + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* scratch = reinterpret_cast<int*>(smem + RING_BYTES + 256);
  int* tp = scratch + 40;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < C::BUFS; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, C::EPI_WARPS);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), TMEM_COLS);
    tmem_relinquish();
  }
  grid_dep_wait();  // the operands come from the previous kernels on the stream
  grid_dep_launch();
  int tiles;
  if (a.offsets != nullptr) {
    const bool ok = block_tile_prefix(a.offsets, a.groups, a.rows, BM, tp, scratch);
    if (!ok && threadIdx.x == 0 && blockIdx.x == 0) set_error(a.err, kErrOffsets);
    tiles = ok ? tp[a.groups] * a.n_tiles : 0;
  } else {
    tiles = static_cast<int>((a.rows + BM - 1) / BM) * a.n_tiles;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_par = 0;
      bool aborted = false;
      for (int L = blockIdx.x; L < tiles && !aborted; L += gridDim.x) {
        const Tile t = decode_tile(L, tp, a);
        const int brow = t.g * a.N + t.nt * BN;
        const int boxes = (t.valid + A_BOX - 1) / A_BOX;
        const uint32_t tx = static_cast<uint32_t>(boxes * A_BOX * BK + BN * BK);
        for (int kb = 0; kb < a.kblocks; ++kb) {
          if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, s_abort)) {
            aborted = true;
            break;
          }
          const uint32_t st = smem_u32(ring + stage * C::STAGE_BYTES);
          const uint32_t fb = full0 + 8 * stage;
          mbar_arrive_expect_tx(fb, tx);
          tma_load_2d(st + A_BYTES, &tmB, fb, kb * BK, brow);
          for (int i = 0; i < boxes; ++i)
            tma_load_2d(st + i * A_BOX * BK, &tmA, fb, kb * BK, static_cast<int>(t.row0) + i * A_BOX);
          armed |= 1u << stage;
          armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (aborted) {
        set_error(a.err, kErrTimeout);
        *s_abort = 1;
        // let every copy this thread started land before the CTA releases its smem
        for (int s = 0; s < C::STAGES; ++s)
          if (armed & (1u << s)) mbar_wait(full0 + 8 * s, (armed_par >> s) & 1, nullptr, kDrainLimitNs);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc = idesc_f32acc(BM, BN, kFmtE4M3);
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool aborted = false;
      for (int L = blockIdx.x; L < tiles && !aborted; L += gridDim.x) {
        for (int kb = 0; kb < a.kblocks; ++kb) {
          if (!mbar_wait(tempty0 + 8 * buf, buf_phase ^ 1, s_abort) ||
              !mbar_wait(full0 + 8 * stage, phase, s_abort)) {
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(ring + stage * C::STAGE_BYTES);
          const uint32_t b0 = a0 + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            tc_mma_f8kind(tmem_base + buf * BN, sdesc_k128(a0 + kk * 32), sdesc_k128(b0 + kk * 32),
                          idesc, kk != 0 ? 1u : 0u);
          tc_commit(empty0 + 8 * stage);
          tc_commit(tfull0 + 8 * buf);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
          if (++buf == C::BUFS) {
            buf = 0;
            buf_phase ^= 1;
          }
        }
      }
      if (aborted) {
        set_error(a.err, kErrTimeout);
        *s_abort = 1;
        // wait for the MMAs already issued before TMEM is freed
        tc_commit(drain);
        mbar_wait(drain, 0, nullptr, kDrainLimitNs);
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int quarter = warp & 3;       // TMEM lane quarter this warp may read
    const int half = (warp - 2) >> 2;   // which 128 columns of the tile
    const int r = quarter * 32 + lane;
    int buf = 0;
    uint32_t buf_phase = 0;
    bool aborted = false;
    for (int L = blockIdx.x; L < tiles && !aborted; L += gridDim.x) {
      const Tile t = decode_tile(L, tp, a);
      const bool row_ok = r < t.valid;
      const bool warp_ok = quarter * 32 < t.valid;
      const int64_t row = t.row0 + (row_ok ? r : 0);
      const int nb = min(t.nt * (BN / 128) + half, a.nblocks - 1);
      const float* as = a.a_scale + row;
      const float* bs = a.b_scale + (static_cast<int64_t>(t.g) * a.nblocks + nb) * a.kblocks;
      uint64_t acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0ull;
      float s_next = __ldg(as) * __ldg(bs);
      for (int kb = 0; kb < a.kblocks; ++kb) {
        const uint64_t s = f2_splat(s_next);
        if (kb + 1 < a.kblocks)
          s_next = __ldg(as + static_cast<int64_t>(kb + 1) * a.rows) * __ldg(bs + kb + 1);
        if (!mbar_wait(tfull0 + 8 * buf, buf_phase, s_abort)) {
          aborted = true;
          break;
        }
        if (warp_ok) {
          tc_fence_after();
          const uint32_t tb = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + buf * BN + half * 128;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(tb + c * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              acc[c * 16 + j] = f2_fma(f2_pack(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])),
                                       s, acc[c * 16 + j]);
          }
          tc_fence_before();
        }
        __syncwarp();
        // relaxed: the TMEM reads are complete (tcgen05.wait::ld) and nothing else is handed on
        if (lane == 0) mbar_arrive_relaxed(tempty0 + 8 * buf);
        if (++buf == C::BUFS) {
          buf = 0;
          buf_phase ^= 1;
        }
      }
      if (aborted) {
        if (lane == 0) set_error(a.err, kErrTimeout);
        *s_abort = 1;
        break;
      }
      const int col = t.nt * BN + half * 128;
      if (row_ok && col < a.N) {
        const int n = min(128, a.N - col);
        const int64_t at = row * a.N + col;
        if (OUT == kFp8OutBf16) {
          store_bf16(a.out, at, acc, n, a.vec32);
        } else if (OUT == kFp8OutF32) {
          store_f32(a.out, at, acc, n, a.vec32);
        } else {
          float* sc = a.out_scale + static_cast<int64_t>(nb) * a.rows + row;
          if (a.act == 2) store_e4m3<2>(a.out, at, sc, acc, n);
          else if (a.act == 1) store_e4m3<1>(a.out, at, sc, acc, n);
          else store_e4m3<0>(a.out, at, sc, acc, n);
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, TMEM_COLS);
}

}  // namespace f8

template <int BN, int OUT>
static cudaError_t launch_tiles(const Fp8GemmProblem& p, f8::Args a, const LaunchCtx& c) {
  CUtensorMap tmA, tmB;
  if (!make_tmap_1b(&tmA, p.a, static_cast<uint64_t>(p.rows), p.K, f8::A_BOX) ||
      !make_tmap_1b(&tmB, p.b, static_cast<uint64_t>(p.groups) * p.N, p.K, BN))
    return cudaErrorInvalidValue;
  a.n_tiles = (p.N + BN - 1) / BN;
  // upper bound of the tile count: sum over groups of ceil(rows / 128)
  const int64_t active = p.rows < p.groups ? p.rows : p.groups;
  const int64_t tiles = (p.offsets == nullptr ? (p.rows + f8::BM - 1) / f8::BM
                                              : p.rows / f8::BM + active) * a.n_tiles;
  const int grid = static_cast<int>(tiles < c.num_sms ? tiles : c.num_sms);
  cudaError_t e = ensure_smem_limit(f8::fp8_gemm_tc_kernel<BN, OUT>, f8::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return launch_kernel(f8::fp8_gemm_tc_kernel<BN, OUT>, dim3(grid), dim3(f8::Cfg<BN>::THREADS),
                       f8::SMEM_BYTES, c, tmA, tmB, a);
}

template <int BN>
static cudaError_t launch_out(const Fp8GemmProblem& p, const f8::Args& a, const LaunchCtx& c) {
  if (p.out_type == kFp8OutBf16) return launch_tiles<BN, kFp8OutBf16>(p, a, c);
  if (p.out_type == kFp8OutF32) return launch_tiles<BN, kFp8OutF32>(p, a, c);
  return launch_tiles<BN, kFp8OutE4m3>(p, a, c);
}

cudaError_t launch_fp8_gemm(const Fp8GemmProblem& p, const LaunchCtx& c) {
  if (p.groups > f8::MAX_GROUPS) return cudaErrorInvalidValue;
  f8::Args a;
  a.offsets = p.offsets;
  a.groups = p.groups;
  a.N = p.N;
  a.kblocks = (p.K + f8::BK - 1) / f8::BK;
  a.n_tiles = 0;
  a.nblocks = (p.N + kScaleBlock - 1) / kScaleBlock;
  a.rows = p.rows;
  a.a_scale = p.a_scale;
  a.b_scale = p.b_scale;
  a.out = p.out;
  a.out_scale = p.out_scale;
  a.act = p.act;
  const int64_t row_bytes = static_cast<int64_t>(p.N) * (p.out_type == kFp8OutF32 ? 4 : 2);
  a.vec32 = row_bytes % 32 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
  a.err = c.err;
  return p.N > 128 ? launch_out<256>(p, a, c) : launch_out<128>(p, a, c);
}

}  // namespace moe
