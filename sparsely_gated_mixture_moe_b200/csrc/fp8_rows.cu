// Quantisation to e4m3 with block scales, and the dispatch of quantised token rows.
//
// quantise:  s = max|v| / 448 over a block (at least 2^-126), q = 448 v / max|v| rounded to
//            nearest even.  A block is 128 consecutive values of an activation row, or
//            128 x 128 of a weight matrix.
// gather:    row s of the permuted batch is token row perm_src[s] / k, scales with it
//            [Switch Transformer, switch_routing: dispatch is a gather of each expert's
//            tokens].
// Both are one pass over their data, bound by memory.
#include "fp8.cuh"
#include "internal.h"

namespace moe {

constexpr int kRowWarps = 8;
constexpr int kChunk = 1024;  // values of a row that one warp quantises: four 16-byte loads a lane

template <typename T>
__global__ void __launch_bounds__(kRowWarps * 32)
    quantize_rows_kernel(const T* __restrict__ x, uint8_t* __restrict__ q,
                         float* __restrict__ scale, int64_t rows, int d, int chunks) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int64_t row = unit / chunks;
  if (row >= rows) return;
  const int col0 = static_cast<int>(unit - row * chunks) * kChunk + lane * 8;
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (col0 + 256 * i < d) {
      load8(x + row * d + col0 + 256 * i, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = col0 + 256 * i;
    float m = kAmaxFloor;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[i][j]));
    m = amax_half_warp(m);
    if (col >= d) continue;
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = exact_quotient(v[i][j], m);
    *reinterpret_cast<uint2*>(q + row * d + col) =
        make_uint2(pack_e4m3x4(r[0], r[1], r[2], r[3]), pack_e4m3x4(r[4], r[5], r[6], r[7]));
    if ((lane & 15) == 0)
      scale[static_cast<int64_t>(col / kScaleBlock) * rows + row] = block_scale(m);
  }
}

// One 128 x 128 block a CTA: 16 lanes a row, each thread 8 rows.
template <typename T>
__global__ void __launch_bounds__(256)
    quantize_weights_kernel(const T* __restrict__ w, uint8_t* __restrict__ q,
                            float* __restrict__ scale, int n, int k, int nb, int kb) {
  __shared__ float warp_max[8];
  grid_dep_wait();
  grid_dep_launch();
  const int bk = blockIdx.x % kb;
  const int bn = (blockIdx.x / kb) % nb;
  const int64_t g = blockIdx.x / (kb * static_cast<int64_t>(nb));
  const int r0 = bn * kScaleBlock + (threadIdx.x >> 4), col = bk * kScaleBlock + (threadIdx.x & 15) * 8;
  float v[8][8];
  float m = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = r0 + 16 * i;
    if (row < n && col < k) {
      load8(w + (g * n + row) * k + col, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[i][j]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, warp_max[i]);
  if (threadIdx.x == 0) scale[(g * nb + bn) * kb + bk] = block_scale(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = r0 + 16 * i;
    if (row >= n || col >= k) continue;
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = exact_quotient(v[i][j], m);
    *reinterpret_cast<uint2*>(q + (g * n + row) * k + col) =
        make_uint2(pack_e4m3x4(r[0], r[1], r[2], r[3]), pack_e4m3x4(r[4], r[5], r[6], r[7]));
  }
}

// 32 permuted rows a CTA: each warp copies four rows in 16-byte pieces, then lane = row for
// the scales, so that a warp writes 128 consecutive bytes of a scale block's column.
__global__ void __launch_bounds__(kRowWarps * 32)
    gather_rows_fp8_kernel(const uint8_t* __restrict__ x, const float* __restrict__ xs,
                           const int32_t* __restrict__ perm_src, const int32_t* __restrict__ n_kept,
                           uint8_t* __restrict__ x_perm, float* __restrict__ xs_perm, int64_t T,
                           int k, int d, int* err) {
  __shared__ int src[32];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = T * k, s0 = static_cast<int64_t>(blockIdx.x) * 32;
  // the number of kept rows and the rows' sources in one round trip
  const int kept = *n_kept, asg = s0 + lane < n ? perm_src[s0 + lane] : -1;
  if (kept < 0 || kept > n) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_error(err, kErrOffsets);
    return;
  }
  if (s0 >= kept) return;
  if (warp == 0) {
    int t = -1;
    if (s0 + lane < kept) {
      if (asg >= 0 && asg < n) t = asg / k;
      else set_error(err, kErrSlot);  // not a permutation written by the permute step
    }
    src[lane] = t;
  }
  __syncthreads();
  const int nv = d / 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = src[warp * 4 + i];
    if (t < 0) continue;
    const uint4* from = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(t) * d);
    uint4* to = reinterpret_cast<uint4*>(x_perm + (s0 + warp * 4 + i) * d);
    for (int v = lane; v < nv; v += 32) to[v] = __ldg(from + v);
  }
  const int blocks = (d + kScaleBlock - 1) / kScaleBlock, t = src[lane];
  if (t >= 0)
    for (int b = warp; b < blocks; b += kRowWarps)
      xs_perm[b * n + s0 + lane] = __ldg(xs + b * T + t);
}

cudaError_t launch_quantize_rows(const void* x, int x_bf16, void* q, float* scale, int64_t rows,
                                 int d, const LaunchCtx& c) {
  const int chunks = (d + kChunk - 1) / kChunk;
  const int64_t blocks = (rows * chunks + kRowWarps - 1) / kRowWarps;
  const dim3 grid(static_cast<unsigned>(blocks)), block(kRowWarps * 32);
  if (x_bf16)
    return launch_kernel(quantize_rows_kernel<__nv_bfloat16>, grid, block, 0, c,
                         static_cast<const __nv_bfloat16*>(x), static_cast<uint8_t*>(q), scale, rows,
                         d, chunks);
  return launch_kernel(quantize_rows_kernel<float>, grid, block, 0, c, static_cast<const float*>(x),
                       static_cast<uint8_t*>(q), scale, rows, d, chunks);
}

cudaError_t launch_quantize_weights(const void* w, int w_bf16, void* q, float* scale,
                                    int64_t groups, int n, int k, const LaunchCtx& c) {
  const int nb = (n + kScaleBlock - 1) / kScaleBlock, kb = (k + kScaleBlock - 1) / kScaleBlock;
  const dim3 grid(static_cast<unsigned>(groups * nb * kb)), block(256);
  if (w_bf16)
    return launch_kernel(quantize_weights_kernel<__nv_bfloat16>, grid, block, 0, c,
                         static_cast<const __nv_bfloat16*>(w), static_cast<uint8_t*>(q), scale, n, k,
                         nb, kb);
  return launch_kernel(quantize_weights_kernel<float>, grid, block, 0, c,
                       static_cast<const float*>(w), static_cast<uint8_t*>(q), scale, n, k, nb, kb);
}

cudaError_t launch_gather_rows_fp8(const void* x, const float* xs, const int32_t* perm_src,
                                   const int32_t* n_kept, void* x_perm, float* xs_perm, int64_t T,
                                   int k, int d, const LaunchCtx& c) {
  const int64_t blocks = (T * k + 31) / 32;
  return launch_kernel(gather_rows_fp8_kernel, dim3(static_cast<unsigned>(blocks)),
                       dim3(kRowWarps * 32), 0, c, static_cast<const uint8_t*>(x), xs, perm_src,
                       n_kept, static_cast<uint8_t*>(x_perm), xs_perm, T, k, d, c.err);
}

}  // namespace moe
