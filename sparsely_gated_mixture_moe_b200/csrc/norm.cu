// Root-mean-square norm with the residual's addition, and its backward.
//
//   forward:   r = x + residual (stored, and normalised as stored), rstd = 1 / sqrt(mean(r^2)
//              + eps), y = r rstd w, in the layer's type and / or in e4m3 with a scale for
//              each block of 128 (both from the fp32 value: one rounding each)
//   backward:  with xhat = r rstd,  dx = dres + rstd (w dy - xhat mean(w dy xhat)),
//              dw = sum over rows of dy xhat
//
// The norm in front of an MoE layer: its 16-bit output feeds the router, its 8-bit output the
// experts.  One pass over the data, bound by memory: a row's values stay in registers (up
// to 32 a thread) between the reduction and the output, 16 lanes hold one scale block.
#include "fp8.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kVec = 4;  // 8-value vectors a thread holds

// Sum over the TPR threads of a row, to all of them, in a fixed order.  `red` holds one
// float for each warp of the block; every thread of the block must call it.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const int w0 = warp / (TPR / 32) * (TPR / 32);
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) v += red[w0 + w];
    __syncthreads();
  }
  return v;
}

template <int TPR>
constexpr int block_threads() { return TPR < 256 ? 256 : TPR; }

template <typename T, int TPR>
__global__ void __launch_bounds__(block_threads<TPR>())
    rmsnorm_kernel(const T* x, const T* residual, const T* __restrict__ weight, T* sum_out,
                   T* __restrict__ y, uint8_t* __restrict__ q, float* __restrict__ scale,
                   float* __restrict__ rstd_out, int64_t rows, int d, float eps) {
  __shared__ float red[block_threads<TPR>() / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (block_threads<TPR>() / TPR) + threadIdx.x / TPR;
  const int col0 = (threadIdx.x % TPR) * 8;
  const bool live = row < rows;
  const int64_t base = row * d;
  float v[kVec][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int col = col0 + i * TPR * 8;
    if (live && col < d) {
      load8(x + base + col, v[i]);
      if (residual != nullptr) {
        float r[8];
        load8(residual + base + col, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += r[j];
        if (sizeof(T) == 2) {
          // the stored sum is what is normalised: the backward reads it back
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = __bfloat162float(__float2bfloat16_rn(v[i][j]));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int col = col0 + i * TPR * 8;
    if (sum_out != nullptr && live && col < d) store8(sum_out + base + col, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  }
  ss = row_sum<TPR>(ss, red);
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(d) + eps);
  if (rstd_out != nullptr && live && col0 == 0) rstd_out[row] = rstd;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int col = col0 + i * TPR * 8;
    if (i * TPR * 8 >= d) break;
    const bool in = live && col < d;
    if (in) {
      float w[8];
      load8(weight + col, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * w[j];
      if (y != nullptr) store8(y + base + col, v[i]);
    }
    if (q != nullptr) {
      float m = kAmaxFloor;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[i][j]));
      m = amax_half_warp(m);
      if (in) {
        const float inv = kE4m3Max / m;
        uint32_t b[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          b[j] = pack_e4m3x4(v[i][4 * j] * inv, v[i][4 * j + 1] * inv, v[i][4 * j + 2] * inv,
                             v[i][4 * j + 3] * inv);
        *reinterpret_cast<uint2*>(q + base + col) = make_uint2(b[0], b[1]);
        if ((threadIdx.x & 15) == 0)
          scale[static_cast<int64_t>(col / kScaleBlock) * rows + row] = block_scale(m);
      }
    }
  }
}

// Each block walks rows blockIdx.x * rows-per-block, + gridDim.x * ..., its threads keeping
// the weight gradient of their columns in registers; the block's sum goes to partial
// [gridDim.x][d], summed in block order by sum_partials_kernel (or is the result itself for
// one block).  Sums are taken in a fixed order: the result does not vary from run to run.
template <typename T, int TPR>
__global__ void __launch_bounds__(block_threads<TPR>())
    rmsnorm_backward_kernel(const T* __restrict__ r, const T* __restrict__ weight,
                            const float* __restrict__ rstd_in, const float* __restrict__ dy,
                            const float* dres, float* dx, float* __restrict__ partial, int64_t rows,
                            int d) {
  constexpr int NT = block_threads<TPR>(), RPB = NT / TPR;
  __shared__ float red[NT / 32];
  __shared__ float fold[RPB > 1 ? NT * 8 : 1];
  grid_dep_wait();
  grid_dep_launch();
  const int sub = threadIdx.x / TPR, col0 = (threadIdx.x % TPR) * 8;
  float dw[kVec][8];
#pragma unroll
  for (int i = 0; i < kVec; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * RPB; r0 < rows;
       r0 += static_cast<int64_t>(gridDim.x) * RPB) {
    const int64_t row = r0 + sub;
    const bool live = row < rows;
    const int64_t base = row * d;
    const float rstd = live ? rstd_in[row] : 0.0f;
    float xh[kVec][8], g[kVec][8];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int col = col0 + i * TPR * 8;
      if (live && col < d) {
        load8(r + base + col, xh[i]);
        load8(dy + base + col, g[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) xh[i][j] = g[i][j] = 0.0f;
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int col = col0 + i * TPR * 8;
      if (col >= d) continue;
      float w[8];  // read again for each row (L1): in registers it would cost occupancy
      load8(weight + col, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] *= rstd;
        dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
        g[i][j] *= w[j];
        dot = fmaf(g[i][j], xh[i][j], dot);
      }
    }
    const float mean = row_sum<TPR>(dot, red) / static_cast<float>(d);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int col = col0 + i * TPR * 8;
      if (!live || col >= d) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = rstd * (g[i][j] - xh[i][j] * mean);
      if (dres != nullptr) {
        float e[8];
        load8(dres + base + col, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += e[j];
      }
      store8(dx + base + col, o);
    }
  }
  if (partial == nullptr) return;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int col = col0 + i * TPR * 8;
    if (RPB > 1) {
      // the block's rows in order
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) fold[threadIdx.x + NT * j] = dw[i][j];
      __syncthreads();
      if (sub == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          for (int s = 1; s < RPB; ++s) dw[i][j] += fold[threadIdx.x + s * TPR + NT * j];
      }
    }
    if (sub == 0 && col < d) store8(partial + static_cast<int64_t>(blockIdx.x) * d + col, dw[i]);
  }
}

// dweight[j] = sum over the n blocks' partials, in a fixed order: 8 threads take every eighth
// partial of a column, then their sums in order.
__global__ void __launch_bounds__(256)
    sum_partials_kernel(const float* __restrict__ partial, float* __restrict__ out, int n, int d) {
  __shared__ float part[8][32];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (col < d)
#pragma unroll 8
    for (int i = g; i < n; i += 8) s += partial[static_cast<int64_t>(i) * d + col];
  part[g][lane] = s;
  __syncthreads();
  if (g == 0 && col < d) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += part[i][lane];
    out[col] = s;
  }
}

// Threads that share a row: the fewest that hold d values, 32 a thread.
int threads_per_row(int d) {
  for (int t : {32, 128, 256})
    if (d <= t * kVec * 8) return t;
  return 512;
}

template <typename T, int TPR>
cudaError_t norm_forward(const NormProblem& p, const LaunchCtx& c) {
  const int rpb = block_threads<TPR>() / TPR;
  return launch_kernel(rmsnorm_kernel<T, TPR>, dim3(static_cast<unsigned>((p.rows + rpb - 1) / rpb)),
                       dim3(block_threads<TPR>()), 0, c, static_cast<const T*>(p.x),
                       static_cast<const T*>(p.residual), static_cast<const T*>(p.weight),
                       static_cast<T*>(p.sum_out), static_cast<T*>(p.y),
                       static_cast<uint8_t*>(p.q), p.scale, p.rstd, p.rows, p.d, p.eps);
}

template <typename T, int TPR>
cudaError_t norm_backward(const NormBackwardProblem& p, const LaunchCtx& c) {
  const int64_t rpb = block_threads<TPR>() / TPR;
  int64_t blocks = (p.rows + rpb - 1) / rpb;
  if (blocks > kNormBackwardBlocks) blocks = kNormBackwardBlocks;
  float* partial = p.dweight == nullptr ? nullptr : blocks == 1 ? p.dweight : p.partial;
  cudaError_t e = launch_kernel(rmsnorm_backward_kernel<T, TPR>, dim3(static_cast<unsigned>(blocks)),
                                dim3(block_threads<TPR>()), 0, c, static_cast<const T*>(p.r),
                                static_cast<const T*>(p.weight), p.rstd, p.dy, p.dres, p.dx, partial,
                                p.rows, p.d);
  if (e != cudaSuccess || p.dweight == nullptr || blocks == 1) return e;
  return launch_kernel(sum_partials_kernel, dim3((p.d + 31) / 32), dim3(256), 0, c,
                       static_cast<const float*>(p.partial), p.dweight, static_cast<int>(blocks), p.d);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormProblem& p, const LaunchCtx& c) {
#define MOE_NORM(TPR)                                                    \
  case TPR:                                                              \
    return p.bf16 ? norm_forward<__nv_bfloat16, TPR>(p, c) : norm_forward<float, TPR>(p, c);
  switch (threads_per_row(p.d)) {
    MOE_NORM(32) MOE_NORM(128) MOE_NORM(256) MOE_NORM(512)
  }
#undef MOE_NORM
  return cudaErrorInvalidValue;
}

cudaError_t launch_rmsnorm_backward(const NormBackwardProblem& p, const LaunchCtx& c) {
#define MOE_NORM(TPR)                                                    \
  case TPR:                                                              \
    return p.bf16 ? norm_backward<__nv_bfloat16, TPR>(p, c) : norm_backward<float, TPR>(p, c);
  switch (threads_per_row(p.d)) {
    MOE_NORM(32) MOE_NORM(128) MOE_NORM(256) MOE_NORM(512)
  }
#undef MOE_NORM
  return cudaErrorInvalidValue;
}

}  // namespace moe
