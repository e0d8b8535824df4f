// C ABI of the norm and the 8-bit operators (declared in include/moe.h): host-side argument
// validation and launches.
#include <limits.h>

#include "internal.h"
#include "moe.h"

namespace moe {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Entry {
  LaunchCtx lc;
  int launches = 0;
  bool ok = false;
  Entry(void* ws, moe_stream_t stream) {
    lc.stream = reinterpret_cast<cudaStream_t>(stream);
    lc.err = static_cast<int*>(ws);
    lc.launches = &launches;
    int dev = 0;
    ok = cudaGetDevice(&dev) == cudaSuccess &&
         cudaDeviceGetAttribute(&lc.num_sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
  }
  moe_status finish(cudaError_t e) {
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    set_last_launch_count(launches);
    return MOE_OK;
  }
};

moe_status nothing_to_do() {
  set_last_launch_count(0);
  return MOE_OK;
}

// Longest row or contraction: block counts and coordinates are 32-bit.
constexpr int64_t kMaxWidth = int64_t{1} << 30;

// rows and columns of a matrix whose rows are read in vectors of `step` values
moe_status check_rows(int64_t rows, int64_t d, int step) {
  if (rows < 0 || d <= 0) return MOE_ERR_INVALID_ARG;
  if (rows >= (int64_t{1} << 31) || d > kMaxWidth || d % step != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_dtype(int32_t dtype) {
  return dtype == MOE_F32 || dtype == MOE_BF16 ? MOE_OK : MOE_ERR_INVALID_ARG;
}

int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

moe_status check_norm(int64_t rows, int32_t d, int32_t dtype) {
  moe_status st = check_rows(rows, d, 8);
  if (st != MOE_OK) return st;
  if ((st = check_dtype(dtype)) != MOE_OK) return st;
  return d > kNormMaxWidth ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status check_product(int64_t rows, int32_t N, int32_t K, int64_t groups, int32_t out_dtype) {
  if (rows < 0 || N <= 0 || K <= 0 || groups <= 0) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_dtype(out_dtype);
  if (st != MOE_OK) return st;
  if (N % 8 != 0 || K % 16 != 0 || K > kMaxWidth || groups > 1024) return MOE_ERR_UNSUPPORTED;
  // rows and weight rows are 32-bit TMA coordinates, tiles are counted in 32 bits
  if (rows >= (int64_t{1} << 31) - 256 || groups * N >= (int64_t{1} << 31) - 256)
    return MOE_ERR_UNSUPPORTED;
  if ((rows / 128 + groups) * blocks_of(N) >= INT_MAX / 2) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_rmsnorm(int64_t rows, int32_t d, int32_t dtype, float eps, const void* x,
                       const void* residual, const void* weight, void* residual_out, void* y,
                       void* y_q, float* y_scale, float* rstd, moe_stream_t stream) {
  moe_status st = check_norm(rows, d, dtype);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
  if ((y_q == nullptr) != (y_scale == nullptr)) return MOE_ERR_INVALID_ARG;
  if (y_q != nullptr && d % 16 != 0) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return nothing_to_do();
  if (!x || !weight || (!y && !y_q && !rstd && !residual_out)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) ||
      !aligned16(y) || !aligned16(y_q))
    return MOE_ERR_INVALID_ARG;
  Entry en(nullptr, stream);
  if (!en.ok) return MOE_ERR_CUDA;
  NormProblem p;
  p.rows = rows;
  p.d = d;
  p.bf16 = dtype == MOE_BF16;
  p.eps = eps;
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.sum_out = residual_out;
  p.y = y;
  p.q = y_q;
  p.scale = y_scale;
  p.rstd = rstd;
  return en.finish(launch_rmsnorm(p, en.lc));
}

size_t moe_rmsnorm_backward_workspace_size(int64_t rows, int32_t d) {
  if (check_norm(rows, d, MOE_F32) != MOE_OK) return 0;
  const int64_t blocks = rows < kNormBackwardBlocks ? (rows > 0 ? rows : 1) : kNormBackwardBlocks;
  return static_cast<size_t>(blocks) * d * 4;
}

moe_status moe_rmsnorm_backward(int64_t rows, int32_t d, int32_t dtype, const void* r,
                                const void* weight, const float* rstd, const float* dy,
                                const float* dresidual, float* dx, float* dweight, void* ws,
                                moe_stream_t stream) {
  moe_status st = check_norm(rows, d, dtype);
  if (st != MOE_OK) return st;
  if (!aligned16(r) || !aligned16(weight) || !aligned16(dy) || !aligned16(dresidual) ||
      !aligned16(dx) || !aligned16(dweight) || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) {
    if (dweight && cudaMemsetAsync(dweight, 0, static_cast<size_t>(d) * 4,
                                   reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
      return MOE_ERR_CUDA;
    return nothing_to_do();
  }
  if (!r || !weight || !rstd || !dy || !dx || (dweight && !ws)) return MOE_ERR_INVALID_ARG;
  Entry en(nullptr, stream);
  if (!en.ok) return MOE_ERR_CUDA;
  NormBackwardProblem p;
  p.rows = rows;
  p.d = d;
  p.bf16 = dtype == MOE_BF16;
  p.r = r;
  p.weight = weight;
  p.rstd = rstd;
  p.dy = dy;
  p.dres = dresidual;
  p.dx = dx;
  p.dweight = dweight;
  p.partial = static_cast<float*>(ws);
  return en.finish(launch_rmsnorm_backward(p, en.lc));
}

moe_status moe_quantize_rows_fp8(int64_t rows, int32_t d, int32_t dtype, const void* x, void* q,
                                 float* scale, moe_stream_t stream) {
  moe_status st = check_rows(rows, d, 16);
  if (st != MOE_OK) return st;
  if ((st = check_dtype(dtype)) != MOE_OK) return st;
  if (rows * ((d + 1023) / 1024) >= (int64_t{1} << 33)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return nothing_to_do();
  if (!x || !q || !scale || !aligned16(x) || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  Entry en(nullptr, stream);
  if (!en.ok) return MOE_ERR_CUDA;
  return en.finish(launch_quantize_rows(x, dtype == MOE_BF16, q, scale, rows, d, en.lc));
}

moe_status moe_quantize_weights_fp8(int64_t groups, int32_t N, int32_t K, int32_t dtype,
                                    const void* w, void* q, float* scale, moe_stream_t stream) {
  if (groups < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_dtype(dtype);
  if (st != MOE_OK) return st;
  if (K % 16 != 0 || N > kMaxWidth || K > kMaxWidth || groups > INT_MAX / (blocks_of(N) * blocks_of(K)))
    return MOE_ERR_UNSUPPORTED;
  if (groups == 0) return nothing_to_do();
  if (!w || !q || !scale || !aligned16(w) || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  Entry en(nullptr, stream);
  if (!en.ok) return MOE_ERR_CUDA;
  return en.finish(launch_quantize_weights(w, dtype == MOE_BF16, q, scale, groups, N, K, en.lc));
}

moe_status moe_gather_rows_fp8(const moe_config* cfg, const void* x_q, const float* x_scale,
                               const int32_t* perm_src, const int32_t* offsets, void* xq_perm,
                               float* xs_perm, void* ws, moe_stream_t stream) {
  const moe_status st = check_config_host(cfg);
  if (st != MOE_OK) return st;
  if (cfg->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (cfg->T == 0) return nothing_to_do();
  if (!x_q || !x_scale || !perm_src || !offsets || !xq_perm || !xs_perm || !ws)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(x_q) || !aligned16(xq_perm) || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  Entry en(ws, stream);
  if (!en.ok) return MOE_ERR_CUDA;
  return en.finish(launch_gather_rows_fp8(x_q, x_scale, perm_src, offsets + cfg->E, xq_perm, xs_perm,
                                          cfg->T, cfg->k, cfg->d_model, en.lc));
}

moe_status moe_grouped_matmul_fp8(int64_t rows, int32_t N, int32_t K, int32_t groups,
                                  const void* a_q, const float* a_scale, const int32_t* offsets,
                                  const void* b_q, const float* b_scale, void* out,
                                  int32_t out_dtype, void* ws, moe_stream_t stream) {
  const moe_status st = check_product(rows, N, K, groups, out_dtype);
  if (st != MOE_OK) return st;
  if (rows == 0) return nothing_to_do();
  if (!a_q || !a_scale || !offsets || !b_q || !b_scale || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned16(a_q) || !aligned16(b_q) || !aligned16(out) || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  Entry en(ws, stream);
  if (!en.ok) return MOE_ERR_CUDA;
  Fp8GemmProblem p;
  p.rows = rows;
  p.N = N;
  p.K = K;
  p.groups = groups;
  p.offsets = offsets;
  p.a = a_q;
  p.a_scale = a_scale;
  p.b = b_q;
  p.b_scale = b_scale;
  p.out_type = out_dtype == MOE_BF16 ? kFp8OutBf16 : kFp8OutF32;
  p.out = out;
  return en.finish(launch_fp8_gemm(p, en.lc));
}

moe_status moe_matmul_fp8(int64_t M, int32_t N, int32_t K, const void* a_q, const float* a_scale,
                          const void* b_q, const float* b_scale, void* out, int32_t out_dtype,
                          void* ws, moe_stream_t stream) {
  const moe_status st = check_product(M, N, K, 1, out_dtype);
  if (st != MOE_OK) return st;
  if (M == 0) return nothing_to_do();
  if (!a_q || !a_scale || !b_q || !b_scale || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned16(a_q) || !aligned16(b_q) || !aligned16(out) || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  Entry en(ws, stream);
  if (!en.ok) return MOE_ERR_CUDA;
  Fp8GemmProblem p;
  p.rows = M;
  p.N = N;
  p.K = K;
  p.a = a_q;
  p.a_scale = a_scale;
  p.b = b_q;
  p.b_scale = b_scale;
  p.out_type = out_dtype == MOE_BF16 ? kFp8OutBf16 : kFp8OutF32;
  p.out = out;
  return en.finish(launch_fp8_gemm(p, en.lc));
}

moe_status moe_expert_ffn_fp8(const moe_config* cfg, const void* x_q, const float* x_scale,
                              const int32_t* offsets, const void* w1_q, const float* w1_scale,
                              const void* w2_q, const float* w2_scale, void* h_q, float* h_scale,
                              void* y_perm, void* ws, moe_stream_t stream) {
  moe_status st = check_config_host(cfg);
  if (st != MOE_OK) return st;
  if (cfg->dtype != MOE_BF16 || cfg->hidden_f16) return MOE_ERR_UNSUPPORTED;
  const int64_t rows = cfg->T * cfg->k;
  if ((st = check_product(rows, cfg->d_ff, cfg->d_model, cfg->E, MOE_F32)) != MOE_OK) return st;
  if ((st = check_product(rows, cfg->d_model, cfg->d_ff, cfg->E, MOE_F32)) != MOE_OK) return st;
  if (cfg->T == 0) return nothing_to_do();
  if (!x_q || !x_scale || !offsets || !w1_q || !w1_scale || !w2_q || !w2_scale || !h_q ||
      !h_scale || !y_perm || !ws)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(x_q) || !aligned16(w1_q) || !aligned16(w2_q) || !aligned16(h_q) ||
      !aligned16(y_perm) || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  Entry en(ws, stream);
  if (!en.ok) return MOE_ERR_CUDA;
  Fp8GemmProblem p;
  p.rows = rows;
  p.N = cfg->d_ff;
  p.K = cfg->d_model;
  p.groups = cfg->E;
  p.offsets = offsets;
  p.a = x_q;
  p.a_scale = x_scale;
  p.b = w1_q;
  p.b_scale = w1_scale;
  p.out_type = kFp8OutE4m3;
  p.act = cfg->act == MOE_ACT_GELU ? 2 : 1;
  p.out = h_q;
  p.out_scale = h_scale;
  cudaError_t e = launch_fp8_gemm(p, en.lc);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  p.N = cfg->d_model;
  p.K = cfg->d_ff;
  p.a = h_q;
  p.a_scale = h_scale;
  p.b = w2_q;
  p.b_scale = w2_scale;
  p.out_type = kFp8OutF32;
  p.out = y_perm;
  p.out_scale = nullptr;
  return en.finish(launch_fp8_gemm(p, en.lc));
}

}  // extern "C"
