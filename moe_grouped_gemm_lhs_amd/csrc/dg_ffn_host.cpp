// dg_ffn_host.cpp -- host side of the feed-forward operators in 8 bits declared in
// include/dg.h: argument validation, workspaces, launches.  As for the other calls,
// validation is pure host code and comes before any device work.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "dg.h"
#include "dg_ffn.h"
#include "dg_ops.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool valid_format(int f) { return f == DG_FP8_E4M3 || f == DG_FP8_E5M2; }
bool valid_dtype(int d) { return d == DG_IN_F32 || d == DG_IN_BF16; }
bool blocks_of_128(int64_t n) { return n > 0 && n % dg::kBlockK == 0; }

// A row stride: the row's length at least, and a multiple of 8 elements (16-byte accesses).
bool stride_ok(int64_t ld, int64_t K) { return ld >= K && ld <= INT32_MAX && ld % 8 == 0; }

bool norm_shape(int64_t T, int64_t K) {
  return T >= 0 && T <= INT32_MAX && blocks_of_128(K) && K <= dg::kNormMaxK;
}

// Rows of H: N columns, of B: 2 N.  32-bit offsets inside a tile's rows and group's scales.
constexpr int64_t kGatedMaxN = (int64_t)1 << 20, kGatedMaxK = (int64_t)1 << 22;
bool gated_shape(int kind, int64_t rows, int64_t N, int64_t K, int64_t G) {
  if (!blocks_of_128(K) || K > kGatedMaxK || N < 0 || N % dg::kBlockK != 0 || N > kGatedMaxN)
    return false;
  if (rows < 0 || rows > INT32_MAX || G < 1 || G > INT32_MAX) return false;
  const int64_t groups = kind == dg::kMasked ? G : 1;
  if ((rows + 63) / 64 * (N / dg::kBlockK + 1) > INT32_MAX / groups) return false;
  return kind != dg::kMasked || rows * G <= INT32_MAX;
}

bool wgrad_shape(int64_t T, int64_t N, int64_t K, int64_t G) {
  if (T < 0 || T > INT32_MAX - dg::kAlignM || N < 0 || K < 0 || N % dg::kBlockK || K % dg::kBlockK)
    return false;
  if (N > kGatedMaxK || K > kGatedMaxK || G < 1 || G > INT32_MAX) return false;
  return (N / dg::kBlockK) * (K / dg::kBlockK) <= (INT32_MAX >> 8) / G;   // tiles of a launch
}

dg_status launched() { return hipGetLastError() == hipSuccess ? DG_OK : DG_ERR_HIP; }

dg_status gated(int kind, const uint8_t* A, int a_format, const float* sA, const uint8_t* B, int b_format,
                const float* sB, const int32_t* rows_of, uint8_t* H, float* sH, int out_format, uint8_t* GU,
                float* sGU, int activation, int64_t rows, int64_t N, int64_t K, int64_t G, void* workspace,
                size_t workspace_bytes, void* stream) {
  if (!gated_shape(kind, rows, N, K, G)) return DG_ERR_SHAPE;
  if (!valid_format(a_format) || !valid_format(b_format) || !valid_format(out_format) ||
      (activation != DG_ACT_SILU && activation != DG_ACT_GELU))
    return DG_ERR_FORMAT;
  if (rows == 0 || N == 0) return DG_OK;
  if (!A || !sA || !B || !sB || !H || !sH || (kind != dg::kDense && !rows_of) ||
      (GU != nullptr) != (sGU != nullptr))
    return DG_ERR_NULL;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(H, 16) || !aligned(GU, 16) || !aligned(sA, 4) ||
      !aligned(sB, 4) || !aligned(sH, 4) || !aligned(sGU, 4) || !aligned(rows_of, 4))
    return DG_ERR_ALIGN;
  const size_t need = dg_gated_workspace_bytes(kind, rows, N, K, G);
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return DG_ERR_WORKSPACE;
  int num_cus = 0;
  const dg_status st = dg::current_gpu(&num_cus);
  if (st != DG_OK) return st;
  dg::GatedArgs a{};
  a.A = A; a.sA = sA; a.B = B; a.sB = sB;
  if (kind == dg::kContiguous) a.group_idx = rows_of;
  if (kind == dg::kMasked) a.masked_m = rows_of;
  a.H = H; a.sH = sH; a.GU = GU; a.sGU = sGU; a.act = activation; a.out_fmt = out_format;
  a.rows = (int)rows; a.N = (int)(2 * N); a.K = (int)K; a.G = (int)G;
  std::unique_lock<std::mutex> together(dg::workspace_mutex(workspace), std::defer_lock);
  if (need > 0) together.lock();
  (void)hipGetLastError();
  dg::launch_gated(a, kind, a_format, b_format, num_cus, workspace, (hipStream_t)stream);
  return launched();
}

dg_status wgrad(const uint8_t* P, int p_format, const float* sP, const uint8_t* Q, int q_format,
                const float* sQ, const int32_t* group_idx, bool grouped, void* dW, int dtype, int accumulate,
                int64_t T, int64_t N, int64_t K, int64_t G, void* workspace, size_t workspace_bytes,
                void* stream) {
  if (!wgrad_shape(T, N, K, G)) return DG_ERR_SHAPE;
  if (!valid_format(p_format) || !valid_format(q_format) || !valid_dtype(dtype)) return DG_ERR_FORMAT;
  if (N == 0 || K == 0 || (T == 0 && accumulate)) return DG_OK;
  if (!dW || (T > 0 && (!P || !sP || !Q || !sQ || (grouped && !group_idx)))) return DG_ERR_NULL;
  if (!aligned(P, 16) || !aligned(Q, 16) || !aligned(dW, 16) || !aligned(sP, 4) || !aligned(sQ, 4) ||
      !aligned(group_idx, 4))
    return DG_ERR_ALIGN;
  const size_t need = dg_wgrad_workspace_bytes(T, N, K, G);
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return DG_ERR_WORKSPACE;
  int num_cus = 0;
  const dg_status st = dg::current_gpu(&num_cus);
  if (st != DG_OK) return st;
  dg::WgradArgs a{};
  a.P = P; a.sP = sP; a.Q = Q; a.sQ = sQ; a.group_idx = grouped ? group_idx : nullptr; a.dW = dW;
  a.partial = (float*)workspace;
  a.T = T; a.N = (int)N; a.K = (int)K; a.G = (int)G;
  a.p_fmt = p_format; a.q_fmt = q_format; a.bf16 = dtype == DG_IN_BF16; a.accumulate = accumulate != 0;
  const dg::WgradPlan plan = dg::wgrad_plan(T, N, K, G);
  a.splits = plan.splits; a.big = plan.big;
  std::unique_lock<std::mutex> together(dg::workspace_mutex(workspace), std::defer_lock);
  if (need > 0) together.lock();
  (void)hipGetLastError();
  dg::launch_wgrad(a, (hipStream_t)stream);
  return launched();
}

}  // namespace

extern "C" {

dg_status dg_rms_norm_fp8(const void *X, int dtype, int64_t ldx, const void *residual, int64_t ld_residual,
                          const void *weight, int weight_dtype, float eps, void *H, int64_t ldh, uint8_t *Q,
                          float *S, int format, uint16_t *Y, int64_t ldy, float *rstd, int64_t T, int64_t K,
                          void *stream) {
  if (!norm_shape(T, K) || !stride_ok(ldx, K) || (residual && (!stride_ok(ld_residual, K) || !stride_ok(ldh, K))) ||
      (Y && !stride_ok(ldy, K)))
    return DG_ERR_SHAPE;
  if (!valid_dtype(dtype) || (weight && !valid_dtype(weight_dtype)) || (Q && !valid_format(format)))
    return DG_ERR_FORMAT;
  if (T == 0) return DG_OK;
  if (!X || (residual != nullptr) != (H != nullptr) || (Q != nullptr) != (S != nullptr)) return DG_ERR_NULL;
  if (!aligned(X, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(H, 16) || !aligned(Q, 8) ||
      !aligned(S, 4) || !aligned(Y, 16) || !aligned(rstd, 4))
    return DG_ERR_ALIGN;
  int num_cus = 0;
  const dg_status st = dg::current_gpu(&num_cus);
  if (st != DG_OK) return st;
  dg::NormArgs a{};
  a.x = X; a.ldx = ldx; a.r = residual; a.ldr = ld_residual; a.w = weight; a.h = H; a.ldh = ldh;
  a.q = Q; a.s = S; a.y = Y; a.ldy = ldy; a.rstd = rstd; a.T = T; a.K = (int)K;
  a.bf16 = dtype == DG_IN_BF16; a.w_bf16 = weight_dtype == DG_IN_BF16; a.fmt = format; a.eps = eps;
  (void)hipGetLastError();
  dg::launch_norm(a, (hipStream_t)stream);
  return launched();
}

size_t dg_rms_norm_backward_workspace_bytes(int64_t T, int64_t K) {
  if (!norm_shape(T, K)) return 0;
  return (size_t)dg::norm_backward_grid(T) * (size_t)K * 4;
}

dg_status dg_rms_norm_backward(const void *grad_y, int dtype, int64_t ld_grad_y, const void *H, int64_t ldh,
                               const float *rstd, const void *weight, int weight_dtype, const void *grad_h,
                               int64_t ld_grad_h, void *grad_x, int64_t ld_grad_x, float *grad_weight, int64_t T,
                               int64_t K, void *workspace, size_t workspace_bytes, void *stream) {
  if (!norm_shape(T, K) || !stride_ok(ld_grad_y, K) || !stride_ok(ldh, K) || !stride_ok(ld_grad_x, K) ||
      (grad_h && !stride_ok(ld_grad_h, K)))
    return DG_ERR_SHAPE;
  if (!valid_dtype(dtype) || (weight && !valid_dtype(weight_dtype))) return DG_ERR_FORMAT;
  if (T == 0 && !grad_weight) return DG_OK;
  if (T > 0 && (!grad_y || !H || !rstd || !grad_x)) return DG_ERR_NULL;
  if (!aligned(grad_y, 16) || !aligned(H, 16) || !aligned(rstd, 4) || !aligned(weight, 16) ||
      !aligned(grad_h, 16) || !aligned(grad_x, 16) || !aligned(grad_weight, 4))
    return DG_ERR_ALIGN;
  const size_t need = grad_weight ? dg_rms_norm_backward_workspace_bytes(T, K) : 0;
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return DG_ERR_WORKSPACE;
  int num_cus = 0;
  const dg_status st = dg::current_gpu(&num_cus);
  if (st != DG_OK) return st;
  dg::NormArgs a{};
  a.x = grad_y; a.ldx = ld_grad_y; a.r = H; a.ldr = ldh; a.w = weight; a.h = grad_x; a.ldh = ld_grad_x;
  a.grad_h = grad_h; a.ld_gh = ld_grad_h; a.rstd = (float *)rstd; a.grad_w = grad_weight;
  a.partial = (float *)workspace; a.T = T; a.K = (int)K; a.bf16 = dtype == DG_IN_BF16;
  a.w_bf16 = weight_dtype == DG_IN_BF16;
  std::unique_lock<std::mutex> together(dg::workspace_mutex(workspace), std::defer_lock);
  if (need > 0) together.lock();
  (void)hipGetLastError();
  dg::launch_norm_backward(a, (hipStream_t)stream);
  return launched();
}

size_t dg_gated_workspace_bytes(int kind, int64_t rows_or_cap, int64_t N, int64_t K, int64_t G) {
  if (kind < dg::kDense || kind > dg::kMasked || !gated_shape(kind, rows_or_cap, N, K, kind == dg::kDense ? 1 : G))
    return 0;
  if (rows_or_cap == 0 || N == 0) return 0;
  return dg::gated_plan(kind, rows_or_cap, N, K, G).bytes;
}

dg_status dg_gated_fp8_nt(const uint8_t *A, int a_format, const float *sA, const uint8_t *B, int b_format,
                          const float *sB, uint8_t *H, float *sH, int out_format, uint8_t *GU, float *sGU,
                          int activation, int64_t M, int64_t N, int64_t K, void *workspace,
                          size_t workspace_bytes, void *stream) {
  return gated(dg::kDense, A, a_format, sA, B, b_format, sB, nullptr, H, sH, out_format, GU, sGU, activation, M,
               N, K, 1, workspace, workspace_bytes, stream);
}

dg_status dg_grouped_gated_fp8_contiguous(const uint8_t *A, int a_format, const float *sA, const uint8_t *B,
                                          int b_format, const float *sB, const int32_t *group_idx, uint8_t *H,
                                          float *sH, int out_format, uint8_t *GU, float *sGU, int activation,
                                          int64_t M_total, int64_t N, int64_t K, int64_t G, void *workspace,
                                          size_t workspace_bytes, void *stream) {
  return gated(dg::kContiguous, A, a_format, sA, B, b_format, sB, group_idx, H, sH, out_format, GU, sGU,
               activation, M_total, N, K, G, workspace, workspace_bytes, stream);
}

dg_status dg_grouped_gated_fp8_masked(const uint8_t *A, int a_format, const float *sA, const uint8_t *B,
                                      int b_format, const float *sB, const int32_t *masked_m, uint8_t *H,
                                      float *sH, int out_format, int activation, int64_t G, int64_t cap,
                                      int64_t N, int64_t K, void *workspace, size_t workspace_bytes,
                                      void *stream) {
  return gated(dg::kMasked, A, a_format, sA, B, b_format, sB, masked_m, H, sH, out_format, nullptr, nullptr,
               activation, cap, N, K, G, workspace, workspace_bytes, stream);
}

dg_status dg_gated_backward(const void *grad_H, int dtype, const uint8_t *GU, int gu_format, const float *sGU,
                            const int32_t *group_idx, int activation, uint8_t *D, float *sD, int out_format,
                            int64_t T, int64_t N, int64_t G, void *stream) {
  if (T < 0 || T > INT32_MAX || N < 0 || N % dg::kBlockK != 0 || N > kGatedMaxN || G < 1 || G > INT32_MAX ||
      T * (N / dg::kBlockK) > ((int64_t)1 << 28))
    return DG_ERR_SHAPE;
  if (!valid_dtype(dtype) || !valid_format(gu_format) || !valid_format(out_format) ||
      (activation != DG_ACT_SILU && activation != DG_ACT_GELU))
    return DG_ERR_FORMAT;
  if (T == 0 || N == 0) return DG_OK;
  if (!grad_H || !GU || !sGU || !D || !sD) return DG_ERR_NULL;
  if (!aligned(grad_H, 16) || !aligned(GU, 16) || !aligned(D, 16) || !aligned(sGU, 4) || !aligned(sD, 4) ||
      !aligned(group_idx, 4))
    return DG_ERR_ALIGN;
  int num_cus = 0;
  const dg_status st = dg::current_gpu(&num_cus);
  if (st != DG_OK) return st;
  dg::GatedBackArgs a{};
  a.dh = grad_H; a.gu = GU; a.sgu = sGU; a.group_idx = group_idx; a.d = D; a.sd = sD; a.T = T; a.N = (int)N;
  a.G = (int)G; a.bf16 = dtype == DG_IN_BF16; a.act = activation; a.gu_fmt = gu_format; a.fmt = out_format;
  (void)hipGetLastError();
  dg::launch_gated_backward(a, (hipStream_t)stream);
  return launched();
}

size_t dg_wgrad_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t G) {
  if (!wgrad_shape(T, N, K, G)) return 0;
  const int splits = dg::wgrad_plan(T, N, K, G).splits;
  return splits > 1 ? (size_t)splits * G * N * K * 4 : 0;
}

dg_status dg_wgrad_fp8(const uint8_t *P, int p_format, const float *sP, const uint8_t *Q, int q_format,
                       const float *sQ, void *dW, int dtype, int accumulate, int64_t T, int64_t N, int64_t K,
                       void *workspace, size_t workspace_bytes, void *stream) {
  return wgrad(P, p_format, sP, Q, q_format, sQ, nullptr, false, dW, dtype, accumulate, T, N, K, 1, workspace,
               workspace_bytes, stream);
}

dg_status dg_grouped_wgrad_fp8_contiguous(const uint8_t *P, int p_format, const float *sP, const uint8_t *Q,
                                          int q_format, const float *sQ, const int32_t *group_idx, void *dW,
                                          int dtype, int accumulate, int64_t M_total, int64_t N, int64_t K,
                                          int64_t G, void *workspace, size_t workspace_bytes, void *stream) {
  return wgrad(P, p_format, sP, Q, q_format, sQ, group_idx, true, dW, dtype, accumulate, M_total, N, K, G,
               workspace, workspace_bytes, stream);
}

}  // extern "C"
