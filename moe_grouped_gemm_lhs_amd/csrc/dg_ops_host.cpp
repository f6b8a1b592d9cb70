// dg_ops_host.cpp -- host side of the gate and the adapters declared in include/dg.h:
// argument validation, launch shapes, launches.  As for the GEMM calls, validation is pure
// host code and comes before any device work.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "dg.h"
#include "dg_internal.h"
#include "dg_ops.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Current device must be gfx950.
dg_status check_device() {
  constexpr int kMaxDevices = 64;
  static int known[kMaxDevices];                 // 0: not looked at, 1: gfx950, 2: another
  static std::mutex mu;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
    (void)hipGetLastError();
    return DG_ERR_DEVICE;
  }
  std::lock_guard<std::mutex> lk(mu);
  if (!known[dev]) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
      (void)hipGetLastError();
      return DG_ERR_DEVICE;
    }
    known[dev] = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
  }
  return known[dev] == 1 ? DG_OK : DG_ERR_DEVICE;
}

bool route_shape(int64_t T, int64_t E, int64_t k, int64_t ld) {
  return T >= 0 && T <= INT32_MAX && E >= 1 && E <= dg::kRouteMaxE && k >= 1 &&
         k <= dg::kRouteMaxK && k <= E && T <= INT32_MAX / k && ld >= E && ld <= INT32_MAX;
}

bool route_format(int dtype, int score) {
  return (dtype == DG_IN_F32 || dtype == DG_IN_BF16) &&
         (score == DG_SCORE_SOFTMAX || score == DG_SCORE_SIGMOID);
}

// Rows that can be read or written four elements at a time.
int route_vec(const void* p, int64_t E, int64_t ld, int bf16) {
  return E % 4 == 0 && ld % 4 == 0 && aligned(p, bf16 ? 8 : 16);
}

bool lora_shape(int64_t T, int64_t N, int64_t K, int64_t R, int64_t L) {
  // K % 128 as for the projection beside which the adapters stand
  return T >= 0 && T <= INT32_MAX - 64 && N >= 0 && N <= ((int64_t)1 << 22) && K > 0 &&
         K % dg::kBlockK == 0 && K <= ((int64_t)1 << 22) && R >= 8 && R <= dg::kLoraMaxR &&
         R % 8 == 0 && L >= 1 && L <= INT32_MAX;
}

}  // namespace

std::mutex& dg::workspace_mutex(const void* workspace) {
  static std::mutex mu[64];
  return mu[((uintptr_t)workspace >> 8) % 64];
}

extern "C" {

size_t dg_moe_route_workspace_bytes(int64_t T, int64_t E) {
  if (!route_shape(T, E, 1, E)) return 0;
  const size_t slots = (size_t)dg::route_slots(T, E);
  return slots ? dg::kRouteWsHeader + slots * (8 * (size_t)E + 4) : 0;
}

dg_status dg_moe_route(const void* logits, int dtype, int64_t ld, const float* bias,
                       const uint8_t* row_valid, int64_t T, int64_t E, int64_t k, int score,
                       int normalize, float scale, float balance, int32_t* ids, float* weights,
                       int32_t* counts, float* loss, float* coef, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (!route_shape(T, E, k, ld)) return DG_ERR_SHAPE;
  if (!route_format(dtype, score)) return DG_ERR_FORMAT;
  if (T == 0 && !counts && !loss && !coef) return DG_OK;
  if (T > 0 && (!logits || !ids || !weights)) return DG_ERR_NULL;
  if ((loss != nullptr) != (coef != nullptr) || (loss && !counts)) return DG_ERR_NULL;
  const int bf16 = dtype == DG_IN_BF16;
  if (!aligned(logits, bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(ids, 4) ||
      !aligned(weights, 4) || !aligned(counts, 4) || !aligned(loss, 4) || !aligned(coef, 4))
    return DG_ERR_ALIGN;
  const size_t need = counts ? dg_moe_route_workspace_bytes(T, E) : 0;
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
    return DG_ERR_WORKSPACE;
  const dg_status st = check_device();
  if (st != DG_OK) return st;
  dg::RouteArgs a{};
  a.logits = logits; a.ld = ld; a.bias = bias; a.row_valid = row_valid; a.T = T;
  a.E = (int)E; a.k = (int)k; a.bf16 = bf16; a.sigmoid = score == DG_SCORE_SIGMOID;
  a.normalize = normalize != 0; a.vec = route_vec(logits, E, ld, bf16);
  a.scale = scale; a.balance = balance; a.ids = ids; a.weights = weights; a.counts = counts;
  a.loss = loss; a.coef = coef; a.workspace = workspace;
  std::unique_lock<std::mutex> together(dg::workspace_mutex(workspace), std::defer_lock);
  if (need > 0) together.lock();
  (void)hipGetLastError();
  dg::launch_route(a, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? DG_OK : DG_ERR_HIP;
}

dg_status dg_moe_route_backward(const void* logits, int dtype, int64_t ld, const uint8_t* row_valid,
                                int64_t T, int64_t E, int64_t k, int score, int normalize,
                                float scale, const int32_t* ids, const float* grad_weights,
                                const float* coef, const float* grad_loss, void* grad_logits,
                                int64_t ld_grad, void* stream) {
  if (!route_shape(T, E, k, ld) || ld_grad < E || ld_grad > INT32_MAX) return DG_ERR_SHAPE;
  if (!route_format(dtype, score)) return DG_ERR_FORMAT;
  if (T == 0) return DG_OK;
  if (!logits || !grad_logits || (grad_weights && !ids) || (grad_loss && !coef)) return DG_ERR_NULL;
  const int bf16 = dtype == DG_IN_BF16;
  if (!aligned(logits, bf16 ? 2 : 4) || !aligned(grad_logits, bf16 ? 2 : 4) || !aligned(ids, 4) ||
      !aligned(grad_weights, 4) || !aligned(coef, 4) || !aligned(grad_loss, 4))
    return DG_ERR_ALIGN;
  const dg_status st = check_device();
  if (st != DG_OK) return st;
  dg::RouteArgs a{};
  a.logits = logits; a.ld = ld; a.row_valid = row_valid; a.T = T; a.E = (int)E; a.k = (int)k;
  a.bf16 = bf16; a.sigmoid = score == DG_SCORE_SIGMOID; a.normalize = normalize != 0;
  a.vec = route_vec(logits, E, ld, bf16); a.scale = scale; a.coef = (float*)coef;
  a.ids_in = ids; a.grad_weights = grad_weights; a.grad_loss = grad_loss;
  a.grad_logits = grad_logits; a.ld_grad = ld_grad;
  a.vec_grad = route_vec(grad_logits, E, ld_grad, bf16);
  (void)hipGetLastError();
  dg::launch_route_backward(a, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? DG_OK : DG_ERR_HIP;
}

size_t dg_lora_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t R, int64_t L) {
  if (!lora_shape(T, N, K, R, L) || T == 0 || N == 0) return 0;
  dg::LoraArgs a{};
  a.T = T; a.N = N; a.K = (int)K; a.R = (int)R;
  dg::lora_plan(&a);
  return (size_t)a.S * T * R * 4 + (size_t)T * 4;
}

dg_status dg_lora_bf16(const uint16_t* X, int64_t ldx, const uint16_t* A, const uint16_t* B,
                       const int32_t* ids, const float* scales, const int32_t* ranks,
                       const uint16_t* base, int64_t ld_base, uint16_t* out, int64_t ld_out,
                       int64_t T, int64_t N, int64_t K, int64_t R, int64_t L, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (!lora_shape(T, N, K, R, L)) return DG_ERR_SHAPE;
  if (ldx < K || ldx > INT32_MAX || ldx % 8 != 0 || ld_out < N || ld_out > INT32_MAX ||
      (base && (ld_base < N || ld_base > INT32_MAX)) ||
      (base == out && base && ld_base != ld_out))
    return DG_ERR_SHAPE;
  if (T == 0 || N == 0) return DG_OK;
  if (!X || !A || !B || !ids || !out) return DG_ERR_NULL;
  if (!aligned(X, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(ids, 4) ||
      !aligned(scales, 4) || !aligned(ranks, 4) || !aligned(base, 2) || !aligned(out, 2))
    return DG_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 16) ||
      workspace_bytes < dg_lora_workspace_bytes(T, N, K, R, L))
    return DG_ERR_WORKSPACE;
  const dg_status st = check_device();
  if (st != DG_OK) return st;
  dg::LoraArgs a{};
  a.x = X; a.ldx = ldx; a.A = A; a.B = B; a.ids = ids; a.scales = scales; a.ranks = ranks;
  a.base = base; a.ld_base = ld_base; a.out = out; a.ld_out = ld_out;
  a.h = (float*)workspace;
  a.T = T; a.N = N; a.K = (int)K; a.R = (int)R; a.L = (int)L;
  dg::lora_plan(&a);
  a.parts = (int*)(a.h + (int64_t)a.S * T * R);
  std::lock_guard<std::mutex> together(dg::workspace_mutex(workspace));
  (void)hipGetLastError();
  dg::launch_lora(a, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? DG_OK : DG_ERR_HIP;
}

}  // extern "C"
