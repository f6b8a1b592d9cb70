// dg_ops.h -- shared between the host side of the gate and the adapters (dg_ops_host.cpp)
// and their kernels (dg_route.hip, dg_lora.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dg {

// First bytes of the gate's workspace, before its workgroups' sums.
constexpr int kRouteWsHeader = 16;

// The gate and its backward pass (defined in dg_route.hip).
constexpr int kRouteMaxK = 16;       // choices a row
constexpr int kRouteMaxE = 1024;     // experts
constexpr int kRouteMaxGrid = 512;   // workgroups
constexpr int64_t kRouteWideWork = (int64_t)1 << 21;   // logits from which V = 32

struct RouteArgs {
  const void* logits;
  int64_t ld;                  // row stride of the logits
  const float* bias;           // E, or nullptr
  const uint8_t* row_valid;    // T, or nullptr
  int64_t T;
  int E, k;
  int bf16, sigmoid, normalize, vec;   // vec: rows may be read four logits at a time
  float scale, balance;
  // forward
  int32_t* ids;
  float* weights;
  int32_t* counts;             // or nullptr
  float* loss;                 // or nullptr
  float* coef;                 // with loss; read in the backward pass (or nullptr)
  void* workspace;
  // backward
  const int32_t* ids_in;
  const float* grad_weights;   // or nullptr
  const float* grad_loss;      // or nullptr (1)
  void* grad_logits;
  int64_t ld_grad;
  int vec_grad;
};

// Workgroups' sums (of E probabilities, E counts and the rows) that the forward pass keeps in
// the workspace for these sizes.
int route_slots(int64_t T, int64_t E);
void launch_route(const RouteArgs& a, hipStream_t stream);
void launch_route_backward(const RouteArgs& a, hipStream_t stream);

// Low-rank adapters (defined in dg_lora.hip).
constexpr int kLoraMaxR = 128;
constexpr int64_t kLoraFewRows = 128;
constexpr int64_t kLoraRows = (int64_t)1 << 20;   // rows of a launch
constexpr int64_t kLoraPastCaches = (int64_t)64 << 20;   // bytes of an output

struct LoraArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* A;
  const uint16_t* B;
  const int32_t* ids;
  const float* scales;         // L, or nullptr (1)
  const int32_t* ranks;        // L, or nullptr (R)
  const uint16_t* base;        // or nullptr (0); may be out
  int64_t ld_base;
  uint16_t* out;
  int64_t ld_out;
  float* h;                    // S x T x R, the workspace
  int64_t h_part;              // elements from one part to the next
  int* parts;                  // T, behind it: parts of a row's sums
  int64_t T, N;
  int K, R, L;
  // the plan for the sizes (lora_plan)
  int mt;                      // first kernel: row tiles of 16 a workgroup; 0: the one for
                               // few rows
  int S;                       // parts of the sums over K, at most
  int grid;                    // workgroups of the first kernel
  int up_mt;                   // second kernel: row tiles of 16 a workgroup
  int up_ct;                   // its column tiles of 16 a wave
  int up_Q;                    // workgroups over the adapters of the same rows
  bool past_caches;            // out is stored past the caches
};

void lora_plan(LoraArgs* a);
void launch_lora(const LoraArgs& a, hipStream_t stream);

}  // namespace dg
