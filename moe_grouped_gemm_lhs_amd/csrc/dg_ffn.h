// dg_ffn.h -- shared between the host side of the feed-forward operators in 8 bits
// (dg_ffn_host.cpp) and their kernels (dg_norm.hip, dg_gated.hip, dg_wgrad.hip).  Not part of
// the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dg_internal.h"

namespace dg {

// Root-mean-square norm (defined in dg_norm.hip).
constexpr int64_t kNormMaxK = 65536;
constexpr int64_t kNormRows = (int64_t)1 << 20;   // rows of a launch
constexpr int64_t kNormFewRows = 1024;  // backward in one launch
constexpr int kNormMaxGrid = 512;       // workgroups that keep sums of a weight's gradient

struct NormArgs {
  const void* x;               // T x K; backward: the gradient by y
  const void* r;               // residual, or nullptr; backward: h
  const void* w;               // K, or nullptr (1)
  void* h;                     // x + r, with r; backward: the gradient by x
  const void* grad_h;          // backward: added to the gradient, or nullptr
  int64_t ldx, ldr, ldh, ldy, ld_gh;
  uint8_t* q;                  // codes, or nullptr
  float* s;                    // their scales
  uint16_t* y;                 // bf16 output, or nullptr
  float* rstd;                 // T, or nullptr; backward: read
  float* grad_w;               // backward: K, or nullptr
  float* partial;              // backward: a row of K sums a workgroup
  int64_t T;
  int K;
  int bf16, w_bf16, fmt;
  float eps;
};

// Workgroups of the backward pass, each of which keeps a row of sums.
int norm_backward_grid(int64_t T);
void launch_norm(const NormArgs& a, hipStream_t stream);
void launch_norm_backward(const NormArgs& a, hipStream_t stream);

// The gated block (defined in dg_gated.hip).
enum Act : int { kActSilu = 0, kActGelu = 1 };

struct GatedArgs : GemmArgs {  // N: rows of B, gate and up together
  uint8_t* H;                  // codes, rows x N/2
  float* sH;
  uint8_t* GU;                 // codes of gate and up, rows x N, or nullptr
  float* sGU;
  int act, out_fmt;
  float* scratch;              // few tiles: parts of sums, the workspace
};

// What runs for these sizes (N: columns of H).
struct GatedPlan {
  int bm;                      // rows of a tile of the split kernels; 0: whole tiles
  size_t bytes;                // of the workspace
};
GatedPlan gated_plan(int kind, int64_t rows, int64_t N, int64_t K, int64_t G);
void launch_gated(GatedArgs& a, int kind, int fmt_a, int fmt_b, int num_cus, void* workspace,
                  hipStream_t stream);

struct GatedBackArgs {
  const void* dh;              // T x N
  const uint8_t* gu;           // T x 2N
  const float* sgu;            // T x 2N/128
  const int32_t* group_idx;    // or nullptr
  uint8_t* d;                  // T x 2N
  float* sd;
  int64_t T;
  int N, G;
  int bf16, act, gu_fmt, fmt;
};
void launch_gated_backward(const GatedBackArgs& a, hipStream_t stream);

// A weight's gradient (defined in dg_wgrad.hip).
struct WgradArgs {
  const uint8_t* P;            // T x N
  const float* sP;
  const uint8_t* Q;            // T x K
  const float* sQ;
  const int32_t* group_idx;    // or nullptr
  void* dW;                    // G x N x K
  float* partial;              // splits x G x N x K, or nullptr
  int64_t T;
  int N, K, G;
  int p_fmt, q_fmt, bf16, accumulate;
  int splits;                  // the plan's
  bool big;
};
struct WgradPlan {
  bool big;                    // tiles of 256 x 256, else 128 x 128
  int splits;                  // parts of the sum over rows
};
WgradPlan wgrad_plan(int64_t T, int64_t N, int64_t K, int64_t G);
void launch_wgrad(const WgradArgs& a, hipStream_t stream);

}  // namespace dg
