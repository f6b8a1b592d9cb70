"""Calls of several host threads that share a workspace on one stream: the launches of a call
that meet in the workspace must be enqueued with none of another call between them.  The host
side is built against launches that only look whether another call is between its own."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_grouped_gemm_lhs_amd", "csrc")
ROCM = "/opt/rocm/include"

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstring>
#include <thread>
#include <vector>

#include <hip/hip_runtime.h>

#include "dg.h"
#include "dg_ops.h"

// A device that there is, and launches in which a call's first and second kernel lie apart.
extern "C" {
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) {
  std::strcpy(p->gcnArchName, "gfx950");
  return hipSuccess;
}
}
static std::atomic<int> inside{0}, calls{0}, between{0};
static void two_launches() {
  if (inside.fetch_add(1) != 0) ++between;
  std::this_thread::sleep_for(std::chrono::milliseconds(1));
  inside.fetch_sub(1);
  ++calls;
}
namespace dg {
int route_slots(int64_t, int64_t) { return 4; }
void launch_route(const RouteArgs&, hipStream_t) { two_launches(); }
void launch_route_backward(const RouteArgs&, hipStream_t) {}
void lora_plan(LoraArgs* a) { a->S = 1; }
void launch_lora(const LoraArgs&, hipStream_t) { two_launches(); }
}  // namespace dg

int main() {
  alignas(16) static char ws[1 << 16];
  void* p = ws;
  uint16_t* h = (uint16_t*)ws;
  std::atomic<int> wrong{0};
  auto work = [&] {
    for (int i = 0; i < 20; ++i) {
      if (dg_moe_route(p, DG_IN_F32, 64, nullptr, nullptr, 64, 64, 4, DG_SCORE_SOFTMAX, 0, 1.0f, 0.0f,
                       (int32_t*)p, (float*)p, (int32_t*)p, nullptr, nullptr, p, sizeof ws, nullptr) != DG_OK)
        ++wrong;
      if (dg_lora_bf16(h, 128, h, h, (int32_t*)p, nullptr, nullptr, nullptr, 0, h, 8, 4, 8, 128, 8, 1, p,
                       sizeof ws, nullptr) != DG_OK)
        ++wrong;
    }
  };
  std::vector<std::thread> threads;
  for (int i = 0; i < 4; ++i) threads.emplace_back(work);
  for (auto& t : threads) t.join();
  std::printf("calls %d wrong %d between %d\n", calls.load(), wrong.load(), between.load());
}
"""


@pytest.mark.skipif(not os.path.exists(os.path.join(ROCM, "hip", "hip_runtime.h")), reason="no HIP headers")
def test_a_calls_launches_follow_each_other(tmp_path):
    src, exe = tmp_path / "threads.cpp", tmp_path / "threads"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-w", "-pthread", "-D__HIP_PLATFORM_AMD__", "-I", ROCM,
                           "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src),
                           os.path.join(CSRC, "dg_ops_host.cpp"), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True, timeout=60).stdout
    assert out.split() == ["calls", "160", "wrong", "0", "between", "0"], out
