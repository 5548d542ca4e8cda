// Host threads that call the library on one stream at once, without a GPU: the
// C-ABI sources are linked with the HIP calls and kernel launches of this file.
// Work enqueued on a stream runs in the order of its launches, so a launch here
// does its work at once: the first writes the call's number to its workspace,
// the second, some time later, must find it there.  Prints "<calls> <wrong>"
// for each entry point.
#include <hip/hip_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <thread>
#include <vector>

#include "../dense_fp32_gemm_f32_amd/csrc/gemm_f32_internal.h"
#include "../dense_fp32_gemm_f32_amd/csrc/grouped_internal.h"
#include "../include/gemm_f32.h"

// ---- the HIP calls of the C-ABI layer ---------------------------------------
extern "C" {
hipError_t hipGetDevice(int* d) { return *d = 0, hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
  std::memset(p, 0, sizeof(*p));
  std::strcpy(p->gcnArchName, "gfx950");
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { return *v = 0, hipSuccess; }
hipError_t hipPointerGetAttributes(hipPointerAttribute_t* a, const void*) {
  a->type = hipMemoryTypeDevice;
  a->device = 0;
  return hipSuccess;
}
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) {
  return *s = hipStreamCaptureStatusNone, hipSuccess;
}
hipError_t hipMalloc(void** p, size_t n) {
  return (*p = std::malloc(n)) ? hipSuccess : hipErrorOutOfMemory;
}
hipError_t hipFree(void* p) { return std::free(p), hipSuccess; }
hipError_t hipMemsetAsync(void* p, int v, size_t n, hipStream_t) {
  return std::memset(p, v, n), hipSuccess;
}
}

// ---- the launches -------------------------------------------------------------
namespace {
std::atomic<int> g_calls{0}, g_wrong{0};
thread_local float* g_part = nullptr;   // the workspace of this thread's last launch

// Two launches that pass a value through the workspace.
hipError_t two_launches(float* part) {
  const float mine = (float)++g_calls;
  g_part = part;
  *(volatile float*)part = mine;
  std::this_thread::sleep_for(std::chrono::microseconds(200));
  if (*(volatile float*)part != mine) ++g_wrong;
  return hipSuccess;
}

gemmf32::SkinnyPlan plan(const gemmf32::Problem&, int) { return {2, 16, 1, 64, 0}; }
hipError_t skinny(const gemmf32::Problem&, const gemmf32::SkinnyPlan&, float* part,
                  const gemmf32::Epilogue&, hipStream_t) {
  return two_launches(part);
}
const gemmf32::SkinnyVariant kSkinny = {"skinnyx_w8_c2_u2_s0_vec", 16, 4, 1, false, false, 0, false,
                                        false, plan, skinny};
}  // namespace

namespace gemmf32 {
int mfma_variant_count() { return 0; }
const MfmaVariant& mfma_variant(int) { std::abort(); }
int mfma_ex_variant_count() { return 0; }
const MfmaExVariant& mfma_ex_variant(int) { std::abort(); }
int skinny_variant_count() { return 1; }
const SkinnyVariant& skinny_variant(int) { return kSkinny; }
hipError_t launch_ref(const Problem&, hipStream_t) { return hipSuccess; }
hipError_t launch_scale(const Problem&, const Epilogue&, hipStream_t) { return hipSuccess; }
hipError_t launch_clock_probe(int, unsigned long long*, hipStream_t) { return hipSuccess; }
int noalloc_scratch(int, hipStream_t, NoallocScratch* out) {
  static float fixed[64];
  out->partials = fixed;
  out->partial_floats = 64;
  return GEMM_F32_OK;
}
ReducePlan plan_reduce(int64_t) { return {}; }
hipError_t launch_reduce_sum(int64_t, const float*, float*, unsigned long long*, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_group_rows(int, int, int, const int*, int*, int*, int*, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_grouped(const GroupedProblem&, const Epilogue&, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_adapters_add(const AdapterProblem&, hipStream_t) { return hipSuccess; }
bool adapters_few(const AdapterProblem&) { return true; }
size_t adapters_few_floats(const AdapterProblem&) { return 64; }
hipError_t launch_adapters_few(const AdapterProblem&, float* part, hipStream_t) {
  return two_launches(part);
}
size_t grouped_wgrad_floats(const GroupedProblem&) { return 64; }
hipError_t launch_grouped_wgrad(const GroupedProblem&, const Epilogue&, float* part,
                                hipStream_t) {
  return two_launches(part);
}
}  // namespace gemmf32

// ---- the calls ------------------------------------------------------------------
namespace {
float* mem(int i) { return reinterpret_cast<float*>((uintptr_t)(i + 1) << 32); }
const int* imem(int i) { return reinterpret_cast<const int*>(mem(i)); }

int adapters(void* stream) {
  return gemm_f32_adapters(0, 8, 32, 64, 4, 2, 8, imem(0), imem(1), nullptr, mem(2), 64, mem(3),
                           32, mem(4), 4, 256, mem(5), 32, 128, nullptr, mem(6), 4, mem(7), 32,
                           stream);
}
int wgrad(void* stream) {
  return gemm_f32_grouped_wgrad(64, 32, 32, 2, imem(0), 1.f, mem(1), 32, 64, nullptr, mem(2), 32,
                                64, nullptr, 0.f, mem(3), 32, 1024, stream);
}
int few_rows(void* stream) {
  return gemm_f32(8, 32, 64, mem(1), 64, mem(2), 32, mem(3), 32, stream);
}
int noalloc(void* stream) {
  return gemm_f32_noalloc(8, 32, 64, mem(1), 64, mem(2), 32, mem(3), 32, stream);
}

void run(const char* name, int (*call)(void*), void* stream) {
  g_calls = g_wrong = 0;
  std::atomic<int> refused{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 4; ++t)
    threads.emplace_back([&] {
      for (int i = 0; i < 50; ++i)
        if (call(stream) != GEMM_F32_OK) ++refused;
    });
  for (auto& t : threads) t.join();
  std::printf("%s calls %d refused %d wrong %d\n", name, g_calls.load(), refused.load(),
              g_wrong.load());
}

// Calls on the two handles of the legacy default stream in turn.
int both_handles(void* stream) {
  static std::atomic<int> n{0};
  (void)stream;
  return noalloc(++n % 2 ? nullptr : (void*)hipStreamLegacy);
}

// Threads that call on hipStreamPerThread, each its own stream: the workspaces
// in use by more than one of them.
void run_per_thread() {
  std::vector<std::thread> threads;
  std::vector<float*> part(4);
  for (int t = 0; t < 4; ++t)
    threads.emplace_back([&part, t] {
      for (int i = 0; i < 2; ++i)
        if (adapters(hipStreamPerThread) == GEMM_F32_OK) part[t] = g_part;
    });
  for (auto& t : threads) t.join();
  int shared = 0;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j) shared += part[i] == part[j];
  std::printf("per_thread got %d shared %d\n", part[0] && part[1] && part[2] && part[3], shared);
}
}  // namespace

int main() {
  for (void* stream : {(void*)nullptr, (void*)0x1000}) {
    run("adapters", adapters, stream);
    run("wgrad", wgrad, stream);
    run("few_rows", few_rows, stream);
    run("noalloc", noalloc, stream);
  }
  run("both_handles", both_handles, nullptr);
  run_per_thread();
  return gemm_f32_release_workspaces();
}
