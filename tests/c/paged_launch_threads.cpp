// The decode attention's host side on a made-up CUDA runtime (no GPU): what two threads that call it at
// once ask of the runtime, with the threads stopped where a scheduler may stop them.
#include <cuda_runtime_api.h>

#include <atomic>
#include <chrono>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <thread>

namespace oasis {
struct PagedShape {
  int B, Hq, Hkv, nb_max, n_pages;
};
cudaError_t launch_paged_decode_attn(const PagedShape&, const uint16_t*, size_t, const uint8_t*, const float*, const int*,
                                     const int*, const int*, const int*, int, float, void*, uint16_t*, unsigned*,
                                     cudaStream_t);
}  // namespace oasis

namespace {
std::mutex mu;
std::string order;                // the threads whose launches came, one letter each
std::atomic<int> limit{48 << 10};  // dynamic shared memory that a launch may have
thread_local char me = '-';
bool pause_limits = false;
void rest(int ms) { std::this_thread::sleep_for(std::chrono::milliseconds(ms)); }
}  // namespace

extern "C" {
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*) {}
cudaError_t __cudaGetKernel(void**, const void*) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(void*, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorNotSupported; }
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, cudaStream_t) { return 1; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaErrorNotSupported; }

cudaError_t cudaGetDevice(int* d) {
  *d = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int value) {
  if (pause_limits && me == 'a') rest(100);  // stopped before its value is taken
  limit = value;
  if (pause_limits && me == 'b') rest(200);  // stopped after
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void*, void**) {
  if ((int)cfg->dynamicSmemBytes > limit) return cudaErrorInvalidValue;
  {
    std::lock_guard<std::mutex> lock(mu);
    order += me;
  }
  rest(20);
  return cudaSuccess;
}
}

int main(int argc, char** argv) {
  const bool limits = argc > 1 && !strcmp(argv[1], "limits");
  pause_limits = limits;
  cudaError_t status[2] = {cudaSuccess, cudaSuccess};
  alignas(16) static char memory[64];
  auto run = [&](char name, int group, int calls) {
    me = name;
    const oasis::PagedShape s{3, 2 * group, 2, 4000, 100};  // a wide table: equal ranges, two launches a call
    for (int i = 0; i < calls; ++i) {
      const cudaError_t e = oasis::launch_paged_decode_attn(s, (const uint16_t*)memory, 256 * group, (const uint8_t*)memory,
                                                            (const float*)memory, (const int*)memory, (const int*)memory,
                                                            nullptr, nullptr, 0, 0.1f, memory, (uint16_t*)memory, nullptr,
                                                            nullptr);
      if (e != cudaSuccess) status[name - 'a'] = e;
    }
  };
  std::thread a([&] { run('a', limits ? 1 : 4, limits ? 1 : 5); });
  std::thread b([&] {
    rest(limits ? 30 : 5);
    run('b', limits ? 8 : 4, limits ? 2 : 5);
  });
  a.join();
  b.join();
  printf("status %d %d\norder %s\n", (int)status[0], (int)status[1], order.c_str());
  return 0;
}
