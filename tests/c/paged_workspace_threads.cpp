// The paged cache's calls that leave something in a workspace between their launches, on a made-up CUDA runtime (no
// GPU): two threads that share a stream and a workspace, each with a call of another kind.
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <chrono>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <thread>

#include "oasis.h"

namespace oasis {
void set_last_error(const std::string& msg) { fprintf(stderr, "%s\n", msg.c_str()); }
}  // namespace oasis

namespace {
std::mutex mu;
std::string order;  // the threads whose launches came, one letter each
thread_local char me = '-';
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

const char* cudaGetErrorName(cudaError_t) { return "error"; }
const char* cudaGetErrorString(cudaError_t) { return "error"; }
cudaError_t cudaGetDevice(int* d) {
  *d = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* fa, const void*) {
  memset(fa, 0, sizeof *fa);
  fa->numRegs = 168;
  return cudaSuccess;
}
CUresult made_up_encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                        const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                        CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(made_up_encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) {
  {
    std::lock_guard<std::mutex> lock(mu);
    order += me;
  }
  rest(20);
  return cudaSuccess;
}
}

namespace {
alignas(256) char memory[64];
const size_t kMuch = size_t(1) << 40;  // bytes of the workspace, which nothing touches

// Sizes whose work is split: each call joins its parts in its last launch.
oasis_status call(const std::string& kind) {
  const oasis_paged_shape s{3, 8, 2, 128, 16, 4000, 100};
  int32_t* ints = reinterpret_cast<int32_t*>(memory);
  if (kind == "resume_kv_q8")
    return oasis_resume_kv_q8(&s, memory, 1024, memory, 256, memory, 256, ints, 50, memory, reinterpret_cast<float*>(memory), ints,
                              ints, 9000, 0.1f, memory, kMuch, memory, 1024, nullptr, nullptr);
  if (kind == "resume_kv_q4")
    return oasis_resume_kv_q4(&s, memory, 1024, memory, 256, memory, 256, ints, 50, memory, memory, ints, ints, 9000, 0.1f, memory,
                              kMuch, memory, 1024, nullptr, nullptr);
  if (kind == "resume")
    return oasis_resume_attn(&s, memory, 1024, memory, 256, memory, 256, ints, 50, ints, 9000, 0.1f, memory, kMuch, memory, 1024,
                             nullptr, nullptr);
  if (kind == "decode_q8")
    return oasis_paged_decode_attn_q8(&s, memory, 1024, memory, reinterpret_cast<float*>(memory), ints, ints, nullptr, nullptr, 0,
                                      0.1f, memory, kMuch, memory, nullptr, nullptr);
  if (kind == "decode_q4")
    return oasis_paged_decode_attn_q4(&s, memory, 1024, memory, memory, ints, ints, nullptr, nullptr, 0, 0.1f, memory, kMuch,
                                      memory, nullptr, nullptr);
  return OASIS_ERR_INVALID;
}
}  // namespace

int main(int argc, char** argv) {
  if (argc != 3) return 2;
  oasis_status status[2] = {OASIS_OK, OASIS_OK};
  auto run = [&](char name) {
    me = name;
    for (int i = 0; i < 5; ++i) {
      const oasis_status st = call(argv[1 + name - 'a']);
      if (st != OASIS_OK) status[name - 'a'] = st;
    }
  };
  std::thread a([&] { run('a'); });
  std::thread b([&] {
    rest(5);
    run('b');
  });
  a.join();
  b.join();
  printf("status %d %d\norder %s\n", (int)status[0], (int)status[1], order.c_str());
  return 0;
}
