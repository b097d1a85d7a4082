// Types and device helpers shared by the paged 8-bit cache's kernels.
#pragma once

#include "common.cuh"

namespace oasis {

struct PagedShape {
  int B, Hq, Hkv, nb_max, n_pages;
  __host__ __device__ int G() const { return Hq / Hkv; }
};

// Exponent range of a page's scale 2^e.  High: 448 * 2^119 = 1.75 * 2^127 is the largest page value
// that fp32 holds (448 * 2^120 does not fit), so the finite bf16 above it (up to 1.9922 * 2^127)
// saturate there, by an eighth at most.  Low: below -60 a page's values are as good as zero.
constexpr int kScaleELow = -60, kScaleEHigh = 119;
constexpr long long kHeadPageBytes = 2LL * kBS * kD;  // keys and values of one head in one page

// 16-byte loads (coherent: see launch_chained); the second leaves no line in L1.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ uint4 load16_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // e in [-126, 127]

// Two e4m3 (low 16 bits of w) -> two halves, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(r) : "r"(w));
  return r;
}

// Two floats -> two e4m3 (round to nearest even, saturating); lo in bits 0..7.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Kernels of a decode step follow each other closely: each is launched while its predecessor in the
// stream still runs (programmatic stream serialization), sets itself up, and waits for the
// predecessor's end before it touches global memory.  What the predecessor writes changes while
// such a kernel lives: so none of its pointers is __restrict__, and no load takes the
// non-coherent path, either of which would let a load pass the wait.
__device__ __forceinline__ void wait_for_predecessor() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
}

template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int cluster,
                           Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

__device__ __forceinline__ void set_err(unsigned* err, unsigned bits) {
  if (err != nullptr && bits) atomicOr(err, bits);
}

}  // namespace oasis
