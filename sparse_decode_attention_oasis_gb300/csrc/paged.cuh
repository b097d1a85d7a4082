// Types and device helpers shared by the kernels of the paged cache, in 8 and in 4 bits.
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

// Pages in 4 bits: groups of 16 dimensions of a token share a scale byte.
constexpr int kGroup = 16, kGroups = kD / kGroup;
constexpr long long kHeadPageBytes4 = kHeadPageBytes / 2;        // codes of one head in one page
constexpr long long kHeadScaleBytes4 = 2LL * kBS * kGroups;      // its scales: keys [token][group], values [group][token]
// A scale byte is an unsigned float with 5 exponent and 3 fraction bits: the half with bits b << 7.  The largest in use,
// 10,240 = 1.25 * 2^13, keeps 6 * scale = 61,440 below fp16's largest value, so that every stored value (2 + 4 significant
// bits, a multiple of 2^-18) is a half, and a bf16, exactly.  0xff (a NaN as a half) marks a group that held a NaN.
constexpr int kScaleByteHigh = 226, kScaleByteNaN = 255;

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

__device__ __forceinline__ uint2 load8_stream(const void* p) {
  uint2 r;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t load2_stream(const void* p) {
  uint16_t r;
  asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=h"(r) : "l"(p) : "memory");
  return r;
}

// Byte kByte of w, two e2m1 codes (the lower in its lower bits) -> two halves, exact.
template <int kByte>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (kByte == 0) asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, a;\n}" : "=r"(r) : "r"(w));
  if constexpr (kByte == 1) asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, b;\n}" : "=r"(r) : "r"(w));
  if constexpr (kByte == 2) asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, c;\n}" : "=r"(r) : "r"(w));
  if constexpr (kByte == 3) asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %1;\n cvt.rn.f16x2.e2m1x2 %0, d;\n}" : "=r"(r) : "r"(w));
  return r;
}

// Scale bytes 0 and 1 of w as the two halves of a word; scale byte kByte of w in both.
__device__ __forceinline__ uint32_t scale_pair(uint32_t w) { return __byte_perm(w, 0, 0x4140) << 7; }
template <int kByte>
__device__ __forceinline__ uint32_t scale_twice(uint32_t w) { return __byte_perm(w, 0, 0x4040 + 0x0101 * kByte) << 7; }

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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

// Held by a call while it issues launches that read what its earlier ones left in the workspace: of two host threads that
// share a stream and a workspace, in whichever of the paged cache's calls, none comes between.
inline std::mutex& workspace_lock() {
  static std::mutex locks[kMaxDevicesCached];
  return locks[current_device()];
}

__device__ __forceinline__ void set_err(unsigned* err, unsigned bits) {
  if (err != nullptr && bits) atomicOr(err, bits);
}

}  // namespace oasis
