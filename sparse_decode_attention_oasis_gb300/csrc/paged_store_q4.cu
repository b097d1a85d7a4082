// New K/V rows quantised into 4-bit pages (oasis_store_kv_q4).
//
// Mathematics: for 16 dimensions of one token of one head, s = the least scale (5 exponent, 3 fraction
// bits) of at least amax / 6 (6: the largest e2m1), y = e2m1(x / s), ties to the even code.  Every
// token has its own scales, so a page's earlier tokens stay as they are, whatever comes later.
// The quotient is formed as x * (1 / s) in fp32, from an approximate reciprocal (2^-22 off at most),
// and rounded to a multiple of 2^-16 by adding and taking away 192; that has one right answer: with 8
// bits in x and 4 in s a quotient is a tie of the codes (a multiple of 1/4) exactly or is 2^-11 away
// from each, and the product is off by less than 2^-19, so ties come out as ties and everything else
// stays on its side.  Likewise amax * fl(1/6) is s where amax is 6 s (fl(1/6) is 2^-25 too large, less
// than half a step at the 4 bits of s), and 2^-8 away from it elsewhere.
//
// A lane has a group, a warp's instruction four rows of one head; rows are independent, so there is no order to keep
// and nothing is read but the rows.
// Bound: HBM, 656 B for a row, head, K and V, with the instructions close behind.  15,600 rows of 8 heads (82 MB):
// 13.9 us, 5.9 TB/s, 0.88 of the measured copy rate (15.7 with a group to a pair of lanes, half the instructions being
// spent twice; 20.2 with two divisions for each group and quotients one by one as well).  4 and 16 rows to a warp take
// 16.8 and 14.0; 32 rows of a decode step: 1.4 us.
#include <cuda_fp16.h>

#include "paged.cuh"

namespace oasis {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 8;  // rows of a warp in long calls

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The byte of the least scale of at least amax / 6, at most the largest one in use.
__device__ __forceinline__ int scale_byte(float amax) {
  const float r = __fmul_rn(amax, 1.0f / 6.0f);
  if (r < 6.103515625e-5f) return (int)ceilf(r * 131072.0f);  // below 2^-14: multiples of 2^-17
  return (int)min((__float_as_uint(r) + 0xfffffu) >> 20, (uint32_t)(kScaleByteHigh + 896)) - 896;  // 896: exponents' bias
}

// a * inv rounded to a multiple of 2^-16, both halves of a pair.
__device__ __forceinline__ void quotients(uint32_t w, uint64_t inv, float& lo, float& hi) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(w << 16), "r"(w & 0xffff0000u));
  asm("{\n .reg .b64 c, d;\n mov.b64 c, {%3, %3};\n mov.b64 d, {%4, %4};\n fma.rn.f32x2 %0, %1, %2, c;\n"
      " add.rn.f32x2 %0, %0, d;\n}"
      : "=l"(x)
      : "l"(x), "l"(inv), "f"(192.0f), "f"(-192.0f));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}

// Eight quotients -> codes, the lowest dimension in the lowest bits; a zero has no sign.
__device__ __forceinline__ uint32_t codes8(const float* y) {
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  const uint32_t some = (w | w >> 1 | w >> 2) & 0x11111111u;
  return w & (0x77777777u | some << 3);
}

// The 16 elements of a group; kWide: rows on 32-byte boundaries.
template <bool kWide>
__device__ __forceinline__ void load_group(const uint16_t* p, uint32_t* w) {
  if constexpr (kWide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 4)  // the second load finds the sectors in L1
      asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "l"(p + 2 * i)
                   : "memory");
  }
}

// grid: x = groups of kWarps * per rows, y = heads * 2 (K, V); per: rows of a warp, 4 or kRows.
template <int kPer, bool kWide>
__global__ void __launch_bounds__(kWarps * 32)
store_kv_q4_kernel(PagedShape s, const uint16_t* k, size_t k_stride, const uint16_t* v, size_t v_stride,
                   const int* slot_map, int n_rows, uint8_t* pages, uint8_t* scales, unsigned* err) {
  wait_for_predecessor();
  const int lane = threadIdx.x & 31, sub = lane >> 3, group = lane & 7;
  const int h = blockIdx.y >> 1, which = blockIdx.y & 1;
  const uint16_t* src = (which ? v : k) + (size_t)h * kD + group * 16;
  const size_t stride = which ? v_stride : k_stride;
  const long long r0 = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kPer;
  const unsigned n_slots = (unsigned)s.n_pages * kBS;
  unsigned bits = 0;
  // of page 0, token 0; a page further is `page_bytes`, `scale_bytes` on
  uint8_t* const codes = pages + (size_t)h * kHeadPageBytes4 + which * (kBS * kD / 2) + group * 8;
  uint8_t* const to = scales + (size_t)h * kHeadScaleBytes4 + which * (kBS * kGroups) + group * (which ? kBS : 1);
  const unsigned page_bytes = s.Hkv * kHeadPageBytes4, scale_bytes = s.Hkv * kHeadScaleBytes4, step = which ? 1 : kGroups;
  if (r0 >= n_rows) return;
  uint32_t x[kPer / 4][8];
  int slot[kPer / 4];
#pragma unroll
  for (int i = 0; i < kPer / 4; ++i) {
    const int r = (int)min(r0 + 4 * i + sub, (long long)n_rows - 1);  // behind the last row: that again, stored nowhere
    slot[i] = r0 + 4 * i + sub < n_rows ? slot_map[r] : -1;
    load_group<kWide>(src + (size_t)r * stride, x[i]);
  }
#pragma unroll
  for (int i = 0; i < kPer / 4; ++i) {
    const uint32_t* w = x[i];
    uint32_t m = 0;
#pragma unroll
    for (int d = 0; d < 8; ++d) m = max_u16x2(m, w[d] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
    const bool nan = m > 0x7f80u;
    const int b = scale_byte(__uint_as_float(m << 16));
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(__half2float(__ushort_as_half((unsigned short)max(b << 7, 128)))));
    uint64_t inv2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(inv2) : "f"(inv));
    float y[16];
#pragma unroll
    for (int d = 0; d < 8; ++d) quotients(w[d], inv2, y[2 * d], y[2 * d + 1]);  // all zeros where b is 0
    const uint2 code = nan ? make_uint2(0u, 0u) : make_uint2(codes8(y), codes8(y + 8));
    const unsigned at = (unsigned)slot[i], page = at / kBS, pos = at % kBS;
    const bool good = at < n_slots;
    bits |= good || slot[i] == -1 ? 0u : (unsigned)OASIS_EW_BAD_SLOT;
    if (good) *reinterpret_cast<uint2*>(codes + (size_t)page * page_bytes + pos * (kD / 2)) = code;
    if (good) to[(size_t)page * scale_bytes + pos * step] = (uint8_t)(nan ? kScaleByteNaN : b);
  }
  if (blockIdx.y == 0) set_err(err, bits);
}

template <bool kWide>
cudaError_t launch(const PagedShape& s, const uint16_t* k, size_t k_stride, const uint16_t* v, size_t v_stride,
                   const int* slot_map, int n_rows, uint8_t* pages, uint8_t* scales, unsigned* err, cudaStream_t stream) {
  // Four rows to a warp while all those warps are resident at once; long calls take kRows for the loads in flight.
  const bool few = ((long long)n_rows + 3) / 4 * s.Hkv * 2 <= (long long)sm_count() * 64;
  const int per = few ? 4 : kRows;
  const dim3 grid((unsigned)(((long long)n_rows + kWarps * per - 1) / (kWarps * per)), (unsigned)(2 * s.Hkv));
  return launch_chained(few ? store_kv_q4_kernel<4, kWide> : store_kv_q4_kernel<kRows, kWide>, grid, dim3(kWarps * 32), 0, stream,
                        1, s, k, k_stride, v, v_stride, slot_map, n_rows, pages, scales, err);
}

}  // namespace

cudaError_t launch_store_kv_q4(const PagedShape& s, const uint16_t* k, size_t k_stride, const uint16_t* v, size_t v_stride,
                               const int* slot_map, int n_rows, uint8_t* pages, uint8_t* scales, unsigned* err,
                               cudaStream_t stream) {
  if (n_rows == 0) return cudaSuccess;
  // 15,600 rows in slices of a fused buffer: 14.2 us on 32-byte boundaries, 15.3 where only 16 bytes can be loaded at once
  const bool wide = (reinterpret_cast<uintptr_t>(k) & 31) == 0 && (reinterpret_cast<uintptr_t>(v) & 31) == 0 &&
                    k_stride % 16 == 0 && v_stride % 16 == 0;
  return (wide ? launch<true> : launch<false>)(s, k, k_stride, v, v_stride, slot_map, n_rows, pages, scales, err, stream);
}

}  // namespace oasis
