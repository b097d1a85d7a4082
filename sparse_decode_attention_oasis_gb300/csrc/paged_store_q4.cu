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
// Two rows of one head to a warp's instruction: 16 lanes of 16 bytes cover a row, a pair of lanes a
// group.  Rows are independent, so there is no order to keep and nothing is read but the rows.
// Bound: HBM, 656 B for a row, head, K and V, with the instructions close behind.  15,600 rows of 8 heads (82 MB):
// 15.6 us, 5.3 TB/s, 0.79 of the measured copy rate (20.2 with two divisions for each group and quotients
// one by one); 4, 16 and 32 rows to a warp take 17.5, 17.9 and 19.6; 32 rows of a decode step: 1.4 us.
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

// grid: x = groups of kWarps * per rows, y = heads * 2 (K, V); per: rows of a warp, 2 or kRows.
template <int kPer>
__global__ void __launch_bounds__(kWarps * 32)
store_kv_q4_kernel(PagedShape s, const uint16_t* k, size_t k_stride, const uint16_t* v, size_t v_stride,
                   const int* slot_map, int n_rows, uint8_t* pages, uint8_t* scales, unsigned* err) {
  wait_for_predecessor();
  const int lane = threadIdx.x & 31, half = lane >> 4, col = lane & 15;
  const int h = blockIdx.y >> 1, which = blockIdx.y & 1;
  const uint16_t* src = (which ? v : k) + (size_t)h * kD + col * 8;
  const size_t stride = which ? v_stride : k_stride;
  const long long r0 = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kPer;
  const unsigned n_slots = (unsigned)s.n_pages * kBS;
  unsigned bits = 0;
  // of page 0, token 0; a page further is `page_bytes`, `scale_bytes` on
  uint8_t* const codes = pages + (size_t)h * kHeadPageBytes4 + which * (kBS * kD / 2) + col * 4;
  uint8_t* const to = scales + (size_t)h * kHeadScaleBytes4 + which * (kBS * kGroups) + (col >> 1) * (which ? kBS : 1);
  const unsigned page_bytes = s.Hkv * kHeadPageBytes4, scale_bytes = s.Hkv * kHeadScaleBytes4, step = which ? 1 : kGroups;
  if (r0 >= n_rows) return;
  uint4 x[kPer / 2];
  int slot[kPer / 2];
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) {
    const long long r = r0 + 2 * i + half;
    slot[i] = r < n_rows ? slot_map[r] : -1;
    x[i] = r < n_rows ? load16_stream(src + (size_t)r * stride) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t m = max_u16x2(max_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                           max_u16x2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    m = max(m & 0xffffu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));  // the group's other lane
    const bool nan = m > 0x7f80u;
    const int b = scale_byte(__uint_as_float(m << 16));
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(__half2float(__ushort_as_half((unsigned short)max(b << 7, 128)))));
    uint64_t inv2;
    asm("mov.b64 %0, {%1, %1};" : "=l"(inv2) : "f"(inv));
    float y[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) quotients(w[d], inv2, y[2 * d], y[2 * d + 1]);  // all zeros where b is 0
    const uint32_t code = nan ? 0u : codes8(y);
    const unsigned at = (unsigned)slot[i], page = at / kBS, pos = at % kBS;
    const bool good = at < n_slots;
    bits |= good || slot[i] == -1 ? 0u : (unsigned)OASIS_EW_BAD_SLOT;
    if (good) *reinterpret_cast<uint32_t*>(codes + (size_t)page * page_bytes + pos * (kD / 2)) = code;
    if (good && (col & 1) == 0) to[(size_t)page * scale_bytes + pos * step] = (uint8_t)(nan ? kScaleByteNaN : b);
  }
  if (blockIdx.y == 0) set_err(err, bits);
}

}  // namespace

cudaError_t launch_store_kv_q4(const PagedShape& s, const uint16_t* k, size_t k_stride, const uint16_t* v, size_t v_stride,
                               const int* slot_map, int n_rows, uint8_t* pages, uint8_t* scales, unsigned* err,
                               cudaStream_t stream) {
  if (n_rows == 0) return cudaSuccess;
  // Two rows to a warp while all those warps are resident at once; long calls take kRows for the loads in flight.
  const long long resident = (long long)sm_count() * 64;
  const bool few = ((long long)n_rows + 1) / 2 * s.Hkv * 2 <= resident;
  const int per = few ? 2 : kRows;
  const dim3 grid((unsigned)(((long long)n_rows + kWarps * per - 1) / (kWarps * per)), (unsigned)(2 * s.Hkv));
  if (few)
    return launch_chained(store_kv_q4_kernel<2>, grid, dim3(kWarps * 32), 0, stream, 1, s, k, k_stride, v, v_stride, slot_map,
                          n_rows, pages, scales, err);
  return launch_chained(store_kv_q4_kernel<kRows>, grid, dim3(kWarps * 32), 0, stream, 1, s, k, k_stride, v, v_stride,
                        slot_map, n_rows, pages, scales, err);
}

}  // namespace oasis
