// New K/V rows quantised into 8-bit pages (oasis_store_kv_q8).
//
// Mathematics: for the rows of one page and one head, e = the least exponent with
// amax <= 448 * 2^e over the tokens that the page then holds (448: the largest
// e4m3), y = e4m3(x * 2^-e).  The scale is a power of two so that x * 2^-e is exact
// in fp32 and the only rounding is the one to e4m3 (3 mantissa bits: half a step is
// 2^-4 of the value), and so that a page whose scale grows by later tokens keeps
// its earlier values exactly, but for those that become subnormal; a scale
// amax/448 would round them a second time.
//
// One warp per (run of rows in one page, head, K or V): 16 lanes cover a row's 256
// bytes in 16-byte loads, two rows to an instruction, held in registers from the
// maximum to the conversion, so that every row is read once.  Bound: HBM.  15,170 tokens of
// 8 heads (93 MB): 17.1 us, 5.5 TB/s, 0.81 of the measured copy rate, of which 2 us are launch
// and first loads; 32 tokens of a decode step: 2.3 us, 4.7 to 6.0 where every page's scale grows.
#include "paged.cuh"

namespace oasis {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The least e with amax <= 448 * 2^e = 1.75 * 2^(e + 8); bits: |x| as bf16 (its
// exponent field E and 7 mantissa bits; infinities and NaN end at the high clamp).
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  const int e = (int)(bits >> 7) - 127 - 8 + ((bits & 0x7f) > 0x60 ? 1 : 0);
  return min(max(e, kScaleELow), kScaleEHigh);
}

// Four e4m3 values times f = 2^de (de < 0), rounded to nearest even again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const uint32_t lo = e4m3x2_to_f16x2(w), hi = e4m3x2_hi_to_f16x2(w);
  float a, b, c, d;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}" : "=f"(a), "=f"(b) : "r"(lo));
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}" : "=f"(c), "=f"(d) : "r"(hi));
  return f32x2_to_e4m3x2(a * f, b * f) | (f32x2_to_e4m3x2(c * f, d * f) << 16);
}

// grid: x = groups of kWarps * rows_per_warp rows, y = heads * 2 (K, V).
__global__ void __launch_bounds__(kWarps * 32)
store_kv_q8_kernel(PagedShape s, const uint16_t* k, size_t k_stride, const uint16_t* v,
                   size_t v_stride, const int* slot_map, int n_rows, int rows_per_warp,
                   uint8_t* pages, float* scales, unsigned* err) {
  wait_for_predecessor();
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y >> 1, which = blockIdx.y & 1;
  const uint16_t* src = which ? v : k;
  const size_t stride = which ? v_stride : k_stride;
  const int r0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * rows_per_warp;
  const int r1 = min(r0 + rows_per_warp, n_rows);
  const int n_slots = s.n_pages * kBS;
  unsigned bits = 0;
  if (r0 >= n_rows) return;

  int r = r0;
  while (r < r1) {
    // lane j looks at row r - 1 + j: a run starts where a slot is on another page than its predecessor's
    const int row = r - 1 + lane;
    const int slot = row >= 0 && row < n_rows ? slot_map[row] : -1;
    const bool good = slot >= 0 && slot < n_slots;
    const int prev = __shfl_up_sync(0xffffffffu, slot, 1);
    const bool same = good && prev >= 0 && prev / kBS == slot / kBS;
    const bool mine = lane >= 1 && row < r1;
    if (mine && slot != -1 && !good) bits |= OASIS_EW_BAD_SLOT;
    if (mine && same && slot != prev + 1) bits |= OASIS_EW_BAD_COUNT;
    const unsigned starts = __ballot_sync(0xffffffffu, mine && good && !same);
    if (starts == 0) {
      r += 31;
      continue;
    }
    const int first = __ffs(starts) - 1;  // the lane of the next run's first row
    const int row_a = r - 1 + first;
    const int slot_a = __shfl_sync(0xffffffffu, slot, first);
    const int page = slot_a / kBS, pos = slot_a % kBS;
    // its length: rows in consecutive positions up to the page's end
    int next = __shfl_sync(0xffffffffu, slot, (first + lane) & 31);
    if (first + kBS > 32) next = row_a + lane < n_rows ? slot_map[row_a + lane] : -1;  // not all of them are at hand
    const unsigned cont = __ballot_sync(0xffffffffu, lane < kBS - pos && next == slot_a + lane);
    const int len = __ffs(~cont) - 1;

    const int half = lane >> 4, col = lane & 15;  // two rows to an instruction, 8 dimensions to a lane
    const uint16_t* base = src + (size_t)row_a * stride + (size_t)h * kD + col * 8;
    uint4 x[kBS / 2];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kBS / 2; ++i) {
      const int t = 2 * i + half;
      x[i] = t < len ? load16_stream(base + (size_t)t * stride) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kBS / 2; ++i) {
      m = max_u16x2(m, max_u16x2(max_u16x2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                 max_u16x2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
    int e = scale_exponent(max(m & 0xffffu, m >> 16));

    const long long head_page = (long long)page * s.Hkv + h;
    uint8_t* dst = pages + head_page * kHeadPageBytes + which * (kBS * kD);
    float* scale = scales + head_page * 2 + which;
    if (pos > 0) {  // the page holds tokens 0 .. pos - 1
      const int e_old = min(max((int)((__float_as_uint(*scale) >> 23) & 0xff) - 127, kScaleELow), kScaleEHigh);
      if (e > e_old) {
        const float f = pow2f(max(e_old - e, -126));  // below 2^-20 every value rounds to zero
        for (int i = lane; i < pos * (kD / 4); i += 32) {
          uint32_t* w = reinterpret_cast<uint32_t*>(dst) + i;
          *w = rescale4(*w, f);
        }
      } else {
        e = e_old;
      }
    }
    __syncwarp();
    if (lane == 0) *scale = pow2f(e);
    const float f = pow2f(-e);
#pragma unroll
    for (int i = 0; i < kBS / 2; ++i) {
      const int t = 2 * i + half;
      if (t < len) {
        uint2 y;
        y.x = f32x2_to_e4m3x2(bf_lo(x[i].x) * f, bf_hi(x[i].x) * f) |
              (f32x2_to_e4m3x2(bf_lo(x[i].y) * f, bf_hi(x[i].y) * f) << 16);
        y.y = f32x2_to_e4m3x2(bf_lo(x[i].z) * f, bf_hi(x[i].z) * f) |
              (f32x2_to_e4m3x2(bf_lo(x[i].w) * f, bf_hi(x[i].w) * f) << 16);
        *reinterpret_cast<uint2*>(dst + (pos + t) * kD + col * 8) = y;
      }
    }
    r = row_a + len;  // rows of a broken run that follow are looked at (and flagged) by the next turn
  }
  if (blockIdx.y == 0) set_err(err, bits);
}

}  // namespace

cudaError_t launch_store_kv_q8(const PagedShape& s, const uint16_t* k, size_t k_stride, const uint16_t* v,
                               size_t v_stride, const int* slot_map, int n_rows, uint8_t* pages, float* scales,
                               unsigned* err, cudaStream_t stream) {
  if (n_rows == 0) return cudaSuccess;
  // A decode step's rows are each a page's run of their own: a warp for each row keeps
  // the loads in flight at once.  A prompt's runs have 16 rows.
  const long long resident = (long long)sm_count() * 32;
  const int per = (long long)n_rows * s.Hkv * 2 <= resident ? 1 : kBS;
  const long long groups = ((long long)n_rows + kWarps * per - 1) / (kWarps * per);
  dim3 grid((unsigned)groups, (unsigned)(2 * s.Hkv));
  return launch_chained(store_kv_q8_kernel, grid, dim3(kWarps * 32), 0, stream, 1, s, k, k_stride, v, v_stride, slot_map,
                        n_rows, per, pages, scales, err);
}

}  // namespace oasis
