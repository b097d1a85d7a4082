// Held tokens read back from their pages as packed bf16 rows, new rows behind them (oasis_read_kv_q8, _q4).
//
// Mathematics: value = code * scale.  e4m3 times a power of two has 4 significant bits, e2m1 times
// a scale of 4 bits has 6, so both are bf16 values exactly and nothing is rounded.
//
// Work: a unit is 16 positions of one request and one KV head, its page's keys and values (or the
// new rows that lie there).  The units of all requests, heads innermost, form one sequence, cut into
// equal ranges for the thread blocks; a block's warps take its units in turn.  Each lane has 32
// dimensions of two tokens, whole 32-byte sectors to a store.
// Bound: HBM, 10.5 KB read and written for a unit in 4 bits, 12.3 in 8.  46,700 tokens of 8 heads in ten requests
// (254 MB, 4 bits): 45 us, 5.7 TB/s, 0.85 of the measured copy rate; 1,000 tokens: 5.3 us, four loads that wait for one
// another.  Blocks of 16 units, so that the ones that finish early make room: one range for each place of the GPU 49 us;
// one unit to a warp 46; two blocks an SM 46 (1,000 tokens: 4.5), four 57.  These are figures of 4 bits; in 8 the same
// 46,700 tokens (296 MB) take 64 us, 4.6 TB/s, 0.69: at three blocks an SM its 80 registers spill 124 bytes.  In a cache of
// 512 slots of which two hold tokens the call takes 10.0 us against 9.3 without the others, of 4,096 25.
#include <cuda_fp16.h>

#include "paged.cuh"

namespace oasis {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 3;
constexpr int kUnits = 2;  // of a warp in long calls of few requests

struct Args {
  const uint8_t* pages;
  const void* scales;  // 8 bits: float, 4 bits: bytes
  const int* table;
  const int* ctx_len;
  const uint16_t *k_new, *v_new;
  size_t k_stride, v_stride;
  const int* new_start;  // NULL: no new rows
  int n_new;
  bool only_new;  // requests without new rows have no rows at all
  int* kv_start;
  uint16_t *k_out, *v_out;
  int n_rows;
  unsigned* err;
};

struct Request {
  int held, fresh;  // tokens in pages, new rows
  int first;        // its first new row
};

__device__ __forceinline__ Request request(const PagedShape& s, const Args& a, int b, unsigned* bits) {
  Request r;
  r.held = (int)min((long long)max(a.ctx_len[b], 0), (long long)s.nb_max * kBS);
  r.fresh = r.first = 0;
  if (a.new_start != nullptr) {
    const int from = a.new_start[b], to = a.new_start[b + 1];
    if (from < 0 || to < from || to > a.n_new) {
      *bits |= OASIS_EW_BAD_COUNT;
    } else {
      r.first = from;
      r.fresh = to - from;
    }
  }
  if (a.only_new && r.fresh == 0) r.held = 0;
  return r;
}

// The block's exclusive prefix of x; total: the sum.
__device__ __forceinline__ long long block_prefix(long long x, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();  // the sums of the call before have been read
  if (lane == 31) warp_sums[warp] = y;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? warp_sums[w] : 0;
    all += warp_sums[w];
  }
  *total = all;
  return before + y - x;
}

__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h) {  // exact for stored values
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(f.x, f.y);
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 32 values of a token: codes of a lane and their scales.
struct Piece4 {
  uint4 code;
  uint32_t scale;  // two bytes
  __device__ __forceinline__ void clear() {
    code = make_uint4(0u, 0u, 0u, 0u);
    scale = 0;
  }
  __device__ __forceinline__ void load(const uint8_t* pages, const void* scales, long long head_page, int which, int t, int c) {
    code = load16_stream(pages + head_page * kHeadPageBytes4 + which * (kBS * kD / 2) + t * (kD / 2) + c * 16);
    const uint8_t* at = static_cast<const uint8_t*>(scales) + head_page * kHeadScaleBytes4 + which * (kBS * kGroups);
    if (which == 0) {
      scale = load2_stream(at + t * kGroups + c * 2);
    } else {
      uint32_t lo, hi;
      asm volatile("ld.global.u8 %0, [%1];" : "=r"(lo) : "l"(at + (2 * c) * kBS + t) : "memory");
      asm volatile("ld.global.u8 %0, [%1];" : "=r"(hi) : "l"(at + (2 * c + 1) * kBS + t) : "memory");
      scale = lo | hi << 8;
    }
  }
  __device__ __forceinline__ void values(int half, uint32_t* w) const {  // 16 of them
    const uint32_t f = half ? scale_twice<1>(scale) : scale_twice<0>(scale);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = word(code, 2 * half + i);
      w[4 * i] = f16x2_to_bf16x2(mul_f16x2(e2m1x2_to_f16x2<0>(x), f));
      w[4 * i + 1] = f16x2_to_bf16x2(mul_f16x2(e2m1x2_to_f16x2<1>(x), f));
      w[4 * i + 2] = f16x2_to_bf16x2(mul_f16x2(e2m1x2_to_f16x2<2>(x), f));
      w[4 * i + 3] = f16x2_to_bf16x2(mul_f16x2(e2m1x2_to_f16x2<3>(x), f));
    }
  }
};
struct Piece8 {
  uint4 code[2];
  float scale;
  __device__ __forceinline__ void clear() {
    code[0] = code[1] = make_uint4(0u, 0u, 0u, 0u);
    scale = 0.f;
  }
  __device__ __forceinline__ void load(const uint8_t* pages, const void* scales, long long head_page, int which, int t, int c) {
    const uint8_t* p = pages + head_page * kHeadPageBytes + which * (kBS * kD) + t * kD + c * 32;
    code[0] = load16_stream(p);
    code[1] = load16_stream(p + 16);
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(scale) : "l"(static_cast<const float*>(scales) + head_page * 2 + which) : "memory");
  }
  __device__ __forceinline__ void values(int half, uint32_t* w) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t x = word(code[half], i >> 1), h = i & 1 ? e4m3x2_hi_to_f16x2(x) : e4m3x2_to_f16x2(x);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      w[i] = pack_bf16x2(f.x * scale, f.y * scale);
    }
  }
};

template <int kBits>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
read_kv_kernel(PagedShape s, Args a) {
  using Piece = std::conditional_t<kBits == 8, Piece8, Piece4>;
  __shared__ long long warp_sums[kWarps];
  __shared__ int unit_start[kThreads], row_start[kThreads], last_end;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) last_end = 0;
  wait_for_predecessor();

  // ---- prefixes over the requests, a chunk of them to a thread
  const int per = (s.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, s.B), b1 = min(b0 + per, s.B);
  unsigned bits = 0;
  long long rows = 0, units = 0, all;
  Request mine = {};  // the chunk's only request
  for (int b = b0; b < b1; ++b) {
    mine = request(s, a, b, &bits);
    rows += (long long)mine.held + mine.fresh;
  }
  auto again = [&](int b) { return per == 1 ? mine : request(s, a, b, &bits); };  // bits of the first pass stay
  const long long row0 = block_prefix(rows, warp_sums, &all);
  // the first request whose rows do not fit, and all behind it, get none
  int end_fits = 0;
  long long at = row0;
  for (int b = b0; b < b1; ++b) {
    const Request r = again(b);
    at += (long long)r.held + r.fresh;
    if (at > a.n_rows) {
      bits |= OASIS_EW_BAD_COUNT;
    } else {
      units += ((long long)r.held + r.fresh + kBS - 1) / kBS;
      end_fits = (int)at;
    }
  }
  if (end_fits > 0) atomicMax(&last_end, end_fits);
  const long long unit0 = block_prefix(units, warp_sums, &all);
  unit_start[tid] = (int)unit0;
  row_start[tid] = (int)min(row0, (long long)a.n_rows);  // chunks that do not fit have no units
  __syncthreads();
  if (blockIdx.x == 0) {
    at = row0;
    if (tid == 0) a.kv_start[0] = 0;
    for (int b = b0; b < b1; ++b) {
      const Request r = again(b);
      at += (long long)r.held + r.fresh;
      a.kv_start[b + 1] = at > a.n_rows ? last_end : (int)at;
    }
    set_err(a.err, bits);
  }

  // ---- this warp's units (32 bits: the rows alone limit them to a 4096th of what the GPU's memory holds)
  const long long total = all * s.Hkv;
  const int lo = (int)(blockIdx.x * total / gridDim.x), hi = (int)((blockIdx.x + 1) * total / gridDim.x);
  int u = lo + warp;
  if (u >= hi) return;
  bits = 0;
  int i = 0, j = kThreads - 1;
  while (i < j) {  // the last chunk that starts at or before the unit
    const int m = (i + j + 1) >> 1;
    if (unit_start[m] <= u / s.Hkv) i = m; else j = m - 1;
  }
  int b = i * per;
  int first_unit = unit_start[i], first_row = row_start[i];
  Request r = request(s, a, b, &bits);
  for (; u < hi; u += kWarps) {
    const int idx = u / s.Hkv, h = u - idx * s.Hkv;
    while (first_unit + (r.held + r.fresh + kBS - 1) / kBS <= idx) {  // requests that fit: sums of 32 bits
      first_unit += (r.held + r.fresh + kBS - 1) / kBS;
      first_row += r.held + r.fresh;
      r = request(s, a, ++b, &bits);
    }
    const int x = idx - first_unit, pos = x * kBS;
    const int n = min(r.held + r.fresh - pos, kBS), held = min(max(r.held - pos, 0), n);
    const size_t row_elems = (size_t)s.Hkv * kD;
    const size_t out0 = (size_t)(first_row + pos) * row_elems + (size_t)h * kD;
    if (held > 0) {
      const int page = a.table[(long long)b * s.nb_max + x], t = lane >> 2, c = lane & 3;
      const bool good = page >= 0 && page < s.n_pages;
      if (!good) bits |= OASIS_EW_BAD_SLOT;
      const long long head_page = (long long)page * s.Hkv + h;
      Piece p[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {  // keys of tokens t and t + 8, values of them
        p[m].clear();
        if (good && t + (m & 1) * 8 < held) p[m].load(a.pages, a.scales, head_page, m >> 1, t + (m & 1) * 8, c);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int tok = t + (m & 1) * 8;
        if (tok >= held) continue;
        uint16_t* dst = (m >> 1 ? a.v_out : a.k_out) + out0 + tok * row_elems + c * 32;
        uint32_t w[8];
        p[m].values(0, w);
        store32(dst, w);
        p[m].values(1, w);
        store32(dst + 16, w);
      }
    }
    if (held < n) {  // new rows: two to an instruction
      const int half = lane >> 4, col = (lane & 15) * 8;
      const size_t from = (size_t)(r.first + (pos + held - r.held));
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {
        const uint16_t* src = (which ? a.v_new : a.k_new) + (size_t)h * kD + col;
        const size_t stride = which ? a.v_stride : a.k_stride;
        uint4 w[kBS / 2];
#pragma unroll
        for (int m = 0; m < kBS / 2; ++m)
          if (held + 2 * m + half < n) w[m] = load16_stream(src + (from + 2 * m + half) * stride);
        uint16_t* dst = (which ? a.v_out : a.k_out) + out0 + col;
#pragma unroll
        for (int m = 0; m < kBS / 2; ++m)
          if (held + 2 * m + half < n) *reinterpret_cast<uint4*>(dst + (held + 2 * m + half) * row_elems) = w[m];
      }
    }
  }
  set_err(a.err, bits);
}

}  // namespace

template <int kBits>
static cudaError_t launch(const PagedShape& s, const Args& a, cudaStream_t stream) {
  // every request may end in a partly filled unit
  const long long units = ((long long)a.n_rows / kBS + (s.B < a.n_rows ? s.B : a.n_rows)) * s.Hkv;
  const long long one = (units + kWarps - 1) / kWarps, most = (long long)kCtasPerSm * sm_count();
  long long grid = one < 1 ? 1 : one < most ? one : most;
  // every block goes over all requests, so where those are many there are no more blocks than places
  if (s.B <= kThreads && (one + kUnits - 1) / kUnits > most) grid = (one + kUnits - 1) / kUnits;
  return launch_chained(read_kv_kernel<kBits>, dim3((unsigned)grid), dim3(kThreads), 0, stream, 1, s, a);
}

cudaError_t launch_read_kv(int bits, const PagedShape& s, const uint8_t* pages, const void* scales, const int* table,
                           const int* ctx, const uint16_t* k_new, size_t k_stride, const uint16_t* v_new, size_t v_stride,
                           const int* new_start, int n_new, bool only_new, int* kv_start, uint16_t* k_out, uint16_t* v_out, int n_rows,
                           unsigned* err, cudaStream_t stream) {
  const Args a{pages, scales, table, ctx, k_new, v_new, k_stride, v_stride, new_start, n_new,
               only_new, kv_start, k_out, v_out, n_rows, err};
  return bits == 8 ? launch<8>(s, a, stream) : launch<4>(s, a, stream);
}

}  // namespace oasis
