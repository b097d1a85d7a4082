// Causal attention over packed prompts (oasis_prompt_attn).
//
// Mathematics: one pass over the keys with the running maximum and sum of a
// softmax, o = sum_j 2^(c s_j - M) v_j / sum_j 2^(c s_j - M), c = scale * log2(e).
//
// Rows: the G query heads of a KV head and consecutive tokens are packed into the
// rows of a tile (row = token * G + head), so that every K/V tile is read once for
// the whole group and a tile of short sequences is not mostly empty.
// Roundings: weights to bf16 for the product with V (2^-9 each, the sums are of the
// unrounded fp32 weights), the output to bf16; scores, maxima, sums and
// accumulators are fp32.
#include "paged.cuh"

namespace oasis {
namespace {

constexpr int kWarps = 4;
constexpr int kTileRows = kWarps * 16;
constexpr int kTileKeys = 32;
constexpr int kPitch = kD + 8;  // shared-memory row pitch in elements

__device__ __forceinline__ void ldsm_x4(uint32_t* r, const uint16_t* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"((uint32_t)__cvta_generic_to_shared(p)));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t* r, const uint16_t* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"((uint32_t)__cvta_generic_to_shared(p)));
}

__global__ void __launch_bounds__(kWarps * 32)
prompt_attn_kernel(PagedShape s, const uint16_t* __restrict__ q, size_t q_stride, const uint16_t* __restrict__ k,
                   size_t k_stride, const uint16_t* __restrict__ v, size_t v_stride,
                   const int* __restrict__ row_start, int n_rows, float scale_log2, uint16_t* __restrict__ out,
                   size_t out_stride, unsigned* __restrict__ err) {
  __shared__ __align__(16) uint16_t ks[kTileKeys * kPitch], vs[kTileKeys * kPitch];
  __shared__ int found[3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = s.Hq / s.Hkv, per = kTileRows / G;  // tokens in a tile
  const int h = blockIdx.y;
  if (tid == 0) {
    int tile = blockIdx.x;
    found[0] = -1;
    for (int b = 0; b < s.B; ++b) {
      const int a = row_start[b], z = row_start[b + 1];
      if (a < 0 || z < a || z > n_rows) {
        if (blockIdx.x == 0 && blockIdx.y == 0) set_err(err, OASIS_EW_BAD_COUNT);
        continue;
      }
      const int n = (z - a + per - 1) / per;
      if (tile < n) {
        found[0] = a;
        found[1] = z;
        found[2] = tile * per;
        break;
      }
      tile -= n;
    }
  }
  __syncthreads();
  if (found[0] < 0) return;
  const int a = found[0], len = found[1] - a, t0 = found[2];

  const int row[2] = {warp * 16 + (lane >> 2), warp * 16 + (lane >> 2) + 8};
  int tok[2];
  bool live[2];
  uint32_t qf[8][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    tok[i] = t0 + row[i] / G;
    live[i] = row[i] < per * G && tok[i] < len;
    const uint16_t* src = q + (size_t)(a + tok[i]) * q_stride + (size_t)(h * G + row[i] % G) * kD + (lane & 3) * 2;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      qf[m][i] = live[i] ? *reinterpret_cast<const uint32_t*>(src + m * 16) : 0u;
      qf[m][2 + i] = live[i] ? *reinterpret_cast<const uint32_t*>(src + m * 16 + 8) : 0u;
    }
  }
  float acc[16][4] = {};
  float top[2] = {neg_inf(), neg_inf()}, sum[2] = {0.f, 0.f};
  const int keys = min(len, t0 + per);
  for (int j0 = 0; j0 < keys; j0 += kTileKeys) {
    __syncthreads();
    for (int i = tid; i < kTileKeys * 16; i += kWarps * 32) {
      const int r = i >> 4, c = (i & 15) * 8;
      const bool in = j0 + r < len;
      const size_t at = (size_t)(a + j0 + r);
      *reinterpret_cast<uint4*>(ks + r * kPitch + c) =
          in ? ldg_nc(k + at * k_stride + (size_t)h * kD + c) : make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(vs + r * kPitch + c) =
          in ? ldg_nc(v + at * v_stride + (size_t)h * kD + c) : make_uint4(0u, 0u, 0u, 0u);
    }
    __syncthreads();
    float sc[4][4] = {};
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int n = 0; n < 4; n += 2) {
        uint32_t r[4];
        ldsm_x4(r, ks + (n * 8 + (lane & 7) + (lane & 16 ? 8 : 0)) * kPitch + m * 16 + (lane & 8));
        mma_bf16_16816(sc[n][0], sc[n][1], sc[n][2], sc[n][3], qf[m][0], qf[m][1], qf[m][2], qf[m][3], r[0], r[1]);
        mma_bf16_16816(sc[n + 1][0], sc[n + 1][1], sc[n + 1][2], sc[n + 1][3], qf[m][0], qf[m][1], qf[m][2], qf[m][3],
                       r[2], r[3]);
      }
    float big[2] = {neg_inf(), neg_inf()};
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j = j0 + n * 8 + (lane & 3) * 2 + (c & 1);
        sc[n][c] = j <= tok[c >> 1] && j < len ? sc[n][c] * scale_log2 : neg_inf();
        big[c >> 1] = fmaxf(big[c >> 1], sc[n][c]);
      }
    float f[2], ref[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      big[i] = fmaxf(big[i], __shfl_xor_sync(0xffffffffu, big[i], 1));
      big[i] = fmaxf(big[i], __shfl_xor_sync(0xffffffffu, big[i], 2));
      const float next = fmaxf(top[i], big[i]);
      f[i] = top[i] == neg_inf() ? 0.f : exp2f(top[i] - next);
      top[i] = next;
      ref[i] = next == neg_inf() ? 0.f : next;
      sum[i] *= f[i];
    }
    uint32_t p[4][2];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        sc[n][c] = exp2f(sc[n][c] - ref[c >> 1]);
        sum[c >> 1] += sc[n][c];
      }
      p[n][0] = pack_bf16x2(sc[n][0], sc[n][1]);
      p[n][1] = pack_bf16x2(sc[n][2], sc[n][3]);
    }
#pragma unroll
    for (int d = 0; d < 16; ++d) {
      acc[d][0] *= f[0];
      acc[d][1] *= f[0];
      acc[d][2] *= f[1];
      acc[d][3] *= f[1];
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int d = 0; d < 16; d += 2) {
        uint32_t r[4];
        ldsm_x4_t(r, vs + (kk * 16 + (lane & 15)) * kPitch + d * 8 + (lane & 16 ? 8 : 0));
        mma_bf16_16816(acc[d][0], acc[d][1], acc[d][2], acc[d][3], p[2 * kk][0], p[2 * kk][1], p[2 * kk + 1][0],
                       p[2 * kk + 1][1], r[0], r[1]);
        mma_bf16_16816(acc[d + 1][0], acc[d + 1][1], acc[d + 1][2], acc[d + 1][3], p[2 * kk][0], p[2 * kk][1],
                       p[2 * kk + 1][0], p[2 * kk + 1][1], r[2], r[3]);
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    if (!live[i]) continue;
    const float inv = sum[i] > 0.f ? 1.0f / sum[i] : 0.f;
    uint16_t* dst = out + (size_t)(a + tok[i]) * out_stride + (size_t)(h * G + row[i] % G) * kD + (lane & 3) * 2;
#pragma unroll
    for (int d = 0; d < 16; ++d)
      *reinterpret_cast<uint32_t*>(dst + d * 8) = pack_bf16x2(acc[d][2 * i] * inv, acc[d][2 * i + 1] * inv);
  }
}

}  // namespace

cudaError_t launch_prompt_attn(const PagedShape& s, const uint16_t* q, size_t q_stride, const uint16_t* k,
                               size_t k_stride, const uint16_t* v, size_t v_stride, const int* row_start, int n_rows,
                               float scale, uint16_t* out, size_t out_stride, unsigned* err, cudaStream_t stream) {
  if (n_rows == 0) return cudaSuccess;
  const int per = kTileRows / s.G();
  // tiles of all sequences: at most one partly filled tile for each
  const long long tiles = (long long)n_rows / per + (s.B < n_rows ? s.B : n_rows);
  dim3 grid((unsigned)tiles, (unsigned)s.Hkv);
  prompt_attn_kernel<<<grid, kWarps * 32, 0, stream>>>(s, q, q_stride, k, k_stride, v, v_stride, row_start, n_rows,
                                                       scale * 1.4426950408889634f, out, out_stride, err);
  return cudaGetLastError();
}

}  // namespace oasis
