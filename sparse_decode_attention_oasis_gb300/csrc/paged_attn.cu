// Decode attention over 8-bit pages (oasis_paged_decode_attn_q8).
//
// Mathematics: a softmax over tokens with a running reference M, one per query
// row: w_t = 2^(c s_t + lv_t - M), o = sum w_t v8_t / sum w_t 2^-lv_t, where
// s_t = q . k8_t * 2^lk_t, lk and lv the exponents of the page's key and value scale
// and c = scale * log2(e).  Taking lv into the exponent keeps the weights of pages
// with different scales inside one fp16 range.  M lies 11 below the score that set it and
// moves only when a score passes it by more than 15, so most pages need no rescaling of
// the accumulators and the largest weight is always 2^11 to 2^15 of fp16's 2^16.
//
// Work: one warp takes one page (16 tokens of one KV head) at a time, straight from
// global memory into mma.sync fragments, without shared memory:
//   S^T[16 tokens x 8 rows]  = K[16 x 128] Q^T       8 x m16n8k16, K the A operand
//   O^T[128 dims x 8 rows]  += V^T[128 x 16] W^T     8 x m16n8k16, V^T the A operand
// The query rows are the narrow side (n = 8 >= G), so nothing is padded to 16 rows.
// The order of dimensions inside a fragment is free as long as both operands share
// it: a lane's 16-byte loads are its fragments' dimensions, every load instruction
// covers whole 32-byte sectors, and V's pairs of tokens need one byte permute each.
// e4m3 converts to fp16 exactly; q is scaled by a power of two for each row so that
// its largest value lies in [2^14, 2^15), then converts to fp16 without rounding
// (bf16 has 8 significant bits, fp16 11; values 2^29 below the row's largest lose
// bits, 2^-40 of the score).  Roundings: w to fp16 for the product with V (2^-11 of its value at
// most; below 2^-25 of the largest weight of the warp's tokens, scales included, 2^-36 of that), the
// output to bf16 (2^-8, which dominates); s, w, the sums and the accumulators are fp32.
// The largest weight near 1 lost the others at 2^-25 of it: beside a leader of 20 nats
// with a zero value nothing was left of its warp's other tokens.  Lifts of 7, 11 and 13 bits cost the same time.
//
// Split: the pages of all (request, KV head) pairs form one sequence, cut into equal
// ranges for the thread blocks and again for their warps, whatever the lengths are.
// A warp writes a pair that lies wholly inside its range; pieces are joined in shared
// memory, and pieces of pairs that cross thread blocks by a second kernel from the
// workspace (two pieces at most for each block, so its size does not depend on the
// context).  Where a pair can have few pages only, a cluster of 1 to 8 blocks takes a pair and
// joins its pieces through distributed shared memory, in one launch.
//
// Bound: HBM, 4 KiB + 8 B for a page and head.  32 requests of 16K tokens, 32/8 heads (1.07
// GB): 170 us, 6.3 TB/s, 0.93 of the measured copy rate; ncu: DRAM bytes equal the
// algorithmic ones, 32% of the issue slots used.  The time is 9 to 12 us (launch, tables and
// first pages 4, the blocks' uneven ends 3, the two joins 4) and the bytes at the copy rate,
// so 128 pages for each of 256 pairs (134 MB) take 30 us; by clusters they take 28, and one
// request of 700 tokens 6.7 against 8.2.  Measured and not kept: pages in a ring of three in shared memory by bulk
// copies (186 against 174 us: the deeper queues end more unevenly), L2 prefetch 2 to 8
// pages ahead (177 to 197), queries loaded before the tables but converted after (205:
// the live registers cost the loop), 4 or 16 warps to a block (no change), one join
// block for all query rows of a pair (1 us more).
#include "paged.cuh"

namespace oasis {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
constexpr int kMinPages = 8;  // pages a thread block gets at least, when there are so few
constexpr int kJoinWarps = 4;
constexpr int kMaxG = 8;
constexpr int kRowFloats = kD + 2;
constexpr float kLift = 11.0f, kMostBits = 15.0f;  // log2 of the weight of the score that sets M, of the largest weight
// The least running reference of a row that has seen a token: a row without tokens keeps -inf and gets zeros, one
// whose scores are all NaN or -inf gets the softmax's NaN (its sum is NaN or 0), however its pages are split.
constexpr float kLowest = -3e38f;

struct Args {
  const uint16_t* q;
  size_t q_stride;
  const uint8_t* pages;
  const float* scales;
  const int* table;
  const int* ctx_len;
  const int* sel;
  const int* nsel;
  int sel_max;
  int team;  // blocks of a cluster
  float scale_log2;
  float* parts;  // [grid][2][G][kRowFloats]
  int2* tails;   // [grid]: the pair whose first piece is a block's tail (-1: none), its last block
  uint16_t* out;
  unsigned* err;
};

__device__ __forceinline__ void mma_f16_16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Pages of pair e = b * Hkv + h.
__device__ __forceinline__ int pair_pages(const PagedShape& s, const Args& a, int e, unsigned* bits) {
  if (a.sel == nullptr) return (int)min(((long long)max(a.ctx_len[e / s.Hkv], 0) + kBS - 1) / kBS, (long long)s.nb_max);
  const int n = a.nsel[e];
  if (n < 0 || n > a.sel_max) {
    *bits |= OASIS_EW_BAD_COUNT;
    return n < 0 ? 0 : a.sel_max;
  }
  return n;
}

// The running state of one warp: rows r0 = 2 (lane % 4) and r0 + 1, dimensions
// 16 (lane / 4) .. + 15 (acc[m][0], [2] and [1], [3]: dimensions 2m, 2m + 1 of the rows).
struct State {
  float acc[8][4];
  float top[2];  // M
  float sum[2];  // this lane's tokens only
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
    top[0] = top[1] = neg_inf();
    sum[0] = sum[1] = 0.f;
  }
};

// What a row's accumulators are multiplied with at the end: 0 where it has no token.
__device__ __forceinline__ float inverse(float top, float sum) { return top == neg_inf() ? 0.f : 1.0f / sum; }

struct Rows {  // a lane's 16-byte pieces of a page's keys and values
  uint4 v[4];
};

// Keys: rows lane / 4 and + 8, dimensions 16 (lane % 4) .. and 64 + 16 (lane % 4) ..
__device__ __forceinline__ void load_keys(Rows& k, const uint8_t* page, int lane) {
  const uint8_t* p = page + (lane >> 2) * kD + (lane & 3) * 16;
  k.v[0] = load16_stream(p);
  k.v[1] = load16_stream(p + 64);
  k.v[2] = load16_stream(p + 8 * kD);
  k.v[3] = load16_stream(p + 8 * kD + 64);
}

// Values: tokens 2 (lane % 4), + 1, + 8, + 9, dimensions 16 (lane / 4) ..
__device__ __forceinline__ void load_values(Rows& v, const uint8_t* page, int lane) {
  const uint8_t* p = page + kBS * kD + (lane & 3) * 2 * kD + (lane >> 2) * 16;
  v.v[0] = load16_stream(p);
  v.v[1] = load16_stream(p + kD);
  v.v[2] = load16_stream(p + 8 * kD);
  v.v[3] = load16_stream(p + 9 * kD);
}

struct Shared {
  float2 top_sum[2 * kWarps][kMaxG];  // of a piece's rows
  long long chunk_start[kThreads + 1];
  long long warp_sums[kWarps];
  long long slot_lo[2 * kWarps], slot_hi[2 * kWarps];
  int slot_pair[2 * kWarps];
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float2 load_remote(const float* mine, unsigned rank) {  // the same place in block `rank`'s shared memory
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}

// kClustered: a cluster of `team` blocks for each pair, else all pages in equal ranges.
template <bool kClustered>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
paged_decode_attn_kernel(PagedShape s, Args a) {
  extern __shared__ __align__(16) float slot_rows[];  // [2 * kWarps][G][kD], then (kClustered) [G][kRowFloats]
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = s.Hq / s.Hkv;
  wait_for_predecessor();
  const int pairs = s.B * s.Hkv;
  const int per = (pairs + kThreads - 1) / kThreads;
  const int team = a.team, rank = blockIdx.x % team;  // kClustered: blocks to a pair, this one's place
  unsigned bits = 0;
  int blocks = 1;
  long long total = 0, c_lo, c_hi;  // pages of all pairs (of this one), this block's range

  if constexpr (kClustered) {
    const int e = blockIdx.x / team;
    total = pair_pages(s, a, e, &bits);
    if (total == 0) {
      set_err(a.err, bits);
      if (rank == 0)
        for (int i = tid; i < G * kD / 8; i += kThreads)
          reinterpret_cast<uint4*>(a.out + (long long)e * G * kD)[i] = make_uint4(0u, 0u, 0u, 0u);
      return;  // the whole cluster
    }
    c_lo = rank * total / team;
    c_hi = (rank + 1) * total / team;
    if (lane < 2) sh.slot_pair[warp * 2 + lane] = -1;
    __syncwarp();
  } else {
    // prefix of the pairs' pages; pairs without pages get their zero rows here
    long long n = 0;
    for (int e = min(tid * per, pairs); e < min((tid + 1) * per, pairs); ++e) {
      const int c = pair_pages(s, a, e, &bits);
      n += c;
      if (c == 0 && e % (int)gridDim.x == (int)blockIdx.x)
        for (int i = 0; i < G * kD / 8; ++i)
          reinterpret_cast<uint4*>(a.out + (long long)e * G * kD)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    long long x = n;
  #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh.warp_sums[warp] = x;
    if (lane < 2) sh.slot_pair[warp * 2 + lane] = -1;
    __syncthreads();
    long long off = 0;
  #pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      off += w < warp ? sh.warp_sums[w] : 0;
      total += sh.warp_sums[w];
    }
    sh.chunk_start[tid] = off + x - n;
    if (tid == 0) sh.chunk_start[kThreads] = total;
    __syncthreads();
    const long long wanted = (total + kMinPages - 1) / kMinPages;
    blocks = wanted < (long long)gridDim.x ? (int)wanted : (int)gridDim.x;
    if ((int)blockIdx.x >= blocks) {
      if (tid == 0) a.tails[blockIdx.x] = make_int2(-1, 0);
      if (blockIdx.x == 0) set_err(a.err, bits);
      return;
    }
    c_lo = blockIdx.x * total / blocks;
    c_hi = (blockIdx.x + 1) * total / blocks;
  }
  const long long w_lo = c_lo + warp * (c_hi - c_lo) / kWarps, w_hi = c_lo + (warp + 1) * (c_hi - c_lo) / kWarps;

  if (w_lo < w_hi) {
    // the pair that holds page w_lo: the last chunk of pairs that starts at or before it, then a walk
    int i = 0, j = kClustered ? 0 : kThreads - 1;
    while (i < j) {
      const int m = (i + j + 1) >> 1;
      if (sh.chunk_start[m] <= w_lo) i = m; else j = m - 1;
    }
    int e = kClustered ? blockIdx.x / team : i * per;
    long long e_lo = kClustered ? 0 : sh.chunk_start[i];
    // with one pair to a chunk the prefix holds its pages
    auto pages_of = [&](int pair) {
      if (kClustered) return (int)total;
      return per == 1 ? (int)(sh.chunk_start[pair + 1] - sh.chunk_start[pair]) : pair_pages(s, a, pair, &bits);
    };
    int count = pages_of(e);
    while (e_lo + count <= w_lo) {
      e_lo += count;
      count = pages_of(++e);
    }
    long long p = w_lo;
    while (true) {
      const int b = e / s.Hkv, h = e - b * s.Hkv;
      const int ctx = (int)min((long long)max(a.ctx_len[b], 0), (long long)s.nb_max * kBS);
      const int nb = (ctx + kBS - 1) / kBS;
      const int first = (int)(p - e_lo), last = (int)min((long long)count, w_hi - e_lo);  // pages of the pair

      // ---- the query row lane / 4, dimensions as for the keys
      uint32_t qf[16];
      float fac[2];
      {
        uint4 w[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) w[m] = make_uint4(0u, 0u, 0u, 0u);
        if ((lane >> 2) < G) {
          const uint16_t* src = a.q + (size_t)b * a.q_stride + (size_t)(h * G + (lane >> 2)) * kD + (lane & 3) * 16;
          w[0] = load16(src);
          w[1] = load16(src + 8);
          w[2] = load16(src + 64);
          w[3] = load16(src + 72);
        }
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const uint32_t v = word(w[c], d) & 0x7fff7fffu;
            m = max(m, max(v & 0xffffu, v >> 16));
          }
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int ex = max((int)(m >> 7) - 127, -112);  // exponent of the row's largest value
        const float f = pow2f(14 - ex);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint32_t v = word(w[c >> 2], c & 3);
          qf[c] = pack_f16x2(bf_lo(v) * f, bf_hi(v) * f);
        }
        const float mine = a.scale_log2 * pow2f(ex - 14);
        fac[0] = __shfl_sync(0xffffffffu, mine, (lane & 3) * 8);
        fac[1] = __shfl_sync(0xffffffffu, mine, (lane & 3) * 8 + 4);
      }

      Rows kr, vr;
      int my_page = -1, my_valid = 0;  // of page (group of 32) + lane
      float2 my_scale = make_float2(1.f, 1.f);
      const long long head_stride = kHeadPageBytes;
      auto lookup = [&](int at) {  // tables of pages at .. at + 31
        my_page = -1;
        my_valid = 0;
        const int idx = at + lane;
        if (idx < last) {
          int blk = idx;
          if (a.sel != nullptr) {
            blk = a.sel[(long long)e * a.sel_max + idx];
            if (blk < 0 || blk >= nb) {
              blk = -1;
              bits |= OASIS_EW_BAD_BLOCK;
            }
          }
          if (blk >= 0) {
            const int pg = a.table[(long long)b * s.nb_max + blk];
            if (pg >= 0 && pg < s.n_pages) {
              my_page = pg;
              my_valid = min(kBS, ctx - blk * kBS);
              my_scale = *reinterpret_cast<const float2*>(a.scales + ((long long)pg * s.Hkv + h) * 2);
            } else {
              bits |= OASIS_EW_BAD_SLOT;
            }
          }
        }
      };
      auto head_page = [&](int page) { return a.pages + ((long long)page * s.Hkv + h) * head_stride; };

      lookup(first);
      int page = __shfl_sync(0xffffffffu, my_page, 0);
      if (page >= 0) {
        load_keys(kr, head_page(page), lane);
        load_values(vr, head_page(page), lane);
      }
      State st;
      st.clear();
      for (int at = first; at < last; ++at) {
        const int in = (at - first) & 31;
        const int valid = __shfl_sync(0xffffffffu, my_valid, in);
        const float ks = __shfl_sync(0xffffffffu, my_scale.x, in), vs = __shfl_sync(0xffffffffu, my_scale.y, in);
        const bool here = page >= 0;
        if (in == 31) lookup(at + 1);
        page = at + 1 < last ? __shfl_sync(0xffffffffu, my_page, (at + 1 - first) & 31) : -1;
        float sc[4] = {0.f, 0.f, 0.f, 0.f};
        if (here) {
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const uint32_t lo = word(kr.v[m >> 2], m & 3), hi = word(kr.v[2 + (m >> 2)], m & 3);
            mma_f16_16816(sc, e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(hi), e4m3x2_hi_to_f16x2(lo),
                          e4m3x2_hi_to_f16x2(hi), qf[2 * m], qf[2 * m + 1]);
          }
        }
        if (page >= 0) load_keys(kr, head_page(page), lane);
        if (here) {
          const int g = lane >> 2;
          const float lv = (float)((int)((__float_as_uint(vs) >> 23) & 0xff) - 127);
          const float f0 = fac[0] * ks, f1 = fac[1] * ks;
          float s0 = fmaf(sc[0], f0, lv), s1 = fmaf(sc[1], f1, lv);
          float s2 = fmaf(sc[2], f0, lv), s3 = fmaf(sc[3], f1, lv);
          if (valid < kBS) {
            if (g >= valid) s0 = s1 = neg_inf();
            if (g + 8 >= valid) s2 = s3 = neg_inf();
            // what lies behind the last token may be NaN: zero times it is not zero
            const int t = (lane & 3) * 2;
            if (t >= valid) vr.v[0] = make_uint4(0u, 0u, 0u, 0u);
            if (t + 1 >= valid) vr.v[1] = make_uint4(0u, 0u, 0u, 0u);
            if (t + 8 >= valid) vr.v[2] = make_uint4(0u, 0u, 0u, 0u);
            if (t + 9 >= valid) vr.v[3] = make_uint4(0u, 0u, 0u, 0u);
          }
          float m0 = fmaxf(fmaxf(s0, s2), kLowest), m1 = fmaxf(fmaxf(s1, s3), kLowest);
          if (__any_sync(0xffffffffu, m0 > st.top[0] + kMostBits || m1 > st.top[1] + kMostBits)) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
              m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
            }
            const float n0 = fmaxf(st.top[0], m0 - kLift), n1 = fmaxf(st.top[1], m1 - kLift);
            const float c0 = exp2f(st.top[0] - n0), c1 = exp2f(st.top[1] - n1);  // 0 for the first page
            st.top[0] = n0;
            st.top[1] = n1;
            st.sum[0] *= c0;
            st.sum[1] *= c1;
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              st.acc[m][0] *= c0;
              st.acc[m][1] *= c1;
              st.acc[m][2] *= c0;
              st.acc[m][3] *= c1;
            }
          }
          const float w0 = exp2f(s0 - st.top[0]), w1 = exp2f(s1 - st.top[1]);
          const float w2 = exp2f(s2 - st.top[0]), w3 = exp2f(s3 - st.top[1]);
          const float iv = pow2f(-(int)lv);
          st.sum[0] = fmaf(w0 + w2, iv, st.sum[0]);
          st.sum[1] = fmaf(w1 + w3, iv, st.sum[1]);
          const uint32_t b0 = transpose_8x8(pack_f16x2(w0, w1)), b1 = transpose_8x8(pack_f16x2(w2, w3));
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t t0 = word(vr.v[0], m), t1 = word(vr.v[1], m), t8 = word(vr.v[2], m), t9 = word(vr.v[3], m);
            const uint32_t p0 = __byte_perm(t0, t1, 0x5140), p1 = __byte_perm(t8, t9, 0x5140);
            const uint32_t p2 = __byte_perm(t0, t1, 0x7362), p3 = __byte_perm(t8, t9, 0x7362);
            mma_f16_16816(st.acc[2 * m], e4m3x2_to_f16x2(p0), e4m3x2_hi_to_f16x2(p0), e4m3x2_to_f16x2(p1),
                          e4m3x2_hi_to_f16x2(p1), b0, b1);
            mma_f16_16816(st.acc[2 * m + 1], e4m3x2_to_f16x2(p2), e4m3x2_hi_to_f16x2(p2), e4m3x2_to_f16x2(p3),
                          e4m3x2_hi_to_f16x2(p3), b0, b1);
          }
        }
        if (page >= 0) load_values(vr, head_page(page), lane);
      }

      // ---- the pair's piece: the output if it is all of it, else a slot
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        st.sum[0] += __shfl_xor_sync(0xffffffffu, st.sum[0], o);
        st.sum[1] += __shfl_xor_sync(0xffffffffu, st.sum[1], o);
      }
      const bool whole = first == 0 && last == count && !(kClustered && team > 1);
      const int which = first == 0 ? 1 : 0, slot = warp * 2 + which;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (lane & 3) * 2 + i;
        if (r >= G) continue;
        if (whole) {
          const float inv = inverse(st.top[i], st.sum[i]);
          uint32_t w[8];
#pragma unroll
          for (int m = 0; m < 8; ++m) w[m] = pack_bf16x2(st.acc[m][i] * inv, st.acc[m][2 + i] * inv);
          uint4* dst = reinterpret_cast<uint4*>(a.out + ((long long)e * G + r) * kD + (lane >> 2) * 16);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          float* row = slot_rows + ((size_t)slot * G + r) * kD + (lane >> 2) * 16;
#pragma unroll
          for (int m = 0; m < 8; m += 2)
            *reinterpret_cast<float4*>(row + 2 * m) =
                make_float4(st.acc[m][i], st.acc[m][2 + i], st.acc[m + 1][i], st.acc[m + 1][2 + i]);
          if (lane < 4) sh.top_sum[slot][r] = make_float2(st.top[i], st.sum[i]);
        }
      }
      if (!whole && lane == 0) {
        sh.slot_pair[slot] = e;
        sh.slot_lo[slot] = e_lo;
        sh.slot_hi[slot] = e_lo + count;
      }
      p = e_lo + last;
      if (p >= w_hi) break;
      do {
        e_lo += count;
        count = pages_of(++e);
      } while (count == 0);
    }
  }
  set_err(a.err, bits);
  __syncthreads();

  // ---- join the warps' pieces: a row of a pair to a warp, four dimensions to a lane
  const int my_pair = lane < 2 * kWarps ? sh.slot_pair[lane] : -1;
  const unsigned same = __match_any_sync(0xffffffffu, my_pair);
  const unsigned leads = __ballot_sync(0xffffffffu, my_pair >= 0 && __ffs(same) - 1 == lane);
  const int units = __popc(leads) * G;
  int2 tail = make_int2(-1, 0);
  if (!kClustered && leads) {  // only the last pair can go on in the next block
    const int lead = 31 - __clz(leads);
    const long long e_hi = sh.slot_hi[lead];
    // its last piece is in the last block whose range starts before e_hi
    if (sh.slot_lo[lead] >= c_lo && e_hi > c_hi)
      tail = make_int2(sh.slot_pair[lead], (int)((e_hi * blocks + total - 1) / total - 1));
  }
  if (!kClustered && tid == 0) a.tails[blockIdx.x] = tail;
  float* piece = slot_rows + (size_t)2 * kWarps * G * kD;  // kClustered: this block's rows
  for (int u = warp; u < units; u += kWarps) {
    const int lead = __fns(leads, 0, u / G + 1), r = u % G;
    const unsigned mask = __shfl_sync(0xffffffffu, same, lead);
    const float2 ts = mask >> lane & 1 ? sh.top_sum[lane][r] : make_float2(neg_inf(), 0.f);
    const float top = warp_max(ts.x);
    const float f = ts.x == neg_inf() ? 0.f : exp2f(ts.x - top);
    const float sum = warp_sum(f * ts.y);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (unsigned left = mask; left; left &= left - 1) {
      const int j = __ffs(left) - 1;
      const float fj = __shfl_sync(0xffffffffu, f, j);
      const float4 v = reinterpret_cast<const float4*>(slot_rows + ((size_t)j * G + r) * kD)[lane];
      o.x = fmaf(fj, v.x, o.x);
      o.y = fmaf(fj, v.y, o.y);
      o.z = fmaf(fj, v.z, o.z);
      o.w = fmaf(fj, v.w, o.w);
    }
    const int e = sh.slot_pair[lead];
    const bool starts = sh.slot_lo[lead] >= c_lo;
    if (starts && sh.slot_hi[lead] <= c_hi && !(kClustered && team > 1)) {
      const float inv = inverse(top, sum);
      reinterpret_cast<uint2*>(a.out + ((long long)e * G + r) * kD)[lane] =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    } else {
      float* row = kClustered ? piece + r * kRowFloats
                              : a.parts + (((long long)blockIdx.x * 2 + (starts ? 1 : 0)) * G + r) * kRowFloats;
      *reinterpret_cast<float2*>(row + lane * 4) = make_float2(o.x, o.y);
      *reinterpret_cast<float2*>(row + lane * 4 + 2) = make_float2(o.z, o.w);
      if (lane == 0) *reinterpret_cast<float2*>(row + kD) = make_float2(top, sum);
    }
  }
  if constexpr (kClustered) {
    if (team == 1) return;
    if (leads == 0)  // no page of the pair for this block
      for (int i = tid; i < G * kRowFloats; i += kThreads) piece[i] = i % kRowFloats == kD ? neg_inf() : 0.f;
    cluster_sync();
    // row r is joined by warp r / team of block r % team
    const int r = warp * team + rank;
    if (r < G) {
      const float* row = piece + r * kRowFloats;
      const float2 ts = lane < team ? load_remote(row + kD, lane) : make_float2(neg_inf(), 0.f);
      const float top = warp_max(ts.x);
      const float f = ts.x == neg_inf() ? 0.f : exp2f(ts.x - top);
      const float sum = warp_sum(f * ts.y);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int c = 0; c < team; ++c) {
        const float fc = __shfl_sync(0xffffffffu, f, c);
        const float2 u = load_remote(row + lane * 4, c), v = load_remote(row + lane * 4 + 2, c);
        o = make_float4(fmaf(fc, u.x, o.x), fmaf(fc, u.y, o.y), fmaf(fc, v.x, o.z), fmaf(fc, v.y, o.w));
      }
      const float inv = inverse(top, sum);
      reinterpret_cast<uint2*>(a.out + ((long long)(blockIdx.x / team) * G + r) * kD)[lane] =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    }
    cluster_sync();  // no block's shared memory goes while another reads it
  }
}

// Joins the pieces of a pair that starts in block blockIdx.x and ends in a later one, one query
// row to a thread block: its warps take every kWarps-th piece, a lane four dimensions.
__global__ void __launch_bounds__(kJoinWarps * 32)
paged_decode_join_kernel(PagedShape s, const float* parts, const int2* tails,
                         uint16_t* out) {
  __shared__ float rows[kJoinWarps][kRowFloats];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = s.Hq / s.Hkv, r = blockIdx.y, first = blockIdx.x;
  wait_for_predecessor();  // the pieces are written
  const int2 t = tails[first];
  if (t.x < 0) return;
  const int n = t.y - first + 1;
  float top = neg_inf(), sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int c = warp; c < n; c += kJoinWarps) {
    const float* row = parts + (((long long)first + c) * 2 + (c == 0 ? 1 : 0)) * G * kRowFloats + r * kRowFloats;
    const float2 ml = *reinterpret_cast<const float2*>(row + kD);
    const float2 a = *reinterpret_cast<const float2*>(row + lane * 4), b = *reinterpret_cast<const float2*>(row + lane * 4 + 2);
    const float next = fmaxf(top, ml.x);
    const float f0 = top == neg_inf() ? 0.f : exp2f(top - next), f1 = ml.x == neg_inf() ? 0.f : exp2f(ml.x - next);
    o[0] = fmaf(o[0], f0, a.x * f1);
    o[1] = fmaf(o[1], f0, a.y * f1);
    o[2] = fmaf(o[2], f0, b.x * f1);
    o[3] = fmaf(o[3], f0, b.y * f1);
    sum = fmaf(sum, f0, ml.y * f1);
    top = next;
  }
  for (int i = 0; i < 4; ++i) rows[warp][lane * 4 + i] = o[i];
  if (lane == 0) {
    rows[warp][kD] = top;
    rows[warp][kD + 1] = sum;
  }
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= kD / 2) return;
  float m = neg_inf();
  for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, rows[w][kD]);
  float l = 0.f, o0 = 0.f, o1 = 0.f;
  if (m != neg_inf()) {
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = exp2f(rows[w][kD] - m);
      l = fmaf(f, rows[w][kD + 1], l);
      o0 = fmaf(f, rows[w][2 * d], o0);
      o1 = fmaf(f, rows[w][2 * d + 1], o1);
    }
  }
  const float inv = inverse(m, l);
  *reinterpret_cast<uint32_t*>(out + ((long long)t.x * G + r) * kD + 2 * d) = pack_bf16x2(o0 * inv, o1 * inv);
}

int most_blocks() { return kCtasPerSm * sm_count(); }

}  // namespace

size_t paged_attn_workspace_bytes(const PagedShape& s) {
  const size_t n = (size_t)most_blocks();
  return n * 2 * s.G() * kRowFloats * sizeof(float) + n * sizeof(int2);
}

cudaError_t launch_paged_decode_attn(const PagedShape& s, const uint16_t* q, size_t q_stride, const uint8_t* pages,
                                     const float* scales, const int* table, const int* ctx, const int* sel,
                                     const int* nsel, int sel_max, float scale, void* ws, uint16_t* out,
                                     unsigned* err, cudaStream_t stream) {
  const int most = most_blocks();
  const long long pages_max = (long long)s.B * s.Hkv * (sel ? sel_max : s.nb_max);
  const long long blocks = (pages_max + kMinPages - 1) / kMinPages;
  const int grid = blocks < most ? (int)blocks : most;
  float* parts = static_cast<float*>(ws);
  Args a{q, q_stride, pages, scales, table, ctx, sel, nsel, sel_max, 1, scale * 1.4426950408889634f, parts,
         reinterpret_cast<int2*>(parts + (size_t)most * 2 * s.G() * kRowFloats), out, err};
  const size_t smem = (size_t)2 * kWarps * s.G() * kD * sizeof(float);
  const long long pairs = (long long)s.B * s.Hkv;
  const int pair_max = sel ? sel_max : s.nb_max;
  // A cluster for each pair needs no prefix over the pairs, no workspace and no second kernel, but leaves blocks
  // idle that other pairs could use: taken while a pair's most pages (by the width of the table or selection; the lengths are
  // not known here) keep its blocks busy for a few us.  32/8 heads, clusters against equal ranges: 1 x 700 tokens 6.7
  // against 8.2 us, 1 x 4,096 9.2 against 11.3, 1 x 8,192 (64 pages for each of 64 blocks) 14.0 against 13.6, 32 x
  // 1,000 16.7 against 19.7.  With more of the places filled the gain lasts longer: of 304, 208 pairs of 96 pages 21.3 against
  // 22.3 and of 128 26.4 against 25.9, 256 pairs of 128 27.8 against 30.3, of 192 38.6 against 40.3, of 256 49.1 against 50.0.
  while (a.team < 8 && pairs * a.team * 2 <= most && pair_max > kMinPages * a.team) a.team *= 2;
  const int team_pages = pairs * a.team * 3 >= most * 2LL ? 128 : 56;  // two thirds of the GPU's places filled, or fewer
  if (pairs * a.team <= most && pair_max <= team_pages * a.team) {
    const size_t with_piece = smem + (size_t)s.G() * kRowFloats * sizeof(float);
    static int attr_cache[kMaxDevicesCached] = {};
    cudaError_t e = ensure_dyn_smem((const void*)paged_decode_attn_kernel<true>, with_piece, attr_cache);
    if (e != cudaSuccess) return e;
    return launch_chained(paged_decode_attn_kernel<true>, dim3((unsigned)(pairs * a.team)), dim3(kThreads), with_piece, stream,
                          a.team, s, a);
  }
  static int attr_cache[kMaxDevicesCached] = {};
  cudaError_t e = ensure_dyn_smem((const void*)paged_decode_attn_kernel<false>, smem, attr_cache);
  if (e != cudaSuccess) return e;
  // the join reads what the kernel before it left in the workspace: of two threads that share a stream, none comes between
  static std::mutex both[kMaxDevicesCached];
  std::lock_guard<std::mutex> lock(both[current_device()]);
  e = launch_chained(paged_decode_attn_kernel<false>, dim3(grid), dim3(kThreads), smem, stream, 1, s, a);
  if (e != cudaSuccess || grid == 1) return e;
  return launch_chained(paged_decode_join_kernel, dim3(grid, s.G()), dim3(kJoinWarps * 32), 0, stream, 1, s, parts, a.tails,
                        out);
}

}  // namespace oasis
