// Decode attention over pages in 8 bits (oasis_paged_decode_attn_q8) and in 4 (oasis_paged_decode_attn_q4).
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
//
// Pages in 4 bits: the same mathematics without page scales (lk, lv = 0): a code times its group's scale has 6 significant
// bits and is a half exactly, so keys and values are scaled before the products and the weights need no exponent of a page.
// A lane's dimensions of a token are whole groups of 16, so it needs two scale bytes for a key and one for a value.  Pages
// pass through shared memory by asynchronous copies, two at a time while the next two are on their way: half the bytes
// of a page in 8 bits want twice as many in flight, more than registers hold (two pages ahead in registers: 123 against 103 us).
// Bound: HBM, 2,304 B for a page and head.  32 requests of 1 to 32K tokens, 32/8 heads (471 MB): 88 us, 5.4 TB/s,
// 0.80 of the measured copy rate; the same copies without any arithmetic 86.  4 us pass before the first pages are there, and
// of an SM's two blocks the one that started first is done at 66, the other at 79 (without arithmetic 65 and 68).  One
// request of 128K tokens, 64/8 heads (151 MB): 38 us.  128 pages for each of 256 pairs (76 MB): 22 us.  A pair costs a
// warp 3 us beside its pages, which a gap in the equal ranges stands for: 17 pairs of one or two pages at one warp made the
// whole call 103 us without gaps, 91 with gaps of 2 pages, 88 with 5.  287 instructions for a page and head (64 conversions, 64
// multiplications by scales, 16 for the exchange of codes between value rows, 16 MMAs): leaving out the conversions or the
// multiplications changes no time.  Measured and not kept (against 91): one page at a time 94, keys and values copied each as soon
// as their places are free 92, scores of the next pages beside the products of these 101, copies that zero instead of branches 93,
// 9 warps to a block 100 (spills), 16 warps to one block 96 (103 where they meet every 8 to 32 pages), 52 to 57% of the
// pages for the first half of the blocks 90 to 96 (in a chain of calls a half is not what an SM got first).
#include <type_traits>

#include "paged.cuh"

namespace oasis {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
constexpr int kMinPages = 8;  // pages a thread block gets at least, when there are so few
constexpr int kPairGap = 5;   // 4 bits: what a pair costs a warp beside its pages, in pages
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
  const void* scales;  // 8 bits: float, 4 bits: bytes
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

// Pages in 4 bits pass through a ring of kStages places in shared memory for each warp: codes of keys, of values, scales.
// A place's value rows are kept in lines of two tokens whose 16-byte pieces are exchanged (xor 2 (line & 3)), so that
// the lanes' 8-byte reads of four lines at a time meet in no bank.
constexpr int kStages = 4;
constexpr int kStageBytes = (int)(kHeadPageBytes4 + kHeadScaleBytes4);

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void lds(uint32_t at, uint32_t* w) {
  if constexpr (kBytes == 16)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
  else if constexpr (kBytes == 8)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
  else
    asm volatile("{\n .reg .u16 h;\n ld.shared.u16 h, [%1];\n cvt.u32.u16 %0, h;\n}" : "=r"(w[0]) : "r"(at));
}

__device__ __forceinline__ float exp2_fast(float x) {  // results below 2^-126 become zero
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// S^T += K Q^T of a page in 4 bits.  A lane has keys lane / 4 and + 8, dimensions 32 (lane % 4) .., two groups of each;
// a step of the product takes 4 of them (step m: 4m ..).
__device__ __forceinline__ void scores4(float* sc, uint32_t place, int lane, const uint32_t* qf) {
  uint32_t k0[4], k1[4], s0, s1;
  lds<16>(place + lane * 16, k0);
  lds<16>(place + lane * 16 + 8 * (kD / 2), k1);
  const uint32_t s = place + (uint32_t)kHeadPageBytes4 + lane * 2;
  lds<2>(s, &s0);
  lds<2>(s + 8 * kGroups, &s1);
#pragma unroll
  for (int half = 0; half < 2; ++half) {  // a group of 16 dimensions
    const uint32_t f0 = half ? scale_twice<1>(s0) : scale_twice<0>(s0);
    const uint32_t f1 = half ? scale_twice<1>(s1) : scale_twice<0>(s1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = k0[2 * half + i], hi = k1[2 * half + i];
      const int m = 4 * half + 2 * i;
      mma_f16_16816(sc, mul_f16x2(e2m1x2_to_f16x2<0>(lo), f0), mul_f16x2(e2m1x2_to_f16x2<0>(hi), f1),
                    mul_f16x2(e2m1x2_to_f16x2<1>(lo), f0), mul_f16x2(e2m1x2_to_f16x2<1>(hi), f1), qf[2 * m], qf[2 * m + 1]);
      mma_f16_16816(sc, mul_f16x2(e2m1x2_to_f16x2<2>(lo), f0), mul_f16x2(e2m1x2_to_f16x2<2>(hi), f1),
                    mul_f16x2(e2m1x2_to_f16x2<3>(lo), f0), mul_f16x2(e2m1x2_to_f16x2<3>(hi), f1), qf[2 * m + 2],
                    qf[2 * m + 3]);
    }
  }
}

// O^T += V^T W^T of a page in 4 bits.  A lane has tokens 2 (lane % 4), + 1, + 8, + 9, dimensions 16 (lane / 4) .., a group.
// Bytes of a token's row hold two dimensions, the product takes pairs of tokens, so the codes of two rows are exchanged
// (lo: the even dimensions of both, hi: the odd ones) before they become halves.  valid: tokens of the page; what lies
// behind them may be NaN, and zero times that is not zero: codes are finite, so it is their scales that become zero.
__device__ __forceinline__ void outputs4(float (*acc)[4], uint32_t place, int lane, int valid, uint32_t b0, uint32_t b1) {
  const int g = lane >> 2, c = lane & 3;
  const uint32_t line = place + kBS * (kD / 2) + c * kD + ((g * 8) ^ (c * 32));
  uint32_t t0[2], t1[2], t8[2], t9[2], s0, s1;
  lds<8>(line, t0);
  lds<8>(place + kBS * (kD / 2) + c * kD + ((kD / 2 + g * 8) ^ (c * 32)), t1);
  lds<8>(line + 4 * kD, t8);
  lds<8>(place + kBS * (kD / 2) + c * kD + ((kD / 2 + g * 8) ^ (c * 32)) + 4 * kD, t9);
  const uint32_t s = place + (uint32_t)kHeadPageBytes4 + kBS * kGroups + g * kBS + c * 2;
  lds<2>(s, &s0);
  lds<2>(s + 8, &s1);
  if (valid < kBS) {
    const int t = c * 2;
    s0 &= t >= valid ? 0u : t + 1 >= valid ? 0xffu : 0xffffu;
    s1 &= t + 8 >= valid ? 0u : t + 9 >= valid ? 0xffu : 0xffffu;
  }
  const uint32_t f0 = scale_pair(s0), f1 = scale_pair(s1);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo0 = (t0[i] & 0x0f0f0f0fu) | (t1[i] << 4 & 0xf0f0f0f0u);
    const uint32_t hi0 = (t0[i] >> 4 & 0x0f0f0f0fu) | (t1[i] & 0xf0f0f0f0u);
    const uint32_t lo1 = (t8[i] & 0x0f0f0f0fu) | (t9[i] << 4 & 0xf0f0f0f0u);
    const uint32_t hi1 = (t8[i] >> 4 & 0x0f0f0f0fu) | (t9[i] & 0xf0f0f0f0u);
    mma_f16_16816(acc[4 * i], mul_f16x2(e2m1x2_to_f16x2<0>(lo0), f0), mul_f16x2(e2m1x2_to_f16x2<0>(hi0), f0),
                  mul_f16x2(e2m1x2_to_f16x2<0>(lo1), f1), mul_f16x2(e2m1x2_to_f16x2<0>(hi1), f1), b0, b1);
    mma_f16_16816(acc[4 * i + 1], mul_f16x2(e2m1x2_to_f16x2<1>(lo0), f0), mul_f16x2(e2m1x2_to_f16x2<1>(hi0), f0),
                  mul_f16x2(e2m1x2_to_f16x2<1>(lo1), f1), mul_f16x2(e2m1x2_to_f16x2<1>(hi1), f1), b0, b1);
    mma_f16_16816(acc[4 * i + 2], mul_f16x2(e2m1x2_to_f16x2<2>(lo0), f0), mul_f16x2(e2m1x2_to_f16x2<2>(hi0), f0),
                  mul_f16x2(e2m1x2_to_f16x2<2>(lo1), f1), mul_f16x2(e2m1x2_to_f16x2<2>(hi1), f1), b0, b1);
    mma_f16_16816(acc[4 * i + 3], mul_f16x2(e2m1x2_to_f16x2<3>(lo0), f0), mul_f16x2(e2m1x2_to_f16x2<3>(hi0), f0),
                  mul_f16x2(e2m1x2_to_f16x2<3>(lo1), f1), mul_f16x2(e2m1x2_to_f16x2<3>(hi1), f1), b0, b1);
  }
}

// Scores of tokens behind a page's last one.
__device__ __forceinline__ void mask4(float* sc, int valid, int lane) {
  const int g = lane >> 2;
  if (g >= valid) sc[0] = sc[1] = neg_inf();
  if (g + 8 >= valid) sc[2] = sc[3] = neg_inf();
}

// Two pages in 4 bits into the running state (two chains of products, one look at the maxima).  v0, v1: their tokens, 0
// where there is no page: what its place holds then weighs nothing.  top: M, kLowest before the first page (scores
// of -inf alone leave it there).
__device__ __forceinline__ void attend4(uint32_t place, int v0, int v1, const uint32_t* qf, const float* f, int lane, State& st,
                                        float* top) {
  float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
  scores4(a, place, lane, qf);
  scores4(b, place + kStageBytes, lane, qf);
  if (v0 + v1 < 2 * kBS) {
    mask4(a, v0, lane);
    mask4(b, v1, lane);
  }
  float m0 = fmaxf(fmaxf(a[0], a[2]), fmaxf(b[0], b[2])) * f[0], m1 = fmaxf(fmaxf(a[1], a[3]), fmaxf(b[1], b[3])) * f[1];
  if (__any_sync(0xffffffffu, m0 > top[0] + kMostBits || m1 > top[1] + kMostBits)) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
      m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
    }
    const float n0 = fmaxf(top[0], m0 - kLift), n1 = fmaxf(top[1], m1 - kLift);
    const float c0 = exp2_fast(top[0] - n0), c1 = exp2_fast(top[1] - n1);  // 0 for the first page
    top[0] = n0;
    top[1] = n1;
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
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = exp2_fast(fmaf(a[i], f[i & 1], -top[i & 1]));
    b[i] = exp2_fast(fmaf(b[i], f[i & 1], -top[i & 1]));
  }
  st.sum[0] += (a[0] + a[2]) + (b[0] + b[2]);
  st.sum[1] += (a[1] + a[3]) + (b[1] + b[3]);
  outputs4(st.acc, place, lane, v0, transpose_8x8(pack_f16x2(a[0], a[1])), transpose_8x8(pack_f16x2(a[2], a[3])));
  outputs4(st.acc, place + kStageBytes, lane, v1, transpose_8x8(pack_f16x2(b[0], b[1])), transpose_8x8(pack_f16x2(b[2], b[3])));
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

// kClustered: a cluster of `team` blocks for each pair, else all pages in equal ranges.  kBits: 8 or 4.
template <bool kClustered, int kBits>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
paged_decode_attn_kernel(PagedShape s, Args a) {
  // 8 bits: rows of slots [2 * kWarps][G][kD], then (kClustered) of the block's piece [G][kRowFloats].
  // 4 bits: rows of every second slot [kWarps][G][kD], then each warp's ring; the other slot of a warp is written when its
  // ring is done with and takes its beginning, the block's piece the end of the first one.
  extern __shared__ __align__(16) float slot_rows[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = s.Hq / s.Hkv;
  auto ring_of = [&](int w) { return reinterpret_cast<uint8_t*>(slot_rows + (size_t)kWarps * G * kD) + w * kStages * kStageBytes; };
  auto slot_at = [&](int slot) {
    if constexpr (kBits == 8) return slot_rows + (size_t)slot * G * kD;
    return slot & 1 ? reinterpret_cast<float*>(ring_of(slot >> 1)) : slot_rows + (size_t)(slot >> 1) * G * kD;
  };
  wait_for_predecessor();
  const int pairs = s.B * s.Hkv;
  const int per = (pairs + kThreads - 1) / kThreads;
  const int team = a.team, rank = blockIdx.x % team;  // kClustered: blocks to a pair, this one's place
  unsigned bits = 0;
  int blocks = 1;
  // Before each pair's pages lies a gap: a warp with many short pairs spends its time on their tables and first pages.
  constexpr int kGap = kBits == 4 && !kClustered ? kPairGap : 0;
  long long total = 0, c_lo, c_hi;  // pages (and gaps) of all pairs (of this one), this block's range

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
      n += c > 0 ? c + kGap : 0;
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
      if (per > 1) return pair_pages(s, a, pair, &bits);
      const int n = (int)(sh.chunk_start[pair + 1] - sh.chunk_start[pair]);
      return kGap ? max(n - kGap, 0) : n;
    };
    auto span = [&](int pages) { return kGap && pages > 0 ? pages + kGap : pages; };
    int count = pages_of(e);
    while (e_lo + span(count) <= w_lo) {
      e_lo += span(count);
      count = pages_of(++e);
    }
    while (true) {
      const long long p_lo = e_lo + kGap;  // the pair's first page
      const int first = (int)max(w_lo - p_lo, 0ll), last = (int)min((long long)count, w_hi - p_lo);  // pages of the pair
      if (kGap == 0 || first < last) {
        const int b = e / s.Hkv, h = e - b * s.Hkv;
        const int ctx = (int)min((long long)max(a.ctx_len[b], 0), (long long)s.nb_max * kBS);
        const int nb = (ctx + kBS - 1) / kBS;

        int my_page = -1, my_valid = 0;  // of page (group of 32) + lane
        float2 my_scale = make_float2(1.f, 1.f);
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
                if constexpr (kBits == 8)
                  my_scale = *reinterpret_cast<const float2*>(static_cast<const float*>(a.scales) + ((long long)pg * s.Hkv + h) * 2);
              } else {
                bits |= OASIS_EW_BAD_SLOT;
              }
            }
          }
        };
        // ---- the query row lane / 4, dimensions as for the keys
        uint32_t qf[16];
        float fac[2];
        auto load_query = [&](uint4 (&w)[4]) {
#pragma unroll
          for (int m = 0; m < 4; ++m) w[m] = make_uint4(0u, 0u, 0u, 0u);
          if ((lane >> 2) < G) {
            constexpr int kPiece = kBits == 8 ? 16 : 32, kNext = kBits == 8 ? 64 : 16;
            const uint16_t* src = a.q + (size_t)b * a.q_stride + (size_t)(h * G + (lane >> 2)) * kD + (lane & 3) * kPiece;
            w[0] = load16(src);
            w[1] = load16(src + 8);
            w[2] = load16(src + kNext);
            w[3] = load16(src + kNext + 8);
          }
        };
        auto convert_query = [&](const uint4 (&w)[4]) {
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
        };

        State st;
        uint4 query[4];
        load_query(query);
        if constexpr (kBits == 8) {
          convert_query(query);
          st.clear();
          Rows kr, vr;
          const long long head_stride = kHeadPageBytes;
          auto head_page = [&](int page) { return a.pages + ((long long)page * s.Hkv + h) * head_stride; };
          lookup(first);
          int page = __shfl_sync(0xffffffffu, my_page, 0);
          if (page >= 0) {
            load_keys(kr, head_page(page), lane);
            load_values(vr, head_page(page), lane);
          }
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
        } else {
          // Two pages at a time, the next two on their way: half as many bytes each as in 8 bits.
          const uint8_t* const codes = a.pages + (long long)h * kHeadPageBytes4 + lane * 16;
          const uint8_t* const scales = static_cast<const uint8_t*>(a.scales) + (long long)h * kHeadScaleBytes4 + (lane & 15) * 16;
          const long long page_bytes = s.Hkv * kHeadPageBytes4, scale_bytes = s.Hkv * kHeadScaleBytes4;
          const uint32_t ring = (uint32_t)__cvta_generic_to_shared(ring_of(warp));
          const uint32_t value_at = kBS * (kD / 2) + (lane >> 3) * kD + ((lane & 7) ^ (lane >> 3) << 1) * 16;
          // a page and its tokens in one word (page * 32 + tokens, 0: none): of page (group of 32) + lane.  The tables of the
          // group after that are on their way as well.
          uint32_t ahead = 0;
          lookup(first);
          auto fetch = [&](int at, uint32_t place) {  // pages at and at + 1: their tokens, 16 bits each
            uint32_t tokens = 0;
            if (at < last) {
              const int in = (at - first) & 31;
              if (in == 0) {
                ahead = my_page < 0 ? 0u : (uint32_t)my_page * 32 + (uint32_t)my_valid;
                lookup(at + 32);
              }
              const uint32_t w0 = __shfl_sync(0xffffffffu, ahead, in), w1 = __shfl_sync(0xffffffffu, ahead, in + 1);
              if (w0) {
                const uint8_t* from = codes + (long long)(w0 >> 5) * page_bytes;
                copy16(place + lane * 16, from);
                copy16(place + lane * 16 + 512, from + 512);
                copy16(place + value_at, from + 1024);
                copy16(place + value_at + 512, from + 1536);
              }
              if (w1) {
                const uint8_t* from = codes + (long long)(w1 >> 5) * page_bytes;
                copy16(place + kStageBytes + lane * 16, from);
                copy16(place + kStageBytes + lane * 16 + 512, from + 512);
                copy16(place + kStageBytes + value_at, from + 1024);
                copy16(place + kStageBytes + value_at + 512, from + 1536);
              }
              const uint32_t mine = lane < 16 ? w0 : w1;  // the first 16 lanes copy the first one's scales
              if (mine)
                copy16(place + (lane < 16 ? 0 : kStageBytes) + (uint32_t)kHeadPageBytes4 + (lane & 15) * 16,
                       scales + (long long)(mine >> 5) * scale_bytes);
              tokens = (w0 & 31) | (w1 & 31) << 16;
            }
            copy_commit();
            return tokens;
          };
          uint32_t seen = 0, tokens = fetch(first, ring), next = fetch(first + 2, ring + 2 * kStageBytes);
          convert_query(query);  // the tables and the first pages are on their way
          st.clear();
          // a score's factor stays normal, so that it leaves an infinity one
          const float f[2] = {fmaxf(fac[0], 1.1754944e-38f), fmaxf(fac[1], 1.1754944e-38f)};
          float top[2] = {kLowest, kLowest};
          uint32_t place = ring;
          for (int at = first; at < last; at += 2) {
            copy_wait<1>();
            __syncwarp();  // the pages have landed for all lanes
            seen |= tokens;
            attend4(place, tokens & 31, tokens >> 16, qf, f, lane, st, top);
            __syncwarp();  // all lanes are done with them
            tokens = next;
            next = fetch(at + 4, place);
            place = place == ring ? ring + 2 * kStageBytes : ring;
          }
          copy_wait<0>();
          if (seen) {
            st.top[0] = top[0];
            st.top[1] = top[1];
          }
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
            float* row = slot_at(slot) + (size_t)r * kD + (lane >> 2) * 16;
#pragma unroll
            for (int m = 0; m < 8; m += 2)
              *reinterpret_cast<float4*>(row + 2 * m) =
                  make_float4(st.acc[m][i], st.acc[m][2 + i], st.acc[m + 1][i], st.acc[m + 1][2 + i]);
            if (lane < 4) sh.top_sum[slot][r] = make_float2(st.top[i], st.sum[i]);
          }
        }
        if (!whole && lane == 0) {
          sh.slot_pair[slot] = e;
          sh.slot_lo[slot] = p_lo;
          sh.slot_hi[slot] = p_lo + count;
        }
      }
      if (p_lo + count >= w_hi) break;
      do {
        e_lo += span(count);
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
  // kClustered: this block's rows
  float* piece = kBits == 8 ? slot_rows + (size_t)2 * kWarps * G * kD
                            : reinterpret_cast<float*>(ring_of(0)) + (size_t)kMaxG * kD;
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
      const float4 v = reinterpret_cast<const float4*>(slot_at(j) + (size_t)r * kD)[lane];
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

// The same for pages in 4 bits, with no more thread blocks than there can be pairs that go on in a later block.  kSpread: a
// block for each of a pair's rows, its pieces spread over the warps (few pairs in many pieces); else one for the
// pair, a row to a warp (many pairs in two pieces).
constexpr int kJoinWarps4 = 8, kJoinThreads4 = kJoinWarps4 * 32;
template <bool kSpread>
__global__ void __launch_bounds__(kJoinThreads4)
paged_decode_join4_kernel(PagedShape s, const float* parts, const int2* tails, int blocks, uint16_t* out) {
  __shared__ float rows[kJoinWarps4][kRowFloats];
  __shared__ int warp_tails[kJoinWarps4], found[3];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = s.Hq / s.Hkv;
  const int wanted = kSpread ? blockIdx.x / G : blockIdx.x;
  wait_for_predecessor();  // the pieces are written
  if (tid == 0) found[0] = -1;
  int before = 0;  // tails of the blocks looked at
  for (int b0 = 0; b0 < blocks; b0 += kJoinThreads4) {
    const int b = b0 + tid;
    const int2 t = b < blocks ? tails[b] : make_int2(-1, 0);
    const unsigned has = __ballot_sync(0xffffffffu, t.x >= 0);
    if (lane == 0) warp_tails[warp] = __popc(has);
    __syncthreads();
    int rank = before + __popc(has & ((1u << lane) - 1));
#pragma unroll
    for (int w = 0; w < kJoinWarps4; ++w) {
      rank += w < warp ? warp_tails[w] : 0;
      before += warp_tails[w];
    }
    if (t.x >= 0 && rank == wanted) {
      found[0] = t.x;
      found[1] = b;
      found[2] = t.y;
    }
    __syncthreads();
  }
  if (found[0] < 0) return;
  const int first = found[1], n = found[2] - first + 1;
  const int r = kSpread ? blockIdx.x % G : warp, c_first = kSpread ? warp : 0;
  constexpr int kStep = kSpread ? kJoinWarps4 : 1, kAtOnce = 5;
  float top = neg_inf(), sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  if (r < G) {
    for (int c0 = c_first; c0 < n; c0 += kStep * kAtOnce) {
      float4 x[kAtOnce];
      float2 ml[kAtOnce];
#pragma unroll
      for (int d = 0; d < kAtOnce; ++d) {
        const int c = min(c0 + d * kStep, n - 1);
        const float* row = parts + ((((long long)first + c) * 2 + (c == 0 ? 1 : 0)) * G + r) * kRowFloats;
        ml[d] = *reinterpret_cast<const float2*>(row + kD);
        const float2 u = *reinterpret_cast<const float2*>(row + lane * 4), v = *reinterpret_cast<const float2*>(row + lane * 4 + 2);
        x[d] = make_float4(u.x, u.y, v.x, v.y);
      }
#pragma unroll
      for (int d = 0; d < kAtOnce; ++d) {
        if (c0 + d * kStep >= n) continue;
        const float next = fmaxf(top, ml[d].x);
        const float f0 = top == neg_inf() ? 0.f : exp2f(top - next), f1 = ml[d].x == neg_inf() ? 0.f : exp2f(ml[d].x - next);
        o[0] = fmaf(o[0], f0, x[d].x * f1);
        o[1] = fmaf(o[1], f0, x[d].y * f1);
        o[2] = fmaf(o[2], f0, x[d].z * f1);
        o[3] = fmaf(o[3], f0, x[d].w * f1);
        sum = fmaf(sum, f0, ml[d].y * f1);
        top = next;
      }
    }
  }
  uint16_t* const dst = out + ((long long)found[0] * G + r) * kD;
  if constexpr (!kSpread) {
    if (r >= G) return;
    const float inv = inverse(top, sum);
    reinterpret_cast<uint2*>(dst)[lane] = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) rows[warp][lane * 4 + i] = o[i];
    if (lane == 0) {
      rows[warp][kD] = top;
      rows[warp][kD + 1] = sum;
    }
    __syncthreads();
    if (tid >= kD / 2) return;
    float m = neg_inf();
#pragma unroll
    for (int w = 0; w < kJoinWarps4; ++w) m = fmaxf(m, rows[w][kD]);
    float l = 0.f, o0 = 0.f, o1 = 0.f;
    if (m != neg_inf()) {
#pragma unroll
      for (int w = 0; w < kJoinWarps4; ++w) {
        const float f = exp2f(rows[w][kD] - m);
        l = fmaf(f, rows[w][kD + 1], l);
        o0 = fmaf(f, rows[w][2 * tid], o0);
        o1 = fmaf(f, rows[w][2 * tid + 1], o1);
      }
    }
    const float inv = inverse(m, l);
    *reinterpret_cast<uint32_t*>(dst + 2 * tid) = pack_bf16x2(o0 * inv, o1 * inv);
  }
}

int most_blocks() { return kCtasPerSm * sm_count(); }

}  // namespace

size_t paged_attn_workspace_bytes(const PagedShape& s) {
  const size_t n = (size_t)most_blocks();
  return n * 2 * s.G() * kRowFloats * sizeof(float) + n * sizeof(int2);
}

namespace {

template <int kBits>
cudaError_t launch_decode(const PagedShape& s, const uint16_t* q, size_t q_stride, const uint8_t* pages, const void* scales,
                          const int* table, const int* ctx, const int* sel, const int* nsel, int sel_max, float scale,
                          void* ws, uint16_t* out, unsigned* err, cudaStream_t stream) {
  const int most = most_blocks();
  const long long pages_max = (long long)s.B * s.Hkv * (sel ? sel_max : s.nb_max);
  const long long blocks = (pages_max + kMinPages - 1) / kMinPages;
  const int grid = blocks < most ? (int)blocks : most;
  float* parts = static_cast<float*>(ws);
  Args a{q, q_stride, pages, scales, table, ctx, sel, nsel, sel_max, 1, scale * 1.4426950408889634f, parts,
         reinterpret_cast<int2*>(parts + (size_t)most * 2 * s.G() * kRowFloats), out, err};
  static_assert(kMaxG * (kD + kRowFloats) * sizeof(float) <= kStages * kStageBytes, "a slot and the piece fit in a ring");
  const size_t slots = (size_t)kWarps * s.G() * kD * sizeof(float);
  const size_t smem = kBits == 8 ? 2 * slots : slots + (size_t)kWarps * kStages * kStageBytes;
  const long long pairs = (long long)s.B * s.Hkv;
  const int pair_max = sel ? sel_max : s.nb_max;
  // A cluster for each pair needs no prefix over the pairs, no workspace and no second kernel, but leaves blocks
  // idle that other pairs could use: taken while a pair's most pages (by the width of the table or selection; the lengths are
  // not known here) keep its blocks busy for a few us.  32/8 heads, clusters against equal ranges: 1 x 700 tokens 6.7
  // against 8.2 us, 1 x 4,096 9.2 against 11.3, 1 x 8,192 (64 pages for each of 64 blocks) 14.0 against 13.6, 32 x
  // 1,000 16.7 against 19.7.  With more of the places filled the gain lasts longer: of 304, 208 pairs of 96 pages 21.3 against
  // 22.3 and of 128 26.4 against 25.9, 256 pairs of 128 27.8 against 30.3, of 192 38.6 against 40.3, of 256 49.1 against 50.0.
  while (a.team < 8 && pairs * a.team * 2 <= most && pair_max > kMinPages * a.team) a.team *= 2;
  // 4 bits: 8 pairs of 512 pages by teams of 8 11.1 against 11.5, of 1,024 15.7 against 13.4; 256 pairs of 128 22.0 against
  // 25.2, of 188 28.4 against 28.9, of 256 35.2 against 36.7.
  const bool filled = pairs * a.team * 3 >= most * 2LL;  // two thirds of the GPU's places, or fewer
  const int team_pages = kBits == 8 ? (filled ? 128 : 56) : filled ? 256 : 72;
  if (pairs * a.team <= most && pair_max <= team_pages * a.team) {
    const size_t with_piece = kBits == 8 ? smem + (size_t)s.G() * kRowFloats * sizeof(float) : smem;
    static int attr_cache[kMaxDevicesCached] = {};
    cudaError_t e = ensure_dyn_smem((const void*)paged_decode_attn_kernel<true, kBits>, with_piece, attr_cache);
    if (e != cudaSuccess) return e;
    return launch_chained(paged_decode_attn_kernel<true, kBits>, dim3((unsigned)(pairs * a.team)), dim3(kThreads), with_piece, stream,
                          a.team, s, a);
  }
  static int attr_cache[kMaxDevicesCached] = {};
  cudaError_t e = ensure_dyn_smem((const void*)paged_decode_attn_kernel<false, kBits>, smem, attr_cache);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(workspace_lock());  // the join reads what the kernel before it left in the workspace
  e = launch_chained(paged_decode_attn_kernel<false, kBits>, dim3(grid), dim3(kThreads), smem, stream, 1, s, a);
  if (e != cudaSuccess || grid == 1) return e;
  if constexpr (kBits == 4) {
    const int tails = pairs < grid ? (int)pairs : grid;
    const bool spread = tails * s.G() <= most;
    return launch_chained(spread ? paged_decode_join4_kernel<true> : paged_decode_join4_kernel<false>,
                          dim3(spread ? tails * s.G() : tails), dim3(kJoinThreads4), 0, stream, 1, s, parts, a.tails, grid, out);
  }
  return launch_chained(paged_decode_join_kernel, dim3(grid, s.G()), dim3(kJoinWarps * 32), 0, stream, 1, s, parts, a.tails,
                        out);
}

}  // namespace

cudaError_t launch_paged_decode_attn(const PagedShape& s, const uint16_t* q, size_t q_stride, const uint8_t* pages,
                                     const float* scales, const int* table, const int* ctx, const int* sel,
                                     const int* nsel, int sel_max, float scale, void* ws, uint16_t* out,
                                     unsigned* err, cudaStream_t stream) {
  return launch_decode<8>(s, q, q_stride, pages, scales, table, ctx, sel, nsel, sel_max, scale, ws, out, err, stream);
}

cudaError_t launch_paged_decode_attn_q4(const PagedShape& s, const uint16_t* q, size_t q_stride, const uint8_t* pages,
                                        const uint8_t* scales, const int* table, const int* ctx, const int* sel,
                                        const int* nsel, int sel_max, float scale, void* ws, uint16_t* out,
                                        unsigned* err, cudaStream_t stream) {
  return launch_decode<4>(s, q, q_stride, pages, scales, table, ctx, sel, nsel, sel_max, scale, ws, out, err, stream);
}

}  // namespace oasis
