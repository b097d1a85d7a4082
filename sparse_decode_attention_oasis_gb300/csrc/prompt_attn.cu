// Causal attention over packed prompts (oasis_prompt_attn): TMA -> shared memory ->
// tcgen05.mma -> TMEM, one persistent thread block per SM.
//
// Mathematics: one pass over the keys with a running reference M and sum of a
// softmax, w_j = 2^(c s_j - M), o = sum_j w_j v_j / sum_j w_j, c = scale * log2(e).  M lies
// 34 above the score that sets it and moves only when a score is more than 8 above that one, so the
// accumulators are rescaled a few times in a whole row, not at every tile; weights of at most 2^-26
// cost no precision in fp32 or bf16 and keep sums of large values finite.
//
// Rows: the G query heads of a KV head and consecutive tokens are packed into the
// rows of a tile (row = token * G + head), so that every K/V tile is read once for
// the whole group and a tile of short sequences is not mostly empty.
// Roundings: weights to bf16 for the product with V (2^-8 of each at most; the sums are of the
// unrounded fp32 weights), the output to bf16; scores, maxima, sums and accumulators
// are fp32.  fp16 weights would keep 3 bits more, but both operands of an MMA have one
// type, and bf16 values do not fit fp16's range.
//
// Roles (384 threads):
//   warps 0..3, 4..7  softmax of row tile 0 and 1: one row to a thread, its 128 scores read
//                     from TMEM, the weights written back to TMEM in bf16 over the scores,
//                     the output row at the end;
//   warps 8, 11       one lane each issues the MMAs of row tile 0 and 1: S_i = Q_i K_j^T, then O_i += P_i V_j
//                     with P_i from TMEM.  While one tile's softmax runs, the tensor cores work for the
//                     other.  The issuing lane's instructions are on the critical path: with one warp for
//                     both tiles and general loops a pair of tiles took 3,200 cycles, so it now is a warp for
//                     each tile, one lane from end to end, and loops without a condition to spare;
//   warp 9            TMA producer: Q tiles, and K and V tiles of 128 tokens in a ring of 5;
//   warp 10           scheduler: finds this block's work items and hands them to the others; and it looks over
//                     the V tiles with tokens that not all rows of an item attend.
// TMEM: two S/P and two O tiles of 128 columns, all 512.  Shared memory: 64 KB of Q and a ring
// of 160 KB.
//
// Zero times NaN is not zero: a masked weight does not keep an infinity or NaN of V out.  So V rows behind
// a sequence's last token (another sequence's, or padding) are zeroed in shared memory before the product, and
// infinities and NaN in rows after an item's first token as well; the output rows that do attend those get them
// back at the block's end, from global memory.  The look at a tile runs beside its scores' product and softmax and
// costs where an item has few tiles: one prompt of 128 tokens 8.1 -> 8.4 us, 16 of 512 52.2 -> 53.4, twelve
// packed 163.5 -> 164.8, one of 16,384 within its noise; what a warp of its own for the ragged tiles saves the producer
// outweighs it for 700 prompts of 20 tokens (108 -> 105).  By the softmax warps at their output it was 8 to 12% more.
//
// Bound: the tensor cores, 4 x 128 x 128 x 128 multiply-adds for a pair of tiles, 2,048 cycles; a
// pair takes 2,300 to 2,600, the chain S -> softmax (1,250 cycles) -> product of one tile being longer than
// twice the other's MMAs; and the power cap: in long calls the SM clock settles at 1.7 to 1.85 GHz.  One
// prompt of 16,384 tokens, 32/8 heads: 1.20 ms (1.83 PFLOP/s, 0.94 of the measured matrix product),
// 1.34 ms in calls that follow each other for seconds; ncu at 8,192 tokens: tensor pipe 78% of
// elapsed cycles, issue slots 45%.  Twelve packed prompts (11,430 tokens): 162 us in a graph, 177 as calls; an item pays
// some 4,000 cycles at its ends beside its tiles.  Measured and not kept: two softmax warps to 32 rows
// (2,300 against 1,500 us then: the issuing lane starves), output by warps of its own (1,250 against
// 1,200: fewer registers for the softmax), 200 or 216 registers for the softmax (3% more), scores
// and weights of a last tile cut to the chunks that hold keys, as branches (1,650) or as a second body
// (packed 210 against 175), only its products cut (within 2% either way), outputs transposed over four lanes
// (packed 181 against 175), the output through a ring place and a tensor store (16 prompts of 512 tokens 51
// against 53, the others the same, for 80 lines of accounting).
// Every wait is bounded: on expiry the block raises OASIS_EW_TIMEOUT, waits (bounded)
// for its own copies and MMAs, frees TMEM and returns.
#include "paged.cuh"
#include "tc.cuh"

namespace oasis {
namespace {

using namespace tc;

constexpr int kTile = 128;                   // rows of a query tile, tokens of a K/V tile
constexpr uint32_t kHalf = kTile * 128;      // bytes of 128 rows x 64 columns
constexpr uint32_t kTileBytes = 2 * kHalf;
constexpr int kRing = 5;
constexpr int kItems = 4;                    // items that the scheduler may be ahead
constexpr int kThreads = 384;
// 168 registers a thread at launch (64,512 in all): 8 warps of 208 and 4 of 88 use them up
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(12 * kLaunchRegs >= 8 * kSoftmaxRegs + 4 * kOtherRegs, "register split");
constexpr int kConsumers = 11;               // warps that read an item: softmax, MMA, producer
constexpr float kSlack = 8.0f;
// 2^26 weights of up to 2^(8 - 34) times the largest bf16 do not pass fp32's largest value.  At the other end products
// of values under 2^-92 leave fp32's normal range.
constexpr float kDrop = 34.0f;
// The least score that sets M: a first tile whose scores are all -inf leaves it there, below every finite score.
constexpr float kLowest = -3e38f;

struct Item {
  int row0;   // first row of the sequence, -1: no more items
  int len;    // its tokens
  int tok0;   // first token of query tile 0
  int h;      // KV head
};

struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[kRing], kv_empty[kRing];
  uint64_t s_full[2], p_full[2][2], o_full[2];  // p_full: the weights of a tile's first and second 64 tokens
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t raw_full[kRing];  // V tiles that the scheduler warp has to look over first
  uint64_t done[2];
  Item items[kItems];
  uint32_t tmem_base;
  int abort_flag;
  int token;  // 1: a row tile's products are being issued
  int cleaned;  // 1: infinities or NaN of V were taken out of a tile
};

constexpr size_t kSmemBytes = 1024 + 2 * (size_t)kTileBytes + kRing * (size_t)kTileBytes + sizeof(Bars);
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a thread block");

// Shared-memory operand descriptors, low word: address and leading offset, high word: the rest.
// Q, K: K-major 128-byte rows, 8-row groups 1,024 B apart.  V: rows are tokens (the contraction),
// 64 dimensions to a 128-byte row: 8-token groups 1,024 B apart, the second 64 dimensions kHalf apart.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t qk_desc_low(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t v_desc_low(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | ((kHalf >> 4) << 16); }

// One elected lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.b32 %0, 1, 0, P;\n}\n" : "=r"(ok));
  return ok != 0;
}

// D (+)= A B, operands given as the low words of their descriptors.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
      "r"(acc ? 1u : 0u), "n"(kDescHigh));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
      "r"(acc ? 1u : 0u), "n"(kDescHigh));
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ bool finite(uint32_t w) { return (w & 0x7f80u) != 0x7f80u && (w & 0x7f800000u) != 0x7f800000u; }
// Whether 16-byte pieces c0 .. c1 - 1 of both halves of a tile hold no infinity and no NaN: one warp.
__device__ __forceinline__ bool all_finite(uint32_t at, int c0, int c1, int lane) {
  uint32_t odd[4] = {0, 0, 0, 0};  // sums of products: not finite if a value is not (or at 2^64, which costs a second look)
  for (int c = c0 + lane; c - lane < c1; c += 2 * 32) {
    uint4 x[4];  // pieces c and c + 32 of both halves; behind the last one, that again
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = lds16(at + (u & 1) * kHalf + min(c + (u >> 1) * 32, c1 - 1) * 16);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      odd[2 * (u & 1)] = fma_bf16x2(x[u].x, x[u].y, odd[2 * (u & 1)]);
      odd[2 * (u & 1) + 1] = fma_bf16x2(x[u].z, x[u].w, odd[2 * (u & 1) + 1]);
    }
  }
  return __all_sync(0xffffffffu, finite(odd[0]) && finite(odd[1]) && finite(odd[2]) && finite(odd[3]));
}

// A pair of bf16 with infinities and NaN as zeros.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

// The first K/V tile of an item with tokens after the item's first one.
__device__ __forceinline__ int first_masked(const Item& it) { return (it.tok0 + 1) / kTile; }

// K/V tiles that query tile i of an item reads (0: the tile has no token).
__device__ __forceinline__ int kv_tiles(const Item& it, int i, int per) {
  const int t0 = it.tok0 + i * per;
  return t0 < it.len ? (min(it.len, t0 + per) + kTile - 1) / kTile : 0;
}

// Work items: two query tiles of one sequence and KV head.  Up to 320 sequences are kept in one
// warp's registers and the items are ordered by their place in the sequence, the last
// (the ones with the most keys) first, so that every block gets an equal share; more sequences are
// walked in their order, 32 at a time.
struct Schedule {
  static constexpr int kKept = 10;  // sequences to a lane
  const int* row_start;
  int B, n_rows, pair;              // pair: tokens of an item
  int lane;
  bool sorted;
  int kept;                         // registers of a lane in use
  int n[kKept];                     // items of sequence lane + 32 i
  int first[kKept], end[kKept];     // its rows
  int most;                         // the most items of a sequence
  int window;                       // unsorted: first sequence of the window, items before it
  int before;
  unsigned bits;

  __device__ int items_of(int b, bool flag) {
    const int a = row_start[b], z = row_start[b + 1];
    if (a < 0 || z < a || z > n_rows) {
      if (flag) bits |= OASIS_EW_BAD_COUNT;
      return 0;
    }
    return (z - a + pair - 1) / pair;
  }
  __device__ void init(const int* rs, int b_, int rows, int pr, int ln) {
    row_start = rs;
    B = b_;
    n_rows = rows;
    pair = pr;
    lane = ln;
    bits = 0;
    sorted = B <= 32 * kKept;
    kept = (B + 31) / 32;
    window = 0;
    before = 0;
    most = 0;
    if (sorted) {
#pragma unroll
      for (int i = 0; i < kKept; ++i) {
        if (i >= kept) break;
        const int b = lane + 32 * i;
        n[i] = b < B ? items_of(b, true) : 0;
        first[i] = b < B ? row_start[b] : 0;
        end[i] = b < B ? row_start[b + 1] : 0;
        most = max(most, n[i]);
      }
      most = (int)__reduce_max_sync(0xffffffffu, (unsigned)most);
    }
  }
  __device__ int at_or_above(int level) const {  // items whose place in their sequence is >= level
    int c = 0;
#pragma unroll
    for (int i = 0; i < kKept; ++i)
      if (i < kept) c += max(n[i] - level, 0);
    return __reduce_add_sync(0xffffffffu, c);
  }
  // Rows a .. z - 1 of the sequence of item idx, and its place there (calls with rising idx); false: there are no more.
  __device__ bool find(int idx, int& a, int& z, int& place) {
    if (sorted) {
      if (idx >= at_or_above(0)) return false;
      int lo = 0, hi = most - 1;  // the highest level with more than idx items at or above it
      while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (at_or_above(m) > idx) lo = m; else hi = m - 1;
      }
      int rank = idx - at_or_above(lo + 1);  // among the sequences that have this level
      place = lo;
#pragma unroll
      for (int i = 0; i < kKept; ++i) {
        if (i >= kept) break;
        const unsigned has = __ballot_sync(0xffffffffu, n[i] > lo);
        const int c = __popc(has);
        if (rank >= 0 && rank < c) {
          const bool mine = n[i] > lo && __popc(has & ((1u << lane) - 1)) == rank;
          const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
          a = __shfl_sync(0xffffffffu, first[i], src);
          z = __shfl_sync(0xffffffffu, end[i], src);
        }
        rank -= c;
      }
      return true;
    }
    while (window < B) {
      const int s = window + lane;
      const int c = s < B ? items_of(s, true) : 0;
      int x = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const int all = __shfl_sync(0xffffffffu, x, 31);
      if (idx < before + all) {
        const int local = idx - before;
        const unsigned has = __ballot_sync(0xffffffffu, x > local);
        const int w = __ffs(has) - 1;
        a = row_start[window + w];
        z = row_start[window + w + 1];
        place = local - __shfl_sync(0xffffffffu, x - c, w);
        return true;
      }
      before += all;
      window += 32;
    }
    return false;
  }
  // Item k of this block (row0 -1: there are no more; calls with rising k): rounds of gridDim.x items, every second one
  // in the other direction (32 bits: the rows of K alone limit items to a 32nd of what the GPU's memory holds).
  __device__ Item item(int k, int heads) {
    const unsigned at = (unsigned)k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    int a = 0, z = 0, place = 0;
    if (!find((int)(at / (unsigned)heads), a, z, place)) return Item{-1, 0, 0, 0};
    return Item{a, z - a, place * pair, (int)(at % (unsigned)heads)};
  }
};

// Adds to a block's output rows what was taken out of V: infinities and NaN of the tokens from an item's second to each
// row's own.  An item to a warp of the first eight, four dimensions to a lane; rare, so out of the kernel's own code.
__device__ __noinline__ void give_back(int sequences, int heads, int G, const int* row_start, int n_rows, const uint16_t* v,
                                       size_t v_stride, uint16_t* out, size_t out_stride) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tokens = 2 * (kTile / G);
  Schedule sch;
  sch.init(row_start, sequences, n_rows, tokens, lane);
  for (int k = 0;; ++k) {
    const Item it = sch.item(k, heads);
    if (it.row0 < 0) return;
    if (k % 8 != warp) continue;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t = it.tok0 + 1; t < min(it.len, it.tok0 + tokens); ++t) {
      const uint2 x = *reinterpret_cast<const uint2*>(v + (size_t)(it.row0 + t) * v_stride + (size_t)it.h * kD + lane * 4);
      const uint32_t w[4] = {x.x << 16, x.x & 0xffff0000u, x.y << 16, x.y & 0xffff0000u};
#pragma unroll
      for (int d = 0; d < 4; ++d)
        if ((w[d] & 0x7f800000u) == 0x7f800000u) sum[d] += __uint_as_float(w[d]);
      if (sum[0] == 0.f && sum[1] == 0.f && sum[2] == 0.f && sum[3] == 0.f) continue;
      for (int g = 0; g < G; ++g) {
        uint2* dst = reinterpret_cast<uint2*>(out + (size_t)(it.row0 + t) * out_stride + (size_t)(it.h * G + g) * kD + lane * 4);
        const uint2 o = *dst;
        *dst = make_uint2(pack_bf16x2(bf_lo(o.x) + sum[0], bf_hi(o.x) + sum[1]),
                          pack_bf16x2(bf_lo(o.y) + sum[2], bf_hi(o.y) + sum[3]));
      }
    }
  }
}

// The scheduler warp: hands out the block's items, and looks over the V tiles with tokens that not all rows of an item
// attend.  False: a wait gave up.  Out of the kernel's own code (56 registers of the warp's 88): inlined, it crowded
// the other roles, and the whole kernel took 4 to 5% longer.
__device__ __noinline__ bool schedule(Bars* bars, uint8_t* ring, int sequences, int heads, int per, const int* row_start,
                                      int n_rows, unsigned* err) {
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort_flag;
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag)) != 0;
  };
  bool ok = true;
  Schedule sch;
  sch.init(row_start, sequences, n_rows, 2 * per, lane);
  unsigned slot = 0, raw_uses = 0;  // ring places of the items before, uses of raw_full (odd: 1)
  // Rows behind the sequence's last token become zeros, infinities and NaN after the item's first token too.
  auto look_over = [&](const Item& it) {
    const int n = max(kv_tiles(it, 0, per), kv_tiles(it, 1, per));
    for (int j = first_masked(it); j < n; ++j) {
      const unsigned place = (slot + 2 * (unsigned)j + 1) % kRing;
      if (!wait_all(&bars->raw_full[place], raw_uses >> place & 1)) return false;
      raw_uses ^= 1u << place;
      uint8_t* buf = ring + (size_t)place * kTileBytes;
      const int held = min(kTile, it.len - j * kTile);                    // rows of the sequence
      const int c0 = max(0, it.tok0 + 1 - j * kTile) * 8, c1 = held * 8;  // in pieces of 16 bytes
      const bool clean = all_finite(smem_u32(buf), c0, c1, lane);
      if (!clean) {
        for (int c = c0 + lane; c < c1; c += 32)
          for (int half = 0; half < 2; ++half) {
            uint4* at = reinterpret_cast<uint4*>(buf + half * kHalf + c * 16);
            const uint4 x = *at;
            *at = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
          }
        if (lane == 0) *reinterpret_cast<volatile int*>(&bars->cleaned) = 1;
      }
      for (int c = c1 + lane; c < kTile * 8; c += 32) {
        *reinterpret_cast<uint4*>(buf + c * 16) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(buf + kHalf + c * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      if (!clean || held < kTile) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->kv_full[place]);
    }
    slot += 2 * (unsigned)n;
    return true;
  };
  // An item's tiles are looked over when the next item is out, so that the producer need not wait for it.
  for (int k = 0;; ++k) {
    const Item it = sch.item(k, heads);
    const int st = k % kItems;
    if (!wait_all(&bars->item_empty[st], ((k / kItems) & 1) ^ 1)) {
      ok = false;
      break;
    }
    if (lane == 0) {
      bars->items[st] = it;
      mbar_arrive(&bars->item_full[st]);
    }
    __syncwarp();
    if (k > 0 && !look_over(bars->items[(k - 1) % kItems])) {
      ok = false;
      break;
    }
    if (it.row0 < 0) break;
  }
  set_err(err, sch.bits);
  return ok;
}

__global__ void __launch_bounds__(kThreads, 1)
prompt_attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, PagedShape s, const uint16_t* v, size_t v_stride,
                   const int* row_start, int n_rows, float scale_log2, uint16_t* out, size_t out_stride,
                   unsigned* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + 2 * kTileBytes;
  Bars* bars = reinterpret_cast<Bars*>(ring + kRing * (size_t)kTileBytes);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = s.Hq / s.Hkv, per = kTile / G;  // per: tokens of a query tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i][0], 4);
      mbar_init(&bars->p_full[i][1], 4);
      mbar_init(&bars->o_full[i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bars->kv_full[i], 1);
      mbar_init(&bars->kv_empty[i], 2);  // both tiles' MMAs
      mbar_init(&bars->raw_full[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->item_empty[i], kConsumers);
    }
    mbar_init(&bars->done[0], 1);
    mbar_init(&bars->done[1], 1);
    bars->abort_flag = 0;
    bars->token = 0;
    bars->cleaned = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem_base)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  wait_for_predecessor();
  bool timed_out = false;

  // Item k of this block, for the warps that consume items: false at the end or on a time-out.
  auto take = [&](int k, Item& it) {
    const int st = k % kItems;
    const bool ok = mbar_wait(&bars->item_full[st], (k / kItems) & 1, abort_flag);
    if (!__all_sync(0xffffffffu, ok)) {
      timed_out = true;
      return false;
    }
    it = bars->items[st];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[st]);
    return it.row0 >= 0;
  };

  // A whole warp waits: the same answer for all lanes.
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag)) != 0;
  };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax and output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int i = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lanes + (uint32_t)i * 128, o_addr = tmem + lanes + 256u + (uint32_t)i * 128;
    const int g = row % G, tok_in = row / G;
    const bool sectors = (reinterpret_cast<uintptr_t>(out) & 31) == 0 && out_stride % 16 == 0;
    unsigned turn = 0, outputs = 0;
    Item it;
    for (int k = 0; take(k, it); ++k) {
      const int n = kv_tiles(it, i, per);
      if (n == 0) continue;
      const int t0 = it.tok0 + i * per, tok = t0 + tok_in;
      float ref = 0.f;
      uint64_t sum_a = 0, sum_b = 0;
      for (int j = 0; j < n; ++j, ++turn) {
        if (!wait_all(&bars->s_full[i], turn & 1)) {
          timed_out = true;
          break;
        }
        tc_fence_after();
        uint32_t x[128];
        tmem_ld32(s_addr, x);
        tmem_ld32(s_addr + 32, x + 32);
        tmem_ld32(s_addr + 64, x + 64);
        tmem_ld32(s_addr + 96, x + 96);
        tmem_wait_ld();
        if (j * kTile + kTile - 1 > t0 || (j + 1) * kTile > it.len) {  // keys in the future or behind the sequence
          const int last = min(tok, it.len - 1) - j * kTile;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > last) x[c] = 0xff800000u;
        }
        float m[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) m[c] = __uint_as_float(x[c]);
#pragma unroll
        for (int c = 8; c < 128; c += 16)
#pragma unroll
          for (int d = 0; d < 8; ++d)
            m[d] = c + 8 < 128 ? max3(m[d], __uint_as_float(x[c + d]), __uint_as_float(x[(c + 8 < 128 ? c + 8 : c) + d]))
                               : fmaxf(m[d], __uint_as_float(x[c + d]));
        const float big = scale_log2 * max3(max3(m[0], m[1], m[2]), max3(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
        if (j == 0) {
          ref = fmaxf(big, kLowest) + kDrop;
        } else if (__any_sync(0xffffffffu, big > ref + (kSlack - kDrop))) {
          // S_j is there, so the product with V_(j-1) is complete and O is at rest until P_j is handed over
          const float next = fmaxf(ref, big + kDrop), f = ex2(ref - next);
          ref = next;
          float a, b;
          unpack2(sum_a, a, b);
          sum_a = pack2(a * f, b * f);
          unpack2(sum_b, a, b);
          sum_b = pack2(a * f, b * f);
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t o[32];
            tmem_ld32(o_addr + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int d = 0; d < 32; ++d) o[d] = __float_as_uint(__uint_as_float(o[d]) * f);
            tmem_st32(o_addr + c, o);
          }
        }
        const uint64_t sc2 = pack2(scale_log2, scale_log2), ref2 = pack2(-ref, -ref);
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
          float a, b, d, e;
          unpack2(fma2(pack2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc2, ref2), a, b);
          unpack2(fma2(pack2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sc2, ref2), d, e);
          a = ex2(a);
          b = ex2(b);
          d = ex2(d);
          e = ex2(e);
          sum_a = add2(sum_a, pack2(a, b));
          sum_b = add2(sum_b, pack2(d, e));
          x[c / 2] = pack_bf16x2(a, b);
          x[c / 2 + 1] = pack_bf16x2(d, e);
          if (c % 64 == 60) {  // the product with the first 64 tokens starts while the others' weights are formed
            tmem_st32(s_addr + c / 64 * 32, x + c / 64 * 32);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_full[i][c / 64]);
          }
        }
      }
      if (timed_out) break;
      if (!wait_all(&bars->o_full[i], outputs & 1)) {
        timed_out = true;
        break;
      }
      ++outputs;
      tc_fence_after();
      float a, b, d, e;
      unpack2(sum_a, a, b);
      unpack2(sum_b, d, e);
      const float total = (a + b) + (d + e);
      const float inv = 1.0f / total;  // every row has a key; no finite score at all gives NaN
      const bool live = row < per * G && tok < it.len;
      uint16_t* dst = out + (size_t)(it.row0 + (live ? tok : 0)) * out_stride + (size_t)(it.h * G + g) * kD;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        tmem_ld32(o_addr + c, o);
        tmem_wait_ld();
        if (live) {
          uint32_t w[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) w[q] = pack_bf16x2(__uint_as_float(o[2 * q]) * inv, __uint_as_float(o[2 * q + 1]) * inv);
          if (sectors) {  // whole 32-byte sectors to an instruction
            store32(dst + c, w);
            store32(dst + c + 16, w + 8);
          } else {
#pragma unroll
            for (int q = 0; q < 16; q += 4)
              *reinterpret_cast<uint4*>(dst + c + 2 * q) = make_uint4(w[q], w[q + 1], w[q + 2], w[q + 3]);
          }
        }
      }
      tc_fence_before();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  }
  if (warp == 8 || warp == 11) {
    // ------------------------------------------------------------ MMA issuer of one row tile: one lane
    const int i = warp == 8 ? 0 : 1;
    const uint32_t id_s = instr_desc(kTile), id_o = instr_desc(kTile) | (1u << 16);
    const uint32_t q_low = qk_desc_low(smem_u32(smem) + (uint32_t)i * kTileBytes), kv0 = smem_u32(ring);
    const uint32_t s_addr = tmem + (uint32_t)i * 128, o_addr = tmem + 256u + (uint32_t)i * 128;
    if (elect_one()) {
      unsigned at = 0, phase = 0;     // ring place of the next K or V tile (K_0 V_0 K_1 V_1 ..), and its phase
      unsigned items = 0, turns = 0;  // Q tiles, S tiles so far
      auto advance = [&] {
        if (++at == kRing) {
          at = 0;
          phase ^= 1;
        }
      };
      auto ready = [&](uint64_t* bar, uint32_t parity) {
        timed_out |= !mbar_wait(bar, parity, abort_flag);
        return !timed_out;
      };
      // One tile's products at a time: what is issued from both at once is executed in turns and ends late for both,
      // which then stay in step, softmax beside softmax and products beside products (some
      // blocks took 25% longer).
      auto take_token = [&] {
        if (atomicExch(&bars->token, 1) == 0) return true;
        const unsigned long long t0 = global_ns();
        unsigned n = 0;
        while (atomicExch(&bars->token, 1) != 0) {
          if ((++n & 63u) == 0 && (*abort_flag || global_ns() - t0 > kWaitNs)) {
            timed_out = true;
            return false;
          }
        }
        return true;
      };
      auto give_token = [&] { *reinterpret_cast<volatile int*>(&bars->token) = 0; };
      auto scores = [&](uint32_t place) {  // S = Q K^T
        const uint32_t kb = qk_desc_low(kv0 + place * kTileBytes);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = ((uint32_t)(kk >> 2) * kHalf + (uint32_t)(kk & 3) * 32u) >> 4;
          mma_ss(s_addr, q_low + off, kb + off, id_s, kk > 0);
        }
        mma_commit(&bars->s_full[i]);
      };
      for (int k = 0;; ++k) {
        const int st = k % kItems;
        if (!ready(&bars->item_full[st], (k / kItems) & 1)) break;
        const Item it = bars->items[st];
        mbar_arrive(&bars->item_empty[st]);
        if (it.row0 < 0) break;
        const int ni = kv_tiles(it, i, per), n = max(kv_tiles(it, 0, per), kv_tiles(it, 1, per));
        if (ni > 0) {
          if (!ready(&bars->q_full[i], items++ & 1) || !ready(&bars->kv_full[at], phase)) break;
          tc_fence_after();
          scores(at);
          if (ni == 1) mma_commit(&bars->q_empty[i]);
          mma_commit(&bars->kv_empty[at]);
          advance();
        }
        for (int j = 1; j <= ni; ++j) {  // P_(j-1) V_(j-1), then S_j
          const uint32_t v_at = at, v_phase = phase;
          advance();
          const uint32_t vb = v_desc_low(kv0 + v_at * kTileBytes), p_phase = turns & 1;
          ++turns;
          if (!ready(&bars->kv_full[v_at], v_phase) || (j < ni && !ready(&bars->kv_full[at], phase)) ||
              !ready(&bars->p_full[i][0], p_phase))
            break;
          tc_fence_after();
          if (!take_token()) break;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_ts(o_addr, s_addr + kk * 8, vb + kk * (2048 >> 4), id_o, kk > 0 || j > 1);
          if (!ready(&bars->p_full[i][1], p_phase)) { give_token(); break; }
          tc_fence_after();
#pragma unroll
          for (int kk = 4; kk < 8; ++kk) mma_ts(o_addr, s_addr + kk * 8, vb + kk * (2048 >> 4), id_o, true);
          if (j < ni) {
            scores(at);
            give_token();
            if (j == ni - 1) mma_commit(&bars->q_empty[i]);
            mma_commit(&bars->kv_empty[at]);
            advance();
          } else {
            mma_commit(&bars->o_full[i]);
            give_token();
          }
          mma_commit(&bars->kv_empty[v_at]);
        }
        // tiles that this row tile does not read: their places are given back in step with the ring
        for (int t = 2 * ni; t < 2 * n && !timed_out; ++t) {
          if (ready(&bars->kv_full[at], phase)) mbar_arrive(&bars->kv_empty[at]);
          advance();
        }
        if (timed_out) break;
      }
      // nothing of this tile is in flight on the tensor cores when it leaves
      mma_commit(&bars->done[i]);
      mbar_drain(&bars->done[i], 0);
    }
    timed_out = __any_sync(0xffffffffu, timed_out);
  } else if (warp == 9) {
    // ------------------------------------------------------------ TMA producer
    unsigned slot = 0, q_uses[2] = {0, 0};
    unsigned raw_uses = 0, raw_now = 0;  // a bit to a ring place: uses for raw_full so far (odd: 1), its latest use is one
    if (lane < 3) {
      const CUtensorMap* map = lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v;
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
    }
    const uint32_t q_bytes = 2u * 128u * (uint32_t)(per * G);
    Item it;
    for (int k = 0; take(k, it) && !timed_out; ++k) {
      const int n = max(kv_tiles(it, 0, per), kv_tiles(it, 1, per));
      for (int j = 0; j < n && !timed_out; ++j) {
        for (int part = 0; part < 2 && !timed_out; ++part, ++slot) {  // K_j, V_j
          const bool q_here = j == 0 && kv_tiles(it, part, per) > 0;   // Q_0 before K_0, Q_1 before V_0
          const bool raw = part == 1 && j >= first_masked(it);         // to be looked over before it is full
          const unsigned place = slot % kRing;
          uint8_t* buf = ring + (size_t)place * kTileBytes;
          bool ok = true;
          if (lane == 0) {
            if (q_here) {
              ok = mbar_wait(&bars->q_empty[part], (q_uses[part] & 1) ^ 1, abort_flag);
              if (ok) {
                uint8_t* qb = smem + (size_t)part * kTileBytes;
                mbar_expect_tx(&bars->q_full[part], q_bytes);
                tma_load_3d(qb, &map_q, 0, it.h * G, it.row0 + it.tok0 + part * per, &bars->q_full[part]);
                tma_load_3d(qb + kHalf, &map_q, 64, it.h * G, it.row0 + it.tok0 + part * per, &bars->q_full[part]);
              }
            }
            ok = ok && mbar_wait(&bars->kv_empty[place], ((slot / kRing) & 1) ^ 1, abort_flag);
            if (ok) {
              uint64_t* bar = raw ? &bars->raw_full[place] : &bars->kv_full[place];
              const CUtensorMap* map = part ? &map_v : &map_k;
              mbar_expect_tx(bar, kTileBytes);
              tma_load_3d(buf, map, 0, it.h, it.row0 + j * kTile, bar);
              tma_load_3d(buf + kHalf, map, 64, it.h, it.row0 + j * kTile, bar);
            }
          }
          if (q_here) ++q_uses[part];
          timed_out = !__all_sync(0xffffffffu, ok);
          if (!timed_out) {
            raw_uses ^= raw ? 1u << place : 0u;
            raw_now = raw ? raw_now | 1u << place : raw_now & ~(1u << place);
          }
        }
      }
    }
    if (timed_out && lane == 0) {  // copies that were issued have to land before the block leaves
      for (unsigned u = slot > kRing ? slot - kRing : 0; u < slot; ++u) {
        const unsigned place = u % kRing;
        if (raw_now >> place & 1) mbar_drain(&bars->raw_full[place], (raw_uses >> place & 1) ^ 1);
        else mbar_drain(&bars->kv_full[place], (u / kRing) & 1);
      }
      for (int i = 0; i < 2; ++i)
        if (q_uses[i]) mbar_drain(&bars->q_full[i], (q_uses[i] - 1) & 1);
    }
    __syncwarp();
  } else if (warp == 10) {
    timed_out = !schedule(bars, ring, s.B, s.Hkv, per, row_start, n_rows, err);
  }

  if (timed_out) {
    *abort_flag = 1;
    if (lane == 0) set_err(err, OASIS_EW_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp < 8 && bars->cleaned)  // the block's outputs are written
    give_back(s.B, s.Hkv, G, row_start, n_rows, v, v_stride, out, out_stride);
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

bool rows_map(CUtensorMap* m, const uint16_t* p, int heads, int n_rows, size_t stride, int box_heads, int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)heads, (cuuint64_t)n_rows};
  const cuuint64_t strides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_prompt_attn(const PagedShape& s, const uint16_t* q, size_t q_stride, const uint16_t* k,
                               size_t k_stride, const uint16_t* v, size_t v_stride, const int* row_start, int n_rows,
                               float scale, uint16_t* out, size_t out_stride, unsigned* err, cudaStream_t stream) {
  if (n_rows == 0) return cudaSuccess;
  if (!encode_fn()) return cudaErrorNotSupported;
  const int G = s.G(), per = kTile / G;
  CUtensorMap mq, mk, mv;
  if (!rows_map(&mq, q, s.Hq, n_rows, q_stride, G, per) || !rows_map(&mk, k, s.Hkv, n_rows, k_stride, 1, kTile) ||
      !rows_map(&mv, v, s.Hkv, n_rows, v_stride, 1, kTile))
    return cudaErrorInvalidValue;
  // items of all sequences: at most one partly filled one for each
  const long long items = ((long long)n_rows / (2 * per) + (s.B < n_rows ? s.B : n_rows)) * s.Hkv;
  const int sms = sm_count();
  const int grid = items < sms ? (int)items : sms;
  static int attr_cache[kMaxDevicesCached] = {};
  cudaError_t e = ensure_dyn_smem((const void*)prompt_attn_kernel, kSmemBytes, attr_cache);
  if (e != cudaSuccess) return e;
  // the roles' register split draws on what the kernel is launched with: a build with fewer would wait for ever
  static int launch_regs[kMaxDevicesCached] = {};
  int& regs = launch_regs[current_device()];
  if (!regs) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, prompt_attn_kernel);
    if (e != cudaSuccess) return e;
    regs = fa.numRegs;
  }
  if (regs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  return launch_chained(prompt_attn_kernel, dim3(grid), dim3(kThreads), kSmemBytes, stream, 1, mq, mk, mv, s, v, v_stride,
                        row_start, n_rows, scale * 1.4426950408889634f, out, out_stride, err);
}

}  // namespace oasis
