// Causal attention over packed prompts (oasis_prompt_attn), and over keys that lie before them as well
// (oasis_resume_attn): TMA -> shared memory ->
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
//
// Keys before the new rows (Piece for Item): few rows may read many keys, so all items' tiles form one sequence, cut into
// ranges of equal cost (Ranges), one for each block; parts of items that cross a border leave their accumulators,
// reference and sum in fp32, and a second kernel joins them.  Two parts at most for a block, 266 KB in all, so
// the workspace does not depend on the sizes.  32/8 heads, with the read-back from 4-bit pages: 2,048 tokens after 30,000
// 630 to 665 us in a graph of 12 calls (1.04 TFLOP, 1.9 PFLOP/s in the kernel's 540 to 565 us; read-back 25 to 30, join 12), up
// to 680 in calls that follow each other for a second, when the power cap has the SM clock at 1.72 GHz, 45 after 6,000
// 28.4 us (6, 15 and 5), eight requests of 1 to 2,000 after up to 12,000 150 us (30, 105, 8); 64/8 heads, 511 after 8,100 and
// 900 after 700 from 8-bit pages 146 us.  Beside the tiles a block pays 5 to 7 us before its first scores and 3 to 4 at
// an item's ends.  The join moves what the parts hold (40 MB where every block has two) at the rate of the L2 and HBM.
// ncu at eight requests: tensor pipe 62% of active cycles, DRAM 37%, issue slots 40%.  A scheduler walks slots without new
// rows one by one, 0.11 us each: two requests of 40 after 4,000 at the ends of 512 slots 84 us, side by side 30.  Measured and not kept: cuts up to 3 or 6
// tiles from an item's end moved there (28.4 -> 29.1 and 32.4 us for 45 tokens, the others within 2%).
// Every wait is bounded: on expiry the block raises OASIS_EW_TIMEOUT, waits (bounded)
// for its own copies and MMAs, frees TMEM and returns.
#include <type_traits>

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

// An item of a call with keys before the new rows, or a part of one: K/V tiles j0 .. j1 - 1 of the sequence.
struct Piece : Item {
  int kv0;     // first K/V row of the sequence
  int past;    // keys before its first query row
  int j0, j1;
  bool whole;  // all tiles of the item
};

__device__ __forceinline__ int past_of(const Item&) { return 0; }
__device__ __forceinline__ int past_of(const Piece& it) { return it.past; }
__device__ __forceinline__ int kv_row(const Item& it) { return it.row0; }
__device__ __forceinline__ int kv_row(const Piece& it) { return it.kv0; }
__device__ __forceinline__ int first_tile(const Item&) { return 0; }
__device__ __forceinline__ int first_tile(const Piece& it) { return it.j0; }

// What the parts of items that cross thread blocks leave for the join.  A block has two places: 0 for a part of an item
// that began in a block before it, 1 for the first part of one that goes on in the next.
struct Tail {
  int row0, len, tok0, h, past;
  int last;    // the block with the item's last tiles, -1: no item goes on from here
  int2 tiles[2];  // j0, j1 of the parts in this block's places, (0, 0): none
};
struct Parts {
  const int* kv_start;
  int n_kv_rows;
  bool unsplit;   // the bounds say that no item is cut: there is no join
  float* o;       // [blocks][2][kD / 8][2 * kTile][8], not divided: what a warp's 32 rows store at once lies together
  float2* stats;  // [blocks][2][2 * kTile]: reference and sum of a row
  Tail* tails;    // [blocks]
  __device__ __forceinline__ size_t row(int block, int place, int r) const {
    return ((size_t)block * 2 + place) * (2 * kTile) + r;
  }
  __device__ __forceinline__ float* o_at(int block, int place, int r, int c) const {  // dimensions c .. of 8 * (c / 8) + 7
    return o + ((((size_t)block * 2 + place) * (kD / 8) + c / 8) * (2 * kTile) + r) * 8 + c % 8;
  }
};

template <class It>
struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[kRing], kv_empty[kRing];
  uint64_t s_full[2], p_full[2][2], o_full[2];  // p_full: the weights of a tile's first and second 64 tokens
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t raw_full[kRing];  // V tiles that the scheduler warp has to look over first
  uint64_t done[2];
  It items[kItems];
  uint32_t tmem_base;
  int abort_flag;
  int token;  // 1: a row tile's products are being issued
  int cleaned;  // 1: infinities or NaN of V were taken out of a tile
};

template <class It>
constexpr size_t kSmemBytes = 1024 + 2 * (size_t)kTileBytes + kRing * (size_t)kTileBytes + sizeof(Bars<It>);
static_assert(kSmemBytes<Piece> <= 227 * 1024, "shared memory of a thread block");

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

// The first K/V tile of an item's sequence with tokens after the item's first one.
template <class It>
__device__ __forceinline__ int first_masked(const It& it) {
  return (past_of(it) + it.tok0 + 1) / kTile;
}

// K/V tiles that query tile i of an item reads (0: the tile has no token).
template <class It>
__device__ __forceinline__ int tiles_of(const It& it, int i, int per) {
  const int t0 = it.tok0 + i * per;
  return t0 < it.len ? (past_of(it) + min(it.len, t0 + per) + kTile - 1) / kTile : 0;
}
__device__ __forceinline__ int kv_tiles(const Item& it, int i, int per) { return tiles_of(it, i, per); }
__device__ __forceinline__ int kv_tiles(const Piece& it, int i, int per) {  // those of this part
  return max(min(tiles_of(it, i, per), it.j1) - it.j0, 0);
}

// Work items: two query tiles of one sequence and KV head.  Up to 320 sequences are kept in one
// warp's registers and the items are ordered by their place in the sequence, the last
// (the ones with the most keys) first, so that every block gets an equal share; more sequences are
// walked in their order, 32 at a time.
struct Schedule {
  using Cost = int;  // none
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

// Where every item can have an SM and no sequence more than kUnsplit keys, no item is cut: that costs a
// long item's time and saves the parts.  Sequences::cost decides it from the starts, so that the caller's bounds and
// padding change no bit of the output; where these alone say so, no join is launched either.  32/8 heads, 4-bit
// pages, device time in a graph (time of a call alone), with no join:
// 20 rows after 300 tokens 16.6 -> 14.0 us (39.6 -> 34.7), 500 without a context 24.3 -> 17.5 (45.5 -> 37.7), 100 after 900
// 23.5 -> 21.6 (44.8 -> 42.5), but 60 after 1,400 24.0 -> 26.7 and after 1,900 25.1 -> 32.4.  With a join that finds
// nothing: 8 x 20 after 600 25.1 -> 22.8, 12 x 10 after 1,000 32.8 -> 29.7, 100 after 900 in a call with room for 4,000 22.7 -> 24.8.
constexpr int kUnsplit = 1024;

// A call with keys before its new rows: its sequences, and what their items cost in keys: past + the keys of the item's last
// row (whole tiles of rows) + kItemCost for its ends, and an eighth less for an item whose second query tile has no token
// (measured: 1.3 us for a K/V tile and both query tiles, 1.1 for one, 2.8 to 3.9 for an item's ends, 1.3 us being 128 keys).
struct Sequences {
  static constexpr int kItemCost = 400;
  const int *q_start, *kv_start;
  int B, n_rows, n_kv_rows, pair, per, heads, lane;
  bool unsplit;  // no item is cut: every item costs 1, borders of equal ranges lie between items
  unsigned bits;

  __device__ void set(const int* qs, const Parts& parts, int b, int rows, int tokens, int hkv, int ln) {
    q_start = qs;
    kv_start = parts.kv_start;
    B = b;
    n_rows = rows;
    n_kv_rows = parts.n_kv_rows;
    unsplit = parts.unsplit;
    per = tokens;
    pair = 2 * tokens;
    heads = hkv;
    lane = ln;
    bits = 0;
  }
  __device__ bool sequence(int s, int& qa, int& n, int& ka, int& before) {
    qa = q_start[s];
    n = q_start[s + 1] - qa;
    ka = kv_start[s];
    const int m = kv_start[s + 1] - ka;
    before = m - n;
    const bool good = qa >= 0 && n >= 0 && q_start[s + 1] <= n_rows && ka >= 0 && m >= n && kv_start[s + 1] <= n_kv_rows;
    if (!good) {
      bits |= OASIS_EW_BAD_COUNT;
      n = 0;
    }
    return n > 0;
  }
  template <class C>
  __device__ C before_place(int p, int keys) const {  // cost of a head's items before place p
    if (unsplit) return p;
    return (C)p * (C)(keys + kItemCost) + (C)pair * ((C)p * (C)(p + 1) / 2);
  }
  // The item at place p of a sequence with n rows.
  template <class C>
  __device__ C item_cost(int p, int n, int keys) const {
    if (unsplit) return 1;
    const C c = (C)(keys + kItemCost) + (C)(p + 1) * (C)pair;
    return p * pair + per >= n ? c - c / 8 : c;
  }
  template <class C>
  __device__ C head_cost(int n, int keys) const {
    const int last = (n - 1) / pair;
    return before_place<C>(last, keys) + item_cost<C>(last, n, keys);
  }
  // The cost of all items, and whether they are cut (unsplit); of_lane: of sequence `lane`; items: how many there are, at
  // most 2^25.
  __device__ long long cost(long long* of_lane, unsigned* items) {
    long long total = 0;
    unsigned many = 0, mine = 0;
    int most = 0;  // keys of a sequence
    *of_lane = 0;
#pragma unroll 4
    for (int s = lane; s < B; s += 32) {
      int qa, n, ka, before;
      const bool some = sequence(s, qa, n, ka, before);
      const long long c = some ? heads * head_cost<long long>(n, before) : 0;
      const unsigned here = (unsigned)heads * (unsigned)((n + pair - 1) / pair);
      total += c;
      many = min(many + here, 1u << 20);
      most = max(most, some ? before + n : 0);
      if (s == lane) {
        *of_lane = c;
        mine = here;
      }
    }
    *items = __reduce_add_sync(0xffffffffu, many);
    if (!unsplit && *items <= gridDim.x && (int)__reduce_max_sync(0xffffffffu, (unsigned)most) <= kUnsplit) {
      unsplit = true;
      *of_lane = mine;
      return *items;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    return total;
  }
};

// The items cut into equal ranges of cost for the thread blocks.  A sequence's items follow each other head by head; an item
// that crosses a range's border is cut at a tile there (not one tile from its ends).  There are as many ranges as pieces of
// kLeast keys fit, or as items if they are more (items of short requests then have an SM each: 13.0 -> 11.3 us), at most one
// to an SM.  kLeast 256, 448 and 768 take 30.5, 29.7 and 29.4 us for 45 rows after 6,000 tokens, 512 28.2.
// C: unsigned where the cost of all items is below 2^31, else long long.  This arithmetic lies before a block's first load:
// with 64 bits alone eight requests take 151 us against 149, 2,048 rows after 30,000 tokens 660 against 649.
constexpr int kLeast = 512;  // least cost of a block's range, where there are no more items than such ranges
template <class C>
struct Ranges : Sequences {
  using Cost = C;
  C lo, hi;        // this block's range
  C share, extra;  // all ranges: `extra` of them are one longer than `share`
  // the sequence at hand
  int b, a, len, kv0, past;
  C start, of_head;  // where it begins, a head's cost
  int h, place;      // the next item
  C at;              // where it begins

  __device__ Ranges() {}
  __device__ explicit Ranges(const Sequences& s) : Sequences(s) {}
  // total, of_lane, items: of Sequences::cost
  __device__ void init(C total, C of_lane, unsigned items) {
    const C pieces = (total + (kLeast - 1)) / kLeast, most = pieces < (C)items ? (C)items : pieces;
    const int blocks = most < (C)gridDim.x ? (int)most : (int)gridDim.x;
    lo = hi = at = 0;
    len = 0;
    if ((int)blockIdx.x >= blocks) return;
    share = total / (C)blocks;
    extra = total - share * (C)blocks;
    lo = begin_of(blockIdx.x);
    hi = begin_of(blockIdx.x + 1);
    // the sequence that holds cost lo
    start = 0;
    for (int w = 0;; w += 32) {
      const int s = w + lane;
      C c = of_lane;
      if (w > 0) {
        int qa, n, ka, before;
        const unsigned keep = bits;  // reported with the cost
        c = s < B && sequence(s, qa, n, ka, before) ? (C)heads * head_cost<C>(n, before) : 0;
        bits = keep;
      }
      C x = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const C y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const unsigned over = __ballot_sync(0xffffffffu, start + x > lo);
      if (over) {
        const int src = __ffs(over) - 1;
        start += __shfl_sync(0xffffffffu, x - c, src);
        take_sequence(w + src);
        break;
      }
      start += __shfl_sync(0xffffffffu, x, 31);
    }
    h = (int)((lo - start) / of_head);
    const C rest = lo - start - (C)h * of_head;
    int p0 = 0, p1 = (len + pair - 1) / pair - 1;  // the last place that begins at or before it
    while (p0 < p1) {
      const int m = (p0 + p1 + 1) >> 1;
      if (before_place<C>(m, past) <= rest) p0 = m; else p1 = m - 1;
    }
    place = p0;
    at = start + (C)h * of_head + before_place<C>(place, past);
  }
  __device__ C begin_of(int block) const { return (C)block * share + ((C)block < extra ? (C)block : extra); }
  __device__ int block_of(C cost) const {
    const C longer = extra * (share + 1);
    return (int)(cost < longer ? cost / (share + 1) : extra + (cost - longer) / share);
  }
  __device__ void take_sequence(int s) {
    b = s;
    const unsigned keep = bits;
    sequence(s, a, len, kv0, past);
    bits = keep;
    of_head = len > 0 ? head_cost<C>(len, past) : 0;
    h = place = 0;
  }
  // The tile at which a border inside an item cuts it, `cost` behind its beginning; half: its second query tile is empty.
  __device__ int cut(int cost, int tiles, bool half) const {
    const int j = min(max((half ? cost + cost / 7 : cost) - kItemCost, 0) / kTile, tiles);
    return j < 2 ? 0 : tiles - j < 2 ? tiles : j;
  }
  // This block's next part (row0 -1: there are no more).  end: where its item ends, of one that goes on behind this block's
  // range and begins in it, else 0.
  __device__ Piece next(C* end) {
    *end = 0;
    while (at < hi) {
      Piece it;
      it.row0 = a;
      it.len = len;
      it.tok0 = place * pair;
      it.h = h;
      it.kv0 = kv0;
      it.past = past;
      const int tiles = max(tiles_of(it, 0, per), tiles_of(it, 1, per));
      const bool half = it.tok0 + per >= len;
      const C from = at, to = start + (C)h * of_head + before_place<C>(place, past) + item_cost<C>(place, len, past);
      at = to;
      if (++place * pair >= len) {
        place = 0;
        if (++h == heads) {
          h = 0;
          start = to;
          len = 0;
          while (len == 0 && at < hi) take_sequence(b + 1);  // below hi there is another one
        }
      }
      it.j0 = from < lo ? cut((int)(lo - from), tiles, half) : 0;
      it.j1 = to > hi ? cut((int)(hi - from), tiles, half) : tiles;
      it.whole = it.j0 == 0 && it.j1 == tiles;
      if (it.j0 >= it.j1) continue;
      if (it.j0 == 0 && !it.whole) *end = to;
      return it;
    }
    Piece none = {};
    none.row0 = -1;
    return none;
  }
};

// Adds to a block's output rows what was taken out of V: infinities and NaN of the tokens from an item's second to each
// row's own.  An item to a warp of the first eight, four dimensions to a lane; rare, so out of the kernel's own code.
template <class It>
__device__ __noinline__ void give_back(int sequences, int heads, int G, const int* row_start, int n_rows, const uint16_t* v,
                                       size_t v_stride, uint16_t* out, size_t out_stride, Parts parts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = kTile / G, tokens = 2 * per;
  std::conditional_t<std::is_same_v<It, Item>, Schedule, Ranges<long long>> sch;
  if constexpr (std::is_same_v<It, Item>) {
    sch.init(row_start, sequences, n_rows, tokens, lane);
  } else {
    sch.set(row_start, parts, sequences, n_rows, per, heads, lane);
    long long of_lane;
    unsigned items;
    const long long total = sch.cost(&of_lane, &items);
    sch.init(total, of_lane, items);
  }
  for (int k = 0;; ++k) {
    It it;
    if constexpr (std::is_same_v<It, Item>) {
      it = sch.item(k, heads);
    } else {
      long long end;
      it = sch.next(&end);
    }
    if (it.row0 < 0) return;
    if (k % 8 != warp) continue;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t = it.tok0 + 1; t < min(it.len, it.tok0 + tokens); ++t) {
      bool here = true;  // the token's key and value are in this part's tiles
      if constexpr (!std::is_same_v<It, Item>) here = it.past + t >= it.j0 * kTile && it.past + t < it.j1 * kTile;
      if (here) {
        const uint2 x = *reinterpret_cast<const uint2*>(v + (size_t)(kv_row(it) + past_of(it) + t) * v_stride +
                                                        (size_t)it.h * kD + lane * 4);
        const uint32_t w[4] = {x.x << 16, x.x & 0xffff0000u, x.y << 16, x.y & 0xffff0000u};
#pragma unroll
        for (int d = 0; d < 4; ++d)
          if ((w[d] & 0x7f800000u) == 0x7f800000u) sum[d] += __uint_as_float(w[d]);
      }
      if (sum[0] == 0.f && sum[1] == 0.f && sum[2] == 0.f && sum[3] == 0.f) continue;
      for (int g = 0; g < G; ++g) {
        if constexpr (!std::is_same_v<It, Item>) {
          if (!it.whole) {
            const int i = (t - it.tok0) / per, r = i * kTile + (t - it.tok0 - i * per) * G + g;
            float4* dst = reinterpret_cast<float4*>(parts.o_at(blockIdx.x, it.j0 == 0, r, lane * 4));
            const float4 o = *dst;
            *dst = make_float4(o.x + sum[0], o.y + sum[1], o.z + sum[2], o.w + sum[3]);
            continue;
          }
        }
        uint2* dst = reinterpret_cast<uint2*>(out + (size_t)(it.row0 + t) * out_stride + (size_t)(it.h * G + g) * kD + lane * 4);
        const uint2 o = *dst;
        *dst = make_uint2(pack_bf16x2(bf_lo(o.x) + sum[0], bf_hi(o.x) + sum[1]),
                          pack_bf16x2(bf_lo(o.y) + sum[2], bf_hi(o.y) + sum[3]));
      }
    }
  }
}

// Hands out the block's items, and looks over the V tiles with tokens that not all rows of an item attend.  False: a
// wait gave up.
template <class It, class Sch>
__device__ __forceinline__ bool hand_out(Sch& sch, Bars<It>* bars, uint8_t* ring, int heads, int per, const Parts& parts,
                                         unsigned* err) {
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort_flag;
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag)) != 0;
  };
  bool ok = true;
  Tail tail = {};
  tail.last = -1;
  unsigned slot = 0, raw_uses = 0;  // ring places of the items before, uses of raw_full (odd: 1)
  // Rows behind the sequence's last token become zeros, infinities and NaN after the item's first token too.
  auto look_over = [&](const It& it) {
    const int n = max(kv_tiles(it, 0, per), kv_tiles(it, 1, per)), j0 = first_tile(it), keys = past_of(it) + it.len;
    for (int j = max(first_masked(it), j0); j < j0 + n; ++j) {
      const unsigned place = (slot + 2 * (unsigned)(j - j0) + 1) % kRing;
      if (!wait_all(&bars->raw_full[place], raw_uses >> place & 1)) return false;
      raw_uses ^= 1u << place;
      uint8_t* buf = ring + (size_t)place * kTileBytes;
      const int held = min(kTile, keys - j * kTile);                                     // rows of the sequence
      const int c0 = max(0, past_of(it) + it.tok0 + 1 - j * kTile) * 8, c1 = held * 8;  // in pieces of 16 bytes
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
    It it;
    [[maybe_unused]] typename Sch::Cost end = 0;
    if constexpr (std::is_same_v<It, Item>) it = sch.item(k, heads);
    else it = sch.next(&end);
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
    if constexpr (!std::is_same_v<It, Item>) {
      if (it.row0 >= 0 && !it.whole) {
        tail.tiles[it.j0 == 0] = make_int2(it.j0, it.j1);
        if (end != 0) {
          tail.row0 = it.row0;
          tail.len = it.len;
          tail.tok0 = it.tok0;
          tail.h = it.h;
          tail.past = it.past;
          tail.last = sch.block_of(end - 1);
        }
      }
    }
    if (k > 0 && !look_over(bars->items[(k - 1) % kItems])) {
      ok = false;
      break;
    }
    if (it.row0 < 0) break;
  }
  if constexpr (std::is_same_v<It, Item>) {
    set_err(err, sch.bits);
  } else {
    if (blockIdx.x == 0) set_err(err, sch.bits);
    if (lane == 0) parts.tails[blockIdx.x] = tail;
  }
  return ok;
}

// The scheduler warp.  Out of the kernel's own code (56 registers of the warp's 88): inlined, it crowded the other roles, and
// the whole kernel took 4 to 5% longer.
template <class It>
__device__ __noinline__ bool schedule(Bars<It>* bars, uint8_t* ring, int sequences, int heads, int per, const int* row_start,
                                      int n_rows, Parts parts, unsigned* err) {
  const int lane = threadIdx.x & 31;
  if constexpr (std::is_same_v<It, Item>) {
    Schedule sch;
    sch.init(row_start, sequences, n_rows, 2 * per, lane);
    return hand_out(sch, bars, ring, heads, per, parts, err);
  } else {
    Sequences all;
    all.set(row_start, parts, sequences, n_rows, per, heads, lane);
    long long of_lane;
    unsigned items;
    const long long total = all.cost(&of_lane, &items);
    if (total >> 31 == 0) {
      Ranges<unsigned> sch(all);
      sch.init((unsigned)total, (unsigned)of_lane, items);
      return hand_out(sch, bars, ring, heads, per, parts, err);
    }
    Ranges<long long> sch(all);
    sch.init(total, of_lane, items);
    return hand_out(sch, bars, ring, heads, per, parts, err);
  }
}

// It: Item, or Piece where keys lie before the new rows (row_start: of the query rows, parts: the rest).
template <class It>
__global__ void __launch_bounds__(kThreads, 1)
prompt_attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, PagedShape s, const uint16_t* v, size_t v_stride,
                   const int* row_start, int n_rows, float scale_log2, uint16_t* out, size_t out_stride,
                   Parts parts, unsigned* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + 2 * kTileBytes;
  Bars<It>* bars = reinterpret_cast<Bars<It>*>(ring + kRing * (size_t)kTileBytes);
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
  auto take = [&](int k, It& it) {
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
    It it;
    for (int k = 0; take(k, it); ++k) {
      const int n = kv_tiles(it, i, per);
      if (n == 0) continue;
      const int t0 = it.tok0 + i * per, tok = t0 + tok_in;
      const int past = past_of(it) - first_tile(it) * kTile;  // keys before the first query row, from this part's first one
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
        if (j * kTile + kTile - 1 > past + t0 || (j + 1) * kTile > past + it.len) {  // in the future or behind the sequence
          const int last = past + min(tok, it.len - 1) - j * kTile;
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
        } else if (__any_sync(0xffffffffu, row < per * G && tok < it.len && big > ref + (kSlack - kDrop))) {
          // rows of no sequence do not ask, whatever they hold: no bit of the others depends on them
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
      if constexpr (std::is_same_v<It, Piece>) {
        if (!it.whole) {
          const bool mine = row < per * G && tok < it.len;
          if (mine) parts.stats[parts.row(blockIdx.x, it.j0 == 0, i * kTile + row)] = make_float2(ref, total);
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t o[32];
            tmem_ld32(o_addr + c, o);
            tmem_wait_ld();
            if (mine) {
#pragma unroll
              for (int q = 0; q < 32; q += 8) store32(parts.o_at(blockIdx.x, it.j0 == 0, i * kTile + row, c + q), o + q);
            }
          }
          tc_fence_before();
          continue;
        }
      }
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
        const It it = bars->items[st];
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
    It it;
    for (int k = 0; take(k, it) && !timed_out; ++k) {
      const int j0 = first_tile(it);
      const int n = max(kv_tiles(it, 0, per), kv_tiles(it, 1, per));
      for (int j = 0; j < n && !timed_out; ++j) {
        for (int part = 0; part < 2 && !timed_out; ++part, ++slot) {  // K_j, V_j
          const bool q_here = j == 0 && kv_tiles(it, part, per) > 0;   // Q_0 before K_0, Q_1 before V_0
          const bool raw = part == 1 && j0 + j >= first_masked(it);         // to be looked over before it is full
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
              tma_load_3d(buf, map, 0, it.h, kv_row(it) + (j0 + j) * kTile, bar);
              tma_load_3d(buf + kHalf, map, 64, it.h, kv_row(it) + (j0 + j) * kTile, bar);
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
    timed_out = !schedule<It>(bars, ring, s.B, s.Hkv, per, row_start, n_rows, parts, err);
  }

  if (timed_out) {
    *abort_flag = 1;
    if (lane == 0) set_err(err, OASIS_EW_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp < 8 && bars->cleaned)  // the block's outputs are written
    give_back<It>(s.B, s.Hkv, G, row_start, n_rows, v, v_stride, out, out_stride, parts);
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

constexpr int kJoinWarps = 8, kJoinThreads = kJoinWarps * 32;
constexpr int kJoinPerSm = 2;
constexpr int kMostBlocks = kJoinThreads;  // thread blocks whose parts a join can take

__device__ __forceinline__ float2 load8(const float2* p) {
  float2 v;
  asm volatile("ld.global.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 load16f(const float* p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}

// kRows rows of an item to a warp, from `row` on: neighbouring rows lie together eight dimensions at a time, so a lane has
// four dimensions of eight in kRows places of one row.  tails: from the item's first block.
template <int kRows>
__device__ __forceinline__ void join_rows(const Parts& parts, const Tail* tails, int first, int row, int rows, int count, int per,
                                          int G, uint16_t* out, size_t out_stride) {
  constexpr int kPlaces = kD / 8 / kRows;  // pieces of eight dimensions that one load of the warp spans
  const int lane = threadIdx.x & 31, mine = row + (lane >> 1) % kRows, c0 = lane / (2 * kRows) * 8 + (lane & 1) * 4;
  const Tail& tail = tails[0];
  const int at = min(mine, rows - 1), i = at / G / per, r = at + i * (kTile - per * G);  // behind the last row: that again
  Piece item = {};
  item.len = tail.len;
  item.tok0 = tail.tok0;
  item.past = tail.past;
  const int tiles = tiles_of(item, i, per);
  float top = neg_inf(), sum = 0.f;
  float4 o[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kAtOnce = 8 / kRows;  // parts whose loads are in flight together
  for (int p0 = 0; p0 < count; p0 += kAtOnce) {
    float2 st[kAtOnce];
    float4 x[kAtOnce][kRows];
#pragma unroll
    for (int d = 0; d < kAtOnce; ++d) {
      const int p = min(p0 + d, count - 1);
      st[d] = load8(parts.stats + parts.row(first + p, p == 0, r));
#pragma unroll
      for (int k = 0; k < kRows; ++k) x[d][k] = load16f(parts.o_at(first + p, p == 0, r, c0 + k * kPlaces * 8));
    }
#pragma unroll
    for (int d = 0; d < kAtOnce; ++d) {
      const int p = min(p0 + d, count - 1);
      const int2 part = tails[p].tiles[p == 0];
      if (p0 + d >= count || min(part.y, tiles) <= part.x) continue;  // no part, or one without tiles of this row
      const float next = fmaxf(top, st[d].x), f0 = ex2(top - next), f1 = ex2(st[d].x - next);
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        o[k] = make_float4(fmaf(o[k].x, f0, x[d][k].x * f1), fmaf(o[k].y, f0, x[d][k].y * f1),
                           fmaf(o[k].z, f0, x[d][k].z * f1), fmaf(o[k].w, f0, x[d][k].w * f1));
      sum = fmaf(sum, f0, st[d].y * f1);
      top = next;
    }
  }
  if (mine >= rows) return;
  const float inv = 1.0f / sum;
  uint16_t* dst = out + (size_t)(tail.row0 + tail.tok0 + at / G) * out_stride + (size_t)(tail.h * G + at % G) * kD + c0;
#pragma unroll
  for (int k = 0; k < kRows; ++k)
    *reinterpret_cast<uint2*>(dst + k * kPlaces * 8) =
        make_uint2(pack_bf16x2(o[k].x * inv, o[k].y * inv), pack_bf16x2(o[k].z * inv, o[k].w * inv));
}

// Joins the parts of items that go on in a later block.  Every thread block lists the items (a tail to a thread); their rows
// are dealt out in units of kJoinWarps rows, or four times as many where there are enough of them to go round.
__global__ void __launch_bounds__(kJoinThreads, kJoinPerSm)
prompt_join_kernel(PagedShape s, Parts parts, int blocks, uint16_t* out, size_t out_stride) {
  __shared__ Tail tails[kMostBlocks];
  __shared__ int unit_end[kMostBlocks], warp_units[kJoinWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = s.Hq / s.Hkv, per = kTile / G;
  wait_for_predecessor();  // the parts are written
  auto rows_of = [&](const Tail& t) { return min(t.len - t.tok0, 2 * per) * G; };
  int rows = 0;
  if (tid < blocks) {
    tails[tid] = parts.tails[tid];
    if (tails[tid].last >= 0) rows = rows_of(tails[tid]);
  }
  const int items = __syncthreads_count(rows > 0);
  const int turns = items * 2 * kTile >= (int)gridDim.x * 2 * kJoinWarps ? 4 : 2;  // rows of a warp
  int n = (rows + kJoinWarps * turns - 1) / (kJoinWarps * turns);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, n, o);
    if (lane >= o) n += y;
  }
  if (lane == 31) warp_units[warp] = n;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    n += w < warp ? warp_units[w] : 0;
    total += warp_units[w];
  }
  unit_end[tid] = n;
  __syncthreads();
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int first = 0, hi = kMostBlocks - 1;  // the first block whose units end behind u
    while (first < hi) {
      const int m = (first + hi) >> 1;
      if (unit_end[m] > u) hi = m; else first = m + 1;
    }
    const int row = ((u - (first ? unit_end[first - 1] : 0)) * kJoinWarps + warp) * turns;
    const int all = rows_of(tails[first]), count = min(tails[first].last, blocks - 1) - first + 1;
    if (row >= all) continue;
    if (turns == 4) join_rows<4>(parts, tails + first, first, row, all, count, per, G, out, out_stride);
    else join_rows<2>(parts, tails + first, first, row, all, count, per, G, out, out_stride);
  }
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

namespace {

template <class It>
cudaError_t launch_attn(const PagedShape& s, const uint16_t* q, size_t q_stride, const uint16_t* k, size_t k_stride,
                        const uint16_t* v, size_t v_stride, const int* row_start, int n_rows, int n_kv_rows, float scale,
                        uint16_t* out, size_t out_stride, const Parts& parts, int grid, unsigned* err, cudaStream_t stream) {
  const int G = s.G(), per = kTile / G;
  CUtensorMap mq, mk, mv;
  if (!rows_map(&mq, q, s.Hq, n_rows, q_stride, G, per) || !rows_map(&mk, k, s.Hkv, n_kv_rows, k_stride, 1, kTile) ||
      !rows_map(&mv, v, s.Hkv, n_kv_rows, v_stride, 1, kTile))
    return cudaErrorInvalidValue;
  static int attr_cache[kMaxDevicesCached] = {};
  cudaError_t e = ensure_dyn_smem((const void*)prompt_attn_kernel<It>, kSmemBytes<It>, attr_cache);
  if (e != cudaSuccess) return e;
  // the roles' register split draws on what the kernel is launched with: a build with fewer would wait for ever
  static int launch_regs[kMaxDevicesCached] = {};
  int& regs = launch_regs[current_device()];
  if (!regs) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, prompt_attn_kernel<It>);
    if (e != cudaSuccess) return e;
    regs = fa.numRegs;
  }
  if (regs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  return launch_chained(prompt_attn_kernel<It>, dim3(grid), dim3(kThreads), kSmemBytes<It>, stream, 1, mq, mk, mv, s, v,
                        v_stride, row_start, n_rows, scale * 1.4426950408889634f, out, out_stride, parts, err);
}

Parts parts_of(void* ws, const int* kv_start, int n_kv_rows) {
  const size_t rows = (size_t)sm_count() * 2 * (2 * kTile);
  Parts p = {};
  p.kv_start = kv_start;
  p.n_kv_rows = n_kv_rows;
  p.o = static_cast<float*>(ws);
  p.stats = reinterpret_cast<float2*>(p.o + rows * kD);
  p.tails = reinterpret_cast<Tail*>(p.stats + rows);
  return p;
}

}  // namespace

cudaError_t launch_prompt_attn(const PagedShape& s, const uint16_t* q, size_t q_stride, const uint16_t* k,
                               size_t k_stride, const uint16_t* v, size_t v_stride, const int* row_start, int n_rows,
                               float scale, uint16_t* out, size_t out_stride, unsigned* err, cudaStream_t stream) {
  if (n_rows == 0) return cudaSuccess;
  if (!encode_fn()) return cudaErrorNotSupported;
  // items of all sequences: at most one partly filled one for each
  const long long items = ((long long)n_rows / (2 * (kTile / s.G())) + (s.B < n_rows ? s.B : n_rows)) * s.Hkv;
  const int sms = sm_count();
  return launch_attn<Item>(s, q, q_stride, k, k_stride, v, v_stride, row_start, n_rows, n_rows, scale, out, out_stride, Parts{},
                           items < sms ? (int)items : sms, err, stream);
}

size_t resume_workspace_bytes() {
  const size_t blocks = (size_t)sm_count();
  return blocks * (2 * (2 * kTile) * (kD * sizeof(float) + sizeof(float2)) + sizeof(Tail));
}

// The join reads what the kernel before it left in the workspace: the caller holds workspace_lock.
cudaError_t launch_resume_attn(const PagedShape& s, const uint16_t* q, size_t q_stride, const uint16_t* k, size_t k_stride,
                               const uint16_t* v, size_t v_stride, const int* q_start, int n_rows, const int* kv_start,
                               int n_kv_rows, float scale, void* ws, uint16_t* out, size_t out_stride, unsigned* err,
                               cudaStream_t stream) {
  if (n_rows == 0 || n_kv_rows == 0) return cudaSuccess;
  if (!encode_fn()) return cudaErrorNotSupported;
  // blocks that the largest cost of these sizes can use: every item with all keys
  const int pair = 2 * (kTile / s.G());
  const long long items = ((long long)n_rows / pair + (s.B < n_rows ? s.B : n_rows)) * s.Hkv;
  const long long pieces = (items * (Sequences::kItemCost + (long long)n_kv_rows + pair) + kLeast - 1) / kLeast;
  const long long most = pieces < items ? items : pieces;
  const int sms = sm_count() < kMostBlocks ? sm_count() : kMostBlocks, grid = most < sms ? (int)most : sms;
  Parts parts = parts_of(ws, kv_start, n_kv_rows);
  parts.unsplit = items <= sms && n_kv_rows <= kUnsplit;
  cudaError_t e = launch_attn<Piece>(s, q, q_stride, k, k_stride, v, v_stride, q_start, n_rows, n_kv_rows, scale, out, out_stride,
                                     parts, grid, err, stream);
  if (e != cudaSuccess || grid == 1 || parts.unsplit) return e;
  return launch_chained(prompt_join_kernel, dim3(kJoinPerSm * sm_count()), dim3(kJoinThreads), 0, stream, 1, s, parts, grid, out,
                        out_stride);
}

}  // namespace oasis
