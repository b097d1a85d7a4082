// Block tables and slot maps built from request lengths (oasis_extend_tables,
// oasis_release_tables).
//
// Mathematics: exclusive prefixes over the requests of need_b = ceil(new/16) -
// ceil(old/16) and of rows_b = new - old; the k-th page of the call is the k-th
// free page from the list's end, row r of request b is position old_b + r -
// start_b.  Whole numbers throughout, no atomics: the result does not depend on
// the order in which thread blocks run.
//
// One launch: every thread block forms the prefixes for itself (2 x 4 bytes per
// request from L2, one scan over 256 threads that each own ceil(B/256) requests)
// and then writes its own 4,096 rows of the slot map, so no block waits for
// another.  Bound: the launch, three scans and two dependent rounds of loads: 3.9 us for 256
// requests of one new token, 9.9 us for 64 prompts of 1.9 million (7.7 MB, 1.5 us at the
// copy rate: the scans' instructions, which every block repeats).
#include "paged.cuh"

namespace oasis {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerCta = 4096;
constexpr int kSpans = 512;  // requests with rows in a block's range that are listed at a time

__device__ __forceinline__ long long shfl_up_ll(long long v, int o) { return __shfl_up_sync(0xffffffffu, v, o); }

// Exclusive scan of one value per thread over the block; total receives the sum.
__device__ long long block_exclusive(long long v, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = shfl_up_ll(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // warp_sums may still be read from an earlier scan
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  long long off = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    off += w < warp ? warp_sums[w] : 0;
    all += warp_sums[w];
  }
  *total = all;
  return off + x - v;
}

struct Growth {
  int old_len, new_len, need;
  bool bad;
};

__device__ __forceinline__ Growth growth(const PagedShape& s, const int* old_len, const int* new_len, int b) {
  Growth g;
  g.old_len = old_len[b];
  g.new_len = new_len[b];
  const long long cap = (long long)s.nb_max * kBS;
  g.bad = g.old_len < 0 || g.new_len < g.old_len || (long long)g.new_len > cap;
  if (g.bad) g.new_len = g.old_len;
  g.need = g.bad ? 0 : (int)(((long long)g.new_len + kBS - 1) / kBS - ((long long)g.old_len + kBS - 1) / kBS);
  return g;
}

struct RowSpan {  // a request with rows in this thread block's range
  int first;   // its first row, from the range's start (negative: before it)
  int b;
  int held;    // tokens that it holds
  int page0;   // its first new page's place in the call, -1: the request got nothing
};

__global__ void __launch_bounds__(kThreads)
extend_tables_kernel(PagedShape s, const int* old_len, const int* new_len,
                     const int* free_pages, const int* n_free_in,
                     int* table, int* len_out, int* n_free_out,
                     int* row_start, int* slot_map, int n_rows, unsigned* err) {
  __shared__ RowSpan spans[kSpans + 1];
  __shared__ long long warp_sums[kThreads / 32];
  __shared__ int taken_max[kThreads / 32];
  wait_for_predecessor();
  const int tid = threadIdx.x;
  const bool first_cta = blockIdx.x == 0;
  const long long lo = (long long)blockIdx.x * kRowsPerCta;
  const long long hi = lo + kRowsPerCta < n_rows ? lo + kRowsPerCta : n_rows;
  const int nf_raw = *n_free_in;
  const int n_free = nf_raw < 0 ? 0 : (nf_raw > s.n_pages ? s.n_pages : nf_raw);
  const int per = (s.B + kThreads - 1) / kThreads;
  const int b_lo = min(tid * per, s.B), b_hi = min(b_lo + per, s.B);

  long long need = 0, rows = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Growth g = growth(s, old_len, new_len, b);
    need += g.need;
    rows += g.new_len - g.old_len;
  }
  long long need_all, rows_all;
  const long long need0 = block_exclusive(need, warp_sums, &need_all);
  const long long row0 = block_exclusive(rows, warp_sums, &rows_all);

  // the requests with rows in [lo, hi), in order; block 0 also writes the per-request outputs
  int mine = 0, taken = 0;
  unsigned bits = first_cta && nf_raw != n_free ? OASIS_EW_BAD_COUNT : 0u;
  {
    long long nd = need0, rw = row0;
    for (int b = b_lo; b < b_hi; ++b) {
      const Growth g = growth(s, old_len, new_len, b);
      const int n = g.new_len - g.old_len;
      if (n > 0 && rw < hi && rw + n > lo) ++mine;
      if (first_cta) {
        const bool no_page = g.need > 0 && nd + g.need > n_free, no_room = rw + n > n_rows;
        if (g.need > 0 && !no_page && !no_room) taken = max(taken, (int)(nd + g.need));
        len_out[b] = no_page || no_room ? g.old_len : g.new_len;
        row_start[b] = (int)min(rw, (long long)n_rows);
        bits |= (no_page ? OASIS_EW_NO_SLOT : 0u) | (g.bad || no_room ? OASIS_EW_BAD_COUNT : 0u);
      }
      nd += g.need;
      rw += n;
    }
  }
  if (first_cta) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
    if ((tid & 31) == 0) taken_max[tid >> 5] = taken;
  }
  __syncthreads();
  if (first_cta && tid == 0) {
    for (int w = 1; w < kThreads / 32; ++w) taken = max(taken, taken_max[w]);
    *n_free_out = n_free - taken;
    row_start[s.B] = (int)min(rows_all, (long long)n_rows);
  }

  const int rows_here = (int)max(0LL, min(hi, rows_all) - lo);  // of requests; the others get -1
  const int rows_end = (int)(hi - lo);
  const bool quads = (reinterpret_cast<uintptr_t>(slot_map) & 15) == 0;  // lo is a multiple of 4
  long long listed_all;
  const int at0 = (int)block_exclusive(mine, warp_sums, &listed_all);
  const int listed = (int)listed_all;
  for (int base = 0; base == 0 || base < listed; base += kSpans) {
    if (base > 0) __syncthreads();  // the spans of the round before are read
    if (mine > 0 && at0 <= base + kSpans && at0 + mine > base) {
      long long nd = need0, rw = row0;
      int at = at0;
      for (int b = b_lo; b < b_hi; ++b) {
        const Growth g = growth(s, old_len, new_len, b);
        const int n = g.new_len - g.old_len;
        if (n > 0 && rw < hi && rw + n > lo) {
          const bool ok = !(g.need > 0 && nd + g.need > n_free) && rw + n <= n_rows;
          if (at >= base && at <= base + kSpans) spans[at - base] = RowSpan{(int)(rw - lo), b, g.old_len, ok ? (int)nd : -1};
          ++at;
        }
        nd += g.need;
        rw += n;
      }
    }
    __syncthreads();
    // the rows of these spans (of the last ones: to the range's end), four to a thread: mostly of one request
    const int count = min(kSpans, listed - base);
    const int row_lo = base == 0 ? 0 : spans[0].first;
    const int row_hi = min(rows_end, base + kSpans < listed ? spans[kSpans].first : kRowsPerCta);
    auto span_of = [&](int r) {  // the last span that starts at or before r
      int i = 0, j = count - 1;
      while (i < j) {
        const int m = (i + j + 1) >> 1;
        if (spans[m].first <= r) i = m; else j = m - 1;
      }
      return i;
    };
    auto page_of = [&](const RowSpan& sp, int x) {  // of block x of the span's request
      const int held = (int)(((long long)sp.held + kBS - 1) / kBS);
      int page = x >= held ? free_pages[n_free - 1 - (sp.page0 + x - held)] : table[(long long)sp.b * s.nb_max + x];
      if (page < 0 || page >= s.n_pages) {
        page = -1;
        bits |= OASIS_EW_BAD_BLOCK;
      }
      return page;
    };
    auto enter = [&](const RowSpan& sp, int x, int page) {  // a block whose first token is a new row
      if ((long long)x * kBS >= sp.held) table[(long long)sp.b * s.nb_max + x] = page;
    };
    auto slot_of = [](int page, int pos) { return page < 0 ? -1 : page * kBS + pos % kBS; };
    // requests of a few rows (a decode step): a row to a thread, or four of them would wait in turn (256 requests
    // of one row: 6.6 against 4.1 us; 64 prompts of 30,000 rows: 8.7 in fours against 12.9)
    const int each = quads && count * 8 <= row_hi - row_lo ? 4 : 1;
    for (int r0 = row_lo / each * each + each * tid; r0 < row_hi; r0 += each * kThreads) {
      const int i = each == 4 && r0 < rows_here ? span_of(max(r0, row_lo)) : 0;
      const int span_end = min(rows_here, i + 1 < count ? spans[i + 1].first : row_hi);
      if (each == 4 && r0 >= row_lo && r0 + 4 <= span_end) {
        const RowSpan sp = spans[i];
        int4 out = make_int4(-1, -1, -1, -1);
        if (sp.page0 >= 0) {
          const int pos = sp.held + r0 - sp.first, x0 = pos / kBS, x1 = (pos + 3) / kBS;
          const int p0 = page_of(sp, x0), p1 = x1 != x0 ? page_of(sp, x1) : p0;
          if (pos % kBS == 0) enter(sp, x0, p0);
          if (x1 != x0) enter(sp, x1, p1);
          out = make_int4(slot_of(p0, pos), slot_of((pos + 1) / kBS == x0 ? p0 : p1, pos + 1),
                          slot_of((pos + 2) / kBS == x0 ? p0 : p1, pos + 2), slot_of(p1, pos + 3));
        }
        *reinterpret_cast<int4*>(slot_map + lo + r0) = out;
        continue;
      }
      for (int r = max(r0, row_lo); r < min(r0 + each, row_hi); ++r) {
        int slot = -1;
        if (r < rows_here) {
          const RowSpan sp = spans[span_of(r)];
          if (sp.page0 >= 0) {
            const int pos = sp.held + r - sp.first, page = page_of(sp, pos / kBS);
            if (pos % kBS == 0) enter(sp, pos / kBS, page);
            slot = slot_of(page, pos);
          }
        }
        slot_map[lo + r] = slot;
      }
    }
  }
  set_err(err, bits);
}

// Request b's released pages go to places n_free + (prefix over requests) of the
// free list; the blocks of a request are copied by one thread block.
__global__ void __launch_bounds__(kThreads)
release_tables_kernel(PagedShape s, const int* len, const int* keep_len,
                      const int* table, int* free_pages,
                      const int* n_free_in, int* n_free_out, unsigned* err) {
  __shared__ long long warp_sums[kThreads / 32];
  __shared__ long long chunk0[kThreads];
  wait_for_predecessor();
  const int tid = threadIdx.x;
  const int nf_raw = *n_free_in;
  const int n_free = nf_raw < 0 ? 0 : (nf_raw > s.n_pages ? s.n_pages : nf_raw);
  const int per = (s.B + kThreads - 1) / kThreads;
  const int b_lo = min(tid * per, s.B), b_hi = min(b_lo + per, s.B);
  unsigned bits = nf_raw != n_free ? OASIS_EW_BAD_COUNT : 0u;
  // a request that keeps keep_len of len tokens is one that grows from keep_len to len
  long long n = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Growth g = growth(s, keep_len, len, b);
    n += g.need;
    if (g.bad) bits |= OASIS_EW_BAD_COUNT;
  }
  long long all;
  chunk0[tid] = block_exclusive(n, warp_sums, &all);
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    const long long left = n_free + all;
    *n_free_out = (int)min(left, (long long)s.n_pages);
    if (left > s.n_pages) bits |= OASIS_EW_NO_SLOT;
  }
  for (int b = blockIdx.x; b < s.B; b += gridDim.x) {
    const Growth g = growth(s, keep_len, len, b);
    if (g.need == 0) continue;
    long long at = n_free + chunk0[b / per];
    for (int c = b / per * per; c < b; ++c) at += growth(s, keep_len, len, c).need;
    const int x0 = (int)(((long long)g.old_len + kBS - 1) / kBS);
    for (int i = tid; i < g.need && at + i < s.n_pages; i += kThreads) {
      int page = table[(long long)b * s.nb_max + x0 + i];
      if (page < 0 || page >= s.n_pages) {
        page = -1;
        bits |= OASIS_EW_BAD_BLOCK;
      }
      free_pages[at + i] = page;
    }
  }
  set_err(err, bits);
}

}  // namespace

cudaError_t launch_extend_tables(const PagedShape& s, const int* old_len, const int* new_len, const int* free_pages,
                                 const int* n_free, int* table, int* len_out, int* n_free_out, int* row_start,
                                 int* slot_map, int n_rows, unsigned* err, cudaStream_t stream) {
  const int grid = n_rows > kRowsPerCta ? (n_rows + kRowsPerCta - 1) / kRowsPerCta : 1;
  return launch_chained(extend_tables_kernel, dim3(grid), dim3(kThreads), 0, stream, 1, s, old_len, new_len, free_pages,
                        n_free, table, len_out, n_free_out, row_start, slot_map, n_rows, err);
}

cudaError_t launch_release_tables(const PagedShape& s, const int* len, const int* keep_len, const int* table,
                                  int* free_pages, const int* n_free, int* n_free_out, unsigned* err,
                                  cudaStream_t stream) {
  const int most = 2 * sm_count();
  const int grid = s.B < most ? s.B : most;
  return launch_chained(release_tables_kernel, dim3(grid), dim3(kThreads), 0, stream, 1, s, len, keep_len, table, free_pages,
                        n_free, n_free_out, err);
}

}  // namespace oasis
