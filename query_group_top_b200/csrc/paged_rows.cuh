// The new tokens of a batch and where their rows lie in a paged cache: shared
// by the append kernel and the attention kernels over the cache.
//
// The batch's new tokens are numbered 0 .. T-1, sequence after sequence:
// sequence b has tokens cu[b] .. cu[b+1]-1, or, without cu, tokens b*g ..
// b*g+g-1 (one step of g tokens each).  seqlens[b] counts the cache rows that
// the sequence holds with its n_b new ones, so new token i of sequence b sits
// at row seqlens[b] - n_b + i, and row r of sequence b is row r % page_size of
// page table[b][r / page_size].
//
// Nothing here trusts what the device arrays hold: a span or a page that does
// not fit is told to the caller (ok = false, row -1), which skips it.  The
// arithmetic is plain C++ so that it is checked on the host as well.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define PIVOT_HD __host__ __device__ __forceinline__
#else
#define PIVOT_HD inline
#endif

namespace pivot {

struct NewSpan {
  int tok0;  // first new token of the sequence
  int n;     // its new tokens
  int len;   // its cache rows, the new ones included
  bool ok;   // false: the lengths contradict each other or the cache; skip the sequence
};

struct PagedRows {
  const int32_t* table;    // [B][max_pages]
  const int32_t* seqlens;  // [B]
  const int32_t* cu;       // [B+1], or null: g tokens each
  int B, T, g;
  int max_pages, num_pages, log2_page;
  int max_len;             // longest sequence that may be read or written

  PIVOT_HD NewSpan span(int b) const {
    const long long lo = cu ? cu[b] : static_cast<long long>(b) * g;
    const long long hi = cu ? cu[b + 1] : lo + g;
    const long long len = seqlens[b];
    const bool in = lo >= 0 && hi >= lo && hi <= T;
    NewSpan s;
    s.tok0 = in ? static_cast<int>(lo) : 0;
    s.n = in ? static_cast<int>(hi - lo) : 0;
    s.len = static_cast<int>(len);
    s.ok = in && len >= hi - lo && len <= max_len;
    return s;
  }
  // The new tokens of sequence b, 0 where its offsets do not fit (span(b).n).
  PIVOT_HD int new_tokens(int b) const {
    if (!cu) return g;
    const long long lo = cu[b], hi = cu[b + 1];
    return lo >= 0 && hi >= lo && hi <= T ? static_cast<int>(hi - lo) : 0;
  }
  // Page that holds row r of sequence b (0 <= r < max_len), or -1 where the
  // table names a page outside the cache.
  PIVOT_HD int page(int b, int r) const {
    const int pg = table[static_cast<long long>(b) * max_pages + (r >> log2_page)];
    return pg >= 0 && pg < num_pages ? pg : -1;
  }
  // Cache row [pages * page_size] of row r of sequence b, or -1.
  PIVOT_HD long long row(int b, int r) const {
    const int pg = page(b, r);
    return pg < 0 ? -1 : (static_cast<long long>(pg) << log2_page) + (r & ((1 << log2_page) - 1));
  }
};

// One sequence's rows: PagedRows::row with the sequence's place in the table
// taken out, in 32 bits (a cache has fewer than 2^31 rows).
struct SequenceRows {
  const int32_t* table;
  int num_pages, log2_page;

  PIVOT_HD SequenceRows(const PagedRows& p, int b)
      : table(p.table + static_cast<long long>(b) * p.max_pages), num_pages(p.num_pages), log2_page(p.log2_page) {}
  PIVOT_HD int row(int r) const { return row_or(r, -1); }
  PIVOT_HD int row_or(int r, int none) const {
    const int pg = table[r >> log2_page];
    return pg >= 0 && pg < num_pages ? (pg << log2_page) + (r & ((1 << log2_page) - 1)) : none;
  }
};

// Rows [0, max_len) that sequences of a cache may use: no more than the table
// covers, in an int.
PIVOT_HD int paged_max_len(int max_pages, int log2_page, int max_seqlen) {
  const long long rows = static_cast<long long>(max_pages) << log2_page;
  return rows < max_seqlen ? static_cast<int>(rows) : max_seqlen;
}

#if defined(__CUDACC__)
// The sequence that token t belongs to (the last b with cu[b] <= t), found by
// the whole warp: 32 probes a round, so two rounds settle 1024 sequences.
__device__ __forceinline__ int find_sequence(const PagedRows& p, int t, int lane) {
  if (!p.cu) return t / p.g;
  int lo = 0, hi = p.B;  // cu[lo] <= t (assumed), the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool below = at < hi && p.cu[at] <= t;
    const unsigned votes = __ballot_sync(0xffffffffu, below) | 1u;
    const int last = 31 - __clz(votes);
    lo += last * step;
    hi = min(hi, lo + step);
  }
  return lo;
}
#endif

}  // namespace pivot
