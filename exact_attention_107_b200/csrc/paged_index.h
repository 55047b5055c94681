// Index arithmetic of the paged cache, plain C++ so that it also compiles for the host.
//
// Pools hold (num_pages, Hkv, 2^shift, D) elements; a sequence's row of the block table names the
// page of positions [i 2^shift, (i + 1) 2^shift).  Tables and lengths are the caller's device
// data: nothing here follows an index before it has been compared with its table.
#pragma once

#ifdef __CUDACC__
#define FA_HD __host__ __device__ __forceinline__
#else
#define FA_HD inline
#endif

namespace fa {

// Page of position p, or -1 where p or the table's entry lies outside.
FA_HD int page_of(const int* row, int width, int shift, int num_pages, long long p) {
  if (p < 0 || (p >> shift) >= width) return -1;
  const int page = row[p >> shift];
  return page >= 0 && page < num_pages ? page : -1;
}

// Row (of D elements) of position p of head hk in a pool; only for page >= 0.
FA_HD long long page_row_of(int page, int Hkv, int hk, long long p, int shift) {
  return ((static_cast<long long>(page) * Hkv + hk) << shift) + (p & ((1LL << shift) - 1));
}

// Where token n of a sequence goes that has `fresh` of the T offered tokens and len with them.
struct AppendSlot {
  bool real;           // n is one of the sequence's new tokens
  long long position;  // its position
  int page;            // -1: not to be written
};
FA_HD AppendSlot append_slot(int len, int fresh, int T, int n, const int* row, int width, int shift, int num_pages) {
  AppendSlot s;
  s.real = n < fresh;
  s.position = static_cast<long long>(len) - fresh + n;
  s.page = s.real && fresh <= T ? page_of(row, width, shift, num_pages, s.position) : -1;
  return s;
}

// Positions [first, end) that a decode row at position p may see; end = p + 1, or 0 for p < 0.
FA_HD int first_seen(int p, int window) { return window > 0 && p >= window ? p - window + 1 : 0; }

// The positions that a decode step of T rows reads of a sequence, and the tiles of `tile` that hold
// them.  Holds for lengths up to the largest int: the tiles are counted from the last position.
struct Span {
  int len, first, tile0, ntiles;
};
FA_HD Span span_of(int seq_len, int positions, int T, int window, int tile) {
  Span s;
  s.len = seq_len < 0 ? 0 : (seq_len < positions ? seq_len : positions);
  s.first = first_seen(s.len - T, window);
  s.tile0 = s.first / tile;
  s.ntiles = s.len == 0 ? 0 : (s.len - 1) / tile + 1 - s.tile0;
  return s;
}

}  // namespace fa
