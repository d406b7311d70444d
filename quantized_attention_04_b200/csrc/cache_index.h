// Index arithmetic of the paged cache, shared by the kernels and (compiled as
// plain C++) by the host tests: which row a slot is, what a sequence's device
// integers may say, and how a run of tiles is cut among blocks.
#pragma once
#include <climits>
#include <cstdint>

#ifdef __CUDACC__
#define SAGE2_HD __host__ __device__ __forceinline__
#else
#define SAGE2_HD inline
#endif

namespace sage2 {

// A paged key/value cache (sage2_cache, checked): rows of d values, row
// ((page*Hkv + h) << page_shift) + slot % page of the pools.
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* ks;               // row scales (e4m3), else null
  float* vs;
  int pages, Hkv, page_shift, d;
  int kv_dtype;            // 0 fp16, 1 bf16, 3 e4m3
};

// Is slot `slot` inside a table row of MP pages?
SAGE2_HD bool slot_inside(int slot, int page_shift, int MP) {
  return slot >= 0 && (slot >> page_shift) < MP;
}
SAGE2_HD bool page_inside(int page, int pages) {
  return static_cast<unsigned>(page) < static_cast<unsigned>(pages);
}
// Row of slot `slot` of head h, given the page it is on.
SAGE2_HD long long row_of(int page, int Hkv, int h, int page_shift, int slot) {
  return (((long long)page * Hkv + h) << page_shift) + (slot & ((1 << page_shift) - 1));
}

// Tokens in the cache and drafted tokens of one sequence.
struct SeqLen {
  int len, n;
};
// Do they fit T drafted tokens and a table of `cap` slots?
SAGE2_HD bool seq_fits(int len, int n, int T, int cap) {
  return n >= 0 && n <= T && len >= 0 && n <= cap && len <= cap - n;
}
// The nearest pair that fits.
SAGE2_HD SeqLen seq_clamped(int len, int n, int T, int cap) {
  SeqLen s;
  const int top = T < cap ? T : cap;
  s.n = n < 0 ? 0 : (n > top ? top : n);
  s.len = len < 0 ? 0 : (len > cap - s.n ? cap - s.n : len);
  return s;
}

// Key tiles of one (head, row tile) pair of a sequence: none if nothing is asked of it.
SAGE2_HD int pair_tiles(SeqLen s, int tile) {
  return s.n == 0 ? 0 : (s.len + s.n + tile - 1) / tile;
}

// `total` tiles are cut among the blocks 0..grid-1 into runs as equal as can be.
SAGE2_HD int run_blocks(long long total, int grid, int least) {
  const long long most = (total + least - 1) / least;
  return (int)(most < grid ? (most < 1 ? 1 : most) : grid);
}
SAGE2_HD long long run_start(long long total, int grid, int c) { return total * c / grid; }
// The block whose run holds tile p.
SAGE2_HD int run_of(long long p, long long total, int grid) {
  return (int)(((p + 1) * grid - 1) / total);
}

}  // namespace sage2
