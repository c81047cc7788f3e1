// How the paged operators cut their work: integer arithmetic only, for the
// kernels and for tests on the host.
#pragma once

#ifdef __CUDACC__
#define GQA_HD __host__ __device__ __forceinline__
#else
#define GQA_HD inline
#endif

namespace gqa {

GQA_HD int least(int a, int b) { return a < b ? a : b; }
GQA_HD int most(int a, int b) { return a > b ? a : b; }
// a / b rounded up, a > 0 up to the largest int
GQA_HD int ceil_div(int a, int b) { return (a - 1) / b + 1; }

// `total` units over `parts` ranges, the first `more` of them one longer.
struct Split {
  int each, more;
  GQA_HD Split(int total, int parts) : each(total / parts), more(total - each * parts) {}
  GQA_HD int start(int c) const { return c * each + least(c, more); }
  GQA_HD int holder(int u) const {  // the range that holds unit u (each > 0)
    const int x = more * (each + 1);
    return u < x ? u / (each + 1) : more + (u - x) / each;
  }
};

// ---- sequence of a packed token: 32-way search of cu[0..B]

// Of the undecided cu[lo + 1 .. lo + size], whether the last of this lane's
// stretch of `step` is at or before m.
GQA_HD bool search_at_or_before(const int* cu, int lo, int size, int step, int lane, int m) {
  const int j = (lane + 1) * step;
  return j <= size && cu[lo + j] <= m;
}
// The number of j in 1..B with cu[j] <= m; count(lo, size, step): lanes for
// which the above holds.
template <class Count>
GQA_HD int search_sequence(int B, Count count) {
  int lo = 0, size = B;
  while (size > 0) {
    const int step = (size + 31) / 32;
    const int n = count(lo, size, step);
    lo += n * step;
    size = least(step - 1, size - n * step);
  }
  return lo;
}

// ---- decode attention: chunks in (sequence, KV head, position) order

// CTAs with a range of `total` > 0 chunks: no more than leave each warp a chunk.
GQA_HD int decode_ctas(int total, int grid, int warps) { return least(grid, ceil_div(total, warps)); }
// The first chunk of a warp's share of [c0, c1); warp = warps: c1.
GQA_HD int warp_start(int c0, int c1, int warp, int warps) { return c0 + (c1 - c0) * warp / warps; }

// ---- packed prefill attention: items cut into equal ranges

constexpr int ITEM_UNITS = 2;  // what an item takes beside its key tiles, in those (2.8 us)
constexpr int MAX_PARTS = 64;  // of an item
constexpr int MIN_TILES = 3;   // key tiles of a part at least

// Units of a range: of half the longest item at least, each item in three at
// most; as short as MAX_PARTS allows. No shorter than the mean of `grid` ranges.
GQA_HD int mean_range(int units, int grid) { return most(ceil_div(units, grid), MIN_TILES); }
GQA_HD int few_parts_range(int mean, int longest) { return most(mean, (longest + 1) / 2); }
GQA_HD int many_parts_range(int mean, int longest) { return most(mean, (longest + MAX_PARTS - 3) / (MAX_PARTS - 2)); }
GQA_HD int range_count(int units, int range, int grid) { return least(grid, most(1, units / range)); }

// An item is its key tiles and, before them, ITEM_UNITS units for what else it
// takes; in (entry, KV head, key tile) order there are cum[e] * n_kv units before
// entry e. Piece of the item with unit u, from u on as far as the range that ends
// at `end` goes: key tiles [j0, j1) of KV head g of the entry (j1 <= j0: none);
// the ranges with a part of the item; the first unit behind the piece.
struct Piece {
  int entry, g, j0, j1, first, last, behind;
};
GQA_HD Piece piece_at(int u, int end, const Split& split, int entries, const int* cum, int n_kv) {
  int lo = 0, hi = entries;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] * n_kv <= u) lo = mid; else hi = mid;
  }
  Piece p;
  const int w = cum[lo + 1] - cum[lo], x = u - cum[lo] * n_kv;
  p.entry = lo;
  p.g = x / w;
  const int base = cum[lo] * n_kv + p.g * w + ITEM_UNITS;  // the unit of the item's first tile
  p.j0 = most(0, u - base);
  p.j1 = least(w - ITEM_UNITS, end - base);
  p.first = split.holder(base);
  p.last = split.holder(base + w - ITEM_UNITS - 1);
  p.behind = least(end, base + w - ITEM_UNITS);
  return p;
}

}  // namespace gqa
