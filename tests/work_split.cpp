// The paged operators' cutting of work (csrc/work_split.h) for tests on the host.
#include "work_split.h"

using namespace gqa;

extern "C" {

void ranges(int total, int parts, int* starts) {  // [parts + 1]
  const Split s(total, parts);
  for (int c = 0; c <= parts; ++c) starts[c] = s.start(c);
}

void holders(int total, int parts, const int* units, int n, int* out) {
  const Split s(total, parts);
  for (int i = 0; i < n; ++i) out[i] = s.holder(units[i]);
}

int ctas(int total, int grid, int warps) { return decode_ctas(total, grid, warps); }

void shares(int c0, int c1, int warps, int* starts) {  // [warps + 1]
  for (int w = 0; w <= warps; ++w) starts[w] = warp_start(c0, c1, w, warps);
}

int sequence(const int* cu, int B, int m) {
  return search_sequence(B, [&](int lo, int size, int step) {
    int n = 0;
    for (int lane = 0; lane < 32; ++lane) n += search_at_or_before(cu, lo, size, step, lane, m);
    return n;
  });
}

int range_units(int units, int grid, int longest, int few) {
  const int mean = mean_range(units, grid);
  return few ? few_parts_range(mean, longest) : many_parts_range(mean, longest);
}
int parts_of(int units, int range, int grid) { return range_count(units, range, grid); }
int item_units() { return ITEM_UNITS; }
int max_parts() { return MAX_PARTS; }

// Every range's pieces in order, as a CTA takes them: (range, entry, g, j0, j1,
// first, last, behind) each; and, after them, that of the range's last unit, as
// the item that goes on behind it is found. Returns how many.
int pieces(int units, int parts, const int* cum, int entries, int n_kv, int* out, int room) {
  const Split s(units, parts);
  int n = 0;
  auto put = [&](int c, const Piece& p) {
    if (n < room) {
      const int v[8] = {c, p.entry, p.g, p.j0, p.j1, p.first, p.last, p.behind};
      for (int i = 0; i < 8; ++i) out[8 * n + i] = v[i];
    }
    ++n;
  };
  for (int c = 0; c < parts; ++c) {
    const int end = s.start(c + 1);
    for (int u = s.start(c); u < end;) {
      const Piece p = piece_at(u, end, s, entries, cum, n_kv);
      put(c, p);
      if (p.behind <= u) return -1;
      u = p.behind;
    }
    put(-1 - c, piece_at(end - 1, end, s, entries, cum, n_kv));
  }
  return n;
}

}  // extern "C"
