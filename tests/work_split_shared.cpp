// The cutting of own rows in the decode attention with shared rows
// (csrc/work_split.h) for tests on the host.
#include "work_split.h"

using namespace gqa;

extern "C" {

int ctas(int total, int grid) { return full_ctas(total, grid, 8); }

// [8 ctas + 1]: the first chunk of each warp, as a CTA shares its range out
void warps(int total, int ctas, int* starts) {
  const Split s(total, ctas);
  for (int c = 0; c < ctas; ++c) {
    const int c0 = s.start(c), c1 = s.start(c + 1), with = least(8, c1 - c0);
    for (int w = 0; w < 8; ++w) starts[8 * c + w] = w < with ? warp_start(c0, c1, w, with) : c1;
  }
  starts[8 * ctas] = total;
}

void span(int first, int end, int total, int ctas, int* out) {
  const WarpSpan w = warps_of(first, end, Split(total, ctas), least(8, total));
  out[0] = w.first;
  out[1] = w.last;
}

}
