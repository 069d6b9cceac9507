// Prints which tile each call of 8-bit integers on standard input is launched with, one call a
// line:  E rows C N gated  ->  tile channels rows stage_bytes stages slots chains once
// (once: an expert's rows are expected to be one tile, and the weights pass the caches)
#include <stdio.h>

#include "../../combine_ep_get_layout_amd/csrc/experts_choice.hpp"

using namespace ep;

template <class D>
static void show(const char* name, int E, long long rows, bool ring) {
  const bool once = ring && 2 * rows <= std::min<long long>(rows, E) * D::BM;
  printf("%s %d %d %d %d %d %d %d\n", name, D::BN, D::BM, D::KB, D::STAGES,
         forward_slots<D, false>(), D::kChains ? 1 : 0, once ? 1 : 0);
}

int main() {
  int E, C, N, gated;
  long long rows;
  while (scanf("%d %lld %d %d %d", &E, &rows, &C, &N, &gated) == 5) {
    switch (choose_forward_int8(E, rows, C, N, gated)) {
      case kLargeTile:
        if (short_int8(C, gated)) show<Big8Dims>("wide", E, rows, false);
        else show<BigDims>("large", E, rows, false);
        break;
      case kMediumTile: show<MediumDims>("medium", E, rows, true); break;
      case kNarrowTile: show<NarrowDims>("narrow", E, rows, true); break;
      case kSmallTile: show<SmallDims>("small", E, rows, true); break;
      case kTinyTile: show<TinyDims>("tiny", E, rows, true); break;
    }
  }
  return 0;
}
