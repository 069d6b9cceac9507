// Prints which tile each call on standard input is launched with, one call a line:
//   forward E rows C wide fp8 fp8_result  ->  tile channels rows stage_bytes stages slots chains
//   dx E rows C O                         ->  the same
//   dw E C O                              ->  tile channels rows
//   dbias E rows N                        ->  channels of a workgroup
#include <stdio.h>
#include <string.h>

#include "../../combine_ep_get_layout_amd/csrc/experts_choice.hpp"

using namespace ep;

template <class D>
static void show(const char* name, int slots, bool chains) {
  printf("%s %d %d %d %d %d %d\n", name, D::BN, D::BM, D::KB, D::STAGES, slots, chains ? 1 : 0);
}

template <bool FP8>
static void forward(int E, long long rows, int C, long long wide, bool fp8_result) {
  typedef typename std::conditional<FP8, Big8Dims, BigDims>::type Large;
  const bool chain = !fp8_result;  // a result in FP8 takes more of the LDS
  switch (choose_forward<FP8>(E, rows, C, wide, fp8_result)) {
#define SHOW(D, name) show<D>(name, forward_slots<D, FP8>(), chain && D::kChains)
    case kLargeTile: SHOW(Large, "large"); break;
    case kMediumTile: SHOW(MediumDims, "medium"); break;
    case kNarrowTile: SHOW(NarrowDims, "narrow"); break;
    case kSmallTile: SHOW(SmallDims, "small"); break;
    case kTinyTile: SHOW(TinyDims, "tiny"); break;
#undef SHOW
  }
}

int main() {
  char op[16];
  while (scanf("%15s", op) == 1) {
    int E, C, O, fp8, result;
    long long rows, wide;
    if (!strcmp(op, "forward")) {
      if (scanf("%d %lld %d %lld %d %d", &E, &rows, &C, &wide, &fp8, &result) != 6) return 1;
      if (fp8) forward<true>(E, rows, C, wide, result);
      else forward<false>(E, rows, C, wide, result);
    } else if (!strcmp(op, "dx")) {
      if (scanf("%d %lld %d %d", &E, &rows, &C, &O) != 4) return 1;
      switch (choose_dx(E, rows, C, O)) {
#define SHOW(D, name) show<D>(name, dx_slots<D>(), D::kChains)
        case kDxBig: SHOW(grad::Big, "big"); break;
        case kDxMedium: SHOW(grad::Medium, "medium"); break;
        case kDxSmall: SHOW(grad::Small, "small"); break;
#undef SHOW
      }
    } else if (!strcmp(op, "dw")) {
      if (scanf("%d %d %d", &E, &C, &O) != 3) return 1;
      switch (choose_dw(E, C, O)) {
#define SHOW(D, name) show<D>(name, 0, false)
        case kDwBig: SHOW(grad::Big, "big"); break;
        case kDwSquare: SHOW(grad::Square, "square"); break;
        case kDwPair: SHOW(grad::Pair, "pair"); break;
#undef SHOW
      }
    } else if (!strcmp(op, "dbias")) {
      if (scanf("%d %lld %d", &E, &rows, &C) != 3) return 1;
      printf("%d\n", choose_dbias(E, rows, C));
    } else {
      return 1;
    }
  }
  return 0;
}
