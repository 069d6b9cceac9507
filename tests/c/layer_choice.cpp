// The layer's choice of kernels.  Prints for each call on standard input, one a line,
//   bytes entries E H I
// the two that its products are launched with, a line each:
//   bytes gated|down|many_gated|many_down form        (bytes 1: weights of 8 bits)
// and with an argument instead those that any call can take.
#include <stdio.h>

#include <set>
#include <string>

#include "../../combine_ep_get_layout_amd/csrc/layer_choice.hpp"

using namespace ep;

static const char* const kGated[] = {"few", "few_split", "some", "most"};
static const char* const kDown[] = {"4", "8", "16", "32"};
static const char* const kMany[] = {"few1", "few2", "rows1", "rows2_once", "rows2"};

static void kernels(bool bytes, int entries, int E, int H, int I, std::string (&out)[2]) {
  const std::string kind = bytes ? "1 " : "0 ";
  if (layer_many(entries, E, I)) {
    out[0] = kind + "many_gated " + kMany[choose_layer_many(true, entries, E, I)];
    out[1] = kind + "many_down " + kMany[choose_layer_many(false, entries, E, H)];
  } else {
    out[0] = kind + "gated " + kGated[choose_layer_gated(bytes, entries, E, I)];
    out[1] = kind + "down " + kDown[choose_layer_down(bytes, entries, E)];
  }
}

int main(int argc, char**) {
  std::string k[2];
  if (argc == 1) {
    int bytes, entries, E, H, I;
    while (scanf("%d %d %d %d %d", &bytes, &entries, &E, &H, &I) == 5) {
      kernels(bytes, entries, E, H, I, k);
      printf("%s\n%s\n", k[0].c_str(), k[1].c_str());
    }
    return 0;
  }
  std::set<std::string> all;
  for (int bytes = 0; bytes < 2; ++bytes)
    for (int entries = 1; entries <= 1024; entries += 1 + entries / 64)
      for (int E = 1; E <= kMaxExperts; E += 1 + E / 32)
        for (int H = 8; H <= 32768; H = H * 3 / 2 / 8 * 8 + 8)
          for (int I = 8; I <= 32768; I = I * 3 / 2 / 8 * 8 + 8) {
            kernels(bytes, entries, E, H, I, k);
            all.insert(k[0]);
            all.insert(k[1]);
          }
  for (const std::string& s : all) printf("%s\n", s.c_str());
  return 0;
}
