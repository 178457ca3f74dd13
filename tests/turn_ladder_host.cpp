// Prints theta^(-r / c) / 2 pi, r = 0 .. c - 1, as the library holds it: two hexadecimal words.
#include <cstdio>
#include <cstdlib>

#include "turn_ladder.h"

int main(int argc, char** argv) {
  if (argc != 3) return 2;
  const float theta = (float)std::atof(argv[1]);
  const int c = std::atoi(argv[2]);
  uint64_t hi[64];
  uint32_t lo[64];
  if (c < 1 || c > 64) return 2;
  oomb::turn_ladder((double)theta, c, hi, lo);
  for (int r = 0; r < c; ++r) std::printf("%016llx %08x\n", (unsigned long long)hi[r], (unsigned)lo[r]);
  return 0;
}
