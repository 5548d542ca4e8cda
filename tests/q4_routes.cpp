// Asks the rules of the 4-bit products which kernel a call takes: "rows N K groups" on
// standard input, the kernel's name on standard output.
#include <cstdio>
#include <iostream>

#include "../dense_fp32_gemm_f32_amd/csrc/q4_routes.h"

int main() {
  gemmf32::Q4Problem p;
  while (std::cin >> p.g.rows >> p.g.N >> p.g.K >> p.g.groups) {
    const auto& t = gemmf32::kQ4Tiles[gemmf32::q4_tile(p)];
    if (gemmf32::q4_few(p))
      std::puts("few");
    else
      std::printf("%dx%d\n", t.rows, t.cols);
  }
  return 0;
}
