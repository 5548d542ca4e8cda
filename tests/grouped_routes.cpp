// Prints the kernel that each call read from the input takes, one a line:
//   product  <N x K> <rows> <N> <K> <groups> <lda> <ldb> <strideB>
//   gradient <rows> <M> <N> <groups> <lda> <ldb>
//   projection <N x K> <M> <N> <K> <lda> <ldb>
// with operands on 16 bytes.
#include <iostream>
#include <string>

#include "../dense_fp32_gemm_f32_amd/csrc/grouped_routes.h"

int main() {
  using namespace gemmf32;
  static const char* const kProduct[] = {"rows", "mixed", "64, 4 floats", "64, 1 float",
                                         "128, 1 float"};
  std::string kind;
  while (std::cin >> kind) {
    GroupedProblem p;
    if (kind == "product") {
      std::cin >> p.tb >> p.rows >> p.N >> p.K >> p.groups >> p.lda >> p.ldb >> p.sb;
      std::cout << kProduct[(int)product_kernel(p)] << "\n";
    } else if (kind == "projection") {
      p.groups = 1;
      std::cin >> p.tb >> p.rows >> p.N >> p.K >> p.lda >> p.ldb;
      std::cout << (projection_grouped(p) ? "grouped" : "fused") << "\n";
    } else {
      std::cin >> p.rows >> p.M >> p.N >> p.groups >> p.lda >> p.ldb;
      const GradientTiles t = gradient_tiles(p);
      if (wgrad_thin(p)) {
        std::cout << "thin\n";
      } else {
        std::cout << (t.large ? "128, " : "64, ") << (t.wide ? "4 floats" : "1 float")
                  << (t.slices > 1 ? ", slices" : "") << "\n";
      }
    }
  }
}
