// Prints the tile and the pieces of K that a product of M x N x K is cut into, for each
// three numbers on the command line.
#include <stdio.h>
#include <stdlib.h>

#include "../../bit_weight_gemm_amd/csrc/mx_plan.h"

int main(int argc, char **argv) {
    for (int i = 1; i + 2 < argc; i += 3) {
        const auto p = biloco::mx::plan_of(atoi(argv[i]), atoi(argv[i + 1]), atoi(argv[i + 2]));
        printf("%d %d\n", p.rows ? 0 : p.bm, p.pieces);
    }
}
