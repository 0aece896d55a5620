// Prints the tile of the kernel for many tokens, "tiles row_waves", of each pair of
// tokens and weight rows given.  Test infrastructure.
#include <cstdio>
#include <cstdlib>

#include "../../mxfp4_block_amax_amd/csrc/fp4_linear.h"

int main(int argc, char **argv) {
    for (int i = 1; i + 1 < argc; i += 2) {
        const fp4dev::Wide w = fp4dev::wide_tile(std::atoll(argv[i]), std::atoll(argv[i + 1]));
        std::printf("%d %d\n", w.tiles, w.row_waves);
    }
}
