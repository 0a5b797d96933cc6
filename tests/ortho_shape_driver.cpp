// Tile choice and estimates of the Newton-Schulz products for problems read from stdin ("batch M N symmetric steps"), for the
// 256 CUs that they were fitted on: "choice us64 us128 us128pairs us256 split" a line.
#include <cstdio>

#include "ortho_shape.h"

int main() {
    long b, m, n, steps;
    int symmetric;
    while (std::scanf("%ld %ld %ld %d %ld", &b, &m, &n, &symmetric, &steps) == 5) {
        const int sides[] = {64, 128, 128, 256};
        std::printf("%d", (int)ortho_tile(b, m, n, symmetric, steps, 256));
        for (int i = 0; i < 4; i++) std::printf(" %.3f", ortho_tile_us((OrthoTile)i, ortho_tiles(b, m, n, symmetric, sides[i]), steps, 256));
        std::printf(" %d\n", symmetric ? (int)ortho_split(ortho_tiles(b, m, n, true, 64), steps, 1 << 20, 256) : 1);
    }
}
