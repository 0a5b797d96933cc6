// Tile choice and estimates of the Newton-Schulz products for problems read from stdin ("batch M N symmetric steps room"), for the
// 256 CUs that they were fitted on: "choice side parts us64 us128 us128pairs us256" a line. Side and parts: of a symmetric product whose
// contraction is shared, with `room` bytes for the sums; 0 and 1 where it is not.
#include <cstdio>

#include "ortho_shape.h"

int main() {
    long b, m, n, steps, room;
    int symmetric;
    while (std::scanf("%ld %ld %ld %d %ld %ld", &b, &m, &n, &symmetric, &steps, &room) == 6) {
        const int sides[] = {64, 128, 128, 256};
        const OrthoSplit split = symmetric ? ortho_split(b, m, steps, room, 256) : OrthoSplit{0, 1};
        std::printf("%d %d %d", (int)ortho_tile(b, m, n, symmetric, steps, 256), split.parts > 1 ? (int)split.side : 0, (int)split.parts);
        for (int i = 0; i < 4; i++) std::printf(" %.3f", ortho_tile_us((OrthoTile)i, ortho_tiles(b, m, n, symmetric, sides[i]), steps, 256));
        std::printf("\n");
    }
}
