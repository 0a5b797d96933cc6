// Host arithmetic of the Newton-Schulz products: which workgroup tile a product gets. No HIP: fitted to times measured on the
// 256 CUs of an MI355X.
#pragma once
#include <stdint.h>

namespace {

// PAIRS: two workgroups to a CU, with half the stages. TAIL: whole rounds of 256, and the rest in quarters of 128.
enum OrthoTile { TILE_64, TILE_128, TILE_128_PAIRS, TILE_256, TILE_256_TAIL };

// Tiles of a batch of M x N products; a symmetric one computes those on and below the diagonal.
inline int64_t ortho_tiles(int64_t batch, int64_t M, int64_t N, bool symmetric, int side) {
    const int64_t m = (M + side - 1) / side, n = (N + side - 1) / side;
    return batch * (symmetric ? m * (m + 1) / 2 : m * n);
}

// Estimated time in us of a product whose contraction has `steps` steps of 64: rounds of tiles over the CUs, each with a fixed
// part (first loads, last stores) and a time for every step that grows with the CUs that are busy (they share caches
// and power). Measured and (estimated), five symmetric products and four others:
//                                    64            128          128 in pairs   256
//   256 x 256, 16 steps              7.5 (8.7)     14.4 (13)     13.8 (14)     20.6 (24)
//   1000 x 2001, 16                  12.2 (12)     14.7 (14)     15 (15)       23.1 (24)
//   1024 x 1024, 64                  15.3 (17)     33.2 (34)     40.8 (37)     66.2 (65)
//   2048 x 2048, 32                  23.6 (22)     21.5 (22)     24.9 (24)     40.1 (38)
//   1536 x 4096, 24                  37.8 (48)     34.2 (35)     27.2 (27)     34.6 (33)
//   8 of 1024 x 2048, 16             62.4 (88)     52 (51)       39.7 (43)     34.8 (34)
//   4096 x 4096, 64                  162 (158)     110 (112)     97.4 (104)    78.3 (77)
//   8 of 2048 x 2048, 112            -             322 (325)     326 (294)     299 (277)
//   8 of 2048 x 7168, 32             -             690 (598)     550 (507)     390 (378)
inline double ortho_tile_us(OrthoTile tile, int64_t tiles, int64_t steps, int64_t cus) {
    const double s = (double)steps;
    if (tile == TILE_64) {                       // one workgroup a CU, or two
        if (tiles <= cus) return 6.0 + 0.17 * s;
        const double fill = (double)tiles / (double)(2 * cus);
        return fill <= 1.0 ? 4.5 + (0.2 + 0.3 * fill) * s : 1.5 + fill * (1.5 + 0.58 * s);
    }
    const int64_t slots = tile == TILE_128_PAIRS ? 2 * cus : cus;
    auto round = [&](double fill) {
        switch (tile) {
            case TILE_128: return 3.0 + (0.42 + 0.15 * fill) * s;
            case TILE_128_PAIRS: return 4.0 + (fill <= 0.5 ? 0.45 + 0.3 * fill : 0.7 + 0.6 * (fill - 0.5)) * s;
            default: return 6.0 + fill + (0.85 + 0.1 * fill + 0.5 * fill * fill) * s;
        }
    };
    const int64_t whole = tiles / slots, rest = tiles % slots;
    return (tile == TILE_256 ? 4.0 : 3.0) + (double)whole * round(1.0) + (rest ? round((double)rest / (double)slots) : 0.0);
}

// The rest of whole rounds of 256 x 256 tiles, in quarters on 128 x 128 tiles, one or two to a CU. Eight symmetric 2048 x 2048
// (288 tiles), 112 steps: 267 us in two launches and 299 in one; 32 steps: 103 and 111 (102 on 128 x 128 tiles alone).
// (Several workgroups to a tile of the rest, as below, took 49 us instead of 68 to 74 in quarters with 112 steps, 28 and 22 with 32;
// but the matrices of a batch would then have their sums in different orders.)
inline OrthoTile ortho_tail_tile(int64_t rest, int64_t cus) { return 4 * rest <= cus ? TILE_128 : TILE_128_PAIRS; }

inline OrthoTile ortho_tile(int64_t batch, int64_t M, int64_t N, bool symmetric, int64_t steps, int64_t cus, double* estimate = nullptr) {
    const OrthoTile shapes[] = {TILE_64, TILE_128, TILE_128_PAIRS, TILE_256};
    const int sides[] = {64, 128, 128, 256};
    OrthoTile best = TILE_64;
    double least = 0.0;
    for (int i = 0; i < 4; i++) {
        const double us = ortho_tile_us(shapes[i], ortho_tiles(batch, M, N, symmetric, sides[i]), steps, cus);
        if (i == 0 || us < least) best = shapes[i], least = us;
    }
    const int64_t big = ortho_tiles(batch, M, N, symmetric, 256), rest = big % cus;
    if (big > cus && rest > 0) {
        const double us = ortho_tile_us(TILE_256, big - rest, steps, cus) + ortho_tile_us(ortho_tail_tile(rest, cus), 4 * rest, steps, cus);
        if (us < least) best = TILE_256_TAIL, least = us;
    }
    if (estimate) *estimate = least;
    return best;
}

// A symmetric product's tiles of `side` whose contraction `parts` workgroups share each, with a second launch that adds their sums;
// parts 1: none. As many parts as CUs, a part of at least eight steps, and `room` bytes for the sums.
struct OrthoSplit {
    int64_t side, parts;
};
// The second launch and the sums' way to the Infinity Cache and back: 4.5 us and 14 for 64 MB. Whole updates by m x n, with one workgroup a tile and with several:
// 64 x 2048 87 and 91 us, 256 x 2048 105 and 100, 64 x 4096 106 and 84, 64 x 16384 221 and 92, 512 x 4096 152 and 139, two of 496 x
// 3973 174 and 167, 640 x 10240 291 and 194; on tiles of 128 1024 x 4096 191 and 217, 1024 x 16384 446 and 387, 1536 x 8192 530 and 445;
// on tiles of 256 2560 x 8192 967 and 1029, 2048 x 16384 1321 and 1106, 3000 x 18432 2721 and 2416.
inline OrthoSplit ortho_split(int64_t batch, int64_t M, int64_t steps, int64_t room, int64_t cus) {
    double least;
    ortho_tile(batch, M, M, true, steps, cus, &least);
    OrthoSplit best = {64, 1};
    for (int64_t side = 64; side <= 256; side *= 2) {
        const int64_t tiles = ortho_tiles(batch, M, M, true, (int)side), bytes = tiles * side * side * 4;
        int64_t parts = cus / tiles;
        if (parts > steps / 8) parts = steps / 8;
        if (parts > room / bytes) parts = room / bytes;
        if (parts < 2) continue;
        const double us = ortho_tile_us(side == 64 ? TILE_64 : side == 128 ? TILE_128 : TILE_256, tiles * parts, (steps + parts - 1) / parts, cus) + 4.5 + (double)(parts * bytes) / 4.7e6;
        if (us < least) best = {side, parts}, least = us;
    }
    return best;
}

}  // namespace
