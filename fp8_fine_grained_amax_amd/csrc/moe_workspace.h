// Host arithmetic of the mixture of experts for a few tokens: how its down-projection is split, and where its workspace's
// parts lie. No HIP: the size query has to give the same answer whichever device is current, so the splits are for
// the 256 CUs of an MI355X.
#pragma once
#include <stdint.h>

namespace {

constexpr int kWords = 64;             // bitmap words: 2048 experts
constexpr int64_t kFusedTokens = 16;   // up to here the activations are quantized inside the two products
constexpr int kDownWaves = 8;

// A model narrow enough to leave CUs without a column block, and with steps enough, has each block's shared between up
// to 8 workgroups.
constexpr int kMaxSplits = 8;

// Workgroups that share a column block of the down-projection: as many as give every CU two, where the blocks alone
// leave half of the CUs without one, and no more than leave each wave four steps. Joining their sums costs another
// launch of 4.5 us. (64 tokens, 64 experts, H = 2048, I = 1024, 64 column blocks: 105 us, split 54 with the join.)
inline int down_splits(int64_t blocks, int64_t slots, int64_t nkb) {
    if (blocks < 1 || blocks > 128) return 1;
    const int64_t by_steps = slots * nkb / (4 * kDownWaves), by_cus = 512 / blocks;
    const int64_t s = by_steps < by_cus ? by_steps : by_cus;
    return s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : (int)s;
}
// 16-row tiles of the down-projection's workgroups: two share the tokens' operands (with up to 16 tokens only where that
// leaves workgroups enough, or they are split).
inline int down_tiles(int64_t T, int64_t H, int64_t slots, int64_t I) {
    return T > kFusedTokens || H >= 4096 || down_splits(H / 32, slots, I / 128) > 1 ? 2 : 1;
}

// What a call launches for its number of experts: at most `slots` of them chosen, and the down-projection's shape.
struct MoeLaunch {
    int64_t slots;
    int tiles, splits;
    MoeLaunch(int64_t T, int topk, int64_t E, int64_t H, int64_t I) {
        slots = T * topk < E ? T * topk : E;
        tiles = down_tiles(T, H, slots, I);
        splits = down_splits(H / (16 * tiles), slots, I / 128);
    }
};

// The slots as the planning launch writes them down for the others, and the activations' codes. A slot's tokens
// have consecutive places, 16 to a tile; the places of a slot's last tile that have no token hold token and pair -1.
struct MoePlan {
    int* used;            // number of slots
    int* list;            // [slots] experts
    int* base;            // [slots + 1] first tile
    int* place;           // [T * topk] place of a choice, or -1
    int* token;           // [tiles * 16]
    int* pair;            // [tiles * 16] choice: token * topk + number
    float* weight;        // [tiles * 16] routing weight
    uint8_t* xq;          // [T][H] codes
    float* sx;            // [H / 128][T]
    uint8_t* hq;          // [tiles][I / 128] operand blocks
    float* sh;
};

inline int64_t pad16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// Workspace: the hidden values in fp32; partial sums of a split down-projection; for more than 16 tokens also the plan and
// the activations' codes. A call's slots are at most its choices, and fewer are never split more often; a slot's tokens
// fill all its tiles but the last. H and I are multiples of 128.
struct MoeWorkspace {
    int64_t rows, slots, tiles, partial, plan, xq, sx, hq, sh, bytes;
    MoeWorkspace(int64_t T, int topk, int64_t H, int64_t I) {
        const MoeLaunch most(T, topk, 32 * kWords, H, I);
        rows = T * topk;
        slots = most.slots;
        tiles = slots + rows / 16;
        partial = rows * I * 4;
        bytes = partial + (most.splits > 1 ? most.splits * T * H * 4 : 0);
        plan = xq = sx = hq = sh = bytes;
        if (T > kFusedTokens) {
            xq = plan + pad16(4 * (2 + 2 * slots + rows + 3 * 16 * tiles));
            sx = xq + T * H;
            hq = sx + pad16(T * (H / 128) * 4);
            sh = hq + tiles * 16 * I;
            bytes = sh + tiles * 16 * (I / 128) * 4;
        }
    }
    MoePlan of(uint8_t* ws) const {
        MoePlan m{};
        m.used = (int*)(ws + plan);
        m.list = m.used + 1;
        m.base = m.list + slots;
        m.place = m.base + slots + 1;
        m.token = m.place + rows;
        m.pair = m.token + 16 * tiles;
        m.weight = (float*)(m.pair + 16 * tiles);
        m.xq = ws + xq;
        m.sx = (float*)(ws + sx);
        m.hq = ws + hq;
        m.sh = (float*)(ws + sh);
        return m;
    }
};

}  // namespace
