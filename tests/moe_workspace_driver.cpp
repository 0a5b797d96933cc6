// The workspace arithmetic of the mixture of experts (fp8_fine_grained_amax_amd/csrc/moe_workspace.h) over every width, also
// those that the entry point refuses, with the checks of the integer operations that the compiler can add: no call divides
// by zero or overflows, and the parts that any number of experts' launches write lie inside the bytes asked for.
#include <stdio.h>
#include <stdlib.h>

#include "moe_workspace.h"

static int g_failures = 0;
static void expect(bool ok, const char* what, int64_t T, int topk, int64_t E, int64_t H, int64_t I) {
    if (ok || g_failures++ > 20) return;
    printf("%s: T %lld topk %d E %lld H %lld I %lld\n", what, (long long)T, topk, (long long)E, (long long)H, (long long)I);
}

static void one(int64_t T, int topk, int64_t H, int64_t I) {
    const MoeWorkspace at(T, topk, H, I);
    expect(at.bytes >= 0 && at.partial == T * topk * I * 4, "sizes", T, topk, 0, H, I);
    expect(T <= kFusedTokens || at.bytes <= at.partial + kMaxSplits * T * H * 4 + 4 * (2 + 51 * at.slots + 5 * at.rows) + 32 + T * H +
                                                T * (H / 128) * 4 + at.tiles * 16 * I + at.tiles * 16 * (I / 128) * 4,
           "no more than the parts", T, topk, 0, H, I);
    if (H % 128 != 0 || I % 128 != 0) return;
    expect(at.partial % 16 == 0 && at.plan % 16 == 0 && at.xq % 16 == 0 && at.sx % 16 == 0 && at.hq % 16 == 0 && at.sh % 16 == 0,
           "alignment", T, topk, 0, H, I);
    if (T > kFusedTokens) {
        const MoePlan m = at.of((uint8_t*)(uintptr_t)4096);
        auto off = [](const void* p) { return (int64_t)(uintptr_t)p - 4096; };
        expect(off(m.used) == at.plan && off(m.list) >= at.plan + 4 && off(m.base) >= off(m.list) + 4 * at.slots &&
                   off(m.place) >= off(m.base) + 4 * (at.slots + 1) && off(m.token) >= off(m.place) + 4 * at.rows &&
                   off(m.pair) >= off(m.token) + 64 * at.tiles && off(m.weight) >= off(m.pair) + 64 * at.tiles &&
                   at.xq >= off(m.weight) + 64 * at.tiles && at.sx >= at.xq + T * H && at.hq >= at.sx + T * (H / 128) * 4 &&
                   at.sh >= at.hq + at.tiles * 16 * I && at.bytes >= at.sh + at.tiles * 16 * (I / 128) * 4,
               "parts of the plan", T, topk, 0, H, I);
    }
    // every number of experts: the partial sums end before the plan begins, the slots and their tiles fit
    for (int64_t E = 1; E <= 32 * kWords; E += E < 80 ? 1 : 61) {
        const MoeLaunch l(T, topk, E, H, I);
        expect(l.slots <= at.slots && l.splits >= 1 && l.splits <= kMaxSplits && (l.tiles == 1 || l.tiles == 2), "launch", T, topk, E, H, I);
        expect(l.splits == 1 || at.partial + l.splits * T * H * 4 <= at.plan, "splits", T, topk, E, H, I);
        // slots with at least one and together `rows` tokens take at most this many tiles of 16
        expect(l.slots + at.rows / 16 <= at.tiles, "tiles", T, topk, E, H, I);
    }
}

int main() {
    const int64_t tokens[] = {0, 1, 2, 8, 15, 16, 17, 33, 64};
    const int choices[] = {1, 2, 3, 8, 32};
    const int64_t far[] = {(1 << 20) - 1, 1 << 20};
    for (int64_t T : tokens)
        for (int topk : choices) {
            for (int64_t H = 0; H <= 300; H++)
                for (int64_t I = 0; I <= 300; I += H % 128 == 0 ? 1 : 37) one(T, topk, H, I);
            for (int64_t H = 0; H <= 8192; H += 128)
                for (int64_t I = 0; I <= 8192; I += 1024) one(T, topk, H, I + (H % 1024));
            for (int64_t H : far)
                for (int64_t I : far) one(T, topk, H, I);
        }
    if (g_failures) return 1;
    printf("moe workspace driver done\n");
    return 0;
}
