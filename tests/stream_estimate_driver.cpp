// Estimated times of the Linear of few rows (fp8_fine_grained_amax_amd/csrc/stream_shape.h) against what no kernel can
// beat: every code of the weight and of the activations read once at the 8 TB/s of an MI355X's memory. With arguments M N K:
// the estimate in us.
#include <stdio.h>
#include <stdlib.h>

#include "stream_shape.h"

int main(int argc, char** argv) {
    if (argc == 4) return printf("%f\n", stream_linear_us(atoll(argv[1]), atoll(argv[2]), atoll(argv[3]))) < 0;
    const int64_t depths[] = {128, 1024, 7168, 16384, 131072, 1 << 24};
    int bad = 0;
    for (int64_t M = 1; M < 2000000; M += M / 3 + 1)
        for (int64_t N = 1; N < 70000; N += N / 3 + 1)
            for (int64_t K : depths) {
                const double us = stream_linear_us(M, N, K), least = ((double)M + (double)N) * (double)K / 8e6;
                if (us >= least || bad++ > 10) continue;
                printf("M %lld N %lld K %lld: estimated %.2f us, %.2f at the memory's peak\n", (long long)M, (long long)N, (long long)K, us, least);
            }
    printf("%d estimates too low\n", bad);
    return bad != 0;
}
