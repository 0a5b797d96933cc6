// Orthogonalised update by Newton-Schulz products (gfx950): A = X X^T, B = a I + b A + c A A, X = B X, a few times over.
//
// Three products a step, m x m x n, m x m x m and m x n x m with m the smaller side, bound by the matrix cores. Operands
// are fp16: bf16's 8 bits make an update 1e-2 off, fp16's 11 bits 1.3e-3 (simulated, 768 x 2048), at the same rate, and the
// range suffices, since |X| <= 1 at the start and the steps keep its singular values below about 1.2. X is held times
// 2^12, whose entries of a large matrix would be denormal otherwise (1e-4), A and B times 2^11 (|B| stays below 30).
// With a I inside B, a and B's diagonal share a rounding; a X beside B X instead is a little less exact where gradients have many
// independent tokens (simulated: 512 x 512 1.31e-3 against 1.23e-3, 256 x 1024 1.47e-3 and 1.09e-3) and more where X X^T is
// diagonal (1.5e-3 and 2.0e-3), and reading X once more at every tile's end took 14 us a round of 256 x 256 tiles.
//
// X X^T and A A (A is symmetric) are products of rows with rows (C[i][j] = sum_k P[i][k] Q[j][k]); they compute the tiles on and
// below the diagonal and write each one twice. B X takes X as it lies: the transposing LDS read turns it on its way into the
// registers, at the same number of bytes a cycle. (From a transposed copy of X, which every product wrote beside
// X itself: 8 x 2048 x 7168 4.02 ms against 3.85, 7168 x 18432 12.67 and 12.44, 512 x 1024 by 8 155 us and 144.)
// Contractions are padded with zeros to multiples of 64.
#include "host_util.h"
#include "mfma_tile.h"
#include "ortho_shape.h"
#include "train_launch.h"

#include <algorithm>
#include <type_traits>

namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int BK = 64;                           // a K step: 128 bytes of a row
constexpr float kScaleX = 4096.0f, kScaleA = 2048.0f;
constexpr int kNormParts = 256;                  // partial sums of a matrix's squares, at most

int64_t pad(int64_t v) { return (v + BK - 1) / BK * BK; }
int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

// A step's products. A and B are symmetric and write each tile twice. The last X leaves as bf16 without padding; the others are
// fp16 with zeros up to their strides. Each has kernels of its own: a small product's time is mostly that of code that
// runs once, and a kernel for all of them has twice as much of it.
enum Product { PRODUCT_A, PRODUCT_B, PRODUCT_X, PRODUCT_LAST };
constexpr bool symmetric(Product P) { return P == PRODUCT_A || P == PRODUCT_B; }

// C = alpha P Q^T of every matrix of a batch; in B, where Q is P, beta P + diag I beside it, and in the last product times beta. A launch begins with the arguments' way
// from the host's memory: 168 bytes of them instead of 104 cost a small product 0.1 to 0.2 us.
struct OrthoGemm {
    const uint16_t *p, *q;                       // fp16 [M][ld]; of A and B [N][ld], of X [ld][ld_q]
    uint16_t* out;                               // [M][ld_out], or turned [N][ld_out]
    int64_t p_batch, q_batch, out_batch;
    int ld, ld_q, ld_out, M, N;
    float alpha, beta, diag;
    int first, count;                            // the 256 x 256 tiles to compute, on tiles of 128 in quarters; count 0: everything
    int turned;                                  // of the last product only
    int tiles, m_tiles;                          // of a matrix, and rows of them; tiles of 256 with a count
};

typedef short v4s __attribute__((ext_vector_type(4)));
// The transposing read. (restrict: without it the compiler waits for all loads to LDS before each.)
__device__ __forceinline__ v2i tr_read(const uint8_t* __restrict__ lds) {
    return __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)lds));
}

// Tile number id (below 2^24) of a lower triangle, row by row: the root is off by one at most.
__device__ __forceinline__ void triangle(int id, int& i, int& j) {
    i = (int)((__builtin_amdgcn_sqrtf(8.0f * (float)id + 1.0f) - 1.0f) * 0.5f);
    i -= i * (i + 1) / 2 > id;
    i += (i + 1) * (i + 2) / 2 <= id;
    j = id - i * (i + 1) / 2;
}
// Matrix and tile number id of a batch; of a symmetric product's lower triangle.
template <Product P>
__device__ __forceinline__ void plain_tile(const OrthoGemm& p, int id, int64_t& batch, int& ti, int& tj) {
    const int b = id / p.tiles, local = id - b * p.tiles;
    batch = b;
    if constexpr (symmetric(P)) {
        triangle(local, ti, tj);
    } else {
        tj = local / p.m_tiles;
        ti = local - tj * p.m_tiles;
    }
}

// Byte of 16-byte chunk c of a row below 16 in a stage. An operand of 16 rows and 32 of the 64 values has row l % 16 and eight of
// them in lane l: the chunks 2 (l / 16) in one operand and 2 (l / 16) + 1 in the other, for both sides alike. (The order of a
// contraction is free. With l / 16 and l / 16 + 4 every read had a two-way bank conflict, 5% of the time.)
__device__ __forceinline__ int frag_at(int row, int c) { return row * 128 + ((c ^ swz128(row)) << 4); }

// The second operand as it lies in X: a stage holds 64 rows (of the contraction) of BN columns, with the pairs of 16-byte chunks
// XORed with bits of the row, so that the eight rows that 32 lanes read at once lie in different banks: the rows 4 i .. + 3 and
// those 16 further on.
template <int BN>
__device__ __forceinline__ int turn_pair(int k) { return BN == 64 ? (k >> 1 & 1) | (k >> 4 & 1) << 1 : (k & 3) | (k >> 4 & 1) << 2; }

// Byte of the second operand that a lane loads for the 1024 bytes number f of a stage, from the tile's first row or column in the
// K step on; past the end the last again.
template <Product P, int BN>
__device__ __forceinline__ uint32_t q_offset(const OrthoGemm& p, int n0, int f, int lane) {
    if constexpr (symmetric(P)) {
        const int row = f * 8 + (lane >> 3), r = n0 + row < p.N ? row : p.N - 1 - n0;
        return (uint32_t)r * (uint32_t)(p.ld * 2) + (((lane & 7) ^ swz128(row)) << 4);
    } else {
        constexpr int CH = BN / 8;
        const int row = f * (64 / CH) + lane / CH, c = 8 * ((lane % CH) ^ (2 * turn_pair<BN>(row))), last = p.ld_q - 8 - n0;
        return (uint32_t)row * (uint32_t)(p.ld_q * 2) + 2 * (uint32_t)(c < last ? c : last);
    }
}
// The tile's part of the second operand, and the bytes from a K step of it to the next.
template <Product P>
__device__ __forceinline__ const uint8_t* q_first(const OrthoGemm& p, int64_t batch, int n0) {
    return (const uint8_t*)(symmetric(P) ? p.p + batch * p.p_batch + (int64_t)n0 * p.ld : p.q + batch * p.q_batch + n0);
}
template <Product P>
__device__ __forceinline__ int64_t q_step(const OrthoGemm& p) { return symmetric(P) ? 2 * BK : 2 * BK * (int64_t)p.ld_q; }

// Where a lane finds the operand of 16 columns, first / 16 + j of the tile, in a stage, and the operand's eight values of half h.
template <Product P, int BN>
__device__ __forceinline__ int q_at(int first, int j, int lane) {
    const int lrow = lane & 15, g16 = lane >> 4;
    if constexpr (symmetric(P)) return (first + 16 * j) * 128 + frag_at(lrow, 2 * g16);
    const int k = 16 * g16 + (lrow >> 2);
    return k * (2 * BN) + ((((first / 16 + j) ^ turn_pair<BN>(k)) * 2 + (lrow >> 1 & 1)) << 4) + (lrow & 1) * 8;
}
template <Product P, int BN>
__device__ __forceinline__ v8h read_q(const uint8_t* st, int at, int h) {
    if constexpr (symmetric(P)) return *reinterpret_cast<const v8h*>(st + (at ^ (h << 4)));
    const v2i a = tr_read(st + at + h * 8 * (2 * BN)), b = tr_read(st + at + (h * 8 + 4) * (2 * BN));
    return __builtin_bit_cast(v8h, v4i{a.x, a.y, b.x, b.y});
}

// The 256 x 256 tile number id of a batch.
template <Product P>
__device__ __forceinline__ void big_tile(const OrthoGemm& p, int id, int64_t& batch, int& ti, int& tj) {
    const int b = id / p.tiles, local = id - b * p.tiles;
    batch = b;
    if constexpr (symmetric(P)) {
        triangle(local, ti, tj);
    } else {
        constexpr int GM = 8;                            // rows of tiles that an XCD's run goes down together
        const int m_tiles = p.m_tiles, n_tiles = (p.N + 255) / 256;
        const int group = local / (GM * n_tiles), first = group * GM, rows = min(m_tiles - first, GM), within = local - group * GM * n_tiles;
        ti = first + within % rows;
        tj = within / rows;
    }
}

template <class T>
__device__ __forceinline__ uint32_t half_bits(float v) { return (uint32_t)__builtin_bit_cast(unsigned short, (T)v); }

// P's elements at the places of a wave's 16 x 16 tiles of B, four to a lane, loaded together (in bounds). (wr, wc): the wave's first row and column
// in the workgroup's tile.
template <Product P, int MSUB, int NSUB>
__device__ __forceinline__ void load_e(const OrthoGemm& p, uint2 (&w)[MSUB][NSUB], int64_t batch, int m0, int n0, int wr, int wc) {
    if constexpr (P != PRODUCT_B) return;
    const int lane = threadIdx.x & 63;
    const uint16_t* e = p.p + batch * p.p_batch + (int64_t)m0 * p.ld;
#pragma unroll
    for (int i = 0; i < MSUB; i++) {
        const int r = wr + 16 * i + (lane & 15);
        const uint32_t row = (uint32_t)(m0 + r < p.M ? r : p.M - 1 - m0) * (uint32_t)p.ld;
#pragma unroll
        for (int j = 0; j < NSUB; j++) {
            const int n = n0 + wc + 16 * j + 4 * (lane >> 4);
            w[i][j] = *reinterpret_cast<const uint2*>(e + (row + (uint32_t)(n < p.ld ? n : 0)));
        }
    }
}

// The end of a workgroup's tile (`diagonal`: of a symmetric product, on the diagonal): alpha acc and what B adds, stored in rows and, turned, in columns. Lane l holds row l % 16 and columns
// 4 (l / 16) .. + 3 of every 16 x 16 tile. The finished tile goes through an LDS image [BM rows][BN / 8 chunks of 8], chunk c
// of row r at c ^ (r % 16) (% 8 with 64 columns), which is read in rows, and in columns by the transposing read: 16 lanes
// read 4 rows x 16 columns, four columns a lane, and each gets one column's four rows.
template <Product P, int BM, int BN, int THREADS, int MSUB, int NSUB>
__device__ __forceinline__ void finish(const OrthoGemm& p, const v4f (&acc)[MSUB][NSUB], const uint2 (&w)[MSUB][NSUB], uint8_t* smem,
                                       int64_t batch, int m0, int n0, int wr, int wc, bool diagonal) {
    constexpr int MIX = BN / 8 < 16 ? BN / 8 - 1 : 15;
    constexpr bool LAST = P == PRODUCT_LAST;
    using T = std::conditional_t<LAST, __bf16, _Float16>;
    const int tid = threadIdx.x, lane = tid & 63, lrow = lane & 15, g16 = lane >> 4;
    [[maybe_unused]] const float diag = diagonal ? p.diag : 0.0f;
#pragma unroll
    for (int i = 0; i < MSUB; i++) {
        const int r = wr + 16 * i + lrow, m = m0 + r;
#pragma unroll
        for (int j = 0; j < NSUB; j++) {
            const int c = wc + 16 * j + 4 * g16, n = n0 + c;
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                v[k] = p.alpha * acc[i][j][k];
                if constexpr (LAST) v[k] *= p.beta;            // the caller's factor: times alpha it may be denormal
                if constexpr (P == PRODUCT_B) {
                    const uint32_t h = k & 2 ? w[i][j].y : w[i][j].x;
                    const float old = (float)__builtin_bit_cast(_Float16, (unsigned short)(k & 1 ? h >> 16 : h));
                    v[k] = __builtin_fmaf(p.beta, old, v[k]) + (m == n + k ? diag : 0.0f);
                }
                if (!LAST && (m >= p.M || n + k >= p.N)) v[k] = 0.0f;      // padding
            }
            *reinterpret_cast<uint2*>(smem + r * (2 * BN) + (((c >> 3) ^ (r & MIX)) << 4) + ((c >> 2) & 1) * 8) =
                make_uint2(half_bits<T>(v[0]) | (half_bits<T>(v[1]) << 16), half_bits<T>(v[2]) | (half_bits<T>(v[3]) << 16));
        }
    }
    __syncthreads();
    // 8 values to a lane; `width`: columns that are there. Without padding rows may begin anywhere.
    auto store = [&](uint16_t* row, int c, int width, uint4 v) {
        if (LAST && ((p.ld_out & 7) || ((uintptr_t)row & 15) || c + 8 > width)) {
            const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 8; k++)
                if (c + k < width) row[c + k] = (uint16_t)(h[k >> 1] >> (16 * (k & 1)));
        } else if (c < width) {
            *reinterpret_cast<uint4*>(row + c) = v;
        }
    };
    if (P != PRODUCT_LAST || !p.turned) {
        constexpr int CH = BN / 8;
        uint16_t* out = p.out + batch * p.out_batch;
        const int width = LAST ? p.N : p.ld_out;
#pragma unroll 4
        for (int it = 0; it < BM * CH / THREADS; it++) {
            const int f = it * THREADS + tid, r = f / CH, c = f % CH;
            if (m0 + r < p.M)
                store(out + (int64_t)(m0 + r) * p.ld_out, n0 + 8 * c, width, *reinterpret_cast<const uint4*>(smem + r * (2 * BN) + ((c ^ (r & MIX)) << 4)));
        }
    }
    if (LAST ? p.turned : symmetric(P) && !diagonal) {
        constexpr int CH = BM / 8;
        uint16_t* out = p.out + batch * p.out_batch;
        const int width = LAST ? p.M : p.ld_out;
#pragma unroll 4
        for (int it = 0; it < BN * CH / THREADS; it++) {
            const int f = it * THREADS + tid, c0 = f / (16 * CH) * 16, r = 8 * (f / 16 % CH), col = c0 + 4 * (lrow & 3);     // column c0 + lrow, rows r .. r + 7
            v2i part[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int row = r + 4 * h + (lrow >> 2);
                part[h] = tr_read(smem + row * (2 * BN) + (((col >> 3) ^ (row & MIX)) << 4) + ((col >> 2) & 1) * 8);
            }
            const int n = n0 + c0 + lrow;
            if (n < p.N) store(out + (int64_t)n * p.ld_out, m0 + r, width, make_uint4(part[0].x, part[0].y, part[1].x, part[1].y));
        }
    }
}

// ------------------------------------------------------------------------------------------------
// 128 x 128 x 64 workgroup tiles: 4 waves (2 x 2) of 64 x 64, STAGES K steps in flight (loads go straight to LDS).
// ------------------------------------------------------------------------------------------------
struct MidTile {
    static constexpr int NTHREADS = 256, BM = 128, BN = 128, SUB = 4, STAGE = (BM + BN) * 128, LOADS = 8;
};

// SPLIT: as small_tile's.
template <Product P, int STAGES, bool SPLIT>
__device__ __forceinline__ void mid_tile(const OrthoGemm& p, v4f* parts, int split) {
    using C = MidTile;
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    int ti, tj, steps = p.ld / BK, part_id = 0, k0 = 0, nkb = steps;
    int64_t batch;
    if constexpr (SPLIT) {
        part_id = xcd_remap((int)blockIdx.x, (int)gridDim.x);
        const int all = (int)gridDim.x / split, part = part_id / all;
        plain_tile<P>(p, part_id - part * all, batch, ti, tj);
        k0 = part * steps / split;
        nkb = (part + 1) * steps / split - k0;
    } else if (p.count) {                                       // quarters of 256 x 256 tiles
        const int id = xcd_remap((int)blockIdx.x, (int)gridDim.x);
        big_tile<P>(p, p.first + (id >> 2), batch, ti, tj);
        ti = 2 * ti + (id >> 1 & 1);
        tj = 2 * tj + (id & 1);
        if (ti * C::BM >= p.M || tj * C::BN >= p.N || (symmetric(P) && tj > ti)) return;
    } else {
        plain_tile<P>(p, xcd_remap((int)blockIdx.x, (int)gridDim.x), batch, ti, tj);
    }
    const int m0 = ti * C::BM, n0 = tj * C::BN;
    const uint8_t* pp = (const uint8_t*)(p.p + batch * p.p_batch + (int64_t)m0 * p.ld) + k0 * 128;
    const uint8_t* qp = q_first<P>(p, batch, n0) + k0 * q_step<P>(p);

    uint32_t a_off[4], b_off[4];
#pragma unroll
    for (int u = 0; u < 4; u++) {
        const int row = (wave + 4 * u) * 8 + (lane >> 3), rm = m0 + row < p.M ? row : p.M - 1 - m0;    // past the end: the last again
        a_off[u] = (uint32_t)rm * (uint32_t)(p.ld * 2) + (((lane & 7) ^ swz128(row)) << 4);
        b_off[u] = q_offset<P, C::BN>(p, n0, wave + 4 * u, lane);
    }
    auto issue = [&](int kb, int slot) {
        const int k = kb < nkb ? kb : nkb - 1;
        uint8_t* st = smem + slot * C::STAGE;
        const auto ra = fg_buffer_rsrc(pp + (int64_t)k * 128), rb = fg_buffer_rsrc(qp + k * q_step<P>(p));
#pragma unroll
        for (int u = 0; u < 4; u++) {
            fg_buffer_load_lds16(ra, st + (wave + 4 * u) * 1024, a_off[u]);
            fg_buffer_load_lds16(rb, st + C::BM * 128 + (wave + 4 * u) * 1024, b_off[u]);
        }
    };
    const int lrow = lane & 15, g16 = lane >> 4;
    const int frag[2] = {frag_at(lrow, 2 * g16), frag_at(lrow, 2 * g16 + 1)};
    int q_frag[C::SUB];
#pragma unroll
    for (int j = 0; j < C::SUB; j++) q_frag[j] = q_at<P, C::BN>(wn * 64, j, lane);
    v8h af[2][C::SUB][2], bf[2][C::SUB][2];
    auto read = [&](int kb, int set) {
        const uint8_t* st = smem + (kb & (STAGES - 1)) * C::STAGE;
#pragma unroll
        for (int i = 0; i < C::SUB; i++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                af[set][i][h] = *reinterpret_cast<const v8h*>(st + (wm * 64 + 16 * i) * 128 + frag[h]);
                bf[set][i][h] = read_q<P, C::BN>(st + C::BM * 128, q_frag[i], h);
            }
    };
    v4f acc[C::SUB][C::SUB];
#pragma unroll
    for (int i = 0; i < C::SUB; i++)
#pragma unroll
        for (int j = 0; j < C::SUB; j++) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    uint2 e[C::SUB][C::SUB];
    if constexpr (!SPLIT) load_e<P>(p, e, batch, m0, n0, wm * 64, wn * 64);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < STAGES; s++) issue(s, s);
    wait_loads<(STAGES - 1) * C::LOADS>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(0, 0);
    // The barrier of step kb says that every wave's part of stage kb + 1 has landed and that stage kb's operands are read,
    // so its slot takes stage kb + STAGES. Every step issues the same loads (past the end the last block's again, into a slot
    // that nobody reads).
    auto step = [&](int kb, auto set_tag) {
        constexpr int set = decltype(set_tag)::value;
        __builtin_amdgcn_sched_barrier(0);
        wait_loads<(STAGES - 2) * C::LOADS>();
        __builtin_amdgcn_s_waitcnt(0xC07F);             // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        issue(kb + STAGES, kb & (STAGES - 1));
        read(kb + 1, set ^ 1);
#pragma unroll
        for (int t = 0; t < C::SUB * C::SUB; t++) {
            const int i = t / C::SUB, j = t % C::SUB;
#pragma unroll
            for (int h = 0; h < 2; h++) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(bf[set][j][h], af[set][i][h], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);   // two MFMAs
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // an LDS read of the next step's operands, of X's two to each
            if (!symmetric(P) && t % 2 == 0) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
    };
    int kb = 0;
    for (; kb + 1 < nkb; kb += 2) {
        step(kb, std::integral_constant<int, 0>{});
        step(kb + 1, std::integral_constant<int, 1>{});
    }
    if (kb < nkb) step(kb, std::integral_constant<int, 0>{});
    __builtin_amdgcn_s_waitcnt(0);
    if constexpr (SPLIT) {                              // a wave's 64 x 64
        v4f* to = parts + ((int64_t)part_id * 4 + wave) * 1024 + lane;
#pragma unroll
        for (int t = 0; t < C::SUB * C::SUB; t++) to[t * 64] = acc[t / C::SUB][t % C::SUB];
    } else {
        __syncthreads();                                // the stages are free
        finish<P, C::BM, C::BN, C::NTHREADS>(p, acc, e, smem, batch, m0, n0, wm * 64, wn * 64, symmetric(P) && ti == tj);
    }
}
template <Product P, int STAGES>
__global__ __launch_bounds__(MidTile::NTHREADS, 4 / STAGES) void fg_ortho_mid_kernel(OrthoGemm p) { mid_tile<P, STAGES, false>(p, nullptr, 1); }

// ------------------------------------------------------------------------------------------------
// 256 x 256 x 64 workgroup tiles: 8 waves (2 x 4) of 128 x 64, two on a SIMD, which take turns: while one issues 32 MFMAs (half
// of its tile's K step, 64 x 64), the other reads its next operands from LDS and issues loads. Two barriers a half keep
// them apart; the waves of the second group are one barrier behind.
//
// The halves are (A0, B) and (A1, B): B's operands are read once a step, and so is each half of A's. Two stages of 64 KB: what both
// groups have read is loaded over at once, A0 and B with the step after next's (in the second half's turn), A1 with the next
// step's (in the first half's), so that a load has at least two of a step's four turns to land. What a half reads is waited
// for in the turn before, in front of a barrier; loads return in order, so the counts of those that may be outstanding are
// fixed: A0 and B are 6 loads of a wave, A1 2. Past the end every step loads the last block again, into a slot that nobody reads:
// asking for the end cost 1.5%.
//
// Measured: B X of 7168 x 18432, 1.33 to 1.45 ms by the gradient's values, 1310 to 1426 TFLOP/s (torch's fp16 product of these
// sizes 1.37 ms). The matrix cores are busy 81% of the cycles at about 1.7 GHz, which the chip's power leaves them; at 8 x 2048 x
// 7168 66% at 1.8 GHz, 1240 TFLOP/s: there a tile has 32 K steps between its first loads and last stores. Turns of 16 MFMAs
// (quarters, half the reads a turn) took 10% longer, MFMAs of 32 x 32 5% (fewer cycles, a lower clock).
// ------------------------------------------------------------------------------------------------
struct BigTile {
    static constexpr int NTHREADS = 512, BM = 256, BN = 256, MSUB = 8, NSUB = 4, STAGE = (BM + BN) * 128, LDS = 2 * STAGE;
};

// SPLIT: as small_tile's.
template <Product P, bool SPLIT>
__device__ __forceinline__ void large_tile(const OrthoGemm& p, v4f* parts, int split) {
    using C = BigTile;
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    int64_t batch;
    int ti, tj;
    const int id = xcd_remap((int)blockIdx.x, (int)gridDim.x), all = SPLIT ? (int)gridDim.x / split : 0, part = SPLIT ? id / all : 0;
    big_tile<P>(p, SPLIT ? id - part * all : id, batch, ti, tj);
    const int steps = p.ld / BK, k0 = SPLIT ? part * steps / split : 0, nkb = SPLIT ? (part + 1) * steps / split - k0 : steps;
    const int m0 = ti * C::BM, n0 = tj * C::BN;
    const uint8_t* pp = (const uint8_t*)(p.p + batch * p.p_batch + (int64_t)m0 * p.ld) + k0 * 128;
    const uint8_t* qp = q_first<P>(p, batch, n0) + k0 * q_step<P>(p);

    // Loads: an instruction fills 8 rows of 128 bytes. A0 is rows [0, 64) and [128, 192) of the tile; a wave loads 16 rows of
    // each half and four parts of B.
    auto a_row = [&](int half, int u) { return (wave >> 2) * 128 + half * 64 + (wave & 3) * 16 + u * 8; };
    auto b_part = [&](int half, int u) { return (wave >> 1) * 8 + half * 4 + (wave & 1) * 2 + u; };
    uint32_t a_off[2][2], b_off[2][2];
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const int ra = a_row(h, u) + (lane >> 3), rm = m0 + ra < p.M ? ra : p.M - 1 - m0;    // past the end: the last again
            a_off[h][u] = (uint32_t)rm * (uint32_t)(p.ld * 2) + (((lane & 7) ^ swz128(ra)) << 4);
            b_off[h][u] = q_offset<P, C::BN>(p, n0, b_part(h, u), lane);
        }
    auto load_a = [&](int kb, int half) {
        const auto rs = fg_buffer_rsrc(pp + (int64_t)(kb < nkb ? kb : nkb - 1) * 128);
#pragma unroll
        for (int u = 0; u < 2; u++) fg_buffer_load_lds16(rs, smem + (kb & 1) * C::STAGE + a_row(half, u) * 128, a_off[half][u]);
    };
    auto load_b = [&](int kb, int half) {
        const auto rs = fg_buffer_rsrc(qp + (kb < nkb ? kb : nkb - 1) * q_step<P>(p));
#pragma unroll
        for (int u = 0; u < 2; u++) fg_buffer_load_lds16(rs, smem + (kb & 1) * C::STAGE + C::BM * 128 + b_part(half, u) * 1024, b_off[half][u]);
    };

    const int lrow = lane & 15, g16 = lane >> 4;
    const int frag[2] = {frag_at(lrow, 2 * g16), frag_at(lrow, 2 * g16 + 1)};
    int q_frag[C::NSUB];
#pragma unroll
    for (int j = 0; j < C::NSUB; j++) q_frag[j] = q_at<P, C::BN>(wn * 64, j, lane);
    v8h af[4][2], bf[C::NSUB][2];                        // a half of A's 16-row operands, and B's
    auto read_a = [&](int kb, int half) {
        const uint8_t* st = smem + (kb & 1) * C::STAGE + (wm * 128 + half * 64) * 128;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int h = 0; h < 2; h++) af[i][h] = *reinterpret_cast<const v8h*>(st + 16 * i * 128 + frag[h]);
    };
    auto read_b = [&](int kb) {
        const uint8_t* st = smem + (kb & 1) * C::STAGE + C::BM * 128;
#pragma unroll
        for (int j = 0; j < C::NSUB; j++)
#pragma unroll
            for (int h = 0; h < 2; h++) bf[j][h] = read_q<P, C::BN>(st, q_frag[j], h);
    };
    v4f acc[C::MSUB][C::NSUB];
#pragma unroll
    for (int i = 0; i < C::MSUB; i++)
#pragma unroll
        for (int j = 0; j < C::NSUB; j++) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    // The turn of the matrix cores: the operands are there (lgkmcnt), and so is what the next turn reads, on every wave.
    auto multiply = [&](int half) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < C::NSUB; j++)
                    acc[4 * half + i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(bf[j][h], af[i][h], acc[4 * half + i][j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    auto load_first = [&](int kb) {
        load_a(kb, 0);
        load_b(kb, 0);
        load_b(kb, 1);
    };
    load_first(0);
    load_a(0, 1);
    load_first(1);
    wait_loads<8>();
    __builtin_amdgcn_s_barrier();
    if (wm == 1) __builtin_amdgcn_s_barrier();           // the second group
    __builtin_amdgcn_sched_barrier(0);
    for (int kb = 0; kb < nkb; kb++) {
        read_b(kb);
        read_a(kb, 0);
        load_a(kb + 1, 1);
        wait_loads<8>();                                 // A1 of this step
        multiply(0);
        read_a(kb, 1);
        load_first(kb + 2);
        wait_loads<8>();                                 // A0 and B of the next step
        multiply(1);
    }
    if (wm == 0) __builtin_amdgcn_s_barrier();           // every wave passes the same number of barriers
    __builtin_amdgcn_s_waitcnt(0);
    if constexpr (SPLIT) {                               // a wave's 128 x 64
#pragma unroll
        for (int i = 0; i < C::MSUB; i++) {
            v4f* to = parts + ((int64_t)id * 16 + (2 * wm + i / 4) * 4 + wn) * 1024 + i % 4 * (C::NSUB * 64) + lane;
#pragma unroll
            for (int j = 0; j < C::NSUB; j++) to[j * 64] = acc[i][j];
        }
    } else {
        __syncthreads();                                 // the stages are free
        uint2 e[C::MSUB][C::NSUB];
        load_e<P>(p, e, batch, m0, n0, wm * 128, wn * 64);
        finish<P, C::BM, C::BN, C::NTHREADS>(p, acc, e, smem, batch, m0, n0, wm * 128, wn * 64, symmetric(P) && ti == tj);
    }
}
template <Product P>
__global__ __launch_bounds__(BigTile::NTHREADS, 1) void fg_ortho_big_kernel(OrthoGemm p) { large_tile<P, false>(p, nullptr, 1); }

// ------------------------------------------------------------------------------------------------
// 64 x 64 workgroup tiles for small matrices: 4 waves, each with a quarter of the contraction (every fourth K step) for the whole
// tile and stages of its own, so that nothing waits for another wave before the sums are joined, in LDS and in the order of
// the waves. A CU loads at about 80 to 95 GB/s, and that bounds the K steps: two stages a wave (SLOTS) gain at most 8% over
// one, which leaves room for a second workgroup on a CU: two stages and one, 1000 x 1000 x 2001, 136 tiles, 10.2 and 11.0 us;
// 1000 x 2001 x 1000, 512 tiles, 14.2 and 11.0. The smallest, 256 x 256 x 256, takes 4.9 us, nearly all of it latency: of the launch,
// the first loads, the join and the stores.
// ------------------------------------------------------------------------------------------------
template <int SLOTS_>
struct SmallTile {
    static constexpr int SLOTS = SLOTS_, NTHREADS = 256, WAVES = 4, SIDE = 64, SUB = 4, STAGE = 2 * SIDE * 128, LOADS = 16;
    static constexpr int LDS = SLOTS == 2 ? WAVES * 2 * STAGE : WAVES * STAGE + 8192;
};

// SPLIT: the contraction's part number id / (tiles of all matrices) of `split`. Its sums go to `parts`: [part][64 x 64 tile][16 x 16
// tile][lane], those of a larger tile row by row.
template <Product P, int SLOTS, bool SPLIT>
__device__ __forceinline__ void small_tile(const OrthoGemm& p, v4f* parts, int split) {
    using C = SmallTile<SLOTS>;
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t batch;
    int ti, tj;
    const int id = xcd_remap((int)blockIdx.x, (int)gridDim.x), all = SPLIT ? (int)gridDim.x / split : 0, part = SPLIT ? id / all : 0;
    plain_tile<P>(p, SPLIT ? id - part * all : id, batch, ti, tj);
    const int steps = p.ld / BK, k0 = SPLIT ? part * steps / split : 0, nkb = SPLIT ? (part + 1) * steps / split - k0 : steps;
    const int m0 = ti * C::SIDE, n0 = tj * C::SIDE;
    const uint8_t* pp = (const uint8_t*)(p.p + batch * p.p_batch + (int64_t)m0 * p.ld) + k0 * 128;
    const uint8_t* qp = q_first<P>(p, batch, n0) + k0 * q_step<P>(p);
    uint8_t* ring = smem + wave * (SLOTS * C::STAGE);

    uint32_t a_off[8], b_off[8];
#pragma unroll
    for (int u = 0; u < 8; u++) {
        const int row = u * 8 + (lane >> 3), rm = m0 + row < p.M ? row : p.M - 1 - m0;    // past the end: the last again
        a_off[u] = (uint32_t)rm * (uint32_t)(p.ld * 2) + (((lane & 7) ^ swz128(row)) << 4);
        b_off[u] = q_offset<P, C::SIDE>(p, n0, u, lane);
    }
    auto issue = [&](int kb, int slot) {
        if (kb >= nkb) return;
        const auto ra = fg_buffer_rsrc(pp + (int64_t)kb * 128), rb = fg_buffer_rsrc(qp + kb * q_step<P>(p));
#pragma unroll
        for (int u = 0; u < 8; u++) {
            fg_buffer_load_lds16(ra, ring + slot * C::STAGE + u * 1024, a_off[u]);
            fg_buffer_load_lds16(rb, ring + slot * C::STAGE + C::SIDE * 128 + u * 1024, b_off[u]);
        }
    };
    const int lrow = lane & 15, g16 = lane >> 4;
    const int frag[2] = {frag_at(lrow, 2 * g16), frag_at(lrow, 2 * g16 + 1)};
    int q_frag[C::SUB];
#pragma unroll
    for (int j = 0; j < C::SUB; j++) q_frag[j] = q_at<P, C::SIDE>(0, j, lane);
    v4f acc[C::SUB][C::SUB];
#pragma unroll
    for (int i = 0; i < C::SUB; i++)
#pragma unroll
        for (int j = 0; j < C::SUB; j++) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    uint2 e[1][C::SUB];                                  // of the strip of 16 rows that the wave ends with
    load_e<P>(p, e, batch, m0, n0, 16 * wave, 0);
    __builtin_amdgcn_sched_barrier(0);
    issue(wave, 0);
    if constexpr (SLOTS == 2) issue(wave + C::WAVES, 1);
    int slot = 0;
    for (int kb = wave; kb < nkb; kb += C::WAVES, slot ^= SLOTS - 1) {
        if (SLOTS == 2 && kb + C::WAVES < nkb) wait_loads<C::LOADS>(); // this step's, with the next one's outstanding
        else wait_loads<0>();
        __builtin_amdgcn_sched_barrier(0);
        const uint8_t* st = ring + slot * C::STAGE;
        v8h af[C::SUB][2], bf[C::SUB][2];
#pragma unroll
        for (int i = 0; i < C::SUB; i++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                af[i][h] = *reinterpret_cast<const v8h*>(st + 16 * i * 128 + frag[h]);
                bf[i][h] = read_q<P, C::SIDE>(st + C::SIDE * 128, q_frag[i], h);
            }
        __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0): the slot is read
        __builtin_amdgcn_sched_barrier(0);
        issue(kb + SLOTS * C::WAVES, slot);
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int i = 0; i < C::SUB; i++)
#pragma unroll
                for (int j = 0; j < C::SUB; j++) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(bf[j][h], af[i][h], acc[i][j], 0, 0, 0);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();                                     // the rings are free
    v4f* red = reinterpret_cast<v4f*>(smem);             // [wave][strip][column tile][lane]
#pragma unroll
    for (int i = 0; i < C::SUB; i++)
#pragma unroll
        for (int j = 0; j < C::SUB; j++) red[((wave * C::SUB + i) * C::SUB + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    v4f sum[1][C::SUB];
#pragma unroll
    for (int j = 0; j < C::SUB; j++) {
        sum[0][j] = red[(wave * C::SUB + j) * 64 + lane];
#pragma unroll
        for (int w = 1; w < C::WAVES; w++) sum[0][j] += red[((w * C::SUB + wave) * C::SUB + j) * 64 + lane];
    }
    if constexpr (SPLIT) {
        v4f* to = parts + (int64_t)id * 1024 + wave * (C::SUB * 64) + lane;
#pragma unroll
        for (int j = 0; j < C::SUB; j++) to[j * 64] = sum[0][j];
    } else {
        finish<P, C::SIDE, C::SIDE, C::NTHREADS>(p, sum, e, smem + C::WAVES * 16384, batch, m0, n0, 16 * wave, 0, symmetric(P) && ti == tj);
    }
}
template <Product P, int SLOTS>
__global__ __launch_bounds__(256, 3 - SLOTS) void fg_ortho_small_kernel(OrthoGemm p) { small_tile<P, SLOTS, false>(p, nullptr, 1); }

// A of few tiles and a long contraction: tiles that several workgroups share, as many as there are CUs. 64 x 16384, one tile of 64 x 64
// and 256 K steps: 5.8 us and 3.4 for the sum of 32 parts; with one workgroup 34 us.
// 1536 x 16384 on tiles of 128, three parts each, 60 us instead of 108; 2048 x 16384 on tiles of 256, seven parts, 90 instead of 133.
__global__ __launch_bounds__(256, 1) void fg_ortho_split_kernel(OrthoGemm p, v4f* parts, int split) {
    small_tile<PRODUCT_A, 2, true>(p, parts, split);
}
__global__ __launch_bounds__(256, 1) void fg_ortho_mid_split_kernel(OrthoGemm p, v4f* parts, int split) {
    mid_tile<PRODUCT_A, 4, true>(p, parts, split);
}
__global__ __launch_bounds__(512, 1) void fg_ortho_big_split_kernel(OrthoGemm p, v4f* parts, int split) {
    large_tile<PRODUCT_A, true>(p, parts, split);
}
// The sum of the parts, in their order, and its end: 16 rows of a 64 x 64 tile a workgroup, four columns a thread. `side`: 64 x 64
// tiles to a side of the split ones, 1, 2 or 4.
__global__ __launch_bounds__(256) void fg_ortho_join_kernel(OrthoGemm p, const v4f* __restrict__ parts, int split, int side) {
    __shared__ __attribute__((aligned(16))) uint16_t turned[64][20];     // [column][row]
    const int tid = threadIdx.x, lane = tid & 63, tile = blockIdx.x >> 2, strip = blockIdx.x & 3;
    const int r = lane & 15, c = 16 * (tid >> 6) + 4 * (lane >> 4);
    int64_t batch;
    int ti, tj;
    const int whole = tile / (side * side), within = tile - whole * side * side;
    plain_tile<PRODUCT_A>(p, whole, batch, ti, tj);
    ti = side * ti + within / side;
    tj = side * tj + within % side;
    if (ti * 64 >= p.M || tj > ti) return;               // nothing, or what the tile across the diagonal writes
    const v4f* from = parts + (int64_t)tile * 1024 + strip * 256 + tid;
    const int64_t next = (int64_t)(gridDim.x >> 2) * 1024;
    v4f sum = {0.f, 0.f, 0.f, 0.f};
    int part = 0;
    for (; part + 8 <= split; part += 8) {
        v4f v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = from[(part + i) * next];
#pragma unroll
        for (int i = 0; i < 8; i++) sum += v[i];
    }
    for (; part < split; part++) sum += from[part * next];
    const int m = ti * 64 + strip * 16 + r, n = tj * 64 + c;
    uint32_t h[4];
#pragma unroll
    for (int k = 0; k < 4; k++) h[k] = m < p.M && n + k < p.N ? half_bits<_Float16>(p.alpha * sum[k]) : 0;
    uint16_t* out = p.out + batch * p.out_batch;
    if (m < p.M) *reinterpret_cast<uint2*>(out + (int64_t)m * p.ld_out + n) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    if (ti == tj) return;
#pragma unroll
    for (int k = 0; k < 4; k++) turned[c + k][r] = (uint16_t)h[k];
    __syncthreads();
    const int col = tid >> 2, r4 = 4 * (tid & 3);
    if (tj * 64 + col < p.N)
        *reinterpret_cast<uint2*>(out + (int64_t)(tj * 64 + col) * p.ld_out + ti * 64 + strip * 16 + r4) = *reinterpret_cast<const uint2*>(&turned[col][r4]);
}

// ------------------------------------------------------------------------------------------------
// The start: |G|, then X. Both are bound by HBM: 8 x 2048 x 7168 f32 99 us (4.8 TB/s) and 120 (5.9).
// ------------------------------------------------------------------------------------------------
// Four neighbouring elements of G from element i on, the first `count` of them; `whole`: all four, aligned to their size.
__device__ __forceinline__ v4f load_g(const FgOrtho& p, int64_t i, int64_t count, bool whole) {
    v4f v = {0.f, 0.f, 0.f, 0.f};
    if (whole) {
        if (!p.g_bf16) return *reinterpret_cast<const v4f*>((const float*)p.g + i);
        const uint2 w = *reinterpret_cast<const uint2*>((const uint16_t*)p.g + i);
        return v4f{fg_bf16_lo(w.x), fg_bf16_hi(w.x), fg_bf16_lo(w.y), fg_bf16_hi(w.y)};
    }
#pragma unroll
    for (int k = 0; k < 4; k++)
        if (k < count) v[k] = p.g_bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p.g)[i + k] << 16) : ((const float*)p.g)[i + k];
    return v;
}
// Whether every four elements from a multiple of four columns on may be loaded at once (but those that the row's end cuts).
__device__ __forceinline__ bool fours_aligned(const FgOrtho& p) { return p.ld % 4 == 0 && ((uintptr_t)p.g & (p.g_bf16 ? 7 : 15)) == 0; }

// Sum over a workgroup of WAVES waves, in every thread.
template <int WAVES>
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
    for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; w++) s += red[w];
    return s;
}

// Squares are summed in 64 bits: an fp32 gradient's may leave 32 bits' range either way. Bound by HBM: 512 threads a workgroup,
// four loads of four elements in flight each.
constexpr int kNormThreads = 512;
__global__ __launch_bounds__(kNormThreads) void fg_ortho_norm_kernel(FgOrtho p, double* __restrict__ partial) {
    __shared__ double red[kNormThreads / 64];
    const int64_t batch = blockIdx.y, fours = (p.K + 3) / 4, total = p.N * fours, step = (int64_t)gridDim.x * kNormThreads;
    const int64_t row_step = step / fours, col_step = step % fours;
    const bool aligned = fours_aligned(p);
    int64_t at = (int64_t)blockIdx.x * kNormThreads + threadIdx.x, row = at / fours, col = at % fours;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    while (at < total) {
        v4f v[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
            v[u] = v4f{0.f, 0.f, 0.f, 0.f};
            if (at < total) v[u] = load_g(p, (batch * p.N + row) * p.ld + 4 * col, p.K - 4 * col, aligned && 4 * col + 4 <= p.K);
            at += step;
            row += row_step;
            col += col_step;
            if (col >= fours) {
                col -= fours;
                row++;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; u++)
#pragma unroll
            for (int k = 0; k < 4; k++) s[k] = __builtin_fma((double)v[u][k], (double)v[u][k], s[k]);
    }
    const double sum = block_sum<kNormThreads / 64>((s[0] + s[1]) + (s[2] + s[3]), red);
    if (threadIdx.x == 0) partial[batch * kNormParts + blockIdx.x] = sum;
}

// 64 x 64 elements of G to X, turned where the rows are the longer side, zeros behind the last row and column; behind the last row
// of X the zeros go to the other buffer of X as well, which later steps read and nothing writes there. A thread takes 4 x 4
// elements. WIDE: X is G as it lies.
template <bool WIDE>
__global__ __launch_bounds__(256) void fg_ortho_start_kernel(FgOrtho p, const double* __restrict__ partial, int parts, uint16_t* x,
                                                             uint16_t* other, int64_t rows, int64_t ld) {
    __shared__ double red[4];
    __shared__ __attribute__((aligned(16))) uint16_t tile[WIDE ? 1 : 64][72];       // [column][row]
    const int64_t batch = blockIdx.y, tiles = (p.K + 63) / 64;
    const int64_t r0 = (int64_t)(blockIdx.x / tiles) * 64, c0 = (int64_t)(blockIdx.x % tiles) * 64;
    const int c = 4 * (threadIdx.x & 15), r = 4 * (threadIdx.x >> 4);
    const bool whole = fours_aligned(p) && c0 + c + 4 <= p.K;
    v4f v[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        v[k] = v4f{0.f, 0.f, 0.f, 0.f};
        if (r0 + r + k < p.N) v[k] = load_g(p, (batch * p.N + r0 + r + k) * p.ld + c0 + c, p.K - c0 - c, whole && c0 + c < p.K);
    }
    const double sum = block_sum<4>((int)threadIdx.x < parts ? partial[batch * kNormParts + threadIdx.x] : 0.0, red);
    // |G| + eps in fp32, and in 64 bits where fp32 has too few bits for it or none: X = G 2^-e inv, whose parts are normal numbers
    // whatever the two are (a factor of 1 / 2^-140 alone would be infinite, and 0 times it NaN).
    const float norm = (float)__builtin_sqrt(sum), rounded = norm + p.eps;
    const double divisor = rounded >= 0x1p-126f && rounded < __builtin_inff() ? (double)rounded : __builtin_sqrt(sum) + (double)p.eps;
    const int e = __builtin_amdgcn_frexp_exp(divisor);
    const float inv = norm < __builtin_inff() ? (float)(1.0 / __builtin_amdgcn_ldexp(divisor, -e)) : __builtin_nanf("");
    uint32_t h[4][4];
#pragma unroll
    for (int k = 0; k < 4; k++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const bool there = r0 + r + k < p.N && c0 + c + j < p.K;     // a factor of NaN leaves the padding 0
            h[k][j] = there ? half_bits<_Float16>(__builtin_amdgcn_ldexpf(v[k][j], -e) * inv * kScaleX) : 0;
        }
    const int64_t m = WIDE ? p.N : p.K;
    x += batch * rows * ld;
    other += batch * rows * ld;
    auto put = [&](int64_t row, int64_t col, uint2 w) {
        *reinterpret_cast<uint2*>(x + row * ld + col) = w;
        if (row >= m) *reinterpret_cast<uint2*>(other + row * ld + col) = w;
    };
    if constexpr (WIDE) {
#pragma unroll
        for (int k = 0; k < 4; k++) put(r0 + r + k, c0 + c, make_uint2(h[k][0] | (h[k][1] << 16), h[k][2] | (h[k][3] << 16)));
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++) *reinterpret_cast<uint2*>(&tile[c + k][r]) = make_uint2(h[0][k] | (h[1][k] << 16), h[2][k] | (h[3][k] << 16));
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int col = (threadIdx.x >> 4) + 16 * k, row = 4 * (threadIdx.x & 15);
            put(c0 + col, r0 + row, *reinterpret_cast<const uint2*>(&tile[col][row]));
        }
    }
}

template <class Tile, class Kernel>
hipError_t launch(Kernel kern, int64_t tiles, int lds, std::atomic<uint64_t>& limit_set, const OrthoGemm& p, hipStream_t stream) {
    const hipError_t e = fg_set_lds_limit_once((const void*)kern, lds, limit_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)tiles), dim3(Tile::NTHREADS), lds, stream, p);
    return hipGetLastError();
}

template <Product P>
hipError_t launch_tile(OrthoTile tile, const OrthoGemm& all, int64_t batch, hipStream_t stream) {
    static std::atomic<uint64_t> limits[5];
    const int side = tile == TILE_64 ? 64 : tile == TILE_256 || all.count ? 256 : 128;
    OrthoGemm p = all;
    p.tiles = (int)ortho_tiles(1, p.M, p.N, symmetric(P), side);
    p.m_tiles = (p.M + side - 1) / side;
    const int64_t tiles = p.tiles * batch, mid = p.count ? 4 * (int64_t)p.count : tiles;
    switch (tile) {
        case TILE_64:
            if (tiles <= fg_device_cus())
                return launch<SmallTile<2>>(fg_ortho_small_kernel<P, 2>, tiles, SmallTile<2>::LDS, limits[0], p, stream);
            return launch<SmallTile<1>>(fg_ortho_small_kernel<P, 1>, tiles, SmallTile<1>::LDS, limits[1], p, stream);
        case TILE_128: return launch<MidTile>(fg_ortho_mid_kernel<P, 4>, mid, 4 * MidTile::STAGE, limits[2], p, stream);
        case TILE_128_PAIRS: return launch<MidTile>(fg_ortho_mid_kernel<P, 2>, mid, 2 * MidTile::STAGE, limits[3], p, stream);
        default: return launch<BigTile>(fg_ortho_big_kernel<P>, p.count ? p.count : tiles, BigTile::LDS, limits[4], p, stream);
    }
}

// parts: what the product does not use otherwise of the workspace, parts_bytes of it.
template <Product P>
hipError_t launch_gemm(const OrthoGemm& p, int64_t batch, hipStream_t stream, void* parts = nullptr, int64_t parts_bytes = 0) {
    const int64_t cus = fg_device_cus();
    if constexpr (P == PRODUCT_A) {
        const OrthoSplit split = ortho_split(batch, p.M, p.ld / BK, parts_bytes, cus);
        if (split.parts > 1) {
            const int64_t tiles = ortho_tiles(batch, p.M, p.N, true, (int)split.side);
            const int size = split.side == 64 ? 0 : split.side == 128 ? 1 : 2, side = 1 << size;
            const auto kern = size == 0 ? fg_ortho_split_kernel : size == 1 ? fg_ortho_mid_split_kernel : fg_ortho_big_split_kernel;
            const int lds = size == 0 ? SmallTile<2>::LDS : size == 1 ? 4 * MidTile::STAGE : BigTile::LDS;
            OrthoGemm g = p;
            g.tiles = (int)(tiles / batch);
            static std::atomic<uint64_t> limits[3];
            if (const hipError_t e = fg_set_lds_limit_once((const void*)kern, lds, limits[size]); e != hipSuccess) return e;
            hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * split.parts)), dim3(size == 2 ? 512 : 256), lds, stream, g, (v4f*)parts, (int)split.parts);
            hipLaunchKernelGGL(fg_ortho_join_kernel, dim3((unsigned)(tiles * side * side * 4)), dim3(256), 0, stream, g, (const v4f*)parts,
                               (int)split.parts, side);
            return hipGetLastError();
        }
    }
    const OrthoTile tile = ortho_tile(batch, p.M, p.N, symmetric(P), p.ld / BK, cus);
    if (tile != TILE_256_TAIL) return launch_tile<P>(tile, p, batch, stream);
    const int64_t all = ortho_tiles(batch, p.M, p.N, symmetric(P), 256), rest = all % cus;
    OrthoGemm part = p;
    part.count = (int)(all - rest);
    if (const hipError_t e = launch_tile<P>(TILE_256, part, batch, stream); e != hipSuccess) return e;
    part.first = part.count;
    part.count = (int)rest;
    return launch_tile<P>(ortho_tail_tile(rest, cus), part, batch, stream);
}

// The workspace: X twice (one is read while the other is written), A, B and the partial sums. X has mp rows, zeros behind its m: B X
// contracts over them.
struct Layout {
    int64_t m, n, mp, np, x0, x1, a, b, partial, bytes;
    Layout(int64_t batch, int64_t N, int64_t K) : m(std::min(N, K)), n(std::max(N, K)), mp(pad(m)), np(pad(n)) {
        int64_t at = 0;
        auto take = [&](int64_t size) {
            const int64_t here = at;
            at += align256(size);
            return here;
        };
        x0 = take(2 * batch * mp * np);
        x1 = take(2 * batch * mp * np);
        a = take(2 * batch * m * mp);
        b = take(2 * batch * m * mp);
        partial = take(8 * batch * kNormParts);
        bytes = at;
    }
};

}  // namespace

int64_t fg_ortho_workspace_bytes(int64_t batch, int64_t N, int64_t K) { return Layout(batch, N, K).bytes; }

hipError_t fg_launch_orthogonalize(const FgOrtho& o, hipStream_t stream) {
    const Layout l(o.batch, o.N, o.K);
    uint8_t* ws = (uint8_t*)o.workspace;
    uint16_t *x = (uint16_t*)(ws + l.x0), *next = (uint16_t*)(ws + l.x1), *a = (uint16_t*)(ws + l.a), *b = (uint16_t*)(ws + l.b);
    double* partial = (double*)(ws + l.partial);
    const bool wide = o.N <= o.K;
    const int parts = (int)std::min<int64_t>(kNormParts, (o.N * ((o.K + 3) / 4) + 2 * kNormThreads - 1) / (2 * kNormThreads));
    hipLaunchKernelGGL(fg_ortho_norm_kernel, dim3(parts, (unsigned)o.batch), dim3(kNormThreads), 0, stream, o, partial);
    const dim3 blocks((unsigned)(((o.N + 63) / 64) * ((o.K + 63) / 64)), (unsigned)o.batch);
    if (wide) hipLaunchKernelGGL(fg_ortho_start_kernel<true>, blocks, dim3(256), 0, stream, o, partial, parts, x, next, l.mp, l.np);
    else hipLaunchKernelGGL(fg_ortho_start_kernel<false>, blocks, dim3(256), 0, stream, o, partial, parts, x, next, l.mp, l.np);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    // A's parts may lie where the next X will, as far as its first rows of zeros.
    const int64_t room = 2 * (l.m == l.mp ? o.batch : 1) * l.m * l.np;
    for (int s = 0; s < o.steps; s++) {
        OrthoGemm g{};
        g.M = g.N = (int)l.m;
        g.p = x; g.ld = (int)l.np; g.p_batch = l.mp * l.np;
        g.out = a; g.ld_out = (int)l.mp; g.out_batch = l.m * l.mp;
        g.alpha = kScaleA / (kScaleX * kScaleX);
        if (const hipError_t e = launch_gemm<PRODUCT_A>(g, o.batch, stream, next, room); e != hipSuccess) return e;
        g.p = a; g.ld = (int)l.mp; g.p_batch = l.m * l.mp;
        g.out = b;
        g.alpha = o.c / kScaleA; g.beta = o.b; g.diag = o.a * kScaleA;
        if (const hipError_t e = launch_gemm<PRODUCT_B>(g, o.batch, stream); e != hipSuccess) return e;
        g.p = b; g.q = x; g.ld_q = (int)l.np; g.q_batch = l.mp * l.np; g.N = (int)l.n;
        if (s + 1 < o.steps) {
            g.out = next; g.ld_out = (int)l.np; g.out_batch = l.mp * l.np;
            g.alpha = 1.0f / kScaleA;
            if (const hipError_t e = launch_gemm<PRODUCT_X>(g, o.batch, stream); e != hipSuccess) return e;
        } else {
            g.out = o.out; g.ld_out = (int)o.K; g.out_batch = o.N * o.K;
            g.turned = !wide;
            g.alpha = 1.0f / (kScaleA * kScaleX); g.beta = o.scale;
            if (const hipError_t e = launch_gemm<PRODUCT_LAST>(g, o.batch, stream); e != hipSuccess) return e;
        }
        std::swap(x, next);
    }
    return hipSuccess;
}
