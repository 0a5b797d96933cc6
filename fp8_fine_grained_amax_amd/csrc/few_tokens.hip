// Feed-forward products for a few tokens (gfx950): a Linear of few rows with its epilogue, and a whole
// mixture-of-experts layer for at most 64 tokens.
//
// With few tokens a product reads its weights once and does little with them: it is bound by the rate at which
// weight codes stream from HBM, not by the matrix cores. So no tile is staged in LDS: a wave keeps 16-row weight
// tiles of one 128-deep K block as MFMA operands in registers, loads them a few K blocks ahead, and the waves
// of a workgroup split the contraction and join their sums through LDS in a fixed order. An MFMA takes weight
// rows as its first operand and tokens as its second, so lane l ends with token l % 16 and four consecutive
// weight rows.
//
// Loads and operands: an MFMA operand has row l % 16 and the bytes [16 g, 16 g + 16) and [64 + 16 g, + 16) of its 128,
// g = l / 16, in lane l. Loaded like that, every lane of a quad reads another row, which a compute unit serves at a
// third of its rate (L2-resident rows: 9.4 TB/s over the card, against 29 with quads that read 64 contiguous
// bytes; from HBM 3.9 to 5.2 against 5.1 to 5.8). So lane l loads row l / 4 and the bytes of g = l % 4, and the
// registers are turned to operands by an exchange over the LDS crossbar (ds_bpermute, eight an operand).
#include "ffn_epilogue.h"
#include "ffn_launch.h"
#include "ffn_math.h"
#include "host_util.h"

hipError_t fg_launch_quant_act_cols(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, int pow2,
                                    uint8_t* q, float* scales, hipStream_t stream);

namespace {

enum { SRC_BF16 = 0, SRC_F32 = 1, SRC_CODES = 2 };
constexpr int BK = FG_GROUP;

// A lane's place in a load of a 16-row tile, and the byte address (4 x lane) that an operand lane takes its bytes from.
__device__ __forceinline__ int load_row(int lane) { return lane >> 2; }
__device__ __forceinline__ int load_group(int lane) { return lane & 3; }
__device__ __forceinline__ int operand_source(int lane) { return 4 * (4 * (lane & 15) + (lane >> 4)); }

__device__ __forceinline__ v8i to_operand(const v4i& lo, const v4i& hi, int source) {
    v8i r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        r[i] = __builtin_amdgcn_ds_bpermute(source, lo[i]);
        r[4 + i] = __builtin_amdgcn_ds_bpermute(source, hi[i]);
    }
    return r;
}

// Hidden values in the workspace: the 32 values of each lane group g of a row's 128 are eight fours, and four j of
// all groups lie next to each other, so that the loads of a quad are contiguous there too. Position of the four
// that begins at k (a multiple of 4).
__device__ __forceinline__ int hidden_at(int k) { return ((k >> 6) * 4 + ((k >> 2) & 3)) * 16 + ((k >> 4) & 3) * 4; }

// One token tile of one K block as it is loaded: this lane's 32 values of its row's 128. `row` is the load row's.
template <int SRC>
struct ActRegs;
template <>
struct ActRegs<SRC_BF16> {
    uint4 v[4];
    __device__ __forceinline__ void load(const uint16_t* row, int64_t k, int lane) {
        const uint16_t* p = row + k + 16 * load_group(lane);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = *reinterpret_cast<const uint4*>(p + (i >> 1) * 64 + (i & 1) * 8);
    }
    __device__ __forceinline__ void get(float (&f)[32]) const {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                f[8 * i + 2 * j] = fg_bf16_lo(w[j]);
                f[8 * i + 2 * j + 1] = fg_bf16_hi(w[j]);
            }
        }
    }
};
template <>
struct ActRegs<SRC_F32> {
    v4f v[8];
    __device__ __forceinline__ void load(const float* row, int64_t k, int lane) {
        const float* p = row + k + 4 * load_group(lane);
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = *reinterpret_cast<const v4f*>(p + 16 * i);
    }
    __device__ __forceinline__ void get(float (&f)[32]) const {
#pragma unroll
        for (int i = 0; i < 32; i++) f[i] = v[i >> 2][i & 3];
    }
};
template <>
struct ActRegs<SRC_CODES> {
    v4i lo, hi;
    float s;          // of the operand's row
    __device__ __forceinline__ void load(const uint8_t* row, const float* scale, int64_t k, int lane) {
        const uint8_t* p = row + k + 16 * load_group(lane);
        lo = *reinterpret_cast<const v4i*>(p);
        hi = *reinterpret_cast<const v4i*>(p + 64);
        s = *scale;
    }
};

// Max over the quad that holds one row (quad_perm [1,0,3,2], [2,3,0,1]).
__device__ __forceinline__ float quad_max(float v) {
    v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false)));
    return __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false)));
}

// The MFMA operand of a token tile and the scale of the lane's operand row; fp32 and bf16 values are quantized
// 1x128 here, as loaded.
template <int SRC>
__device__ __forceinline__ v8i act_operand(const ActRegs<SRC>& r, int pow2, int source, float& s) {
    if constexpr (SRC == SRC_CODES) {
        s = r.s;
        return to_operand(r.lo, r.hi, source);
    } else {
        float f[32];
        r.get(f);
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; i++) m = __builtin_fmaxf(m, __builtin_fabsf(f[i]));
        const float own = fg_scale_from_amax(quad_max(m), pow2);
        const fg_divisor d = fg_divisor_of(own);
        const bool small = fg_any_small(own);
        v4i c[2];
        if (!small) {
#pragma unroll
            for (int i = 0; i < 8; i++) c[i >> 2][i & 3] = (int)fg_quant4<false>(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3], d);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) c[i >> 2][i & 3] = (int)fg_quant4<true>(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3], d);
        }
        s = __int_as_float(__builtin_amdgcn_ds_bpermute(source, __float_as_int(own)));
        return to_operand(c[0], c[1], source);
    }
}

// One K block as loaded: RT weight tiles of 16 rows, their block scales (RT / SG tiles share one) and NT token
// tiles.
template <int RT, int SG, int NT, int SRC>
struct StepRegs {
    v4i w[RT][2];
    float ws[SG];
    ActRegs<SRC> x[NT];
};

// Not a non-temporal load: the two halves of a line come from two instructions, and only a cached line is fetched once.
__device__ __forceinline__ v4i load_weight(const uint8_t* p) { return *reinterpret_cast<const v4i*>(p); }

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// A lane's 32 codes as the bf16 values they stand for (exact), for four 32-deep bf16 MFMAs.
struct WideOperand {
    v8bf v[4];
    __device__ __forceinline__ explicit WideOperand(const v8i& q) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const v2bf lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[i], 1.0f, false);
            const v2bf hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[i], 1.0f, true);
            v[i >> 1][4 * (i & 1)] = lo[0];
            v[i >> 1][4 * (i & 1) + 1] = lo[1];
            v[i >> 1][4 * (i & 1) + 2] = hi[0];
            v[i >> 1][4 * (i & 1) + 3] = hi[1];
        }
    }
};

// acc += sW sX P_b for every tile of a step; `tiles` has a bit for each token tile that holds a token in use.
// EXACT: P_b by bf16 MFMAs. The FP8 MFMAs align the 32 products of a chunk and cut off what falls below, 1.5e-5 of
// the block's sum; that moves about one in 2000 of the values that are quantized next over a border between two
// codes (a mixture's output 2.7e-3 off instead of the 1.7e-3 of its own rounding). The bf16 ones sum exactly to fp32
// (1e-8), and the matrix cores have the time: 0.2 of a weight stream's.
template <int RT, int SG, int NT, int SRC, bool EXACT>
__device__ __forceinline__ void consume(const StepRegs<RT, SG, NT, SRC>& b, int pow2, int tiles, int source,
                                        v4f (&acc)[RT][NT]) {
    v8i w[RT];
#pragma unroll
    for (int r = 0; r < RT; r++) w[r] = to_operand(b.w[r][0], b.w[r][1], source);
    if constexpr (EXACT) {
        v8i x[NT];
        float s[NT];
#pragma unroll
        for (int t = 0; t < NT; t++) x[t] = act_operand<SRC>(b.x[t], pow2, source, s[t]);
#pragma unroll
        for (int r = 0; r < RT; r++) {
            const WideOperand wr(w[r]);
#pragma unroll
            for (int t = 0; t < NT; t++) {
                if (NT > 1 && !((tiles >> t) & 1)) continue;
                const WideOperand xt(x[t]);
                v4f part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 4; i++) part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wr.v[i], xt.v[i], part, 0, 0, 0);
                const float f = s[t] * b.ws[r * SG / RT];
#pragma unroll
                for (int q = 0; q < 4; q++) acc[r][t][q] = __builtin_fmaf(part[q], f, acc[r][t][q]);
            }
        }
    } else {
#pragma unroll
        for (int t = 0; t < NT; t++) {
            if (NT > 1 && !((tiles >> t) & 1)) continue;
            float s;
            const v8i x = act_operand<SRC>(b.x[t], pow2, source, s);
#pragma unroll
            for (int r = 0; r < RT; r++) {
                const v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[r], x, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, 127);
                const float f = s * b.ws[r * SG / RT];
#pragma unroll
                for (int q = 0; q < 4; q++) acc[r][t][q] = __builtin_fmaf(part[q], f, acc[r][t][q]);
            }
        }
    }
}

// A zero that the compiler takes for a lane's own value: a load at a uniform address plus this stays a vector
// load, whose wait counts only the loads before it. (Scalar loads return out of order, so waiting for one waits
// for all that were issued ahead.)
__device__ __forceinline__ int lane_zero() {
    int z = 0;
    asm("" : "+v"(z));
    return z;
}

// Runs steps [k0, k1) with DEPTH steps' loads in flight. load(buffer) loads the next step (and, past the end, the
// last one again: every pass of the loop issues the same loads, so that the waits can count them); use(buffer)
// is called for the steps in order.
template <int DEPTH, class Regs, class Load, class Use>
__device__ __forceinline__ void stream_steps(int k0, int k1, Load&& load, Use&& use) {
    Regs buf[DEPTH];
    if (k0 >= k1) return;
    // The order of the loads is kept by scheduling fences: a wait for one counts the ones behind it.
#pragma unroll
    for (int i = 0; i < DEPTH; i++) {
        load(buf[i]);
        __builtin_amdgcn_sched_barrier(0);
    }
    for (int k = k0; k < k1; k += DEPTH) {
#pragma unroll
        for (int i = 0; i < DEPTH; i++) {
            if (k + i < k1) use(buf[i]);
            __builtin_amdgcn_sched_barrier(0);
            load(buf[i]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// ---------------------------------------------------------------------------------------------------------
// A Linear of few rows: y = act(x . W^T + bias) + residual. A workgroup owns 16 RT output columns and 16 NT
// tokens; its waves split the contraction.
// ---------------------------------------------------------------------------------------------------------
template <int RT, int NT, int NW, int DEPTH>
__global__ __launch_bounds__(NW * 64) void fg_stream_linear_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ sx,
                                                                   const uint8_t* __restrict__ wq, const float* __restrict__ sw,
                                                                   int64_t M, int64_t N, int64_t K, FgEpilogue ep, void* y,
                                                                   int out_bf16) {
    __shared__ float red[NW][RT * NT * 4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4, z = lane_zero(), source = operand_source(lane);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RT), m0 = (int64_t)blockIdx.y * (16 * NT);
    const int nkb = (int)(K / BK);
    const int k0 = (int)((int64_t)nkb * wave / NW), k1 = (int)((int64_t)nkb * (wave + 1) / NW);

    const uint8_t* wp[RT];
    const uint8_t* xp[NT];
    int64_t xm[NT];
#pragma unroll
    for (int r = 0; r < RT; r++) {
        const int64_t n = n0 + 16 * r + load_row(lane);         // columns past N read the last one again
        wp[r] = wq + (n < N ? n : N - 1) * K + 16 * load_group(lane);
    }
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int64_t m = m0 + 16 * t + l16, r = m0 + 16 * t + load_row(lane);     // and rows past M
        xm[t] = m < M ? m : M - 1;
        xp[t] = xq + (r < M ? r : M - 1) * K;
    }
    const float* sp = sw + (n0 / 128) * nkb + z;
    const int left = (int)((M - m0 + 15) / 16);       // token tiles with a row
    const int tiles = left >= NT ? (1 << NT) - 1 : (1 << left) - 1;

    v4f acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};

    using Regs = StepRegs<RT, 1, NT, SRC_CODES>;
    int lk = k0;
    stream_steps<DEPTH, Regs>(k0, k1,
        [&](Regs& b) {
            const int64_t k = (int64_t)lk * BK;
#pragma unroll
            for (int r = 0; r < RT; r++) {
                b.w[r][0] = load_weight(wp[r] + k);
                b.w[r][1] = load_weight(wp[r] + k + 64);
            }
            b.ws[0] = sp[lk];
#pragma unroll
            for (int t = 0; t < NT; t++) b.x[t].load(xp[t], sx + (int64_t)lk * M + xm[t], k, lane);
            lk = lk + 1 < k1 ? lk + 1 : lk;
        },
        [&](Regs& b) { consume<RT, 1, NT, SRC_CODES, false>(b, 0, tiles, source, acc); });

#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int q = 0; q < 4; q++) red[wave][(r * NT + t) * 4 + q][lane] = acc[r][t][q];
    __syncthreads();
    for (int id = wave; id < RT * NT; id += NW) {
        const int r = id / NT, t = id % NT;
        const int64_t m = m0 + 16 * t + l16, n = n0 + 16 * r + 4 * g;
        if (m >= M || n >= N) continue;
        v4f v = {0.f, 0.f, 0.f, 0.f}, res = {0.f, 0.f, 0.f, 0.f};
        if (ep.bias) v = fg_load_four(ep.bias, n, ep.bias_bf16, ep.vector_ok, N - n);
        if (ep.residual) res = fg_load_four(ep.residual, m * ep.ld_res + n, ep.residual_bf16, ep.vector_ok, N - n);
#pragma unroll
        for (int q = 0; q < 4; q++) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; w++) sum += red[w][id * 4 + q][lane];
            v[q] = fg_act_any(ep.act, sum + v[q]) + res[q];
        }
        if (out_bf16) {
            uint16_t* o = (uint16_t*)y + m * N + n;
            if ((N & 3) == 0) {
                *reinterpret_cast<uint2*>(o) = make_uint2(fg_bf16_bits(v[0]) | (fg_bf16_bits(v[1]) << 16),
                                                          fg_bf16_bits(v[2]) | (fg_bf16_bits(v[3]) << 16));
            } else {
#pragma unroll
                for (int q = 0; q < 4; q++)
                    if (n + q < N) o[q] = (uint16_t)fg_bf16_bits(v[q]);
            }
        } else {
            float* o = (float*)y + m * N + n;
            if ((N & 3) == 0) {
                *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int q = 0; q < 4; q++)
                    if (n + q < N) o[q] = v[q];
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------------------
// Mixture of experts.
//
// The experts that some token chose are numbered in ascending order (their slots). Token t sits in column
// t % 16 of token tile t / 16 for every expert, so tokens are neither sorted nor counted: a column whose token
// did not choose the expert computes something that nobody reads.
//   up:   workgroup = (16 RG hidden columns, slot): gate and up rows together, act(gate) * up to the workspace in
//         fp32, in the row of the first of the token's choices that names the expert.
//   down: workgroup = 16 RT output columns, all slots: the waves split the slots' K blocks between them, fold each
//         expert's sums into the tokens' with the routing weight, and join at the end.
// ---------------------------------------------------------------------------------------------------------
constexpr int kWords = 64;          // bitmap words: 2048 experts

// The chosen experts as a bitmap in LDS with the count of the ones before each word; returns how many there
// are. Ends with a barrier. `ids` is a copy of the choices in LDS.
__device__ __forceinline__ int route(const FgMoe& p, int* ids, uint32_t* words, int* before, int tid, int threads) {
    const int n = (int)p.T * p.topk;
    if (tid < kWords) words[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += threads) {
        const int e = p.ids[i];
        ids[i] = e;
        if ((uint32_t)e < (uint32_t)p.E) atomicOr(&words[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (tid < 64) {
        const int c = __popc(words[tid]);
        int sum = c;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(sum, d);
            if (tid >= d) sum += o;
        }
        before[tid] = sum - c;
        if (tid == 63) before[64] = sum;
    }
    __syncthreads();
    return before[64];
}

// Position of bit number n (from 0) of a word that has more than n set.
__device__ __forceinline__ int nth_bit(uint32_t w, int n) {
    for (; n > 0; n--) w &= w - 1;
    return __ffs((int)w) - 1;
}

template <int RG, int NT, int NW, int DEPTH, int SRC>
__global__ __launch_bounds__(NW * 64) void fg_moe_up_kernel(FgMoe p, const uint8_t* __restrict__ xq, const float* __restrict__ sx,
                                                            float* __restrict__ h) {
    constexpr int RT = 2 * RG;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    float* red = reinterpret_cast<float*>(smem);                          // [NW][RT * NT * 4][64]
    int* ids = reinterpret_cast<int*>(red + NW * RT * NT * 4 * 64);       // [T * topk]
    __shared__ uint32_t words[kWords];
    __shared__ int before[kWords + 1];
    __shared__ int choice[64];          // first choice of each token that names the expert, or -1
    __shared__ unsigned long long in_use;
    __shared__ int expert;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4, z = lane_zero(), source = operand_source(lane);
    const int nblk = (int)(p.I / (16 * RG));
    const int slot = (int)blockIdx.x / nblk;
    const int64_t n0 = (int64_t)((int)blockIdx.x % nblk) * (16 * RG);

    const int used = route(p, ids, words, before, tid, NW * 64);
    if (slot >= used) return;
    if (tid < kWords && before[tid] <= slot && slot < before[tid + 1]) expert = 32 * tid + nth_bit(words[tid], slot - before[tid]);
    __syncthreads();
    const int e = __builtin_amdgcn_readfirstlane(expert);
    if (tid < 64) {
        int c = -1;
        if (tid < p.T)
            for (int j = p.topk - 1; j >= 0; j--)
                if (ids[tid * p.topk + j] == e) c = j;
        choice[tid] = c;
        const uint64_t m = __builtin_amdgcn_ballot_w64(c >= 0);
        if (tid == 0) in_use = m;
    }
    __syncthreads();
    const uint64_t mask = in_use;
    const int first = __ffsll((unsigned long long)mask) - 1;
    int tiles = 0;
#pragma unroll
    for (int t = 0; t < NT; t++)
        if ((mask >> (16 * t)) & 0xFFFF) tiles |= 1 << t;
    tiles = __builtin_amdgcn_readfirstlane(tiles);

    const int nkb = (int)(p.H / BK);
    const int k0 = nkb * wave / NW, k1 = nkb * (wave + 1) / NW;
    const uint8_t* wp[RT];
#pragma unroll
    for (int r = 0; r < RT; r++) {
        const int64_t n = (r < RG ? 0 : p.I) + n0 + 16 * (r % RG) + load_row(lane);
        wp[r] = p.w1q + ((int64_t)e * 2 * p.I + n) * p.H + 16 * load_group(lane);
    }
    const float* sp[2];
#pragma unroll
    for (int s = 0; s < 2; s++) sp[s] = p.s1 + ((int64_t)e * 2 * (p.I / 128) + (s * p.I + n0) / 128) * nkb + z;
    // columns not in use read the first token's row: valid memory, no extra traffic
    auto token_of = [&](int t) { return ((mask >> t) & 1) ? t : first; };
    int xt[NT], xr[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        xt[t] = token_of(16 * t + l16);
        xr[t] = token_of(16 * t + load_row(lane));
    }

    v4f acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};

    using Regs = StepRegs<RT, 2, NT, SRC>;
    int lk = k0;
    stream_steps<DEPTH, Regs>(k0, k1,
        [&](Regs& b) {
            const int64_t k = (int64_t)lk * BK;
#pragma unroll
            for (int r = 0; r < RT; r++) {
                b.w[r][0] = load_weight(wp[r] + k);
                b.w[r][1] = load_weight(wp[r] + k + 64);
            }
            b.ws[0] = sp[0][lk];
            b.ws[1] = sp[1][lk];
#pragma unroll
            for (int t = 0; t < NT; t++) {
                if constexpr (SRC == SRC_CODES) b.x[t].load(xq + xr[t] * p.H, sx + lk * p.T + xt[t], k, lane);
                else b.x[t].load(p.x + xr[t] * p.ld_x, k, lane);
            }
            lk = lk + 1 < k1 ? lk + 1 : lk;
        },
        [&](Regs& b) { consume<RT, 2, NT, SRC, true>(b, p.pow2, tiles, source, acc); });

#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int q = 0; q < 4; q++) red[((wave * RT + r) * NT + t) * 256 + q * 64 + lane] = acc[r][t][q];
    __syncthreads();
    for (int id = wave; id < RG * NT; id += NW) {
        const int r = id / NT, t = id % NT;
        const int c = choice[16 * t + l16];
        if (c < 0) continue;
        v4f v;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; w++) {
                gate += red[((w * RT + r) * NT + t) * 256 + q * 64 + lane];
                up += red[((w * RT + RG + r) * NT + t) * 256 + q * 64 + lane];
            }
            v[q] = fg_act_any(p.act, gate) * up;
        }
        const int64_t n = n0 + 16 * r + 4 * g;
        *reinterpret_cast<v4f*>(h + ((int64_t)(16 * t + l16) * p.topk + c) * p.I + (n & ~127) + hidden_at((int)(n & 127))) = v;
    }
}

// fp32 rows -> 1x128 codes and scales, one 16-lane group a tile; rows of choices that name no local expert, or
// one that an earlier choice of the token named, were not written and are skipped.
__global__ __launch_bounds__(256) void fg_moe_quant_kernel(FgMoe p, const float* __restrict__ h, uint8_t* __restrict__ hq,
                                                           float* __restrict__ sh) {
    const int lane16 = threadIdx.x & 15;
    const int64_t groups = p.I / FG_GROUP, rows = p.T * p.topk;
    const int64_t id = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int64_t r = id / groups, g = id % groups;
    bool ok = r < rows;
    if (ok) {
        const int e = p.ids[r], j = (int)(r % p.topk);
        ok = (uint32_t)e < (uint32_t)p.E;
        for (int i = 1; i <= j; i++) ok = ok && p.ids[r - i] != e;
    }
    float f[8];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const v4f v = ok ? *reinterpret_cast<const v4f*>(h + r * p.I + g * FG_GROUP + hidden_at(lane16 * 8 + 4 * i)) : v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; q++) f[4 * i + q] = v[q];
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) m = __builtin_fmaxf(m, __builtin_fabsf(f[i]));
    const float s = fg_scale_from_amax(fg_row16_max(m), p.pow2);
    const fg_divisor d = fg_divisor_of(s);
    const bool small = fg_any_small(s);
    const uint2 c = make_uint2(fg_quant4(f[0], f[1], f[2], f[3], d, small), fg_quant4(f[4], f[5], f[6], f[7], d, small));
    if (!ok) return;
    *reinterpret_cast<uint2*>(hq + r * p.I + g * FG_GROUP + lane16 * 8) = c;
    if (lane16 == 0) sh[g * rows + r] = s;
}

template <int RT, int NT, int NW, int DEPTH, int SRC>
__global__ __launch_bounds__(NW * 64) void fg_moe_down_kernel(FgMoe p, const float* __restrict__ h, const uint8_t* __restrict__ hq,
                                                              const float* __restrict__ sh) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int n_pairs = (int)p.T * p.topk;
    const int max_used = n_pairs < p.E ? n_pairs : p.E;
    float* red = reinterpret_cast<float*>(smem);                          // [NW][RT * NT * 4][64], once the rest is done with
    int* ids = reinterpret_cast<int*>(smem);                              // [T * topk]
    float* weight = reinterpret_cast<float*>(ids + n_pairs);              // [T * topk]
    int* list = reinterpret_cast<int*>(weight + n_pairs);                 // [max_used] experts by slot
    int8_t* choice = reinterpret_cast<int8_t*>(list + max_used);          // [max_used][16 NT], as in the up kernel
    __shared__ uint32_t words[kWords];
    __shared__ int before[kWords + 1];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4, z = lane_zero(), source = operand_source(lane);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);

    for (int i = tid; i < n_pairs; i += NW * 64) weight[i] = p.weights[i];
    const int used = route(p, ids, words, before, tid, NW * 64);
    for (int i = tid; i < used * 16 * NT; i += NW * 64) choice[i] = -1;
    if (tid < kWords) {
        uint32_t w = words[tid];
        for (int s = before[tid]; w; s++, w &= w - 1) list[s] = 32 * tid + __ffs((int)w) - 1;
    }
    __syncthreads();
    for (int i = tid; i < n_pairs; i += NW * 64) {
        const int e = ids[i], t = i / p.topk, j = i % p.topk;
        bool mine = (uint32_t)e < (uint32_t)p.E;
        for (int k = 1; k <= j; k++) mine = mine && ids[i - k] != e;       // the first choice that names e
        if (mine) choice[(before[e >> 5] + __popc(words[e >> 5] & ((1u << (e & 31)) - 1))) * (16 * NT) + t] = (int8_t)j;
    }
    __syncthreads();

    const int nkb = (int)(p.I / BK);
    const int steps = used * nkb;
    const int k0 = (int)((int64_t)steps * wave / NW), k1 = (int)((int64_t)steps * (wave + 1) / NW);
    v4f acc[RT][NT], sum[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[r][t] = sum[r][t] = v4f{0.f, 0.f, 0.f, 0.f};

    // The loader's place: slot and K block, with the lane's pointers for the slot.
    using Regs = StepRegs<RT, 1, NT, SRC>;
    int ls = nkb > 0 ? k0 / nkb : 0, lk = nkb > 0 ? k0 % nkb : 0, left = k1 - k0;
    const uint8_t* wp = nullptr;
    const float* sp = nullptr;
    int row[NT], lrow[NT];              // rows of the columns' tokens, and of those that this lane loads
    auto enter = [&](int s) {
        const int e = __builtin_amdgcn_readfirstlane(list[s]);
        wp = p.w2q + ((int64_t)e * p.H + n0 + load_row(lane)) * p.I + 16 * load_group(lane);
        sp = p.s2 + ((int64_t)e * (p.H / 128) + n0 / 128) * nkb + z;
        // columns not in use read a row that some token of the tile uses, or (no tile) the slot's first
        const int8_t* c = choice + s * (16 * NT);
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const int j = c[16 * t + l16];
            const uint64_t m = __builtin_amdgcn_ballot_w64(j >= 0);
            const int own = (16 * t + l16) * p.topk + j;
            const int any = m ? __builtin_amdgcn_readlane(own, __ffsll((unsigned long long)m) - 1) : -1;
            row[t] = j >= 0 ? own : any;
        }
        int some = -1;
#pragma unroll
        for (int t = 0; t < NT; t++) some = some >= 0 ? some : __builtin_amdgcn_readlane(row[t], 0);
#pragma unroll
        for (int t = 0; t < NT; t++) {
            row[t] = row[t] >= 0 ? row[t] : some;
            lrow[t] = __shfl(row[t], load_row(lane));
        }
    };
    if (k0 < k1) enter(ls);
    // The consumer's place, with the slot's token tiles.
    int cs = ls, ck = lk, done = 0, tiles = 0;
    auto tiles_of = [&](int s) {
        int m = 0;
        for (int t = 0; t < NT; t++)
            if (__builtin_amdgcn_ballot_w64(choice[s * (16 * NT) + 16 * t + l16] >= 0)) m |= 1 << t;
        return __builtin_amdgcn_readfirstlane(m);
    };
    if (NT > 1 && k0 < k1) tiles = tiles_of(cs);
    stream_steps<DEPTH, Regs>(k0, k1,
        [&](Regs& b) {
            const int64_t k = (int64_t)lk * BK;
#pragma unroll
            for (int r = 0; r < RT; r++) {
                b.w[r][0] = load_weight(wp + 16 * r * p.I + k);
                b.w[r][1] = load_weight(wp + 16 * r * p.I + k + 64);
            }
            b.ws[0] = sp[lk];
#pragma unroll
            for (int t = 0; t < NT; t++) {
                if constexpr (SRC == SRC_CODES) b.x[t].load(hq + lrow[t] * p.I, sh + (int64_t)lk * n_pairs + row[t], k, lane);
                else b.x[t].load(h + lrow[t] * p.I, k, lane);
            }
            if (left > 1) {
                left--;
                if (++lk == nkb) {
                    lk = 0;
                    enter(++ls);
                }
            }
        },
        [&](Regs& b) {
            consume<RT, 1, NT, SRC, false>(b, p.pow2, tiles, source, acc);
            done++;
            ck++;
            if (ck == nkb || done == k1 - k0) {     // the wave's share of this expert is complete: weigh it
                const int e = list[cs];
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    const int tok = 16 * t + l16;
                    const bool in_use = choice[cs * (16 * NT) + tok] >= 0;
                    float w = 0.0f;
                    if (in_use)
                        for (int j = 0; j < p.topk; j++)
                            if (ids[tok * p.topk + j] == e) w += weight[tok * p.topk + j];
#pragma unroll
                    for (int r = 0; r < RT; r++)
#pragma unroll
                        for (int q = 0; q < 4; q++) {
                            sum[r][t][q] = in_use ? __builtin_fmaf(w, acc[r][t][q], sum[r][t][q]) : sum[r][t][q];
                            acc[r][t][q] = 0.0f;
                        }
                }
                ck = 0;
                cs++;
                if (NT > 1 && done < k1 - k0) tiles = tiles_of(cs);
            }
        });

    __syncthreads();                     // every wave has read its choices and weights
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int q = 0; q < 4; q++) red[((wave * RT + r) * NT + t) * 256 + q * 64 + lane] = sum[r][t][q];
    __syncthreads();
    for (int id = wave; id < RT * NT; id += NW) {
        const int r = id / NT, t = id % NT;
        const int64_t tok = 16 * t + l16, n = n0 + 16 * r + 4 * g;
        if (tok >= p.T) continue;
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; q++) {
            v[q] = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; w++) v[q] += red[((w * RT + r) * NT + t) * 256 + q * 64 + lane];
        }
        if (p.out_bf16) {
            uint16_t* o = (uint16_t*)p.y + tok * p.ld_y + n;
            const uint32_t lo = fg_bf16_bits(v[0]) | (fg_bf16_bits(v[1]) << 16), hi = fg_bf16_bits(v[2]) | (fg_bf16_bits(v[3]) << 16);
            if ((p.ld_y & 3) == 0) {
                *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
            } else {
                o[0] = (uint16_t)lo;
                o[1] = (uint16_t)(lo >> 16);
                o[2] = (uint16_t)hi;
                o[3] = (uint16_t)(hi >> 16);
            }
        } else {
            float* o = (float*)p.y + tok * p.ld_y + n;
            if ((p.ld_y & 3) == 0) {
                *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int q = 0; q < 4; q++) o[q] = v[q];
            }
        }
    }
}

template <int RT, int NT, int NW, int DEPTH>
hipError_t launch_linear(const uint8_t* xq, const float* sx, const uint8_t* wq, const float* sw, int64_t M, int64_t N,
                         int64_t K, const FgEpilogue& e, void* y, int out_bf16, hipStream_t stream) {
    const dim3 grid((unsigned)((N + 16 * RT - 1) / (16 * RT)), (unsigned)((M + 16 * NT - 1) / (16 * NT)));
    hipLaunchKernelGGL((fg_stream_linear_kernel<RT, NT, NW, DEPTH>), grid, dim3(NW * 64), 0, stream, xq, sx, wq, sw, M, N, K,
                       e, y, out_bf16);
    return hipGetLastError();
}

template <class Kernel>
hipError_t raise_lds(Kernel kern, int bytes, std::atomic<uint64_t>& done) {
    return bytes > 65536 ? fg_set_lds_limit_once((const void*)kern, 156 * 1024, done) : hipSuccess;
}

template <int RG, int NT, int NW, int DEPTH, int SRC>
hipError_t launch_up(const FgMoe& p, const uint8_t* xq, const float* sx, float* h, int64_t slots, hipStream_t stream) {
    auto kern = fg_moe_up_kernel<RG, NT, NW, DEPTH, SRC>;
    const int lds = NW * 2 * RG * NT * 1024 + (int)p.T * p.topk * 4;
    static std::atomic<uint64_t> lds_limit_set{0};
    const hipError_t e = raise_lds(kern, lds, lds_limit_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)(slots * (p.I / (16 * RG)))), dim3(NW * 64), lds, stream, p, xq, sx, h);
    return hipGetLastError();
}

template <int RT, int NT, int NW, int DEPTH, int SRC>
hipError_t launch_down(const FgMoe& p, const float* h, const uint8_t* hq, const float* sh, int64_t slots, hipStream_t stream) {
    auto kern = fg_moe_down_kernel<RT, NT, NW, DEPTH, SRC>;
    const int sums = NW * RT * NT * 1024, lists = (int)(p.T * p.topk * 8 + slots * (4 + 16 * NT));
    const int lds = sums > lists ? sums : lists;      // at most 2048 * 76 = 152 KB
    static std::atomic<uint64_t> lds_limit_set{0};
    const hipError_t e = raise_lds(kern, lds, lds_limit_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)(p.H / (16 * RT))), dim3(NW * 64), lds, stream, p, h, hq, sh);
    return hipGetLastError();
}

constexpr int64_t kWideLinear = 4096;  // output columns from which a Linear's workgroups take 32 of them
constexpr int64_t kFusedTokens = 16;   // up to here the activations are quantized inside the two products

int64_t pad16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// Workspace: the hidden values in fp32; for more than 16 tokens also the codes and scales of x and of them.
struct MoeWorkspace {
    int64_t h, xq, sx, hq, sh, bytes;
    MoeWorkspace(int64_t T, int topk, int64_t H, int64_t I) {
        const int64_t rows = T * topk;
        h = 0;
        bytes = rows * I * 4;
        xq = sx = hq = sh = bytes;
        if (T > kFusedTokens) {
            sx = xq + pad16(T * H);
            hq = sx + pad16(H / 128 * T * 4);
            sh = hq + pad16(rows * I);
            bytes = sh + pad16(I / 128 * rows * 4);
        }
    }
};

template <int NT>
hipError_t moe_with_codes(const FgMoe& p, uint8_t* ws, const MoeWorkspace& at, int64_t slots, hipStream_t stream) {
    float* h = (float*)(ws + at.h);
    hipError_t e = fg_launch_quant_act_cols(p.x, p.T, p.H, p.ld_x, p.pow2, ws + at.xq, (float*)(ws + at.sx), stream);
    if (e != hipSuccess) return e;
    if (p.I > 0) {
        e = launch_up<2, NT, 4, 1, SRC_CODES>(p, ws + at.xq, (const float*)(ws + at.sx), h, slots, stream);
        if (e != hipSuccess) return e;
        const int64_t tiles = p.T * p.topk * (p.I / FG_GROUP);
        hipLaunchKernelGGL(fg_moe_quant_kernel, dim3((unsigned)((tiles + 15) / 16)), dim3(256), 0, stream, p, h, ws + at.hq,
                           (float*)(ws + at.sh));
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return launch_down<2, NT, 8, 2, SRC_CODES>(p, h, ws + at.hq, (const float*)(ws + at.sh), slots, stream);
}

}  // namespace

// Estimated time in us of the weight-streaming Linear: 4 us of launch and latency, then a pass over the weights for
// every 64 rows, the first from HBM and the others from the caches at about the same 5.2 TB/s (3.2 where N leaves 16-row
// workgroups only), and an LDS exchange that the tokens' operands add to the first pass. Measured: N = 18432,
// K = 7168: 31 us at M = 16, 48 at 64, 66 at 128, 115 at 256; N = K = 7168: 13.5, 19.5, 29.5, 48.5.
double fg_stream_linear_us(int64_t M, int64_t N, int64_t K) {
    const double pass = (double)N * (double)K / (N >= kWideLinear ? 5.2e6 : 3.2e6);
    return 4.0 + pass * (M <= 16 ? 1.0 : M <= 32 ? 1.2 : (double)((M + 63) / 64) + 0.6);
}

hipError_t fg_launch_stream_linear(const uint8_t* xq, const float* sx, const uint8_t* wq, const float* sw, int64_t M,
                                   int64_t N, int64_t K, const FgEpilogue& e, void* y, int out_bf16, hipStream_t stream) {
    // 32 output columns a workgroup share each token tile's loads and exchange (N = 7168, K = 18432, M = 16: 28.4 us
    // against 35.7 with 16), where that leaves workgroups enough; 8 waves split the contraction of the others.
    if (N >= kWideLinear) {
        if (M <= 16) return launch_linear<2, 1, 4, 2>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
        if (M <= 32) return launch_linear<2, 2, 8, 2>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
        return launch_linear<2, 4, 8, 1>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
    }
    if (M <= 16) return launch_linear<1, 1, 8, 1>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
    if (M <= 32) return launch_linear<1, 2, 8, 1>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
    return launch_linear<1, 4, 8, 1>(xq, sx, wq, sw, M, N, K, e, y, out_bf16, stream);
}

int64_t fg_moe_workspace_bytes(int64_t T, int topk, int64_t H, int64_t I) { return MoeWorkspace(T, topk, H, I).bytes; }

hipError_t fg_launch_moe_few_tokens(const FgMoe& p, hipStream_t stream) {
    const MoeWorkspace at(p.T, p.topk, p.H, p.I);
    uint8_t* ws = (uint8_t*)p.workspace;
    const int64_t pairs = p.T * p.topk, slots = pairs < p.E ? pairs : p.E;
    if (p.T > 32) return moe_with_codes<4>(p, ws, at, slots, stream);
    if (p.T > kFusedTokens) return moe_with_codes<2>(p, ws, at, slots, stream);
    float* h = (float*)(ws + at.h);
    const bool wide_up = slots * (p.I / 32) >= 256, wide_down = p.H >= 32 * 128;
    if (p.I > 0) {
        const hipError_t e = wide_up ? launch_up<2, 1, 4, 2, SRC_BF16>(p, nullptr, nullptr, h, slots, stream)
                                     : launch_up<1, 1, 8, 1, SRC_BF16>(p, nullptr, nullptr, h, slots, stream);
        if (e != hipSuccess) return e;
    }
    return wide_down ? launch_down<2, 1, 8, 2, SRC_F32>(p, h, nullptr, nullptr, slots, stream)
                     : launch_down<1, 1, 8, 1, SRC_F32>(p, h, nullptr, nullptr, slots, stream);
}
