// A whole mixture-of-experts feed-forward for at most 64 tokens (gfx950): bound by the rate at which the chosen experts'
// weights stream from HBM (see weight_stream.h).
//
// The experts that some token chose are numbered (their slots): in ascending order, or with at most 64 choices in that of
// their first ones.
//   up:   workgroup = (32 or 16 hidden columns, slot): gate and up rows together, act(gate) * up to the workspace in
//         fp32, in the row of the first of the token's choices that names the expert.
//   down: workgroup = 32 or 16 output columns, all slots: the waves split the slots' K blocks between them, weigh each
//         expert's sums into the tokens' with the routing weight, and join at the end.
//
// Up to 16 tokens these two launches are all. Token t sits in column t of the one token tile for every expert, so tokens
// are neither sorted nor counted (a column whose token did not choose the expert computes something that nobody
// reads); every workgroup works the slots out for itself and quantizes the activations that it needs as it loads them.
//
// For more tokens that work would be done too often, and most columns would stand idle: 64 tokens with 8 choices
// among 64 experts give each expert 8. Two small launches go between: one quantizes x and writes down for each slot its
// tokens, closely packed into tiles of 16 (MoePlan), one quantizes the hidden values as MFMA operands in that order. A
// slot then runs with 1, 2 or 4 token tiles.
//
// Measured, H = 7168, I = 2048. One token, 8 experts: up 44.4 us (235 MB, 5.3 TB/s), down 28.1 (117 MB, 4.2 TB/s; 224
// workgroups for 256 CUs, and the experts' list before the first load). 64 tokens, 8 choices of 64 experts, 16 of them
// here: plan 8.1, up 87 (470 MB, 5.4 TB/s), quantize 4.8, down 48.6 (235 MB, 4.8 TB/s); with the fused launches 162 in
// all instead of 147.
#include "ffn_launch.h"
#include "host_util.h"
#include "moe_workspace.h"
#include "weight_stream.h"

#include <type_traits>

namespace {

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

// Slot of an expert that some token chose.
__device__ __forceinline__ int slot_of_expert(const uint32_t* words, const int* before, int e) {
    return before[e >> 5] + __popc(words[e >> 5] & ((1u << (e & 31)) - 1));
}

// Whether choice i names an expert here that no earlier choice of its token names.
__device__ __forceinline__ bool first_choice(const FgMoe& p, const int* ids, int i) {
    bool first = (uint32_t)ids[i] < (uint32_t)p.E;
    for (int k = 1; k <= i % p.topk; k++) first = first && ids[i - k] != ids[i];
    return first;
}

// At most 64 choices: a lane holds each, and every wave finds the slots by itself, in the order in which the choices first
// name the experts, without LDS or a barrier (one token, 2 of 8 experts, H = 1024, I = 512: the up kernel
// 4.9 us instead of 5.8, the down kernel 4.8 instead of 5.6).
constexpr int kLaneChoices = 64;

__device__ __forceinline__ int lane_choice(const FgMoe& p, int n, int lane) {
    const int id = lane < n ? p.ids[lane] : -1;
    return (uint32_t)id < (uint32_t)p.E ? id : -1;
}

// Takes the next expert out of `left`, the lanes whose choices still want one (not 0); `same`: the lanes that chose it.
__device__ __forceinline__ int next_expert(int id, uint64_t& left, uint64_t& same) {
    const int e = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
    same = __builtin_amdgcn_ballot_w64(id == e);
    left &= ~same;
    return e;
}

// The first of token t's choices among them, or -1.
__device__ __forceinline__ int choice_among(const FgMoe& p, uint64_t same, int t) {
    const uint64_t own = t < p.T ? (same >> (t * p.topk)) & ((1ull << p.topk) - 1) : 0;
    return own ? __ffsll((unsigned long long)own) - 1 : -1;
}

// Position of bit number n (from 0) of a word that has more than n set.
__device__ __forceinline__ int nth_bit(uint32_t w, int n) {
    for (; n > 0; n--) w &= w - 1;
    return __ffs((int)w) - 1;
}

// Eight values of each lane, 16 lanes a 1x128 tile -> its codes and the tile's scale.
__device__ __forceinline__ uint2 quant_tile(const float (&f)[8], int pow2, float& s) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) m = __builtin_fmaxf(m, __builtin_fabsf(f[i]));
    s = fg_scale_from_amax(fg_row16_max(m), pow2);
    const fg_divisor d = fg_divisor_of(s);
    const bool small = fg_any_small(s);
    return make_uint2(fg_quant4(f[0], f[1], f[2], f[3], d, small), fg_quant4(f[4], f[5], f[6], f[7], d, small));
}

__device__ __forceinline__ void store_four(const FgMoe& p, int64_t tok, int64_t n, const float (&v)[4]) {
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

// ---- up to 16 tokens ------------------------------------------------------------------------------------

template <int RG, int NW, int DEPTH>
__global__ __launch_bounds__(NW * 64) void fg_moe_up_kernel(FgMoe p, float* __restrict__ h) {
    constexpr int RT = 2 * RG;
    __shared__ float red[NW][RT][4][64];
    __shared__ int ids[16 * 32];
    __shared__ uint32_t words[kWords];
    __shared__ int before[kWords + 1];
    __shared__ int expert;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4, z = lane_zero(), source = operand_source(lane);
    const int nblk = (int)(p.I / (16 * RG));
    const int slot = (int)blockIdx.x / nblk;
    const int64_t n0 = (int64_t)((int)blockIdx.x % nblk) * (16 * RG);

    int e, c;                           // the expert, and token l16's choice of it or -1
    const int n_pairs = (int)p.T * p.topk;
    if (n_pairs <= kLaneChoices) {
        const int id = lane_choice(p, n_pairs, lane);
        uint64_t left = __builtin_amdgcn_ballot_w64(id >= 0), same = 0;
        e = -1;
        for (int s = 0; s <= slot; s++) {
            if (!left) return;
            e = next_expert(id, left, same);
        }
        c = choice_among(p, same, l16);
    } else {
        const int used = route(p, ids, words, before, tid, NW * 64);
        if (slot >= used) return;
        if (tid < kWords && before[tid] <= slot && slot < before[tid + 1]) expert = 32 * tid + nth_bit(words[tid], slot - before[tid]);
        __syncthreads();
        e = __builtin_amdgcn_readfirstlane(expert);
        c = -1;
        if (l16 < p.T)
            for (int j = p.topk - 1; j >= 0; j--)
                if (ids[l16 * p.topk + j] == e) c = j;
    }
    // columns not in use read the first token's row: valid memory, no extra traffic
    const uint32_t mask = (uint32_t)__builtin_amdgcn_ballot_w64(c >= 0) & 0xFFFF;
    const int xr = (mask >> load_row(lane)) & 1 ? load_row(lane) : __ffs((int)mask) - 1;

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

    v4f acc[RT][1];
#pragma unroll
    for (int r = 0; r < RT; r++) acc[r][0] = v4f{0.f, 0.f, 0.f, 0.f};
    using Regs = StepRegs<RT, 2, 1, SRC_BF16>;
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
            b.x[0].load(p.x + xr * p.ld_x, k, lane);
            lk = lk + 1 < k1 ? lk + 1 : lk;
        },
        [&](Regs& b) { consume<RT, 2, 1, SRC_BF16, true>(b, p.pow2, 1, source, acc); });

#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int q = 0; q < 4; q++) red[wave][r][q][lane] = acc[r][0][q];
    __syncthreads();
    if (c < 0) return;
    for (int r = wave; r < RG; r += NW) {
        v4f v;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; w++) {
                gate += red[w][r][q][lane];
                up += red[w][RG + r][q][lane];
            }
            v[q] = fg_act_any(p.act, gate) * up;
        }
        const int64_t n = n0 + 16 * r + 4 * g;
        *reinterpret_cast<v4f*>(h + ((int64_t)l16 * p.topk + c) * p.I + (n & ~127) + hidden_at((int)(n & 127))) = v;
    }
}

template <int RT, int NW, int DEPTH>
__global__ __launch_bounds__(NW * 64) void fg_moe_down_kernel(FgMoe p, const float* __restrict__ h, float* __restrict__ partial) {
    __shared__ float red[NW][RT][4][64];
    __shared__ int ids[16 * 32];
    __shared__ float weight[16 * 32];
    __shared__ int list[16 * 32];                 // experts by slot
    __shared__ int8_t choice[16 * 32][16];        // [slot][token]: its first choice of the expert, or -1
    __shared__ uint32_t words[kWords];
    __shared__ int before[kWords + 1];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4, z = lane_zero(), source = operand_source(lane);
    const int n_pairs = (int)p.T * p.topk;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);

    for (int i = tid; i < n_pairs; i += NW * 64) weight[i] = p.weights[i];
    int used = 0;
    if (n_pairs <= kLaneChoices) {
        const int id = lane_choice(p, n_pairs, lane);
        if (wave == 0) ids[lane] = id;
        uint64_t left = __builtin_amdgcn_ballot_w64(id >= 0), same;
        for (; left; used++) {
            const int e = next_expert(id, left, same);
            if (used % NW != wave) continue;
            const int c = choice_among(p, same, l16);
            if (lane < 16) choice[used][lane] = (int8_t)c;
            if (lane == 0) list[used] = e;
        }
    } else {
        used = route(p, ids, words, before, tid, NW * 64);
        for (int i = tid; i < used * 4; i += NW * 64) reinterpret_cast<int*>(choice)[i] = -1;
        if (tid < kWords) {
            uint32_t w = words[tid];
            for (int s = before[tid]; w; s++, w &= w - 1) list[s] = 32 * tid + __ffs((int)w) - 1;
        }
        __syncthreads();
        for (int i = tid; i < n_pairs; i += NW * 64)
            if (first_choice(p, ids, i)) choice[slot_of_expert(words, before, ids[i])][i / p.topk] = (int8_t)(i % p.topk);
    }
    __syncthreads();

    const int nkb = (int)(p.I / BK);
    const int steps = used * nkb;
    // this wave's share of all slots' K blocks, over the workgroups of one column block (grid y)
    const int parts = NW * (int)gridDim.y, part = (int)blockIdx.y * NW + wave;
    const int k0 = (int)((int64_t)steps * part / parts), k1 = (int)((int64_t)steps * (part + 1) / parts);
    v4f acc[RT][1], sum[RT];
#pragma unroll
    for (int r = 0; r < RT; r++) acc[r][0] = sum[r] = v4f{0.f, 0.f, 0.f, 0.f};

    // The loader's place: slot and K block, with the lane's pointers for the slot.
    using Regs = StepRegs<RT, 1, 1, SRC_F32>;
    int ls = nkb > 0 ? k0 / nkb : 0, lk = nkb > 0 ? k0 % nkb : 0, left = k1 - k0;
    const uint8_t* wp = nullptr;
    const float* sp = nullptr;
    const float* hp = nullptr;
    auto enter = [&](int s) {
        const int e = __builtin_amdgcn_readfirstlane(list[s]);
        wp = p.w2q + ((int64_t)e * p.H + n0 + load_row(lane)) * p.I + 16 * load_group(lane);
        sp = p.s2 + ((int64_t)e * (p.H / 128) + n0 / 128) * nkb + z;
        // columns not in use read the row of one that is
        const int tok = load_row(lane), j = choice[s][tok], own = tok * p.topk + j;
        const uint64_t m = __builtin_amdgcn_ballot_w64(j >= 0);
        const int any = __builtin_amdgcn_readlane(own, __ffsll((unsigned long long)m) - 1);
        hp = h + (int64_t)(j >= 0 ? own : any) * p.I;
    };
    if (k0 < k1) enter(ls);
    int cs = ls, ck = lk, done = 0;               // the consumer's place
    stream_steps<DEPTH, Regs>(k0, k1,
        [&](Regs& b) {
            const int64_t k = (int64_t)lk * BK;
#pragma unroll
            for (int r = 0; r < RT; r++) {
                b.w[r][0] = load_weight(wp + 16 * r * p.I + k);
                b.w[r][1] = load_weight(wp + 16 * r * p.I + k + 64);
            }
            b.ws[0] = sp[lk];
            b.x[0].load(hp, k, lane);
            if (left > 1) {
                left--;
                if (++lk == nkb) {
                    lk = 0;
                    enter(++ls);
                }
            }
        },
        [&](Regs& b) {
            consume<RT, 1, 1, SRC_F32, false>(b, p.pow2, 1, source, acc);
            done++;
            ck++;
            if (ck == nkb || done == k1 - k0) {     // the wave's share of this expert is complete: weigh it
                const int e = list[cs];
                const bool in_use = choice[cs][l16] >= 0;
                float w = 0.0f;
                if (in_use)
                    for (int j = 0; j < p.topk; j++)
                        if (ids[l16 * p.topk + j] == e) w += weight[l16 * p.topk + j];
#pragma unroll
                for (int r = 0; r < RT; r++)
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        sum[r][q] = in_use ? __builtin_fmaf(w, acc[r][0][q], sum[r][q]) : sum[r][q];
                        acc[r][0][q] = 0.0f;
                    }
                ck = 0;
                cs++;
            }
        });

#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int q = 0; q < 4; q++) red[wave][r][q][lane] = sum[r][q];
    __syncthreads();
    if (l16 >= p.T) return;
    for (int r = wave; r < RT; r += NW) {
        const int64_t n = n0 + 16 * r + 4 * g;
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; q++) {
            v[q] = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; w++) v[q] += red[w][r][q][lane];
        }
        if (gridDim.y > 1) *reinterpret_cast<float4*>(partial + ((int64_t)blockIdx.y * p.T + l16) * p.H + n) = make_float4(v[0], v[1], v[2], v[3]);
        else store_four(p, l16, n, v);
    }
}

// ---- more tokens ------------------------------------------------------------------------------------------

constexpr int kMaxPairs = 64 * 32;

// The last workgroup writes the slots down; the others quantize x.
__global__ __launch_bounds__(256) void fg_moe_plan_kernel(FgMoe p, MoePlan plan) {
    __shared__ int ids[kMaxPairs];
    __shared__ uint32_t words[kWords];
    __shared__ int before[kWords + 1];
    __shared__ uint32_t tokens[kMaxPairs][2];     // [slot] bitmap of its tokens
    __shared__ int base[kMaxPairs + 1];
    __shared__ float weights[kMaxPairs];
    const int tid = threadIdx.x;
    if (blockIdx.x < gridDim.x - 1) {
        const int lane16 = tid & 15, groups = (int)(p.H / BK);
        const int id = (int)blockIdx.x * 16 + (tid >> 4), t = id / groups, g = id % groups;
        const bool ok = t < p.T;
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (ok) {
            const uint4 v = *reinterpret_cast<const uint4*>(p.x + t * p.ld_x + g * BK + 8 * lane16);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 8; i++) f[i] = (i & 1) ? fg_bf16_hi(w[i >> 1]) : fg_bf16_lo(w[i >> 1]);
        }
        float s;
        const uint2 c = quant_tile(f, p.pow2, s);
        if (!ok) return;
        *reinterpret_cast<uint2*>(plan.xq + t * p.H + g * BK + 8 * lane16) = c;
        if (lane16 == 0) plan.sx[g * p.T + t] = s;
        return;
    }
    const int n = (int)p.T * p.topk;
    for (int i = tid; i < n; i += 256) weights[i] = p.weights[i];
    const int used = route(p, ids, words, before, tid, 256);
    for (int i = tid; i < used; i += 256) tokens[i][0] = tokens[i][1] = 0;
    if (tid < kWords) {
        uint32_t w = words[tid];
        for (int s = before[tid]; w; s++, w &= w - 1) plan.list[s] = 32 * tid + __ffs((int)w) - 1;
    }
    __syncthreads();
    for (int i = tid; i < n; i += 256)
        if ((uint32_t)ids[i] < (uint32_t)p.E) {
            const int t = i / p.topk;
            atomicOr(&tokens[slot_of_expert(words, before, ids[i])][t >> 5], 1u << (t & 31));
        }
    __syncthreads();
    if (tid < 64) {
        // tiles before each slot: a lane adds up its run of slots, the wave the lanes
        const int run = (used + 63) / 64, s0 = tid * run < used ? tid * run : used, s1 = s0 + run < used ? s0 + run : used;
        int sum = 0;
        for (int s = s0; s < s1; s++) sum += (__popc(tokens[s][0]) + __popc(tokens[s][1]) + 15) / 16;
        int all = sum;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(all, d);
            if (tid >= d) all += o;
        }
        int b = all - sum;
        for (int s = s0; s < s1; s++) {
            base[s] = b;
            b += (__popc(tokens[s][0]) + __popc(tokens[s][1]) + 15) / 16;
        }
        if (tid == 63) base[used] = all;
    }
    __syncthreads();
    for (int s = tid; s <= used; s += 256) plan.base[s] = base[s];
    if (tid == 0) *plan.used = used;
    for (int i = tid; i < 16 * base[used]; i += 256) {      // places without a token keep this
        plan.token[i] = plan.pair[i] = -1;
        plan.weight[i] = 0.0f;
    }
    __syncthreads();
    for (int i = tid; i < n; i += 256) {
        int place = -1;
        if (first_choice(p, ids, i)) {
            const int e = ids[i], t = i / p.topk, s = slot_of_expert(words, before, e);
            const uint32_t low = t < 32 ? 0 : tokens[s][0], at = tokens[s][t >> 5] & ((1u << (t & 31)) - 1);
            place = 16 * base[s] + __popc(low) + __popc(at);
            float w = 0.0f;
            for (int j = 0; j < p.topk; j++)
                if (ids[t * p.topk + j] == e) w += weights[t * p.topk + j];
            plan.token[place] = t;
            plan.pair[place] = i;
            plan.weight[place] = w;
        }
        plan.place[i] = place;
    }
}

// Runs a slot's steps [k0, k1) with NT token tiles: weight rows of RT tiles at wp (lane's own), their block scales at sp,
// activations through x(regs, tile, k block).
template <int RT, int SG, int NT, int DEPTH, int SRC, bool EXACT, class LoadX>
__device__ __forceinline__ void stream_slot(const uint8_t* const (&wp)[RT], const float* const (&sp)[SG], int k0, int k1,
                                            int source, LoadX&& load_x, v4f (&acc)[RT][NT]) {
    using Regs = StepRegs<RT, SG, NT, SRC>;
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[r][t] = v4f{0.f, 0.f, 0.f, 0.f};
    int lk = k0;
    stream_steps<DEPTH, Regs>(k0, k1,
        [&](Regs& b) {
            const int64_t k = (int64_t)lk * BK;
#pragma unroll
            for (int r = 0; r < RT; r++) {
                b.w[r][0] = load_weight(wp[r] + k);
                b.w[r][1] = load_weight(wp[r] + k + 64);
            }
#pragma unroll
            for (int s = 0; s < SG; s++) b.ws[s] = sp[s][lk];
#pragma unroll
            for (int t = 0; t < NT; t++) load_x(b.x[t], t, lk);
            lk = lk + 1 < k1 ? lk + 1 : lk;
        },
        [&](Regs& b) { consume<RT, SG, NT, SRC, EXACT>(b, 0, (1 << NT) - 1, source, acc); });
}

template <int RG, int NW>
__global__ __launch_bounds__(NW * 64) void fg_moe_up_many_kernel(FgMoe p, MoePlan plan, float* __restrict__ h) {
    constexpr int RT = 2 * RG;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    float* red = reinterpret_cast<float*>(smem);                          // [NW][gate, up][tile][4][64]

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4, z = lane_zero(), source = operand_source(lane);
    const int nblk = (int)(p.I / (16 * RG));
    const int slot = (int)blockIdx.x / nblk;
    const int64_t n0 = (int64_t)((int)blockIdx.x % nblk) * (16 * RG);
    if (slot >= *plan.used) return;
    const int e = plan.list[slot], tile0 = plan.base[slot], nt = plan.base[slot + 1] - tile0;

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

    auto run = [&](auto count) {
        constexpr int NT = decltype(count)::value;
        // Places without a token read the slot's first one (three tiles run as four, the last one without a token).
        const uint8_t* xp[NT];
        int xt[NT];
        const int some = plan.token[16 * tile0];
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const int a = t < nt ? plan.token[16 * (tile0 + t) + load_row(lane)] : -1, b = t < nt ? plan.token[16 * (tile0 + t) + l16] : -1;
            xp[t] = plan.xq + (a >= 0 ? a : some) * p.H;
            xt[t] = b >= 0 ? b : some;
        }
        v4f acc[RT][NT];
        stream_slot<RT, 2, NT, NT == 1 ? 2 : 1, SRC_ROWS, true>(wp, sp, k0, k1, source,
            [&](ActRegs<SRC_ROWS>& x, int t, int k) { x.load(xp[t], plan.sx + k * p.T + xt[t], (int64_t)k * BK, lane); }, acc);
#pragma unroll
        for (int r = 0; r < RG; r++) {
            if (r > 0) __syncthreads();             // the last pass's sums are read
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    red[((wave * 2 + 0) * NT + t) * 256 + q * 64 + lane] = acc[r][t][q];
                    red[((wave * 2 + 1) * NT + t) * 256 + q * 64 + lane] = acc[RG + r][t][q];
                }
            __syncthreads();
            for (int t = wave; t < NT && t < nt; t += NW) {
                const int pair = plan.pair[16 * (tile0 + t) + l16];
                if (pair < 0) continue;
                v4f v;
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    float gate = 0.0f, up = 0.0f;
#pragma unroll
                    for (int w = 0; w < NW; w++) {
                        gate += red[((w * 2 + 0) * NT + t) * 256 + q * 64 + lane];
                        up += red[((w * 2 + 1) * NT + t) * 256 + q * 64 + lane];
                    }
                    v[q] = fg_act_any(p.act, gate) * up;
                }
                const int64_t n = n0 + 16 * r + 4 * g;
                *reinterpret_cast<v4f*>(h + (int64_t)pair * p.I + (n & ~127) + hidden_at((int)(n & 127))) = v;
            }
        }
    };
    if (nt == 1) run(std::integral_constant<int, 1>{});
    else if (nt == 2) run(std::integral_constant<int, 2>{});
    else run(std::integral_constant<int, 4>{});
}

// The hidden values of the choices that have a place, as operands.
__global__ __launch_bounds__(256) void fg_moe_quant_kernel(FgMoe p, MoePlan plan, const float* __restrict__ h) {
    const int lane16 = threadIdx.x & 15;
    const int64_t groups = p.I / BK, rows = p.T * p.topk;
    const int64_t id = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4), r = id / groups, g = id % groups;
    const int place = r < rows ? plan.place[r] : -1;
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (place >= 0) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const v4f v = *reinterpret_cast<const v4f*>(h + r * p.I + g * BK + hidden_at(lane16 * 8 + 4 * i));
#pragma unroll
            for (int q = 0; q < 4; q++) f[4 * i + q] = v[q];
        }
    }
    float s;
    const uint2 c = quant_tile(f, p.pow2, s);
    if (place < 0) return;
    const int64_t block = (int64_t)(place >> 4) * groups + g;
    *reinterpret_cast<uint2*>(plan.hq + block * 2048 + operand_at(place & 15, 8 * lane16)) = c;
    if (lane16 == 0) plan.sh[block * 16 + (place & 15)] = s;
}

// The waves' sums of the tokens lie in LDS, [wave][64 tokens][16 RT columns], rows 16 bytes longer than that so that 16
// tokens' 16-byte pieces spread over the banks. A slot's tokens are different ones, so its lanes never meet.
template <int RT, int NW>
__global__ __launch_bounds__(NW * 64) void fg_moe_down_many_kernel(FgMoe p, MoePlan plan, float* __restrict__ partial) {
    constexpr int ROW = 16 * RT + 4;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4, z = lane_zero(), source = operand_source(lane);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);
    const int tokens = (int)p.T;
    float* sums = reinterpret_cast<float*>(smem);                         // [NW][tokens][ROW]
    float* own = sums + wave * tokens * ROW;
    for (int i = lane; i < tokens * ROW / 4; i += 64) reinterpret_cast<v4f*>(own)[i] = v4f{0.f, 0.f, 0.f, 0.f};

    const int nkb = (int)(p.I / BK), used = *plan.used;
    const int steps = used * nkb;
    // this wave's share of all slots' K blocks, over the workgroups of one column block (grid y)
    const int parts = NW * (int)gridDim.y, part = (int)blockIdx.y * NW + wave;
    const int k0 = (int)((int64_t)steps * part / parts), k1 = (int)((int64_t)steps * (part + 1) / parts);
    for (int k = k0; k < k1;) {
        const int slot = k / nkb, ka = k % nkb, kb = k1 - k < nkb - ka ? ka + (k1 - k) : nkb;
        k += kb - ka;
        const int e = plan.list[slot], tile0 = plan.base[slot], nt = plan.base[slot + 1] - tile0;
        const uint8_t* wp[RT];
#pragma unroll
        for (int r = 0; r < RT; r++) wp[r] = p.w2q + ((int64_t)e * p.H + n0 + 16 * r + load_row(lane)) * p.I + 16 * load_group(lane);
        const float* sp[1] = {p.s2 + ((int64_t)e * (p.H / 128) + n0 / 128) * nkb + z};
        auto run = [&](auto count) {
            constexpr int NT = decltype(count)::value;
            int tok[NT];
            float w[NT];
#pragma unroll
            for (int t = 0; t < NT; t++) {
                tok[t] = t < nt ? plan.token[16 * (tile0 + t) + l16] : -1;
                w[t] = t < nt ? plan.weight[16 * (tile0 + t) + l16] : 0.0f;
            }
            v4f acc[RT][NT];
            stream_slot<RT, 1, NT, NT == 4 ? 2 : 3, SRC_OPERAND, false>(wp, sp, ka, kb, source,
                [&](ActRegs<SRC_OPERAND>& x, int t, int kk) {
                    x.load(plan.hq, plan.sh, (int64_t)(tile0 + (t < nt ? t : 0)) * nkb + kk, lane);
                }, acc);
#pragma unroll
            for (int t = 0; t < NT; t++) {
                if (tok[t] < 0) continue;
#pragma unroll
                for (int r = 0; r < RT; r++) {
                    v4f* s = reinterpret_cast<v4f*>(own + tok[t] * ROW + 16 * r + 4 * g);
                    v4f v = *s;
#pragma unroll
                    for (int q = 0; q < 4; q++) v[q] = __builtin_fmaf(w[t], acc[r][t][q], v[q]);
                    *s = v;
                }
            }
        };
        if (nt == 1) run(std::integral_constant<int, 1>{});
        else if (nt == 2) run(std::integral_constant<int, 2>{});
        else run(std::integral_constant<int, 4>{});
    }
    __syncthreads();
    for (int i = tid; i < tokens * 4 * RT; i += NW * 64) {
        const int tok = i / (4 * RT), n = i % (4 * RT) * 4;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; w++) {
            const v4f s = *reinterpret_cast<const v4f*>(sums + (w * tokens + tok) * ROW + n);
#pragma unroll
            for (int q = 0; q < 4; q++) v[q] += s[q];
        }
        if (gridDim.y > 1) *reinterpret_cast<float4*>(partial + ((int64_t)blockIdx.y * p.T + tok) * p.H + n0 + n) = make_float4(v[0], v[1], v[2], v[3]);
        else store_four(p, tok, n0 + n, v);
    }
}

// ---- launches ---------------------------------------------------------------------------------------------

// Joins the partial sums of the down-projection's workgroups, in order.
__global__ __launch_bounds__(256) void fg_moe_join_kernel(FgMoe p, const float* __restrict__ partial, int splits) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, tok = id / (p.H / 4), n = id % (p.H / 4) * 4;
    if (tok >= p.T) return;
    v4f part[kMaxSplits];
#pragma unroll
    for (int i = 0; i < kMaxSplits; i++)          // all loads at once; those past the last split read it again
        part[i] = *reinterpret_cast<const v4f*>(partial + ((i < splits ? i : splits - 1) * p.T + tok) * p.H + n);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kMaxSplits; i++)
#pragma unroll
        for (int q = 0; q < 4; q++) v[q] += i < splits ? part[i][q] : 0.0f;
    store_four(p, tok, n, v);
}

template <class Kernel>
hipError_t raise_lds(Kernel kern, int bytes, std::atomic<uint64_t>& done) {
    return bytes > 65536 ? fg_set_lds_limit_once((const void*)kern, 128 * 1024, done) : hipSuccess;
}

template <int RG, int NW, int DEPTH>
hipError_t launch_up(const FgMoe& p, float* h, int64_t slots, hipStream_t stream) {
    hipLaunchKernelGGL((fg_moe_up_kernel<RG, NW, DEPTH>), dim3((unsigned)(slots * (p.I / (16 * RG)))), dim3(NW * 64), 0, stream, p, h);
    return hipGetLastError();
}

template <int RT, int DEPTH>
hipError_t launch_down(const FgMoe& p, const float* h, float* partial, int splits, hipStream_t stream) {
    hipLaunchKernelGGL((fg_moe_down_kernel<RT, kDownWaves, DEPTH>), dim3((unsigned)(p.H / (16 * RT)), (unsigned)splits),
                       dim3(kDownWaves * 64), 0, stream, p, h, partial);
    return hipGetLastError();
}

template <int RG, int NW>
hipError_t launch_up_many(const FgMoe& p, const MoePlan& plan, float* h, int64_t slots, hipStream_t stream) {
    const int lds = NW * 2 * (p.T > 32 ? 4 : 2) * 1024;
    hipLaunchKernelGGL((fg_moe_up_many_kernel<RG, NW>), dim3((unsigned)(slots * (p.I / (16 * RG)))), dim3(NW * 64), lds, stream, p, plan, h);
    return hipGetLastError();
}

template <int RT>
hipError_t launch_down_many(const FgMoe& p, const MoePlan& plan, float* partial, int splits, hipStream_t stream) {
    auto kern = fg_moe_down_many_kernel<RT, kDownWaves>;
    const int lds = kDownWaves * (int)p.T * (16 * RT + 4) * 4;
    static std::atomic<uint64_t> lds_limit_set{0};
    const hipError_t e = raise_lds(kern, lds, lds_limit_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)(p.H / (16 * RT)), (unsigned)splits), dim3(kDownWaves * 64), lds, stream, p, plan, partial);
    return hipGetLastError();
}

}  // namespace

int64_t fg_moe_workspace_bytes(int64_t T, int topk, int64_t H, int64_t I) { return MoeWorkspace(T, topk, H, I).bytes; }

hipError_t fg_launch_moe_few_tokens(const FgMoe& p, hipStream_t stream) {
    const MoeWorkspace at(p.T, p.topk, p.H, p.I);
    uint8_t* ws = (uint8_t*)p.workspace;
    float *h = (float*)ws, *partial = (float*)(ws + at.partial);
    const MoeLaunch shape(p.T, p.topk, p.E, p.H, p.I);
    const int64_t slots = shape.slots;
    const int tiles = shape.tiles, splits = shape.splits;
    hipError_t e = hipSuccess;
    if (p.T <= kFusedTokens) {
        // 32 gate and 32 up rows a workgroup (they share the token's quantization) where that leaves three quarters of the CUs
        // one: 6 experts, H = 2048, I = 1024 (192 workgroups) 21.5 us for the call against 24.0; 2 experts, H = 4096,
        // I = 2048 (128) 23.2 against 21.6 with 16 rows
        if (p.I > 0) e = 4 * slots * (p.I / 32) >= 3 * fg_device_cus() ? launch_up<2, 4, 2>(p, h, slots, stream) : launch_up<1, 8, 1>(p, h, slots, stream);
        if (e == hipSuccess)
            e = tiles == 2 ? launch_down<2, 2>(p, h, partial, splits, stream) : launch_down<1, 1>(p, h, partial, splits, stream);
    } else {
        const MoePlan plan = at.of(ws);
        const int64_t x_tiles = p.T * (p.H / BK), h_tiles = at.rows * (p.I / BK);
        hipLaunchKernelGGL(fg_moe_plan_kernel, dim3((unsigned)((x_tiles + 15) / 16 + 1)), dim3(256), 0, stream, p, plan);
        e = hipGetLastError();
        if (e == hipSuccess && p.I > 0) e = launch_up_many<2, 4>(p, plan, h, slots, stream);
        if (e == hipSuccess && p.I > 0) {
            hipLaunchKernelGGL(fg_moe_quant_kernel, dim3((unsigned)((h_tiles + 15) / 16)), dim3(256), 0, stream, p, plan, h);
            e = hipGetLastError();
        }
        if (e == hipSuccess) e = launch_down_many<2>(p, plan, partial, splits, stream);
    }
    if (e != hipSuccess || splits == 1) return e;
    hipLaunchKernelGGL(fg_moe_join_kernel, dim3((unsigned)((p.T * p.H / 4 + 255) / 256)), dim3(256), 0, stream, p, partial, splits);
    return hipGetLastError();
}
