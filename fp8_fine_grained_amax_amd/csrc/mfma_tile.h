// Device helpers of the kernels that tile a matrix product: workgroups to XCDs, loads straight to LDS, and the order of an operand's
// rows there.
#pragma once
#include "common.h"

// The LDS swizzle of rows of 128 bytes. gfx950 serves a ds_read_b128 16 lanes (256 B, all 64 banks) at a time, and the 8 rows
// one direct-load instruction writes as 128 B per row. For a [rows][128 B] tile the 16 B chunk c of row r
// is stored at c ^ swz128(r): rows r..r+15 read at one logical chunk land on 16 distinct (row parity,
// chunk) bank groups.
__device__ __forceinline__ int swz128(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// Workgroups are dispatched round-robin over the 8 XCDs (workgroup b runs on XCD b % 8, each XCD with its
// own L2). Map workgroup b of a grid of `total` to a logical tile id so that every XCD holds one contiguous
// range of ids: XCD x gets ids [x * (total / 8) + min(x, total % 8), ...), one per workgroup it runs.
__device__ __forceinline__ int xcd_remap(int b, int total) {
    const int x = b & 7, local = b >> 3;
    const int base = total >> 3, extra = total & 7;
    return x * base + (x < extra ? x : extra) + local;
}

// Raw buffer descriptor over [base, base + 2^32 - 1): stride 0, no swizzle; the range check never
// triggers for the 32-bit offsets the kernels use (the host bounds the sizes so they stay below 2^32).
// The base is wave-uniform by construction; taking it through readfirstlane states so, and the descriptor
// then lives in SGPRs without a per-lane loop.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t fg_buffer_rsrc(const void* base) {
    const uint64_t u = (uint64_t)base;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
    void* b = (void*)(((uint64_t)hi << 32) | lo);
    return __builtin_amdgcn_make_buffer_rsrc(b, (short)0, (int)0xFFFFFFFFu, 0x00020000);
}

// 16-byte direct-to-LDS buffer load (lane l lands at byte 16 l of the LDS destination). The call is
// compiled in the device pass only: the host pass checks this builtin's size operand against its own
// target, rejects 16 without a diagnostic and then drops every kernel that uses it from the host object.
__device__ __forceinline__ void fg_buffer_load_lds16(__amdgpu_buffer_rsrc_t rs, void* lds, uint32_t voffset) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, FG_LDS(lds), 16, voffset, 0, 0, 0);
#endif
}

// s_waitcnt with only the vector-memory count set.
template <int N>
__device__ __forceinline__ void wait_loads() {
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
