// lora.hpp -- the second low-rank product, shared by lora_expand and the GEMM
// that adds it to its accumulators: delta[m] = scale[a] (H[m] B[a]^T) by bf16
// MFMAs.
//
// H is fp32 and the MFMA takes bf16, so scale * H is split into two bf16,
// hi = bf16(v) and lo = bf16(v - hi), with a product each: together they carry
// v to 2^-17 relative, while one bf16 alone would add an error of 2^-9 to every
// delta before the sum is rounded to bf16.  R is small next to K and N: the
// second product is 2 % of the GEMM with adapters at R = 64 (5 of 256 us).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// A buffer descriptor of `bytes` from base on, past which loads read zero and stores
// are dropped.  Every descriptor is workgroup- or wave-uniform; readfirstlane says so to the
// compiler, which otherwise may keep one in VGPRs and wrap each load through
// it in a loop over distinct values.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *base, int64_t bytes) {
    int32_t n = bytes > 0x7FFFFFFFll ? 0x7FFFFFFF : (bytes > 0 ? (int32_t)bytes : 0);
    const uint64_t b = (uint64_t)base;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
    n = __builtin_amdgcn_readfirstlane(n);
    return __builtin_amdgcn_make_buffer_rsrc((void *)(((uint64_t)hi << 32) | lo), (short)0, n,
                                             0x00020000);
}

typedef __attribute__((address_space(3))) void lds_void;

// A workgroup barrier that leaves vector memory operations in flight:
// __syncthreads() also fences global memory, which makes the compiler wait
// for every outstanding store before it.  The caller waits for what the
// barrier must cover (its DMA) with its own s_waitcnt; the LDS reads issued
// before are waited for here, and the empty asm statements keep the compiler
// from moving memory accesses across the barrier.
__device__ __forceinline__ void barrier_lds_only() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0); vmcnt and expcnt not waited for
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A byte offset past every descriptor, the largest included.
constexpr int OUT_OF_RANGE = (int)0x80000000;

// Column, within a wave's 64, of fragment row r of MFMA sub-tile j: lane l
// then holds columns 8 (l/16) .. +8 in sub-tiles 0 and 1 and 32 + 8 (l/16)
// .. +8 in sub-tiles 2 and 3 (the GEMM's order of B rows within a wave).
__device__ __forceinline__ int lora_col(int j, int r) {
    return 32 * (j >> 1) + 8 * (r >> 2) + 4 * (j & 1) + (r & 3);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Adapter a's rows of B for the columns from n on (n < N).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t lora_rsrc(const LoraArgs &g, int a, int64_t n, int64_t N) {
    return make_rsrc(g.B + ((int64_t)a * N + n) * g.R, (N - n) * g.R * 2);
}

// Eight ranks from r on of the descriptor's row c; zero past N, and past R by an
// offset out of range.  (A branch or a select after the load would keep the compiler
// from issuing loads together.)
__device__ __forceinline__ v8bf lora_load_b(__amdgpu_buffer_rsrc_t b, int c, int r, int R) {
    return __builtin_bit_cast(v8bf,
                              __builtin_amdgcn_raw_buffer_load_b128(b, r < R ? (c * R + r) * 2 : OUT_OF_RANGE, 0, 0));
}

// scale * H[m, r .. r+8) split in two; zero for a row that is not the
// adapter's (live == false) and past R.
struct LoraH {
    v4f a, b;
};
__device__ __forceinline__ LoraH lora_load_h(const LoraArgs &g, int64_t m, bool live, int r) {
    const bool ok = live && r < g.R;
    const v4f *p = (const v4f *)(g.H + (ok ? m * g.R + r : 0));
    LoraH h = {p[0], p[1]};
#pragma unroll
    for (int e = 0; e < 4; e++) {
        h.a[e] = ok ? h.a[e] : 0.f;
        h.b[e] = ok ? h.b[e] : 0.f;
    }
    return h;
}
__device__ __forceinline__ void lora_split(const LoraH &h, float s, v8bf &hi, v8bf &lo) {
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const float v = s * (e < 4 ? h.a[e & 3] : h.b[e & 3]);
        hi[e] = (__bf16)v;
        lo[e] = (__bf16)(v - (float)hi[e]);
    }
}
