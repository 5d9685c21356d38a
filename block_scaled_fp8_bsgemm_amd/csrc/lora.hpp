// lora.hpp -- the second low-rank product, shared by lora_expand and the GEMM
// that adds it to its accumulators: delta[m] = scale[a] (H[m] B[a]^T) by bf16
// MFMAs.
//
// H is fp32 and the MFMA takes bf16, so scale * H is split into two bf16,
// hi = bf16(v) and lo = bf16(v - hi), with a product each: together they carry
// v to 2^-17 relative, while one bf16 alone would add an error of 2^-9 to every
// delta before the sum is rounded to bf16.  R is small next to K and N, and
// the products are a few percent of what these kernels wait for.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// Column, within a wave's 64, of fragment row r of MFMA sub-tile j: lane l
// then holds columns 8 (l/16) .. +8 in sub-tiles 0 and 1 and 32 + 8 (l/16)
// .. +8 in sub-tiles 2 and 3 (the GEMM's order of B rows within a wave).
__device__ __forceinline__ int lora_col(int j, int r) {
    return 32 * (j >> 1) + 8 * (r >> 2) + 4 * (j & 1) + (r & 3);
}

// Row n of adapter a's B; a column past N takes the last one, whose result
// is not stored.
__device__ __forceinline__ const uint16_t *lora_brow(const LoraArgs &g, int a, int64_t n, int64_t N) {
    return g.B + ((int64_t)a * N + (n < N ? n : N - 1)) * g.R;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Loads whose lanes may have nothing to load take a valid address all the same
// and select zero afterwards: a branch around each load would keep the compiler from
// issuing them together.
__device__ __forceinline__ v8bf lora_load_b(const uint16_t *row, int r, int R) {
    const u32x4 v = *(const u32x4 *)(row + (r < R ? r : 0));
    const u32x4 z = {0u, 0u, 0u, 0u};
    return __builtin_bit_cast(v8bf, r < R ? v : z);
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
