// resnorm.hip -- what lies between two blocks of a layer stack, in one pass
// over the row (gfx950):
//
//   p = y / rms(y) * post_w          norm after the block (or p = y)
//   h = alpha * resid + beta * gate * p            the residual stream
//   z = h / rms(h) * pre_w           norm before the next block
//   q = e4m3(z / s)                  the next projection's fp8 operand
//
// with rms(v) = sqrt(mean(v^2) + eps).  y is the block's bf16 output, or the
// gathered fp8 wire that rowdq_e4m3 takes; q has the block scales of actq_e4m3
// (1x128 fp32) or mxq_e4m3 (1x32 E8M0).  Everything between the loads and the
// stores is fp32: each stored value is rounded once, so z and q are those of
// the unrounded h, and q is not taken from a rounded z.
//
// A row stays in its workgroup's registers from load to store, so each byte is
// moved once: the kernel is bound by HBM.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "codec.hpp"
#include "launch.hpp"

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void widen(u32x4 w, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
        v[2 * e] = bf16_lo(w[e]);
        v[2 * e + 1] = bf16_hi(w[e]);
    }
}

__device__ __forceinline__ void decode(u32x2 c, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 2; e++) {
        const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[e], false);
        const v2f b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[e], true);
        v[4 * e] = a[0]; v[4 * e + 1] = a[1];
        v[4 * e + 2] = b[0]; v[4 * e + 3] = b[1];
    }
}

__device__ __forceinline__ u32x4 narrow(const float (&v)[8]) {
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; e++) o[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
    return o;
}

// The sum over the T lanes of a row (T = 64: one wave, no LDS).  A second use
// of red needs no barrier of its own after the first one's reads: it takes
// another slot.
template <int T>
__device__ __forceinline__ float row_sum(float v, float *red) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < T / 64; w++) v += red[w];
    }
    return v;
}

// amax over the G lanes of a scale block (G a power of two, blocks aligned)
template <int G>
__device__ __forceinline__ float group_max(float m) {
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    return m;
}

// T lanes per row, CPT packs of 8 values to a lane (pack tid + T i): rows of
// up to 8 T CPT values.  WIRE: y is e4m3 codes with a row scale.  RES32: the
// residual stream is fp32.  QB: 0, or the scale block of q.
template <int T, int CPT, bool WIRE, bool RES32, int QB>
__global__ void __launch_bounds__(T < 256 ? 256 : T) resnorm_kernel(ResnormArgs g) {
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    __shared__ float red[2][T / 64];
    const int tid = threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / T;
    if (row >= g.rows) return;   // whole waves: T >= 64
    const int64_t base = row * g.nch;
    const float inv_n = 1.0f / (float)(g.nch * 8);

    float v[CPT][8], r[CPT][8];
#pragma unroll
    for (int i = 0; i < CPT; i++) {
        const int c = tid + T * i;
#pragma unroll
        for (int e = 0; e < 8; e++) v[i][e] = r[i][e] = 0.f;
        if (c >= g.nch) continue;
        if constexpr (WIRE) decode(__builtin_nontemporal_load((const u32x2 *)g.y + base + c), v[i]);
        else widen(__builtin_nontemporal_load((const u32x4 *)g.y + base + c), v[i]);
        if constexpr (RES32) {
            const u32x4 a = __builtin_nontemporal_load((const u32x4 *)g.resid + 2 * (base + c));
            const u32x4 b = __builtin_nontemporal_load((const u32x4 *)g.resid + 2 * (base + c) + 1);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                r[i][e] = __uint_as_float(a[e]);
                r[i][4 + e] = __uint_as_float(b[e]);
            }
        } else {
            widen(__builtin_nontemporal_load((const u32x4 *)g.resid + base + c), r[i]);
        }
    }
    if constexpr (WIRE) {
        const float s = g.y_scale[row];
#pragma unroll
        for (int i = 0; i < CPT; i++)
#pragma unroll
            for (int e = 0; e < 8; e++) v[i][e] *= s;
    }
    float mul = g.beta;
    if (g.post_w) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < CPT; i++)
#pragma unroll
            for (int e = 0; e < 8; e++) ss += v[i][e] * v[i][e];
        mul *= 1.0f / sqrtf(row_sum<T>(ss, red[0]) * inv_n + g.eps);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; i++) {
        const int c = tid + T * i;
        if (c >= g.nch) continue;
        if (g.post_w) {
            float w[8];
            widen(((const u32x4 *)g.post_w)[c], w);
#pragma unroll
            for (int e = 0; e < 8; e++) v[i][e] *= w[e];
        }
        if (g.gate) {
            float w[8];
            widen(*((const u32x4 *)(g.gate + row * g.gate_row) + c), w);
#pragma unroll
            for (int e = 0; e < 8; e++) v[i][e] *= w[e];
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
            v[i][e] = g.alpha * r[i][e] + mul * v[i][e];
            ss += v[i][e] * v[i][e];
        }
        if constexpr (RES32) {
            u32x4 a, b;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                a[e] = __float_as_uint(v[i][e]);
                b[e] = __float_as_uint(v[i][4 + e]);
            }
            __builtin_nontemporal_store(a, (u32x4 *)g.resid_out + 2 * (base + c));
            __builtin_nontemporal_store(b, (u32x4 *)g.resid_out + 2 * (base + c) + 1);
        } else {
            __builtin_nontemporal_store(narrow(v[i]), (u32x4 *)g.resid_out + base + c);
        }
    }
    if (QB == 0 && !g.z) return;
    const float rs = 1.0f / sqrtf(row_sum<T>(ss, red[1]) * inv_n + g.eps);
#pragma unroll
    for (int i = 0; i < CPT; i++) {
        const int c = tid + T * i;
        if (c >= g.nch) continue;   // whole scale blocks: N is a multiple of QB
        float w[8], amax = 0.f;
#pragma unroll
        for (int e = 0; e < 8; e++) w[e] = 1.f;
        if (g.pre_w) widen(((const u32x4 *)g.pre_w)[c], w);
#pragma unroll
        for (int e = 0; e < 8; e++) {
            v[i][e] *= rs * w[e];
            amax = fmaxf(amax, fabsf(v[i][e]));
        }
        if (g.z) __builtin_nontemporal_store(narrow(v[i]), (u32x4 *)g.z + base + c);
        if constexpr (QB == 128) {
            const float s = group_max<16>(amax) / 448.0f;
            if ((c & 15) == 0) ((float *)g.q_scale)[(base + c) >> 4] = s;
            const double R = s != 0.0f ? 1.0 / (double)s : 0.0;
            u32x2 o;
#pragma unroll
            for (int e = 0; e < 2; e++)
                o[e] = pack_e4m3x4_sat(wire_quotient(v[i][4 * e], R), wire_quotient(v[i][4 * e + 1], R),
                                       wire_quotient(v[i][4 * e + 2], R), wire_quotient(v[i][4 * e + 3], R));
            if (s == 0.0f) o = (u32x2){0u, 0u};
            __builtin_nontemporal_store(o, (u32x2 *)g.q + base + c);
        } else if constexpr (QB == 32) {
            // the smallest k with amax <= 448 * 2^k, from amax's IEEE bits
            const float m = group_max<4>(amax);
            const uint32_t bits = __float_as_uint(m);
            const int ef = (int)(bits >> 23);
            int k = (ef - 127) - ((bits & 0x7FFFFFu) > 0x600000u ? 7 : 8);
            if (ef == 0 || k < -127) k = -127;
            if (k > 120) k = 120;   // an infinite or NaN amax
            if ((c & 3) == 0) ((uint8_t *)g.q_scale)[(base + c) >> 2] = m == 0.0f ? 0 : (uint8_t)(k + 127);
            const float inv = __uint_as_float((uint32_t)(127 - k) << 23);   // 2^-k
            u32x2 o;
#pragma unroll
            for (int e = 0; e < 2; e++)
                o[e] = pack_e4m3x4(v[i][4 * e] * inv, v[i][4 * e + 1] * inv, v[i][4 * e + 2] * inv,
                                   v[i][4 * e + 3] * inv);
            if (m == 0.0f) o = (u32x2){0u, 0u};
            __builtin_nontemporal_store(o, (u32x2 *)g.q + base + c);
        }
    }
}

template <int T, int CPT, bool WIRE, bool RES32>
int launch_q(const ResnormArgs &g, int q_block, dim3 grid, dim3 block, hipStream_t stream) {
    if (q_block == 128) return bs_enqueue(resnorm_kernel<T, CPT, WIRE, RES32, 128>, grid, block, stream, g);
    if (q_block == 32) return bs_enqueue(resnorm_kernel<T, CPT, WIRE, RES32, 32>, grid, block, stream, g);
    return bs_enqueue(resnorm_kernel<T, CPT, WIRE, RES32, 0>, grid, block, stream, g);
}

template <int T, int CPT>
int launch_t(const ResnormArgs &g, bool resid_f32, int q_block, hipStream_t stream) {
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    const dim3 grid((unsigned)((g.rows + ROWS - 1) / ROWS)), block(T < 256 ? 256 : T);
    if (g.y_scale)
        return resid_f32 ? launch_q<T, CPT, true, true>(g, q_block, grid, block, stream)
                         : launch_q<T, CPT, true, false>(g, q_block, grid, block, stream);
    return resid_f32 ? launch_q<T, CPT, false, true>(g, q_block, grid, block, stream)
                     : launch_q<T, CPT, false, false>(g, q_block, grid, block, stream);
}

}  // namespace

int bs_launch_resnorm(const ResnormArgs &g, bool resid_f32, int q_block, hipStream_t stream) {
    if (g.rows > 0x7FFFFFFF) return -1;
    if (g.nch <= 128) return launch_t<64, 2>(g, resid_f32, q_block, stream);
    if (g.nch <= 512) return launch_t<256, 2>(g, resid_f32, q_block, stream);
    if (g.nch <= 1024) return launch_t<256, 4>(g, resid_f32, q_block, stream);
    return launch_t<512, 4>(g, resid_f32, q_block, stream);
}
