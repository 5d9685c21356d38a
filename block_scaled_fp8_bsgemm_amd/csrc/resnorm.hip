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
// moved once: the kernel is bound by HBM.  16384 wire rows of 7168 with a bf16
// residual to 1x128 codes: 118 us, 6.0 TB/s, reading and writing its 676 MiB once; 4096
// bf16 rows of 5120 with an fp32 residual to bf16 and 1x32 codes: 50 us, 5.5 TB/s;
// one row of 7168: 4.7 us.
#include <float.h>
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

// The sum of a row's squares from each lane's P partial sums, one for every two of its
// packs.  A row's 128 consecutive packs are summed over 64 lanes, two packs to each,
// and those sums are added in the order of the packs: the same additions whether a
// lane holds two packs (P = 1, a wave covers 128) or four (P = 2, 256), so a row's result
// does not depend on how many rows the call has.  WAVE: the row is one wave's;
// otherwise the workgroup's waves meet in red, another one for each use, which needs
// no barrier after the reads.
template <bool WAVE, int P>
__device__ __forceinline__ float row_sum(float (&v)[P], float *red) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
#pragma unroll
        for (int h = 0; h < P; h++) v[h] += __shfl_xor(v[h], off, 64);
    if constexpr (WAVE) {
        static_assert(P == 1, "a wave's row has at most 128 packs");
        return v[0];
    } else {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int h = 0; h < P; h++) red[(threadIdx.x >> 6) * P + h] = v[h];
        }
        __syncthreads();
        float sum = 0.f;
        for (unsigned w = 0; w < blockDim.x / 64; w++)
#pragma unroll
            for (int h = 0; h < P; h++) sum += red[w * P + h];
        return sum;
    }
}

// 1 / rms of a row whose squares sum to `sum`.  Where finite values of 2^57 and more
// take that sum past fp32, the row's values are multiplied by 2^-80 and summed
// again, and the result is the reciprocal for the smaller values: their normed ones
// are the same.  Only such rows, and those that are not finite, take the second sum.
template <int CPT, bool WAVE>
__device__ __forceinline__ float inv_rms(float sum, float (&v)[CPT][8], int first, const ResnormArgs &g, float *red) {
    const float inv_n = 1.0f / (float)(g.nch * 8);
    float eps = g.eps;
    if (!(sum <= FLT_MAX)) {   // the same for all of the row's lanes
        float ss[CPT / 2];
#pragma unroll
        for (int i = 0; i < CPT; i++) {
            float sq = 0.f;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                v[i][e] *= 0x1p-80f;
                sq += v[i][e] * v[i][e];
            }
            if (i % 2 == 0) ss[i / 2] = 0.f;
            ss[i / 2] += first + 64 * i < g.nch ? sq : 0.f;
        }
        sum = row_sum<WAVE>(ss, red);
        eps = eps * 0x1p-80f * 0x1p-80f;
    }
    return 1.0f / sqrtf(sum * inv_n + eps);
}

// The larger of two values, NaN if either is (fmaxf drops NaN, and a block of
// NaN would get the scale 0 of a block of zeros).
__device__ __forceinline__ float nan_max(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// amax over the G lanes of a scale block (G a power of two, blocks aligned)
template <int G>
__device__ __forceinline__ float group_max(float m) {
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1) m = nan_max(m, __shfl_xor(m, off, 64));
    return m;
}

// CPT packs of 8 values to a lane, 64 CPT consecutive packs to a wave (lane l its
// packs l + 64 i).  WAVE: a wave takes a whole row, four rows to a workgroup;
// otherwise the workgroup's waves share one.  WIRE: y is e4m3 codes with a row scale.
// RES32: the residual stream is fp32.  QB: 0, or the scale block of q.
//
// Every load, the weights' and the gate's too, goes out before the first
// reduction.  A lane past the row's end loads the last pack, counts as zero and
// stores nothing, so that no load is behind a branch.
template <int CPT, bool WAVE, bool WIRE, bool RES32, int QB>
__global__ void __launch_bounds__(512) resnorm_kernel(ResnormArgs g) {
    constexpr int P = CPT / 2;   // partial sums of squares to a lane
    __shared__ float red[4][8 * P];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int first = lane + (WAVE ? 0 : wave * 64 * CPT);
    const int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
    if (row >= g.rows) return;   // whole waves of a WAVE workgroup
    const int64_t base = row * g.nch;

    u32x4 yw[CPT], ra[CPT], rb[CPT], pw[CPT], gw[CPT], ww[CPT];
    const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};   // bf16 1.0
#pragma unroll
    for (int i = 0; i < CPT; i++) {
        const int c = min(first + 64 * i, g.nch - 1);
        if constexpr (WIRE) {
            const u32x2 q = __builtin_nontemporal_load((const u32x2 *)g.y + base + c);
            yw[i] = (u32x4){q[0], q[1], 0u, 0u};
        } else {
            yw[i] = __builtin_nontemporal_load((const u32x4 *)g.y + base + c);
        }
        if constexpr (RES32) {
            // each of the two takes every other 16 bytes, so the lines have to stay in L1
            // between them: non-temporal they took 56.6 us against 49.8 (4096 x 5120)
            ra[i] = *((const u32x4 *)g.resid + 2 * (base + c));
            rb[i] = *((const u32x4 *)g.resid + 2 * (base + c) + 1);
        } else {
            ra[i] = __builtin_nontemporal_load((const u32x4 *)g.resid + base + c);
        }
    }
    const float ys = WIRE ? g.y_scale[row] : 1.0f;
#pragma unroll
    for (int i = 0; i < CPT; i++) {
        const int c = min(first + 64 * i, g.nch - 1);
        pw[i] = g.post_w ? ((const u32x4 *)g.post_w)[c] : ones;
        gw[i] = g.gate ? *((const u32x4 *)(g.gate + row * g.gate_row) + c) : ones;
        ww[i] = g.pre_w ? ((const u32x4 *)g.pre_w)[c] : ones;
    }

    float v[CPT][8];
    float mul = g.beta;
    float ss[P];
#pragma unroll
    for (int h = 0; h < P; h++) ss[h] = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; i++) {
        if constexpr (WIRE) decode((u32x2){yw[i][0], yw[i][1]}, v[i]);
        else widen(yw[i], v[i]);
        const float live = first + 64 * i < g.nch ? 1.f : 0.f;
        float sq = 0.f;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            if (WIRE) v[i][e] *= ys;
            sq += v[i][e] * v[i][e];
        }
        ss[i / 2] += live != 0.f ? sq : 0.f;
    }
    if (g.post_w) mul *= inv_rms<CPT, WAVE>(row_sum<WAVE>(ss, red[0]), v, first, g, red[2]);
#pragma unroll
    for (int h = 0; h < P; h++) ss[h] = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; i++) {
        const int c = first + 64 * i;
        float p[8], q[8], r[8], sq = 0.f;
        widen(pw[i], p);
        widen(gw[i], q);
        if constexpr (RES32) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                r[e] = __uint_as_float(ra[i][e]);
                r[4 + e] = __uint_as_float(rb[i][e]);
            }
        } else {
            widen(ra[i], r);
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
            v[i][e] = g.alpha * r[e] + mul * (v[i][e] * p[e] * q[e]);
            sq += v[i][e] * v[i][e];
        }
        if (c >= g.nch) continue;
        ss[i / 2] += sq;
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
    const float rs = inv_rms<CPT, WAVE>(row_sum<WAVE>(ss, red[1]), v, first, g, red[3]);
#pragma unroll
    for (int i = 0; i < CPT; i++) {
        const int c = first + 64 * i;
        if (c >= g.nch) continue;   // whole scale blocks: N is a multiple of QB
        float w[8], amax = 0.f;
        widen(ww[i], w);
#pragma unroll
        for (int e = 0; e < 8; e++) {
            v[i][e] *= rs * w[e];
            amax = nan_max(amax, fabsf(v[i][e]));
        }
        if (g.z) __builtin_nontemporal_store(narrow(v[i]), (u32x4 *)g.z + base + c);
        if constexpr (QB == 128) {
            const float s = group_max<16>(amax) / 448.0f;
            if ((c & 15) == 0) ((float *)g.q_scale)[(base + c) >> 4] = s;
            u32x2 o = {0u, 0u};
            if (!(s < 0x1p-126f)) {
                // z * (1/s): z is itself rounded, so a quotient exact to the last bit
                // would say no more; |z| / s stays below 448.0002.  A NaN scale gives NaN
                // codes, an infinite one a NaN code where z is infinite and 0 elsewhere.
                const float inv = 1.0f / s;
#pragma unroll
                for (int e = 0; e < 2; e++)
                    o[e] = pack_e4m3x4(v[i][4 * e] * inv, v[i][4 * e + 1] * inv, v[i][4 * e + 2] * inv,
                                       v[i][4 * e + 3] * inv);
            } else if (s != 0.0f) {   // a subnormal scale, whose reciprocal may not exist in fp32
                const double R = 1.0 / (double)s;
#pragma unroll
                for (int e = 0; e < 2; e++)
                    o[e] = pack_e4m3x4_sat(wire_quotient(v[i][4 * e], R), wire_quotient(v[i][4 * e + 1], R),
                                           wire_quotient(v[i][4 * e + 2], R), wire_quotient(v[i][4 * e + 3], R));
            }
            __builtin_nontemporal_store(o, (u32x2 *)g.q + base + c);
        } else if constexpr (QB == 32) {
            // the smallest k with amax <= 448 * 2^k, from amax's IEEE bits
            const float m = group_max<4>(amax);
            const uint32_t bits = __float_as_uint(m);
            const int ef = (int)(bits >> 23);
            int k = (ef - 127) - ((bits & 0x7FFFFFu) > 0x600000u ? 7 : 8);
            if (ef == 0 || k < -127) k = -127;
            const bool nan = ef == 255;   // NaN or infinite: E8M0's NaN, and NaN codes
            if ((c & 3) == 0)
                ((uint8_t *)g.q_scale)[(base + c) >> 2] = m == 0.0f ? 0 : nan ? 0xFF : (uint8_t)(k + 127);
            const float inv = nan ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(127 - k) << 23);   // 2^-k
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

template <int CPT, bool WAVE, bool WIRE, bool RES32>
int launch_q(const ResnormArgs &g, int q_block, dim3 grid, dim3 block, hipStream_t stream) {
    if (q_block == 128) return bs_enqueue(resnorm_kernel<CPT, WAVE, WIRE, RES32, 128>, grid, block, stream, g);
    if (q_block == 32) return bs_enqueue(resnorm_kernel<CPT, WAVE, WIRE, RES32, 32>, grid, block, stream, g);
    return bs_enqueue(resnorm_kernel<CPT, WAVE, WIRE, RES32, 0>, grid, block, stream, g);
}

template <int CPT, bool WAVE>
int launch_t(const ResnormArgs &g, bool resid_f32, int q_block, hipStream_t stream) {
    const dim3 grid((unsigned)(WAVE ? (g.rows + 3) / 4 : g.rows));
    const dim3 block(WAVE ? 256 : (g.nch + 64 * CPT - 1) / (64 * CPT) * 64);
    if (g.y_scale)
        return resid_f32 ? launch_q<CPT, WAVE, true, true>(g, q_block, grid, block, stream)
                         : launch_q<CPT, WAVE, true, false>(g, q_block, grid, block, stream);
    return resid_f32 ? launch_q<CPT, WAVE, false, true>(g, q_block, grid, block, stream)
                     : launch_q<CPT, WAVE, false, false>(g, q_block, grid, block, stream);
}

// The call's rows from `first` on, `rows` of them at most.
ResnormArgs rows_from(ResnormArgs g, int64_t first, int64_t rows, bool resid_f32, int q_block) {
    const int64_t at = first * g.nch * 8;
    g.y = (const uint8_t *)g.y + at * (g.y_scale ? 1 : 2);
    if (g.y_scale) g.y_scale += first;
    if (g.gate) g.gate += first * g.gate_row;
    g.resid = (const uint8_t *)g.resid + at * (resid_f32 ? 4 : 2);
    g.resid_out = (uint8_t *)g.resid_out + at * (resid_f32 ? 4 : 2);
    if (g.z) g.z += at;
    if (g.q) g.q += at;
    if (q_block) g.q_scale = (uint8_t *)g.q_scale + at / 32;   // n / 128 fp32, or n / 32 bytes
    g.rows = g.rows - first < rows ? g.rows - first : rows;
    return g;
}

}  // namespace

int bs_launch_resnorm(const ResnormArgs &all, bool resid_f32, int q_block, hipStream_t stream) {
    // A launch holds fewer than 2^32 lanes, and a row has at most 512: more rows than
    // 2^22 go in several launches.
    constexpr int64_t ROWS = (int64_t)1 << 22;
    for (int64_t first = 0; first < all.rows; first += ROWS) {
        const ResnormArgs g = rows_from(all, first, ROWS, resid_f32, q_block);
        // a row has as few lanes as hold it in CPT packs each, so that few are idle
        // (N = 7168: 7 waves of 2 packs, or 4 of 4).  Few rows want the shorter chain
        // of 2 packs, many the fewer waves to join: graph launches of wire rows to
        // codes at N = 7168, us for 2 packs / 4: 1 row 3.8 / 4.8, 64 rows 4.1 / 5.1, 511
        // rows 6.7 / 6.9, 1024 rows 11.2 / 10.7, 16384 rows 119 / 117.
        const int rc = g.nch <= 128                       ? launch_t<2, true>(g, resid_f32, q_block, stream)
                       : g.nch <= 1024 && all.rows < 512 ? launch_t<2, false>(g, resid_f32, q_block, stream)
                                                          : launch_t<4, false>(g, resid_f32, q_block, stream);
        if (rc != 0) return rc;
    }
    return 0;
}
