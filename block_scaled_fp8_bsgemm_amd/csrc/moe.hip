// moe.hip -- the experts of a feed-forward block (gfx950):
//
//   moe_route   a token's experts and their weights from the router's logits
//   moe_fp8     out[m] = base[m] + sum_e w[m,e] W2[e] (act(W1[e] x[m]) * (W3[e] x[m]))
//               for a few tokens, the experts' weights e4m3 with fp32 128x128 scales
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.hpp"
#include "codec.hpp"
#include "launch.hpp"
#include "lora.hpp"

namespace {

// ------------------------------------------------------------------ route --

// A key's order as an unsigned integer: larger key, larger integer; 0 is kept for
// experts that cannot be chosen.
__device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);   // -0 ranks as 0
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered(uint64_t k) {
    return __builtin_bit_cast(double, (k >> 63) ? k & 0x7FFFFFFFFFFFFFFFull : ~k);
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int off) {
    return (uint64_t)__shfl_xor((unsigned long long)v, off, 64);
}

__device__ __forceinline__ float load_logit(const RouteArgs &g, int64_t row, int e) {
    const int64_t i = row * g.E + e;
    return g.bf16 ? bf16_lo(((const uint16_t *)g.logits)[i]) : ((const float *)g.logits)[i];
}

// One wave to a row, four rows to a workgroup, experts lane, lane + 64, ... to a lane
// (EPL of them).  Keys are fp64: a chosen expert's key may lie next to one that is
// not chosen, and which of two fp32 keys is larger would go by their roundings.
template <int EPL>
__global__ void __launch_bounds__(256) moe_route_kernel(RouteArgs g) {
    __shared__ uint64_t skey[4][EPL * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = (int64_t)blockIdx.x * 4 + wave;
    if (row >= g.rows) return;   // no barrier below: waves share nothing
    float x[EPL];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = lane + 64 * i;
        x[i] = e < g.E ? load_logit(g, row, e) : -INFINITY;
        top = fmaxf(top, x[i]);
    }
    double inv_sum = 1.0;
    if (g.softmax) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; i++) sum += lane + 64 * i < g.E ? exp((double)x[i] - (double)top) : 0.0;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
        inv_sum = 1.0 / sum;
    }
    const auto score = [&](float v) {
        return g.softmax ? exp((double)v - (double)top) * inv_sum : 1.0 / (1.0 + exp(-(double)v));
    };
    uint64_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = lane + 64 * i;
        bool ok = e < g.E && x[i] > -INFINITY;
        double k = x[i];
        if (g.bias || g.groups > 1) k = score(x[i]);
        if (g.bias) {
            const float b = e < g.E ? g.bias[e] : 0.f;
            ok = ok && b > -INFINITY;
            k += (double)b;
        }
        key[i] = ok && k == k ? ordered(k) : 0;
    }
    if (g.groups > 1) {
#pragma unroll
        for (int i = 0; i < EPL; i++) skey[wave][lane + 64 * i] = key[i];
        __builtin_amdgcn_wave_barrier();
        uint64_t best = 0, second = 0;
        if (lane < g.groups)
            for (int i = 0; i < g.per_group; i++) {
                const uint64_t k = skey[wave][lane * g.per_group + i];
                if (k > best) {
                    second = best;
                    best = k;
                } else if (k > second) {
                    second = k;
                }
            }
        uint64_t rank_key = 0;   // of the sum of the group's largest keys
        if (best) rank_key = ordered(unordered(best) + (g.group_top == 2 && second ? unordered(second) : 0.0));
        int ahead = 0;
        for (int j = 0; j < g.groups; j++) {
            const uint64_t k = (uint64_t)__shfl((unsigned long long)rank_key, j, 64);
            ahead += k > rank_key || (k == rank_key && j < lane) ? 1 : 0;
        }
        const uint64_t keep = __ballot(rank_key != 0 && ahead < g.topk_groups);
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const unsigned grp = ((unsigned)(lane + 64 * i) * g.group_mul) >> 20;
            if (!((keep >> (grp & 63)) & 1)) key[i] = 0;
        }
    }
    int mine = -1;   // lane k's: the expert chosen k-th
    for (int k = 0; k < g.topk; k++) {
        uint64_t best = 0;
        int at = -1;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (key[i] > best) {
                best = key[i];
                at = lane + 64 * i;
            }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const uint64_t b = shfl_xor64(best, off);
            const int a = __shfl_xor(at, off, 64);
            if (b > best || (b == best && (unsigned)a < (unsigned)at)) {
                best = b;
                at = a;
            }
        }
        if (lane == k) mine = at;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (at == lane + 64 * i) key[i] = 0;
    }
    double w = mine >= 0 ? score(load_logit(g, row, mine)) : 0.0;
    if (g.renorm) {
        double sum = w;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
        w = sum == 0.0 ? 0.0 : w / sum;
    }
    if (lane < g.topk) {
        g.ids[row * g.topk + lane] = mine;
        g.weights[row * g.topk + lane] = (float)(w * (double)g.scale);
    }
}

// ---------------------------------------------------------------- experts --
//
// Few tokens are bound by the weights' bytes, 3 D I of each expert in use, so
// neither product rounds its other operand: x is bf16 as it comes, h is fp32 in two
// bf16 (hi + lo, 17 bits), and a weight's e4m3 code is a bf16 value exactly.  Products
// are bf16 MFMAs with fp32 sums, one scale for 64 deep pieces of a 128 x 128 block.
//
//   moe_up    one workgroup: one expert, 16 columns of W1 and the same of W3; its waves
//             split D, and their sums are added in wave order
//   moe_down  one workgroup: 32 columns of out, all experts in ascending order; its
//             waves split I, each with sums of its own for every token, added in wave
//             order at the end
//
// How D and I are split does not depend on the tokens, so a token's result is the
// same in every batch, and nothing is summed by atomics.

constexpr int MOE_WAVES = 8, MOE_NT = MOE_WAVES * 64;
constexpr int MOE_PAIRS = 1024;   // most M * topk
constexpr int MOE_ROWS = 128;     // most M

// The workspace: the experts in use and their tokens, written by moe_up for moe_down,
// and h in two planes of bf16 [M * topk, I].
struct MoeEntry {
    int at;     // token | pair << 8, pair = token * topk + slot
    float w;
};
struct MoeList {
    int *count;         // number of experts in use
    int *expert, *n;    // [slots]: each one's number and how many tokens it has
    MoeEntry *entry;    // [slots][M]
};
__device__ __forceinline__ MoeList moe_list(const MoeArgs &g) {
    MoeList l;
    l.count = (int *)g.ws;
    l.expert = l.count + 64;
    l.n = l.expert + g.slots;
    l.entry = (MoeEntry *)(l.n + g.slots);
    return l;
}

// Sixteen e4m3 codes as bf16, in order.
__device__ __forceinline__ void widen16(u32x4 c, v8bf (&v)[2]) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[e], 1.0f, false);
        const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[e], 1.0f, true);
        v8bf &o = v[e >> 1];
        o[4 * (e & 1)] = a[0]; o[4 * (e & 1) + 1] = a[1];
        o[4 * (e & 1) + 2] = b[0]; o[4 * (e & 1) + 3] = b[1];
    }
}

__device__ __forceinline__ void fold(v4f &acc, const v4f &p, float s) {
#pragma unroll
    for (int e = 0; e < 4; e++) acc[e] = __builtin_fmaf(p[e], s, acc[e]);
}

// The tokens of one workgroup's expert, found from the ids alone.
struct MoeShared {
    int ids[MOE_PAIRS];
    unsigned used[32];          // a bit for each expert
    int expert, n;
    MoeEntry entry[MOE_ROWS];
};

// Finds the `slot`-th expert in use and its tokens (ascending).  False if there are no
// more.  A token that names an expert in several slots counts once, by the first,
// with the sum of their weights.
__device__ __forceinline__ bool moe_find(MoeShared &s, const MoeArgs &g, int slot) {
    const int tid = threadIdx.x, lane = tid & 63, pairs = g.M * g.topk;
    if (tid < 32) s.used[tid] = 0;
    __syncthreads();
    for (int i = tid; i < pairs; i += MOE_NT) {
        const int e = g.ids[i];
        const bool ok = (unsigned)e < (unsigned)g.E;
        s.ids[i] = ok ? e : -1;
        if (ok) atomicOr(&s.used[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    // every wave: the slot-th set bit of the 32 words
    unsigned word = lane < 32 ? s.used[lane] : 0;
    int upto = __popc(word);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up(upto, off, 64);
        if (lane >= off) upto += v;
    }
    const uint64_t hit = __ballot(lane < 32 && upto > slot);
    const int total = __builtin_amdgcn_readlane(upto, 31);
    if (slot == 0 && tid == 0 && blockIdx.x == 0) *moe_list(g).count = total;
    if (!hit) return false;
    const int l = __ffsll((unsigned long long)hit) - 1;
    int skip = slot - (__builtin_amdgcn_readlane(upto, l) - __popc(__builtin_amdgcn_readlane((int)word, l)));
    unsigned w = (unsigned)__builtin_amdgcn_readlane((int)word, l);
    while (skip-- > 0) w &= w - 1;
    const int expert = 32 * l + __ffs(w) - 1;
    if (tid < 64) {   // its tokens
        int n = 0;
        for (int m0 = 0; m0 < g.M; m0 += 64) {
            const int m = m0 + lane;
            int first = -1;
            float weight = 0.f;
            if (m < g.M)
                for (int k = 0; k < g.topk; k++)
                    if (s.ids[m * g.topk + k] == expert) {
                        weight += g.weights[m * g.topk + k];
                        if (first < 0) first = m * g.topk + k;
                    }
            const uint64_t b = __ballot(first >= 0);
            if (first >= 0) s.entry[n + __popcll(b & ((1ull << lane) - 1))] = MoeEntry{m | first << 8, weight};
            n += __popcll(b);
        }
        if (lane == 0) {
            s.expert = expert;
            s.n = n;
        }
    }
    __syncthreads();
    return true;
}

// A wave's share of `units` pieces of 64.
__device__ __forceinline__ int share(int units, int wave) { return units * wave / MOE_WAVES; }

// RT x 16 tokens of the workgroup's expert against its 16 + 16 columns.
template <int RT, int DEPTH>
__device__ __forceinline__ void moe_up_rows(MoeShared &s, v4f (*part)[2 * RT][64], const MoeArgs &g, int r0, int c0,
                                            int wave, int lane) {
    const int fr = lane & 15, fg = lane >> 4;
    const int64_t D = g.D;
    const int e = s.expert, n = s.n;
    const uint8_t *w[2];
    const float *sc[2];
    const int DB = (int)(D / 128);
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int64_t col = ((int64_t)e * 2 + h) * g.I + c0;
        w[h] = g.W13 + (col + fr) * D + 16 * fg;
        sc[h] = g.s13 + col / 128 * DB;
    }
    const uint16_t *x[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) x[i] = g.x + (s.entry[min(r0 + 16 * i + fr, n - 1)].at & 255) * D + 16 * fg;
    v4f acc[2][RT];
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
        for (int i = 0; i < RT; i++) acc[h][i] = (v4f){0.f, 0.f, 0.f, 0.f};
    const int units = DB * 2, first = share(units, wave), end = share(units, wave + 1);
    u32x4 wv[DEPTH][2];
    v8bf xv[DEPTH][RT][2];
    const auto load = [&](int d, int u) {
        u = min(u, end - 1);
#pragma unroll
        for (int h = 0; h < 2; h++) wv[d][h] = __builtin_nontemporal_load((const u32x4 *)(w[h] + 64 * (int64_t)u));
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int q = 0; q < 2; q++) xv[d][i][q] = *(const v8bf *)(x[i] + 64 * (int64_t)u + 8 * q);
    };
    if (first < end) {
#pragma unroll
        for (int d = 0; d < DEPTH; d++) load(d, first + d);
        for (int u0 = first; u0 < end; u0 += DEPTH) {
#pragma unroll
            for (int d = 0; d < DEPTH; d++) {
                const int u = u0 + d;
                if (u >= end) break;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    v8bf wb[2];
                    widen16(wv[d][h], wb);
                    const float scale = sc[h][u >> 1];
#pragma unroll
                    for (int i = 0; i < RT; i++) {
                        v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int q = 0; q < 2; q++)
                            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[q], xv[d][i][q], p, 0, 0, 0);
                        fold(acc[h][i], p, scale);
                    }
                }
                load(d, u + DEPTH);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
        for (int i = 0; i < RT; i++) part[wave][h * RT + i][lane] = acc[h][i];
    __syncthreads();
    if (wave < RT) {
        const int row = r0 + 16 * wave + fr;
        v4f t[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            t[h] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int v = 0; v < MOE_WAVES; v++) t[h] += part[v][h * RT + wave][lane];
        }
        float a[4] = {t[0][0], t[0][1], t[0][2], t[0][3]};
        act_all(a, g.act);
        if (row < n) {
            typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
            v4bf hi, lo;
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const float h = a[q] * t[1][q];
                hi[q] = (__bf16)h;
                lo[q] = (__bf16)(h - (float)hi[q]);
            }
            const int64_t at = (int64_t)(s.entry[row].at >> 8) * g.I + c0 + 4 * fg;
            *(v4bf *)(g.h + at) = hi;
            *(v4bf *)(g.h + g.plane + at) = lo;
        }
    }
    __syncthreads();
}

template <int RTMAX>
__global__ void __launch_bounds__(MOE_NT) moe_up_kernel(MoeArgs g) {
    __shared__ MoeShared s;
    __shared__ v4f part[MOE_WAVES][2 * RTMAX][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = blockIdx.y;
    if (!moe_find(s, g, slot)) return;
    const int n = s.n;
    if (blockIdx.x == 0) {   // the list for moe_down
        const MoeList l = moe_list(g);
        if (threadIdx.x == 0) {
            l.expert[slot] = s.expert;
            l.n[slot] = n;
        }
        if ((int)threadIdx.x < n) l.entry[(int64_t)slot * g.M + threadIdx.x] = s.entry[threadIdx.x];
    }
    const int c0 = blockIdx.x * 16;
    for (int r0 = 0; r0 < n; r0 += 16 * RTMAX) {
        if (RTMAX == 1 || n - r0 <= 16)
            moe_up_rows<1, 4>(s, (v4f(*)[2][64])part, g, r0, c0, wave, lane);
        else if (RTMAX == 2 || n - r0 <= 32)
            moe_up_rows<2, 3>(s, (v4f(*)[4][64])part, g, r0, c0, wave, lane);
        else
            moe_up_rows<RTMAX, 2>(s, part, g, r0, c0, wave, lane);
    }
}

constexpr int DOWN_CT = 2, DOWN_COLS = 16 * DOWN_CT, DOWN_UNITS = 4;
constexpr int DOWN_PITCH = DOWN_COLS + 4;   // floats of a token's sums: rows in different banks

template <int MMAX>
__global__ void __launch_bounds__(MOE_NT) moe_down_kernel(MoeArgs g) {
    __shared__ __attribute__((aligned(16))) float sum[MOE_WAVES][MMAX][DOWN_PITCH];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fg = lane >> 4;
    const int64_t I = g.I;
    const int IB = (int)(I / 128), units = IB * 2;
    const int first = share(units, wave), end = share(units, wave + 1);
    const int64_t n0 = (int64_t)blockIdx.x * DOWN_COLS;
    for (int i = lane; i < MMAX * DOWN_PITCH / 4; i += 64) ((v4f *)sum[wave])[i] = (v4f){0.f, 0.f, 0.f, 0.f};
    const MoeList l = moe_list(g);
    const int experts = min(*l.count, g.slots);
    for (int t = 0; t < experts; t++) {
        const int e = l.expert[t], n = l.n[t];
        const MoeEntry *entry = l.entry + (int64_t)t * g.M;
        const uint8_t *w = g.W2 + ((int64_t)e * g.D + n0 + fr) * I + 16 * fg;
        const float *sc = g.s2 + ((int64_t)e * (g.D / 128) + n0 / 128) * IB;
        for (int u0 = first; u0 < end; u0 += DOWN_UNITS) {
            u32x4 wv[DOWN_UNITS][DOWN_CT];
#pragma unroll
            for (int u = 0; u < DOWN_UNITS; u++)
#pragma unroll
                for (int j = 0; j < DOWN_CT; j++)
                    wv[u][j] = __builtin_nontemporal_load((const u32x4 *)(w + j * 16 * I + 64 * (int64_t)min(u0 + u, end - 1)));
            for (int r0 = 0; r0 < n; r0 += 16) {
                const MoeEntry x = entry[min(r0 + fr, n - 1)];
                const uint16_t *h = g.h + (int64_t)(x.at >> 8) * I + 16 * fg;
                v4f acc[DOWN_CT];
#pragma unroll
                for (int j = 0; j < DOWN_CT; j++) acc[j] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int u = 0; u < DOWN_UNITS; u++) {
                    if (u0 + u >= end) break;
                    v8bf hv[2][2];
#pragma unroll
                    for (int p = 0; p < 2; p++)
#pragma unroll
                        for (int q = 0; q < 2; q++)
                            hv[p][q] = *(const v8bf *)(h + p * g.plane + 64 * (int64_t)(u0 + u) + 8 * q);
                    const float scale = sc[(u0 + u) >> 1];
#pragma unroll
                    for (int j = 0; j < DOWN_CT; j++) {
                        v8bf wb[2];
                        widen16(wv[u][j], wb);
                        v4f p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int q = 0; q < 2; q++)
#pragma unroll
                            for (int z = 0; z < 2; z++)
                                p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[q], hv[z][q], p, 0, 0, 0);
                        fold(acc[j], p, scale);
                    }
                }
                if (r0 + fr < n) {
                    float *row = &sum[wave][x.at & 255][4 * fg];
#pragma unroll
                    for (int j = 0; j < DOWN_CT; j++) {
                        v4f *d = (v4f *)(row + 16 * j);
                        v4f v = *d;
                        fold(v, acc[j], x.w);
                        *d = v;
                    }
                }
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g.M * (DOWN_COLS / 4); i += MOE_NT) {
        const int m = i / (DOWN_COLS / 4), c = i % (DOWN_COLS / 4) * 4;
        v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < MOE_WAVES; q++) v += *(const v4f *)&sum[q][m][c];
        const int64_t at = m * g.D + n0 + c;
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        if (g.base) {
            const u32x2 b = *(const u32x2 *)(g.base + at);
            v[0] += bf16_lo(b[0]); v[1] += bf16_hi(b[0]);
            v[2] += bf16_lo(b[1]); v[3] += bf16_hi(b[1]);
        }
        *(u32x2 *)(g.out + at) = (u32x2){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
}

}  // namespace

int bs_launch_moe_route(RouteArgs g, hipStream_t stream) {
    constexpr int64_t ROWS = (int64_t)1 << 25;   // a launch holds fewer than 2^32 lanes
    const RouteArgs all = g;
    for (int64_t first = 0; first < all.rows; first += ROWS) {
        g.rows = all.rows - first < ROWS ? all.rows - first : ROWS;
        g.logits = (const uint8_t *)all.logits + first * all.E * (all.bf16 ? 2 : 4);
        g.ids = all.ids + first * all.topk;
        g.weights = all.weights + first * all.topk;
        const dim3 grid((unsigned)((g.rows + 3) / 4)), block(256);
        const int rc = g.E <= 64    ? bs_enqueue(moe_route_kernel<1>, grid, block, stream, g)
                       : g.E <= 128 ? bs_enqueue(moe_route_kernel<2>, grid, block, stream, g)
                       : g.E <= 256 ? bs_enqueue(moe_route_kernel<4>, grid, block, stream, g)
                       : g.E <= 512 ? bs_enqueue(moe_route_kernel<8>, grid, block, stream, g)
                                    : bs_enqueue(moe_route_kernel<16>, grid, block, stream, g);
        if (rc != 0) return rc;
    }
    return 0;
}

// Bytes of the list, then of the two planes of h.
static int64_t moe_list_bytes(int64_t M, int64_t slots) {
    const int64_t n = 256 + slots * 8 + slots * M * (int64_t)sizeof(MoeEntry);
    return (n + 255) / 256 * 256;
}
int64_t bs_moe_workspace(int64_t M, int64_t topk, int64_t E, int64_t I) {
    const int64_t slots = E < M * topk ? E : M * topk;
    return moe_list_bytes(M, slots) + 4 * M * topk * I;
}

int bs_launch_moe(MoeArgs g, hipStream_t stream) {
    g.slots = g.E < g.M * g.topk ? g.E : g.M * g.topk;
    g.h = (uint16_t *)((uint8_t *)g.ws + moe_list_bytes(g.M, g.slots));
    g.plane = (int64_t)g.M * g.topk * g.I;
    const dim3 up((unsigned)(g.I / 16), (unsigned)g.slots), down((unsigned)(g.D / DOWN_COLS)), block(MOE_NT);
    int rc = g.M <= 16 ? bs_enqueue(moe_up_kernel<1>, up, block, stream, g)
                       : bs_enqueue(moe_up_kernel<4>, up, block, stream, g);
    if (rc != 0) return rc;
    if (g.M <= 16) return bs_enqueue(moe_down_kernel<16>, down, block, stream, g);
    if (g.M <= 64) return bs_enqueue(moe_down_kernel<64>, down, block, stream, g);
    return bs_enqueue(moe_down_kernel<128>, down, block, stream, g);
}
