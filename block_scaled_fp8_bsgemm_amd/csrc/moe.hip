// moe.hip -- the experts of a feed-forward block (gfx950):
//
//   moe_route   a token's experts and their weights from the router's logits
//   moe_fp8     out[m] = base[m] + sum_e w[m,e] W2[e] (act(W1[e] x[m]) * (W3[e] x[m]))
//               for a few tokens, the experts' weights e4m3 with fp32 128x128 scales
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "act.hpp"
#include "codec.hpp"
#include "launch.hpp"
#include "lora.hpp"

namespace {

// ------------------------------------------------------------------ route --

// One wave to a row, four rows to a workgroup; expert e is lane e / EPL's, so the lowest
// lane that has the largest key has the lowest such expert.
//
// Keys are fp64 by their definition: a chosen expert's key may lie next to one that is
// not chosen, and which of two fp32 keys is larger goes by their roundings.  Without bias
// and groups the key is the logit itself and fp32 is exact.  Otherwise a row is chosen
// by fp32 keys first, and where two keys (or two groups' sums) that the choice or its
// order compares lie closer than what fp32 may be off (route_close), it is chosen again by
// fp64 keys.  That happens to about one row in a hundred of 256 experts with random
// logits; an fp64 exponential for every expert took as long as all the rest.
//
// The selection's instructions bound it, about 900 a row: 16384 rows of 256 experts, sigmoid,
// bias, 4 of 8 groups, 8 experts 24 us (17.8 MB; all by fp64 keys 45), 3001 rows of 60 experts by
// their logits 4.0, 64 rows of 256 with groups 8.8 if one of them needs fp64 keys, else 5.

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_from(int old, int v) {
    return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xF, false);
}
// op over the wave's lanes, left in lane 63: from 1, 2, 4, 8 lanes below within each 16, then
// the 16 below's last lane, then the 32 below's.  `none` stands in where there is no lane.
template <typename Op>
__device__ __forceinline__ int wave_reduce(int v, int none, Op op) {
    v = op(v, dpp_from<0x111, 0xF>(none, v));
    v = op(v, dpp_from<0x112, 0xF>(none, v));
    v = op(v, dpp_from<0x114, 0xF>(none, v));
    v = op(v, dpp_from<0x118, 0xF>(none, v));
    v = op(v, dpp_from<0x142, 0xA>(none, v));
    v = op(v, dpp_from<0x143, 0xC>(none, v));
    return __builtin_amdgcn_readlane(v, 63);
}
constexpr int KEY_NONE = INT_MIN;
__device__ __forceinline__ int wave_max(int v) {
    return wave_reduce(v, KEY_NONE, [](int a, int b) { return max(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
    return __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(int, v), 0, [](int a, int b) {
                                  return __builtin_bit_cast(int, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
                              }));
}
template <int CTRL, int ROWS> __device__ __forceinline__ double max_from(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)dpp_from<CTRL, ROWS>((int)b, (int)b);
    const uint32_t hi = (uint32_t)dpp_from<CTRL, ROWS>((int)(b >> 32), (int)(b >> 32));
    const double o = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    return o > v ? o : v;
}
__device__ __forceinline__ double wave_max(double v) {
    v = max_from<0x111, 0xF>(v);
    v = max_from<0x112, 0xF>(v);
    v = max_from<0x114, 0xF>(v);
    v = max_from<0x118, 0xF>(v);
    v = max_from<0x142, 0xA>(v);
    v = max_from<0x143, 0xC>(v);
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)b, 63), hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// An fp32 key as an integer of the same order (-0 as 0), and back.
__device__ __forceinline__ int ordered(float v) {
    const int b = __builtin_bit_cast(int, v + 0.0f);
    return b ^ (b >> 31 & 0x7FFFFFFF);
}
__device__ __forceinline__ float unordered(int k) { return __builtin_bit_cast(float, k ^ (k >> 31 & 0x7FFFFFFF)); }

__device__ __forceinline__ int first_lane(uint64_t lanes) { return __ffsll((unsigned long long)lanes) - 1; }

// Whether two keys, or sums of two, a that fp32 puts first and b, may be in the other order
// by fp64.  An exponential e^-t by the hardware's and its reciprocal are off by (3 t + 5)
// 2^-24 relative, and softmax's sum by less than 50 2^-24.  So with a bias a sigmoid is off by
// less than 2^-21, all softmax scores together by less than 2^-18, and the key's own rounding is
// 2^-24 of it; the margin is twice as much for either two.  Without one a score is off by
// less than 2^-16 of itself, an eighth of the margin, but only where it is a normal number:
// the hardware gives zero below 2^-126, off by all of its value.  So nothing up to 2^-100 is
// decided here; above that a sum's lost second key is 2^-26 of it.
__device__ __forceinline__ bool route_close(float a, float b, bool biased) {
    const float part = biased ? 0x1p-17f : 0x1p-13f, least = biased ? 0x1p-17f : 0x1p-100f;
    return !(a - b > __builtin_fmaf(part, fabsf(a) + fabsf(b), least));
}

// The largest and second largest key of group `lane`, by way of LDS.
template <typename K>
__device__ __forceinline__ void group_best(const K *key, const RouteArgs &g, int lane, K none, K &best, K &second) {
    K a = none, b = none;
    if (lane < g.groups)
        for (int i = 0; i < g.per_group; i++) {
            const K k = key[lane * g.per_group + i];
            const K low = k < a ? k : a;
            b = low > b ? low : b;
            a = k > a ? k : a;
        }
    best = a;
    second = b;
}

template <int EPL> __device__ __forceinline__ bool group_kept(uint64_t keep, const RouteArgs &g, int lane, int i) {
    const unsigned group = ((unsigned)(lane * EPL + i) * g.group_mul) >> 20;
    return keep >> (group & 63) & 1;
}

// Chooses by fp64 keys: lane k has the k-th expert, or -1.
template <int EPL>
__device__ __forceinline__ int choose_f64(const float (&x)[EPL], const RouteArgs &g, double top, double *lds, int lane) {
    double inv_sum = 1.0;
    if (g.softmax) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; i++) sum += lane * EPL + i < g.E ? exp((double)x[i] - top) : 0.0;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
        inv_sum = 1.0 / sum;
    }
    const double none = -INFINITY;
    double key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = lane * EPL + i;
        const float b = g.bias && e < g.E ? g.bias[e] : 0.f;
        double k = g.softmax ? exp((double)x[i] - top) * inv_sum : 1.0 / (1.0 + exp(-(double)x[i]));
        if (g.bias) k += (double)b;
        key[i] = e < g.E && x[i] > -INFINITY && b > -INFINITY && k == k ? k : none;
    }
    if (g.groups > 1) {
#pragma unroll
        for (int i = 0; i < EPL; i++) lds[lane * EPL + i] = key[i];
        __builtin_amdgcn_wave_barrier();
        double best, second;
        group_best(lds, g, lane, none, best, second);
        if (g.group_top == 2 && second > none) best += second;
        uint64_t keep = 0;
        for (int k = 0; k < g.topk_groups; k++) {
            const double m = wave_max(best);
            if (m == none) break;
            const int l = first_lane(__ballot(best == m));
            keep |= 1ull << l;
            if (lane == l) best = none;
        }
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (!group_kept<EPL>(keep, g, lane, i)) key[i] = none;
    }
    int mine = -1;
    for (int k = 0; k < g.topk; k++) {
        double m = key[0];
#pragma unroll
        for (int i = 1; i < EPL; i++) m = key[i] > m ? key[i] : m;
        const double best = wave_max(m);
        if (best == none) break;
        const int l = first_lane(__ballot(m == best));
        int at = EPL - 1;
#pragma unroll
        for (int i = EPL - 2; i >= 0; i--) at = key[i] == best ? i : at;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (lane == l && at == i) key[i] = none;
        const int e = l * EPL + __builtin_amdgcn_readlane(at, l);
        if (lane == k) mine = e;
    }
    return mine;
}

// Lanes l ^ 1, l ^ 2, l ^ 7 and l ^ 15 (an exchange of pairs, quads and eights whose lanes are
// alike).
template <int CTRL> __device__ __forceinline__ void merge_from(int &best, int &second) {
    const int b = dpp_from<CTRL, 0xF>(KEY_NONE, best), c = dpp_from<CTRL, 0xF>(KEY_NONE, second);
    second = max(min(best, b), max(second, c));
    best = max(best, b);
}

// The sum of a group's largest keys, or its largest, as an ordered key.
__device__ __forceinline__ int group_score(int best, int second, const RouteArgs &g) {
    return g.group_top == 2 && second != KEY_NONE ? ordered(unordered(best) + unordered(second)) : best;
}

// The same by fp32 keys; ok is false where they do not decide it.  Keys are kept as
// integers, each lane's in descending order with the lower expert first, so that a lane's
// best is its first.
template <int EPL>
__device__ __forceinline__ int choose_f32(const float (&x)[EPL], const RouteArgs &g, float top, int *lds, int lane,
                                          bool &ok) {
    constexpr float LOG2E = 1.44269504f;
    const bool plain = !g.bias && g.groups == 1, biased = g.bias != nullptr;
    int key[EPL];
    if (plain) {
#pragma unroll
        for (int i = 0; i < EPL; i++) key[i] = x[i] > -INFINITY ? ordered(x[i]) : KEY_NONE;   // nor NaN
    } else {
        float s[EPL], sum = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            s[i] = g.softmax ? exp2_fast((x[i] - top) * LOG2E) : rcp_fast(1.0f + exp2_fast(-LOG2E * x[i]));
            sum += lane * EPL + i < g.E ? s[i] : 0.f;
        }
        const float inv = g.softmax && biased ? rcp_fast(wave_sum(sum)) : 1.0f;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const int e = lane * EPL + i;
            const float b = biased && e < g.E ? g.bias[e] : 0.f;
            key[i] = x[i] > -INFINITY && b > -INFINITY ? ordered(s[i] * inv + b) : KEY_NONE;
        }
    }
    ok = plain || !g.softmax || top < INFINITY;
    if (g.groups > 1) {
        // the topk_groups best, one by one, and the first one that is left out
        const int lanes = g.per_group / EPL;   // to a group
        int best = key[0], second = KEY_NONE, m, last = 0, k = 0;
        const bool whole = lanes * EPL == g.per_group && (lanes & (lanes - 1)) == 0 && lanes <= 16;
        if (whole) {   // between the group's lanes, and its score in each of them
#pragma unroll
            for (int i = 1; i < EPL; i++) {
                second = max(second, min(best, key[i]));
                best = max(best, key[i]);
            }
            if (lanes > 1) merge_from<0xB1>(best, second);
            if (lanes > 2) merge_from<0x4E>(best, second);
            if (lanes > 4) merge_from<0x141>(best, second);
            if (lanes > 8) merge_from<0x140>(best, second);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; i++) lds[lane * EPL + i] = key[i];
            __builtin_amdgcn_wave_barrier();
            group_best(lds, g, lane, KEY_NONE, best, second);
        }
        int score = best == KEY_NONE ? KEY_NONE : group_score(best, second, g);
        const int own = whole ? lane & -lanes : lane;   // the first lane of the lane's group
        uint64_t keep = 0;
        for (; k < g.topk_groups; k++) {
            m = wave_max(score);
            if (m == KEY_NONE) break;
            const int l = first_lane(__ballot(score == m));
            keep |= 1ull << l;
            if (own == l) score = KEY_NONE;
            last = m;
        }
        // The last kept and the first left out decide.  But a sum of two keys of either sign is
        // off by what they are, which may be far more than the sum and another from group to
        // group; then the least that any kept sum can be lies above the most that any other can.
        const bool pair = g.group_top == 2 && second != KEY_NONE;
        if (biased && __ballot(pair && (best ^ second) < 0)) {
            const float mag = best == KEY_NONE ? 0.f : fabsf(unordered(best)) + (pair ? fabsf(unordered(second)) : 0.f);
            const float off = 0x1p-18f * (1.0f + mag), v = unordered(group_score(best, second, g));
            const bool kept = keep >> own & 1;
            // an infinite bound decides nothing, nor does one that is not a number
            const int least = kept ? ordered(off < INFINITY ? -v + off : INFINITY) : KEY_NONE;
            const int most = kept || best == KEY_NONE ? KEY_NONE : ordered(off < INFINITY ? v + off : INFINITY);
            const int l = wave_max(least), h = wave_max(most);
            if (h != KEY_NONE && !(-unordered(l) > unordered(h))) ok = false;
        } else if (k == g.topk_groups) {
            m = wave_max(score);
            if (m != KEY_NONE && route_close(unordered(last), unordered(m), biased)) ok = false;
        }
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (!(whole ? keep >> own & 1 : group_kept<EPL>(keep, g, lane, i))) key[i] = KEY_NONE;
    }
    int id[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) id[i] = i;
#pragma unroll
    for (int i = 1; i < EPL; i++)   // insertion: stable
#pragma unroll
        for (int j = i; j > 0; j--) {
            const bool swap = key[j] > key[j - 1];
            const int a = key[j], b = key[j - 1], c = id[j], d = id[j - 1];
            key[j] = swap ? b : a;
            key[j - 1] = swap ? a : b;
            id[j] = swap ? d : c;
            id[j - 1] = swap ? c : d;
        }
    int mine = -1, chosen = KEY_NONE, m = KEY_NONE;   // lane k's expert and key
    for (int k = 0; k < g.topk; k++) {
        m = wave_max(key[0]);
        if (m == KEY_NONE) break;
        const int l = first_lane(__ballot(key[0] == m));
        const int e = l * EPL + __builtin_amdgcn_readlane(id[0], l);
        if (lane == k) {
            mine = e;
            chosen = m;
        }
        if (lane == l) {
#pragma unroll
            for (int i = 0; i + 1 < EPL; i++) {
                key[i] = key[i + 1];
                id[i] = id[i + 1];
            }
            key[EPL - 1] = KEY_NONE;
        }
    }
    if (!plain && m != KEY_NONE) {
        m = wave_max(key[0]);   // the first one that is left out
        int after = __shfl(chosen, lane + 1 < 64 ? lane + 1 : lane, 64);
        if (lane == g.topk - 1) after = m;
        const bool close = chosen != KEY_NONE && after != KEY_NONE && lane < g.topk &&
                           route_close(unordered(chosen), unordered(after), biased);
        if (__ballot(close)) ok = false;
    } else if (!plain) {   // fewer than topk: all of them, in order
        const int after = __shfl(chosen, lane + 1 < 64 ? lane + 1 : lane, 64);
        if (__ballot(chosen != KEY_NONE && after != KEY_NONE && lane < 63 &&
                     route_close(unordered(chosen), unordered(after), biased)))
            ok = false;
    }
    return mine;
}

__device__ __forceinline__ float load_logit(const RouteArgs &g, int64_t row, int e) {
    const int64_t i = row * g.E + e;
    return g.bf16 ? bf16_lo(((const uint16_t *)g.logits)[i]) : ((const float *)g.logits)[i];
}

// VEC: fp32 logits whose lanes' EPL are whole and aligned.
//
// The weights are fp64 exponentials and quotients, for topk lanes of a wave: with up to 16
// experts chosen one wave does them for the workgroup's four rows.
template <int EPL, bool VEC>
__global__ void __launch_bounds__(256) moe_route_kernel(RouteArgs g) {
    __shared__ double lds[4][EPL * 64];
    __shared__ int chosen[4][64];
    __shared__ double sums[4];   // softmax: of the row's exponentials, less its largest logit
    __shared__ float tops[4];    // and that, NaN if a logit is
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row0 = (int64_t)blockIdx.x * 4, row = row0 + wave;
    if (row < g.rows) {
        float x[EPL];
        if constexpr (VEC) {
            typedef float vec __attribute__((ext_vector_type(EPL == 1 ? 1 : EPL == 2 ? 2 : 4)));
            constexpr int V = EPL < 4 ? EPL : 4;
            const bool in = lane * EPL < g.E;
#pragma unroll
            for (int i = 0; i < EPL; i += V) {
                vec v;
                if (in) v = *(const vec *)((const float *)g.logits + row * g.E + lane * EPL + i);
#pragma unroll
                for (int e = 0; e < V; e++) x[i + e] = in ? v[e] : -INFINITY;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; i++) x[i] = lane * EPL + i < g.E ? load_logit(g, row, lane * EPL + i) : -INFINITY;
        }
        float top = 0.f;
        bool nan = false;
        if (g.softmax) {
            int m = KEY_NONE;
#pragma unroll
            for (int i = 0; i < EPL; i++) {
                m = x[i] == x[i] ? max(m, ordered(x[i])) : m;
                nan |= x[i] != x[i];
            }
            m = wave_max(m);
            top = m == KEY_NONE ? -INFINITY : unordered(m);
            nan = __ballot(nan) != 0;
        }
        bool ok;
        int mine = choose_f32<EPL>(x, g, nan ? INFINITY : top, (int *)lds[wave], lane, ok);
        if (!ok) mine = choose_f64<EPL>(x, g, top, lds[wave], lane);
        chosen[wave][lane] = mine;
        if (g.softmax) {
            if (!g.renorm) {
                double sum = 0.0;
#pragma unroll
                for (int i = 0; i < EPL; i++) sum += lane * EPL + i < g.E ? exp((double)x[i] - (double)top) : 0.0;
#pragma unroll
                for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
                if (lane == 0) sums[wave] = sum;
            }
            if (lane == 0) tops[wave] = nan ? NAN : top;
        }
    }
    __syncthreads();
    const bool shared = g.topk <= 16;
    if (shared && wave > 0) return;
    const int r = shared ? lane >> 4 : wave, k = shared ? lane & 15 : lane;
    const bool live = k < g.topk && row0 + r < g.rows;
    const int mine = live ? chosen[r][k] : -1;
    double w = 0.0;
    if (mine >= 0) {
        const double v = load_logit(g, row0 + r, mine);
        if (g.softmax) {
            w = exp(v - (double)tops[r]);
            if (!g.renorm) w /= sums[r];
        } else {
            w = 1.0 / (1.0 + exp(-v));
        }
    }
    if (g.renorm) {
        double sum = w;
        for (int off = 1; off < g.topk; off <<= 1) sum += __shfl_xor(sum, off, 64);
        w = mine < 0 || sum == 0.0 ? 0.0 : w / sum;   // an empty slot's beside a sum of NaN, too
    }
    if (live) {
        g.ids[(row0 + r) * g.topk + k] = mine;
        g.weights[(row0 + r) * g.topk + k] = (float)(w * (double)g.scale);
    }
}

// ---------------------------------------------------------------- experts --
//
// Few tokens are bound by the weights' bytes, 3 D I of each expert in use, so
// neither product rounds its other operand: x is bf16 as it comes, h is fp32 in two
// bf16 (hi + lo, 17 bits), and a weight's e4m3 code is a bf16 value exactly.  Products
// are bf16 MFMAs with fp32 sums, one scale for each 64 deep piece of a 128 x 128 block.
//
//   moe_up    an item is one expert, 16 columns of W1 and the same of W3.  The waves split D,
//             and their sums are added in wave order.  Two workgroups for each CU: up to 16
//             tokens both are on it, above that (178 VGPRs) one behind the other
//   moe_down  a workgroup: 16 or 32 columns of out and one class of the experts; an item is
//             one of them, in ascending order.  The waves split I; each has its own sums for
//             every token, weighted, and these are added in wave order at the end
//   moe_join  with more classes than one: their sums, in order
//
// An expert's weights are read once for each 32 (moe_up) and 16 (moe_down) of its tokens:
// 128 tokens of 8 experts, D = 7168, I = 2048, take 205 us, where reading them once would
// take 57.
//
// How D and I are split does not depend on the tokens, so a token's result is the
// same in every batch, and no sum depends on timing.
//
// Measured, up / down, D = 7168, I = 2048: one token of 8 experts 44.0 / 24.3 us (5.3 and 4.8
// TB/s), 16 tokens of 64 experts, 8 each, 278 / 147 (6.0 and 5.6), 128 tokens of 32 experts here of
// 256 165 / 120 (5.7 and 3.9: their sums fill LDS, so the workgroups have 16 columns, and 448 of
// them share 256 CUs).  Reading the experts' rows and nothing else reaches 6.2 TB/s, in any
// pattern of 128 bytes or more; 64-byte pieces a fifth less.  5 tokens of 16 experts of 1024 x 384,
// 7.0 / 7.7 and 2.6 to join: making the lists takes 2, a round of loads 1, an item's sums 1.
//
// The weights come by DMA into two slots of LDS for each wave, 32 rows x 128 bytes (or 16 x
// 256) to a slot, and the other operand to registers, also for one slot ahead: a wave multiplies
// one slot while the next is on its way, through the boundaries of items too, and
// waits for its own loads alone, by their number.  A wave with a share issues every load
// whether or not there is something to load, then out of its descriptor's range, so that
// the number is known where they are waited for; one without a share loads nothing.

constexpr int MOE_WAVES = 8, MOE_NT = MOE_WAVES * 64;
constexpr int MOE_PAIRS = 1024;      // most M * topk, and most experts
constexpr int SLOT = 4096;           // bytes: T tiles of 16 rows of SU 64-byte units
template <int T> constexpr int SU = 4 / T;
__shared__ __attribute__((aligned(1024))) uint8_t sW0[MOE_WAVES * SLOT];
__shared__ __attribute__((aligned(1024))) uint8_t sW1[MOE_WAVES * SLOT];
template <int ST> __device__ __forceinline__ uint8_t *slot_of(int wave) { return (ST ? sW1 : sW0) + wave * SLOT; }

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

// acc += s p.  The empty statement keeps the sum in its block: moved behind a branch (to the
// next tile, or past the last unit), it was compiled without the wait states that reading
// an MFMA's result takes on the branch's other way, and read it too early.  (A test searches
// the assembly for such reads.)
__device__ __forceinline__ void fold(v4f &acc, const v4f &p, float s) {
#pragma unroll
    for (int e = 0; e < 4; e++) acc[e] = __builtin_fmaf(p[e], s, acc[e]);
    asm volatile("" : "+v"(acc));
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ float lane_value(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// The experts in use, ascending, and their tokens.
struct MoeLists {
    unsigned item[MOE_PAIRS];   // expert | number of its tokens << 10 | first of them in at << 18
    int at[MOE_PAIRS];          // token | pair << 8, pair = token * topk + slot
    float w[MOE_PAIRS];         // moe_down: the token's weight
    int count;
};

// Up to FEW_PAIRS pairs, by one wave: lane i has pair i, and goes through the others'.  A token
// that names an expert in several slots counts once, by the first, with the sum of their
// weights, in order.  In all of the call, so / by the sort below: 2 pairs 12.7 / 14.5 us, 8 pairs
// 17.1 / 18.9 and, of 7168 x 2048, 69.8 / 70.6; but 10 pairs 16.4 / 16.1, 32 pairs 23.2 / 17.6.
constexpr int FEW_PAIRS = 8;
__device__ __forceinline__ void few_lists(MoeLists &l, const MoeArgs &g, bool weights, int classes, int rest) {
    const int i = threadIdx.x, pairs = g.M * g.topk, m = i / g.topk;
    int e = -1;
    float given = 0.f;
    if (i < pairs) {
        e = g.ids[i];
        if (weights) given = g.weights[i];
        if (!((unsigned)e < (unsigned)g.E && e % classes == rest)) e = -1;
    }
    bool first = e >= 0;
    float w = 0.f;
    for (int k = 0; k < pairs; k++) {
        const bool same = __builtin_amdgcn_readlane(e, k) == e && __builtin_amdgcn_readlane(m, k) == m;
        first = first && !(same && k < i);
        if (weights) w += same && k >= i ? lane_value(given, k) : 0.f;
    }
    // the expert's tokens, those of lanes before this one, and those of lower experts
    int n = 0, place = 0, before = 0;
    for (uint64_t left = __ballot(first); left; left &= left - 1) {
        const int k = __ffsll((unsigned long long)left) - 1, other = __builtin_amdgcn_readlane(e, k);
        n += other == e;
        place += other == e && k < i;
        before += other < e;
    }
    const uint64_t leaders = __ballot(first && place == 0);
    int item = 0;
    for (uint64_t left = leaders; left; left &= left - 1)
        item += __builtin_amdgcn_readlane(e, __ffsll((unsigned long long)left) - 1) < e;
    if (first) {
        l.at[before + place] = m | i << 8;
        l.w[before + place] = w;
        if (place == 0) l.item[item] = (unsigned)e | (unsigned)n << 10 | (unsigned)before << 18;
    }
    if (i == 0) l.count = __popcll(leaders);
}

// Every workgroup makes them, from the ids: a counting sort in LDS, in slots that no
// weights are in yet (scratch).  A token that names an expert in several slots counts once, by
// the first, with the sum of their weights.  The tokens of an expert stand in the order
// that its counter gave them, which no result depends on: a token has its own column
// of an MFMA, and its own sums.
//
// Of the experts whose number is `rest` modulo `classes` alone.
__device__ __forceinline__ void moe_lists(MoeLists &l, int *scratch, const MoeArgs &g, bool weights, int classes,
                                          int rest) {
    if (g.M * g.topk <= FEW_PAIRS) {
        if (threadIdx.x < 64) few_lists(l, g, weights, classes, rest);
        __syncthreads();
        return;
    }
    int *ids = scratch, *hist = ids + MOE_PAIRS, *total = hist + MOE_PAIRS;
    float *given = (float *)(total + MOE_WAVES);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, pairs = g.M * g.topk;
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int i = tid + j * MOE_NT;
        hist[i] = 0;
        if (i < pairs) {
            const int e = g.ids[i];
            if (weights) given[i] = g.weights[i];
            ids[i] = (unsigned)e < (unsigned)g.E && e % classes == rest ? e : -1;
        }
    }
    __syncthreads();
    int mine[2];   // the pair's expert, if it is the first of its token to name it
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int i = tid + j * MOE_NT;
        mine[j] = i < pairs ? ids[i] : -1;
        for (int k = i - i % g.topk; k < i && mine[j] >= 0; k++)
            if (ids[k] == mine[j]) mine[j] = -1;
        if (mine[j] >= 0) atomicAdd(&hist[mine[j]], 1);
    }
    __syncthreads();
    // experts 2 tid and 2 tid + 1: tokens, and experts in use (<< 16), before them
    const int n0 = hist[2 * tid], n1 = hist[2 * tid + 1];
    const int own = n0 + n1 + (((n0 != 0) + (n1 != 0)) << 16);
    int before = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(before, off, 64);
        if (lane >= off) before += v;
    }
    if (lane == 63) total[wave] = before;
    __syncthreads();
    before -= own;
    for (int w = 0; w < wave; w++) before += total[w];
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int n = j ? n1 : n0;
        if (n) {
            l.item[before >> 16] = (unsigned)(2 * tid + j) | (unsigned)n << 10 | (unsigned)(before & 0xFFFF) << 18;
            hist[2 * tid + j] = before & 0xFFFF;
            before += n + (1 << 16);
        }
    }
    if (tid == MOE_NT - 1) l.count = before >> 16;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; j++) {
        if (mine[j] < 0) continue;
        const int i = tid + j * MOE_NT, m = i / g.topk, pos = atomicAdd(&hist[mine[j]], 1);
        l.at[pos] = m | i << 8;
        if (weights) {
            float w = 0.f;
            for (int k = i; k < (m + 1) * g.topk; k++)
                if (ids[k] == mine[j]) w += given[k];
            l.w[pos] = w;
        }
    }
    __syncthreads();
}

// Where a wave's share of `blocks` 128 deep blocks begins, in units of 64, and the slots that the
// largest share fills.  With fewer blocks than waves some have none, and load nothing.
__device__ __forceinline__ int share(int blocks, int wave) { return blocks * wave / MOE_WAVES * 2; }
template <int T> __device__ __forceinline__ int stages_of(int blocks) {
    return ((blocks + MOE_WAVES - 1) / MOE_WAVES * 2 + SU<T> - 1) / SU<T>;
}

// T tiles of 16 rows of `pitch` bytes each.
template <int T> struct Tiles {
    __amdgpu_buffer_rsrc_t r[T];
};

// A lane's byte offsets in the SU instructions of a tile, each of whole row segments of
// 64 SU bytes, 16 bytes a lane.  A row's chunks are permuted by its number so that the 16
// rows of a fragment read lie in different banks: chunk c of row r is at place c ^ r of
// the 16 (SU = 4), or c ^ (r / 2) of the 8 (SU = 2, two rows to the banks).
template <int T> __device__ __forceinline__ int place(int r, int c) { return SU<T> == 4 ? c ^ r : c ^ (r >> 1); }
template <int T> struct LaneOffsets {
    int off[SU<T>], chunk[SU<T>];
};
template <int T>
__device__ __forceinline__ LaneOffsets<T> lane_offsets(int pitch, int lane) {
    LaneOffsets<T> o;
#pragma unroll
    for (int i = 0; i < SU<T>; i++) {
        const int row = 16 / SU<T> * i + lane / (4 * SU<T>);
        o.chunk[i] = place<T>(row, lane % (4 * SU<T>));
        o.off[i] = row * pitch + o.chunk[i] * 16;
    }
    return o;
}

// 16 bytes of each lane to consecutive places of LDS.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint8_t *to, int off, int at) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)to, 16, off, at, 0, 0);
}

// `units` pieces of 64 bytes from unit u0 on into slot ST.
template <int ST, int T>
__device__ __forceinline__ void moe_dma(const Tiles<T> &t, const LaneOffsets<T> &o, int u0, int units, int wave) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the slot's last reads are done
#pragma unroll
    for (int h = 0; h < T; h++)
#pragma unroll
        for (int i = 0; i < SU<T>; i++) {
            const int off = o.chunk[i] < 4 * units ? o.off[i] : OUT_OF_RANGE;
            dma16(t.r[h], slot_of<ST>(wave) + (h * SU<T> + i) * 1024, off, u0 * 64);
        }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// All vector memory operations but the last N are done.
template <int N>
__device__ __forceinline__ void wait_all_but() {
    static_assert(N < 64, "vmcnt has 6 bits");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
    asm volatile("" ::: "memory");
}

// Row fr's 16 codes of unit q, tile h, of slot ST.
template <int ST, int T>
__device__ __forceinline__ void slot_frag(v8bf (&w)[2], int h, int q, int wave, int fr, int fg) {
    widen16(*(const u32x4 *)(slot_of<ST>(wave) + (h * 16 + fr) * 64 * SU<T> + place<T>(fr, 4 * q + fg) * 16), w);
}

__device__ __forceinline__ v8bf load_v8(__amdgpu_buffer_rsrc_t r, int off, int at) {
    return __builtin_bit_cast(v8bf, __builtin_amdgcn_raw_buffer_load_b128(r, off, at, 0));
}

// The other operand's rows come in groups of 16 / Z, each row in Z pieces of 8 values for
// every 16 of a unit: x in two (its first and second 8), h in four (the two 8s of its
// high parts, then of its low parts).  The 16 columns of an MFMA are a group's row and
// piece, column Z r + z: one instruction loads a unit for all of them, however few rows
// there are, where a piece to an instruction takes Z of them, mostly for rows that are
// not there, and a CU's rate of loads would bound the kernel.  The weights' first 8 of each 16 go
// with even pieces and the second 8 with odd ones; the pieces' sums are added at the end.
__device__ __forceinline__ void group_unit(v4f &acc, const v8bf (&w)[2], const v8bf &x, float scale, bool odd) {
    const v4f zero = {0.f, 0.f, 0.f, 0.f};
    const v4f p0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[0], x, zero, 0, 0, 0);
    const v4f p1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[1], x, zero, 0, 0, 0);
    v4f p;
#pragma unroll
    for (int e = 0; e < 4; e++) p[e] = odd ? p1[e] : p0[e];
    fold(acc, p, scale);
}
template <int CTRL> __device__ __forceinline__ float quad_perm(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
// The sum of a row's Z pieces, in each of its lanes.
template <int Z> __device__ __forceinline__ v4f add_pieces(v4f v) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
        v[e] += quad_perm<0xB1>(v[e]);                // lanes 1, 0, 3, 2
        if (Z == 4) v[e] += quad_perm<0x4E>(v[e]);    // lanes 2, 3, 0, 1
    }
    return v;
}

// Units of stage `a`, an even number.
template <int T, typename At, typename Work>
__device__ __forceinline__ int units_of(const At &a, const Work &w) {
    return a.n > 0 ? min(max(w.end - (w.first + a.k * SU<T>), 0), SU<T>) : 0;
}

// All loads of a stage but the next one's are done: those are `groups` for each unit, the
// scales and the slot's.
template <int T, int MAX>
__device__ __forceinline__ void wait_stage(int groups) {
    constexpr int N = 1 + SLOT / 1024;
    if constexpr (MAX == 1) {
        wait_all_but<SU<T> + N>();
    } else {
        if (groups >= MAX) wait_all_but<SU<T> * MAX + N>();
        else wait_stage<T, MAX - 1>(groups);
    }
}

// ----------------------------------------------------------------- moe_up --

// Where a wave is in its work: item `it` (expert, 16 columns from c0 on), the expert's
// tokens from r0 on (in up to G groups of 8), stage k of the wave's share of D.
template <int G> struct UpAt {
    int it, r0, k, expert, first, n, c0, groups;
    int off[G];   // byte offset of the lane's token's x; out of range past the last one
};
struct UpWork {
    const MoeLists *l;
    __amdgpu_buffer_rsrc_t x;
    int items, blocks, stages, first, end;   // blocks: of 16 columns
    int fr, fg, wave, lane;
};

template <int G>
__device__ __forceinline__ void up_tokens(UpAt<G> &a, const UpWork &w, int64_t D) {
    a.groups = min(max((a.n - a.r0 + 7) >> 3, 1), G);
#pragma unroll
    for (int i = 0; i < G; i++) {
        const int row = a.r0 + 8 * i + (w.fr >> 1);
        a.off[i] = row < a.n ? (w.l->at[a.first + row] & 255) * (int)D * 2 + 32 * w.fg + 16 * (w.fr & 1) : OUT_OF_RANGE;
    }
}
template <int G>
__device__ __forceinline__ void up_item(UpAt<G> &a, const UpWork &w, int64_t D) {
    if (a.it >= w.items) {
        a.n = 0;
    } else {
        const int t = a.it / w.blocks;
        a.c0 = (a.it - t * w.blocks) * 16;
        const unsigned item = (unsigned)uniform((int)w.l->item[t]);
        a.expert = item & 1023;
        a.n = item >> 10 & 255;
        a.first = item >> 18;
    }
    up_tokens<G>(a, w, D);
}
template <int G>
__device__ __forceinline__ void up_next(UpAt<G> &a, const UpWork &w, int64_t D) {
    if (++a.k < w.stages) return;
    a.k = 0;
    a.r0 += 8 * G;
    if (a.r0 < a.n) {
        up_tokens<G>(a, w, D);
        return;
    }
    a.r0 = 0;
    a.it += gridDim.x;
    up_item<G>(a, w, D);
}

template <int G> struct UpRegs {
    v8bf x[2][G];
    float sc;   // lane h: the scale of the block, tile h
};

// Loads of stage `a` into slot ST and r.
template <int G, int ST>
__device__ __forceinline__ void up_load(UpRegs<G> &r, const UpAt<G> &a, const UpWork &w, const MoeArgs &g,
                                        const LaneOffsets<2> &o) {
    const int64_t row = (int64_t)a.expert * 2 * g.I + a.c0;
    const int u0 = w.first + a.k * SU<2>;
    const int units = units_of<2>(a, w);
#pragma unroll
    for (int i = 0; i < G; i++) {
        if (i >= a.groups) break;
#pragma unroll
        for (int q = 0; q < SU<2>; q++)
            r.x[q][i] = load_v8(w.x, units ? a.off[i] : OUT_OF_RANGE, (u0 + q) * 128);
    }
    const int64_t DB = g.D / 128;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(g.s13 + row / 128 * DB, (g.I / 128 * DB + DB) * 4);
    r.sc = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                         rs, w.lane < units ? (w.lane * (int)(g.I / 128 * DB) + u0 / 2) * 4 : OUT_OF_RANGE, 0, 0));
    const Tiles<2> t = {make_rsrc(g.W13 + row * g.D, 16 * g.D), make_rsrc(g.W13 + (row + g.I) * g.D, 16 * g.D)};
    moe_dma<ST, 2>(t, o, u0, units, w.wave);
}

// The sums of an item's tokens, added over the waves by way of slot ST, which they have
// just read; act, product, and h as 64 bytes for each 16 columns: their high parts, then
// their low parts.
template <int G, int ST>
__device__ __forceinline__ void up_finish(const v4f (&acc)[2][G], const UpAt<G> &a, const UpWork &w, const MoeArgs &g) {
    constexpr int TP = (G + 1) / 2;   // tiles of two groups: even lanes have one's rows, odd lanes the other's
    static_assert(2 * TP * 1024 <= SLOT, "a wave's tiles fit a slot");
    v4f *own = (v4f *)slot_of<ST>(w.wave);
#pragma unroll
    for (int j = 0; j < TP; j++) {
        if (2 * j >= a.groups) break;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const v4f even = add_pieces<2>(acc[h][2 * j]), odd = add_pieces<2>(acc[h][2 * j + 1]);
            v4f v;
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = w.fr & 1 ? odd[e] : even[e];
            own[(h * TP + j) * 64 + w.lane] = v;
        }
    }
    barrier_lds_only();
    const int j = (w.wave - a.it) & (MOE_WAVES - 1);   // another wave from item to item
    if (j < TP && 2 * j < a.groups) {
        const int row = a.r0 + 8 * (2 * j + (w.fr & 1)) + (w.fr >> 1);
        v4f t[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            t[h] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int v = 0; v < MOE_WAVES; v++) t[h] += ((const v4f *)slot_of<ST>(v))[(h * TP + j) * 64 + w.lane];
        }
        float v[4] = {t[0][0], t[0][1], t[0][2], t[0][3]};
        act_all(v, g.act);
        if (row < a.n) {
            typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
            v4bf hi, lo;
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const float h = v[q] * t[1][q];
                hi[q] = (__bf16)h;
                lo[q] = (__bf16)(h - (float)hi[q]);
            }
            uint16_t *to = g.h + ((int64_t)(w.l->at[a.first + row] >> 8) * g.I + a.c0) * 2 + 4 * w.fg;
            *(v4bf *)to = hi;
            *(v4bf *)(to + 16) = lo;
        }
    }
    barrier_lds_only();
}

// One stage, in slot ST, the next one's loads first.  False after the last.
template <int G, int ST>
__device__ __forceinline__ bool up_stage(v4f (&acc)[2][G], UpRegs<G> (&r)[2], UpAt<G> &a, UpAt<G> &next,
                                         const UpWork &w, const MoeArgs &g, const LaneOffsets<2> &o) {
    up_load<G, ST ^ 1>(r[ST ^ 1], next, w, g, o);
    wait_stage<2, G>(next.groups);
    const int units = units_of<2>(a, w);
#pragma unroll
    for (int q = 0; q < SU<2>; q++) {
        if (q >= units) break;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            v8bf wb[2];
            slot_frag<ST, 2>(wb, h, q, w.wave, w.fr, w.fg);
            const float scale = lane_value(r[ST].sc, h);
#pragma unroll
            for (int i = 0; i < G; i++) {
                if (i >= a.groups) break;
                group_unit(acc[h][i], wb, r[ST].x[q][i], scale, w.fr & 1);
            }
        }
    }
    if (a.k == w.stages - 1) {
        up_finish<G, ST>(acc, a, w, g);
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int i = 0; i < G; i++) acc[h][i] = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    a = next;
    up_next<G>(next, w, g.D);
    return a.it < w.items;
}

template <int G>
__global__ void __launch_bounds__(MOE_NT) moe_up_kernel(MoeArgs g) {
    __shared__ MoeLists l;
    moe_lists(l, (int *)slot_of<0>(0), g, false, 1, 0);
    UpWork w;
    w.l = &l;
    w.lane = threadIdx.x & 63;
    w.wave = uniform(threadIdx.x >> 6);
    w.fr = w.lane & 15;
    w.fg = w.lane >> 4;
    w.x = make_rsrc(g.x, g.M * g.D * 2);
    w.blocks = (int)(g.I / 16);
    w.items = uniform(l.count) * w.blocks;
    const int blocks = (int)(g.D / 128);
    w.stages = stages_of<2>(blocks);
    w.first = share(blocks, w.wave);
    w.end = share(blocks, w.wave + 1);
    const LaneOffsets<2> o = lane_offsets<2>((int)g.D, w.lane);
    UpAt<G> a = {};
    a.it = blockIdx.x;
    if (a.it >= w.items) return;
    up_item<G>(a, w, g.D);
    v4f acc[2][G];
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
        for (int i = 0; i < G; i++) acc[h][i] = (v4f){0.f, 0.f, 0.f, 0.f};
    if (w.first == w.end) {   // no share: its part in the others' sums
        for (int stage = 0; a.it < w.items; stage++) {
            if (a.k == w.stages - 1) {
                if (stage & 1) up_finish<G, 1>(acc, a, w, g);
                else up_finish<G, 0>(acc, a, w, g);
            }
            up_next<G>(a, w, g.D);
        }
        return;
    }
    UpAt<G> next = a;
    UpRegs<G> r[2];
    up_load<G, 0>(r[0], next, w, g, o);
    up_next<G>(next, w, g.D);
    while (up_stage<G, 0>(acc, r, a, next, w, g, o) && up_stage<G, 1>(acc, r, a, next, w, g, o)) {
    }
    wait_all_but<0>();   // the last (empty) DMA is retired
}

// --------------------------------------------------------------- moe_down --

// Where a wave is: expert t of the list, its tokens from r0 on (in up to four groups of
// 4), stage k of the wave's share of I.
constexpr int DG = 4;
struct DownAt {
    int t, r0, k, expert, first, n, groups;
    int off[DG];   // byte offset of the lane's token's h
};
struct DownWork {
    const MoeLists *l;
    __amdgpu_buffer_rsrc_t h;
    int count, stages, first, end;
    int64_t n0;
    int fr, fg, wave, lane;
};

__device__ __forceinline__ void down_tokens(DownAt &a, const DownWork &w, int64_t I) {
    a.groups = min(max((a.n - a.r0 + 3) >> 2, 1), DG);
#pragma unroll
    for (int i = 0; i < DG; i++) {
        const int row = a.r0 + 4 * i + (w.fr >> 2);
        a.off[i] = row < a.n ? (w.l->at[a.first + row] >> 8) * (int)I * 4 + 64 * w.fg + 16 * (w.fr & 3) : OUT_OF_RANGE;
    }
}
__device__ __forceinline__ void down_item(DownAt &a, const DownWork &w, int64_t I) {
    if (a.t >= w.count) {
        a.n = 0;
    } else {
        const unsigned item = (unsigned)uniform((int)w.l->item[a.t]);
        a.expert = item & 1023;
        a.n = item >> 10 & 255;
        a.first = item >> 18;
    }
    down_tokens(a, w, I);
}
__device__ __forceinline__ void down_next(DownAt &a, const DownWork &w, int64_t I) {
    if (++a.k < w.stages) return;
    a.k = 0;
    a.r0 += 4 * DG;
    if (a.r0 < a.n) {
        down_tokens(a, w, I);
        return;
    }
    a.r0 = 0;
    a.t++;
    down_item(a, w, I);
}

template <int T> struct DownRegs {
    v8bf h[SU<T>][DG];
    float sc;        // lane q: the scale of unit q
};

// T: tiles of 16 columns to a workgroup.
template <int T, int ST>
__device__ __forceinline__ void down_load(DownRegs<T> &r, const DownAt &a, const DownWork &w, const MoeArgs &g,
                                          const LaneOffsets<T> &o) {
    const int64_t row = (int64_t)a.expert * g.D + w.n0;
    const int u0 = w.first + a.k * SU<T>;
    const int units = units_of<T>(a, w);
#pragma unroll
    for (int i = 0; i < DG; i++) {
        if (i >= a.groups) break;
#pragma unroll
        for (int q = 0; q < SU<T>; q++)
            r.h[q][i] = load_v8(w.h, q < units ? a.off[i] : OUT_OF_RANGE, (u0 + q) * 256);
    }
    const int64_t IB = g.I / 128;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(g.s2 + row / 128 * IB, IB * 4);
    r.sc = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                         rs, w.lane < units ? (u0 + w.lane) / 2 * 4 : OUT_OF_RANGE, 0, 0));
    Tiles<T> t;
#pragma unroll
    for (int j = 0; j < T; j++) t.r[j] = make_rsrc(g.W2 + (row + 16 * j) * g.I, 16 * g.I);
    moe_dma<ST, T>(t, o, u0, units, w.wave);
}

// One stage, in slot ST, the next one's loads first.  False after the last.  sum: the
// wave's own sums, 16 T columns of each token; of a token m, four columns c are at place
// c ^ (m % 4).
template <int T, int ST>
__device__ __forceinline__ bool down_stage(v4f (&acc)[T][DG], DownRegs<T> (&r)[2], DownAt &a, DownAt &next, v4f *sum,
                                           const DownWork &w, const MoeArgs &g, const LaneOffsets<T> &o) {
    down_load<T, ST ^ 1>(r[ST ^ 1], next, w, g, o);
    wait_stage<T, DG>(next.groups);
    const int units = units_of<T>(a, w);
#pragma unroll
    for (int q = 0; q < SU<T>; q++) {
        if (q >= units) break;
        const float scale = lane_value(r[ST].sc, q);
#pragma unroll
        for (int j = 0; j < T; j++) {
            v8bf wb[2];
            slot_frag<ST, T>(wb, j, q, w.wave, w.fr, w.fg);
#pragma unroll
            for (int i = 0; i < DG; i++) {
                if (i >= a.groups) break;
                group_unit(acc[j][i], wb, r[ST].h[q][i], scale, w.fr & 1);
            }
        }
    }
    if (a.k == w.stages - 1) {
#pragma unroll
        for (int i = 0; i < DG; i++) {
            if (i >= a.groups) break;
            const int row = a.r0 + 4 * i + (w.fr >> 2);
            const bool mine = (w.fr & 3) == 0 && row < a.n;
            const int m = mine ? w.l->at[a.first + row] & 255 : 0;
            const float weight = mine ? w.l->w[a.first + row] : 0.f;
#pragma unroll
            for (int j = 0; j < T; j++) {
                const v4f t = add_pieces<4>(acc[j][i]);
                if (mine) {
                    v4f *d = sum + m * 4 * T + 4 * j + (w.fg ^ (m & 3));
                    v4f s = *d;
                    fold(s, t, weight);
                    *d = s;
                }
                acc[j][i] = (v4f){0.f, 0.f, 0.f, 0.f};
            }
        }
    }
    a = next;
    down_next(next, w, g.I);
    return a.t < w.count;
}

// base + v as four elements of out.
__device__ __forceinline__ void moe_store(const MoeArgs &g, int64_t at, v4f v) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    if (g.base) {
        const u32x2 b = *(const u32x2 *)(g.base + at);
        v[0] += bf16_lo(b[0]); v[1] += bf16_hi(b[0]);
        v[2] += bf16_lo(b[1]); v[3] += bf16_hi(b[1]);
    }
    *(u32x2 *)(g.out + at) = (u32x2){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

template <int T, int MMAX>
__global__ void __launch_bounds__(MOE_NT) moe_down_kernel(MoeArgs g) {
    __shared__ MoeLists l;
    __shared__ v4f sum[MOE_WAVES][MMAX * 4 * T];
    for (int i = threadIdx.x; i < MOE_WAVES * MMAX * 4 * T; i += MOE_NT) sum[0][i] = (v4f){0.f, 0.f, 0.f, 0.f};
    moe_lists(l, (int *)slot_of<0>(0), g, true, (int)gridDim.y, (int)blockIdx.y);
    DownWork w;
    w.l = &l;
    w.lane = threadIdx.x & 63;
    w.wave = uniform(threadIdx.x >> 6);
    w.fr = w.lane & 15;
    w.fg = w.lane >> 4;
    w.h = make_rsrc(g.h, (int64_t)g.M * g.topk * g.I * 4);
    w.count = uniform(l.count);
    w.n0 = (int64_t)blockIdx.x * 16 * T;
    const int blocks = (int)(g.I / 128);
    w.stages = stages_of<T>(blocks);
    w.first = share(blocks, w.wave);
    w.end = share(blocks, w.wave + 1);
    const LaneOffsets<T> o = lane_offsets<T>((int)g.I, w.lane);
    DownAt a = {};
    if (w.count > 0 && w.first < w.end) {
        down_item(a, w, g.I);
        DownAt next = a;
        DownRegs<T> r[2];
        v4f acc[T][DG];
#pragma unroll
        for (int j = 0; j < T; j++)
#pragma unroll
            for (int i = 0; i < DG; i++) acc[j][i] = (v4f){0.f, 0.f, 0.f, 0.f};
        down_load<T, 0>(r[0], next, w, g, o);
        down_next(next, w, g.I);
        while (down_stage<T, 0>(acc, r, a, next, sum[w.wave], w, g, o) &&
               down_stage<T, 1>(acc, r, a, next, sum[w.wave], w, g, o)) {
        }
        wait_all_but<0>();   // the last (empty) DMA is retired
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g.M * 4 * T; i += MOE_NT) {
        const int m = i / (4 * T), c = i % (4 * T);
        v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < MOE_WAVES; k++) v += sum[k][m * 4 * T + (c ^ (m & 3))];
        const int64_t at = m * g.D + w.n0 + 4 * c;
        if (gridDim.y > 1) *(v4f *)(g.part + (int64_t)blockIdx.y * g.M * g.D + at) = v;
        else moe_store(g, at, v);
    }
}

// The classes' sums, in their order.
__global__ void __launch_bounds__(64) moe_join_kernel(MoeArgs g, int classes) {
    const int64_t n = g.M * g.D, at = ((int64_t)blockIdx.x * 64 + threadIdx.x) * 4;
    if (at >= n) return;
    v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int k = 0; k < classes; k++) v += *(const v4f *)(g.part + k * n + at);
    moe_store(g, at, v);
}

}  // namespace

template <int EPL>
static int launch_route(const RouteArgs &g, hipStream_t stream) {
    const dim3 grid((unsigned)((g.rows + 3) / 4)), block(256);
    if (!g.bf16 && g.E % EPL == 0 && ((uintptr_t)g.logits & 15) == 0 && (EPL < 4 || g.E % 4 == 0))
        return bs_enqueue(moe_route_kernel<EPL, true>, grid, block, stream, g);
    return bs_enqueue(moe_route_kernel<EPL, false>, grid, block, stream, g);
}

int bs_launch_moe_route(RouteArgs g, hipStream_t stream) {
    constexpr int64_t ROWS = (int64_t)1 << 25;   // a launch holds fewer than 2^32 lanes
    const RouteArgs all = g;
    for (int64_t first = 0; first < all.rows; first += ROWS) {
        g.rows = all.rows - first < ROWS ? all.rows - first : ROWS;
        g.logits = (const uint8_t *)all.logits + first * all.E * (all.bf16 ? 2 : 4);
        g.ids = all.ids + first * all.topk;
        g.weights = all.weights + first * all.topk;
        const int rc = g.E <= 64    ? launch_route<1>(g, stream)
                       : g.E <= 128 ? launch_route<2>(g, stream)
                       : g.E <= 256 ? launch_route<4>(g, stream)
                       : g.E <= 512 ? launch_route<8>(g, stream)
                                    : launch_route<16>(g, stream);
        if (rc != 0) return rc;
    }
    return 0;
}

// Classes that the experts are split into by their numbers, each with workgroups of its
// own: with few columns the workgroups are few, and each takes about 1 us an expert.  In all,
// without / with: 40 tokens of 59 experts, D = 128, I = 384 102 / 33 us; 5 tokens of 16, 1024 x 384
// 21.3 / 16.2; 16 tokens of 64, 4096 x 1536 260 / 206; but one token of 2 of 16, 1024 x 512 13.7 /
// 14.4 (the join is a launch of 3 us; 12.7 since few_lists).  Half as many classes 33, 17.6, 260; twice as many 33, 16.1,
// 213, and at D = 7168, where one is enough, 441 against 428 for 16 tokens of 64 experts.
constexpr int CLASS_COLUMNS = 8192;   // about 256 workgroups of 32 columns
static int moe_classes(int64_t E, int64_t D) {
    const int64_t most = (E + 1) / 2, c = CLASS_COLUMNS / D;   // two experts to a class
    return (int)(c < 1 || most < 1 ? 1 : c < most ? c : most);
}

// h: 32 bits for each of its values, of every pair; then each class's sums, fp32 [M, D].
int64_t bs_moe_workspace(int64_t M, int64_t topk, int64_t E, int64_t I) {
    return 4 * M * topk * I + (E > 2 ? 4 * CLASS_COLUMNS * M : 0);
}

template <int T, int MMAX>
static int launch_down(const MoeArgs &g, int classes, hipStream_t stream) {
    return bs_enqueue(moe_down_kernel<T, MMAX>, dim3((unsigned)(g.D / (16 * T)), (unsigned)classes), dim3(MOE_NT), stream, g);
}

int bs_launch_moe(const MoeArgs &args, hipStream_t stream) {
    MoeArgs g = args;
    g.part = (float *)(g.h + 2 * (int64_t)g.M * g.topk * g.I);
    const int64_t slots = g.E < g.M * g.topk ? g.E : g.M * g.topk, items = slots * (g.I / 16);
    const int64_t wgs = 2 * (int64_t)bs_stream_cus(stream);
    const dim3 up((unsigned)(items < wgs ? items : wgs)), block(MOE_NT);
    int rc = g.M <= 16 ? bs_enqueue(moe_up_kernel<2>, up, block, stream, g)
                       : bs_enqueue(moe_up_kernel<4>, up, block, stream, g);
    if (rc != 0) return rc;
    // 32 columns to a workgroup while its waves' sums of all tokens fit beside the slots
    const int classes = moe_classes(g.E, g.D);
    rc = g.M <= 16   ? launch_down<2, 16>(g, classes, stream)
         : g.M <= 64 ? launch_down<2, 64>(g, classes, stream)
                     : launch_down<1, 128>(g, classes, stream);
    if (rc != 0 || classes == 1) return rc;
    return bs_enqueue(moe_join_kernel, dim3((unsigned)((g.M * g.D / 4 + 63) / 64)), dim3(64), stream, g, classes);
}
