// lora.hip -- low-rank adapters of many requests beside a shared projection
// (gfx950).  Row m of a batch uses adapter id(m) (or none), and adds
//
//   scale[a] * ( x[m] A[a]^T ) B[a]^T,   A[a] [R, K], B[a] [N, R], a = id(m)
//
// to its row of the shared product.  Three kernels, each one launch:
//
//   lora_plan    orders the rows by adapter (a stable counting sort)
//   lora_shrink  H[m] = x[m] A[a]^T, fp32
//   lora_expand  out[m] = base[m] + scale[a] (H[m] B[a]^T), bf16 row bands
//
// shrink and expand walk tiles of rows that share one adapter, taken from the
// plan, so an adapter's weights are read once per tile whatever order its rows
// have in the batch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "codec.hpp"
#include "launch.hpp"
#include "lora.hpp"

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------- plan --

// plan = start[0 .. L+1], order[0 .. M): with key(m) = id(m) for an id in
// [0, L) and L otherwise, start[a] is the number of rows with key < a and
// order lists the rows by key, rows of one key in ascending order.
//
// Workgroup a places key a alone: it counts the rows with smaller keys, which
// is start[a], and writes its own rows behind them.  No workgroup waits for
// another and nothing is summed atomically, so the result is deterministic
// and one launch does it; the price is that each of the L + 1 workgroups reads
// all ids (64 KiB at M = 16384, from L2).  A wave takes 1024 consecutive rows
// of a panel, 64 per step, so counts and ranks within a step are ballots, and
// only 16 wave totals go through LDS.  A batch of one panel is read once and
// stays in registers.
constexpr int PLAN_STEPS = 16, PLAN_WAVES = 16, PLAN_PANEL = PLAN_STEPS * PLAN_WAVES * 64;

__device__ __forceinline__ void plan_load(int (&key)[PLAN_STEPS], const int32_t *ids, int64_t first, int64_t M,
                                          int L) {
#pragma unroll
    for (int i = 0; i < PLAN_STEPS; i++) {
        const int64_t m = first + 64 * i;
        key[i] = L + 1;   // past the end: no group's
        if (m < M) {
            const int id = ids[m];
            key[i] = (uint32_t)id < (uint32_t)L ? id : L;
        }
    }
}

__global__ void __launch_bounds__(PLAN_WAVES * 64)
lora_plan_kernel(const int32_t *__restrict__ ids, int32_t *__restrict__ plan, int64_t M, int L) {
    __shared__ int tot[PLAN_WAVES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int a = blockIdx.x;
    const int64_t mine = (int64_t)wave * (PLAN_STEPS * 64) + lane;
    int32_t *order = plan + L + 2;
    int key[PLAN_STEPS];
    int less = 0;
    for (int64_t p = 0; p < M; p += PLAN_PANEL) {
        plan_load(key, ids, p + mine, M, L);
#pragma unroll
        for (int i = 0; i < PLAN_STEPS; i++) less += __popcll(__ballot(key[i] < a));
    }
    if (lane == 0) tot[wave] = less;
    __syncthreads();
    int pos = 0;
#pragma unroll
    for (int w = 0; w < PLAN_WAVES; w++) pos += tot[w];
    if (threadIdx.x == 0) {
        plan[a] = pos;
        if (a == L) plan[L + 1] = (int32_t)M;
    }
    for (int64_t p = 0; p < M; p += PLAN_PANEL) {
        if (M > PLAN_PANEL) plan_load(key, ids, p + mine, M, L);
        int n = 0;
#pragma unroll
        for (int i = 0; i < PLAN_STEPS; i++) n += __popcll(__ballot(key[i] == a));
        __syncthreads();
        if (lane == 0) tot[wave] = n;
        __syncthreads();
        int at = pos;
#pragma unroll
        for (int w = 0; w < PLAN_WAVES; w++) {
            at += w < wave ? tot[w] : 0;
            pos += tot[w];
        }
#pragma unroll
        for (int i = 0; i < PLAN_STEPS; i++) {
            const uint64_t b = __ballot(key[i] == a);
            if (key[i] == a) order[at + __popcll(b & ((1ull << lane) - 1))] = (int32_t)(p + mine + 64 * i);
            at += __popcll(b);
        }
    }
}

// A tile of at most T rows of one group: positions [first, first + count) of
// order.  group == L is the rows without an adapter; count == 0 means that
// there is no such tile.
struct RowTile {
    int group, first, count;
};

// Tile t of the plan, groups in order, ceil(rows / T) tiles to each.  Every
// wave finds it by itself, 64 groups at a time, by a prefix sum over the
// groups' tile counts.  What the plan holds is clamped to [0, M], so that no
// content of it leads outside the buffers.
template <int T>
__device__ __forceinline__ RowTile find_tile(const int32_t *plan, int M, int L, int t, int lane) {
    int before = 0;
    for (int g0 = 0; g0 <= L; g0 += 64) {
        const int g = g0 + lane;
        int s0 = 0, n = 0;
        if (g <= L) {
            s0 = min(max(plan[g], 0), M);
            n = min(max(plan[g + 1], s0), M) - s0;
        }
        const int tiles = (n + T - 1) / T;
        int upto = tiles;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(upto, off, 64);
            if (lane >= off) upto += v;
        }
        const uint64_t hit = __ballot(before + upto > t);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            const int skip = t - before - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(tiles, l));
            RowTile r;
            r.group = g0 + l;
            r.first = __builtin_amdgcn_readlane(s0, l) + skip * T;
            r.count = min(T, __builtin_amdgcn_readlane(n, l) - skip * T);
            return r;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return RowTile{0, 0, 0};
}

// The most tiles that M rows in L + 1 groups can make.
inline int64_t max_tiles(int64_t M, int64_t L, int T) { return M / T + (L + 1 < M ? L + 1 : M); }

// The batch row at position p of order; M (no row) outside the tile or for an
// entry that is no row.
__device__ __forceinline__ int tile_row(const int32_t *order, const RowTile &t, int i, int M) {
    if (i >= t.count) return M;
    const int m = order[t.first + i];
    return (uint32_t)m < (uint32_t)M ? m : M;
}

// ----------------------------------------------------------------- shrink --

struct ShrinkArgs {
    const uint16_t *x;      // bf16 [M, K]
    const uint16_t *A;      // bf16 [L, R, K]
    const int32_t *plan;
    float *H;               // fp32 [M, R]
    int M, L, R;
    int64_t K;
};

// Eight bf16 of a row from k on, zero past its end (K % 8 == 0).
__device__ __forceinline__ v8bf load_k(const uint16_t *row, int64_t k, int64_t K) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k < K) v = *(const u32x4 *)(row + k);
    return __builtin_bit_cast(v8bf, v);
}

// One workgroup: 16 RT rows of one adapter, 16 CT columns of H.  Its W waves
// take the K axis in turns of 64 and their partial sums are added in wave
// order through LDS, so a short batch still spreads K over a CU's waves and
// the result does not depend on timing.  A lane takes 16 consecutive k of a
// row in each turn, its first eight to one MFMA and the rest to a second: the
// contraction may take k in any order as long as both operands do, and a
// row's four lanes so read 128 consecutive bytes.  The adapter's rows are the
// MFMA's first operand, which leaves a lane four consecutive columns of one
// row of H.
template <int RT, int CT, int W>
__global__ void __launch_bounds__(W * 64) lora_shrink_kernel(ShrinkArgs g) {
    __shared__ v4f part[W][RT * CT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fg = lane >> 4;
    const RowTile t = find_tile<16 * RT>(g.plan, g.M, g.L, blockIdx.x, lane);
    if (t.count <= 0) return;
    const int32_t *order = g.plan + g.L + 2;
    const int c0 = blockIdx.y * 16 * CT;
    int row[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) row[i] = tile_row(order, t, 16 * i + fr, g.M);
    if (t.group < g.L) {
        const uint16_t *xr[RT], *ar[CT];
#pragma unroll
        for (int i = 0; i < RT; i++) xr[i] = g.x + (int64_t)(row[i] < g.M ? row[i] : 0) * g.K;
#pragma unroll
        for (int j = 0; j < CT; j++)
            ar[j] = g.A + ((int64_t)t.group * g.R + min(c0 + 16 * j + fr, g.R - 1)) * g.K;
        v4f acc[RT][CT];
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int j = 0; j < CT; j++) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
        for (int64_t k0 = wave * 64; k0 < g.K; k0 += W * 64) {
            const int64_t k = k0 + 16 * fg;
            v8bf xv[RT][2], av[CT][2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
#pragma unroll
                for (int i = 0; i < RT; i++) xv[i][h] = load_k(xr[i], k + 8 * h, g.K);
#pragma unroll
                for (int j = 0; j < CT; j++) av[j][h] = load_k(ar[j], k + 8 * h, g.K);
            }
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int i = 0; i < RT; i++)
#pragma unroll
                    for (int j = 0; j < CT; j++)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[j][h], xv[i][h], acc[i][j], 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int j = 0; j < CT; j++) part[wave][i * CT + j][lane] = acc[i][j];
    }
    __syncthreads();
    for (int s = wave; s < RT * CT; s += W) {
        v4f sum = {0.f, 0.f, 0.f, 0.f};
        if (t.group < g.L) {
#pragma unroll
            for (int w = 0; w < W; w++) sum += part[w][s][lane];
        }
        const int c = c0 + 16 * (s % CT) + 4 * fg;
        const int m = tile_row(order, t, 16 * (s / CT) + fr, g.M);
        if (m < g.M && c < g.R) *(v4f *)(g.H + (int64_t)m * g.R + c) = sum;
    }
}

// ----------------------------------------------------------------- expand --

struct ExpandArgs {
    LoraArgs lora;
    const int32_t *plan;
    const uint16_t *base;   // bf16 row bands
    uint16_t *out;
    int M, col_blocks;
    int64_t N, band_rows, band_stride;
};

// One workgroup: 16 RT rows of one adapter, 256 columns, 64 to a wave.  The
// B rows are the MFMA's first operand, its fragment rows taken in the order
// of lora_col, so that a lane holds 8 consecutive columns of a row in each
// half of the wave's 64 and moves base and out in 16-byte pieces.  base is
// loaded before the products and added to them in fp32; out is rounded once.
template <int RT>
__global__ void __launch_bounds__(256) lora_expand_kernel(ExpandArgs g) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fg = lane >> 4;
    const int tile = (int)(blockIdx.x / (unsigned)g.col_blocks);
    const RowTile t = find_tile<16 * RT>(g.plan, g.M, g.lora.L, tile, lane);
    if (t.count <= 0) return;
    const bool has = t.group < g.lora.L;
    if (!has && g.base == g.out) return;   // rows without an adapter, in place
    const int32_t *order = g.plan + g.lora.L + 2;
    const int64_t n0 = (int64_t)((int)blockIdx.x - tile * g.col_blocks) * 256 + wave * 64;
    int row[RT];
    int64_t at[RT];
    u32x4 bv[RT][2];
#pragma unroll
    for (int i = 0; i < RT; i++) {
        row[i] = tile_row(order, t, 16 * i + fr, g.M);
        const int64_t band = row[i] / g.band_rows;
        at[i] = band * g.band_stride + (row[i] - band * g.band_rows) * g.N + n0 + 8 * fg;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            bv[i][h] = (u32x4){0u, 0u, 0u, 0u};
            if (row[i] < g.M && n0 + 8 * fg + 32 * h < g.N)
                bv[i][h] = __builtin_nontemporal_load((const u32x4 *)(g.base + at[i] + 32 * h));
        }
    }
    v4f acc[RT][4];
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    if (has) {
        const float s = g.lora.scale ? g.lora.scale[t.group] : 1.0f;
        const uint16_t *br[4];
#pragma unroll
        for (int j = 0; j < 4; j++) br[j] = lora_brow(g.lora, t.group, n0 + lora_col(j, fr), g.N);
        for (int r0 = 0; r0 < g.lora.R; r0 += 32) {
            const int r = r0 + 8 * fg;
            v8bf b[4];
#pragma unroll
            for (int j = 0; j < 4; j++) b[j] = lora_load_b(br[j], r, g.lora.R);
#pragma unroll
            for (int i = 0; i < RT; i++) {
                v8bf hi, lo;
                lora_load_h(g.lora, row[i], row[i] < g.M, r, s, hi, lo);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], hi, acc[i][j], 0, 0, 0);
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], lo, acc[i][j], 0, 0, 0);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
            if (row[i] >= g.M || n0 + 8 * fg + 32 * h >= g.N) continue;
            u32x4 o;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const v4f &c = acc[i][2 * h + (e >> 1)];
                o[e] = pack_bf16x2(bf16_lo(bv[i][h][e]) + c[2 * (e & 1)], bf16_hi(bv[i][h][e]) + c[2 * (e & 1) + 1]);
            }
            __builtin_nontemporal_store(has ? o : bv[i][h], (u32x4 *)(g.out + at[i] + 32 * h));
        }
}

}  // namespace

int bs_launch_lora_plan(const int32_t *ids, int32_t *plan, int64_t M, int L, hipStream_t stream) {
    return bs_enqueue(lora_plan_kernel, dim3(L + 1), dim3(PLAN_WAVES * 64), stream, ids, plan, M, L);
}

int bs_launch_lora_shrink(const uint16_t *x, const uint16_t *A, const int32_t *plan, float *H, int64_t M, int64_t K,
                          int L, int R, hipStream_t stream) {
    const ShrinkArgs g = {x, A, plan, H, (int)M, L, R, K};
    const dim3 grid((unsigned)max_tiles(M, L, 16), (unsigned)((R + 63) / 64));
    return bs_enqueue(lora_shrink_kernel<1, 4, 8>, grid, dim3(512), stream, g);
}

int bs_launch_lora_expand(const LoraArgs &lora, const int32_t *plan, const uint16_t *base, uint16_t *out, int64_t M,
                          int64_t N, int64_t band_rows, int64_t band_stride, hipStream_t stream) {
    const int64_t cols = (N + 255) / 256, blocks = max_tiles(M, lora.L, 16) * cols;
    if (blocks > 0x7FFFFFFF) return -1;
    const ExpandArgs g = {lora, plan, base, out, (int)M, (int)cols, N, band_rows, band_stride};
    return bs_enqueue(lora_expand_kernel<1>, dim3((unsigned)blocks), dim3(256), stream, g);
}
