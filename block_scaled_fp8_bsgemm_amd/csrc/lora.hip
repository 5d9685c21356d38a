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
// stays in registers.  64 rows and 8 adapters: 4.4 us, 16384 rows and 64
// adapters: 5.8, of which a launch that does nothing takes about 3.
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

// Workgroups of at most 512 lanes in a grid of x by y (or z) of them: a launch
// holds fewer than 2^32 lanes along x, which the tiles of 2^29 rows pass.
constexpr int64_t GRID_X = (int64_t)1 << 22;
inline unsigned grid_x(int64_t n) { return (unsigned)(n < GRID_X ? n : GRID_X); }
inline unsigned grid_more(int64_t n) { return (unsigned)((n + GRID_X - 1) / GRID_X); }

// The batch row of the tile's row `lane`, one load for the wave; M (no row) past
// the tile's count or for an entry that is no row.  Any lane's is then had by a
// shuffle.
__device__ __forceinline__ int tile_rows(const int32_t *order, const RowTile &t, int lane, int M) {
    const int m = order[t.first + min(lane, t.count - 1)];
    return lane < t.count && (uint32_t)m < (uint32_t)M ? m : M;
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

// Eight bf16 of a row from k on.  TAIL: zero past its end (K % 8 == 0).
template <bool TAIL>
__device__ __forceinline__ v8bf load_k(const uint16_t *row, int64_t k, int64_t K) {
    const u32x4 v = *(const u32x4 *)(row + (TAIL && k >= K ? 0 : k));
    const u32x4 z = {0u, 0u, 0u, 0u};
    return __builtin_bit_cast(v8bf, TAIL && k >= K ? z : v);
}

// UN turns of a wave, `step` apart from k on: every load before the first product.
template <int RT, int CT, int UN, bool TAIL>
__device__ __forceinline__ void shrink_steps(v4f (&acc)[RT][CT], const uint16_t *const (&xr)[RT],
                                             const uint16_t *const (&ar)[CT], int64_t k, int64_t step, int64_t K) {
    v8bf xv[UN][RT][2], av[UN][CT][2];
#pragma unroll
    for (int u = 0; u < UN; u++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int i = 0; i < RT; i++) xv[u][i][h] = load_k<TAIL>(xr[i], k + u * step + 32 * h, K);
#pragma unroll
            for (int j = 0; j < CT; j++) av[u][j][h] = load_k<TAIL>(ar[j], k + u * step + 32 * h, K);
        }
    __builtin_amdgcn_sched_barrier(0);   // the loads stay ahead of the products
#pragma unroll
    for (int u = 0; u < UN; u++)
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int i = 0; i < RT; i++)
#pragma unroll
                for (int j = 0; j < CT; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[u][j][h], xv[u][i][h], acc[i][j], 0, 0, 0);
}

// One workgroup: 16 RT rows of one adapter, 16 CT columns of H.  Its W waves
// take the K axis in turns of 64 and their partial sums are added in wave
// order through LDS, so a short batch still spreads K over a CU's waves and
// the result does not depend on timing.  A turn is two MFMAs of 32 k: for each a
// row's four lanes read 64 consecutive bytes, the two loads its 128.  The adapter's
// rows are the MFMA's first operand, which leaves a lane four consecutive columns of
// one row of H.
template <int RT, int CT, int W, int UN>
__global__ void __launch_bounds__(W * 64) lora_shrink_kernel(ShrinkArgs g) {
    __shared__ v4f part[W][RT * CT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fg = lane >> 4;
    const RowTile t = find_tile<16 * RT>(g.plan, g.M, g.L, blockIdx.z * GRID_X + blockIdx.x, lane);
    if (t.count <= 0) return;
    const int32_t *order = g.plan + g.L + 2;
    const int c0 = blockIdx.y * 16 * CT;
    const int rows = tile_rows(order, t, lane, g.M);
    int row[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) row[i] = __shfl(rows, 16 * i + fr, 64);
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
        int64_t k = wave * 64;
        for (; k + (UN - 1) * W * 64 + 64 <= g.K; k += UN * W * 64)
            shrink_steps<RT, CT, UN, false>(acc, xr, ar, k + 8 * fg, W * 64, g.K);
        for (; k < g.K; k += W * 64) shrink_steps<RT, CT, 1, true>(acc, xr, ar, k + 8 * fg, 0, g.K);
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
        const int m = __shfl(rows, 16 * (s / CT) + fr, 64);
        if (m < g.M && c < g.R) *(v4f *)(g.H + (int64_t)m * g.R + c) = sum;
    }
}

// ----------------------------------------------------------------- expand --

struct ExpandArgs {
    LoraArgs lora;
    const int32_t *plan;
    const uint16_t *base;   // bf16 row bands
    uint16_t *out;
    int M, band_rows;
    int col_blocks, chunks;   // workgroups along N, and 256-column chunks to each
    int64_t N, band_gap;
};

// Lanes l and l ^ 8 exchange v (a DPP rotation by 8 within each 16 lanes).
__device__ __forceinline__ u32x4 swap8(u32x4 v) {
    u32x4 r;
#pragma unroll
    for (int e = 0; e < 4; e++) r[e] = (uint32_t)__builtin_amdgcn_mov_dpp((int)v[e], 0x128, 0xF, 0xF, false);
    return r;
}

// One workgroup: 16 RT rows of one adapter and `chunks` column chunks of 256,
// 64 columns to a wave.  The rows' scale * H is split into its two bf16 once
// and kept in LDS for all of them: row i is 2 NCH 16-byte pieces, hi's pieces
// 0 .. NCH - 1 before lo's, each at its number xor (i mod 16), so that the 16 rows
// of a fragment read lie in different banks.
//
// The B rows are the MFMA's first operand, its fragment rows taken in the order
// of lora_col, so that lane l = r + 16 g holds 16-byte pieces g and 4 + g of
// row r's 128 bytes.  base and out move in whole 128-byte row segments, eight
// rows to an instruction: X covers rows 0..7 of a 16-row group, lanes r < 8
// piece g and lanes r >= 8 piece 4 + g of row r % 8, and Y rows 8..15 with the
// pieces the other way round; one exchange between lanes l and l ^ 8 goes from
// either form to the other.  base is loaded before the products and added to
// them in fp32; out is rounded once.
template <int RT, int RMAX>
__global__ void __launch_bounds__(256) lora_expand_kernel(ExpandArgs g) {
    constexpr int NCH = RMAX / 8;
    __shared__ u32x4 sh[16 * RT * 2 * NCH];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fg = lane >> 4;
    const unsigned wg = blockIdx.y * (unsigned)GRID_X + blockIdx.x;
    const int tile = (int)(wg / (unsigned)g.col_blocks);
    const RowTile t = find_tile<16 * RT>(g.plan, g.M, g.lora.L, tile, lane);
    if (t.count <= 0) return;
    const bool has = t.group < g.lora.L;
    if (!has && g.base == g.out) return;   // rows without an adapter, in place
    const int rows = tile_rows(g.plan + g.lora.L + 2, t, lane, g.M);
    if (has) {
        const float s = g.lora.scale ? g.lora.scale[t.group] : 1.0f;
#pragma unroll
        for (int k = 0; k < (16 * RT * NCH + 255) / 256; k++) {
            const int i = (threadIdx.x + 256 * k) / NCH, c = threadIdx.x % NCH;
            if (i >= 16 * RT) break;   // whole waves: NCH divides 64
            const int m = __shfl(rows, i, 64);
            v8bf hi, lo;
            lora_split(lora_load_h(g.lora, m, m < g.M, 8 * c), s, hi, lo);
            sh[i * 2 * NCH + (c ^ (i & 15))] = __builtin_bit_cast(u32x4, hi);
            sh[i * 2 * NCH + ((NCH + c) ^ (i & 15))] = __builtin_bit_cast(u32x4, lo);
        }
        __syncthreads();
    }
    const bool up = fr >= 8;
    int64_t at[RT][2];     // first element of the X and Y rows; negative: no row
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int m = __shfl(rows, 16 * i + 8 * h + (fr & 7), 64);
            // band_gap: what a band's stride has beyond its rows
            const int64_t gap = g.band_gap ? g.band_gap * ((uint32_t)m / (uint32_t)g.band_rows) : 0;
            at[i][h] = m < g.M ? m * g.N + gap : -1;
        }
    const int64_t first = (int64_t)((int)wg - tile * g.col_blocks) * g.chunks;
    const int64_t end = min((first + g.chunks) * 256, g.N);
    const int dx = 8 * fg + (up ? 32 : 0), dy = 8 * fg + (up ? 0 : 32);
    const int64_t c0 = first * 256;
    const __amdgpu_buffer_rsrc_t rB = lora_rsrc(g.lora, has ? t.group : 0, c0, g.N);
    auto load_b = [&](v8bf(&b)[4], int64_t n, int r0) {
#pragma unroll
        for (int j = 0; j < 4; j++)
            b[j] = lora_load_b(rB, (int)(n - c0) + lora_col(j, fr), r0 + 8 * fg, g.lora.R);
    };
    v8bf bnext[4];
    if (has) load_b(bnext, first * 256 + wave * 64, 0);
    for (int64_t n0 = first * 256 + wave * 64; n0 < end; n0 += 256) {
        u32x4 xy[RT][2];   // base's pieces (anything where there are none)
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int64_t n = n0 + (h ? dy : dx);
                xy[i][h] = __builtin_nontemporal_load(
                    (const u32x4 *)(g.base + (at[i][h] >= 0 && n < g.N ? at[i][h] + n : 0)));
            }
        if (has) {
            v4f acc[RT][4];
#pragma unroll
            for (int i = 0; i < RT; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
            for (int r0 = 0; r0 < g.lora.R; r0 += 32) {
                const int r = r0 + 8 * fg;
                v8bf b[4];
#pragma unroll
                for (int j = 0; j < 4; j++) b[j] = bnext[j];
                const bool last = r0 + 32 >= g.lora.R;
                load_b(bnext, last ? n0 + 256 : n0, last ? 0 : r0 + 32);
#pragma unroll
                for (int i = 0; i < RT; i++) {
                    const u32x4 *row = sh + (16 * i + fr) * 2 * NCH;
                    const v8bf hi = __builtin_bit_cast(v8bf, row[(r / 8) ^ fr]);
                    const v8bf lo = __builtin_bit_cast(v8bf, row[(NCH + r / 8) ^ fr]);
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], hi, acc[i][j], 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], lo, acc[i][j], 0, 0, 0);
                }
            }
#pragma unroll
            for (int i = 0; i < RT; i++) {
                const u32x4 lo = up ? xy[i][1] : xy[i][0], hi = swap8(up ? xy[i][0] : xy[i][1]);
                u32x4 o[2];
#pragma unroll
                for (int h = 0; h < 2; h++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const uint32_t w = h ? hi[e] : lo[e];
                        const v4f &c = acc[i][2 * h + (e >> 1)];
                        o[h][e] = pack_bf16x2(bf16_lo(w) + c[2 * (e & 1)], bf16_hi(w) + c[2 * (e & 1) + 1]);
                    }
                const u32x4 oh = swap8(o[1]);
                xy[i][0] = up ? oh : o[0];
                xy[i][1] = up ? o[0] : oh;
            }
        }
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int64_t n = n0 + (h ? dy : dx);
                if (at[i][h] >= 0 && n < g.N)
                    __builtin_nontemporal_store(xy[i][h], (u32x4 *)(g.out + at[i][h] + n));
            }
    }
}

}  // namespace

int bs_launch_lora_plan(const int32_t *ids, int32_t *plan, int64_t M, int L, hipStream_t stream) {
    return bs_enqueue(lora_plan_kernel, dim3(L + 1), dim3(PLAN_WAVES * 64), stream, ids, plan, M, L);
}

template <int RT, int CT, int UN>
static int launch_shrink(const ShrinkArgs &g, hipStream_t stream) {
    constexpr int W = 8;
    const int64_t tiles = max_tiles(g.M, g.L, 16 * RT);
    const dim3 grid(grid_x(tiles), (unsigned)((g.R + 16 * CT - 1) / (16 * CT)), grid_more(tiles));
    return bs_enqueue(lora_shrink_kernel<RT, CT, W, UN>, grid, dim3(64 * W), stream, g);
}

// Long batches take 64 rows and 64 ranks a workgroup, which reads x once per 64 ranks
// and A once per 64 rows.  Its 128 KiB of partial sums leave a CU one workgroup, so
// more than 256 tiles with an adapter take a second round: M = 16384, K = 2048, R = 64
// takes 20 us up to there and 33 with an adapter on each of its rows, strewn over
// eight (R = 128: 38 and 51; R = 256: 73 and 87).  Shorter batches spread the ranks over
// workgroups, since one CU then waits for fewer of A's bytes.  Graph launches at
// K = 2048, R = 64, 8 adapters, us for (64 rows, 64 ranks) / (16, 64) / (16, 32) /
// (16, 16): M = 16384: 20.4 / 37.6 / 44.6 / 56.3; M = 4096: 18.5 / 12.8 / 14.5 / 19.6;
// M = 1024: 18.0 / 12.5 / 9.0 / 10.9; M = 256, mixed: 15.4 / 11.7 / 8.5 / 6.8.
int bs_launch_lora_shrink(const uint16_t *x, const uint16_t *A, const int32_t *plan, float *H, int64_t M, int64_t K,
                          int L, int R, hipStream_t stream) {
    const ShrinkArgs g = {x, A, plan, H, (int)M, L, R, K};
    if (M >= 8192) return launch_shrink<4, 4, 1>(g, stream);
    if (M >= 2048) return launch_shrink<1, 4, 2>(g, stream);
    if (M >= 512) return launch_shrink<1, 2, 2>(g, stream);
    return launch_shrink<1, 1, 4>(g, stream);
}

template <int RT, int RMAX>
static int launch_expand(ExpandArgs g, hipStream_t stream) {
    const int64_t cols = (g.N + 255) / 256, tiles = max_tiles(g.M, g.lora.L, 16 * RT);
    // A workgroup takes as many column chunks as leave about 1024 of them, two rounds
    // of the 512 that the registers let a device hold at RT = 4: a long run of
    // chunks pays for finding the tile and splitting its H once.  M = 16384,
    // N = 5120, 8 adapters of rank 32 / 64 / 128: 79.6 / 86.8 / 104.9 us, against
    // 84.5 / 87.1 / 103.4 at 512 workgroups, 80.5 / 92.0 / 111.8 at 2048 and 90.0 /
    // 97.4 / 117.8 at one chunk to each.
    int64_t chunks = tiles * cols / 1024;
    chunks = chunks < 1 ? 1 : chunks > cols ? cols : chunks;
    if (chunks > 4096) chunks = 4096;   // offsets within a workgroup's part of B: below 2^30
    g.chunks = (int)chunks;
    g.col_blocks = (int)((cols + chunks - 1) / chunks);
    const int64_t n = tiles * g.col_blocks;
    if (n > 0x7FFFFFFF) return -1;
    return bs_enqueue(lora_expand_kernel<RT, RMAX>, dim3(grid_x(n), grid_more(n)), dim3(256), stream, g);
}

template <int RT>
static int launch_expand_r(const ExpandArgs &g, hipStream_t stream) {
    if (g.lora.R <= 64) return launch_expand<RT, 64>(g, stream);
    if (g.lora.R <= 128) return launch_expand<RT, 128>(g, stream);
    return launch_expand<RT, 256>(g, stream);
}

int bs_launch_lora_expand(const LoraArgs &lora, const int32_t *plan, const uint16_t *base, uint16_t *out, int64_t M,
                          int64_t N, int64_t band_rows, int64_t band_stride, hipStream_t stream) {
    const ExpandArgs g = {lora, plan, base, out, (int)M, (int)band_rows, 0, 0, N, band_stride - band_rows * N};
    // 64-row tiles once an adapter has 32 rows on average and there is work for every
    // CU.  R = 64, rows mixed, 16-row tiles / 64-row, us by graph launches: N = 7168, 8
    // adapters, M = 128: 8.4 / 8.7, 512: 13.0 / 10.5, 2048: 31.5 / 23.5; 32 adapters,
    // M = 512: 17.6 / 19.1, 2048: 42.7 / 27.1; N = 1024, M = 512: 5.3 / 7.9, 2048: 8.0 /
    // 8.4, 8192: 19.6 / 14.1.  32-row tiles lie between the two.
    if (M >= 32 * (int64_t)(lora.L + 1) && M * N >= (int64_t)1 << 21) return launch_expand_r<4>(g, stream);
    return launch_expand_r<1>(g, stream);
}
