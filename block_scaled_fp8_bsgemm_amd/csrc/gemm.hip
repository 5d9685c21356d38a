// gemm.hip -- block-scale fp8 GEMM with a destination-major band epilogue
// for gfx950 (MI355X).
//
// Computes C = A * B^T for A [M,K] e4m3 with one fp32 scale per 1x128 block
// and B [N,K] e4m3 with one fp32 scale per 128x128 block, accumulating in
// fp32 and writing bf16 ("MORI GEMM + All-Reduce Benchmark", "Running the
// benchmark", --quant blockscale; sglang PR 40757, "What").  Each 128-deep K
// block of a 16x16 output sub-tile is one v_mfma_f32_16x16x128_f8f6f4 into a
// zeroed fp32 temporary; its result is folded into the running accumulator
// with one fma by the block's combined scale a_scale[m,kb] * b_scale[n/128,kb],
// K blocks in ascending order.  The epilogue writes each output row straight
// into its destination's row band (sglang PR 40757, "What": the GEMM writes
// each destination's row band as its own unit).
//
// Tiling (one workgroup = 8 waves = 512 lanes, one 256x256 output tile):
//  - per K block the A tile [256 x 128 B] and B tile [256 x 128 B] are staged
//    in LDS, double buffered (2 x 64 KiB); rows are placed in even / odd
//    128-byte slots and 16-byte chunks XOR-swizzled (swz) so that every MFMA
//    operand read is served without bank conflicts;
//  - global loads use buffer descriptors that end where the matrix ends, so
//    rows past M (a ragged last tile) read as zero without any branch;
//  - waves form a 2 (M) x 4 (N) grid of 128 x 64 wave tiles (8 x 4 MFMA
//    sub-tiles, 128 fp32 accumulator registers per lane);
//  - the MFMA takes the B fragment as its first operand, so each lane ends up
//    holding 4 consecutive output columns of one output row: one combined
//    scale per lane per sub-tile row;
//  - the K block's a_scale values of the tile's 256 rows and its b_scale
//    values are DMA'd into LDS with the operands; each wave forms its rows'
//    combined scales a_scale * b_scale in registers;
//  - at the end each wave stores its 128 x 64 bf16 sub-tile straight from
//    the accumulators as whole 128-byte row segments of the destination
//    band, eight rows per instruction (B's rows are staged in an order that
//    makes this possible; non-temporal stores in the blockscale kernels);
//  - workgroup -> tile mapping is XCD-aware: workgroups are dealt to the 8
//    XCDs round-robin, so each XCD is given a contiguous run of tiles, ordered
//    in groups of 4 M-tiles so that concurrently running tiles share A and B
//    panels in that XCD's L2 (its 32 concurrent tiles span 4 M-tiles x 8
//    N-tiles; measured faster than 8 x 4, 2 x 16 or 1 x 32).
//
// When K / 128 is even (the benchmark's K = 2048) and each operand stays
// under 2^31 bytes, the blockscale and mxfp8 GEMMs run as persistent kernels
// instead: one workgroup per CU walks several tiles, so the workgroup launch
// is not paid per tile, a tile's last K block already loads the next tile's
// first, and a finished tile's stores drain under the next tile's first K
// block (in the blockscale one, half of them go out between its MFMAs).
// Results are bit-identical to the tile kernels'.
//
// A second blockscale kernel reads B in a prepacked form (the same bytes in the
// MFMA's operand order, written once by bprepack_kernel) straight into
// registers instead of staging it in LDS; its results are bit-identical.
//
// The same tile kernel is also built for the mxfp8 variant (sglang PR 43480,
// "What" and "Not in this PR": e4m3 operands with one E8M0 scale byte per
// 1x32 block of A's and B's rows): there the scales are applied by the scaled
// MFMA v_mfma_scale_f32_16x16x128_f8f6f4 itself, the MFMAs accumulate
// directly, and the stage's scale piece carries the tile rows' scale bytes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "act.hpp"
#include "codec.hpp"
#include "launch.hpp"
#include "lora.hpp"

namespace {

constexpr int BM = 256, BN = 256, BK = 128;
constexpr int NTHREADS = 512;
constexpr int WM = 128, WN = 64;        // wave tile
constexpr int TM = WM / 16, TN = WN / 16;
constexpr int GROUP_M = 4;
constexpr int NUM_XCD = 8;

typedef int v8i __attribute__((ext_vector_type(8)));

struct GemmArgs {
    const uint8_t *A;
    const void *sa;         // blockscale: fp32 [M, K/128]; mxfp8: E8M0 bytes [M, K/32]
    const uint8_t *B;
    const void *sb;         // blockscale: fp32 [N/128, K/128]; mxfp8: E8M0 bytes [N, K/32]
    uint16_t *C;
    int64_t M, N, K;
    int64_t band_rows, band_stride;
    int KB;                 // K / 128
    int NB;                 // N / 128
    int tiles_m, tiles_n;
};

// The two pipeline stages are distinct LDS objects so that the compiler can
// tell a DMA into one stage from reads of the other and does not serialise
// them with a wait.
__shared__ __attribute__((aligned(1024))) uint8_t sA0[BM * BK];
__shared__ __attribute__((aligned(1024))) uint8_t sA1[BM * BK];
__shared__ __attribute__((aligned(1024))) uint8_t sB0[BN * BK];
__shared__ __attribute__((aligned(1024))) uint8_t sB1[BN * BK];
// scales per stage, one dword per entry: blockscale: [0, 256) a_scale of the
// tile's rows (in the order of sa_row); [256, 512) four 64-entry slots filled by waves 4..7 with
// b_scale, of which entries 256 and 257 (the tile's two 128-column blocks) are
// read.  mxfp8: [0, 256) the K block's 4 E8M0 bytes of each A row, [256, 512)
// those of each B row.
constexpr int SCALES = BM + 256;
__shared__ __attribute__((aligned(1024))) float sS0[SCALES];
__shared__ __attribute__((aligned(1024))) float sS1[SCALES];

template <int ST> __device__ __forceinline__ uint8_t *stA() { return ST ? sA1 : sA0; }
template <int ST> __device__ __forceinline__ uint8_t *stB() { return ST ? sB1 : sB0; }
template <int ST> __device__ __forceinline__ float *stS() { return ST ? sS1 : sS0; }


// Byte offset of 16-byte chunk `c` (0..7) of tile row `r` inside a staged
// [rows x 128 B] operand tile.  An MFMA fragment read (ds_read_b128) has each
// 16-lane quarter read one chunk of 16 consecutive rows.  Within every 16-row
// group, rows 0-7 go to the even 128-byte slots and rows 8-15 to the odd
// ones, and chunks are XOR-swizzled by the row's low three bits: lanes 0-7 of
// a quarter then read banks 0-31 and lanes 8-15 banks 32-63, each half
// without conflicts, each lane from a different slot row.  Measured, this
// reads at the LDS's full rate; the plain row-major XOR swizzle, which also
// puts the 16 lanes in 64 distinct banks, reads at about half of it.
__device__ __forceinline__ int lds_slot(int r) { return (r & ~15) | ((r & 7) << 1) | ((r >> 3) & 1); }
__device__ __forceinline__ int swz(int r, int c) { return lds_slot(r) * 128 + ((c ^ (r & 7)) << 4); }

// B's rows are staged in a permuted order so that the epilogue can store C
// straight from the accumulators.  Each wave's 64 output columns are four
// 16-column MFMA sub-tiles j, and the MFMA leaves lane l with 4 consecutive
// columns 4 (l/16) .. +4 of its sub-tile.  If sub-tile j's fragment row r is
// B row brow_j(r) = 32 (j/2) + 8 (r/4) + 4 (j%2) + r%4 of the wave's 64, then
// lane l's columns of sub-tiles 0 and 1 are the 8 consecutive columns
// 8 (l/16) .. +8 and those of sub-tiles 2 and 3 the 8 at 32 + 8 (l/16): two
// 16-byte stores per lane and row group.  brow_of(R) applies this to LDS row
// R = 64 w + 16 j + r of the staged B tile; it is a permutation within each
// 64-row group, so each wave's columns still lie in one 128-column b_scale
// block.
__device__ __forceinline__ int brow_of(int R) {
    const int j = (R >> 4) & 3, r = R & 15;
    return (R & ~63) + 32 * (j >> 1) + 8 * (r >> 2) + 4 * (j & 1) + (r & 3);
}

// A tile's operand descriptors: its row panels of A and B, and its scales.
struct Panels {
    __amdgpu_buffer_rsrc_t rA, rB, rS;   // rS: a_scale (waves 0..3) or b_scale (4..7)
};

struct Loader {
    Panels P;                            // the current tile's
    __amdgpu_buffer_rsrc_t rZ;           // zero-size: every load through it reads nothing
    int poff;    // prepacked B: this lane's byte offset in its wave's first fragment
    int pstep;   // prepacked B: bytes from one 16-row group to the next (K/128 * 2 KiB)
    int voff;    // this lane's byte offset of its chunk in the A row panel (even slots i)
    int voff1;   // the same for odd slots i (the lane's chunk with bit 2 flipped)
    int voffB;   // the same two for the B panel, whose rows are fetched in the
    int voffB1;  //   permuted order of brow_of (see there)
    int k4;      // 4 rows of a panel, in bytes
    int soff;    // this lane's byte offset of its scale (a_scale row, or b_scale block)
    int ldsq;    // byte offset of this wave's first 1 KiB LDS slot
    int sdst;    // byte offset of this wave's 256-byte scale slot
};

// A tile's byte offsets in A, in B and in this wave's scales, or the change
// of them from one tile to another (persistent kernels).
struct TileOff {
    int a, b, s;
};

// One DMA instruction of a stage load: pieces 0..7 are the A and B slots
// i = piece / 2 (A for even pieces, B for odd), piece 8 the scales.  A block
// past the end (valid == false) goes through the zero-size descriptor: the
// loads touch no memory and the stage is not read again.  d moves the
// lanes' offsets to another tile of the same whole-matrix descriptors.
template <int ST, int PIECE>
__device__ __forceinline__ void dma_piece(const Loader &L, const Panels &P, int kb, bool valid,
                                          const TileOff &d = TileOff{0, 0, 0}) {
    const int koff = kb * BK;
    if (PIECE < 8) {
        const int i = PIECE >> 1;
        const int q = L.ldsq + i * 1024;
        if (PIECE & 1) {
            // B: slot i's global rows are those of slot 0 plus 0, 8, 4, 12
            const int vo = ((i & 1) ? L.voffB1 : L.voffB) + (2 * (i & 1) + (i >> 1)) * L.k4 + d.b;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(valid ? P.rB : L.rZ, (lds_void *)(stB<ST>() + q),
                                                     16, vo, koff, 0, 0);
        } else {
            // A: slot i's rows are those of slot 0 plus 0, 4, 16, 20 (see load_stage)
            const int vo = ((i & 1) ? L.voff1 : L.voff) + (4 * (i >> 1) + (i & 1)) * L.k4 + d.a;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(valid ? P.rA : L.rZ, (lds_void *)(stA<ST>() + q),
                                                     16, vo, koff, 0, 0);
        }
    } else {
        // blockscale: waves 0..3 fetch a_scale of rows 64w..64w+63, waves
        // 4..7 b_scale of the column blocks from the tile's first one on;
        // mxfp8: waves 0..3 fetch the 4 scale bytes of the K block for A rows
        // 64w.., waves 4..7 for B rows 64(w-4)..  Each wave fills its own
        // 256-byte slot; no branch: every wave issues exactly one.
        __builtin_amdgcn_raw_ptr_buffer_load_lds(valid ? P.rS : L.rZ,
                                                 (lds_void *)((uint8_t *)stS<ST>() + L.sdst), 4,
                                                 L.soff + d.s, kb * 4, 0, 0);
    }
}

// DMA the K block kb of the A and B panels and of the scales into stage ST.
// One buffer_load ... lds writes 64 lanes x 16 B = 1 KiB of LDS in lane order:
// eight 128-byte row slots, lane l on slot l/8 at physical chunk l%8.  Wave w's
// slot i (0..3) covers LDS slots 32w + 8i .. 32w + 8i + 7, which hold tile rows
// 32w + {0, 4, 16, 20}[i] + (l/16) + 8 * ((l/8) % 2) (lds_slot inverted), so
// every instruction still fetches eight whole 128-byte row segments; the lane
// fetches logical chunk (l%8) ^ (row & 7) of its row, which realises the
// swizzle.  B's LDS row R holds the tile's B row brow_of(R) (a permutation
// within each 64-row group), so slot i of wave w fetches B rows 32w + {0, 8,
// 4, 12}[i] + (l/16) + 16 * ((l/8) % 2).
template <int ST>
__device__ __forceinline__ void load_stage(const Loader &L, int kb, bool valid = true) {
    dma_piece<ST, 0>(L, L.P, kb, valid); dma_piece<ST, 1>(L, L.P, kb, valid);
    dma_piece<ST, 2>(L, L.P, kb, valid); dma_piece<ST, 3>(L, L.P, kb, valid);
    dma_piece<ST, 4>(L, L.P, kb, valid); dma_piece<ST, 5>(L, L.P, kb, valid);
    dma_piece<ST, 6>(L, L.P, kb, valid); dma_piece<ST, 7>(L, L.P, kb, valid);
    dma_piece<ST, 8>(L, L.P, kb, valid);
}

// One MFMA operand fragment: lane l's 32 bytes of a 16-row fragment are row
// r's 16-byte chunks g and g + 4 (g = l / 16), i.e. K [16g, 16g+16) and
// [64+16g, 64+16g+16) of the 128-deep block.  The 16x16x128 fp8 MFMA adds its
// products into the fp32 result in 16-slot passes taken from the bytes 0-15
// of lane groups 0..3 first, then from their bytes 16-31 (measured on the
// device, with and without scales); with this placement the passes cover K
// in ascending order, 16 at a time.  The scaled MFMA takes the lane's scale
// byte for K group g, which this placement also satisfies.
__device__ __forceinline__ v8i lds_frag(const uint8_t *st, int r, int g) {
    const u32x4 lo = *(const u32x4 *)(st + swz(r, g));
    const u32x4 hi = *(const u32x4 *)(st + swz(r, g + 4));
    return (v8i){(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                 (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

__device__ __forceinline__ void fold4(v4f &acc, const v4f &p, float s) {
#pragma unroll
    for (int e = 0; e < 4; e++) acc[e] = __builtin_fmaf(p[e], s, acc[e]);
}

__device__ __forceinline__ void wait_dma_and_sync() {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's DMAs have landed
    __syncthreads();                     // ... and every other wave's; LDS reads are done
}

// The scales of one K block for this wave's rows: a_scale of its 8 row
// groups (lane row m = 16 i + lane % 16 of the wave tile) and b_scale of its
// column block; their products are the combined scales s[i].
struct RawScales {
    float sa[TM];
    float sb, sb1;   // sb1: gated products only
};

// The a_scale slots hold the tile's 256 rows so that a lane's 8 values
// (row 128 wm + 16 i + frow, i = 0..7; q = 16 wm + frow) are two 16-byte
// pieces, i = 0..3 at slot 4 q and i = 4..7 at slot 128 + 4 q: two reads
// instead of eight, and consecutive lanes read consecutive 16-byte pieces
// (no bank conflicts).  Slot p holds row sa_row(p).
__device__ __forceinline__ int sa_row(int p) {
    const int q = (p >> 2) & 31, i = ((p >> 7) << 2) | (p & 3);
    return (q >> 4) * WM + i * 16 + (q & 15);
}

// The mxfp8 scale slots (4 bytes each: a row's scale bytes of the K block)
// hold the tile's 256 A rows, then its 256 B rows, so that the 8 A rows of a
// lane (row 128 wm + 16 i + frow, i = 0..7) sit in 8 consecutive slots, and
// so do its 4 B rows (the B rows of LDS rows 64 wn + 16 j + frow, j = 0..3):
// three 16-byte reads instead of twelve byte reads.  Slot p (waves 0..3 fill
// 0..255, waves 4..7 256..511) holds tile row mx_scale_row(p) of A or B.
__device__ __forceinline__ int mx_scale_row(int p) {
    if (p < BM) return (p & 128) | ((p & 7) << 4) | ((p >> 3) & 15);
    const int q = p - BM;
    return brow_of((q & ~63) | ((q & 3) << 4) | ((q >> 2) & 15));
}

template <int ST>
__device__ __forceinline__ void read_a_scales(RawScales &r, int wm, int frow) {
    const float *sc = stS<ST>();
    typedef float v4s __attribute__((ext_vector_type(4)));
    const v4s *q = (const v4s *)sc + (wm * 16 + frow);
    const v4s lo = q[0], hi = q[32];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        r.sa[i] = lo[i];
        r.sa[4 + i] = hi[i];
    }
}

template <int ST>
__device__ __forceinline__ void read_scales(RawScales &r, int wm, int wn, int frow) {
    // this wave's 64 columns lie inside one 128-column b_scale block
    r.sb = stS<ST>()[BM + (wn >> 1)];   // wave 4's slot: entries BM, BM+1
    read_a_scales<ST>(r, wm, frow);
}

__device__ __forceinline__ void combine_scales(float (&s)[TM], const RawScales &r) {
#pragma unroll
    for (int i = 0; i < TM; i++) s[i] = r.sa[i] * r.sb;
}

// A K block's combined scales: of row group i and column sub-tile j at(i, j).  Sub-tiles
// share the wave's one column block, except in a gated product (GLU), whose sub-tiles
// 0 and 1 are gate columns and 2 and 3 up columns, in another block: there the
// product of the two scales is formed at each use, for want of 8 registers.
template <bool GLU> struct Scales {
    float s[TM];
    __device__ __forceinline__ float at(int i, int) const { return s[i]; }
    __device__ __forceinline__ void set(const RawScales &r) { combine_scales(s, r); }
};
template <> struct Scales<true> {
    float sa[TM], sb[2];
    __device__ __forceinline__ float at(int i, int j) const { return sa[i] * sb[j >> 1]; }
    __device__ __forceinline__ void set(const RawScales &r) {
#pragma unroll
        for (int i = 0; i < TM; i++) sa[i] = r.sa[i];
        sb[0] = r.sb;
        sb[1] = r.sb1;
    }
};

// Row group 7's scales of the previous block, for its last three products.
template <bool GLU> struct TailScale {
    float s;
    __device__ __forceinline__ float at(int) const { return s; }
    __device__ __forceinline__ void set(const Scales<GLU> &c) { s = c.at(TM - 1, 0); }
};
template <> struct TailScale<true> {
    float s[2];
    __device__ __forceinline__ float at(int j) const { return s[j >> 1]; }
    __device__ __forceinline__ void set(const Scales<true> &c) {
        s[0] = c.at(TM - 1, 0);
        s[1] = c.at(TM - 1, 2);
    }
};

template <int ST, bool GLU>
__device__ __forceinline__ void read_block_scales(RawScales &r, int wm, int wn, int frow) {
    if constexpr (GLU) {   // wave 4's slot: entries BM (gate) and BM + 1 (up)
        r.sb = stS<ST>()[BM];
        r.sb1 = stS<ST>()[BM + 1];
        read_a_scales<ST>(r, wm, frow);
    } else {
        read_scales<ST>(r, wm, wn, frow);
    }
}

// The first fragments of the K block in stage ST, in the order the first
// MFMAs use them (A row group 0, then B column groups 0..3), then the scales.
template <int ST, bool GLU>
__device__ __forceinline__ void read_head(v8i &a, v8i (&bf)[TN], Scales<GLU> &s, int wm, int wn,
                                          int frow, int fc) {
    a = lds_frag(stA<ST>(), wm * WM + frow, fc);
#pragma unroll
    for (int j = 0; j < TN; j++) bf[j] = lds_frag(stB<ST>(), wn * WN + j * 16 + frow, fc);
    RawScales r;
    read_block_scales<ST, GLU>(r, wm, wn, frow);
    s.set(r);
}

// ---- mxfp8 --------------------------------------------------------------
// The scaled MFMA takes lane l's 32 bytes of a 16-row fragment as the K
// values [16g, 16g+16) and [64+16g, 64+16g+16) of row l%16 (g = l/16), the
// placement lds_frag gives, and lane l's scale byte as the E8M0 scale of that
// row's 32-wide block g: byte g of the row's 4 scale bytes for the K block.
// The scale bytes are held four to a register: byte i % 4 of a[i / 4] for A
// row group i, byte j of b for B column group j.  The scaled MFMA's op_sel
// picks the byte (mx_mfma), so a wave holds 3 registers of scales, not 12.
struct MxScales {
    int a[TM / 4];   // A rows of the wave's 8 row groups
    int b;           // B rows of its 4 column groups
};

// byte g of each of the four dwords of v, packed (byte i from dword i)
__device__ __forceinline__ int byte_g4(const u32x4 &v, int g) {
    // v_perm selects bytes of {hi, lo}: selector byte k in 0..7 picks that
    // byte, 0x0C gives 0
    const uint32_t s01 = 0x0C0C0400u + (uint32_t)g * 0x0101u;            // bytes g, 4 + g
    const uint32_t s23 = 0x04000C0Cu + (uint32_t)g * 0x01010000u;        // bytes 2, 3
    const uint32_t t01 = __builtin_amdgcn_perm(v[1], v[0], s01);
    const uint32_t t23 = __builtin_amdgcn_perm(v[3], v[2], s23);
    return (int)(t01 | t23);
}

template <int ST>
__device__ __forceinline__ void read_mx_scales(MxScales &x, int wm, int wn, int frow, int g) {
    // the slots of the lane's 8 A rows and of its 4 B rows are contiguous
    // (mx_scale_row): 32 and 16 bytes, each dword a row's 4 group bytes
    const uint8_t *sc = (const uint8_t *)stS<ST>();
    const u32x4 a0 = *(const u32x4 *)(sc + (wm * WM + frow * 8) * 4);
    const u32x4 a1 = *(const u32x4 *)(sc + (wm * WM + frow * 8) * 4 + 16);
    const u32x4 b = *(const u32x4 *)(sc + (BM + wn * WN + frow * 4) * 4);
    x.a[0] = byte_g4(a0, g);
    x.a[1] = byte_g4(a1, g);
    x.b = byte_g4(b, g);
}

// The scaled MFMA of A row group i and B column group j (both compile-time
// after unrolling), each scale byte selected by op_sel.
template <int OB>
__device__ __forceinline__ v4f mx_mfma_j(const v8i &b, const v8i &a, const v4f &c, int sb, int sa, int i) {
    switch (i & 3) {
    case 0: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, OB, sb, 0, sa);
    case 1: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, OB, sb, 1, sa);
    case 2: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, OB, sb, 2, sa);
    default: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, OB, sb, 3, sa);
    }
}
__device__ __forceinline__ v4f mx_mfma(const v8i &b, const v8i &a, const v4f &c, const MxScales &x, int i,
                                       int j) {
    const int sa = x.a[i >> 2];
    switch (j) {
    case 0: return mx_mfma_j<0>(b, a, c, x.b, sa, i);
    case 1: return mx_mfma_j<1>(b, a, c, x.b, sa, i);
    case 2: return mx_mfma_j<2>(b, a, c, x.b, sa, i);
    default: return mx_mfma_j<3>(b, a, c, x.b, sa, i);
    }
}

template <int ST>
__device__ __forceinline__ void read_head_mx(v8i &a, v8i (&bf)[TN], MxScales &x, int wm, int wn,
                                             int frow, int g) {
    a = lds_frag(stA<ST>(), wm * WM + frow, g);
#pragma unroll
    for (int j = 0; j < TN; j++) bf[j] = lds_frag(stB<ST>(), wn * WN + j * 16 + frow, g);
    read_mx_scales<ST>(x, wm, wn, frow, g);
}

// DMA of block kb + 1 into stage ST ^ 1 during the first nine MFMAs of block
// kb (see kblock); dma_block takes the block, its validity and the tile's
// panels explicitly.
template <int ST>
__device__ __forceinline__ void dma_block(const Loader &L, const Panels &P, int k, int kload, bool v,
                                          const TileOff &d = TileOff{0, 0, 0}) {
    if (k < 9) {
        if (k == 0) dma_piece<ST ^ 1, 8>(L, P, kload, v, d);
        if (k == 1) dma_piece<ST ^ 1, 0>(L, P, kload, v, d);
        if (k == 2) dma_piece<ST ^ 1, 1>(L, P, kload, v, d);
        if (k == 3) dma_piece<ST ^ 1, 2>(L, P, kload, v, d);
        if (k == 4) dma_piece<ST ^ 1, 3>(L, P, kload, v, d);
        if (k == 5) dma_piece<ST ^ 1, 4>(L, P, kload, v, d);
        if (k == 6) dma_piece<ST ^ 1, 5>(L, P, kload, v, d);
        if (k == 7) dma_piece<ST ^ 1, 6>(L, P, kload, v, d);
        if (k == 8) dma_piece<ST ^ 1, 7>(L, P, kload, v, d);
    }
}

// One mxfp8 K block from stage ST: the same schedule as the blockscale kblock
// below (A fragments one row group ahead, barrier after row group 6, the next
// block's head read between the MFMAs of row group 7, its DMA of block kload
// (moved by d to another tile) during the first nine MFMAs), but the block
// scales are applied inside the MFMA and each MFMA accumulates straight into
// its accumulator: no fold.
template <int ST>
__device__ __forceinline__ void kblock_mx(v4f (&acc)[TM][TN], v8i &a, v8i (&bf)[TN], MxScales &x,
                                          const Loader &L, int kload, bool vload, int wm, int wn,
                                          int frow, int g, const TileOff &d = TileOff{0, 0, 0}) {
    const uint8_t *as = stA<ST>();
    v8i an = a;
    v8i a_next = a;
    MxScales xn;
#pragma unroll
    for (int i = 0; i < TM; i++) {
        const v8i af = an;
        if (i + 1 < TM) an = lds_frag(as, wm * WM + (i + 1) * 16 + frow, g);
        if (i == TM - 1) {
            wait_dma_and_sync();
            a_next = lds_frag(stA<ST ^ 1>(), wm * WM + frow, g);
            read_mx_scales<ST ^ 1>(xn, wm, wn, frow, g);
        }
#pragma unroll
        for (int j = 0; j < TN; j++) {
            const int k = i * TN + j;
            acc[i][j] = mx_mfma(bf[j], af, acc[i][j], x, i, j);
            if (i == TM - 1) bf[j] = lds_frag(stB<ST ^ 1>(), wn * WN + j * 16 + frow, g);
            dma_block<ST>(L, L.P, k, kload, vload, d);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    x = xn;
    a = a_next;
}

// ---- blockscale with prepacked B -----------------------------------------
// The prepacked weight holds, for each 16-row group of B and K block, the
// 2 KiB the MFMA takes as its B operand, in lane order and split in two
// 1 KiB halves: half h, lane l = 16 g + r: bytes [16 g + 64 h, 16 g + 64 h + 16)
// of the 128-byte K segment of the group's fragment row r, which is B row
// brow_of(16 nt + r) (the order the LDS-staged kernels stage B in).  A wave loads its fragment j of block kb
// straight into registers with two fully coalesced 1 KiB loads; B needs no
// LDS and no DMA.  A block past the end loads through the zero-size
// descriptor.
template <int H>
__device__ __forceinline__ void load_bp_half(const Loader &L, v8i &f, int j, int kb, bool valid) {
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(valid ? L.P.rB : L.rZ, L.poff + H * 1024,
                                                          j * L.pstep + kb * 2048, 0);
#pragma unroll
    for (int e = 0; e < 4; e++) f[4 * H + e] = (int)v[e];
}

// The loads of block kb + 1 during the first MFMAs of block kb: the B
// fragments into the registers block kb - 1 used, the A slots and scales by
// DMA into the other stage (unread since the previous block's barrier).
template <int ST>
__device__ __forceinline__ void load_next_pb(const Loader &L, v8i (&bn)[TN], int k, int kb,
                                             int KB) {
    const bool v = kb + 1 < KB;
    if (k < 8) {
        if (k & 1) load_bp_half<1>(L, bn[k >> 1], k >> 1, kb + 1, v);
        else load_bp_half<0>(L, bn[k >> 1], k >> 1, kb + 1, v);
    }
    if (k == 0) dma_piece<ST ^ 1, 8>(L, L.P, kb + 1, v);
    if (k == 1) dma_piece<ST ^ 1, 0>(L, L.P, kb + 1, v);
    if (k == 2) dma_piece<ST ^ 1, 2>(L, L.P, kb + 1, v);
    if (k == 3) dma_piece<ST ^ 1, 4>(L, L.P, kb + 1, v);
    if (k == 4) dma_piece<ST ^ 1, 6>(L, L.P, kb + 1, v);
}

// The first K block of a tile: A slots and scales by DMA into stage ST, the
// B fragments into b; then the head reads (A row group 0, the scales).
template <int ST>
__device__ __forceinline__ void load_first_pb(const Loader &L, v8i (&b)[TN]) {
    dma_piece<ST, 8>(L, L.P, 0, true);
    dma_piece<ST, 0>(L, L.P, 0, true); dma_piece<ST, 2>(L, L.P, 0, true);
    dma_piece<ST, 4>(L, L.P, 0, true); dma_piece<ST, 6>(L, L.P, 0, true);
#pragma unroll
    for (int j = 0; j < TN; j++) {
        load_bp_half<0>(L, b[j], j, 0, true);
        load_bp_half<1>(L, b[j], j, 0, true);
    }
}

template <int ST>
__device__ __forceinline__ void read_head_pb(v8i &a, float (&s)[TM], int wm, int wn, int frow,
                                             int fc) {
    a = lds_frag(stA<ST>(), wm * WM + frow, fc);
    RawScales r;
    read_scales<ST>(r, wm, wn, frow);
    combine_scales(s, r);
}

// One K block as kblock below, with the B fragments of this block in bc and
// those of the next block loaded into bn.
template <int ST>
__device__ __forceinline__ void kblock_pb(v4f (&acc)[TM][TN], v4f (&p)[4], float &s_tail, v8i &a,
                                          const v8i (&bc)[TN], v8i (&bn)[TN], float (&s)[TM],
                                          const Loader &L, int kb, int KB, int wm, int wn,
                                          int frow, int fc) {
    const uint8_t *as = stA<ST>();
    v8i an = a;
    v8i a_next = a;
    RawScales rn;
#pragma unroll
    for (int i = 0; i < TM; i++) {
        const v8i af = an;
        if (i + 1 < TM) an = lds_frag(as, wm * WM + (i + 1) * 16 + frow, fc);
        if (i == TM - 1) {
            wait_dma_and_sync();
            a_next = lds_frag(stA<ST ^ 1>(), wm * WM + frow, fc);
            read_scales<ST ^ 1>(rn, wm, wn, frow);
        }
#pragma unroll
        for (int j = 0; j < TN; j++) {
            const int k = i * TN + j;
            p[k & 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                bc[j], af, (v4f){0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
            if (k >= 3) {
                const int kp = k - 3;
                fold4(acc[kp / TN][kp % TN], p[kp & 3], s[kp / TN]);
            } else {
                fold4(acc[TM - 1][k + 1], p[(k + 1) & 3], s_tail);
            }
            load_next_pb<ST>(L, bn, k, kb, KB);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    s_tail = s[TM - 1];
    combine_scales(s, rn);
    a = a_next;
}

// One K block from stage ST: 8 x 4 MFMAs per wave, each into a zeroed
// temporary p[k % 4] that is folded into its accumulator (one fma per
// element, by the row's combined scale) three MFMAs later, when it is
// certainly complete.  The fold pipeline runs on across K blocks: the last
// three products of a block are folded during the first MFMAs of the next,
// with that block's row-group-7 scale s_tail.
//
// The next K block kb + 1 goes to the other stage, which nobody reads after
// the previous block's barrier: its DMA is issued one instruction after each
// of nine consecutive MFMAs from MFMA SHIFT on (0 or DMA_SHIFT, see
// gemm_persistent).  After row group 6 (every fragment of this
// stage is then in registers) each wave waits for its DMA and the waves meet
// at a barrier; the reads of block kb + 1's first fragments and scales then go
// out between the MFMAs of row group 7, so that its MFMAs find them landed.
// The block loaded is block kload of the panels P, moved by d to another
// tile: the persistent kernel's last block of a tile loads the next tile's
// block 0, whose head it then reads.  After the last tile the DMA goes
// nowhere and those reads fetch unused values.  NEXT = false leaves both out:
// the other stage is then filled by the caller (the adapters' H, before this
// block) and waited for at the barrier.
template <int ST, int SHIFT = 0, bool NEXT = true, bool GLU>
__device__ __forceinline__ void kblock(v4f (&acc)[TM][TN], v4f (&p)[4], TailScale<GLU> &s_tail, v8i &a,
                                       v8i (&bf)[TN], Scales<GLU> &s, const Loader &L,
                                       const Panels &P, int kload, bool vload, int wm, int wn,
                                       int frow, int fc, const TileOff &d = TileOff{0, 0, 0}) {
    const uint8_t *as = stA<ST>();
    v8i an = a;
    v8i a_next = a;
    RawScales rn;
#pragma unroll
    for (int i = 0; i < TM; i++) {
        const v8i af = an;
        if (i + 1 < TM) an = lds_frag(as, wm * WM + (i + 1) * 16 + frow, fc);
        if (i == TM - 1) {
            wait_dma_and_sync();
            if constexpr (NEXT) {
                a_next = lds_frag(stA<ST ^ 1>(), wm * WM + frow, fc);
                read_block_scales<ST ^ 1, GLU>(rn, wm, wn, frow);
            }
        }
#pragma unroll
        for (int j = 0; j < TN; j++) {
            const int k = i * TN + j;
            p[k & 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                bf[j], af, (v4f){0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
            if (k >= 3) {
                const int kp = k - 3;
                fold4(acc[kp / TN][kp % TN], p[kp & 3], s.at(kp / TN, kp % TN));
            } else {
                // products 29, 30, 31 of the previous block: row group 7
                fold4(acc[TM - 1][k + 1], p[(k + 1) & 3], s_tail.at(k + 1));
            }
            if (NEXT && i == TM - 1) {
                bf[j] = lds_frag(stB<ST ^ 1>(), wn * WN + j * 16 + frow, fc);
            }
            // the DMA of the next block (kload, normally kb + 1) into the
            // other stage (unread since the previous block's barrier), one
            // instruction after each of nine consecutive MFMAs from MFMA
            // SHIFT on, away from the head reads of row group 7
            if (NEXT && k >= SHIFT) dma_block<ST>(L, P, k - SHIFT, kload, vload, d);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    s_tail.set(s);
    if constexpr (NEXT) s.set(rn);
    a = a_next;
}

constexpr int MODE_BS = 0, MODE_PB = 1, MODE_MX = 2;

// Workgroup (or, in the persistent kernel, virtual workgroup) b -> tile,
// XCD-aware and grouped: b runs on XCD b % 8, which is given the contiguous
// run of tiles [x * per_xcd, (x + 1) * per_xcd), ordered in groups of GROUP_M
// M-tiles.  False for the padding workgroups past the last tile.
template <int COLS = BN>
__device__ __forceinline__ bool tile_of(const GemmArgs &g, int b, int64_t &m0, int64_t &n0) {
    const int T = g.tiles_m * g.tiles_n;
    const int per_xcd = (T + NUM_XCD - 1) / NUM_XCD;
    if (b >= per_xcd * NUM_XCD) return false;
    const int t = (b % NUM_XCD) * per_xcd + b / NUM_XCD;
    if (t >= T) return false;
    const int group = t / (GROUP_M * g.tiles_n);
    const int first_m = group * GROUP_M;
    const int gm = min(GROUP_M, g.tiles_m - first_m);
    const int local = t - group * GROUP_M * g.tiles_n;
    m0 = (int64_t)(first_m + local % gm) * BM;
    n0 = (int64_t)(local / gm) * COLS;
    return true;
}

// The tile-dependent part of the loader in the tile kernels: descriptors of
// the tile's row panels and scales, zero past the end of the matrices.
template <int MODE, bool GLU = false>
__device__ __forceinline__ Panels panels_of(const GemmArgs &g, int64_t m0, int64_t n0, int wave) {
    const int64_t K = g.K;
    Panels P;
    P.rA = make_rsrc(g.A + m0 * K, (g.M - m0) * K);
    if (GLU)   // even waves stage gate rows, odd ones up rows
        P.rB = make_rsrc(g.B + (n0 + (wave & 1) * g.N) * K, (g.N - n0) * K);
    else if (MODE == MODE_PB)
        P.rB = make_rsrc(g.B + (n0 / 16) * ((int64_t)g.KB * 2048), (g.N - n0) * K);
    else
        P.rB = make_rsrc(g.B + n0 * K, (g.N - n0) * K);
    if (MODE == MODE_MX) {
        const int KQ = (int)(K / 32);   // mxfp8 scale bytes per row
        P.rS = wave < 4 ? make_rsrc((const uint8_t *)g.sa + m0 * KQ, (g.M - m0) * KQ)
                        : make_rsrc((const uint8_t *)g.sb + n0 * KQ, (g.N - n0) * KQ);
    } else {
        const int nb0 = (int)(n0 / 128);
        P.rS = wave < 4 ? make_rsrc((const float *)g.sa + m0 * g.KB, (g.M - m0) * g.KB * 4)
                        : make_rsrc((const float *)g.sb + (int64_t)nb0 * g.KB,
                                    (int64_t)((GLU ? 2 : 1) * g.NB - nb0) * g.KB * 4);
    }
    return P;
}

// The lane-dependent part, the same for every tile.  GLU: the up rows lie N rows
// behind the gate rows (WHOLE: in the same descriptor), and of the scale blocks wave 4's
// lane 0 fetches the gate columns' and lane 1 the up columns'.
template <int MODE, bool GLU = false, bool WHOLE = false>
__device__ __forceinline__ void init_loader(Loader &L, const GemmArgs &g, int wave, int lane) {
    const int K = (int)g.K;
    L.rZ = make_rsrc(g.A, 0);
    L.ldsq = wave * 4096;
    if (MODE == MODE_PB) {
        L.pstep = g.KB * 2048;
        L.poff = (wave & 3) * TN * L.pstep + lane * 16;
    }
    // slot 0's row and chunk of this lane (see load_stage); the odd slots'
    // rows are 4 further on, so their row & 7 has bit 2 set
    const int row = wave * 32 + (lane >> 4) + 8 * ((lane >> 3) & 1);
    const int chunk = (lane & 7) ^ (lane >> 4);
    L.voff = row * K + chunk * 16;
    L.voff1 = L.voff ^ 64;
    const int rowB = (GLU ? (wave >> 1) * 32 + (WHOLE ? (wave & 1) * (int)g.N : 0) : wave * 32) + (lane >> 4) +
                     16 * ((lane >> 3) & 1);   // = brow_of(LDS row)
    L.voffB = rowB * K + chunk * 16;
    L.voffB1 = L.voffB ^ 64;
    L.k4 = 4 * K;
    // blockscale: waves 0..3 fetch a_scale in the slot order of sa_row;
    // mxfp8: each row's 4 scale bytes in the slot order of mx_scale_row
    L.soff = MODE == MODE_MX ? mx_scale_row(wave * 64 + lane) * (K / 32)
                             : (wave < 4 ? sa_row(wave * 64 + lane) : GLU ? (lane & 1) * g.NB : lane) * g.KB * 4;
    L.sdst = wave * 256;
}

// The persistent kernels' descriptors cover whole matrices (each
// under 2^31 bytes, which the host checks), and a tile is a byte offset in
// the lanes' offsets: range-checked like them, so rows past the end still
// read zeros, and a tile change needs no new descriptor.
template <int MODE, bool GLU = false>
__device__ __forceinline__ Panels whole_panels(const GemmArgs &g, int wave) {
    Panels P;
    P.rA = make_rsrc(g.A, g.M * g.K);
    P.rB = make_rsrc(g.B, (GLU ? 2 : 1) * g.N * g.K);
    if (MODE == MODE_MX)
        P.rS = wave < 4 ? make_rsrc(g.sa, g.M * (g.K / 32)) : make_rsrc(g.sb, g.N * (g.K / 32));
    else
        P.rS = wave < 4 ? make_rsrc(g.sa, g.M * g.KB * 4)
                        : make_rsrc(g.sb, (int64_t)(GLU ? 2 : 1) * g.NB * g.KB * 4);
    return P;
}

// Tile (m0, n0)'s offsets for whole_panels: A's and B's row panels, and the
// scales this wave fetches (a_scale rows for waves 0..3, b_scale column
// blocks for 4..7).
template <int MODE>
__device__ __forceinline__ TileOff tile_off(const GemmArgs &g, int64_t m0, int64_t n0, int wave) {
    TileOff t;
    t.a = (int)(m0 * g.K);
    t.b = (int)(n0 * g.K);
    if (MODE == MODE_MX)
        t.s = (int)((wave < 4 ? m0 : n0) * (g.K / 32));
    else
        t.s = wave < 4 ? (int)(m0 * g.KB * 4) : (int)((n0 / 128) * g.KB * 4);
    return t;
}

__device__ __forceinline__ void shift_loader(Loader &L, const TileOff &d) {
    L.voff += d.a;
    L.voff1 += d.a;
    L.voffB += d.b;
    L.voffB1 += d.b;
    L.soff += d.s;
}

// Where the epilogue's stores go.  Row m0 + ml of a tile lies in band
// d0 + (r0 + ml) / band_rows at row (r0 + ml) % band_rows, with d0, r0 those
// of the tile's first row (rows < 2^31): one division per tile.  With bands
// of at least 256 rows a tile crosses at most one band boundary, at tile row
// mlb: rows before it are at element off0 + ml * N of C, rows from it on at
// off1 + ml * N, so each stored row costs a compare, a select and an add.
struct BandOut {
    int64_t off0, off1, lane_off, n;
    uint32_t br, d0, r0;
    int mlb, rows, ml0;
    bool col_ok;
};
__device__ __forceinline__ BandOut band_out(const GemmArgs &g, int64_t m0, int64_t n, int ml0) {
    BandOut o;
    o.n = n;
    o.ml0 = ml0;
    o.br = (uint32_t)g.band_rows;
    o.d0 = __builtin_amdgcn_readfirstlane((uint32_t)m0 / o.br);
    o.r0 = (uint32_t)m0 - o.d0 * o.br;
    o.rows = (int)(g.M - m0 < BM ? g.M - m0 : BM);   // tile rows inside M
    o.col_ok = n < g.N;
    o.lane_off = (int64_t)ml0 * g.N + n;
    o.off0 = (int64_t)o.d0 * g.band_stride + (int64_t)o.r0 * g.N;
    o.off1 = (int64_t)(o.d0 + 1) * g.band_stride - (int64_t)(o.br - o.r0) * g.N;
    o.mlb = o.br - o.r0 < (uint32_t)BM ? (int)(o.br - o.r0) : BM;
    return o;
}
template <int MODE>
__device__ __forceinline__ void store_piece(uint16_t *dst, u32x4 v) {
    // C is written once.  Inside the wo_b step, storing it non-temporally
    // made both the blockscale GEMM and the fused reduce that follows it
    // faster (step 338 -> 331 us); the mxfp8 GEMM, measured on its own,
    // was slower with it (162 -> 167 us) and keeps ordinary stores.
    if constexpr (MODE == MODE_MX) *(u32x4 *)dst = v;
    else __builtin_nontemporal_store(v, (u32x4 *)dst);
}

// Store one 16-byte piece of tile row ml = o.ml0 + dml (dml a constant) at
// column o.n + dn.
template <int MODE>
__device__ __forceinline__ void band_store(const GemmArgs &g, const BandOut &o, int dml, int dn, u32x4 v) {
    const int ml = o.ml0 + dml;
    if (ml >= o.rows || !o.col_ok) return;
    uint16_t *dst;
    if (o.br >= BM) {
        dst = g.C + ((ml < o.mlb ? o.off0 : o.off1) + o.lane_off + (int64_t)dml * g.N + dn);
    } else {
        const uint32_t rr = o.r0 + (uint32_t)ml;
        dst = g.C + ((int64_t)(o.d0 + rr / o.br) * g.band_stride + (int64_t)(rr % o.br) * g.N + o.n + dn);
    }
    store_piece<MODE>(dst, v);
}

// The epilogue: each wave's 128 x 64 bf16 sub-tile goes from the accumulators
// straight to the destination band, without LDS.  With B's rows staged in the
// order of brow_of, lane l = r + 16 g (r < 16) holds for row group i the 8
// consecutive columns 8 g .. +8 ("piece" g of the row's 8 16-byte pieces) of
// tile row 16 i + r in sub-tiles 0 and 1 (lo), and piece 4 + g in sub-tiles 2
// and 3 (hi).  Lanes l and l ^ 8 (rows r and r ^ 8) trade their hi pieces
// with one DPP row rotation by 8; then the lanes with r < 8 hold pieces g and
// 4 + g of row r and the lanes with r >= 8 pieces 4 + g and g of row r - 8
// (the X store), and likewise for rows r + 8 (the Y store).  Each store
// instruction so writes 8 whole 128-byte row segments, which measured faster
// than 16 half rows.  A wave's columns are either all inside N or all past it
// (N % 128 == 0).
__device__ __forceinline__ u32x4 swap_rows8(u32x4 v) {
    u32x4 r;
#pragma unroll
    for (int e = 0; e < 4; e++)   // row_ror:8 within each 16-lane row: lane l reads lane l ^ 8
        r[e] = (uint32_t)__builtin_amdgcn_mov_dpp((int)v[e], 0x128, 0xF, 0xF, false);
    return r;
}

// The pieces lane l stores for row group i: x for tile row 16 i + (l % 8) at
// column piece px, y for tile row 16 i + 8 + (l % 8) at piece px +- 4.
__device__ __forceinline__ void tile_pieces(const v4f (&acc)[TM][TN], int i, bool up, u32x4 &x, u32x4 &y) {
    const u32x4 lo = {pack_bf16x2(acc[i][0][0], acc[i][0][1]), pack_bf16x2(acc[i][0][2], acc[i][0][3]),
                      pack_bf16x2(acc[i][1][0], acc[i][1][1]), pack_bf16x2(acc[i][1][2], acc[i][1][3])};
    const u32x4 hi = swap_rows8(
        (u32x4){pack_bf16x2(acc[i][2][0], acc[i][2][1]), pack_bf16x2(acc[i][2][2], acc[i][2][3]),
                pack_bf16x2(acc[i][3][0], acc[i][3][1]), pack_bf16x2(acc[i][3][2], acc[i][3][3])});
#pragma unroll
    for (int e = 0; e < 4; e++) {
        x[e] = up ? hi[e] : lo[e];
        y[e] = up ? lo[e] : hi[e];
    }
}

// Whether every row and column of the tile is inside the matrix and the
// bands are contiguous (C is then plain row-major [M, N]): the epilogue of
// such a tile takes the fast path of store_tile, and every lane issues all
// 2 * TM of its stores.
template <int COLS = BN>
__device__ __forceinline__ bool tile_is_plain(const GemmArgs &g, int64_t m0, int64_t n0) {
    return m0 + BM <= g.M && n0 + COLS <= g.N && g.band_stride == g.band_rows * g.N;
}

// WIDE: rows may be more than 2^24 elements long.
template <int MODE, bool WIDE = true>
__device__ __forceinline__ void store_tile(const v4f (&acc)[TM][TN], const GemmArgs &g, int64_t m0,
                                           int64_t n0, int wave, int lane) {
    // opaque to the compiler, so that the addresses below are formed here
    // rather than hoisted out of a tile loop and kept live across it
    asm volatile("" : "+v"(lane));
    const int wm = wave >> 2, wn = wave & 3;
    const bool up = (lane >> 3) & 1;                 // r >= 8
    const int px = (lane >> 4) + (up ? 4 : 0);       // piece of the X store
    const int dny = up ? -32 : 32;                   // the Y store's piece, in columns from X's
    if ((!WIDE || g.N <= (int64_t)1 << 24) && tile_is_plain(g, m0, n0)) {
        // row-major C, no bounds: a uniform base per row group and one
        // 32-bit lane offset (rows 0 .. 143 of N elements)
        const uint32_t lx = (uint32_t)((wm * WM + (lane & 7)) * g.N + wn * WN + px * 8);
        const uint32_t ly = lx + (uint32_t)(8 * g.N + dny);
        uint16_t *base = g.C + m0 * g.N + n0;
#pragma unroll
        for (int i = 0; i < TM; i++) {
            u32x4 x, y;
            tile_pieces(acc, i, up, x, y);
            uint16_t *bi = base + (int64_t)i * 16 * g.N;
            store_piece<MODE>(bi + lx, x);
            store_piece<MODE>(bi + ly, y);
        }
        return;
    }
    const BandOut o = band_out(g, m0, n0 + wn * WN + px * 8, wm * WM + (lane & 7));
#pragma unroll
    for (int i = 0; i < TM; i++) {
        u32x4 x, y;
        tile_pieces(acc, i, up, x, y);
        band_store<MODE>(g, o, i * 16, 0, x);
        band_store<MODE>(g, o, i * 16 + 8, dny, y);
    }
}

// ---- bias, activation and residual -------------------------------------------
// The epilogue of bsgemm_fp8_act, on the finished fp32 accumulators before the one
// rounding to bf16:
//
//   t = acc + bias,  v = act(t)  or, gated (GLU),  v = act(t_gate) * t_up
//   C = alpha * resid + beta * v
//
// GLU: B has 2 N rows, gate rows first.  A tile's 256 rows of B are then 128 gate and
// the same 128 up columns, 32 and 32 to a wave: staged so that sub-tiles 0 and 1
// are gate columns in the order that brow_of gives them, and 2 and 3 the up columns of
// the same ones, a lane holds both of each of its 8 columns and the product stays in
// its registers.
enum { EPI_NONE, EPI_ACT, EPI_RESID, EPI_GLU };   // EPI_RESID: EPI_ACT with a residual

struct ActArgs {
    const uint16_t *bias;    // bf16 [N] (GLU: [2 N]) or null
    const uint16_t *resid;   // bf16 bands as C, or null; may be C
    float alpha, beta;
    int act;
};
struct ActGemmArgs {
    GemmArgs g;
    ActArgs q;
};

// Eight columns: t in place of their results.  bias, resid: 8 packed bf16 (zeros where
// there are none).
__device__ __forceinline__ void add8(float (&t)[8], u32x4 b) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
        t[2 * e] += bf16_lo(b[e]);
        t[2 * e + 1] += bf16_hi(b[e]);
    }
}
// N values v: alpha r + beta v, rounded after beta v and once more, or beta v.
template <int N, typename Bits>
__device__ __forceinline__ void join(float (&v)[N], Bits r, const ActArgs &q) {
#pragma clang fp contract(off)
#pragma unroll
    for (int e = 0; e < N; e++) v[e] = q.beta * v[e];
    if (q.resid) {
#pragma unroll
        for (int e = 0; e < N; e++) v[e] = __builtin_fmaf(q.alpha, e & 1 ? bf16_hi(r[e >> 1]) : bf16_lo(r[e >> 1]), v[e]);
    }
}
__device__ __forceinline__ u32x4 load_bias8(const ActArgs &q, int64_t n) {
    return q.bias ? *(const u32x4 *)(q.bias + n) : (u32x4){0u, 0u, 0u, 0u};
}
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
    return (u32x4){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// Element of C of row ml = o.ml0 + dml of a tile, column o.n + dn; negative past M.
__device__ __forceinline__ int64_t band_at(const GemmArgs &g, const BandOut &o, int dml, int dn) {
    const int ml = o.ml0 + dml;
    if (ml >= o.rows) return -1;
    if (o.br >= BM) return (ml < o.mlb ? o.off0 : o.off1) + o.lane_off + (int64_t)dml * g.N + dn;
    const uint32_t rr = o.r0 + (uint32_t)ml;
    return (int64_t)(o.d0 + rr / o.br) * g.band_stride + (int64_t)(rr % o.br) * g.N + o.n + dn;
}
__device__ __forceinline__ u32x4 load_resid8(const ActArgs &q, int64_t at) {
    return __builtin_nontemporal_load((const u32x4 *)(q.resid + (at < 0 ? 0 : at)));
}

// A tile's accumulators in place of their results (GLU: in sub-tiles 0 and 1).  The
// residual comes in the pieces of the store (tile_pieces), whole 128-byte row segments,
// BATCH row groups at a time, and goes to its columns' lanes by the same exchange.  Four
// at a time: M = 16384, N = 7168, K = 2048 with a residual 256 to 268 us on one card or
// another, 1 % and 2 % less than with eight and two, against 229 to 236 without bias, activation
// and residual.  What is left is the read of the residual after the products, 235 MB or 44 us
// at the rate of a large copy, of which about a third is behind the tiles of other CUs.  Half of it by
// DMA into the free stage during the last K block took 276 for 264 (264 non-temporal), and one
// kernel with and without a residual 264 for 256.
template <int EPI, int BATCH>
__device__ __forceinline__ void act_tile(v4f (&acc)[TM][TN], const GemmArgs &g, const ActArgs &q, int64_t m0,
                                         int64_t n0, int wave, int lane) {
    constexpr bool GLU = EPI == EPI_GLU;
    asm volatile("" : "+v"(lane));   // addresses formed here, not hoisted
    const int wm = wave >> 2, wn = wave & 3, frow = lane & 15, fg = lane >> 4;
    const bool up = (lane >> 3) & 1;
    const int64_t n = n0 + wn * (GLU ? 32 : 64);
    if (n >= g.N) return;   // N % 128 == 0: all of the wave's columns
    const u32x4 b0 = load_bias8(q, n + 8 * fg), b1 = load_bias8(q, n + 8 * fg + (GLU ? g.N : 32));
    const BandOut o = GLU ? band_out(g, m0, n + 8 * fg, wm * WM + frow)
                          : band_out(g, m0, n + 8 * fg + (up ? 32 : 0), wm * WM + (lane & 7));
#pragma unroll
    for (int h = 0; h < TM; h += BATCH) {
        u32x4 r[BATCH][2] = {};
        if (EPI == EPI_RESID || (GLU && q.resid)) {
#pragma unroll
            for (int i = 0; i < BATCH; i++)
#pragma unroll
                for (int y = 0; y < (GLU ? 1 : 2); y++)
                    r[i][y] = load_resid8(q, band_at(g, o, (h + i) * 16 + 8 * y, y ? (up ? -32 : 32) : 0));
        }
#pragma unroll
        for (int i = 0; i < BATCH; i++) {
            v4f(&c)[TN] = acc[h + i];
            u32x4 ra = r[i][0], rb = r[i][1];
            if (EPI == EPI_RESID) {
                ra = up ? r[i][1] : r[i][0];
                rb = swap_rows8(up ? r[i][0] : r[i][1]);
            }
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = c[e >> 2][e & 3];
            add8(v, b0);
            act_all(v, q.act);
            if constexpr (GLU) {
                float u[8];
#pragma unroll
                for (int e = 0; e < 8; e++) u[e] = c[2 + (e >> 2)][e & 3];
                add8(u, b1);
#pragma unroll
                for (int e = 0; e < 8; e++) v[e] *= u[e];
            }
            join(v, ra, q);
#pragma unroll
            for (int e = 0; e < 8; e++) c[e >> 2][e & 3] = v[e];
            if constexpr (!GLU) {
#pragma unroll
                for (int e = 0; e < 8; e++) v[e] = c[2 + (e >> 2)][e & 3];
                add8(v, b1);
                act_all(v, q.act);
                join(v, rb, q);
#pragma unroll
                for (int e = 0; e < 8; e++) c[2 + (e >> 2)][e & 3] = v[e];
            }
        }
    }
}

// The lane's 8 columns of a gated row group.
__device__ __forceinline__ u32x4 gated_piece(const v4f (&acc)[TM][TN], int i) {
    return (u32x4){pack_bf16x2(acc[i][0][0], acc[i][0][1]), pack_bf16x2(acc[i][0][2], acc[i][0][3]),
                   pack_bf16x2(acc[i][1][0], acc[i][1][1]), pack_bf16x2(acc[i][1][2], acc[i][1][3])};
}

// The gated tile's store: 64 bytes of 16 rows to an instruction.
__device__ __forceinline__ void store_gated_tile(const v4f (&acc)[TM][TN], const GemmArgs &g, int64_t m0, int64_t n0,
                                                 int wave, int lane) {
    asm volatile("" : "+v"(lane));
    const BandOut o = band_out(g, m0, n0 + (wave & 3) * 32 + (lane >> 4) * 8, (wave >> 2) * WM + (lane & 15));
#pragma unroll
    for (int i = 0; i < TM; i++) band_store<MODE_BS>(g, o, i * 16, 0, gated_piece(acc, i));
}

// ---- adapters --------------------------------------------------------------
struct LoraGemmArgs {
    LoraArgs lora;
    const int32_t *ids;     // int32 [M]: a row's adapter; outside [0, L): none
};

// Adds scale[a] (H[m] B[a]^T), a = ids[m], to the finished accumulators of a
// tile, in fp32, before the one rounding to bf16.
//
// 64 ranks at a time: the tile's 256 rows of H come by DMA into a stage, 32
// ranks (128 bytes a row) into its A part and 32 into its B part, in the row
// slots of the A tile.  The first 64 go to stage 1 during the last K block,
// which takes no next block there; later ones to the two stages in turn, during the
// products of those before.  A wave then turns the rows it loaded into scale *
// value split in two bf16, in place: of every two 16-byte chunks, eight ranks,
// the first gets the hi parts and the second the lo parts.  So the split is done
// once for the four waves that share the rows.
//
// A wave goes through the distinct adapters of its 128 rows (one or two in a
// prefill chunk, whose requests are runs of rows).  For each it has the
// adapter's 64 columns of B in registers, in the sub-tiles' own column order,
// and gives every 16-row group that has such a row its products, which only the
// adapter's own rows keep: a row takes nothing from another adapter, be its weights
// NaN, and a row of no adapter keeps its product bit for bit.
//
// Measured at M = 16384, N = 7168, K = 2048, 8 adapters in runs, against 213 us
// without adapters: R = 16 / 64 / 128: 235 / 253 / 287 us; every row its own
// draw of the 8 adapters, R = 64: 401 (keeping other rows' sums took 3 and 34 us
// over adding them zeros, which let one adapter's NaN into its neighbours).  What
// is left at R = 64 is B's latency (14 us), the split (7), the second product (5)
// and the fragments' reads (5), from copies with one of them left out.  This stands in the tile kernel:
// in the persistent one it spilled 64 to 95 registers and took 277 us.

// ids of the tile's rows, loaded with the tile's first K block
__shared__ int32_t sI[BM];
__shared__ float sR[BM];   // and their adapters' scales, before the last K block

// Waves 0..3 take 64 each; rows past M read as 0 and are told apart by their number.
__device__ __forceinline__ void load_ids(const GemmArgs &g, const LoraGemmArgs &q, int64_t m0, int wave, int lane) {
    if (wave < 4)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(q.ids + m0, (g.M - m0 < BM ? g.M - m0 : BM) * 4),
                                                 (lds_void *)&sI[wave * 64], 4, (wave * 64 + lane) * 4, 0, 0, 0);
}

// A tile row's adapter, -1 if it has none.
__device__ __forceinline__ int id_of(const GemmArgs &g, const LoraGemmArgs &q, int64_t m0, int r) {
    const int a = sI[r];
    return m0 + r < g.M && (uint32_t)a < (uint32_t)q.lora.L ? a : -1;
}

__device__ __forceinline__ bool tile_has_adapter(const GemmArgs &g, const LoraGemmArgs &q, int64_t m0, int lane) {
    bool has = false;
#pragma unroll
    for (int h = 0; h < 4; h++) has |= id_of(g, q, m0, 64 * h + lane) >= 0;
    return __ballot(has) != 0;
}

// H's ranks rc .. rc+63 into stage ST: slot i of wave w as in load_stage; a chunk
// past R goes out of the descriptor's range and reads as zero.
template <int ST>
__device__ __forceinline__ void lora_dma(const GemmArgs &g, const LoraGemmArgs &q, int64_t m0, int rc, int wave,
                                         int lane) {
    asm volatile("" : "+v"(lane));   // addresses formed here, not hoisted
    const int R = q.lora.R;
    const __amdgpu_buffer_rsrc_t rH = make_rsrc(q.lora.H + m0 * R, (g.M - m0 < BM ? g.M - m0 : BM) * R * 4);
#pragma unroll
    for (int h = 0; h < 2; h++) {
        if (rc + 32 * h >= R) break;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int row = wave * 32 + (lane >> 4) + 8 * ((lane >> 3) & 1) + 16 * (i >> 1) + 4 * (i & 1);
            const int r = rc + 32 * h + 4 * ((lane & 7) ^ (lane >> 4) ^ (4 * (i & 1)));
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rH, (lds_void *)((h ? stB<ST>() : stA<ST>()) + wave * 4096 + i * 1024), 16,
                r < R ? (row * R + r) * 4 : OUT_OF_RANGE, 0, 0, 0);
        }
    }
}

// One lane's 32 values of a row: the row's 128 bytes in st, split in place.
__device__ __forceinline__ void lora_split_row(uint8_t *st, int r, float s) {
#pragma unroll
    for (int c = 0; c < 4; c++) {
        u32x4 *p0 = (u32x4 *)(st + swz(r, 2 * c)), *p1 = (u32x4 *)(st + swz(r, 2 * c + 1));
        LoraH h;
        h.a = __builtin_bit_cast(v4f, *p0);
        h.b = __builtin_bit_cast(v4f, *p1);
        v8bf hi, lo;
        lora_split(h, s, hi, lo);
        *p0 = __builtin_bit_cast(u32x4, hi);
        *p1 = __builtin_bit_cast(u32x4, lo);
    }
}

// A wave's adapters: of its 128 rows, and the first one's B, which is loaded a
// step ahead.
struct LoraWave {
    int id[2];       // adapters of rows lane and 64 + lane
    int first;       // the first of them
    v8bf b0[TN];     // its B for the coming ranks rc .. rc+31
};

// Half h of ranks rc .. rc+63 of adapter a's B, for the wave's columns from n on;
// zero past R and N.
__device__ __forceinline__ void lora_b(v8bf (&b)[TN], const GemmArgs &g, const LoraGemmArgs &q, int a, int64_t n,
                                       int rc, int h, int lane) {
    const int R = q.lora.R, r = rc + 32 * h + 8 * (lane >> 4);
    if (rc + 32 * h >= R) return;
    const __amdgpu_buffer_rsrc_t rB = lora_rsrc(q.lora, a, n, g.N);
#pragma unroll
    for (int j = 0; j < TN; j++) b[j] = lora_load_b(rB, lora_col(j, lane & 15), r, R);
}

__device__ __forceinline__ int lora_first(const int (&id)[2], const uint64_t (&todo)[2]) {
    return todo[0] ? __builtin_amdgcn_readlane(id[0], __ffsll((unsigned long long)todo[0]) - 1)
                   : __builtin_amdgcn_readlane(id[1], __ffsll((unsigned long long)todo[1]) - 1);
}

// The wave's adapters from the ids in LDS, and the first one's B for ranks 0..31.
__device__ __forceinline__ void lora_begin(LoraWave &w, const GemmArgs &g, const LoraGemmArgs &q, int64_t m0,
                                           int64_t n, int wm, int lane) {
    w.id[0] = id_of(g, q, m0, wm * WM + lane);
    w.id[1] = id_of(g, q, m0, wm * WM + 64 + lane);
    const uint64_t all[2] = {__ballot(w.id[0] >= 0), __ballot(w.id[1] >= 0)};
    w.first = -1;
    if (all[0] | all[1]) {
        w.first = lora_first(w.id, all);
        lora_b(w.b0, g, q, w.first, n, 0, 0, lane);
    }
}

// The products of ranks rc .. rc+63, whose H is in stage ST.
template <int ST>
__device__ __forceinline__ void lora_chunk(v4f (&acc)[TM][TN], LoraWave &w, const GemmArgs &g, const LoraGemmArgs &q,
                                           float cs, int64_t n, int rc, int wm, int wave, int lane) {
    const int frow = lane & 15, fg = lane >> 4;
    const int R = q.lora.R;
    v8bf b1[TN];
    if (w.first >= 0) lora_b(b1, g, q, w.first, n, rc, 1, lane);
    // the first 32 lanes take the A part's rows, the others the B part's, of the
    // rows this wave loaded
    const int crow = wave * 32 + (lane & 31);
    if (lane < 32) lora_split_row(stA<ST>(), crow, cs);
    else if (rc + 32 < R) lora_split_row(stB<ST>(), crow, cs);
    barrier_lds_only();
    auto half = [&](int h, const v8bf(&b)[TN], const uint64_t (&mine)[2]) {
        if (rc + 32 * h >= R) return;
#pragma unroll
        for (int i = 0; i < TM; i++) {
            const uint32_t rows = (uint32_t)(mine[i >> 2] >> (16 * (i & 3))) & 0xFFFFu;
            if (!rows) continue;
            const bool live = (rows >> frow) & 1;
            const uint8_t *st = h ? stB<ST>() : stA<ST>();
            const int r = wm * WM + 16 * i + frow;
            const v8bf hi = *(const v8bf *)(st + swz(r, 2 * fg)), lo = *(const v8bf *)(st + swz(r, 2 * fg + 1));
            v4f t[TN];
#pragma unroll
            for (int j = 0; j < TN; j++) t[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], hi, acc[i][j], 0, 0, 0);
#pragma unroll
            for (int j = 0; j < TN; j++) t[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], lo, t[j], 0, 0, 0);
            // a lane's sums are those of row frow: other adapters' rows keep theirs
#pragma unroll
            for (int j = 0; j < TN; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) acc[i][j][e] = live ? t[j][e] : acc[i][j][e];
        }
    };
    if (w.first < 0) return;
    uint64_t todo[2] = {__ballot(w.id[0] >= 0), __ballot(w.id[1] >= 0)};
    int a = w.first;
    for (;;) {
        const uint64_t mine[2] = {__ballot(w.id[0] == a), __ballot(w.id[1] == a)};
        todo[0] &= ~mine[0];
        todo[1] &= ~mine[1];
        const bool more = (todo[0] | todo[1]) != 0;
        half(0, w.b0, mine);
        // a half's registers are free for what comes next: the next adapter, or the
        // first one's next ranks
        if (more) a = lora_first(w.id, todo);
        lora_b(w.b0, g, q, more ? a : w.first, n, more ? rc : rc + 64, 0, lane);
        half(1, b1, mine);
        if (!more) break;
        lora_b(b1, g, q, a, n, rc, 1, lane);
    }
}

// All ranks; the first 64 are in stage 1, and every wave has passed a barrier since.
__device__ __forceinline__ void lora_add(v4f (&acc)[TM][TN], const GemmArgs &g, const LoraGemmArgs &q, int64_t m0,
                                         int64_t n, int wm, int wave, int lane) {
    asm volatile("" : "+v"(lane));   // addresses formed here, not hoisted
    LoraWave w;
    lora_begin(w, g, q, m0, n, wm, lane);
    const int R = q.lora.R;
    const float cs = sR[wave * 32 + (lane & 31)];   // the scale of the row this lane splits
    for (int rc = 0;;) {
        if (rc + 64 < R) lora_dma<0>(g, q, m0, rc + 64, wave, lane);
        lora_chunk<1>(acc, w, g, q, cs, n, rc, wm, wave, lane);
        if ((rc += 64) >= R) return;
        wait_dma_and_sync();   // the next ranks are in, and these are read
        if (rc + 64 < R) lora_dma<1>(g, q, m0, rc + 64, wave, lane);
        lora_chunk<0>(acc, w, g, q, cs, n, rc, wm, wave, lane);
        if ((rc += 64) >= R) return;
        wait_dma_and_sync();
    }
}

// One 256x256 output tile.  MODE_BS: blockscale operands, A and B staged in
// LDS; MODE_PB: blockscale with the prepacked B loaded into registers;
// MODE_MX: mxfp8 operands (E8M0 scales per 1x32 block, applied by the scaled
// MFMA).
template <int MODE, bool LORA = false, int EPI = EPI_NONE>
__device__ __forceinline__ void gemm_tile(const GemmArgs &g, const LoraGemmArgs &q = {}, const ActArgs &ep = {}) {
    constexpr bool GLU = EPI == EPI_GLU;
    int64_t m0, n0;
    if (!tile_of<GLU ? BN / 2 : BN>(g, blockIdx.x, m0, n0)) return;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // wave-uniform: keep in SGPRs
    const int wm = wave >> 2, wn = wave & 3;
    const int KB = g.KB;
    constexpr bool MX = MODE == MODE_MX;

    if constexpr (LORA) load_ids(g, q, m0, wave, lane);
    bool any = false;   // whether a row of the tile has an adapter
    Loader L;
    init_loader<MODE, GLU>(L, g, wave, lane);
    L.P = panels_of<MODE, GLU>(g, m0, n0, wave);

    const int frow = lane & 15;
    const int fc = lane >> 4;   // the lane group: K chunks fc and fc + 4
    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};

    if constexpr (MODE == MODE_PB) {
        // stage 1 runs with the B registers bA, stage 0 with bB
        v8i a, bA[TN], bB[TN];
        float s[TM];
        if (KB & 1) {
            load_first_pb<0>(L, bB);
            wait_dma_and_sync();
            read_head_pb<0>(a, s, wm, wn, frow, fc);
        } else {
            load_first_pb<1>(L, bA);
            wait_dma_and_sync();
            read_head_pb<1>(a, s, wm, wn, frow, fc);
        }
        v4f p[4];
#pragma unroll
        for (int q = 0; q < 4; q++) p[q] = (v4f){0.f, 0.f, 0.f, 0.f};
        float s_tail = 0.f;
        int kb = 0;
        if (KB & 1) {
            kblock_pb<0>(acc, p, s_tail, a, bB, bA, s, L, 0, KB, wm, wn, frow, fc);
            kb = 1;
        }
        for (; kb < KB; kb += 2) {
            kblock_pb<1>(acc, p, s_tail, a, bA, bB, s, L, kb, KB, wm, wn, frow, fc);
            kblock_pb<0>(acc, p, s_tail, a, bB, bA, s, L, kb + 1, KB, wm, wn, frow, fc);
        }
#pragma unroll
        for (int j = 1; j < TN; j++) fold4(acc[TM - 1][j], p[(TM * TN - TN + j) & 3], s_tail);
    } else if constexpr (MX) {
        const int gq = lane >> 4;
        v8i a, bf[TN];
        MxScales x;
        if (KB & 1) {
            load_stage<0>(L, 0);
            wait_dma_and_sync();
            read_head_mx<0>(a, bf, x, wm, wn, frow, gq);
        } else {
            load_stage<1>(L, 0);
            wait_dma_and_sync();
            read_head_mx<1>(a, bf, x, wm, wn, frow, gq);
        }
        int kb = 0;
        if (KB & 1) {
            kblock_mx<0>(acc, a, bf, x, L, 1, 1 < KB, wm, wn, frow, gq);
            kb = 1;
        }
        for (; kb < KB; kb += 2) {
            kblock_mx<1>(acc, a, bf, x, L, kb + 1, kb + 1 < KB, wm, wn, frow, gq);
            kblock_mx<0>(acc, a, bf, x, L, kb + 2, kb + 2 < KB, wm, wn, frow, gq);
        }
    } else {

    // K block kb sits in stage (kb + KB + 1) % 2, so that the blocks after
    // an odd first one come in (stage 1, stage 0) pairs.  The first block is
    // loaded and read before the loop; each block then starts the DMA of the
    // next one (see kblock).
    v8i a, bf[TN];
    Scales<GLU> s;
    if (KB & 1) {
        load_stage<0>(L, 0);
        wait_dma_and_sync();
        read_head<0>(a, bf, s, wm, wn, frow, fc);
    } else {
        load_stage<1>(L, 0);
        wait_dma_and_sync();
        read_head<1>(a, bf, s, wm, wn, frow, fc);
    }

    float scale = 1.0f;   // of tile row tid's adapter, for tid < 256
    if constexpr (LORA) {
        any = tile_has_adapter(g, q, m0, lane);
        if (any && q.lora.scale) scale = q.lora.scale[max(id_of(g, q, m0, tid & (BM - 1)), 0)];
    }
    // nothing pending before the first block: its first three folds add 0 * 0
    v4f p[4];
#pragma unroll
    for (int q = 0; q < 4; q++) p[q] = (v4f){0.f, 0.f, 0.f, 0.f};
    TailScale<GLU> s_tail = {};

    int kb = 0;
    if (KB & 1) {
        kblock<0>(acc, p, s_tail, a, bf, s, L, L.P, 1, 1 < KB, wm, wn, frow, fc);
        kb = 1;
    }
    for (; kb < KB - (LORA ? 2 : 0); kb += 2) {
        kblock<1>(acc, p, s_tail, a, bf, s, L, L.P, kb + 1, kb + 1 < KB, wm, wn, frow, fc);
        kblock<0>(acc, p, s_tail, a, bf, s, L, L.P, kb + 2, kb + 2 < KB, wm, wn, frow, fc);
    }
    if constexpr (LORA) {
        if (tid < BM) sR[tid] = scale;
        if (kb < KB) {   // the last two blocks, the second without a successor
            kblock<1>(acc, p, s_tail, a, bf, s, L, L.P, kb + 1, true, wm, wn, frow, fc);
            if (any) lora_dma<1>(g, q, m0, 0, wave, lane);
            kblock<0, 0, false>(acc, p, s_tail, a, bf, s, L, L.P, 0, false, wm, wn, frow, fc);
        } else if (any) {   // K = 128: nothing to hide the load behind
            lora_dma<1>(g, q, m0, 0, wave, lane);
            wait_dma_and_sync();
        }
    }
#pragma unroll
    for (int j = 1; j < TN; j++) fold4(acc[TM - 1][j], p[(TM * TN - TN + j) & 3], s_tail.at(j));
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the last (empty) DMA is retired

    if constexpr (LORA) {
        if (any) lora_add(acc, g, q, m0, n0 + wn * WN, wm, wave, lane);
    }
    if constexpr (EPI != EPI_NONE) act_tile<EPI, 4>(acc, g, ep, m0, n0, wave, lane);
    if constexpr (GLU) store_gated_tile(acc, g, m0, n0, wave, lane);
    else store_tile<MODE>(acc, g, m0, n0, wave, lane);
}

// A plain tile's epilogue is split in two, so that neither end of a tile
// boundary waits idle.  Its row groups 0 .. TAIL_RG - 1 are stored at the end
// of the tile (in gemm_persistent, after the K loop), behind the next tile's
// first DMA and while it lands; the rest go out inside the next tile's first
// K block (kblock_first).  TAIL_RG = 4 measured 1-2 % faster than 0, 2, 6 or
// 8.
constexpr int TAIL_RG = 4;

// The lane's two store offsets in a row group of a plain tile, in elements
// (see store_tile), and its half.
struct PlainOffsets {
    uint32_t lx, ly;
    bool up;
};
template <bool GLU = false>
__device__ __forceinline__ PlainOffsets plain_offsets(int64_t N, int wm, int wn, int lane) {
    asm volatile("" : "+v"(lane));   // formed here, per tile, not hoisted
    PlainOffsets o;
    if constexpr (GLU) {   // one piece of the lane's row
        o.lx = o.ly = (uint32_t)((wm * WM + (lane & 15)) * N + wn * 32 + (lane >> 4) * 8);
        o.up = false;
        return o;
    }
    o.up = (lane >> 3) & 1;
    const int px = (lane >> 4) + (o.up ? 4 : 0);
    o.lx = (uint32_t)((wm * WM + (lane & 7)) * N + wn * WN + px * 8);
    o.ly = o.lx + (uint32_t)(8 * N + (o.up ? -32 : 32));
    return o;
}

// Row group i of a plain tile (i a constant once the caller's loop is
// unrolled), stored non-temporally through rC (a descriptor of C from the
// tile's first element on), or through the zero-size descriptor, which
// stores nothing but issues the same two instructions.
template <bool GLU = false>
__device__ __forceinline__ void plain_store_rg(const v4f (&acc)[TM][TN], int i, __amdgpu_buffer_rsrc_t rC,
                                               int64_t N, const PlainOffsets &o) {
    if constexpr (GLU) {
        __builtin_amdgcn_raw_buffer_store_b128(gated_piece(acc, i), rC, 2 * ((uint32_t)(i * 16 * N) + o.lx), 0, 2);
        return;
    }
    u32x4 x, y;
    tile_pieces(acc, i, o.up, x, y);
    const uint32_t ri = (uint32_t)(i * 16 * N);   // the row group's first element
    __builtin_amdgcn_raw_buffer_store_b128(x, rC, 2 * (ri + o.lx), 0, 2);   // 2: nt
    __builtin_amdgcn_raw_buffer_store_b128(y, rC, 2 * (ri + o.ly), 0, 2);
}

// The first K block of every tile in the persistent blockscale kernel.  It
// carries no products over from a previous block, and the first fold of each
// sub-tile, three MFMAs after its MFMA as in kblock, sets the accumulator to
// fma(p, s, +0), which is what folding into a zeroed accumulator gives; the
// last three sub-tiles, whose first fold is the next block's, are zeroed
// here.  So the accumulators may still hold the previous tile when the block
// starts: if that tile was a plain one (see tile_is_plain), the stores of
// its row group i >= TAIL_RG go out here, just before MFMA 4 i, the last
// reads of those accumulators, and drain while the new tile's MFMAs run.  rC
// is a descriptor of the previous tile's part of C from its first element
// on (row-major C: contiguous bands), or the zero-size one when there is
// nothing to store: the stores are always issued, so that every wave runs
// the same instructions and the vector memory count below is exact.  The
// DMA of block 1 goes out after MFMAs 0..8 as in kblock, before the stores of
// row groups 4..6, so at the barrier before row group 7 this wave's DMA has
// landed once at most those 6 stores are outstanding (vector memory
// operations retire in issue order).
template <int ST, bool GLU>
__device__ __forceinline__ void kblock_first(v4f (&acc)[TM][TN], v4f (&p)[4], TailScale<GLU> &s_tail, v8i &a,
                                             v8i (&bf)[TN], Scales<GLU> &s, const Loader &L,
                                             const Panels &P, int kload, bool vload, int wm, int wn,
                                             int frow, int fc, __amdgpu_buffer_rsrc_t rC,
                                             int64_t N, const PlainOffsets &o) {
    static_assert(TAIL_RG >= 3 && TAIL_RG <= 6, "the wait below counts the stores of row groups TAIL_RG..6");
    const uint8_t *as = stA<ST>();
    v8i an = a;
    v8i a_next = a;
    RawScales rn;
#pragma unroll
    for (int i = 0; i < TM; i++) {
        const v8i af = an;
        if (i + 1 < TM) an = lds_frag(as, wm * WM + (i + 1) * 16 + frow, fc);
        if (i == TM - 1) {
            // vmcnt: the stores of row groups TAIL_RG..6, two (GLU: one) to each, may remain
            __builtin_amdgcn_s_waitcnt(0x0F70 | ((GLU ? 1 : 2) * (7 - TAIL_RG)));
            barrier_lds_only();
            a_next = lds_frag(stA<ST ^ 1>(), wm * WM + frow, fc);
            read_block_scales<ST ^ 1, GLU>(rn, wm, wn, frow);
        }
#pragma unroll
        for (int j = 0; j < TN; j++) {
            const int k = i * TN + j;
            if (j == 0 && i >= TAIL_RG) plain_store_rg<GLU>(acc, i, rC, N, o);
            if (j == 0 && i == TM - 1) {
                // products 29..31 are first folded by the next block, which
                // adds them (fma into the accumulator): start those at zero
#pragma unroll
                for (int jj = 1; jj < TN; jj++) acc[i][jj] = (v4f){0.f, 0.f, 0.f, 0.f};
            }
            p[k & 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                bf[j], af, (v4f){0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
            if (k >= 3) {
                const int kp = k - 3;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    acc[kp / TN][kp % TN][e] = __builtin_fmaf(p[kp & 3][e], s.at(kp / TN, kp % TN), 0.0f);
            }
            if (i == TM - 1) {
                bf[j] = lds_frag(stB<ST ^ 1>(), wn * WN + j * 16 + frow, fc);
            }
            dma_block<ST>(L, P, k, kload, vload);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    s_tail.set(s);
    s.set(rn);
    a = a_next;
}

// ---- persistent kernels (K / 128 even; blockscale and mxfp8) ----
// One workgroup per CU walks the tiles of virtual workgroups b, b + G,
// b + 2G, ... (G = grid size, a multiple of 8, so every tile stays on the XCD
// the non-persistent mapping gives it).  The K blocks of successive tiles form
// one stream; block 0 of every tile sits in stage 1, its last block in stage
// 0.  The descriptors cover whole matrices, so the last K block of a tile
// DMAs the next tile's block 0 (its lanes' offsets moved by dn) as any block
// DMAs its successor, and reads its head.  (Switching descriptors inside the
// K loop instead made the compiler spill hundreds of VGPRs.)  Blockscale: a
// plain tile then stores half of its row groups at once and the other half
// inside the next tile's first K block (kblock_first), between its MFMAs.
// mxfp8: a plain tile stores all of them at once, and they drain under the
// next tile's first K block.  The last tile and tiles that are not plain
// store everything at once.
// The blockscale kernel runs one copy of this body per row half of the wave
// grid (WMC = wm, a compile-time constant: each wave executes straight-line
// code with its row offsets folded), and the second half issues its K
// blocks' DMA DMA_SHIFT MFMAs later than the first, so that the two waves of
// a SIMD do not stall on DMA issue at the same time (together ≈ 3 % faster,
// bit-identical; a shift of 8 was slower).  WMC = -1: one body, wm at run
// time (mxfp8).
constexpr int DMA_SHIFT = 4;

template <int MODE, int WMC, int EPI = EPI_NONE>
__device__ __forceinline__ void gemm_persistent(const GemmArgs &g) {
    constexpr bool GLU = EPI == EPI_GLU;
    constexpr int COLS = GLU ? BN / 2 : BN;
    constexpr int DSH = WMC == 1 ? DMA_SHIFT : 0;
    constexpr bool MX = MODE == MODE_MX;
    int vb = blockIdx.x;
    int64_t m0, n0;
    if (!tile_of<COLS>(g, vb, m0, n0)) return;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // wave-uniform: keep in SGPRs
    const int wm = WMC >= 0 ? WMC : wave >> 2;
    const int wn = wave & 3;
    const int KB = g.KB;   // even, at least 2
    const int frow = lane & 15;
    const int fc = lane >> 4;   // the lane group: K chunks fc and fc + 4

    Loader L;
    init_loader<MODE, GLU, true>(L, g, wave, lane);
    L.P = whole_panels<MODE, GLU>(g, wave);
    shift_loader(L, tile_off<MODE>(g, m0, n0, wave));

    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};

    // block 0 of every tile sits in stage 1 (K / 128 even)
    const int gq = lane >> 4;   // mxfp8: the lane's 32-wide K group
    v8i a, bf[TN];
    Scales<GLU> s;
    MxScales x;
    load_stage<1>(L, 0);
    wait_dma_and_sync();
    if constexpr (MX) read_head_mx<1>(a, bf, x, wm, wn, frow, gq);
    else read_head<1>(a, bf, s, wm, wn, frow, fc);

    v4f p[4];
#pragma unroll
    for (int q = 0; q < 4; q++) p[q] = (v4f){0.f, 0.f, 0.f, 0.f};
    TailScale<GLU> s_tail = {};

    // The kernel's only argument, read in place from the kernarg segment
    // where each tile needs it (scalar loads), rather than held in SGPRs
    // across the K loop.
    typedef const __attribute__((address_space(4))) GemmArgs *KArgs;
    const KArgs gp = (KArgs)__builtin_amdgcn_kernarg_segment_ptr();
    auto args = [gp]() {
        KArgs q = gp;
        asm volatile("" : "+s"(q));
        return *(const GemmArgs *)q;
    };
    // blockscale: whether the accumulators hold the previous tile, whose
    // stores then go out inside this tile's first K block (kblock_first), and
    // that tile's origin
    bool pend = false;
    int64_t pm0 = 0, pn0 = 0;
    // the tile after this one and the move of the loader's offsets from
    // this tile to it (zero if there is none); found at the tile boundary,
    // so that only three offsets stay live across the K loop
    int64_t m0n = 0, n0n = 0;
    bool has_next = false;
    TileOff dn = {0, 0, 0};
    auto find_next = [&]() {
        const GemmArgs gt = args();
        has_next = __builtin_amdgcn_readfirstlane((int)tile_of<COLS>(gt, vb + (int)gridDim.x, m0n, n0n));
        dn = TileOff{0, 0, 0};
        if (has_next) {
            const TileOff tn = tile_off<MODE>(gt, m0n, n0n, wave), tc = tile_off<MODE>(gt, m0, n0, wave);
            dn.a = __builtin_amdgcn_readfirstlane(tn.a - tc.a);
            dn.b = __builtin_amdgcn_readfirstlane(tn.b - tc.b);
            dn.s = __builtin_amdgcn_readfirstlane(tn.s - tc.s);
        }
    };
    find_next();
    for (;;) {
        if constexpr (MX) {
            const TileOff d0 = {0, 0, 0};
            for (int kb = 0; kb < KB; kb += 2) {
                kblock_mx<1>(acc, a, bf, x, L, kb + 1, true, wm, wn, frow, gq);
                kblock_mx<0>(acc, a, bf, x, L, kb + 2 < KB ? kb + 2 : 0, kb + 2 < KB || has_next, wm, wn,
                             frow, gq, kb + 2 < KB ? d0 : dn);
            }
            shift_loader(L, dn);
        } else {
            {
                const GemmArgs gt = args();
                const PlainOffsets o = plain_offsets<GLU>(gt.N, wm, wn, lane);
                const __amdgpu_buffer_rsrc_t rC =
                    pend ? make_rsrc(gt.C + pm0 * gt.N + pn0, (gt.M - pm0) * gt.N * 2) : L.rZ;
                kblock_first<1>(acc, p, s_tail, a, bf, s, L, L.P, 1, true, wm, wn, frow, fc, rC,
                                gt.N, o);
            }
            // The last block (always in stage 0) DMAs the next tile's block
            // 0 into stage 1, as any block DMAs its successor, and its head
            // reads fetch that block's first fragments and scales.
            const TileOff d0 = {0, 0, 0};
            kblock<0, DSH>(acc, p, s_tail, a, bf, s, L, L.P, 2 < KB ? 2 : 0, 2 < KB || has_next, wm, wn,
                           frow, fc, 2 < KB ? d0 : dn);
            for (int kb = 2; kb < KB; kb += 2) {
                kblock<1, DSH>(acc, p, s_tail, a, bf, s, L, L.P, kb + 1, true, wm, wn, frow, fc);
                kblock<0, DSH>(acc, p, s_tail, a, bf, s, L, L.P, kb + 2 < KB ? kb + 2 : 0,
                               kb + 2 < KB || has_next, wm, wn, frow, fc, kb + 2 < KB ? d0 : dn);
            }
            shift_loader(L, dn);
        }
        if constexpr (!MX) {
            // the last three products of the tile (kblock_first carries none)
#pragma unroll
            for (int j = 1; j < TN; j++) fold4(acc[TM - 1][j], p[(TM * TN - TN + j) & 3], s_tail.at(j));
        }

        if constexpr (MX) {
            // The last tile and tiles that are not plain store here; a plain
            // one stores its 2 * TM pieces per lane (other tiles issue the
            // same instructions through the zero-size descriptor, so that
            // every path issues the same vector memory operations), and they
            // drain under the next tile's first K block, whose block 0 and
            // head are already in.
            const bool plain = tile_is_plain(args(), m0, n0);
            if (!has_next || !plain) store_tile<MODE, false>(acc, args(), m0, n0, wave, lane);
            if (!has_next) break;
            {
                const GemmArgs gt = args();
                const PlainOffsets o = plain_offsets(gt.N, wm, wn, lane);
                const __amdgpu_buffer_rsrc_t rT =
                    plain ? make_rsrc(gt.C + m0 * gt.N + n0, (gt.M - m0) * gt.N * 2) : L.rZ;
#pragma unroll
                for (int i = 0; i < TM; i++) plain_store_rg(acc, i, rT, gt.N, o);
            }
#pragma unroll
            for (int i = 0; i < TM; i++)
#pragma unroll
                for (int j = 0; j < TN; j++) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
        } else {
            // The last tile and tiles that are not plain store here.  A
            // plain tile stores its row groups 0 .. TAIL_RG - 1 here and the
            // rest inside the next tile's first K block.  Every path issues
            // those 2 * TAIL_RG stores (other tiles through the zero-size
            // descriptor), so that the vector memory count of the next
            // tile's first block is exact.  The next tile's block 0 and its
            // head are already in (the last K block loaded them).
            if constexpr (EPI != EPI_NONE) {
                typedef const __attribute__((address_space(4))) ActGemmArgs *ActKArgs;
                ActKArgs ka = (ActKArgs)gp;
                asm volatile("" : "+s"(ka));
                const ActGemmArgs at = *(const ActGemmArgs *)ka;
                act_tile<EPI, 2>(acc, at.g, at.q, m0, n0, wave, lane);
            }
            const bool plain = tile_is_plain<COLS>(args(), m0, n0);
            if (!has_next || !plain) {
                if constexpr (GLU) store_gated_tile(acc, args(), m0, n0, wave, lane);
                else store_tile<MODE, false>(acc, args(), m0, n0, wave, lane);
            }
            if (!has_next) break;
            {
                const GemmArgs gt = args();
                const PlainOffsets o = plain_offsets<GLU>(gt.N, wm, wn, lane);
                const __amdgpu_buffer_rsrc_t rT =
                    plain ? make_rsrc(gt.C + m0 * gt.N + n0, (gt.M - m0) * gt.N * 2) : L.rZ;
#pragma unroll
                for (int i = 0; i < TAIL_RG; i++) plain_store_rg<GLU>(acc, i, rT, gt.N, o);
            }
            pend = plain;
            pm0 = m0;
            pn0 = n0;
        }
        vb += (int)gridDim.x;
        m0 = m0n;
        n0 = n0n;
        find_next();
    }
}

__global__ void __launch_bounds__(NTHREADS) bsgemm_persistent_kernel(GemmArgs g) {
    // wm = wave / 4 = threadIdx.x / 256, the same for every lane of a wave
    if (__builtin_amdgcn_readfirstlane(threadIdx.x >> 8)) gemm_persistent<MODE_BS, 1>(g);
    else gemm_persistent<MODE_BS, 0>(g);
}
__global__ void __launch_bounds__(NTHREADS) bsgemm_act_persistent_kernel(ActGemmArgs a) {
    if (__builtin_amdgcn_readfirstlane(threadIdx.x >> 8)) gemm_persistent<MODE_BS, 1, EPI_GLU>(a.g);
    else gemm_persistent<MODE_BS, 0, EPI_GLU>(a.g);
}
__global__ void __launch_bounds__(NTHREADS) mxgemm_persistent_kernel(GemmArgs g) {
    gemm_persistent<MODE_MX, -1>(g);
}

__global__ void __launch_bounds__(NTHREADS) bsgemm_tile_kernel(GemmArgs g) { gemm_tile<MODE_BS>(g); }

__global__ void __launch_bounds__(NTHREADS) bsgemm_lora_tile_kernel(GemmArgs g, LoraGemmArgs q) {
    gemm_tile<MODE_BS, true>(g, q);
}

template <int EPI>
__global__ void __launch_bounds__(NTHREADS) bsgemm_act_tile_kernel(ActGemmArgs a) {
    gemm_tile<MODE_BS, false, EPI>(a.g, {}, a.q);
}

__global__ void __launch_bounds__(NTHREADS) bsgemm_pb_tile_kernel(GemmArgs g) { gemm_tile<MODE_PB>(g); }

__global__ void __launch_bounds__(NTHREADS) mxgemm_tile_kernel(GemmArgs g) { gemm_tile<MODE_MX>(g); }

// Workgroup -> tile of rows x cols.  Workgroups are dealt to the XCDs in turn, and a
// column's row tiles follow each other on one XCD, whose L2 serves B to all but the
// first.  Where the columns divide by the XCDs they are dealt in turn, which reads
// the weight evenly (N = 7168: M = 1 7.1 us, M = 64 14.2, against 7.7 and 15.1 by
// runs); otherwise each XCD gets a contiguous run of tiles, so that none idles
// (N = 384, K = 256, M = 5733: 9.6 us against 16.0).  False for the workgroups past
// the last tile.
__device__ __forceinline__ bool column_tile(const GemmArgs &g, int rows, int cols, int64_t &m0, int64_t &n0) {
    const int tm = (int)((g.M + rows - 1) / rows), tn = (int)(g.N / cols);
    const int xcd = (int)(blockIdx.x % NUM_XCD), turn = (int)(blockIdx.x / NUM_XCD);
    const bool even = tn % NUM_XCD == 0;
    const int t = even ? turn : xcd * (int)(gridDim.x / NUM_XCD) + turn;
    m0 = (int64_t)(t % tm) * rows;
    n0 = (int64_t)(even ? t / tm * NUM_XCD + xcd : t / tm) * cols;
    return n0 < g.N;
}

// ---- few rows, with adapters -------------------------------------------------
// The 256-row tile leaves a short batch on N / 256 of the CUs, waiting for B.
// Here a wave takes 16 RG rows x 16 CG columns by itself, straight from global
// memory to registers, D K blocks ahead, one wave to a workgroup (two or four
// side by side took 1.3 to 2.5 times as long: they wait on one CU).  Each K block is
// the same MFMA on the same fragments, folded in the same order, so the sums are
// those of the other kernels bit for bit.  The 16-column sub-tiles take B's rows in
// the order of lora_col, two sub-tiles to a 16-byte piece of C.

template <int RG, int CG>
struct ShortBlock {
    v8i a[RG], b[CG];
    float sa[RG], sb;
};

__device__ __forceinline__ v8i frag_of(__amdgpu_buffer_rsrc_t r, int off, int k) {
    const u32x4 lo = __builtin_amdgcn_raw_buffer_load_b128(r, off, k, 0);
    const u32x4 hi = __builtin_amdgcn_raw_buffer_load_b128(r, off + 64, k, 0);
    return (v8i){(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// The adapters of a wave's 16 RG rows from m0 on (rows_in of them inside M) and 16 CG
// columns from n on, added to its finished accumulators: four adapters at a time, so
// that a batch of single tokens does not wait for each one's B in turn; H of the
// wave's rows is loaded and split once per 32 ranks.
template <int RG, int CG>
__device__ __forceinline__ void wave_adapters(v4f (&acc)[RG][CG], const GemmArgs &g, const LoraGemmArgs &q, int64_t m0,
                                              int64_t n, int rows_in, int lane) {
    const int frow = lane & 15, fg = lane >> 4;
    const int R = q.lora.R;
    int id = -1;
    if (lane < rows_in) id = q.ids[m0 + lane];
    if ((uint32_t)id >= (uint32_t)q.lora.L) id = -1;
    const uint64_t all = __ballot(id >= 0);
    if (all) {
        float s[RG];
        int idr[RG];
#pragma unroll
        for (int i = 0; i < RG; i++) {
            idr[i] = __shfl(id, 16 * i + frow, 64);
            s[i] = q.lora.scale ? q.lora.scale[max(idr[i], 0)] : 1.0f;
        }
        for (int r0 = 0; r0 < R; r0 += 32) {
            const int r = r0 + 8 * fg;
            v8bf hi[RG], lo[RG];
#pragma unroll
            for (int i = 0; i < RG; i++)
                lora_split(lora_load_h(q.lora, m0 + 16 * i + frow, idr[i] >= 0, r), s[i], hi[i], lo[i]);
            uint64_t todo = all;
            while (todo) {
                int a[4];
                v8bf b[4][CG];
#pragma unroll
                for (int t = 0; t < 4; t++) {
                    a[t] = -2;   // no row's
                    if (!todo) continue;
                    a[t] = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)todo) - 1);
                    todo &= ~__ballot(id == a[t]);
                    const __amdgpu_buffer_rsrc_t rL = lora_rsrc(q.lora, a[t], n, g.N);
#pragma unroll
                    for (int j = 0; j < CG; j++) b[t][j] = lora_load_b(rL, lora_col(j, frow), r, R);
                }
#pragma unroll
                for (int t = 0; t < 4; t++) {
                    if (a[t] < 0) continue;
#pragma unroll
                    for (int i = 0; i < RG; i++) {
                        // a lane's sums are those of row frow: other adapters' rows keep theirs
                        const bool live = idr[i] == a[t];
#pragma unroll
                        for (int j = 0; j < CG; j++) {
                            v4f x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[t][j], hi[i], acc[i][j], 0, 0, 0);
                            x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[t][j], lo[i], x, 0, 0, 0);
#pragma unroll
                            for (int e = 0; e < 4; e++) acc[i][j][e] = live ? x[e] : acc[i][j][e];
                        }
                    }
                }
            }
        }
    }
}

template <int RG, int CG>
__device__ __forceinline__ void wave_store(const v4f (&acc)[RG][CG], const GemmArgs &g, int64_t m0, int64_t n,
                                           int rows_in, int lane) {
    const int frow = lane & 15, fg = lane >> 4;
#pragma unroll
    for (int i = 0; i < RG; i++) {
        if (16 * i + frow >= rows_in) continue;
        const uint32_t m = (uint32_t)(m0 + 16 * i + frow), br = (uint32_t)g.band_rows, d = m / br;
        uint16_t *row = g.C + (int64_t)d * g.band_stride + (int64_t)(m - d * br) * g.N + n + 8 * fg;
#pragma unroll
        for (int j = 0; j < CG; j += 2) {
            const u32x4 o = {pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3]),
                             pack_bf16x2(acc[i][j + 1][0], acc[i][j + 1][1]),
                             pack_bf16x2(acc[i][j + 1][2], acc[i][j + 1][3])};
            *(u32x4 *)(row + 16 * j) = o;
        }
    }
}

template <int RG, int CG, int D>
__global__ void __launch_bounds__(64) bsgemm_lora_short_kernel(GemmArgs g, LoraGemmArgs q) {
    const int lane = threadIdx.x;
    const int frow = lane & 15, fg = lane >> 4;
    int64_t m0, n;
    if (!column_tile(g, 16 * RG, 16 * CG, m0, n)) return;
    const int rows_in = (int)(g.M - m0 < 16 * RG ? g.M - m0 : 16 * RG);
    const int K = (int)g.K, KB = g.KB;
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.A + m0 * K, (int64_t)rows_in * K);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.B + n * K, (int64_t)(16 * CG) * K);
    const __amdgpu_buffer_rsrc_t rS = make_rsrc((const float *)g.sa + m0 * KB, (int64_t)rows_in * KB * 4);
    const float *sb = (const float *)g.sb + n / 128 * KB;
    const int offA = frow * K + 16 * fg;
    int offB[CG];
#pragma unroll
    for (int j = 0; j < CG; j++) offB[j] = lora_col(j, frow) * K + 16 * fg;

    // a block past the last one loads that again, and is not used
    auto load = [&](ShortBlock<RG, CG> &x, int kb) {
        kb = min(kb, KB - 1);
#pragma unroll
        for (int j = 0; j < CG; j++) x.b[j] = frag_of(rB, offB[j], kb * 128);
#pragma unroll
        for (int i = 0; i < RG; i++) x.a[i] = frag_of(rA, offA + i * 16 * K, kb * 128);
#pragma unroll
        for (int i = 0; i < RG; i++)
            x.sa[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rS, (16 * i + frow) * KB * 4, kb * 4, 0));
        x.sb = sb[kb];
    };
    v4f acc[RG][CG];
#pragma unroll
    for (int i = 0; i < RG; i++)
#pragma unroll
        for (int j = 0; j < CG; j++) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    ShortBlock<RG, CG> x[D];
#pragma unroll
    for (int d = 0; d < D; d++) load(x[d], d);
    for (int kb = 0; kb < KB; kb += D) {
#pragma unroll
        for (int d = 0; d < D; d++) {
            if (kb + d >= KB) break;
            v4f p[RG][CG];
#pragma unroll
            for (int i = 0; i < RG; i++)
#pragma unroll
                for (int j = 0; j < CG; j++)
                    p[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        x[d].b[j], x[d].a[i], (v4f){0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < RG; i++) {
                const float s = x[d].sa[i] * x[d].sb;
#pragma unroll
                for (int j = 0; j < CG; j++) fold4(acc[i][j], p[i][j], s);
            }
            load(x[d], kb + d + D);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    wave_adapters<RG, CG>(acc, g, q, m0, n, rows_in, lane);
    wave_store<RG, CG>(acc, g, m0, n, rows_in, lane);
}

// ---- middling batches, with adapters -----------------------------------------
// 64 rows x 128 columns to a workgroup of 8 waves (2 x 4, 32 x 32 each), A, B and
// the row scales staged by DMA three K blocks deep: too few tiles of 256 rows to
// fill the CUs, too many rows for every wave to load its own fragments.  A stage is
// one LDS object (so that the compiler can tell the DMA into one from the reads of
// another): 8 KiB of A and 16 KiB of B in the slots of lds_slot, then each wave's
// copy of the 64 rows' scales.  Three stages let two workgroups share a CU; four
// took as long for one workgroup to a CU and 28 against 22 us for two.
//
// At K block kb a wave waits until its own DMA of kb has landed (that of the next
// block may be in flight), meets the others, whose reads of block kb - 1 are then
// done too, sends block kb + 2 to the stage kb - 1 was in, and multiplies.  Blocks
// past the last load that one again, so that the count is the same throughout.
// Same MFMAs, folds and order as the other kernels: the sums are theirs bit for bit.
constexpr int MID_BM = 64, MID_BN = 128, MID_STAGES = 3, MID_DMA = 4;   // MID_DMA: a wave's DMA per block
constexpr int MID_STAGE = (MID_BM + MID_BN) * BK + 8 * 256;
__shared__ __attribute__((aligned(1024))) uint8_t sM0[MID_STAGE];
__shared__ __attribute__((aligned(1024))) uint8_t sM1[MID_STAGE];
__shared__ __attribute__((aligned(1024))) uint8_t sM2[MID_STAGE];
template <int ST> __device__ __forceinline__ uint8_t *stM() {
    return ST == 0 ? sM0 : ST == 1 ? sM1 : sM2;
}

struct MidLoader {
    __amdgpu_buffer_rsrc_t rA, rB, rS;
    int offA, offB[2], offS, wave;
};

// The row in LDS slot s (lds_slot inverted).
__device__ __forceinline__ int slot_row(int s) { return (s & ~15) | ((s & 15) >> 1) | ((s & 1) << 3); }

template <int ST>
__device__ __forceinline__ void mid_load(const MidLoader &L, int kb) {
    uint8_t *st = stM<ST>();
    __builtin_amdgcn_raw_ptr_buffer_load_lds(L.rA, (lds_void *)(st + L.wave * 1024), 16, L.offA, kb * BK, 0, 0);
#pragma unroll
    for (int i = 0; i < 2; i++)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(L.rB, (lds_void *)(st + MID_BM * BK + (2 * L.wave + i) * 1024), 16,
                                                 L.offB[i], kb * BK, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(L.rS, (lds_void *)(st + (MID_BM + MID_BN) * BK + L.wave * 256), 4, L.offS,
                                             kb * 4, 0, 0);
}

// b_scale of the K blocks from `first` on, one to a lane (of gate and up columns).
// Loaded at each block they come between the blocks' DMA, and waiting for them is
// waiting for all DMA on its way (0.65 us a block); so they are loaded for MID_RUN blocks
// at a time.
constexpr int MID_RUN = 63;   // a multiple of the stages, at most a wave's lanes
struct MidScales {
    int first;
    float s[2];
    __device__ __forceinline__ float at(int h, int kb) const {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, s[h]), kb - first));
    }
};

template <int ST, bool GLU>
__device__ __forceinline__ void mid_block(v4f (&acc)[2][2], const MidLoader &L, int kb, int KB, const MidScales &sb,
                                          int lane) {
    const int frow = lane & 15, fg = lane >> 4, wm = L.wave >> 2, wn = L.wave & 3;
    __builtin_amdgcn_s_waitcnt(0x0F70 | (MID_DMA * (MID_STAGES - 2)));   // vmcnt: block kb is in
    barrier_lds_only();
    mid_load<(ST + MID_STAGES - 1) % MID_STAGES>(L, min(kb + MID_STAGES - 1, KB - 1));
    const uint8_t *st = stM<ST>();
    const float *sc = (const float *)(st + (MID_BM + MID_BN) * BK + L.wave * 256);
    const float sbk = sb.at(0, kb), sbk1 = GLU ? sb.at(1, kb) : 0.f;
    v8i a[2], b[2];
    float s[2][2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        a[i] = lds_frag(st, wm * 32 + i * 16 + frow, fg);
        b[i] = lds_frag(st + MID_BM * BK, wn * 32 + i * 16 + frow, fg);
        const float sa = sc[wm * 32 + i * 16 + frow];
        s[i][0] = sa * sbk;
        s[i][1] = GLU ? sa * sbk1 : s[i][0];
    }
    v4f p[2][2];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++)
            p[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j], a[i], (v4f){0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0,
                                                                       0, 0);
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) fold4(acc[i][j], p[i][j], s[i][j]);
}

// The sums of one tile of 64 rows and 128 rows of B (GLU: 64 gate and the same 64 up
// columns, 16 and 16 to a wave in its two sub-tiles).
template <bool GLU>
__device__ __forceinline__ void mid_sums(v4f (&acc)[2][2], const GemmArgs &g, int64_t m0, int64_t n0, int rows_in,
                                         int wave, int lane) {
    const int K = (int)g.K, KB = g.KB;
    MidLoader L;
    L.wave = wave;
    L.rA = make_rsrc(g.A + m0 * K, (int64_t)rows_in * K);
    if (GLU) L.rB = make_rsrc(g.B + (n0 + (wave & 1) * g.N) * K, (int64_t)(MID_BN / 2) * K);
    else L.rB = make_rsrc(g.B + n0 * K, (int64_t)MID_BN * K);
    L.rS = make_rsrc((const float *)g.sa + m0 * KB, (int64_t)rows_in * KB * 4);
    const int ra = slot_row(8 * wave + (lane >> 3));
    L.offA = ra * K + ((lane & 7) ^ (ra & 7)) * 16;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        // LDS row r holds B row lora_col of its sub-tile, within the wave's 32 columns
        // (GLU: row r % 16 of the wave's 16, from the gate or the up rows)
        const int r = slot_row(8 * (2 * wave + i) + (lane >> 3));
        const int row = GLU ? (r >> 5) * 16 + (r & 15) : (r & ~31) + lora_col((r >> 4) & 1, r & 15);
        L.offB[i] = row * K + ((lane & 7) ^ (r & 7)) * 16;
    }
    L.offS = lane * KB * 4;
    const float *sb = (const float *)g.sb + n0 / 128 * KB, *sb1 = sb + (int64_t)g.NB * KB;
    MidScales b = {};
    const auto scales = [&](int kb) {
        const int k = min(kb + lane, KB - 1);
        b.first = kb;
        b.s[0] = sb[k];
        if (GLU) b.s[1] = sb1[k];
    };
    scales(0);
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    mid_load<0>(L, 0);
    mid_load<1>(L, min(1, KB - 1));
    for (int kb = 0;;) {
        const int end = min(kb + MID_RUN, KB);
        for (; kb < end; kb += MID_STAGES) {
            mid_block<0, GLU>(acc, L, kb, KB, b, lane);
            if (kb + 1 < KB) mid_block<1, GLU>(acc, L, kb + 1, KB, b, lane);
            if (kb + 2 < KB) mid_block<2, GLU>(acc, L, kb + 2, KB, b, lane);
        }
        if (kb >= KB) break;
        scales(kb);
        __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0), so that the loop need not wait for them
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): the DMA past the last block is retired
}

__global__ void __launch_bounds__(NTHREADS) bsgemm_lora_mid_kernel(GemmArgs g, LoraGemmArgs q) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t m0, n0;
    if (!column_tile(g, MID_BM, MID_BN, m0, n0)) return;
    const int rows_in = (int)(g.M - m0 < MID_BM ? g.M - m0 : MID_BM);
    v4f acc[2][2];
    mid_sums<false>(acc, g, m0, n0, rows_in, wave, lane);
    const int64_t mw = m0 + 32 * (wave >> 2), nw = n0 + 32 * (wave & 3);
    const int rw = rows_in - 32 * (wave >> 2);
    if (rw <= 0) return;
    wave_adapters<2, 2>(acc, g, q, mw, nw, rw < 32 ? rw : 32, lane);
    wave_store<2, 2>(acc, g, mw, nw, rw < 32 ? rw : 32, lane);
}

// Element of C of row m, column n.
__device__ __forceinline__ int64_t element_at(const GemmArgs &g, uint32_t m, int64_t n) {
    const uint32_t br = (uint32_t)g.band_rows, d = m / br;
    return (int64_t)d * g.band_stride + (int64_t)(m - d * br) * g.N + n;
}

template <bool GLU>
__global__ void __launch_bounds__(NTHREADS) bsgemm_act_mid_kernel(ActGemmArgs a) {
    const GemmArgs &g = a.g;
    const ActArgs &q = a.q;
    const int lane = threadIdx.x & 63, frow = lane & 15, fg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t m0, n0;
    if (!column_tile(g, MID_BM, GLU ? MID_BN / 2 : MID_BN, m0, n0)) return;
    const int rows_in = (int)(g.M - m0 < MID_BM ? g.M - m0 : MID_BM);
    v4f acc[2][2];
    mid_sums<GLU>(acc, g, m0, n0, rows_in, wave, lane);
    // a lane's columns: 8 of the wave's 32 (GLU: 4 of its 16, gate and up)
    const int64_t n = n0 + (GLU ? 16 * (wave & 3) + 4 * fg : 32 * (wave & 3) + 8 * fg);
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    u32x4 bias = {0u, 0u, 0u, 0u};
    if constexpr (GLU) {
        if (q.bias) {
            const u32x2 b0 = *(const u32x2 *)(q.bias + n), b1 = *(const u32x2 *)(q.bias + g.N + n);
            bias = (u32x4){b0[0], b0[1], b1[0], b1[1]};
        }
    } else {
        bias = load_bias8(q, n);
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int row = 32 * (wave >> 2) + 16 * i + frow;
        if (row >= rows_in) continue;
        const int64_t at = element_at(g, (uint32_t)(m0 + row), n);
        float t[8];
#pragma unroll
        for (int e = 0; e < 8; e++) t[e] = acc[i][e >> 2][e & 3];
        add8(t, bias);
        if constexpr (GLU) {
            float v[4] = {t[0], t[1], t[2], t[3]};
            act_all(v, q.act);
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] *= t[4 + e];
            u32x2 r = {0u, 0u};
            if (q.resid) r = *(const u32x2 *)(q.resid + at);
            join(v, r, q);
            *(u32x2 *)(g.C + at) = (u32x2){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        } else {
            act_all(t, q.act);
            u32x4 r = {0u, 0u, 0u, 0u};
            if (q.resid) r = *(const u32x4 *)(q.resid + at);
            join(t, r, q);
            *(u32x4 *)(g.C + at) = pack8(t);
        }
    }
}

// ---- few rows, with bias, activation and residual ------------------------------
// 16 RG rows by 16 CT rows of B to a workgroup (GLU: of each 16, 8 gate rows and the up
// rows of the same columns).  Its eight waves take the K blocks in turn, so that
// all of a turn's loads are on their way together, where one wave for all of K waits for
// a few blocks at a time.  The block products go to LDS, one of every wave's,
// and are folded in ascending order of K by a lane for each four elements, so the sums
// are those of the other kernels bit for bit.
//
// A weight's read bounds it.  M = 1, gated, N = 2048, K = 7168: 29 MB in 7.8 us, of which an
// empty launch takes 3; M = 64,
// N = 7168, K = 2048: 9.6 us, 16.7 MB.  The next turn's loads are on their way while one is
// multiplied and folded; loads past the last turn, unused, cost what used ones do.
template <int RG, int CT, bool GLU>
__global__ void __launch_bounds__(NTHREADS) bsgemm_act_rows_kernel(ActGemmArgs a) {
    constexpr int W = 8, COLS = (GLU ? 8 : 16) * CT, UNITS = RG * CT * 64, PER = (UNITS + NTHREADS - 1) / NTHREADS;
    constexpr int SB = GLU ? 2 : 1, SAS = (W * RG * 16 + NTHREADS - 1) / NTHREADS;
    __shared__ v4f prod[2][W][CT][RG][64];
    __shared__ float scale[2][W][SB][RG * 16];
    const GemmArgs &g = a.g;
    const ActArgs &q = a.q;
    const int tid = threadIdx.x, lane = tid & 63, frow = lane & 15, fg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * COLS, m0 = (int64_t)blockIdx.y * (16 * RG), K = g.K;
    const int rows_in = (int)(g.M - m0 < 16 * RG ? g.M - m0 : 16 * RG);
    const int KB = g.KB, turns = (KB + W - 1) / W;
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.A + m0 * K, rows_in * K);
    const __amdgpu_buffer_rsrc_t rS = make_rsrc((const float *)g.sa + m0 * KB, (int64_t)rows_in * KB * 4);
    const uint8_t *B[CT];
#pragma unroll
    for (int j = 0; j < CT; j++)
        B[j] = g.B + (GLU ? n0 + 8 * j + (frow & 7) + (frow >> 3) * g.N : n0 + 16 * j + frow) * K + 16 * fg;
    const float *sb = (const float *)g.sb + n0 / 128 * KB, *sb1 = sb + (int64_t)g.NB * KB;

    v8i x[RG], b[CT];
    float s[SAS], sbv[SAS][SB];
    // nothing past the last block: a load costs the CU's 16 cycles even if it is not used
    const auto load = [&](int t) {
        const int kb = t * W + wave;
        if (t >= turns) return;
#pragma unroll
        for (int e = 0; e < SAS; e++) {   // the scales of one row and block of the turn
            const int id = tid + e * NTHREADS, r = id / W, k = min(t * W + id % W, KB - 1);
            s[e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rS, (r * KB + k) * 4, 0, 0));
            sbv[e][0] = sb[k];
            if (GLU) sbv[e][SB - 1] = sb1[k];
        }
        if (kb >= KB) return;
#pragma unroll
        for (int j = 0; j < CT; j++) {
            const u32x4 lo = *(const u32x4 *)(B[j] + (int64_t)kb * 128), hi = *(const u32x4 *)(B[j] + (int64_t)kb * 128 + 64);
            b[j] = (v8i){(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
        }
#pragma unroll
        for (int i = 0; i < RG; i++) x[i] = frag_of(rA, (16 * i + frow) * (int)K + 16 * fg, kb * 128);
    };
    v4f acc[PER];
#pragma unroll
    for (int p = 0; p < PER; p++) acc[p] = (v4f){0.f, 0.f, 0.f, 0.f};
    load(0);
    for (int t = 0; t < turns; t++) {
        const int buf = t & 1;
#pragma unroll
        for (int j = 0; j < CT; j++)
#pragma unroll
            for (int i = 0; i < RG; i++)
                prod[buf][wave][j][i][lane] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    b[j], x[i], (v4f){0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < SAS; e++) {
            const int id = tid + e * NTHREADS;
            if (id < W * RG * 16) {
#pragma unroll
                for (int h = 0; h < SB; h++) scale[buf][id % W][h][id / W] = s[e] * sbv[e][h];
            }
        }
        load(t + 1);
        __builtin_amdgcn_sched_barrier(0);
        barrier_lds_only();   // and turn t - 1 is folded: its buffer is free for t + 1
        const int blocks = min(KB - t * W, W);
#pragma unroll
        for (int p = 0; p < PER; p++) {
            const int id = tid + p * NTHREADS;
            if (id >= UNITS) break;
            const int i = (id >> 6) % RG, j = id / (64 * RG);
            const int h = GLU ? fg >> 1 : 0;
            if (blocks == W) {
#pragma unroll
                for (int k = 0; k < W; k++)
                    fold4(acc[p], prod[buf][k][j][i][lane], scale[buf][k][h][16 * i + frow]);
            } else {
                for (int k = 0; k < blocks; k++)
                    fold4(acc[p], prod[buf][k][j][i][lane], scale[buf][k][h][16 * i + frow]);
            }
        }
    }
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int p = 0; p < PER; p++) {
        const int id = tid + p * NTHREADS;
        if (id >= UNITS) break;   // whole waves
        const int i = (id >> 6) % RG, j = id / (64 * RG), row = 16 * i + frow;
        float v[4] = {acc[p][0], acc[p][1], acc[p][2], acc[p][3]}, u[4];
        const int64_t n = n0 + (GLU ? 8 * j : 16 * j) + 4 * (GLU ? fg & 1 : fg);
        if (q.bias) {
            const u32x2 bv = *(const u32x2 *)(q.bias + n + (GLU && fg >= 2 ? g.N : 0));
            v[0] += bf16_lo(bv[0]); v[1] += bf16_hi(bv[0]);
            v[2] += bf16_lo(bv[1]); v[3] += bf16_hi(bv[1]);
        }
        if constexpr (GLU) {   // the up values of a lane's columns are 32 lanes on
#pragma unroll
            for (int e = 0; e < 4; e++) u[e] = __shfl_down(v[e], 32, 64);
            if (fg >= 2) continue;
        }
        if (row >= rows_in) continue;
        act_all(v, q.act);
        const int64_t at = element_at(g, (uint32_t)(m0 + row), n);
        u32x2 r = {0u, 0u};
        if (q.resid) r = *(const u32x2 *)(q.resid + at);
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (GLU) v[e] *= u[e];
        join(v, r, q);
        *(u32x2 *)(g.C + at) = (u32x2){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
}

// B [N, K] -> the prepacked layout [N/16][K/128][2][64][16 B]: unit u of the
// output (16 bytes) is half h, lane l = 16 g + r of 16-row group nt and K
// block kb, and holds bytes [16 g + 64 h, +16) of row brow_of(16 nt + r)'s K
// block kb (the two halves of lane l are the chunks lds_frag gives it; the
// rows are those the LDS-staged kernel places in the same fragment slot).
// One lane per output unit: the writes are contiguous, the reads 16-byte
// aligned gathers.
__global__ void __launch_bounds__(256)
bprepack_kernel(const u32x4 *__restrict__ B, u32x4 *__restrict__ Bp, int64_t units, int64_t K) {
    const int64_t KB = K / 128;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units;
         u += (int64_t)gridDim.x * 256) {
        const int l = (int)(u & 63);
        const int h = (int)((u >> 6) & 1);
        const int64_t blk = u >> 7;          // nt * KB + kb
        const int64_t nt = blk / KB, kb = blk - nt * KB;
        const int64_t row = (nt & ~(int64_t)3) * 16 + brow_of((int)((nt & 3) * 16 + (l & 15)));
        const int64_t col = kb * 128 + 16 * (l >> 4) + 64 * h;
        Bp[u] = B[(row * K + col) >> 4];
    }
}

}  // namespace

static GemmArgs gemm_args(const uint8_t *A, const void *sa, const uint8_t *B, const void *sb,
                          uint16_t *C, int64_t M, int64_t N, int64_t K, int64_t band_rows,
                          int64_t band_stride) {
    GemmArgs g;
    g.A = A; g.sa = sa; g.B = B; g.sb = sb; g.C = C;
    g.M = M; g.N = N; g.K = K;
    g.band_rows = band_rows; g.band_stride = band_stride;
    g.KB = (int)(K / 128);
    g.NB = (int)(N / 128);
    g.tiles_m = (int)((M + BM - 1) / BM);
    g.tiles_n = (int)((N + BN - 1) / BN);
    return g;
}

static int gemm_grid(const GemmArgs &g) {
    const int T = g.tiles_m * g.tiles_n;
    return ((T + NUM_XCD - 1) / NUM_XCD) * NUM_XCD;
}

// CUs of the device a stream belongs to, asked once per device and kept
// (an atomic per device: concurrent first calls store the same value).
static std::atomic<int> g_cus[64];

int bs_stream_cus(hipStream_t stream) {
    hipDevice_t dev = 0;
    if (hipStreamGetDevice(stream, &dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int cus = g_cus[dev].load(std::memory_order_relaxed);
    if (cus == 0) {
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            cus < NUM_XCD)
            cus = 256;
        g_cus[dev].store(cus, std::memory_order_relaxed);
    }
    return cus;
}

// The persistent kernels' grid: one workgroup per CU of the stream's device,
// a multiple of 8 so that the XCD of each tile is the one the non-persistent
// launch gives it.
static int persistent_grid(const GemmArgs &g, hipStream_t stream) {
    const int grid = gemm_grid(g), per = bs_stream_cus(stream) / NUM_XCD * NUM_XCD;
    return grid < per ? grid : per;
}

// Whether the persistent kernels take a product: they address each operand through one
// descriptor with 31-bit lane offsets, the rows of a ragged last tile included, and a whole
// tile's rows of C through another, past whose 2^31 bytes a store is dropped (N = 4210688
// is the widest).
static bool persistent_fits(const GemmArgs &g, int64_t rows_of_B) {
    const int64_t lim = 0x7FFFFFFF;
    return g.KB % 2 == 0 && (g.M + BM) * g.K <= lim && (rows_of_B + BN) * g.K <= lim && ((BM - 1) * g.N + BN) * 2 <= lim;
}

int bs_launch_gemm(const uint8_t *A, const float *sa, const uint8_t *B, const float *sb,
                   uint16_t *C, int64_t M, int64_t N, int64_t K, int64_t band_rows,
                   int64_t band_stride, hipStream_t stream) {
    const GemmArgs g = gemm_args(A, sa, B, sb, C, M, N, K, band_rows, band_stride);
    if (persistent_fits(g, N))
        return bs_enqueue(bsgemm_persistent_kernel, dim3(persistent_grid(g, stream)), dim3(NTHREADS),
                          stream, g);
    return bs_enqueue(bsgemm_tile_kernel, dim3(gemm_grid(g)), dim3(NTHREADS), stream, g);
}

int bs_launch_gemm_lora(const uint8_t *A, const float *sa, const uint8_t *B, const float *sb, uint16_t *C,
                        const LoraArgs &lora, const int32_t *ids, int64_t M, int64_t N, int64_t K, int64_t band_rows,
                        int64_t band_stride, hipStream_t stream) {
    const GemmArgs g = gemm_args(A, sa, B, sb, C, M, N, K, band_rows, band_stride);
    const LoraGemmArgs q = {lora, ids};
    // Short batches by waves of 16 x 32 or 32 x 64 while that takes at most two or one
    // of them to a CU, middling ones by 64 x 128 tiles while that takes at most two.
    // K = 2048, R = 16, us by graph launches, 16 x 32 / 32 x 64 / 64 x 128 / 256 x 256:
    // N = 7168, M = 16: 9.9 / 14.9 / 12.4 / 29; M = 64: 19.6 / 14.8 / 13.3 / 30;
    // M = 200: 49 / 34 / 13.6 / 31; M = 512: 109 / 55 / 21 / 31; M = 1024: 216 / 122 /
    // 39 / 32; N = 1024, M = 256: 11.0 / 12.3 / 11.1 / 29; M = 512: 19.0 / 12.8 / 11.6 /
    // 29; M = 2048: - / - / 14.0 / 30; M = 4096: - / - / 23 / 30.
    const auto count = [&](int rows, int cols) { return N / cols * ((M + rows - 1) / rows); };
    const auto grid_of = [&](int rows, int cols) {
        return dim3((unsigned)((count(rows, cols) + NUM_XCD - 1) / NUM_XCD * NUM_XCD));
    };
    if (count(16, 32) <= 512)
        return bs_enqueue(bsgemm_lora_short_kernel<1, 2, 4>, grid_of(16, 32), dim3(64), stream, g, q);
    if (count(32, 64) <= 256)
        return bs_enqueue(bsgemm_lora_short_kernel<2, 4, 3>, grid_of(32, 64), dim3(64), stream, g, q);
    if (count(MID_BM, MID_BN) <= 512)
        return bs_enqueue(bsgemm_lora_mid_kernel, grid_of(MID_BM, MID_BN), dim3(NTHREADS), stream, g, q);
    return bs_enqueue(bsgemm_lora_tile_kernel, dim3(gemm_grid(g)), dim3(NTHREADS), stream, g, q);
}

// Workgroups of the few-rows kernel in a column and in a row of them.
static int64_t act_rows_x(const GemmArgs &g, bool gated, int CT) { return g.N / ((gated ? 8 : 16) * CT); }
static int64_t act_rows_y(const GemmArgs &g, int RG) { return (g.M + 16 * RG - 1) / (16 * RG); }

template <int RG, int CT>
static int launch_act_rows(const ActGemmArgs &a, bool gated, hipStream_t stream) {
    const dim3 grid((unsigned)act_rows_x(a.g, gated, CT), (unsigned)act_rows_y(a.g, RG));
    if (gated) return bs_enqueue(bsgemm_act_rows_kernel<RG, CT, true>, grid, dim3(NTHREADS), stream, a);
    return bs_enqueue(bsgemm_act_rows_kernel<RG, CT, false>, grid, dim3(NTHREADS), stream, a);
}

// Two of the 16 rows of B to a workgroup, which then reads A half as often, if that leaves
// enough workgroups.  One / two, us: N = 7168, K = 2048 (448 of one): M = 1 6.2 / 5.9, M = 16
// 7.5 / 6.5, M = 64 13.0 / 9.6; gated N = 2048, K = 7168 (256): M = 1 8.0 / 10.7, M = 16 10.1 /
// 12.9, M = 64 19.8 / 22.6; N = 1024, K = 1024 (64): M = 1 3.5 / 4.0, M = 64 5.2 / 5.8.
template <int RG>
static int launch_act_rows(const ActGemmArgs &a, bool gated, hipStream_t stream) {
    return act_rows_x(a.g, gated, 1) * act_rows_y(a.g, RG) >= 448 ? launch_act_rows<RG, 2>(a, gated, stream)
                                                                   : launch_act_rows<RG, 1>(a, gated, stream);
}

int bs_launch_gemm_act(const uint8_t *A, const float *sa, const uint8_t *B, const float *sb, const uint16_t *bias,
                       const uint16_t *resid, uint16_t *C, int64_t M, int64_t N, int64_t K, int act, bool gated,
                       float alpha, float beta, int64_t band_rows, int64_t band_stride, hipStream_t stream) {
    GemmArgs g = gemm_args(A, sa, B, sb, C, M, N, K, band_rows, band_stride);
    if (gated) g.tiles_n = (int)(N / (BN / 2));
    const ActGemmArgs a = {g, {bias, resid, alpha, beta, act}};
    const auto count = [&](int rows, int cols) { return N / cols * ((M + rows - 1) / rows); };
    const int mid_cols = gated ? MID_BN / 2 : MID_BN;
    const int64_t rows4 = act_rows_x(g, gated, 2) * act_rows_y(g, 4);
    // Few rows by the kernel that splits K over a workgroup's waves, 16, 32 or 64 rows to
    // one and the last while there is at most one of them to a CU; more by 64 x 128 tiles
    // while that takes one row of them or at most two to a CU; else whole tiles.  us by graph
    // launches, fewest rows that hold M / 64 rows / 64 x 128 / 256 x 256, with a residual,
    // N = 7168, K = 2048: M = 16: 6.5 / 7.3 / 10.2 / 29; M = 32: 7.6 / 8.1 / 11.2 / 29; M = 64:
    // 9.6 / 9.6 / 12.3 / 30; M = 128: - / 16.8 / 12.6 / 31; M = 512: - / 53 / 21 / 34; M =
    // 1024: - / 102 / 37 / 35; gated, N = 2048, K = 7168: M = 16: 10.0 / 12.9 / 24 / 71; M =
    // 128: - / 23 / 29 / 73; M = 256: - / 43 / 30 / 77; M = 512: - / 82 / 30 / 77; wide, K = 2048,
    // M = 64: N = 28672: - / 30 / 13.8 / 28; N = 131072: - / - / 64 / 82 (M = 128: 93 / 86).
    if (N < (int64_t)1 << 25) {   // a launch holds fewer than 2^32 lanes
        if (M <= 16) return launch_act_rows<1>(a, gated, stream);
        if (M <= 32) return launch_act_rows<2>(a, gated, stream);
        if (rows4 <= 256) return launch_act_rows<4>(a, gated, stream);
    }
    const int64_t mid = count(MID_BM, mid_cols), mid_grid = (mid + NUM_XCD - 1) / NUM_XCD * NUM_XCD;
    if (mid <= 512 || (M <= MID_BM && lanes_fit(mid_grid, NTHREADS))) {
        const dim3 grid((unsigned)mid_grid);
        return gated ? bs_enqueue(bsgemm_act_mid_kernel<true>, grid, dim3(NTHREADS), stream, a)
                     : bs_enqueue(bsgemm_act_mid_kernel<false>, grid, dim3(NTHREADS), stream, a);
    }
    // The gated epilogue fits beside the persistent kernel's carried products (M = 16384,
    // N = 2048: K = 2048 125 us against the tile kernel's 131, K = 7168 426 against 429); the
    // plain one, with twice the columns to a lane, spilled 38 to 86 registers there.
    if (gated && persistent_fits(g, 2 * N))
        return bs_enqueue(bsgemm_act_persistent_kernel, dim3(persistent_grid(g, stream)), dim3(NTHREADS), stream, a);
    const dim3 grid(gemm_grid(g));
    return gated   ? bs_enqueue(bsgemm_act_tile_kernel<EPI_GLU>, grid, dim3(NTHREADS), stream, a)
           : resid ? bs_enqueue(bsgemm_act_tile_kernel<EPI_RESID>, grid, dim3(NTHREADS), stream, a)
                   : bs_enqueue(bsgemm_act_tile_kernel<EPI_ACT>, grid, dim3(NTHREADS), stream, a);
}

int bs_launch_gemm_pb(const uint8_t *A, const float *sa, const uint8_t *Bp, const float *sb,
                      uint16_t *C, int64_t M, int64_t N, int64_t K, int64_t band_rows,
                      int64_t band_stride, hipStream_t stream) {
    const GemmArgs g = gemm_args(A, sa, Bp, sb, C, M, N, K, band_rows, band_stride);
    return bs_enqueue(bsgemm_pb_tile_kernel, dim3(gemm_grid(g)), dim3(NTHREADS), stream, g);
}

int bs_launch_bprepack(const uint8_t *B, uint8_t *Bp, int64_t N, int64_t K, hipStream_t stream) {
    const int64_t units = N * K / 16;
    int64_t blocks = (units + 255) / 256;
    if (blocks > 65536) blocks = 65536;
    return bs_enqueue(bprepack_kernel, dim3((unsigned)blocks), dim3(256), stream, (const u32x4 *)B,
                      (u32x4 *)Bp, units, K);
}

int bs_launch_mxgemm(const uint8_t *A, const uint8_t *sa, const uint8_t *B, const uint8_t *sb,
                     uint16_t *C, int64_t M, int64_t N, int64_t K, int64_t band_rows,
                     int64_t band_stride, hipStream_t stream) {
    const GemmArgs g = gemm_args(A, sa, B, sb, C, M, N, K, band_rows, band_stride);
    if (persistent_fits(g, N))
        return bs_enqueue(mxgemm_persistent_kernel, dim3(persistent_grid(g, stream)), dim3(NTHREADS),
                          stream, g);
    return bs_enqueue(mxgemm_tile_kernel, dim3(gemm_grid(g)), dim3(NTHREADS), stream, g);
}
