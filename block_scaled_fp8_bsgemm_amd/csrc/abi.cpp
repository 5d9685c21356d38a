// abi.cpp -- the extern "C" entry points of libbsgemm (declared, with their
// contracts, in include/bsgemm.h).  Every argument is checked on the host
// before anything is enqueued; a rejected call launches nothing and writes
// nothing.  The kernels themselves live in gemm.hip, stream.hip, lora.hip,
// resnorm.hip and moe.hip.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "bsgemm.h"
#include "launch.hpp"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;   // rows / columns per matrix
constexpr int64_t kMaxK = (int64_t)1 << 22;     // keeps in-tile byte offsets in 32 bits
constexpr int64_t kMaxRows = (int64_t)1 << 30;  // rows of a batch with adapters (32-bit positions)
constexpr int64_t kMaxAdapters = 4096;
constexpr int64_t kMaxRank = 256;
constexpr int64_t kMaxNorm = 16384;             // a normed row: it stays in one workgroup's registers
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxTopk = 64;                // a chosen expert to a lane
constexpr int64_t kMaxTokens = 128, kMaxPairs = 1024;   // moe_fp8: the lists that its workgroups hold
constexpr int64_t kMaxWidth = 65536;            // moe_fp8: D and I
constexpr int32_t kActs = 5;

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void *p, int64_t bytes) {
    uintptr_t a = (uintptr_t)p;
    return Range{a, a + (uintptr_t)(bytes > 0 ? bytes : 0)};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Whether one launch holds the products' tiles of 256 x 256, 512 lanes to each: their number
// is rounded up to a multiple of the 8 XCDs, and the lanes stay fewer than 2^32.
inline bool tiles_fit(int64_t M, int64_t rows_of_B) {
    return (M + 255) / 256 * ((rows_of_B + 255) / 256) <= ((int64_t)1 << 23) - 8;
}

inline hipStream_t as_stream(void *s) { return (hipStream_t)s; }

}  // namespace

extern "C" {

const char *bs_status_str(bs_status status) {
    switch (status) {
        case BS_OK: return "ok";
        case BS_ERR_INVALID: return "invalid argument (null pointer, negative size, bad count or overlapping buffers)";
        case BS_ERR_UNSUPPORTED: return "unsupported shape, stride or alignment";
        case BS_ERR_LAUNCH: return "the HIP runtime rejected the kernel launch";
    }
    return "unknown status";
}

}  // extern "C"

namespace {

// Validation shared by the blockscale GEMM entry points: B is either the
// weight [N, K] row-major or its prepacked form, the same N * K bytes.  `more`
// checks what an entry point takes besides, given C's range.
template <typename Launch, typename More>
bs_status blockscale_gemm(Launch launch, More more, const uint8_t *A, const float *a_scale,
                          const uint8_t *B, const float *b_scale, uint16_t *C, int64_t M,
                          int64_t N, int64_t K, int32_t bands, int64_t band_stride,
                          void *stream) {
    if (!A || !a_scale || !B || !b_scale || !C) return BS_ERR_INVALID;
    if (M < 0 || N <= 0 || K <= 0 || bands < 1 || band_stride < 0) return BS_ERR_INVALID;
    if (N % 128 || K % 128 || bands > 64) return BS_ERR_UNSUPPORTED;
    if (M >= kMaxDim || N >= kMaxDim || K > kMaxK || !tiles_fit(M, N)) return BS_ERR_UNSUPPORTED;
    if (M % bands) return BS_ERR_UNSUPPORTED;
    const int64_t band_rows = M / bands;
    const int64_t stride = band_stride == 0 ? band_rows * N : band_stride;
    if (stride < band_rows * N || stride % 8) return BS_ERR_UNSUPPORTED;
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(a_scale, 4) ||
        !aligned(b_scale, 4))
        return BS_ERR_UNSUPPORTED;
    const int64_t KB = K / 128, NB = N / 128;
    const Range rc = range_of(C, ((bands - 1) * stride + band_rows * N) * 2);
    if (overlap(rc, range_of(A, M * K)) || overlap(rc, range_of(B, N * K)) ||
        overlap(rc, range_of(a_scale, M * KB * 4)) || overlap(rc, range_of(b_scale, NB * KB * 4)))
        return BS_ERR_INVALID;
    if (const bs_status st = more(rc); st != BS_OK) return st;
    if (M == 0) return BS_OK;
    return launch(A, a_scale, B, b_scale, C, M, N, K, band_rows == 0 ? 1 : band_rows, stride,
                  as_stream(stream)) == 0
               ? BS_OK
               : BS_ERR_LAUNCH;
}

// What the low-rank entry points share: counts of adapters and ranks.
bs_status lora_dims(int64_t M, int64_t L, int64_t R) {
    if (M < 0 || L <= 0 || R <= 0) return BS_ERR_INVALID;
    if (M >= kMaxRows || L > kMaxAdapters || R % 8 || R > kMaxRank) return BS_ERR_UNSUPPORTED;
    return BS_OK;
}

}  // namespace

extern "C" {

bs_status bsgemm_fp8(const uint8_t *A, const float *a_scale, const uint8_t *B, const float *b_scale,
                     uint16_t *C, int64_t M, int64_t N, int64_t K, int32_t bands,
                     int64_t band_stride, void *stream) {
    return blockscale_gemm(bs_launch_gemm, [](Range) { return BS_OK; }, A, a_scale, B, b_scale, C, M,
                           N, K, bands, band_stride, stream);
}

bs_status bsgemm_fp8_pb(const uint8_t *A, const float *a_scale, const uint8_t *Bp,
                        const float *b_scale, uint16_t *C, int64_t M, int64_t N, int64_t K,
                        int32_t bands, int64_t band_stride, void *stream) {
    return blockscale_gemm(bs_launch_gemm_pb, [](Range) { return BS_OK; }, A, a_scale, Bp, b_scale,
                           C, M, N, K, bands, band_stride, stream);
}

bs_status bprepack_e4m3(const uint8_t *B, uint8_t *Bp, int64_t N, int64_t K, void *stream) {
    if (!B || !Bp || N <= 0 || K <= 0) return BS_ERR_INVALID;
    if (N % 128 || K % 128 || N >= kMaxDim || K > kMaxK) return BS_ERR_UNSUPPORTED;
    if (!aligned(B, 16) || !aligned(Bp, 16)) return BS_ERR_UNSUPPORTED;
    if (overlap(range_of(B, N * K), range_of(Bp, N * K))) return BS_ERR_INVALID;
    return bs_launch_bprepack(B, Bp, N, K, as_stream(stream)) == 0 ? BS_OK : BS_ERR_LAUNCH;
}

bs_status mxgemm_fp8(const uint8_t *A, const uint8_t *a_scale, const uint8_t *B, const uint8_t *b_scale,
                     uint16_t *C, int64_t M, int64_t N, int64_t K, int32_t bands,
                     int64_t band_stride, void *stream) {
    if (!A || !a_scale || !B || !b_scale || !C) return BS_ERR_INVALID;
    if (M < 0 || N <= 0 || K <= 0 || bands < 1 || band_stride < 0) return BS_ERR_INVALID;
    if (N % 128 || K % 128 || bands > 64) return BS_ERR_UNSUPPORTED;
    if (M >= kMaxDim || N >= kMaxDim || K > kMaxK || !tiles_fit(M, N)) return BS_ERR_UNSUPPORTED;
    if (M % bands) return BS_ERR_UNSUPPORTED;
    const int64_t band_rows = M / bands;
    const int64_t stride = band_stride == 0 ? band_rows * N : band_stride;
    if (stride < band_rows * N || stride % 8) return BS_ERR_UNSUPPORTED;
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(a_scale, 4) ||
        !aligned(b_scale, 4))
        return BS_ERR_UNSUPPORTED;
    const int64_t KQ = K / 32;
    const Range rc = range_of(C, ((bands - 1) * stride + band_rows * N) * 2);
    if (overlap(rc, range_of(A, M * K)) || overlap(rc, range_of(B, N * K)) ||
        overlap(rc, range_of(a_scale, M * KQ)) || overlap(rc, range_of(b_scale, N * KQ)))
        return BS_ERR_INVALID;
    if (M == 0) return BS_OK;
    return bs_launch_mxgemm(A, a_scale, B, b_scale, C, M, N, K, band_rows == 0 ? 1 : band_rows,
                            stride, as_stream(stream)) == 0
               ? BS_OK
               : BS_ERR_LAUNCH;
}

bs_status band_reduce(const uint16_t *const *parts, int32_t P, uint16_t *out, int64_t rows,
                      int64_t N, void *stream) {
    if (!parts || !out || P < 1 || P > 16 || rows < 0 || N <= 0) return BS_ERR_INVALID;
    for (int p = 0; p < P; p++)
        if (!parts[p]) return BS_ERR_INVALID;
    if (N % 8 || rows >= kMaxDim * 8 || N >= kMaxDim) return BS_ERR_UNSUPPORTED;
    if (!aligned(out, 16)) return BS_ERR_UNSUPPORTED;
    for (int p = 0; p < P; p++)
        if (!aligned(parts[p], 16)) return BS_ERR_UNSUPPORTED;
    const Range ro = range_of(out, rows * N * 2);
    for (int p = 0; p < P; p++)
        if (overlap(ro, range_of(parts[p], rows * N * 2))) return BS_ERR_INVALID;
    if (rows == 0) return BS_OK;
    return bs_launch_band_reduce(parts, P, out, rows, N, as_stream(stream)) == 0 ? BS_OK : BS_ERR_LAUNCH;
}

bs_status band_rowq_e4m3(const uint16_t *const *parts, int32_t P, uint8_t *q, float *scale,
                         int64_t rows, int64_t N, void *stream) {
    if (!parts || !q || !scale || P < 1 || P > 16 || rows < 0 || N <= 0) return BS_ERR_INVALID;
    for (int p = 0; p < P; p++)
        if (!parts[p]) return BS_ERR_INVALID;
    if (N % 8 || N > 8192 || rows >= kMaxDim) return BS_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(scale, 4)) return BS_ERR_UNSUPPORTED;
    for (int p = 0; p < P; p++)
        if (!aligned(parts[p], 16)) return BS_ERR_UNSUPPORTED;
    const Range rq = range_of(q, rows * N), rs = range_of(scale, rows * 4);
    if (overlap(rq, rs)) return BS_ERR_INVALID;
    for (int p = 0; p < P; p++) {
        const Range rp = range_of(parts[p], rows * N * 2);
        if (overlap(rq, rp) || overlap(rs, rp)) return BS_ERR_INVALID;
    }
    if (rows == 0) return BS_OK;
    return bs_launch_band_rowq(parts, P, q, scale, rows, N, as_stream(stream)) == 0 ? BS_OK
                                                                                     : BS_ERR_LAUNCH;
}

bs_status rowq_e4m3(const uint16_t *x, uint8_t *q, float *scale, int64_t rows, int64_t N,
                    void *stream) {
    if (!x || !q || !scale || rows < 0 || N <= 0) return BS_ERR_INVALID;
    if (N % 8 || N / 8 >= kMaxDim || rows >= kMaxDim * 8) return BS_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return BS_ERR_UNSUPPORTED;
    const Range rx = range_of(x, rows * N * 2), rq = range_of(q, rows * N), rs = range_of(scale, rows * 4);
    if (overlap(rq, rx) || overlap(rs, rx) || overlap(rq, rs)) return BS_ERR_INVALID;
    if (rows == 0) return BS_OK;
    return bs_launch_rowq(x, q, scale, rows, N, as_stream(stream)) == 0 ? BS_OK : BS_ERR_LAUNCH;
}

bs_status rowdq_e4m3(const uint8_t *q, const float *scale, uint16_t *y, int64_t rows, int64_t N,
                     void *stream) {
    if (!q || !scale || !y || rows < 0 || N <= 0) return BS_ERR_INVALID;
    if (N % 8 || N / 8 >= kMaxDim || rows >= kMaxDim * 8) return BS_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(y, 16) || !aligned(scale, 4)) return BS_ERR_UNSUPPORTED;
    const Range ry = range_of(y, rows * N * 2);
    if (overlap(ry, range_of(q, rows * N)) || overlap(ry, range_of(scale, rows * 4))) return BS_ERR_INVALID;
    if (rows == 0) return BS_OK;
    return bs_launch_rowdq(q, scale, y, rows, N, as_stream(stream)) == 0 ? BS_OK : BS_ERR_LAUNCH;
}

bs_status blockq_e4m3(const float *x, uint8_t *q, float *scale, int64_t rows, int64_t cols,
                      int32_t block_rows, void *stream) {
    if (!x || !q || !scale || rows < 0 || cols <= 0) return BS_ERR_INVALID;
    if (block_rows != 1 && block_rows != 128) return BS_ERR_UNSUPPORTED;
    if (cols % 128 || cols >= kMaxDim || rows >= kMaxDim) return BS_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return BS_ERR_UNSUPPORTED;
    const int64_t nscale = ((rows + block_rows - 1) / block_rows) * (cols / 128);
    const Range rx = range_of(x, rows * cols * 4), rq = range_of(q, rows * cols),
                rs = range_of(scale, nscale * 4);
    if (overlap(rq, rx) || overlap(rs, rx) || overlap(rq, rs)) return BS_ERR_INVALID;
    if (rows == 0) return BS_OK;
    return bs_launch_blockq(x, q, scale, rows, cols, block_rows, as_stream(stream)) == 0 ? BS_OK
                                                                                         : BS_ERR_LAUNCH;
}

bs_status actq_e4m3(const uint16_t *x, uint8_t *q, float *scale, int64_t rows, int64_t cols,
                    void *stream) {
    if (!x || !q || !scale || rows < 0 || cols <= 0) return BS_ERR_INVALID;
    if (cols % 128 || cols >= kMaxDim || rows >= kMaxDim) return BS_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return BS_ERR_UNSUPPORTED;
    const Range rx = range_of(x, rows * cols * 2), rq = range_of(q, rows * cols),
                rs = range_of(scale, rows * (cols / 128) * 4);
    if (overlap(rq, rx) || overlap(rs, rx) || overlap(rq, rs)) return BS_ERR_INVALID;
    if (rows == 0) return BS_OK;
    return bs_launch_actq(x, q, scale, rows, cols, as_stream(stream)) == 0 ? BS_OK : BS_ERR_LAUNCH;
}

bs_status mxq_e4m3(const uint16_t *x, uint8_t *q, uint8_t *scale, int64_t rows, int64_t cols,
                   void *stream) {
    if (!x || !q || !scale || rows < 0 || cols <= 0) return BS_ERR_INVALID;
    if (cols % 32 || cols >= kMaxDim || rows >= kMaxDim) return BS_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(q, 16)) return BS_ERR_UNSUPPORTED;
    const Range rx = range_of(x, rows * cols * 2), rq = range_of(q, rows * cols),
                rs = range_of(scale, rows * (cols / 32));
    if (overlap(rq, rx) || overlap(rs, rx) || overlap(rq, rs)) return BS_ERR_INVALID;
    if (rows == 0) return BS_OK;
    return bs_launch_mxq(x, q, scale, rows, cols, as_stream(stream)) == 0 ? BS_OK : BS_ERR_LAUNCH;
}

bs_status lora_plan(const int32_t *ids, int32_t *plan, int64_t M, int64_t n_adapters, void *stream) {
    if (!plan || (!ids && M > 0) || M < 0 || n_adapters <= 0) return BS_ERR_INVALID;
    if (M >= kMaxRows || n_adapters > kMaxAdapters) return BS_ERR_UNSUPPORTED;
    if (!aligned(ids, 4) || !aligned(plan, 4)) return BS_ERR_UNSUPPORTED;
    if (overlap(range_of(plan, (n_adapters + 2 + M) * 4), range_of(ids, M * 4))) return BS_ERR_INVALID;
    return bs_launch_lora_plan(ids, plan, M, (int)n_adapters, as_stream(stream)) == 0 ? BS_OK : BS_ERR_LAUNCH;
}

bs_status lora_shrink(const uint16_t *x, const uint16_t *A, const int32_t *plan, float *H, int64_t M, int64_t K,
                      int64_t n_adapters, int64_t R, void *stream) {
    if (!x || !A || !plan || !H || K <= 0) return BS_ERR_INVALID;
    if (const bs_status st = lora_dims(M, n_adapters, R); st != BS_OK) return st;
    if (K % 8 || K > kMaxK) return BS_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(A, 16) || !aligned(H, 16) || !aligned(plan, 4)) return BS_ERR_UNSUPPORTED;
    const Range rh = range_of(H, M * R * 4);
    if (overlap(rh, range_of(x, M * K * 2)) || overlap(rh, range_of(A, n_adapters * R * K * 2)) ||
        overlap(rh, range_of(plan, (n_adapters + 2 + M) * 4)))
        return BS_ERR_INVALID;
    if (M == 0) return BS_OK;
    return bs_launch_lora_shrink(x, A, plan, H, M, K, (int)n_adapters, (int)R, as_stream(stream)) == 0
               ? BS_OK
               : BS_ERR_LAUNCH;
}

bs_status lora_expand(const float *H, const uint16_t *B, const float *scale, const int32_t *plan,
                      const uint16_t *base, uint16_t *out, int64_t M, int64_t N, int64_t n_adapters, int64_t R,
                      int32_t bands, int64_t band_stride, void *stream) {
    if (!H || !B || !plan || !base || !out || N <= 0 || bands < 1 || band_stride < 0) return BS_ERR_INVALID;
    if (const bs_status st = lora_dims(M, n_adapters, R); st != BS_OK) return st;
    if (N % 8 || N >= kMaxDim || bands > 64 || M % bands) return BS_ERR_UNSUPPORTED;
    const int64_t band_rows = M / bands;
    const int64_t stride = band_stride == 0 ? band_rows * N : band_stride;
    if (stride < band_rows * N || stride % 8) return BS_ERR_UNSUPPORTED;
    if (!aligned(H, 16) || !aligned(B, 16) || !aligned(base, 16) || !aligned(out, 16) || !aligned(plan, 4) ||
        !aligned(scale, 4))
        return BS_ERR_UNSUPPORTED;
    const int64_t bytes = ((bands - 1) * stride + band_rows * N) * 2;
    const Range ro = range_of(out, bytes);
    if ((base != out && overlap(ro, range_of(base, bytes))) || overlap(ro, range_of(H, M * R * 4)) ||
        overlap(ro, range_of(B, n_adapters * N * R * 2)) || overlap(ro, range_of(scale, scale ? n_adapters * 4 : 0)) ||
        overlap(ro, range_of(plan, (n_adapters + 2 + M) * 4)))
        return BS_ERR_INVALID;
    if (M == 0) return BS_OK;
    const LoraArgs lora = {H, B, scale, (int)n_adapters, (int)R};
    return bs_launch_lora_expand(lora, plan, base, out, M, N, band_rows, stride, as_stream(stream)) == 0
               ? BS_OK
               : BS_ERR_LAUNCH;
}

bs_status bsgemm_fp8_lora(const uint8_t *A, const float *a_scale, const uint8_t *B, const float *b_scale,
                          const float *H, const uint16_t *lora_B, const float *lora_scale, const int32_t *ids,
                          uint16_t *C, int64_t M, int64_t N, int64_t K, int64_t n_adapters, int64_t R, int32_t bands,
                          int64_t band_stride, void *stream) {
    if (!H || !lora_B || !ids) return BS_ERR_INVALID;
    if (const bs_status st = lora_dims(M, n_adapters, R); st != BS_OK) return st;
    if (!aligned(H, 16) || !aligned(lora_B, 16) || !aligned(lora_scale, 4) || !aligned(ids, 4))
        return BS_ERR_UNSUPPORTED;
    const LoraArgs lora = {H, lora_B, lora_scale, (int)n_adapters, (int)R};
    const auto more = [&](Range rc) {
        const bool hit = overlap(rc, range_of(H, M * R * 4)) || overlap(rc, range_of(lora_B, n_adapters * N * R * 2)) ||
                         overlap(rc, range_of(lora_scale, lora_scale ? n_adapters * 4 : 0)) ||
                         overlap(rc, range_of(ids, M * 4));
        return hit ? BS_ERR_INVALID : BS_OK;
    };
    const auto launch = [&](const uint8_t *a, const float *sa, const uint8_t *b, const float *sb, uint16_t *c,
                            int64_t m, int64_t n, int64_t k, int64_t band_rows, int64_t stride, hipStream_t st) {
        return bs_launch_gemm_lora(a, sa, b, sb, c, lora, ids, m, n, k, band_rows, stride, st);
    };
    return blockscale_gemm(launch, more, A, a_scale, B, b_scale, C, M, N, K, bands, band_stride, stream);
}

bs_status resnorm(const void *y, const float *y_scale, const void *resid, const uint16_t *post_w,
                  const uint16_t *gate, int64_t gate_row, const uint16_t *pre_w, void *resid_out, uint16_t *z,
                  uint8_t *q, void *q_scale, int64_t rows, int64_t N, int32_t resid_f32, int32_t q_block, float alpha,
                  float beta, float eps, void *stream) {
    if (!y || !resid || !resid_out || rows < 0 || N <= 0 || gate_row < 0) return BS_ERR_INVALID;
    if (resid_f32 != 0 && resid_f32 != 1) return BS_ERR_INVALID;
    if (q_block != 0 && q_block != 32 && q_block != 128) return BS_ERR_UNSUPPORTED;
    if ((q_block != 0) != (q != nullptr) || (q_block != 0) != (q_scale != nullptr)) return BS_ERR_INVALID;
    if (!(eps > 0.0f) || !std::isfinite(eps) || !std::isfinite(alpha) || !std::isfinite(beta)) return BS_ERR_INVALID;
    if (N % 8 || N > kMaxNorm || rows >= kMaxDim || (q_block && N % q_block)) return BS_ERR_UNSUPPORTED;
    if (gate_row != 0 && gate_row != N) return BS_ERR_UNSUPPORTED;
    const void *p16[] = {y, resid, post_w, gate, pre_w, resid_out, z, q};
    for (const void *p : p16)
        if (!aligned(p, 16)) return BS_ERR_UNSUPPORTED;
    if (!aligned(y_scale, 4) || !aligned(q_scale, q_block == 128 ? 4 : 1)) return BS_ERR_UNSUPPORTED;
    const int64_t n = rows * N, rb = n * (resid_f32 ? 4 : 2);
    const Range in[] = {range_of(y, y_scale ? n : n * 2), range_of(y_scale, y_scale ? rows * 4 : 0),
                        range_of(post_w, post_w ? N * 2 : 0), range_of(gate, !gate ? 0 : gate_row ? n * 2 : N * 2),
                        range_of(pre_w, pre_w ? N * 2 : 0), range_of(resid, rb)};
    const Range out[] = {range_of(resid_out, rb), range_of(z, z ? n * 2 : 0), range_of(q, q ? n : 0),
                         range_of(q_scale, q_block ? n / 32 : 0) /* n / 128 fp32, or n / 32 bytes */};
    for (int i = 0; i < 4; i++) {
        for (int j = 0; j < 6; j++)   // the residual may be updated in place
            if (overlap(out[i], in[j]) && !(i == 0 && j == 5 && resid == resid_out)) return BS_ERR_INVALID;
        for (int j = i + 1; j < 4; j++)
            if (overlap(out[i], out[j])) return BS_ERR_INVALID;
    }
    if (rows == 0) return BS_OK;
    const ResnormArgs g = {y, y_scale, post_w, gate, resid, resid_out, pre_w, z, q, q_scale,
                           rows, gate_row, (int)(N / 8), alpha, beta, eps};
    return bs_launch_resnorm(g, resid_f32 != 0, q_block, as_stream(stream)) == 0 ? BS_OK : BS_ERR_LAUNCH;
}

bs_status bsgemm_fp8_act(const uint8_t *A, const float *a_scale, const uint8_t *B, const float *b_scale,
                         const uint16_t *bias, const uint16_t *resid, uint16_t *C, int64_t M, int64_t N, int64_t K,
                         int32_t act, int32_t gated, float alpha, float beta, int32_t bands, int64_t band_stride,
                         void *stream) {
    if (act < 0 || act >= kActs || (gated != 0 && gated != 1)) return BS_ERR_INVALID;
    if (!std::isfinite(alpha) || !std::isfinite(beta)) return BS_ERR_INVALID;
    if (N > 0 && N < kMaxDim && M > 0 && M < kMaxDim) {
        const int64_t rows = gated ? 2 * N : N;   // of B
        if (rows >= kMaxDim || !tiles_fit(M, rows)) return BS_ERR_UNSUPPORTED;
    }
    if (!aligned(bias, 16) || !aligned(resid, 16)) return BS_ERR_UNSUPPORTED;
    const auto more = [&](Range rc) {
        const Range rr = range_of(resid, resid ? (int64_t)(rc.hi - rc.lo) : 0);
        if (overlap(rc, range_of(bias, bias ? (gated ? 2 : 1) * N * 2 : 0)) || (resid != C && overlap(rc, rr)) ||
            (gated && (overlap(rc, range_of(B, 2 * N * K)) || overlap(rc, range_of(b_scale, N / 64 * (K / 128) * 4)))))
            return BS_ERR_INVALID;
        return BS_OK;
    };
    const auto launch = [&](const uint8_t *a, const float *sa, const uint8_t *b, const float *sb, uint16_t *c,
                            int64_t m, int64_t n, int64_t k, int64_t band_rows, int64_t stride, hipStream_t st) {
        return bs_launch_gemm_act(a, sa, b, sb, bias, resid, c, m, n, k, act, gated != 0, alpha, beta, band_rows,
                                  stride, st);
    };
    return blockscale_gemm(launch, more, A, a_scale, B, b_scale, C, M, N, K, bands, band_stride, stream);
}

bs_status moe_route(const void *logits, const float *bias, int32_t *ids, float *weights, int64_t rows, int64_t E,
                    int32_t topk, int32_t logits_bf16, int32_t score, int32_t groups, int32_t topk_groups,
                    int32_t group_top, int32_t renorm, float scale, void *stream) {
    if (((!logits || !ids || !weights) && rows != 0) || rows < 0 || E <= 0 || topk < 1 || groups < 1)
        return BS_ERR_INVALID;
    if ((logits_bf16 | score | renorm) & ~1) return BS_ERR_INVALID;
    if (topk > E || topk_groups < 1 || topk_groups > groups || !std::isfinite(scale)) return BS_ERR_INVALID;
    if (group_top != 1 && group_top != 2) return BS_ERR_INVALID;
    if (E > kMaxExperts || topk > kMaxTopk || groups > 64 || E % groups || rows >= ((int64_t)1 << 40) / E)
        return BS_ERR_UNSUPPORTED;
    if (!aligned(logits, logits_bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return BS_ERR_UNSUPPORTED;
    const Range ri = range_of(ids, rows * topk * 4), rw = range_of(weights, rows * topk * 4);
    const Range in[] = {range_of(logits, rows * E * (logits_bf16 ? 2 : 4)), range_of(bias, bias ? E * 4 : 0)};
    for (const Range &r : in)
        if (overlap(ri, r) || overlap(rw, r)) return BS_ERR_INVALID;
    if (overlap(ri, rw)) return BS_ERR_INVALID;
    if (rows == 0) return BS_OK;
    const int per = (int)(E / groups);
    // floor(e * mul / 2^20) = e / per for e < 1024: mul exceeds 2^20 / per by less than
    // one, so e * mul / 2^20 exceeds e / per by less than 2^-10 <= 1 / per
    const unsigned mul = ((1u << 20) + (unsigned)per - 1) / (unsigned)per;
    const RouteArgs g = {logits, bias, ids, weights, rows, (int)E, topk, logits_bf16, score == 0, groups, topk_groups,
                         group_top, renorm, per, mul, scale};
    return bs_launch_moe_route(g, as_stream(stream)) == 0 ? BS_OK : BS_ERR_LAUNCH;
}

}  // extern "C"

namespace {

bs_status moe_dims(int64_t M, int64_t topk, int64_t E, int64_t I) {
    if (M < 0 || topk <= 0 || E <= 0 || I <= 0) return BS_ERR_INVALID;
    if (M > kMaxTokens || topk > kMaxTopk || M * topk > kMaxPairs || E > kMaxExperts) return BS_ERR_UNSUPPORTED;
    if (I % 128 || I > kMaxWidth) return BS_ERR_UNSUPPORTED;
    return BS_OK;
}

}  // namespace

extern "C" {

bs_status moe_fp8_workspace(int64_t M, int64_t topk, int64_t E, int64_t I, int64_t *bytes) {
    if (!bytes) return BS_ERR_INVALID;
    if (const bs_status st = moe_dims(M, topk, E, I); st != BS_OK) return st;
    *bytes = bs_moe_workspace(M, topk, E, I);
    return BS_OK;
}

bs_status moe_fp8(const uint16_t *x, const int32_t *ids, const float *weights, const uint8_t *W13, const float *s13,
                  const uint8_t *W2, const float *s2, const uint16_t *base, uint16_t *out, void *ws, int64_t M,
                  int64_t topk, int64_t E, int64_t D, int64_t I, int32_t act, void *stream) {
    if (!W13 || !s13 || !W2 || !s2 || D <= 0 || act < 0 || act >= kActs) return BS_ERR_INVALID;
    if (const bs_status st = moe_dims(M, topk, E, I); st != BS_OK) return st;
    if (D % 128 || D > kMaxWidth) return BS_ERR_UNSUPPORTED;
    if (M == 0) return BS_OK;
    if (!x || !ids || !weights || !out || !ws) return BS_ERR_INVALID;
    const void *p16[] = {x, W13, W2, base, out, ws};
    for (const void *p : p16)
        if (!aligned(p, 16)) return BS_ERR_UNSUPPORTED;
    const void *p4[] = {ids, weights, s13, s2};
    for (const void *p : p4)
        if (!aligned(p, 4)) return BS_ERR_UNSUPPORTED;
    const int64_t blocks = E * (I / 128) * (D / 128);
    const Range in[] = {range_of(x, M * D * 2), range_of(ids, M * topk * 4), range_of(weights, M * topk * 4),
                        range_of(W13, 2 * E * I * D), range_of(s13, 2 * blocks * 4), range_of(W2, E * I * D),
                        range_of(s2, blocks * 4), range_of(base, base ? M * D * 2 : 0)};
    const Range ro = range_of(out, M * D * 2), rws = range_of(ws, bs_moe_workspace(M, topk, E, I));
    if (overlap(ro, rws)) return BS_ERR_INVALID;
    for (int i = 0; i < 8; i++)
        if (overlap(rws, in[i]) || (overlap(ro, in[i]) && !(i == 7 && base == out))) return BS_ERR_INVALID;
    const MoeArgs g = {x, ids, weights, W13, s13, W2, s2, base, out, (uint16_t *)ws, nullptr, (int)M, (int)topk, (int)E, act, D, I};
    return bs_launch_moe(g, as_stream(stream)) == 0 ? BS_OK : BS_ERR_LAUNCH;
}

}  // extern "C"
