// launch.hpp -- internal launchers behind the C ABI (arguments already
// validated by abi.cpp).  Each returns 0 when the launch was accepted.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

int bs_launch_gemm(const uint8_t *A, const float *sa, const uint8_t *B, const float *sb,
                   uint16_t *C, int64_t M, int64_t N, int64_t K, int64_t band_rows,
                   int64_t band_stride, hipStream_t stream);

int bs_launch_gemm_pb(const uint8_t *A, const float *sa, const uint8_t *Bp, const float *sb,
                      uint16_t *C, int64_t M, int64_t N, int64_t K, int64_t band_rows,
                      int64_t band_stride, hipStream_t stream);
int bs_launch_bprepack(const uint8_t *B, uint8_t *Bp, int64_t N, int64_t K, hipStream_t stream);
int bs_launch_mxgemm(const uint8_t *A, const uint8_t *sa, const uint8_t *B, const uint8_t *sb,
                     uint16_t *C, int64_t M, int64_t N, int64_t K, int64_t band_rows,
                     int64_t band_stride, hipStream_t stream);
int bs_launch_band_reduce(const uint16_t *const *parts, int P, uint16_t *out, int64_t rows,
                          int64_t N, hipStream_t stream);

int bs_launch_rowq(const uint16_t *x, uint8_t *q, float *scale, int64_t rows, int64_t N,
                   hipStream_t stream);

int bs_launch_rowdq(const uint8_t *q, const float *scale, uint16_t *y, int64_t rows, int64_t N,
                    hipStream_t stream);

int bs_launch_blockq(const float *x, uint8_t *q, float *scale, int64_t rows, int64_t cols,
                     int block_rows, hipStream_t stream);
int bs_launch_band_rowq(const uint16_t *const *parts, int P, uint8_t *q, float *scale, int64_t rows,
                        int64_t N, hipStream_t stream);
int bs_launch_actq(const uint16_t *x, uint8_t *q, float *scale, int64_t rows, int64_t cols,
                   hipStream_t stream);
int bs_launch_mxq(const uint16_t *x, uint8_t *q, uint8_t *e, int64_t rows, int64_t cols,
                  hipStream_t stream);

// The low-rank adapters of a batch: what lora_expand and the GEMM with
// adapters read besides the row each adapter belongs to.
struct LoraArgs {
    const float *H;         // fp32 [M, R]: x A[a]^T of each row
    const uint16_t *B;      // bf16 [L, N, R]
    const float *scale;     // fp32 [L]; null: 1
    int L, R;
};
int bs_launch_lora_plan(const int32_t *ids, int32_t *plan, int64_t M, int L, hipStream_t stream);
int bs_launch_lora_shrink(const uint16_t *x, const uint16_t *A, const int32_t *plan, float *H, int64_t M, int64_t K,
                          int L, int R, hipStream_t stream);
int bs_launch_lora_expand(const LoraArgs &lora, const int32_t *plan, const uint16_t *base, uint16_t *out, int64_t M,
                          int64_t N, int64_t band_rows, int64_t band_stride, hipStream_t stream);
int bs_launch_gemm_lora(const uint8_t *A, const float *sa, const uint8_t *B, const float *sb, uint16_t *C,
                        const LoraArgs &lora, const int32_t *ids, int64_t M, int64_t N, int64_t K, int64_t band_rows,
                        int64_t band_stride, hipStream_t stream);

// One row of resnorm, see resnorm.hip.
struct ResnormArgs {
    const void *y;            // bf16 [rows, N], or e4m3 codes with y_scale
    const float *y_scale;     // fp32 [rows]; null: y is bf16
    const uint16_t *post_w;   // bf16 [N]; null: no norm after the block
    const uint16_t *gate;     // bf16 [N] (gate_row == 0) or [rows, N]; null: 1
    const void *resid;        // bf16 or fp32 [rows, N]
    void *resid_out;          // the same type
    const uint16_t *pre_w;    // bf16 [N]; null: 1
    uint16_t *z;              // bf16 [rows, N] or null
    uint8_t *q;               // e4m3 [rows, N] or null
    void *q_scale;            // fp32 [rows, N/128] or E8M0 [rows, N/32]
    int64_t rows, gate_row;
    int nch;                  // N / 8
    float alpha, beta, eps;
};
int bs_launch_resnorm(const ResnormArgs &g, bool resid_f32, int q_block, hipStream_t stream);

#include <tuple>

// Enqueue `kernel` with hipLaunchKernel and report that launch's own status
// (not a sticky error left by an unrelated earlier call).  No dimension may hold 2^32
// lanes or more: the runtime refuses that or, seen too, runs their number modulo
// 2^32 and reports success.
template <typename... KArgs, typename... Args>
int bs_enqueue(void (*kernel)(KArgs...), dim3 grid, dim3 block, hipStream_t stream, Args... args) {
    static_assert(sizeof...(KArgs) == sizeof...(Args), "kernel argument count");
    std::tuple<KArgs...> a(args...);
    hipError_t rc = hipSuccess;
    std::apply(
        [&](auto &...e) {
            void *argv[] = {(void *)&e...};
            rc = hipLaunchKernel((const void *)kernel, grid, block, argv, 0, stream);
        },
        a);
    return rc == hipSuccess ? 0 : -1;
}
