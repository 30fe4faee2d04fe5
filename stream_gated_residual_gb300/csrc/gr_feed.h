// Internal declarations of the gated feed-forward sublayer and of the products on FP8 blocks.
#pragma once

#include <stdint.h>

#include "gr_internal.h"

namespace gr {

constexpr int kBlock = 128;   // channels of an FP8 block

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// FP8 blocks of `n_matrix` matrices [rows][cols] (gr_blocks.cu).
cudaError_t launch_encode_blocks(int64_t n_matrix, int64_t rows, int64_t cols, int block_rows, int dtype,
                                 const void* m, uint8_t* codes, uint8_t* scales, cudaStream_t st);

// Scales as the products on tensor cores take them: the tokens' in words of four blocks, 512 bytes for 128 rows with
// row r's word at 16 (r % 32) + 4 (r / 32), [ceil(rows / 128)][scale_steps(k)][512]; the weights' in rows of whole words.
inline int scale_steps(int64_t k) { return int(ceil_div(ceil_div(k, kBlock), 4)); }
inline int scale_pitch(int64_t k) { return 4 * scale_steps(k); }
inline size_t token_scale_bytes(int64_t rows, int64_t k) { return size_t(ceil_div(rows, kBlock)) * scale_steps(k) * 512; }
struct Fp8Product {
    const uint8_t *tokens, *token_scales, *weights, *weight_scales;
    bool token_rows = false;   // token_scales in plain rows (tc_takes_rows): no launch before laid anything out
};
// Whether a product takes both operands' scales as the encoder left them: few tokens, rows of whole words.
bool tc_takes_rows(int64_t N, int64_t K, const uint8_t* a_scales, const uint8_t* b_scales);
// Rows of scales [rows][blocks] to be laid out: as tokens, or with the weights' pitch.
struct ScaleRows {
    const uint8_t* from;
    uint8_t* to;
    int64_t rows;
    int blocks;
    bool tokens;
};
// Lays out up to two sets of scales and, where x is not null, encodes the bf16 rows x [n][cols] in blocks of one row.
cudaError_t launch_fp8_operands(const void* x, int64_t n, int64_t cols, uint8_t* codes, uint8_t* token_scales,
                                const ScaleRows& a, const ScaleRows& b, cudaStream_t st);

// Products on the tcgen05 tensor cores, bf16 (gr_feed_tc.cu); `ws` as tc_feed_workspace says (this and the other
// workspace functions: SIZE_MAX for calls that are too large to be planned). `tokens`: of a
// product whose other dimensions are the weights' (few of them go in parts over k), else INT64_MAX. Each
// tc_product is a programmatic dependent of the launch before it on `st`, which must be this file's.
cudaError_t tc_gated(int64_t N, int D, int F, int act, const void* x, const void* w_in, void* h, void* pre,
                     float* ws, cudaStream_t st);
cudaError_t tc_gated_grad(int64_t N, int D, int F, int act, const void* dy, const void* w_out, const void* pre,
                          void* dpre, void* h, float* ws, cudaStream_t st);
cudaError_t tc_product(int64_t M, int64_t N, int64_t K, int64_t tokens, const void* a, bool a_k, const void* b,
                       bool b_k, void* out, float* ws, cudaStream_t st);
// On FP8 blocks, programmatic dependents of the launch that laid out their scales (if one did); h in blocks of one row, its
// scales laid out as the tokens of the next product; out bf16.
cudaError_t tc_gated_fp8(int64_t N, int D, int F, int act, const Fp8Product& in, uint8_t* h, uint8_t* hs, float* ws,
                         cudaStream_t st);
cudaError_t tc_product_fp8(int64_t N, int64_t O, int64_t K, const Fp8Product& in, void* out, float* ws,
                           cudaStream_t st);
size_t tc_product_fp8_workspace(int64_t N, int64_t O, int64_t K);
size_t tc_feed_fp8_workspace(int64_t N, int D, int F);
size_t tc_feed_workspace(int64_t N, int D, int F, bool gradient);
// fp32: both passes, every operand as three bf16 terms.
size_t f32_feed_workspace(int64_t N, int D, int F, bool gradient);
cudaError_t f32_feed_forward(int64_t N, int64_t D, int64_t F, int act, const float* x, const float* w_in,
                             const float* w_out, float* y, float* pre, void* ws, cudaStream_t st);
cudaError_t f32_feed_backward(int64_t N, int64_t D, int64_t F, int act, const float* dy, const float* x,
                              const float* w_in, const float* w_out, const float* pre, float* dx, float* dw_in,
                              float* dw_out, void* ws, cudaStream_t st);
// Status bits of the bounded waits of gr_feed_tc.cu (0 = none; -1 = could not be read).
int feed_status(bool clear);

#ifdef __CUDACC__
// The byte of a token's block among scales of `steps` steps.
__device__ __forceinline__ int64_t scale_at(int64_t row, uint32_t block, int steps) {
    return ((row >> 7) * steps + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (block & 3);
}
// Φ(g) in fp32. By erfc and not by 1 + erf, which cancels below zero: at g = -5 a tenth of the value is lost, below -5.6
// all of it. What is left is the argument's rounding, up to g^2 + 1 units.
__device__ __forceinline__ float normal_below(float g) { return 0.5f * erfcf(g * -0.70710678118654752f); }
// The activations and their slopes in fp32 with the accurate expf and erfcf.
template <int ACT> __device__ __forceinline__ float activate(float g) {
    if constexpr (ACT == GR_SILU) return g / (1.0f + expf(-g));
    else return g * normal_below(g);
}
template <int ACT> __device__ __forceinline__ float activate_slope(float g) {
    if constexpr (ACT == GR_SILU) {
        const float s = 1.0f / (1.0f + expf(-g));
        return s * (1.0f + g * (1.0f - s));
    } else {
        return normal_below(g) + g * expf(-0.5f * g * g) * 0.39894228040143268f;
    }
}
#endif

}  // namespace gr
