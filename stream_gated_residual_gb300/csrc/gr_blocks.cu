// FP8 blocks: matrices as e4m3 codes with a power-of-two scale for each 128 channels of a row (activations)
// or each 128 x 128 values (weights). A block's exponent is the smallest e with its largest magnitude at most
// 448·2^e, so no value is clipped; its codes are v/2^e rounded to nearest even. One pass: a block's values
// stay in registers between their maximum and their codes.
#include "gr_feed.h"
#include "gr_ptx.cuh"
#include "gr_blocks.cuh"

namespace gr {
namespace {

__device__ __forceinline__ void load16(const float* p, float (&v)[4]) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&v)[4], float inv) {
    *reinterpret_cast<uint32_t*>(p) = block_codes4(v, inv);
}
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&v)[8], float inv) {
    *reinterpret_cast<uint2*>(p) = make_uint2(block_codes4(v, inv), block_codes4(v + 4, inv));
}

constexpr int kThreads = 256;

// Blocks of one row: 16 bytes a lane, so 16 lanes (bf16) or 32 (fp32) hold a block. Each group of lanes reads two blocks
// before it encodes the first: 16384 bf16 rows of 4096 take 43 us (one block at a time 47, four 42; 128 rows 1.9 us,
// with four 2.3). TOKENS: scales as a product takes them.
constexpr int kPer = 2;
template <typename T, bool TOKENS>
__device__ __forceinline__ void encode_rows(const T* __restrict__ m, uint8_t* __restrict__ codes,
                                            uint8_t* __restrict__ scales, uint32_t blocks, int64_t cols, uint32_t nb,
                                            uint32_t cta) {
    constexpr int kV = 16 / sizeof(T), kLanes = kBlock / kV, kGroups = kThreads / kLanes;
    const int lane = threadIdx.x % kLanes;
    const uint32_t first = cta * (kGroups * kPer) + threadIdx.x / kLanes;
    float v[kPer][kV];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t at = first + i * kGroups, row = at / nb, c = (at - row * nb) * kBlock + lane * kV;
#pragma unroll
        for (int k = 0; k < kV; ++k) v[i][k] = 0.0f;
        if (at < blocks && c < cols) load16(m + row * cols + c, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t at = first + i * kGroups, row = at / nb, b = at - row * nb, c = b * kBlock + lane * kV;
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kV; ++k) top = max(top, block_mag(v[i][k]));
#pragma unroll
        for (int d = kLanes / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
        float inv;
        const uint8_t s = block_scale(top, inv);
        if (at < blocks && c < cols) store_codes(codes + row * cols + c, v[i], inv);
        if (lane == 0 && at < blocks) scales[TOKENS ? scale_at(row, b, int(nb + 3) / 4) : at] = s;
    }
}
template <typename T>
constexpr int kRowsPerCta = kThreads / (kBlock / (16 / int(sizeof(T)))) * kPer;   // blocks

template <typename T>
__global__ void __launch_bounds__(kThreads)
encode_rows_kernel(const T* __restrict__ m, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                   uint32_t blocks, int64_t cols, uint32_t nb) {
    encode_rows<T, false>(m, codes, scales, blocks, cols, nb, blockIdx.x);
}

// The operands of products on FP8 blocks: CTAs for the scales' words first, then for x's blocks.
__device__ __forceinline__ void lay_out(const ScaleRows& s, int64_t i) {
    const int steps = (s.blocks + 3) / 4;
    const int64_t row = i / steps;
    if (row >= s.rows) return;
    const int st = int(i - row * steps);
    uint32_t v = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (st * 4 + k < s.blocks) v |= uint32_t(s.from[row * s.blocks + st * 4 + k]) << (8 * k);
    *reinterpret_cast<uint32_t*>(s.to + (s.tokens ? scale_at(row, st * 4, steps) : i * 4)) = v;
}
__global__ void __launch_bounds__(kThreads)
fp8_operands_kernel(const __nv_bfloat16* __restrict__ x, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                    uint32_t blocks, int64_t cols, uint32_t nb, const ScaleRows a, const ScaleRows b, int64_t ctas_a,
                    int64_t ctas_b) {
    dep_launch_dependents();
    const int64_t c = blockIdx.x;
    if (c < ctas_a) lay_out(a, c * kThreads + threadIdx.x);
    else if (c < ctas_a + ctas_b) lay_out(b, (c - ctas_a) * kThreads + threadIdx.x);
    else encode_rows<__nv_bfloat16, true>(x, codes, scales, blocks, cols, nb, uint32_t(c - ctas_a - ctas_b));
}

// Blocks of 128 rows: a CTA each, the block in registers between its maximum and its codes. 16384 x 7184 fp32 take 95
// us, 6.2 TB/s (256 threads 113 us, 1024 100).
constexpr int kTileThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kTileThreads)
encode_tiles_kernel(const T* __restrict__ m, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                    int64_t rows, int64_t cols, int64_t nb, int64_t tiles_r) {
    constexpr int kV = 16 / sizeof(T), kLanes = kBlock / kV, kRows = kTileThreads / kLanes, kN = kBlock / kRows;
    __shared__ uint32_t part[kTileThreads / 32];
    const int64_t tile = blockIdx.x, which = tile / (nb * tiles_r), r = tile / nb % tiles_r, b = tile % nb;
    const int64_t row0 = which * rows + r * kBlock;
    const int last = int(min(int64_t(kBlock), rows - r * kBlock));
    const int lane = threadIdx.x % kLanes, first = threadIdx.x / kLanes;
    const int64_t c = b * kBlock + lane * kV;
    float v[kN][kV] = {};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (c < cols && first + i * kRows < last) load16(m + (row0 + first + i * kRows) * cols + c, v[i]);
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < kV; ++j) top = max(top, block_mag(v[i][j]));
    top = __reduce_max_sync(~0u, top);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTileThreads / 32; ++i) top = max(top, part[i]);
    float inv;
    const uint8_t s = block_scale(top, inv);
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (c < cols && first + i * kRows < last)
            store_codes(codes + (row0 + first + i * kRows) * cols + c, v[i], inv);
    if (threadIdx.x == 0) scales[tile] = s;
}

template <typename T>
cudaError_t encode(int64_t n_matrix, int64_t rows, int64_t cols, int block_rows, const T* m, uint8_t* codes,
                   uint8_t* scales, cudaStream_t st) {
    const int64_t nb = ceil_div(cols, kBlock);
    if (block_rows == 1) {
        const int64_t blocks = n_matrix * rows * nb, grid = ceil_div(blocks, kRowsPerCta<T>);
        if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
        encode_rows_kernel<<<unsigned(grid), kThreads, 0, st>>>(m, codes, scales, uint32_t(blocks), cols, uint32_t(nb));
    } else {
        const int64_t tiles_r = ceil_div(rows, kBlock), grid = n_matrix * tiles_r * nb;
        if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
        encode_tiles_kernel<<<unsigned(grid), kTileThreads, 0, st>>>(m, codes, scales, rows, cols, nb, tiles_r);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_encode_blocks(int64_t n_matrix, int64_t rows, int64_t cols, int block_rows, int dtype,
                                 const void* m, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
    return dtype == GR_F32 ? encode(n_matrix, rows, cols, block_rows, static_cast<const float*>(m), codes, scales, st)
                           : encode(n_matrix, rows, cols, block_rows, static_cast<const __nv_bfloat16*>(m), codes,
                                    scales, st);
}

cudaError_t launch_fp8_operands(const void* x, int64_t n, int64_t cols, uint8_t* codes, uint8_t* token_scales,
                                const ScaleRows& a, const ScaleRows& b, cudaStream_t st) {
    auto ctas = [](const ScaleRows& s) { return ceil_div(s.rows * ((s.blocks + 3) / 4), kThreads); };
    const int64_t nb = ceil_div(cols, kBlock), blocks = x ? n * nb : 0;
    const int64_t grid = ctas(a) + ctas(b) + ceil_div(blocks, kRowsPerCta<__nv_bfloat16>);
    if (grid > 0x7fffffffLL || blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    fp8_operands_kernel<<<unsigned(grid), kThreads, 0, st>>>(static_cast<const __nv_bfloat16*>(x), codes, token_scales,
                                                             uint32_t(blocks), cols, uint32_t(nb), a, b, ctas(a), ctas(b));
    return cudaGetLastError();
}

}  // namespace gr
