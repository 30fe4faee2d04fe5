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

// Blocks of one row: 16 bytes a lane, so 16 lanes (bf16) or 32 (fp32) hold a block.
template <typename T>
__global__ void __launch_bounds__(kThreads)
encode_rows_kernel(const T* __restrict__ m, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                   int64_t blocks, int64_t cols, int nb, int pitch) {
    dep_launch_dependents();
    constexpr int kV = 16 / sizeof(T), kLanes = kBlock / kV;
    const int64_t at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
    const int lane = threadIdx.x % kLanes;
    const int64_t row = at / nb, c = (at - row * nb) * kBlock + lane * kV;
    const bool in = at < blocks && c < cols;
    float v[kV] = {};
    if (in) load16(m + row * cols + c, v);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kV; ++i) top = max(top, block_mag(v[i]));
#pragma unroll
    for (int d = kLanes / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
    float inv;
    const uint8_t s = block_scale(top, inv);
    if (in) store_codes(codes + row * cols + c, v, inv);
    if (lane == 0 && at < blocks) scales[row * pitch + (at - row * nb)] = s;
}

// Blocks of 128 rows: a CTA each, 64 values a thread.
template <typename T>
__global__ void __launch_bounds__(kThreads)
encode_tiles_kernel(const T* __restrict__ m, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                    int64_t rows, int64_t cols, int64_t nb, int64_t tiles_r) {
    constexpr int kV = 16 / sizeof(T), kLanes = kBlock / kV, kRows = kThreads / kLanes, kN = kBlock / kRows;
    __shared__ uint32_t part[kThreads / 32];
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
    for (int i = 0; i < kThreads / 32; ++i) top = max(top, part[i]);
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
                   uint8_t* scales, int pitch, cudaStream_t st) {
    const int64_t nb = ceil_div(cols, kBlock);
    int64_t grid;
    if (block_rows == 1) {
        const int64_t blocks = n_matrix * rows * nb;
        grid = ceil_div(blocks, kThreads / (kBlock / (16 / sizeof(T))));
        if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
        encode_rows_kernel<<<unsigned(grid), kThreads, 0, st>>>(m, codes, scales, blocks, cols, int(nb), pitch);
    } else {
        const int64_t tiles_r = ceil_div(rows, kBlock);
        grid = n_matrix * tiles_r * nb;
        if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
        encode_tiles_kernel<<<unsigned(grid), kThreads, 0, st>>>(m, codes, scales, rows, cols, nb, tiles_r);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_encode_blocks(int64_t n_matrix, int64_t rows, int64_t cols, int block_rows, int dtype,
                                 const void* m, uint8_t* codes, uint8_t* scales, int pitch, cudaStream_t st) {
    return dtype == GR_F32 ? encode(n_matrix, rows, cols, block_rows, static_cast<const float*>(m), codes, scales,
                                    pitch, st)
                           : encode(n_matrix, rows, cols, block_rows, static_cast<const __nv_bfloat16*>(m), codes,
                                    scales, pitch, st);
}

}  // namespace gr
