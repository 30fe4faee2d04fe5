// Layer norm of rows x[n][g][:], g < G groups with a weight row each (G = 1: a plain stream, G = 4:
// each branch of a state with its own gain), and its gradient.
// The norm at the end of a stack, before its logits: "Residual" (rainlin-net.pages.dev/llm-inference/residual),
// §2.2 has y = F(Norm(x)) and leaves the norm open. The Gated Residual's own norm is the RMS norm inside
// its read; a layer norm of each branch is this library's choice for a readout. (A page that normalises
// every channel stream with a LayerNorm, m.lqnn.cn/news/232857, describes another method.)
//   forward   μ = mean x, v = mean (x − μ)², r = 1/√(v + eps), x̂ = (x − μ) r, y = x̂ w_g + b_g
//   backward  u = dy w_g, dx = r (u − mean u − x̂ mean(u x̂)), dw_g = Σ_n dy x̂, db_g = Σ_n dy
//
// Both are one pass over HBM: a block holds a row in registers (16 channels a thread), the next
// row's loads are in flight while this one is reduced, and the weights stay in registers for all
// rows of the block. The variance is summed from x − μ, not as a difference of moments. The
// gradient's dw and db are summed per block in registers over its rows, written once as partial
// rows, and a second kernel adds those in a fixed order, so two runs give the same bits.
#include <math.h>

#include <atomic>

#include "gr_internal.h"
#include "gr_ptx.cuh"

namespace gr {
namespace {

constexpr int kSmall = 256, kLarge = 768;   // threads a block at most: D <= 4096, D <= 12288

// 8 channels as loaded (bf16: 4 registers, fp32: 8), so a prefetched row costs no more than its bytes.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void load_kept(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z,
        v[7] = b.w;
    }
};
template <> struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        u = __ldcs(reinterpret_cast<const uint4*>(p));
    }
    __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
};
__device__ __forceinline__ void put8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void put8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]),
                                              pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7]));
}

// Sums over the block, the same in every thread. `slot` alternates between calls (four of 32
// floats), so one barrier a call is enough: a slot is written again only after the barrier of
// the call in between.
__device__ __forceinline__ float block_sum(float v, float* slot, int warps) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) slot[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? slot[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* slot, int warps) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (warps == 1) return make_float2(a, b);
    const int lane = threadIdx.x & 31;
    if (lane == 0) slot[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 s = lane < warps ? slot[lane] : make_float2(0.0f, 0.0f);
    a = s.x, b = s.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return make_float2(a, b);
}

// A thread's two groups of 8 channels: c0 and c0 + 8·blockDim.
template <typename T> struct Row {
    Raw8<T> v[2];
    __device__ __forceinline__ void load(const T* p, int c0, int c1, int D) {
        if (c0 < D) v[0].load(p + c0);
        else v[0].zero();
        if (c1 < D) v[1].load(p + c1);
        else v[1].zero();
    }
};

template <typename T, int MAXT>
__global__ void __launch_bounds__(MAXT)
norm_kernel(int64_t N, int D, int G, float eps, const T* __restrict__ x,
            const float* __restrict__ w, const float* __restrict__ b, T* __restrict__ y,
            float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float slots[4][32];
    const int warps = blockDim.x >> 5;
    const int g = blockIdx.x % G;
    const int64_t first = blockIdx.x / G, step = gridDim.x / G;
    const int c0 = threadIdx.x * 8, c1 = c0 + blockDim.x * 8;
    Row<T> row;   // the next row, on its way (two of them ahead took 8% longer: fewer blocks an SM)
    if (first < N) row.load(x + (first * G + g) * int64_t(D), c0, c1, D);
    Raw8<float> wr[2], br[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int c = k ? c1 : c0;
        wr[k].zero();
        br[k].zero();
        if (c < D) {
            wr[k].load_kept(w + int64_t(g) * D + c);
            if (b) br[k].load_kept(b + int64_t(g) * D + c);
        }
    }
    const float inv_d = 1.0f / float(D);
    int turn = 0;
    for (int64_t n = first; n < N; n += step) {
        float v[2][8];
        row.v[0].get(v[0]);
        row.v[1].get(v[1]);
        if (n + step < N) row.load(x + ((n + step) * G + g) * int64_t(D), c0, c1, D);
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[0][k] + v[1][k];
        const float mu = block_sum(s, slots[turn], warps) * inv_d;
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if ((k ? c1 : c0) < D) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[k][j] -= mu;
                    s = fmaf(v[k][j], v[k][j], s);
                }
            }
        }
        const float var = block_sum(s, slots[turn + 1], warps) * inv_d;
        turn ^= 2;
        const float r = 1.0f / sqrtf(var + eps);
        const int64_t at = n * G + g;
        if (threadIdx.x == 0) {
            if (mean) mean[at] = mu;
            if (rstd) rstd[at] = r;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = k ? c1 : c0;
            if (c < D) {
                float wv[8], bv[8];
                wr[k].get(wv);
                br[k].get(bv);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[k][j] = fmaf(v[k][j] * r, wv[j], bv[j]);
                put8(y + at * D + c, v[k]);
            }
        }
    }
}

// part: [blocks][2 or 1][D] — the block's share of dw, then of db.
template <typename T, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == kSmall ? 2 : 1)
norm_backward_kernel(int64_t N, int D, int G, const float* __restrict__ dy,
                     const T* __restrict__ x, const float* __restrict__ w,
                     const float* __restrict__ mean, const float* __restrict__ rstd,
                     float* __restrict__ dx, float* __restrict__ part, bool bias) {
    __shared__ float2 slots[2][32];
    constexpr bool kAhead = MAXT == kSmall;   // the large block has no registers to prefetch into
    dep_launch_dependents();
    const int warps = blockDim.x >> 5;
    const int g = blockIdx.x % G;
    const int64_t first = blockIdx.x / G, step = gridDim.x / G;
    const int c0 = threadIdx.x * 8, c1 = c0 + blockDim.x * 8;
    Row<T> xr;
    Row<float> dr;
    float mu = 0.0f, r = 0.0f;
    auto fetch = [&](int64_t n) {
        const int64_t at = n * G + g;
        xr.load(x + at * D, c0, c1, D);
        dr.load(dy + at * D, c0, c1, D);
        mu = __ldg(mean + at);
        r = __ldg(rstd + at);
    };
    if (kAhead && first < N) fetch(first);
    Raw8<float> wr[2];
    float dw[2][8] = {}, db[2][8] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        wr[k].zero();
        if ((k ? c1 : c0) < D) wr[k].load_kept(w + int64_t(g) * D + (k ? c1 : c0));
    }
    const float inv_d = 1.0f / float(D);
    int turn = 0;
    for (int64_t n = first; n < N; n += step) {
        if (!kAhead) fetch(n);
        float xh[2][8], u[2][8];
        const float rn = r;
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float wv[8];
            xr.v[k].get(xh[k]);
            dr.v[k].get(u[k]);
            wr[k].get(wv);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[k][j] = (xh[k][j] - mu) * r;
                // channels past D have dy = 0 and w = 0: they add nothing anywhere
                dw[k][j] = fmaf(u[k][j], xh[k][j], dw[k][j]);
                db[k][j] += u[k][j];
                u[k][j] *= wv[j];
                s1 += u[k][j];
                s2 = fmaf(u[k][j], xh[k][j], s2);
            }
        }
        if (kAhead && n + step < N) fetch(n + step);
        const float2 m = block_sum2(s1, s2, slots[turn], warps);
        turn ^= 1;
        const float m1 = m.x * inv_d, m2 = m.y * inv_d;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = k ? c1 : c0;
            if (c < D) {
#pragma unroll
                for (int j = 0; j < 8; ++j) u[k][j] = rn * (u[k][j] - m1 - xh[k][j] * m2);
                put8(dx + (n * G + g) * D + c, u[k]);
            }
        }
    }
    float* p = part + int64_t(blockIdx.x) * (bias ? 2 : 1) * D;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int c = k ? c1 : c0;
        if (c < D) {
            put8(p + c, dw[k]);
            if (bias) put8(p + D + c, db[k]);
        }
    }
}

// dw and db: 32 channels a block, its 32 groups of 8 threads take the partial rows in turn (blocks g,
// g + G, ...) and are added up in a fixed tree. (128 channels and 8 groups a block took 12 us for the
// 304 rows of D = 4096, four times as long: too few loads in flight.)
__global__ void __launch_bounds__(256)
norm_reduce_kernel(int blocks, int D, int G, bool bias, const float* __restrict__ part,
                   float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float4 sums[8][8];
    dep_wait();
    const int col = threadIdx.x & 7, q = threadIdx.x >> 3;
    const int c = (blockIdx.x * 8 + col) * 4, g = blockIdx.y, which = blockIdx.z;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < D) {
        const int64_t rows = bias ? 2 : 1;
#pragma unroll 10
        for (int k = g + G * q; k < blocks; k += 32 * G) {
            const float4 v =
                *reinterpret_cast<const float4*>(part + (int64_t(k) * rows + which) * D + c);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, o), s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
        s.z += __shfl_xor_sync(0xffffffffu, s.z, o), s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
    }
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) < 8) sums[w][col] = s;
    __syncthreads();
    if (threadIdx.x < 8 && c < D) {
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            const float4 v = sums[k][col];
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        *reinterpret_cast<float4*>((which ? db : dw) + int64_t(g) * D + c) = s;
    }
}

int threads_of(int D) { return ((D + 15) / 16 + 31) / 32 * 32; }

// Persistent grids: a multiple of G blocks, at most what the device holds at once (asked once per
// kernel and block size; `known` is the kernel's table).
template <typename K>
int resident_blocks(K kern, std::atomic<int>* known, int threads, int G, int64_t N) {
    int per_sm = known[threads / 32].load(std::memory_order_relaxed);
    if (per_sm == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0) != cudaSuccess ||
            per_sm < 1)
            per_sm = 1;
        known[threads / 32].store(per_sm, std::memory_order_relaxed);
    }
    int64_t most = int64_t(per_sm) * sm_count() / G;
    if (most < 1) most = 1;
    return int((N < most ? N : most) * G);
}

template <typename T>
cudaError_t norm_typed(int64_t N, int D, int G, float eps, const void* x, const float* w,
                       const float* b, void* y, float* mean, float* rstd, cudaStream_t st) {
    const int threads = threads_of(D);
    auto kern = threads <= kSmall ? norm_kernel<T, kSmall> : norm_kernel<T, kLarge>;
    static std::atomic<int> known[kLarge / 32 + 1];   // by warps, which also tell the kernel
    const int blocks = resident_blocks(kern, known, threads, G, N);
    kern<<<blocks, threads, 0, st>>>(N, D, G, eps, static_cast<const T*>(x), w, b,
                                     static_cast<T*>(y), mean, rstd);
    return cudaGetLastError();
}

// Blocks of the gradient kernel: two an SM, a multiple of G. That is what its registers allow at 256 threads
// (D near 4096: 16384 rows in 117 us cold, floor 99). Narrower blocks would leave room for more of them, and
// too few rows are on their way (D = 2048: 74 us of 50, 1024: 59 of 25, 512: 49 of 12); wider ones hold no
// next row and spill 76 to 84 bytes (D = 7168: 348 of 173, 12288: 545 of 297). The bound is what the
// workspace is sized for without a device.
constexpr int kMostBlocks = 320;
int backward_blocks(int64_t N, int G) {
    int64_t most = int64_t(sm_count()) * 2;
    most = (most < kMostBlocks ? most : kMostBlocks) / G;
    if (most < 1) most = 1;
    return int((N < most ? N : most) * G);
}

}  // namespace

cudaError_t launch_layer_norm(int64_t N, int D, int G, int dtype, float eps, const void* x,
                              const float* w, const float* b, void* y, float* mean, float* rstd,
                              cudaStream_t st) {
    return dtype == GR_BF16 ? norm_typed<__nv_bfloat16>(N, D, G, eps, x, w, b, y, mean, rstd, st)
                            : norm_typed<float>(N, D, G, eps, x, w, b, y, mean, rstd, st);
}

// Two partial rows [D] a block of the largest grid.
size_t layer_norm_backward_workspace(int64_t N, int D, int G) {
    const int64_t blocks = N < kMostBlocks / G ? N * G : kMostBlocks;
    return align256(size_t(blocks) * 2 * D * 4);
}

cudaError_t launch_layer_norm_backward(int64_t N, int D, int G, int dtype, const float* dy,
                                       const void* x, const float* w, const float* mean,
                                       const float* rstd, float* dx, float* dw, float* db,
                                       void* workspace, cudaStream_t st) {
    float* part = static_cast<float*>(workspace);
    const int threads = threads_of(D);
    const bool bias = db != nullptr;
    int blocks = 0;
    if (N > 0) {
        blocks = backward_blocks(N, G);
        if (dtype == GR_BF16) {
            auto kern = threads <= kSmall ? norm_backward_kernel<__nv_bfloat16, kSmall>
                                          : norm_backward_kernel<__nv_bfloat16, kLarge>;
            kern<<<blocks, threads, 0, st>>>(N, D, G, dy, static_cast<const __nv_bfloat16*>(x), w,
                                             mean, rstd, dx, part, bias);
        } else {
            auto kern = threads <= kSmall ? norm_backward_kernel<float, kSmall>
                                          : norm_backward_kernel<float, kLarge>;
            kern<<<blocks, threads, 0, st>>>(N, D, G, dy, static_cast<const float*>(x), w, mean,
                                             rstd, dx, part, bias);
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((D + 31) / 32, G, bias ? 2 : 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = N > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, norm_reduce_kernel, blocks, D, G, bias,
                              static_cast<const float*>(part), dw, db);
}

}  // namespace gr
