// The feed-forward sublayer's products on CUDA cores: fp32 FMAs on tiles of 128 x 128, any size.
//
//     out[m][n] = Σ_k A[m][k] B[n][k]
//
// each operand with k contiguous in memory, or m (n). Both tiles go through shared memory as [k][row], 16 k at
// a time, the next ones on their way from global memory meanwhile; a thread holds 8 x 8 sums.
#include <math.h>

#include "gr_feed.h"

namespace gr {
namespace {

constexpr int kT = 128, kK = 16, kThreads = 256;

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
}

// An operand: a tile's row r at memory row row(t0, r) (negative: none), four values of it from k on.
template <typename T> struct KMajor {
    static constexpr bool kContiguousK = true;
    const T* p;
    int64_t rows, k;
    __device__ int64_t row(int64_t t0, int r) const { return t0 + r < rows ? t0 + r : -1; }
    __device__ void get(int64_t row, int64_t at, float (&v)[4]) const {
        if (row >= 0 && at < k) load4(p + row * k + at, v);
    }
};
// The gate's rows in the lower half of the tile, the up projection's in the upper: a thread has both of a channel.
template <typename T> struct GatePair {
    static constexpr bool kContiguousK = true;
    const T* p;
    int64_t f, k;
    __device__ int64_t row(int64_t t0, int r) const {
        const int64_t c = (t0 >> 1) + (r & 63);
        return c < f ? c + (r >> 6) * f : -1;
    }
    __device__ void get(int64_t row, int64_t at, float (&v)[4]) const {
        if (row >= 0 && at < k) load4(p + row * k + at, v);
    }
};
template <typename T> struct RowMajor {
    static constexpr bool kContiguousK = false;
    const T* p;
    int64_t rows, k;
    __device__ void get(int64_t row, int64_t at, float (&v)[4]) const {
        if (row < rows && at < k) load4(p + at * rows + row, v);
    }
};
// What becomes of a thread's sums of row m, columns n..n+3 and n+64.. of the tile at n0.
template <typename T> struct Store {
    T* out;
    int64_t n;
    __device__ void put(int64_t m, int64_t n0, int c, const float (&lo)[4], const float (&hi)[4]) const {
        if (n0 + c < n) store4(out + m * n + n0 + c, lo);
        if (n0 + 64 + c < n) store4(out + m * n + n0 + 64 + c, hi);
    }
};
template <typename T, typename H, int ACT> struct Gated {
    H* h;
    T* pre;
    int64_t f;
    __device__ void put(int64_t m, int64_t n0, int c, const float (&g)[4], const float (&u)[4]) const {
        const int64_t ch = n0 / 2 + c;
        if (ch >= f) return;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = activate<ACT>(g[i]) * u[i];
        store4(h + m * f + ch, v);
        if (pre) {
            store4(pre + 2 * m * f + ch, g);
            store4(pre + (2 * m + 1) * f + ch, u);
        }
    }
};
template <typename T, int ACT> struct GatedGrad {
    const T* pre;
    T *dpre, *h;
    int64_t f;
    __device__ void four(int64_t m, int64_t ch, const float (&dh)[4]) const {
        if (ch >= f) return;
        float g[4], u[4], v[4];
        load4(pre + 2 * m * f + ch, g);
        load4(pre + (2 * m + 1) * f + ch, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = dh[i] * u[i] * activate_slope<ACT>(g[i]);
        store4(dpre + 2 * m * f + ch, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = activate<ACT>(g[i]), v[i] = dh[i] * g[i];
        store4(dpre + (2 * m + 1) * f + ch, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = g[i] * u[i];
        store4(h + m * f + ch, v);
    }
    __device__ void put(int64_t m, int64_t n0, int c, const float (&lo)[4], const float (&hi)[4]) const {
        four(m, n0 + c, lo);
        four(m, n0 + 64 + c, hi);
    }
};

template <class O> __device__ __forceinline__ void fetch(const O& o, int64_t t0, int64_t k0, float (&v)[2][4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = threadIdx.x + i * kThreads;
        v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.0f;
        if constexpr (O::kContiguousK) o.get(o.row(t0, at >> 2), k0 + (at & 3) * 4, v[i]);
        else o.get(t0 + (at & 31) * 4, k0 + (at >> 5), v[i]);
    }
}
template <class O> __device__ __forceinline__ void put(float (*s)[kT + 4], const float (&v)[2][4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = threadIdx.x + i * kThreads;
        if constexpr (O::kContiguousK) {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[(at & 3) * 4 + j][at >> 2] = v[i][j];
        } else {
            *reinterpret_cast<float4*>(&s[at >> 5][(at & 31) * 4]) =
                make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        }
    }
}

// grid: the tiles, those of n first (blockIdx.x = tile of n + tiles of n · tile of m).
template <class A, class B, class E>
__global__ void __launch_bounds__(kThreads) simt_kernel(A a, B b, E e, int64_t M, int64_t tiles_n, int64_t K) {
    __shared__ __align__(16) float as[2][kK][kT + 4], bs[2][kK][kT + 4];
    const int64_t m0 = int64_t(blockIdx.x) / tiles_n * kT, n0 = int64_t(blockIdx.x) % tiles_n * kT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[8][8] = {}, ra[2][4], rb[2][4];
    fetch(a, m0, 0, ra);
    fetch(b, n0, 0, rb);
    int buf = 0;
    for (int64_t k0 = 0; k0 < K; k0 += kK, buf ^= 1) {
        put<A>(as[buf], ra);
        put<B>(bs[buf], rb);
        __syncthreads();
        if (k0 + kK < K) {
            fetch(a, m0, k0 + kK, ra);
            fetch(b, n0, k0 + kK, rb);
        }
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            float x[8], y[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 p = *reinterpret_cast<const float4*>(&as[buf][k][h * 64 + ty * 4]);
                const float4 q = *reinterpret_cast<const float4*>(&bs[buf][k][h * 64 + tx * 4]);
                x[h * 4] = p.x, x[h * 4 + 1] = p.y, x[h * 4 + 2] = p.z, x[h * 4 + 3] = p.w;
                y[h * 4] = q.x, y[h * 4 + 1] = q.y, y[h * 4 + 2] = q.z, y[h * 4 + 3] = q.w;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t m = m0 + (i >> 2) * 64 + ty * 4 + (i & 3);
        if (m >= M) continue;
        const float lo[4] = {acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
        const float hi[4] = {acc[i][4], acc[i][5], acc[i][6], acc[i][7]};
        e.put(m, n0, tx * 4, lo, hi);
    }
}

template <class A, class B, class E>
cudaError_t run(const A& a, const B& b, const E& e, int64_t M, int64_t N, int64_t K, cudaStream_t st) {
    const int64_t tn = ceil_div(N, kT), tiles = ceil_div(M, kT) * tn;
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
    simt_kernel<<<unsigned(tiles), kThreads, 0, st>>>(a, b, e, M, tn, K);
    return cudaGetLastError();
}

template <typename T, int ACT>
cudaError_t gated(int64_t N, int D, int F, const void* x, const void* w, void* h, void* pre, cudaStream_t st) {
    return run(KMajor<T>{static_cast<const T*>(x), N, D}, GatePair<T>{static_cast<const T*>(w), F, D},
               Gated<T, T, ACT>{static_cast<T*>(h), static_cast<T*>(pre), F}, N, ceil_div(F, 64) * 128, D, st);
}
template <typename T, int ACT>
cudaError_t gated_grad(int64_t N, int D, int F, const void* dy, const void* w, const void* pre, void* dpre,
                       void* h, cudaStream_t st) {
    return run(KMajor<T>{static_cast<const T*>(dy), N, D}, RowMajor<T>{static_cast<const T*>(w), F, D},
               GatedGrad<T, ACT>{static_cast<const T*>(pre), static_cast<T*>(dpre), static_cast<T*>(h), F}, N, F,
               D, st);
}
template <typename T>
cudaError_t product(int64_t M, int64_t N, int64_t K, const void* a, bool a_k, const void* b, bool b_k, void* out,
                    cudaStream_t st) {
    const Store<T> e{static_cast<T*>(out), N};
    const KMajor<T> ak{static_cast<const T*>(a), M, K}, bk{static_cast<const T*>(b), N, K};
    const RowMajor<T> am{static_cast<const T*>(a), M, K}, bn{static_cast<const T*>(b), N, K};
    if (a_k) return b_k ? run(ak, bk, e, M, N, K, st) : run(ak, bn, e, M, N, K, st);
    return b_k ? cudaErrorInvalidValue : run(am, bn, e, M, N, K, st);
}

}  // namespace

#define GR_BY_TYPE(f, ...)                                                                  \
    (dtype == GR_F32 ? (act == GR_SILU ? f<float, GR_SILU>(__VA_ARGS__)                     \
                                       : f<float, GR_GELU>(__VA_ARGS__))                    \
                     : (act == GR_SILU ? f<__nv_bfloat16, GR_SILU>(__VA_ARGS__)             \
                                       : f<__nv_bfloat16, GR_GELU>(__VA_ARGS__)))

cudaError_t simt_gated(int64_t N, int D, int F, int dtype, int act, const void* x, const void* w_in, void* h,
                       void* pre, cudaStream_t st) {
    return GR_BY_TYPE(gated, N, D, F, x, w_in, h, pre, st);
}

cudaError_t simt_gated_grad(int64_t N, int D, int F, int dtype, int act, const void* dy, const void* w_out,
                            const void* pre, void* dpre, void* h, cudaStream_t st) {
    return GR_BY_TYPE(gated_grad, N, D, F, dy, w_out, pre, dpre, h, st);
}

cudaError_t simt_product(int64_t M, int64_t N, int64_t K, int dtype, const void* a, bool a_k, const void* b,
                         bool b_k, void* out, cudaStream_t st) {
    return dtype == GR_F32 ? product<float>(M, N, K, a, a_k, b, b_k, out, st)
                           : product<__nv_bfloat16>(M, N, K, a, a_k, b, b_k, out, st);
}

}  // namespace gr
