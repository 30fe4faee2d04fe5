// Linear attention with a decay for each head, on CUDA cores: the chunked form for every type, head
// size and length, and the recurrent form for single tokens.
//   "【论文解读】 Qwen3.8 Flash Next" (wkq9411.github.io), §一 uses a linear-attention token mixer
//   as the sublayer F between a Gated Residual's read and write. Per sequence and head, with
//   λ = exp(log_decay_h) <= 1:
//     S_t = λ S_{t−1} + k_t v_tᵀ,   o_t = scale · S_tᵀ q_t
// The chunked form takes 32 tokens at a time: the scores of the tokens among themselves, masked and
// decayed, times the values, plus the state before the chunk read through λ^age; then the state
// moves on by the whole chunk. Everything is fp32; each output is rounded once.
#include <math.h>

#include "gr_internal.h"
#include "gr_mixer.h"

namespace gr {
namespace {

constexpr int kC = 32;      // tokens a chunk
constexpr int kCols = 64;   // columns of c (and M) a block
constexpr int kCs = kCols + 4;
constexpr int kThreads = 256;

size_t simt_smem(int da) {
    return sizeof(float) * (size_t(2) * kC * (da + 4) + size_t(kC) * kCs + size_t(kC) * (kC + 1) +
                            size_t(da) * kCs + kC + 2);
}

template <typename T>
__device__ __forceinline__ void stage_rows(const MixRows& r, int64_t row0, int len, int head, int d0,
                                           int d, int dmax, float* dst, int pitch) {
    const T* base = static_cast<const T*>(r.p) + head * r.hs + d0;
    for (int i = threadIdx.x; i < kC * d; i += kThreads) {
        const int t = i / d, c = i - t * d;
        dst[t * pitch + c] = t < len && d0 + c < dmax ? to_f32(base[(row0 + t) * r.ts + c]) : 0.0f;
    }
}

// One block a (sequence, head, 64 columns). Scores of j > i (or j < i backwards) are never formed
// into products, so what stands in a later row cannot reach an earlier output.
template <typename T>
__global__ void __launch_bounds__(kThreads) mix_simt_kernel(const MixArgs p) {
    extern __shared__ float sm[];
    const int da = p.da, ap = da + 4;
    float* A = sm;
    float* B = A + kC * ap;
    float* C = B + kC * ap;
    float* P = C + kC * kCs;
    float* M = P + kC * (kC + 1);
    float* pw = M + da * kCs;      // λ^0 .. λ^32
    const int tid = threadIdx.x;
    const int b = blockIdx.x / p.n_heads, h = blockIdx.x - b * p.n_heads;
    const int e0 = blockIdx.y * kCols;
    const int cols = min(kCols, p.dc - e0);
    const float g = p.log_decay[h];
    int64_t begin, end;
    mix_span(p, b, begin, end);
    const int64_t mbase = (int64_t(b) * p.n_heads + h) * int64_t(p.da) * p.dc;
    for (int i = tid; i <= kC; i += kThreads) pw[i] = decay_pow(g, i);
    for (int i = tid; i < da * kCs; i += kThreads) {
        const int d = i / kCs, e = i - d * kCs;
        M[i] = p.m_in && e < cols ? p.m_in[mbase + int64_t(d) * p.mr + int64_t(e0 + e) * p.mc] : 0.0f;
    }
    const int64_t chunks = (end - begin + kC - 1) / kC;
    const int ti = tid >> 4, tj = tid & 15;
    for (int64_t n = 0; n < chunks; ++n) {
        const int64_t ck = p.reverse ? chunks - 1 - n : n;
        const int64_t row0 = begin + ck * kC;
        const int len = int(min(int64_t(kC), end - row0));
        const int late = p.reverse && n == 0 ? 1 : 0;   // M_in enters the last token undecayed
        __syncthreads();
        stage_rows<T>(p.a, row0, len, h, 0, da, da, A, ap);
        stage_rows<T>(p.b, row0, len, h, 0, da, da, B, ap);
        stage_rows<T>(p.c, row0, len, h, e0, kCols, p.dc, C, kCs);
        __syncthreads();
        // scores: rows 2ti, 2ti + 1, columns tj, tj + 16
        {
            float s[2][2] = {};
            const float* a0 = A + (2 * ti) * ap;
            const float* b0 = B + tj * ap;
            for (int d = 0; d < da; d += 4) {
                const float4 x0 = *reinterpret_cast<const float4*>(a0 + d);
                const float4 x1 = *reinterpret_cast<const float4*>(a0 + ap + d);
                const float4 y0 = *reinterpret_cast<const float4*>(b0 + d);
                const float4 y1 = *reinterpret_cast<const float4*>(b0 + 16 * ap + d);
                s[0][0] = fmaf(x0.x, y0.x, fmaf(x0.y, y0.y, fmaf(x0.z, y0.z, fmaf(x0.w, y0.w, s[0][0]))));
                s[0][1] = fmaf(x0.x, y1.x, fmaf(x0.y, y1.y, fmaf(x0.z, y1.z, fmaf(x0.w, y1.w, s[0][1]))));
                s[1][0] = fmaf(x1.x, y0.x, fmaf(x1.y, y0.y, fmaf(x1.z, y0.z, fmaf(x1.w, y0.w, s[1][0]))));
                s[1][1] = fmaf(x1.x, y1.x, fmaf(x1.y, y1.y, fmaf(x1.z, y1.z, fmaf(x1.w, y1.w, s[1][1]))));
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int i = 2 * ti + x, j = tj + 16 * y;
                    const int gap = p.reverse ? j - i : i - j;
                    P[i * (kC + 1) + j] = gap >= 0 ? s[x][y] * (pw[gap] * p.weight) : 0.0f;
                }
        }
        __syncthreads();
        // outputs: rows 2ti, 2ti + 1, columns 4tj .. 4tj + 3
        {
            const int i0 = 2 * ti, e = 4 * tj;
            float o[2][4] = {}, m[2][4] = {};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int i = i0 + x;
                const int j0 = p.reverse ? i : 0, j1 = p.reverse ? len : i + 1;
                for (int j = j0; j < j1; ++j) {
                    const float w = P[i * (kC + 1) + j];
                    const float4 c = *reinterpret_cast<const float4*>(C + j * kCs + e);
                    o[x][0] = fmaf(w, c.x, o[x][0]), o[x][1] = fmaf(w, c.y, o[x][1]);
                    o[x][2] = fmaf(w, c.z, o[x][2]), o[x][3] = fmaf(w, c.w, o[x][3]);
                }
            }
            for (int d = 0; d < da; ++d) {
                const float4 s = *reinterpret_cast<const float4*>(M + d * kCs + e);
                const float a0 = A[i0 * ap + d], a1 = A[(i0 + 1) * ap + d];
                m[0][0] = fmaf(a0, s.x, m[0][0]), m[0][1] = fmaf(a0, s.y, m[0][1]);
                m[0][2] = fmaf(a0, s.z, m[0][2]), m[0][3] = fmaf(a0, s.w, m[0][3]);
                m[1][0] = fmaf(a1, s.x, m[1][0]), m[1][1] = fmaf(a1, s.y, m[1][1]);
                m[1][2] = fmaf(a1, s.z, m[1][2]), m[1][3] = fmaf(a1, s.w, m[1][3]);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int i = i0 + x;
                if (i < len && e < cols) {
                    const float w = pw[p.reverse ? len - i - late : i + 1];
                    T* dst = static_cast<T*>(p.out.p) + (row0 + i) * p.out.ts + h * p.out.hs + e0 + e;
#pragma unroll
                    for (int k = 0; k < 4; ++k) dst[k] = from_f32<T>(p.outer * fmaf(w, m[x][k], o[x][k]));
                }
            }
        }
        __syncthreads();
        // the state: rows ti + 16k (four at a time), columns 4tj .. 4tj + 3
        {
            const float keep = pw[len - late];
            const int e = 4 * tj;
            for (int d0 = ti; d0 < da; d0 += 64) {
                float m[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int d = d0 + 16 * k;
                    const float4 s = d < da ? *reinterpret_cast<const float4*>(M + d * kCs + e)
                                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    m[k][0] = keep * s.x, m[k][1] = keep * s.y, m[k][2] = keep * s.z,
                    m[k][3] = keep * s.w;
                }
                for (int j = 0; j < len; ++j) {
                    const float w = p.weight * pw[p.reverse ? j : len - 1 - j];
                    const float4 c = *reinterpret_cast<const float4*>(C + j * kCs + e);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int d = d0 + 16 * k;
                        const float x = d < da ? B[j * ap + d] * w : 0.0f;
                        m[k][0] = fmaf(x, c.x, m[k][0]), m[k][1] = fmaf(x, c.y, m[k][1]);
                        m[k][2] = fmaf(x, c.z, m[k][2]), m[k][3] = fmaf(x, c.w, m[k][3]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int d = d0 + 16 * k;
                    if (d < da)
                        *reinterpret_cast<float4*>(M + d * kCs + e) =
                            make_float4(m[k][0], m[k][1], m[k][2], m[k][3]);
                }
            }
        }
    }
    __syncthreads();
    if (p.m_out) {
        // backwards, λ once more takes the gradient to the state before the first token (an empty
        // sequence passes its state through)
        const float last = p.reverse && chunks > 0 ? decay_pow(g, 1) : 1.0f;
        for (int i = tid; i < da * kCs; i += kThreads) {
            const int d = i / kCs, e = i - d * kCs;
            if (e < cols) p.m_out[mbase + int64_t(d) * p.mr + int64_t(e0 + e) * p.mc] = last * M[i];
        }
    }
}

// One token of one request and head a block: the state [dk][dv] passes through registers once
// (S' = λ S + k vᵀ, written back), four columns a thread, and o = scale · qᵀ S' is summed over the
// rows in registers and then over the block's row groups in order.
template <typename T>
__global__ void __launch_bounds__(kThreads)
mix_step_kernel(int n_heads, int dk, int dv, float scale, MixRows q, MixRows k, MixRows v,
                const float* __restrict__ log_decay, float* __restrict__ state, int64_t n_slots,
                const int32_t* __restrict__ slots, MixRows o) {
    __shared__ float qs[256], ks[256];
    __shared__ float4 sums[kThreads];
    const int64_t n = blockIdx.x / n_heads;
    const int h = int(blockIdx.x - n * n_heads), tid = threadIdx.x;
    const int64_t slot = slots ? int64_t(slots[n]) : n;
    T* out = static_cast<T*>(o.p) + n * o.ts + h * o.hs;
    if (slot < 0 || slot >= n_slots) {
        for (int e = tid; e < dv; e += blockDim.x) out[e] = from_f32<T>(0.0f);
        return;
    }
    const int vecs = dv >> 2, groups = blockDim.x / vecs;
    const int cg = tid % vecs, rg = tid / vecs;
    float4* S = reinterpret_cast<float4*>(state + (slot * n_heads + h) * int64_t(dk) * dv) + cg;
    for (int d = tid; d < dk; d += blockDim.x) {
        qs[d] = to_f32((static_cast<const T*>(q.p) + n * q.ts + h * q.hs)[d]);
        ks[d] = to_f32((static_cast<const T*>(k.p) + n * k.ts + h * k.hs)[d]);
    }
    const T* vp = static_cast<const T*>(v.p) + n * v.ts + h * v.hs + 4 * cg;
    const float4 ve = make_float4(to_f32(vp[0]), to_f32(vp[1]), to_f32(vp[2]), to_f32(vp[3]));
    const float lam = decay_pow(log_decay[h], 1);
    __syncthreads();
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int kU = 8;   // rows in flight a thread
    for (int d0 = rg; d0 < dk; d0 += kU * groups) {
        float4 s[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int d = d0 + u * groups;
            if (d < dk) s[u] = S[int64_t(d) * vecs];
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int d = d0 + u * groups;
            if (d < dk) {
                const float kd = ks[d], qd = qs[d];
                s[u].x = fmaf(lam, s[u].x, kd * ve.x), s[u].y = fmaf(lam, s[u].y, kd * ve.y);
                s[u].z = fmaf(lam, s[u].z, kd * ve.z), s[u].w = fmaf(lam, s[u].w, kd * ve.w);
                S[int64_t(d) * vecs] = s[u];
                acc.x = fmaf(qd, s[u].x, acc.x), acc.y = fmaf(qd, s[u].y, acc.y);
                acc.z = fmaf(qd, s[u].z, acc.z), acc.w = fmaf(qd, s[u].w, acc.w);
            }
        }
    }
    sums[tid] = acc;
    __syncthreads();
    if (rg == 0) {
        for (int r = 1; r < groups; ++r) {
            const float4 x = sums[r * vecs + cg];
            acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
        }
        out[4 * cg] = from_f32<T>(scale * acc.x), out[4 * cg + 1] = from_f32<T>(scale * acc.y);
        out[4 * cg + 2] = from_f32<T>(scale * acc.z), out[4 * cg + 3] = from_f32<T>(scale * acc.w);
    }
}

}  // namespace

cudaError_t launch_mix_simt(const MixArgs& p, cudaStream_t st) {
    if (p.n_seqs == 0) return cudaSuccess;
    const size_t smem = simt_smem(p.da);
    auto kern = p.dtype == GR_BF16 ? mix_simt_kernel<__nv_bfloat16> : mix_simt_kernel<float>;
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    const dim3 grid(unsigned(p.n_seqs) * p.n_heads, (p.dc + kCols - 1) / kCols);
    kern<<<grid, kThreads, smem, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_mix_step(int64_t n, int n_heads, int dk, int dv, int dtype, float scale,
                            MixRows q, MixRows k, MixRows v, const float* log_decay, float* state,
                            int64_t n_slots, const int32_t* slots, MixRows o, cudaStream_t st) {
    const int vecs = dv / 4;
    const int threads = kThreads / vecs * vecs;
    auto kern = dtype == GR_BF16 ? mix_step_kernel<__nv_bfloat16> : mix_step_kernel<float>;
    kern<<<unsigned(n * n_heads), threads, 0, st>>>(n_heads, dk, dv, scale, q, k, v, log_decay, state,
                                                    n_slots, slots, o);
    return cudaGetLastError();
}

}  // namespace gr
