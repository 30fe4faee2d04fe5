// Linear attention with a decay for each head, on CUDA cores: the chunked form for every type, head
// size and length, and the recurrent form for single tokens.
//   "【论文解读】 Qwen3.8 Flash Next" (wkq9411.github.io), §一 uses a linear-attention token mixer
//   as the sublayer F between a Gated Residual's read and write. Per sequence and head, with
//   λ = exp(log_decay_h) <= 1:
//     S_t = λ S_{t−1} + k_t v_tᵀ,   o_t = scale · S_tᵀ q_t
// The chunked form takes 64 tokens at a time (32 where the head is wider than 128): the scores of the
// tokens among themselves, masked and decayed, times the values, plus the state before the chunk read
// through λ^age; then the state moves on by the whole chunk. Everything is fp32; each output is rounded
// once. A block holds 64 columns of the values and the state; every product is a 4 × 4 (2 × 4) tile a
// thread from 16-byte reads of shared memory, which then keep up with the fp32 units (scalar reads of a
// 2 × 4 tile took five times as long). Long prompts of few heads are cut into segments as on the tensor
// cores.
#include <math.h>
#include <string.h>

#include "gr_internal.h"
#include "gr_mixer.h"
#include "gr_ptx.cuh"

namespace gr {
namespace {

constexpr int kCols = 64;   // columns of c (and M) a block
constexpr int kCs = kCols + 4;
constexpr int kThreads = 256;

int chunk_of(int da) { return da <= 128 ? 64 : 32; }

size_t simt_smem(int da) {
    const size_t c = chunk_of(da);
    return sizeof(float) * (2 * c * (da + 4) + c * kCs + c * (c + 4) + size_t(da) * kCs + c + 4);
}

// Rows row0 .. row0 + len of one head's channels d0 .. d0 + d as fp32, eight at a time; zeros behind.
template <typename T>
__device__ __forceinline__ void stage_rows(const MixRows& r, int64_t row0, int rows, int len, int head,
                                           int d0, int d, int dmax, float* dst, int pitch) {
    const T* base = static_cast<const T*>(r.p) + head * r.hs + d0;
    const int per = d / 8;
    for (int i = threadIdx.x; i < rows * per; i += kThreads) {
        const int t = i / per, c = (i - t * per) * 8;
        float v[8] = {};
        if (t < len && d0 + c < dmax) {
            const T* s = base + (row0 + t) * r.ts + c;
            if constexpr (sizeof(T) == 2) {
                const uint4 u = *reinterpret_cast<const uint4*>(s);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) unf2(bf2_to_f2(w[k]), v[2 * k], v[2 * k + 1]);
            } else {
                const float4 a = reinterpret_cast<const float4*>(s)[0];
                const float4 b = reinterpret_cast<const float4*>(s)[1];
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z,
                v[7] = b.w;
            }
        }
        float4* q = reinterpret_cast<float4*>(dst + t * pitch + c);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}
__device__ __forceinline__ void add4(float (&o)[4], float w, float4 c) {
    o[0] = fmaf(w, c.x, o[0]), o[1] = fmaf(w, c.y, o[1]);
    o[2] = fmaf(w, c.z, o[2]), o[3] = fmaf(w, c.w, o[3]);
}

struct Pass {
    MixArgs p;
    Segments sg;
    float *slots, *firsts;
};

// One block a (segment, head, 64 columns). Scores of j > i (or j < i backwards) are zero and their
// products are left out, so what stands in a later row cannot reach an earlier output. kSum: only the
// segment's own sum, written to its slot.
template <typename T, int kC, bool kSum>
__global__ void __launch_bounds__(kThreads) mix_simt_kernel(const __grid_constant__ Pass L) {
    constexpr int kR = kC / 16;          // rows a thread
    constexpr int kP = kC + 4;
    const MixArgs& p = L.p;
    extern __shared__ __align__(16) float sm[];
    const int da = p.da, ap = da + 4;
    float* A = sm;
    float* B = A + kC * ap;
    float* C = B + kC * ap;
    float* P = C + kC * kCs;
    float* M = P + kC * kP;
    float* pw = M + da * kCs;            // λ^0 .. λ^kC
    __shared__ int found[4];
    const int tid = threadIdx.x, h = blockIdx.x % p.n_heads;
    if (tid < 32) {
        int seq = 0, seg = 0, index = 0;
        const bool ok = find_segment<kSum>(p, L.sg, blockIdx.x / p.n_heads, seq, seg, index);
        if (tid == 0) found[0] = ok, found[1] = seq, found[2] = seg, found[3] = index;
    }
    __syncthreads();
    if (kSum) dep_launch_dependents();
    if (!found[0]) return;   // the grid is an upper bound
    const int b = found[1], seg = found[2];
    const int e0 = blockIdx.y * kCols;
    const int cols = min(kCols, p.dc - e0);
    const float g = p.log_decay[h];
    int64_t begin, end;
    mix_span(p, b, begin, end);
    const int64_t all = (end - begin + kC - 1) / kC, n0 = int64_t(seg) * L.sg.per_seg;
    const int64_t n1 = min(all, n0 + L.sg.per_seg);
    const bool last = n0 + L.sg.per_seg >= all;
    const int64_t one = int64_t(p.da) * p.dc, mbase = (int64_t(b) * p.n_heads + h) * one;
    float* const slot = L.slots + (int64_t(found[3]) * p.n_heads + h) * one;
    // the state before the segment: its predecessor's slot, m_in, or m_in's copy
    const float* from = seg > 0 ? slot - p.n_heads * one : p.m_in ? p.m_in + mbase : nullptr;
    int mr = seg > 0 ? p.dc : p.mr, mc = seg > 0 ? 1 : p.mc;
    if (seg == 0 && !last && L.firsts) from = L.firsts + mbase, mr = p.dc, mc = 1;
    for (int i = tid; i <= kC; i += kThreads) pw[i] = decay_pow(g, i);
    for (int i = tid; i < da * kCs; i += kThreads) {
        const int d = i / kCs, e = i - d * kCs;
        M[i] = !kSum && from && e < cols ? from[int64_t(d) * mr + int64_t(e0 + e) * mc] : 0.0f;
    }
    const int ti = tid >> 4, tj = tid & 15;
    for (int64_t n = n0; n < n1; ++n) {
        const int64_t ck = p.reverse ? all - 1 - n : n;
        const int64_t row0 = begin + ck * kC;
        const int len = int(min(int64_t(kC), end - row0));
        const int late = p.reverse && n == 0 ? 1 : 0;   // M_in enters the last token undecayed
        __syncthreads();
        if (!kSum) stage_rows<T>(p.a, row0, kC, len, h, 0, da, da, A, ap);
        stage_rows<T>(p.b, row0, kC, len, h, 0, da, da, B, ap);
        stage_rows<T>(p.c, row0, kC, len, h, e0, kCols, p.dc, C, kCs);
        __syncthreads();
        if (!kSum) {
            // scores: rows ti·kR .., columns tj + 16y
            float s[kR][kR] = {};
            const float* a0 = A + ti * kR * ap;
            const float* b0 = B + tj * ap;
            for (int d = 0; d < da; d += 4) {
                float4 x[kR], y[kR];
#pragma unroll
                for (int k = 0; k < kR; ++k) x[k] = ld4(a0 + k * ap + d), y[k] = ld4(b0 + 16 * k * ap + d);
#pragma unroll
                for (int k = 0; k < kR; ++k)
#pragma unroll
                    for (int l = 0; l < kR; ++l) s[k][l] = dot4(x[k], y[l], s[k][l]);
            }
#pragma unroll
            for (int k = 0; k < kR; ++k)
#pragma unroll
                for (int l = 0; l < kR; ++l) {
                    const int i = ti * kR + k, j = tj + 16 * l;
                    const int gap = p.reverse ? j - i : i - j;
                    P[i * kP + j] = gap >= 0 ? s[k][l] * (pw[gap] * p.weight) : 0.0f;
                }
            __syncthreads();
            // outputs: rows ti·kR .., columns 4tj .. 4tj + 3
            const int i0 = ti * kR, e = 4 * tj;
            float o[kR][4] = {}, m[kR][4] = {};
            // the columns every row of the tile takes kR at a time (where the tiles begin), the tile's own
            // one by one
            const int j0 = p.reverse ? i0 + kR : 0, j1 = p.reverse ? len : i0;
            for (int j = j0; j < j1; j += kR) {
                float w[kR][kR];
#pragma unroll
                for (int k = 0; k < kR; ++k) {
                    const float* q = P + (i0 + k) * kP + j;
                    if constexpr (kR == 4) {
                        const float4 v = ld4(q);
                        w[k][0] = v.x, w[k][1] = v.y, w[k][2] = v.z, w[k][3] = v.w;
                    } else {
#pragma unroll
                        for (int l = 0; l < kR; ++l) w[k][l] = q[l];
                    }
                }
#pragma unroll
                for (int l = 0; l < kR; ++l) {
                    // (rows past the sequence's end are zero in C, and in P's columns)
                    const float4 c = ld4(C + (j + l) * kCs + e);
#pragma unroll
                    for (int k = 0; k < kR; ++k) add4(o[k], w[k][l], c);
                }
            }
#pragma unroll
            for (int l = 0; l < kR; ++l) {
                const float4 c = ld4(C + (i0 + l) * kCs + e);
#pragma unroll
                for (int k = 0; k < kR; ++k)
                    if (p.reverse ? l >= k : l <= k) add4(o[k], P[(i0 + k) * kP + i0 + l], c);
            }
            for (int d = 0; d < da; d += 4) {
                float4 x[kR];
#pragma unroll
                for (int k = 0; k < kR; ++k) x[k] = ld4(A + (i0 + k) * ap + d);
#pragma unroll
                for (int l = 0; l < 4; ++l) {
                    const float4 s4 = ld4(M + (d + l) * kCs + e);
#pragma unroll
                    for (int k = 0; k < kR; ++k)
                        add4(m[k], l == 0 ? x[k].x : l == 1 ? x[k].y : l == 2 ? x[k].z : x[k].w, s4);
                }
            }
#pragma unroll
            for (int k = 0; k < kR; ++k) {
                const int i = i0 + k;
                if (i < len && e < cols) {
                    const float w = pw[p.reverse ? len - i - late : i + 1];
                    T* dst = static_cast<T*>(p.out.p) + (row0 + i) * p.out.ts + h * p.out.hs + e0 + e;
                    float v[4];
#pragma unroll
                    for (int l = 0; l < 4; ++l) v[l] = p.outer * fmaf(w, m[k][l], o[k][l]);
                    if constexpr (sizeof(T) == 2)
                        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]));
                    else
                        *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
                }
            }
            __syncthreads();
        }
        // the state: rows 4ti + 64k .., columns 4tj .. 4tj + 3
        const float keep = pw[len - late];
        const int e = 4 * tj;
        for (int d = 4 * ti; d < da; d += 64) {
            float m[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 s = ld4(M + (d + k) * kCs + e);
                m[k][0] = keep * s.x, m[k][1] = keep * s.y, m[k][2] = keep * s.z, m[k][3] = keep * s.w;
            }
#pragma unroll 4
            for (int j = 0; j < len; ++j) {
                const float w = p.weight * pw[p.reverse ? j : len - 1 - j];
                const float4 x = ld4(B + j * ap + d), c = ld4(C + j * kCs + e);
                add4(m[0], x.x * w, c), add4(m[1], x.y * w, c), add4(m[2], x.z * w, c), add4(m[3], x.w * w, c);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<float4*>(M + (d + k) * kCs + e) =
                    make_float4(m[k][0], m[k][1], m[k][2], m[k][3]);
        }
    }
    __syncthreads();
    if (kSum || (last && p.m_out)) {
        // backwards, λ once more takes the gradient to the state before the first token (an empty
        // sequence passes its state through)
        const float w = !kSum && p.reverse && all > 0 ? decay_pow(g, 1) : 1.0f;
        float* to = kSum ? slot : p.m_out + mbase;
        const int tr = kSum ? p.dc : p.mr, tc = kSum ? 1 : p.mc;
        for (int i = tid; i < da * kCs; i += kThreads) {
            const int d = i / kCs, e = i - d * kCs;
            if (e < cols) to[int64_t(d) * tr + int64_t(e0 + e) * tc] = w * M[i];
        }
    }
}

struct Scan {
    MixArgs pass[kMostPasses];
    Segments sg;
    float *slots, *firsts;
    int64_t units;
};

// The segments' sums to the states after them: one thread four elements of a (cut sequence, head), the
// loads of four segments on their way together.
__global__ void __launch_bounds__(256) mix_scan_kernel(const __grid_constant__ Scan L) {
    const MixArgs& p = L.pass[blockIdx.z];
    const Segments sg = L.sg;
    float* const firsts = p.m_in && p.m_in == p.m_out ? L.firsts : nullptr;
    const int want = blockIdx.x / p.n_heads, h = blockIdx.x - want * p.n_heads;
    const int one = p.da * p.dc;
    float* const slots = L.slots + int64_t(blockIdx.z) * L.units * one;
    const int at = (blockIdx.y * 256 + threadIdx.x) * 4;
    // the want-th of the sequences that are cut, and the segments before its own
    __shared__ int found;
    __shared__ int64_t segments_before;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int seq = -1, cut = 0;
        int64_t before = 0;
        for (int b0 = 0; b0 < p.n_seqs && seq < 0; b0 += 32) {
            int n = 0;
            if (b0 + lane < p.n_seqs) {
                int64_t x, y;
                mix_span(p, b0 + lane, x, y);
                n = sg.count(x, y);
            }
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            const unsigned cuts = __ballot_sync(0xffffffffu, n > 1);
            const int mine = cut + __popc(cuts & ((1u << lane) - 1u));
            const unsigned hit = __ballot_sync(0xffffffffu, n > 1 && mine == want);
            if (hit) {
                const int l = __ffs(hit) - 1;
                seq = b0 + l;
                before += __shfl_sync(0xffffffffu, inc - n, l);
            } else {
                before += __shfl_sync(0xffffffffu, inc, 31);
                cut += __popc(cuts);
            }
        }
        if (lane == 0) found = seq, segments_before = before;
    }
    __syncthreads();
    const int b = found;
    const int64_t first = segments_before;
    if (b < 0 || at >= one) return;   // the grid is an upper bound
    dep_wait();
    int64_t begin, end;
    mix_span(p, b, begin, end);
    const int n = sg.count(begin, end);
    // starts that do not ascend may name more segments than the workspace has slots
    if ((first + n) * p.n_heads > L.units) return;
    const float g = p.log_decay[h];
    float m[4] = {};
    if (p.m_in) {
        const float* s = p.m_in + (int64_t(b) * p.n_heads + h) * one;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = (at + k) / p.dc, j = (at + k) - i * p.dc;
            m[k] = s[int64_t(i) * p.mr + int64_t(j) * p.mc];
        }
    }
    if (firsts)
        *reinterpret_cast<float4*>(firsts + (int64_t(b) * p.n_heads + h) * one + at) =
            make_float4(m[0], m[1], m[2], m[3]);
    const int64_t full = int64_t(sg.per_seg) * sg.chunk;
    // backwards the first segment holds the sequence's partial chunk, and its state enters undecayed
    const int64_t chunks = (end - begin + sg.chunk - 1) / sg.chunk;
    const int64_t len0 = p.reverse ? full - (chunks * sg.chunk - (end - begin)) - 1 : full;
    const float l0 = decay_pow(g, len0), lf = decay_pow(g, full);
    const int64_t step = int64_t(p.n_heads) * one;
    float* s = slots + (first * p.n_heads + h) * one + at;
    constexpr int kU = 4;
    for (int i = 0; i < n - 1; i += kU) {
        float4 v[kU];
#pragma unroll
        for (int k = 0; k < kU; ++k)
            if (i + k < n - 1) v[k] = __ldcg(reinterpret_cast<const float4*>(s + (i + k) * step));
#pragma unroll
        for (int k = 0; k < kU; ++k)
            if (i + k < n - 1) {
                const float w = i + k == 0 ? l0 : lf;
                m[0] = fmaf(w, m[0], v[k].x), m[1] = fmaf(w, m[1], v[k].y);
                m[2] = fmaf(w, m[2], v[k].z), m[3] = fmaf(w, m[3], v[k].w);
                *reinterpret_cast<float4*>(s + (i + k) * step) = make_float4(m[0], m[1], m[2], m[3]);
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

cudaError_t launch_mix_scan(const MixArgs* pass, int passes, const Segments& sg, float* slots,
                            float* firsts, int64_t units, cudaStream_t st) {
    Scan L;
    memset(&L, 0, sizeof(L));
    for (int i = 0; i < passes; ++i) L.pass[i] = pass[i];
    L.sg = sg;
    L.slots = slots;
    L.firsts = firsts;
    L.units = units;
    const unsigned sums = mix_sums(pass->n_tokens, pass->n_heads, sg);
    const unsigned rows = unsigned(pass->n_seqs) * pass->n_heads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sums < rows ? sums : rows, (pass->da * pass->dc + 1023) / 1024, passes);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mix_scan_kernel, L);
}

namespace {

Segments simt_plan(int64_t N, int n_seqs, int H, int da, int dc) {
    return mix_plan(N, n_seqs, int64_t(H) * ((dc + kCols - 1) / kCols), chunk_of(da));
}

template <typename T, int kC> cudaError_t simt(const MixArgs& p, float* slots, cudaStream_t st) {
    Pass L;
    memset(&L, 0, sizeof(L));
    L.p = p;
    L.sg = simt_plan(p.n_tokens, p.n_seqs, p.n_heads, p.da, p.dc);
    L.slots = slots;
    const int64_t units = mix_units(p.n_tokens, p.n_seqs, p.n_heads, L.sg);
    const size_t smem = simt_smem(p.da);
    const unsigned slices = (p.dc + kCols - 1) / kCols;
    auto kern = mix_simt_kernel<T, kC, false>;
    auto sum = mix_simt_kernel<T, kC, true>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e == cudaSuccess && mix_cuts(p.n_tokens, L.sg)) {
        if (p.m_in && p.m_in == p.m_out) L.firsts = slots + units * p.da * int64_t(p.dc);
        e = cudaFuncSetAttribute(sum, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
        sum<<<dim3(mix_sums(p.n_tokens, p.n_heads, L.sg), slices), kThreads, smem, st>>>(L);
        e = cudaGetLastError();
        if (e == cudaSuccess) e = launch_mix_scan(&p, 1, L.sg, slots, L.firsts, units, st);
    }
    if (e != cudaSuccess) return e;
    kern<<<dim3(unsigned(units), slices), kThreads, smem, st>>>(L);
    return cudaGetLastError();
}

}  // namespace

// The slots and a copy of the first states.
size_t mix_simt_workspace(int64_t N, int n_seqs, int H, int da, int dc) {
    if (N == 0 || n_seqs == 0) return 0;
    const Segments sg = simt_plan(N, n_seqs, H, da, dc);
    if (!mix_cuts(N, sg)) return 0;
    return align256(size_t(mix_units(N, n_seqs, H, sg) + int64_t(n_seqs) * H) * da * dc * 4);
}

cudaError_t launch_mix_simt(const MixArgs& p, void* workspace, cudaStream_t st) {
    if (p.n_seqs == 0) return cudaSuccess;
    float* slots = static_cast<float*>(workspace);
    if (chunk_of(p.da) == 64)
        return p.dtype == GR_BF16 ? simt<__nv_bfloat16, 64>(p, slots, st) : simt<float, 64>(p, slots, st);
    return p.dtype == GR_BF16 ? simt<__nv_bfloat16, 32>(p, slots, st) : simt<float, 32>(p, slots, st);
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
