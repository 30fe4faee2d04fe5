// The state a stack starts from and the gradient of the table it comes from.
//   "【论文解读】 Qwen3.8 Flash Next" (wkq9411.github.io), §二.6 starts every branch at the token's
//   embedding: R_i^(0)[t] = scale · E[id_t], i = 0..n_b-1 (n_b = 4, or 1 for a plain stream).
//   Its gradient: dE[v] = scale · Σ_{t: id_t = v} Σ_i dR_i[t].
// An id outside [0, V) reads no row (its state is zero) and has no gradient.
//
// The gradient is summed by sorted tokens, so no atomics touch it and two runs give the same bits:
//   1. sort_fill_kernel   one CTA a tile of <= 16384 tokens sorts (id, position) by id, stably, in
//                         shared memory; the other CTAs zero dE meanwhile (the sort hides there).
//   2. run_sum_kernel     pieces of consecutive sorted positions × 512 channels: the rows of a run
//                         (equal ids) are summed in registers in ascending t. A run inside the piece
//                         goes to dE, one that crosses the piece's ends leaves a partial row.
//   3. run_join_kernel    the piece a crossing run starts in adds up the run's partial rows, always in
//                         the same order.
// Tiles after the first add to dE, one after another.
#include <math.h>

#include "gr_internal.h"
#include "gr_ptx.cuh"

namespace gr {
namespace {

// ---- lookup ---------------------------------------------------------------------------------------

template <typename T> __device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <> __device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}

template <typename T> struct Vec8;
template <> struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ explicit Vec8(const float (&v)[8])
        : a(make_float4(v[0], v[1], v[2], v[3])), b(make_float4(v[4], v[5], v[6], v[7])) {}
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
};
template <> struct Vec8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ explicit Vec8(const float (&v)[8])
        : u(make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]),
                       pack_bf2(v[6], v[7]))) {}
    __device__ __forceinline__ void store(__nv_bfloat16* p) const {
        *reinterpret_cast<uint4*>(p) = u;
    }
};

// A warp a token, 8 channels a lane and step: one 16-byte (bf16) or 32-byte (fp32) read of the
// row, scaled in fp32 and rounded once, then one store a branch.
template <typename TI, typename TE, typename TR, int NB>
__global__ void __launch_bounds__(256)
embed_kernel(int64_t N, int64_t V, int D, float scale, const TI* __restrict__ ids,
             const TE* __restrict__ E, TR* __restrict__ R, int split) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t = unit / split;
    const int part = int(unit - t * split);
    if (t >= N) return;
    const int64_t id = int64_t(ids[t]);
    const bool in = id >= 0 && id < V;
    const TE* row = E + (in ? id : 0) * D;
    TR* out = R + t * NB * int64_t(D);
#pragma unroll 2
    for (int c = (part * 32 + lane) * 8; c < D; c += split * 256) {
        float v[8] = {};
        if (in) {
            load8(row + c, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= scale;
        }
        const Vec8<TR> o(v);
#pragma unroll
        for (int i = 0; i < NB; ++i) o.store(out + int64_t(i) * D + c);
    }
}

template <typename TI, typename TE, typename TR>
void embed_nb(int64_t N, int64_t V, int D, int nb, float scale, const void* ids, const void* E,
              void* R, cudaStream_t st) {
    // warps a token: enough of them that a few tokens still spread over the SMs
    int split = 1;
    while (split * 256 < D && N * split < int64_t(sm_count()) * 32) split *= 2;
    const int64_t blocks = (N * split + 7) / 8;
    const TI* i = static_cast<const TI*>(ids);
    const TE* e = static_cast<const TE*>(E);
    TR* r = static_cast<TR*>(R);
    if (nb == 1)
        embed_kernel<TI, TE, TR, 1><<<unsigned(blocks), 256, 0, st>>>(N, V, D, scale, i, e, r, split);
    else
        embed_kernel<TI, TE, TR, 4><<<unsigned(blocks), 256, 0, st>>>(N, V, D, scale, i, e, r, split);
}

template <typename TI>
void embed_types(int64_t N, int64_t V, int D, int nb, int table_dtype, int state_dtype,
                 float scale, const void* ids, const void* E, void* R, cudaStream_t st) {
    using B = __nv_bfloat16;
    if (table_dtype == GR_F32 && state_dtype == GR_F32)
        embed_nb<TI, float, float>(N, V, D, nb, scale, ids, E, R, st);
    else if (table_dtype == GR_F32)
        embed_nb<TI, float, B>(N, V, D, nb, scale, ids, E, R, st);
    else if (state_dtype == GR_F32)
        embed_nb<TI, B, float>(N, V, D, nb, scale, ids, E, R, st);
    else
        embed_nb<TI, B, B>(N, V, D, nb, scale, ids, E, R, st);
}

// ---- the gradient's sort ------------------------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortItems = 16;                          // a thread's items at most
constexpr int kSortTile = kSortThreads * kSortItems;    // 16384: tokens of one tile
constexpr int kSortBits = 5;
constexpr int kDigits = 1 << kSortBits;
// Items lie in shared memory with a gap after every 16, so that threads reading 16 in a row meet no
// bank twice.
__device__ __forceinline__ int at(int i) { return i + (i >> 4); }
constexpr int kSortSlots = kSortTile + kSortTile / 16;
// keys, positions, the threads' digit counts, the scan's warp sums
constexpr size_t kSortSmem =
    size_t(kSortSlots) * 6 + size_t(kDigits) * kSortThreads * 2 + 32 * sizeof(uint32_t);

// Stable radix sort of a tile's (id, position), 5 bits a pass, least significant first. A thread holds
// consecutive items and counts its own digits one after another, so an item's rank among its thread's
// equal digits comes with the count, and a scan of the counts in (digit, thread) order gives the
// places: warp d scans digit d's counts. Few items take few of the threads, 4 to 8 each. (Ranks from warp-wide matches of 8-bit digits took 56 us for 16384 uniform ids of 15 bits: a
// match costs a step for every distinct digit in the warp.) Ids outside [0, V) take the key V.
template <typename TI>
__device__ void sort_tile(const TI* __restrict__ ids, int64_t V, int n, int passes,
                          uint32_t* __restrict__ out_id, uint32_t* __restrict__ out_pos, char* smem) {
    uint32_t* skey = reinterpret_cast<uint32_t*>(smem);
    uint16_t* spos = reinterpret_cast<uint16_t*>(smem + size_t(kSortSlots) * 4);
    uint16_t* cnt = reinterpret_cast<uint16_t*>(smem + size_t(kSortSlots) * 6);   // [digit][thread]
    uint32_t* wsum = reinterpret_cast<uint32_t*>(cnt + size_t(kDigits) * kSortThreads);
    static_assert(kDigits == kSortThreads / 32, "a warp a digit");
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    int holders = 32;                                   // threads that hold items
    while (holders < kSortThreads && holders * 8 < n) holders *= 2;
    const int per = (n + holders - 1) / holders;        // items of each
    const bool holds = tid < holders;
    for (int i = tid; i < per * holders; i += kSortThreads) {
        uint32_t key = 0xffffffffu;   // past the tile: sorts behind every key and is not written
        if (i < n) {
            const int64_t id = int64_t(ids[i]);
            key = uint32_t(id >= 0 && id < V ? id : V);
        }
        skey[at(i)] = key;
        spos[at(i)] = uint16_t(i);
    }
    const int quads = holders / 8;                      // 16-byte groups of a digit's counts
    uint4* const counts = reinterpret_cast<uint4*>(cnt);
    for (int p = 0; p < passes; ++p) {
        for (int i = tid; i < kDigits * quads; i += kSortThreads) counts[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        uint32_t key[kSortItems];
        uint32_t pos[kSortItems / 2], rank[kSortItems / 4];   // two and four to a register
        if (holds) {
#pragma unroll
            for (int j = 0; j < kSortItems; ++j) {
                if (j % 2 == 0) pos[j / 2] = 0;
                if (j % 4 == 0) rank[j / 4] = 0;
                if (j < per) {
                    const int i = at(tid * per + j);
                    key[j] = skey[i];
                    pos[j / 2] |= uint32_t(spos[i]) << (16 * (j & 1));
                    uint16_t* c = cnt + ((key[j] >> (kSortBits * p)) & (kDigits - 1)) * holders + tid;
                    const uint32_t r = *c;
                    *c = uint16_t(r + 1);
                    rank[j / 4] |= r << (8 * (j & 3));
                }
            }
        }
        __syncthreads();
        // exclusive scan within digit w, then of the digits' sums
        uint32_t sum = 0;
        for (int i0 = 0; i0 < quads; i0 += 32) {
            const int i = w * quads + i0 + lane;
            const uint4 u = i0 + lane < quads ? counts[i] : make_uint4(0, 0, 0, 0);
            const uint32_t pk[4] = {u.x, u.y, u.z, u.w};
            uint32_t t = u.x + u.y + u.z + u.w;   // halves of at most 16 · 4 each: no carry
            t = (t & 0xffffu) + (t >> 16);
            uint32_t inc = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += x;
            }
            uint32_t base = sum + inc - t, q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t next = base + (pk[k] & 0xffffu);
                q[k] = (base & 0xffffu) | (next << 16);
                base = next + (pk[k] >> 16);
            }
            if (i0 + lane < quads) counts[i] = make_uint4(q[0], q[1], q[2], q[3]);
            sum += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) wsum[w] = sum;
        __syncthreads();
        if (w == 0) {
            const uint32_t t = wsum[lane];
            uint32_t x = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            wsum[lane] = x - t;
        }
        __syncthreads();
        if (holds) {
#pragma unroll
            for (int j = 0; j < kSortItems; ++j) {
                if (j < per) {
                    const uint32_t d = (key[j] >> (kSortBits * p)) & (kDigits - 1);
                    const int to = at(int(wsum[d] + cnt[d * holders + tid] + ((rank[j / 4] >> (8 * (j & 3))) & 255u)));
                    skey[to] = key[j];
                    spos[to] = uint16_t(pos[j / 2] >> (16 * (j & 1)));
                }
            }
        }
        __syncthreads();
    }
    for (int i = tid; i < n; i += kSortThreads) {
        out_id[i] = skey[at(i)];
        out_pos[i] = spos[at(i)];
    }
}

template <typename TI>
__global__ void __launch_bounds__(kSortThreads, 1)
sort_fill_kernel(const TI* __restrict__ ids, int64_t N, int64_t V, int passes,
                 uint32_t* __restrict__ sorted_id, uint32_t* __restrict__ sorted_pos, int tiles,
                 float4* __restrict__ fill, int64_t n4) {
    extern __shared__ __align__(16) char smem[];
    dep_launch_dependents();
    if (int(blockIdx.x) < tiles) {
        const int64_t t0 = int64_t(blockIdx.x) * kSortTile;
        const int n = int(N - t0 < kSortTile ? N - t0 : kSortTile);
        sort_tile(ids + t0, V, n, passes, sorted_id + t0, sorted_pos + t0, smem);
    } else if (fill) {
        const int64_t step = int64_t(gridDim.x - tiles) * kSortThreads;
        for (int64_t i = int64_t(blockIdx.x - tiles) * kSortThreads + threadIdx.x; i < n4; i += step)
            fill[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
}

// ---- the gradient's sums --------------------------------------------------------------------------

constexpr int kSumThreads = 128;   // × 4 channels
constexpr int kBatch = 4;          // rows whose loads are in flight together

template <int NB>
__device__ __forceinline__ float4 row_sum(const float* __restrict__ dR, int64_t t, int D, int c) {
    const float* p = dR + t * NB * int64_t(D) + c;
    float4 s = __ldcs(reinterpret_cast<const float4*>(p));
#pragma unroll
    for (int i = 1; i < NB; ++i) {
        const float4 b = __ldcs(reinterpret_cast<const float4*>(p + int64_t(i) * D));
        s.x += b.x, s.y += b.y, s.z += b.z, s.w += b.w;
    }
    return s;
}

__device__ __forceinline__ void flush(float* __restrict__ dst, float4 a, float scale, bool add) {
    float4* p = reinterpret_cast<float4*>(dst);
    a.x *= scale, a.y *= scale, a.z *= scale, a.w *= scale;
    if (add) {
        const float4 b = *p;
        a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
    }
    *p = a;
}

// Partial rows: piece p's row 2p is its share of a run that began in an earlier piece, row 2p+1 of
// a run that begins in it and goes on (a piece inside one run only has row 2p).
template <int NB>
__global__ void __launch_bounds__(kSumThreads)
run_sum_kernel(const float* __restrict__ dR, const uint32_t* __restrict__ sid,
               const uint32_t* __restrict__ spos, int n, int64_t V, int D, int piece, float scale,
               bool add, float* __restrict__ dE, float* __restrict__ part) {
    dep_wait();
    dep_launch_dependents();
    const int i0 = blockIdx.x * piece, i1 = min(i0 + piece, n);
    const int c = (blockIdx.y * kSumThreads + threadIdx.x) * 4;
    if (c >= D) return;
    uint32_t cur = sid[i0];
    bool from_before = i0 > 0 && sid[i0 - 1] == cur;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = i0; i < i1; i += kBatch) {
        float4 x[kBatch];
        uint32_t id[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            id[k] = i + k < i1 ? sid[i + k] : 0xffffffffu;
            x[k] = id[k] < V ? row_sum<NB>(dR, spos[i + k], D, c)
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (i + k >= i1) break;
            if (id[k] != cur) {
                if (cur < V) {
                    if (from_before)
                        *reinterpret_cast<float4*>(part + int64_t(2 * blockIdx.x) * D + c) = acc;
                    else
                        flush(dE + int64_t(cur) * D + c, acc, scale, add);
                }
                cur = id[k];
                from_before = false;
                acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            acc.x += x[k].x, acc.y += x[k].y, acc.z += x[k].z, acc.w += x[k].w;
        }
    }
    if (cur < V) {
        const bool goes_on = i1 < n && sid[i1] == cur;
        if (from_before || goes_on)
            *reinterpret_cast<float4*>(part + int64_t(2 * blockIdx.x + (from_before ? 0 : 1)) * D + c) =
                acc;
        else
            flush(dE + int64_t(cur) * D + c, acc, scale, add);
    }
}

// Four groups of threads take a run's pieces in turn and are added up in order.
constexpr int kJoinGroups = 4;
__global__ void __launch_bounds__(kSumThreads * kJoinGroups)
run_join_kernel(const uint32_t* __restrict__ sid, int n, int64_t V, int D, int piece, float scale,
                bool add, float* __restrict__ dE, const float* __restrict__ part) {
    __shared__ float4 sums[kJoinGroups][kSumThreads];
    dep_wait();
    const int p = blockIdx.x, i0 = p * piece, i1 = i0 + piece;
    if (i1 >= n) return;
    const uint32_t id = sid[i1], before = sid[i1 - 1], head = sid[i0], prev = p > 0 ? sid[i0 - 1] : ~id;
    // the run that crosses this piece's end has to begin inside it
    if (id >= V || before != id || (head == id && prev == id)) return;
    const int t = threadIdx.x % kSumThreads, group = threadIdx.x / kSumThreads;
    const int c = (blockIdx.y * kSumThreads + t) * 4;
    // the run's end by bisection: the first sorted index > i1 whose id differs
    int lo = i1 + 1, hi = n;
    while (lo < hi) {
        const int m = (lo + hi) >> 1;
        if (sid[m] == id) lo = m + 1;
        else hi = m;
    }
    const int pieces = (lo - 1) / piece - p + 1;   // with a share of the run, this one first
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < D) {
#pragma unroll 8
        for (int q = group; q < pieces; q += kJoinGroups) {
            const int64_t row = 2 * int64_t(p + q) + (q == 0 ? 1 : 0);
            const float4 b = *reinterpret_cast<const float4*>(part + row * D + c);
            acc.x += b.x, acc.y += b.y, acc.z += b.z, acc.w += b.w;
        }
    }
    sums[group][t] = acc;
    __syncthreads();
    if (group > 0 || c >= D) return;
#pragma unroll
    for (int k = 1; k < kJoinGroups; ++k) {
        const float4 b = sums[k][t];
        acc.x += b.x, acc.y += b.y, acc.z += b.z, acc.w += b.w;
    }
    flush(dE + int64_t(id) * D + c, acc, scale, add);
}

// Sorted positions a CTA of the sums takes: 64 for large tiles (few partial rows), fewer where the
// pieces would not fill the SMs (a constant, so that the workspace can be sized without a device).
int piece_of(int64_t n, int D) {
    constexpr int64_t kSms = 152;
    const int64_t cols = (D + kSumThreads * 4 - 1) / (kSumThreads * 4);
    int piece = 64;
    while (piece > 4 && (n + piece - 1) / piece * cols < kSms * 4) piece /= 2;
    return piece;
}
int64_t pieces_of(int64_t n, int D) {
    const int piece = piece_of(n, D);
    return (n + piece - 1) / piece;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem,
                         cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

template <typename TI>
cudaError_t sort_fill(int64_t N, int64_t V, const void* ids, uint32_t* sid, uint32_t* spos,
                      float* fill, int64_t fill_n, cudaStream_t st) {
    int passes = 1;   // the keys are 0 .. V
    while ((uint64_t(V) >> (kSortBits * passes)) != 0) ++passes;
    const int tiles = int((N + kSortTile - 1) / kSortTile);
    const int64_t n4 = fill_n / 4;
    int64_t fillers = fill ? (n4 + kSortThreads * 4 - 1) / (kSortThreads * 4) : 0;
    const int64_t most = int64_t(sm_count()) * 4;
    fillers = fillers < most ? fillers : most;
    auto kern = sort_fill_kernel<TI>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(kSortSmem));
    if (e != cudaSuccess) return e;
    kern<<<unsigned(tiles + fillers), kSortThreads, kSortSmem, st>>>(
        static_cast<const TI*>(ids), N, V, passes, sid, spos, tiles, reinterpret_cast<float4*>(fill),
        n4);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embed(int64_t N, int64_t V, int D, int nb, int table_dtype, int state_dtype,
                         int id_bits, float scale, const void* ids, const void* table, void* R,
                         cudaStream_t st) {
    if (id_bits == 32)
        embed_types<int32_t>(N, V, D, nb, table_dtype, state_dtype, scale, ids, table, R, st);
    else
        embed_types<int64_t>(N, V, D, nb, table_dtype, state_dtype, scale, ids, table, R, st);
    return cudaGetLastError();
}

// The sorted ids and positions [N] each, then two partial rows [D] a piece, for the whole tiles or the
// last one (a smaller tile may have more pieces), whichever have more.
size_t embed_backward_workspace(int64_t N, int D) {
    const int64_t whole = N < kSortTile ? 0 : pieces_of(kSortTile, D);
    const int64_t last = pieces_of(N % kSortTile, D);
    const int64_t pieces = whole > last ? whole : last;
    return 2 * align256(size_t(N) * 4) + align256(size_t(2 * pieces) * D * 4);
}

cudaError_t launch_embed_backward(int64_t N, int64_t V, int D, int nb, int id_bits, float scale,
                                  const float* dR, const void* ids, float* dE, bool accumulate,
                                  void* workspace, cudaStream_t st) {
    char* ws = static_cast<char*>(workspace);
    uint32_t* sid = reinterpret_cast<uint32_t*>(ws);
    uint32_t* spos = reinterpret_cast<uint32_t*>(ws + align256(size_t(N) * 4));
    float* part = reinterpret_cast<float*>(ws + 2 * align256(size_t(N) * 4));
    float* fill = accumulate ? nullptr : dE;
    cudaError_t e = id_bits == 32 ? sort_fill<int32_t>(N, V, ids, sid, spos, fill, V * D, st)
                                  : sort_fill<int64_t>(N, V, ids, sid, spos, fill, V * D, st);
    for (int64_t t0 = 0; e == cudaSuccess && t0 < N; t0 += kSortTile) {
        const int n = int(N - t0 < kSortTile ? N - t0 : kSortTile);
        const int piece = piece_of(n, D);
        const dim3 grid(pieces_of(n, D), (D + kSumThreads * 4 - 1) / (kSumThreads * 4));
        const float* rows = dR + t0 * nb * int64_t(D);
        const bool add = accumulate || t0 > 0;
        e = launch_after(nb == 1 ? run_sum_kernel<1> : run_sum_kernel<4>, grid, kSumThreads, 0, st,
                         rows, sid + t0, spos + t0, n, V, D, piece, scale, add, dE, part);
        if (e == cudaSuccess)
            e = launch_after(run_join_kernel, grid, kSumThreads * kJoinGroups, 0, st, sid + t0, n, V, D, piece,
                             scale, add, dE, part);
    }
    return e;
}

}  // namespace gr
