// The feed-forward sublayer's products on the 5th-generation tensor cores (tcgen05, operands staged by TMA,
// accumulators in tensor memory): bf16, FP8 blocks, and fp32 as three bf16 terms.
//
//     C[m][n] = Σ_k A[m][k] B[n][k]
//
// Two CTAs on neighbouring SMs form one tile of 256 x 256 (cta_group::2): each holds 128 rows of A and half of B's
// rows, so an operand byte that reaches an SM is used for 256 rows of the other operand, and an SM loads 32 KB for
// 512 cycles of MMAs. A persistent grid of pairs; in each CTA one warp feeds a ring of stages by TMA, one (of the
// pair's first CTA) issues the MMAs, eight drain the accumulator: two accumulators in tensor memory, so the MMAs of
// the next tile run meanwhile.
//
// Bound by the tensor pipe with many tokens: 16384 x 4096 x 22016 in bf16 takes 1.52 ms (1.94 PFLOP/s, the pipe 95%
// active at 1.64 GHz), the same in FP8 0.88 ms (3.4 PFLOP/s, 77% active at 1.75 GHz). With few tokens they become C's
// columns and the weights' bytes bound it: 268 MB for 64 tokens in 43.5 us from the first load to the last sum, the
// partial sums of ranges of k joined by a second launch (2 us when it follows at once).
#include <atomic>

#include "gr_feed.h"
#include "gr_ptx.cuh"
#include "gr_blocks.cuh"
#include "gr_tc.cuh"

namespace gr {
namespace {

// ---- the two-CTA forms (cta_group::2) -----------------------------------------------------------
__device__ __forceinline__ void tmem_alloc2(uint32_t* slot, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D (+)= A · Bᵀ over both CTAs: A's and B's halves at the same shared-memory offsets in each, D's rows 0-127 in
// the first CTA's tensor memory, 128-255 in the second's. Issued by one thread of the first.
__device__ __forceinline__ void tc_mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Arrives once on `bar` of both CTAs when every MMA (and copy) this thread issued before has completed.
__device__ __forceinline__ void tc_commit2(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(uint16_t(3))
        : "memory");
}
// TMA loads into this CTA's shared memory whose bytes complete on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_pair_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_pair_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
// Bounded wait on a phase. Acquires at CTA scope: what is handed over here is TMA's, the tensor cores' or, scales, read
// by them.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    long long t0 = 0;
    for (int k = 0;; ++k) {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p;\n"
            " mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}"
            : "=r"(done)
            : "r"(a), "r"(parity), "r"(kSuspendNs)
            : "memory");
        if (done) return true;
        if (k == 0) t0 = clock64();
        else if (clock64() - t0 > kWaitLimit) {
            atomicOr(&g_wait_status, 1u);
            return false;
        }
    }
}
// The same by a whole warp, with one answer: its lanes leave their loops together.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) { return __all_sync(~0u, wait_on(bar, parity)); }
// One lane of a warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(~0u, v, 0); }
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Shared-memory descriptor of an MN-major operand in the 128-byte swizzled layout: 64 elements of M or N in
// each 128-byte row, a row for each k; blocks of 64 elements `block` bytes apart, groups of 8 k 1024.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t block) {
    uint64_t d = 0;
    d |= uint64_t((saddr >> 4) & 0x3FFFu);
    d |= uint64_t((block >> 4) & 0x3FFFu) << 16;
    d |= uint64_t((1024u >> 4) & 0x3FFFu) << 32;
    d |= uint64_t(1u) << 46;
    d |= uint64_t(2u) << 61;
    return d;
}

// ---- FP8 blocks: kind::mxf8f6f4 with a power-of-two scale for each row and 32 k ------------------
// The scales lie in tensor memory: row r of 128 in column r / 32, lane r % 32 (of every quadrant), a byte for each
// of four blocks of k. Both operands e4m3; the descriptor names the byte.
__device__ __forceinline__ uint32_t idesc_fp8(int N, int step) {
    return (uint32_t(step) << 4) | (uint32_t(N >> 3) << 17) | (1u << 23) | (16u << 24) | (uint32_t(step) << 29);
}
__device__ __forceinline__ void tc_mma2_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::
            "r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}
// 512 bytes (the scales of 128 rows) of shared memory into four columns of every quadrant, in both CTAs.
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint32_t saddr) {
    uint64_t d = 0;
    d |= uint64_t((saddr >> 4) & 0x3FFFu);
    d |= uint64_t((128u >> 4) & 0x3FFFu) << 32;   // 8 rows of 16 bytes
    d |= uint64_t(1u) << 46;
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// ---- what a launch computes ---------------------------------------------------------------------
enum Mode {
    kStore,    // C as bf16
    kGated,    // B: 128 rows of the gate's weights in the first CTA, the up projection's in the second
    kGrad,     // C = dh: with pre, dgate, dup and h
    kPart,     // C's sums over a range of k, fp32, to the workspace
};

// The scales of a product's operands. The tokens' as the tensor cores take them: for each 128 rows and four blocks of
// k 512 bytes, row r's word at 16 (r % 32) + 4 (r / 32). The weights' in rows of whole words, one for each `per` rows'
// (a matrix') 128. token_pitch: few tokens may also come in rows of whole words.
struct Scales {
    const uint8_t *tokens, *weights;
    int64_t n_tokens, n_weights, per;
    int pitch, token_pitch;
    __device__ const uint8_t* weight_row(uint32_t row) const {
        const uint32_t m = uint32_t(per), which = row / m;
        return weights + int64_t(which * ((m + kBlock - 1) / kBlock) + (row - which * m) / kBlock) * pitch;
    }
};

struct Args {
    int nk;                 // blocks of 64 k (FP8: 128), 128 bytes of a row
    int tiles_m, tiles_n;   // of 256 x bn
    int bn;                 // columns of a tile: kPart 16 .. 256, else 256 (kGated: 128 channels)
    int group;              // row tiles that are taken together
    int stages;
    int act;
    int keep;               // kGated: write pre
    int whole_a, whole_b;   // MN-major operands of whole groups of 64 rows: a box of both groups at once
    int early;              // A is not the launch before's: its first stages are read ahead of it
    int trigger;            // the next launch may start beside this one
    // Tiles 0 .. whole - 1 are done by a pair each; the others' steps of k, one after another, in even ranges
    uint32_t whole;
    // chunk > 0: no tile is whole; a pair's in turn are chunks of so many blocks, of all tiles their first, then their next
    uint32_t chunk, chunks, tiles;
    uint32_t turns;         // whole tiles, or chunks
    uint32_t steps;         // of a tile: nk in steps of one block (FP8: four, what a word of scales covers)
    uint32_t range, longer; // steps of a range; the first `longer` have one more
    int slots;              // partial tiles a pair's range may have
    float* part;
    int64_t rows, cols;     // of C (kGated: channels of h): boxes that start behind them are not stored
    Scales scales;          // FP8
    uint8_t* hs;            // FP8 kGated: h's scales, as a product's tokens
    int hs_steps;
    __host__ __device__ uint32_t begin(uint32_t pair) const { return pair * range + (pair < longer ? pair : longer); }
    // The pair whose range holds a step.
    __device__ uint32_t owner(uint32_t step) const {
        const uint32_t split = longer * (range + 1);
        return step < split ? step / (range + 1) : longer + (step - split) / range;
    }
    // Tile t's place: groups of row tiles, so that the tiles in flight share rows of both operands in the L2.
    __device__ void place(uint32_t t, int& m, int& n) const {
        const uint32_t per = uint32_t(group) * uint32_t(tiles_n), g = t / per, r = t - g * per;
        const uint32_t rows = min(uint32_t(group), uint32_t(tiles_m) - g * group);
        n = int(r / rows), m = int(g * group + r % rows);
    }
};

constexpr int kThreads = 320;      // FP8: a warp more
constexpr uint32_t kColScales = 256;   // FP8: the scales' columns, behind the accumulators'
constexpr int kScaleSlot = 512 + 1024; // of a step of four blocks: 128 rows of A, 256 of B
constexpr int kTileM = 256, kRowsA = 128, kBoxA = kRowsA * 128;
constexpr int kMaxStages = 12;
constexpr int kScaleSlots = 8;
constexpr int kAuxBytes = 640, kAuxFp8 = kAuxBytes + 2048 + kScaleSlots * kScaleSlot;
constexpr int kSmemMax = 232448;

// Staging for the outputs of a warp: kStore and kGated a box of 32 rows x 64 columns (FP8 h: of bytes), kGrad two of
// them.
__host__ __device__ constexpr int stage_out(int mode, bool fp8) {
    return mode == kPart ? 0 : mode == kGrad ? 2 * 4096 : mode == kGated && fp8 ? 2048 : 4096;
}

struct Aux {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2], done, loaded[8];
    uint64_t scales_full[kScaleSlots], scales_empty[kScaleSlots], top_full[4];
    uint32_t tmem;
};
static_assert(sizeof(Aux) <= kAuxBytes, "aux");
// FP8, behind it: the rows' largest magnitudes in the two halves of a block [2][2][128], then the slots of scales.

// A pair's pieces of work, in the order all its roles go through them.
struct Unit {
    int m, n, k0, k1;
    int slot;   // of the partial tiles; -1: a whole tile
};
template <int STEP> struct Units {
    const Args& a;
    uint32_t tile, pairs, at, end;
    int slot;
    __device__ Units(const Args& a, uint32_t pair, uint32_t pairs)
        : a(a), tile(pair), pairs(pairs), at(a.begin(pair)), end(a.begin(pair + 1)), slot(int(pair) * a.slots) {}
    __device__ bool next(Unit& u) {
        if (tile < a.turns) {
            uint32_t t = tile;
            u.k0 = 0, u.k1 = a.nk, u.slot = -1;
            if (a.chunk) {
                const uint32_t c = tile / a.tiles;
                t -= c * a.tiles;
                u.k0 = int(c * a.chunk), u.k1 = min(u.k0 + int(a.chunk), a.nk), u.slot = int(t * a.chunks + c);
            }
            a.place(t, u.m, u.n);
            tile += pairs;
            return true;
        }
        if (at >= end) return false;
        const uint32_t t = at / a.steps, s0 = at - t * a.steps, s1 = min(a.steps, s0 + end - at);
        a.place(a.whole + t, u.m, u.n);
        u.k0 = int(s0) * STEP, u.k1 = min(int(s1) * STEP, a.nk);
        u.slot = slot++;
        at += s1 - s0;
        return true;
    }
};

__device__ __forceinline__ void pack8(uint4& v, const float (&f)[8]) {
    v = make_uint4(pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7]));
}
// σ(g) of a value whose product is rounded to bf16 or coarser: exp by the hardware's 2^x, off by (2 + |g|) units, and a
// division that gives 0 where 1 + exp(-g) is above 2^126.
__device__ __forceinline__ float fast_sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }
// Φ(g) and exp(-g²/2) of such a value. With a = |g| and t = 1 / (1 + 0.28 a), Φ(-a) = exp(-a²/2) t Q(t): Q is the
// polynomial of degree 8 nearest to erfcx(a / √2) / 2t over all t in (0, 1] (least squares, weighted anew until the
// relative error was even: 1.7e-7), so nothing cancels below zero, where 1 + erf has no digits left from g = -5.6 on. Off
// by up to 10 units for a < 6, 18 at 10, from the exponent's rounding. erfcf in its place is as good and spills 750 bytes
// in the 64-fold epilogue: 16384 tokens of 512 x 2048 took 257 us, now 127 (1 + erf 136).
__device__ __forceinline__ void normal_both(float g, float& below, float& bell) {
    const float t = __fdividef(1.0f, fmaf(0.28f, fabsf(g), 1.0f));
    bell = __expf(-0.5f * g * g);
    float q = 0.0247199573f;
    q = fmaf(q, t, -0.093593061f);
    q = fmaf(q, t, 0.0924280286f);
    q = fmaf(q, t, -0.00644911174f);
    q = fmaf(q, t, 0.0727749839f);
    q = fmaf(q, t, 0.0836308002f);
    q = fmaf(q, t, 0.103084661f);
    q = fmaf(q, t, 0.111699805f);
    q = fmaf(q, t, 0.111703858f);
    q *= bell * t;
    below = g > 0.0f ? 1.0f - q : q;
}
// f(g) and f'(g)
__device__ __forceinline__ void act_both(int act, float g, float& a, float& slope) {
    if (act == GR_SILU) {
        const float s = fast_sigmoid(g);
        a = g * s;
        slope = fmaf(a, 1.0f - s, s);
    } else {
        float below, bell;
        normal_both(g, below, bell);
        a = g * below;
        slope = fmaf(g * 0.39894228040143268f, bell, below);
    }
}
__device__ __forceinline__ float act_of(int act, float g) {
    if (act == GR_SILU) return g * fast_sigmoid(g);
    float below, bell;
    normal_both(g, below, bell);
    return g * below;
}
__device__ __forceinline__ void st_shared16(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// tmA: K-major {k, row} box {64, 128}, MN-major {row, k} box {64, 64} or, of whole groups of 64 rows, {row % 64, k,
// row / 64} box {64, 64, 2}. tmB: the same over bn / 2 rows (kGated: {k,
// channel, matrix} box {64, 128, 1}). tmC0: C, or h; tmC1: pre; tmC2: dpre.
// TERMS 3 (kPart): each operand as three bf16 matrices one after another, {.., matrix} boxes.
// FP8: codes, both operands K-major, boxes of 128 k; tmC0 of kGated: h's codes.
template <int MODE, bool FP8, bool A_MN, bool B_MN, int TERMS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(FP8 ? kThreads + 32 : kThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
            const __grid_constant__ CUtensorMap tmC0, const __grid_constant__ CUtensorMap tmC1,
            const __grid_constant__ CUtensorMap tmC2, const __grid_constant__ Args args) {
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int rows_b = args.bn / 2, box_b = rows_b * 128, stage = TERMS * (kBoxA + box_b), stages = args.stages;
    uint8_t* out = sm + stages * stage;
    Aux& x = *reinterpret_cast<Aux*>(out + 8 * stage_out(MODE, FP8));
    uint32_t* const tops = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(&x) + kAuxBytes);
    uint8_t* const sf = reinterpret_cast<uint8_t*>(tops + 512);
    constexpr int kK = FP8 ? 128 : 64;
    // The scales take columns behind 256: one accumulator of up to 256 columns, or two of 128.
    const int accs = FP8 && args.bn > 128 ? 1 : 2, acc_cols = FP8 ? 128 : 256;
    // A tensor core cuts off what an addition to its accumulator shifts out, up to two units in its last place. Few enough of
    // them (kLongest) are nothing beside a rounding to bf16, but not for fp32, so there an accumulator takes four blocks at
    // most (16 additions, 2.8e-7), and those sums are added up with rounding.
    constexpr int kRun = TERMS > 1 ? 4 : 1 << 30;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool first = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&x.full[s], 1), mbar_init(&x.empty[s], 1);
        for (int b = 0; b < 2; ++b) mbar_init(&x.acc_full[b], 1), mbar_init(&x.acc_empty[b], 16);
        for (int i = 0; i < kScaleSlots; ++i) mbar_init(&x.scales_full[i], 2), mbar_init(&x.scales_empty[i], 1);
        for (int q = 0; q < 4; ++q) mbar_init(&x.top_full[q], 2);
        for (int w = 0; w < 8; ++w) mbar_init(&x.loaded[w], 1);
        mbar_init(&x.done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc2(&x.tmem, 512);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = x.tmem;
    // The next launch waits for this one's end in its turn. What the launch before wrote (or still reads) is touched
    // after dep_wait only.
    if (args.trigger) dep_launch_dependents();
    if (warp != 0) dep_wait();

    Units<FP8 ? 4 : 1> units(args, cluster_id_x(), ncluster_x());
    Unit u;
    // The producer's and the issuer's whole warps run their loops and one lane issues: descriptors and addresses stay in
    // uniform registers (from a branch of one lane a stage took the issuer 1000 cycles, twice what its MMAs take).
    if (warp == 0) {
        const bool leader = elect_one();
        const uint32_t bytes = 2u * uint32_t(stage);
        const uint32_t bar0 = map_rank(smem_u32(&x.full[0]), 0);   // the first CTA's barriers count both CTAs' bytes
        uint32_t g = 0, s = 0, lap = 0;                            // block, its stage, how often the ring went round
        auto load_a = [&](uint32_t s, int m0, int kb) {
            if (first) mbar_expect_tx(&x.full[s], bytes);
            uint8_t* pa = sm + s * stage;
            if constexpr (TERMS > 1) {
#pragma unroll
                for (int t = 0; t < TERMS; ++t, pa += kBoxA) {
                    tma_pair_3d(pa, &tmA, A_MN ? m0 : kb * kK, A_MN ? kb * kK : m0, t, bar0 + s * 8);
                    if (A_MN) tma_pair_3d(pa + 8192, &tmA, m0 + 64, kb * kK, t, bar0 + s * 8);
                }
            } else if constexpr (A_MN) {
                if (args.whole_a) {
                    tma_pair_3d(pa, &tmA, 0, kb * kK, m0 >> 6, bar0 + s * 8);
                } else {
                    tma_pair_2d(pa, &tmA, m0, kb * kK, bar0 + s * 8);
                    tma_pair_2d(pa + 8192, &tmA, m0 + 64, kb * kK, bar0 + s * 8);
                }
            } else {
                tma_pair_2d(pa, &tmA, kb * kK, m0, bar0 + s * 8);
            }
        };
        auto load_b = [&](uint32_t s, int n0, int kb) {
            uint8_t* pb = sm + s * stage + TERMS * kBoxA;
            if constexpr (TERMS > 1) {
#pragma unroll
                for (int t = 0; t < TERMS; ++t, pb += box_b)
                    tma_pair_3d(pb, &tmB, B_MN ? n0 : kb * kK, B_MN ? kb * kK : n0, t, bar0 + s * 8);
            } else if constexpr (MODE == kGated) {
                tma_pair_3d(pb, &tmB, kb * kK, n0, int(rank), bar0 + s * 8);
            } else if constexpr (B_MN) {
                if (args.whole_b)
                    tma_pair_3d(pb, &tmB, 0, kb * kK, n0 >> 6, bar0 + s * 8);
                else
                    for (int i = 0; i < rows_b; i += 64) tma_pair_2d(pb + i * 128, &tmB, n0 + i, kb * kK, bar0 + s * 8);
            } else {
                tma_pair_2d(pb, &tmB, kb * kK, n0, bar0 + s * 8);
            }
        };
        bool more = units.next(u);
        int ahead = 0;   // blocks of the first unit whose A is on its way already
        if (args.early && more) {
            const int m0 = uniform(u.m * kTileM + int(rank) * kRowsA), k0 = uniform(u.k0);
            ahead = min(stages, uniform(u.k1) - k0);
            if (leader)
                for (int i = 0; i < ahead; ++i) load_a(i, m0, k0 + i);
        }
        dep_wait();
        fence_async_global();
        for (bool ok = true; ok && more; more = units.next(u)) {
            const int m0 = uniform(u.m * kTileM + int(rank) * kRowsA);
            const int n0 = uniform(u.n * (MODE == kGated ? 128 : args.bn) + (MODE == kGated ? 0 : int(rank) * rows_b));
            const int k0 = uniform(u.k0), k1 = uniform(u.k1);
            for (int kb = k0; kb < k1; ++kb, ++g) {
                if (lap > 0 && !wait_warp(&x.empty[s], (lap - 1) & 1)) {
                    ok = false;
                    break;
                }
                if (leader) {
                    if (g >= uint32_t(ahead)) load_a(s, m0, kb);
                    load_b(s, n0, kb);
                }
                if (++s == uint32_t(stages)) s = 0, ++lap;
            }
        }
        // no copy is under way when the CTAs leave: the first CTA sees both CTAs' arrive
        if (first)
            for (uint32_t i = g > uint32_t(stages) ? g - stages : 0; i < g; ++i)
                wait_warp(&x.full[i % stages], (i / stages) & 1);
    } else if (warp == 1) {
        if (first) {
            const bool leader = elect_one();
            const uint32_t idesc = FP8 ? idesc_fp8(args.bn, 0)
                                       : idesc_bf16_f32(256, args.bn) | (A_MN ? 1u << 15 : 0) | (B_MN ? 1u << 16 : 0);
            const uint32_t base = smem_u32(sm), sf0 = smem_u32(sf), copies = 1 + (args.bn + 127) / 128;
            const uint64_t da0 = A_MN ? sdesc_mn(base, 8192) : sdesc_sw128(base);
            const uint64_t db0 = B_MN ? sdesc_mn(base + TERMS * kBoxA, 8192) : sdesc_sw128(base + TERMS * kBoxA);
            const uint32_t hop = uint32_t(stage) >> 4;   // from a stage to the next, in a descriptor
            uint32_t s = 0, lap = 0, q = 0;              // stage, laps, steps of scales
            bool ok = true;
            for (int j = 0; ok && units.next(u);) {
                const int all = uniform(u.k1 - u.k0);
                for (int from = 0; ok && from < all; from += kRun, ++j) {
                    const int b = j % accs, blocks = min(kRun, all - from);
                    if (j >= accs && !wait_warp(&x.acc_empty[b], (j / accs - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + b * acc_cols;
                    for (int kb = 0; kb < blocks; ++kb) {
                        const uint32_t step = uint32_t(kb) & 3;
                        if (FP8 && step == 0) {
                            // the scales of this and the next three blocks; the copies run in order with the MMAs
                            if (!wait_warp(&x.scales_full[q % kScaleSlots], (q / kScaleSlots) & 1)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            if (leader)
                                for (uint32_t i = 0; i < copies; ++i)
                                    tc_copy_scales(tmem + kColScales + (q & 1) * 16 + i * 4,
                                                   sf0 + (q % kScaleSlots) * kScaleSlot + i * 512);
                            ++q;
                        }
                        if (!wait_warp(&x.full[s], lap & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (leader) {
                            const uint64_t da = da0 + s * hop, db = db0 + s * hop;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint64_t a = da + k * (A_MN ? 128 : 2), bb = db + k * (B_MN ? 128 : 2);
                                if constexpr (TERMS > 1) {
                                    // the product of the first terms, and beside it the five that are smaller
#pragma unroll
                                    for (int ta = 0; ta < TERMS; ++ta)
#pragma unroll
                                        for (int tb = 0; ta + tb < TERMS; ++tb)
                                            tc_mma2(d + (ta + tb > 0 ? 128 : 0), a + ta * (kBoxA >> 4),
                                                    bb + tb * (uint32_t(box_b) >> 4), idesc,
                                                    kb > 0 || k > 0 || ta + tb > 1 || ta > 0);
                                } else if constexpr (FP8) {
                                    const uint32_t sfa = tmem + kColScales + ((q - 1) & 1) * 16;
                                    tc_mma2_fp8(d, a, bb, idesc | (step << 4) | (step << 29), sfa, sfa + 4, kb > 0 || k > 0);
                                } else {
                                    tc_mma2(d, a, bb, idesc, kb > 0 || k > 0);
                                }
                            }
                            tc_commit2(&x.empty[s]);
                            if (FP8 && (step == 3 || kb + 1 == blocks)) tc_commit2(&x.scales_empty[(q - 1) % kScaleSlots]);
                        }
                        if (++s == uint32_t(stages)) s = 0, ++lap;
                    }
                    if (ok && leader) tc_commit2(&x.acc_full[b]);
                }
            }
            if (leader) tc_commit2(&x.done);
            wait_warp(&x.done, 0);
        }
    } else if (FP8 && warp == 10) {
        // Scales: a word (four blocks) for each of 128 rows of A and bn of B into shared memory. Rows behind the last have any scales: their rows or columns of C may
        // come out NaN, and are not stored.
        constexpr bool kTokensB = MODE == kPart;   // else A's rows are the tokens
        const Scales& sc = args.scales;
        const uint32_t steps = args.steps;
        const uint8_t *pw[8], *pt[8];   // the lane's rows of weights in the tile, and (kPart) of tokens
        const uint32_t hop = sc.token_pitch ? 4 : 512;   // from a step's words of the tokens to the next's
        int64_t t0 = 0;                 // the tile's first token
        auto find = [&](const Unit& t) {
            t0 = kTokensB ? int64_t(t.n) * args.bn : int64_t(t.m) * kTileM + rank * kRowsA;
            const int64_t w0 = kTokensB ? int64_t(t.m) * kTileM + rank * kRowsA : int64_t(t.n) * args.bn;
#pragma unroll
            for (int i = 0; i < (kTokensB ? 4 : 8); ++i) {
                const int r = i * 32 + lane;
                int64_t row = w0 + r;
                if (MODE == kGated) {
                    const int64_t ch = int64_t(t.n) * 128 + (r & 127);
                    row = ch < sc.per ? ch + (r >> 7) * sc.per : sc.n_weights;
                }
                pw[i] = row < sc.n_weights ? sc.weight_row(uint32_t(row)) : sc.weights;
            }
            if constexpr (kTokensB) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t row = t0 + i * 32;   // 32 rows from a multiple of 32 on
                    pt[i] = row + lane >= sc.n_tokens ? sc.tokens
                            : sc.token_pitch          ? sc.tokens + (row + lane) * sc.token_pitch
                                                      : sc.tokens + (row >> 7) * steps * 512 + lane * 16 + ((row >> 5) & 3) * 4;
                }
            }
        };
        auto copy4 = [](uint32_t to, const uint8_t* p) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(p) : "memory");
        };
        auto copy_step = [&](uint32_t at, int kb) {
            const uint32_t st = uint32_t(kb) >> 2, w = kTokensB ? at : at + 512, to = kTokensB ? at + 512 : at;
#pragma unroll
            for (int i = 0; i < (kTokensB ? 4 : 8); ++i) copy4(w + (i >> 2) * 512 + (i & 3) * 4, pw[i] + kb);
            if constexpr (kTokensB) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i * 32 < args.bn) copy4(to + (i >> 2) * 512 + (i & 3) * 4, pt[i] + st * hop);
            } else if (t0 < sc.n_tokens) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to),
                             "l"(sc.tokens + ((t0 >> 7) * steps + st) * 512 + lane * 16)
                             : "memory");
            }
        };
        // Half of the slots at a time: the fence that hands copied words to the tensor cores waits for every copy under
        // way, so copies of a step at a time would each take a trip to the L2 (16384 tokens of 4096 x 11008: 1.59 ms, so 1.55).
        constexpr uint32_t kBatch = kScaleSlots / 2;
        uint32_t q = 0;
        bool more = units.next(u), ok = true;
        int kb = u.k0;
        if (more) find(u);
        while (ok && more) {
            const uint32_t begin = q;
            for (uint32_t i = 0; ok && more && i < kBatch; ++i, ++q) {
                const uint32_t slot = q % kScaleSlots;
                if (q >= kScaleSlots) ok = wait_warp(&x.scales_empty[slot], ((q / kScaleSlots) - 1) & 1);
                if (ok) copy_step(smem_u32(sf) + slot * kScaleSlot + lane * 16, kb);
                kb += 4;
                if (kb >= u.k1) {
                    more = units.next(u);
                    kb = u.k0;
                    if (more) find(u);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_shared();
            __syncwarp();
            if (lane == 0 && ok)
                for (uint32_t i = begin; i < q; ++i)
                    arrive_remote(map_rank(smem_u32(&x.scales_full[i % kScaleSlots]), 0));
        }
    } else {
        const int w = warp - 2, half = w >> 2, quad = warp & 3;
        const uint32_t mine = smem_u32(out) + w * stage_out(MODE, FP8);
        uint8_t* const minep = out + w * stage_out(MODE, FP8);
        const uint32_t lanes = uint32_t(quad) << 21;   // lane field of a tensor-memory address: quad * 32 << 16
        auto row_of = [&](const Unit& t) { return t.m * kTileM + int(rank) * kRowsA + quad * 32; };
        // kGrad: gate and up of 64 channels of the warp's rows into its two boxes, which dgate and dup leave from, then h
        uint32_t reads = 0, used = 0;
        auto read_pre = [&](int row, int ch, int which) {
            if (lane == 0) {
                if (which) mbar_expect_tx(&x.loaded[w], 8192);
                tma_load_3d(minep + which * 4096, &tmC1, ch, which, row, &x.loaded[w]);
            }
            reads += which;
        };
        bool more = units.next(u);
        if (MODE == kGrad && more && u.slot < 0) {
            read_pre(row_of(u), u.n * 256 + half * 128, 1);
            read_pre(row_of(u), u.n * 256 + half * 128, 0);
        }
        for (int j = 0; more; ++j) {
            const int b = j % accs;
            const Unit now = u;
            if (!wait_warp(&x.acc_full[b], (j / accs) & 1)) break;
            tc_fence_after();
            const uint32_t acc = tmem + b * acc_cols + lanes;
            const int row = row_of(now);   // the warp's first
            auto drained = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_remote(map_rank(smem_u32(&x.acc_empty[b]), 0));
            };
            // 64 columns of fp32 as a bf16 box, stored once it is written
            auto put_box = [&](const float (&v)[64], auto&& store) {
                if (lane == 0) bulk_wait_read<0>();
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    st_shared16(mine + swz(lane, c),
                                make_uint4(pack_bf2(v[8 * c], v[8 * c + 1]), pack_bf2(v[8 * c + 2], v[8 * c + 3]),
                                           pack_bf2(v[8 * c + 4], v[8 * c + 5]),
                                           pack_bf2(v[8 * c + 6], v[8 * c + 7])));
                fence_async_shared();
                __syncwarp();
                if (lane == 0 && row < args.rows) {
                    store();
                    bulk_commit();
                }
            };
            auto get64 = [&](uint32_t col, float (&v)[64]) {
                uint32_t r[4][16];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld16_nowait(acc + col + i * 16, r[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    tmem_wait_ld(r[i]);
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[i * 16 + k] = __uint_as_float(r[i][k]);
                }
            };
            // twice 64 columns, all on their way at once
            auto get128 = [&](uint32_t col, uint32_t col2, float (&v)[64], float (&v2)[64]) {
                uint32_t r[8][16];
#pragma unroll
                for (int i = 0; i < 8; ++i) tmem_ld16_nowait(acc + (i < 4 ? col : col2) + (i & 3) * 16, r[i]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    tmem_wait_ld(r[i]);
#pragma unroll
                    for (int k = 0; k < 16; ++k) (i < 4 ? v : v2)[(i & 3) * 16 + k] = __uint_as_float(r[i][k]);
                }
            };
            // a partial tile's sums: [256 / 8 columns][256 rows][8]
            auto put_part = [&](uint32_t col, const float (&v)[64]) {
                float4* p = reinterpret_cast<float4*>(args.part) +
                            int64_t(now.slot) * (kTileM * 64) +
                            (int64_t(col >> 3) * kTileM + int(rank) * kRowsA + quad * 32 + lane) * 2;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    p[(i >> 1) * (kTileM * 2) + (i & 1)] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            };
            if (MODE != kPart && now.slot >= 0) {
                float v[64];
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    const uint32_t col = half * 128 + i * 64;
                    get64(col, v);
                    if (i == 1) drained();
                    put_part(col, v);
                }
            } else if constexpr (MODE == kStore) {
                const int col = now.n * 256 + half * 128;
                auto put = [&](const float (&v)[64], int i) {
                    put_box(v, [&] {
                        if (col + i * 64 < args.cols) tma_store_2d(&tmC0, minep, col + i * 64, row);
                    });
                };
                float v[64];
                if constexpr (FP8) {   // one accumulator: the next tile waits for it
                    float v2[64];
                    get128(half * 128, half * 128 + 64, v, v2);
                    drained();
                    put(v, 0);
                    put(v2, 1);
                } else {
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        get64(half * 128 + i * 64, v);
                        if (i == 1) drained();
                        put(v, i);
                    }
                }
            } else if constexpr (MODE == kGated) {
                const int col = now.n * 128 + half * 64;
                float ga[64], up[64];
                get128(half * 64, 128 + half * 64, ga, up);
                drained();
                const bool in = col < args.cols;
                if (args.keep && in) {
                    put_box(ga, [&] { tma_store_3d(&tmC1, minep, col, 0, row); });
                    put_box(up, [&] { tma_store_3d(&tmC1, minep, col, 1, row); });
                }
                if (args.act == GR_SILU) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) ga[i] = act_of(GR_SILU, ga[i]) * up[i];
                } else {
                    // eight at a time, behind a branch that the compiler does not see through: their many values in
                    // flight next to 128 registers would be spilled
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        int act;
                        asm volatile("mov.b32 %0, %1;" : "=r"(act) : "r"(args.act));
                        if (act == GR_GELU)
#pragma unroll
                            for (int i = 8 * c; i < 8 * c + 8; ++i) ga[i] = act_of(GR_GELU, ga[i]) * up[i];
                    }
                }
                if constexpr (FP8) {
                    if (col + 64 > args.cols)   // channels behind the last are not the block's
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (col + i >= args.cols) ga[i] = 0.0f;
                    // the block's largest magnitude: this half's and the other's, from the warp that has the same rows
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < 64; ++i) top = max(top, block_mag(ga[i]));
                    uint32_t* t = tops + (j & 1) * 256 + quad * 32 + lane;
                    t[half * 128] = top;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x.top_full[quad]);
                    if (!wait_warp(&x.top_full[quad], j & 1)) break;
                    top = max(top, *const_cast<volatile uint32_t*>(t + (half ^ 1) * 128));
                    float inv;
                    const uint8_t e = block_scale(top, inv);
                    if (half == 0 && row + lane < args.rows)
                        args.hs[scale_at(row + lane, now.n, args.hs_steps)] = e;
                    if (lane == 0) bulk_wait_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        st_shared16(mine + swz64(lane, c),
                                    make_uint4(block_codes4(ga + 16 * c, inv), block_codes4(ga + 16 * c + 4, inv),
                                               block_codes4(ga + 16 * c + 8, inv),
                                               block_codes4(ga + 16 * c + 12, inv)));
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0 && in && row < args.rows) {
                        tma_store_2d(&tmC0, minep, col, row);
                        bulk_commit();
                    }
                } else if (in) put_box(ga, [&] { tma_store_2d(&tmC0, minep, col, row); });
            } else if constexpr (MODE == kGrad) {
                const int col = now.n * 256 + half * 128;
                // the tile after this one, whose first values are read behind this one's last
                Units<1> peek = units;
                Unit after;
                const bool follows = peek.next(after) && after.slot < 0;
                bool ok = true;
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    float dh[64];
                    get64(half * 128 + i * 64, dh);
                    if (i == 1) drained();
                    ok = ok && wait_warp(&x.loaded[w], used & 1);
                    ++used;
                    uint4 h[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        float g[8], p[8], a[8], s[8];
                        unpack8(ld_shared16(mine + swz(lane, c)), g);
                        unpack8(ld_shared16(mine + 4096 + swz(lane, c)), p);
                        if (args.act == GR_SILU) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) act_both(GR_SILU, g[k], a[k], s[k]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k) act_both(GR_GELU, g[k], a[k], s[k]);
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            s[k] *= dh[c * 8 + k] * p[k];
                            p[k] *= a[k];
                            a[k] *= dh[c * 8 + k];
                        }
                        uint4 v;
                        pack8(v, s);
                        st_shared16(mine + swz(lane, c), v);
                        pack8(v, a);
                        st_shared16(mine + 4096 + swz(lane, c), v);
                        pack8(h[c], p);
                    }
                    const int ch = col + i * 64;
                    const bool in = ok && row < args.rows && ch < args.cols;
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if (in) {
                            tma_store_3d(&tmC2, minep, ch, 0, row);
                            tma_store_3d(&tmC2, minep + 4096, ch, 1, row);
                            bulk_commit();
                        }
                        bulk_wait_read<0>();
                    }
                    __syncwarp();
                    // h after them, from the gate's box; the next 64 channels, of this tile or of the next whole one
                    const bool next = i == 0 || follows;
                    const int next_row = i == 0 ? row : row_of(after);
                    const int next_ch = i == 0 ? col + 64 : after.n * 256 + half * 128;
                    if (next) read_pre(next_row, next_ch, 1);
#pragma unroll
                    for (int c = 0; c < 8; ++c) st_shared16(mine + swz(lane, c), h[c]);
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if (in) {
                            tma_store_2d(&tmC0, minep, ch, row);
                            bulk_commit();
                        }
                        if (next) bulk_wait_read<0>();
                    }
                    if (next) read_pre(next_row, next_ch, 0);
                }
                if (!ok) break;
            } else if constexpr (TERMS > 1) {
                // sums of runs, added up in registers: every other 16 columns of up to 128
                float sum[4][16];
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int k = 0; k < 16; ++k) sum[c][k] = 0.0f;
                bool ok = true;
                for (int from = now.k0;; ++j) {
                    const uint32_t at = tmem + (j % accs) * acc_cols + lanes;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (half * 16 + c * 32 >= args.bn) continue;
                        float lead[16], rest[16];
                        tmem_ld16(at + half * 16 + c * 32, lead);
                        tmem_ld16(at + 128 + half * 16 + c * 32, rest);
#pragma unroll
                        for (int k = 0; k < 16; ++k) sum[c][k] += lead[k] + rest[k];
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_remote(map_rank(smem_u32(&x.acc_empty[j % accs]), 0));
                    from += kRun;
                    if (from >= now.k1) break;
                    ok = wait_warp(&x.acc_full[(j + 1) % accs], ((j + 1) / accs) & 1);
                    if (!ok) break;
                    tc_fence_after();
                }
                if (!ok) break;
                float* p = args.part + int64_t(now.slot) * (int64_t(kTileM) * args.bn) +
                           int(rank) * kRowsA + quad * 32 + lane;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (half * 16 + c * 32 >= args.bn) continue;
#pragma unroll
                    for (int k = 0; k < 16; ++k) p[int64_t(half * 16 + c * 32 + k) * kTileM] = sum[c][k];
                }
            } else {
                float* p = args.part + int64_t(now.slot) * (int64_t(kTileM) * args.bn) +
                           int(rank) * kRowsA + quad * 32 + lane;
                for (int c = half * 16; c < args.bn; c += 32) {
                    float v[16];
                    tmem_ld16(acc + c, v);
#pragma unroll
                    for (int k = 0; k < 16; ++k) p[int64_t(c + k) * kTileM] = v[k];
                }
                drained();
            }
            more = units.next(u);
        }
        for (; used < reads; ++used) wait_warp(&x.loaded[w], used & 1);   // after a wait that ran out
        if (lane == 0) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc2(tmem, 512);
}

// ---- the sums of the pairs' parts ---------------------------------------------------------------
// A tile that is not whole is spread over the pairs whose ranges of k meet it, in order: the first of them may have
// begun with earlier tiles, for the others it is their first partial tile.
struct JoinArgs {
    Args a;                      // of the products
    int64_t rows, cols;          // of the output (h's channels)
    __nv_bfloat16 *out, *pre_out;
    const __nv_bfloat16* pre;
    __nv_bfloat16* dpre;         // fp32: out (but kJoinStore's) and dpre as three terms
    float *out_f32, *pre_f32;    // fp32: C, and pre
    uint8_t *codes, *scales;     // h in FP8 blocks
    int scale_steps;
};

// Where the partial sums of one place of a tile lie (t counted from the first that is not whole, `at` in fours): found
// before the products are waited for.
struct Sums {
    const float4 *from, *rest;
    int64_t hop;
    uint32_t more;
    __device__ Sums(const Args& a, uint32_t t, int64_t at) {
        const uint32_t first = a.owner(t * a.steps), last = a.owner(t * a.steps + a.steps - 1);
        const int64_t tile = int64_t(kTileM) * a.bn / 4;
        hop = a.slots * tile;
        const float4* p = reinterpret_cast<const float4*>(a.part) + at;
        from = p + first * hop + (t - a.begin(first) / a.steps) * tile;
        rest = p + (first + 1) * hop;
        more = last - first;
    }
    template <int FOURS> __device__ __forceinline__ void add(float (&v)[4 * FOURS]) const {
        float4 s[FOURS];
#pragma unroll
        for (int i = 0; i < FOURS; ++i) s[i] = __ldcg(from + i);
        const float4* q = rest;
#pragma unroll 4
        for (uint32_t c = 0; c < more; ++c, q += hop) {
#pragma unroll
            for (int i = 0; i < FOURS; ++i) {
                const float4 w = __ldcg(q + i);
                s[i].x += w.x, s[i].y += w.y, s[i].z += w.z, s[i].w += w.w;
            }
        }
#pragma unroll
        for (int i = 0; i < FOURS; ++i)
            v[4 * i] = s[i].x, v[4 * i + 1] = s[i].y, v[4 * i + 2] = s[i].z, v[4 * i + 3] = s[i].w;
    }
};
template <int N> __device__ __forceinline__ void put_bf16(__nv_bfloat16* p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
        *reinterpret_cast<uint2*>(p + i) = make_uint2(pack_bf2(v[i], v[i + 1]), pack_bf2(v[i + 2], v[i + 3]));
}
template <int N> __device__ __forceinline__ void get_bf16(const __nv_bfloat16* p, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p + i);
        v[i] = __uint_as_float(u.x << 16), v[i + 1] = __uint_as_float(u.x & 0xffff0000u);
        v[i + 2] = __uint_as_float(u.y << 16), v[i + 3] = __uint_as_float(u.y & 0xffff0000u);
    }
}
// What the epilogues do with whole tiles, on N neighbouring channels of a token.
template <int N>
__device__ __forceinline__ void finish_gated(const JoinArgs& j, int64_t token, int64_t ch, float (&g)[N], float (&up)[N]) {
    if (j.pre_out) {
        put_bf16(j.pre_out + 2 * token * j.rows + ch, g);
        put_bf16(j.pre_out + (2 * token + 1) * j.rows + ch, up);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) g[k] = act_of(j.a.act, g[k]) * up[k];
}
template <int N>
__device__ __forceinline__ void finish_grad(const JoinArgs& j, int64_t token, int64_t ch, float (&dh)[N]) {
    float g[N], p[N], s[N];
    get_bf16(j.pre + 2 * token * j.rows + ch, g);
    get_bf16(j.pre + (2 * token + 1) * j.rows + ch, p);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float a, slope;
        act_both(j.a.act, g[k], a, slope);
        s[k] = slope * (dh[k] * p[k]);
        p[k] *= a;
        dh[k] *= a;
    }
    put_bf16(j.dpre + 2 * token * j.rows + ch, s);
    put_bf16(j.dpre + (2 * token + 1) * j.rows + ch, dh);
    put_bf16(j.out + token * j.rows + ch, p);
}
// N channels of each of LANES neighbouring lanes, a block of 128, as codes.
template <int N, int LANES>
__device__ __forceinline__ void finish_fp8(const JoinArgs& j, int64_t token, int64_t ch, const float (&h)[N], bool in) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) top = max(top, block_mag(h[k]));
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
    float inv;
    const uint8_t e = block_scale(top, inv);
    if (!in) return;
#pragma unroll
    for (int k = 0; k < N; k += 4)
        *reinterpret_cast<uint32_t*>(j.codes + token * j.rows + ch + k) = block_codes4(h + k, inv);
    if ((ch & (kBlock - 1)) == 0) j.scales[scale_at(token, uint32_t(ch / kBlock), j.scale_steps)] = e;
}

// fp32: an operand of a product as three bf16 terms, each the rounding of what the ones before leave (the first
// towards zero where it would become infinite): 24 bits and more, below 2^-110 to half of bf16's last place, 2^-134. What
// is not finite is the first term alone.
__device__ __forceinline__ void terms_of(float v, __nv_bfloat16 (&t)[3]) {
    t[0] = __float2bfloat16_rn(v);
    if ((__float_as_uint(v) & 0x7f800000u) == 0x7f800000u) {
        t[1] = t[2] = __float2bfloat16_rn(0.0f);
        return;
    }
    if ((__bfloat16_as_ushort(t[0]) & 0x7f80) == 0x7f80) t[0] = __float2bfloat16_rz(v);
    const float r = v - __bfloat162float(t[0]);
    t[1] = __float2bfloat16_rn(r);
    t[2] = __float2bfloat16_rn(r - __bfloat162float(t[1]));
}
__device__ __forceinline__ void put_terms(__nv_bfloat16* p, int64_t hop, const float (&v)[4]) {
    __nv_bfloat16 t[4][3];
#pragma unroll
    for (int k = 0; k < 4; ++k) terms_of(v[k], t[k]);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const __nv_bfloat162 a(t[0][i], t[1][i]), b(t[2][i], t[3][i]);
        *reinterpret_cast<uint2*>(p + i * hop) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                            *reinterpret_cast<const uint32_t*>(&b));
    }
}
struct Cut {
    const float* from;
    __nv_bfloat16* to;
    int64_t n;   // a multiple of 8
};
struct Cuts {
    Cut c[3];
};
__global__ void __launch_bounds__(256) terms_kernel(const Cuts cuts) {
    dep_launch_dependents();
    int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const Cut& c = cuts.c[k];
        if (i >= 0 && i < c.n) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(c.from + i));
            const float v[4] = {f.x, f.y, f.z, f.w};
            put_terms(c.to + i, c.n, v);
        }
        i -= c.n;
    }
}
__device__ __forceinline__ void put_f32(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void finish_gated_f32(const JoinArgs& j, int64_t token, int64_t ch, float (&g)[4],
                                                 const float (&up)[4]) {
    if (j.pre_f32) {
        put_f32(j.pre_f32 + 2 * token * j.rows + ch, g);
        put_f32(j.pre_f32 + (2 * token + 1) * j.rows + ch, up);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        g[k] = (j.a.act == GR_SILU ? activate<GR_SILU>(g[k]) : activate<GR_GELU>(g[k])) * up[k];
    put_terms(j.out + token * j.rows + ch, j.rows * j.cols, g);
}
__device__ __forceinline__ void finish_grad_f32(const JoinArgs& j, int64_t token, int64_t ch, float (&dh)[4]) {
    const float* q = j.pre_f32 + 2 * token * j.rows + ch;
    const float4 g4 = *reinterpret_cast<const float4*>(q), p4 = *reinterpret_cast<const float4*>(q + j.rows);
    const float g[4] = {g4.x, g4.y, g4.z, g4.w}, p[4] = {p4.x, p4.y, p4.z, p4.w};
    float s[4], h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const bool silu = j.a.act == GR_SILU;
        const float a = silu ? activate<GR_SILU>(g[k]) : activate<GR_GELU>(g[k]);
        s[k] = dh[k] * p[k] * (silu ? activate_slope<GR_SILU>(g[k]) : activate_slope<GR_GELU>(g[k]));
        h[k] = a * p[k];
        dh[k] *= a;
    }
    const int64_t hop = 2 * j.rows * j.cols;
    put_terms(j.dpre + 2 * token * j.rows + ch, hop, s);
    put_terms(j.dpre + (2 * token + 1) * j.rows + ch, hop, dh);
    put_terms(j.out + token * j.rows + ch, j.rows * j.cols, h);
}

// After kPart: C's rows are the output's channels, contiguous, its columns the tokens. A thread has four rows of a
// column; in FP8 a warp has a block.
enum Join { kJoinStore, kJoinGated, kJoinGrad, kJoinGatedFp8 };
constexpr int kJoinThreads = 128;

template <int JOIN, bool F32>
__global__ void __launch_bounds__(kJoinThreads) join_columns_kernel(const __grid_constant__ JoinArgs j) {
    dep_launch_dependents();
    constexpr bool kPair = JOIN == kJoinGated || JOIN == kJoinGatedFp8;
    const Args& a = j.a;
    const uint32_t rows = uint32_t(j.rows), lines = JOIN == kJoinGatedFp8 ? (rows + kBlock - 1) / kBlock * kBlock : rows;
    const uint32_t i = blockIdx.x * kJoinThreads + threadIdx.x, col = i / (lines / 4), row = (i - col * (lines / 4)) * 4;
    const bool in = col < uint32_t(j.cols) && row < rows;
    const uint32_t tn = col / uint32_t(a.bn), up_row = rows + row;
    const int64_t at = int64_t(col - tn * a.bn) * kTileM;
    const Sums s(a, in ? tn * a.tiles_m + row / kTileM : 0, (at + row % kTileM) / 4);
    const Sums su(a, in && kPair ? tn * a.tiles_m + up_row / kTileM : 0, (at + up_row % kTileM) / 4);
    dep_wait();
    if (JOIN != kJoinGatedFp8 && !in) return;
    float v[4] = {}, up[4];
    if (in) s.add<1>(v);
    if constexpr (kPair) {
        if (in) {
            su.add<1>(up);
            if constexpr (F32) finish_gated_f32(j, col, row, v, up);
            else finish_gated(j, col, row, v, up);
        }
    }
    if constexpr (JOIN == kJoinGatedFp8) finish_fp8<4, 32>(j, col, row, v, in);
    else if constexpr (JOIN == kJoinGrad && F32) finish_grad_f32(j, col, row, v);
    else if constexpr (JOIN == kJoinGrad) finish_grad(j, col, row, v);
    else if constexpr (JOIN == kJoinGated && F32) return;
    else if constexpr (F32) put_f32(j.out_f32 + int64_t(col) * rows + row, v);
    else put_bf16(j.out + int64_t(col) * rows + row, v);
}

// After the other modes: the tiles behind the whole ones, C as the output. A thread has eight columns of a row.
template <int JOIN> __global__ void __launch_bounds__(kJoinThreads) join_tiles_kernel(const __grid_constant__ JoinArgs j) {
    dep_launch_dependents();
    constexpr bool kPair = JOIN == kJoinGated || JOIN == kJoinGatedFp8;
    constexpr uint32_t kCols = kPair ? 128 : 256, kPer = kCols / 8, kBlocks = kTileM * kPer / kJoinThreads;
    const Args& a = j.a;
    const uint32_t t = blockIdx.x / kBlocks, i = (blockIdx.x - t * kBlocks) * kJoinThreads + threadIdx.x;
    const uint32_t r = i / kPer, c = i % kPer * 8;
    int m, n;
    a.place(a.whole + t, m, n);
    const int64_t row = int64_t(m) * kTileM + r, col = int64_t(n) * kCols + c;
    const bool in = row < a.rows && col < a.cols;
    const Sums s(a, t, (int64_t(c >> 3) * kTileM + r) * 2);
    dep_wait();
    if (JOIN != kJoinGatedFp8 && !in) return;
    float v[8] = {}, up[8];
    if (in) s.add<2>(v);
    if constexpr (kPair) {
        if (in) {
            const Sums su(a, t, (int64_t((c + 128) >> 3) * kTileM + r) * 2);
            su.add<2>(up);
            finish_gated(j, row, col, v, up);
        }
    }
    if constexpr (JOIN == kJoinGatedFp8) finish_fp8<8, 16>(j, row, col, v, in);
    else if constexpr (JOIN == kJoinGrad) finish_grad(j, row, col, v);
    else put_bf16(j.out + row * a.cols + col, v);
}

// ---- host ---------------------------------------------------------------------------------------
bool map_box(CUtensorMap* m, CUtensorMapDataType type, const void* p, int nd, const cuuint64_t* dims,
             const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(m, type, cuuint32_t(nd), const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// A bf16 matrix [rows][cols] in boxes of box_rows x box_cols.
bool map_bf16(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int box_rows, int box_cols) {
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)}, strides[1] = {cuuint64_t(cols) * 2};
    const cuuint32_t box[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)};
    return map_box(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, 2, dims, strides, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
}
// [a][b][cols] with boxes over one of a or b.
bool map_bf16_3d(CUtensorMap* m, const void* p, int64_t a, int64_t b, int64_t cols, int box_a, int box_b,
                 int box_cols) {
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(b), cuuint64_t(a)};
    const cuuint64_t strides[2] = {cuuint64_t(cols) * 2, cuuint64_t(cols * b) * 2};
    const cuuint32_t box[3] = {cuuint32_t(box_cols), cuuint32_t(box_b), cuuint32_t(box_a)};
    return map_box(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, 3, dims, strides, box,
                   CU_TENSOR_MAP_SWIZZLE_128B);
}

// A bf16 matrix [k][rows], rows a multiple of 64, as [rows / 64][k][64]: boxes of `groups` x 64 k x 64 rows, each group
// where a box of its own would lie.
bool map_groups(CUtensorMap* m, const void* p, int64_t k, int64_t rows, int groups) {
    const cuuint64_t dims[3] = {64, cuuint64_t(k), cuuint64_t(rows / 64)};
    const cuuint64_t strides[2] = {cuuint64_t(rows) * 2, 128};
    const cuuint32_t box[3] = {64, 64, cuuint32_t(groups)};
    return map_box(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// Codes [rows][cols] in boxes of 128 (64: h's) columns.
bool map_codes(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int box_rows, int box_cols) {
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)}, strides[1] = {cuuint64_t(cols)};
    const cuuint32_t box[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)};
    return map_box(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, 2, dims, strides, box,
                   box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}
bool map_codes_pair(CUtensorMap* m, const void* p, int64_t rows, int64_t cols) {
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), 2};
    const cuuint64_t strides[2] = {cuuint64_t(cols), cuuint64_t(cols * rows)};
    const cuuint32_t box[3] = {128, 128, 1};
    return map_box(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), unsigned grid, int threads, size_t smem, cudaStream_t st,
                   bool programmatic, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = programmatic ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// SM pairs of the current device; where there is none (workspace sizes asked on a host without a GPU), a GB300's.
int pairs_of() {
    const int n = sm_count() / 2;
    return n > 0 ? n : 76;
}

// Up to so many tokens they are C's columns: the block of 4096 x 11008 on 512 tokens takes 112 us (by tiles 122), on
// 640 173 (131).
constexpr int kFewTokens = 512;

// An operand's memory and its rows along M or N.
struct Operand {
    const void* p;
    int64_t rows;
};

template <int MODE, bool FP8, int TERMS>
int stages_for(int bn) {
    const int stage = TERMS * (kBoxA + bn / 2 * 128);
    const int room = (kSmemMax - 1024 - (FP8 ? kAuxFp8 : kAuxBytes) - 8 * stage_out(MODE, FP8)) / stage;
    return room > kMaxStages ? kMaxStages : room;
}

// How a product is divided: the tiles, the pairs, the partial tiles.
struct Plan {
    Args a{};
    bool columns = false;   // kPart
    int pairs = 0;
    uint32_t rest = 0;      // tiles in parts
    size_t bytes = 0;       // of the parts; kTooLarge where tiles or steps pass 32 bits (no memory holds such a call)
};
constexpr size_t kTooLarge = SIZE_MAX;

template <int MODE, bool FP8, bool A_MN, bool B_MN, int TERMS = 1>
cudaError_t launch_pairs(const Operand& a, const Operand& b, int64_t K, const Plan& p, const CUtensorMap& c0,
                         const CUtensorMap& c1, const CUtensorMap& c2, cudaStream_t st, bool programmatic) {
    CUtensorMap ma, mb;
    Args args = p.a;
    const int rows_b = args.bn / 2;
    bool ok;
    if constexpr (FP8) {
        ok = map_codes(&ma, a.p, a.rows, K, kRowsA, 128) &&
             (MODE == kGated ? map_codes_pair(&mb, b.p, b.rows, K) : map_codes(&mb, b.p, b.rows, K, rows_b, 128));
    } else if constexpr (TERMS > 1) {
        ok = (A_MN ? map_bf16_3d(&ma, a.p, TERMS, K, a.rows, 1, 64, 64)
                   : map_bf16_3d(&ma, a.p, TERMS, a.rows, K, 1, kRowsA, 64)) &&
             (B_MN ? map_bf16_3d(&mb, b.p, TERMS, K, b.rows, 1, 64, 64)
                   : map_bf16_3d(&mb, b.p, TERMS, b.rows, K, 1, rows_b, 64));
    } else {
        args.whole_a = A_MN && a.rows % 64 == 0;
        args.whole_b = B_MN && b.rows % 64 == 0 && rows_b % 64 == 0;
        ok = args.whole_a ? map_groups(&ma, a.p, K, a.rows, kRowsA / 64)
             : A_MN       ? map_bf16(&ma, a.p, K, a.rows, 64, 64)
                          : map_bf16(&ma, a.p, a.rows, K, kRowsA, 64);
        if (MODE == kGated)
            ok = ok && map_bf16_3d(&mb, b.p, 2, b.rows, K, 1, 128, 64);
        else
            ok = ok && (args.whole_b ? map_groups(&mb, b.p, K, b.rows, rows_b / 64)
                        : B_MN       ? map_bf16(&mb, b.p, K, b.rows, 64, 64)
                                     : map_bf16(&mb, b.p, b.rows, K, rows_b, 64));
    }
    if (!ok) return cudaErrorInvalidValue;
    args.stages = stages_for<MODE, FP8, TERMS>(args.bn);
    const size_t smem = 1024 + size_t(args.stages) * TERMS * (kBoxA + rows_b * 128) + 8 * stage_out(MODE, FP8) +
                        (FP8 ? kAuxFp8 : kAuxBytes);
    // The shared memory's limit is raised once a device.
    static std::atomic<uint64_t> raised{0};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (device & 63);
    if (device > 63 || !(raised.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(pair_kernel<MODE, FP8, A_MN, B_MN, TERMS>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        if (e != cudaSuccess) return e;
        if (device <= 63) raised.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch(pair_kernel<MODE, FP8, A_MN, B_MN, TERMS>, unsigned(2 * p.pairs), FP8 ? kThreads + 32 : kThreads, smem, st,
                  programmatic, ma, mb, c0, c1, c2, args);
}

// ---- plans ----
// The tiles behind `whole` in ranges of at least `least` steps.
void spread(Plan& p, int64_t tiles, int64_t whole, int least) {
    if (tiles > 0xffffffffLL || (tiles - whole) * p.a.steps > 0xffffffffLL) {
        p.pairs = 1;
        p.bytes = kTooLarge;
        return;
    }
    p.a.whole = p.a.turns = uint32_t(whole);
    p.a.tiles = uint32_t(tiles);
    p.rest = uint32_t(tiles - whole);
    p.pairs = pairs_of();
    const int64_t total = int64_t(p.rest) * p.a.steps;
    if (whole == 0) {
        const int64_t most = ceil_div(total, least);
        p.pairs = int(most < p.pairs ? most : p.pairs);
    }
    p.a.range = uint32_t(total / p.pairs), p.a.longer = uint32_t(total % p.pairs);
    p.a.slots = int(ceil_div(ceil_div(total, p.pairs), p.a.steps)) + 1;
    p.bytes = p.rest ? size_t(p.pairs) * p.a.slots * kTileM * p.a.bn * 4 : 0;
}

// How many blocks of k an accumulator takes in bf16 and FP8. Each addition of 16 products (FP8: 32) is cut to its last
// place: on sums of one sign that took 1.1 to 1.7 units of the sum so far, so that in one accumulator the weights'
// gradients of a million tokens came out 4.0e-3 to 6.6e-3 short, more than half a unit of bf16, and of this many blocks at a
// time up to 3.8e-4.
constexpr int kLongest = 1024;
static_assert(GR_MAX_FF / 128 <= kLongest, "FP8 needs no chunks");

// A product whose accumulators would take more goes in chunks of k whose sums are added up like other parts. All tiles
// are at the same chunk, so that they share their operands' reads in the L2; chunks as long as keeps the pairs busy. The
// gradient of 131072 tokens of 2560 x 10240 takes 27.0 ms (26.8 in one accumulator a tile), of 65536 13.3 either way.
void bound(Plan& p) {
    const int64_t tiles = p.a.tiles, pairs = pairs_of(), nk = p.a.nk;
    if (p.bytes == kTooLarge || nk <= kLongest || (p.a.whole == 0 && p.a.range < uint32_t(kLongest))) return;
    int64_t best = INT64_MAX;
    const int64_t fewest = ceil_div(nk, kLongest);
    for (int64_t c = fewest; c == fewest || (c < fewest + 64 && c <= nk / 256); ++c) {
        const int64_t chunk = ceil_div(nk, c), chunks = ceil_div(nk, chunk), turns = tiles * chunks;
        const int64_t time = ceil_div(turns, pairs) * (chunk + 16);   // the parts' stores: about 16 blocks
        if (time >= best - best / 32) continue;                      // more parts only where they save some time
        best = time;
        p.a.chunk = uint32_t(chunk), p.a.chunks = uint32_t(chunks);
        p.a.turns = uint32_t(turns);
        p.bytes = size_t(turns) * kTileM * p.a.bn * 4;
        if (turns > 0x7fffffffLL) p.bytes = kTooLarge;
    }
    p.a.whole = p.a.range = p.a.longer = 0;
    p.rest = uint32_t(tiles);
    p.pairs = int(p.a.turns < uint32_t(pairs) ? p.a.turns : pairs);
}

// Whole tiles of 256 x 256 (kGated: 128 channels), a pair each, as long as there are as many as pairs. The last ones,
// fewer than that, are a pair's each too, or divided along k among all the pairs where that is expected to be shorter:
// the parts and their sums cost about as much as 80 blocks of k (25 us), and pairs that are at different k share no
// reads of the L2, so that operands beyond it are read from memory more than once. Divided and not, us: dx of 8192 x
// 2560 x 10240 446 + 9 and 480, of 1536 tokens 136 + 13 and 95.
Plan plan_tiles(int64_t rows, int64_t cols, int64_t K, int per_tile, bool fp8) {
    Plan p;
    p.a.nk = int(ceil_div(K, fp8 ? 128 : 64));
    p.a.steps = fp8 ? uint32_t(ceil_div(p.a.nk, 4)) : uint32_t(p.a.nk);
    p.a.tiles_m = int(ceil_div(rows, kTileM));
    p.a.tiles_n = int(ceil_div(cols, per_tile));
    p.a.bn = 256;
    p.a.group = 8;
    p.a.rows = rows, p.a.cols = cols;
    const int64_t tiles = int64_t(p.a.tiles_m) * p.a.tiles_n, pairs = pairs_of(), rest = tiles % pairs;
    const double range = double(rest) * p.a.nk / double(pairs);
    const bool resident = (rows + cols * (256 / per_tile)) * K * (fp8 ? 1 : 2) <= (60 << 20);
    const bool divide = range >= 2 && range * (resident ? 1.0 : 1.4) + 80 < p.a.nk;
    spread(p, tiles, divide ? tiles - rest : tiles, fp8 ? 1 : 4);
    if (tiles < p.pairs && !divide) p.pairs = int(tiles);
    bound(p);
    // Not where the sums of parts come next: their CTAs, waiting beside the products, make them slower (the gradient of
    // 16384 tokens of 256 x 1024: 205 us instead of 126).
    p.a.trigger = p.rest == 0;
    return p;
}

// Few tokens: C's rows are the weights' and its columns the tokens, in tiles of as few columns as the steps of 16 (FP8:
// 32; 128 where the tokens' operand is not K-major) allow; all of them in parts.
Plan plan_columns(int64_t rows, int64_t tokens, int64_t K, int step, bool fp8, int most = 256) {
    Plan p;
    p.columns = true;
    p.a.nk = int(ceil_div(K, fp8 ? 128 : 64));
    p.a.steps = fp8 ? uint32_t(ceil_div(p.a.nk, 4)) : uint32_t(p.a.nk);
    p.a.tiles_m = int(ceil_div(rows, kTileM));
    p.a.tiles_n = int(ceil_div(tokens, most));
    p.a.bn = int(ceil_div(ceil_div(tokens, p.a.tiles_n), step) * step);
    p.a.tiles_n = int(ceil_div(tokens, p.a.bn));
    p.a.group = p.a.tiles_m;   // tile t: row tile t % tiles_m
    // The weights are read ahead and the sums' CTAs wait beside the products: 64 tokens of 256 x 1024 take 11.6 us (13.3
    // without the trigger), of 4096 x 16384 80 (83), 1000 fp32 tokens of 512 x 2048 as long as without.
    p.a.early = p.a.trigger = 1;
    spread(p, int64_t(p.a.tiles_m) * p.a.tiles_n, 0, fp8 ? 1 : 4);
    return p;
}

const CUtensorMap kNone = {};

template <int JOIN, bool F32 = false> cudaError_t join(const Plan& p, JoinArgs j, cudaStream_t st) {
    j.a = p.a;
    if (p.a.chunk) {   // a tile's chunks as ranges of one step each
        j.a.steps = p.a.chunks;
        j.a.range = 1;
        j.a.slots = 1;
    }
    if (F32 || p.columns) {
        const int64_t lines = JOIN == kJoinGatedFp8 ? ceil_div(j.rows, kBlock) * kBlock : j.rows;
        if (lines / 4 * j.cols > 0xffffffffLL - kJoinThreads) return cudaErrorInvalidValue;
        return launch(join_columns_kernel<JOIN, F32>, unsigned(ceil_div(lines / 4 * j.cols, kJoinThreads)), kJoinThreads, 0,
                      st, true, j);
    }
    const int blocks = kTileM * (JOIN == kJoinGated || JOIN == kJoinGatedFp8 ? 16 : 32) / kJoinThreads;
    return p.rest ? launch(join_tiles_kernel<JOIN>, p.rest * blocks, kJoinThreads, 0, st, true, j) : cudaSuccess;
}

bool few(int64_t tokens) { return tokens <= kFewTokens; }

// C [M][N] = A Bᵀ.
Plan plan_product(int64_t M, int64_t N, int64_t K, int64_t tokens, bool fp8) {
    if (!few(tokens)) return plan_tiles(M, N, K, 256, fp8);
    Plan p = plan_columns(N, M, K, fp8 ? 32 : 16, fp8);
    bound(p);
    return p;
}
template <bool A_K, bool B_K>
cudaError_t product(const void* a, const void* b, void* out, int64_t M, int64_t N, int64_t K, int64_t tokens,
                    float* ws, cudaStream_t st) {
    Plan p = plan_product(M, N, K, tokens, false);
    p.a.part = ws;
    JoinArgs j{};
    j.out = static_cast<__nv_bfloat16*>(out);
    j.rows = N, j.cols = M;
    cudaError_t e;
    if (p.columns) {
        if constexpr (A_K)
            e = launch_pairs<kPart, false, !B_K, false>({b, N}, {a, M}, K, p, kNone, kNone, kNone, st, true);
        else
            e = cudaErrorInvalidValue;
    } else {
        CUtensorMap c;
        if (!map_bf16(&c, out, M, N, 32, 64)) return cudaErrorInvalidValue;
        e = launch_pairs<kStore, false, !A_K, !B_K>({a, M}, {b, N}, K, p, c, kNone, kNone, st, true);
    }
    return e != cudaSuccess ? e : join<kJoinStore>(p, j, st);
}

Plan plan_gated(int64_t N, int64_t D, int64_t F, bool fp8) {
    return few(N) ? plan_columns(2 * F, N, D, fp8 ? 32 : 16, fp8) : plan_tiles(N, F, D, 128, fp8);
}
Plan plan_grad(int64_t N, int64_t D, int64_t F) {
    return few(N) ? plan_columns(F, N, D, 16, false) : plan_tiles(N, F, D, 256, false);
}

}  // namespace

cudaError_t tc_gated(int64_t N, int D, int F, int act, const void* x, const void* w_in, void* h, void* pre,
                     float* ws, cudaStream_t st) {
    Plan p = plan_gated(N, D, F, false);
    p.a.part = ws, p.a.act = act, p.a.keep = pre != nullptr;
    JoinArgs j{};
    j.out = static_cast<__nv_bfloat16*>(h), j.pre_out = static_cast<__nv_bfloat16*>(pre);
    j.rows = F, j.cols = N;
    cudaError_t e;
    if (p.columns) {
        e = launch_pairs<kPart, false, false, false>({w_in, 2 * int64_t(F)}, {x, N}, D, p, kNone, kNone, kNone, st, false);
    } else {
        CUtensorMap c, cp = kNone;
        if (!map_bf16(&c, h, N, F, 32, 64) || (pre && !map_bf16_3d(&cp, pre, N, 2, F, 32, 1, 64)))
            return cudaErrorInvalidValue;
        e = launch_pairs<kGated, false, false, false>({x, N}, {w_in, F}, D, p, c, cp, kNone, st, false);
    }
    return e != cudaSuccess ? e : join<kJoinGated>(p, j, st);
}

cudaError_t tc_gated_grad(int64_t N, int D, int F, int act, const void* dy, const void* w_out, const void* pre,
                          void* dpre, void* h, float* ws, cudaStream_t st) {
    Plan p = plan_grad(N, D, F);
    p.a.part = ws, p.a.act = act;
    JoinArgs j{};
    j.out = static_cast<__nv_bfloat16*>(h), j.dpre = static_cast<__nv_bfloat16*>(dpre), j.pre = static_cast<const __nv_bfloat16*>(pre);
    j.rows = F, j.cols = N;
    cudaError_t e;
    if (p.columns) {
        e = launch_pairs<kPart, false, true, false>({w_out, F}, {dy, N}, D, p, kNone, kNone, kNone, st, false);
    } else {
        CUtensorMap c, cp, cd;
        if (!map_bf16(&c, h, N, F, 32, 64) || !map_bf16_3d(&cp, pre, N, 2, F, 32, 1, 64) || !map_bf16_3d(&cd, dpre, N, 2, F, 32, 1, 64))
            return cudaErrorInvalidValue;
        e = launch_pairs<kGrad, false, false, true>({dy, N}, {w_out, F}, D, p, c, cp, cd, st, false);
    }
    return e != cudaSuccess ? e : join<kJoinGrad>(p, j, st);
}

cudaError_t tc_product(int64_t M, int64_t N, int64_t K, int64_t tokens, const void* a, bool a_k, const void* b,
                       bool b_k, void* out, float* ws, cudaStream_t st) {
    if (a_k)
        return b_k ? product<true, true>(a, b, out, M, N, K, tokens, ws, st)
                   : product<true, false>(a, b, out, M, N, K, tokens, ws, st);
    return b_k ? cudaErrorInvalidValue : product<false, false>(a, b, out, M, N, K, tokens, ws, st);
}

size_t tc_feed_workspace(int64_t N, int D, int F, bool gradient) {
    size_t need = 0;
    auto cover = [&](const Plan& p) { need = p.bytes > need ? p.bytes : need; };
    if (gradient) {
        cover(plan_grad(N, D, F));
        cover(plan_product(N, D, 2 * int64_t(F), N, false));
        cover(plan_product(2 * int64_t(F), D, N, INT64_MAX, false));
        cover(plan_product(D, F, N, INT64_MAX, false));
    } else {
        cover(plan_gated(N, D, F, false));
        cover(plan_product(N, D, F, N, false));
    }
    return need;
}

namespace {

// ---- fp32 ----
// The same steps with every operand as three bf16 terms and all of C in parts, whatever its size: fp32 stands for small
// models and checks.
template <bool A_K, bool B_K> Plan plan_f32(int64_t rows, int64_t cols, int64_t K) {
    Plan p = plan_columns(rows, cols, K, B_K ? 16 : 128, false, 128);
    p.a.early = 0;   // the operands' terms are of launches before
    return p;
}
// C [N][M] (C's rows along M, contiguous) = B Aᵀ.
template <int JOIN, bool A_K, bool B_K>
cudaError_t product_f32(const __nv_bfloat16* a, const __nv_bfloat16* b, int64_t M, int64_t N, int64_t K, int act,
                        JoinArgs j, float* ws, cudaStream_t st) {
    Plan p = plan_f32<A_K, B_K>(M, N, K);
    p.a.part = ws, p.a.act = act;
    const cudaError_t e = launch_pairs<kPart, false, !A_K, !B_K, 3>({a, M}, {b, N}, K, p, kNone, kNone, kNone, st, true);
    return e != cudaSuccess ? e : join<JOIN, true>(p, j, st);
}
cudaError_t cut_terms(const Cuts& c, cudaStream_t st) {
    const int64_t n = c.c[0].n + c.c[1].n + c.c[2].n, grid = ceil_div(n / 4, 256);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch(terms_kernel, unsigned(grid), 256, 0, st, false, c);
}

// The terms of a call's operands in its workspace, and the parts.
struct TermParts {
    __nv_bfloat16 *x, *w_in, *w_out, *h, *dy = nullptr, *dpre = nullptr;
    float* parts = nullptr;
    size_t bytes = 0;
    TermParts(int64_t N, int64_t D, int64_t F, bool gradient, void* ws) {
        char* base = static_cast<char*>(ws);
        auto take = [&](int64_t n, size_t width) {
            char* p = base ? base + bytes : nullptr;
            bytes += align256(size_t(n) * width);
            return p;
        };
        auto terms = [&](int64_t n) { return reinterpret_cast<__nv_bfloat16*>(take(n, 6)); };
        x = terms(N * D), w_in = terms(2 * F * D), w_out = terms(D * F), h = terms(N * F);
        if (gradient) dy = terms(N * D), dpre = terms(2 * N * F);
        size_t need = 0;
        auto cover = [&](const Plan& p) { need = p.bytes > need ? p.bytes : need; };
        if (gradient) {
            cover(plan_f32<false, true>(F, N, D));
            cover(plan_f32<false, true>(D, N, 2 * F));
            cover(plan_f32<false, false>(D, 2 * F, N));
            cover(plan_f32<false, false>(F, D, N));
        } else {
            cover(plan_f32<true, true>(2 * F, N, D));
            cover(plan_f32<true, true>(D, N, F));
        }
        // the joins count their threads, four rows of a column each, in 32 bits
        if (need == kTooLarge || N * (D > F ? D : F) > (int64_t(1) << 34) - 1024) bytes = kTooLarge;
        else parts = reinterpret_cast<float*>(take(int64_t(need), 1));
    }
};

}  // namespace

size_t f32_feed_workspace(int64_t N, int D, int F, bool gradient) { return TermParts(N, D, F, gradient, nullptr).bytes; }

cudaError_t f32_feed_forward(int64_t N, int64_t D, int64_t F, int act, const float* x, const float* w_in,
                             const float* w_out, float* y, float* pre, void* ws, cudaStream_t st) {
    const TermParts t(N, D, F, false, ws);
    cudaError_t e = cut_terms({{{x, t.x, N * D}, {w_in, t.w_in, 2 * F * D}, {w_out, t.w_out, D * F}}}, st);
    JoinArgs j{};
    j.out = t.h, j.pre_f32 = pre, j.rows = F, j.cols = N;
    if (e == cudaSuccess) e = product_f32<kJoinGated, true, true>(t.w_in, t.x, 2 * F, N, D, act, j, t.parts, st);
    j.out_f32 = y, j.rows = D, j.cols = N;
    if (e == cudaSuccess) e = product_f32<kJoinStore, true, true>(t.w_out, t.h, D, N, F, act, j, t.parts, st);
    return e;
}

cudaError_t f32_feed_backward(int64_t N, int64_t D, int64_t F, int act, const float* dy, const float* x,
                              const float* w_in, const float* w_out, const float* pre, float* dx, float* dw_in,
                              float* dw_out, void* ws, cudaStream_t st) {
    const TermParts t(N, D, F, true, ws);
    cudaError_t e = cut_terms({{{dy, t.dy, N * D}, {w_out, t.w_out, D * F}, {x, t.x, N * D}}}, st);
    if (e == cudaSuccess) e = cut_terms({{{w_in, t.w_in, 2 * F * D}, {}, {}}}, st);
    JoinArgs j{};
    j.out = t.h, j.dpre = t.dpre, j.pre_f32 = const_cast<float*>(pre), j.rows = F, j.cols = N;
    if (e == cudaSuccess) e = product_f32<kJoinGrad, false, true>(t.w_out, t.dy, F, N, D, act, j, t.parts, st);
    j.out_f32 = dx, j.rows = D, j.cols = N;
    if (e == cudaSuccess) e = product_f32<kJoinStore, false, true>(t.w_in, t.dpre, D, N, 2 * F, act, j, t.parts, st);
    j.out_f32 = dw_in, j.rows = D, j.cols = 2 * F;
    if (e == cudaSuccess) e = product_f32<kJoinStore, false, false>(t.x, t.dpre, D, 2 * F, N, act, j, t.parts, st);
    j.out_f32 = dw_out, j.rows = F, j.cols = D;
    if (e == cudaSuccess) e = product_f32<kJoinStore, false, false>(t.h, t.dy, F, D, N, act, j, t.parts, st);
    return e;
}

// ---- FP8 ----
cudaError_t tc_gated_fp8(int64_t N, int D, int F, int act, const Fp8Product& in, uint8_t* h, uint8_t* hs, float* ws,
                         cudaStream_t st) {
    Plan p = plan_gated(N, D, F, true);
    p.a.part = ws, p.a.act = act;
    p.a.scales = {in.token_scales, in.weight_scales, N, 2 * int64_t(F), F, scale_pitch(D), 0};
    JoinArgs j{};
    j.codes = h, j.scales = hs, j.scale_steps = scale_steps(F);
    j.rows = F, j.cols = N;
    cudaError_t e;
    if (p.columns) {
        e = launch_pairs<kPart, true, false, false>({in.weights, 2 * int64_t(F)}, {in.tokens, N}, D, p, kNone, kNone, kNone,
                                                    st, true);
    } else {
        CUtensorMap c;
        if (!map_codes(&c, h, N, F, 32, 64)) return cudaErrorInvalidValue;
        p.a.hs = hs, p.a.hs_steps = scale_steps(F);
        e = launch_pairs<kGated, true, false, false>({in.tokens, N}, {in.weights, F}, D, p, c, kNone, kNone, st, true);
    }
    return e != cudaSuccess ? e : join<kJoinGatedFp8>(p, j, st);
}

cudaError_t tc_product_fp8(int64_t N, int64_t O, int64_t K, const Fp8Product& in, void* out, float* ws,
                           cudaStream_t st) {
    Plan p = plan_product(N, O, K, N, true);
    p.a.part = ws;
    p.a.scales = {in.token_scales, in.weight_scales, N, O, O, scale_pitch(K), in.token_rows ? scale_pitch(K) : 0};
    JoinArgs j{};
    j.out = static_cast<__nv_bfloat16*>(out);
    j.rows = O, j.cols = N;
    cudaError_t e;
    if (p.columns) {
        e = launch_pairs<kPart, true, false, false>({in.weights, O}, {in.tokens, N}, K, p, kNone, kNone, kNone, st,
                                                    !in.token_rows);
    } else {
        CUtensorMap c;
        if (!map_bf16(&c, out, N, O, 32, 64)) return cudaErrorInvalidValue;
        e = launch_pairs<kStore, true, false, false>({in.tokens, N}, {in.weights, O}, K, p, c, kNone, kNone, st,
                                                    !in.token_rows);
    }
    return e != cudaSuccess ? e : join<kJoinStore>(p, j, st);
}

bool tc_takes_rows(int64_t N, int64_t K, const uint8_t* a_scales, const uint8_t* b_scales) {
    return few(N) && ceil_div(K, kBlock) % 4 == 0 &&
           ((reinterpret_cast<uintptr_t>(a_scales) | reinterpret_cast<uintptr_t>(b_scales)) & 3) == 0;
}
size_t tc_product_fp8_workspace(int64_t N, int64_t O, int64_t K) { return plan_product(N, O, K, N, true).bytes; }
size_t tc_feed_fp8_workspace(int64_t N, int D, int F) {
    const size_t in = plan_gated(N, D, F, true).bytes, down = plan_product(N, D, F, N, true).bytes;
    return in > down ? in : down;
}

int feed_status(bool clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_status, sizeof(v)) != cudaSuccess) return -1;
    if (clear && v) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_wait_status, &z, sizeof(z)) != cudaSuccess) return -1;
    }
    return int(v);
}

}  // namespace gr
