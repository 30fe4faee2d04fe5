// The feed-forward sublayer's products on the 5th-generation tensor cores (tcgen05, operands staged by TMA,
// accumulators in tensor memory), bf16 and FP8 blocks:
//
//     C[m][n] = Σ_k A[m][k] B[n][k]
//
// Two CTAs on neighbouring SMs form one tile of 256 x 256 (cta_group::2): each holds 128 rows of A and half of
// B's rows, so an operand byte that reaches an SM is used for 256 rows of the other operand, and an SM loads 32
// KB for 512 cycles of MMAs. A persistent grid of pairs; in each CTA one warp feeds a ring of stages by TMA, one
// (of the pair's first CTA) issues the MMAs, eight drain the accumulator: two accumulators in tensor memory, so
// the MMAs of the next tile run meanwhile.
#include <string.h>

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
// of four steps of k. Both operands e4m3; the descriptor names the byte.
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

// Where the scale bytes of an operand's rows lie: `per` rows a matrix, `block` rows a scale row.
struct Scales {
    const uint8_t* p;
    int64_t rows, per;
    int block, pitch;
    __device__ const uint8_t* at(int64_t row) const {
        if (block == 1) return p + row * pitch;
        const uint32_t r = uint32_t(row), m = uint32_t(per), which = r / m;
        return p + int64_t(which * ((m + kBlock - 1) / kBlock) + (r - which * m) / kBlock) * pitch;
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
    int steps;              // kPart: nk in steps of one block (FP8: four, what a word of scales covers)
    int64_t total;          // kPart: tiles · steps, divided evenly among the pairs
    int slots;              // kPart: partial tiles a pair may write
    float* part;
    int64_t rows, cols;     // of C (kGated: channels of h): boxes that start behind them are not stored
    Scales sa, sb;          // FP8
    uint8_t* hs;            // FP8 kGated: h's scales
    int hs_pitch;
};

constexpr int kThreads = 320;      // FP8: a warp more
constexpr uint32_t kColScales = 256;   // FP8: the scales' columns, behind the accumulators'
constexpr int kScaleSlot = 512 + 1024; // of a step of four blocks: 128 rows of A, 256 of B
constexpr int kTileM = 256, kRowsA = 128, kBoxA = kRowsA * 128;
constexpr int kMaxStages = 12;
constexpr int kAuxBytes = 512, kAuxFp8 = 512 + 2048 + 2 * kScaleSlot;
constexpr int kSmemMax = 232448;

// Staging for the outputs of a warp: kStore and kGated one box of 32 rows x 64 columns, twice; kGrad three boxes
// of 32 rows x 32 columns.
__host__ __device__ constexpr int stage_out(int mode) {
    return mode == kPart ? 0 : mode == kGrad ? 3 * 2048 : 4096;
}

struct Aux {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2], done, loaded[8];
    uint64_t scales_full[2], scales_empty[2], top_full[4];
    uint32_t tmem;
};
static_assert(sizeof(Aux) <= kAuxBytes, "aux");
// FP8, behind it: the rows' largest magnitudes in the two halves of a block [2][2][128], then two slots of scales.

// A pair's pieces of work, in the order all its roles go through them.
struct Unit {
    int m, n, k0, k1;
};
template <int MODE, int STEP> struct Units {
    const Args& a;
    int pair, pairs;
    int64_t at, end;
    int j = 0;
    __device__ Units(const Args& a, int pair, int pairs) : a(a), pair(pair), pairs(pairs) {
        at = MODE == kPart ? a.total * pair / pairs : pair;
        end = MODE == kPart ? a.total * (pair + 1) / pairs : int64_t(a.tiles_m) * a.tiles_n;
    }
    __device__ bool next(Unit& u) {
        if (at >= end) return false;
        if constexpr (MODE == kPart) {
            const int64_t t = at / a.steps, s0 = at - t * a.steps, s1 = min(int64_t(a.steps), s0 + end - at);
            u.k0 = int(s0) * STEP, u.k1 = min(int(s1) * STEP, a.nk);
            u.m = int(t % a.tiles_m), u.n = int(t / a.tiles_m);
            at += s1 - s0;
        } else {
            // groups of row tiles, so that the tiles in flight share rows of both operands in the L2
            const int64_t per = int64_t(a.group) * a.tiles_n, g = at / per, r = at - g * per;
            const int rows = min(a.group, a.tiles_m - int(g) * a.group);
            u.m = int(g) * a.group + int(r % rows), u.n = int(r / rows);
            u.k0 = 0, u.k1 = a.nk;
            at += pairs;
        }
        ++j;
        return true;
    }
};

__device__ __forceinline__ void pack8(uint4& v, const float (&f)[8]) {
    v = make_uint4(pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7]));
}
__device__ __forceinline__ float act_of(int act, float g) {
    return act == GR_SILU ? activate<GR_SILU>(g) : activate<GR_GELU>(g);
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

// tmA: K-major {k, row} box {64, 128}, MN-major {row, k} box {64, 64}. tmB: the same over bn / 2 rows (kGated: {k,
// channel, matrix} box {64, 128, 1}). tmC0: C, or h; tmC1: pre (kGated; kGrad: read); tmC2: dpre.
// FP8: codes, both operands K-major, boxes of 128 k; tmC0 of kGated: h's codes.
template <int MODE, bool FP8, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(FP8 ? kThreads + 32 : kThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
            const __grid_constant__ CUtensorMap tmC0, const __grid_constant__ CUtensorMap tmC1,
            const __grid_constant__ CUtensorMap tmC2, const __grid_constant__ Args args) {
    extern __shared__ uint8_t raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int rows_b = args.bn / 2, box_b = rows_b * 128, stage = kBoxA + box_b, stages = args.stages;
    uint8_t* out = sm + stages * stage;
    Aux& x = *reinterpret_cast<Aux*>(out + 8 * stage_out(MODE));
    uint32_t* const tops = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(&x) + kAuxBytes);
    uint8_t* const sf = reinterpret_cast<uint8_t*>(tops + 512);
    constexpr int kK = FP8 ? 128 : 64;
    // The scales take columns behind 256: one accumulator of up to 256 columns, or two of 128.
    const int accs = FP8 && args.bn > 128 ? 1 : 2, acc_cols = FP8 ? 128 : 256;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool first = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&x.full[s], 1), mbar_init(&x.empty[s], 1);
        for (int b = 0; b < 2; ++b) mbar_init(&x.acc_full[b], 1), mbar_init(&x.acc_empty[b], 16);
        for (int w = 0; w < 8; ++w) mbar_init(&x.loaded[w], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&x.scales_full[i], 2), mbar_init(&x.scales_empty[i], 1);
        for (int q = 0; q < 4; ++q) mbar_init(&x.top_full[q], 2);
        mbar_init(&x.done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc2(&x.tmem, 512);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = x.tmem;
    // what the launches before this one wrote is read from here on
    dep_wait();
    fence_async_global();
    dep_launch_dependents();

    Units<MODE, FP8 ? 4 : 1> units(args, int(cluster_id_x()), int(ncluster_x()));
    Unit u;
    if (warp == 0) {
        if (lane == 0) {
            const uint32_t bytes = 2u * uint32_t(stage);
            uint32_t g = 0;
            bool ok = true;
            while (ok && units.next(u)) {
                const int m0 = u.m * kTileM + int(rank) * kRowsA;
                const int n0 = u.n * (MODE == kGated ? 128 : args.bn) + (MODE == kGated ? 0 : int(rank) * rows_b);
                for (int kb = u.k0; kb < u.k1; ++kb, ++g) {
                    const uint32_t s = g % stages;
                    if (g >= uint32_t(stages) && !mbar_wait(&x.empty[s], ((g / stages) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    // the first CTA's barrier counts both CTAs' bytes
                    if (first) mbar_expect_tx(&x.full[s], bytes);
                    const uint32_t bar = map_rank(smem_u32(&x.full[s]), 0);
                    uint8_t *pa = sm + s * stage, *pb = pa + kBoxA;
                    if constexpr (A_MN) {
                        tma_pair_2d(pa, &tmA, m0, kb * kK, bar);
                        tma_pair_2d(pa + 8192, &tmA, m0 + 64, kb * kK, bar);
                    } else {
                        tma_pair_2d(pa, &tmA, kb * kK, m0, bar);
                    }
                    if constexpr (MODE == kGated) {
                        tma_pair_3d(pb, &tmB, kb * kK, n0, int(rank), bar);
                    } else if constexpr (B_MN) {
                        for (int i = 0; i < rows_b; i += 64)
                            tma_pair_2d(pb + i * 128, &tmB, n0 + i, kb * kK, bar);
                    } else {
                        tma_pair_2d(pb, &tmB, kb * kK, n0, bar);
                    }
                }
            }
            // no copy is under way when the CTAs leave: the first CTA sees both CTAs' arrive
            if (first)
                for (uint32_t i = g > uint32_t(stages) ? g - stages : 0; i < g; ++i)
                    mbar_wait(&x.full[i % stages], (i / stages) & 1);
        }
    } else if (warp == 1) {
        if (first && lane == 0) {
            const uint32_t idesc = idesc_bf16_f32(256, args.bn) | (A_MN ? 1u << 15 : 0) | (B_MN ? 1u << 16 : 0);
            uint32_t g = 0, q = 0;
            bool ok = true;
            for (int j = 0; ok && units.next(u); ++j) {
                const int b = j % accs;
                if (j >= accs && !mbar_wait(&x.acc_empty[b], (j / accs - 1) & 1)) break;
                tc_fence_after();
                const uint32_t d = tmem + b * acc_cols;
                for (int kb = u.k0; kb < u.k1; ++kb, ++g) {
                    const uint32_t s = g % stages, step = uint32_t(kb - u.k0) & 3;
                    if (FP8 && step == 0) {
                        // the scales of this and the next three blocks; the copies run in order with the MMAs
                        if (!mbar_wait(&x.scales_full[q & 1], (q >> 1) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t at = smem_u32(sf) + (q & 1) * kScaleSlot, to = tmem + kColScales + (q & 1) * 16;
                        for (int i = 0; i < 1 + (args.bn + 127) / 128; ++i) tc_copy_scales(to + i * 4, at + i * 512);
                        ++q;
                    }
                    if (!mbar_wait(&x.full[s], (g / stages) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t pa = smem_u32(sm + s * stage), pb = pa + kBoxA;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (FP8) {
                            const uint32_t sfa = tmem + kColScales + ((q - 1) & 1) * 16;
                            tc_mma2_fp8(d, sdesc_sw128(pa + k * 32), sdesc_sw128(pb + k * 32),
                                        idesc_fp8(args.bn, int(step)), sfa, sfa + 4, kb > u.k0 || k > 0);
                        } else {
                            tc_mma2(d, A_MN ? sdesc_mn(pa + k * 2048, 8192) : sdesc_sw128(pa + k * 32),
                                    B_MN ? sdesc_mn(pb + k * 2048, 8192) : sdesc_sw128(pb + k * 32), idesc,
                                    kb > u.k0 || k > 0);
                        }
                    }
                    tc_commit2(&x.empty[s]);
                    if (FP8 && (step == 3 || kb + 1 == u.k1)) tc_commit2(&x.scales_empty[(q - 1) & 1]);
                }
                if (ok) tc_commit2(&x.acc_full[b]);
            }
            tc_commit2(&x.done);
            mbar_wait(&x.done, 0);
        }
    } else if (FP8 && warp == 10) {
        // Scales: four bytes (blocks) of 128 rows of A and bn of B into shared memory, where row r's word lies at
        // 16 (r % 32) + 4 (r / 32) of its 128 rows. The next step's are on their way while a slot is waited for.
        struct Words {
            uint32_t a[4], b[8];
        };
        const Scales &sa = args.sa, &sb = args.sb;
        const bool whole_a = ((reinterpret_cast<uintptr_t>(sa.p) | sa.pitch) & 3) == 0;
        const bool whole_b = ((reinterpret_cast<uintptr_t>(sb.p) | sb.pitch) & 3) == 0;
        // a lane's rows of a tile: where their scales begin, null behind the last row
        const uint8_t *pa[4], *pb[8];
        auto find = [&](const Unit& t) {
            const int64_t m0 = int64_t(t.m) * kTileM + rank * kRowsA;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = m0 + i * 32 + lane;
                pa[i] = row < sa.rows ? sa.at(row) : nullptr;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = i * 32 + lane;
                int64_t row = int64_t(t.n) * args.bn + r;
                if (MODE == kGated) {
                    const int64_t ch = int64_t(t.n) * 128 + (r & 127);
                    row = ch < sb.per ? ch + (r >> 7) * sb.per : sb.rows;
                }
                pb[i] = r < args.bn && row < sb.rows ? sb.at(row) : nullptr;
            }
        };
        auto word = [&](const uint8_t* p, bool whole, int kb) -> uint32_t {
            if (!p) return 0x7f7f7f7fu;
            p += kb;
            if (whole) return *reinterpret_cast<const uint32_t*>(p);   // within the padded row
            uint32_t v = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (kb + i < args.nk) v |= uint32_t(p[i]) << (8 * i);
            return v;
        };
        auto fetch = [&](int kb, Words& v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v.a[i] = word(pa[i], whole_a, kb);
#pragma unroll
            for (int i = 0; i < 8; ++i) v.b[i] = word(pb[i], whole_b, kb);
        };
        Words v;
        uint32_t q = 0;
        bool more = units.next(u);
        int kb = u.k0;
        if (more) find(u), fetch(kb, v);
        while (more) {
            const Words now = v;
            kb += 4;
            if (kb >= u.k1) {
                more = units.next(u);
                kb = u.k0;
                if (more) find(u);
            }
            if (more) fetch(kb, v);
            if (q >= 2 && !mbar_wait(&x.scales_empty[q & 1], ((q >> 1) - 1) & 1)) break;
            const uint32_t at = smem_u32(sf) + (q & 1) * kScaleSlot + lane * 16;
            st_shared16(at, make_uint4(now.a[0], now.a[1], now.a[2], now.a[3]));
            st_shared16(at + 512, make_uint4(now.b[0], now.b[1], now.b[2], now.b[3]));
            st_shared16(at + 1024, make_uint4(now.b[4], now.b[5], now.b[6], now.b[7]));
            fence_async_shared();
            __syncwarp();
            if (lane == 0) arrive_remote(map_rank(smem_u32(&x.scales_full[q & 1]), 0));
            ++q;
        }
    } else {
        const int w = warp - 2, half = w >> 2, quad = warp & 3;
        const uint32_t mine = smem_u32(out) + w * stage_out(MODE);
        uint8_t* const minep = out + w * stage_out(MODE);
        const uint32_t lanes = uint32_t(quad) << 21;   // lane field of a tensor-memory address: quad * 32 << 16
        // kGrad: pre's boxes of the next 32 channels, read ahead
        uint32_t loads = 0, waits = 0;
        auto load_pre = [&](int row, int ch) {
            ++loads;
            if (lane == 0) {
                bulk_wait_read<0>();
                mbar_expect_tx(&x.loaded[w], 4096);
                tma_load_3d(minep, &tmC1, ch, 0, row, &x.loaded[w]);
                tma_load_3d(minep + 2048, &tmC1, ch, 1, row, &x.loaded[w]);
            }
        };
        bool more = units.next(u);
        if (MODE == kGrad && more)
            load_pre(u.m * kTileM + int(rank) * kRowsA + quad * 32, u.n * 256 + half * 128);
        for (int j = 0; more; ++j) {
            const int b = j % accs;
            const Unit now = u;
            if (!mbar_wait(&x.acc_full[b], (j / accs) & 1)) break;
            tc_fence_after();
            const uint32_t acc = tmem + b * acc_cols + lanes;
            const int row = now.m * kTileM + int(rank) * kRowsA + quad * 32;   // the warp's first
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
            if constexpr (MODE == kStore) {
                const int col = now.n * 256 + half * 128;
                float v[64];
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    get64(half * 128 + i * 64, v);
                    if (i == 1) drained();
                    put_box(v, [&] {
                        if (col + i * 64 < args.cols) tma_store_2d(&tmC0, minep, col + i * 64, row);
                    });
                }
            } else if constexpr (MODE == kGated) {
                const int col = now.n * 128 + half * 64;
                float ga[64], up[64];
                get64(half * 64, ga);
                get64(128 + half * 64, up);
                drained();
                const bool in = col < args.cols;
                if (args.keep && in) {
                    put_box(ga, [&] { tma_store_3d(&tmC1, minep, col, 0, row); });
                    put_box(up, [&] { tma_store_3d(&tmC1, minep, col, 1, row); });
                }
                if (args.act == GR_SILU) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) ga[i] = activate<GR_SILU>(ga[i]) * up[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 64; ++i) ga[i] = activate<GR_GELU>(ga[i]) * up[i];
                }
                if constexpr (FP8) {
                    // the block's largest magnitude: this half's and the other's, from the warp that has the same rows
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < 64; ++i) top = max(top, block_mag(ga[i]));
                    uint32_t* t = tops + (j & 1) * 256 + quad * 32 + lane;
                    t[half * 128] = top;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x.top_full[quad]);
                    if (!mbar_wait(&x.top_full[quad], j & 1)) break;
                    top = max(top, *const_cast<volatile uint32_t*>(t + (half ^ 1) * 128));
                    float inv;
                    const uint8_t e = block_scale(top, inv);
                    if (half == 0 && row + lane < args.rows)
                        args.hs[int64_t(row + lane) * args.hs_pitch + now.n] = e;
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
                more = units.next(u);
                bool ok = true;
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    float dh[32];
                    {
                        uint32_t r[2][16];
                        tmem_ld16_nowait(acc + half * 128 + i * 32, r[0]);
                        tmem_ld16_nowait(acc + half * 128 + i * 32 + 16, r[1]);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            tmem_wait_ld(r[q]);
#pragma unroll
                            for (int k = 0; k < 16; ++k) dh[q * 16 + k] = __uint_as_float(r[q][k]);
                        }
                    }
                    if (i == 3) drained();
                    ok = ok && mbar_wait(&x.loaded[w], waits++ & 1);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float g[8], p[8], a[8], s[8];
                        unpack8(ld_shared16(mine + swz64(lane, c)), g);
                        unpack8(ld_shared16(mine + 2048 + swz64(lane, c)), p);
                        if (args.act == GR_SILU) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                a[k] = activate<GR_SILU>(g[k]);
                                s[k] = activate_slope<GR_SILU>(g[k]);
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                a[k] = activate<GR_GELU>(g[k]);
                                s[k] = activate_slope<GR_GELU>(g[k]);
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            s[k] *= dh[c * 8 + k] * p[k];
                            p[k] *= a[k];
                            a[k] *= dh[c * 8 + k];
                        }
                        uint4 v;
                        pack8(v, s);
                        st_shared16(mine + swz64(lane, c), v);
                        pack8(v, a);
                        st_shared16(mine + 2048 + swz64(lane, c), v);
                        pack8(v, p);
                        st_shared16(mine + 4096 + swz64(lane, c), v);
                    }
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0 && ok && row < args.rows && col + i * 32 < args.cols) {
                        tma_store_3d(&tmC2, minep, col + i * 32, 0, row);
                        tma_store_3d(&tmC2, minep + 2048, col + i * 32, 1, row);
                        tma_store_2d(&tmC0, minep + 4096, col + i * 32, row);
                        bulk_commit();
                    }
                    if (ok && i < 3)
                        load_pre(row, col + (i + 1) * 32);
                    else if (ok && more)
                        load_pre(u.m * kTileM + int(rank) * kRowsA + quad * 32, u.n * 256 + half * 128);
                }
                if (!ok) break;
            } else {
                float* p = args.part + (int64_t(cluster_id_x()) * args.slots + j) * (int64_t(kTileM) * args.bn) +
                           int(rank) * kRowsA + quad * 32 + lane;
                for (int c = half * 16; c < args.bn; c += 32) {
                    float v[16];
                    tmem_ld16(acc + c, v);
#pragma unroll
                    for (int k = 0; k < 16; ++k) p[int64_t(c + k) * kTileM] = v[k];
                }
                drained();
            }
            if (MODE != kGrad) more = units.next(u);
        }
        if (MODE == kGrad && waits < loads) mbar_wait(&x.loaded[w], waits & 1);
        if (lane == 0) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc2(tmem, 512);
}

// ---- the sums of the pairs' parts ---------------------------------------------------------------
// C's tile t of kPart is spread over the pairs whose ranges of k meet it, in order; a pair's slots hold its tiles
// [column][256 rows]. Four rows of a column a thread, rows contiguous in the output.
enum Join { kJoinStore, kJoinGated, kJoinGrad, kJoinGatedFp8 };

struct JoinArgs {
    const float* part;
    int64_t total, rows, cols;   // of the output (kJoinGated: channels)
    int steps, tiles_m, bn, slots, pairs, act;
    __nv_bfloat16 *out, *pre_out;
    const __nv_bfloat16* pre;
    __nv_bfloat16* dpre;
    uint8_t *codes, *scales;     // kJoinGatedFp8: h
    int pitch;
};

__device__ __forceinline__ float4 joined(const JoinArgs& a, int64_t row, int64_t col) {
    const int64_t tn = col / a.bn, t = tn * a.tiles_m + row / kTileM, k0 = t * a.steps;
    const int64_t at = (col - tn * a.bn) * kTileM + row % kTileM, tile = int64_t(kTileM) * a.bn;
    int64_t c = ((k0 + 1) * a.pairs - 1) / a.total;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (; c < a.pairs; ++c) {
        const int64_t begin = a.total * c / a.pairs;
        if (begin >= k0 + a.steps) break;
        const int64_t slot = c * a.slots + (t - begin / a.steps);
        const float4 v = __ldcs(reinterpret_cast<const float4*>(a.part + slot * tile + at));
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    return s;
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, float a, float b, float c, float d) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf2(a, b), pack_bf2(c, d));
}
__device__ __forceinline__ void get4(const __nv_bfloat16* p, float (&v)[4]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
}

template <int JOIN>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinArgs a) {
    dep_wait();
    dep_launch_dependents();
    const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (i >= a.rows * a.cols) return;
    const int64_t col = i / a.rows, row = i - col * a.rows;
    const float4 s = joined(a, row, col);
    if constexpr (JOIN == kJoinStore) {
        put4(a.out + i, s.x, s.y, s.z, s.w);
    } else if constexpr (JOIN == kJoinGated) {
        const float4 p = joined(a, a.rows + row, col);
        const float g[4] = {s.x, s.y, s.z, s.w}, up[4] = {p.x, p.y, p.z, p.w};
        float h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = act_of(a.act, g[k]) * up[k];
        put4(a.out + i, h[0], h[1], h[2], h[3]);
        if (a.pre_out) {
            put4(a.pre_out + 2 * col * a.rows + row, g[0], g[1], g[2], g[3]);
            put4(a.pre_out + (2 * col + 1) * a.rows + row, up[0], up[1], up[2], up[3]);
        }
    } else {
        const float dh[4] = {s.x, s.y, s.z, s.w};
        float g[4], p[4], f[4], d[4];
        get4(a.pre + 2 * col * a.rows + row, g);
        get4(a.pre + (2 * col + 1) * a.rows + row, p);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = act_of(a.act, g[k]);
            d[k] = dh[k] * p[k] * (a.act == GR_SILU ? activate_slope<GR_SILU>(g[k]) : activate_slope<GR_GELU>(g[k]));
            p[k] *= f[k];
            f[k] *= dh[k];
        }
        put4(a.dpre + 2 * col * a.rows + row, d[0], d[1], d[2], d[3]);
        put4(a.dpre + (2 * col + 1) * a.rows + row, f[0], f[1], f[2], f[3]);
        put4(a.out + i, p[0], p[1], p[2], p[3]);
    }
}

// h in blocks of 128 channels of a column, a warp each.
__global__ void __launch_bounds__(256) join_fp8_kernel(const __grid_constant__ JoinArgs a) {
    dep_wait();
    dep_launch_dependents();
    const int nb = int((a.rows + kBlock - 1) / kBlock);
    const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) / 32;
    if (i >= a.cols * nb) return;
    const int lane = threadIdx.x & 31;
    const int64_t col = i / nb, row = (i - col * nb) * kBlock + lane * 4;
    float h[4] = {};
    if (row < a.rows) {
        const float4 s = joined(a, row, col), p = joined(a, a.rows + row, col);
        const float g[4] = {s.x, s.y, s.z, s.w}, up[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = act_of(a.act, g[k]) * up[k];
    }
    uint32_t top = max(max(block_mag(h[0]), block_mag(h[1])), max(block_mag(h[2]), block_mag(h[3])));
    top = __reduce_max_sync(~0u, top);
    float inv;
    const uint8_t e = block_scale(top, inv);
    if (row < a.rows) *reinterpret_cast<uint32_t*>(a.codes + col * a.rows + row) = block_codes4(h, inv);
    if (lane == 0) a.scales[col * a.pitch + (i - col * nb)] = e;
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
                   box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}
// [a][b][cols] with boxes over one of a or b.
bool map_bf16_3d(CUtensorMap* m, const void* p, int64_t a, int64_t b, int64_t cols, int box_a, int box_b,
                 int box_cols) {
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(b), cuuint64_t(a)};
    const cuuint64_t strides[2] = {cuuint64_t(cols) * 2, cuuint64_t(cols * b) * 2};
    const cuuint32_t box[3] = {cuuint32_t(box_cols), cuuint32_t(box_b), cuuint32_t(box_a)};
    return map_box(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, 3, dims, strides, box,
                   box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
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
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
    }
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

int pairs_of() { return sm_count() / 2; }

// An operand's memory and its rows along M or N.
struct Operand {
    const void* p;
    int64_t rows;
};

template <int MODE, bool FP8>
int stages_for(int bn) {
    const int stage = kBoxA + bn / 2 * 128;
    const int room = (kSmemMax - 1024 - (FP8 ? kAuxFp8 : kAuxBytes) - 8 * stage_out(MODE)) / stage;
    return room > kMaxStages ? kMaxStages : room;
}

template <int MODE, bool FP8, bool A_MN, bool B_MN>
cudaError_t launch_pairs(const Operand& a, const Operand& b, int64_t K, Args args, int pairs, const CUtensorMap& c0,
                         const CUtensorMap& c1, const CUtensorMap& c2, cudaStream_t st, bool programmatic) {
    CUtensorMap ma, mb;
    const int rows_b = args.bn / 2;
    bool ok;
    if constexpr (FP8) {
        ok = map_codes(&ma, a.p, a.rows, K, kRowsA, 128) &&
             (MODE == kGated ? map_codes_pair(&mb, b.p, b.rows, K) : map_codes(&mb, b.p, b.rows, K, rows_b, 128));
    } else {
        ok = A_MN ? map_bf16(&ma, a.p, K, a.rows, 64, 64) : map_bf16(&ma, a.p, a.rows, K, kRowsA, 64);
        if (MODE == kGated)
            ok = ok && map_bf16_3d(&mb, b.p, 2, b.rows, K, 1, 128, 64);
        else
            ok = ok && (B_MN ? map_bf16(&mb, b.p, K, b.rows, 64, 64) : map_bf16(&mb, b.p, b.rows, K, rows_b, 64));
    }
    if (!ok) return cudaErrorInvalidValue;
    args.stages = stages_for<MODE, FP8>(args.bn);
    const size_t smem = 1024 + size_t(args.stages) * (kBoxA + rows_b * 128) + 8 * stage_out(MODE) +
                        (FP8 ? kAuxFp8 : kAuxBytes);
    return launch(pair_kernel<MODE, FP8, A_MN, B_MN>, unsigned(2 * pairs), FP8 ? kThreads + 32 : kThreads, smem, st,
                  programmatic, ma, mb, c0, c1, c2, args);
}

// ---- whole tiles ----
Args whole(int64_t rows, int64_t cols, int64_t K, int per_tile, int kk = 64) {
    Args a{};
    a.nk = int(ceil_div(K, kk));
    a.tiles_m = int(ceil_div(rows, kTileM));
    a.tiles_n = int(ceil_div(cols, per_tile));
    a.bn = 256;
    a.group = 8;
    return a;
}
int pairs_for(const Args& a) {
    const int64_t tiles = int64_t(a.tiles_m) * a.tiles_n;
    return int(tiles < pairs_of() ? tiles : pairs_of());
}

// ---- parts ----
struct Parts {
    Args a{};
    int pairs = 0;
    size_t bytes = 0;
};
// C [rows][cols] over K in parts: the tiles' columns as even as the steps of 16 (FP8: 32; 128) allow, k divided among
// the pairs in ranges of at least four blocks.
Parts parts_of(int64_t rows, int64_t cols, int64_t K, int step, bool fp8 = false) {
    Parts p;
    p.a.nk = int(ceil_div(K, fp8 ? 128 : 64));
    p.a.steps = fp8 ? int(ceil_div(p.a.nk, 4)) : p.a.nk;
    p.a.tiles_m = int(ceil_div(rows, kTileM));
    p.a.tiles_n = int(ceil_div(cols, 256));
    p.a.bn = int(ceil_div(ceil_div(cols, p.a.tiles_n), step) * step);
    p.a.tiles_n = int(ceil_div(cols, p.a.bn));
    p.a.total = int64_t(p.a.tiles_m) * p.a.tiles_n * p.a.steps;
    const int64_t most = fp8 ? p.a.total : ceil_div(p.a.total, 4);
    p.pairs = int(most < pairs_of() ? most : pairs_of());
    p.a.slots = int(ceil_div(ceil_div(p.a.total, p.pairs), p.a.steps)) + 1;
    p.bytes = size_t(p.pairs) * p.a.slots * kTileM * p.a.bn * 4;
    return p;
}

JoinArgs join_args(const Parts& p, float* ws, int64_t rows, int64_t cols, int act) {
    JoinArgs j{};
    j.part = ws;
    j.total = p.a.total, j.rows = rows, j.cols = cols;
    j.steps = p.a.steps, j.tiles_m = p.a.tiles_m, j.bn = p.a.bn, j.slots = p.a.slots, j.pairs = p.pairs, j.act = act;
    return j;
}
template <int JOIN>
cudaError_t join(const Parts& p, float* ws, int64_t rows, int64_t cols, int act, void* out, const void* pre,
                 void* pre_out, void* dpre, cudaStream_t st) {
    JoinArgs j = join_args(p, ws, rows, cols, act);
    j.out = static_cast<__nv_bfloat16*>(out);
    j.pre_out = static_cast<__nv_bfloat16*>(pre_out);
    j.pre = static_cast<const __nv_bfloat16*>(pre);
    j.dpre = static_cast<__nv_bfloat16*>(dpre);
    return launch(join_kernel<JOIN>, unsigned(ceil_div(rows * cols / 4, 256)), 256, 0, st, true, j);
}

// Whether a product goes in parts. Its tokens are the columns of the parts' form.
bool in_parts(int64_t tokens, const Args& direct) {
    const int64_t tiles = int64_t(direct.tiles_m) * direct.tiles_n, slots = ceil_div(tiles, pairs_of()) * pairs_of();
    return tokens <= 256 || tiles * 10 < slots * 7;
}

const CUtensorMap kNone = {};

// C [M][N] = A Bᵀ as whole tiles, or in parts as Cᵀ with the rows along N.
template <bool A_K, bool B_K>
cudaError_t product(const void* a, const void* b, void* out, int64_t M, int64_t N, int64_t K, int64_t tokens,
                    float* ws, cudaStream_t st, bool programmatic) {
    Args w = whole(M, N, K, 256);
    if (!in_parts(tokens, w)) {
        CUtensorMap c;
        if (!map_bf16(&c, out, M, N, 32, 64)) return cudaErrorInvalidValue;
        w.rows = M, w.cols = N;
        return launch_pairs<kStore, false, !A_K, !B_K>({a, M}, {b, N}, K, w, pairs_for(w), c, kNone, kNone, st,
                                                programmatic);
    }
    Parts p = parts_of(N, M, K, A_K ? 16 : 128);
    p.a.part = ws;
    const cudaError_t e = launch_pairs<kPart, false, !B_K, !A_K>({b, N}, {a, M}, K, p.a, p.pairs, kNone, kNone, kNone, st,
                                                          programmatic);
    return e != cudaSuccess ? e : join<kJoinStore>(p, ws, N, M, 0, out, nullptr, nullptr, nullptr, st);
}
size_t product_bytes(int64_t M, int64_t N, int64_t K, int64_t tokens, bool a_k) {
    return in_parts(tokens, whole(M, N, K, 256)) ? parts_of(N, M, K, a_k ? 16 : 128).bytes : 0;
}

}  // namespace

cudaError_t tc_gated(int64_t N, int D, int F, int act, const void* x, const void* w_in, void* h, void* pre,
                     float* ws, cudaStream_t st) {
    Args w = whole(N, F, D, 128);
    if (!in_parts(N, w)) {
        CUtensorMap c, cp = kNone;
        if (!map_bf16(&c, h, N, F, 32, 64) || (pre && !map_bf16_3d(&cp, pre, N, 2, F, 32, 1, 64)))
            return cudaErrorInvalidValue;
        w.rows = N, w.cols = F, w.act = act, w.keep = pre != nullptr;
        return launch_pairs<kGated, false, false, false>({x, N}, {w_in, F}, D, w, pairs_for(w), c, cp, kNone, st, false);
    }
    Parts p = parts_of(2 * int64_t(F), N, D, 16);
    p.a.part = ws;
    const cudaError_t e = launch_pairs<kPart, false, false, false>({w_in, 2 * int64_t(F)}, {x, N}, D, p.a, p.pairs, kNone,
                                                            kNone, kNone, st, false);
    return e != cudaSuccess ? e : join<kJoinGated>(p, ws, F, N, act, h, nullptr, pre, nullptr, st);
}

cudaError_t tc_gated_grad(int64_t N, int D, int F, int act, const void* dy, const void* w_out, const void* pre,
                          void* dpre, void* h, float* ws, cudaStream_t st) {
    Args w = whole(N, F, D, 256);
    if (!in_parts(N, w)) {
        CUtensorMap c, cp, cd;
        if (!map_bf16(&c, h, N, F, 32, 32) || !map_bf16_3d(&cp, pre, N, 2, F, 32, 1, 32) ||
            !map_bf16_3d(&cd, dpre, N, 2, F, 32, 1, 32))
            return cudaErrorInvalidValue;
        w.rows = N, w.cols = F, w.act = act;
        return launch_pairs<kGrad, false, false, true>({dy, N}, {w_out, F}, D, w, pairs_for(w), c, cp, cd, st, false);
    }
    Parts p = parts_of(F, N, D, 16);
    p.a.part = ws;
    const cudaError_t e = launch_pairs<kPart, false, true, false>({w_out, F}, {dy, N}, D, p.a, p.pairs, kNone, kNone,
                                                           kNone, st, false);
    return e != cudaSuccess ? e : join<kJoinGrad>(p, ws, F, N, act, h, pre, nullptr, dpre, st);
}

cudaError_t tc_product(int64_t M, int64_t N, int64_t K, int64_t tokens, const void* a, bool a_k, const void* b,
                       bool b_k, void* out, float* ws, cudaStream_t st) {
    if (a_k)
        return b_k ? product<true, true>(a, b, out, M, N, K, tokens, ws, st, true)
                   : product<true, false>(a, b, out, M, N, K, tokens, ws, st, true);
    return b_k ? cudaErrorInvalidValue : product<false, false>(a, b, out, M, N, K, tokens, ws, st, true);
}

// ---- FP8 ----
cudaError_t tc_gated_fp8(int64_t N, int D, int F, int act, Fp8Matrix x, int x_pitch, Fp8Matrix w_in, uint8_t* h,
                         uint8_t* hs, int hs_pitch, float* ws, cudaStream_t st, bool programmatic) {
    const int db = int(ceil_div(D, kBlock));
    const Scales sx{x.scales, N, N, 1, x_pitch}, sw{w_in.scales, 2 * int64_t(F), F, kBlock, db};
    Args w = whole(N, F, D, 128, 128);
    if (!in_parts(N, w)) {
        CUtensorMap c;
        if (!map_codes(&c, h, N, F, 32, 64)) return cudaErrorInvalidValue;
        w.rows = N, w.cols = F, w.act = act, w.sa = sx, w.sb = sw, w.hs = hs, w.hs_pitch = hs_pitch;
        return launch_pairs<kGated, true, false, false>({x.codes, N}, {w_in.codes, F}, D, w, pairs_for(w), c, kNone,
                                                        kNone, st, programmatic);
    }
    Parts p = parts_of(2 * int64_t(F), N, D, 32, true);
    p.a.part = ws, p.a.sa = sw, p.a.sb = sx;
    cudaError_t e = launch_pairs<kPart, true, false, false>({w_in.codes, 2 * int64_t(F)}, {x.codes, N}, D, p.a,
                                                            p.pairs, kNone, kNone, kNone, st, programmatic);
    if (e != cudaSuccess) return e;
    JoinArgs j = join_args(p, ws, F, N, act);
    j.codes = h, j.scales = hs, j.pitch = hs_pitch;
    return launch(join_fp8_kernel, unsigned(ceil_div(N * ceil_div(F, kBlock), 8)), 256, 0, st, true, j);
}

cudaError_t tc_product_fp8(int64_t N, int64_t O, int64_t K, Fp8Matrix a, int a_pitch, Fp8Matrix b, void* out,
                           float* ws, cudaStream_t st, bool programmatic) {
    const int kb = int(ceil_div(K, kBlock));
    const Scales sa{a.scales, N, N, 1, a_pitch}, sb{b.scales, O, O, kBlock, kb};
    Args w = whole(N, O, K, 256, 128);
    if (!in_parts(N, w)) {
        CUtensorMap c;
        if (!map_bf16(&c, out, N, O, 32, 64)) return cudaErrorInvalidValue;
        w.rows = N, w.cols = O, w.sa = sa, w.sb = sb;
        return launch_pairs<kStore, true, false, false>({a.codes, N}, {b.codes, O}, K, w, pairs_for(w), c, kNone,
                                                        kNone, st, programmatic);
    }
    Parts p = parts_of(O, N, K, 32, true);
    p.a.part = ws, p.a.sa = sb, p.a.sb = sa;
    const cudaError_t e = launch_pairs<kPart, true, false, false>({b.codes, O}, {a.codes, N}, K, p.a, p.pairs, kNone,
                                                                  kNone, kNone, st, programmatic);
    return e != cudaSuccess ? e : join<kJoinStore>(p, ws, O, N, 0, out, nullptr, nullptr, nullptr, st);
}

size_t tc_product_fp8_workspace(int64_t N, int64_t O, int64_t K) {
    return in_parts(N, whole(N, O, K, 256, 128)) ? parts_of(O, N, K, 32, true).bytes : 0;
}
size_t tc_feed_fp8_workspace(int64_t N, int D, int F) {
    const size_t down = tc_product_fp8_workspace(N, D, F);
    const size_t in = in_parts(N, whole(N, F, D, 128, 128)) ? parts_of(2 * int64_t(F), N, D, 32, true).bytes : 0;
    return in > down ? in : down;
}

size_t tc_feed_workspace(int64_t N, int D, int F, bool gradient) {
    size_t need = 0;
    auto cover = [&](size_t n) { need = n > need ? n : need; };
    if (gradient) {
        if (in_parts(N, whole(N, F, D, 256))) cover(parts_of(F, N, D, 16).bytes);
        cover(product_bytes(N, D, 2 * int64_t(F), N, true));
        cover(product_bytes(2 * int64_t(F), D, N, INT64_MAX, false));
        cover(product_bytes(D, F, N, INT64_MAX, false));
    } else {
        if (in_parts(N, whole(N, F, D, 128))) cover(parts_of(2 * int64_t(F), N, D, 16).bytes);
        cover(product_bytes(N, D, F, N, true));
    }
    return need;
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
