// Linear attention with a decay for each head on the 5th-generation tensor cores (tcgen05,
// accumulators in tensor memory, operands staged by TMA): bf16 rows, head sizes 64 and 128. The
// masked, decayed product of gr_mixer.h, in chunks of 128 tokens; a prompt and each of its three
// gradients is one pass of it.
//
// A chunk's rows i = 0..127 (λ the head's decay, M the state before the chunk):
//     P_ij  = outer weight λ^{i−j} (a_i·b_j) for j <= i           MMA 1, then WG A (mask, decay, bf16)
//     out_i = Σ_j P_ij c_j + outer λ^{i+1} (Mᵀ a_i)               MMA 4 and MMA 2, then WG A
//     M'    = λ^len M + Σ_j b_j (weight λ^{len−1−j} c_j)ᵀ         WG V0, V1 scale c, MMA 3, then WG M
// (backwards in time the exponents run the other way.) No exponent is negative, so no decay overflows.
//
// The state M stays in registers, in fp32, for all chunks of a segment. Its update is a product of
// bf16 operands, so the decayed values are split into three bf16 terms (24 bits together): the
// state's error is that of fp32 (two terms leave 2.2e-6 of it). P and the copy of M that the outputs read
// are rounded to bf16 once, each in its own share of the output: with the output's own rounding 1.41 times
// that one's error alone.
//
// One CTA an SM (its shared memory and all 512 columns of tensor memory). At head size 128 a chunk moves
// 128 KB, 2.9 us at an SM's share of the measured copy bandwidth, and takes 3072 cycles (1.6 us) of the
// tensor cores; it is done every 3.9 us (8192 tokens of 152 heads: 249 us, 5.1 TB/s; head size 64: 182 us).
// What bounds it are the 13 thousand warp instructions between the MMAs, at 6.6 cycles an instruction and
// 41% of the issue slots, most of them the split of the decayed values. Each step has a warpgroup of its
// own and works ahead of the next. Measured and not kept: outputs staged in c's tile and stored by
// TMA (277 us: the tile's next load waits for them), the roles on seven warpgroups with M in tensor memory
// (277 us), on three (377 us); M added up by the MMAs in tensor memory would round with every one.
//
// Prompts with too few heads and sequences to fill the SMs are cut into segments: a first launch
// forms each segment's own sum, a scan turns the sums into the states the segments start from, and the pass
// runs on all segments at once (32768 tokens of 32 heads: 144 + 8 + 241 us; uncut 945 us).
//
// Warps: 0 TMA producer, 1 issuer of the scores' and outputs' MMAs (owns the tensor memory), 2 issuer
// of the state's MMAs, 4-7 WG A (scores and outputs), 8-15 WG V0 and V1 (decayed values, in turn),
// 16-19 WG M (the state). The state's chain and the outputs' meet only where MMA 2 reads M. Every
// mbarrier wait is bounded; when one runs out the status bit is set, all roles leave their loops, and
// copies and MMAs in flight are waited for.
#include <math.h>
#include <string.h>

#include <atomic>

#include "gr_internal.h"
#include "gr_mixer.h"
#include "gr_ptx.cuh"
#include "gr_tc.cuh"

namespace gr {
namespace {

constexpr int kChunk = 128;
constexpr int kBox = kChunk * 128;        // 128 rows of 64 bf16 channels
constexpr int kThreads = 640;
constexpr int kSub = 16;                  // tokens of one step of the state's MMA

// Tensor-memory columns: scores (then P in their place), Σ P c, Mᵀ a, the state's update.
constexpr uint32_t kColS = 0, kColO = 128, kColE = 256, kColU = 384;

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzled layout: 64 elements
// of M or N in each 128-byte row, a row for each k. Leading byte offset: between blocks of 64
// elements of M or N; stride byte offset: between groups of 8 k (1024, one swizzle atom).
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= uint64_t((saddr >> 4) & 0x3FFFu);
    d |= uint64_t((block_bytes >> 4) & 0x3FFFu) << 16;
    d |= uint64_t((1024u >> 4) & 0x3FFFu) << 32;
    d |= uint64_t(1u) << 46;
    d |= uint64_t(2u) << 61;
    return d;
}
constexpr uint32_t kMnA = 1u << 15, kMnB = 1u << 16;   // A, B given MN-major

template <int DA, int DC> struct Smem {
    static constexpr int kA = DA / 64 * kBox, kB = kA, kC = DC / 64 * kBox;
    static constexpr int kTerm = DC / 64 * kSub * 128;   // one bf16 term of a step's values
    static constexpr int kV = 3 * kTerm;
    static constexpr int kM = DC / 64 * DA * 128;
    static constexpr int b = kA, c = b + 2 * kB, v = c + 2 * kC, m = v + 2 * kV, aux = m + kM;
    static constexpr int kAux = 7168;
    // a head size of 64 still runs MMAs over 128 rows of b: the second 64-channel block it names
    // is the 16 KB behind the tile, whatever they hold, and its result rows are not used
    static constexpr int total = aux + kAux + 1024;
};

struct Aux {
    uint64_t a_full, a_empty, b_full[2], b_empty[2], c_full[2], c_empty[2];
    uint64_t s_full, p_ready, o_full, o_free, v_ready[2], v_free[2], u_full, u_free, m_ready, m_free,
        c_seen, c_clean[2], done;
    uint32_t tmem;
    int dead;
    int seq, seg, index;
    alignas(16) float pw[kChunk + 4];   // λ^0 .. λ^128
    alignas(16) float rev[32];          // λ^31 .. λ^0
    // a block of 32 rows and columns on the diagonal: outer weight λ^|i−j| (rows 16 bytes off a multiple of
    // 128, so that the lanes' 16-byte reads of one column group meet no bank twice)
    alignas(16) float diag[32][36];
    // By n & 3, which no other chunk writes before chunk n's outputs are out (WG V at chunk n + 3 has
    // seen PV of n + 1 done, and that waits for the outputs of n):
    int bad[4];                // n + 1 when chunk n's values are not all finite
    uint8_t first[4][128];     // by column: the first such row, in the order of time
};
static_assert(sizeof(Aux) <= 7168, "aux");

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* dead) {
    const uint32_t a = smem_u32(bar);
    long long t0 = 0;
    for (int k = 0;; ++k) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n"
            " mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(a), "r"(parity), "r"(kSuspendNs)
            : "memory");
        if (ok) return true;
        if (*dead) return false;
        if (k == 0) t0 = clock64();
        if (clock64() - t0 > kWaitLimit) {
            *dead = 1;
            atomicOr(&g_wait_status, 1u);
            return false;
        }
    }
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
// The same for a whole warp: the answer is the same in all lanes, which have come together again.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* dead) {
    return __all_sync(0xffffffffu, wait(bar, parity, dead));
}

// 32 bytes at once: a thread's own row is written in whole sectors.
__device__ __forceinline__ void st_row32(void* p, const uint32_t (&u)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]),
                 "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}
// One lane of the (whole) warp, the same every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
    return p != 0;
}
template <int N> __device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ uint32_t upper_halves(uint64_t v) {
    return __byte_perm(uint32_t(v), uint32_t(v >> 32), 0x7632);
}

// A bf16 pair times w as three (or two) bf16 pairs: 8 bits of the fp32 product's 24 each, cut off, so
// that three sum to the product exactly; of two the second is rounded. `seen` turns NaN where the pair
// is not finite.
template <int kTerms>
__device__ __forceinline__ void split_terms(uint32_t u, uint64_t w2, uint32_t& t0, uint32_t& t1, uint32_t& t2,
                                      uint64_t& seen) {
    const uint64_t keep = 0xffff0000ffff0000ull, minus = f2(-1.0f, -1.0f);
    uint64_t v = mul2(bf2_to_f2(u), w2);
    seen = fma2(v, 0ull, seen);
    t0 = upper_halves(v);
    v = fma2(v & keep, minus, v);
    if (kTerms == 2) {
        t1 = f2_to_bf2(v);
    } else {
        t1 = upper_halves(v);
        v = fma2(v & keep, minus, v);
        t2 = upper_halves(v);
    }
}

struct Launch {
    CUtensorMap rows[4];             // the distinct row arguments
    MixArgs pass[kMostPasses];
    int a[kMostPasses], b[kMostPasses], c[kMostPasses];   // the passes' maps
    Segments sg;
    float* slots;                    // [pass][segment][head] states
    float* firsts;                   // a copy of m_in, see mix_scan_kernel; else null
    int64_t units;                   // slots of a pass
};

// kSum: only the segment's own sum (no outputs), written to its slot; else the pass, which reads its first
// state from the slot of the segment before, or from m_in.
// kTerms: bf16 terms of the decayed values. Three where the state is a result; where only outputs read
// it, through a rounding to bf16, two (relative error 2^-17) leave that rounding as it is.
// kFine: P and the state's copy as two bf16 terms each, so that only the output's own rounding is left:
// 1.00 times its error. Rounded once, the norm of the error is 1.41 times that (± 0.04 over 160 rows of a
// head, ± 0.01 over 2048), a single row's up to 2.6 times, however many rows the call has. P's second
// term lies in the columns of its own scores, the state's in the second stage of b, which leaves b with one:
// launch_mix_tc says which calls can afford that.
template <int DA, int DC, bool kSum, int kTerms, int kPass, bool kFine>
__device__ __forceinline__ void mix_pass(const Launch& L) {
    const MixArgs& p = L.pass[kPass];
    const CUtensorMap &tmA = L.rows[L.a[kPass]], &tmB = L.rows[L.b[kPass]], &tmC = L.rows[L.c[kPass]];
    const Segments sg = L.sg;
    float* const slots = L.slots + int64_t(kPass) * L.units * (DA * DC);
    const float* const firsts = p.m_in && p.m_in == p.m_out ? L.firsts : nullptr;
    using S = Smem<DA, DC>;
    extern __shared__ __align__(1024) char raw[];
    char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);   // the swizzle's atoms
    Aux& x = *reinterpret_cast<Aux*>(sm + S::aux);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % p.n_heads;
    const float g = p.log_decay[h], intra = p.weight * p.outer;

    if (warp == 0) {
        int seq = 0, seg = 0, index = 0;
        const bool found = find_segment<kSum>(p, sg, blockIdx.x / p.n_heads, seq, seg, index);
        if (lane == 0) {
            x.seq = found ? seq : -1;
            x.seg = seg;
            x.index = index;
            x.dead = 0;
            x.bad[0] = x.bad[1] = x.bad[2] = x.bad[3] = 0;
            mbar_init(&x.a_full, 1), mbar_init(&x.a_empty, 1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mbar_init(&x.b_full[i], 1), mbar_init(&x.b_empty[i], kSum ? 1 : 2);
                mbar_init(&x.c_full[i], 1), mbar_init(&x.c_empty[i], 1);
                mbar_init(&x.v_ready[i], 4), mbar_init(&x.v_free[i], 1);
            }
            mbar_init(&x.s_full, 1), mbar_init(&x.p_ready, 4), mbar_init(&x.o_full, 2);
            mbar_init(&x.o_free, 4), mbar_init(&x.u_full, 1), mbar_init(&x.u_free, 4);
            mbar_init(&x.m_ready, 4), mbar_init(&x.m_free, 1), mbar_init(&x.c_seen, 8);
            mbar_init(&x.c_clean[0], 8), mbar_init(&x.c_clean[1], 8);
            mbar_init(&x.done, 2);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    __syncthreads();
    if (kSum) dep_launch_dependents();
    const int seq = x.seq, seg = x.seg;
    int64_t begin = 0, end = 0;
    if (seq >= 0) mix_span(p, seq, begin, end);
    const int64_t all = (end - begin + kChunk - 1) / kChunk;   // the sequence's chunks
    const int64_t n0 = int64_t(seg) * sg.per_seg;              // the segment's first, in time
    const bool last_seg = n0 + sg.per_seg >= all;
    if (seq < 0) return;   // the grid is an upper bound
    float* const slot = slots + (int64_t(x.index) * p.n_heads + h) * (DA * DC);   // of this segment
    const int chunks = int(min(int64_t(sg.per_seg), all - n0));
    const bool rev = p.reverse;
    // the chunk at step n of this segment: its first row, its rows, and whether the state enters
    // its last token undecayed
    auto row_of = [&](int n) { return begin + (rev ? all - 1 - (n0 + n) : n0 + n) * kChunk; };
    auto len_of = [&](int64_t row) { return int(min(int64_t(kChunk), end - row)); };
    auto load = [&](const CUtensorMap* map, int boxes, int at, uint64_t* bar, int n) {
        mbar_expect_tx(bar, boxes * kBox);
        for (int k = 0; k < boxes; ++k)
            tma_load_3d(sm + at + k * kBox, map, k * 64, h, int(row_of(n)), bar);
    };
    if (warp == 0 && lane == 0 && chunks > 0) {
        // the first chunk is on its way while the tables are made
        load(&tmB, DA / 64, S::b, &x.b_full[0], 0);
        load(&tmC, DC / 64, S::c, &x.c_full[0], 0);
        if (!kSum) load(&tmA, DA / 64, 0, &x.a_full, 0);
    }
    if (warp == 1) {
        tmem_alloc(&x.tmem, 512);
        tmem_relinquish();
    } else if (warp > 1) {
        for (int i = tid - 64; i <= kChunk; i += kThreads - 64) x.pw[i] = decay_pow(g, i);
        for (int i = tid - 64; i < 32; i += kThreads - 64) x.rev[i] = decay_pow(g, 31 - i);
        for (int i = tid - 64; i < 1024; i += kThreads - 64) {
            const int d = (i >> 5) - (i & 31);
            x.diag[i >> 5][i & 31] = intra * decay_pow(g, d < 0 ? -d : d);
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, x.tmem, 0);
    const bool from_slot = seg > 0;
    const bool has_in = !kSum && (from_slot || p.m_in != nullptr);
    // b's stage at step n and its parity: kFine's second stage holds the state's second term
    auto b_at = [](int n) { return kFine ? 0 : n & 1; };
    auto b_par = [](int n) { return uint32_t(kFine ? n : n >> 1) & 1u; };
    // whether the state after step n is still read (by the next chunk, or as a result)
    const bool wants_last = kSum || (last_seg && p.m_out != nullptr);

    if (warp < 4) {
        reg_dec<56>();
        if (warp == 0 && lane == 0) {
            // ---- producer -----------------------------------------------------------------------
            for (int n = 1; n < chunks; ++n) {
                const int st = n & 1;
                const uint32_t use2 = uint32_t(n >> 1) & 1u;
                if (n >= (kFine ? 1 : 2) && !wait(&x.b_empty[b_at(n)], b_par(n) ^ 1u, &x.dead)) break;
                load(&tmB, DA / 64, S::b + b_at(n) * S::kB, &x.b_full[b_at(n)], n);
                if (n >= 2 && !wait(&x.c_empty[st], use2 ^ 1u, &x.dead)) break;
                load(&tmC, DC / 64, S::c + st * S::kC, &x.c_full[st], n);
                if (kSum) continue;
                if (!wait(&x.a_empty, uint32_t(n - 1) & 1u, &x.dead)) break;
                load(&tmA, DA / 64, 0, &x.a_full, n);
            }
            if (x.dead) {
                // nobody consumes any more: let every copy land before the memory is given up
                const long long t0 = clock64();
                while (clock64() - t0 < kWaitLimit / 100) {
                }
            }
        } else if (warp == 1) {
            // ---- scores and outputs -------------------------------------------------------------
            // The whole warp runs the loop and one lane issues: descriptors and addresses stay in
            // uniform registers (issued from a branch of one lane, an MMA took about 120 cycles)
            const bool leader = elect_one();
            const uint32_t base = smem_u32(sm);
            const uint32_t a0 = base, m0 = base + S::m;
            constexpr uint32_t iS = idesc_bf16_f32(128, 128);
            constexpr uint32_t iE = idesc_bf16_f32(128, DC) | kMnB;
            uint32_t e_n = 0;
            for (int n = 0; !kSum && n < chunks; ++n) {
                const int st = n & 1;
                const uint32_t par2 = uint32_t(n >> 1) & 1u, par = uint32_t(n) & 1u;
                const uint32_t b0 = base + S::b + b_at(n) * S::kB, c0 = base + S::c + st * S::kC;
                if (!wait_warp(&x.b_full[b_at(n)], b_par(n), &x.dead)) break;
                if (!wait_warp(&x.a_full, par, &x.dead)) break;
                // the scores take the place of the last chunk's P
                if (n > 0 && !wait_warp(&x.o_full, par ^ 1u, &x.dead)) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int k = 0; k < DA / 16; ++k) {
                        const uint32_t off = (k >> 2) * kBox + (k & 3) * 32;
                        tc_mma(tm + kColS, sdesc_sw128(a0 + off), sdesc_sw128(b0 + off), iS, k > 0);
                    }
                    tc_commit(&x.s_full);
                    tc_commit(&x.b_empty[b_at(n)]);
                }
                if (n > 0 || has_in) {
                    if (!wait_warp(&x.m_ready, e_n & 1u, &x.dead)) break;
                    // the last chunk's outputs have been read
                    if (n > 0 && !wait_warp(&x.o_free, par ^ 1u, &x.dead)) break;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < DA / 16; ++k) {
                            const uint32_t off = (k >> 2) * kBox + (k & 3) * 32;
                            tc_mma(tm + kColE, sdesc_sw128(a0 + off), sdesc_mn(m0 + k * 2048, DA * 128),
                                   iE, k > 0);
                            if (kFine)
                                tc_mma(tm + kColE, sdesc_sw128(a0 + off),
                                       sdesc_mn(base + S::b + S::kB + k * 2048, DA * 128), iE, 1);
                        }
                        tc_commit(&x.m_free);
                    }
                    ++e_n;
                }
                if (leader) tc_commit(&x.a_empty);
                if (!wait_warp(&x.c_clean[st], par2, &x.dead)) break;
                // hands on what c_clean told (x.bad, x.first) with the outputs
                if (leader) mbar_arrive(&x.o_full);
                if (n > 0 && !wait_warp(&x.o_free, par ^ 1u, &x.dead)) break;
                if (!wait_warp(&x.p_ready, par, &x.dead)) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int k = 0; k < kChunk / 16; ++k)
                        if (kFine) {
                            const uint32_t at = tm + kColS + (k >> 1) * 32 + (k & 1) * 8;
                            tc_mma_ts(tm + kColO, at, sdesc_mn(c0 + k * 2048, kBox), iE, k > 0);
                            tc_mma_ts(tm + kColO, at + 16, sdesc_mn(c0 + k * 2048, kBox), iE, 1);
                        } else {
                            tc_mma_ts(tm + kColO, tm + kColS + k * 8, sdesc_mn(c0 + k * 2048, kBox), iE,
                                      k > 0);
                        }
                    tc_commit(&x.o_full);
                    tc_commit(&x.c_empty[st]);
                }
            }
            if (leader) tc_commit(&x.done);
            int never = 0;
            wait_warp(&x.done, 0, &never);
        } else if (warp == 2) {
            // ---- the state's update -------------------------------------------------------------
            const bool leader = elect_one();
            const uint32_t base = smem_u32(sm);
            constexpr uint32_t iU = idesc_bf16_f32(128, DC) | kMnA | kMnB;
            uint32_t v_use = 0;    // rounds of the two buffers so far
            for (int n = 0; n < chunks; ++n) {
                const int st = n & 1;
                const uint32_t b0 = base + S::b + b_at(n) * S::kB;
                if (!wait_warp(&x.b_full[b_at(n)], b_par(n), &x.dead)) break;
                if (n + 1 < chunks || wants_last) {
                    if (n > 0 && !wait_warp(&x.u_free, uint32_t(n - 1) & 1u, &x.dead)) break;
                    bool ok = true;
                    for (int s = 0; ok && s < kChunk / kSub; s += 2, ++v_use) {
#pragma unroll
                        for (int buf = 0; buf < 2; ++buf) {
                            if (!(ok = wait_warp(&x.v_ready[buf], v_use & 1u, &x.dead))) break;
                            tc_fence_after();
                            if (leader) {
                                const uint64_t ad = sdesc_mn(b0 + (s + buf) * 2048, kBox);
#pragma unroll
                                for (int t = 0; t < kTerms; ++t)
                                    tc_mma(tm + kColU, ad,
                                           sdesc_mn(base + S::v + buf * S::kV + t * S::kTerm, kSub * 128),
                                           iU, s > 0 || buf > 0 || t > 0);
                                tc_commit(&x.v_free[buf]);
                            }
                        }
                    }
                    if (!ok) break;
                    if (leader) tc_commit(&x.u_full);
                }
                if (leader) {
                    tc_commit(&x.b_empty[b_at(n)]);
                    if (kSum) tc_commit(&x.c_empty[st]);
                }
            }
            if (leader) tc_commit(&x.done);
            int never = 0;
            wait_warp(&x.done, 0, &never);
        }
        __syncwarp();
    } else if (warp < 8) {
        // 56 + 120 + 2 · 56 + 192 registers a thread: the launch's 5 · 96
        reg_inc<120>();
        if (!kSum) {
            // ---- WG A: scores to P, outputs ---------------------------------------------------------
            const int wq = warp - 4, i = wq * 32 + lane;
            const uint32_t tl = tm + (uint32_t(wq * 32) << 16);
            char* out0 = static_cast<char*>(p.out.p) + int64_t(h) * p.out.hs * 2;
            const bool wide = ((reinterpret_cast<uintptr_t>(out0) | uintptr_t(p.out.ts * 2)) & 31u) == 0;
            for (int n = 0; n < chunks; ++n) {
                const uint32_t par = uint32_t(n) & 1u;
                const int64_t row = row_of(n);
                const int len = len_of(row);
                const int late = rev && seg == 0 && n == 0 ? 1 : 0;
                const bool read_m = n > 0 || has_in;
                if (!wait_warp(&x.s_full, par, &x.dead)) break;
                tc_fence_after();
#pragma unroll 1
                for (int jb = 0; jb < 4; ++jb) {
                    uint32_t q[16], q2[16];
                    const bool off = rev ? jb > wq : jb < wq;
                    if (off || jb == wq) {
                        uint32_t r[32];
                        tmem_ld32(tl + kColS + jb * 32, r);
                        // λ^|i−j|: off the diagonal the row's distance to the block times the column's
                        // within it
                        const float rw =
                            !off ? 1.0f : intra * (rev ? x.pw[jb * 32 - i] : x.pw[i - jb * 32 - 31]);
                        const float4* cw =
                            reinterpret_cast<const float4*>(!off ? x.diag[lane] : rev ? x.pw : x.rev);
                        const uint64_t rw2 = f2(rw, rw);
                        tmem_wait32(r);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 c = cw[j];
                            const uint64_t u = mul2(f2(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1])),
                                                    mul2(f2(c.x, c.y), rw2));
                            const uint64_t v =
                                mul2(f2(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])),
                                     mul2(f2(c.z, c.w), rw2));
                            q[2 * j] = f2_to_bf2(u), q[2 * j + 1] = f2_to_bf2(v);
                            if (kFine) {
                                const uint64_t minus = f2(-1.0f, -1.0f);
                                q2[2 * j] = f2_to_bf2(fma2(bf2_to_f2(q[2 * j]), minus, u));
                                q2[2 * j + 1] = f2_to_bf2(fma2(bf2_to_f2(q[2 * j + 1]), minus, v));
                            }
                        }
                        // the columns of later (backwards: earlier) rows are cut off, whatever they hold, and,
                        // backwards, those past the sequence's end (forwards no valid row reaches them)
                        const int live = rev ? len - jb * 32 : 32;
                        if (!off || live < 32) {
                            const int from = rev && !off ? lane : 0, to = rev || off ? live : lane + 1;
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const uint32_t keep = (2 * j >= from && 2 * j < to ? 0xffffu : 0u) |
                                                      (2 * j + 1 >= from && 2 * j + 1 < to ? 0xffff0000u : 0u);
                                q[j] &= keep;
                                if (kFine) q2[j] &= keep;
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) q[j] = q2[j] = 0;
                    }
                    if (kFine) {
                        tmem_st16(tl + kColS + jb * 32, q);
                        tmem_st16(tl + kColS + jb * 32 + 16, q2);
                    } else {
                        // P's columns lie below the scores that are still to be read
                        tmem_st16(tl + kColS + jb * 16, q);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&x.p_ready);
                if (!wait_warp(&x.o_full, par, &x.dead)) break;
                tc_fence_after();
                const bool bad = x.bad[n & 3] == n + 1;
                const bool live = i < len;
                const float ew = live ? p.outer * x.pw[rev ? len - i - late : i + 1] : 0.0f;
                const uint64_t ew2 = f2(ew, ew);
                char* dst = out0 + (row + i) * p.out.ts * 2;
                const int ti = rev ? kChunk - 1 - i : i;
                // 16 columns at a time, the next ones on their way
                uint32_t o[2][16], m[2][16];
#pragma unroll
                for (int k = 0; k < 16; ++k) m[0][k] = m[1][k] = 0;
                auto fetch = [&](int e, int k2) {
                    tmem_ld16_nowait(tl + kColO + e, o[k2]);
                    if (read_m) tmem_ld16_nowait(tl + kColE + e, m[k2]);
                };
                fetch(0, 0);
#pragma unroll 1
                for (int e0 = 0; e0 < DC; e0 += 32) {
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        const int e = e0 + 16 * k2;
                        tmem_wait_ld(o[k2]);
                        if (read_m) tmem_wait_ld(m[k2]);
                        if (e + 16 < DC) fetch(e + 16, k2 ^ 1);
                        if (bad) {
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                if (ti >= int(x.first[n & 3][e + k])) o[k2][k] = 0x7fffffffu;
                        }
                        if (k2 == 1 && e + 16 == DC) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&x.o_free);
                        }
                        if (live) {
                            uint32_t u[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                u[k] = f2_to_bf2(fma2(
                                    ew2,
                                    f2(__uint_as_float(m[k2][2 * k]), __uint_as_float(m[k2][2 * k + 1])),
                                    f2(__uint_as_float(o[k2][2 * k]), __uint_as_float(o[k2][2 * k + 1]))));
                            if (wide) {
                                st_row32(dst + e * 2, u);
                            } else {
                                reinterpret_cast<uint4*>(dst + e * 2)[0] =
                                    make_uint4(u[0], u[1], u[2], u[3]);
                                reinterpret_cast<uint4*>(dst + e * 2)[1] =
                                    make_uint4(u[4], u[5], u[6], u[7]);
                            }
                        }
                    }
                }
            }
        }
    } else if (warp < 16) {
        reg_dec<56>();
        // ---- WG V0, V1: decayed values; V0 takes the even steps, V1 the odd ones, each with a buffer ----
        const int buf = warp >= 12, t = (tid - 256) & 127;
        const int vr = t >> 3, vc = t & 7;   // its row of a step and 16-byte column
        char* vt = sm + S::v + buf * S::kV + swz(vr, vc);
        uint32_t v_use = 0;
        for (int n = 0; n < chunks; ++n) {
            const int st = n & 1;
            const uint32_t par2 = uint32_t(n >> 1) & 1u, par = uint32_t(n) & 1u;
            const int len = len_of(row_of(n));
            const bool need_u = n + 1 < chunks || wants_last;
            char* ct = sm + S::c + st * S::kC;
            char* bt = sm + S::b + b_at(n) * S::kB;
            if (!wait_warp(&x.c_full[st], par2, &x.dead)) break;
            if (len < kChunk && !wait_warp(&x.b_full[b_at(n)], b_par(n), &x.dead)) break;
            bool ok = true;
            uint64_t seen = 0;
#pragma unroll 1
            for (int s = buf; s < kChunk / kSub; s += 2) {
                const int r = s * kSub + vr;
                if (r >= len) {
                    // rows past the sequence's end may hold anything: they become zero
#pragma unroll
                    for (int k = 0; k < DC / 64; ++k)
                        *reinterpret_cast<uint4*>(ct + k * kBox + swz(r, vc)) = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int k = 0; k < DA / 64; ++k)
                        *reinterpret_cast<uint4*>(bt + k * kBox + swz(r, vc)) = make_uint4(0, 0, 0, 0);
                }
                // split before the wait for the buffer, so that only stores lie between the MMAs
                const float w = p.weight * (r < len ? x.pw[rev ? r : len - 1 - r] : 0.0f);
                const uint64_t w2 = f2(w, w);
                uint4 a[DC / 64], b[DC / 64], c[DC / 64];
#pragma unroll
                for (int k = 0; k < DC / 64; ++k) {
                    const uint4 u = *reinterpret_cast<const uint4*>(ct + k * kBox + swz(r, vc));
                    split_terms<kTerms>(u.x, w2, a[k].x, b[k].x, c[k].x, seen);
                    split_terms<kTerms>(u.y, w2, a[k].y, b[k].y, c[k].y, seen);
                    split_terms<kTerms>(u.z, w2, a[k].z, b[k].z, c[k].z, seen);
                    split_terms<kTerms>(u.w, w2, a[k].w, b[k].w, c[k].w, seen);
                }
                if (need_u) {
                    if (v_use >= 1 && !(ok = wait_warp(&x.v_free[buf], (v_use - 1) & 1u, &x.dead))) break;
#pragma unroll
                    for (int k = 0; k < DC / 64; ++k) {
                        char* q = vt + k * (kSub * 128);
                        *reinterpret_cast<uint4*>(q) = a[k];
                        *reinterpret_cast<uint4*>(q + S::kTerm) = b[k];
                        if (kTerms > 2) *reinterpret_cast<uint4*>(q + 2 * S::kTerm) = c[k];
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x.v_ready[buf]);
                    ++v_use;
                }
            }
            if (!ok) break;
            if (!kSum) {
                // all values seen: a chunk with one that is not finite takes the slow way before its
                // product is formed (0 times such a value would reach earlier rows)
                float s0, s1;
                unf2(seen, s0, s1);
                const bool odd = __any_sync(0xffffffffu, !(s0 == 0.0f && s1 == 0.0f));
                if (lane == 0) {
                    if (odd) x.bad[n & 3] = n + 1;
                    mbar_arrive(&x.c_seen);
                }
                if (!wait_warp(&x.c_seen, par, &x.dead)) break;
                if (buf == 0 && x.bad[n & 3] == n + 1) {
                    for (int e = t; e < DC; e += 128) {
                        int f = kChunk;
                        for (int j = 0; j < len; ++j) {
                            unsigned short* q = reinterpret_cast<unsigned short*>(
                                                    ct + (e >> 6) * kBox + swz(j, (e >> 3) & 7)) +
                                                (e & 7);
                            if ((*q & 0x7f80u) != 0x7f80u) continue;
                            f = min(f, rev ? kChunk - 1 - j : j);
                            *q = 0;   // the product is formed without it
                        }
                        x.first[n & 3][e] = uint8_t(f);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&x.c_clean[st]);
            }
        }
    } else {
        reg_inc<192>();
        // ---- WG M: the state ------------------------------------------------------------------------
        const int wq = warp - 16, d = tid - 512;
        const uint32_t tl = tm + (uint32_t(wq * 32) << 16);
        const bool owns = d < DA;            // thread d holds the state's row d
        float M[DC];
#pragma unroll
        for (int e = 0; e < DC; ++e) M[e] = 0.0f;
        const int64_t one = int64_t(DA) * DC;
        if (has_in && owns) {
            const bool copied = firsts && !last_seg;
            if (from_slot || copied) {
                const float* from = from_slot ? slot - p.n_heads * one
                                              : firsts + (int64_t(seq) * p.n_heads + h) * one;
                const float4* s = reinterpret_cast<const float4*>(from + int64_t(d) * DC);
#pragma unroll
                for (int e = 0; e < DC / 4; ++e) {
                    const float4 v = __ldcg(s + e);
                    M[4 * e] = v.x, M[4 * e + 1] = v.y, M[4 * e + 2] = v.z, M[4 * e + 3] = v.w;
                }
            } else {
                const float* s = p.m_in + (int64_t(seq) * p.n_heads + h) * one + int64_t(d) * p.mr;
#pragma unroll
                for (int e = 0; e < DC; ++e) M[e] = s[int64_t(e) * p.mc];
            }
        }
        // the state as the MMA reads it: row d of 64-column boxes, bf16
        auto publish = [&]() {
            if (owns) {
#pragma unroll
                for (int k = 0; k < DC / 8; ++k) {
                    const uint4 u = make_uint4(pack_bf2(M[8 * k], M[8 * k + 1]),
                                               pack_bf2(M[8 * k + 2], M[8 * k + 3]),
                                               pack_bf2(M[8 * k + 4], M[8 * k + 5]),
                                               pack_bf2(M[8 * k + 6], M[8 * k + 7]));
                    const int at = (k >> 3) * (DA * 128) + swz(d, k & 7);
                    *reinterpret_cast<uint4*>(sm + S::m + at) = u;
                    if (kFine) {
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                        uint32_t v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            v[j] = f2_to_bf2(fma2(bf2_to_f2(w[j]), f2(-1.0f, -1.0f),
                                                  f2(M[8 * k + 2 * j], M[8 * k + 2 * j + 1])));
                        *reinterpret_cast<uint4*>(sm + S::b + S::kB + at) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.m_ready);
        };
        if (has_in && chunks > 0) publish();
        uint32_t published = has_in ? 1u : 0u;
        int n = 0;
        for (; n < chunks && (n + 1 < chunks || wants_last); ++n) {
            const int len = len_of(row_of(n));
            const int late = rev && seg == 0 && n == 0 ? 1 : 0;
            const float keep = x.pw[len - late];
            if (!wait_warp(&x.u_full, uint32_t(n) & 1u, &x.dead)) break;
            tc_fence_after();
            const uint64_t keep2 = f2(keep, keep);
#pragma unroll
            for (int e = 0; e < DC; e += 16) {
                uint32_t u[16];
                tmem_ld16_nowait(tl + kColU + e, u);
                tmem_wait_ld(u);
#pragma unroll
                for (int k = 0; k < 16; k += 2)
                    unf2(fma2(keep2, f2(M[e + k], M[e + k + 1]),
                              f2(__uint_as_float(u[k]), __uint_as_float(u[k + 1]))),
                         M[e + k], M[e + k + 1]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.u_free);
            if (!kSum && n + 1 < chunks) {
                if (published > 0 && !wait_warp(&x.m_free, (published - 1) & 1u, &x.dead)) break;
                publish();
                ++published;
            }
        }
        if (n == chunks && owns) {
            if (kSum) {
                float* s = slot + int64_t(d) * DC;
#pragma unroll
                for (int e = 0; e < DC; e += 8) {
                    uint32_t u[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(M[e + k]);
                    st_row32(s + e, u);
                }
            } else if (last_seg && p.m_out) {
                // backwards, λ once more takes the gradient to the state before the first token
                const float w = rev && end > begin ? x.pw[1] : 1.0f;
                float* s = p.m_out + (int64_t(seq) * p.n_heads + h) * one + int64_t(d) * p.mr;
                if (p.mc == 1) {
#pragma unroll
                    for (int e = 0; e < DC; e += 4)
                        *reinterpret_cast<float4*>(s + e) =
                            make_float4(w * M[e], w * M[e + 1], w * M[e + 2], w * M[e + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < DC; ++e) s[int64_t(e) * p.mc] = w * M[e];
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// blockIdx.y is the pass. Each has its code by itself, so that its arguments stay constants of the launch
// and branches on them uniform ones (read through an index, a chunk took a quarter longer).
template <int DA, int DC, bool kSum, int kTerms, int kPasses, bool kFine>
__global__ void __launch_bounds__(kThreads, 1) mix_tc_kernel(const __grid_constant__ Launch L) {
    if (kPasses == 1 || blockIdx.y == 0) mix_pass<DA, DC, kSum, kTerms, 0, kFine>(L);
    else if (blockIdx.y == 1) mix_pass<DA, DC, kSum, kTerms, 1, kFine>(L);
    else mix_pass<DA, DC, kSum, kTerms, 2, kFine>(L);
}

bool map_rows(CUtensorMap* m, const MixRows& r, int64_t N, int H, int d) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(H), cuuint64_t(N)};
    const cuuint64_t strides[2] = {cuuint64_t(r.hs) * 2, cuuint64_t(r.ts) * 2};
    const cuuint32_t box[3] = {64, 1, kChunk};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, r.p, dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                   Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

template <int DA, int DC, int kTerms, int kPasses, bool kFine>
cudaError_t run(const MixArgs* pass, float* slots, cudaStream_t st) {
    constexpr int passes = kPasses;
    const MixArgs& p = pass[0];
    Launch L;
    memset(&L, 0, sizeof(L));
    int maps = 0;
    MixRows seen[4];
    int width[4];
    auto map_of = [&](const MixRows& r, int d) {
        for (int i = 0; i < maps; ++i)
            if (seen[i].p == r.p && seen[i].ts == r.ts && seen[i].hs == r.hs && width[i] == d) return i;
        if (maps == 4 || !map_rows(&L.rows[maps], r, p.n_tokens, p.n_heads, d)) return -1;
        seen[maps] = r;
        width[maps] = d;
        return maps++;
    };
    for (int i = 0; i < passes; ++i) {
        L.pass[i] = pass[i];
        L.a[i] = map_of(pass[i].a, DA);
        L.b[i] = map_of(pass[i].b, DA);
        L.c[i] = map_of(pass[i].c, DC);
        if (L.a[i] < 0 || L.b[i] < 0 || L.c[i] < 0) return cudaErrorInvalidValue;
    }
    L.sg = mix_plan(p.n_tokens, p.n_seqs, int64_t(p.n_heads) * passes, kChunk);
    L.units = mix_units(p.n_tokens, p.n_seqs, p.n_heads, L.sg);
    const bool split = mix_cuts(p.n_tokens, L.sg);
    L.slots = slots;
    L.firsts = split ? slots + passes * L.units * int64_t(DA * DC) : nullptr;
    const dim3 grid(unsigned(L.units), passes);
    constexpr int smem = Smem<DA, DC>::total;
    static_assert(smem <= 232448, "shared memory");
    static_assert(Smem<DA, DC>::kM <= Smem<DA, DC>::kB, "the state's second term");
    static std::atomic<uint64_t> ready;   // a bit for each device whose kernels have their shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev > 63 || !(ready.load(std::memory_order_relaxed) >> dev & 1))) {
        e = cudaFuncSetAttribute(mix_tc_kernel<DA, DC, false, kTerms, kPasses, kFine>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(mix_tc_kernel<DA, DC, true, kTerms, kPasses, false>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && dev <= 63) ready.fetch_or(uint64_t(1) << dev);
    }
    if (e == cudaSuccess && split) {
        const dim3 sums(mix_sums(p.n_tokens, p.n_heads, L.sg), passes);
        e = launch(mix_tc_kernel<DA, DC, true, kTerms, kPasses, false>, sums, kThreads, smem, st, L);
        if (e == cudaSuccess)
            e = launch_mix_scan(L.pass, passes, L.sg, slots, L.firsts, L.units, st);
    }
    // (launched after the scan in the plain order: as its programmatic dependent a gradient of 96 uncut
    // rows took 176 us against 142)
    if (e == cudaSuccess)
        e = launch(mix_tc_kernel<DA, DC, false, kTerms, kPasses, kFine>, grid, kThreads, smem, st, L);
    return e;
}

template <int DA, int DC, int kPasses>
cudaError_t choose(int how, const MixArgs* p, float* slots, cudaStream_t st) {
    return how == 0   ? run<DA, DC, 3, kPasses, true>(p, slots, st)
           : how == 1 ? run<DA, DC, 2, kPasses, false>(p, slots, st)
                      : run<DA, DC, 3, kPasses, false>(p, slots, st);
}

}  // namespace

bool mix_tc_supported(const MixArgs& p) {
    const int64_t most = int64_t(1) << 38;   // a tensor map's strides are below 2^40 bytes
    for (const MixRows* r : {&p.a, &p.b, &p.c})
        if (r->ts > most || r->hs > most) return false;
    return p.dtype == GR_BF16 && (p.da == 64 || p.da == 128) && (p.dc == 64 || p.dc == 128) &&
           p.n_tokens > 0 && p.n_seqs > 0 &&
           mix_units(p.n_tokens, p.n_seqs, p.n_heads, {1, kChunk}) <= 0x7fffffff;
}

// The slots of all passes and, for one of them, a copy of its first states.
size_t mix_tc_workspace(int64_t N, int n_seqs, int H, int da, int dc, int passes) {
    if (N == 0 || n_seqs == 0) return 0;
    const Segments sg = mix_plan(N, n_seqs, int64_t(H) * passes, kChunk);
    if (!mix_cuts(N, sg)) return 0;
    return align256(size_t(passes * mix_units(N, n_seqs, H, sg) + int64_t(n_seqs) * H) * da * dc * 4);
}

cudaError_t launch_mix_tc(const MixArgs* p, int passes, void* workspace, cudaStream_t st) {
    float* slots = static_cast<float*>(workspace);
    bool state = false;
    for (int i = 0; i < passes; ++i) state = state || p[i].m_out;
    // Fine where it costs little, up to a chunk of tokens or the rows of 16 chunks: such calls wait more
    // than they compute (the gradient of 512 tokens of 4 heads of 128 takes 23 us instead of 21, the prompt
    // 25 instead of 24). Larger ones do not (8192 tokens of 152 heads: 315 us instead of 248). The rule
    // looks at the call, so the same sequence may be fine alone and not among others.
    const bool fine = p->n_tokens <= kChunk || p->n_tokens * p->n_heads <= 16 * kChunk;
    // 0: fine (whatever its terms: three), 1: two terms, 2: three
    const int how = fine ? 0 : state ? 2 : 1;
    if (passes == 3 && p->da == p->dc)
        return p->da == 128 ? choose<128, 128, 3>(how, p, slots, st) : choose<64, 64, 3>(how, p, slots, st);
    if (passes != 1) return cudaErrorInvalidValue;
    if (p->da == 128)
        return p->dc == 128 ? choose<128, 128, 1>(how, p, slots, st) : choose<128, 64, 1>(how, p, slots, st);
    return p->dc == 128 ? choose<64, 128, 1>(how, p, slots, st) : choose<64, 64, 1>(how, p, slots, st);
}

int mixer_status(bool clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_status, sizeof(v)) != cudaSuccess) return -1;
    if (clear && v) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_wait_status, &z, sizeof(z)) != cudaSuccess) return -1;
    }
    return int(v);
}

}  // namespace gr
