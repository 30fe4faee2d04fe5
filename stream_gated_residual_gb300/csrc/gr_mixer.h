// The linear-attention mixer's internal interface: one masked, decayed product over a packed batch
// of sequences, which the forward pass and all three gradients are instances of.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gr {

// Rows [n_tokens][n_heads][d] at any 16-byte aligned token and head strides (in elements).
struct MixRows {
    void* p;
    int64_t ts, hs;
};

// For every sequence (rows starts[b] .. starts[b+1]) and head, with λ = exp(log_decay[h]):
//   forwards   M_t = λ M_{t−1} + weight b_t c_tᵀ,   out_t = outer M_tᵀ a_t
//              = outer [ weight Σ_{s<=t} λ^{t−s} (a_t·b_s) c_s + λ^{t+1} M_inᵀ a_t ]
//   backwards  the same with the order of the tokens reversed (s >= t), except that M_in enters the
//              last token undecayed (it is the gradient of the state after that token):
//              the exponent of its decay is T − 1 − t
// a, b have da channels, c and out dc; M is [da][dc]. M_in and M_out are fp32 [B][H][da·dc] with the
// element (i, j) at i·mr + j·mc; either may be null. Forwards M_out = M after the last token;
// backwards it is λ·M after the first one (the gradient of the state before it).
struct MixArgs {
    int64_t n_tokens;
    int n_seqs, n_heads, da, dc, dtype;
    MixRows a, b, c, out;
    const float* log_decay;
    const int32_t* starts;   // null: one sequence of all tokens
    const float* m_in;
    float* m_out;
    int mr, mc;
    float weight, outer;
    bool reverse;
};

// Sequence b's rows [begin, end), clamped to the packed rows so that no entry of `starts` can lead
// outside them.
__device__ __forceinline__ void mix_span(const MixArgs& p, int b, int64_t& begin, int64_t& end) {
    begin = 0;
    end = p.n_tokens;
    if (p.starts) {
        begin = max(int64_t(0), min(int64_t(p.starts[b]), p.n_tokens));
        end = max(begin, min(int64_t(p.starts[b + 1]), p.n_tokens));
    }
}
// λ^n as exp(n·log λ), λ^0 = 1 also for λ = 0.
__device__ __forceinline__ float decay_pow(float log_decay, int64_t n) {
    return n == 0 ? 1.0f : expf(float(n) * log_decay);
}

// Where a CTA works: segment `seg` (in the order of time it is processed) of sequence `seq`. Every
// sequence has at least one segment, so that an empty one passes its state on.
struct Segments {
    int per_seg;   // chunks of a segment
    int chunk;     // tokens of a chunk
    __device__ __forceinline__ int count(int64_t begin, int64_t end) const {
        const int64_t chunks = (end - begin + chunk - 1) / chunk;
        const int64_t n = (chunks + per_seg - 1) / per_seg;
        return n > 0 ? int(n) : 1;
    }
};

// The whole warp finds the sequence that holds segment `want`, 32 sequences at a time; `index` is the
// segment's place among all. kSum counts only the segments that have a successor: those whose sum is
// needed.
template <bool kSum>
__device__ __forceinline__ bool find_segment(const MixArgs& p, const Segments& sg, int want, int& seq,
                                             int& seg, int& index) {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int b0 = 0; b0 < p.n_seqs; b0 += 32) {
        const int b = b0 + lane;
        int n = 0;
        if (b < p.n_seqs) {
            int64_t x, y;
            mix_span(p, b, x, y);
            n = sg.count(x, y) - (kSum ? 1 : 0);
        }
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        const bool mine = n > 0 && want >= before + inc - n && want < before + inc;
        const unsigned hit = __ballot_sync(0xffffffffu, mine);
        if (hit) {
            const int l = __ffs(hit) - 1;
            seq = b0 + l;
            seg = want - before - (__shfl_sync(0xffffffffu, inc, l) - __shfl_sync(0xffffffffu, n, l));
            index = want + (kSum ? seq : 0);
            return true;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
}

// Chunks a segment. A unit (a segment of a head) takes its chunks one after another, one unit an SM at a
// time; cutting a sequence costs a second pass over b and c of all but its last segment, and two
// launches. The host knows the sequences' number and sum, not their lengths:
//   - too few of them to fill the SMs (rows < 152): taken as equally long, cut so that the estimated time
//     is least (32768 tokens, 32 heads of 128: 256 chunks uncut 945 us, in 4 segments 403, in 9 388);
//   - enough of them: only a sequence longer than twice an SM's even share of all chunks is cut, which
//     bounds what a single long one can cost (equal ones are never cut).
inline int64_t mix_plan_evenly(int64_t N, int n_seqs, int64_t heads, int chunk) {
    constexpr int kSms = 152;   // blocks the segments are planned for
    const int64_t rows = n_seqs * heads;
    const int64_t mean = (N + n_seqs - 1) / n_seqs;
    const int64_t chunks = (mean + chunk - 1) / chunk;
    if (rows >= kSms) {
        const int64_t total = (N / chunk + n_seqs) * heads;
        return 2 * ((total + kSms - 1) / kSms);
    }
    if (chunks <= 1) return 1;
    int64_t most = (6 * kSms + rows - 1) / rows;
    most = most < chunks ? most : chunks;
    int64_t best = chunks;
    double least = 1e300;
    for (int64_t n = 1; n <= most; ++n) {
        const int64_t per = (chunks + n - 1) / n, segs = (chunks + per - 1) / per;
        const int64_t waves = (rows * segs + kSms - 1) / kSms;
        const int64_t waves1 = (rows * (segs - 1) + kSms - 1) / kSms;
        // in units of a chunk's time (about 4 us): 2 a unit to start and drain; sums 0.6 of a chunk
        double t = waves * (per + 2.0);
        if (segs > 1) t += waves1 * (0.6 * per + 1.5) + 2.0;
        if (t < least) least = t, best = per;
    }
    return best;
}

inline Segments mix_plan(int64_t N, int n_seqs, int64_t heads, int chunk) {
    int64_t per = mix_plan_evenly(N, n_seqs, heads, chunk);
    // several sequences, but none can be twice as long: not cut, which saves the two launches that
    // would look for one that is (13 us of 140 for the gradient of 2 · 4096 tokens, 16 heads of 128)
    if (n_seqs > 1 && N <= 2 * per * chunk) per = N / chunk + 1;
    return {int(per < 1 << 26 ? per : 1 << 26), chunk};
}

// An upper bound of the segments of all sequences, times the heads (the slots of a pass).
inline int64_t mix_units(int64_t N, int n_seqs, int H, const Segments& sg) {
    return (N / (int64_t(sg.per_seg) * sg.chunk) + n_seqs) * H;
}
// Whether any sequence can have a second segment: none is longer than all tokens.
inline bool mix_cuts(int64_t N, const Segments& sg) { return N > int64_t(sg.per_seg) * sg.chunk; }
// The blocks of the segments with a successor: each is a whole one.
inline unsigned mix_sums(int64_t N, int H, const Segments& sg) {
    return unsigned(N / (int64_t(sg.per_seg) * sg.chunk)) * H;
}

// The segments' sums to the states after them, in place (gr_mixer.cu): slot s of a sequence and head
// becomes λ^len_s (state before s) + slot s; the last segment's slot is not used. slots
// [pass][units][da·dc], segments of all sequences in order, each with n_heads slots. `firsts`, for the pass
// whose m_out is m_in itself, takes a copy of m_in [B][H][da·dc] for the first segments: their sequence's last
// segment may be done before they start. Launched as the programmatic dependent of the sums.
constexpr int kMostPasses = 3;
cudaError_t launch_mix_scan(const MixArgs* pass, int passes, const Segments& sg, float* slots,
                            float* firsts, int64_t units, cudaStream_t st);

// CUDA-core form: every type, head size and length (gr_mixer.cu); workspace as below.
size_t mix_simt_workspace(int64_t n_tokens, int n_seqs, int n_heads, int da, int dc);
cudaError_t launch_mix_simt(const MixArgs& p, void* workspace, cudaStream_t st);

// Tensor-core form (gr_mixer_tc.cu): bf16, da and dc 64 or 128. One pass, or three over the same packed
// sequences in one launch (the gradient's dq, dk and dv where da == dc): same da, dc, heads and starts;
// no pass's m_out may be another one's m_in. The workspace holds the segments' states where prompts
// are cut.
bool mix_tc_supported(const MixArgs& p);
size_t mix_tc_workspace(int64_t n_tokens, int n_seqs, int n_heads, int da, int dc, int passes);
cudaError_t launch_mix_tc(const MixArgs* p, int passes, void* workspace, cudaStream_t st);
int mixer_status(bool clear);

// One token a request, the fp32 states read and written in place (gr_mixer.cu).
cudaError_t launch_mix_step(int64_t n, int n_heads, int dk, int dv, int dtype, float scale,
                            MixRows q, MixRows k, MixRows v, const float* log_decay, float* state,
                            int64_t n_slots, const int32_t* slots, MixRows o, cudaStream_t st);

}  // namespace gr
