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

// CUDA-core form: every type, head size and length (gr_mixer.cu).
cudaError_t launch_mix_simt(const MixArgs& p, cudaStream_t st);

// Tensor-core form (gr_mixer_tc.cu): bf16, da and dc 64 or 128. One pass, or three over the same packed
// sequences in one launch (the gradient's dq, dk and dv where da == dc): same da, dc, heads and starts;
// no pass's m_out may be another one's m_in. The workspace holds the segments' states where prompts
// are cut.
constexpr int kMostPasses = 3;
bool mix_tc_supported(const MixArgs& p);
size_t mix_tc_workspace(int64_t n_tokens, int n_seqs, int n_heads, int da, int dc, int passes);
cudaError_t launch_mix_tc(const MixArgs* p, int passes, void* workspace, cudaStream_t st);
int mixer_status(bool clear);

// One token a request, the fp32 states read and written in place (gr_mixer.cu).
cudaError_t launch_mix_step(int64_t n, int n_heads, int dk, int dv, int dtype, float scale,
                            MixRows q, MixRows k, MixRows v, const float* log_decay, float* state,
                            int64_t n_slots, const int32_t* slots, MixRows o, cudaStream_t st);

}  // namespace gr
