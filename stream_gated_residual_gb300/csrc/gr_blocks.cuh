// The rule of FP8 blocks, for the units that write them (after gr_ptx.cuh).
#pragma once

namespace gr {
namespace {

// Magnitudes compare as their bits do; infinity and NaN lie above every finite one.
__device__ __forceinline__ uint32_t block_mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The biased exponent of a block from its largest magnitude's bits, and the factor 2^-e (0: not finite).
__device__ __forceinline__ uint8_t block_scale(uint32_t top, float& inv) {
    if (top >= 0x7f800000u) {
        inv = 0.0f;
        return 255;
    }
    const int e = fp8_block_exp(__uint_as_float(top));
    inv = pow2f(-e);
    return uint8_t(e + 127);
}
__device__ __forceinline__ uint32_t block_codes4(const float* v, float inv) {
    if (inv == 0.0f) return 0x7f7f7f7fu;
    return uint32_t(f2_to_e4m3x2(v[0] * inv, v[1] * inv)) |
           (uint32_t(f2_to_e4m3x2(v[2] * inv, v[3] * inv)) << 16);
}

}  // namespace
}  // namespace gr
