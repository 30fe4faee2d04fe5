// Host-side checks that the decoder parts' C entries share.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "gr_internal.h"

namespace gr {
namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t width(int dtype) { return dtype == GR_BF16 ? 2 : 4; }
inline bool real_dtype(int dtype) { return dtype == GR_F32 || dtype == GR_BF16; }
inline int as_status(cudaError_t e) { return e == cudaSuccess ? GR_OK : GR_E_CUDA; }

// A buffer of a call: where it starts and how many bytes the call may touch.
struct Span {
    const void* p;
    size_t n;
};
inline bool meet(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}

}  // namespace
}  // namespace gr
