// Internal interface of the window kernel (sq_window.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sq_internal.h"

namespace sqk {

constexpr int kWindowMax = SQ_WINDOW_MAX;

struct WindowArgs {
    const uint8_t *base;   // the pool: packed (strides in bytes) or fp32 (in floats)
    int64_t slot_stride;
    const int32_t *slot, *lens;
    int32_t n, length, n_heads, n_key_heads;
    const void *q, *k, *v, *beta, *g;
    void *y;               // or null
    float *S_out;          // or null
};

// tab: the packed pool's heads; null for an fp32 pool.
hipError_t launch_window(const WindowArgs &a, const HeadTable *tab, int d, bool kda, bool f32, bool y_f32, hipStream_t stream);

} // namespace sqk
