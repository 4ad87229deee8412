// Internal interface of the draft check (sq_verify.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sq_internal.h"

namespace sqk {

constexpr float kLog2e = 1.44269504088896340736f;

struct VerifyArgs {
    const void *target, *draft;              // logits; draft or null
    int64_t target_stride, draft_stride;     // elements from row to row
    const int32_t *tokens, *lens;            // lens or null
    const float *accept_u, *sample_e;        // null where greedy
    int32_t n, m, vocab;
    float inv_temperature;
    int32_t *accepted, *next;
    // workspace: per (row, split) a maximum and a sum (greedy: its index); per
    // (request, split) the best score and its token
    float2 *stats;
    uint64_t *best;
    int32_t splits, sample_splits;           // workgroups per row, per request
};

constexpr int kVerifySplits = 64;    // at most
constexpr int kVerifySegment = 4096; // at least so many logits per workgroup

struct VerifyLayout { size_t stats, best, bytes; };
inline VerifyLayout verify_layout(int64_t n, int64_t m) {
    VerifyLayout l;
    l.stats = 0;
    l.best = l.stats + (size_t)(n * (2 * m + 1) * kVerifySplits) * sizeof(float2);
    l.bytes = (l.best + (size_t)(n * kVerifySplits) * sizeof(uint64_t) + 255) / 256 * 256;
    return l;
}

hipError_t launch_verify(const VerifyArgs &a, bool f32, bool greedy, hipStream_t stream);

} // namespace sqk
