// Argument checks that the C-ABI files share (sq_api.cpp, sq_block_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <exception>
#include <vector>

#include "sq.h"

namespace sqk {

// Sets sq_last_error()'s text; returns st.
sq_status fail(sq_status st, const char *fmt, ...);
sq_status hip_fail(hipError_t e, const char *what);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Debug mode: with SQ_DEBUG set to a value other than "0" in the
// environment (read at each call), every compute entry point on a pool first
// runs sq_check_slots on its slot indices (which synchronises the stream) and
// enqueues nothing if one is out of range or repeated: overlapping slots would
// make the in-place update race.
bool debug_slots();

// Host memory for the debug checks' lists: no exception may leave through a C entry point.
template <typename T> sq_status host_list(std::vector<T> &v, size_t n) {
    try {
        v.resize(n);
    } catch (const std::exception &) {
        return fail(SQ_ENOMEM, "no host memory for a list of %zu entries", n);
    }
    return SQ_OK;
}

// A scratch buffer of at least `need` bytes.
sq_status check_work(const char *name, const void *p, size_t have, size_t need);
// With SQ_DEBUG: the sequence list on the host (synchronises the stream).
sq_status check_sequences(int32_t n_seq, int64_t n_tokens, const int32_t *cu, hipStream_t stream);
// The slots on the host (synchronises the stream): distinct, and, unless others are left out, inside [0, n_slots).
sq_status check_slot_list(const int32_t *slot_idx, int32_t n, int32_t n_slots, bool others, hipStream_t stream);

} // namespace sqk
