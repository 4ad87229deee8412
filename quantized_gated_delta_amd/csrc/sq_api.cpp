// C ABI of the packed low-bit recurrent-state pool (declared in include/sq.h).
//
// Host side only: argument validation, the pool layout, error text and
// kernel launches on the caller's stream.  The library owns no device
// memory; every device buffer comes from the caller.
#include "sq.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <exception>
#include <new>
#include <vector>

#include "sq_check.h"
#include "sq_internal.h"
#include "sq_seq.h"
#include "sq_verify.h"
#include "sq_window.h"

struct sq_pool {
    sq_pool_desc desc;          // head_bits points at bits below
    uint8_t bits[sqk::kMaxHeads];
    sqk::PoolView view;
    sqk::HeadTable tab;
    int64_t rec_bytes[sqk::kMaxHeads];
    size_t bytes;               // n_slots * slot_stride
    bool row_mixed;             // some head has per-key-row widths
};

namespace {
thread_local char g_err[512] = "";
} // namespace

namespace sqk {

sq_status fail(sq_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return st;
}

sq_status hip_fail(hipError_t e, const char *what) {
    return fail(SQ_EHIP, "%s: %s (%d)", what, hipGetErrorString(e), (int)e);
}

bool debug_slots() {
    const char *v = std::getenv("SQ_DEBUG");
    return v && v[0] && !(v[0] == '0' && v[1] == 0);
}

sq_status check_work(const char *name, const void *p, size_t have, size_t need) {
    if (need == 0) return SQ_OK;
    if (!p) return fail(SQ_EINVAL, "%s is NULL", name);
    if (!aligned(p, 256)) return fail(SQ_EINVAL, "%s is not 256-byte aligned", name);
    if (have < need) return fail(SQ_ENOMEM, "%s has %zu bytes, %zu are needed", name, have, need);
    return SQ_OK;
}

sq_status check_sequences(int32_t n_seq, int64_t n_tokens, const int32_t *cu, hipStream_t stream) {
    std::vector<int32_t> host;
    sq_status st = host_list(host, (size_t)n_seq + 1);
    if (st) return st;
    hipError_t e = hipStreamSynchronize(stream);
    if (e != hipSuccess) return hip_fail(e, "hipStreamSynchronize");
    e = hipMemcpy(host.data(), cu, sizeof(int32_t) * host.size(), hipMemcpyDeviceToHost);
    if (e != hipSuccess) return hip_fail(e, "hipMemcpy(cu)");
    for (int32_t i = 0; i <= n_seq; ++i)
        if (host[(size_t)i] < (i ? host[(size_t)i - 1] : 0) || host[(size_t)i] > n_tokens)
            return fail(SQ_EINVAL, "cu[%d] = %d must be non-decreasing within [0, %lld]", i, host[(size_t)i],
                        (long long)n_tokens);
    return SQ_OK;
}

sq_status check_slot_list(const int32_t *slot_idx, int32_t n, int32_t n_slots, bool others, hipStream_t stream) {
    std::vector<int32_t> host;
    std::vector<uint8_t> seen;  // zeros
    sq_status st;
    if ((st = host_list(host, (size_t)n)) || (st = host_list(seen, (size_t)n_slots))) return st;
    hipError_t e = hipStreamSynchronize(stream);
    if (e != hipSuccess) return hip_fail(e, "hipStreamSynchronize");
    e = hipMemcpy(host.data(), slot_idx, sizeof(int32_t) * (size_t)n, hipMemcpyDeviceToHost);
    if (e != hipSuccess) return hip_fail(e, "hipMemcpy(slot_idx)");
    for (int32_t i = 0; i < n; ++i) {
        const int32_t s = host[(size_t)i];
        if (s < 0 || s >= n_slots) {
            if (others) continue;
            return fail(SQ_EINVAL, "slot_idx[%d] = %d is outside [0, %d)", i, s, n_slots);
        }
        if (seen[(size_t)s]) return fail(SQ_EINVAL, "slot_idx[%d] = %d is repeated", i, s);
        seen[(size_t)s] = 1;
    }
    return SQ_OK;
}

} // namespace sqk

using sqk::aligned;
using sqk::check_sequences;
using sqk::check_slot_list;
using sqk::check_work;
using sqk::debug_slots;
using sqk::fail;
using sqk::hip_fail;

namespace {

// Rows of one head with per-key-row widths: non-decreasing widths in
// {4, 6, 8} that change only at multiples of the rows a wavefront holds per
// row slot (d / 16 at d = 128, d / 4 at d = 64).  Returns the 4- and 6-bit
// row counts.
sq_status row_split(const sq_pool_desc *d, const uint8_t *row_bits, int h, uint8_t *n4,
                    uint8_t *n6) {
    const int dk = d->d_k, grain = dk == 128 ? 8 : 16;
    const uint8_t *w = row_bits + (size_t)h * dk;
    int c4 = 0, c6 = 0;
    for (int i = 0; i < dk; ++i) {
        if (w[i] != 4 && w[i] != 6 && w[i] != 8)
            return fail(SQ_EUNSUPPORTED, "row_bits[%d][%d] = %d, must be 4, 6 or 8", h, i, w[i]);
        if (i > 0 && w[i] < w[i - 1])
            return fail(SQ_EUNSUPPORTED, "row_bits[%d] must be non-decreasing (row %d)", h, i);
        if (i > 0 && w[i] != w[i - 1] && i % grain != 0)
            return fail(SQ_EUNSUPPORTED,
                        "row_bits[%d] changes width at row %d, not a multiple of %d", h, i, grain);
        c4 += w[i] == 4;
        c6 += w[i] == 6;
    }
    *n4 = (uint8_t)c4;
    *n6 = (uint8_t)c6;
    return SQ_OK;
}

sq_status check_desc(const sq_pool_desc *d, const uint8_t *row_bits = nullptr) {
    if (!d) return fail(SQ_EINVAL, "desc is NULL");
    if (d->n_slots < 1) return fail(SQ_EINVAL, "n_slots must be >= 1 (got %d)", d->n_slots);
    if (d->n_heads < 1 || d->n_heads > sqk::kMaxHeads)
        return fail(SQ_EUNSUPPORTED, "n_heads must be in [1, %d] (got %d)", sqk::kMaxHeads, d->n_heads);
    if (d->d_k != d->d_v)
        return fail(SQ_EUNSUPPORTED, "d_k must equal d_v (got %d, %d)", d->d_k, d->d_v);
    if (d->d_k != 64 && d->d_k != 128)
        return fail(SQ_EUNSUPPORTED, "d_k = d_v must be 64 or 128 (got %d)", d->d_k);
    if (d->gate != SQ_GATE_GDN && d->gate != SQ_GATE_KDA)
        return fail(SQ_EINVAL, "gate must be SQ_GATE_GDN or SQ_GATE_KDA (got %d)", (int)d->gate);
    if (!d->head_bits) return fail(SQ_EINVAL, "head_bits is NULL");
    for (int h = 0; h < d->n_heads; ++h) {
        const int b = d->head_bits[h];
        if (b == 0) {
            if (!row_bits)
                return fail(SQ_EINVAL, "head_bits[%d] = 0 needs per-row widths (row_bits)", h);
            uint8_t n4, n6;
            sq_status st = row_split(d, row_bits, h, &n4, &n6);
            if (st) return st;
        } else if (b != 4 && b != 6 && b != 8 && b != 16) {
            return fail(SQ_EUNSUPPORTED, "head_bits[%d] = %d, must be 4, 6, 8 or 16", h, b);
        }
    }
    return SQ_OK;
}

// Layout: per slot, head records back to back in head order.  row_bits is
// read only for heads whose head_bits is 0 (already validated).
int64_t layout(const sq_pool_desc *d, const uint8_t *row_bits, int64_t *off, int64_t *rec,
               uint8_t *n4 = nullptr, uint8_t *n6 = nullptr) {
    int64_t pos = 0;
    for (int h = 0; h < d->n_heads; ++h) {
        int64_t rb;
        uint8_t a = 0, b = 0;
        if (d->head_bits[h] == 0) {
            row_split(d, row_bits, h, &a, &b);
            rb = sqk::record_bytes_rows(a, b, d->d_k);
        } else {
            rb = sqk::record_bytes(d->head_bits[h], d->d_k);
        }
        if (n4) n4[h] = a;
        if (n6) n6[h] = b;
        if (off) off[h] = pos;
        if (rec) rec[h] = rb;
        pos += rb;
    }
    return pos;
}

sq_status check_rows(const sq_pool *p, const int32_t *slot_idx, int32_t n) {
    if (!p) return fail(SQ_EINVAL, "pool is NULL");
    if (n < 0) return fail(SQ_EINVAL, "n must be >= 0 (got %d)", n);
    if (n > p->desc.n_slots)
        return fail(SQ_EINVAL, "n = %d exceeds n_slots = %d (slots must be distinct)", n, p->desc.n_slots);
    if ((int64_t)n * p->desc.n_heads > 0x7FFFFFFFll)
        return fail(SQ_EUNSUPPORTED, "n * n_heads exceeds the grid limit");
    if (n > 0 && !slot_idx) return fail(SQ_EINVAL, "slot_idx is NULL");
    if (n > 0 && !aligned(slot_idx, 4)) return fail(SQ_EINVAL, "slot_idx is not 4-byte aligned");
    return SQ_OK;
}

sq_status check_io(const char *name, const void *p, bool need) {
    if (!need) return SQ_OK;
    if (!p) return fail(SQ_EINVAL, "%s is NULL", name);
    if (!aligned(p, 16)) return fail(SQ_EINVAL, "%s is not 16-byte aligned", name);
    return SQ_OK;
}

sq_status check_step_io(const void *q, const void *k, const void *v, const void *beta,
                        const void *g, sq_dtype in_dtype, const void *y, sq_dtype y_dtype) {
    if (in_dtype != SQ_F32 && in_dtype != SQ_BF16)
        return fail(SQ_EINVAL, "in_dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)in_dtype);
    if (y_dtype != SQ_F32 && y_dtype != SQ_BF16)
        return fail(SQ_EINVAL, "y_dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)y_dtype);
    sq_status st;
    if ((st = check_io("q", q, true)) || (st = check_io("k", k, true)) ||
        (st = check_io("v", v, true)) || (st = check_io("beta", beta, true)) ||
        (st = check_io("g", g, true)) || (st = check_io("y", y, true)))
        return st;
    return SQ_OK;
}

sq_status check_seq(const sq_seq_desc *d) {
    if (!d) return fail(SQ_EINVAL, "desc is NULL");
    if (d->n_seq < 0) return fail(SQ_EINVAL, "n_seq must be >= 0 (got %d)", d->n_seq);
    if (d->n_tokens < 0) return fail(SQ_EINVAL, "n_tokens must be >= 0 (got %lld)", (long long)d->n_tokens);
    if (d->n_heads < 1) return fail(SQ_EINVAL, "n_heads must be >= 1 (got %d)", d->n_heads);
    if (d->n_key_heads < 1 || d->n_heads % d->n_key_heads != 0)
        return fail(SQ_EINVAL, "n_key_heads = %d is not a divisor of n_heads = %d", d->n_key_heads, d->n_heads);
    if (d->d_k != d->d_v) return fail(SQ_EUNSUPPORTED, "d_k must equal d_v (got %d, %d)", d->d_k, d->d_v);
    if (d->d_k != 64 && d->d_k != 128)
        return fail(SQ_EUNSUPPORTED, "d_k = d_v must be 64 or 128 (got %d)", d->d_k);
    if (d->gate != SQ_GATE_GDN && d->gate != SQ_GATE_KDA)
        return fail(SQ_EINVAL, "gate must be SQ_GATE_GDN or SQ_GATE_KDA (got %d)", (int)d->gate);
    if (d->in_dtype != SQ_F32 && d->in_dtype != SQ_BF16)
        return fail(SQ_EINVAL, "in_dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)d->in_dtype);
    if (d->y_dtype != SQ_F32 && d->y_dtype != SQ_BF16)
        return fail(SQ_EINVAL, "y_dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)d->y_dtype);
    if (d->n_tokens > 0x7FFFFFFFll - 64) return fail(SQ_EUNSUPPORTED, "n_tokens exceeds 2^31 - 65");
    // grids: one workgroup per (chunk slot, head) and per (sequence, head, 16 columns)
    const int64_t slots = sqk::chunk_slots(d->n_tokens, d->n_seq);
    if (slots * d->n_heads > 0x7FFFFFFFll || (int64_t)d->n_seq * d->n_heads > 0x7FFFFFFFll / 8 - 8)
        return fail(SQ_EUNSUPPORTED, "n_tokens or n_seq times n_heads exceeds the grid limit");
    const int64_t per16 = d->in_dtype == SQ_BF16 ? 8 : 4, dense_k = (int64_t)d->n_key_heads * d->d_k,
                  dense_v = (int64_t)d->n_heads * d->d_v;
    const struct { const char *name; int64_t stride, dense; } st[3] = {
        {"q_stride", d->q_stride, dense_k}, {"k_stride", d->k_stride, dense_k}, {"v_stride", d->v_stride, dense_v}};
    for (const auto &s : st)
        if (s.stride != 0 && (s.stride < s.dense || s.stride % per16 != 0 || s.stride > 1 << 24))
            return fail(SQ_EINVAL, "%s = %lld must be 0 or a multiple of %lld, at least %lld and at most 2^24", s.name,
                        (long long)s.stride, (long long)per16, (long long)s.dense);
    if (dense_v > 1 << 24) return fail(SQ_EUNSUPPORTED, "n_heads * d_v exceeds 2^24");  // 32-bit offsets within a chunk
    return SQ_OK;
}

sqk::SeqArgs seq_args(const sq_seq_desc *d, const int32_t *cu, const void *q, const void *k, const void *v,
                      const void *beta, const void *g, const float *S0, void *work) {
    sqk::SeqArgs a{};
    a.q = q; a.k = k; a.v = v; a.beta = beta; a.g = g;
    a.q_stride = d->q_stride ? d->q_stride : (int64_t)d->n_key_heads * d->d_k;
    a.k_stride = d->k_stride ? d->k_stride : (int64_t)d->n_key_heads * d->d_k;
    a.v_stride = d->v_stride ? d->v_stride : (int64_t)d->n_heads * d->d_v;
    a.cu = cu;
    a.n_seq = d->n_seq;
    a.n_heads = d->n_heads;
    a.n_key_heads = d->n_key_heads;
    a.n_tokens = d->n_tokens;
    a.S0 = S0;
    a.work = static_cast<uint8_t *>(work);
    return a;
}

// beta, GDN's g and their gradients: read and written by the element.
sq_status check_elems(const sq_seq_desc *d, const char *name, const void *p, bool row_of_channels) {
    if (d->n_tokens == 0) return SQ_OK;
    if (row_of_channels) return check_io(name, p, true);
    if (!p) return fail(SQ_EINVAL, "%s is NULL", name);
    const int size = d->in_dtype == SQ_F32 ? 4 : 2;
    if (!aligned(p, size)) return fail(SQ_EINVAL, "%s is not %d-byte aligned", name, size);
    return SQ_OK;
}

// Pointers that every sequence call takes.
sq_status check_seq_io(const sq_seq_desc *d, const int32_t *cu, const void *q, const void *k, const void *v,
                       const void *beta, const void *g, const float *S0) {
    sq_status st;
    const bool any = d->n_tokens > 0;
    if (!cu) return fail(SQ_EINVAL, "cu is NULL");
    if (!aligned(cu, 4)) return fail(SQ_EINVAL, "cu is not 4-byte aligned");
    if ((st = check_io("q", q, any)) || (st = check_io("k", k, any)) || (st = check_io("v", v, any)) ||
        (st = check_elems(d, "beta", beta, false)) || (st = check_elems(d, "g", g, d->gate == SQ_GATE_KDA)) ||
        (st = check_io("S0", S0, S0 != nullptr)))
        return st;
    return SQ_OK;
}

// What both window calls check besides the pool.
sq_status check_window(int32_t length, const int32_t *lens, int32_t n_heads, int32_t n_key_heads, const void *q,
                       const void *k, const void *v, const void *beta, const void *g, sq_dtype in_dtype,
                       const void *y, sq_dtype y_dtype, const float *S_out) {
    if (length < 1 || length > SQ_WINDOW_MAX)
        return fail(SQ_EINVAL, "length must be in [1, %d] (got %d)", SQ_WINDOW_MAX, length);
    if (n_key_heads < 1 || n_heads % n_key_heads != 0)
        return fail(SQ_EINVAL, "n_key_heads = %d is not a divisor of n_heads = %d", n_key_heads, n_heads);
    if (in_dtype != SQ_F32 && in_dtype != SQ_BF16)
        return fail(SQ_EINVAL, "in_dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)in_dtype);
    if (y_dtype != SQ_F32 && y_dtype != SQ_BF16)
        return fail(SQ_EINVAL, "y_dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)y_dtype);
    if (!y && !S_out) return fail(SQ_EINVAL, "y and S_out are both NULL");
    if (lens && !aligned(lens, 4)) return fail(SQ_EINVAL, "lens is not 4-byte aligned");
    sq_status st;
    if ((st = check_io("q", q, y != nullptr)) || (st = check_io("k", k, true)) || (st = check_io("v", v, true)) ||
        (st = check_io("beta", beta, true)) || (st = check_io("g", g, true)) || (st = check_io("y", y, y != nullptr)) ||
        (st = check_io("S_out", S_out, S_out != nullptr)))
        return st;
    return SQ_OK;
}

sqk::WindowArgs window_args(const void *base, int64_t slot_stride, const int32_t *slot_idx, int32_t n, int32_t length,
                            const int32_t *lens, int32_t n_heads, int32_t n_key_heads, const void *q, const void *k,
                            const void *v, const void *beta, const void *g, void *y, float *S_out) {
    sqk::WindowArgs a;
    a.base = static_cast<const uint8_t *>(base);
    a.slot_stride = slot_stride;
    a.slot = slot_idx; a.lens = lens;
    a.n = n; a.length = length; a.n_heads = n_heads; a.n_key_heads = n_key_heads;
    a.q = q; a.k = k; a.v = v; a.beta = beta; a.g = g;
    a.y = y; a.S_out = S_out;
    return a;
}

} // namespace

extern "C" {

const char *sq_last_error(void) { return g_err; }

const char *sq_version(void) { return "sq 0.1 (gfx950)"; }

sq_status sq_pool_bytes_rows(const sq_pool_desc *desc, const uint8_t *row_bits, size_t *bytes) {
    sq_status st = check_desc(desc, row_bits);
    if (st) return st;
    if (!bytes) return fail(SQ_EINVAL, "bytes is NULL");
    const int64_t stride = layout(desc, row_bits, nullptr, nullptr);
    if ((uint64_t)desc->n_slots > (uint64_t)INT64_MAX / (uint64_t)stride)
        return fail(SQ_ENOMEM, "pool size overflows");
    *bytes = (size_t)((int64_t)desc->n_slots * stride);
    return SQ_OK;
}

sq_status sq_pool_bytes(const sq_pool_desc *desc, size_t *bytes) {
    return sq_pool_bytes_rows(desc, nullptr, bytes);
}

sq_status sq_pool_create_rows(const sq_pool_desc *desc, const uint8_t *row_bits, void *dev_buf,
                              size_t bytes, sq_pool **out) {
    if (!out) return fail(SQ_EINVAL, "out is NULL");
    *out = nullptr;
    size_t need = 0;
    sq_status st = sq_pool_bytes_rows(desc, row_bits, &need);
    if (st) return st;
    if (!dev_buf) return fail(SQ_EINVAL, "dev_buf is NULL");
    if (!aligned(dev_buf, 256)) return fail(SQ_EINVAL, "dev_buf is not 256-byte aligned");
    if (bytes < need) return fail(SQ_ENOMEM, "buffer has %zu bytes, pool needs %zu", bytes, need);
    sq_pool *p = new (std::nothrow) sq_pool;
    if (!p) return fail(SQ_ENOMEM, "host allocation failed");
    std::memset(p, 0, sizeof *p);
    p->desc = *desc;
    std::memcpy(p->bits, desc->head_bits, (size_t)desc->n_heads);
    p->desc.head_bits = p->bits;
    uint8_t n4[sqk::kMaxHeads] = {}, n6[sqk::kMaxHeads] = {};
    const int64_t stride = layout(desc, row_bits, p->tab.off, p->rec_bytes, n4, n6);
    for (int h = 0; h < desc->n_heads; ++h) {
        p->tab.info[h] = sqk::head_info(desc->head_bits[h], n4[h], n6[h]);
        p->row_mixed |= desc->head_bits[h] == 0;
    }
    int s = 0;
    while ((1 << s) < desc->n_heads) ++s;
    p->view.h_shift = 31 + s;
    p->view.h_magic = (uint32_t)((((uint64_t)1 << (31 + s)) + (uint64_t)desc->n_heads - 1) /
                                 (uint64_t)desc->n_heads);
    p->view.row_mixed = p->row_mixed;
    p->view.base = static_cast<uint8_t *>(dev_buf);
    p->view.slot_stride = stride;
    p->view.n_heads = desc->n_heads;
    p->view.d = desc->d_k;
    p->bytes = need;
    *out = p;
    return SQ_OK;
}

sq_status sq_pool_create(const sq_pool_desc *desc, void *dev_buf, size_t bytes, sq_pool **out) {
    return sq_pool_create_rows(desc, nullptr, dev_buf, bytes, out);
}

sq_status sq_pool_destroy(sq_pool *pool) {
    delete pool;
    return SQ_OK;
}

sq_status sq_pool_layout(const sq_pool *pool, int64_t *slot_stride, int64_t *head_off,
                         int64_t *record_bytes) {
    if (!pool) return fail(SQ_EINVAL, "pool is NULL");
    if (slot_stride) *slot_stride = pool->view.slot_stride;
    for (int h = 0; h < pool->desc.n_heads; ++h) {
        if (head_off) head_off[h] = pool->tab.off[h];
        if (record_bytes) record_bytes[h] = pool->rec_bytes[h];
    }
    return SQ_OK;
}

sq_status sq_pool_set_row_impact(sq_pool *pool, const float *impact) {
    if (!pool) return fail(SQ_EINVAL, "pool is NULL");
    if (impact && !aligned(impact, 16)) return fail(SQ_EINVAL, "impact is not 16-byte aligned");
    pool->view.impact = impact;
    return SQ_OK;
}

sq_status sq_quant_state(sq_pool *pool, const int32_t *slot_idx, int32_t n, const float *S,
                         hipStream_t stream) {
    sq_status st = check_rows(pool, slot_idx, n);
    if (st) return st;
    if (n == 0) return SQ_OK;
    if (debug_slots() && (st = sq_check_slots(pool, slot_idx, n, stream))) return st;
    if ((st = check_io("S", S, true))) return st;
    const hipError_t e = sqk::launch_quant_state(pool->view, pool->tab, slot_idx, n, S, stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "quant_state launch");
}

sq_status sq_dequant_state(const sq_pool *pool, const int32_t *slot_idx, int32_t n, float *S,
                           hipStream_t stream) {
    sq_status st = check_rows(pool, slot_idx, n);
    if (st) return st;
    if (n == 0) return SQ_OK;
    if (debug_slots() && (st = sq_check_slots(pool, slot_idx, n, stream))) return st;
    if ((st = check_io("S", S, true))) return st;
    const hipError_t e = sqk::launch_dequant_state(pool->view, pool->tab, slot_idx, n, S, stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "dequant_state launch");
}

sq_status sq_decode_step(sq_pool *pool, const int32_t *slot_idx, int32_t n, const void *q,
                         const void *k, const void *v, const void *beta, const void *g,
                         sq_dtype in_dtype, void *y, sq_dtype y_dtype, hipStream_t stream) {
    sq_status st = check_rows(pool, slot_idx, n);
    if (st) return st;
    if (n == 0) return SQ_OK;
    if (debug_slots() && (st = sq_check_slots(pool, slot_idx, n, stream))) return st;
    if ((st = check_step_io(q, k, v, beta, g, in_dtype, y, y_dtype))) return st;
    sqk::StepIO io;
    io.slot = slot_idx;
    io.q = q; io.k = k; io.v = v; io.beta = beta; io.g = g; io.y = y;
    io.n = n;
    io.in_bf16 = in_dtype == SQ_BF16;
    io.y_bf16 = y_dtype == SQ_BF16;
    io.kda = pool->desc.gate == SQ_GATE_KDA;
    io.s_out = nullptr;
    const hipError_t e = sqk::launch_decode(pool->view, pool->tab, io, stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "decode_step launch");
}

sq_status sq_decode_update(const sq_pool *pool, const int32_t *slot_idx, int32_t n, const void *q,
                           const void *k, const void *v, const void *beta, const void *g,
                           sq_dtype in_dtype, void *y, sq_dtype y_dtype, float *S_out,
                           hipStream_t stream) {
    sq_status st = check_rows(pool, slot_idx, n);
    if (st) return st;
    if (n == 0) return SQ_OK;
    if (debug_slots() && (st = sq_check_slots(pool, slot_idx, n, stream))) return st;
    if ((st = check_step_io(q, k, v, beta, g, in_dtype, y, y_dtype))) return st;
    if ((st = check_io("S_out", S_out, true))) return st;
    sqk::StepIO io;
    io.slot = slot_idx;
    io.q = q; io.k = k; io.v = v; io.beta = beta; io.g = g; io.y = y;
    io.n = n;
    io.in_bf16 = in_dtype == SQ_BF16;
    io.y_bf16 = y_dtype == SQ_BF16;
    io.kda = pool->desc.gate == SQ_GATE_KDA;
    io.s_out = S_out;
    const hipError_t e = sqk::launch_decode_update(pool->view, pool->tab, io, stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "decode_update launch");
}

sq_status sq_split_step_noalloc(sq_pool *pool, const int32_t *slot_idx, int32_t n, const void *q,
                                const void *k, const void *v, const void *beta, const void *g,
                                sq_dtype in_dtype, void *y, sq_dtype y_dtype, hipStream_t stream) {
    sq_status st = check_rows(pool, slot_idx, n);
    if (st) return st;
    if (n == 0) return SQ_OK;
    if (debug_slots() && (st = sq_check_slots(pool, slot_idx, n, stream))) return st;
    const uint64_t need = (uint64_t)n * (uint64_t)pool->desc.n_heads * (uint64_t)pool->desc.d_k *
                          (uint64_t)pool->desc.d_v * sizeof(float);
    if (need > (uint64_t)SQ_SPLIT_SCRATCH_BYTES)
        return fail(SQ_ENOMEM,
                    "S' of %d requests x %d heads needs %llu bytes, the static buffer holds %llu "
                    "(at most %llu requests of this pool per call)",
                    n, pool->desc.n_heads, (unsigned long long)need,
                    (unsigned long long)SQ_SPLIT_SCRATCH_BYTES,
                    (unsigned long long)(SQ_SPLIT_SCRATCH_BYTES /
                                         ((uint64_t)pool->desc.n_heads * pool->desc.d_k *
                                          pool->desc.d_v * sizeof(float))));
    if ((st = check_step_io(q, k, v, beta, g, in_dtype, y, y_dtype))) return st;
    sqk::StepIO io;
    io.slot = slot_idx;
    io.q = q; io.k = k; io.v = v; io.beta = beta; io.g = g; io.y = y;
    io.n = n;
    io.in_bf16 = in_dtype == SQ_BF16;
    io.y_bf16 = y_dtype == SQ_BF16;
    io.kda = pool->desc.gate == SQ_GATE_KDA;
    io.s_out = nullptr;
    const hipError_t e = sqk::launch_split_step_scratch(pool->view, pool->tab, io, stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "split_step_noalloc launch");
}

sq_status sq_f32_decode_step(float *state_pool, int32_t n_slots, int32_t n_heads, int32_t d_k,
                             int32_t d_v, sq_gate gate, const int32_t *slot_idx, int32_t n,
                             const void *q, const void *k, const void *v, const void *beta,
                             const void *g, sq_dtype in_dtype, void *y, sq_dtype y_dtype,
                             hipStream_t stream) {
    if (n_slots < 1) return fail(SQ_EINVAL, "n_slots must be >= 1 (got %d)", n_slots);
    if (n_heads < 1) return fail(SQ_EINVAL, "n_heads must be >= 1 (got %d)", n_heads);
    if (d_k != d_v) return fail(SQ_EUNSUPPORTED, "d_k must equal d_v (got %d, %d)", d_k, d_v);
    if (d_k != 64 && d_k != 128) return fail(SQ_EUNSUPPORTED, "d must be 64 or 128 (got %d)", d_k);
    if (gate != SQ_GATE_GDN && gate != SQ_GATE_KDA)
        return fail(SQ_EINVAL, "gate must be SQ_GATE_GDN or SQ_GATE_KDA (got %d)", (int)gate);
    if (n < 0) return fail(SQ_EINVAL, "n must be >= 0 (got %d)", n);
    if (n > n_slots) return fail(SQ_EINVAL, "n = %d exceeds n_slots = %d", n, n_slots);
    if ((int64_t)n * n_heads > 0x7FFFFFFFll) return fail(SQ_EUNSUPPORTED, "grid too large");
    if (n == 0) return SQ_OK;
    if (!slot_idx) return fail(SQ_EINVAL, "slot_idx is NULL");
    sq_status st;
    if ((st = check_io("state_pool", state_pool, true))) return st;
    if ((st = check_step_io(q, k, v, beta, g, in_dtype, y, y_dtype))) return st;
    sqk::StepIO io;
    io.slot = slot_idx;
    io.q = q; io.k = k; io.v = v; io.beta = beta; io.g = g; io.y = y;
    io.n = n;
    io.in_bf16 = in_dtype == SQ_BF16;
    io.y_bf16 = y_dtype == SQ_BF16;
    io.kda = gate == SQ_GATE_KDA;
    const int64_t stride = (int64_t)n_heads * d_k * d_v;
    const hipError_t e = sqk::launch_f32_decode(state_pool, stride, n_heads, d_k, io, stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "f32_decode_step launch");
}

sq_status sq_check_slots(const sq_pool *pool, const int32_t *slot_idx, int32_t n,
                         hipStream_t stream) {
    sq_status st = check_rows(pool, slot_idx, n);
    if (st) return st;
    if (n == 0) return SQ_OK;
    return check_slot_list(slot_idx, n, pool->desc.n_slots, false, stream);
}

sq_status sq_chunk_bytes(const sq_seq_desc *desc, size_t *work, size_t *save) {
    sq_status st = check_seq(desc);
    if (st) return st;
    if (!work) return fail(SQ_EINVAL, "work is NULL");
    const bool kda = desc->gate == SQ_GATE_KDA, f32 = desc->in_dtype == SQ_F32;
    const int64_t blocks = sqk::chunk_slots(desc->n_tokens, desc->n_seq) * desc->n_heads;
    int64_t block = sqk::forward_layout(desc->d_k, kda, f32, desc->y_dtype == SQ_F32 ? 3 : 2).block;
    if (save) {
        const int64_t back = sqk::backward_layout(desc->d_k, kda, f32).block;
        block = back > block ? back : block;
        *save = (size_t)(blocks * sqk::save_layout(desc->d_k).block);
    }
    *work = (size_t)(blocks * block);
    return SQ_OK;
}

sq_status sq_chunk_forward(const sq_seq_desc *desc, const int32_t *cu, const void *q, const void *k, const void *v,
                           const void *beta, const void *g, const float *S0, void *y, float *S_out, void *save,
                           size_t save_bytes, void *work, size_t work_bytes, hipStream_t stream) {
    size_t need = 0, both = 0, keep = 0;
    sq_status st = sq_chunk_bytes(desc, &need, nullptr);
    if (st || (st = sq_chunk_bytes(desc, &both, &keep))) return st;
    if (desc->n_seq == 0) return SQ_OK;
    if ((st = check_seq_io(desc, cu, q, k, v, beta, g, S0)) || (st = check_io("y", y, desc->n_tokens > 0)) ||
        (st = check_io("S_out", S_out, S_out != nullptr)) || (st = check_work("work", work, work_bytes, need)) ||
        (save && (st = check_work("save", save, save_bytes, keep))))
        return st;
    if (debug_slots() && (st = check_sequences(desc->n_seq, desc->n_tokens, cu, stream))) return st;
    sqk::SeqArgs a = seq_args(desc, cu, q, k, v, beta, g, S0, work);
    a.y = y;
    a.S_out = S_out;
    a.save = static_cast<uint8_t *>(save);
    const hipError_t e = sqk::launch_chunk_forward(a, desc->d_k, desc->gate == SQ_GATE_KDA, desc->in_dtype == SQ_F32,
                                                   desc->y_dtype == SQ_F32, stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "chunk_forward launch");
}

sq_status sq_chunk_backward(const sq_seq_desc *desc, const int32_t *cu, const void *q, const void *k, const void *v,
                            const void *beta, const void *g, const void *dy, const float *dS_out, const void *save,
                            size_t save_bytes, void *dq, void *dk, void *dv, void *dbeta, void *dg, float *dS0,
                            void *work, size_t work_bytes, hipStream_t stream) {
    size_t need = 0, keep = 0;
    sq_status st = sq_chunk_bytes(desc, &need, &keep);
    if (st) return st;
    if (desc->n_seq == 0) return SQ_OK;
    const bool any = desc->n_tokens > 0;
    if ((st = check_seq_io(desc, cu, q, k, v, beta, g, nullptr)) || (st = check_io("dy", dy, any)) ||
        (st = check_io("dS_out", dS_out, dS_out != nullptr)) || (st = check_io("dq", dq, any)) ||
        (st = check_io("dk", dk, any)) || (st = check_io("dv", dv, any)) || (st = check_elems(desc, "dbeta", dbeta, false)) ||
        (st = check_elems(desc, "dg", dg, desc->gate == SQ_GATE_KDA)) || (st = check_io("dS0", dS0, dS0 != nullptr)) ||
        (st = check_work("save", save, save_bytes, keep)) || (st = check_work("work", work, work_bytes, need)))
        return st;
    if (debug_slots() && (st = check_sequences(desc->n_seq, desc->n_tokens, cu, stream))) return st;
    sqk::SeqArgs a = seq_args(desc, cu, q, k, v, beta, g, nullptr, work);
    a.save = static_cast<uint8_t *>(const_cast<void *>(save));
    a.dy = dy; a.dS_out = dS_out;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dbeta = dbeta; a.dg = dg; a.dS0 = dS0;
    const hipError_t e = sqk::launch_chunk_backward(a, desc->d_k, desc->gate == SQ_GATE_KDA,
                                                    desc->in_dtype == SQ_F32, stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "chunk_backward launch");
}

sq_status sq_window_update(const sq_pool *pool, const int32_t *slot_idx, int32_t n, int32_t length,
                           const int32_t *lens, int32_t n_key_heads, const void *q, const void *k, const void *v,
                           const void *beta, const void *g, sq_dtype in_dtype, void *y, sq_dtype y_dtype,
                           float *S_out, hipStream_t stream) {
    sq_status st = check_rows(pool, slot_idx, n);
    if (st) return st;
    if (n == 0) return SQ_OK;
    if ((st = check_window(length, lens, pool->desc.n_heads, n_key_heads, q, k, v, beta, g, in_dtype, y, y_dtype, S_out)))
        return st;
    if (debug_slots() && (st = sq_check_slots(pool, slot_idx, n, stream))) return st;
    const sqk::WindowArgs a = window_args(pool->view.base, pool->view.slot_stride, slot_idx, n, length, lens,
                                          pool->desc.n_heads, n_key_heads, q, k, v, beta, g, y, S_out);
    const hipError_t e = sqk::launch_window(a, &pool->tab, pool->desc.d_k, pool->desc.gate == SQ_GATE_KDA,
                                            in_dtype == SQ_F32, y_dtype == SQ_F32, stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "window_update launch");
}

sq_status sq_f32_window_update(const float *state_pool, int32_t n_slots, int32_t n_heads, int32_t n_key_heads,
                               int32_t d_k, int32_t d_v, sq_gate gate, const int32_t *slot_idx, int32_t n,
                               int32_t length, const int32_t *lens, const void *q, const void *k, const void *v,
                               const void *beta, const void *g, sq_dtype in_dtype, void *y, sq_dtype y_dtype,
                               float *S_out, hipStream_t stream) {
    if (n_slots < 1) return fail(SQ_EINVAL, "n_slots must be >= 1 (got %d)", n_slots);
    if (n_heads < 1) return fail(SQ_EINVAL, "n_heads must be >= 1 (got %d)", n_heads);
    if (d_k != d_v) return fail(SQ_EUNSUPPORTED, "d_k must equal d_v (got %d, %d)", d_k, d_v);
    if (d_k != 64 && d_k != 128) return fail(SQ_EUNSUPPORTED, "d must be 64 or 128 (got %d)", d_k);
    if (gate != SQ_GATE_GDN && gate != SQ_GATE_KDA)
        return fail(SQ_EINVAL, "gate must be SQ_GATE_GDN or SQ_GATE_KDA (got %d)", (int)gate);
    if (n < 0) return fail(SQ_EINVAL, "n must be >= 0 (got %d)", n);
    if (n > n_slots) return fail(SQ_EINVAL, "n = %d exceeds n_slots = %d", n, n_slots);
    if ((int64_t)n * n_heads > 0x7FFFFFFFll) return fail(SQ_EUNSUPPORTED, "grid too large");
    if (n == 0) return SQ_OK;
    if (!slot_idx) return fail(SQ_EINVAL, "slot_idx is NULL");
    sq_status st;
    if ((st = check_io("state_pool", state_pool, true)) ||
        (st = check_window(length, lens, n_heads, n_key_heads, q, k, v, beta, g, in_dtype, y, y_dtype, S_out)))
        return st;
    const sqk::WindowArgs a = window_args(state_pool, (int64_t)n_heads * d_k * d_v, slot_idx, n, length, lens, n_heads,
                                          n_key_heads, q, k, v, beta, g, y, S_out);
    const hipError_t e = sqk::launch_window(a, nullptr, d_k, gate == SQ_GATE_KDA, in_dtype == SQ_F32,
                                            y_dtype == SQ_F32, stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "f32_window_update launch");
}

sq_status sq_verify_bytes(int32_t n, int32_t m, size_t *bytes) {
    if (n < 0) return fail(SQ_EINVAL, "n must be >= 0 (got %d)", n);
    if (m < 1 || m > SQ_DRAFT_MAX) return fail(SQ_EINVAL, "m must be in [1, %d] (got %d)", SQ_DRAFT_MAX, m);
    if (!bytes) return fail(SQ_EINVAL, "bytes is NULL");
    *bytes = sqk::verify_layout(n, m).bytes;
    return SQ_OK;
}

sq_status sq_verify_draft(int32_t n, int32_t m, int32_t vocab, const void *target, int64_t target_stride,
                          const void *draft, int64_t draft_stride, sq_dtype logits_dtype, const int32_t *tokens,
                          const int32_t *lens, const float *accept_u, const float *sample_e, float temperature,
                          int32_t *accepted, int32_t *next, void *work, size_t work_bytes, hipStream_t stream) {
    size_t need = 0;
    sq_status st = sq_verify_bytes(n, m, &need);
    if (st) return st;
    if (vocab < 1 || vocab > 0x7FFFFFFF - 65536) return fail(SQ_EINVAL, "vocab = %d is out of range", vocab);
    if (logits_dtype != SQ_F32 && logits_dtype != SQ_BF16)
        return fail(SQ_EINVAL, "logits_dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)logits_dtype);
    // the kernels scale logits by log2(e) / T
    if (!(temperature >= 0.f) || std::isinf(temperature) || (temperature > 0.f && std::isinf(1.f / temperature * sqk::kLog2e)))
        return fail(SQ_EINVAL, "temperature = %g must be 0 or a positive number, and 1 / temperature within fp32", (double)temperature);
    if ((target_stride && target_stride < vocab) || (draft && draft_stride && draft_stride < vocab) ||
        target_stride > INT64_MAX / 16 / 65536 || draft_stride > INT64_MAX / 16 / 65536)
        return fail(SQ_EINVAL, "a row stride must be 0 or at least vocab = %d", vocab);
    if (n == 0) return SQ_OK;
    if ((int64_t)n * (2 * m + 1) > 65535) return fail(SQ_EUNSUPPORTED, "n * (2 m + 1) exceeds 65535 rows");
    const bool greedy = temperature == 0.f;
    const uintptr_t e = logits_dtype == SQ_F32 ? 4 : 2;
    const struct { const char *name; const void *p; bool need; uintptr_t align; } io[8] = {
        {"target", target, true, e}, {"draft", draft, false, e}, {"tokens", tokens, true, 4}, {"lens", lens, false, 4},
        {"accept_u", accept_u, !greedy, 4}, {"sample_e", sample_e, !greedy, 4}, {"accepted", accepted, true, 4}, {"next", next, true, 4}};
    for (const auto &x : io) {
        if (x.need && !x.p) return fail(SQ_EINVAL, "%s is NULL", x.name);
        if (x.p && !aligned(x.p, x.align)) return fail(SQ_EINVAL, "%s is not %d-byte aligned", x.name, (int)x.align);
    }
    if ((st = check_work("work", work, work_bytes, need))) return st;
    // written by one workgroup of a request while its others read the lists
    const struct { const char *name; const void *p; size_t count; } list[4] = {
        {"accepted", accepted, (size_t)n}, {"next", next, (size_t)n}, {"tokens", tokens, (size_t)n * m}, {"lens", lens, lens ? (size_t)n : 0}};
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 4; ++j) {
            const uintptr_t x = reinterpret_cast<uintptr_t>(list[i].p), y = reinterpret_cast<uintptr_t>(list[j].p);
            if (x < y + 4 * list[j].count && y < x + 4 * list[i].count && list[j].count)
                return fail(SQ_EINVAL, "%s and %s overlap", list[i].name, list[j].name);
        }
    const sqk::VerifyLayout lay = sqk::verify_layout(n, m);
    uint8_t *base = static_cast<uint8_t *>(work);
    sqk::VerifyArgs a{};
    a.target = target; a.draft = greedy ? nullptr : draft;
    a.target_stride = target_stride ? target_stride : vocab;
    a.draft_stride = draft_stride ? draft_stride : vocab;
    a.tokens = tokens; a.lens = lens; a.accept_u = accept_u; a.sample_e = sample_e;
    a.n = n; a.m = m; a.vocab = vocab;
    a.inv_temperature = greedy ? 1.f : 1.f / temperature;
    a.accepted = accepted; a.next = next;
    a.stats = reinterpret_cast<float2 *>(base + lay.stats);
    a.best = reinterpret_cast<uint64_t *>(base + lay.best);
    const hipError_t err = sqk::launch_verify(a, logits_dtype == SQ_F32, greedy, stream);
    return err == hipSuccess ? SQ_OK : hip_fail(err, "verify_draft launch");
}

sq_status sq_device_copy(const void *src, void *dst, size_t bytes, hipStream_t stream) {
    if (bytes == 0) return SQ_OK;
    if (!src || !dst) return fail(SQ_EINVAL, "src or dst is NULL");
    if (!aligned(src, 16) || !aligned(dst, 16)) return fail(SQ_EINVAL, "buffers are not 16-byte aligned");
    if (bytes % 16) return fail(SQ_EINVAL, "bytes (%zu) is not a multiple of 16", bytes);
    const hipError_t e = sqk::launch_stream_copy(src, dst, (uint64_t)(bytes / 16), stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "stream copy launch");
}

sq_status sq_issue_probe(int op, float *sink, hipStream_t stream) {
    if (op < 0 || op >= SQ_PROBE_COUNT) return fail(SQ_EINVAL, "op = %d is not a probe class", op);
    if (!sink) return fail(SQ_EINVAL, "sink is NULL");
    if (!aligned(sink, 4)) return fail(SQ_EINVAL, "sink is not 4-byte aligned");
    const hipError_t e = sqk::launch_issue_probe(op, sink, stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "issue probe launch");
}

sq_status sq_arith_selfcheck(uint64_t *counts, hipStream_t stream) {
    if (!counts) return fail(SQ_EINVAL, "counts is NULL");
    if (!aligned(counts, 8)) return fail(SQ_EINVAL, "counts is not 8-byte aligned");
    const hipError_t e =
        sqk::launch_arith_selfcheck(reinterpret_cast<unsigned long long *>(counts), stream);
    return e == hipSuccess ? SQ_OK : hip_fail(e, "arith_selfcheck launch");
}

} // extern "C"
