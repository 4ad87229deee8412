// C ABI of the operators around a recurrent layer (declared in include/sq.h): the short
// convolution, the selective scan, the norms.  Host side only, as sq_api.cpp.
#include "sq.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "sq_block.h"
#include "sq_check.h"
#include "sq_scan.h"

using sqk::aligned;
using sqk::check_sequences;
using sqk::check_slot_list;
using sqk::check_work;
using sqk::debug_slots;
using sqk::fail;
using sqk::hip_fail;

namespace {

constexpr int64_t kMaxTokens = 0x7FFFFFFFll - 65536;  // block numbers and ends of blocks stay in 32 bits
constexpr int64_t kMaxStride = 1 << 24;
constexpr int64_t kMaxThreads = 0xFFFFFFFFll;  // of a grid's axis

int size_of(sq_dtype t) { return t == SQ_F32 ? 4 : 2; }
bool is_type(sq_dtype t) { return t == SQ_F32 || t == SQ_BF16; }

// One argument: `rows` rows of `row` bytes, `stride` bytes apart.
struct Arg {
    const char *name;
    const void *p;
    bool need, written;
    int64_t rows, row, stride;
    uintptr_t align;
};
Arg dense(const char *name, const void *p, bool need, bool written, int64_t bytes, uintptr_t align) {
    return Arg{name, p, need, written, bytes > 0 ? 1 : 0, bytes, bytes, align};
}

bool overlap(const Arg &a, const Arg &b) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.row <= 0 || b.row <= 0) return false;
    const intptr_t x = reinterpret_cast<intptr_t>(a.p), y = reinterpret_cast<intptr_t>(b.p);
    if (x >= y + (b.rows - 1) * b.stride + b.row || y >= x + (a.rows - 1) * a.stride + a.row) return false;
    if (a.rows > 1 && b.rows > 1 && a.stride == b.stride) {  // parts of one wider tensor
        const int64_t d = ((y - x) % a.stride + a.stride) % a.stride;
        return !(d >= a.row && d + b.row <= a.stride);
    }
    return true;
}

// NULL, alignment, and outputs that share memory with anything else.  same: pairs of names that may be
// the very same tensor.
struct Same { const char *a, *b; };
template <int N, int M> sq_status check_args(const Arg (&args)[N], const Same (&same)[M]) {
    for (const Arg &a : args) {
        if (a.need && a.rows > 0 && !a.p) return fail(SQ_EINVAL, "%s is NULL", a.name);
        if (a.p && !aligned(a.p, a.align)) return fail(SQ_EINVAL, "%s is not %d-byte aligned", a.name, (int)a.align);
    }
    for (int i = 0; i < N; ++i)
        for (int j = i + 1; j < N; ++j) {
            if (!(args[i].written || args[j].written) || !overlap(args[i], args[j])) continue;
            bool fine = false;
            for (const Same &s : same)
                fine |= args[i].p == args[j].p && args[i].row == args[j].row && args[i].rows == args[j].rows && args[i].stride == args[j].stride &&
                        ((s.a == args[i].name && s.b == args[j].name) || (s.a == args[j].name && s.b == args[i].name));
            if (!fine) return fail(SQ_EINVAL, "%s and %s overlap", args[i].name, args[j].name);
        }
    return SQ_OK;
}
// Names of arguments that `Same` refers to: compared by address.
const char kS0[] = "S0", kS_out[] = "S_out", kdS0[] = "dS0", kdS_out[] = "dS_out", kx[] = "x", ky[] = "y", kdy[] = "dy", kdx[] = "dx";
const char kr[] = "r", kr_out[] = "r_out", kdr[] = "dr", kdr_out[] = "dr_out", kdh[] = "dh", kd_o[] = "d_o";
const Same kNone[1] = {{nullptr, nullptr}};

// A token stride: 0 for dense rows, else at least a row and a multiple of `per`.
sq_status check_stride(const char *name, int64_t stride, int64_t row, int64_t per) {
    if (stride != 0 && (stride < row || stride % per != 0 || stride > kMaxStride))
        return fail(SQ_EINVAL, "%s = %lld must be 0 or a multiple of %lld, at least %lld and at most 2^24", name, (long long)stride,
                    (long long)per, (long long)row);
    return SQ_OK;
}
int64_t stride_or(int64_t stride, int64_t row) { return stride ? stride : row; }

sq_status check_batch(int32_t n_seq, int64_t n_tokens) {
    if (n_seq < 0) return fail(SQ_EINVAL, "n_seq must be >= 0 (got %d)", n_seq);
    if (n_tokens < 0) return fail(SQ_EINVAL, "n_tokens must be >= 0 (got %lld)", (long long)n_tokens);
    if (n_tokens >= kMaxTokens) return fail(SQ_EUNSUPPORTED, "n_tokens exceeds 2^31 - 2^16");
    return SQ_OK;
}
// cu, which the kernels read all along.
Arg list_of(const int32_t *cu, int32_t n_seq) { return dense("cu", cu, true, false, 4 * ((int64_t)n_seq + 1), 4); }
sq_status check_step(const void *pool, int32_t n_slots, const int32_t *slot_idx, int32_t n) {
    if (n_slots < 1) return fail(SQ_EINVAL, "n_slots must be >= 1 (got %d)", n_slots);
    if (n < 0) return fail(SQ_EINVAL, "n must be >= 0 (got %d)", n);
    if (n == 0) return SQ_OK;
    if (!pool) return fail(SQ_EINVAL, "pool is NULL");
    if (!slot_idx) return fail(SQ_EINVAL, "slot_idx is NULL");
    if (!aligned(slot_idx, 4)) return fail(SQ_EINVAL, "slot_idx is not 4-byte aligned");
    return SQ_OK;
}

// ------------------------------------------------------------------ convolution
sq_status check_conv(const sq_conv_desc *d, bool batch) {
    if (!d) return fail(SQ_EINVAL, "desc is NULL");
    sq_status st;
    if (batch && (st = check_batch(d->n_seq, d->n_tokens))) return st;
    if (d->n_channels < 1 || d->n_channels > (1 << 23)) return fail(SQ_EINVAL, "n_channels = %d must be in [1, 2^23]", d->n_channels);
    if (d->width < 2 || d->width > 4) return fail(SQ_EUNSUPPORTED, "width must be 2, 3 or 4 (got %d)", d->width);
    if (d->act != SQ_ACT_NONE && d->act != SQ_ACT_SILU) return fail(SQ_EUNSUPPORTED, "act must be SQ_ACT_NONE or SQ_ACT_SILU (got %d)", (int)d->act);
    if (!is_type(d->dtype)) return fail(SQ_EINVAL, "dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)d->dtype);
    if (batch && sqk::block_slots(d->n_tokens, d->n_seq, 6) > kMaxThreads / 256) return fail(SQ_EUNSUPPORTED, "n_tokens / 64 + n_seq exceeds the grid limit");
    return check_stride("x_stride", d->x_stride, d->n_channels, 1);
}
sqk::ConvArgs conv_args(const sq_conv_desc *d, const int32_t *cu, const void *x, const float *weight, const float *bias) {
    sqk::ConvArgs a{};
    a.seqs = sqk::Ragged{cu, d->n_seq, (int32_t)d->n_tokens};
    a.x = x; a.weight = weight; a.bias = bias;
    a.x_stride = stride_or(d->x_stride, d->n_channels);
    a.channels = d->n_channels; a.width = d->width; a.silu = d->act == SQ_ACT_SILU;
    return a;
}
// Whether rows can be loaded 16 bytes at a time: all of them aligned, and whole vectors.
template <int N> bool vectors(sq_dtype t, int64_t row, int64_t stride, const void *const (&p)[N]) {
    const int64_t per = 16 / size_of(t);
    bool fine = row % 8 == 0 && stride % per == 0;
    for (const void *q : p) fine &= aligned(q, 16);
    return fine;
}

// ------------------------------------------------------------------ scan
sq_status check_scan(const sq_scan_desc *d, bool batch) {
    if (!d) return fail(SQ_EINVAL, "desc is NULL");
    sq_status st;
    if (batch && (st = check_batch(d->n_seq, d->n_tokens))) return st;
    if (d->n_heads < 1 || d->n_heads > 16384) return fail(SQ_EINVAL, "n_heads = %d must be in [1, 16384]", d->n_heads);
    if (d->n_groups < 1 || d->n_heads % d->n_groups != 0)
        return fail(SQ_EINVAL, "n_groups = %d is not a divisor of n_heads = %d", d->n_groups, d->n_heads);
    if (d->d_state != 64 && d->d_state != 128) return fail(SQ_EUNSUPPORTED, "d_state must be 64 or 128 (got %d)", d->d_state);
    if (d->d_head != 64 && d->d_head != 128) return fail(SQ_EUNSUPPORTED, "d_head must be 64 or 128 (got %d)", d->d_head);
    if (d->softplus != 0 && d->softplus != 1) return fail(SQ_EINVAL, "softplus must be 0 or 1 (got %d)", d->softplus);
    if (!is_type(d->in_dtype)) return fail(SQ_EINVAL, "in_dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)d->in_dtype);
    if (!is_type(d->y_dtype)) return fail(SQ_EINVAL, "y_dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)d->y_dtype);
    const int64_t per = 16 / size_of(d->in_dtype), wide = (int64_t)d->n_heads * d->d_head, keys = (int64_t)d->n_groups * d->d_state;
    if ((st = check_stride("x_stride", d->x_stride, wide, per)) || (st = check_stride("dt_stride", d->dt_stride, d->n_heads, 1)) ||
        (st = check_stride("b_stride", d->b_stride, keys, per)) || (st = check_stride("c_stride", d->c_stride, keys, per)) ||
        (st = check_stride("dx_stride", d->dx_stride, wide, per)) || (st = check_stride("ddt_stride", d->ddt_stride, d->n_heads, 1)) ||
        (st = check_stride("db_stride", d->db_stride, keys, per)) || (st = check_stride("dc_stride", d->dc_stride, keys, per)))
        return st;
    if (wide > kMaxStride || keys > kMaxStride) return fail(SQ_EUNSUPPORTED, "n_heads * d_head or n_groups * d_state exceeds 2^24");  // 32-bit offsets within a chunk
    if (batch) {
        const sqk::ScanPlan p = sqk::scan_plan(*d);
        if (p.seg_slots > kMaxThreads / 256 / ((p.parts + 7) / 8 * 8) || p.chunk_slots > kMaxThreads / 512 / ((int64_t)d->n_groups * p.subsets))
            return fail(SQ_EUNSUPPORTED, "n_tokens or n_seq times n_heads exceeds the grid limit");
    }
    return SQ_OK;
}
size_t scan_work(const sqk::ScanPlan &p, bool train) {
    return (size_t)(p.state_bytes + p.fade_bytes + (train ? p.save_bytes + p.group_bytes + p.dots_bytes + p.head_bytes : 0));
}
sqk::ScanArgs scan_args(const sq_scan_desc *d, const int32_t *cu, const void *x, const void *raw, const float *A, const void *B, const void *C,
                        const float *D, const float *bias, void *work) {
    sqk::ScanArgs a{};
    const int64_t wide = (int64_t)d->n_heads * d->d_head, keys = (int64_t)d->n_groups * d->d_state;
    a.seqs = sqk::Ragged{cu, d->n_seq, (int32_t)d->n_tokens};
    a.x = x; a.raw = raw; a.A = A; a.B = B; a.C = C; a.D = D; a.bias = bias;
    a.x_stride = stride_or(d->x_stride, wide); a.dt_stride = stride_or(d->dt_stride, d->n_heads);
    a.b_stride = stride_or(d->b_stride, keys); a.c_stride = stride_or(d->c_stride, keys);
    a.dx_stride = stride_or(d->dx_stride, wide); a.ddt_stride = stride_or(d->ddt_stride, d->n_heads);
    a.db_stride = stride_or(d->db_stride, keys); a.dc_stride = stride_or(d->dc_stride, keys);
    a.n_heads = d->n_heads; a.n_groups = d->n_groups; a.d_head = d->d_head; a.softplus = d->softplus;
    if (work) {
        const sqk::ScanPlan p = sqk::scan_plan(*d);
        uint8_t *base = static_cast<uint8_t *>(work);
        a.seg_shift = p.seg_shift;
        a.segments = d->n_tokens > ((int64_t)1 << p.seg_shift);
        a.seg_state = reinterpret_cast<float *>(base);
        a.seg_fade = reinterpret_cast<float *>(base += p.state_bytes);
        a.grad_save = base += p.fade_bytes;
        a.group_part = reinterpret_cast<float *>(base += p.save_bytes);
        a.dots = reinterpret_cast<float *>(base += p.group_bytes);
        a.head_part = reinterpret_cast<float *>(base += p.dots_bytes);
        a.chunk_parts = p.chunk_slots * p.parts;
        a.subsets = p.subsets;
    }
    return a;
}

// ------------------------------------------------------------------ norms
sq_status check_norm(int32_t d, float eps, sq_dtype t) {
    if (d < 1 || d > sqk::kNormMax) return fail(SQ_EUNSUPPORTED, "d must be in [1, %d] (got %d)", sqk::kNormMax, d);
    if (!(eps >= 0.f) || std::isinf(eps)) return fail(SQ_EINVAL, "eps = %g must be a finite number from 0 on", (double)eps);
    if (!is_type(t)) return fail(SQ_EINVAL, "dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)t);
    return SQ_OK;
}
sq_status check_gate(const sq_gated_norm_desc *d) {
    if (!d) return fail(SQ_EINVAL, "desc is NULL");
    sq_status st = check_norm(d->d, d->eps, d->dtype);
    if (st) return st;
    if (d->n_groups < 1 || d->n_groups > 65535) return fail(SQ_EINVAL, "n_groups = %d must be in [1, 65535]", d->n_groups);
    if (d->n_tokens < 0 || d->n_tokens > 0x7FFFFFFFll / d->n_groups) return fail(SQ_EINVAL, "n_tokens * n_groups must be in [0, 2^31)");
    if (d->act != SQ_ACT_NONE && d->act != SQ_ACT_SILU && d->act != SQ_ACT_SIGMOID) return fail(SQ_EINVAL, "act = %d is none of sq_act", (int)d->act);
    const int64_t wide = (int64_t)d->n_groups * d->d;
    if (wide > kMaxStride) return fail(SQ_EUNSUPPORTED, "n_groups * d exceeds 2^24");
    if ((st = check_stride("x_stride", d->x_stride, wide, 1)) || (st = check_stride("z_stride", d->z_stride, wide, 1)) ||
        (st = check_stride("dx_stride", d->dx_stride, wide, 1)) || (st = check_stride("dz_stride", d->dz_stride, wide, 1)))
        return st;
    return SQ_OK;
}
sqk::GateArgs gate_args(const sq_gated_norm_desc *d, const void *x, const void *z, const float *weight) {
    sqk::GateArgs a{};
    const int64_t wide = (int64_t)d->n_groups * d->d;
    a.x = x; a.z = d->act == SQ_ACT_NONE ? nullptr : z; a.weight = weight;
    a.n_tokens = d->n_tokens;
    a.x_stride = stride_or(d->x_stride, wide); a.z_stride = stride_or(d->z_stride, wide);
    a.dx_stride = stride_or(d->dx_stride, wide); a.dz_stride = stride_or(d->dz_stride, wide);
    a.groups = d->n_groups; a.d = d->d; a.act = d->act; a.eps = d->eps;
    return a;
}
int64_t gate_rows(const sq_gated_norm_desc *d) { return d->shared_weight ? d->n_tokens * d->n_groups : d->n_tokens; }
sq_status check_residual(const sq_residual_norm_desc *d) {
    if (!d) return fail(SQ_EINVAL, "desc is NULL");
    const sq_status st = check_norm(d->d, d->eps, d->dtype);
    if (st) return st;
    if (!is_type(d->res_dtype)) return fail(SQ_EINVAL, "res_dtype must be SQ_F32 or SQ_BF16 (got %d)", (int)d->res_dtype);
    if (d->n_rows < 0 || d->n_rows > 0x7FFFFFFFll) return fail(SQ_EINVAL, "n_rows must be in [0, 2^31)");
    return SQ_OK;
}

} // namespace

extern "C" {

sq_status sq_conv_bytes(const sq_conv_desc *desc, size_t *work) {
    sq_status st = check_conv(desc, true);
    if (st) return st;
    if (!work) return fail(SQ_EINVAL, "work is NULL");
    *work = (size_t)sqk::conv_partials(desc->n_tokens, desc->n_seq, desc->n_channels) * desc->n_channels * (desc->width + 1) * sizeof(float);
    return SQ_OK;
}

sq_status sq_conv_forward(const sq_conv_desc *desc, const int32_t *cu, const void *x, const float *weight, const float *bias,
                          const void *S0, void *y, void *S_out, hipStream_t stream) {
    sq_status st = check_conv(desc, true);
    if (st) return st;
    if (desc->n_seq == 0) return SQ_OK;
    const int e = size_of(desc->dtype);
    const int64_t c = desc->n_channels, n = desc->n_tokens, xs = stride_or(desc->x_stride, c), state = desc->n_seq * (int64_t)(desc->width - 1) * c * e;
    const Arg args[] = {list_of(cu, desc->n_seq), {kx, x, true, false, n, c * e, xs * e, (uintptr_t)e}, dense("weight", weight, true, false, c * desc->width * 4, 4),
                        dense("bias", bias, false, false, c * 4, 4), dense(kS0, S0, false, false, state, e),
                        dense(ky, y, true, true, n * c * e, e), dense(kS_out, S_out, false, true, state, e)};
    if ((st = check_args(args, kNone))) return st;
    if (debug_slots() && (st = check_sequences(desc->n_seq, desc->n_tokens, cu, stream))) return st;
    sqk::ConvArgs a = conv_args(desc, cu, x, weight, bias);
    a.S0 = S0; a.y = y; a.S_out = S_out;
    const void *const p[] = {x, S0, y, S_out, weight};
    const hipError_t err = sqk::launch_conv_forward(a, desc->dtype == SQ_F32, vectors(desc->dtype, c, xs, p), stream);
    return err == hipSuccess ? SQ_OK : hip_fail(err, "conv_forward launch");
}

sq_status sq_conv_backward(const sq_conv_desc *desc, const int32_t *cu, const void *x, const float *weight, const float *bias,
                           const void *S0, const void *dy, const void *dS_out, void *dx, float *dweight, float *dbias, void *dS0,
                           void *work, size_t work_bytes, hipStream_t stream) {
    size_t need = 0;
    sq_status st = sq_conv_bytes(desc, &need);
    if (st) return st;
    if (desc->n_seq == 0) {
        if (!aligned(dweight, 4) || !aligned(dbias, 4)) return fail(SQ_EINVAL, "dweight or dbias is not 4-byte aligned");
        sqk::ConvArgs a = conv_args(desc, nullptr, nullptr, nullptr, nullptr);
        a.dweight = dweight; a.dbias = dbias;
        const hipError_t err = sqk::launch_conv_sums(a, 0, stream);
        return err == hipSuccess ? SQ_OK : hip_fail(err, "conv_backward launch");
    }
    const int e = size_of(desc->dtype);
    const int64_t c = desc->n_channels, n = desc->n_tokens, xs = stride_or(desc->x_stride, c), state = desc->n_seq * (int64_t)(desc->width - 1) * c * e;
    const Arg args[] = {list_of(cu, desc->n_seq), {kx, x, true, false, n, c * e, xs * e, (uintptr_t)e}, dense("weight", weight, true, false, c * desc->width * 4, 4),
                        dense("bias", bias, false, false, c * 4, 4), dense(kS0, S0, false, false, state, e),
                        dense(kdy, dy, true, false, n * c * e, e), dense(kdS_out, dS_out, false, false, state, e),
                        dense(kdx, dx, true, true, n * c * e, e), dense("dweight", dweight, true, true, c * desc->width * 4, 4),
                        dense("dbias", dbias, false, true, c * 4, 4), dense(kdS0, dS0, false, true, state, e),
                        dense("work", work, false, true, (int64_t)need, 1)};
    if ((st = check_work("work", work, work_bytes, need)) || (st = check_args(args, kNone))) return st;
    if (debug_slots() && (st = check_sequences(desc->n_seq, desc->n_tokens, cu, stream))) return st;
    sqk::ConvArgs a = conv_args(desc, cu, x, weight, bias);
    a.S0 = S0; a.dy = dy; a.dS_out = dS_out; a.dx = dx; a.dweight = dweight; a.dbias = dbias; a.dS0 = dS0;
    a.partial = static_cast<float *>(work);
    const void *const p[] = {x, S0, dy, dS_out, dx, dS0, weight};
    const hipError_t err = sqk::launch_conv_backward(a, desc->dtype == SQ_F32, vectors(desc->dtype, c, xs, p), stream);
    return err == hipSuccess ? SQ_OK : hip_fail(err, "conv_backward launch");
}

sq_status sq_conv_step(const sq_conv_desc *desc, void *pool, int32_t n_slots, const int32_t *slot_idx, int32_t n, const void *x,
                       const float *weight, const float *bias, void *y, hipStream_t stream) {
    sq_status st = check_conv(desc, false);
    if (st || (st = check_step(pool, n_slots, slot_idx, n))) return st;
    if (n == 0) return SQ_OK;
    if (n > (1 << 27) - 8) return fail(SQ_EUNSUPPORTED, "n exceeds the grid limit");  // 8 requests to a workgroup where there are many
    const int e = size_of(desc->dtype);
    const int64_t c = desc->n_channels, xs = stride_or(desc->x_stride, c);
    const Arg args[] = {{kx, x, true, false, n, c * e, xs * e, (uintptr_t)e}, dense("weight", weight, true, false, c * desc->width * 4, 4),
                        dense("bias", bias, false, false, c * 4, 4), dense("pool", pool, true, true, (int64_t)n_slots * (desc->width - 1) * c * e, e),
                        dense(ky, y, true, true, n * c * e, e), dense("slot_idx", slot_idx, true, false, 4ll * n, 4)};
    if ((st = check_args(args, kNone))) return st;
    if (debug_slots() && (st = check_slot_list(slot_idx, n, n_slots, true, stream))) return st;
    sqk::ConvArgs a = conv_args(desc, nullptr, x, weight, bias);
    a.pool = pool; a.slot = slot_idx; a.n = n; a.n_slots = n_slots; a.y = y;
    const void *const p[] = {x, pool, y, weight};
    const hipError_t err = sqk::launch_conv_step(a, desc->dtype == SQ_F32, vectors(desc->dtype, c, xs, p), stream);
    return err == hipSuccess ? SQ_OK : hip_fail(err, "conv_step launch");
}

sq_status sq_scan_bytes(const sq_scan_desc *desc, size_t *work, size_t *save) {
    sq_status st = check_scan(desc, true);
    if (st) return st;
    if (!work) return fail(SQ_EINVAL, "work is NULL");
    const sqk::ScanPlan p = sqk::scan_plan(*desc);
    *work = scan_work(p, save != nullptr);
    if (save) *save = (size_t)p.save_bytes;
    return SQ_OK;
}

sq_status sq_scan_forward(const sq_scan_desc *desc, const int32_t *cu, const void *x, const void *raw, const float *A, const void *B,
                          const void *C, const float *D, const float *dt_bias, const float *S0, void *y, float *S_out, void *save,
                          size_t save_bytes, void *work, size_t work_bytes, hipStream_t stream) {
    size_t need = 0, both = 0, keep = 0;
    sq_status st = sq_scan_bytes(desc, &need, nullptr);
    if (st || (st = sq_scan_bytes(desc, &both, &keep))) return st;
    if (desc->n_seq == 0) return SQ_OK;
    const int e = size_of(desc->in_dtype), ey = size_of(desc->y_dtype);
    const int64_t n = desc->n_tokens, h = desc->n_heads, wide = h * desc->d_head, keys = (int64_t)desc->n_groups * desc->d_state;
    const int64_t state = desc->n_seq * h * desc->d_state * desc->d_head * 4;
    const Arg args[] = {list_of(cu, desc->n_seq), {kx, x, true, false, n, wide * e, stride_or(desc->x_stride, wide) * e, 16}, {"raw", raw, true, false, n, h * e, stride_or(desc->dt_stride, h) * e, (uintptr_t)e},
                        dense("A", A, true, false, h * 4, 4), {"B", B, true, false, n, keys * e, stride_or(desc->b_stride, keys) * e, 16},
                        {"C", C, true, false, n, keys * e, stride_or(desc->c_stride, keys) * e, 16}, dense("D", D, false, false, h * 4, 4),
                        dense("dt_bias", dt_bias, false, false, h * 4, 4), dense(kS0, S0, false, false, state, 16), dense(ky, y, true, true, n * wide * ey, 16),
                        dense(kS_out, S_out, false, true, state, 16), dense("save", save, false, true, (int64_t)keep, 1), dense("work", work, false, true, (int64_t)need, 1)};
    const Same same[] = {{kS0, kS_out}};
    if ((st = check_work("work", work, work_bytes, need)) || (save && (st = check_work("save", save, save_bytes, keep))) ||
        (st = check_args(args, same)))
        return st;
    if (debug_slots() && (st = check_sequences(desc->n_seq, desc->n_tokens, cu, stream))) return st;
    sqk::ScanArgs a = scan_args(desc, cu, x, raw, A, B, C, D, dt_bias, work);
    a.S0 = S0; a.y = y; a.S_out = S_out; a.save = static_cast<uint8_t *>(save);
    const hipError_t err = sqk::launch_scan_forward(a, desc->d_state, desc->in_dtype == SQ_F32, desc->y_dtype == SQ_F32, stream);
    return err == hipSuccess ? SQ_OK : hip_fail(err, "scan_forward launch");
}

sq_status sq_scan_backward(const sq_scan_desc *desc, const int32_t *cu, const void *x, const void *raw, const float *A, const void *B,
                           const void *C, const float *D, const float *dt_bias, const void *dy, const float *dS_out, const void *save,
                           size_t save_bytes, void *dx, void *draw, float *dA, void *dB, void *dC, float *dD, float *ddt_bias, float *dS0,
                           void *work, size_t work_bytes, hipStream_t stream) {
    size_t need = 0, keep = 0;
    sq_status st = sq_scan_bytes(desc, &need, &keep);
    if (st) return st;
    if (desc->n_seq == 0) {
        if (!aligned(dA, 4) || !aligned(dD, 4) || !aligned(ddt_bias, 4)) return fail(SQ_EINVAL, "dA, dD or ddt_bias is not 4-byte aligned");
        const int64_t h = desc->n_heads;
        const sqk::SumArgs s[3] = {{nullptr, dA, 0, h, h}, {nullptr, dD, 0, h, h}, {nullptr, ddt_bias, 0, h, h}};
        const hipError_t err = sqk::launch_column_sums(s, 3, stream);
        return err == hipSuccess ? SQ_OK : hip_fail(err, "scan_backward launch");
    }
    const int e = size_of(desc->in_dtype);
    const int64_t n = desc->n_tokens, h = desc->n_heads, wide = h * desc->d_head, keys = (int64_t)desc->n_groups * desc->d_state;
    const int64_t state = desc->n_seq * h * desc->d_state * desc->d_head * 4;
    const Arg args[] = {list_of(cu, desc->n_seq), {kx, x, true, false, n, wide * e, stride_or(desc->x_stride, wide) * e, 16}, {"raw", raw, true, false, n, h * e, stride_or(desc->dt_stride, h) * e, (uintptr_t)e},
                        dense("A", A, true, false, h * 4, 4), {"B", B, true, false, n, keys * e, stride_or(desc->b_stride, keys) * e, 16},
                        {"C", C, true, false, n, keys * e, stride_or(desc->c_stride, keys) * e, 16}, dense("D", D, false, false, h * 4, 4),
                        dense("dt_bias", dt_bias, false, false, h * 4, 4), dense(kdy, dy, true, false, n * wide * e, 16),
                        dense(kdS_out, dS_out, false, false, state, 16), dense("save", save, false, false, (int64_t)keep, 1),
                        {kdx, dx, true, true, n, wide * e, stride_or(desc->dx_stride, wide) * e, 16},
                        {"draw", draw, true, true, n, h * e, stride_or(desc->ddt_stride, h) * e, (uintptr_t)e}, dense("dA", dA, true, true, h * 4, 4),
                        {"dB", dB, true, true, n, keys * e, stride_or(desc->db_stride, keys) * e, 16}, {"dC", dC, true, true, n, keys * e, stride_or(desc->dc_stride, keys) * e, 16},
                        dense("dD", dD, false, true, h * 4, 4), dense("ddt_bias", ddt_bias, false, true, h * 4, 4), dense(kdS0, dS0, false, true, state, 16),
                        dense("work", work, false, true, (int64_t)need, 1)};
    const Same same[] = {{kdS0, kdS_out}};
    if ((st = check_work("work", work, work_bytes, need)) || (st = check_work("save", save, save_bytes, keep)) ||
        (st = check_args(args, same)))
        return st;
    if (debug_slots() && (st = check_sequences(desc->n_seq, desc->n_tokens, cu, stream))) return st;
    sqk::ScanArgs a = scan_args(desc, cu, x, raw, A, B, C, D, dt_bias, work);
    a.save = static_cast<uint8_t *>(const_cast<void *>(save));
    a.dy = dy; a.dS_out = dS_out; a.dx = dx; a.draw = draw; a.dA = dA; a.dB = dB; a.dC = dC; a.dD = dD; a.dbias = ddt_bias; a.dS0 = dS0;
    const hipError_t err = sqk::launch_scan_backward(a, desc->d_state, desc->in_dtype == SQ_F32, stream);
    return err == hipSuccess ? SQ_OK : hip_fail(err, "scan_backward launch");
}

sq_status sq_scan_step(const sq_scan_desc *desc, float *state_pool, int32_t n_slots, const int32_t *slot_idx, int32_t n, const void *x,
                       const void *raw, const float *A, const void *B, const void *C, const float *D, const float *dt_bias, void *y,
                       hipStream_t stream) {
    sq_status st = check_scan(desc, false);
    if (st || (st = check_step(state_pool, n_slots, slot_idx, n))) return st;
    if (n == 0) return SQ_OK;
    const int e = size_of(desc->in_dtype), ey = size_of(desc->y_dtype);
    const int64_t h = desc->n_heads, wide = h * desc->d_head, keys = (int64_t)desc->n_groups * desc->d_state;
    if (n * h > kMaxThreads / 256) return fail(SQ_EUNSUPPORTED, "n * n_heads exceeds the grid limit");
    const Arg args[] = {{kx, x, true, false, n, wide * e, stride_or(desc->x_stride, wide) * e, 16}, {"raw", raw, true, false, n, h * e, stride_or(desc->dt_stride, h) * e, (uintptr_t)e},
                        dense("A", A, true, false, h * 4, 4), {"B", B, true, false, n, keys * e, stride_or(desc->b_stride, keys) * e, 16},
                        {"C", C, true, false, n, keys * e, stride_or(desc->c_stride, keys) * e, 16}, dense("D", D, false, false, h * 4, 4),
                        dense("dt_bias", dt_bias, false, false, h * 4, 4), dense(ky, y, true, true, n * wide * ey, 16),
                        dense("state_pool", state_pool, true, true, n_slots * h * desc->d_state * desc->d_head * 4, 16),
                        dense("slot_idx", slot_idx, true, false, 4ll * n, 4)};
    if ((st = check_args(args, kNone))) return st;
    if (debug_slots() && (st = check_slot_list(slot_idx, n, n_slots, true, stream))) return st;
    sqk::ScanArgs a = scan_args(desc, nullptr, x, raw, A, B, C, D, dt_bias, nullptr);
    a.pool = state_pool; a.slot = slot_idx; a.n = n; a.n_slots = n_slots; a.y = y;
    const hipError_t err = sqk::launch_scan_step(a, desc->d_state, desc->in_dtype == SQ_F32, desc->y_dtype == SQ_F32, stream);
    return err == hipSuccess ? SQ_OK : hip_fail(err, "scan_step launch");
}

sq_status sq_gated_norm_bytes(const sq_gated_norm_desc *desc, size_t *work) {
    sq_status st = check_gate(desc);
    if (st) return st;
    if (!work) return fail(SQ_EINVAL, "work is NULL");
    *work = (size_t)sqk::norm_blocks(gate_rows(desc), desc->d, desc->shared_weight ? 1 : desc->n_groups) * (desc->shared_weight ? 1 : desc->n_groups) * desc->d * sizeof(float);
    return SQ_OK;
}

sq_status sq_gated_norm_forward(const sq_gated_norm_desc *desc, const void *x, const void *z, const float *weight, void *y, hipStream_t stream) {
    sq_status st = check_gate(desc);
    if (st) return st;
    if (desc->n_tokens == 0) return SQ_OK;
    const int e = size_of(desc->dtype);
    const int64_t n = desc->n_tokens, wide = (int64_t)desc->n_groups * desc->d, xs = stride_or(desc->x_stride, wide), zs = stride_or(desc->z_stride, wide);
    const bool gate = desc->act != SQ_ACT_NONE;
    if (!gate && z) return fail(SQ_EINVAL, "z is given, but act is SQ_ACT_NONE");
    const Arg args[] = {{kx, x, true, false, n, wide * e, xs * e, (uintptr_t)e}, {"z", z, gate, false, n, wide * e, zs * e, (uintptr_t)e},
                        dense("weight", weight, false, false, (desc->shared_weight ? desc->d : wide) * 4, 4), {ky, y, true, true, n, wide * e, wide * e, (uintptr_t)e}};
    const Same same[] = {{kx, ky}};
    if ((st = check_args(args, same))) return st;
    sqk::GateArgs a = gate_args(desc, x, z, weight);
    a.y = y;
    const void *const p[] = {x, z, y, weight};
    const bool vec = vectors(desc->dtype, desc->d, xs, p) && (zs * e) % 16 == 0;
    const hipError_t err = sqk::launch_gate_forward(a, desc->dtype == SQ_F32, vec, desc->gate_first && gate, desc->shared_weight, stream);
    return err == hipSuccess ? SQ_OK : hip_fail(err, "gated_norm_forward launch");
}

sq_status sq_gated_norm_backward(const sq_gated_norm_desc *desc, const void *x, const void *z, const float *weight, const void *dy, void *dx,
                                 void *dz, float *dweight, void *work, size_t work_bytes, hipStream_t stream) {
    size_t need = 0;
    sq_status st = sq_gated_norm_bytes(desc, &need);
    if (st) return st;
    const int e = size_of(desc->dtype);
    const int64_t n = desc->n_tokens, wide = (int64_t)desc->n_groups * desc->d, xs = stride_or(desc->x_stride, wide), zs = stride_or(desc->z_stride, wide);
    const int64_t dxs = stride_or(desc->dx_stride, wide), dzs = stride_or(desc->dz_stride, wide);
    const bool gate = desc->act != SQ_ACT_NONE;
    if (!gate && (z || dz)) return fail(SQ_EINVAL, "z or dz is given, but act is SQ_ACT_NONE");
    const Arg args[] = {{kx, x, true, false, n, wide * e, xs * e, (uintptr_t)e}, {"z", z, gate, false, n, wide * e, zs * e, (uintptr_t)e},
                        dense("weight", weight, false, false, (desc->shared_weight ? desc->d : wide) * 4, 4), {kdy, dy, true, false, n, wide * e, wide * e, (uintptr_t)e},
                        {kdx, dx, true, true, n, wide * e, dxs * e, (uintptr_t)e}, {"dz", dz, gate, true, n, wide * e, dzs * e, (uintptr_t)e},
                        dense("dweight", dweight, false, true, (desc->shared_weight ? desc->d : wide) * 4, 4), dense("work", dweight ? work : nullptr, false, true, (int64_t)need, 1)};
    const Same same[] = {{kdy, kdx}};
    if ((dweight && (st = check_work("work", work, work_bytes, need))) || (st = check_args(args, same))) return st;
    sqk::GateArgs a = gate_args(desc, x, z, weight);
    a.dy = dy; a.dx = dx; a.dz = dz; a.dweight = dweight; a.partial = static_cast<float *>(work);
    const void *const p[] = {x, z, dy, dx, dz, weight};
    const bool vec = vectors(desc->dtype, desc->d, xs, p) && (zs * e) % 16 == 0 && (dxs * e) % 16 == 0 && (dzs * e) % 16 == 0;
    const hipError_t err = sqk::launch_gate_backward(a, desc->dtype == SQ_F32, vec, desc->gate_first && gate, desc->shared_weight, stream);
    return err == hipSuccess ? SQ_OK : hip_fail(err, "gated_norm_backward launch");
}

sq_status sq_residual_norm_bytes(const sq_residual_norm_desc *desc, size_t *work) {
    sq_status st = check_residual(desc);
    if (st) return st;
    if (!work) return fail(SQ_EINVAL, "work is NULL");
    *work = (size_t)sqk::norm_blocks(desc->n_rows, desc->d, 1) * 3 * desc->d * sizeof(float);
    return SQ_OK;
}

sq_status sq_residual_norm_forward(const sq_residual_norm_desc *desc, const void *o, const void *r, const float *post_weight,
                                   const float *scale, const float *weight, void *r_out, void *h, hipStream_t stream) {
    sq_status st = check_residual(desc);
    if (st) return st;
    if (desc->n_rows == 0) return SQ_OK;
    const int e = size_of(desc->dtype), er = size_of(desc->res_dtype);
    const int64_t n = desc->n_rows, d = desc->d;
    const Arg args[] = {dense("o", o, true, false, n * d * e, e), dense(kr, r, false, false, n * d * er, er),
                        dense("post_weight", post_weight, false, false, d * 4, 4), dense("scale", scale, false, false, d * 4, 4),
                        dense("weight", weight, false, false, d * 4, 4), dense(kr_out, r_out, true, true, n * d * er, er),
                        dense("h", h, false, true, n * d * e, e)};
    const Same same[] = {{kr, kr_out}};
    if ((st = check_args(args, same))) return st;
    sqk::ResidualArgs a{};
    a.o = o; a.r = r; a.post = post_weight; a.scale = scale; a.weight = weight; a.r_out = r_out; a.h = h;
    a.n_rows = n; a.d = desc->d; a.eps = desc->eps;
    const void *const p[] = {o, r, r_out, h, post_weight, scale, weight};
    const hipError_t err = sqk::launch_residual_forward(a, desc->dtype == SQ_F32, desc->res_dtype == SQ_F32, vectors(desc->dtype, d, 0, p), stream);
    return err == hipSuccess ? SQ_OK : hip_fail(err, "residual_norm_forward launch");
}

sq_status sq_residual_norm_backward(const sq_residual_norm_desc *desc, const void *o, const void *r, const float *post_weight,
                                    const float *scale, const float *weight, const void *dh, const void *dr_out, void *d_o, void *dr,
                                    float *dpost_weight, float *dscale, float *dweight, void *work, size_t work_bytes, hipStream_t stream) {
    size_t need = 0;
    sq_status st = sq_residual_norm_bytes(desc, &need);
    if (st) return st;
    if (dpost_weight && !post_weight) return fail(SQ_EINVAL, "dpost_weight is given, but post_weight is NULL");
    const bool sums = dpost_weight || dscale || dweight;  // over the rows, in the workspace
    const int e = size_of(desc->dtype), er = size_of(desc->res_dtype);
    const int64_t n = desc->n_rows, d = desc->d;
    const Arg args[] = {dense("o", o, true, false, n * d * e, e), dense(kr, r, false, false, n * d * er, er),
                        dense("post_weight", post_weight, false, false, d * 4, 4), dense("scale", scale, false, false, d * 4, 4),
                        dense("weight", weight, false, false, d * 4, 4), dense(kdh, dh, false, false, n * d * e, e),
                        dense(kdr_out, dr_out, false, false, n * d * er, er), dense(kd_o, d_o, true, true, n * d * e, e),
                        dense(kdr, dr, false, true, n * d * er, er), dense("dpost_weight", dpost_weight, false, true, d * 4, 4),
                        dense("dscale", dscale, false, true, d * 4, 4), dense("dweight", dweight, false, true, d * 4, 4),
                        dense("work", sums ? work : nullptr, false, true, (int64_t)need, 1)};
    const Same same[] = {{kdr, kdr_out}, {kdh, kd_o}};
    if ((sums && (st = check_work("work", work, work_bytes, need))) || (st = check_args(args, same))) return st;
    sqk::ResidualArgs a{};
    a.o = o; a.r = r; a.post = post_weight; a.scale = scale; a.weight = weight; a.dh = dh; a.dr_out = dr_out;
    a.d_o = d_o; a.dr = dr; a.dpost = dpost_weight; a.dscale = dscale; a.dweight = dweight; a.partial = static_cast<float *>(work);
    a.n_rows = n; a.d = desc->d; a.eps = desc->eps;
    const void *const p[] = {o, r, dh, dr_out, d_o, dr, post_weight, scale, weight};
    const hipError_t err = sqk::launch_residual_backward(a, desc->dtype == SQ_F32, desc->res_dtype == SQ_F32, vectors(desc->dtype, d, 0, p), stream);
    return err == hipSuccess ? SQ_OK : hip_fail(err, "residual_norm_backward launch");
}

} // extern "C"
