// Shared by the kernels around a recurrent layer (sq_conv.hip, sq_norm.hip, sq_scan.hip):
// their arguments, ragged batches cut into blocks of tokens, vectors of 8 elements, and the
// activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sq.h"
#include "sq_seq.h"

namespace sqk {

// ------------------------------------------------------------------ ragged batches
// Sequence s owns the block slots from cu[s] >> shift + s: one at least, enough for its
// tokens, and none of another sequence, without a prefix sum over lengths on the host.
struct Ragged {
    const int32_t *cu;  // [n_seq + 1]
    int32_t n_seq, n_tokens;
};
struct Block {
    int32_t seq;   // negative: an idle slot
    int32_t t0;    // first token of the sequence
    int32_t len;   // tokens of the sequence
    int32_t c;     // the block's number in it
};
inline int64_t block_slots(int64_t n_tokens, int32_t n_seq, int shift) { return (n_tokens >> shift) + n_seq; }

// Offsets are held inside the tokens, so that a wrong list cannot make a kernel leave its buffers.
__device__ __forceinline__ void ragged_span(const Ragged &a, int32_t s, int32_t &lo, int32_t &len) {
    const int32_t n = a.n_tokens;
    int32_t hi = a.cu[s + 1];
    lo = a.cu[s];
    lo = lo < 0 ? 0 : lo > n ? n : lo;
    hi = hi < lo ? lo : hi > n ? n : hi;
    len = hi - lo;
}

// The block on slot x, for a whole wave: its lanes probe 64 sequences at a time.  The first
// block of a sequence without tokens is no idle slot: its state is still handed on.
__device__ __forceinline__ Block block_at(const Ragged &a, int64_t x, int shift) {
    const int l = threadIdx.x & 63;
    int32_t lo = 0, n = a.n_seq, t0, len;
    while (n > 64) {  // the last probed s whose first slot is not behind x
        const int32_t step = (n + 63) >> 6, s = lo + l * step;
        ragged_span(a, min(s, a.n_seq - 1), t0, len);
        const bool before = l * step < n && (int64_t)(t0 >> shift) + s <= x;
        const int k = max(__popcll(__ballot(before)) - 1, 0);
        lo += k * step;
        n = min(step, n - k * step);
    }
    ragged_span(a, min(lo + l, a.n_seq - 1), t0, len);
    const int k = max(__popcll(__ballot(l < n && (int64_t)(t0 >> shift) + lo + l <= x)) - 1, 0);
    Block b;
    b.t0 = __builtin_amdgcn_readlane(t0, k);
    b.len = __builtin_amdgcn_readlane(len, k);
    const int64_t c = x - ((int64_t)(b.t0 >> shift) + lo + k);
    const bool live = c == 0 || (c > 0 && (c << shift) < b.len);
    b.seq = live ? lo + k : -1;
    b.c = live ? (int32_t)c : 0;
    return b;
}

// ------------------------------------------------------------------ vectors of elements
// What N elements (4 or 8) are loaded as.
template <bool F32, int N> struct Raw { uint32_t v[N * (F32 ? 4 : 2) / 4]; };
template <bool F32> using Raw8 = Raw<F32, 8>;

// Elements i .. i + N - 1 of p.  VEC: 16-byte loads (8 bytes for 4 of bf16; aligned, all inside); otherwise element by
// element, those from `left` on as zeros.
template <bool F32, bool VEC, int N> __device__ __forceinline__ Raw<F32, N> load_n(const void *p, int64_t i, int left) {
    Raw<F32, N> r;
    constexpr int WORDS = sizeof(r.v) / 4;
    if constexpr (VEC) {
        const Elem<F32> *q = static_cast<const Elem<F32> *>(p) + i;
        if constexpr (WORDS == 2) {
            *reinterpret_cast<uint2 *>(r.v) = *reinterpret_cast<const uint2 *>(q);
        } else {
#pragma unroll
            for (int k = 0; k < WORDS; k += 4) *reinterpret_cast<uint4 *>(r.v + k) = reinterpret_cast<const uint4 *>(q)[k / 4];
        }
    } else {
        uint32_t x[N];
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = e < left ? ld_raw<F32>(p, i + e) : 0u;
#pragma unroll
        for (int k = 0; k < WORDS; ++k) r.v[k] = F32 ? x[k] : x[2 * k] | x[2 * k + 1] << 16;
    }
    return r;
}
template <bool F32, int N> __device__ __forceinline__ void widen_n(const Raw<F32, N> &r, float (&x)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = __uint_as_float(F32 ? r.v[e] : e & 1 ? r.v[e / 2] & 0xffff0000u : r.v[e / 2] << 16);
}
template <bool F32, bool VEC, int N> __device__ __forceinline__ void store_n(void *p, int64_t i, const float (&x)[N], int left) {
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            const f4 v{x[k], x[k + 1], x[k + 2], x[k + 3]};
            if constexpr (F32 || N == 4) st_elem4<F32>(p, i + k, v);
        }
        if constexpr (!F32 && N == 8) *reinterpret_cast<bf8 *>(static_cast<__bf16 *>(p) + i) = make_frag<false, 1>(x).t[0];
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < left) st_elem<F32>(p, i + e, x[e]);
    }
}
template <bool F32, bool VEC> __device__ __forceinline__ Raw8<F32> load8(const void *p, int64_t i, int left) { return load_n<F32, VEC, 8>(p, i, left); }
template <bool F32> __device__ __forceinline__ void widen8(const Raw8<F32> &r, float (&x)[8]) { widen_n<F32, 8>(r, x); }
template <bool F32, bool VEC> __device__ __forceinline__ void store8(void *p, int64_t i, const float (&x)[8], int left) { store_n<F32, VEC, 8>(p, i, x, left); }

// ------------------------------------------------------------------ sums over lanes
// Sums over 16 neighbouring lanes, to all of them, by rotations within the row; and over all 64.
template <int N> __device__ __forceinline__ float rotated(float x) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), 0x120 + N, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_sum(float x) {
    x += rotated<8>(x);
    x += rotated<4>(x);
    x += rotated<2>(x);
    return x + rotated<1>(x);
}
// ... over lanes 16 apart
__device__ __forceinline__ float rows_sum(float x) {
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}

// ------------------------------------------------------------------ activations
// e^-z by the hardware's exponential, for results of type F32 or bf16.  Its argument t is rounded, which is |z| 2^-24 of the
// result.  For fp32, what -z is beyond t ln 2 is put back (ln 2's own rounding, |z| 2^-28, stays), but where 2^t leaves
// fp32's range, so that infinities give 0 and infinity.  For bf16, 2^-17 at most next to its 2^-9, it stays (convolution in
// training, 8192 x 8192, 171 us, with it 176).
template <bool F32> __device__ __forceinline__ float exp_neg(float z) {
    const float t = -1.44269504088896340736f * z, r = __builtin_amdgcn_exp2f(t);
    if (!F32) return r;
    const float e = fmaf(r, fmaf(t, -0.69314718055994530942f, -z), r);
    return fabsf(t) < 126.f ? e : r;
}
// 1 / (1 + e^-z) to 2^-21 (bf16: 2^-17) of itself from z = -87 on (below that, less than 2^-125, it may be 0); a NaN stays one.
template <bool F32> __device__ __forceinline__ float sigmoid_of(float z) { return __builtin_amdgcn_rcpf(1.f + exp_neg<F32>(z)); }
// act(z) and its derivative; none: 1 and 0 (no gate).
template <bool F32> __device__ __forceinline__ float gate_of(int act, float z) {
    const float s = sigmoid_of<F32>(z);
    return act == SQ_ACT_SILU ? z * s : s;
}
template <bool F32> __device__ __forceinline__ void gate_and_slope(int act, float z, float &value, float &slope) {
    const float e = exp_neg<F32>(z), s = __builtin_amdgcn_rcpf(1.f + e);
    // 1 - sigma = e^-z sigma: as a difference it would have few bits where sigma is near 1.  Where e^-z is infinite sigma is 0,
    // and so is the slope
    const float rest = fminf(e, 3e38f) * s;
    value = act == SQ_ACT_SILU ? z * s : s;
    slope = act == SQ_ACT_SILU ? fmaf(value, rest, s) : s * rest;
}

// ------------------------------------------------------------------ arguments
struct ConvArgs {
    Ragged seqs;
    const void *x, *S0, *dy, *dS_out;
    const float *weight, *bias;
    void *y, *S_out, *dx, *dS0;
    float *dweight, *dbias, *partial;
    int64_t x_stride;
    int32_t channels, width, silu;
    // step
    void *pool;
    const int32_t *slot;
    int32_t n, n_slots;
};
// Most workgroups along the tokens of the backward pass of a batch of up to these sizes: each leaves its sums over tokens in
// `partial`.
int64_t conv_partials(int64_t n_tokens, int32_t n_seq, int32_t channels);
hipError_t launch_conv_forward(const ConvArgs &a, bool f32, bool vec, hipStream_t stream);
hipError_t launch_conv_backward(const ConvArgs &a, bool f32, bool vec, hipStream_t stream);
hipError_t launch_conv_sums(const ConvArgs &a, int blocks, hipStream_t stream);  // blocks 0: zeros
hipError_t launch_conv_step(const ConvArgs &a, bool f32, bool vec, hipStream_t stream);

struct GateArgs {
    const void *x, *z, *dy;
    const float *weight;
    void *y, *dx, *dz;
    float *dweight, *partial;
    int64_t n_tokens, x_stride, z_stride, dx_stride, dz_stride;
    int32_t groups, d, act;
    float eps;
};
struct ResidualArgs {
    const void *o, *r, *dh, *dr_out;
    const float *post, *scale, *weight;
    void *r_out, *h, *d_o, *dr;
    float *dpost, *dscale, *dweight, *partial;
    int64_t n_rows;
    int32_t d;
    float eps;
};
constexpr int kNormMax = 16384;  // longest row: 1024 threads of 16 elements
// Workgroups of a backward pass along the rows (512 in all groups that have weights of their own): each leaves its sums
// over rows in `partial`.
int norm_blocks(int64_t rows, int32_t d, int32_t groups);
hipError_t launch_gate_forward(const GateArgs &a, bool f32, bool vec, bool first, bool shared, hipStream_t stream);
hipError_t launch_gate_backward(const GateArgs &a, bool f32, bool vec, bool first, bool shared, hipStream_t stream);
hipError_t launch_residual_forward(const ResidualArgs &a, bool f32, bool res_f32, bool vec, hipStream_t stream);
hipError_t launch_residual_backward(const ResidualArgs &a, bool f32, bool res_f32, bool vec, hipStream_t stream);

// out[j] = sum over i of part[i][j], in a fixed order: the second half of every gradient that is a sum
// over tokens.
struct SumArgs {
    const float *part;
    float *out;
    int64_t rows, cols, row_stride;
};
hipError_t launch_column_sums(const SumArgs *a, int count, hipStream_t stream);

} // namespace sqk
