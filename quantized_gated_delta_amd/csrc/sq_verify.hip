// Drafted tokens against the target's probabilities, with given random numbers.
//
// For request b with drafted tokens x_0 .. x_{len-1}, target logits in len + 1 rows
// and draft logits in len rows, p = softmax(target / T), q = softmax(draft / T):
//   token i stands if all before it do and u_i q_i(x_i) < p_i(x_i);
//   the token after the accepted a is the argmax over v of r(v) / e(v), with
//   r = max(p_a - q_a, 0) where one was rejected (a < len), p_len otherwise.
// With u uniform and e exponential this draws from p exactly, and needs no sum
// over r: the argmax of r / e is a draw from r's normalisation.  Without draft
// logits q_i is 1 at x_i: the draft was certain.  T = 0: the argmax of the target decides
// both.  Ties go to the lower token.
//
// Bound by reading each logit once: kernel 1 takes every row's maximum and sum in one
// pass (running maximum, sum rescaled when it grows), a row split over
// several workgroups where there are few rows.  Kernel 2 joins the parts,
// decides, and reads the one row that the next token is drawn from.  Where
// several workgroups share it, kernel 3 takes the best of their parts: the end
// of a kernel orders their writes before its reads on every XCD (instead, an atomic
// maximum that the last workgroup by a counter read: 24 us for kernel 2 with 64
// requests of 131072 tokens, where kernels 2 and 3 take 17 + 4).
//
// Measured: 64 requests of 4 drafted tokens, 131072 logits each, bf16, with draft logits
// 27 + 17 + 4 us (kernel 1 at 5.5 TB/s, 2 at 4.0); 256 requests, 50001 logits, fp32, 28 + 20 + 5 us;
// one greedy request, 32000 logits, 4 + 3 us, less than the host takes to ask for it.
#include <float.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sq_verify.h"

namespace sqk {
namespace {

// Eight consecutive logits of a row whose start may have any alignment; NaN
// counts as minus infinity, plus infinity as the largest finite value.
template <bool F32> __device__ __forceinline__ void load8(const void *base, int64_t at, float (&x)[8]) {
    if constexpr (F32) {
        typedef float v4 __attribute__((ext_vector_type(4), aligned(4)));
        const float *p = static_cast<const float *>(base) + at;
        const v4 a = *reinterpret_cast<const v4 *>(p), b = *reinterpret_cast<const v4 *>(p + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < 4 ? a[i] : b[i - 4];
    } else {
        typedef __bf16 v8 __attribute__((ext_vector_type(8), aligned(2)));
        const v8 a = *reinterpret_cast<const v8 *>(static_cast<const __bf16 *>(base) + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)a[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -INFINITY), FLT_MAX);
}
template <bool F32> __device__ __forceinline__ float load1(const void *base, int64_t at) {
    float x;
    if constexpr (F32) x = static_cast<const float *>(base)[at];
    else x = (float)static_cast<const __bf16 *>(base)[at];
    return fminf(fmaxf(x, -INFINITY), FLT_MAX);
}

// e^{(x - m) / T}, c = log2(e) / T; a row without any finite logit has m = -inf and no probabilities.
__device__ __forceinline__ float weight(float x, float m, float c) { return m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((x - m) * c); }

// (maximum, sum) of two parts of a row.
__device__ __forceinline__ float2 join(float2 a, float2 b, float c) {
    const float m = fmaxf(a.x, b.x);
    return make_float2(m, a.y * weight(a.x, m, c) + b.y * weight(b.x, m, c));
}
// The better of two (score, token) pairs: the higher score, then the lower token.
__device__ __forceinline__ float2 better(float2 a, float2 b) {
    const int i = __float_as_int(a.y), j = __float_as_int(b.y);
    return b.x > a.x || (b.x == a.x && j < i) ? b : a;
}
__device__ __forceinline__ float2 shfl_xor2(float2 v, int off) { return make_float2(__shfl_xor(v.x, off), __shfl_xor(v.y, off)); }

constexpr int kNone = 0x7fffffff;  // no token
__device__ __forceinline__ float2 no_token() { return make_float2(-INFINITY, __int_as_float(kNone)); }

template <bool GREEDY> __device__ __forceinline__ float2 merge(float2 a, float2 b, float c) { return GREEDY ? better(a, b) : join(a, b, c); }

// Over the 256 threads; the result in thread 0.
template <bool GREEDY> __device__ __forceinline__ float2 reduce(float2 v, float c, float2 *s, int t) {
#pragma unroll
    for (int off = 32; off; off >>= 1) v = merge<GREEDY>(v, shfl_xor2(v, off), c);
    if ((t & 63) == 0) s[t >> 6] = v;
    __syncthreads();
    if (t == 0) v = merge<GREEDY>(merge<GREEDY>(s[0], s[1], c), merge<GREEDY>(s[2], s[3], c), c);
    return v;
}

// The part of `vocab` that workgroup `part` of `parts` takes, in multiples of 8.
__device__ __forceinline__ void segment(int vocab, int part, int parts, int &lo, int &hi) {
    const int each = ((vocab + 7) / 8 + parts - 1) / parts * 8;
    lo = min(vocab, part * each);
    hi = min(vocab, lo + each);
}

__device__ __forceinline__ int length_of(const VerifyArgs &a, int b) { return a.lens ? min(max(a.lens[b], 0), a.m) : a.m; }

template <bool F32, bool GREEDY> __global__ __launch_bounds__(256) void stats_kernel(VerifyArgs a) {
    __shared__ float2 s[4];
    const int t = threadIdx.x, part = blockIdx.x;
    const int64_t row = blockIdx.y, targets = (int64_t)a.n * (a.m + 1);
    const bool is_draft = row >= targets;
    const int b = is_draft ? (int)((row - targets) / a.m) : (int)(row / (a.m + 1));
    const int i = is_draft ? (int)((row - targets) % a.m) : (int)(row % (a.m + 1));
    const int len = length_of(a, b);
    if (is_draft ? i >= len : i > len) return;  // a row that nothing is decided by
    const void *base = is_draft ? a.draft : a.target;
    const int64_t at = is_draft ? (row - targets) * a.draft_stride : row * a.target_stride;
    const float c = a.inv_temperature * kLog2e;
    int lo, hi;
    segment(a.vocab, part, a.splits, lo, hi);
    float2 best = GREEDY ? no_token() : make_float2(-INFINITY, 0.f);
    constexpr int U = 4;
    int v = lo + 8 * t;
    for (; v + (U - 1) * 2048 + 8 <= hi; v += U * 2048) {
        float x[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) load8<F32>(base, at + v + u * 2048, x[u]);
        float m = x[0][0];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, x[u][j]);
        if constexpr (GREEDY) {
            if (m > best.x) {
                best.x = m;
#pragma unroll
                for (int u = U - 1; u >= 0; --u)
#pragma unroll
                    for (int j = 7; j >= 0; --j)
                        if (x[u][j] == m) best.y = __int_as_float(v + u * 2048 + j);
            }
        } else if (fmaxf(m, best.x) > -INFINITY) {
            if (m > best.x) best = make_float2(m, best.y * weight(best.x, m, c));
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += __builtin_amdgcn_exp2f((x[u][j] - best.x) * c);
            best.y += sum;
        }
    }
    for (; v < hi; v += 2048) {
        float x[8];
        if (v + 8 <= hi) {
            load8<F32>(base, at + v, x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = v + j < hi ? load1<F32>(base, at + v + j) : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (GREEDY) {
                if (x[j] > best.x) best = make_float2(x[j], __int_as_float(v + j));
            } else if (x[j] > -INFINITY) {
                best = join(best, make_float2(x[j], 1.f), c);
            }
        }
    }
    best = reduce<GREEDY>(best, c, s, t);
    if (t == 0) a.stats[row * a.splits + part] = best;
}

// How many of request b's tokens stand, by the whole workgroup.
struct DecideLds {
    float2 target[SQ_DRAFT_MAX + 1], draft[SQ_DRAFT_MAX];  // maximum and sum (greedy: token) of each row
    uint64_t best[4];
    int ok[SQ_DRAFT_MAX];
};
template <bool F32, bool GREEDY> __device__ __forceinline__ int decide(const VerifyArgs &a, int b, DecideLds &s, int t) {
    const int w = t >> 6, l = t & 63, len = length_of(a, b);
    const float c = a.inv_temperature * kLog2e;
    const int64_t targets = (int64_t)a.n * (a.m + 1);
    // a row's parts, one wave per row
    for (int i = w; i < 2 * len + 1; i += 4) {
        const bool is_draft = i > len;
        if (is_draft && (GREEDY || !a.draft)) break;
        const int64_t row = is_draft ? targets + (int64_t)b * a.m + (i - len - 1) : (int64_t)b * (a.m + 1) + i;
        float2 v = l < a.splits ? a.stats[row * a.splits + l] : GREEDY ? no_token() : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int off = 32; off; off >>= 1) v = merge<GREEDY>(v, shfl_xor2(v, off), c);
        if (l == 0) (is_draft ? s.draft[i - len - 1] : s.target[i]) = v;
    }
    __syncthreads();
    if (t < len) {
        const int x = a.tokens[(int64_t)b * a.m + t];
        bool ok = false;
        if (x >= 0 && x < a.vocab) {  // a token outside the vocabulary is rejected
            const float2 of_t = s.target[t];
            if constexpr (GREEDY) {
                ok = __float_as_int(of_t.y) == x;
            } else {
                const int64_t row = (int64_t)b * (a.m + 1) + t;
                const float p = of_t.y > 0.f ? weight(load1<F32>(a.target, row * a.target_stride + x), of_t.x, c) / of_t.y : 0.f;
                float q = 1.f;
                if (a.draft) {
                    const int64_t dr = (int64_t)b * a.m + t;
                    const float2 of_d = s.draft[t];
                    q = of_d.y > 0.f ? weight(load1<F32>(a.draft, dr * a.draft_stride + x), of_d.x, c) / of_d.y : 0.f;
                }
                ok = a.accept_u[(int64_t)b * a.m + t] * q < p;
            }
        }
        s.ok[t] = ok;
    }
    __syncthreads();
    int acc = 0;
    while (acc < len && s.ok[acc]) ++acc;
    return acc;
}

// The best of r / e (whole: of p / e) over the tokens lo .. hi - 1, by the whole
// workgroup, as (score, token) ordered as one integer: scores are not negative, the
// lower token is the larger; 0 where no score is above 0.
template <bool F32> __device__ __forceinline__ uint64_t draw(const VerifyArgs &a, int b, int acc, DecideLds &s, int lo, int hi, bool whole, int t) {
    const float c = a.inv_temperature * kLog2e;
    const int64_t trow = ((int64_t)b * (a.m + 1) + acc) * a.target_stride;
    const int64_t drow = ((int64_t)b * a.m + acc) * a.draft_stride;
    const bool rejected = acc < length_of(a, b), less = rejected && a.draft;
    const int bad = rejected ? a.tokens[(int64_t)b * a.m + acc] : -1;
    // a row without probabilities: its weights come out as NaN (never above 0) or are held to 0
    const float tm = s.target[acc].x, ti = s.target[acc].y > 0.f ? 1.f / s.target[acc].y : 0.f;
    const bool has_q = less && s.draft[acc].y > 0.f;
    const float dm = has_q ? s.draft[acc].x : 0.f, di = has_q ? 1.f / s.draft[acc].y : 0.f;
    const float *noise = a.sample_e + (int64_t)b * a.vocab;
    float score = 0.f;
    int token = kNone;
    for (int v = lo + 8 * t; v < hi; v += 2048) {
        float x[8], q[8], e[8];
        if (v + 8 <= hi) {
            load8<F32>(a.target, trow + v, x);
            if (less) load8<F32>(a.draft, drow + v, q);
            load8<true>(noise, v, e);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = v + j < hi;
                x[j] = in ? load1<F32>(a.target, trow + v + j) : -INFINITY;
                q[j] = in && less ? load1<F32>(a.draft, drow + v + j) : -INFINITY;
                e[j] = in ? noise[v + j] : 1.f;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float r = __builtin_amdgcn_exp2f((x[j] - tm) * c) * ti;
            if (!whole) r -= less ? __builtin_amdgcn_exp2f((q[j] - dm) * c) * di : v + j == bad ? 1.f : 0.f;
            r = fmaxf(r, 0.f) * __builtin_amdgcn_rcpf(e[j]);  // held to 0 first: noise below 0 takes a token out
            if (r > score) score = r, token = v + j;
        }
    }
    uint64_t best = token == kNone ? 0 : (uint64_t)__float_as_uint(score) << 32 | (uint32_t)(kNone - token);
#pragma unroll
    for (int off = 32; off; off >>= 1) {
        const uint64_t other = __shfl_xor((unsigned long long)best, off);
        best = other > best ? other : best;
    }
    __syncthreads();
    if ((t & 63) == 0) s.best[t >> 6] = best;
    __syncthreads();
    best = s.best[0];
    for (int i = 1; i < 4; ++i) best = s.best[i] > best ? s.best[i] : best;
    return best;
}
__device__ __forceinline__ int token_of(uint64_t best) { return best == 0 ? -1 : kNone - (int)(uint32_t)best; }

template <bool F32, bool GREEDY> __global__ __launch_bounds__(256) void decide_kernel(VerifyArgs a) {
    __shared__ DecideLds s;
    const int t = threadIdx.x, part = blockIdx.x, b = blockIdx.y;
    const int acc = decide<F32, GREEDY>(a, b, s, t);
    if (part == 0 && t == 0) a.accepted[b] = acc;
    if constexpr (GREEDY) {
        const int token = __float_as_int(s.target[acc].y);
        if (t == 0) a.next[b] = token == kNone ? -1 : token;
    } else {
        int lo, hi;
        segment(a.vocab, part, a.sample_splits, lo, hi);
        uint64_t best = draw<F32>(a, b, acc, s, lo, hi, false, t);
        if (a.sample_splits > 1) {
            if (t == 0) a.best[(int64_t)b * a.sample_splits + part] = best;
            return;
        }
        if (best == 0) best = draw<F32>(a, b, acc, s, 0, a.vocab, true, t);  // nothing left of p after q: from p itself
        if (t == 0) a.next[b] = token_of(best);
    }
}

// The best of a request's parts.
template <bool F32> __global__ __launch_bounds__(256) void pick_kernel(VerifyArgs a) {
    __shared__ DecideLds s;
    const int t = threadIdx.x, b = blockIdx.x;
    uint64_t best = (t & 63) < a.sample_splits ? a.best[(int64_t)b * a.sample_splits + (t & 63)] : 0;
#pragma unroll
    for (int off = 32; off; off >>= 1) {
        const uint64_t other = __shfl_xor((unsigned long long)best, off);
        best = other > best ? other : best;
    }
    if (best == 0) {  // in every wave alike: nothing left of p after q, from p itself
        const int acc = decide<F32, false>(a, b, s, t);
        best = draw<F32>(a, b, acc, s, 0, a.vocab, true, t);
    }
    if (t == 0) a.next[b] = token_of(best);
}

template <bool F32, bool GREEDY> hipError_t verify(const VerifyArgs &a, hipStream_t stream) {
    const int64_t rows = (int64_t)a.n * (a.m + 1) + (a.draft && !GREEDY ? (int64_t)a.n * a.m : 0);
    hipLaunchKernelGGL((stats_kernel<F32, GREEDY>), dim3(a.splits, (uint32_t)rows), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((decide_kernel<F32, GREEDY>), dim3(GREEDY ? 1 : a.sample_splits, a.n), dim3(256), 0, stream, a);
    if constexpr (!GREEDY)
        if (a.sample_splits > 1) hipLaunchKernelGGL((pick_kernel<F32>), dim3(a.n), dim3(256), 0, stream, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_verify(const VerifyArgs &args, bool f32, bool greedy, hipStream_t stream) {
    VerifyArgs a = args;
    // enough workgroups to fill the GPU, segments long enough to be worth one
    const int64_t rows = (int64_t)a.n * (a.m + 1) + (a.draft && !greedy ? (int64_t)a.n * a.m : 0);
    const int most = (a.vocab + kVerifySegment - 1) / kVerifySegment;
    auto parts = [&](int64_t have) {
        const int64_t want = (2048 + have - 1) / have;
        return (int32_t)(want < most ? (want < kVerifySplits ? want : kVerifySplits) : (most < kVerifySplits ? most : kVerifySplits));
    };
    a.splits = parts(rows);
    a.sample_splits = parts(a.n);
    if (f32) return greedy ? verify<true, true>(a, stream) : verify<true, false>(a, stream);
    return greedy ? verify<false, true>(a, stream) : verify<false, false>(a, stream);
}

} // namespace sqk
