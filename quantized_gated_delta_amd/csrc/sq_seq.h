// Shared by the sequence kernels (sq_chunk.hip, sq_chunk_bwd.hip, sq_window.hip):
// operand fragments of the matrix cores, their LDS layout, and the chunk map.
//
// Precision.  A product of two fp32 matrices on the bf16 matrix cores takes
// each operand as a sum of bf16 terms, x = x0 + x1 + x2 with x0 = bf16(x),
// x1 = bf16(x - x0), ...: three terms hold all 24 bits of an fp32, two hold
// 16 (relative error 2^-17).  mma<P> sums the products a_i b_j with i + j < P.
//   P = 3  whatever reaches a state or an fp32 result (fp32-accurate);
//   P = 2  what only reaches a result that is rounded to bf16 at the end
//          (2^-17 against that rounding's 2^-9).
// bf16 inputs are one term and exact, so a product with them costs P matrix
// instructions instead of P (P + 1) / 2.  fp32 inputs use the fp32 matrix
// instruction: 16 times slower than one bf16 product, 2.7 times slower than the
// six of P = 3, but exact in its operands and free of the splitting.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <type_traits>

#include "sq_internal.h"

namespace sqk {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int kChunk = 64;  // tokens of a chunk

template <bool F32> struct ElemOf { typedef uint16_t type; };
template <> struct ElemOf<true> { typedef float type; };
template <bool F32> using Elem = typename ElemOf<F32>::type;

// One lane's part of a 16 x 32 operand (A: row l % 16; B: column l % 16),
// elements 8 (l / 16) .. + 7 of the contracted axis: N bf16 terms, or fp32.
template <bool F32, int N> struct Frag { bf8 t[N]; };
template <int N> struct Frag<true, N> { f4 v[2]; };

template <int P, int NA, int NB>
__device__ __forceinline__ f4 mma(const Frag<false, NA> &a, const Frag<false, NB> &b, f4 c) {
#pragma unroll
    for (int s = P - 1; s >= 0; --s)  // small products first
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
                c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.t[i], b.t[s - i], c, 0, 0, 0);
    return c;
}
template <int P, int NA, int NB>
__device__ __forceinline__ f4 mma(const Frag<true, NA> &a, const Frag<true, NB> &b, f4 c) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i / 4][i % 4], b.v[i / 4][i % 4], c, 0, 0, 0);
    return c;
}

// Contraction over 16: a in memory order (row l % 16, elements 4 (l / 16) .. + 3),
// b as the result layout leaves it (column l % 16, rows 4 (l / 16) .. + 3).
__device__ __forceinline__ f4 mma16(f4 a, f4 b, f4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
}

// x as N bf16 terms, the largest first.
template <int N> __device__ __forceinline__ void split(float x, __bf16 (&t)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i] = (__bf16)x;
        x -= (float)t[i];
    }
}

// Two at a time: the conversion instruction takes a pair.
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));
template <int N> __device__ __forceinline__ void split2(f2 x, bf2 (&t)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i] = __builtin_convertvector(x, bf2);
        if (i + 1 < N) x -= __builtin_convertvector(t[i], f2);
    }
}
template <int N> __device__ __forceinline__ void split4(f4 x, bf4 (&t)[N]) {
    bf2 a[N], b[N];
    split2<N>(f2{x[0], x[1]}, a);
    split2<N>(f2{x[2], x[3]}, b);
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = __builtin_shufflevector(a[i], b[i], 0, 1, 2, 3);
}

template <int N> __device__ __forceinline__ Frag<false, N> frag_of(const float (&x)[8], Frag<false, N> *) {
    Frag<false, N> f;
    bf4 a[N], b[N];
    split4<N>(f4{x[0], x[1], x[2], x[3]}, a);
    split4<N>(f4{x[4], x[5], x[6], x[7]}, b);
#pragma unroll
    for (int p = 0; p < N; ++p) f.t[p] = __builtin_shufflevector(a[p], b[p], 0, 1, 2, 3, 4, 5, 6, 7);
    return f;
}
template <int N> __device__ __forceinline__ Frag<true, N> frag_of(const float (&x)[8], Frag<true, N> *) {
    Frag<true, N> f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i / 4][i % 4] = x[i];
    return f;
}
template <bool F32, int N> __device__ __forceinline__ Frag<F32, N> make_frag(const float (&x)[8]) {
    return frag_of(x, (Frag<F32, N> *)nullptr);
}

template <int N>
__device__ __forceinline__ Frag<false, N> frag_at(const uint16_t *p, int64_t plane, Frag<false, N> *) {
    Frag<false, N> f;
#pragma unroll
    for (int i = 0; i < N; ++i) f.t[i] = *reinterpret_cast<const bf8 *>(p + i * plane);
    return f;
}
template <int N>
__device__ __forceinline__ Frag<true, N> frag_at(const float *p, int64_t, Frag<true, N> *) {
    Frag<true, N> f;
    f.v[0] = *reinterpret_cast<const f4 *>(p);
    f.v[1] = *reinterpret_cast<const f4 *>(p + 4);
    return f;
}
// A fragment at p; the terms of bf16 are `plane` elements apart.
template <bool F32, int N> __device__ __forceinline__ Frag<F32, N> load_frag(const Elem<F32> *p, int64_t plane) {
    return frag_at(p, plane, (Frag<F32, N> *)nullptr);
}
template <int N> __device__ __forceinline__ void zero(Frag<false, N> &f) {
#pragma unroll
    for (int p = 0; p < N; ++p) f.t[p] = bf8{};
}
template <int N> __device__ __forceinline__ void zero(Frag<true, N> &f) { f.v[0] = f.v[1] = f4{}; }

// The elements of a single-term fragment as fp32.
__device__ __forceinline__ void widen(const Frag<false, 1> &f, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)f.t[0][i];
}
__device__ __forceinline__ void widen(const Frag<true, 1> &f, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = f.v[i / 4][i % 4];
}

// A matrix in LDS as [column][K] (an operand whose contracted axis is
// contiguous), N terms one after another.  Rows are padded by 16 bytes: the
// 16 columns of a fragment read then start 4 banks apart.
template <bool F32, int N, int K, int COLS> struct LdsMat {
    typedef Elem<F32> E;
    static constexpr int ROW = F32 ? K + 4 : K + 8;
    static constexpr int PLANE = COLS * ROW;
    static constexpr int BYTES = F32 ? PLANE * 4 : N * PLANE * 2;
    __device__ __forceinline__ static Frag<F32, N> get(const E *m, int col, int k) {
        return load_frag<F32, N>(m + col * ROW + k, PLANE);
    }
    // four consecutive elements of one column, as the result layout holds them
    __device__ __forceinline__ static void put4(E *m, int col, int k, f4 x) {
        if constexpr (F32) {
            *reinterpret_cast<f4 *>(m + col * ROW + k) = x;
        } else {
            bf4 v[N];
            split4<N>(x, v);
#pragma unroll
            for (int p = 0; p < N; ++p) *reinterpret_cast<bf4 *>(m + p * PLANE + col * ROW + k) = v[p];
        }
    }
};

template <bool F32> __device__ __forceinline__ float ld_elem(const void *p, int64_t i) {
    if constexpr (F32)
        return static_cast<const float *>(p)[i];
    else
        return (float)static_cast<const __bf16 *>(p)[i];
}
// The same in two parts, the load and the widening, so that several loads are
// in flight before the first is waited for.
template <bool F32> using RawOf = std::conditional_t<F32, uint32_t, uint16_t>;
template <bool F32> __device__ __forceinline__ uint32_t ld_raw(const void *p, int64_t i) { return static_cast<const RawOf<F32> *>(p)[i]; }
template <bool F32> __device__ __forceinline__ float of_raw(uint32_t x) { return __uint_as_float(F32 ? x : x << 16); }
template <bool F32> __device__ __forceinline__ void st_elem(void *p, int64_t i, float x) {
    if constexpr (F32)
        static_cast<float *>(p)[i] = x;
    else
        static_cast<__bf16 *>(p)[i] = (__bf16)x;
}
template <bool F32> __device__ __forceinline__ void st_elem4(void *p, int64_t i, f4 x) {
    if constexpr (F32) {
        *reinterpret_cast<f4 *>(static_cast<float *>(p) + i) = x;
    } else {
        bf4 v[1];
        split4<1>(x, v);
        *reinterpret_cast<bf4 *>(static_cast<__bf16 *>(p) + i) = v[0];
    }
}

// An address as a wave's base and a lane's 32-bit byte offset: the load takes
// both as they are, where a 64-bit sum would cost vector instructions.
template <typename T> __device__ __forceinline__ const T *at_bytes(const void *base, uint32_t bytes) {
    return reinterpret_cast<const T *>(static_cast<const char *>(base) + bytes);
}
template <typename T> __device__ __forceinline__ T *at_bytes(void *base, uint32_t bytes) {
    return reinterpret_cast<T *>(static_cast<char *>(base) + bytes);
}

// Operands in the workspace lie as the fragments are read: for every 16 rows
// and 32 contracted elements, the terms one after another, each 64 lanes of
// 16 bytes (fp32: two halves of 64 lanes of 16 bytes).  A wave's load is then 1 KB
// of consecutive bytes; rows in memory order would make it 16 half cache lines.
// KB: fragments along the contracted axis.
template <bool F32, int N, int KB> struct Operand {
    static constexpr int SIZE = F32 ? 512 : 512 * N;  // elements of a fragment
    __device__ __forceinline__ static Frag<F32, N> get(const Elem<F32> *m, int tile, int kb, int lane) {
        Frag<F32, N> f;
        const Elem<F32> *p = m + (tile * KB + kb) * SIZE;
        if constexpr (F32) {
            f.v[0] = *at_bytes<f4>(p, 16u * lane);
            f.v[1] = *at_bytes<f4>(p + 256, 16u * lane);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) f.t[i] = *at_bytes<bf8>(p + 512 * i, 16u * lane);
        }
        return f;
    }
    __device__ __forceinline__ static void put(Elem<F32> *m, int tile, int kb, int lane, const Frag<F32, N> &f) {
        Elem<F32> *p = m + (tile * KB + kb) * SIZE;
        if constexpr (F32) {
            *at_bytes<f4>(p, 16u * lane) = f.v[0];
            *at_bytes<f4>(p + 256, 16u * lane) = f.v[1];
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) *at_bytes<bf8>(p + 512 * i, 16u * lane) = f.t[i];
        }
    }
    // row `row`, contracted elements k .. k + 7 (k a multiple of 8)
    __device__ __forceinline__ static void put8(Elem<F32> *m, int row, int k, const float (&x)[8]) {
        const int lane = (k & 31) / 8 * 16 + (row & 15);
        Elem<F32> *p = m + ((row >> 4) * KB + (k >> 5)) * SIZE;
        if constexpr (F32) {
            *reinterpret_cast<f4 *>(p + 4 * lane) = f4{x[0], x[1], x[2], x[3]};
            *reinterpret_cast<f4 *>(p + 256 + 4 * lane) = f4{x[4], x[5], x[6], x[7]};
        } else {
            const Frag<false, N> f = make_frag<false, N>(x);
#pragma unroll
            for (int i = 0; i < N; ++i) *reinterpret_cast<bf8 *>(p + 512 * i + 8 * lane) = f.t[i];
        }
    }
};

// Four consecutive contracted elements k .. k + 3 of one row, N terms: what a lane
// of a transposed 16 x 16 result tile holds.
template <bool F32, int N, int KB> __device__ __forceinline__ uint32_t operand4(int row, int k) {  // bytes
    const uint32_t lane = (k & 31) / 8 * 16 + (row & 15), half = k >> 2 & 1;
    const uint32_t frag = ((row >> 4) * KB + (k >> 5)) * (Operand<F32, N, KB>::SIZE * (uint32_t)sizeof(Elem<F32>));
    return frag + 16 * lane + (F32 ? 1024 : 8) * half;
}
template <bool F32, int N, int KB> __device__ __forceinline__ void put_operand4(Elem<F32> *m, int row, int k, f4 x) {
    const uint32_t at = operand4<F32, N, KB>(row, k);
    if constexpr (F32) {
        *at_bytes<f4>(m, at) = x;
    } else {
        bf4 v[N];
        split4<N>(x, v);
#pragma unroll
        for (int n = 0; n < N; ++n) *at_bytes<bf4>(m + 512 * n, at) = v[n];
    }
}
// ... read back in two parts, the load and the sum of the terms.
template <bool F32, int N> struct Raw4 { bf4 t[N]; };
template <int N> struct Raw4<true, N> { f4 t; };
template <bool F32, int N, int KB> __device__ __forceinline__ Raw4<F32, N> get_operand4(const Elem<F32> *m, int row, int k) {
    const uint32_t at = operand4<F32, N, KB>(row, k);
    Raw4<F32, N> x;
    if constexpr (F32) {
        x.t = *at_bytes<f4>(m, at);
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n) x.t[n] = *at_bytes<bf4>(m + 512 * n, at);
    }
    return x;
}
template <int N> __device__ __forceinline__ f4 sum_of(const Raw4<true, N> &x) { return x.t; }
template <int N> __device__ __forceinline__ f4 sum_of(const Raw4<false, N> &x) {
    f4 y{};
#pragma unroll
    for (int n = N - 1; n >= 0; --n) y += __builtin_convertvector(x.t[n], f4);
    return y;
}

// A 16 x 16 result tile turned around through a wave's own LDS (16 x 20
// floats): in, column l % 16 and rows 4 (l / 16) .. + 3; out, row l % 16 and
// columns 4 (l / 16) .. + 3.
__device__ __forceinline__ f4 turn(float *s, f4 x, int l) {
    const int r = l & 15, g4 = (l >> 4) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) s[(g4 + i) * 20 + r] = x[i];
    __builtin_amdgcn_wave_barrier();
    const f4 y = *reinterpret_cast<const f4 *>(s + r * 20 + g4);
    __builtin_amdgcn_wave_barrier();
    return y;
}

// exp(x) for x <= 0 (or moderate x > 0): the hardware exponential of x log2(e)
// with the rounding error of that product put back; relative error about 2^-22.
__device__ __forceinline__ float exp_of(float x) {
    const float l = 1.44269504088896340736f, ln2 = 0.69314718055994530942f;
    const float t = x * l;
    const float e = fmaf(x, l, -t) + x * 1.925963033500011e-8f;  // log2(e) - l
    const float r = __builtin_amdgcn_exp2f(t);
    return fmaf(r, e * ln2, r);
}

// What the sequence kernels are given.  Chunks are numbered without a prefix
// sum over lengths on the host: sequence s owns the chunk slots from
// cu[s] / 64 + s, which never overlap; slots that no chunk falls on stay idle.
struct SeqArgs {
    const void *q, *k, *v, *beta, *g;
    int64_t q_stride, k_stride, v_stride;  // elements from token to token
    const int32_t *cu;                     // [n_seq + 1]
    int32_t n_seq, n_heads, n_key_heads;
    int64_t n_tokens;
    const float *S0;
    float *S_out;
    void *y;
    uint8_t *work;   // operands of the scan, per (chunk slot, head)
    uint8_t *save;   // what the backward pass needs of the forward, or null
    // backward
    const void *dy;
    const float *dS_out;
    void *dq, *dk, *dv, *dbeta, *dg;
    float *dS0;
};

struct SeqSpan {
    int32_t seq;
    int64_t t0;      // first token
    int32_t len;     // tokens of the sequence
    int64_t slot0;   // its first chunk slot
};

// Sequence s.  Offsets are held inside the tokens, so that a wrong list
// cannot make a kernel leave its buffers.
__device__ __forceinline__ SeqSpan seq_span(const SeqArgs &a, int32_t s) {
    SeqSpan r;
    const int32_t n = (int32_t)a.n_tokens;
    int32_t lo = a.cu[s], hi = a.cu[s + 1];
    lo = lo < 0 ? 0 : lo > n ? n : lo;
    hi = hi < lo ? lo : hi > n ? n : hi;
    r.seq = s;
    r.t0 = lo;
    r.len = hi - lo;
    r.slot0 = (int64_t)(lo / kChunk) + s;
    return r;
}
// ... of a sequence that the whole wave asks for, in scalar registers: every address
// that follows from it is then formed by the scalar unit.
__device__ __forceinline__ SeqSpan wave_span(const SeqArgs &a, int32_t s) {
    SeqSpan r = seq_span(a, s);
    r.seq = s;
    r.t0 = __builtin_amdgcn_readfirstlane((int)r.t0);
    r.len = __builtin_amdgcn_readfirstlane(r.len);
    r.slot0 = r.t0 / kChunk + s;
    return r;
}

// The sequence that owns chunk slot x, and the chunk's number in it (negative
// where x is idle).  The 64 lanes of a wave probe 64 sequences at a time: two dependent
// loads for up to 64 sequences, where a binary search would wait for six.
__device__ __forceinline__ int32_t chunk_at(const SeqArgs &a, int64_t x, SeqSpan &r) {
    const int l = threadIdx.x & 63;
    int32_t lo = 0, n = a.n_seq;
    while (n > 64) {  // the last probed s with slot0(s) <= x
        const int32_t step = (n + 63) >> 6, s = lo + l * step;
        const bool before = l * step < n && seq_span(a, min(s, a.n_seq - 1)).slot0 <= x;
        const int k = max(__popcll(__ballot(before)) - 1, 0);
        lo += k * step;
        n = min(step, n - k * step);
    }
    const SeqSpan mine = seq_span(a, min(lo + l, a.n_seq - 1));
    const int k = max(__popcll(__ballot(l < n && mine.slot0 <= x)) - 1, 0);
    r.seq = lo + k;
    r.t0 = __builtin_amdgcn_readlane((int)mine.t0, k);
    r.len = __builtin_amdgcn_readlane(mine.len, k);
    r.slot0 = r.t0 / kChunk + r.seq;
    const int64_t c = x - r.slot0;
    return c >= 0 && c * kChunk < r.len ? (int32_t)c : -1;
}

// Layout of the workspace: per (chunk slot, head) one block of operand planes.
// bf16: `terms` planes each; fp32: one plane of floats.
struct ChunkLayout {
    // offsets in bytes within a block
    int64_t M, P, K, Q, KT, gates, block;
};

__host__ __device__ constexpr int64_t plane_bytes(bool f32, int terms, int rows, int cols) {
    return (int64_t)rows * cols * (f32 ? 4 : 2 * terms);
}

// Forward operands: M and P (64 x 64), the decayed keys and queries (KDA:
// 64 x d each), the keys as [channel][token] (GDN: undecayed, KDA: decayed to the
// chunk's end), and the gates' factors in fp32: GDN e^G, e^{G_C - G}, beta
// (64 each); KDA beta (64) and e^{G_C} (d).
__host__ __device__ constexpr ChunkLayout forward_layout(int d, bool kda, bool f32, int y_terms) {
    ChunkLayout l{};
    int64_t at = 0;
    l.M = at, at += plane_bytes(f32, 3, kChunk, kChunk);
    l.P = at, at += plane_bytes(f32, y_terms, kChunk, kChunk);
    l.KT = at, at += plane_bytes(f32, kda ? 3 : 1, d, kChunk);
    if (kda) {
        l.K = at, at += plane_bytes(f32, 3, kChunk, d);
        l.Q = at, at += plane_bytes(f32, y_terms, kChunk, d);
    }
    l.gates = at, at += 4 * (3 * kChunk + d);
    l.block = (at + 255) / 256 * 256;
    return l;
}

// What the forward pass leaves for the backward, per (chunk slot, head): the
// state at the chunk's start as an operand [channel][column] and E as
// [token][column], two terms each (as many bytes as fp32).
constexpr int kSaveTerms = 2;
struct SaveLayout { int64_t S, E, block; };
__host__ __device__ constexpr SaveLayout save_layout(int d) {
    SaveLayout l{};
    l.S = 0;
    l.E = (int64_t)d * d * 4;
    l.block = l.E + (int64_t)kChunk * d * 4;
    return l;
}

// Backward operands, per (chunk slot, head): M and P transposed, keys and
// queries as [channel][token] (KDA: decayed from the chunk's start), KDA's keys
// decayed to the chunk's end, the gates' factors as forward, and what the
// backward scan leaves for the gradients: the state's gradient at the chunk's end
// and v's, two terms each, the parts of beta's gradient per 16 columns, and room to
// add up q's and k's gradients over heads that share a key head.
struct BackwardLayout {
    int64_t MT, PT, KT, QT, K, gates, dS, dV, dbeta, sum, block;
};
__host__ __device__ constexpr BackwardLayout backward_layout(int d, bool kda, bool f32) {
    BackwardLayout l{};
    int64_t at = 0;
    l.MT = at, at += plane_bytes(f32, 3, kChunk, kChunk);
    l.PT = at, at += plane_bytes(f32, 3, kChunk, kChunk);
    l.KT = at, at += plane_bytes(f32, kda ? 3 : 1, d, kChunk);
    l.QT = at, at += plane_bytes(f32, kda ? 3 : 1, d, kChunk);
    if (kda) l.K = at, at += plane_bytes(f32, 3, kChunk, d);
    l.dS = at, at += plane_bytes(f32, kSaveTerms, d, d);
    l.dV = at, at += plane_bytes(f32, kSaveTerms, kChunk, d);
    l.gates = at, at += 4 * (3 * kChunk + d);
    l.dbeta = at, at += 4 * kChunk * (d / 16);
    l.sum = at, at += 2 * 4 * kChunk * d;
    l.block = (at + 255) / 256 * 256;
    return l;
}

inline int64_t chunk_slots(int64_t n_tokens, int32_t n_seq) { return n_tokens / kChunk + n_seq; }

hipError_t launch_chunk_forward(const SeqArgs &a, int d, bool kda, bool f32, bool y_f32, hipStream_t stream);
hipError_t launch_chunk_backward(const SeqArgs &a, int d, bool kda, bool f32, hipStream_t stream);

} // namespace sqk
