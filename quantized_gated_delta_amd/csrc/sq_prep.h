// First phase of the chunked gated Delta rule: what depends on one chunk's
// keys, queries and gates alone, for every chunk in parallel.
//
//   B_ij = sum_c k_ic k_jc e^{G_ic - G_jc}  (j < i)     G: sum of the log-gates in the chunk
//   P_ij = sum_c q_ic k_jc e^{G_ic - G_jc}  (j <= i)
//   M    = -B - B diag(beta) M              (strictly lower)
//
// M carries no factor beta on its left, so that both (I + B diag(beta))^-1 =
// I + M diag(beta) and (I + diag(beta) B)^-1 = I + diag(beta) M follow from it
// without a division (a beta of 0 is a token that writes nothing).
//
// M is solved in 16 x 16 blocks: the four diagonal blocks of I + B diag(beta)
// are inverted by forward substitution, one per wave, then wave w takes block
// column w down the rows with the fp32 matrix instruction, whose result
// layout is the next product's operand layout: no exchange between waves.
//
// No exponential of a positive sum is taken where it could overflow: decays
// between 16-token blocks go through the sum at the later block's start (both
// factors at most 1).  Inside a block KDA uses the same product with the block's
// start as reference while no channel loses more than e^-kBlockRange over the block, and
// exponentials of each pair's own sum otherwise.
#pragma once

#include "sq_seq.h"

namespace sqk {

constexpr float kBlockRange = 60.f;
// Log-gates below this are as good as minus infinity: e^-150 is 0 in fp32.
constexpr float kGateFloor = -150.f;

constexpr int kBRow = 68;  // floats in a row of a 64 x 64 matrix in LDS

// Inverse of the unit lower triangular block I + B diag(beta) of one wave's
// 16 tokens; inv: [16][20].
__device__ __forceinline__ void invert_block(const float *sB, const float *sBeta, float *inv, int w, int l) {
    const int c = l & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float s = i == c ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < i; ++j) s = fmaf(-sB[(16 * w + i) * kBRow + 16 * w + j] * sBeta[16 * w + j], x[j], s);
        x[i] = s;
    }
    if (l < 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) inv[i * 20 + c] = x[i];
    }
}

// Block column w of M in the result layout: m[I] for row blocks I >= w.
__device__ __forceinline__ void solve_column(const float *sB, const float *sBeta, const float *sInv, int w, int l, f4 (&m)[4]) {
    const int r = l & 15, g4 = (l >> 4) * 4;
#pragma unroll
    for (int I = 0; I < 4; ++I) {
        m[I] = f4{};
        if (I < w) continue;
        f4 acc;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = -sB[(16 * I + g4 + i) * kBRow + 16 * w + r];
#pragma unroll
        for (int J = 0; J < 3; ++J) {
            if (J < w || J >= I) continue;
            f4 n = *reinterpret_cast<const f4 *>(sB + (16 * I + r) * kBRow + 16 * J + g4);
#pragma unroll
            for (int i = 0; i < 4; ++i) n[i] *= -sBeta[16 * J + g4 + i];
            acc = mma16(n, m[J], acc);
        }
        const f4 v = *reinterpret_cast<const f4 *>(sInv + I * 320 + r * 20 + g4);
        m[I] = mma16(v, acc, f4{});
    }
}

// A 64 x 64 matrix in LDS as an operand; TRANS: its transpose.
template <bool F32, int N, bool TRANS>
__device__ __forceinline__ void write_square(const float *s, Elem<F32> *out, int t) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int u = t + 256 * n, row = (u >> 7) * 16 + (u & 15), k = (u >> 4 & 7) * 8;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = TRANS ? s[(k + i) * kBRow + row] : s[row * kBRow + k + i];
        Operand<F32, N, 2>::put8(out, row, k, x);
    }
}

// Row `row` of the tokens t0 .. of a [token][head][d] input as an operand
// fragment; zero from the sequence's end on.
template <bool F32>
__device__ __forceinline__ Frag<F32, 1> token_frag(const void *base, int64_t stride, int64_t t0, int rows, int row, int64_t at) {
    Frag<F32, 1> f;
    if (row < rows)
        f = load_frag<F32, 1>(static_cast<const Elem<F32> *>(base) + (t0 + row) * stride + at, 0);
    else
        zero(f);
    return f;
}

// The chunk's keys or queries as [channel][token], through LDS (s: 64 rows of
// D + 16 bytes).  All threads call it.
template <int D, bool F32>
__device__ __forceinline__ void write_transposed(const void *base, int64_t stride, int64_t t0, int rows, int head, Elem<F32> *s,
                                                 Elem<F32> *out, int t) {
    constexpr int ROW = D + 16 / (int)sizeof(Elem<F32>), U = D / 8;
    for (int u = t; u < kChunk * U; u += 256) {
        const int row = u / U, c = u % U * 8;
        const Frag<F32, 1> f = token_frag<F32>(base, stride, t0, rows, row, (int64_t)head * D + c);
        if constexpr (F32) {
            *reinterpret_cast<f4 *>(s + row * ROW + c) = f.v[0];
            *reinterpret_cast<f4 *>(s + row * ROW + c + 4) = f.v[1];
        } else {
            *reinterpret_cast<bf8 *>(s + row * ROW + c) = f.t[0];
        }
    }
    __syncthreads();
    for (int u = t; u < D * 8; u += 256) {
        const int ch = (u >> 7) * 16 + (u & 15), k = (u >> 4 & 7) * 8;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = ld_elem<F32>(s, (k + i) * ROW + ch);
        Operand<F32, 1, 2>::put8(out, ch, k, x);
    }
    __syncthreads();
}

// GDN: sums of the log-gates (in double: differences of sums lose nothing) and
// beta of one chunk, by the first wave.
template <bool F32>
__device__ __forceinline__ void gates_gdn(const SeqArgs &a, int64_t t0, int rows, int h, double *sG, float *sBeta, int t) {
    if (t < kChunk) {
        double g = 0.;
        float b = 0.f;
        if (t < rows) {
            g = (double)fmaxf(ld_elem<F32>(a.g, (t0 + t) * a.n_heads + h), kGateFloor);
            b = ld_elem<F32>(a.beta, (t0 + t) * a.n_heads + h);
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const double up = __shfl_up(g, off);
            if (t >= off) g += up;
        }
        sG[t] = g;
        sBeta[t] = b;
    }
}

// GDN: B and P of one chunk into LDS (wave w: token rows 16 w .. + 15; blocks
// above the diagonal are set to zero).
template <int D, bool F32>
__device__ __forceinline__ void pairs_gdn(const SeqArgs &a, int64_t t0, int rows, int hk, const double *sG, float *sB, float *sP, int w, int l) {
    constexpr int KB = D / 32;
    const int r = l & 15, g8 = (l >> 4) * 8, g4 = (l >> 4) * 4;
    Frag<F32, 1> fk[KB], fq[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const int64_t at = (int64_t)hk * D + kb * 32 + g8;
        fk[kb] = token_frag<F32>(a.k, a.k_stride, t0, rows, 16 * w + r, at);
        fq[kb] = token_frag<F32>(a.q, a.q_stride, t0, rows, 16 * w + r, at);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f4 kk{}, qk{};
        if (j <= w) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const Frag<F32, 1> b = token_frag<F32>(a.k, a.k_stride, t0, rows, 16 * j + r, (int64_t)hk * D + kb * 32 + g8);
                kk = mma<1>(fk[kb], b, kk);
                qk = mma<1>(fq[kb], b, qk);
            }
        }
        const int col = 16 * j + r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * w + g4 + i;
            const float e = col <= row ? exp_of((float)(sG[row] - sG[col])) : 0.f;
            sB[row * kBRow + col] = col < row ? kk[i] * e : 0.f;
            sP[row * kBRow + col] = col <= row ? qk[i] * e : 0.f;
        }
    }
}

// KDA: the chunk's keys, queries (as fp32 or bf16) and, per 16-token block and
// channel, the sums of the log-gates up to a token (L) and after it (R) in LDS.
template <int D, bool F32> struct KdaLds {
    static constexpr int ROW = D + 16 / (int)sizeof(Elem<F32>), GROW = D + 4;
    union {
        struct { Elem<F32> k[kChunk * ROW], q[kChunk * ROW]; };
        struct { float B[kChunk * kBRow], P[kChunk * kBRow]; };  // after k and q were read
    };
    float L[kChunk * GROW], R[kChunk * GROW];
    float beta[kChunk];
    float range[4];  // the largest loss over a block, per block
};

template <int D, bool F32>
__device__ __forceinline__ void load_kda(const SeqArgs &a, int64_t t0, int rows, int h, int hk, KdaLds<D, F32> &s, int t) {
    constexpr int ROW = KdaLds<D, F32>::ROW, GROW = KdaLds<D, F32>::GROW, U = D / 8;
    for (int u = t; u < kChunk * U; u += 256) {
        const int row = u / U, c = u % U * 8;
        const Frag<F32, 1> fk = token_frag<F32>(a.k, a.k_stride, t0, rows, row, (int64_t)hk * D + c);
        const Frag<F32, 1> fq = token_frag<F32>(a.q, a.q_stride, t0, rows, row, (int64_t)hk * D + c);
        float g[8];
        if (row < rows)
            widen(load_frag<F32, 1>(static_cast<const Elem<F32> *>(a.g) + ((t0 + row) * a.n_heads + h) * D + c, 0), g);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = 0.f;
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                *reinterpret_cast<f4 *>(s.k + row * ROW + c + 4 * i) = fk.v[i];
                *reinterpret_cast<f4 *>(s.q + row * ROW + c + 4 * i) = fq.v[i];
            }
        } else {
            *reinterpret_cast<bf8 *>(s.k + row * ROW + c) = fk.t[0];
            *reinterpret_cast<bf8 *>(s.q + row * ROW + c) = fq.t[0];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s.L[row * GROW + c + i] = fmaxf(g[i], kGateFloor);
    }
    if (t < kChunk) s.beta[t] = t < rows ? ld_elem<F32>(a.beta, (t0 + t) * a.n_heads + h) : 0.f;
    if (t < 4) s.range[t] = 0.f;
    __syncthreads();
    for (int u = t; u < 4 * D; u += 256) {
        const int blk = u / D, c = u % D;
        float *L = s.L + blk * 16 * GROW + c, *R = s.R + blk * 16 * GROW + c;
        float g[16], up = 0.f, down = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = L[i * GROW];
#pragma unroll
        for (int i = 0; i < 16; ++i) up += g[i], L[i * GROW] = up;
#pragma unroll
        for (int i = 15; i >= 0; --i) R[i * GROW] = down, down += g[i];
        // non-negative floats order as their bits do
        atomicMax(reinterpret_cast<int *>(&s.range[blk]), __float_as_int(fmaxf(-up, 0.f)));
    }
    __syncthreads();
}

// Eight channels of a token with a decay each: x_c e^{G}, where the exponent is
// the sum from the token's block's start (MODE 0), from the chunk's start (1),
// to the chunk's end (2), or from the token to block I's start (3).
template <int D, bool F32, int MODE>
__device__ __forceinline__ void decayed8(const KdaLds<D, F32> &s, const Elem<F32> *x, int tok, int c, int I, float (&out)[8]) {
    constexpr int ROW = KdaLds<D, F32>::ROW, GROW = KdaLds<D, F32>::GROW;
    const float *E = (MODE >= 2 ? s.R : s.L) + tok * GROW + c;
    const int blk = tok >> 4;
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = E[i];
    if (MODE == 1)
        for (int b = 0; b < blk; ++b)
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] += s.L[(16 * b + 15) * GROW + c + i];
    if (MODE >= 2)
        for (int b = blk + 1; b < (MODE == 2 ? 4 : I); ++b)
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] += s.L[(16 * b + 15) * GROW + c + i];
    widen(load_frag<F32, 1>(x + tok * ROW + c, 0), out);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] *= exp_of(e[i]);
}

// The diagonal 16 x 16 blocks of B and P by each pair's own sum of log-gates,
// for gates too strong for a common reference: a lane holds D / 64 channels,
// sums over channels go across the wave.  Results in the matrix instruction's layout.
template <int D, bool F32>
__device__ __forceinline__ void diagonal_kda(const SeqArgs &a, int64_t t0, int rows, int h, const KdaLds<D, F32> &s, int w, int l, f4 &dk, f4 &dq) {
    constexpr int ROW = KdaLds<D, F32>::ROW, NC = D / 64;
    float g[NC][16];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int row = 16 * w + i;
            g[n][i] = row < rows ? fmaxf(ld_elem<F32>(a.g, ((t0 + row) * a.n_heads + h) * D + 64 * n + l), kGateFloor) : 0.f;
        }
#pragma unroll 1
    for (int j = 0; j < 16; ++j) {
        float e[NC], kj[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            e[n] = 0.f;
            kj[n] = ld_elem<F32>(s.k, (16 * w + j) * ROW + 64 * n + l);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < j) continue;
            float sk = 0.f, sq = 0.f;
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                if (i > j) e[n] += g[n][i];
                const float x = kj[n] * exp_of(e[n]);
                sk = fmaf(x, ld_elem<F32>(s.k, (16 * w + i) * ROW + 64 * n + l), sk);
                sq = fmaf(x, ld_elem<F32>(s.q, (16 * w + i) * ROW + 64 * n + l), sq);
            }
#pragma unroll
            for (int off = 32; off; off >>= 1) {
                sk += __shfl_xor(sk, off);
                sq += __shfl_xor(sq, off);
            }
            if (l == (i / 4) * 16 + j) dk[i % 4] = sk, dq[i % 4] = sq;
        }
    }
}

// KDA: B and P of one chunk into LDS, over the keys and queries there (sB, sP
// share their place; all threads call it).  PQ: terms that P is accurate to.
template <int D, bool F32, int PQ>
__device__ __forceinline__ void pairs_kda(const SeqArgs &a, int64_t t0, int rows, int h, KdaLds<D, F32> &s, int w, int l) {
    constexpr int KB = D / 32, ROW = KdaLds<D, F32>::ROW, GROW = KdaLds<D, F32>::GROW;
    const int r = l & 15, g8 = (l >> 4) * 8, g4 = (l >> 4) * 4;
    const bool fast = s.range[w] <= kBlockRange;
    f4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f4{};
#pragma unroll 1
    for (int kb = 0; kb < KB; ++kb) {
        const int c = kb * 32 + g8;
        float x[8];
        decayed8<D, F32, 0>(s, s.k, 16 * w + r, c, 0, x);
        const Frag<F32, 3> fk = make_frag<F32, 3>(x);
        decayed8<D, F32, 0>(s, s.q, 16 * w + r, c, 0, x);
        const Frag<F32, PQ> fq = make_frag<F32, PQ>(x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j > w || (j == w && !fast)) continue;
            if (j < w) {
                decayed8<D, F32, 3>(s, s.k, 16 * j + r, c, w, x);
            } else {  // e^{-L}: the same block's start as reference
                widen(load_frag<F32, 1>(s.k + (16 * w + r) * ROW + c, 0), x);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= exp_of(-s.L[(16 * w + r) * GROW + c + i]);
            }
            const Frag<F32, 3> fb = make_frag<F32, 3>(x);
            kk[j] = mma<3>(fk, fb, kk[j]);
            qk[j] = mma<PQ>(fq, fb, qk[j]);
        }
    }
    f4 dk{}, dq{};
    if (!fast) diagonal_kda<D, F32>(a, t0, rows, h, s, w, l, dk, dq);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int col = 16 * j + r;
        const bool diag = j == w && !fast;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * w + g4 + i;
            s.B[row * kBRow + col] = col < row ? (diag ? dk[i] : kk[j][i]) : 0.f;
            s.P[row * kBRow + col] = col <= row ? (diag ? dq[i] : qk[j][i]) : 0.f;
        }
    }
}

} // namespace sqk
