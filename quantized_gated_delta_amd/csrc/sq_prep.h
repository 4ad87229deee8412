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
// between 16-token blocks go through the ends of the blocks between them (every
// factor at most 1).  Inside a block KDA uses the same product with the block's
// start as reference while no channel loses more than e^-kBlockRange over the block, and
// exponentials of each pair's own sum otherwise.
//
// Bound by memory for GDN (forward 124 us for 12001 tokens x 48 heads, 5.3 TB/s with what it
// writes), by vector issue and latency for KDA, whose keys and queries are written decayed, in
// three terms (214 us for 8192 tokens x 32 heads, 4 TB/s).  What a chunk writes is read by
// the scan's slices, which would otherwise repeat its products eight times.
#pragma once

#include "sq_seq.h"

namespace sqk {

constexpr float kBlockRange = 60.f;
// Log-gates below this are as good as minus infinity: e^-150 is 0 in fp32.
constexpr float kGateFloor = -150.f;
// Not fmaxf, which would take the floor for a NaN and so forget the state without a word.
__device__ __forceinline__ float floor_gate(float g) { return __builtin_elementwise_maximum(g, kGateFloor); }

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

// Block (I, J) of a 64 x 64 matrix from the result layout into an operand; TRANS:
// into the operand of its transpose, which is what the layout already holds.
template <bool F32, int N, bool TRANS>
__device__ __forceinline__ void put_block(Elem<F32> *out, int I, int J, f4 x, float *tile, int l) {
    const int r = l & 15, g4 = (l >> 4) * 4;
    if (TRANS) put_operand4<F32, N, 2>(out, 16 * J + r, 16 * I + g4, x);
    else put_operand4<F32, N, 2>(out, 16 * I + r, 16 * J + g4, turn(tile, x, l));
}

// What a chunk's pairs come to.  Wave w holds blocks (w, j <= w) of B and P in the result
// layout, zero above the diagonal; writes P and M as operands (TRANS: their transposes).
// A fragment spans two blocks, so of the zero half the blocks beside the diagonal ones of
// even rows are written too.
template <bool F32, int N, bool TRANS>
__device__ __forceinline__ void solve_pairs(const f4 (&B)[4], const f4 (&P)[4], float *sB, const float *sBeta, float *sInv, float *tile, Elem<F32> *outP,
                                            Elem<F32> *outM, int w, int l) {
    const int r = l & 15, g4 = (l >> 4) * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j > (w | 1)) continue;
        put_block<F32, N, TRANS>(outP, w, j, P[j], tile, l);
        if (j <= w)
#pragma unroll
            for (int i = 0; i < 4; ++i) sB[(16 * w + g4 + i) * kBRow + 16 * j + r] = B[j][i];
    }
    __builtin_amdgcn_wave_barrier();
    invert_block(sB, sBeta, sInv + w * 320, w, l);
    __syncthreads();
    f4 m[4];
    solve_column(sB, sBeta, sInv, w, l, m);
#pragma unroll
    for (int I = 0; I < 4; ++I)
        if (I >= (w & ~1)) put_block<F32, 3, TRANS>(outM, I, w, m[I], tile, l);
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

// The chunk's keys or queries in LDS, [token][D] padded by 16 bytes.
template <int D, bool F32> struct TokenTile {
    static constexpr int ROW = D + 16 / (int)sizeof(Elem<F32>), UNITS = kChunk * D / 8 / 256;
    Frag<F32, 1> f[UNITS];
    __device__ __forceinline__ void load(const void *base, int64_t stride, int64_t t0, int rows, int head, int t) {
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
            const int u = t + 256 * n;
            f[n] = token_frag<F32>(base, stride, t0, rows, u / (D / 8), (int64_t)head * D + u % (D / 8) * 8);
        }
    }
    __device__ __forceinline__ void store(Elem<F32> *s, int t) const {
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
            const int u = t + 256 * n;
            Elem<F32> *p = s + u / (D / 8) * ROW + u % (D / 8) * 8;
            if constexpr (F32) {
                *reinterpret_cast<f4 *>(p) = f[n].v[0];
                *reinterpret_cast<f4 *>(p + 4) = f[n].v[1];
            } else {
                *reinterpret_cast<bf8 *>(p) = f[n].t[0];
            }
        }
    }
};
// ... as the operand [channel][token].
template <int D, bool F32> __device__ __forceinline__ void write_transposed(const Elem<F32> *s, Elem<F32> *out, int t) {
    constexpr int ROW = TokenTile<D, F32>::ROW;
    for (int u = t; u < D * 8; u += 256) {
        const int ch = (u >> 7) * 16 + (u & 15), k = (u >> 4 & 7) * 8;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = ld_elem<F32>(s, (k + i) * ROW + ch);
        Operand<F32, 1, 2>::put8(out, ch, k, x);
    }
}

// GDN: sums of the log-gates (in double: differences of sums lose nothing) and
// beta of one chunk, by the first wave: the loads, and what follows them.
struct GatesOf { float g, beta; };
template <bool F32> __device__ __forceinline__ GatesOf load_gates(const SeqArgs &a, int64_t t0, int rows, int h, int t) {
    GatesOf x{};
    if (t < rows) x = {ld_elem<F32>(a.g, (t0 + t) * a.n_heads + h), ld_elem<F32>(a.beta, (t0 + t) * a.n_heads + h)};
    return x;
}
__device__ __forceinline__ void gates_gdn(GatesOf x, int rows, double *sG, float *sBeta, int t) {
    if (t < kChunk) {
        double g = t < rows ? (double)floor_gate(x.g) : 0.;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const double up = __shfl_up(g, off);
            if (t >= off) g += up;
        }
        sG[t] = g;
        sBeta[t] = x.beta;
    }
}

// GDN: blocks (w, j <= w) of B and P; fq: the wave's queries, s: the chunk's keys.
template <int D, bool F32>
__device__ __forceinline__ void pairs_gdn(const Elem<F32> *s, const Frag<F32, 1> (&fq)[D / 32], const double *sG, f4 (&B)[4], f4 (&P)[4], int w, int l) {
    constexpr int KB = D / 32, ROW = TokenTile<D, F32>::ROW;
    const int r = l & 15, g8 = (l >> 4) * 8, g4 = (l >> 4) * 4;
    Frag<F32, 1> fk[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) fk[kb] = load_frag<F32, 1>(s + (16 * w + r) * ROW + 32 * kb + g8, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        B[j] = P[j] = f4{};
        if (j > w) continue;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const Frag<F32, 1> b = load_frag<F32, 1>(s + (16 * j + r) * ROW + 32 * kb + g8, 0);
            B[j] = mma<1>(fk[kb], b, B[j]);
            P[j] = mma<1>(fq[kb], b, P[j]);
        }
        const int col = 16 * j + r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * w + g4 + i;
            const float e = col <= row ? exp_of((float)(sG[row] - sG[col])) : 0.f;
            B[j][i] = col < row ? B[j][i] * e : 0.f;
            P[j][i] = col <= row ? P[j][i] * e : 0.f;
        }
    }
}

// One chunk of GDN, forward (K as [channel][token] once per key head, P, M, gates) or backward
// (Q as [channel][token] too, the transposes of P and M).
template <int D, bool F32, int N, bool BWD>
__device__ __forceinline__ void prepare_gdn(const SeqArgs &a, uint8_t *work, int64_t block, int64_t oP, int64_t oM, int64_t oKT, int64_t oQT, int64_t oGates) {
    typedef Elem<F32> E;
    typedef TokenTile<D, F32> Tile;
    constexpr int KB = D / 32;
    __shared__ union {
        __attribute__((aligned(16))) E k[kChunk * Tile::ROW];
        float B[kChunk * kBRow];  // after k was read
    } s;
    __shared__ __attribute__((aligned(16))) E sQ[BWD ? kChunk * Tile::ROW : 8];
    __shared__ __attribute__((aligned(16))) float sInv[4 * 320], sTurn[4 * 320], sBeta[kChunk];
    __shared__ double sG[kChunk];
    const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63;
    const int64_t x = blockIdx.x / (uint32_t)a.n_heads;
    const int h = blockIdx.x % (uint32_t)a.n_heads, share = a.n_heads / a.n_key_heads, hk = h / share;
    SeqSpan sp;
    const int32_t c = chunk_at(a, x, sp);
    if (c < 0) return;
    const int64_t t0 = sp.t0 + (int64_t)c * kChunk;
    const int rows = min(kChunk, sp.len - c * kChunk);
    uint8_t *out = work + (x * a.n_heads + h) * block;
    const bool first = h == hk * share;  // its block holds what the heads of a key head share

    Tile tk, tq;
    Frag<F32, 1> fq[KB];
    tk.load(a.k, a.k_stride, t0, rows, hk, t);
    if (BWD && first) tq.load(a.q, a.q_stride, t0, rows, hk, t);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
        fq[kb] = token_frag<F32>(a.q, a.q_stride, t0, rows, 16 * w + (l & 15), (int64_t)hk * D + kb * 32 + (l >> 4) * 8);
    gates_gdn(load_gates<F32>(a, t0, rows, h, t), rows, sG, sBeta, t);
    tk.store(s.k, t);
    if (BWD && first) tq.store(sQ, t);
    __syncthreads();
    f4 B[4], P[4];
    pairs_gdn<D, F32>(s.k, fq, sG, B, P, w, l);
    if (first) {
        write_transposed<D, F32>(s.k, reinterpret_cast<E *>(out + oKT), t);
        if (BWD) write_transposed<D, F32>(sQ, reinterpret_cast<E *>(out + oQT), t);
    }
    if (t < kChunk) {
        float *gt = reinterpret_cast<float *>(out + oGates);
        gt[t] = exp_of((float)sG[t]);
        gt[kChunk + t] = exp_of((float)(sG[kChunk - 1] - sG[t]));
        gt[2 * kChunk + t] = sBeta[t];
    }
    __syncthreads();
    solve_pairs<F32, N, BWD>(B, P, s.B, sBeta, sInv, sTurn + w * 320, reinterpret_cast<E *>(out + oP), reinterpret_cast<E *>(out + oM), w, l);
}

// ---- KDA.  Lane l of wave w holds token 16 w + l % 16, channels 32 kb + 8 (l / 16) .. + 7:
// an operand fragment's places, so what it decays is an operand as it stands.  Sums of log-gates
// over a 16-token block are scans over 16 lanes.

// Sum over the lanes of a group of 16 up to (from) this one.
template <int CTRL> __device__ __forceinline__ float add_dpp(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float scan_up(float x) {
    x = add_dpp<0x111>(x);
    x = add_dpp<0x112>(x);
    x = add_dpp<0x114>(x);
    return add_dpp<0x118>(x);
}
__device__ __forceinline__ float scan_after(float x) {  // without the lane itself
    x = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x101, 0xf, 0xf, true));
    x = add_dpp<0x101>(x);
    x = add_dpp<0x102>(x);
    x = add_dpp<0x104>(x);
    return add_dpp<0x108>(x);
}

// The diagonal block of B and P of a wave by each pair's own sum of log-gates, for gates too
// strong for a common reference: a lane holds D / 64 channels, sums over channels
// go across the wave.
template <int D, bool F32>
__device__ __forceinline__ void diagonal_kda(const SeqArgs &a, int64_t t0, int rows, int h, int hk, int w, int l, f4 &dk, f4 &dq) {
    constexpr int NC = D / 64;
    uint32_t g[NC][16], k[NC][16], q[NC][16];
    const int64_t first = t0 + 16 * w;
    const int n = rows - 16 * w;  // tokens of the block
    dk = dq = f4{};
    if (n <= 0) return;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int64_t tok = first + min(i, n - 1);
            g[c][i] = ld_raw<F32>(a.g, (tok * a.n_heads + h) * D + 64 * c + l);
            k[c][i] = ld_raw<F32>(a.k, tok * a.k_stride + (int64_t)hk * D + 64 * c + l);
            q[c][i] = ld_raw<F32>(a.q, tok * a.q_stride + (int64_t)hk * D + 64 * c + l);
        }
#pragma unroll 1
    for (int j = 0; j < min(n, 16); ++j) {
        float e[NC], kj[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            e[c] = 0.f;
            kj[c] = ld_elem<F32>(a.k, (first + j) * a.k_stride + (int64_t)hk * D + 64 * c + l);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < j || i >= n) continue;
            float sk = 0.f, sq = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (i > j) e[c] += floor_gate(of_raw<F32>(g[c][i]));
                const float x = kj[c] * exp_of(e[c]);
                sk = fmaf(x, of_raw<F32>(k[c][i]), sk);
                sq = fmaf(x, of_raw<F32>(q[c][i]), sq);
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

template <int D, bool F32, int N, bool BWD>
__device__ __forceinline__ void prepare_kda(const SeqArgs &a, uint8_t *work, int64_t block, int64_t oP, int64_t oM, int64_t oK, int64_t oQ, int64_t oKT, int64_t oQT,
                                            int64_t oGates) {
    typedef Elem<F32> E;
    constexpr int KB = D / 32, ZROW = D + 4;
    __shared__ union {
        __attribute__((aligned(16))) float z[kChunk * ZROW];  // [token][channel]
        float B[kChunk * kBRow];
    } s;
    __shared__ __attribute__((aligned(16))) float sInv[4 * 320], sTurn[4 * 320], sBeta[kChunk], sT[4 * D];  // sT: e^(a block's sum)
    const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63, r = l & 15, g8 = (l >> 4) * 8, g4 = (l >> 4) * 4;
    const int64_t x = blockIdx.x / (uint32_t)a.n_heads;
    const int h = blockIdx.x % (uint32_t)a.n_heads, hk = h / (a.n_heads / a.n_key_heads);
    SeqSpan sp;
    const int32_t c = chunk_at(a, x, sp);
    if (c < 0) return;
    const int64_t t0 = sp.t0 + (int64_t)c * kChunk;
    const int rows = min(kChunk, sp.len - c * kChunk);
    uint8_t *out = work + (x * a.n_heads + h) * block;

    Frag<F32, 1> rk[KB], rq[KB], rg[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const int at = kb * 32 + g8;
        rg[kb] = token_frag<F32>(a.g, (int64_t)a.n_heads * D, t0, rows, 16 * w + r, (int64_t)h * D + at);
        rk[kb] = token_frag<F32>(a.k, a.k_stride, t0, rows, 16 * w + r, (int64_t)hk * D + at);
        rq[kb] = token_frag<F32>(a.q, a.q_stride, t0, rows, 16 * w + r, (int64_t)hk * D + at);
    }
    if (t < kChunk) sBeta[t] = t < rows ? ld_elem<F32>(a.beta, (t0 + t) * a.n_heads + h) : 0.f;
    // e^L (the log-gates of the block up to the token), e^-L, k e^R (R: after the token) to LDS
    float eL[KB][8], iL[KB][8];
    bool weak = true;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        float g[8], k[8], z[8];
        widen(rg[kb], g);
        widen(rk[kb], k);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[i] = floor_gate(g[i]);
            const float L = scan_up(g[i]);
            eL[kb][i] = exp_of(L);
            iL[kb][i] = exp_of(fminf(-L, kBlockRange));
            weak &= L >= -kBlockRange;
            z[i] = k[i] * exp_of(scan_after(g[i]));
        }
        float *p = s.z + (16 * w + r) * ZROW + 32 * kb + g8;
        *reinterpret_cast<f4 *>(p) = f4{z[0], z[1], z[2], z[3]};
        *reinterpret_cast<f4 *>(p + 4) = f4{z[4], z[5], z[6], z[7]};
        if (r == 15) {
            p = sT + w * D + 32 * kb + g8;
            *reinterpret_cast<f4 *>(p) = f4{eL[kb][0], eL[kb][1], eL[kb][2], eL[kb][3]};
            *reinterpret_cast<f4 *>(p + 4) = f4{eL[kb][4], eL[kb][5], eL[kb][6], eL[kb][7]};
        }
    }
    const bool fast = __all(weak);
    __syncthreads();

    // ---- operands by token, and the pairs
    f4 B[4], P[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) B[j] = P[j] = f4{};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const int at = 32 * kb + g8;
        float k[8], q[8], kl[8], ql[8], m[8];
        widen(rk[kb], k);
        widen(rq[kb], q);
#pragma unroll
        for (int i = 0; i < 8; ++i) kl[i] = k[i] * eL[kb][i], ql[i] = q[i] * eL[kb][i], m[i] = 1.f;
        const Frag<F32, 3> fk = make_frag<F32, 3>(kl);
        const Frag<F32, N> fq = make_frag<F32, N>(ql);
        if (fast) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = k[i] * iL[kb][i];
            const Frag<F32, 3> fb = make_frag<F32, 3>(y);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j == w) B[j] = mma<3>(fk, fb, B[j]), P[j] = mma<N>(fq, fb, P[j]);
        }
        // blocks before this one, the nearest first: m grows into the decay in between
#pragma unroll
        for (int j = 2; j >= 0; --j) {
            if (j >= w) continue;
            float y[8], f[8];
            const float *p = s.z + (16 * j + r) * ZROW + at, *pt = sT + j * D + at;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = p[i] * m[i], f[i] = pt[i];
            const Frag<F32, 3> fb = make_frag<F32, 3>(y);
            B[j] = mma<3>(fk, fb, B[j]);
            P[j] = mma<N>(fq, fb, P[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] *= f[i];
        }
        // m is now the decay from the chunk's start to the block's
        if (BWD) {
            float y[8];
            const float *p = s.z + (16 * w + r) * ZROW + at;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = p[i];
            for (int b = w + 1; b < 4; ++b)
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= sT[b * D + at + i];
            Operand<F32, 3, KB>::put8(reinterpret_cast<E *>(out + oK), 16 * w + r, at, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) eL[kb][i] *= m[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) kl[i] *= m[i], ql[i] *= m[i];
            Operand<F32, 3, KB>::put8(reinterpret_cast<E *>(out + oK), 16 * w + r, at, kl);
            Operand<F32, N, KB>::put8(reinterpret_cast<E *>(out + oQ), 16 * w + r, at, ql);
        }
    }
    if (!fast) {
        f4 dk, dq;
        diagonal_kda<D, F32>(a, t0, rows, h, hk, w, l, dk, dq);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j == w) B[j] = dk, P[j] = dq;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * w + g4 + i, col = 16 * j + r;
            if (col >= row) B[j][i] = 0.f;
            if (col > row) P[j][i] = 0.f;
        }
    float *gt = reinterpret_cast<float *>(out + oGates);
    if (t < kChunk) gt[t] = sBeta[t];
    if (t < D) gt[kChunk + t] = sT[t] * sT[D + t] * sT[2 * D + t] * sT[3 * D + t];

    // ---- operands by channel, through LDS
    auto by_channel = [&](int64_t o, bool to_end) {
        for (int u = t; u < D * 8; u += 256) {
            const int ch = (u >> 7) * 16 + (u & 15), k8 = (u >> 4 & 7) * 8;
            float m = 1.f, v[8];
            if (to_end)
                for (int b = (k8 >> 4) + 1; b < 4; ++b) m *= sT[b * D + ch];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = s.z[(k8 + i) * ZROW + ch] * m;
            Operand<F32, 3, 2>::put8(reinterpret_cast<E *>(out + o), ch, k8, v);
        }
    };
    if (BWD) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                float y[8];
                widen(which ? rq[kb] : rk[kb], y);
                float *p = s.z + (16 * w + r) * ZROW + 32 * kb + g8;
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= eL[kb][i];
                *reinterpret_cast<f4 *>(p) = f4{y[0], y[1], y[2], y[3]};
                *reinterpret_cast<f4 *>(p + 4) = f4{y[4], y[5], y[6], y[7]};
            }
            __syncthreads();
            by_channel(which ? oQT : oKT, false);
        }
    } else {
        by_channel(oKT, true);
    }
    __syncthreads();
    solve_pairs<F32, N, BWD>(B, P, s.B, sBeta, sInv, sTurn + w * 320, reinterpret_cast<E *>(out + oP), reinterpret_cast<E *>(out + oM), w, l);
}

} // namespace sqk
