// The gated Delta rule over a window of up to 16 tokens per request, read from
// the packed pool (or an fp32 one): the recurrent form for drafted tokens.
//
// The window is one chunk in the sense of sq_chunk.hip: a state is read once for
// all its tokens instead of once per token, and the tokens' look-ups and
// read-outs are one product each on the matrix cores.  With the state as
// S_ij = r_i code_ij c_j, codes of 4, 6 and 8 bits are exact in one bf16 term, r goes to the
// keys and c to the result:
//   (K e^G S)_tj = c_j sum_i (k_ti e^{G_ti} r_i) code_ij.
// A binary16 state takes two terms (exact), an fp32 state three.
//
// One workgroup per (request, head); wave w owns 16-column tiles of the
// state, all rows, in the matrix instruction's result layout, which is also the operand
// layout once the contracted axis is read in that order.  Codes get there
// through LDS: a lane unpacks 4 rows x 16 columns and writes the four rows'
// bytes of a column as one word.
//
// Measured (d 128, bf16, 48 heads, 6 bits): 512 requests of 5 tokens 212 us (453 MB, 2.1 TB/s), 8
// requests 8.9 us; KDA, 128 requests x 32 heads of up to 4 tokens with S_out, 133 us (343 MB, 2.6 TB/s).
// Bound by vector issue and latency: unpacking, the keys' terms and the window's small triangular
// products are 858 vector instructions of each wave at 5 tokens and 6 bits, issued in 0.68
// of the cycles of busy CUs; the matrix cores are busy in 0.27 of them (KDA with S_out: 0.31 and 0.30, two
// workgroups per CU).
#include "sq_prep.h"
#include "sq_window.h"

#include <type_traits>

namespace sqk {
namespace {

constexpr int kW = kWindowMax;  // 16 rows of the matrix instruction

// Eight LDS elements in the order of two result tiles: rows 4 g .. + 3 of tile
// 2 kb and of tile 2 kb + 1.
template <int N, int ROW> __device__ __forceinline__ Frag<false, N> get_tiles(const uint16_t *m, int row, int kb, int g4) {
    Frag<false, N> f;
#pragma unroll
    for (int p = 0; p < N; ++p) {
        const bf4 a = *reinterpret_cast<const bf4 *>(m + p * 16 * ROW + row * ROW + 32 * kb + g4);
        const bf4 b = *reinterpret_cast<const bf4 *>(m + p * 16 * ROW + row * ROW + 32 * kb + 16 + g4);
        f.t[p] = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return f;
}
template <int N> __device__ __forceinline__ Frag<false, N> tiles_frag(f4 a, f4 b) {
    const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return make_frag<false, N>(x);
}

// The codes of 4 rows x 16 columns as they lie in a record: 16 codes are
// bits / 2 words of a row.
struct Codes { uint32_t w[4][4]; };

template <int BITS> __device__ __forceinline__ int code_of(const uint32_t (&w)[4], int n) {
    const int bit = n * BITS, k = bit >> 5, off = bit & 31;
    uint32_t x = w[k] >> off;
    if (off + BITS > 32) x |= w[k + 1] << (32 - off);
    return (int)(x << (32 - BITS)) >> (32 - BITS);
}
template <int D, int BITS> __device__ __forceinline__ void load_codes(const uint8_t *p, int cg, Codes &c) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < BITS / 2; ++j) c.w[i][j] = reinterpret_cast<const uint32_t *>(p + i * (D * BITS / 8) + cg * 2 * BITS)[j];
}
// ... into LDS as [column][row] bytes, sign-extended: a word holds a column's four rows.
template <int D, int BITS> __device__ __forceinline__ void spread_codes(const Codes &c, int cg, int row0, uint32_t *sC) {
    constexpr int CW = D / 4 + 1;
#pragma unroll
    for (int n = 0; n < 16; ++n) {
        const uint32_t b = ((uint32_t)code_of<BITS>(c.w[0], n) & 255) | ((uint32_t)code_of<BITS>(c.w[1], n) & 255) << 8 |
                           ((uint32_t)code_of<BITS>(c.w[2], n) & 255) << 16 | (uint32_t)code_of<BITS>(c.w[3], n) << 24;
        sC[(16 * cg + n) * CW + row0 / 4] = b;
    }
}

// KEEP: S_out is wanted.  One thread per channel prepares the keys, one the
// queries, while all unpack; after one barrier each wave works alone: it forms the
// pairs of tokens for itself (16 x 16, cheaper than waiting for another wave).
template <int D, bool KDA, bool F32, bool YF32, bool POOL32, bool KEEP>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void window_kernel(WindowArgs a, HeadTable tab) {
    constexpr int MT = D / 16, NT = D / 64, KB = D / 32, EROW = D + 4, KROW = D + 8, CW = D / 4 + 1;
    // terms that y and the differences to v are accurate to; the latter the same whether or
    // not S_out is wanted, so that y is the same to the bit
    constexpr int NQ = YF32 ? 3 : 2, NK = 3;
    __shared__ uint32_t sC[POOL32 ? 1 : D * CW];
    __shared__ __attribute__((aligned(16))) uint16_t sK[NK * kW * KROW], sQ[NQ * kW * KROW];
    __shared__ __attribute__((aligned(16))) float sE[KDA ? 3 * kW * EROW : 4];  // keys times e^L, e^-L, queries times e^L
    __shared__ __attribute__((aligned(16))) float sOut[KEEP ? D * 20 : 4];      // keys decayed to the window's end, [channel][token]
    __shared__ __attribute__((aligned(16))) float sFade[KEEP ? D : 4], sr[KEEP ? D : 4];
    __shared__ __attribute__((aligned(16))) float sBeta[kW];
    __shared__ int sSlow[2];
    const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63, r = l & 15, g4 = (l >> 4) * 4, g8 = (l >> 4) * 8;
    // the waves' tiles to turn, in place of the keys once every wave has read them: GDN then has four workgroups
    // per CU for three (274 -> 234 us for 512 requests of 5 tokens), with S_out three for two
    float *tile = reinterpret_cast<float *>(sK) + w * 320;
    static_assert(sizeof(sK) >= 4 * 320 * sizeof(float), "");
    const int b = blockIdx.x / (uint32_t)a.n_heads, h = blockIdx.x % (uint32_t)a.n_heads;
    const int hk = h / (a.n_heads / a.n_key_heads);
    const int L = a.length, len = a.lens ? min(max(a.lens[b], 0), L) : L;
    const int64_t slot = a.slot[b], tok0 = (int64_t)b * L;

    uint32_t bits = 32, n4 = 0, n6 = 0;
    const uint8_t *rec = nullptr;
    int64_t codes = 0;
    if constexpr (!POOL32) {
        bits = tab.info[h] & 255, n4 = tab.info[h] >> 8 & 255, n6 = tab.info[h] >> 16 & 255;
        rec = a.base + slot * a.slot_stride + tab.off[h];
        codes = bits == 0 ? (int64_t)D * (4 * n4 + 6 * n6 + 8 * (D - n4 - n6)) / 8 : (int64_t)D * D * bits / 8;
    }
    const bool scaled = !POOL32 && bits != 16;

    // the raw keys and queries of token r for the pairs (GDN), the columns' scales
    Frag<F32, 1> rk[KDA ? 1 : KB], rq[KDA ? 1 : KB];
    if constexpr (!KDA) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int64_t at = ((tok0 + r) * a.n_key_heads + hk) * D + 32 * kb + g8;
            zero(rk[kb]), zero(rq[kb]);
            if (r < len) {
                rk[kb] = load_frag<F32, 1>(static_cast<const Elem<F32> *>(a.k) + at, 0);
                if (a.y) rq[kb] = load_frag<F32, 1>(static_cast<const Elem<F32> *>(a.q) + at, 0);
            }
        }
    }
    float cs[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) cs[n] = scaled ? reinterpret_cast<const float *>(rec + codes)[D + (w * NT + n) * 16 + r] : 1.f;
    f4 S[POOL32 ? NT : 1][POOL32 ? MT : 1];
    if constexpr (POOL32) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float *p = reinterpret_cast<const float *>(a.base) + slot * a.slot_stride + (int64_t)h * D * D + (w * NT + n) * 16 + r;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[n][m][i] = p[(16 * m + g4 + i) * D];
        }
    }

    // this thread's codes (D = 64: threads 128 .. 191); four rows share a width
    Codes raw;
    const int unit = D == 128 ? t : t - 128, cg = unit % (D / 16), row0 = unit / (D / 16) * 4;
    uint32_t width = 0;
    if constexpr (!POOL32)
        if (bits != 16 && unit >= 0 && unit < D / 4 * (D / 16)) {
            width = bits ? bits : row0 < (int)n4 ? 4 : row0 < (int)(n4 + n6) ? 6 : 8;
            const uint8_t *p = rec;
            if (bits == 0) {  // rows of 4, then of 6, then of 8 bits
                if (width == 4) p += row0 * (D / 2);
                else if (width == 6) p += n4 * (D / 2) + (row0 - n4) * (D * 6 / 8);
                else p += n4 * (D / 2) + n6 * (D * 6 / 8) + (row0 - n4 - n6) * D;
            } else {
                p += row0 * (D / 8) * bits;
            }
            if (width == 6) load_codes<D, 6>(p, cg, raw);
            else if (width == 4) load_codes<D, 4>(p, cg, raw);
            else load_codes<D, 8>(p, cg, raw);
        }

    // ---- a thread per channel: the decayed keys (threads below D), the decayed queries (the next D)
    const int ch = t % D;
    const bool keys = t < D;
    uint32_t rg[KDA ? kW : 1] = {}, rx[kW] = {}, rv[NT][4];
    if constexpr (!KDA) rg[0] = ld_raw<F32>(a.g, (tok0 + min(r, L - 1)) * a.n_heads + h);
    {
        const void *src = keys || !a.y ? a.k : a.q;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            if (i % 4 == 0 && i >= len) break;
            // past the last token: that one again, its value is not used
            const int64_t tok = tok0 + min(i, len - 1);
            if constexpr (KDA) rg[i] = ld_raw<F32>(a.g, (tok * a.n_heads + h) * D + ch);
            rx[i] = ld_raw<F32>(src, (tok * a.n_key_heads + hk) * D + ch);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                rv[n][i] = ld_raw<F32>(a.v, ((tok0 + min(g4 + i, L - 1)) * a.n_heads + h) * D + (w * NT + n) * 16 + r);
    }
    const uint32_t rbeta = t < kW ? ld_raw<F32>(a.beta, (tok0 + min(t, L - 1)) * a.n_heads + h) : 0;
    const float scale = scaled ? reinterpret_cast<const float *>(rec + codes)[ch] : 1.f;

    // ---- pairs of tokens (GDN): B and P in the result layout, and the sum of the
    // log-gates up to token r in every lane, in double: differences of sums lose nothing
    f4 kk{}, qk{};
    double up = 0.;
    float eup = 1.f, edown = 1.f;  // the decay up to token r and after it
    if constexpr (!KDA) {
        up = r < len ? (double)floor_gate(of_raw<F32>(rg[0])) : 0.;
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) {
            const double x = __shfl_up(up, off, 16);
            if (r >= off) up += x;
        }
        eup = exp_of((float)up), edown = exp_of((float)(__shfl(up, 15, 16) - up));
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            if constexpr (F32) {
                float x[8];
                widen(rk[kb], x);
                const Frag<false, 3> fk = make_frag<false, 3>(x);
                widen(rq[kb], x);
                kk = mma<3>(fk, fk, kk);
                qk = mma<3>(make_frag<false, 3>(x), fk, qk);
            } else {
                kk = mma<1>(rk[kb], rk[kb], kk);
                qk = mma<1>(rq[kb], rk[kb], qk);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = g4 + i;
            const double to = __shfl(up, row, 16);
            const float d = exp_of(row < len && r <= row ? (float)(to - up) : 0.f);
            kk[i] *= d, qk[i] *= d;
        }
    }

    if (t < 2 * D) {
        float sum = 0.f, low = 0.f;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            if (i >= len) break;
            float e, x = of_raw<F32>(rx[i]);
            if constexpr (KDA) {
                sum += floor_gate(of_raw<F32>(rg[i]));
                low = fminf(low, sum);  // not the last sum alone: a gate above 1 may raise it again
                e = x * exp_of(sum);
            } else {
                e = x * __shfl(eup, i, 16);
            }
            __bf16 v[3];
            split<3>(e * scale, v);
            __bf16 *at = reinterpret_cast<__bf16 *>(keys ? sK : sQ) + i * KROW + ch;
#pragma unroll
            for (int p = 0; p < 3; ++p)
                if (p < (keys ? NK : NQ)) at[p * kW * KROW] = v[p];
            if constexpr (KDA) {
                sE[(keys ? 0 : 2) * kW * EROW + i * EROW + ch] = e;
                if (keys) sE[kW * EROW + i * EROW + ch] = x * exp_of(-sum);
            } else if (KEEP && keys) {
                sOut[ch * 20 + i] = x * __shfl(edown, i, 16);
            }
        }
        if (KDA && keys) {
            const bool slow = __any(low < -kBlockRange);
            if (l == 0) sSlow[w] = slow;
        }
        if constexpr (KEEP) {
            if (keys) {
                if constexpr (KDA) {
                    float after = 0.f;
#pragma unroll
                    for (int i = kW - 1; i >= 0; --i) {
                        if (i >= len) continue;
                        sOut[ch * 20 + i] = of_raw<F32>(rx[i]) * exp_of(after);
                        after += floor_gate(of_raw<F32>(rg[i]));
                    }
                }
                for (int i = len; i < kW; ++i) sOut[ch * 20 + i] = 0.f;
                sFade[ch] = KDA ? exp_of(sum) : __shfl(eup, 15, 16), sr[ch] = scale;
            }
        }
    }
    if (t < kW) sBeta[t] = t < len ? of_raw<F32>(rbeta) : 0.f;
    if constexpr (!POOL32) {
        if (width == 6) spread_codes<D, 6>(raw, cg, row0, sC);
        else if (width == 4) spread_codes<D, 4>(raw, cg, row0, sC);
        else if (width == 8) spread_codes<D, 8>(raw, cg, row0, sC);
    }
    __syncthreads();

    // a tile of the state in the result layout: rows 16 m + 4 (l / 16) .. + 3 of this wave's columns
    auto state = [&](int n, int m) {
        if constexpr (POOL32) {
            return S[n][m];
        } else {
            const int col = (w * NT + n) * 16 + r;
            f4 x;
            if (bits == 16) {
                const _Float16 *p = reinterpret_cast<const _Float16 *>(rec) + col;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = (float)p[(16 * m + g4 + i) * D];
            } else {
                const uint32_t c = sC[col * CW + 4 * m + (l >> 4)];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(c >> (8 * i));
            }
            return x;
        }
    };

    // ---- look-up and read-out of every token
    f4 ks[NT], y[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) ks[n] = y[n] = f4{};
    auto products = [&](auto terms) {
        constexpr int N = decltype(terms)::value;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const Frag<false, NK> fk = get_tiles<NK, KROW>(sK, r, kb, g4);
            const Frag<false, NQ> fq = get_tiles<NQ, KROW>(sQ, r, kb, g4);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const Frag<false, N> fs = tiles_frag<N>(state(n, 2 * kb), state(n, 2 * kb + 1));
                ks[n] = mma<NK>(fk, fs, ks[n]);
                y[n] = mma<NQ>(fq, fs, y[n]);
            }
        }
    };
    if constexpr (POOL32) {
        products(std::integral_constant<int, 3>());
    } else {
        if (bits == 16) products(std::integral_constant<int, 2>());
        else products(std::integral_constant<int, 1>());
    }

    // ---- pairs of tokens (KDA)
    if constexpr (!KDA) {
    } else if (!(sSlow[0] | (D == 128 ? sSlow[1] : 0))) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int at = r * EROW + 16 * m + g4;
            const f4 inv = *reinterpret_cast<const f4 *>(sE + kW * EROW + at);
            kk = mma16(*reinterpret_cast<const f4 *>(sE + at), inv, kk);
            qk = mma16(*reinterpret_cast<const f4 *>(sE + 2 * kW * EROW + at), inv, qk);
        }
    } else {  // strong gates: each pair by its own sum of log-gates
        for (int j = 0; j < len; ++j) {
            float e[D / 64], kj[D / 64];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                e[c] = 0.f;
                kj[c] = ld_elem<F32>(a.k, ((tok0 + j) * a.n_key_heads + hk) * D + 64 * c + l);
            }
            for (int i = j; i < len; ++i) {
                float sk = 0.f, sq = 0.f;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    if (i > j) e[c] += floor_gate(ld_elem<F32>(a.g, ((tok0 + i) * a.n_heads + h) * D + 64 * c + l));
                    const int64_t at = ((tok0 + i) * a.n_key_heads + hk) * D + 64 * c + l;
                    const float x = kj[c] * exp_of(e[c]);
                    sk = fmaf(x, ld_elem<F32>(a.k, at), sk);
                    if (a.y) sq = fmaf(x, ld_elem<F32>(a.q, at), sq);
                }
#pragma unroll
                for (int off = 32; off; off >>= 1) sk += __shfl_xor(sk, off), sq += __shfl_xor(sq, off);
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    if (g4 + n == i && r == j) kk[n] = sk, qk[n] = sq;
            }
        }
    }
    __syncthreads();
    // M = -B - N M with N = B diag(beta), by forward substitution, four tokens at a time: a lane holds the four rows of
    // its column, what later rows take of them is one product.  (I - N)(I + N^2)(I + N^4)(I + N^8) for (I + N)^-1 is
    // not good enough: for keys that resemble each other its partial products grow and cancel, which costs 16 tokens
    // two digits.
    const f4 beta = *reinterpret_cast<const f4 *>(sBeta + g4);
    f4 m;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = g4 + i;
        const float x = row < len && r < row ? kk[i] : 0.f;
        m[i] = -x;
        tile[row * 20 + r] = x * sBeta[r];
        if (!(row < len && r <= row)) qk[i] = 0.f;
    }
    __builtin_amdgcn_wave_barrier();
    const f4 later = -*reinterpret_cast<const f4 *>(tile + r * 20 + g4);
    f4 own[4];  // -N within these four tokens
#pragma unroll
    for (int i = 1; i < 4; ++i) own[i] = -*reinterpret_cast<const f4 *>(tile + (g4 + i) * 20 + g4);
    __builtin_amdgcn_wave_barrier();
    auto within = [&](f4 x) {
        x[1] = fmaf(own[1][0], x[0], x[1]);
        x[2] = fmaf(own[2][1], x[1], fmaf(own[2][0], x[0], x[2]));
        x[3] = fmaf(own[3][2], x[2], fmaf(own[3][1], x[1], fmaf(own[3][0], x[0], x[3])));
        return x;
    };
#pragma unroll
    for (int J = 0; J < 3; ++J) {
        if (4 * J + 4 >= len) break;
        m = mma16(g4 == 4 * J && r >= 4 * J + 4 ? later : f4{}, within(m), m);
    }
    m = within(m);
    const f4 fm = turn(tile, m, l), fp = turn(tile, qk, l);

#pragma unroll
    for (int n = 0; n < NT; ++n) {
        f4 e;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = g4 + i;
            e[i] = tok < len ? of_raw<F32>(rv[n][i]) - cs[n] * ks[n][i] : 0.f;
            y[n][i] = tok < len ? y[n][i] * cs[n] : 0.f;
        }
        const f4 u = beta * mma16(fm, beta * e, e);
        if (a.y) {
            const f4 out = turn(tile, mma16(fp, u, y[n]), l);
            if (r < L) st_elem4<YF32>(a.y, ((tok0 + r) * a.n_heads + h) * D + (w * NT + n) * 16 + g4, out);
        }
        if constexpr (KEEP) {
            float *p = a.S_out + ((int64_t)b * a.n_heads + h) * D * D + (w * NT + n) * 16 + g4;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const f4 s0 = state(n, m);
                f4 s;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * m + g4 + i;
                    // the product as sq_dequant_state rounds it
                    s[i] = sFade[row] * (POOL32 ? s0[i] : (float)(((double)s0[i] * sr[row]) * cs[n]));
                }
                s = mma16(*reinterpret_cast<const f4 *>(sOut + (16 * m + r) * 20 + g4), u, s);
                *reinterpret_cast<f4 *>(p + (int64_t)(16 * m + r) * D) = turn(tile, s, l);
            }
        }
    }
}

template <int D, bool POOL32, bool KDA, bool F32, bool YF32>
hipError_t launch(const WindowArgs &a, const HeadTable &tab, hipStream_t stream) {
    const dim3 grid((uint32_t)a.n * a.n_heads);
    if (a.S_out) hipLaunchKernelGGL((window_kernel<D, KDA, F32, YF32, POOL32, true>), grid, dim3(256), 0, stream, a, tab);
    else hipLaunchKernelGGL((window_kernel<D, KDA, F32, YF32, POOL32, false>), grid, dim3(256), 0, stream, a, tab);
    return hipGetLastError();
}

template <int D, bool POOL32, bool KDA>
hipError_t window_types(const WindowArgs &a, const HeadTable &tab, bool f32, bool y_f32, hipStream_t stream) {
    if (f32) return y_f32 ? launch<D, POOL32, KDA, true, true>(a, tab, stream) : launch<D, POOL32, KDA, true, false>(a, tab, stream);
    return y_f32 ? launch<D, POOL32, KDA, false, true>(a, tab, stream) : launch<D, POOL32, KDA, false, false>(a, tab, stream);
}

template <int D, bool POOL32>
hipError_t window(const WindowArgs &a, const HeadTable &tab, bool kda, bool f32, bool y_f32, hipStream_t stream) {
    return kda ? window_types<D, POOL32, true>(a, tab, f32, y_f32, stream) : window_types<D, POOL32, false>(a, tab, f32, y_f32, stream);
}

} // namespace

hipError_t launch_window(const WindowArgs &a, const HeadTable *tab, int d, bool kda, bool f32, bool y_f32, hipStream_t stream) {
    static const HeadTable none{};
    if (tab) return d == 128 ? window<128, false>(a, *tab, kda, f32, y_f32, stream) : window<64, false>(a, *tab, kda, f32, y_f32, stream);
    return d == 128 ? window<128, true>(a, none, kda, f32, y_f32, stream) : window<64, true>(a, none, kda, f32, y_f32, stream);
}

} // namespace sqk
