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

// 16 codes of BITS bits from consecutive bytes, as sign-extended bytes.
template <int BITS> struct Row16 { uint32_t w[BITS / 2]; };
template <int BITS> __device__ __forceinline__ int code_of(const Row16<BITS> &s, int n) {
    const int bit = n * BITS, k = bit >> 5, off = bit & 31;
    uint32_t x = s.w[k] >> off;
    if (off + BITS > 32) x |= s.w[k + 1] << (32 - off);
    return (int)(x << (32 - BITS)) >> (32 - BITS);
}

// Rows row0 .. + 3, columns 16 cg .. + 15 into LDS as [column][row] bytes.
template <int D, int BITS> __device__ __forceinline__ void unpack4x16(const uint8_t *p, int cg, int row0, uint32_t *sC) {
    constexpr int CW = D / 4 + 1, RB = D * BITS / 8;
    Row16<BITS> s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < BITS / 2; ++j) s[i].w[j] = reinterpret_cast<const uint32_t *>(p + i * RB + cg * 2 * BITS)[j];
#pragma unroll
    for (int n = 0; n < 16; ++n) {
        const uint32_t b = ((uint32_t)code_of<BITS>(s[0], n) & 255) | ((uint32_t)code_of<BITS>(s[1], n) & 255) << 8 |
                           ((uint32_t)code_of<BITS>(s[2], n) & 255) << 16 | (uint32_t)code_of<BITS>(s[3], n) << 24;
        sC[(16 * cg + n) * CW + row0 / 4] = b;
    }
}

template <int D, bool KDA, bool F32, bool YF32, bool POOL32>
__global__ __launch_bounds__(256) void window_kernel(WindowArgs a, HeadTable tab) {
    constexpr int MT = D / 16, NT = D / 64, KB = D / 32, GROW = D + 4, KROW = D + 8, CW = D / 4 + 1;
    constexpr int NQ = YF32 ? 3 : 2;
    __shared__ uint32_t sC[POOL32 ? 1 : D * CW];
    __shared__ float sL[kW * GROW], sR[kW * GROW];
    __shared__ uint16_t sK[3 * kW * KROW], sQ[NQ * kW * KROW];
    __shared__ float sOut[D * 20];  // keys decayed to the window's end, [channel][token]
    __shared__ float sM[16 * 20], sP[16 * 20], sB[16 * kBRow], sInv[16 * 20], sBeta[kW];
    __shared__ float sr[D], sc[D], sRange;
    const int t = threadIdx.x, w = t >> 6, l = t & 63, r = l & 15, g4 = (l >> 4) * 4, g8 = (l >> 4) * 8;
    const int b = blockIdx.x / (uint32_t)a.n_heads, h = blockIdx.x % (uint32_t)a.n_heads;
    const int hk = h / (a.n_heads / a.n_key_heads);
    const int L = a.length, len = a.lens ? min(max(a.lens[b], 0), L) : L;
    const int64_t slot = a.slot[b];

    // ---- the state: codes to LDS, scales
    uint32_t bits = 32, n4 = 0, n6 = 0;
    const uint8_t *rec = nullptr;
    if constexpr (!POOL32) {
        bits = tab.info[h] & 255, n4 = tab.info[h] >> 8 & 255, n6 = tab.info[h] >> 16 & 255;
        rec = a.base + slot * a.slot_stride + tab.off[h];
        if (bits != 16) {
            int64_t codes = (int64_t)D * D * bits / 8;
            if (bits == 0) codes = (int64_t)D * (4 * n4 + 6 * n6 + 8 * (D - n4 - n6)) / 8;
            if (t < D / 4 * (D / 16)) {
                const int cg = t % (D / 16), row0 = t / (D / 16) * 4;
                if (bits == 6) {
                    unpack4x16<D, 6>(rec + row0 * (D * 6 / 8), cg, row0, sC);
                } else if (bits == 4) {
                    unpack4x16<D, 4>(rec + row0 * (D * 4 / 8), cg, row0, sC);
                } else if (bits == 8) {
                    unpack4x16<D, 8>(rec + row0 * D, cg, row0, sC);
                } else if (row0 < (int)n4) {  // per-row widths: four rows share one
                    unpack4x16<D, 4>(rec + row0 * (D / 2), cg, row0, sC);
                } else if (row0 < (int)(n4 + n6)) {
                    unpack4x16<D, 6>(rec + n4 * (D / 2) + (row0 - n4) * (D * 6 / 8), cg, row0, sC);
                } else {
                    unpack4x16<D, 8>(rec + n4 * (D / 2) + n6 * (D * 6 / 8) + (row0 - n4 - n6) * D, cg, row0, sC);
                }
            }
            if (t < D) {
                sr[t] = reinterpret_cast<const float *>(rec + codes)[t];
                sc[t] = reinterpret_cast<const float *>(rec + codes)[D + t];
            }
        } else if (t < D) {
            sr[t] = sc[t] = 1.f;
        }
    } else if (t < D) {
        sr[t] = sc[t] = 1.f;
    }

    // ---- sums of the log-gates up to a token and after it
    if (t == 0) sRange = 0.f;
    const int64_t tok0 = (int64_t)b * L;
    if (t < D) {
        float g[kW], up = 0.f, down = 0.f;
#pragma unroll
        for (int i = 0; i < kW; ++i)
            g[i] = i < len ? fmaxf(ld_elem<F32>(a.g, ((tok0 + i) * a.n_heads + h) * (KDA ? D : 1) + (KDA ? t : 0)), kGateFloor) : 0.f;
#pragma unroll
        for (int i = 0; i < kW; ++i) up += g[i], sL[i * GROW + t] = up;
#pragma unroll
        for (int i = kW - 1; i >= 0; --i) sR[i * GROW + t] = down, down += g[i];
    }
    if (t < kW) sBeta[t] = t < len ? ld_elem<F32>(a.beta, (tok0 + t) * a.n_heads + h) : 0.f;
    __syncthreads();
    if (t < D) atomicMax(reinterpret_cast<int *>(&sRange), __float_as_int(fmaxf(-sL[(kW - 1) * GROW + t], 0.f)));

    // ---- the decayed keys and queries
    for (int u = t; u < kW * D / 8; u += 256) {
        const int i = u / (D / 8), c = u % (D / 8) * 8;
        float k[8] = {}, q[8] = {}, x[8];
        if (i < len) {
            const int64_t at = ((tok0 + i) * a.n_key_heads + hk) * D + c;
            widen(load_frag<F32, 1>(static_cast<const Elem<F32> *>(a.k) + at, 0), k);
            if (a.y) widen(load_frag<F32, 1>(static_cast<const Elem<F32> *>(a.q) + at, 0), q);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = exp_of(sL[i * GROW + c + j]) * sr[c + j];
            sOut[(c + j) * 20 + i] = k[j] * exp_of(sR[i * GROW + c + j]);
            x[j] = k[j] * d;
            q[j] *= d;
        }
        const Frag<false, 3> fk = make_frag<false, 3>(x);
        const Frag<false, NQ> fq = make_frag<false, NQ>(q);
#pragma unroll
        for (int p = 0; p < 3; ++p) *reinterpret_cast<bf8 *>(sK + p * kW * KROW + i * KROW + c) = fk.t[p];
#pragma unroll
        for (int p = 0; p < NQ; ++p) *reinterpret_cast<bf8 *>(sQ + p * kW * KROW + i * KROW + c) = fq.t[p];
    }
    __syncthreads();

    // ---- B and M (wave 0), P (wave 1): pairs of tokens
    if (w < 2) {
        const void *left = w == 0 ? a.k : a.q;
        f4 acc{};
        const bool fast = !KDA || sRange <= kBlockRange;
        auto row8 = [&](const void *p, int i, int c, float (&x)[8]) {
            if (i < len && (w == 0 || a.y))
                widen(load_frag<F32, 1>(static_cast<const Elem<F32> *>(p) + ((tok0 + i) * a.n_key_heads + hk) * D + c, 0), x);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = 0.f;
        };
        if (fast) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const int c = 32 * kb + g8;
                float x[8], y[8];
                row8(left, r, c, x);
                row8(a.k, r, c, y);
                if constexpr (KDA) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float e = sL[r * GROW + c + j];
                        x[j] *= exp_of(e);
                        y[j] *= exp_of(-e);
                    }
                }
                if constexpr (KDA || F32)
                    acc = mma<3>(make_frag<false, 3>(x), make_frag<false, 3>(y), acc);
                else
                    acc = mma<1>(make_frag<false, 1>(x), make_frag<false, 1>(y), acc);
            }
            if constexpr (!KDA) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // the smaller of the two differences that give the sum over (r, row]
                    const int row = g4 + i;
                    const float e = row < r ? 0.f : sL[row * GROW] - sL[r * GROW], f = row < r ? 0.f : sR[r * GROW] - sR[row * GROW];
                    acc[i] *= exp_of(sL[r * GROW] > sR[row * GROW] ? e : f);
                }
            }
        } else {
            for (int u = 0; u < 136; ++u) {
                int i = 0, j = u;
                while (j > i) j -= ++i;
                float s = 0.f;
                if (i < len) {
                    for (int c = l; c < D; c += 64) {
                        float e = 0.f;
                        for (int m = j + 1; m <= i; ++m) e += fmaxf(ld_elem<F32>(a.g, ((tok0 + m) * a.n_heads + h) * D + c), kGateFloor);
                        if (w == 0 || a.y)
                            s = fmaf(ld_elem<F32>(left, ((tok0 + i) * a.n_key_heads + hk) * D + c) * exp_of(e),
                                     ld_elem<F32>(a.k, ((tok0 + j) * a.n_key_heads + hk) * D + c), s);
                    }
                }
#pragma unroll
                for (int off = 32; off; off >>= 1) s += __shfl_xor(s, off);
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    if (g4 + n == i && r == j) acc[n] = s;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = g4 + i;
            if (w == 0) sB[row * kBRow + r] = r < row ? acc[i] : 0.f;
            else sP[row * 20 + r] = r <= row ? acc[i] : 0.f;
        }
    }
    __syncthreads();
    if (w == 0) {
        invert_block(sB, sBeta, sInv, 0, l);
        __builtin_amdgcn_wave_barrier();
        f4 nb;  // M = -(I + B diag(beta))^-1 B
#pragma unroll
        for (int i = 0; i < 4; ++i) nb[i] = -sB[(g4 + i) * kBRow + r];
        const f4 m = mma16(*reinterpret_cast<const f4 *>(sInv + r * 20 + g4), nb, f4{});
#pragma unroll
        for (int i = 0; i < 4; ++i) sM[(g4 + i) * 20 + r] = m[i];
    }

    // ---- the state's columns of this wave, in the result layout
    f4 S[NT][MT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int col = (w * NT + n) * 16 + r;
        if constexpr (POOL32) {
            const float *p = reinterpret_cast<const float *>(a.base) + slot * a.slot_stride + (int64_t)h * D * D + col;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[n][m][i] = p[(16 * m + g4 + i) * D];
        } else if (bits == 16) {
            const _Float16 *p = reinterpret_cast<const _Float16 *>(rec) + col;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[n][m][i] = (float)p[(16 * m + g4 + i) * D];
        } else {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint32_t x = sC[col * CW + 4 * m + (l >> 4)];
#pragma unroll
                for (int i = 0; i < 4; ++i) S[n][m][i] = (float)(int8_t)(x >> (8 * i));
            }
        }
    }

    // ---- look-up and read-out of every token
    f4 ks[NT], y[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) ks[n] = y[n] = f4{};
    auto products = [&](auto terms) {
        constexpr int N = decltype(terms)::value;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const Frag<false, 3> fk = get_tiles<3, KROW>(sK, r, kb, g4);
            const Frag<false, NQ> fq = get_tiles<NQ, KROW>(sQ, r, kb, g4);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const Frag<false, N> fs = tiles_frag<N>(S[n][2 * kb], S[n][2 * kb + 1]);
                ks[n] = mma<3>(fk, fs, ks[n]);
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
    __syncthreads();  // M

    const f4 fm = *reinterpret_cast<const f4 *>(sM + r * 20 + g4), fp = *reinterpret_cast<const f4 *>(sP + r * 20 + g4);
    const f4 beta = *reinterpret_cast<const f4 *>(sBeta + g4);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int col = (w * NT + n) * 16 + r;
        const float c = sc[col];
        f4 e;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = g4 + i;
            const float v = tok < len ? ld_elem<F32>(a.v, ((tok0 + tok) * a.n_heads + h) * D + col) : 0.f;
            e[i] = v - c * ks[n][i];
        }
        const f4 u = beta * mma16(fm, beta * e, e);
        if (a.y) {
            const f4 out = mma16(fp, u, y[n] * c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (g4 + i < L) st_elem<YF32>(a.y, ((tok0 + g4 + i) * a.n_heads + h) * D + col, g4 + i < len ? out[i] : 0.f);
        }
        if (a.S_out) {
            float *p = a.S_out + ((int64_t)b * a.n_heads + h) * D * D + col;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                f4 s;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * m + g4 + i;
                    // the product as sq_dequant_state rounds it
                    s[i] = exp_of(sL[(kW - 1) * GROW + row]) * (POOL32 ? S[n][m][i] : (float)(((double)S[n][m][i] * sr[row]) * c));
                }
                s = mma16(*reinterpret_cast<const f4 *>(sOut + (16 * m + r) * 20 + g4), u, s);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[(int64_t)(16 * m + g4 + i) * D] = s[i];
            }
        }
    }
}

template <int D, bool POOL32, bool KDA, bool F32, bool YF32>
hipError_t launch(const WindowArgs &a, const HeadTable &tab, hipStream_t stream) {
    hipLaunchKernelGGL((window_kernel<D, KDA, F32, YF32, POOL32>), dim3((uint32_t)a.n * a.n_heads), dim3(256), 0, stream, a, tab);
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
