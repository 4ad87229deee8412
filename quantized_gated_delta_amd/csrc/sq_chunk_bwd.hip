// Gradients of the chunked gated Delta rule (sq_chunk.hip, sq_prep.h for the notation).
//
// With dY the gradient of y and dS_C that of a chunk's final state,
//   dU  = P^T dY + (K e^{G_C - G}) dS_C
//   dF  = dU + M^T diag(beta) dU            dV = diag(beta) dF     dbeta_i = E_i . dF_i
//   dS0 = diag(e^{G_C}) dS_C + (Q e^G)^T dY - (K e^G)^T dV
//   dP  = dY U^T (j <= i)                   dB = -dV U^T (j < i)
//   dq_i = e^{G_i} dY_i S0^T + sum_j dP_ij k_j e^{G_i - G_j}
//   dk   = row + col,  row_i = -e^{G_i} dV_i S0^T + sum_{j<i} dB_ij k_j e^{G_i - G_j}
//                      col_j = e^{G_C - G_j} U_j dS_C^T + sum_{i>j} dB_ij k_i e^{G_i - G_j}
//                                                        + sum_{i>=j} dP_ij q_i e^{G_i - G_j}
//   dg_t = sum_{i >= t} X_i + sum_{j < t} Z_j + e^{G_C} rowsum(S0 dS_C)   (GDN: summed over channels)
//     Z_j = k_j (the first term of col_j),  X_i = q_i dq_i + k_i (row_i - the other terms of col_i)
// dF needs no division by beta: M has no beta on its left.  A pair (i, i) has no decay:
// it is left out of X, where it would stand with both signs, and what runs to the chunk's
// end is summed from the front, so that strong gates (small dg) keep their accuracy.
//
// Three kernels: the operands (prep, all chunks in parallel), a scan from the last
// chunk to the first that carries dS and leaves dV and each chunk's dS, shaped like the forward
// scan (16 columns of the state per workgroup, rows over its four waves), and
// the gradients of q, k, beta and g (all chunks in parallel), which read the states that
// the forward pass saved.  The heads that share a key head are added up in the
// registers of one workgroup: in a fixed order, without another pass.
//
// Measured (d 128, bf16): GDN, 8192 tokens in 4 sequences, 32 heads on 16 key heads, 68 + 384 + 291 us;
// KDA, 4001 tokens in 3, 32 heads, 111 + 277 + 224 us.  The scan is bound as the
// forward one.  The gradients move 1.46 GB (GDN) and 0.64 GB: 5.0 TB/s of the 5.8 that a copy
// reaches, and 2.9 TB/s, where the latency of the products between tokens is the rest.
#include "sq_prep.h"

namespace sqk {
namespace {

template <int D, bool F32> __global__ __launch_bounds__(256) void prep_gdn_bwd_kernel(SeqArgs a) {
    constexpr BackwardLayout lay = backward_layout(D, false, F32);
    prepare_gdn<D, F32, 3, true>(a, a.work, lay.block, lay.PT, lay.MT, lay.KT, lay.QT, lay.gates);
}

template <int D, bool F32> __global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void prep_kda_bwd_kernel(SeqArgs a) {
    constexpr BackwardLayout lay = backward_layout(D, true, F32);
    prepare_kda<D, F32, 3, true>(a, a.work, lay.block, lay.PT, lay.MT, lay.K, 0, lay.KT, lay.QT, lay.gates);
}

// One (sequence, head), 16 NCT columns of the state's gradient, all chunks backwards.
template <int D, bool KDA, bool F32, int NCT> __global__ __launch_bounds__(256) void scan_bwd_kernel(SeqArgs a) {
    typedef Elem<F32> E;
    constexpr BackwardLayout lay = backward_layout(D, KDA, F32);
    constexpr SaveLayout save = save_layout(D);
    constexpr int MT = D / 64, KB = D / 32, COLS = 16 * NCT, SLICES = D / COLS, KN = KDA ? 3 : 1;
    typedef LdsMat<F32, 3, D, COLS> SMat;
    typedef LdsMat<F32, 3, kChunk, COLS> XMat;
    typedef LdsMat<F32, 1, kChunk, COLS> YMat;
    constexpr int GY = KDA ? 0 : XMat::BYTES;
    __shared__ __attribute__((aligned(16))) uint8_t lds[SMat::BYTES + 2 * XMat::BYTES + 2 * YMat::BYTES + GY];
    __shared__ __attribute__((aligned(16))) float sTurn[4 * 320];
    E *sS = reinterpret_cast<E *>(lds), *sX = reinterpret_cast<E *>(lds + SMat::BYTES);
    E *sU = reinterpret_cast<E *>(lds + SMat::BYTES + XMat::BYTES);
    E *sYg = reinterpret_cast<E *>(lds + SMat::BYTES + 2 * XMat::BYTES + 2 * YMat::BYTES);

    const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63, r = l & 15, g4 = (l >> 4) * 4, g8 = (l >> 4) * 8;
    float *tile = sTurn + w * 320;
    const uint32_t pairs = (uint32_t)a.n_seq * a.n_heads, j = blockIdx.x >> 3;
    const uint32_t pair = j / SLICES * 8 + (blockIdx.x & 7);
    if (pair >= pairs) return;
    const int c0 = (int)(j % SLICES) * COLS;
    const int h = pair % (uint32_t)a.n_heads, share = a.n_heads / a.n_key_heads, hk = h / share;
    const SeqSpan sp = wave_span(a, pair / (uint32_t)a.n_heads);
    const int n_chunks = (sp.len + kChunk - 1) / kChunk;
    const int64_t state = (int64_t)pair * D * D;

    f4 S[MT][NCT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NCT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                S[m][n][i] = a.dS_out ? a.dS_out[state + (int64_t)((w * MT + m) * 16 + g4 + i) * D + c0 + 16 * n + r] : 0.f;

    Frag<F32, KN> fK[KB], fKT[MT][2], fQT[MT][2];
    Frag<F32, 3> fM[2], fP[2];
    uint32_t rdy[NCT][4];  // as loaded: widening them at once would wait for them at once
    Raw4<F32, kSaveTerms> fe[NCT];
    struct Gates { f4 eg, ec, beta, fade[MT]; float fade1; } gt{}, gt_next{};

    auto block_of = [&](int c, int head) { return a.work + ((sp.slot0 + c) * a.n_heads + head) * lay.block; };
    auto rows_of = [&](int c) { return min(kChunk, sp.len - c * kChunk); };
    auto load_k = [&](int c) {
        if constexpr (KDA) {
            const E *b = reinterpret_cast<const E *>(block_of(c, h) + lay.K);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) fK[kb] = Operand<F32, KN, KB>::get(b, w, kb, l);
        } else {
            // past the end: the last token again; its beta is 0, so its dV is 0 too
            const void *pk = static_cast<const E *>(a.k) + (sp.t0 + (int64_t)c * kChunk) * a.k_stride + (int64_t)hk * D;
            const uint32_t row = min(16 * w + r, rows_of(c) - 1);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
                fK[kb] = load_frag<F32, KN>(at_bytes<E>(pk, (row * (uint32_t)a.k_stride + kb * 32 + g8) * (uint32_t)sizeof(E)), 0);
        }
    };
    auto load_dy = [&](int c) {
        const int rows = rows_of(c);
        const void *py = static_cast<const E *>(a.dy) + ((sp.t0 + (int64_t)c * kChunk) * a.n_heads + h) * D + c0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * w + g4 + i;
            const uint32_t at = min(row, rows - 1) * (uint32_t)(a.n_heads * D) + r;
#pragma unroll
            for (int n = 0; n < NCT; ++n) rdy[n][i] = ld_raw<F32>(at_bytes<E>(py, (at + 16 * n) * (uint32_t)sizeof(E)), 0);
        }
    };
    auto load_e = [&](int c) {
        const E *b = reinterpret_cast<const E *>(a.save + ((sp.slot0 + c) * a.n_heads + h) * save.block + save.E);
#pragma unroll
        for (int n = 0; n < NCT; ++n) fe[n] = get_operand4<F32, kSaveTerms, KB>(b, 16 * w + r, c0 + 16 * n + g4);
    };
    auto load_gates = [&](int c) {
        const float *p = reinterpret_cast<const float *>(block_of(c, h) + lay.gates);
        Gates x{};
        if constexpr (KDA) {
            x.beta = *reinterpret_cast<const f4 *>(p + 16 * w + g4);
#pragma unroll
            for (int m = 0; m < MT; ++m) x.fade[m] = *reinterpret_cast<const f4 *>(p + kChunk + (w * MT + m) * 16 + g4);
        } else {
            x.eg = *reinterpret_cast<const f4 *>(p + 16 * w + g4);
            x.ec = *reinterpret_cast<const f4 *>(p + kChunk + 16 * w + g4);
            x.beta = *reinterpret_cast<const f4 *>(p + 2 * kChunk + 16 * w + g4);
            x.fade1 = p[kChunk - 1];
        }
        return x;
    };
    // M^T and P^T: nothing left of the diagonal
    auto load_m = [&](int c) {
        const E *b = reinterpret_cast<const E *>(block_of(c, h) + lay.MT);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (kb == 1 || w < 2) fM[kb] = Operand<F32, 3, 2>::get(b, w, kb, l);
    };
    auto load_p = [&](int c) {
        const E *b = reinterpret_cast<const E *>(block_of(c, h) + lay.PT);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (kb == 1 || w < 2) fP[kb] = Operand<F32, 3, 2>::get(b, w, kb, l);
    };
    auto load_t = [&](int c) {
        const uint8_t *b = block_of(c, KDA ? h : hk * share);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                fKT[m][kb] = Operand<F32, KN, 2>::get(reinterpret_cast<const E *>(b + lay.KT), w * MT + m, kb, l);
                fQT[m][kb] = Operand<F32, KN, 2>::get(reinterpret_cast<const E *>(b + lay.QT), w * MT + m, kb, l);
            }
    };
    const int last = n_chunks - 1;
    if (n_chunks > 0) gt = load_gates(last), load_dy(last), load_k(last), load_p(last), load_m(last), load_e(last), load_t(last);

    // KDA's operands of the chunk after next to L2, a share by each slice, as in the forward scan
    const uint32_t part = j % SLICES;
    constexpr uint32_t kLines = (lay.dS + 127) / 128, kTouch = KDA ? (kLines + 256 * SLICES - 1) / (256 * SLICES) : 0;
    uint32_t touched[kTouch + 1] = {};
    auto touch = [&](int c) {
#pragma unroll
        for (uint32_t i = 0; i < kTouch; ++i) {
            const uint32_t line = (t + 256 * i) * SLICES + part;
            if (line < kLines) touched[i] = *at_bytes<uint32_t>(block_of(c, h), line * 128);
        }
    };
    for (int c = last; c >= 0; --c) {
        const int next = max(c - 1, 0), rows = rows_of(c);
        uint8_t *blk = block_of(c, h);
        // two places in turn: the last chunk's may still be read
        E *sY = reinterpret_cast<E *>(lds + SMat::BYTES + 2 * XMat::BYTES + (c & 1) * YMat::BYTES);
        gt_next = load_gates(next);
        f4 dy[NCT];
#pragma unroll
        for (int n = 0; n < NCT; ++n) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                SMat::put4(sS, 16 * n + r, (w * MT + m) * 16 + g4, S[m][n]);
                put_operand4<F32, kSaveTerms, KB>(reinterpret_cast<E *>(blk + lay.dS), (w * MT + m) * 16 + r, c0 + 16 * n + g4, turn(tile, S[m][n], l));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) dy[n][i] = 16 * w + g4 + i < rows ? of_raw<F32>(rdy[n][i]) : 0.f;
            YMat::put4(sY, 16 * n + r, 16 * w + g4, dy[n]);
        }
        __syncthreads();
        f4 du[NCT];
#pragma unroll
        for (int n = 0; n < NCT; ++n) {
            du[n] = f4{};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) du[n] = mma<3>(fK[kb], SMat::get(sS, 16 * n + r, kb * 32 + g8), du[n]);
            if (!KDA) du[n] *= gt.ec;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (kb == 1 || w < 2) du[n] = mma<3>(fP[kb], YMat::get(sY, 16 * n + r, kb * 32 + g8), du[n]);
            XMat::put4(sX, 16 * n + r, 16 * w + g4, du[n] * gt.beta);
            if constexpr (!KDA) XMat::put4(sYg, 16 * n + r, 16 * w + g4, dy[n] * gt.eg);
        }
        load_k(next);
        load_p(next);
        load_dy(next);
        __syncthreads();
        float db = 0.f;
        E *pv = static_cast<E *>(a.dv) + ((sp.t0 + (int64_t)c * kChunk) * a.n_heads + h) * D + c0;
#pragma unroll
        for (int n = 0; n < NCT; ++n) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (kb == 1 || w < 2) du[n] = mma<3>(fM[kb], XMat::get(sX, 16 * n + r, kb * 32 + g8), du[n]);  // dF
            const f4 dv = du[n] * gt.beta;
            XMat::put4(sU, 16 * n + r, 16 * w + g4, KDA ? -dv : -(dv * gt.eg));
            const f4 df = turn(tile, du[n], l), tv = turn(tile, dv, l), e = sum_of(fe[n]);
#pragma unroll
            for (int i = 0; i < 4; ++i) db = fmaf(df[i], e[i], db);
            put_operand4<F32, kSaveTerms, KB>(reinterpret_cast<E *>(blk + lay.dV), 16 * w + r, c0 + 16 * n + g4, tv);
            if (16 * w + r < rows)
                st_elem4<F32>(at_bytes<char>(pv, ((16 * w + r) * (uint32_t)(a.n_heads * D) + 16 * n + g4) * (uint32_t)sizeof(E)), 0, tv);
        }
        db += __shfl_xor(db, 16);
        db += __shfl_xor(db, 32);
        if (l < 16) reinterpret_cast<float *>(blk + lay.dbeta)[c0 / COLS * kChunk + 16 * w + r] = db;
        load_m(next);
        load_e(next);
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NCT; ++n) {
                S[m][n] = KDA ? S[m][n] * gt.fade[m] : S[m][n] * gt.fade1;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    if constexpr (KDA) S[m][n] = mma<3>(fQT[m][kb], YMat::get(sY, 16 * n + r, kb * 32 + g8), S[m][n]);
                    else S[m][n] = mma<3>(fQT[m][kb], XMat::get(sYg, 16 * n + r, kb * 32 + g8), S[m][n]);
                    S[m][n] = mma<3>(fKT[m][kb], XMat::get(sU, 16 * n + r, kb * 32 + g8), S[m][n]);
                }
            }
        load_t(next);
#pragma unroll
        for (uint32_t i = 0; i < kTouch; ++i) asm volatile("" ::"v"(touched[i]));  // so that the loads are not dropped
        touch(max(c - 2, 0));
        gt = gt_next;
    }
    if (a.dS0)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NCT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a.dS0[state + (int64_t)((w * MT + m) * 16 + g4 + i) * D + c0 + 16 * n + r] = S[m][n][i];
}

// Gradients of q, k, beta and g of one chunk and key head.  Wave w: tokens 16 w .. + 15, whose
// dY, dV and E stay in registers while the states go by, 16 channels at a time.
// SLICES: the parts of beta's gradient that the scan left.
//
// GDN: the decayed dP and dB as bf16 pairs in registers against the keys and
// queries by channel.  All that the four waves share goes once from memory through the LDS,
// asked for two steps before it is used, so that two workgroups share a CU (each wave
// its own loads, one workgroup: 451 us for 8192 tokens x 32 heads, d 128; this 291 us, 5.0 TB/s).
template <int D, bool F32> struct GradLds {
    static constexpr int STATE = 64 * D, TOKENS = F32 ? 4096 : 2048;  // bytes of 16 channels
    static constexpr int SLOT = 2 * STATE + 2 * TOKENS;               // S0, dS, keys, queries
    static constexpr int TURN = 4 * 320, PAIRS = 2 * kChunk * kBRow;
    static_assert(PAIRS >= TURN && 2 * SLOT >= 4 * STATE, "");
    // dP and dB, then each wave's tile to turn; E, then two slots
    __attribute__((aligned(16))) float pairs[PAIRS];
    __attribute__((aligned(16))) uint8_t slots[2 * SLOT];
    __attribute__((aligned(16))) float beta[kChunk], diag[kChunk], in[kChunk], to[kChunk], X[kChunk], Z[kChunk], end[4];
    double G[kChunk];
};

template <int D, bool F32, int SLICES>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(F32 && D == 128 ? 1 : 2))) void grad_gdn_kernel(SeqArgs a) {
    typedef Elem<F32> E;
    constexpr BackwardLayout lay = backward_layout(D, false, F32);
    constexpr SaveLayout save = save_layout(D);
    typedef GradLds<D, F32> Lds;
    constexpr int KB = D / 32, NT = D / 16, N2 = kSaveTerms, PS = D / 64, PT = F32 ? 2 : 1;
    __shared__ Lds s;
    float *sP = s.pairs, *sB = s.pairs + kChunk * kBRow;
    E *sE = reinterpret_cast<E *>(s.slots);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t x = blockIdx.x / (uint32_t)a.n_key_heads;
    const int hk = blockIdx.x % (uint32_t)a.n_key_heads, share = a.n_heads / a.n_key_heads;
    SeqSpan sp;
    const int32_t c = chunk_at(a, x, sp);
    if (c < 0) return;
    const int64_t t0 = sp.t0 + (int64_t)c * kChunk;
    const int rows = min(kChunk, sp.len - c * kChunk);
    uint8_t *shared_blk = a.work + (x * a.n_heads + hk * share) * lay.block;

    for (int h = hk * share; h < (hk + 1) * share; ++h) {
        // opaque, or every address made of it would be kept over the loop, in more registers than there are
        int t = threadIdx.x;
        asm("" : "+v"(t));
        const int l = t & 63, r = l & 15, g4 = (l >> 4) * 4, g8 = (l >> 4) * 8;
        // the sums over the heads that share the key head; every lane adds to what it wrote itself
        f4 *sums = reinterpret_cast<f4 *>(shared_blk + lay.sum) + t;
        const bool head0 = h == hk * share, headn = h + 1 == (hk + 1) * share;
        const uint8_t *blk = a.work + (x * a.n_heads + h) * lay.block, *sv = a.save + (x * a.n_heads + h) * save.block;
        const E *pE = reinterpret_cast<const E *>(sv + save.E), *pdV = reinterpret_cast<const E *>(blk + lay.dV);
        // this thread's share of 16 channels, from memory and to the LDS
        f4 part[2 * PS + PT], sum_q{}, sum_k{};
        auto load_part = [&](int n) {
#pragma unroll
            for (int i = 0; i < PS; ++i) {
                part[i] = *at_bytes<f4>(sv + save.S + n * Lds::STATE, 16u * (t + 256 * i));
                part[PS + i] = *at_bytes<f4>(blk + lay.dS + n * Lds::STATE, 16u * (t + 256 * i));
            }
            if constexpr (F32) {
                part[2 * PS] = *at_bytes<f4>(shared_blk + lay.KT + n * Lds::TOKENS, 16u * t);
                part[2 * PS + PT - 1] = *at_bytes<f4>(shared_blk + lay.QT + n * Lds::TOKENS, 16u * t);
            } else {
                part[2 * PS] = *at_bytes<f4>(shared_blk + (w < 2 ? lay.KT : lay.QT) + n * Lds::TOKENS, 16u * (t & 127));
            }
        };
        auto load_sums = [&](int n) {
            if (!head0) sum_q = sums[512 * n], sum_k = sums[512 * n + 256];
        };
        auto store_part = [&](int slot) {
#pragma unroll
            for (int i = 0; i < 2 * PS + PT; ++i) *reinterpret_cast<f4 *>(s.slots + slot * Lds::SLOT + 16 * (t + 256 * i)) = part[i];
        };

        const GatesOf gates = load_gates<F32>(a, t0, rows, h, t);
        Frag<F32, 1> fy[KB];
        Frag<F32, N2> fv[KB], fe[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            fe[kb] = Operand<F32, N2, KB>::get(pE, w, kb, l);
            fy[kb] = token_frag<F32>(a.dy, (int64_t)a.n_heads * D, t0, rows, 16 * w + r, (int64_t)h * D + kb * 32 + g8);
            fv[kb] = Operand<F32, N2, KB>::get(pdV, w, kb, l);
        }
        load_part(0);
        float db[SLICES];
        if (t < rows)
#pragma unroll
            for (int i = 0; i < SLICES; ++i) db[i] = reinterpret_cast<const float *>(blk + lay.dbeta)[i * kChunk + t];
        __syncthreads();  // the last head's LDS is done with
        gates_gdn(gates, rows, s.G, s.beta, t);
        if (w == 0) {  // decay from the chunk's start; to its end, and beta
            __builtin_amdgcn_wave_barrier();
            s.in[t] = exp_of((float)s.G[t]);
            s.to[t] = exp_of((float)(s.G[kChunk - 1] - s.G[t])) * gates.beta;
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) Operand<F32, N2, KB>::put(sE, w, kb, l, fe[kb]);
        __syncthreads();
        // ---- the pairs' gradients with their decay, rows of this wave
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f4 p{}, b{};
            if (j <= w) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const Frag<F32, N2> f = Operand<F32, N2, KB>::get(sE, j, kb, l);
                    p = mma<N2>(fy[kb], f, p);
                    b = mma<N2>(fv[kb], f, b);
                }
            }
            const int col = 16 * j + r;
            const double to_col = s.G[col];
            const float beta = s.beta[col];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * w + g4 + i;
                const float e = beta * exp_of((float)(s.G[row] - to_col));
                if (j == w && col == row) s.diag[row] = p[i] * e;
                sP[row * kBRow + col] = col < row ? p[i] * e : 0.f;
                sB[row * kBRow + col] = col < row ? -b[i] * e : 0.f;
            }
        }
        if (t < rows) {
#pragma unroll
            for (int i = 1; i < SLICES; ++i) db[0] += db[i];
            st_elem<F32>(a.dbeta, (t0 + t) * a.n_heads + h, db[0]);
        }
        __syncthreads();
        // Fragments kb of dP's and dB's rows of this wave's tokens, and of their columns.
        // Below the diagonal, a wave needs both rows or both columns, never all four.
        auto pairs = [&](const float *m, int kb, bool columns) {
            float u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = columns ? m[(32 * kb + g8 + i) * kBRow + 16 * w + r] : m[(16 * w + r) * kBRow + 32 * kb + g8 + i];
            return make_frag<F32, N2>(u);
        };
        const bool late = w >= 2;  // rows 1, else columns 0
        const Frag<F32, N2> rP = pairs(sP, 0, false), rB = pairs(sB, 0, false), cP = pairs(sP, 1, true), cB = pairs(sB, 1, true);
        const Frag<F32, N2> xP = late ? pairs(sP, 1, false) : pairs(sP, 0, true), xB = late ? pairs(sB, 1, false) : pairs(sB, 0, true);
        f4 X{}, Z{};     // summed over channels, this wave's tokens
        float tail = 0.f;  // S0 . dS
        store_part(0);
        load_part(1);
        load_sums(0);
        __syncthreads();
#pragma unroll 1
        for (int n = 0; n < NT; ++n) {
            const uint8_t *slot = s.slots + (n & 1) * Lds::SLOT;
            const E *tS = reinterpret_cast<const E *>(slot), *tdS = reinterpret_cast<const E *>(slot + Lds::STATE);
            const E *tK = reinterpret_cast<const E *>(slot + 2 * Lds::STATE), *tQ = reinterpret_cast<const E *>(slot + 2 * Lds::STATE + Lds::TOKENS);
            f4 dq{}, row{}, end{}, col{};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const Frag<F32, N2> f0 = Operand<F32, N2, KB>::get(tS, 0, kb, l), f1 = Operand<F32, N2, KB>::get(tdS, 0, kb, l);
                dq = mma<N2>(fy[kb], f0, dq);
                row = mma<N2>(fv[kb], f0, row);
                end = mma<N2>(fe[kb], f1, end);
            }
            const f4 in = *reinterpret_cast<const f4 *>(s.in + 16 * w + g4);
            dq *= in, row *= -in, end *= *reinterpret_cast<const f4 *>(s.to + 16 * w + g4);
            const Frag<F32, 1> k0 = Operand<F32, 1, 2>::get(tK, 0, 0, l), k1 = Operand<F32, 1, 2>::get(tK, 0, 1, l);
            const Frag<F32, 1> q0 = Operand<F32, 1, 2>::get(tQ, 0, 0, l), q1 = Operand<F32, 1, 2>::get(tQ, 0, 1, l);
            dq = mma<N2>(rP, k0, dq), row = mma<N2>(rB, k0, row);
            col = mma<N2>(cB, k1, col), col = mma<N2>(cP, q1, col);
            if (late) dq = mma<N2>(xP, k1, dq), row = mma<N2>(xB, k1, row);
            else col = mma<N2>(xB, k0, col), col = mma<N2>(xP, q0, col);
            const f4 kt = sum_of(get_operand4<F32, 1, 2>(tK, r, 16 * w + g4)), qt = sum_of(get_operand4<F32, 1, 2>(tQ, r, 16 * w + g4));
            X += qt * dq + kt * (row - col), Z += kt * end;
            const f4 diag = *reinterpret_cast<const f4 *>(s.diag + 16 * w + g4);
            dq += diag * kt + sum_q;
            f4 dk = row + col + end + diag * qt + sum_k;
            if (headn) {
                const f4 oq = turn(s.pairs + 320 * w, dq, l), ok = turn(s.pairs + 320 * w, dk, l);
                if (16 * w + r < rows) {
                    const int64_t at = ((t0 + 16 * w + r) * a.n_key_heads + hk) * D + 16 * n + g4;
                    st_elem4<F32>(a.dq, at, oq);
                    st_elem4<F32>(a.dk, at, ok);
                }
            } else {
                sums[512 * n] = dq, sums[512 * n + 256] = dk;
            }
            if (w < KB) {  // 32 columns to each wave
                const Frag<F32, N2> f0 = Operand<F32, N2, KB>::get(tS, 0, w, l), f1 = Operand<F32, N2, KB>::get(tdS, 0, w, l);
                float dot = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (F32) dot = fmaf(f0.v[i / 4][i % 4], f1.v[i / 4][i % 4], dot);
                    else dot = fmaf((float)f0.t[0][i] + (float)f0.t[1][i], (float)f1.t[0][i] + (float)f1.t[1][i], dot);
                }
                tail += dot;
            }
            store_part(~n & 1);
            load_part(min(n + 2, NT - 1));
            load_sums(min(n + 1, NT - 1));
            __syncthreads();
        }
#pragma unroll
        for (int off = 1; off < 16; off <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) X[i] += __shfl_xor(X[i], off), Z[i] += __shfl_xor(Z[i], off);
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) tail += __shfl_xor(tail, off);
        if (r == 0) {
            *reinterpret_cast<f4 *>(s.X + 16 * w + g4) = X;
            *reinterpret_cast<f4 *>(s.Z + 16 * w + g4) = Z;
        }
        if (l == 0) s.end[w] = tail;
        __syncthreads();
        if (t < kChunk) {
            float after = s.X[t], before = t ? s.Z[t - 1] : 0.f;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const float y = __shfl_down(after, off), z = __shfl_up(before, off);
                if (t + off < 64) after += y;
                if (t >= off) before += z;
            }
            const float start = (s.end[0] + s.end[1] + s.end[2] + s.end[3]) * exp_of((float)s.G[kChunk - 1]);
            if (t < rows) st_elem<F32>(a.dg, (t0 + t) * a.n_heads + h, after + before + start);
        }
    }
}

// KDA: 16 by 16 tokens in fp32, the decays put on keys and queries.  e^L and e^R of the
// chunk fill the LDS for one workgroup per CU: eight waves, the last four with the same tokens
// as the first and the other half of the channels, so that two share a SIMD (four waves, each
// with its own loads of the states: 389 us for 4001 tokens x 32 heads, d 128; this 224 us).
template <int D, bool F32> struct GradKdaLds {
    static constexpr bool KQ = !(F32 && D == 128);  // keys and queries fit beside the rest
    static constexpr int ROW = TokenTile<D, F32>::ROW, GROW = D + 4;
    static constexpr int STATE = 64 * D;  // bytes of 16 channels
    union {
        struct { __attribute__((aligned(16))) float dP[kChunk * kBRow], dB[kChunk * kBRow]; };
        __attribute__((aligned(16))) uint8_t states[4 * STATE];  // S0 and dS of 32 channels
    };
    float ownP[4][16 * 17], ownB[4][16 * 17];  // the blocks on the diagonal
    __attribute__((aligned(16))) Elem<F32> k[KQ ? kChunk * ROW : 8], q[KQ ? kChunk * ROW : 8];
    // L: the log-gates of a token's block up to it, R: after it
    float eL[kChunk * GROW], eR[kChunk * GROW];
    __attribute__((aligned(16))) float turn[8][320];
    __attribute__((aligned(16))) float beta[kChunk], diag[kChunk], end[2][D];
    int strong[4];
};

template <int D, bool F32, int SLICES>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void grad_kda_kernel(SeqArgs a) {
    typedef Elem<F32> E;
    constexpr BackwardLayout lay = backward_layout(D, true, F32);
    constexpr SaveLayout save = save_layout(D);
    typedef GradKdaLds<D, F32> Lds;
    constexpr int KB = D / 32, NT = D / 16, ROW = Lds::ROW, GROW = Lds::GROW, N2 = kSaveTerms;
    __shared__ Lds s;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave & 3, half = wave >> 2;
    const int64_t x = blockIdx.x / (uint32_t)a.n_key_heads;
    const int hk = blockIdx.x % (uint32_t)a.n_key_heads, share = a.n_heads / a.n_key_heads;
    SeqSpan sp;
    const int32_t c = chunk_at(a, x, sp);
    if (c < 0) return;
    const int64_t t0 = sp.t0 + (int64_t)c * kChunk;
    const int rows = min(kChunk, sp.len - c * kChunk);

    if constexpr (Lds::KQ) {
        TokenTile<D, F32> tile;
        tile.load(half ? a.q : a.k, half ? a.q_stride : a.k_stride, t0, rows, hk, threadIdx.x & 255);
        tile.store(half ? s.q : s.k, threadIdx.x & 255);
    }
    auto key = [&](int tok, int ch) {
        if constexpr (Lds::KQ) return ld_elem<F32>(s.k, tok * ROW + ch);
        else return tok < rows ? ld_elem<F32>(a.k, (t0 + tok) * a.k_stride + (int64_t)hk * D + ch) : 0.f;
    };
    auto query = [&](int tok, int ch) {
        if constexpr (Lds::KQ) return ld_elem<F32>(s.q, tok * ROW + ch);
        else return tok < rows ? ld_elem<F32>(a.q, (t0 + tok) * a.q_stride + (int64_t)hk * D + ch) : 0.f;
    };
    for (int h = hk * share; h < (hk + 1) * share; ++h) {
        // opaque, as above
        int t = threadIdx.x;
        asm("" : "+v"(t));
        const int l = t & 63, r = l & 15, g4 = (l >> 4) * 4, g8 = (l >> 4) * 8;
        // the sums over the heads that share the key head; every lane adds to what it wrote itself
        f4 *sums = reinterpret_cast<f4 *>(a.work + (x * a.n_heads + hk * share) * lay.block + lay.sum) + (t & 255);
        const uint8_t *blk = a.work + (x * a.n_heads + h) * lay.block, *sv = a.save + (x * a.n_heads + h) * save.block;
        const E *pE = reinterpret_cast<const E *>(sv + save.E), *pdV = reinterpret_cast<const E *>(blk + lay.dV);
        // ---- everything that is waited for once per head
        // a block of tokens and a channel to each thread (d = 64: the last block several times, with the
        // same values); 32-bit offsets within a chunk
        int gb = min(t / D, 3), gch = t % D;
        const uint32_t gate_row = (uint32_t)a.n_heads * D;
        const void *gates = static_cast<const E *>(a.g) + (t0 * a.n_heads + h) * D;
        uint32_t raw[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            raw[i] = *at_bytes<RawOf<F32>>(gates, (uint32_t)sizeof(E) * (min(16 * gb + i, rows - 1) * gate_row + gch));
        const float beta = t < rows ? ld_elem<F32>(a.beta, (t0 + t) * a.n_heads + h) : 0.f;
        Frag<F32, 1> fy[KB];
        Frag<F32, N2> fv[KB], fe[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            fe[kb] = Operand<F32, N2, KB>::get(pE, w, kb, l);
            fy[kb] = token_frag<F32>(a.dy, (int64_t)a.n_heads * D, t0, rows, 16 * w + r, (int64_t)h * D + kb * 32 + g8);
            fv[kb] = Operand<F32, N2, KB>::get(pdV, w, kb, l);
        }
        // this thread's share of the states of 32 channels, from memory and to the LDS
        constexpr int PS = D / 64;
        f4 part[2 * PS];
        auto load_part = [&](int step) {
#pragma unroll
            for (int i = 0; i < PS; ++i) {
                part[i] = *at_bytes<f4>(sv + save.S + 2 * step * Lds::STATE, 16u * (t + 512 * i));
                part[PS + i] = *at_bytes<f4>(blk + lay.dS + 2 * step * Lds::STATE, 16u * (t + 512 * i));
            }
        };
        auto store_part = [&]() {
#pragma unroll
            for (int i = 0; i < 2 * PS; ++i) *reinterpret_cast<f4 *>(s.states + 16 * (t + 512 * i)) = part[i];
        };
        E *tS = reinterpret_cast<E *>(s.states), *tdS = reinterpret_cast<E *>(s.states + 2 * Lds::STATE);
        // cleared on this side of the barrier, set on the other: the last head's readers are two barriers back
        if (t < 4) s.strong[t] = 0;
        __syncthreads();  // the last head's LDS is done with
        if (t < kChunk) s.beta[t] = beta;
        float up = 0.f, low = 0.f, down = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (16 * gb + i >= rows) raw[i] = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            up += floor_gate(of_raw<F32>(raw[i]));
            low = fminf(low, up);  // not the last sum alone: a gate above 1 may raise it again
            s.eL[(16 * gb + i) * GROW + gch] = exp_of(up);
        }
#pragma unroll
        for (int i = 15; i >= 0; --i) {
            s.eR[(16 * gb + i) * GROW + gch] = exp_of(down);
            down += floor_gate(of_raw<F32>(raw[i]));
        }
        if (low < -kBlockRange) s.strong[gb] = 1;
        float db[SLICES];
#pragma unroll
        for (int i = 0; i < SLICES; ++i) db[i] = reinterpret_cast<const float *>(blk + lay.dbeta)[i * kChunk + t % kChunk];
        if (half == 0)  // E to every wave
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) Operand<F32, N2, KB>::put(tS, w, kb, l, fe[kb]);
        __syncthreads();
        // ---- the pairs' gradients, rows of this wave, two blocks of columns
        f4 p[2]{}, b[2]{};
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (2 * half + j <= w)
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const Frag<F32, N2> f = Operand<F32, N2, KB>::get(tS, 2 * half + j, kb, l);
                    p[j] = mma<N2>(fy[kb], f, p[j]);
                    b[j] = mma<N2>(fv[kb], f, b[j]);
                }
        load_part(0);
        if (t < rows) {
#pragma unroll
            for (int i = 1; i < SLICES; ++i) db[0] += db[i];
            st_elem<F32>(a.dbeta, (t0 + t) * a.n_heads + h, db[0]);
        }
        __syncthreads();
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            const int j = 2 * half + jj;
            const int col = 16 * j + r;
            const float beta = s.beta[col];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * w + g4 + i;
                const float e = col <= row ? beta : 0.f;
                const float dp = col < row ? p[jj][i] * e : 0.f, db = col < row ? -b[jj][i] * e : 0.f;
                s.dP[row * kBRow + col] = dp;
                s.dB[row * kBRow + col] = db;
                if (j == w) {
                    s.ownP[w][(g4 + i) * 17 + r] = dp, s.ownB[w][(g4 + i) * 17 + r] = db;
                    if (col == row) s.diag[row] = p[jj][i] * e;
                }
            }
        }
        __syncthreads();
        const bool fast = !s.strong[w];
        // this wave's rows and columns of its own block; of the other three the rows if before, else the columns
        auto rows_of = [&](const float *m, int J) { return *reinterpret_cast<const f4 *>(m + (16 * w + r) * kBRow + 16 * J + g4); };
        auto columns_of = [&](const float *m, int J) {
            f4 x;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = m[(16 * J + g4 + i) * kBRow + 16 * w + r];
            return x;
        };
        const f4 rowP = rows_of(s.dP, w), rowB = rows_of(s.dB, w), colP = columns_of(s.dP, w), colB = columns_of(s.dB, w);
        f4 bP[3], bB[3];
#pragma unroll
        for (int u = 0; u < 3; ++u) {
            if (u < w) bP[u] = rows_of(s.dP, u), bB[u] = rows_of(s.dB, u);
            else bP[u] = columns_of(s.dP, u + 1), bB[u] = columns_of(s.dB, u + 1);
        }
        __syncthreads();
        store_part();
        load_part(1);
        __syncthreads();
#pragma unroll 1
        for (int n = half; n < NT; n += 2) {
            const int ch = 16 * n + r;
            // ---- through the states
            f4 dq{}, row{}, col{};
            float dot = 0.f;  // S0 . dS of one channel, this lane's columns; by the waves with the fewest pairs
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const Frag<F32, N2> f0 = Operand<F32, N2, KB>::get(tS, half, kb, l), f1 = Operand<F32, N2, KB>::get(tdS, half, kb, l);
                dq = mma<N2>(fy[kb], f0, dq);
                row = mma<N2>(fv[kb], f0, row);
                col = mma<N2>(fe[kb], f1, col);
            }
            if (w >= 2) {
#pragma unroll
                for (int u = 0; u < KB / 2; ++u) {
                    const int kb = (w - 2) * (KB / 2) + u;
                    const Frag<F32, N2> f0 = Operand<F32, N2, KB>::get(tS, half, kb, l), f1 = Operand<F32, N2, KB>::get(tdS, half, kb, l);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if constexpr (F32) dot = fmaf(f0.v[i / 4][i % 4], f1.v[i / 4][i % 4], dot);
                        else dot = fmaf((float)f0.t[0][i] + (float)f0.t[1][i], (float)f1.t[0][i] + (float)f1.t[1][i], dot);
                    }
                }
                dot += __shfl_xor(dot, 16);
                dot += __shfl_xor(dot, 32);
            }
            f4 eL, eR, kt, qt;
            float block[4];  // the decay over each block of 16 tokens
#pragma unroll
            for (int b = 0; b < 4; ++b) block[b] = s.eL[(16 * b + 15) * GROW + ch];
            float lo = 1.f, hi = 1.f;
#pragma unroll
            for (int b = 0; b < 4; ++b) lo *= b < w ? block[b] : 1.f, hi *= b > w ? block[b] : 1.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = 16 * w + g4 + i;
                eL[i] = s.eL[tok * GROW + ch], eR[i] = s.eR[tok * GROW + ch];
                dq[i] *= eL[i] * lo;
                row[i] *= -eL[i] * lo;
                col[i] *= eR[i] * hi * s.beta[tok];
            }
            if (w >= 2 && l < 16) s.end[w - 2][ch] = dot * block[0] * block[1] * block[2] * block[3];
#pragma unroll
            for (int i = 0; i < 4; ++i) kt[i] = key(16 * w + g4 + i, ch), qt[i] = query(16 * w + g4 + i, ch);
            const f4 to_end = col;  // what runs to the chunk's end
            col = f4{};
            // ---- between the chunk's tokens
            f4 from{}, back{};  // dq and row without e^L
#pragma unroll
            for (int u = 0; u < 3; ++u) {
                const int J = u < w ? u : u + 1;
                float m = 1.f;  // the decay between the blocks
#pragma unroll
                for (int b = 1; b < 3; ++b) m *= (J < b && b < w) || (w < b && b < J) ? block[b] : 1.f;
                f4 kj, e;
                if (u < w) {  // rows of this wave against keys of block J
#pragma unroll
                    for (int i = 0; i < 4; ++i) kj[i] = key(16 * J + g4 + i, ch), e[i] = s.eR[(16 * J + g4 + i) * GROW + ch];
                    kj *= e * m;
                    from = mma16(bP[u], kj, from);
                    back = mma16(bB[u], kj, back);
                } else {  // keys of this wave against rows of block J
                    f4 qj;
#pragma unroll
                    for (int i = 0; i < 4; ++i) kj[i] = key(16 * J + g4 + i, ch), qj[i] = query(16 * J + g4 + i, ch), e[i] = s.eL[(16 * J + g4 + i) * GROW + ch];
                    e *= m;
                    col = mma16(bB[u], kj * e, col);
                    col = mma16(bP[u], qj * e, col);
                }
            }
            col *= eR;
            if (fast) {
                f4 inv;
#pragma unroll
                for (int i = 0; i < 4; ++i) inv[i] = __builtin_amdgcn_rcpf(eL[i]);
                from = mma16(rowP, kt * inv, from);
                back = mma16(rowB, kt * inv, back);
                col += inv * mma16(colP, qt * eL, mma16(colB, kt * eL, f4{}));
            }
            dq += eL * from, row += eL * back;
            if (!fast) {  // strong gates: the block's pairs one by one, each by its own sum of log-gates
                float *gs = s.turn[wave];  // [token][channel]
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = 16 * w + g4 + i;
                    gs[(g4 + i) * 20 + r] = tok < rows ? floor_gate(ld_elem<F32>(a.g, ((t0 + tok) * a.n_heads + h) * D + ch)) : 0.f;
                }
                __builtin_amdgcn_wave_barrier();
#pragma unroll 1
                for (int j = 0; j < 15; ++j) {
                    float e = 0.f, sum = 0.f;
                    const float kj = key(16 * w + j, ch);
#pragma unroll 1
                    for (int i = j + 1; i < 16; ++i) {
                        e += gs[i * 20 + r];
                        const float d = exp_of(e), p = d * s.ownP[w][i * 17 + j], b = d * s.ownB[w][i * 17 + j];
                        sum = fmaf(b, key(16 * w + i, ch), fmaf(p, query(16 * w + i, ch), sum));
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const bool mine = g4 + y == i;
                            dq[y] += mine ? p * kj : 0.f;
                            row[y] += mine ? b * kj : 0.f;
                        }
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y) col[y] += g4 + y == j ? sum : 0.f;
                }
            }
            const f4 gx = qt * dq + kt * (row - col), gz = kt * to_end;
            const f4 diag = *reinterpret_cast<const f4 *>(s.diag + 16 * w + g4);
            dq += diag * kt;
            f4 dk = row + col + to_end + diag * qt;
            if (share > 1) {
                if (h > hk * share) dq += sums[512 * n], dk += sums[512 * n + 256];
                if (h + 1 < (hk + 1) * share) sums[512 * n] = dq, sums[512 * n + 256] = dk;
            }
            if (h + 1 == (hk + 1) * share) {
                const f4 oq = turn(s.turn[wave], dq, l), ok = turn(s.turn[wave], dk, l);
                if (16 * w + r < rows) {
                    const int64_t at = ((t0 + 16 * w + r) * a.n_key_heads + hk) * D + 16 * n + g4;
                    st_elem4<F32>(a.dq, at, oq);
                    st_elem4<F32>(a.dk, at, ok);
                }
            }
            // in the place of e^L and e^R, once every wave has read them for these channels
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) s.eL[(16 * w + g4 + i) * GROW + ch] = gx[i], s.eR[(16 * w + g4 + i) * GROW + ch] = gz[i];
            store_part();
            load_part(min(n / 2 + 2, NT / 2 - 1));
            __syncthreads();
        }
        asm("" : "+v"(gb), "+v"(gch));  // as above
        // dg: what comes after a token and what came before it, 16 tokens to a thread
        float y[16], z[16], ys = 0.f, zs = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = s.eL[(16 * gb + i) * GROW + gch], z[i] = s.eR[(16 * gb + i) * GROW + gch];
#pragma unroll
        for (int i = 0; i < 16; ++i) ys += y[15 - i], zs += z[i];
        s.dP[gb * D + gch] = ys, s.dB[gb * D + gch] = zs;
        __syncthreads();
        void *dgates = static_cast<E *>(a.dg) + (t0 * a.n_heads + h) * D;
        float before = s.end[0][gch] + s.end[1][gch], after = 0.f;
#pragma unroll
        for (int b = 0; b < 3; ++b)
            if (b < gb) before += s.dB[b * D + gch];
#pragma unroll
        for (int b = 3; b > 0; --b)
            if (b > gb) after += s.dP[b * D + gch];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float now = z[i];
            z[i] = before, before += now;
        }
#pragma unroll
        for (int i = 15; i >= 0; --i) {
            after += y[i];
            if (16 * gb + i < rows) st_elem<F32>(at_bytes<E>(dgates, (uint32_t)sizeof(E) * ((16 * gb + i) * gate_row + gch)), 0, after + z[i]);
        }
    }
}

template <int D, bool KDA, bool F32> hipError_t backward(const SeqArgs &a, hipStream_t stream) {
    constexpr int NCT = 1;
    const int64_t slots = chunk_slots(a.n_tokens, a.n_seq);
    hipError_t e = hipSuccess;
    if (a.n_tokens > 0) {
        const dim3 grid((uint32_t)(slots * a.n_heads));
        if constexpr (KDA) hipLaunchKernelGGL((prep_kda_bwd_kernel<D, F32>), grid, dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((prep_gdn_bwd_kernel<D, F32>), grid, dim3(256), 0, stream, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const uint32_t pairs = (uint32_t)a.n_seq * a.n_heads;
    hipLaunchKernelGGL((scan_bwd_kernel<D, KDA, F32, NCT>), dim3((pairs + 7) / 8 * 8 * (D / (16 * NCT))), dim3(256), 0, stream, a);
    if ((e = hipGetLastError()) != hipSuccess || a.n_tokens == 0) return e;
    const dim3 grid((uint32_t)(slots * a.n_key_heads));
    if constexpr (KDA) hipLaunchKernelGGL((grad_kda_kernel<D, F32, D / (16 * NCT)>), grid, dim3(512), 0, stream, a);
    else hipLaunchKernelGGL((grad_gdn_kernel<D, F32, D / (16 * NCT)>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_chunk_backward(const SeqArgs &a, int d, bool kda, bool f32, hipStream_t stream) {
    if (d == 128) {
        if (kda) return f32 ? backward<128, true, true>(a, stream) : backward<128, true, false>(a, stream);
        return f32 ? backward<128, false, true>(a, stream) : backward<128, false, false>(a, stream);
    }
    if (kda) return f32 ? backward<64, true, true>(a, stream) : backward<64, true, false>(a, stream);
    return f32 ? backward<64, false, true>(a, stream) : backward<64, false, false>(a, stream);
}

} // namespace sqk
