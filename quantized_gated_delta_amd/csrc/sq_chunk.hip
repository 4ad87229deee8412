// The gated Delta rule over whole sequences, forward, in chunks of 64 tokens.
//
// Within a chunk that starts at state S0 (ta-paperlens page, mechanism section,
// for the recurrence), with the notation of sq_prep.h,
//   R' = V - (K e^G) S0        X = diag(beta) R'
//   E  = R' + M X              U = diag(beta) E
//   y  = (Q e^G) S0 + P U      S_C = diag(e^{G_C}) S0 + (K e^{G_C - G})^T U
// Two kernels: prep (sq_prep.h: M, P and the decayed keys and queries, every chunk
// in parallel) and scan, which walks the chunks of one (sequence, head).
//
// The scan is bound by its chain of dependent products (three per chunk) when
// there are few (sequence, head) pairs, so a workgroup holds only 16 NCT columns
// of the state (columns never interact) and splits every product's rows over
// its four waves: wave w owns tokens 16 w .. 16 w + 15 of each chunk and rows
// w d / 4 .. of the state.  The state stays in registers as fp32 accumulators.  What
// another wave needs next (S, X, U) goes through LDS in the layout that is both the
// result's and the next operand's; the left operands come from HBM
// straight into fragments, the next chunk's issued right after their last use.
//
// Measured (d 128, bf16): GDN, 12 sequences of 12001 tokens in all, 48 heads, prep
// 124 us (0.65 GB, 5.3 TB/s: bound by memory) and scan 479 us; KDA, one sequence of 8192
// tokens, 32 heads, prep 214 and scan 384 us.  The scan is bound by latency: its waves spend
// 0.42 to 0.62 of their cycles unable to issue (behind the three products that wait for each
// other), 0.21 to 0.27 waiting for memory, LDS and barriers.  No unit is near its rate: matrix cores
// 0.12 to 0.26 busy, vector issue 0.18 to 0.36, HBM 2.2 to 2.9 TB/s, L2 7 TB/s (GDN) to 16 TB/s (KDA,
// whose slices read 168 KB per chunk and workgroup for GDN's 78).
// 64 tokens per chunk: the pairs' work grows with the chunk, the number of dependent steps
// falls with it, and 64 is what four waves of 16 rows hold.
#include "sq_prep.h"

namespace sqk {
namespace {

template <int D, bool F32, int N> __global__ __launch_bounds__(256) void prep_gdn_kernel(SeqArgs a) {
    constexpr ChunkLayout lay = forward_layout(D, false, F32, N);
    prepare_gdn<D, F32, N, false>(a, a.work, lay.block, lay.P, lay.M, lay.KT, 0, lay.gates);
}

template <int D, bool F32, int N> __global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void prep_kda_kernel(SeqArgs a) {
    constexpr ChunkLayout lay = forward_layout(D, true, F32, N);
    prepare_kda<D, F32, N, false>(a, a.work, lay.block, lay.P, lay.M, lay.K, lay.Q, lay.KT, 0, lay.gates);
}

// One (sequence, head), 16 NCT columns of its state, all chunks.  NTY: terms
// that y is accurate to.
template <int D, bool KDA, bool F32, int NTY, bool YF32, int NCT>
__global__ __launch_bounds__(256) void scan_kernel(SeqArgs a) {
    typedef Elem<F32> E;
    constexpr ChunkLayout lay = forward_layout(D, KDA, F32, NTY);
    constexpr SaveLayout save = save_layout(D);
    constexpr int MT = D / 64, KB = D / 32, COLS = 16 * NCT, SLICES = D / COLS;
    constexpr int KN = KDA ? 3 : 1, QN = KDA ? NTY : 1;
    typedef LdsMat<F32, 3, D, COLS> SMat;
    typedef LdsMat<F32, 3, kChunk, COLS> XMat;
    typedef LdsMat<F32, NTY, kChunk, COLS> YMat;
    __shared__ __attribute__((aligned(16))) uint8_t lds[SMat::BYTES + 2 * XMat::BYTES + (KDA ? 0 : YMat::BYTES)];
    __shared__ __attribute__((aligned(16))) float sTurn[4 * 320];
    E *sS = reinterpret_cast<E *>(lds), *sX = reinterpret_cast<E *>(lds + SMat::BYTES);
    E *sU = reinterpret_cast<E *>(lds + SMat::BYTES + XMat::BYTES);
    E *sY = KDA ? sU : reinterpret_cast<E *>(lds + SMat::BYTES + 2 * XMat::BYTES);

    const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63, r = l & 15, g4 = (l >> 4) * 4, g8 = (l >> 4) * 8;
    // the slices of one (sequence, head) read the same operands: workgroups go
    // to the 8 XCDs in turn, so they are 8 apart to share an L2
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
                S[m][n][i] = a.S0 ? a.S0[state + (int64_t)((w * MT + m) * 16 + g4 + i) * D + c0 + 16 * n + r] : 0.f;

    Frag<F32, KN> fK[KB], fKT[MT][2];
    Frag<F32, QN> fQ[KB];
    Frag<F32, 3> fM[2];
    Frag<F32, NTY> fP[2];
    uint32_t v[NCT][4];  // as loaded: widening them at once would wait for them at once
    // the gates' factors are needed early in a chunk: they are fetched a whole chunk ahead
    struct Gates { f4 eg, ec, beta, fade[MT]; float fade1, eq; } gt{}, gt_next{};

    auto block_of = [&](int c, int head) { return a.work + ((sp.slot0 + c) * a.n_heads + head) * lay.block; };
    auto rows_of = [&](int c) { return min(kChunk, sp.len - c * kChunk); };
    auto load_kq = [&](int c, int kb) {
        if constexpr (KDA) {
            const uint8_t *b = block_of(c, h);
            fK[kb] = Operand<F32, KN, KB>::get(reinterpret_cast<const E *>(b + lay.K), w, kb, l);
            fQ[kb] = Operand<F32, QN, KB>::get(reinterpret_cast<const E *>(b + lay.Q), w, kb, l);
        } else {
            // past the end: the last token again; its beta is 0 there and its y is not stored
            const int64_t tok = sp.t0 + (int64_t)c * kChunk, at = (int64_t)hk * D + kb * 32;
            const uint32_t row = min(16 * w + r, rows_of(c) - 1);
            const void *pk = static_cast<const E *>(a.k) + tok * a.k_stride + at, *pq = static_cast<const E *>(a.q) + tok * a.q_stride + at;
            fK[kb] = load_frag<F32, KN>(at_bytes<E>(pk, (row * (uint32_t)a.k_stride + g8) * (uint32_t)sizeof(E)), 0);
            fQ[kb] = load_frag<F32, QN>(at_bytes<E>(pq, (row * (uint32_t)a.q_stride + g8) * (uint32_t)sizeof(E)), 0);
        }
    };
    auto load_v = [&](int c) {
        const int last = rows_of(c) - 1;
        const void *pv = static_cast<const E *>(a.v) + (sp.t0 + (int64_t)c * kChunk) * a.v_stride + (int64_t)h * D + c0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t row = min(16 * w + g4 + i, last);
#pragma unroll
            for (int n = 0; n < NCT; ++n) v[n][i] = ld_raw<F32>(at_bytes<E>(pv, (row * (uint32_t)a.v_stride + 16 * n + r) * (uint32_t)sizeof(E)), 0);
        }
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
            x.eq = p[16 * w + r];
            x.fade1 = p[kChunk - 1];
        }
        return x;
    };
    auto load_m = [&](int c) {
        const E *b = reinterpret_cast<const E *>(block_of(c, h) + lay.M);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (kb == 0 || w >= 2) fM[kb] = Operand<F32, 3, 2>::get(b, w, kb, l);
    };
    auto load_p = [&](int c) {
        const E *b = reinterpret_cast<const E *>(block_of(c, h) + lay.P);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (kb == 0 || w >= 2) fP[kb] = Operand<F32, NTY, 2>::get(b, w, kb, l);
    };
    auto load_kt = [&](int c, int m) {
        const E *b = reinterpret_cast<const E *>(block_of(c, KDA ? h : hk * share) + lay.KT);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) fKT[m][kb] = Operand<F32, KN, 2>::get(b, w * MT + m, kb, l);
    };
    if (n_chunks > 0) {
        gt = load_gates(0);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) load_kq(0, kb);
        load_v(0), load_m(0), load_p(0);
#pragma unroll
        for (int m = 0; m < MT; ++m) load_kt(0, m);
    }

    // The slices of a (sequence, head) walk in step, so each operand would be waited for from
    // HBM by all of them: each touches its share of the lines of the chunk after next, which
    // brings them to the L2 that the slices share.  KDA alone: 412 -> 370 us for 8192
    // tokens x 32 heads; GDN's operands are half as many bytes (479 -> 508 us).
    const uint32_t part = j % SLICES;
    constexpr uint32_t kLines = (lay.block + 127) / 128, kTouch = KDA ? (kLines + 256 * SLICES - 1) / (256 * SLICES) : 0;
    uint32_t touched[kTouch + 1] = {};
    auto touch = [&](int c) {
#pragma unroll
        for (uint32_t i = 0; i < kTouch; ++i) {
            const uint32_t line = (t + 256 * i) * SLICES + part;
            if (line < kLines) touched[i] = *at_bytes<uint32_t>(block_of(c, h), line * 128);
        }
    };
    for (int c = 0; c < n_chunks; ++c) {
        const int next = min(c + 1, n_chunks - 1), rows = rows_of(c);
        gt_next = load_gates(next);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NCT; ++n) SMat::put4(sS, 16 * n + r, (w * MT + m) * 16 + g4, S[m][n]);
        uint8_t *keep = a.save + ((sp.slot0 + c) * a.n_heads + h) * save.block;
        if (a.save)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NCT; ++n)
                    put_operand4<F32, kSaveTerms, KB>(reinterpret_cast<E *>(keep + save.S), (w * MT + m) * 16 + r, c0 + 16 * n + g4,
                                                      turn(sTurn + w * 320, S[m][n], l));
        __syncthreads();
        // y is formed with its columns as the result's rows: a lane then holds four neighbours of one token
        f4 ks[NCT], y[NCT];
#pragma unroll
        for (int n = 0; n < NCT; ++n) ks[n] = y[n] = f4{};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
            for (int n = 0; n < NCT; ++n) {
                const Frag<F32, 3> fs = SMat::get(sS, 16 * n + r, kb * 32 + g8);
                ks[n] = mma<3>(fK[kb], fs, ks[n]);
                y[n] = mma<NTY>(fs, fQ[kb], y[n]);
            }
            load_kq(next, kb);  // between the products: a load that waits for its turn then waits beside them
        }
        f4 e[NCT];
#pragma unroll
        for (int n = 0; n < NCT; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) e[n][i] = of_raw<F32>(v[n][i]) - (KDA ? ks[n][i] : gt.eg[i] * ks[n][i]);
            XMat::put4(sX, 16 * n + r, 16 * w + g4, e[n] * gt.beta);
        }
        __syncthreads();
        load_v(next);
#pragma unroll
        for (int n = 0; n < NCT; ++n) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (kb == 0 || w >= 2) e[n] = mma<3>(fM[kb], XMat::get(sX, 16 * n + r, kb * 32 + g8), e[n]);
            if (a.save)
                put_operand4<F32, kSaveTerms, KB>(reinterpret_cast<E *>(keep + save.E), 16 * w + r, c0 + 16 * n + g4,
                                                  turn(sTurn + w * 320, e[n], l));
            const f4 u = e[n] * gt.beta;
            if constexpr (KDA) {
                XMat::put4(sU, 16 * n + r, 16 * w + g4, u);
            } else {
                XMat::put4(sU, 16 * n + r, 16 * w + g4, u * gt.ec);
                YMat::put4(sY, 16 * n + r, 16 * w + g4, u);
            }
        }
        load_m(next);
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int n = 0; n < NCT; ++n) {
                S[m][n] = KDA ? S[m][n] * gt.fade[m] : S[m][n] * gt.fade1;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
                    S[m][n] = mma<3>(fKT[m][kb], XMat::get(sU, 16 * n + r, kb * 32 + g8), S[m][n]);
            }
            load_kt(next, m);
        }
        char *py = static_cast<char *>(a.y) + (((sp.t0 + (int64_t)c * kChunk) * a.n_heads + h) * D + c0) * (YF32 ? 4 : 2);
#pragma unroll
        for (int n = 0; n < NCT; ++n) {
            if (!KDA) y[n] *= gt.eq;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (kb == 0 || w >= 2) {
                    if constexpr (KDA)
                        y[n] = mma<NTY>(XMat::get(sU, 16 * n + r, kb * 32 + g8), fP[kb], y[n]);
                    else
                        y[n] = mma<NTY>(YMat::get(sY, 16 * n + r, kb * 32 + g8), fP[kb], y[n]);
                }
            if (16 * w + r < rows)
                st_elem4<YF32>(at_bytes<char>(py, ((16 * w + r) * (uint32_t)(a.n_heads * D) + 16 * n + g4) * (YF32 ? 4u : 2u)), 0, y[n]);
        }
        load_p(next);
#pragma unroll
        for (uint32_t i = 0; i < kTouch; ++i) asm volatile("" ::"v"(touched[i]));  // so that the loads are not dropped
        touch(min(c + 2, n_chunks - 1));
        gt = gt_next;
    }
    if (a.S_out)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NCT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a.S_out[state + (int64_t)((w * MT + m) * 16 + g4 + i) * D + c0 + 16 * n + r] = S[m][n][i];
}

template <int D, bool KDA, bool F32, int NTY, bool YF32, int NCT>
void launch_scan(const SeqArgs &a, hipStream_t stream) {
    const uint32_t pairs = (uint32_t)a.n_seq * a.n_heads;
    const uint32_t grid = (pairs + 7) / 8 * 8 * (D / (16 * NCT));
    hipLaunchKernelGGL((scan_kernel<D, KDA, F32, NTY, YF32, NCT>), dim3(grid), dim3(256), 0, stream, a);
}

template <int D, bool KDA, bool F32, bool YF32> hipError_t forward(const SeqArgs &a, hipStream_t stream) {
    constexpr int NTY = YF32 ? 3 : 2;
    const uint32_t blocks = (uint32_t)(chunk_slots(a.n_tokens, a.n_seq) * a.n_heads);
    if (a.n_tokens > 0) {
        if constexpr (KDA)
            hipLaunchKernelGGL((prep_kda_kernel<D, F32, NTY>), dim3(blocks), dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL((prep_gdn_kernel<D, F32, NTY>), dim3(blocks), dim3(256), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // 32 columns read the operands half as often for the same work, but leave half the
    // workgroups: worth it once 16 columns would give 8 workgroups per CU
    // (48 heads x 12 sequences: 487 against 660 us; 32 x 4: 401 against 377 us;
    // one sequence of 32 heads, KDA: 489 against 374 us).  The rule does not look at lengths, though
    // one long sequence among very many short ones has the chain of a single one.
    if (a.n_seq * (int64_t)a.n_heads * (D / 16) >= 2048) launch_scan<D, KDA, F32, NTY, YF32, 2>(a, stream);
    else launch_scan<D, KDA, F32, NTY, YF32, 1>(a, stream);
    return hipGetLastError();
}

template <int D, bool KDA> hipError_t forward_types(const SeqArgs &a, bool f32, bool y_f32, hipStream_t stream) {
    if (f32) return y_f32 ? forward<D, KDA, true, true>(a, stream) : forward<D, KDA, true, false>(a, stream);
    return y_f32 ? forward<D, KDA, false, true>(a, stream) : forward<D, KDA, false, false>(a, stream);
}

} // namespace

hipError_t launch_chunk_forward(const SeqArgs &a, int d, bool kda, bool f32, bool y_f32, hipStream_t stream) {
    if (d == 128) return kda ? forward_types<128, true>(a, f32, y_f32, stream) : forward_types<128, false>(a, f32, y_f32, stream);
    return kda ? forward_types<64, true>(a, f32, y_f32, stream) : forward_types<64, false>(a, f32, y_f32, stream);
}

} // namespace sqk
