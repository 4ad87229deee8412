// The selective state-space scan over whole sequences, in chunks of 64 tokens, and its step.
//
// Within a chunk that starts at state S0, G the running sum of dt A and L_ij = e^{G_i - G_j},
//   y_i = e^{G_i} S0^T C_i + sum_{j <= i} (C_i . B_j) L_ij dt_j x_j + D x_i
//   S_end = e^{G_end} S0 + sum_j e^{G_end - G_j} dt_j B_j x_j^T
// Nothing but the state's own decay waits for the state, so a wave keeps 16 columns of it (all d_state rows, fp32) in
// registers from chunk to chunk: the result of the update is, as it stands, the left operand of the
// reading (its rows in the order of two result tiles, in which C is read too).  The four
// waves of a workgroup share a chunk's C, B, x, gates and pairs through LDS.
//
// A workgroup walks one segment of one sequence for 64 columns of one head.  Where sequences are
// cut (scan_plan), a first pass forms each segment's own state, a second one walks the segments
// (S = e^{G} S + own), and the main pass starts from those.
// The gradients' pass back over the chunks is the same recurrence with C, dy and e^G for B, x and
// e^{G_end - G} dt, from the last chunk to the first.
#include "sq_scan.h"

namespace sqk {
namespace {

// What a pass over the chunks does: form a segment's own state; form y; the same two backwards.
enum Pass { kOwn, kMain, kOwnBack, kMainBack };

template <int N, bool F32, int NTY, bool YF32, int PASS> __global__ __launch_bounds__(256) void scan_kernel(ScanArgs a) {
    typedef Elem<F32> E;
    constexpr bool BACK = PASS >= kOwnBack, Y = PASS == kMain, OWN = PASS == kOwn || PASS == kOwnBack;
    constexpr int MT = N / 16, KB = N / 32;
    typedef TokenMat<F32, N> KeyMat;
    typedef TokenMat<F32, kHeadPart> XMat;
    typedef LdsMat<F32, NTY, 64, 64> PairMat;
    __shared__ __attribute__((aligned(16))) E sK[KeyMat::SIZE], sX[XMat::SIZE];
    __shared__ __attribute__((aligned(16))) E sC[Y ? KeyMat::SIZE : 8];
    __shared__ __attribute__((aligned(16))) uint8_t sP[Y ? PairMat::BYTES : 16];
    __shared__ Gates gates[2];
    __shared__ __attribute__((aligned(16))) float sTurn[OWN ? 4 : 4 * 320];

    const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63, r = l & 15, g4 = (l >> 4) * 4, g8 = (l >> 4) * 8;
    // the heads of a group read the same B and C: workgroups go to the 8 XCDs in turn, and each
    // XCD gets neighbouring heads
    const int parts = a.n_heads * (a.d_head / kHeadPart), each = (parts + 7) / 8;
    const uint32_t turn_of = blockIdx.x >> 3;
    const int part = (blockIdx.x & 7) * each + turn_of % each;
    if (part >= parts) return;
    const int64_t slot = turn_of / each;
    const Block b = block_at(a.seqs, slot, a.seg_shift);
    if (b.seq < 0) return;
    const Part pt = part_of(a, part);
    const int begin = b.c << a.seg_shift, len = min(b.len - begin, 1 << a.seg_shift), n_chunks = (len + 63) >> 6;
    const bool last = begin + (1 << a.seg_shift) >= b.len;
    const int64_t t0 = (int64_t)b.t0 + begin, at = state_at<N>(a, b.seq, pt);
    const int64_t chunk0 = ((int64_t)(b.t0 >> 6) + b.seq + (begin >> 6)) * parts + part;  // + c * parts
    float *seg = a.seg_state + (slot * parts + part) * N * kHeadPart;

    f4 S[MT];
    const float *from = OWN ? nullptr : a.segments ? seg : (BACK ? a.dS_out : a.S0);
    {
        const int64_t row = a.segments ? kHeadPart : a.d_head;
        const float *p = from ? (a.segments ? from : from + at) : nullptr;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[m][i] = p ? p[(16 * m + g4 + i) * row + 16 * w + r] : 0.f;
    }
    const float A = a.A[pt.head], bias = a.bias ? a.bias[pt.head] : 0.f, D = Y && a.D ? a.D[pt.head] : 0.f;
    const void *keys = BACK ? a.C : a.B, *xs = BACK ? a.dy : a.x;
    const int64_t key_stride = BACK ? a.c_stride : a.b_stride, x_stride = BACK ? (int64_t)a.n_heads * a.d_head : a.x_stride;

    Staged<F32, N, 256> rK, rC;
    Staged<F32, kHeadPart, 256> rX;
    auto rows_of = [&](int c) { return min(64, len - c * 64); };
    auto load = [&](int c) {
        const int64_t tok = t0 + (int64_t)c * 64;
        const int rows = rows_of(c);
        rK.load(static_cast<const E *>(keys) + tok * key_stride + (int64_t)pt.group * N, key_stride, rows, t);
        rX.load(static_cast<const E *>(xs) + tok * x_stride + (int64_t)pt.head * a.d_head + pt.col, x_stride, rows, t);
        if (Y) rC.load(static_cast<const E *>(a.C) + tok * a.c_stride + (int64_t)pt.group * N, a.c_stride, rows, t);
    };
    auto load_raw = [&](int c) {
        const int rows = rows_of(c);
        return ld_elem<F32>(a.raw, (t0 + (int64_t)c * 64 + min(l, rows - 1)) * a.dt_stride + pt.head);
    };
    const int first = BACK ? n_chunks - 1 : 0, step = BACK ? -1 : 1;
    if (n_chunks > 0) {
        load(first);
        if (w == 0) make_gates(gates[0], l, l < rows_of(first), load_raw(first), bias, A, a.softplus);
    }
    if (Y) {  // the tiles beside the diagonal that a contraction over 32 tokens meets and no pair fills
        if (w < 2) PairMat::put4(reinterpret_cast<E *>(sP), 32 * w + r, 32 * w + 16 + g4, f4{});
    }
    float fade = 1.f;
    for (int k = 0; k < n_chunks; ++k) {
        const int c = first + k * step, rows = rows_of(c);
        const Gates &g = gates[k & 1];
        rK.store(sK, t);
        rX.store(sX, t);
        if (Y) rC.store(sC, t);
        __syncthreads();
        if (k + 1 < n_chunks) {
            load(c + step);
            if (w == (k & 3)) make_gates(gates[~k & 1], l, l < rows_of(c + step), load_raw(c + step), bias, A, a.softplus);
        }
        uint8_t *keep = BACK ? a.grad_save : a.save;
        if (!OWN && keep) {
            E *p = reinterpret_cast<E *>(keep + (chunk0 + (int64_t)c * parts) * N * kHeadPart * 4);
#pragma unroll
            for (int m = 0; m < MT; ++m)
                put_operand4<F32, kSaveTerms, 2>(p, 16 * m + r, 16 * w + g4, turn(sTurn + w * 320, S[m], l));
        }
        if (Y) {
            // pairs, as the operand of x: token i's row holds (C_i . B_j) L_ij dt_j
            for (int n = w; n < 10; n += 4) {
                int it, jt;
                pair_tile(n, it, jt);
                f4 p{};
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
                    p = mma<1>(KeyMat::get(sK, 16 * jt + r, 32 * kb + g8), KeyMat::get(sC, 16 * it + r, 32 * kb + g8), p);
                const int i = 16 * it + r;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 16 * jt + g4 + e;
                    p[e] = j <= i ? p[e] * decay_of(g, i, j) * g.dt[j] : 0.f;
                }
                PairMat::put4(reinterpret_cast<E *>(sP), i, 16 * jt + g4, p);
            }
            __syncthreads();
        }
        Frag<F32, 1> fx[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) fx[kb] = get_t<F32, 1>(sX, XMat::ROW, 0, 32 * kb, 16 * w, l);
        if (Y) {
            // transposed, y's columns as the result's rows: a lane then holds four neighbours of one token
            f4 y[4] = {};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                float s[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = S[2 * kb + e / 4][e % 4];
                const Frag<F32, NTY> fs = make_frag<F32, NTY>(s);
#pragma unroll
                for (int it = 0; it < 4; ++it) y[it] = mma<NTY>(fs, KeyMat::get_split(sC, 16 * it + r, 32 * kb + g4), y[it]);
            }
            char *py = static_cast<char *>(a.y) + ((t0 + (int64_t)c * 64) * a.n_heads + pt.head) * a.d_head * (YF32 ? 4 : 2);
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int i = 16 * it + r;
                y[it] *= g.in[i];
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
                    if (kb == 0 || it >= 2) y[it] = mma<NTY>(fx[kb], PairMat::get(reinterpret_cast<E *>(sP), i, 32 * kb + g8), y[it]);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[it][e] = fmaf(D, ld_elem<F32>(sX, i * XMat::ROW + 16 * w + g4 + e), y[it][e]);
                if (i < rows) st_elem4<YF32>(py, (int64_t)i * a.n_heads * a.d_head + pt.col + 16 * w + g4, y[it]);
            }
        }
        // the state: the scaled x as the right operand, three terms, so that the state has fp32 accuracy
        Frag<F32, 3> fs[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            float v[8];
            widen(fx[kb], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int j = 32 * kb + g8 + e;
                v[e] *= BACK ? g.in[j] : g.out[j] * g.dt[j];
            }
            fs[kb] = make_frag<F32, 3>(v);
        }
        const float whole = g.in[63];
        fade *= whole;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            S[m] *= whole;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) S[m] = mma<3>(get_t<F32, 1>(sK, KeyMat::ROW, 0, 32 * kb, 16 * m, l), fs[kb], S[m]);
        }
        __syncthreads();
    }
    float *to = OWN ? seg : BACK ? (b.c == 0 ? a.dS0 : nullptr) : (last ? a.S_out : nullptr);
    if (to) {
        const int64_t row = OWN ? kHeadPart : a.d_head;
        if (!OWN) to += at;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) to[(16 * m + g4 + i) * row + 16 * w + r] = S[m][i];
    }
    if (OWN && t == 0) a.seg_fade[slot * parts + part] = fade;
}

// States at the segments' starts (BACK: their gradients at the segments' ends) in the place of the segments' own.
template <int N, bool BACK> __global__ __launch_bounds__(256) void join_kernel(ScanArgs a) {
    const int parts = a.n_heads * (a.d_head / kHeadPart), part = blockIdx.y;
    const int e = (blockIdx.z * 256 + threadIdx.x) * 4, n = e / kHeadPart, p = e % kHeadPart;
    const int s = blockIdx.x;
    int32_t lo, len;
    ragged_span(a.seqs, s, lo, len);
    const Part pt = part_of(a, part);
    const int count = max(1, (len + (1 << a.seg_shift) - 1) >> a.seg_shift);
    const int64_t slot0 = (int64_t)(lo >> a.seg_shift) + s;
    const float *start = BACK ? a.dS_out : a.S0;
    f4 S{};
    if (start) S = *reinterpret_cast<const f4 *>(start + state_at<N>(a, s, pt) + (int64_t)n * a.d_head + p);
    for (int k = 0; k < count; ++k) {
        const int64_t x = (slot0 + (BACK ? count - 1 - k : k)) * parts + part;
        f4 *q = reinterpret_cast<f4 *>(a.seg_state + x * N * kHeadPart + e);
        const f4 own = *q;
        *q = S;
        S = S * a.seg_fade[x] + own;
    }
}

template <int N, bool F32, int NTY, bool YF32, int PASS> hipError_t launch_pass(const ScanArgs &a, hipStream_t stream) {
    const int64_t parts = (int64_t)a.n_heads * (a.d_head / kHeadPart), slots = block_slots(a.seqs.n_tokens, a.seqs.n_seq, a.seg_shift);
    hipLaunchKernelGGL((scan_kernel<N, F32, NTY, YF32, PASS>), dim3((uint32_t)((parts + 7) / 8 * 8 * slots)), dim3(256), 0, stream, a);
    return hipGetLastError();
}
template <int N, bool BACK> hipError_t launch_join(const ScanArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL((join_kernel<N, BACK>), dim3(a.seqs.n_seq, a.n_heads * (a.d_head / kHeadPart), N * kHeadPart / 1024), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <int N, bool F32, bool YF32> hipError_t forward(const ScanArgs &a, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.segments && ((e = launch_pass<N, F32, 2, false, kOwn>(a, stream)) != hipSuccess || (e = launch_join<N, false>(a, stream)) != hipSuccess)) return e;
    return launch_pass<N, F32, YF32 ? 3 : 2, YF32, kMain>(a, stream);
}
template <int N, bool F32> hipError_t back(const ScanArgs &a, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.segments && ((e = launch_pass<N, F32, 2, false, kOwnBack>(a, stream)) != hipSuccess || (e = launch_join<N, true>(a, stream)) != hipSuccess)) return e;
    return launch_pass<N, F32, 2, false, kMainBack>(a, stream);
}

// One token of one head a workgroup; a thread has 4 columns of every 16th (d_head 128: 8th) row.  Bound by memory: the
// state goes through registers once.
template <int N, int P, bool F32, bool YF32> __global__ __launch_bounds__(256) void step_kernel(ScanArgs a) {
    constexpr int LANES = P / 4, ROWS = 256 / LANES, COUNT = N / ROWS;
    __shared__ float sB[N], sC[N], sum[4][P];
    const int t = threadIdx.x, w = t >> 6, l = t & 63;
    const int req = blockIdx.x / a.n_heads, h = blockIdx.x - req * a.n_heads, group = h / (a.n_heads / a.n_groups);
    const int32_t slot = a.slot[req];
    if (slot < 0 || slot >= a.n_slots) return;
    const int col = (t % LANES) * 4, row = t / LANES;
    float *p = a.pool + ((int64_t)slot * a.n_heads + h) * N * P + row * P + col;
    f4 S[COUNT];
#pragma unroll
    for (int i = 0; i < COUNT; ++i) S[i] = *reinterpret_cast<const f4 *>(p + i * ROWS * P);
    for (int i = t; i < N; i += 256) {
        sB[i] = ld_elem<F32>(a.B, req * a.b_stride + (int64_t)group * N + i);
        sC[i] = ld_elem<F32>(a.C, req * a.c_stride + (int64_t)group * N + i);
    }
    const float v = ld_elem<F32>(a.raw, req * a.dt_stride + h) + (a.bias ? a.bias[h] : 0.f);
    const float dt = a.softplus ? softplus_of(v) : v, s = dt * a.A[h], fade = expf(s < -150.f ? -150.f : s);
    f4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = ld_elem<F32>(a.x, req * a.x_stride + (int64_t)h * P + col + e);
    __syncthreads();
    f4 y{};
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
        const int n = row + i * ROWS;
        const float k = dt * sB[n], c = sC[n];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            S[i][e] = fmaf(S[i][e], fade, k * x[e]);
            y[e] = fmaf(S[i][e], c, y[e]);
        }
        *reinterpret_cast<f4 *>(p + i * ROWS * P) = S[i];
    }
#pragma unroll
    for (int m = LANES; m < 64; m <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += __shfl_xor(y[e], m, 64);
    if (l < LANES) *reinterpret_cast<f4 *>(&sum[w][col]) = y;
    __syncthreads();
    if (t < P) {
        const float D = a.D ? a.D[h] : 0.f, xt = ld_elem<F32>(a.x, req * a.x_stride + (int64_t)h * P + t);
        st_elem<YF32>(a.y, (int64_t)blockIdx.x * P + t, fmaf(D, xt, (sum[0][t] + sum[1][t]) + (sum[2][t] + sum[3][t])));
    }
}

template <int N, int P, bool F32> hipError_t step(const ScanArgs &a, bool y_f32, hipStream_t stream) {
    const dim3 grid((uint32_t)a.n * a.n_heads);
    if (y_f32) hipLaunchKernelGGL((step_kernel<N, P, F32, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((step_kernel<N, P, F32, false>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

} // namespace

ScanPlan scan_plan(const sq_scan_desc &d) {
    ScanPlan p{};
    p.parts = (int64_t)d.n_heads * (d.d_head / kHeadPart);
    const int64_t state = (int64_t)d.d_state * kHeadPart * 4;
    // segments of at least 256 tokens, as many as make about 1024 workgroups
    p.seg_shift = kSegMin;
    while (p.seg_shift < 30 && (d.n_tokens >> p.seg_shift) * p.parts > 1024) ++p.seg_shift;
    p.seg_slots = block_slots(d.n_tokens, d.n_seq, p.seg_shift);
    p.chunk_slots = block_slots(d.n_tokens, d.n_seq, 6);
    // the slots of any smaller batch too: at most 1024 workgroups' or one to 256 tokens
    const int64_t by_tokens = d.n_tokens >> kSegMin, by_parts = 1024 / p.parts + 1, most = (by_tokens < by_parts ? by_tokens : by_parts) + d.n_seq;
    p.state_bytes = most * p.parts * state;
    p.fade_bytes = (most * p.parts * 4 + 255) / 256 * 256;
    p.save_bytes = p.chunk_slots * p.parts * state;
    // the gradients' workgroups: a chunk and a subset of a group's heads, 512 to 1023 of them where there are so
    // many heads; the sums over a subset then take less than 1024 x 64 rows of d_state, in smaller batches too
    const int64_t share = d.n_heads / d.n_groups, units = p.chunk_slots * d.n_groups, rows = d.n_tokens * d.n_heads;
    p.subsets = 1;
    while (p.subsets * 2 <= share && units * p.subsets < 512) p.subsets *= 2;
    p.group_bytes = (rows < 1024 * 64 ? rows : 1024 * 64) * d.d_state * 2 * 4;
    p.head_bytes = (3 * 4 * p.chunk_slots * d.n_heads + 255) / 256 * 256;
    return p;
}

hipError_t launch_scan_forward(const ScanArgs &a, int d_state, bool f32, bool y_f32, hipStream_t stream) {
    if (d_state == 128) {
        if (f32) return y_f32 ? forward<128, true, true>(a, stream) : forward<128, true, false>(a, stream);
        return y_f32 ? forward<128, false, true>(a, stream) : forward<128, false, false>(a, stream);
    }
    if (f32) return y_f32 ? forward<64, true, true>(a, stream) : forward<64, true, false>(a, stream);
    return y_f32 ? forward<64, false, true>(a, stream) : forward<64, false, false>(a, stream);
}

hipError_t launch_scan_states_back(const ScanArgs &a, int d_state, bool f32, hipStream_t stream) {
    if (d_state == 128) return f32 ? back<128, true>(a, stream) : back<128, false>(a, stream);
    return f32 ? back<64, true>(a, stream) : back<64, false>(a, stream);
}

hipError_t launch_scan_step(const ScanArgs &a, int d_state, bool f32, bool y_f32, hipStream_t stream) {
    if (d_state == 128) {
        if (a.d_head == 128) return f32 ? step<128, 128, true>(a, y_f32, stream) : step<128, 128, false>(a, y_f32, stream);
        return f32 ? step<128, 64, true>(a, y_f32, stream) : step<128, 64, false>(a, y_f32, stream);
    }
    if (a.d_head == 128) return f32 ? step<64, 128, true>(a, y_f32, stream) : step<64, 128, false>(a, y_f32, stream);
    return f32 ? step<64, 64, true>(a, y_f32, stream) : step<64, 64, false>(a, y_f32, stream);
}

} // namespace sqk
