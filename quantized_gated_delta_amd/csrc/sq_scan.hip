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
// The gradients' pass back over the chunks is the same with C, dy and e^G for B, x and e^{G_end - G} dt, from the
// last chunk to the first, and what it reads with B is x's gradient: with dS the gradient of the state at a chunk's end,
//   U_j = sum_{i >= j} (C_i . B_j) L_ij dy_i + e^{G_end - G_j} dS^T B_j,   dx_j = D dy_j + dt_j U_j
// It leaves dS, and the dots of x_j with U_j and with its second part, for the other gradients (sq_scan_bwd.hip).
#include "sq_scan.h"

#include <cstdint>

namespace sqk {
namespace {

// What a pass over the chunks does: form a segment's own state; form y; the same two backwards.
enum Pass { kOwn, kMain, kOwnBack, kMainBack };
constexpr int kGates = 4;  // chunks whose gates are formed at once, one by each wave

// The main passes, forwards and (in brackets) backwards.  The state takes up the keys K = B [C] with the
// columns X = x [dy], and is read by the queries Q = C [B]; a query meets the keys of its own
// chunk up to [from] its own place in `pairs`.  NT: terms that the results are accurate to.
// What bounds it: two workgroups to a CU by registers and LDS (fp32 with d_state 128: one, of 107 KB), which hold LDS (0.44 of the cycles) and vector instructions
// (0.39) busy with the matrix units at 0.21; a chunk takes 8000 cycles alone.  8192 tokens x 64 heads, d_state 128, d_head
// 64, bf16: own pass 44 us, main pass 100 to 105; x 32 heads in training, with the states saved: 28, 74 to 81, back 27 and 91
// to 100.
template <int N, bool F32, int NT, bool YF32, int PASS, bool SAVE>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) void scan_kernel(ScanArgs a) {
    typedef Elem<F32> E;
    constexpr bool BACK = PASS >= kOwnBack, READ = PASS == kMain || PASS == kMainBack;
    constexpr int MT = N / 16, KB = N / 32;
    typedef TokenMat<F32, N> KeyMat;
    typedef TokenMat<F32, kHeadPart> XMat;
    typedef LdsMat<F32, NT, 64, 64> PairMat;
    __shared__ __attribute__((aligned(16))) E sK[KeyMat::SIZE], sX[XMat::SIZE];
    __shared__ __attribute__((aligned(16))) E sQ[READ ? KeyMat::SIZE : 8];
    __shared__ __attribute__((aligned(16))) E pairs[READ ? PairMat::BYTES / sizeof(E) : 8];  // [query][key]
    __shared__ Gates gates[kGates];
    __shared__ float dots[2][PASS == kMainBack ? 4 : 1][64];

    const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63, r = l & 15, g4 = (l >> 4) * 4;
    // the heads of a group read the same B and C: workgroups go to the 8 XCDs in turn, and each
    // XCD gets neighbouring heads
    const int parts = a.n_heads * (a.d_head / kHeadPart), each = (parts + 7) / 8;
    const uint32_t turn_of = blockIdx.x >> 3;
    const uint32_t slot = __builtin_amdgcn_readfirstlane(turn_of / each);
    const int part = (blockIdx.x & 7) * each + (turn_of - slot * each);
    if (part >= parts) return;
    const Block b = block_at(a.seqs, slot, a.seg_shift);
    if (b.seq < 0) return;
    const Part pt = part_of(a, part);
    const int begin = b.c << a.seg_shift, len = min(b.len - begin, 1 << a.seg_shift), n_chunks = (len + 63) >> 6;
    const int64_t t0 = (int64_t)b.t0 + begin, at = state_at<N>(a, b.seq, pt);
    const int64_t chunk0 = ((int64_t)(b.t0 >> 6) + b.seq + (begin >> 6)) * parts + part;  // + c * parts
    float *seg = a.seg_state + ((int64_t)slot * parts + part) * N * kHeadPart;

    // the state: a wave has 16 columns, a lane rows 16 m + 4 (l / 16) .. + 3 of column l % 16, times sign_of(m)
    f4 S[MT];
    {
        const float *start = BACK ? a.dS_out : a.S0, *p = !READ ? nullptr : a.segments ? seg : start ? start + at : nullptr;
        const int64_t row = a.segments ? kHeadPart : a.d_head;
#pragma unroll
        for (int m = 0; m < MT; ++m) S[m] = f4{};
        if (p) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[m][i] = p[(16 * m + g4 + i) * row + 16 * w + r];
#pragma unroll
            for (int m = 1; m < MT; m += 2) S[m] = -S[m];
        }
    }
    const float A = a.A[pt.head], bias = a.bias ? a.bias[pt.head] : 0.f, D = READ && a.D ? a.D[pt.head] : 0.f;
    const int64_t y_stride = (int64_t)a.n_heads * a.d_head, column = (int64_t)pt.head * a.d_head + pt.col;
    const int64_t k_stride = BACK ? a.c_stride : a.b_stride, q_stride = BACK ? a.b_stride : a.c_stride, x_stride = BACK ? y_stride : a.x_stride;
    constexpr int OUT = BACK ? sizeof(E) : YF32 ? 4 : 2;  // bytes of an element of y [of x's gradient]
    const int64_t out_stride = BACK ? a.dx_stride : y_stride;
    const uint32_t out_bytes = (uint32_t)out_stride * OUT;
    const E *pk = static_cast<const E *>(BACK ? a.C : a.B) + t0 * k_stride + (int64_t)pt.group * N;
    const E *pq = static_cast<const E *>(BACK ? a.B : a.C) + t0 * q_stride + (int64_t)pt.group * N;
    const E *px = static_cast<const E *>(BACK ? a.dy : a.x) + t0 * x_stride + column;

    const int first = BACK ? n_chunks - 1 : 0, step = BACK ? -1 : 1;
    auto rows_of = [&](int c) { return min(64, len - c * 64); };
    Staged<F32, N, 256> rK, rQ;
    Staged<F32, kHeadPart, 256> rX;
    Raw<F32, 4> next_x[PASS == kMainBack ? 4 : 1];  // what U's dots are with: a lane's four columns of a token of each tile
    auto load = [&](int c) {
        const int rows = rows_of(c);
        if (PASS == kMainBack)
#pragma unroll
            for (int qt = 0; qt < 4; ++qt)
                next_x[qt] = load_n<F32, true, 4>(at_bytes<E>(static_cast<const E *>(a.x) + (t0 + (int64_t)c * 64) * a.x_stride + column,
                                                             (min(16 * qt + r, rows - 1) * (uint32_t)a.x_stride + 16 * w + g4) * (uint32_t)sizeof(E)), 0, 4);
        rK.load(pk + (int64_t)c * 64 * k_stride, (uint32_t)k_stride, rows, t);
        rX.load(px + (int64_t)c * 64 * x_stride, (uint32_t)x_stride, rows, t);
        if (READ) rQ.load(pq + (int64_t)c * 64 * q_stride, (uint32_t)q_stride, rows, t);
    };
    // what wave w forms gates from: its chunk of the kGates from the k-th on
    float raw = 0.f;
    auto load_raw = [&](int k) {
        if (k + w < n_chunks) {
            const int c = first + (k + w) * step;
            raw = ld_elem<F32>(a.raw, (t0 + (int64_t)c * 64 + min(l, rows_of(c) - 1)) * a.dt_stride + pt.head);
        }
    };
    load_raw(0);
    if (n_chunks > 0) load(first);
    // tiles beside the diagonal that a contraction over 32 keys meets and no pair fills
    if (READ && w < 2) PairMat::put4(pairs, 32 * w + (BACK ? 16 : 0) + r, 32 * w + (BACK ? 0 : 16) + g4, f4{});
    float fade = 1.f;
    for (int k = 0; k < n_chunks; ++k) {
        const int c = first + k * step, rows = rows_of(c);
        const Gates &g = gates[k % kGates];
        // addresses in LDS are formed again for each chunk where there is no room to keep them
        int lane = threadIdx.x;
        if (PASS == kMainBack) asm volatile("" : "+v"(lane));
        const int t = lane, l = t & 63, r = l & 15, g4 = (l >> 4) * 4, g8 = (l >> 4) * 8;
        // signs: the state's odd tiles of rows are turned, and so is what every second tile of queries reads
        rK.template store<false, true>(sK, t);
        rX.clear(rows, t);  // behind the end: what nothing is taken up of
        rX.store(sX, t);
        if (READ) rQ.template store<true, true>(sQ, t);
        if (k % kGates == 0 && k + w < n_chunks) make_gates(gates[w], l, l < rows_of(first + (k + w) * step), raw, bias, A, a.softplus);
        Raw<F32, 4> this_x[PASS == kMainBack ? 4 : 1];
#pragma unroll
        for (int qt = 0; qt < (PASS == kMainBack ? 4 : 1); ++qt) this_x[qt] = next_x[qt];
        __syncthreads();
        if (k % kGates == 0) load_raw(k + kGates);
        if (k + 1 < n_chunks) load(c + step);
        if (SAVE) {  // [row][column], fp32
            float *keep = reinterpret_cast<float *>(BACK ? a.grad_save : a.save) + (chunk0 + (int64_t)c * parts) * N * kHeadPart;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) *at_bytes<float>(keep + (16 * m + i) * kHeadPart, (g4 * kHeadPart + 16 * w + r) * 4) = sign_of(m) * S[m][i];
        }
        if (READ) {
            // ten tiles: w, w + 4, w + 8; the last one three times rather than behind a branch, so that each step is
            // taken for a wave's three together
            int kt[3], qt[3];
            f4 p[3] = {};
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                int hi, lo;
                pair_tile(min(w + 4 * j, 9), hi, lo);
                kt[j] = BACK ? hi : lo, qt[j] = BACK ? lo : hi;
            }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                Frag<F32, 1> fk[3], fq[3];
#pragma unroll
                for (int j = 0; j < 3; ++j) fk[j] = KeyMat::get(sK, 16 * kt[j] + r, 32 * kb + g8), fq[j] = KeyMat::get(sQ, 16 * qt[j] + r, 32 * kb + g8);
                mma_all<1, 3, false, false>(fk, fq, p);
            }
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                if (!BACK) p[j] *= *reinterpret_cast<const f4 *>(&g.dt[16 * kt[j] + g4]);
                p[j] = decayed<BACK>(g, p[j], 16 * kt[j] + g4, 16 * qt[j] + r);  // behind dt, whose NaN stays with the pairs that meet
            }
#pragma unroll
            for (int j = 0; j < 3; ++j) PairMat::put4(pairs, 16 * qt[j] + r, 16 * kt[j] + g4, p[j]);
            __syncthreads();
        }
        Frag<F32, 1> fx[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) fx[kb] = get_t<F32, 1>(sX, XMat::ROW, 0, 32 * kb, 16 * w, l);
        if (READ) {
            // transposed, the result's columns as its rows: a lane then holds four neighbours of one token
            f4 y[4] = {}, y_out[4];
            // a block's operands, the next one's on their way (main pass 87 -> 81 us, pass back, which has fewer registers
            // left, 100 without and 102 with; 8192 tokens x 32 heads)
            constexpr bool AHEAD = PASS == kMain;
            Frag<F32, 1> fq[AHEAD ? 2 : 1][4];
            auto queries = [&](int kb) {
#pragma unroll
                for (int qt = 0; qt < 4; ++qt) fq[AHEAD ? kb & 1 : 0][qt] = KeyMat::get_split(sQ, 16 * qt + r, 32 * kb + g4);
            };
            if (AHEAD) queries(0);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                if (!AHEAD) queries(kb);
                else if (kb + 1 < KB) queries(kb + 1);
                __builtin_amdgcn_sched_barrier(0);  // all blocks' operands at once would not fit the registers
                float s[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = S[2 * kb + e / 4][e % 4];
                const Frag<F32, NT> fs = make_frag<F32, NT>(s);
                mma_all<NT, 4, true, false>(&fs, fq[AHEAD ? kb & 1 : 0], y);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int qt = 0; qt < 4; ++qt) {
                const int q = 16 * qt + r;
                y[qt] *= BACK ? g.out[q] : g.in[q];
                const f4 own = load4<F32>(sX + XMat::at(q) * XMat::ROW + 16 * w + g4);
                float x[4], z = 0.f, u = 0.f;
                if (BACK) {
                    widen_n<F32, 4>(this_x[PASS == kMainBack ? qt : 0], x);
                    z = sign_of(qt) * ((x[0] * y[qt][0] + x[1] * y[qt][1]) + (x[2] * y[qt][2] + x[3] * y[qt][3]));
                }
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
                    if (BACK ? kb == 1 || qt < 2 : kb == 0 || qt >= 2) y[qt] = mma<NT>(fx[kb], PairMat::get(pairs, q, 32 * kb + g8), y[qt]);
                y[qt] *= sign_of(qt);
                if (BACK) {
                    u = (x[0] * y[qt][0] + x[1] * y[qt][1]) + (x[2] * y[qt][2] + x[3] * y[qt][3]);
                    z = rows_sum(z), u = rows_sum(u);
                    if (l < 16) dots[0][w][q] = z * g.dt[q], dots[1][w][q] = u;
                    y[qt] *= g.dt[q];
                }
                y[qt] += own * D;
                y_out[qt] = y[qt];
            }
            // whole chunks store without branches, so that the next one's loads are waited for by count and
            // not for the stores behind them
            char *py = static_cast<char *>(BACK ? a.dx : a.y) + ((t0 + (int64_t)c * 64) * out_stride + column) * OUT;
            if (rows == 64) {
#pragma unroll
                for (int qt = 0; qt < 4; ++qt) st_elem4<OUT == 4>(at_bytes<char>(py, (16 * qt + r) * out_bytes + (16 * w + g4) * OUT), 0, y_out[qt]);
            } else {
#pragma unroll
                for (int qt = 0; qt < 4; ++qt)
                    if (16 * qt + r < rows) st_elem4<OUT == 4>(at_bytes<char>(py, (16 * qt + r) * out_bytes + (16 * w + g4) * OUT), 0, y_out[qt]);
                __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
            }
        }
        // the state: the scaled X as the right operand, three terms, so that the state has fp32 accuracy
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
        for (int m = 0; m < MT; ++m) S[m] *= whole;
        if (READ) {
            constexpr bool AHEAD = PASS == kMain;
            Frag<F32, 1> fk[AHEAD ? 2 : 1][4];  // of four tiles of rows
            auto keys = [&](int n) {
#pragma unroll
                for (int m = 0; m < 4; ++m) fk[AHEAD ? n & 1 : 0][m] = get_t<F32, 1>(sK, KeyMat::ROW, 0, 32 * (n & 1), 16 * (n / 2 * 4 + m), l);
            };
            if (AHEAD) keys(0);
#pragma unroll
            for (int n = 0; n < MT / 2; ++n) {
                if (!AHEAD) keys(n);
                else if (n + 1 < MT / 2) keys(n + 1);
                __builtin_amdgcn_sched_barrier(0);
                mma_all<3, 4, false, true>(fk[AHEAD ? n & 1 : 0], &fs[n & 1], S + n / 2 * 4);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {  // as the compiler orders it: 28 us, in the order above 29 (8192 tokens x 32 heads)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) S[m] = mma<3>(get_t<F32, 1>(sK, KeyMat::ROW, 0, 32 * kb, 16 * m, l), fs[kb], S[m]);
                if (m % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
        }
        __syncthreads();
        if (PASS == kMainBack) {  // 0: z, 1: u; waves 2 and 3 store the same again
            const int n = w & 1;
            a.dots[(n * a.chunk_parts + chunk0 + (int64_t)c * parts) * 64 + l] = (dots[n][0][l] + dots[n][1][l]) + (dots[n][2][l] + dots[n][3][l]);
        }
    }
    const bool end = BACK ? b.c == 0 : b.len - begin <= 1 << a.seg_shift;
    float *to = !READ ? seg : !end ? nullptr : BACK ? a.dS0 : a.S_out;
    if (to) {
        const int64_t row = READ ? a.d_head : kHeadPart;
        if (READ) to += at;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) to[(16 * m + g4 + i) * row + 16 * w + r] = sign_of(m) * S[m][i];
    }
    if (!READ && t == 0) a.seg_fade[(int64_t)slot * parts + part] = fade;
}

// States at the segments' starts (BACK: their gradients at the segments' ends) in the place of the segments' own: bound by
// memory and its latency (8 segments of 64 heads, 34 MB: 7 us).
template <int N, bool BACK> __global__ __launch_bounds__(256) void join_kernel(ScanArgs a) {
    const int parts = a.n_heads * (a.d_head / kHeadPart), part = blockIdx.y;
    const int e = (blockIdx.z * 256 + threadIdx.x) * 4, n = e / kHeadPart, p = e % kHeadPart;
    const int s = blockIdx.x;
    int32_t lo, len;
    ragged_span(a.seqs, s, lo, len);
    const Part pt = part_of(a, part);
    const int count = max(1, ((len - 1) >> a.seg_shift) + 1);
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

template <int N, bool F32, int NT, bool YF32, int PASS, bool SAVE = false> hipError_t launch_pass(const ScanArgs &a, hipStream_t stream) {
    const int64_t parts = (int64_t)a.n_heads * (a.d_head / kHeadPart), slots = block_slots(a.seqs.n_tokens, a.seqs.n_seq, a.seg_shift);
    hipLaunchKernelGGL((scan_kernel<N, F32, NT, YF32, PASS, SAVE>), dim3((uint32_t)((parts + 7) / 8 * 8 * slots)), dim3(256), 0, stream, a);
    return hipGetLastError();
}
template <int N, bool BACK> hipError_t launch_join(const ScanArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL((join_kernel<N, BACK>), dim3(a.seqs.n_seq, a.n_heads * (a.d_head / kHeadPart), N * kHeadPart / 1024), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <int N, bool F32, bool YF32> hipError_t forward(const ScanArgs &a, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.segments && ((e = launch_pass<N, F32, 2, false, kOwn>(a, stream)) != hipSuccess || (e = launch_join<N, false>(a, stream)) != hipSuccess)) return e;
    constexpr int NT = YF32 ? 3 : 2;
    return a.save ? launch_pass<N, F32, NT, YF32, kMain, true>(a, stream) : launch_pass<N, F32, NT, YF32, kMain>(a, stream);
}
template <int N, bool F32> hipError_t back(const ScanArgs &a, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.segments && ((e = launch_pass<N, F32, 2, false, kOwnBack>(a, stream)) != hipSuccess || (e = launch_join<N, true>(a, stream)) != hipSuccess)) return e;
    return launch_pass<N, F32, 3, false, kMainBack, true>(a, stream);
}

// One token of one head a workgroup; a thread has 4 columns of every 16th (d_head 128: 8th) row.  Bound by memory: the
// state goes through registers once, past the caches, which no other reader would find it in (512 requests x 64 heads, 2.1 GB:
// 385 us, 5.6 TB/s; through the caches 417).
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
    for (int i = 0; i < COUNT; ++i) S[i] = __builtin_nontemporal_load(reinterpret_cast<const f4 *>(p + i * ROWS * P));
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
        __builtin_nontemporal_store(S[i], reinterpret_cast<f4 *>(p + i * ROWS * P));
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
    // segments of at least 256 tokens, as many as make 512 workgroups, two to a CU (1024: as long in the passes over the
    // chunks, and twice as many states to join, 15 us for 8 at 8192 tokens x 32 heads)
    p.seg_shift = kSegMin;
    while (p.seg_shift < 30 && (d.n_tokens >> p.seg_shift) * p.parts > kSegGroups) ++p.seg_shift;
    p.seg_slots = block_slots(d.n_tokens, d.n_seq, p.seg_shift);
    p.chunk_slots = block_slots(d.n_tokens, d.n_seq, 6);
    // the slots of any smaller batch too: at most those workgroups' or one to 256 tokens
    const int64_t by_tokens = d.n_tokens >> kSegMin, by_parts = kSegGroups / p.parts + 1, most = (by_tokens < by_parts ? by_tokens : by_parts) + d.n_seq;
    p.state_bytes = most * p.parts * state;
    p.fade_bytes = (most * p.parts * 4 + 255) / 256 * 256;
    p.save_bytes = p.chunk_slots * p.parts * state;
    // the gradients' workgroups, one to a CU: a chunk and a subset of a group's heads.  Of up to 1023 workgroups (the sums over
    // a subset then take less than 1024 x 64 rows of d_state, in smaller batches too), as many subsets as
    // take the fewest rounds of 256 times heads, with two heads' time to begin and end (132 chunks x 32 heads, when the kernel
    // took 183 us with 3 subsets: 4, which need a third round, 195; now 166 with 3)
    const int64_t share = d.n_heads / d.n_groups, units = p.chunk_slots * d.n_groups, rows = d.n_tokens * d.n_heads;
    p.subsets = 1;
    int64_t least = INT64_MAX;
    for (int64_t n = 1; n <= share && (n == 1 || units * n < 1024); ++n) {
        const int64_t cost = (units * n + 255) / 256 * ((share + n - 1) / n + 2);
        if (cost < least) least = cost, p.subsets = (int)n;
    }
    p.group_bytes = (rows < 1024 * 64 ? rows : 1024 * 64) * d.d_state * 2 * 4;
    p.dots_bytes = 2 * 4 * 64 * p.chunk_slots * p.parts;
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
