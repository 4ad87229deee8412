// Gradients of the selective state-space scan, chunk by chunk, all chunks in parallel.
//
// With the chunk's state S0 at its start (saved by the forward pass), the gradient dS of its state at the
// end (left by the pass back, sq_scan.hip), L_ij = e^{G_i - G_j}, o_j = e^{G_end - G_j}, per head:
//   U_j  = sum_{i >= j} (C_i . B_j) L_ij dy_i + o_j dS^T B_j          dx_j = D dy_j + dt_j U_j
//   V_ij = L_ij dt_j (dy_i . x_j)                                     (i >= j)
//   dC_i = sum_j V_ij B_j + e^{G_i} S0 dy_i,   dB_j = sum_i V_ij C_i + dt_j o_j dS x_j    (summed over a group's heads)
// and of the decays, W_ij = V_ij (C_i . B_j), r_i = e^{G_i} C_i . (S0 dy_i), z_j = dt_j o_j x_j . (dS^T B_j):
//   dg_t = sum_{i >= t > j} W_ij + sum_{i >= t} r_i + sum_{j < t} z_j + e^{G_end} <S0, dS>
//   ddt_j = U_j . x_j + A dg_j,   dA = sum dt dg,   draw = ddt sigma(raw + bias),   dbias = sum draw,   dD = sum dy . x
// The first sum of dg_t is sum_{i >= t} (sum_{j < i} W_ij) - sum_{j >= t} (sum_{i > j} W_ij): pairs (i, i) are in
// neither, so that strong decays, where all others are small, keep a small dg's accuracy.
// dC and dB share V's sum over the heads, so their products over pairs of tokens are formed once for a group.
//
// A workgroup has a chunk and some heads of a group, one after another; dB and dC stay in registers.
// Eight waves: in the products over the state, wave w has 16 of its rows; in U, 16 columns.
#include "sq_scan.h"

namespace sqk {
namespace {

constexpr int kThreads = 512;

template <int N, bool F32> struct GradLds {
    typedef Elem<F32> E;
    E B[TokenMat<F32, N>::SIZE], C[TokenMat<F32, N>::SIZE];
    E x[TokenMat<F32, kHeadPart>::SIZE], dy[TokenMat<F32, kHeadPart>::SIZE];
    E dS[LdsMat<F32, 2, kHeadPart, N>::BYTES / sizeof(E)];   // [row of the state][column], two terms
    E pair[LdsMat<F32, 2, 64, 64>::BYTES / sizeof(E)];       // [j][i]
    Gates g;
    float row[10][16], col[10][16], diag[64];  // sums of W over a tile's rows and columns; dy . x
    float r[N / 16][64], z[4][64], u[4][64], e[N / 16];
};

template <int N, bool F32> __global__ __launch_bounds__(kThreads) void grad_kernel(ScanArgs a, int64_t slots) {
    typedef Elem<F32> E;
    constexpr int NT = N / 16, KB = N / 32, TT = NT / 2;  // TT: token tiles of a wave in the products over the state
    typedef TokenMat<F32, N> KeyMat;
    typedef TokenMat<F32, kHeadPart> XMat;
    typedef LdsMat<F32, 2, kHeadPart, N> StateMat;
    typedef LdsMat<F32, 2, 64, 64> PairMat;
    typedef Operand<F32, kSaveTerms, 2> Saved;
    __shared__ __attribute__((aligned(16))) GradLds<N, F32> s;

    const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63, r = l & 15, g4 = (l >> 4) * 4, g8 = (l >> 4) * 8;
    const uint32_t sets = (uint32_t)a.n_groups * a.subsets;
    const int64_t slot = blockIdx.x / sets;
    const int set = (int)(blockIdx.x % sets), subset = set % a.subsets, group = set / a.subsets;
    const int halves = a.d_head / kHeadPart, share = a.n_heads / a.n_groups, parts = a.n_heads * halves;
    const int h0 = group * share + share * subset / a.subsets, h1 = group * share + share * (subset + 1) / a.subsets;
    const Block b = block_at(a.seqs, slot, 6);
    const int rows = b.seq < 0 ? 0 : min(64, b.len - b.c * 64);
    if (rows <= 0) {  // its sums are read all the same
        for (int i = t; i < 3 * (h1 - h0); i += kThreads) a.head_part[(i % 3 * slots + slot) * a.n_heads + h0 + i / 3] = 0.f;
        return;
    }
    const int64_t t0 = (int64_t)b.t0 + b.c * 64, y_stride = (int64_t)a.n_heads * a.d_head;
    Staged<F32, N, kThreads> rB, rC;
    Staged<F32, kHeadPart, kThreads> rX, rY;
    rB.load(static_cast<const E *>(a.B) + t0 * a.b_stride + (int64_t)group * N, a.b_stride, rows, t);
    rC.load(static_cast<const E *>(a.C) + t0 * a.c_stride + (int64_t)group * N, a.c_stride, rows, t);
    rB.store(s.B, t);
    rC.store(s.C, t);
    if (w < 2) PairMat::put4(s.pair, 32 * w + 16 + r, 32 * w + g4, f4{});  // (i tile, j tile) = (0, 1), (2, 3): no pairs
    __syncthreads();

    // the pairs of tokens, tiles w and w + 8 of ten: rows i, columns j
    f4 cb[2], V[2] = {};
    int it[2], jt[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int n = min(w + 8 * k, 9);
        pair_tile(n, it[k], jt[k]);
        cb[k] = f4{};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) cb[k] = mma<1>(KeyMat::get(s.C, 16 * it[k] + r, 32 * kb + g8), KeyMat::get(s.B, 16 * jt[k] + r, 32 * kb + g8), cb[k]);
    }
    const int tiles = w < 2 ? 2 : 1;
    // the products over the state: rows 16 nt .., token tiles tt0 ..
    const int nt = w % NT, tt0 = w / NT * TT;
    f4 dB[TT] = {}, dC[TT] = {};
    float ddt = 0.f, dyx = 0.f, dg = 0.f;  // wave 0: a head's sums, a token to a lane

    for (int v = h0 * halves; v < h1 * halves; ++v) {
        const Part pt = part_of(a, v);
        const int64_t col = (int64_t)pt.head * a.d_head + pt.col;
        rX.load(static_cast<const E *>(a.x) + t0 * a.x_stride + col, a.x_stride, rows, t);
        rY.load(static_cast<const E *>(a.dy) + t0 * y_stride + col, y_stride, rows, t);
        const int64_t at = (slot * parts + v) * N * kHeadPart * 4;
        Frag<F32, 2> fS[2], fD[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            fS[kb] = Saved::get(reinterpret_cast<const E *>(a.save + at), nt, kb, l);
            fD[kb] = Saved::get(reinterpret_cast<const E *>(a.grad_save + at), nt, kb, l);
        }
        const float A = a.A[pt.head], bias = a.bias ? a.bias[pt.head] : 0.f, D = a.D ? a.D[pt.head] : 0.f;
        float raw = 0.f;
        if (w == 0) {
            raw = ld_elem<F32>(a.raw, (t0 + min(l, rows - 1)) * a.dt_stride + pt.head);
            make_gates(s.g, l, l < rows, raw, bias, A, a.softplus);
        }
        rX.store(s.x, t);
        rY.store(s.dy, t);
        if (tt0 == 0)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                E *p = s.dS + (16 * nt + r) * StateMat::ROW + 32 * kb + g8;
                if constexpr (F32) {
                    *reinterpret_cast<f4 *>(p) = fD[kb].v[0];
                    *reinterpret_cast<f4 *>(p + 4) = fD[kb].v[1];
                } else {
                    *reinterpret_cast<bf8 *>(p) = fD[kb].t[0];
                    *reinterpret_cast<bf8 *>(p + StateMat::PLANE) = fD[kb].t[1];
                }
            }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k < tiles) {
                f4 xy{};
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) xy = mma<1>(XMat::get(s.dy, 16 * it[k] + r, 32 * kb + g8), XMat::get(s.x, 16 * jt[k] + r, 32 * kb + g8), xy);
                const int j = 16 * jt[k] + r;
                const float dt = s.g.dt[j];
                f4 m, W;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 16 * it[k] + g4 + e;
                    const float L = i >= j ? decay_of(s.g, i, j) : 0.f;
                    m[e] = i >= j ? L * cb[k][e] : 0.f;
                    const float vv = i >= j ? L * dt * xy[e] : 0.f;
                    V[k][e] += vv;
                    W[e] = i > j ? vv * cb[k][e] : 0.f;
                    if (i == j) s.diag[i] = xy[e];
                }
                PairMat::put4(s.pair, j, 16 * it[k] + g4, m);
                float down = (W[0] + W[1]) + (W[2] + W[3]);
                down += __shfl_xor(down, 16, 64);
                down += __shfl_xor(down, 32, 64);
#pragma unroll
                for (int q = 1; q < 16; q <<= 1)
#pragma unroll
                    for (int e = 0; e < 4; ++e) W[e] += __shfl_xor(W[e], q, 64);
                const int n = w + 8 * k;
                if (l < 16) s.col[n][l] = down;
                if (r == 0) *reinterpret_cast<f4 *>(&s.row[n][g4]) = W;
            }
        }
        {
            float e = 0.f;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if constexpr (F32)
                        e = fmaf(fS[kb].v[k / 4][k % 4], fD[kb].v[k / 4][k % 4], e);
                    else
                        e = fmaf((float)fS[kb].t[0][k] + (float)fS[kb].t[1][k], (float)fD[kb].t[0][k] + (float)fD[kb].t[1][k], e);
                }
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) e += __shfl_xor(e, m, 64);
            if (tt0 == 0 && l == 0) s.e[nt] = e;
        }
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            const int i = 16 * (tt0 + k) + r;
            f4 c{}, d{};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                c = mma<2>(fS[kb], XMat::get(s.dy, i, 32 * kb + g8), c);
                d = mma<2>(fD[kb], XMat::get(s.x, i, 32 * kb + g8), d);
            }
            c *= s.g.in[i];
            dC[k] += c;
            dB[k] += d * (s.g.out[i] * s.g.dt[i]);
            float dot = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) dot = fmaf(c[e], ld_elem<F32>(s.C, i * KeyMat::ROW + 16 * nt + g4 + e), dot);
            dot += __shfl_xor(dot, 16, 64);
            dot += __shfl_xor(dot, 32, 64);
            if (l < 16) s.r[nt][i] = dot;
        }
        __syncthreads();
        {   // U, transposed: columns 16 pc .. of the head's part as the result's rows, token tiles jt0, jt0 + 1
            const int pc = w & 3, jt0 = w >> 2 << 1;
            f4 up[2] = {}, us[2] = {};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const Frag<F32, 1> f = get_t<F32, 1>(s.dy, XMat::ROW, 0, 32 * kb, 16 * pc, l);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (kb == 1 || jt0 == 0) up[k] = mma<2>(f, PairMat::get(s.pair, 16 * (jt0 + k) + r, 32 * kb + g8), up[k]);
            }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const Frag<F32, 2> f = get_t<F32, 2>(s.dS, StateMat::ROW, StateMat::PLANE, 32 * kb, 16 * pc, l);
#pragma unroll
                for (int k = 0; k < 2; ++k) us[k] = mma<2>(f, KeyMat::get(s.B, 16 * (jt0 + k) + r, 32 * kb + g8), us[k]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int j = 16 * (jt0 + k) + r, p = 16 * pc + g4;
                const float dt = s.g.dt[j];
                us[k] *= s.g.out[j];
                f4 dx;
                float z = 0.f, u = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = ld_elem<F32>(s.x, j * XMat::ROW + p + e), both = up[k][e] + us[k][e];
                    z = fmaf(us[k][e], x, z);
                    u = fmaf(both, x, u);
                    dx[e] = fmaf(dt, both, D * ld_elem<F32>(s.dy, j * XMat::ROW + p + e));
                }
                z += __shfl_xor(z, 16, 64);
                z += __shfl_xor(z, 32, 64);
                u += __shfl_xor(u, 16, 64);
                u += __shfl_xor(u, 32, 64);
                if (l < 16) s.z[pc][j] = z * dt, s.u[pc][j] = u;
                if (j < rows) st_elem4<F32>(a.dx, (t0 + j) * a.dx_stride + col + p, dx);
            }
        }
        __syncthreads();
        if (w == 0) {
            // a token to a lane; both parts of a head of 128 add to the same sums
            const int ti = l >> 4;
            float up = 0.f, down = 0.f, ri = 0.f, e = 0.f;
            for (int k = 0; k <= ti; ++k) up += s.row[ti * (ti + 1) / 2 + k][r];
            for (int k = ti; k < 4; ++k) down += s.col[k * (k + 1) / 2 + ti][r];
#pragma unroll
            for (int k = 0; k < NT; ++k) ri += s.r[k][l], e += s.e[k];
            const float z = (s.z[0][l] + s.z[1][l]) + (s.z[2][l] + s.z[3][l]);
            ddt += (s.u[0][l] + s.u[1][l]) + (s.u[2][l] + s.u[3][l]);
            dyx += s.diag[l];
            // sums from t on, as the whole less those before t
            const double f = (double)up + ri - down, before = wave_scan(f, l), zs = wave_scan((double)z, l);
            dg += (float)(__shfl(before, 63, 64) - before + f + (zs - z) + (double)s.g.in[63] * e);
            if (pt.col + kHeadPart == a.d_head) {
                const float dt = s.g.dt[l], v0 = raw + bias;
                float draw = fmaf(A, dg, ddt);
                if (a.softplus) draw *= sigmoid_of(v0);
                if (l >= rows) draw = 0.f;
                else st_elem<F32>(a.draw, (t0 + l) * a.ddt_stride + pt.head, draw);
                float sums[3] = {dt * dg, draw, dyx};
#pragma unroll
                for (int m = 1; m < 64; m <<= 1)
#pragma unroll
                    for (int k = 0; k < 3; ++k) sums[k] += __shfl_xor(sums[k], m, 64);
                if (l == 0)
#pragma unroll
                    for (int k = 0; k < 3; ++k) a.head_part[(k * slots + slot) * a.n_heads + pt.head] = sums[k];
                ddt = dyx = dg = 0.f;
            }
        }
        __syncthreads();
    }
    // the pairs' part of dB and dC, for all heads at once
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (k < tiles) PairMat::put4(s.pair, 16 * jt[k] + r, 16 * it[k] + g4, V[k]);
    __syncthreads();
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
        const Frag<F32, 1> fB = get_t<F32, 1>(s.B, KeyMat::ROW, 0, 32 * kb, 16 * nt, l), fC = get_t<F32, 1>(s.C, KeyMat::ROW, 0, 32 * kb, 16 * nt, l);
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            const int tile = tt0 + k;
            if (kb == 0 || tile >= 2) dC[k] = mma<2>(fB, get_t<F32, 2>(s.pair, PairMat::ROW, PairMat::PLANE, 32 * kb, 16 * tile, l), dC[k]);
            if (kb == 1 || tile < 2) dB[k] = mma<2>(fC, PairMat::get(s.pair, 16 * tile + r, 32 * kb + g8), dB[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < TT; ++k) {
        const int i = 16 * (tt0 + k) + r, n = 16 * nt + g4;
        if (i >= rows) continue;
        if (a.subsets > 1) {
            const int64_t plane = (int64_t)a.seqs.n_tokens * a.n_groups * N, at = ((t0 + i) * a.n_groups + group) * N + n;
            *reinterpret_cast<f4 *>(a.group_part + subset * plane + at) = dB[k];
            *reinterpret_cast<f4 *>(a.group_part + (a.subsets + subset) * plane + at) = dC[k];
        } else {
            st_elem4<F32>(a.dB, (t0 + i) * a.db_stride + (int64_t)group * N + n, dB[k]);
            st_elem4<F32>(a.dC, (t0 + i) * a.dc_stride + (int64_t)group * N + n, dC[k]);
        }
    }
}

// dB and dC of a group: its subsets' sums added up, in their order.
template <int N, bool F32> __global__ __launch_bounds__(256) void group_sum_kernel(ScanArgs a) {
    const Block b = block_at(a.seqs, blockIdx.x, 6);
    if (b.seq < 0) return;
    const int rows = min(64, b.len - b.c * 64), group = blockIdx.y;
    const int64_t t0 = (int64_t)b.t0 + b.c * 64, plane = (int64_t)a.seqs.n_tokens * a.n_groups * N;
    const float *part = a.group_part + blockIdx.z * a.subsets * plane;
    void *out = blockIdx.z ? a.dC : a.dB;
    const int64_t stride = blockIdx.z ? a.dc_stride : a.db_stride;
    for (int i = threadIdx.x; i < rows * N / 4; i += 256) {
        const int row = i / (N / 4), n = i % (N / 4) * 4;
        const int64_t at = ((t0 + row) * a.n_groups + group) * N + n;
        f4 sum{};
        for (int k = 0; k < a.subsets; ++k) sum += *reinterpret_cast<const f4 *>(part + k * plane + at);
        st_elem4<F32>(out, (t0 + row) * stride + (int64_t)group * N + n, sum);
    }
}

template <int N, bool F32> hipError_t gradients(const ScanArgs &a, hipStream_t stream) {
    const uint32_t slots = (uint32_t)block_slots(a.seqs.n_tokens, a.seqs.n_seq, 6);
    hipLaunchKernelGGL((grad_kernel<N, F32>), dim3(slots * a.n_groups * a.subsets), dim3(kThreads), 0, stream, a, (int64_t)slots);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.subsets > 1) {
        hipLaunchKernelGGL((group_sum_kernel<N, F32>), dim3(slots, a.n_groups, 2), dim3(256), 0, stream, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int64_t plane = (int64_t)slots * a.n_heads;
    const SumArgs s[3] = {{a.head_part, a.dA, slots, a.n_heads, a.n_heads}, {a.head_part + plane, a.dbias, slots, a.n_heads, a.n_heads},
                          {a.head_part + 2 * plane, a.dD, slots, a.n_heads, a.n_heads}};
    return launch_column_sums(s, 3, stream);
}

} // namespace

hipError_t launch_scan_backward(const ScanArgs &a, int d_state, bool f32, hipStream_t stream) {
    const hipError_t e = launch_scan_states_back(a, d_state, f32, stream);
    if (e != hipSuccess) return e;
    if (d_state == 128) return f32 ? gradients<128, true>(a, stream) : gradients<128, false>(a, stream);
    return f32 ? gradients<64, true>(a, stream) : gradients<64, false>(a, stream);
}

} // namespace sqk
