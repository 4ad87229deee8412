// Gradients of the selective state-space scan, chunk by chunk, all chunks in parallel.
//
// With the chunk's state S0 at its start (saved by the forward pass), the gradient dS of its state at the
// end, U and x's gradient (left by the pass back, sq_scan.hip), L_ij = e^{G_i - G_j}, o_j = e^{G_end - G_j}, per head:
//   V_ij = L_ij dt_j (dy_i . x_j)                                     (i >= j)
//   dC_i = sum_j V_ij B_j + e^{G_i} S0 dy_i,   dB_j = sum_i V_ij C_i + dt_j o_j dS x_j    (summed over a group's heads)
// and of the decays, W_ij = V_ij (C_i . B_j), r_i = e^{G_i} C_i . (S0 dy_i), z_j = dt_j o_j x_j . (dS^T B_j):
//   dg_t = sum_{i >= t > j} W_ij + sum_{i >= t} r_i + sum_{j < t} z_j + e^{G_end} <S0, dS>
//   ddt_j = U_j . x_j + A dg_j,   dA = sum dt dg,   draw = ddt sigma(raw + bias),   dbias = sum draw,   dD = sum dy . x
// The first sum of dg_t is formed without differences, from a 16 x 16 tile's sums over rows and columns where
// t is beside the tile's diagonal, and on the diagonal from its sums over i >= t of each column: as a difference of sums
// over the chunk, rounding errors of all its pairs would reach every t (dbias 1.0e-6 off for 4.2e-7, fp32, d_state 64).
// dC and dB share V's sum over the heads, so their products over pairs of tokens are formed once for a group.
//
// A workgroup has a chunk and some heads of a group, one part after another; dB and dC stay in registers.
// Eight waves: in the products over the state, wave w has 16 of its rows; the next part's states and tokens
// are in flight meanwhile.  Of kBatch parts at once, each wave forms the gates of one before, and its dg after.
// One workgroup to a CU, whose waves wait 0.59 of their cycles: for the states' 64 KB a head (8192 tokens x 32 heads, d_state
// 128, d_head 64, bf16, 330 MB: 166 us, 2.0 TB/s; 153 with them in L2), at the barriers, and in 396 workgroups on 256 CUs.
#include "sq_scan.h"

namespace sqk {
namespace {

constexpr int kThreads = 512, kBatch = 8;

// The decay from token j to a token i behind it; 0 where `live` is false.  (sq_scan.h's `decayed` is no faster here, with a wave's
// one or two tiles beside its products over the state, and takes registers that are short: 170 us for 166.)
__device__ __forceinline__ float decay_of(const Gates &g, int i, int j, bool live) {
    const float d = (g.hi[i] - g.hi[j]) + (g.lo[i] - g.lo[j]);
    return __builtin_amdgcn_exp2f(live ? d : -__builtin_inff());
}

template <int N, bool F32> struct GradLds {
    typedef Elem<F32> E;
    E B[TokenMat<F32, N, false>::SIZE], C[TokenMat<F32, N, false>::SIZE];
    E x[TokenMat<F32, kHeadPart, false>::SIZE], dy[TokenMat<F32, kHeadPart, false>::SIZE];  // at the end V, [j][i]
    Gates g[kBatch];
    // of two parts in turn: sums of W over a tile's rows (on the diagonal: what dg has of it), its columns and all of it;
    // dy . x; r and <S0, dS> by rows of the state
    struct Sums { float row[10][16], col[10][16], all[10], diag[64], r[N / 16][64], e[N / 16]; } sums[2];
    float pairs[kBatch][64], r[kBatch][64], diag[kBatch][64], e[kBatch];  // of a batch: dg's sums of W, r, dy . x, <S0, dS>
};

// Eight values of a row of a state in fp32, and the same as an operand.
struct Row8 { f4 v[2]; };
__device__ __forceinline__ Row8 load_row8(const float *p) { return Row8{{*reinterpret_cast<const f4 *>(p), *reinterpret_cast<const f4 *>(p + 4)}}; }
template <bool F32, int NT> __device__ __forceinline__ Frag<F32, NT> operand_of(const Row8 &x) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x.v[e / 4][e % 4];
    return make_frag<F32, NT>(v);
}

template <int N, bool F32>
__global__ __launch_bounds__(kThreads) void grad_kernel(ScanArgs a, int64_t slots) {
    typedef Elem<F32> E;
    constexpr int NT = N / 16, KB = N / 32, TT = NT / 2;  // TT: token tiles of a wave in the products over the state
    typedef TokenMat<F32, N, false> KeyMat;
    typedef TokenMat<F32, kHeadPart, false> XMat;
    typedef LdsMat<F32, 2, 64, 64> PairMat;
    __shared__ __attribute__((aligned(16))) GradLds<N, F32> s;
    static_assert(sizeof(s.x) + sizeof(s.dy) >= PairMat::BYTES, "V takes the place of x and dy");

    const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l = t & 63, r = l & 15, g4 = (l >> 4) * 4, g8 = (l >> 4) * 8;
    const uint32_t sets = (uint32_t)a.n_groups * a.subsets;
    const int64_t slot = __builtin_amdgcn_readfirstlane(blockIdx.x / sets);
    const int set = (int)(blockIdx.x - (uint32_t)slot * sets), group = __builtin_amdgcn_readfirstlane(set / a.subsets), subset = set - group * a.subsets;
    const int halves = a.d_head / kHeadPart, share = a.n_heads / a.n_groups, parts = a.n_heads * halves;
    const int h0 = group * share + __builtin_amdgcn_readfirstlane(share * subset / a.subsets),
              h1 = group * share + __builtin_amdgcn_readfirstlane(share * (subset + 1) / a.subsets);
    const Block b = block_at(a.seqs, slot, 6);
    const int rows = b.seq < 0 ? 0 : min(64, b.len - b.c * 64);
    if (rows <= 0) {  // its sums are read all the same
        for (int i = t; i < 3 * (h1 - h0); i += kThreads) a.head_part[(i % 3 * slots + slot) * a.n_heads + h0 + i / 3] = 0.f;
        return;
    }
    const int64_t t0 = (int64_t)b.t0 + b.c * 64, y_stride = (int64_t)a.n_heads * a.d_head;
    // the products over the state: rows 16 nt .., token tiles tt0 ..
    const int nt = w % NT, tt0 = w / NT * TT, v0 = h0 * halves, v1 = h1 * halves;

    Staged<F32, kHeadPart, kThreads, false> rX, rY;
    Row8 rS[2], rD[2];
    auto load = [&](int v, int t, int r, int g8) {
        const Part pt = part_of(a, v);
        const int64_t col = (int64_t)pt.head * a.d_head + pt.col;
        rX.load(static_cast<const E *>(a.x) + t0 * a.x_stride + col, (uint32_t)a.x_stride, rows, t);
        rY.load(static_cast<const E *>(a.dy) + t0 * y_stride + col, (uint32_t)y_stride, rows, t);
        const int64_t at = ((slot * parts + v) * N + 16 * nt + r) * kHeadPart + g8;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            rS[kb] = load_row8(reinterpret_cast<const float *>(a.save) + at + 32 * kb);
            rD[kb] = load_row8(reinterpret_cast<const float *>(a.grad_save) + at + 32 * kb);
        }
    };
    {
        Staged<F32, N, kThreads, false> rB, rC;
        rB.load(static_cast<const E *>(a.B) + t0 * a.b_stride + (int64_t)group * N, (uint32_t)a.b_stride, rows, t);
        rC.load(static_cast<const E *>(a.C) + t0 * a.c_stride + (int64_t)group * N, (uint32_t)a.c_stride, rows, t);
        load(v0, t, r, g8);
        rB.store(s.B, t);
        rC.store(s.C, t);
    }
    __syncthreads();

    // the pairs of tokens, tiles w and w + 8 of ten: rows i, columns j
    f4 cb[2], V[2] = {};
    int it[2], jt[2];
    const int tiles = w < 2 ? 2 : 1;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        pair_tile(min(w + 8 * k, 9), it[k], jt[k]);
        cb[k] = f4{};
        if (k < tiles)
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) cb[k] = mma<1>(KeyMat::get(s.C, 16 * it[k] + r, 32 * kb + g8), KeyMat::get(s.B, 16 * jt[k] + r, 32 * kb + g8), cb[k]);
    }
    f4 dB[TT] = {}, dC[TT] = {};

    for (int first = v0; first < v1; first += kBatch) {
        const int count = min(kBatch, v1 - first);
        float raw = 0.f, bias = 0.f, A = 0.f, z = 0.f, u = 0.f;  // of part first + w, a token to a lane
        if (w < count) {
            const Part pt = part_of(a, first + w);
            raw = ld_elem<F32>(a.raw, (t0 + min(l, rows - 1)) * a.dt_stride + pt.head);
            bias = a.bias ? a.bias[pt.head] : 0.f;
            A = a.A[pt.head];
            for (int k = max(0, w + 1 - halves); k <= w; ++k) {  // with the head's first part, if this is its second
                const int64_t at = (slot * parts + first + k) * 64 + l;
                z += a.dots[at];
                u += a.dots[a.chunk_parts * 64 + at];
            }
            make_gates(s.g[w], l, l < rows, raw, bias, A, a.softplus);
        }
        for (int q = 0; q < count; ++q) {
            // addresses in LDS are formed again for each part: kept from part to part, they would be spilled, and reading
            // them back would wait for the next part's loads
            int lane = threadIdx.x;
            asm volatile("" : "+v"(lane));
            const int t = lane, l = t & 63, r = l & 15, g4 = (l >> 4) * 4, g8 = (l >> 4) * 8;
            const Gates &g = s.g[q];
            auto &sum = s.sums[q & 1];
            rX.clear(rows, t);
            rY.clear(rows, t);
            rX.store(s.x, t);
            rY.template store<true>(s.dy, t);
            const Frag<F32, 3> fS[2] = {operand_of<F32, 3>(rS[0]), operand_of<F32, 3>(rS[1])};
            const Frag<F32, 2> fD[2] = {operand_of<F32, 2>(rD[0]), operand_of<F32, 2>(rD[1])};
            float e0 = 0.f;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int k = 0; k < 8; ++k) e0 = fmaf(rS[kb].v[k / 4][k % 4], rD[kb].v[k / 4][k % 4], e0);
            __syncthreads();
            if (first + q + 1 < v1) load(first + q + 1, t, r, g8);
            sum.e[nt] = rows_sum(row_sum(e0));  // waves with the same rows of the state: the same
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (k < tiles) {
                    f4 xy{};
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb) xy = mma<1>(XMat::get(s.dy, 16 * it[k] + r, 32 * kb + g8), XMat::get(s.x, 16 * jt[k] + r, 32 * kb + g8), xy);
                    const int j = 16 * jt[k] + r;
                    const float dt = g.dt[j];
                    xy *= sign_of(it[k]);
                    f4 W;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = 16 * it[k] + g4 + e;
                        const float L = decay_of(g, i, j, i >= j) * dt, vv = i >= j ? L * xy[e] : 0.f;
                        V[k][e] += vv;
                        W[e] = i > j ? vv * cb[k][e] : 0.f;
                    }
                    if (it[k] == jt[k]) {  // dy . x: the diagonal, a lane of each row of 16
                        const int e = r - g4;
                        const float d = e == 0 ? xy[0] : e == 1 ? xy[1] : e == 2 ? xy[2] : xy[3];
                        if (e >= 0 && e < 4) sum.diag[j] = d;
                    }
                    float down = (W[0] + W[1]) + (W[2] + W[3]);
                    if (it[k] == jt[k]) {  // the sums of column j over rows i, i + 1, ..., where j < i
                        const float d1 = __shfl_down(down, 16, 64), d2 = __shfl_down(down, 32, 64), d3 = __shfl_down(down, 48, 64);
                        float below = (l < 48 ? d1 : 0.f) + (l < 32 ? d2 : 0.f) + (l < 16 ? d3 : 0.f);
#pragma unroll
                        for (int e = 3; e >= 0; --e) {
                            below += W[e];
                            W[e] = r < g4 + e ? below : 0.f;
                        }
                    }
                    down = rows_sum(down);
                    const float all = row_sum(down);
#pragma unroll
                    for (int e = 0; e < 4; ++e) W[e] = row_sum(W[e]);
                    const int n = w + 8 * k;  // lanes that have the same sum store it all
                    sum.col[n][r] = down;
                    sum.all[n] = all;
                    *reinterpret_cast<f4 *>(&sum.row[n][g4]) = W;
                }
            }
#pragma unroll
            for (int k = 0; k < TT; ++k) {
                const int i = 16 * (tt0 + k) + r;
                f4 c{}, d{};
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    c = mma<3>(fS[kb], XMat::get(s.dy, i, 32 * kb + g8), c);
                    d = mma<2>(fD[kb], XMat::get(s.x, i, 32 * kb + g8), d);
                }
                c *= sign_of(tt0 + k) * g.in[i];
                dC[k] += c;
                dB[k] += d * (g.out[i] * g.dt[i]);
                const f4 key = load4<F32>(s.C + i * KeyMat::ROW + 16 * nt + g4);
                float dot = (c[0] * key[0] + c[1] * key[1]) + (c[2] * key[2] + c[3] * key[3]);
                sum.r[nt][i] = rows_sum(dot);
            }
            __syncthreads();
            if (w == q) {  // a token to a lane
                // tiles of t's rows: sums over i >= t; of its columns: over j < t; with t between their rows and columns: all
                const int ti = l >> 4;
                float up = 0.f, down = 0.f, all = sum.row[ti * (ti + 1) / 2 + ti][r], ri = 0.f, e = 0.f;
                for (int k = 0; k < ti; ++k) {
                    up += sum.row[ti * (ti + 1) / 2 + k][r];
                    for (int i = ti + 1; i < 4; ++i) all += sum.all[i * (i + 1) / 2 + k];
                }
                for (int k = ti + 1; k < 4; ++k) down += sum.col[k * (k + 1) / 2 + ti][r];
                float before = __shfl_up(down, 1, 16);
                before = r ? before : 0.f;
#pragma unroll
                for (int m = 1; m < 16; m <<= 1) {
                    const float x = __shfl_down(up, m, 16), y = __shfl_up(before, m, 16);
                    up += r + m < 16 ? x : 0.f;
                    before += r >= m ? y : 0.f;
                }
#pragma unroll
                for (int k = 0; k < NT; ++k) ri += sum.r[k][l], e += sum.e[k];
                s.pairs[q][l] = up + before + all;
                s.r[q][l] = ri;
                s.diag[q][l] = sum.diag[l];
                if (l == 0) s.e[q] = e;
            }
        }
        __syncthreads();
        if (w < count) {
            const Part pt = part_of(a, first + w);
            if (pt.col + kHeadPart == a.d_head) {
                float pairs = 0.f, ri = 0.f, e = 0.f, dyx = 0.f;
                for (int k = max(0, w + 1 - halves); k <= w; ++k) pairs += s.pairs[k][l], ri += s.r[k][l], e += s.e[k], dyx += s.diag[k][l];
                // r's sum from t on, as the whole less what is before t (exact in fp64)
                const double rs = wave_scan((double)ri, l), zs = wave_scan((double)z, l);
                const float dg = (float)((double)pairs + (__shfl(rs, 63, 64) - rs + (double)ri) + (zs - (double)z) + (double)s.g[w].in[63] * e), dt = s.g[w].dt[l];
                float draw = fmaf(A, dg, u);
                if (a.softplus) draw *= sigmoid_of<F32>(raw + bias);
                if (l >= rows) draw = 0.f;
                else st_elem<F32>(a.draw, (t0 + l) * a.ddt_stride + pt.head, draw);
                float sums[3] = {dt * dg, draw, dyx};
#pragma unroll
                for (int k = 0; k < 3; ++k) sums[k] = rows_sum(row_sum(sums[k]));
                if (l == 0)
#pragma unroll
                    for (int k = 0; k < 3; ++k) a.head_part[(k * slots + slot) * a.n_heads + pt.head] = sums[k];
            }
        }
        __syncthreads();
    }
    // the pairs' part of dB and dC, for all heads at once
    E *pair = s.x;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (k < tiles) PairMat::put4(pair, 16 * jt[k] + r, 16 * it[k] + g4, V[k]);
    if (w < 2) PairMat::put4(pair, 32 * w + 16 + r, 32 * w + g4, f4{});  // (i tile, j tile) = (0, 1), (2, 3): no pairs
    __syncthreads();
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
        const Frag<F32, 1> fB = get_t<F32, 1, false>(s.B, KeyMat::ROW, 0, 32 * kb, 16 * nt, l), fC = get_t<F32, 1, false>(s.C, KeyMat::ROW, 0, 32 * kb, 16 * nt, l);
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            const int tile = tt0 + k;
            if (kb == 0 || tile >= 2) dC[k] = mma<2>(fB, get_t<F32, 2, false>(pair, PairMat::ROW, PairMat::PLANE, 32 * kb, 16 * tile, l), dC[k]);
            if (kb == 1 || tile < 2) dB[k] = mma<2>(fC, PairMat::get(pair, 16 * tile + r, 32 * kb + g8), dB[k]);
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
