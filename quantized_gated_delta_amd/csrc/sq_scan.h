// The selective state-space scan's kernels (sq_scan.hip, sq_scan_bwd.hip): arguments, workspaces, a chunk's gates.
#pragma once

#include "sq_block.h"

namespace sqk {

constexpr int kHeadPart = 64;  // columns of a state that a workgroup has: a head of 128 is two parts, which share its gates
constexpr int kSegMin = 8;     // shortest segment of a long sequence: 256 tokens
constexpr int kSegGroups = 512;  // workgroups that sequences are cut into segments for

struct ScanArgs {
    Ragged seqs;
    const void *x, *raw, *B, *C;
    const float *A, *D, *bias, *S0;
    void *y;
    float *S_out;
    int64_t x_stride, dt_stride, b_stride, c_stride;
    int32_t n_heads, n_groups, d_head, softplus;  // d_head: 64 or 128
    int32_t seg_shift, segments;  // log2 of a segment's tokens; segments: more than one to some sequence
    float *seg_state, *seg_fade;  // [segment slot][part of a head]: states at the segments' starts, decays over them
    uint8_t *save, *grad_save;    // [chunk slot][part][d_state][64] fp32: states at the chunks' starts; their gradients at the chunks' ends
    // backward
    const void *dy;
    const float *dS_out;
    void *dx, *draw, *dB, *dC;
    float *dA, *dD, *dbias, *dS0;
    int64_t dx_stride, ddt_stride, db_stride, dc_stride;
    int32_t subsets;              // of a group's heads, a workgroup each
    float *group_part;            // [2][subsets][n_tokens][n_groups][d_state]: dB and dC of a subset (subsets > 1)
    float *dots;                  // [2][chunk slot][part][64]: what the pass back leaves of x's dots with U
    int64_t chunk_parts;          // chunk slots x parts
    float *head_part;             // [3][chunk slots][n_heads]: sums over a chunk of dA, dbias and dD
    // step
    float *pool;
    const int32_t *slot;
    int32_t n, n_slots;
};

// How a call is cut up.  Segments: a workgroup walks the chunks of one, so a long sequence is cut where
// there would be too few workgroups to fill the card; its states at the segments' starts
// then come from a pass that forms states alone (about half the work of the whole).
struct ScanPlan {
    int seg_shift, subsets;
    int64_t parts, seg_slots, chunk_slots, state_bytes, fade_bytes, save_bytes, group_bytes, dots_bytes, head_bytes;
};
ScanPlan scan_plan(const sq_scan_desc &d);

hipError_t launch_scan_forward(const ScanArgs &a, int d_state, bool f32, bool y_f32, hipStream_t stream);
hipError_t launch_scan_states_back(const ScanArgs &a, int d_state, bool f32, hipStream_t stream);
hipError_t launch_scan_backward(const ScanArgs &a, int d_state, bool f32, hipStream_t stream);
hipError_t launch_scan_step(const ScanArgs &a, int d_state, bool f32, bool y_f32, hipStream_t stream);

// ------------------------------------------------------------------ device
// log(1 + e^v); from 20 on that is v to one part in 10^10.
__device__ __forceinline__ float softplus_of(float v) { return v > 20.f ? v : log1pf(expf(v)); }

// A chunk's gates in LDS.  G: the running sum of dt A over the chunk, times log2(e), as the sum of two floats, so that
// a difference of two is exact to fp32 wherever it is small, also behind a strong decay.
struct Gates {
    float hi[64], lo[64];  // G
    float dt[64];
    float in[64];          // e^G: from the chunk's start to a token
    float out[64];         // e^{G_end - G}: from a token to the chunk's end
};
// x times the decays between four neighbouring tokens from `four` on and token `one`; LATER: the four are the later ones.
// Pairs that do not meet get 0 by a choice between two values: as `live ? x * decay : 0`, each of the four, its loads
// with it, goes behind a branch of its own (64 x 64 pairs of a chunk: 3000 cycles for 1750).
template <bool LATER> __device__ __forceinline__ f4 decayed(const Gates &g, f4 x, int four, int one) {
    const f4 hi = *reinterpret_cast<const f4 *>(&g.hi[four]), lo = *reinterpret_cast<const f4 *>(&g.lo[four]);
    const float one_hi = g.hi[one], one_lo = g.lo[one];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float d = LATER ? (hi[e] - one_hi) + (lo[e] - one_lo) : (one_hi - hi[e]) + (one_lo - lo[e]);
        const float v = x[e] * __builtin_amdgcn_exp2f(d);
        x[e] = (LATER ? four + e >= one : four + e <= one) ? v : 0.f;
    }
    return x;
}

// Inclusive sums over the lanes of a wave.
__device__ __forceinline__ double wave_scan(double v, int l) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double u = __shfl_up(v, m, 64);
        if (l >= m) v += u;
    }
    return v;
}

// 2^x of an fp64 x: its leading float goes through the hardware's exponential, the rest is first order.
__device__ __forceinline__ float exp2_of(double x) {
    const float hi = (float)x, r = __builtin_amdgcn_exp2f(hi);
    return fmaf(r, (float)(x - (double)hi) * 0.69314718055994530942f, r);
}

// One wave forms a chunk's gates, a token to a lane; live: the token is one of the sequence's.
// Others have no time: they change nothing.
__device__ __forceinline__ void make_gates(Gates &g, int l, bool live, float raw, float bias, float A, int softplus) {
    const float v = raw + bias;
    const float dt = live ? (softplus ? softplus_of(v) : v) : 0.f;
    double s = (double)dt * (double)A;
    s = s < -150.0 ? -150.0 : s;  // a NaN stays one
    if (!live) s = 0.0;
    const double G = wave_scan(s * 1.4426950408889634074, l), end = __shfl(G, 63, 64);
    const float hi = (float)G;
    g.hi[l] = hi;
    g.lo[l] = (float)(G - (double)hi);
    g.dt[l] = dt;
    g.in[l] = exp2_of(G);
    g.out[l] = exp2_of(end - G);
}

// Where row `row` of a PLACED token matrix lies in LDS: of each eight, the first four on the even places, so that the transposing
// loads, which take four rows at once, two of those fours for 32 lanes, meet every bank once (passes over the chunks: 2 %
// less; not where such loads are few, as addresses then cost more).
__device__ __forceinline__ int place_of(int row) { return (row & ~7) | (row & 3) << 1 | (row >> 2 & 1); }

// A matrix of 64 rows (tokens) in LDS, rows as they lie in memory and padded by 16 bytes.
template <bool F32, int COLS, bool PLACED = true> struct TokenMat {
    typedef Elem<F32> E;
    static constexpr int ROW = COLS + (F32 ? 4 : 8), SIZE = 64 * ROW;
    static constexpr int VECS = COLS * (int)sizeof(E) / 16;  // 16-byte vectors of a row
    __device__ __forceinline__ static int at(int row) { return PLACED ? place_of(row) : row; }
    // row `row`, elements k .. k + 7 of the contracted axis
    __device__ __forceinline__ static Frag<F32, 1> get(const E *m, int row, int k) { return load_frag<F32, 1>(m + at(row) * ROW + k, 0); }
    // ... elements k .. k + 3 and k + 16 .. k + 19: the order in which two result tiles hold 32 rows
    __device__ __forceinline__ static Frag<F32, 1> get_split(const E *m, int row, int k) {
        Frag<F32, 1> f;
        const E *p = m + at(row) * ROW + k;
        if constexpr (F32) {
            f.v[0] = *reinterpret_cast<const f4 *>(p);
            f.v[1] = *reinterpret_cast<const f4 *>(p + 16);
        } else {
            f.t[0] = __builtin_shufflevector(*reinterpret_cast<const bf4 *>(p), *reinterpret_cast<const bf4 *>(p + 16), 0, 1, 2, 3, 4, 5, 6, 7);
        }
        return f;
    }
};

template <bool F32> __device__ __forceinline__ f4 load4(const Elem<F32> *p) {
    if constexpr (F32) return *reinterpret_cast<const f4 *>(p);
    else return __builtin_convertvector(*reinterpret_cast<const bf4 *>(p), f4);
}

// c[n] += a[n] b[n], or with one a or b for all: products of the same terms one after another, so that each
// accumulates while the others are issued (with their operands loaded ahead: the state's reading 2000 cycles for 1420 of a
// chunk, its update 1450 for 1120).
template <int P, int COUNT, bool ONE_A, bool ONE_B, int NA, int NB>
__device__ __forceinline__ void mma_all(const Frag<false, NA> *a, const Frag<false, NB> *b, f4 *c) {
#pragma unroll
    for (int s = P - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
#pragma unroll
                for (int n = 0; n < COUNT; ++n)
                    c[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[ONE_A ? 0 : n].t[i], b[ONE_B ? 0 : n].t[s - i], c[n], 0, 0, 0);
}
template <int P, int COUNT, bool ONE_A, bool ONE_B, int NA, int NB>
__device__ __forceinline__ void mma_all(const Frag<true, NA> *a, const Frag<true, NB> *b, f4 *c) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int n = 0; n < COUNT; ++n)
            c[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[ONE_A ? 0 : n].v[i / 4][i % 4], b[ONE_B ? 0 : n].v[i / 4][i % 4], c[n], 0, 0, 0);
}

typedef short s4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4v lds_s4v;
// A fragment of the transposed matrix: row (lane) l % 16 is column col0 + l % 16 of m, contracted elements
// are its rows row0 + 8 (l / 16) .. + 7.  bf16: the transposing LDS load, where 16 lanes take 4 rows of 16.
template <bool F32, int N, bool PLACED = true> __device__ __forceinline__ Frag<F32, N> get_t(const Elem<F32> *m, int row_size, int plane, int row0, int col0, int l) {
    Frag<F32, N> f;
    const int r = l & 15, g = l >> 4;
    if constexpr (F32) {
        const float *p = m + (row0 + 8 * g) * row_size + col0 + r;
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e / 4][e % 4] = p[(PLACED ? place_of(e) : e) * row_size];
    } else {
        const uint16_t *p = m + (row0 + 8 * g + (r >> 2) * (PLACED ? 2 : 1)) * row_size + col0 + (r & 3) * 4;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const s4v a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v *)(p + n * plane));
            const s4v b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v *)(p + n * plane + (PLACED ? 1 : 4) * row_size));
            f.t[n] = __builtin_bit_cast(bf8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
    return f;
}

// The 16 x 16 tiles (it, jt), jt <= it, of 64 x 64 pairs of tokens, numbered row by row.
__device__ __forceinline__ void pair_tile(int n, int &it, int &jt) {
    it = n >= 6 ? 3 : n >= 3 ? 2 : n >= 1 ? 1 : 0;
    jt = n - it * (it + 1) / 2;
}

// The bf16 matrix instructions round sums downwards, about 2^-25 on average: nothing next to a result, but the
// same way for all tokens and rows, so that it shows in sums over many (dbias 2e-6 off for 3e-7).  What such sums are
// formed from is therefore computed with the other sign for every second tile of 16 tokens or rows of the state.
__device__ __forceinline__ float sign_of(int tile) { return tile & 1 ? -1.f : 1.f; }

// Vectors of a token matrix as a workgroup of T threads loads them: from memory into
// registers (behind the last row: it again), and from there into LDS.
template <bool F32, int COLS, int T, bool PLACED = true> struct Staged {
    typedef TokenMat<F32, COLS, PLACED> M;
    static constexpr int COUNT = 64 * M::VECS / T;
    uint4 v[COUNT];
    __device__ __forceinline__ void load(const void *base, uint32_t stride, int rows, int t) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            const uint32_t row = min((i * T + t) / M::VECS, rows - 1), col = (i * T + t) % M::VECS;
            v[i] = *at_bytes<uint4>(base, row * (stride * (uint32_t)sizeof(Elem<F32>)) + col * 16);
        }
    }
    // rows from `rows` on as zeros
    __device__ __forceinline__ void clear(int rows, int t) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            const bool live = (i * T + t) / M::VECS < rows;
            v[i] = uint4{live ? v[i].x : 0u, live ? v[i].y : 0u, live ? v[i].z : 0u, live ? v[i].w : 0u};
        }
    }
    // TURN_ROWS, TURN_COLS: rows and columns 16 .. 31, 48 .. 63, ... with their signs turned, see sign_of
    template <bool TURN_ROWS = false, bool TURN_COLS = false> __device__ __forceinline__ void store(Elem<F32> *m, int t) const {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            const int row = (i * T + t) / M::VECS, col = (i * T + t) % M::VECS;
            const int turned = (TURN_ROWS ? row : 0) ^ (TURN_COLS ? col * 16 / (int)sizeof(Elem<F32>) : 0);
            const uint32_t flip = turned & 16 ? (F32 ? 0x80000000u : 0x80008000u) : 0u;
            *(reinterpret_cast<uint4 *>(m + M::at(row) * M::ROW) + col) = uint4{v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip};
        }
    }
};

// What a part of a head is: its head, group and first column.  The same for a whole wave, so in scalar registers, where
// a division alone would not leave them: every address that follows is then formed by the scalar unit.
struct Part { int head, group, col; };
__device__ __forceinline__ Part part_of(const ScanArgs &a, int part) {
    const bool whole = a.d_head == kHeadPart;
    Part p;
    p.head = whole ? part : part >> 1;
    p.col = whole ? 0 : (part & 1) * kHeadPart;
    p.group = __builtin_amdgcn_readfirstlane(p.head / (a.n_heads / a.n_groups));
    return p;
}
// Element (0, 0) of a part's state in [sequence][head][d_state][d_head].
template <int N> __device__ __forceinline__ int64_t state_at(const ScanArgs &a, int seq, const Part &p) {
    return ((int64_t)seq * a.n_heads + p.head) * N * a.d_head + p.col;
}

} // namespace sqk
