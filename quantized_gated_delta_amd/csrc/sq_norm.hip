// The norms around a block, with its gate and its residual scale, and their gradients.
//
// Gated norm, per row of d (one group of a token):
//   y = n w act(z),  n = x rs,  rs = (mean x^2 + eps)^-1/2        (norm, then gate)
//   y = n w,         n = u rs,  u = x act(z)                      (gate, then norm)
// With t the gradient that reaches n (dy w act(z); dy w),  rs (t - n mean(t n)) reaches x (u);
// mean(t n) = rs mean(t x), so one pass over the row gives both sums, of x^2 and of t x.
// Residual norm, per row:
//   a = o, or no wp with no = o ro;  r' = r + s a;  h = n w with n = r' rs
//   T = dr' + rs (dh w - n mean(dh w n));  dr = T;  ds = sum T a;  da = s T;
//   do = da, or ro (da wp - no mean(da wp no));  dwp = sum da no;  dw = sum dh n
// The backward pass starts from o and r, not from a stored r': as many bytes, and no rounding
// of r' to its type in between.
//
// All of it is bound by memory: a row lies in the registers of 1 to 1024 threads, 8 elements (16 above
// 8192 columns) each, is read once and written once.  Sums over a row go through the wave's lanes and, for
// rows of more than 512, through LDS.  A workgroup walks over rows, the next one's loads in flight while it works on
// one: the parameters are then loaded once, and what waits for a row's sums does not wait for memory too.  A thread
// keeps its columns from row to row, so the sums over rows stay in registers until a workgroup's end and are then
// added up in a fixed order.
#include "sq_block.h"

namespace sqk {
namespace {

// Sums of N values over the `width` threads of a row (a power of two; neighbours).  A row wider than a wave
// has the workgroup to itself.  turn: counts the calls, so that one barrier is enough: a second call
// writes to the other half of lds, a third one comes behind the second one's barrier.
template <int N> __device__ __forceinline__ void row_sums(float (&v)[N], int width, float *lds, int &turn) {
    if (width >= 16) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = row_sum(v[i]);
        if (width >= 32)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], 16, 64);
        if (width >= 64)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], 32, 64);
    } else {
        for (int m = 1; m < width; m <<= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], m, 64);
    }
    if (width > 64) {
        const int w = threadIdx.x >> 6, waves = width >> 6;
        float *p = lds + (turn++ & 1) * 32;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) p[i * 16 + w] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.f;
            for (int k = 0; k < waves; ++k) s += p[i * 16 + k];
            v[i] = s;
        }
    }
}
constexpr int kSumLds = 64;

// The part of a workgroup that a thread is: row `sub` of those handled at once, columns from
// `col` on.  width: threads of a row.
struct Place { int width, sub, rows, col; };
template <int K> __device__ __forceinline__ Place place_of(int d) {
    Place p;
    p.width = 1;
    while (p.width * 8 * K < d) p.width <<= 1;
    p.rows = blockDim.x / p.width;
    p.sub = threadIdx.x / p.width;
    p.col = (threadIdx.x % p.width) * 8;  // vector k: col + k * width * 8
    return p;
}

// Columns of a vector that lie inside the row.
__device__ __forceinline__ int left_of(int d, int col) { return min(8, d - col); }

template <bool F32, bool VEC, int K>
__device__ __forceinline__ void load_row(Raw8<F32> (&r)[K], const void *p, int64_t at, const Place &pl, int d) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = pl.col + k * pl.width * 8;
        r[k] = c < d ? load8<F32, VEC>(p, at + c, left_of(d, c)) : Raw8<F32>{};
    }
}
// Parameters of a thread's columns; `other` where there are none, and 0 behind the row's end.  VEC: d is a multiple
// of 8 and p, like all tensors, 16-byte aligned.
template <bool VEC, int K> __device__ __forceinline__ void load_weights(float (&w)[8 * K], const float *p, const Place &pl, int d, float other) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = pl.col + k * pl.width * 8;
        if (VEC && p) {
            widen8<true>(c < d ? load8<true, true>(p, c, 8) : Raw8<true>{}, *reinterpret_cast<float (*)[8]>(&w[8 * k]));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[8 * k + e] = c + e < d ? (p ? p[c + e] : other) : 0.f;
        }
    }
}
template <bool F32, bool VEC, int K>
__device__ __forceinline__ void store_row(void *p, int64_t at, const float (&x)[8 * K], const Place &pl, int d) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = pl.col + k * pl.width * 8;
        if (c < d) {
            const float (&v)[8] = *reinterpret_cast<const float (*)[8]>(&x[8 * k]);
            store8<F32, VEC>(p, at + c, v, left_of(d, c));
        }
    }
}
template <bool F32, int K> __device__ __forceinline__ void widen_row(const Raw8<F32> (&r)[K], float (&x)[8 * K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) widen8<F32>(r[k], *reinterpret_cast<float (*)[8]>(&x[8 * k]));
}

// 1 / sqrt(mean + eps), correctly rounded in both steps: one of each for a row.
__device__ __forceinline__ float rstd_of(float sum, int d, float eps) { return 1.f / sqrtf(sum / (float)d + eps); }

// A workgroup's sums over its rows, N lists of columns: the rows that it handles at once are
// added through LDS, one after another, and thread row 0 stores.
template <int K, int N>
__device__ __forceinline__ void store_sums(float (&s)[N][8 * K], float *const (&out)[N], const Place &pl, int d, float *lds) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if (!out[n]) continue;
        for (int other = 1; other < pl.rows; ++other) {  // rows > 1: at most 512 columns
            __syncthreads();
            if (pl.sub == other)
#pragma unroll
                for (int e = 0; e < 8 * K; ++e) lds[(threadIdx.x % pl.width) * 8 * K + e] = s[n][e];
            __syncthreads();
            if (pl.sub == 0)
#pragma unroll
                for (int e = 0; e < 8 * K; ++e) s[n][e] += lds[(threadIdx.x % pl.width) * 8 * K + e];
        }
        if (pl.sub == 0)
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = pl.col + k * pl.width * 8 + e;
                    if (c < d) out[n][c] = s[n][8 * k + e];
                }
    }
}

// Row i of the gated norm's rows: shared weights number them over tokens and groups, weights of a
// group's own over the tokens of group blockIdx.y.
struct RowAt { int64_t token, group; };
template <bool SHARED> __device__ __forceinline__ RowAt row_at(const GateArgs &a, uint32_t i) {
    if (!SHARED) return RowAt{i, blockIdx.y};
    if (a.groups == 1) return RowAt{i, 0};
    const uint32_t token = i / (uint32_t)a.groups;
    return RowAt{token, i - token * a.groups};
}

// Rows of one turn of a workgroup, those of the turn after it in flight.
template <bool F32, int K> struct GateRow { Raw8<F32> x[K], z[K]; };
template <bool F32, bool VEC, bool SHARED, int K> __device__ __forceinline__ void load_gate_row(GateRow<F32, K> &r, const GateArgs &a, uint32_t i, const Place &pl) {
    const RowAt at = row_at<SHARED>(a, i);
    load_row<F32, VEC, K>(r.x, a.x, at.token * a.x_stride + at.group * a.d, pl, a.d);
    if (a.z) load_row<F32, VEC, K>(r.z, a.z, at.token * a.z_stride + at.group * a.d, pl, a.d);
}

// 8192 x 32 rows of 128: 40 us, 5.1 TB/s (a workgroup for each 16 rows, without walking: 74).
template <bool F32, bool VEC, bool FIRST, bool SHARED, int K, int T>
__global__ __launch_bounds__(T) void gate_forward_kernel(GateArgs a, uint32_t rows) {
    __shared__ float lds[kSumLds];
    int turn = 0;
    const Place pl = place_of<K>(a.d);
    float w[8 * K];
    load_weights<VEC, K>(w, a.weight ? a.weight + (SHARED ? 0 : (int64_t)blockIdx.y * a.d) : nullptr, pl, a.d, 1.f);
    const uint32_t step = gridDim.x * pl.rows, last = rows - 1;
    GateRow<F32, K> next{};
    load_gate_row<F32, VEC, SHARED, K>(next, a, min(blockIdx.x * pl.rows + pl.sub, last), pl);
    for (uint32_t i0 = blockIdx.x * pl.rows; i0 < rows; i0 += step) {  // the same turns for all threads: the sums have barriers
        const GateRow<F32, K> row = next;
        const uint32_t i = i0 + pl.sub;
        if (i0 + step < rows) load_gate_row<F32, VEC, SHARED, K>(next, a, min(i + step, last), pl);
        float x[8 * K], z[8 * K];
        widen_row<F32, K>(row.x, x);
        widen_row<F32, K>(row.z, z);
        if (a.z)
#pragma unroll
            for (int e = 0; e < 8 * K; ++e) z[e] = gate_of<F32>(a.act, z[e]);
        float s[1] = {0.f};
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) {
            if (FIRST && a.z) x[e] *= z[e];
            s[0] = fmaf(x[e], x[e], s[0]);
        }
        row_sums<1>(s, pl.width, lds, turn);
        const float rs = rstd_of(s[0], a.d, a.eps);
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) {
            x[e] = x[e] * rs * w[e];
            if (!FIRST && a.z) x[e] *= z[e];
        }
        if (i < rows) {
            const RowAt at = row_at<SHARED>(a, i);
            store_row<F32, VEC, K>(a.y, (at.token * a.groups + at.group) * a.d, x, pl, a.d);
        }
    }
}

// 8192 x 32 rows of 128: 67 us, 5.0 TB/s.
template <bool F32, bool VEC, bool FIRST, bool SHARED, int K, int T>
__global__ __launch_bounds__(T) void gate_backward_kernel(GateArgs a, uint32_t rows) {
    __shared__ float lds[512 * K + kSumLds];
    int turn = 0;
    const Place pl = place_of<K>(a.d);
    const float over = 1.f / (float)a.d;
    float w[8 * K], dw[1][8 * K] = {};
    load_weights<VEC, K>(w, a.weight ? a.weight + (SHARED ? 0 : (int64_t)blockIdx.y * a.d) : nullptr, pl, a.d, 1.f);
    const uint32_t step = gridDim.x * pl.rows, last = rows - 1;
    GateRow<F32, K> next{};
    Raw8<F32> next_dy[K] = {};
    auto load = [&](uint32_t i) {
        load_gate_row<F32, VEC, SHARED, K>(next, a, i, pl);
        const RowAt at = row_at<SHARED>(a, i);
        load_row<F32, VEC, K>(next_dy, a.dy, (at.token * a.groups + at.group) * a.d, pl, a.d);
    };
    if (rows) load(min(blockIdx.x * pl.rows + pl.sub, last));
    for (uint32_t i0 = blockIdx.x * pl.rows; i0 < rows; i0 += step) {
        const uint32_t i = i0 + pl.sub;
        const bool live = i < rows;
        float x[8 * K], z[8 * K], dy[8 * K], act[8 * K], slope[8 * K];
        widen_row<F32, K>(next.x, x);
        widen_row<F32, K>(next.z, z);
        widen_row<F32, K>(next_dy, dy);
        if (i0 + step < rows) load(min(i + step, last));
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) {
            act[e] = 1.f, slope[e] = 0.f;
            if (a.z) gate_and_slope<F32>(a.act, z[e], act[e], slope[e]);
            const float u = FIRST ? x[e] * act[e] : x[e], t = FIRST ? dy[e] * w[e] : dy[e] * w[e] * act[e];
            s[0] = fmaf(u, u, s[0]);
            s[1] = fmaf(t, u, s[1]);
        }
        row_sums<2>(s, pl.width, lds + 512 * K, turn);
        const float rs = rstd_of(s[0], a.d, a.eps), c = s[1] * rs * over;
        float dx[8 * K], dz[8 * K];
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) {
            if (FIRST) {
                const float n = x[e] * act[e] * rs, du = rs * fmaf(-n, c, dy[e] * w[e]);
                dx[e] = du * act[e];
                dz[e] = du * x[e] * slope[e];
                if (live) dw[0][e] = fmaf(dy[e], n, dw[0][e]);
            } else {
                const float n = x[e] * rs;
                dx[e] = rs * fmaf(-n, c, dy[e] * w[e] * act[e]);
                dz[e] = dy[e] * n * w[e] * slope[e];
                if (live) dw[0][e] = fmaf(dy[e] * act[e], n, dw[0][e]);
            }
        }
        if (live) {
            const RowAt at = row_at<SHARED>(a, i);
            store_row<F32, VEC, K>(a.dx, at.token * a.dx_stride + at.group * a.d, dx, pl, a.d);
            if (a.dz) store_row<F32, VEC, K>(a.dz, at.token * a.dz_stride + at.group * a.d, dz, pl, a.d);
        }
    }
    float *const out[1] = {a.dweight ? a.partial + ((int64_t)blockIdx.x * gridDim.y + blockIdx.y) * a.d : nullptr};
    store_sums<K, 1>(dw, out, pl, a.d, lds);
}

// 8192 rows of 4096, o in bf16, r in fp32 (403 MB): 66 us (a workgroup a row, without walking: 205).
template <bool F32, bool RF32, bool VEC, int K, int T> __global__ __launch_bounds__(T) void residual_forward_kernel(ResidualArgs a) {
    __shared__ float lds[kSumLds];
    int turn = 0;
    const Place pl = place_of<K>(a.d);
    const uint32_t rows = (uint32_t)a.n_rows, step = gridDim.x * pl.rows, last = rows - 1;
    float post[8 * K], scale[8 * K], w[8 * K];
    load_weights<VEC, K>(post, a.post, pl, a.d, 1.f);
    load_weights<VEC, K>(scale, a.scale, pl, a.d, 1.f);
    load_weights<VEC, K>(w, a.weight, pl, a.d, 1.f);
    Raw8<F32> next_o[K];
    Raw8<RF32> next_r[K] = {};
    auto load = [&](uint32_t i) {
        load_row<F32, VEC, K>(next_o, a.o, (int64_t)i * a.d, pl, a.d);
        if (a.r) load_row<RF32, VEC, K>(next_r, a.r, (int64_t)i * a.d, pl, a.d);
    };
    load(min(blockIdx.x * pl.rows + pl.sub, last));
    for (uint32_t i0 = blockIdx.x * pl.rows; i0 < rows; i0 += step) {
        const uint32_t i = i0 + pl.sub;
        const int64_t at = (int64_t)i * a.d;
        float o[8 * K], r[8 * K], s[1] = {0.f};
        widen_row<F32, K>(next_o, o);
        widen_row<RF32, K>(next_r, r);
        if (i0 + step < rows) load(min(i + step, last));
        if (a.post) {
#pragma unroll
            for (int e = 0; e < 8 * K; ++e) s[0] = fmaf(o[e], o[e], s[0]);
            row_sums<1>(s, pl.width, lds, turn);
            const float rs = rstd_of(s[0], a.d, a.eps);
#pragma unroll
            for (int e = 0; e < 8 * K; ++e) o[e] = o[e] * rs * post[e];
        }
        s[0] = 0.f;
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) {
            r[e] = fmaf(scale[e], o[e], r[e]);
            s[0] = fmaf(r[e], r[e], s[0]);
        }
        if (i < rows) store_row<RF32, VEC, K>(a.r_out, at, r, pl, a.d);
        if (!a.h) continue;
        row_sums<1>(s, pl.width, lds, turn);
        const float rs = rstd_of(s[0], a.d, a.eps);
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) r[e] = r[e] * rs * w[e];
        if (i < rows) store_row<F32, VEC, K>(a.h, at, r, pl, a.d);
    }
}

// The same rows (604 MB): 133 us, 4.5 TB/s; three sums over the row wait for each other, two workgroups to a CU.
template <bool F32, bool RF32, bool VEC, int K, int T>
__global__ __launch_bounds__(T) __attribute__((amdgpu_waves_per_eu(K == 1 ? 4 : 2))) void residual_backward_kernel(ResidualArgs a) {
    __shared__ float lds[512 * K + kSumLds];
    // a thread's parameters, in LDS where there is room for all of them: in registers, one workgroup of 512 would fill a CU
    constexpr bool IN_LDS = K == 1;
    __shared__ __attribute__((aligned(16))) float params[3][2][IN_LDS ? T : 1][4];
    int turn = 0;
    const Place pl = place_of<K>(a.d);
    const float over = 1.f / (float)a.d;
    const uint32_t rows = (uint32_t)a.n_rows, step = gridDim.x * pl.rows, last = rows - 1;
    float kept[IN_LDS ? 1 : 3][8 * K], sums[3][8 * K] = {};
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        float (&v)[8 * K] = kept[IN_LDS ? 0 : n];
        load_weights<VEC, K>(v, n == 0 ? a.post : n == 1 ? a.scale : a.weight, pl, a.d, 1.f);
        if constexpr (IN_LDS)
#pragma unroll
            for (int h = 0; h < 2; ++h) *reinterpret_cast<f4 *>(params[n][h][threadIdx.x]) = f4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    }
    auto param = [&](int n, int e) { return IN_LDS ? params[n][e >> 2][threadIdx.x][e & 3] : kept[IN_LDS ? 0 : n][e]; };
    constexpr int POST = 0, SCALE = 1, WEIGHT = 2;
    Raw8<F32> next_o[K], next_h[K] = {};
    Raw8<RF32> next_r[K] = {}, next_d[K] = {};
    auto load = [&](uint32_t i) {
        const int64_t at = (int64_t)i * a.d;
        load_row<F32, VEC, K>(next_o, a.o, at, pl, a.d);
        if (a.r) load_row<RF32, VEC, K>(next_r, a.r, at, pl, a.d);
        if (a.dh) load_row<F32, VEC, K>(next_h, a.dh, at, pl, a.d);
        if (a.dr_out) load_row<RF32, VEC, K>(next_d, a.dr_out, at, pl, a.d);
    };
    if (rows) load(min(blockIdx.x * pl.rows + pl.sub, last));
    for (uint32_t i0 = blockIdx.x * pl.rows; i0 < rows; i0 += step) {
        const uint32_t i = i0 + pl.sub;
        const bool live = i < rows;
        const int64_t at = (int64_t)i * a.d;
        float o[8 * K], r[8 * K], dh[8 * K], t[8 * K];
        widen_row<F32, K>(next_o, o);
        widen_row<RF32, K>(next_r, r);
        widen_row<F32, K>(next_h, dh);
        widen_row<RF32, K>(next_d, t);
        if (i0 + step < rows) load(min(i + step, last));
        float so[1] = {0.f}, s[2] = {0.f, 0.f};
        float rso = 1.f;
        if (a.post) {
#pragma unroll
            for (int e = 0; e < 8 * K; ++e) so[0] = fmaf(o[e], o[e], so[0]);
            row_sums<1>(so, pl.width, lds + 512 * K, turn);
            rso = rstd_of(so[0], a.d, a.eps);
        }
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) {
            o[e] *= rso;  // the norm behind the block, without its weight
            r[e] = fmaf(param(SCALE, e), a.post ? o[e] * param(POST, e) : o[e], r[e]);
            s[0] = fmaf(r[e], r[e], s[0]);
            s[1] = fmaf(dh[e] * param(WEIGHT, e), r[e], s[1]);
        }
        if (a.dh) {
            row_sums<2>(s, pl.width, lds + 512 * K, turn);
            const float rs = rstd_of(s[0], a.d, a.eps), c = s[1] * rs * over;
#pragma unroll
            for (int e = 0; e < 8 * K; ++e) {
                const float n = r[e] * rs;
                t[e] = fmaf(rs, fmaf(-n, c, dh[e] * param(WEIGHT, e)), t[e]);
                if (live) sums[2][e] = fmaf(dh[e], n, sums[2][e]);
            }
        }
        if (live && a.dr) store_row<RF32, VEC, K>(a.dr, at, t, pl, a.d);
        so[0] = 0.f;
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) {
            if (live) sums[1][e] = fmaf(t[e], a.post ? o[e] * param(POST, e) : o[e], sums[1][e]);
            t[e] *= param(SCALE, e);
            if (a.post) {
                if (live) sums[0][e] = fmaf(t[e], o[e], sums[0][e]);
                t[e] *= param(POST, e);
                so[0] = fmaf(t[e], o[e], so[0]);
            }
        }
        if (a.post) {
            row_sums<1>(so, pl.width, lds + 512 * K, turn);
            const float c = so[0] * over;
#pragma unroll
            for (int e = 0; e < 8 * K; ++e) t[e] = rso * fmaf(-o[e], c, t[e]);
        }
        if (live) store_row<F32, VEC, K>(a.d_o, at, t, pl, a.d);
    }
    const int64_t part = (int64_t)gridDim.x * a.d, mine = (int64_t)blockIdx.x * a.d;
    float *const out[3] = {a.dpost ? a.partial + mine : nullptr, a.dscale ? a.partial + part + mine : nullptr,
                           a.dweight ? a.partial + 2 * part + mine : nullptr};
    store_sums<K, 3>(sums, out, pl, a.d, lds);
}

struct SumList { SumArgs a[4]; };
// 16 columns to a workgroup, and 16 threads to a column: thread k adds the rows k, k + 16, ..., eight of them in flight.
__global__ __launch_bounds__(256) void column_sums_kernel(SumList list) {
    __shared__ float lds[16][17];
    const SumArgs &a = list.a[blockIdx.y];
    const int k = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t c = (int64_t)blockIdx.x * 16 + l;
    if ((int64_t)blockIdx.x * 16 >= a.cols) return;
    float s[8] = {};
    if (c < a.cols)
        for (int64_t i = k; i < a.rows; i += 128)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] += i + 16 * j < a.rows ? a.part[(i + 16 * j) * a.row_stride + c] : 0.f;
    lds[k][l] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    __syncthreads();
    if (k == 0 && c < a.cols) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) sum += lds[j][l];
        a.out[c] = sum;
    }
}

int row_width(int d, int k) {
    int width = 1;
    while (width * 8 * k < d) width <<= 1;
    return width;
}
// Threads of a workgroup: 256 that share rows of up to a wave, or those of one wider row.
int threads_of(int d, int k) { return row_width(d, k) > 64 ? row_width(d, k) : 256; }
int rows_at_once(int d, int k) { return threads_of(d, k) / row_width(d, k); }
int vectors_of(int d) { return d > 4096 ? 2 : 1; }

// The kernel's template arguments from truth values.
template <typename F> void pick(bool b, F f) {
    if (b) f(std::true_type{});
    else f(std::false_type{});
}

} // namespace

// Vectors of a thread and most threads of a workgroup: rows of up to 4096 columns are one vector of 8 to each of up to 512
// threads, longer ones two.  What spills, in bytes a lane: above 8192 columns, with 1024 threads and so 128 registers, all passes
// back (gated 136 to 372, residual 544 to 700) and the residual forward with o and r in fp32 (28); the residual pass back at
// up to 4096 columns, held to four waves per SIMD, in all types but bf16 with an fp32 residual (40 to 64; without 16-byte loads
// all, 72 to 128) and from there to 8192 in all but bf16 throughout (32 to 108).
template <int KK, int TT> struct RowShape { static constexpr int K = KK, T = TT; };
template <typename F> void pick_row(int d, F f) {
    if (d <= 4096) f(RowShape<1, 512>{});
    else if (d <= 8192) f(RowShape<2, 512>{});
    else f(RowShape<2, 1024>{});
}

// Workgroups of a forward pass: as many as fit the card at 2048 threads a CU, so that each walks over as many rows as
// there are left to it.
static uint32_t forward_blocks(int64_t rows, int32_t d, int64_t at_most) {
    const int k = vectors_of(d);
    const int64_t turns = (rows + rows_at_once(d, k) - 1) / rows_at_once(d, k), fit = 256 * (2048 / threads_of(d, k)) / at_most;
    return (uint32_t)(turns < fit ? turns : fit > 1 ? fit : 1);
}

int norm_blocks(int64_t rows, int32_t d, int32_t groups) {
    const int64_t turns = (rows + rows_at_once(d, vectors_of(d)) - 1) / rows_at_once(d, vectors_of(d)), most = groups < 512 ? 512 / groups : 1;
    return (int)(turns < 1 ? 1 : turns < most ? turns : most);
}

hipError_t launch_column_sums(const SumArgs *a, int count, hipStream_t stream) {
    SumList list{};
    int64_t cols = 0;
    int n = 0;
    for (int i = 0; i < count; ++i)
        if (a[i].out) {
            list.a[n++] = a[i];
            cols = a[i].cols > cols ? a[i].cols : cols;
        }
    if (!n) return hipSuccess;
    hipLaunchKernelGGL(column_sums_kernel, dim3((uint32_t)((cols + 15) / 16), n), dim3(256), 0, stream, list);
    return hipGetLastError();
}

hipError_t launch_gate_forward(const GateArgs &a, bool f32, bool vec, bool first, bool shared, hipStream_t stream) {
    const int k = vectors_of(a.d);
    const int64_t rows = shared ? a.n_tokens * a.groups : a.n_tokens;
    const dim3 grid(forward_blocks(rows, a.d, shared ? 1 : a.groups), shared ? 1 : a.groups), block(threads_of(a.d, k));
    pick(f32, [&](auto F) { pick(vec, [&](auto V) { pick(first, [&](auto G) { pick(shared, [&](auto S) { pick_row(a.d, [&](auto R) {
        hipLaunchKernelGGL((gate_forward_kernel<F.value, V.value, G.value, S.value, R.K, R.T>), grid, block, 0, stream, a, (uint32_t)rows);
    }); }); }); }); });
    return hipGetLastError();
}

hipError_t launch_gate_backward(const GateArgs &a, bool f32, bool vec, bool first, bool shared, hipStream_t stream) {
    const int k = vectors_of(a.d);
    const int64_t rows = shared ? a.n_tokens * a.groups : a.n_tokens;
    const int blocks = norm_blocks(rows, a.d, shared ? 1 : a.groups);
    const dim3 grid(blocks, shared ? 1 : a.groups), block(threads_of(a.d, k));
    pick(f32, [&](auto F) { pick(vec, [&](auto V) { pick(first, [&](auto G) { pick(shared, [&](auto S) { pick_row(a.d, [&](auto R) {
        hipLaunchKernelGGL((gate_backward_kernel<F.value, V.value, G.value, S.value, R.K, R.T>), grid, block, 0, stream, a, (uint32_t)rows);
    }); }); }); }); });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t cols = (int64_t)a.d * (shared ? 1 : a.groups);
    const SumArgs s[1] = {{a.partial, a.dweight, blocks, cols, cols}};
    return launch_column_sums(s, 1, stream);
}

hipError_t launch_residual_forward(const ResidualArgs &a, bool f32, bool res_f32, bool vec, hipStream_t stream) {
    const int k = vectors_of(a.d);
    const dim3 grid(forward_blocks(a.n_rows, a.d, 1)), block(threads_of(a.d, k));
    pick(f32, [&](auto F) { pick(res_f32, [&](auto R) { pick(vec, [&](auto V) { pick_row(a.d, [&](auto W) {
        hipLaunchKernelGGL((residual_forward_kernel<F.value, R.value, V.value, W.K, W.T>), grid, block, 0, stream, a);
    }); }); }); });
    return hipGetLastError();
}

hipError_t launch_residual_backward(const ResidualArgs &a, bool f32, bool res_f32, bool vec, hipStream_t stream) {
    const int k = vectors_of(a.d), blocks = norm_blocks(a.n_rows, a.d, 1);
    const dim3 grid(blocks), block(threads_of(a.d, k));
    pick(f32, [&](auto F) { pick(res_f32, [&](auto R) { pick(vec, [&](auto V) { pick_row(a.d, [&](auto W) {
        hipLaunchKernelGGL((residual_backward_kernel<F.value, R.value, V.value, W.K, W.T>), grid, block, 0, stream, a);
    }); }); }); });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t part = (int64_t)blocks * a.d;
    const SumArgs s[3] = {{a.partial, a.dpost, blocks, a.d, a.d}, {a.partial + part, a.dscale, blocks, a.d, a.d},
                          {a.partial + 2 * part, a.dweight, blocks, a.d, a.d}};
    return launch_column_sums(s, 3, stream);
}

} // namespace sqk
