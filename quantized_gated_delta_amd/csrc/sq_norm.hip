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
// rows of more than 512, through LDS.  A thread keeps its columns from row to row, so the sums over
// rows stay in registers until a workgroup's end and are then added up in a fixed order.
#include "sq_block.h"

namespace sqk {
namespace {

// Sums of N values over the `width` threads of a row (a power of two; neighbours).  A row wider than a wave
// has the workgroup to itself.
template <int N> __device__ __forceinline__ void row_sums(float (&v)[N], int width, float *lds) {
    const int in_wave = min(width, 64);
    for (int m = 1; m < in_wave; m <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], m, 64);
    if (width > 64) {
        const int w = threadIdx.x >> 6, waves = width >> 6;
        __syncthreads();  // the last sums' readers
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) lds[i * 16 + w] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.f;
            for (int k = 0; k < waves; ++k) s += lds[i * 16 + k];
            v[i] = s;
        }
    }
}

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
template <int K> __device__ __forceinline__ void load_weights(float (&w)[8 * K], const float *p, const Place &pl, int d, float other) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = pl.col + k * pl.width * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[8 * k + e] = c + e < d ? (p ? p[c + e] : other) : 0.f;
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
__device__ __forceinline__ void row_at(const GateArgs &a, bool shared, int64_t i, int64_t &token, int &group) {
    if (!shared) {
        token = i;
        group = blockIdx.y;
    } else if (a.groups == 1) {
        token = i;
        group = 0;
    } else {
        token = i / a.groups;
        group = (int)(i - token * a.groups);
    }
}

template <bool F32, bool VEC, bool FIRST, bool SHARED, int K>
__global__ __launch_bounds__(1024) void gate_forward_kernel(GateArgs a) {
    __shared__ float lds[16];
    const Place pl = place_of<K>(a.d);
    const int64_t rows = SHARED ? a.n_tokens * a.groups : a.n_tokens;
    const int64_t i = (int64_t)blockIdx.x * pl.rows + pl.sub;
    const bool live = i < rows;
    int64_t token;
    int group;
    row_at(a, SHARED, live ? i : 0, token, group);
    float w[8 * K], x[8 * K], z[8 * K];
    Raw8<F32> rx[K], rz[K] = {};
    load_row<F32, VEC, K>(rx, a.x, token * a.x_stride + (int64_t)group * a.d, pl, a.d);
    if (a.z) load_row<F32, VEC, K>(rz, a.z, token * a.z_stride + (int64_t)group * a.d, pl, a.d);
    load_weights<K>(w, a.weight ? a.weight + (SHARED ? 0 : (int64_t)group * a.d) : nullptr, pl, a.d, 1.f);
    widen_row<F32, K>(rx, x);
    widen_row<F32, K>(rz, z);
    if (a.z)
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) z[e] = gate_of(a.act, z[e]);
    float s[1] = {0.f};
#pragma unroll
    for (int e = 0; e < 8 * K; ++e) {
        if (FIRST && a.z) x[e] *= z[e];
        s[0] = fmaf(x[e], x[e], s[0]);
    }
    row_sums<1>(s, pl.width, lds);
    const float rs = rstd_of(s[0], a.d, a.eps);
#pragma unroll
    for (int e = 0; e < 8 * K; ++e) {
        x[e] = x[e] * rs * w[e];
        if (!FIRST && a.z) x[e] *= z[e];
    }
    if (live) store_row<F32, VEC, K>(a.y, (token * a.groups + group) * a.d, x, pl, a.d);
}

template <bool F32, bool VEC, bool FIRST, bool SHARED, int K>
__global__ __launch_bounds__(1024) void gate_backward_kernel(GateArgs a) {
    __shared__ float lds[512 * K + 32];
    const Place pl = place_of<K>(a.d);
    const int64_t rows = SHARED ? a.n_tokens * a.groups : a.n_tokens;
    const float over = 1.f / (float)a.d;
    float w[8 * K], dw[1][8 * K] = {};
    load_weights<K>(w, a.weight ? a.weight + (SHARED ? 0 : (int64_t)blockIdx.y * a.d) : nullptr, pl, a.d, 1.f);
    // every thread of a workgroup makes the same turns: the sums have barriers
    for (int64_t i0 = (int64_t)blockIdx.x * pl.rows; i0 < rows; i0 += (int64_t)gridDim.x * pl.rows) {
        const int64_t i = i0 + pl.sub;
        const bool live = i < rows;
        int64_t token;
        int group;
        row_at(a, SHARED, live ? i : 0, token, group);
        Raw8<F32> rx[K], rz[K] = {}, ry[K];
        load_row<F32, VEC, K>(rx, a.x, token * a.x_stride + (int64_t)group * a.d, pl, a.d);
        if (a.z) load_row<F32, VEC, K>(rz, a.z, token * a.z_stride + (int64_t)group * a.d, pl, a.d);
        load_row<F32, VEC, K>(ry, a.dy, (token * a.groups + group) * a.d, pl, a.d);
        float x[8 * K], z[8 * K], dy[8 * K], act[8 * K], slope[8 * K];
        widen_row<F32, K>(rx, x);
        widen_row<F32, K>(rz, z);
        widen_row<F32, K>(ry, dy);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) {
            act[e] = 1.f, slope[e] = 0.f;
            if (a.z) gate_and_slope(a.act, z[e], act[e], slope[e]);
            const float u = FIRST ? x[e] * act[e] : x[e], t = FIRST ? dy[e] * w[e] : dy[e] * w[e] * act[e];
            s[0] = fmaf(u, u, s[0]);
            s[1] = fmaf(t, u, s[1]);
        }
        row_sums<2>(s, pl.width, lds + 512 * K);
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
            store_row<F32, VEC, K>(a.dx, token * a.dx_stride + (int64_t)group * a.d, dx, pl, a.d);
            if (a.dz) store_row<F32, VEC, K>(a.dz, token * a.dz_stride + (int64_t)group * a.d, dz, pl, a.d);
        }
    }
    float *const out[1] = {a.dweight ? a.partial + ((int64_t)blockIdx.x * gridDim.y + blockIdx.y) * a.d : nullptr};
    store_sums<K, 1>(dw, out, pl, a.d, lds);
}

template <bool F32, bool RF32, bool VEC, int K> __global__ __launch_bounds__(1024) void residual_forward_kernel(ResidualArgs a) {
    __shared__ float lds[16];
    const Place pl = place_of<K>(a.d);
    const int64_t i = (int64_t)blockIdx.x * pl.rows + pl.sub;
    const bool live = i < a.n_rows;
    const int64_t at = (live ? i : 0) * a.d;
    Raw8<F32> ro[K];
    Raw8<RF32> rr[K] = {};
    load_row<F32, VEC, K>(ro, a.o, at, pl, a.d);
    if (a.r) load_row<RF32, VEC, K>(rr, a.r, at, pl, a.d);
    float o[8 * K], r[8 * K], w[8 * K], s[1] = {0.f};
    widen_row<F32, K>(ro, o);
    widen_row<RF32, K>(rr, r);
    if (a.post) {
        load_weights<K>(w, a.post, pl, a.d, 1.f);
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) s[0] = fmaf(o[e], o[e], s[0]);
        row_sums<1>(s, pl.width, lds);
        const float rs = rstd_of(s[0], a.d, a.eps);
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) o[e] = o[e] * rs * w[e];
    }
    load_weights<K>(w, a.scale, pl, a.d, 1.f);
    s[0] = 0.f;
#pragma unroll
    for (int e = 0; e < 8 * K; ++e) {
        r[e] = fmaf(w[e], o[e], r[e]);
        s[0] = fmaf(r[e], r[e], s[0]);
    }
    if (live) store_row<RF32, VEC, K>(a.r_out, at, r, pl, a.d);
    if (!a.h) return;
    load_weights<K>(w, a.weight, pl, a.d, 1.f);
    row_sums<1>(s, pl.width, lds);
    const float rs = rstd_of(s[0], a.d, a.eps);
#pragma unroll
    for (int e = 0; e < 8 * K; ++e) r[e] = r[e] * rs * w[e];
    if (live) store_row<F32, VEC, K>(a.h, at, r, pl, a.d);
}

template <bool F32, bool RF32, bool VEC, int K> __global__ __launch_bounds__(1024) void residual_backward_kernel(ResidualArgs a) {
    __shared__ float lds[512 * K + 32];
    const Place pl = place_of<K>(a.d);
    const float over = 1.f / (float)a.d;
    float post[8 * K], scale[8 * K], w[8 * K], sums[3][8 * K] = {};
    load_weights<K>(post, a.post, pl, a.d, 1.f);
    load_weights<K>(scale, a.scale, pl, a.d, 1.f);
    load_weights<K>(w, a.weight, pl, a.d, 1.f);
    for (int64_t i0 = (int64_t)blockIdx.x * pl.rows; i0 < a.n_rows; i0 += (int64_t)gridDim.x * pl.rows) {
        const bool live = i0 + pl.sub < a.n_rows;
        const int64_t at = (live ? i0 + pl.sub : 0) * a.d;
        Raw8<F32> ro[K], rh[K] = {};
        Raw8<RF32> rr[K] = {}, rd[K] = {};
        load_row<F32, VEC, K>(ro, a.o, at, pl, a.d);
        if (a.r) load_row<RF32, VEC, K>(rr, a.r, at, pl, a.d);
        if (a.dh) load_row<F32, VEC, K>(rh, a.dh, at, pl, a.d);
        if (a.dr_out) load_row<RF32, VEC, K>(rd, a.dr_out, at, pl, a.d);
        float o[8 * K], r[8 * K], dh[8 * K], t[8 * K];
        widen_row<F32, K>(ro, o);
        widen_row<RF32, K>(rr, r);
        widen_row<F32, K>(rh, dh);
        widen_row<RF32, K>(rd, t);
        float so[1] = {0.f}, s[2] = {0.f, 0.f};
        float rso = 1.f;
        if (a.post) {
#pragma unroll
            for (int e = 0; e < 8 * K; ++e) so[0] = fmaf(o[e], o[e], so[0]);
            row_sums<1>(so, pl.width, lds + 512 * K);
            rso = rstd_of(so[0], a.d, a.eps);
        }
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) {
            o[e] *= rso;  // the norm behind the block, without its weight
            r[e] = fmaf(scale[e], a.post ? o[e] * post[e] : o[e], r[e]);
            s[0] = fmaf(r[e], r[e], s[0]);
            s[1] = fmaf(dh[e] * w[e], r[e], s[1]);
        }
        if (a.dh) {
            row_sums<2>(s, pl.width, lds + 512 * K);
            const float rs = rstd_of(s[0], a.d, a.eps), c = s[1] * rs * over;
#pragma unroll
            for (int e = 0; e < 8 * K; ++e) {
                const float n = r[e] * rs;
                t[e] = fmaf(rs, fmaf(-n, c, dh[e] * w[e]), t[e]);
                if (live) sums[2][e] = fmaf(dh[e], n, sums[2][e]);
            }
        }
        if (live && a.dr) store_row<RF32, VEC, K>(a.dr, at, t, pl, a.d);
        so[0] = 0.f;
#pragma unroll
        for (int e = 0; e < 8 * K; ++e) {
            if (live) sums[1][e] = fmaf(t[e], a.post ? o[e] * post[e] : o[e], sums[1][e]);
            t[e] *= scale[e];
            if (a.post) {
                if (live) sums[0][e] = fmaf(t[e], o[e], sums[0][e]);
                t[e] *= post[e];
                so[0] = fmaf(t[e], o[e], so[0]);
            }
        }
        if (a.post) {
            row_sums<1>(so, pl.width, lds + 512 * K);
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
// 64 columns and 4 waves to a workgroup: wave w adds the rows w, w + 4, ...
__global__ __launch_bounds__(256) void column_sums_kernel(SumList list) {
    __shared__ float lds[4][64];
    const SumArgs &a = list.a[blockIdx.y];
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int64_t c = (int64_t)blockIdx.x * 64 + l;
    if ((int64_t)blockIdx.x * 64 >= a.cols) return;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < a.cols) {
        int64_t i = w;
        for (; i + 12 < a.rows; i += 16)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += a.part[(i + 4 * k) * a.row_stride + c];
        for (int k = 0; i < a.rows; i += 4, ++k) s[k] += a.part[i * a.row_stride + c];
    }
    lds[w][l] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (w == 0 && c < a.cols) a.out[c] = (lds[0][l] + lds[1][l]) + (lds[2][l] + lds[3][l]);
}

int row_width(int d, int k) {
    int width = 1;
    while (width * 8 * k < d) width <<= 1;
    return width;
}
// Threads of a workgroup: 256 that share rows of up to a wave, or those of one wider row.
int threads_of(int d, int k) { return row_width(d, k) > 64 ? row_width(d, k) : 256; }
int rows_at_once(int d, int k) { return threads_of(d, k) / row_width(d, k); }
int vectors_of(int d) { return d > 8192 ? 2 : 1; }

// The kernel's template arguments from truth values.
template <typename F> void pick(bool b, F f) {
    if (b) f(std::true_type{});
    else f(std::false_type{});
}

} // namespace

int norm_blocks(int64_t rows, int32_t d) {
    const int64_t turns = (rows + rows_at_once(d, vectors_of(d)) - 1) / rows_at_once(d, vectors_of(d));
    return (int)(turns < 512 ? (turns > 0 ? turns : 1) : 512);
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
    hipLaunchKernelGGL(column_sums_kernel, dim3((uint32_t)((cols + 63) / 64), n), dim3(256), 0, stream, list);
    return hipGetLastError();
}

hipError_t launch_gate_forward(const GateArgs &a, bool f32, bool vec, bool first, bool shared, hipStream_t stream) {
    const int k = vectors_of(a.d), at_once = rows_at_once(a.d, k);
    const int64_t rows = shared ? a.n_tokens * a.groups : a.n_tokens;
    const dim3 grid((uint32_t)((rows + at_once - 1) / at_once), shared ? 1 : a.groups), block(threads_of(a.d, k));
    pick(f32, [&](auto F) { pick(vec, [&](auto V) { pick(first, [&](auto G) { pick(shared, [&](auto S) { pick(k == 1, [&](auto O) {
        hipLaunchKernelGGL((gate_forward_kernel<F.value, V.value, G.value, S.value, O.value ? 1 : 2>), grid, block, 0, stream, a);
    }); }); }); }); });
    return hipGetLastError();
}

hipError_t launch_gate_backward(const GateArgs &a, bool f32, bool vec, bool first, bool shared, hipStream_t stream) {
    const int k = vectors_of(a.d);
    const int64_t rows = shared ? a.n_tokens * a.groups : a.n_tokens;
    const int blocks = norm_blocks(rows, a.d);
    const dim3 grid(blocks, shared ? 1 : a.groups), block(threads_of(a.d, k));
    pick(f32, [&](auto F) { pick(vec, [&](auto V) { pick(first, [&](auto G) { pick(shared, [&](auto S) { pick(k == 1, [&](auto O) {
        hipLaunchKernelGGL((gate_backward_kernel<F.value, V.value, G.value, S.value, O.value ? 1 : 2>), grid, block, 0, stream, a);
    }); }); }); }); });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t cols = (int64_t)a.d * (shared ? 1 : a.groups);
    const SumArgs s[1] = {{a.partial, a.dweight, blocks, cols, cols}};
    return launch_column_sums(s, 1, stream);
}

hipError_t launch_residual_forward(const ResidualArgs &a, bool f32, bool res_f32, bool vec, hipStream_t stream) {
    const int k = vectors_of(a.d), at_once = rows_at_once(a.d, k);
    const dim3 grid((uint32_t)((a.n_rows + at_once - 1) / at_once)), block(threads_of(a.d, k));
    pick(f32, [&](auto F) { pick(res_f32, [&](auto R) { pick(vec, [&](auto V) { pick(k == 1, [&](auto O) {
        hipLaunchKernelGGL((residual_forward_kernel<F.value, R.value, V.value, O.value ? 1 : 2>), grid, block, 0, stream, a);
    }); }); }); });
    return hipGetLastError();
}

hipError_t launch_residual_backward(const ResidualArgs &a, bool f32, bool res_f32, bool vec, hipStream_t stream) {
    const int k = vectors_of(a.d), blocks = norm_blocks(a.n_rows, a.d);
    const dim3 grid(blocks), block(threads_of(a.d, k));
    pick(f32, [&](auto F) { pick(res_f32, [&](auto R) { pick(vec, [&](auto V) { pick(k == 1, [&](auto O) {
        hipLaunchKernelGGL((residual_backward_kernel<F.value, R.value, V.value, O.value ? 1 : 2>), grid, block, 0, stream, a);
    }); }); }); });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t part = (int64_t)blocks * a.d;
    const SumArgs s[3] = {{a.partial, a.dpost, blocks, a.d, a.d}, {a.partial + part, a.dscale, blocks, a.d, a.d},
                          {a.partial + 2 * part, a.dweight, blocks, a.d, a.d}};
    return launch_column_sums(s, 3, stream);
}

} // namespace sqk
