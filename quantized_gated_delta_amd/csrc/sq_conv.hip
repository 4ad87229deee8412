// A short causal convolution of every channel with its own W taps, over ragged sequences:
//   p[t] = b + sum_k w[W-1-k] x[t-k]   (k = 0 .. W-1; before the sequence: the rows of S0)
//   y = p, or p sigma(p);  S_out: the last W - 1 inputs.
// Gradients, with dp = dy act'(p) formed again from x:
//   dx[t] = sum_k w[W-1-k] dp[t+k] (+ what reaches x[t] through S_out),  dw[W-1-k] = sum_t dp[t] x[t-k],
//   db = sum_t dp[t];  dS0 is dx at the W - 1 places before the sequence.
//
// Bound by memory: one input and one output per element and a handful of operations.  A lane has 8
// neighbouring channels (16 bytes of bf16) and walks a run of tokens with the last W - 1 inputs in
// registers, so an input is read (W - 1 + run) / run times, and that by a lane of the same L2.
#include "sq_block.h"

namespace sqk {
namespace {

constexpr int kRunShift = 4, kRun = 1 << kRunShift;          // tokens of a lane, forward
constexpr int kBlockShift = kRunShift + 2;                   // ... of a workgroup's four waves
constexpr int kBackShift = 5, kBackRun = 1 << kBackShift;    // backward
constexpr int kBackBlockShift = kBackShift + 2;

// Row `at` of sequence b as the convolution sees it: a token, a row of S0 before them, or zeros.
template <bool F32, bool VEC, int W>
__device__ __forceinline__ Raw8<F32> input_row(const ConvArgs &a, const Block &b, int at, int c0, int left) {
    if (at >= 0) return load8<F32, VEC>(a.x, (int64_t)(b.t0 + at) * a.x_stride + c0, left);
    if (a.S0) return load8<F32, VEC>(a.S0, ((int64_t)b.seq * (W - 1) + W - 1 + at) * a.channels + c0, left);
    return Raw8<F32>{};
}

template <int W> __device__ __forceinline__ void load_taps(const ConvArgs &a, int c0, int left, float (&w)[W][8], float (&bias)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = e < left ? a.weight[(int64_t)(c0 + e) * W + j] : 0.f;
        bias[e] = a.bias && e < left ? a.bias[c0 + e] : 0.f;
    }
}

template <bool F32, bool VEC, int W> __global__ __launch_bounds__(256) void conv_forward_kernel(ConvArgs a) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
    const Block b = block_at(a.seqs, blockIdx.x, kBlockShift);
    const int c0 = (blockIdx.y * 64 + l) * 8, left = a.channels - c0;
    if (b.seq < 0 || left <= 0) return;
    const int first = (b.c << kBlockShift) + wave * kRun, last = min(first + kRun, b.len);
    const bool ends = wave == 0 && ((b.c + 1) << kBlockShift) >= b.len;  // the sequence's last block
    if (a.S_out && ends)
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            float v[8];
            widen8<F32>(input_row<F32, VEC, W>(a, b, b.len - (W - 1) + i, c0, left), v);
            store8<F32, VEC>(a.S_out, ((int64_t)b.seq * (W - 1) + i) * a.channels + c0, v, left);
        }
    if (first >= last) return;
    float w[W][8], bias[8], x[W][8];  // x: the input and those before it, the oldest first
    load_taps<W>(a, c0, left, w, bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) widen8<F32>(input_row<F32, VEC, W>(a, b, first - (W - 1) + j, c0, left), x[j]);
    constexpr int kAhead = 8;  // loads in flight
    for (int t0 = first; t0 < last; t0 += kAhead) {
        Raw8<F32> raw[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) raw[i] = load8<F32, VEC>(a.x, (int64_t)(b.t0 + min(t0 + i, last - 1)) * a.x_stride + c0, left);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            widen8<F32>(raw[i], x[W - 1]);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float p = bias[e];
#pragma unroll
                for (int j = 0; j < W; ++j) p = fmaf(w[j][e], x[j][e], p);
                y[e] = a.silu ? gate_of(SQ_ACT_SILU, p) : p;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) x[j][e] = x[j + 1][e];
            }
            if (t0 + i < last) store8<F32, VEC>(a.y, (int64_t)(b.t0 + t0 + i) * a.channels + c0, y, left);
        }
    }
}

// Every workgroup walks the blocks blockIdx.x, + gridDim.x, ... and leaves its sums of dw and db in
// partial[blockIdx.x][channels][W + 1].
template <bool F32, bool VEC, int W> __global__ __launch_bounds__(256) void conv_backward_kernel(ConvArgs a, int64_t slots) {
    __shared__ float lds[64 * 8 * (W + 1)];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
    const int c0 = (blockIdx.y * 64 + l) * 8, left = a.channels - c0;
    float w[W][8], bias[8], dw[W + 1][8] = {};
    load_taps<W>(a, c0, left, w, bias);
    for (int64_t slot = blockIdx.x; slot < slots; slot += gridDim.x) {
        const Block b = block_at(a.seqs, slot, kBackBlockShift);
        if (b.seq < 0) continue;
        const int first = (b.c << kBackBlockShift) + wave * kBackRun, last = min(first + kBackRun, b.len);
        const bool begins = first == 0;
        if (first >= last && !begins) continue;
        if (left <= 0) continue;
        // gradient of input `at` (a token, or before them a row of S0), sum: what came through the taps
        auto store = [&](int at, float (&sum)[8]) {
            const int row = at - (b.len - (W - 1));  // its row of S_out
            if (a.dS_out && row >= 0) {
                float v[8];
                widen8<F32>(load8<F32, VEC>(a.dS_out, ((int64_t)b.seq * (W - 1) + row) * a.channels + c0, left), v);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += v[e];
            }
            if (at >= 0) store8<F32, VEC>(a.dx, (int64_t)(b.t0 + at) * a.channels + c0, sum, left);
            else if (a.dS0) store8<F32, VEC>(a.dS0, ((int64_t)b.seq * (W - 1) + W - 1 + at) * a.channels + c0, sum, left);
        };
        // x: inputs t - W + 1 .. t; d: dp of t - W + 1 .. t, as far as they are known
        float x[W][8], d[W][8] = {};
#pragma unroll
        for (int j = 0; j < W - 1; ++j) widen8<F32>(input_row<F32, VEC, W>(a, b, first - (W - 1) + j, c0, left), x[j]);
        // dp of the W - 1 tokens behind the run reaches its last inputs; the first run also has the
        // inputs before the sequence
        constexpr int kAhead = 4;
        const int stop = last + W - 1;
        for (int t0 = first; t0 < stop; t0 += kAhead) {
            Raw8<F32> rx[kAhead] = {}, ry[kAhead] = {};
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int t = t0 + i;
                if (t < b.len && t < stop) {
                    rx[i] = load8<F32, VEC>(a.x, (int64_t)(b.t0 + t) * a.x_stride + c0, left);
                    ry[i] = load8<F32, VEC>(a.dy, (int64_t)(b.t0 + t) * a.channels + c0, left);
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int t = t0 + i;
                if (t < stop) {
                    float dy[8], sum[8];
                    widen8<F32>(rx[i], x[W - 1]);
                    widen8<F32>(ry[i], dy);
                    const bool inside = t < b.len, mine = t < last;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float p = bias[e], value, slope = 1.f;
#pragma unroll
                        for (int j = 0; j < W; ++j) p = fmaf(w[j][e], x[j][e], p);
                        if (a.silu) gate_and_slope(SQ_ACT_SILU, p, value, slope);
                        d[W - 1][e] = inside ? dy[e] * slope : 0.f;
                        if (mine) {
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[j][e] = fmaf(d[W - 1][e], x[j][e], dw[j][e]);
                            dw[W][e] += d[W - 1][e];
                        }
                        // input t - W + 1 has all its dp now: d[j] meets tap W - 1 - j
                        sum[e] = 0.f;
#pragma unroll
                        for (int j = 0; j < W; ++j) sum[e] = fmaf(w[W - 1 - j][e], d[j][e], sum[e]);
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) x[j][e] = x[j + 1][e], d[j][e] = d[j + 1][e];
                    }
                    const int at = t - (W - 1);
                    if (at >= first || begins) store(at, sum);
                }
            }
        }
    }
    // the four waves' sums, in their order
    const int64_t row = (int64_t)a.channels * (W + 1);
#pragma unroll 1
    for (int other = 0; other < 4; ++other) {
        if (wave == other)
#pragma unroll
            for (int j = 0; j <= W; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float &s = lds[(j * 8 + e) * 64 + l];
                    s = (other ? s : 0.f) + dw[j][e];
                }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < 64 * 8 * (W + 1); i += 256) {
        const int lane = i & 63, e = i >> 6 & 7, j = i >> 9, c = (blockIdx.y * 64 + lane) * 8 + e;
        if (c < a.channels) a.partial[blockIdx.x * row + (int64_t)j * a.channels + c] = lds[i];
    }
}

// partial[blocks][W + 1][channels] into dweight [channels][W] and dbias.
template <int W> __global__ __launch_bounds__(256) void conv_sums_kernel(ConvArgs a, int blocks) {
    __shared__ float lds[4][64];
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63, c = blockIdx.x * 64 + l, j = blockIdx.y;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < a.channels) {
        const float *p = a.partial + (int64_t)j * a.channels + c;
        const int64_t row = (int64_t)a.channels * (W + 1);
        int i = w;
        for (; i + 12 < blocks; i += 16)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += p[(i + 4 * k) * row];
        for (int k = 0; i < blocks; i += 4, ++k) s[k] += p[i * row];
    }
    lds[w][l] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (w == 0 && c < a.channels) {
        const float sum = (lds[0][l] + lds[1][l]) + (lds[2][l] + lds[3][l]);
        if (j < W) a.dweight[(int64_t)c * W + j] = sum;
        else if (a.dbias) a.dbias[c] = sum;
    }
}

// One token a request on a pool of the last inputs [n_slots, W - 1, channels], in place.
template <bool F32, bool VEC, int W> __global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a) {
    const int per_row = (a.channels + 7) / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)a.n * per_row) return;
    const int r = (int)(i / per_row), c0 = (int)(i - (int64_t)r * per_row) * 8, left = a.channels - c0;
    const int32_t slot = a.slot[r];
    if (slot < 0 || slot >= a.n_slots) return;
    const int64_t at = (int64_t)slot * (W - 1) * a.channels + c0;
    Raw8<F32> raw[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) raw[j] = load8<F32, VEC>(a.pool, at + (int64_t)j * a.channels, left);
    raw[W - 1] = load8<F32, VEC>(a.x, r * a.x_stride + c0, left);
    float w[W][8], p[8];
    load_taps<W>(a, c0, left, w, p);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float x[8];
        widen8<F32>(raw[j], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = fmaf(w[j][e], x[e], p[e]);
        if (j > 0) store8<F32, VEC>(a.pool, at + (int64_t)(j - 1) * a.channels, x, left);
    }
    if (a.silu)
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = gate_of(SQ_ACT_SILU, p[e]);
    store8<F32, VEC>(a.y, (int64_t)r * a.channels + c0, p, left);
}

template <typename F> void pick(bool b, F f) {
    if (b) f(std::true_type{});
    else f(std::false_type{});
}
template <typename F> void pick_width(int w, F f) {
    if (w == 2) f(std::integral_constant<int, 2>{});
    else if (w == 3) f(std::integral_constant<int, 3>{});
    else f(std::integral_constant<int, 4>{});
}
uint32_t tiles_of(int channels) { return (channels + 511) / 512; }

} // namespace

// About 2048 workgroups in all: two rounds of four per CU.
int conv_blocks(int64_t n_tokens, int32_t n_seq, int32_t channels) {
    const int64_t slots = block_slots(n_tokens, n_seq, kBackBlockShift), most = 2048 / tiles_of(channels);
    const int64_t blocks = slots < most ? slots : most;
    return (int)(blocks < 1 ? 1 : blocks);
}

hipError_t launch_conv_forward(const ConvArgs &a, bool f32, bool vec, hipStream_t stream) {
    const dim3 grid((uint32_t)block_slots(a.seqs.n_tokens, a.seqs.n_seq, kBlockShift), tiles_of(a.channels));
    pick(f32, [&](auto F) { pick(vec, [&](auto V) { pick_width(a.width, [&](auto W) {
        hipLaunchKernelGGL((conv_forward_kernel<F.value, V.value, W.value>), grid, dim3(256), 0, stream, a);
    }); }); });
    return hipGetLastError();
}

hipError_t launch_conv_backward(const ConvArgs &a, bool f32, bool vec, hipStream_t stream) {
    const int64_t slots = block_slots(a.seqs.n_tokens, a.seqs.n_seq, kBackBlockShift);
    const int blocks = conv_blocks(a.seqs.n_tokens, a.seqs.n_seq, a.channels);
    const dim3 grid(blocks, tiles_of(a.channels));
    pick(f32, [&](auto F) { pick(vec, [&](auto V) { pick_width(a.width, [&](auto W) {
        hipLaunchKernelGGL((conv_backward_kernel<F.value, V.value, W.value>), grid, dim3(256), 0, stream, a, slots);
    }); }); });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    pick_width(a.width, [&](auto W) {
        hipLaunchKernelGGL(conv_sums_kernel<W.value>, dim3((a.channels + 63) / 64, W.value + 1), dim3(256), 0, stream, a, blocks);
    });
    return hipGetLastError();
}

hipError_t launch_conv_step(const ConvArgs &a, bool f32, bool vec, hipStream_t stream) {
    const int64_t lanes = (int64_t)a.n * ((a.channels + 7) / 8);
    pick(f32, [&](auto F) { pick(vec, [&](auto V) { pick_width(a.width, [&](auto W) {
        hipLaunchKernelGGL((conv_step_kernel<F.value, V.value, W.value>), dim3((uint32_t)((lanes + 255) / 256)), dim3(256), 0, stream, a);
    }); }); });
    return hipGetLastError();
}

} // namespace sqk
