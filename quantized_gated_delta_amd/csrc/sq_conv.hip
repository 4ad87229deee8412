// A short causal convolution of every channel with its own W taps, over ragged sequences:
//   p[t] = b + sum_k w[W-1-k] x[t-k]   (k = 0 .. W-1; before the sequence: the rows of S0)
//   y = p, or p sigma(p);  S_out: the last W - 1 inputs.
// Gradients, with dp = dy act'(p) formed again from x:
//   dx[t] = sum_k w[W-1-k] dp[t+k] (+ what reaches x[t] through S_out),  dw[W-1-k] = sum_t dp[t] x[t-k],
//   db = sum_t dp[t];  dS0 is dx at the W - 1 places before the sequence.
//
// Bound by memory: one input and one output per element and a handful of operations.  A lane has 8
// neighbouring channels (16 bytes of bf16; backwards 4, whose sums and windows then leave room for three waves per SIMD: four at
// width 2 in bf16, two at width 4 in fp32) and walks a run of tokens with the last W - 1 inputs in registers, so an input is read (W - 1 + run) / run times, and
// that by a lane of the same L2.
#include "sq_block.h"

#include <algorithm>

namespace sqk {
namespace {

constexpr int kRunShift = 4, kRun = 1 << kRunShift;          // tokens of a lane, forward
constexpr int kBlockShift = kRunShift + 2;                   // ... of a workgroup's four waves
constexpr int kBackShift = 5, kBackRun = 1 << kBackShift;    // backward
constexpr int kBackBlockShift = kBackShift + 2;
constexpr int kWide = 8, kNarrow = 4;                        // channels of a lane, forward and backward
constexpr int kStepRows = 8;                                 // most requests of a lane in a step

// Row `at` of sequence b as the convolution sees it: a token, a row of S0 before them, or zeros.
template <bool F32, bool VEC, int W, int N>
__device__ __forceinline__ Raw<F32, N> input_row(const ConvArgs &a, const Block &b, int at, int c0, int left) {
    if (at >= 0) return load_n<F32, VEC, N>(a.x, (int64_t)(b.t0 + at) * a.x_stride + c0, left);
    if (a.S0) return load_n<F32, VEC, N>(a.S0, ((int64_t)b.seq * (W - 1) + W - 1 + at) * a.channels + c0, left);
    return Raw<F32, N>{};
}

// The taps and biases of a lane's channels.  Taps of neighbouring channels lie one after another: 16 bytes at a time.
template <bool VEC, int W, int N> __device__ __forceinline__ void load_taps(const ConvArgs &a, int c0, int left, float (&w)[W][N], float (&bias)[N]) {
    float flat[W * N];
    const float *p = a.weight + (int64_t)c0 * W;
#pragma unroll
    for (int i = 0; i < W * N; i += 4) {
        if constexpr (VEC) {
            *reinterpret_cast<f4 *>(flat + i) = *reinterpret_cast<const f4 *>(p + i);
        } else {
#pragma unroll
            for (int k = i; k < i + 4; ++k) flat[k] = k < left * W ? p[k] : 0.f;
        }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = flat[e * W + j];
        bias[e] = a.bias && e < left ? a.bias[c0 + e] : 0.f;
    }
}

// 8 loads of a lane in flight: 105 us for 12001 tokens x 10240 channels, 4.7 TB/s (8192 x 8192: 60 us, 4.5 TB/s).
template <bool F32, bool VEC, int W> __global__ __launch_bounds__(256) void conv_forward_kernel(ConvArgs a) {
    constexpr int N = kWide;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
    const Block b = block_at(a.seqs, blockIdx.x, kBlockShift);
    const int c0 = (blockIdx.y * 64 + l) * N, left = a.channels - c0;
    if (b.seq < 0 || left <= 0) return;
    const int first = (b.c << kBlockShift) + wave * kRun, last = min(first + kRun, b.len);
    const bool ends = wave == 0 && ((b.c + 1) << kBlockShift) >= b.len;  // the sequence's last block
    if (a.S_out && ends)
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            float v[N];
            widen_n<F32, N>(input_row<F32, VEC, W, N>(a, b, b.len - (W - 1) + i, c0, left), v);
            store_n<F32, VEC, N>(a.S_out, ((int64_t)b.seq * (W - 1) + i) * a.channels + c0, v, left);
        }
    if (first >= last) return;
    float w[W][N], bias[N], x[4][N];  // x: input t of a run lies in x[(t - first) % 4], so that no window moves
    Raw<F32, N> before[W - 1];
#pragma unroll
    for (int k = 1; k < W; ++k) before[k - 1] = input_row<F32, VEC, W, N>(a, b, first - k, c0, left);
    load_taps<VEC, W, N>(a, c0, left, w, bias);
#pragma unroll
    for (int k = 1; k < W; ++k) widen_n<F32, N>(before[k - 1], x[4 - k]);
    constexpr int kAhead = 8;  // loads in flight
    for (int t0 = first; t0 < last; t0 += kAhead) {
        Raw<F32, N> raw[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) raw[i] = load_n<F32, VEC, N>(a.x, (int64_t)(b.t0 + min(t0 + i, last - 1)) * a.x_stride + c0, left);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            widen_n<F32, N>(raw[i], x[i & 3]);
            float y[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float p = bias[e];
#pragma unroll
                for (int k = 0; k < W; ++k) p = fmaf(w[W - 1 - k][e], x[(i - k) & 3][e], p);
                y[e] = a.silu ? gate_of<F32>(SQ_ACT_SILU, p) : p;
            }
            if (t0 + i < last) store_n<F32, VEC, N>(a.y, (int64_t)(b.t0 + t0 + i) * a.channels + c0, y, left);
        }
    }
}

// Every workgroup walks the blocks blockIdx.x, + gridDim.x, ... and leaves its sums of dw and db in
// partial[blockIdx.x][W + 1][channels].  With 4 channels to a lane its sums and windows fit beside the loads in flight: 102 us
// for 8192 tokens x 8192 channels, 3.9 TB/s (8 channels: 170; held to four waves per SIMD, it spills: 320).  Its
// instructions are 0.35 of the waves' cycles.
template <bool F32, bool VEC, int W>
__global__ __launch_bounds__(256) void conv_backward_kernel(ConvArgs a, int64_t slots) {
    constexpr int N = kNarrow;
    __shared__ float lds[64 * N * (W + 1)];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
    const int c0 = (blockIdx.y * 64 + l) * N, left = a.channels - c0;
    float w[W][N] = {}, bias[N] = {}, dw[W + 1][N] = {};
    if (left > 0) load_taps<VEC, W, N>(a, c0, left, w, bias);
    for (int64_t slot = blockIdx.x; slot < slots; slot += gridDim.x) {
        const Block b = block_at(a.seqs, slot, kBackBlockShift);
        if (b.seq < 0) continue;
        const int first = (b.c << kBackBlockShift) + wave * kBackRun, last = min(first + kBackRun, b.len);
        const bool begins = first == 0;
        if (first >= last && !begins) continue;
        if (left <= 0) continue;
        // gradient of input `at` (a token, or before them a row of S0), sum: what came through the taps
        auto store = [&](int at, float (&sum)[N]) {
            const int row = at - (b.len - (W - 1));  // its row of S_out
            if (a.dS_out && row >= 0) {
                float v[N];
                widen_n<F32, N>(load_n<F32, VEC, N>(a.dS_out, ((int64_t)b.seq * (W - 1) + row) * a.channels + c0, left), v);
#pragma unroll
                for (int e = 0; e < N; ++e) sum[e] += v[e];
            }
            if (at >= 0) store_n<F32, VEC, N>(a.dx, (int64_t)(b.t0 + at) * a.channels + c0, sum, left);
            else if (a.dS0) store_n<F32, VEC, N>(a.dS0, ((int64_t)b.seq * (W - 1) + W - 1 + at) * a.channels + c0, sum, left);
        };
        // x, d: input and dp of token t of the run in [(t - first) % 4], so that no window moves
        float x[4][N], d[4][N] = {};
#pragma unroll
        for (int k = 1; k < W; ++k) widen_n<F32, N>(input_row<F32, VEC, W, N>(a, b, first - k, c0, left), x[4 - k]);
        Raw<F32, N> rx[4] = {}, ry[4] = {};
        auto load = [&](int t0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = min(t0 + i, b.len - 1);  // past the end: not used
                if (b.len > 0) {
                    rx[i] = load_n<F32, VEC, N>(a.x, (int64_t)(b.t0 + t) * a.x_stride + c0, left);
                    ry[i] = load_n<F32, VEC, N>(a.dy, (int64_t)(b.t0 + t) * a.channels + c0, left);
                }
            }
        };
        // four tokens from t0 on.  WHOLE: all of the run, none among its first W - 1, so that what they reach is the run's too
        auto four = [&](int t0, int stop, auto whole) {
            constexpr bool WHOLE = decltype(whole)::value;
            Raw<F32, N> cx[4], cy[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) cx[i] = rx[i], cy[i] = ry[i];
            if (t0 + 4 < stop) load(t0 + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = t0 + i;
                if (!WHOLE && t >= stop) break;
                float dy[N], sum[N];
                widen_n<F32, N>(cx[i], x[i]);
                widen_n<F32, N>(cy[i], dy);
                const bool inside = WHOLE || t < b.len, mine = WHOLE || t < last;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    float p = bias[e], value, slope = 1.f;
#pragma unroll
                    for (int k = 0; k < W; ++k) p = fmaf(w[W - 1 - k][e], x[(i - k) & 3][e], p);
                    if (a.silu) gate_and_slope<F32>(SQ_ACT_SILU, p, value, slope);
                    d[i][e] = inside ? dy[e] * slope : 0.f;
                    if (mine) {
#pragma unroll
                        for (int k = 0; k < W; ++k) dw[W - 1 - k][e] = fmaf(d[i][e], x[(i - k) & 3][e], dw[W - 1 - k][e]);
                        dw[W][e] += d[i][e];
                    }
                    // input t - W + 1 has all its dp now: that of k tokens before t meets tap k
                    sum[e] = 0.f;
#pragma unroll
                    for (int k = W - 1; k >= 0; --k) sum[e] = fmaf(w[k][e], d[(i - k) & 3][e], sum[e]);
                }
                const int at = t - (W - 1);
                if (WHOLE || at >= first || begins) store(at, sum);
            }
        };
        // dp of the W - 1 tokens behind the run reaches its last inputs; the first run also has the
        // inputs before the sequence
        const int stop = last + W - 1;
        load(first);
        four(first, stop, std::false_type{});
        int t0 = first + 4;
        for (; t0 + 4 <= last; t0 += 4) four(t0, stop, std::true_type{});
        for (; t0 < stop; t0 += 4) four(t0, stop, std::false_type{});
    }
    // the four waves' sums, in their order
    const int64_t row = (int64_t)a.channels * (W + 1);
#pragma unroll 1
    for (int other = 0; other < 4; ++other) {
        if (wave == other)
#pragma unroll
            for (int j = 0; j <= W; ++j)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    float &s = lds[(j * N + e) * 64 + l];
                    s = (other ? s : 0.f) + dw[j][e];
                }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < 64 * N * (W + 1); i += 256) {
        const int lane = i / N % 64, e = i % N, j = i / (64 * N), c = (blockIdx.y * 64 + lane) * N + e;
        if (c < a.channels) a.partial[blockIdx.x * row + (int64_t)j * a.channels + c] = lds[(j * N + e) * 64 + lane];
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
        if (j == W) {
            if (a.dbias) a.dbias[c] = sum;
        } else if (a.dweight) {
            a.dweight[(int64_t)c * W + j] = sum;
        }
    }
}

// One token a request on a pool of the last inputs [n_slots, W - 1, channels], in place.  A lane has the
// same 8 channels of `rows` requests, whose taps it loads once (512 requests x 10240 channels, 84 MB: 17.4 us, 4.8 TB/s;
// a request a lane 42).
template <bool F32, bool VEC, int W> __global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a, int rows) {
    constexpr int N = kWide;
    const int c0 = (blockIdx.y * 256 + threadIdx.x) * N, left = a.channels - c0, r0 = blockIdx.x * rows;
    if (left <= 0) return;
    float w[W][N], bias[N];
    load_taps<VEC, W, N>(a, c0, left, w, bias);
    for (int r = r0; r < min(r0 + rows, a.n); ++r) {
        const int32_t slot = a.slot[r];
        if (slot < 0 || slot >= a.n_slots) continue;
        const int64_t at = (int64_t)slot * (W - 1) * a.channels + c0;
        Raw<F32, N> raw[W];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) raw[j] = load_n<F32, VEC, N>(a.pool, at + (int64_t)j * a.channels, left);
        raw[W - 1] = load_n<F32, VEC, N>(a.x, r * a.x_stride + c0, left);
        float p[N];
#pragma unroll
        for (int e = 0; e < N; ++e) p[e] = bias[e];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float x[N];
            widen_n<F32, N>(raw[j], x);
#pragma unroll
            for (int e = 0; e < N; ++e) p[e] = fmaf(w[j][e], x[e], p[e]);
            if (j > 0) store_n<F32, VEC, N>(a.pool, at + (int64_t)(j - 1) * a.channels, x, left);
        }
        if (a.silu)
#pragma unroll
            for (int e = 0; e < N; ++e) p[e] = gate_of<F32>(SQ_ACT_SILU, p[e]);
        store_n<F32, VEC, N>(a.y, (int64_t)r * a.channels + c0, p, left);
    }
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
uint32_t tiles_of(int channels, int per_lane) { return (channels + 64 * per_lane - 1) / (64 * per_lane); }

} // namespace

// Up to 4096 workgroups in all ...
static int64_t most_blocks(int32_t channels) { return std::max<int64_t>(4096 / tiles_of(channels, kNarrow), 1); }
int64_t conv_partials(int64_t n_tokens, int32_t n_seq, int32_t channels) {
    return std::max<int64_t>(std::min(block_slots(n_tokens, n_seq, kBackBlockShift), most_blocks(channels)), 1);
}
// ... each with as many blocks of tokens as the others: just behind a full turn of them, fewer than a smaller batch has.
static int conv_blocks(int64_t slots, int32_t channels) {
    const int64_t turns = (slots + most_blocks(channels) - 1) / most_blocks(channels);
    return (int)(turns > 0 ? (slots + turns - 1) / turns : 1);
}

hipError_t launch_conv_forward(const ConvArgs &a, bool f32, bool vec, hipStream_t stream) {
    const dim3 grid((uint32_t)block_slots(a.seqs.n_tokens, a.seqs.n_seq, kBlockShift), tiles_of(a.channels, kWide));
    pick(f32, [&](auto F) { pick(vec, [&](auto V) { pick_width(a.width, [&](auto W) {
        hipLaunchKernelGGL((conv_forward_kernel<F.value, V.value, W.value>), grid, dim3(256), 0, stream, a);
    }); }); });
    return hipGetLastError();
}

hipError_t launch_conv_backward(const ConvArgs &a, bool f32, bool vec, hipStream_t stream) {
    const int64_t slots = block_slots(a.seqs.n_tokens, a.seqs.n_seq, kBackBlockShift);
    const int blocks = conv_blocks(slots, a.channels);
    const dim3 grid(blocks, tiles_of(a.channels, kNarrow));
    pick(f32, [&](auto F) { pick(vec, [&](auto V) { pick_width(a.width, [&](auto W) {
        hipLaunchKernelGGL((conv_backward_kernel<F.value, V.value, W.value>), grid, dim3(256), 0, stream, a, slots);
    }); }); });
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? launch_conv_sums(a, blocks, stream) : e;
}

hipError_t launch_conv_sums(const ConvArgs &a, int blocks, hipStream_t stream) {
    if (!a.dweight && !a.dbias) return hipSuccess;
    pick_width(a.width, [&](auto W) {
        hipLaunchKernelGGL(conv_sums_kernel<W.value>, dim3((a.channels + 63) / 64, W.value + 1), dim3(256), 0, stream, a, blocks);
    });
    return hipGetLastError();
}

hipError_t launch_conv_step(const ConvArgs &a, bool f32, bool vec, hipStream_t stream) {
    // as many requests to a lane as leave 512 lanes to a CU
    const int tiles = (a.channels + 256 * kWide - 1) / (256 * kWide);
    const int64_t most = (int64_t)a.n * tiles / 512;
    const int rows = most < 1 ? 1 : most < kStepRows ? (int)most : kStepRows;
    const dim3 grid((a.n + rows - 1) / rows, tiles);
    pick(f32, [&](auto F) { pick(vec, [&](auto V) { pick_width(a.width, [&](auto W) {
        hipLaunchKernelGGL((conv_step_kernel<F.value, V.value, W.value>), grid, dim3(256), 0, stream, a, rows);
    }); }); });
    return hipGetLastError();
}

} // namespace sqk
