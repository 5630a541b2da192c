// layer_norm.hip -- layer norm over the channels of a row, and its gradients.
//
//   n = (x - mean) / sqrt(var + eps),  out = n weight + bias
//   d = weight dout,  dx = (d - mean(d) - n mean(d n)) / sqrt(var + eps)
//   dweight = sum dout n,  dbias = sum dout
//
// Bound by memory: 8 (forward) or 14 (backward) operations a channel against 2
// or 3 activations moved.  A row is in registers, eight neighbouring channels
// a lane, so it is read once and the variance is that of the differences from
// the mean.  Rows of up to 512 channels have 16, 32 or 64 lanes of a wave,
// longer ones a workgroup.
#include <hip/hip_runtime.h>

#include "row_device.hpp"

namespace dwps {
namespace {

struct LayerArgs {
    const void *x;
    int64_t x_stride;
    const float *weight, *bias;
    uint32_t tokens, channels;
    float eps, inv;  // 1 / channels
    float count;     // channels: the mean of equal channels is what they are
};

// The sums of a row's lanes, in every one of them; G 0: of the workgroup.
template <int G, int n>
__device__ __forceinline__ void row_sums_of(float (&v)[n], float (*shared)[kMostWaves]) {
    if constexpr (G == 0) {
        group_totals<n>(v, shared);
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            v[i] = row_total(v[i]);
            float w = v[i];
            if (G >= 32) swap_rows(v[i], w), v[i] += w;
            w = v[i];
            if (G >= 64) swap_halves(v[i], w), v[i] += w;
        }
    }
}

// R rows at once: their loads are on their way together, and G 0 has a barrier
// for all their sums.  A workgroup has 256 / G rows R times (G 0: R rows,
// blockDim.x threads with K times 8 channels each).  16384 rows of 4096 channels
// in bf16: 48 us, 5.6 TB/s, with 2 rows (1 row 52, 4 rows 50; 3 rows in all: 2.9
// us, 2.4 with 1); 131072 rows of 128: 11 to 14 us.  8192 rows of 5120: 41 us, 4.1
// TB/s: of workgroups of 10 waves a CU holds two, 20 of its 32 waves (wave cycles over
// busy cycles: 5.0 a SIMD, 7.2 with workgroups of 8 or 16).
template <class T, int G, int K, int R>
__global__ __launch_bounds__(G ? 256 : 64 * kMostWaves) void layer_norm_kernel(LayerArgs a, uint32_t first,
                                                                              T *__restrict__ out) {
    constexpr int V = kVec;
    constexpr uint32_t kRows = G ? 256u / (G ? G : 1) : 1u;
    __shared__ float sh[2][R][kMostWaves];
    const uint32_t lane = G ? threadIdx.x % (G ? G : 1) : threadIdx.x, lanes = G ? G : blockDim.x;
    const int64_t C = a.channels, t0 = (int64_t)(first + blockIdx.x) * (kRows * R) + (G ? threadIdx.x / (G ? G : 1) : 0u);
    float x[R][K][V], w[K][V], b[K][V];
    uint32_t have[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t c = (k * lanes + lane) * V;
        have[k] = c < a.channels ? a.channels - c : 0u;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t t = t0 + i * kRows;
            load_n<T, V>(x[i][k], at_row<T>(a.x, t < (int64_t)a.tokens ? t : 0, a.x_stride, c), have[k], 0.0f);
        }
        load_n<float, V>(w[k], at_col(a.weight, c), have[k], 1.0f);
        load_n<float, V>(b[k], at_col(a.bias, c), have[k], 0.0f);
    }
    float sum[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        sum[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) sum[i] += x[i][k][j];
    }
    row_sums_of<G, R>(sum, sh[0]);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float mean = sum[i] / a.count;
        sum[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                x[i][k][j] = (uint32_t)j < have[k] ? x[i][k][j] - mean : 0.0f;
                sum[i] = __builtin_fmaf(x[i][k][j], x[i][k][j], sum[i]);
            }
    }
    row_sums_of<G, R>(sum, sh[1]);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[i], a.inv, a.eps));
        const int64_t t = t0 + i * kRows;
        if (t >= (int64_t)a.tokens) break;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) x[i][k][j] = __builtin_fmaf(x[i][k][j] * r, w[k][j], b[k][j]);
            store_n<T, V>(out + t * C + (k * lanes + lane) * V, x[i][k], have[k]);
        }
    }
}

// A workgroup takes every gridDim.x-th set of rows, the next one's loads on
// their way (WHOLE: rows of whole vectors), and keeps its sums over rows in
// registers; part[workgroup][dweight, dbias][channel].  8192 rows of 5120
// channels in bf16: 57 us, 4.4 TB/s: the next row's loads wait for two barriers.
// fp32 rows of more than 8192 channels in whole vectors spill 19 of 128 registers.
template <class T, int G, int K, bool WHOLE>
__global__ __launch_bounds__(G ? 256 : 64 * kMostWaves) void layer_norm_bwd_kernel(LayerArgs a, const T *__restrict__ dout,
                                                                                  T *__restrict__ dx, float *__restrict__ part,
                                                                                  uint32_t *hdr, uint32_t words) {
    constexpr int V = kVec;
    constexpr uint32_t kRows = G ? 256u / (G ? G : 1) : 1u;
    __shared__ float sh[2][2][kMostWaves];
    if (blockIdx.x == 0 && threadIdx.x == 0) mark_plain(hdr, words);
    const uint32_t lane = G ? threadIdx.x % (G ? G : 1) : threadIdx.x, lanes = G ? G : blockDim.x;
    const uint32_t own = G ? threadIdx.x / (G ? G : 1) : 0u;
    const int64_t C = a.channels, step = (int64_t)gridDim.x * kRows;
    float acc[2][K][V], weight[K][V];
    uint32_t have[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t c = (k * lanes + lane) * V;
        have[k] = c < a.channels ? a.channels - c : 0u;
        load_n<float, V>(weight[k], at_col(a.weight, c), have[k], 1.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[0][k][j] = acc[1][k][j] = 0.0f;
    }
    struct Row {
        Raw8<T> x[K], g[K];
    } next;
    auto fetch = [&](int64_t t) {
        if (t >= (int64_t)a.tokens) t = 0;  // dropped
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t c = have[k] ? (k * lanes + lane) * V : 0u;
            next.x[k].load(static_cast<const T *>(a.x) + t * a.x_stride + c);
            next.g[k].load(dout + t * C + c);
        }
    };
    int64_t t = (int64_t)blockIdx.x * kRows + own;
    if (WHOLE) fetch(t);
    // a set of rows begins below the last row; those of its rows past it count nothing
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < (int64_t)a.tokens; t0 += step, t += step) {
        const bool there = t < (int64_t)a.tokens;
        float x[K][V], g[K][V], sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (WHOLE) {
                next.x[k].values(x[k]);
                next.g[k].values(g[k]);
            } else {
                const int64_t c = (k * lanes + lane) * V, from = there ? t : 0;
                load_n<T, V>(x[k], at_row<T>(a.x, from, a.x_stride, (uint32_t)c), have[k], 0.0f);
                load_n<T, V>(g[k], dout + from * C + c, have[k], 0.0f);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (!there || (WHOLE && !have[k])) x[k][j] = g[k][j] = 0.0f;
                sum[0] += x[k][j];
                sum[1] = __builtin_fmaf(weight[k][j], g[k][j], sum[1]);
            }
        }
        if (WHOLE) fetch(t + step);
        row_sums_of<G, 2>(sum, sh[0]);
        const float mean = sum[0] / a.count, lean = sum[1] * a.inv;
        sum[0] = sum[1] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                x[k][j] = (uint32_t)j < have[k] ? x[k][j] - mean : 0.0f;
                sum[0] = __builtin_fmaf(x[k][j], x[k][j], sum[0]);
                sum[1] = __builtin_fmaf(weight[k][j] * g[k][j], x[k][j], sum[1]);
            }
        row_sums_of<G, 2>(sum, sh[1]);
        // 0 for a row that is not there, also where eps is 0
        const float r = there ? __builtin_amdgcn_rsqf(__builtin_fmaf(sum[0], a.inv, a.eps)) : 0.0f, tilt = sum[1] * a.inv * r * r;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                acc[0][k][j] = __builtin_fmaf(g[k][j], x[k][j] * r, acc[0][k][j]);
                acc[1][k][j] += g[k][j];
                x[k][j] = r * __builtin_fmaf(-x[k][j], tilt, __builtin_fmaf(weight[k][j], g[k][j], -lean));
            }
            if (there) store_n<T, V>(dx + t * C + (k * lanes + lane) * V, x[k], have[k]);
        }
    }
    if constexpr (G != 0) {
        // the rows' sums of a workgroup meet in shared memory, G lanes a set
        constexpr uint32_t kSets = 256u / (G ? G : 1);
        __shared__ float meet[2][256 * V];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int j = 0; j < V; ++j) meet[w][j * 256 + threadIdx.x] = acc[w][0][j];
        __syncthreads();
        for (uint32_t c = threadIdx.x; c < 2u * a.channels; c += 256u) {
            const uint32_t w = c >= a.channels ? 1u : 0u, col = c - w * a.channels;
            float v = 0.0f;
            for (uint32_t i = 0; i < kSets; ++i) v += meet[w][(col % V) * 256u + i * (G ? G : 1) + col / V];
            part[(int64_t)blockIdx.x * 2 * C + c] = v;
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int w = 0; w < 2; ++w)
                store_n<float, V>(part + ((int64_t)blockIdx.x * 2 + w) * C + (k * lanes + lane) * V, acc[w][k], have[k]);
    }
}

// 16 columns a workgroup, so that few channels too are summed by many: 128
// channels of 1024 workgroups 3.9 us, with 64 columns a workgroup of 4 waves 12.6.
__global__ __launch_bounds__(1024) void layer_params_kernel(const float *__restrict__ part, uint32_t rows, uint32_t channels,
                                                            float *__restrict__ dweight, float *__restrict__ dbias) {
    __shared__ float s[64][17];
    const uint32_t lane = threadIdx.x & 15u, set = threadIdx.x >> 4;
    const uint32_t cols = 2u * channels, col = blockIdx.x * 16u + lane;
    s[set][lane] = col < cols ? column_sum(part + col, set, 64u, rows, cols) : 0.0f;
    __syncthreads();
    if (threadIdx.x >= 256u) return;
    // 16 lanes a column, four sets each
    const uint32_t c = threadIdx.x >> 4, to_col = blockIdx.x * 16u + c;
    const float v = row_total((s[lane][c] + s[lane + 16u][c]) + (s[lane + 32u][c] + s[lane + 48u][c]));
    if (lane || to_col >= cols) return;
    float *to = to_col < channels ? dweight : dbias;
    if (to) to[to_col < channels ? to_col : to_col - channels] = v;
}

// Calls f(lanes a row, or 0 for a workgroup, vectors a thread, threads).
template <class F>
ps_status with_rows(uint32_t channels, F f) {
    auto is = [](auto i) { return i; };
    typedef std::integral_constant<int, 1> One;
    if (channels <= 16u * kVec) return f(is(std::integral_constant<int, 16>()), One(), 256u);
    if (channels <= 32u * kVec) return f(is(std::integral_constant<int, 32>()), One(), 256u);
    if (channels <= 64u * kVec) return f(is(std::integral_constant<int, 64>()), One(), 256u);
    const uint32_t wave = 64u * kVec;
    if (channels <= wave * kMostWaves)
        return f(std::integral_constant<int, 0>(), One(), (uint32_t)ceil_div(channels, wave) * 64u);
    return f(std::integral_constant<int, 0>(), std::integral_constant<int, 2>(), (uint32_t)ceil_div(channels, 2u * wave) * 64u);
}

// Workgroups that share the rows backwards: 16 waves or more a CU where the
// registers hold them (8192 rows of 5120 channels, 10 waves a workgroup: 72 us
// with one a CU, 57 with two, 70 with four), and four sets of rows each, down to
// one a CU: what a workgroup leaves has to be read again (2047 rows of 1537: the
// sums over workgroups 4.2 us, 6.3 with two sets each, 3.8 with eight, which
// takes 3 us longer before).
uint32_t layer_bwd_groups(const ps_layer_input *in) {
    uint32_t groups = 0;
    with_rows(in->channels, [&](auto lanes, auto k, uint32_t threads) {
        constexpr uint32_t G = decltype(lanes)::value;
        const uint32_t held = (decltype(k)::value == 1 ? 28u : 16u) * 64u / threads, wanted = (uint32_t)ceil_div(1024u, threads);
        const uint64_t sets = ceil_div(in->tokens, G ? 256u / (G ? G : 1u) : 1u), most = 256u * (wanted < held ? wanted : held);
        uint64_t n = ceil_div(sets, 4u);
        if (n < 256u) n = sets < 256u ? sets : 256u;
        groups = (uint32_t)(n < most ? n : most);
        return PS_OK;
    });
    return groups;
}

ps_status layer_sizes(const ps_layer_input *in) {
    if (!in) return PS_ERR_NULL;
    if (!dtype_bytes(in->dtype)) return PS_ERR_UNSUPPORTED;
    const int64_t c = in->channels;
    if (in->tokens > kBlockMaxTokens || c == 0 || c > PS_NORM_MAX_CHANNELS || in->x_stride < c || in->x_stride > kBlockMaxStride)
        return PS_ERR_SIZE;
    return PS_OK;
}

ps_status layer_pointers(const ps_layer_input *in) {
    if (in->tokens && !in->x) return PS_ERR_NULL;
    if (!aligned(in->x, dtype_bytes(in->dtype)) || !aligned(in->weight, 4) || !aligned(in->bias, 4)) return PS_ERR_ALIGNMENT;
    return PS_OK;
}

LayerArgs layer_args(const ps_layer_input *in) {
    LayerArgs a{};
    a.x = in->x, a.x_stride = in->x_stride;
    a.weight = in->weight, a.bias = in->bias;
    a.tokens = (uint32_t)in->tokens, a.channels = in->channels;
    a.eps = in->eps, a.inv = 1.0f / (float)in->channels, a.count = (float)in->channels;
    return a;
}

}  // namespace
}  // namespace dwps

using namespace dwps;

extern "C" ps_status ps_layer_norm(const ps_layer_input *in, void *out, void *stream) {
    ps_status st = layer_sizes(in);
    if (st != PS_OK) return st;
    if ((st = layer_pointers(in)) != PS_OK) return st;
    if (!in->tokens) return PS_OK;
    const size_t e = dtype_bytes(in->dtype), c = in->channels;
    if (!out) return PS_ERR_NULL;
    if (!aligned(out, e)) return PS_ERR_ALIGNMENT;
    if (outputs_overlap({{out, in->tokens * c * e}},
                        {{in->x, rows_bytes(in->tokens, in->x_stride, c, e)}, {in->weight, c * 4u}, {in->bias, c * 4u}}))
        return PS_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const LayerArgs a = layer_args(in);
    return with_type(in->dtype, [&](auto zero) {
        using T = decltype(zero);
        return with_rows(in->channels, [&](auto lanes, auto k, uint32_t threads) {
            constexpr int G = decltype(lanes)::value, R = G ? 4 : 2;
            constexpr uint32_t rows = G ? 256u / (G ? G : 1) * R : R;
            timing_begin(s);
            launch_in_parts(ceil_div(in->tokens, rows), 1u, threads, [&](uint32_t first, uint32_t grid) {
                hipLaunchKernelGGL((layer_norm_kernel<T, G, decltype(k)::value, R>), dim3(grid), dim3(threads), 0, s, a, first,
                                   static_cast<T *>(out));
            });
            timing_end(s);
            return launch_status();
        });
    });
}

extern "C" ps_status ps_layer_norm_bwd(void *ws, size_t *ws_bytes, const ps_layer_input *in, const void *dout, void *dx,
                                       float *dweight, float *dbias, void *stream) {
    ps_status st = layer_sizes(in);
    if (st != PS_OK) return st;
    const uint32_t groups = layer_bwd_groups(in);
    PlainWs plan;
    const size_t part_at = plan.take((size_t)groups * 2u * in->channels * 4u);
    bool query = false;
    st = workspace_protocol(ws, ws_bytes, plan.at, &query);
    if (st != PS_OK || query) return st;
    if ((st = layer_pointers(in)) != PS_OK) return st;
    const size_t e = dtype_bytes(in->dtype), c = in->channels, cells = in->tokens * c * e;
    if (in->tokens && (!dout || !dx)) return PS_ERR_NULL;
    if (!aligned(ws, 16) || !aligned(dout, e) || !aligned(dx, e) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return PS_ERR_ALIGNMENT;
    if (outputs_overlap({{dx, cells}, {dweight, c * 4u}, {dbias, c * 4u}},
                        {{in->x, rows_bytes(in->tokens, in->x_stride, c, e)}, {in->weight, c * 4u}, {in->bias, c * 4u},
                         {dout, cells}}))
        return PS_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const LayerArgs a = layer_args(in);
    return with_type(in->dtype, [&](auto zero) {
        using T = decltype(zero);
        return with_rows(in->channels, [&](auto lanes, auto k, uint32_t threads) {
            constexpr int G = decltype(lanes)::value, K = decltype(k)::value;
            float *part = ws_at<float>(ws, part_at);
            timing_begin(s);
            auto launch = [&](auto whole) {
                hipLaunchKernelGGL((layer_norm_bwd_kernel<T, G, K, decltype(whole)::value>), dim3(groups), dim3(threads), 0, s, a,
                                   static_cast<const T *>(dout), static_cast<T *>(dx), part, ws_counter(ws), plan.words());
            };
            if (groups && in->channels % kVec == 0u) launch(std::true_type());
            else if (groups) launch(std::false_type());
            if (dweight || dbias)
                hipLaunchKernelGGL(layer_params_kernel, dim3((uint32_t)ceil_div(2u * in->channels, 16)), dim3(1024), 0, s, part,
                                   groups, in->channels, dweight, dbias);
            timing_end(s);
            return launch_status();
        });
    });
}
