// block_norm.hip -- the norms around a block with its gate and residual sum,
// and their gradients.
//
//   residual_out = residual + scale sigmoid(gate) post y / rms(y)
//   out          = pre residual_out / rms(residual_out)
//
// Bound by memory: 16 (forward) or 45 (backward) operations for every channel
// of a token against 5 or 8 activations moved.  A workgroup holds a row in
// registers, so the row is read once for both norms; the sums over the row
// are wave sums joined in shared memory.
#include <hip/hip_runtime.h>

#include "row_device.hpp"

namespace dwps {
namespace {

struct NormArgs {
    const void *y, *gate, *residual;
    int64_t y_stride, gate_stride, residual_stride;
    const float *scale, *post, *pre;
    uint32_t tokens, channels;
    uint32_t first;  // row of the launch's first workgroup
    float eps, inv;  // 1 / channels
};

// One row: blockDim.x threads with K times 8 neighbouring channels each.
// 16384 x 4096, bf16: 129 to 133 us (5 TB/s); 256 threads with two vectors 151 us.
template <class T, class R, int K>
__global__ __launch_bounds__(64 * kMostWaves) void norm_kernel(NormArgs a, R *__restrict__ res_out, T *__restrict__ out) {
    constexpr int V = kVec;
    __shared__ float sh[2][1][kMostWaves];
    const int64_t t = a.first + blockIdx.x, C = a.channels;
    float q[K][V], r[K][V], sum[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t c = (k * blockDim.x + threadIdx.x) * V, have = c < a.channels ? a.channels - c : 0u;
        float y[V], z[V], s[V], w[V];
        load_n<T, V>(y, at_row<T>(a.y, t, a.y_stride, c), have, 0.0f);
        load_n<T, V>(z, at_row<T>(a.gate, t, a.gate_stride, c), have, 0.0f);
        load_n<R, V>(r[k], at_row<R>(a.residual, t, a.residual_stride, c), have, 0.0f);
        load_n<float, V>(s, at_col(a.scale, c), have, 1.0f);
        load_n<float, V>(w, at_col(a.post, c), have, 1.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sum[0] = __builtin_fmaf(y[i], y[i], sum[0]);
            q[k][i] = (a.gate ? s[i] * sigmoid(z[i]) : s[i]) * (y[i] * w[i]);
        }
    }
    group_totals<1>(sum, sh[0]);
    const float ry = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[0], a.inv, a.eps));
    sum[0] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t c = (k * blockDim.x + threadIdx.x) * V, have = c < a.channels ? a.channels - c : 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            r[k][i] = __builtin_fmaf(q[k][i], ry, r[k][i]);
            sum[0] = __builtin_fmaf(r[k][i], r[k][i], sum[0]);
        }
        store_n<R, V>(res_out + t * C + c, r[k], have);
    }
    group_totals<1>(sum, sh[1]);
    const float rr = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[0], a.inv, a.eps));
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t c = (k * blockDim.x + threadIdx.x) * V, have = c < a.channels ? a.channels - c : 0u;
        float w[V];
        load_n<float, V>(w, at_col(a.pre, c), have, 1.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] *= r[k][i] * rr;
        store_n<T, V>(out + t * C + c, w, have);
    }
}

// Gradients.  With r = residual_out, ry and rr the two reciprocal norms,
// s = sigmoid(gate), w = pre dout:
//   dr = dresidual_out + rr (w - r rr^2 mean(w r))
//   u = scale s post dr,  dy = ry (u - y ry^2 mean(u y))
//   dgate = scale dr y ry post s (1 - s)
//   dscale = sum dr s y ry post,  dpost = sum scale dr s y ry,  dpre = sum dout r rr
// A workgroup takes every gridDim.x-th row and keeps its sums over rows in
// registers; part[workgroup][dscale, dpost, dpre][channel].  The next row's
// loads are on their way while one is worked on (WHOLE: rows of whole
// vectors, one a thread; others load their own).  8192 x 5120, bf16 with an
// fp32 residual: 177 to 191 us and 5 us for the sums (4.7 TB/s or more); without
// the next row on its way and with 20 channels a thread 535 us.

template <class T, class R, int MOST, int K, bool WHOLE>
__global__ __launch_bounds__(MOST) void norm_bwd_kernel(NormArgs a, const T *__restrict__ dout,
                                                                   const R *__restrict__ dres, T *__restrict__ dy,
                                                                   T *__restrict__ dgate, R *__restrict__ dr_out,
                                                                   float *__restrict__ part, uint32_t *hdr,
                                                                   uint32_t words) {
    constexpr int V = kVec;
    __shared__ float sh[2][3][kMostWaves];
    if (blockIdx.x == 0 && threadIdx.x == 0) mark_plain(hdr, words);
    const int64_t C = a.channels;
    float acc[3][K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[0][k][i] = acc[1][k][i] = acc[2][k][i] = 0.0f;
    struct Row {
        Raw8<T> y[K], z[K], g[K];
        Raw8<R> r[K], d[K];
    } next;
    auto fetch = [&](int64_t t) {
        if (t >= (int64_t)a.tokens) t = blockIdx.x;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            uint32_t c = (k * blockDim.x + threadIdx.x) * V;
            if (c >= a.channels) c = 0u;  // dropped
            next.y[k].load(static_cast<const T *>(a.y) + t * a.y_stride + c);
            next.z[k].load(a.gate ? static_cast<const T *>(a.gate) + t * a.gate_stride + c : dout + t * C + c);
            next.r[k].load(static_cast<const R *>(a.residual) + t * a.residual_stride + c);
            next.g[k].load(dout + t * C + c);
            next.d[k].load(dres ? dres + t * C + c : static_cast<const R *>(a.residual) + t * a.residual_stride + c);
        }
    };
    if (WHOLE) fetch(blockIdx.x);
    for (int64_t t = blockIdx.x; t < (int64_t)a.tokens; t += gridDim.x) {
        float y[K][V], z[K][V], r[K][V], g[K][V], d[K][V], sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t c = (k * blockDim.x + threadIdx.x) * V, have = c < a.channels ? a.channels - c : 0u;
            float w[V];
            if (WHOLE) {
                next.y[k].values(y[k]);
                next.z[k].values(z[k]);
                next.r[k].values(r[k]);
                next.g[k].values(g[k]);
                next.d[k].values(d[k]);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (!have) y[k][i] = z[k][i] = r[k][i] = g[k][i] = 0.0f;
                    if (!have || !dres) d[k][i] = 0.0f;
                }
            } else {
                load_n<T, V>(y[k], at_row<T>(a.y, t, a.y_stride, c), have, 0.0f);
                load_n<T, V>(z[k], at_row<T>(a.gate, t, a.gate_stride, c), have, 0.0f);
                load_n<R, V>(r[k], at_row<R>(a.residual, t, a.residual_stride, c), have, 0.0f);
                load_n<T, V>(g[k], dout + t * C + c, have, 0.0f);
                load_n<R, V>(d[k], dres ? dres + t * C + c : nullptr, have, 0.0f);
            }
            load_n<float, V>(w, at_col(a.pre, c), have, 1.0f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sum[0] = __builtin_fmaf(y[k][i], y[k][i], sum[0]);
                sum[1] = __builtin_fmaf(r[k][i], r[k][i], sum[1]);
                sum[2] = __builtin_fmaf(w[i] * g[k][i], r[k][i], sum[2]);
            }
        }
        if (WHOLE) fetch(t + gridDim.x);
        group_totals<3>(sum, sh[0]);
        const float ry = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[0], a.inv, a.eps));
        const float rr = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[1], a.inv, a.eps));
        const float lean = rr * rr * (sum[2] * a.inv);
        float tilt[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t c = (k * blockDim.x + threadIdx.x) * V, have = c < a.channels ? a.channels - c : 0u;
            float w[V], s[V], po[V], dg[V];
            load_n<float, V>(w, at_col(a.pre, c), have, 1.0f);
            load_n<float, V>(s, at_col(a.scale, c), have, 1.0f);
            load_n<float, V>(po, at_col(a.post, c), have, 1.0f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float dr = __builtin_fmaf(rr, __builtin_fmaf(-r[k][i], lean, w[i] * g[k][i]), d[k][i]);
                acc[2][k][i] = __builtin_fmaf(g[k][i], r[k][i] * rr, acc[2][k][i]);
                const float sg = a.gate ? sigmoid(z[k][i]) : 1.0f, unit = y[k][i] * ry;
                const float along = dr * sg * unit;
                acc[0][k][i] = __builtin_fmaf(along, po[i], acc[0][k][i]);
                acc[1][k][i] = __builtin_fmaf(along, s[i], acc[1][k][i]);
                dg[i] = along * s[i] * po[i] * (1.0f - sg);
                const float u = s[i] * dr * sg * po[i];
                tilt[0] = __builtin_fmaf(u, y[k][i], tilt[0]);
                d[k][i] = dr;
                z[k][i] = u;
            }
            store_n<R, V>(dr_out + t * C + c, d[k], have);
            if (dgate) store_n<T, V>(dgate + t * C + c, dg, have);
        }
        group_totals<1>(tilt, sh[1]);
        const float turn = ry * ry * (tilt[0] * a.inv);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t c = (k * blockDim.x + threadIdx.x) * V, have = c < a.channels ? a.channels - c : 0u;
#pragma unroll
            for (int i = 0; i < V; ++i) y[k][i] = ry * __builtin_fmaf(-y[k][i], turn, z[k][i]);
            store_n<T, V>(dy + t * C + c, y[k], have);
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const uint32_t c = (k * blockDim.x + threadIdx.x) * V, have = c < a.channels ? a.channels - c : 0u;
#pragma unroll
        for (int w = 0; w < 3; ++w) store_n<float, V>(part + ((int64_t)blockIdx.x * 3 + w) * C + c, acc[w][k], have);
    }
}

__global__ __launch_bounds__(256) void norm_params_kernel(const float *__restrict__ part, uint32_t rows,
                                                          uint32_t channels, float *__restrict__ dscale,
                                                          float *__restrict__ dpost, float *__restrict__ dpre) {
    __shared__ float s[4][64];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t cols = 3u * channels, col = blockIdx.x * 64u + lane;
    float v = col < cols ? column_sum(part + col, wave, 4u, rows, cols) : 0.0f;
    s[wave][lane] = v;
    __syncthreads();
    if (wave == 0u && col < cols) {
        v = ((s[0][lane] + s[1][lane]) + s[2][lane]) + s[3][lane];
        const uint32_t which = col / channels, c = col % channels;
        float *to = which == 0u ? dscale : which == 1u ? dpost : dpre;
        if (to) to[c] = v;
    }
}

constexpr int kBwdWaves = 12;  // of the backward pass on a CU, 3 on each SIMD

// Workgroups that share the rows: as many as the GPU holds at once, up to 4
// on a CU.
uint32_t bwd_groups(const ps_norm_input *in) {
    const uint32_t most = kBwdWaves, waves = (uint32_t)ceil_div(in->channels, 64u * kVec);
    const uint32_t each = most / (waves < most ? waves : most);
    const uint32_t groups = 256u * (each < 4u ? each : 4u);
    return in->tokens < groups ? (uint32_t)in->tokens : groups;
}

ps_status norm_sizes(const ps_norm_input *in) {
    if (!in) return PS_ERR_NULL;
    if (!dtype_bytes(in->dtype) || (in->residual_dtype != in->dtype && in->residual_dtype != PS_F32))
        return PS_ERR_UNSUPPORTED;
    const int64_t c = in->channels;
    if (in->tokens > kBlockMaxTokens || c == 0 || c > PS_NORM_MAX_CHANNELS || in->y_stride < c ||
        (in->gate && (in->gate_stride < c || in->gate_stride > kBlockMaxStride)) || in->residual_stride < c ||
        in->y_stride > kBlockMaxStride || in->residual_stride > kBlockMaxStride)
        return PS_ERR_SIZE;
    return PS_OK;
}

ps_status norm_pointers(const ps_norm_input *in) {
    const size_t e = dtype_bytes(in->dtype);
    if (in->tokens && (!in->y || !in->residual)) return PS_ERR_NULL;
    if (!aligned(in->y, e) || !aligned(in->gate, e) || !aligned(in->residual, dtype_bytes(in->residual_dtype)) ||
        !aligned(in->scale, 4) || !aligned(in->post_weight, 4) || !aligned(in->pre_weight, 4))
        return PS_ERR_ALIGNMENT;
    return PS_OK;
}

// Bytes of a call's arrays; cells and res: packed rows of the two types.
struct NormBytes {
    size_t y, gate, residual, cells, res, weight;
    explicit NormBytes(const ps_norm_input *in) {
        const size_t e = dtype_bytes(in->dtype), re = dtype_bytes(in->residual_dtype), c = in->channels;
        y = rows_bytes(in->tokens, in->y_stride, c, e);
        gate = rows_bytes(in->tokens, in->gate_stride, c, e);
        residual = rows_bytes(in->tokens, in->residual_stride, c, re);
        cells = in->tokens * c * e;
        res = in->tokens * c * re;
        weight = c * 4u;
    }
};

NormArgs norm_args(const ps_norm_input *in) {
    NormArgs a{};
    a.y = in->y, a.gate = in->gate, a.residual = in->residual;
    a.y_stride = in->y_stride, a.gate_stride = in->gate_stride, a.residual_stride = in->residual_stride;
    a.scale = in->scale, a.post = in->post_weight, a.pre = in->pre_weight;
    a.tokens = (uint32_t)in->tokens, a.channels = in->channels;
    a.eps = in->eps;
    a.inv = 1.0f / (float)in->channels;
    return a;
}

// Calls f(vectors per thread as a constant, threads): one vector a thread up
// to 8192 channels, two above.
template <class F>
ps_status with_shape(uint32_t channels, F f) {
    const uint32_t wave = 64u * kVec;
    if (channels <= wave * kMostWaves)
        return f(std::integral_constant<int, 1>(), (uint32_t)ceil_div(channels, wave) * 64u);
    return f(std::integral_constant<int, 2>(), (uint32_t)ceil_div(channels, 2u * wave) * 64u);
}

// The same for the backward pass: f(most threads, vectors per thread,
// threads).  A row of one vector a thread and its sums take up to 168
// registers, of which a SIMD holds 3 waves: one vector up to kBwdWaves, then
// 512 threads with two (231 registers, no room for the next row), and 1024 with
// two above 8192 channels, whose 128 registers spill 400 bytes a lane in the
// row loop.  8192 rows, bf16 with an fp32 residual, us: 5632 channels 208 (two
// vectors 311), 6144 224 (310), 8192 348, 16384 1685.
template <class F>
ps_status with_bwd_shape(uint32_t channels, F f) {
    auto threads = [&](uint32_t k) { return (uint32_t)ceil_div(channels, k * 64u * kVec) * 64u; };
    typedef std::integral_constant<int, 1> One;
    typedef std::integral_constant<int, 2> Two;
    if (channels <= 256u * kVec) return f(std::integral_constant<int, 256>(), One(), threads(1));
    constexpr int kMost = 64 * kBwdWaves;
    if (channels <= (uint32_t)kMost * kVec) return f(std::integral_constant<int, kMost>(), One(), threads(1));
    if (channels <= 1024u * kVec) return f(std::integral_constant<int, 512>(), Two(), threads(2));
    return f(std::integral_constant<int, 1024>(), Two(), threads(2));
}

template <class F>
ps_status with_norm_types(const ps_norm_input *in, F f) {
    return with_type(in->dtype, [&](auto zero) {
        using T = decltype(zero);
        if (in->residual_dtype == PS_F32) return f(T(), float());
        return f(T(), T());
    });
}

}  // namespace
}  // namespace dwps

using namespace dwps;

extern "C" ps_status ps_block_norm(const ps_norm_input *in, void *residual_out, void *out, void *stream) {
    ps_status st = norm_sizes(in);
    if (st != PS_OK) return st;
    if ((st = norm_pointers(in)) != PS_OK) return st;
    if (!in->tokens) return PS_OK;
    const size_t e = dtype_bytes(in->dtype), re = dtype_bytes(in->residual_dtype);
    if (!residual_out || !out) return PS_ERR_NULL;
    if (!aligned(residual_out, re) || !aligned(out, e)) return PS_ERR_ALIGNMENT;
    const NormBytes n(in);
    if (outputs_overlap({{residual_out, n.res}, {out, n.cells}},
                        {{in->y, n.y}, {in->gate, n.gate}, {in->residual, n.residual}, {in->scale, n.weight},
                         {in->post_weight, n.weight}, {in->pre_weight, n.weight}}))
        return PS_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    NormArgs a = norm_args(in);
    return with_norm_types(in, [&](auto zt, auto zr) {
        using T = decltype(zt);
        using R = decltype(zr);
        return with_shape(in->channels, [&](auto k, uint32_t threads) {
            timing_begin(s);
            launch_in_parts(a.tokens, 1u, threads, [&](uint32_t first, uint32_t grid) {
                a.first = first;
                hipLaunchKernelGGL((norm_kernel<T, R, decltype(k)::value>), dim3(grid), dim3(threads), 0, s, a,
                                   static_cast<R *>(residual_out), static_cast<T *>(out));
            });
            timing_end(s);
            return launch_status();
        });
    });
}

extern "C" ps_status ps_block_norm_bwd(void *ws, size_t *ws_bytes, const ps_norm_input *in, const void *dout,
                                       const void *dresidual_out, const ps_norm_grads *grads, void *stream) {
    ps_status st = norm_sizes(in);
    if (st != PS_OK) return st;
    const uint32_t groups = bwd_groups(in);
    PlainWs plan;
    const size_t part_at = plan.take((size_t)groups * 3u * in->channels * 4u);
    bool query = false;
    st = workspace_protocol(ws, ws_bytes, plan.at, &query);
    if (st != PS_OK || query) return st;
    if ((st = norm_pointers(in)) != PS_OK) return st;
    const size_t e = dtype_bytes(in->dtype), re = dtype_bytes(in->residual_dtype);
    if (!grads || (in->tokens && (!dout || !grads->dy || !grads->dresidual))) return PS_ERR_NULL;
    if (!aligned(ws, 16) || !aligned(dout, e) || !aligned(dresidual_out, re) || !aligned(grads->dy, e) ||
        !aligned(grads->dgate, e) || !aligned(grads->dresidual, re) || !aligned(grads->dscale, 4) ||
        !aligned(grads->dpost_weight, 4) || !aligned(grads->dpre_weight, 4))
        return PS_ERR_ALIGNMENT;
    const NormBytes n(in);
    if (outputs_overlap({{grads->dy, n.cells}, {in->gate ? grads->dgate : nullptr, n.cells}, {grads->dresidual, n.res},
                         {grads->dscale, n.weight}, {grads->dpost_weight, n.weight}, {grads->dpre_weight, n.weight}},
                        {{in->y, n.y}, {in->gate, n.gate}, {in->residual, n.residual}, {in->scale, n.weight},
                         {in->post_weight, n.weight}, {in->pre_weight, n.weight}, {dout, n.cells}, {dresidual_out, n.res}}))
        return PS_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const NormArgs a = norm_args(in);
    return with_norm_types(in, [&](auto zt, auto zr) {
        using T = decltype(zt);
        using R = decltype(zr);
        return with_bwd_shape(in->channels, [&](auto most, auto k, uint32_t threads) {
            constexpr int K = decltype(k)::value;
            float *part = ws_at<float>(ws, part_at);
            timing_begin(s);
            auto launch = [&](auto whole) {
                hipLaunchKernelGGL((norm_bwd_kernel<T, R, decltype(most)::value, K, decltype(whole)::value>),
                                   dim3(groups), dim3(threads), 0, s, a,
                                   static_cast<const T *>(dout), static_cast<const R *>(dresidual_out),
                                   static_cast<T *>(grads->dy), in->gate ? static_cast<T *>(grads->dgate) : nullptr,
                                   static_cast<R *>(grads->dresidual), part, ws_counter(ws), plan.words());
            };
            // a second vector leaves no registers for the next row
            if (groups && K == 1 && in->channels % kVec == 0u) launch(std::integral_constant<bool, K == 1>());
            else if (groups) launch(std::false_type());
            if (grads->dscale || grads->dpost_weight || grads->dpre_weight)
                hipLaunchKernelGGL(norm_params_kernel, dim3((uint32_t)ceil_div(3u * in->channels, 64)), dim3(256), 0, s,
                                   part, groups, in->channels, grads->dscale, grads->dpost_weight, grads->dpre_weight);
            timing_end(s);
            return launch_status();
        });
    });
}
