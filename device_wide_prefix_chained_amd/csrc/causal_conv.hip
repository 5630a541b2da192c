// causal_conv.hip -- the short causal convolution of a state space block:
// forward, backward and the form for single tokens.
//
//   pre[t, d] = bias[d] + sum_k weight[d, k] x[t - (W - 1) + k, d]
//   out[t, d] = silu(pre[t, d])
//
// Bound by memory: 2 W + 5 operations for two activations moved.  A thread
// owns 16 bytes of neighbouring channels and walks down a piece of one
// sequence, the last W rows in registers and the next four on their way, so
// every row is read once but for the W - 1 rows before each piece.
// 16384 x 4096 in 13 sequences, bf16, W = 4: 53 us (5.0 TB/s), 55 to 61 us a
// call among others; pieces of 16 to 64 rows and 2 to 8 rows ahead are within 10%.
#include <hip/hip_runtime.h>

#include "block_device.hpp"

namespace dwps {
namespace {

struct ConvArgs {
    const void *x, *initial;
    const float *weight, *bias;
    const uint32_t *offsets;
    int64_t x_stride;
    uint32_t tokens, channels, num_seqs;
    uint32_t first;      // piece (rows' share, for single tokens) of the launch's first workgroup
    uint32_t shift;      // log2 of the rows of a piece
    uint32_t col_blocks; // workgroups side by side
};

constexpr int kConvThreads = 64;

// V neighbouring channels as they were loaded: 16-bit types stay packed until
// they are used, so that nothing waits for them before.
template <class T, int V>
struct RawRow {
    Pack<T, V> r;
    __device__ __forceinline__ void load(const T *p) { r = *reinterpret_cast<const Pack<T, V> *>(p); }
    __device__ __forceinline__ void values(float (&o)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = (float)r.v[i];
    }
};
template <class T>
struct RawRowPacked {
    typedef uint32_t words __attribute__((ext_vector_type(4)));
    typedef words words_at_2 __attribute__((aligned(2), may_alias));
    words w;
    __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const words_at_2 *>(p); }
    __device__ __forceinline__ void values(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t b = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
            o[i] = (float)__builtin_bit_cast(T, b);
        }
    }
};
template <>
struct RawRow<bf16_t, 8> : RawRowPacked<bf16_t> {};
template <>
struct RawRow<f16_t, 8> : RawRowPacked<f16_t> {};

template <class T, int V>
__device__ __forceinline__ void load_row(float (&v)[V], const T *p) {
    RawRow<T, V> r;
    r.load(p);
    r.values(v);
}
template <class T, int V>
__device__ __forceinline__ void store_row(T *p, const float (&v)[V]) {
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = (T)v[i];
    *reinterpret_cast<Pack<T, V> *>(p) = r;
}

// The thread's first channel.  The last thread of a row steps back to end
// with the row: it and its neighbour compute the same values of the channels
// they share (the first `shared` ones), and no thread has a part of a vector.
template <int V>
__device__ __forceinline__ bool own_channels(const ConvArgs &a, uint32_t block, uint32_t &c, uint32_t *shared = nullptr) {
    const uint32_t own = (block * kConvThreads + threadIdx.x) * V;
    if (own >= a.channels) return false;
    c = own + V > a.channels ? a.channels - V : own;
    if (shared) *shared = own - c;
    return true;
}
// The same, of the channels that the thread shares with no other.
template <class T, int V>
__device__ __forceinline__ void store_own(T *p, const float (&v)[V], uint32_t shared) {
    if (shared == 0u) {
        store_row<T, V>(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if ((uint32_t)i >= shared) p[i] = (T)v[i];
}

// Row r (any row from seq_lo - (W - 1) on) of the sequence: an input row, an
// initial row, or zeros.
template <class T, int V, int W>
__device__ __forceinline__ void past_row(float (&v)[V], const ConvArgs &a, const Piece &q, int64_t r, uint32_t c) {
    if (r >= (int64_t)q.seq_lo) {
        load_row<T, V>(v, static_cast<const T *>(a.x) + r * a.x_stride + c);
    } else if (a.initial) {
        const int64_t j = (int64_t)(W - 1) + r - (int64_t)q.seq_lo;
        load_row<T, V>(v, static_cast<const T *>(a.initial) + ((int64_t)q.seq * (W - 1) + j) * a.channels + c);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.0f;
    }
}

template <int V, int W>
__device__ __forceinline__ void load_weights(float (&w)[W][V], float (&b)[V], const ConvArgs &a, uint32_t c) {
    const Pack<float, V * W> all = *reinterpret_cast<const Pack<float, V * W> *>(a.weight + (int64_t)c * W);
    if (a.bias) {
        const Pack<float, V> r = *reinterpret_cast<const Pack<float, V> *>(a.bias + c);
#pragma unroll
        for (int i = 0; i < V; ++i) b[i] = r.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) b[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][i] = all.v[i * W + k];
}

constexpr int kRows = 4;  // rows loaded ahead

template <class T, int V, int W>
__global__ __launch_bounds__(kConvThreads) void conv_kernel(ConvArgs a, T *__restrict__ out, T *__restrict__ fin) {
    const Piece q = find_piece(a.offsets, a.num_seqs, a.tokens, a.shift, a.first + blockIdx.x / a.col_blocks);
    uint32_t c;
    if (!q.any || !own_channels<V>(a, blockIdx.x % a.col_blocks, c)) return;
    const int64_t C = a.channels;
    const T *x = static_cast<const T *>(a.x) + c;
    RawRow<T, V> next[kRows];
    auto fetch = [&](uint32_t t) {  // rows past the last repeat it
#pragma unroll
        for (int i = 0; i < kRows; ++i) next[i].load(x + (int64_t)(t + i < q.hi ? t + i : q.hi - 1u) * a.x_stride);
    };
    if (q.lo < q.hi) fetch(q.lo);
    float w[W][V], bias[V], win[W][V];  // win[k]: the row W - 1 - k before the present one
    load_weights<V, W>(w, bias, a, c);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) past_row<T, V, W>(win[k + 1], a, q, (int64_t)q.lo - (W - 1) + k, c);
    auto step = [&](const RawRow<T, V> &r, uint32_t t) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) win[k][i] = win[k + 1][i];
        r.values(win[W - 1]);
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float pre = bias[i];
#pragma unroll
            for (int k = 0; k < W; ++k) pre = __builtin_fmaf(w[k][i], win[k][i], pre);
            o[i] = silu(pre);
        }
        store_row<T, V>(out + (int64_t)t * C + c, o);
    };
    uint32_t t = q.lo;
    for (; t + kRows <= q.hi; t += kRows) {
        RawRow<T, V> now[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) now[i] = next[i];
        fetch(t + kRows);
#pragma unroll
        for (int i = 0; i < kRows; ++i) step(now[i], t + i);
    }
#pragma unroll
    for (int i = 0; i < kRows - 1; ++i)
        if (t + i < q.hi) step(next[i], t + i);
    if (fin && q.hi == q.seq_hi) {
#pragma unroll
        for (int k = 1; k < W; ++k) store_row<T, V>(fin + ((int64_t)q.seq * (W - 1) + k - 1) * C + c, win[k]);
    }
}

// Backward.  With g[t] = dout[t] silu'(pre[t]):
//   dx[t] = sum_k weight[k] g[t + W - 1 - k]   (rows past the sequence: 0)
//   dweight[k] = sum_t g[t] x[t - (W - 1) + k],  dbias = sum_t g[t]
// and the rows before the sequence's first (dinitial) as dx.  A piece walks
// W - 1 rows past its end for the g its last rows need, and sums dweight and
// dbias over its own rows into part[piece][k][channel] (k = W: dbias).
// 6001 x 1537, fp32, W = 3: 28 us and 4 us for the sums over pieces.
template <class T, int V, int W>
__global__ __launch_bounds__(kConvThreads) void conv_bwd_kernel(ConvArgs a, const T *__restrict__ dout,
                                                                T *__restrict__ dx, T *__restrict__ dinit,
                                                                float *__restrict__ part, uint32_t *hdr,
                                                                uint32_t words) {
    if (blockIdx.x == 0 && threadIdx.x == 0) mark_plain(hdr, words);
    const uint32_t p = a.first + blockIdx.x / a.col_blocks;
    const Piece q = find_piece(a.offsets, a.num_seqs, a.tokens, a.shift, p);
    uint32_t c;
    if (!own_channels<V>(a, blockIdx.x % a.col_blocks, c)) return;
    const int64_t C = a.channels;
    const T *x = static_cast<const T *>(a.x) + c, *gy = dout + c;
    float w[W][V], bias[V], win[W][V], gw[W][V], sum[W + 1][V];
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) sum[k][i] = 0.0f;
    if (q.any) {
        struct Rows {
            RawRow<T, V> x[kRows], g[kRows];
        } next;
        auto fetch = [&](uint32_t t) {  // rows past the sequence's last repeat it
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int64_t r = t + i < q.seq_hi ? t + i : q.seq_hi - 1u;
                next.x[i].load(x + r * a.x_stride);
                next.g[i].load(gy + r * C);
            }
        };
        if (q.lo < q.seq_hi) fetch(q.lo);
        load_weights<V, W>(w, bias, a, c);
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) gw[k][i] = 0.0f;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) past_row<T, V, W>(win[k + 1], a, q, (int64_t)q.lo - (W - 1) + k, c);
        auto step = [&](const RawRow<T, V> &rx, const RawRow<T, V> &rg, uint32_t t) {
            // the row's own g, 0 past the sequence
            float g[V];
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    win[k][i] = win[k + 1][i];
                    gw[k][i] = gw[k + 1][i];
                }
            rx.values(win[W - 1]);
            rg.values(g);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float pre = bias[i];
#pragma unroll
                for (int k = 0; k < W; ++k) pre = __builtin_fmaf(w[k][i], win[k][i], pre);
                gw[W - 1][i] = t < q.seq_hi ? g[i] * dsilu(pre, sigmoid(pre)) : 0.0f;
            }
            if (t < q.hi) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
#pragma unroll
                    for (int k = 0; k < W; ++k) sum[k][i] = __builtin_fmaf(gw[W - 1][i], win[k][i], sum[k][i]);
                    sum[W][i] += gw[W - 1][i];
                }
            }
            // the row that now has all its g: gw[j] is g of row r + j
            const int64_t r = (int64_t)t - (W - 1);
            if (r >= (int64_t)q.lo || (dinit && q.lo == q.seq_lo)) {
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    o[i] = 0.0f;
#pragma unroll
                    for (int k = 0; k < W; ++k) o[i] = __builtin_fmaf(w[k][i], gw[W - 1 - k][i], o[i]);
                }
                T *to = r >= (int64_t)q.lo ? dx + r * C
                                           : dinit + ((int64_t)q.seq * (W - 1) + (r - (int64_t)q.lo + (W - 1))) * C;
                store_row<T, V>(to + c, o);
            }
        };
        const uint32_t end = q.hi + (W - 1);
        if (q.lo < q.seq_hi) {
            uint32_t t = q.lo;
            for (; t + kRows <= end; t += kRows) {
                const Rows now = next;
                fetch(t + kRows);
#pragma unroll
                for (int i = 0; i < kRows; ++i) step(now.x[i], now.g[i], t + i);
            }
#pragma unroll
            for (int i = 0; i < kRows - 1; ++i)
                if (t + i < end) step(next.x[i], next.g[i], t + i);
        } else if (dinit) {  // an empty sequence gives its initial rows nothing
            const float none[V] = {};
            for (int k = 0; k < W - 1; ++k) store_row<T, V>(dinit + ((int64_t)q.seq * (W - 1) + k) * C + c, none);
        }
    }
#pragma unroll
    for (int k = 0; k <= W; ++k) store_row<float, V>(part + ((int64_t)p * (W + 1) + k) * C + c, sum[k]);
}

// Sums part over the pieces: columns are the (k, channel) pairs.  Each of
// four waves sums every fourth piece of 64 columns, then the four are added
// in order.
__global__ __launch_bounds__(256) void conv_params_kernel(const float *__restrict__ part, uint32_t pieces, uint32_t width,
                                                          uint32_t channels, float *__restrict__ dweight,
                                                          float *__restrict__ dbias) {
    __shared__ float s[4][64];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint64_t cols = (uint64_t)(width + 1u) * channels, col = (uint64_t)blockIdx.x * 64u + lane;
    float v = col < cols ? column_sum(part + col, wave, 4u, pieces, cols) : 0.0f;
    s[wave][lane] = v;
    __syncthreads();
    if (wave == 0u && col < cols) {
        v = ((s[0][lane] + s[1][lane]) + s[2][lane]) + s[3][lane];
        const uint32_t k = (uint32_t)(col / channels), c = (uint32_t)(col % channels);
        if (k < width) dweight[(uint64_t)c * width + k] = v;
        else if (dbias) dbias[c] = v;
    }
}

// One token for each row: W - 1 rows of state in, W - 1 out.  A workgroup
// takes `each` rows, so that the weights, which are as large as the states of
// a row in fp32, are read once for them.  The state may be updated in place,
// so every channel has one thread that stores it, and what a thread reads of
// the others' does not matter.  384 rows x 8192, bf16, W = 4: 15 us (3.4 TB/s),
// 11 us (4.5 TB/s) with a part of it in the cache.
template <class T, int V, int W>
__global__ __launch_bounds__(kConvThreads) void conv_step_kernel(ConvArgs a, const T *state, T *new_state,
                                                                 const int32_t *__restrict__ slots, uint32_t pool,
                                                                 T *__restrict__ out, uint32_t each) {
    uint32_t c, shared;
    if (!own_channels<V>(a, blockIdx.x % a.col_blocks, c, &shared)) return;
    const int64_t C = a.channels;
    const uint32_t i0 = (a.first + blockIdx.x / a.col_blocks) * each, i1 = i0 + each < a.tokens ? i0 + each : a.tokens;
    struct Rows {
        RawRow<T, V> x, s[W];
        int64_t slot;
    };
    auto fetch = [&](Rows &r, uint32_t i) {
        if (i >= i1) i = i1 - 1u;
        const int64_t slot = slots ? (int64_t)slots[i] : (int64_t)i;
        r.slot = slot >= 0 && slot < (int64_t)pool ? slot : -1;
        r.x.load(static_cast<const T *>(a.x) + (int64_t)i * a.x_stride + c);
        if (W > 1 && pool) {  // padding reads a slot that exists and drops it
            const int64_t from = r.slot < 0 ? 0 : r.slot;
#pragma unroll
            for (int k = 0; k < W - 1; ++k) r.s[k].load(state + (from * (W - 1) + k) * C + c);
        }
    };
    Rows next;
    fetch(next, i0);
    float w[W][V], bias[V];
    load_weights<V, W>(w, bias, a, c);
    for (uint32_t i = i0; i < i1; ++i) {
        const Rows now = next;
        fetch(next, i + 1u);
        float win[W][V], o[V];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            now.s[k].values(win[k]);
#pragma unroll
            for (int j = 0; j < V; ++j) win[k][j] = now.slot < 0 ? 0.0f : win[k][j];
        }
        now.x.values(win[W - 1]);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float pre = bias[j];
#pragma unroll
            for (int k = 0; k < W; ++k) pre = __builtin_fmaf(w[k][j], win[k][j], pre);
            o[j] = silu(pre);
        }
        store_own<T, V>(out + (int64_t)i * C + c, o, shared);
        if (now.slot >= 0) {
#pragma unroll
            for (int k = 1; k < W; ++k) store_own<T, V>(new_state + (now.slot * (W - 1) + k - 1) * C + c, win[k], shared);
        }
    }
}

// Calls f with the width as a constant.
template <class F>
ps_status with_width(uint32_t width, F f) {
    switch (width) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    case 8: return f(std::integral_constant<int, 8>());
    default: return PS_ERR_SIZE;
    }
}

// Calls f with a value of the activations' type, the width and the channels
// of a thread (16 bytes, or one where a row is shorter) as constants.
template <class T>
constexpr int kVec = 16 / (int)sizeof(T);
uint32_t vec_of(const ps_conv_input *in) {
    const uint32_t v = 16u / (uint32_t)dtype_bytes(in->dtype);
    return in->channels < v ? 1u : v;
}
template <class F>
ps_status with_conv(const ps_conv_input *in, F f) {
    return with_type(in->dtype, [&](auto zero) {
        using T = decltype(zero);
        return with_width(in->width, [&](auto w) {
            if (vec_of(in) == 1u) return f(zero, w, std::integral_constant<int, 1>());
            return f(zero, w, std::integral_constant<int, kVec<T>>());
        });
    });
}

// Sizes and types alone.
ps_status conv_sizes(const ps_conv_input *in, bool packed) {
    if (!in) return PS_ERR_NULL;
    if (!dtype_bytes(in->dtype)) return PS_ERR_UNSUPPORTED;
    if (in->tokens > kBlockMaxTokens || in->channels == 0u || in->channels > kBlockMaxChannels || in->width == 0u ||
        in->width > PS_CONV_MAX_WIDTH || in->num_seqs > kBlockMaxSeqs || in->x_stride < (int64_t)in->channels ||
        in->x_stride > kBlockMaxStride)
        return PS_ERR_SIZE;
    if (packed && !in->offsets && in->num_seqs > 1u) return PS_ERR_SIZE;
    return PS_OK;
}

ps_status conv_pointers(const ps_conv_input *in) {
    const size_t e = dtype_bytes(in->dtype);
    if (!in->weight || (in->tokens && !in->x)) return PS_ERR_NULL;
    if (!aligned(in->x, e) || !aligned(in->weight, 4) || !aligned(in->bias, 4) || !aligned(in->offsets, 4) ||
        !aligned(in->initial, e))
        return PS_ERR_ALIGNMENT;
    return PS_OK;
}

ConvArgs conv_args(const ps_conv_input *in, uint32_t shift) {
    const uint32_t vec = vec_of(in);
    ConvArgs a{};
    a.x = in->x;
    a.initial = in->width > 1u ? in->initial : nullptr;
    a.weight = in->weight;
    a.bias = in->bias;
    a.offsets = in->offsets;
    a.x_stride = in->x_stride;
    a.tokens = (uint32_t)in->tokens;
    a.channels = in->channels;
    a.num_seqs = in->offsets ? in->num_seqs : 1u;
    a.shift = shift;
    a.col_blocks = (uint32_t)ceil_div(in->channels, (uint64_t)vec * kConvThreads);
    return a;
}

// Rows of a piece, as a power of two.  Forward: as many (8 to 64) as leave
// 4096 waves, 4 on each SIMD.  Backward: 32, more where there would be above
// 512 cells.  A piece leaves width + 1 rows of partial sums, and each sequence
// beyond the cells adds a piece, so many short sequences cost that much more.
uint32_t conv_shift(const ps_conv_input *in) {
    const uint64_t cols = ceil_div(in->channels, (uint64_t)vec_of(in) * kConvThreads);
    uint32_t shift = 3u;
    while (shift < 6u && (in->tokens >> (shift + 1u)) * cols >= 4096u) ++shift;
    return shift;
}
uint32_t conv_bwd_shift(const ps_conv_input *in) {
    uint32_t shift = 5u;
    while ((in->tokens >> shift) > 512u) ++shift;
    return shift;
}

// Bytes of a call's arrays; edge: initial, final and dinitial.
struct ConvBytes {
    size_t x, out, weight, bias, offsets, edge;
    explicit ConvBytes(const ps_conv_input *in) {
        const size_t e = dtype_bytes(in->dtype), c = in->channels;
        x = rows_bytes(in->tokens, in->x_stride, c, e);
        out = in->tokens * c * e;
        weight = c * in->width * 4u;
        bias = c * 4u;
        offsets = ((size_t)in->num_seqs + 1u) * 4u;
        edge = (in->offsets ? in->num_seqs : 1u) * (in->width - 1u) * c * e;
    }
};

}  // namespace
}  // namespace dwps

using namespace dwps;

extern "C" ps_status ps_causal_conv(const ps_conv_input *in, void *out, void *final, void *stream) {
    ps_status st = conv_sizes(in, true);
    if (st != PS_OK) return st;
    if ((st = conv_pointers(in)) != PS_OK) return st;
    const size_t e = dtype_bytes(in->dtype);
    if (in->tokens && !out) return PS_ERR_NULL;
    if (!aligned(out, e) || !aligned(final, e)) return PS_ERR_ALIGNMENT;
    const ConvBytes n(in);
    if (outputs_overlap({{out, n.out}, {final, n.edge}},
                        {{in->x, n.x}, {in->weight, n.weight}, {in->bias, n.bias}, {in->offsets, n.offsets}, {in->initial, n.edge}}))
        return PS_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    ConvArgs a = conv_args(in, conv_shift(in));
    const uint64_t pieces = piece_count(in->tokens, a.num_seqs, in->offsets != nullptr, a.shift);
    if (!pieces) return PS_OK;
    return with_conv(in, [&](auto zero, auto w, auto v) {
        using T = decltype(zero);
        constexpr int W = decltype(w)::value, V = decltype(v)::value;
        timing_begin(s);
        launch_in_parts(pieces, a.col_blocks, kConvThreads, [&](uint32_t first, uint32_t grid) {
            a.first = first;
            hipLaunchKernelGGL((conv_kernel<T, V, W>), dim3(grid), dim3(kConvThreads), 0, s, a, static_cast<T *>(out),
                               W > 1 ? static_cast<T *>(final) : nullptr);
        });
        timing_end(s);
        return launch_status();
    });
}

extern "C" ps_status ps_causal_conv_bwd(void *ws, size_t *ws_bytes, const ps_conv_input *in, const void *dout, void *dx,
                                        float *dweight, float *dbias, void *dinitial, void *stream) {
    ps_status st = conv_sizes(in, true);
    if (st != PS_OK) return st;
    const size_t e = dtype_bytes(in->dtype);
    ConvArgs a = conv_args(in, conv_bwd_shift(in));
    const uint64_t pieces = piece_count(in->tokens, a.num_seqs, in->offsets != nullptr, a.shift);
    PlainWs plan;
    const size_t part_at = plan.take(pieces * (in->width + 1u) * in->channels * 4u);
    bool query = false;
    st = workspace_protocol(ws, ws_bytes, plan.at, &query);
    if (st != PS_OK || query) return st;
    if ((st = conv_pointers(in)) != PS_OK) return st;
    if (!dweight || (in->tokens && (!dout || !dx))) return PS_ERR_NULL;
    if (!aligned(ws, 16) || !aligned(dout, e) || !aligned(dx, e) || !aligned(dweight, 4) || !aligned(dbias, 4) ||
        !aligned(dinitial, e))
        return PS_ERR_ALIGNMENT;
    const ConvBytes n(in);
    if (outputs_overlap({{dx, n.out}, {dweight, n.weight}, {dbias, n.bias}, {dinitial, n.edge}},
                        {{in->x, n.x}, {in->weight, n.weight}, {in->bias, n.bias}, {in->offsets, n.offsets},
                         {in->initial, n.edge}, {dout, n.out}}))
        return PS_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return with_conv(in, [&](auto zero, auto w, auto v) {
        using T = decltype(zero);
        constexpr int W = decltype(w)::value, V = decltype(v)::value;
        float *part = ws_at<float>(ws, part_at);
        timing_begin(s);
        launch_in_parts(pieces, a.col_blocks, kConvThreads, [&](uint32_t first, uint32_t grid) {
            a.first = first;
            hipLaunchKernelGGL((conv_bwd_kernel<T, V, W>), dim3(grid), dim3(kConvThreads), 0, s, a,
                               static_cast<const T *>(dout), static_cast<T *>(dx),
                               W > 1 ? static_cast<T *>(dinitial) : nullptr, part, ws_counter(ws), plan.words());
        });
        hipLaunchKernelGGL(conv_params_kernel, dim3((uint32_t)ceil_div((uint64_t)(in->width + 1u) * in->channels, 64)),
                           dim3(256), 0, s, part, (uint32_t)pieces, in->width, in->channels, dweight, dbias);
        timing_end(s);
        return launch_status();
    });
}

extern "C" ps_status ps_causal_conv_step(const ps_conv_input *in, const void *state, void *new_state,
                                         const int32_t *slots, uint32_t pool, void *out, void *stream) {
    ps_status st = conv_sizes(in, false);
    if (st != PS_OK) return st;
    if ((st = conv_pointers(in)) != PS_OK) return st;
    const size_t e = dtype_bytes(in->dtype);
    if (in->tokens && (!out || (in->width > 1u && pool && (!state || !new_state)))) return PS_ERR_NULL;
    if (!aligned(out, e) || !aligned(state, e) || !aligned(new_state, e) || !aligned(slots, 4)) return PS_ERR_ALIGNMENT;
    if (!slots && in->tokens > pool) return PS_ERR_SIZE;
    const ConvBytes n(in);
    const size_t state_bytes = (size_t)pool * (in->width - 1u) * in->channels * e;
    if (outputs_overlap({{out, n.out}, {new_state, state_bytes}},
                        {{in->x, n.x}, {in->weight, n.weight}, {in->bias, n.bias}, {slots, in->tokens * 4u},
                         {state != new_state ? state : nullptr, state_bytes}}))
        return PS_ERR_ALIAS;
    if (!in->tokens) return PS_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    ConvArgs a = conv_args(in, 0u);
    // up to 4 rows a workgroup, while 2 waves are left for each SIMD
    const uint64_t share = in->tokens * a.col_blocks / 2048u;
    const uint32_t each = share < 1u ? 1u : share > 4u ? 4u : (uint32_t)share;
    return with_conv(in, [&](auto zero, auto w, auto v) {
        using T = decltype(zero);
        constexpr int W = decltype(w)::value, V = decltype(v)::value;
        timing_begin(s);
        launch_in_parts(ceil_div(in->tokens, each), a.col_blocks, kConvThreads, [&](uint32_t first, uint32_t grid) {
            a.first = first;
            hipLaunchKernelGGL((conv_step_kernel<T, V, W>), dim3(grid), dim3(kConvThreads), 0, s, a,
                               static_cast<const T *>(state), static_cast<T *>(new_state), slots, pool,
                               static_cast<T *>(out), each);
        });
        timing_end(s);
        return launch_status();
    });
}
