// gated_delta.hip -- the gated delta rule over packed sequences, and for
// single tokens.
//
//   S' = exp(g) S,  u = beta (v - S'^T k),  S = S' + k u^T,  out = scale S^T q
//
// Prompts run in two launches: every chunk of 64 rows is prepared by itself
// (delta_block.hpp), then a workgroup walks over a sequence's chunks with 64 or
// 128 columns of a head's state in its registers.
#include <hip/hip_runtime.h>

#include "delta_block.hpp"

namespace dwps {

ps_status delta_sizes(const ps_delta_input *in) {
    if (!in) return PS_ERR_NULL;
    if (!dtype_bytes(in->dtype)) return PS_ERR_UNSUPPORTED;
    const int64_t kd = in->key_dim, vd = in->value_dim, kh = in->kheads, h = in->heads;
    if (in->tokens > kBlockMaxTokens || in->num_seqs > kBlockMaxSeqs || (!in->offsets && in->num_seqs > 1u) || kd == 0 ||
        kd > PS_DELTA_MAX_DIM || vd == 0 || vd > PS_DELTA_MAX_DIM || kh == 0 || h == 0 || h > PS_DELTA_MAX_HEADS ||
        h % kh != 0)
        return PS_ERR_SIZE;
    auto bad = [](int64_t stride, int64_t row) { return stride < row || stride > kBlockMaxStride; };
    if (bad(in->q_stride, kh * kd) || bad(in->k_stride, kh * kd) || bad(in->v_stride, h * vd) || bad(in->g_stride, h) ||
        bad(in->beta_stride, h))
        return PS_ERR_SIZE;
    return PS_OK;
}

ps_status delta_pointers(const ps_delta_input *in) {
    const size_t e = dtype_bytes(in->dtype);
    if (in->tokens && (!in->q || !in->k || !in->v || !in->g || !in->beta)) return PS_ERR_NULL;
    if (!aligned(in->q, e) || !aligned(in->k, e) || !aligned(in->v, e) || !aligned(in->g, 4) || !aligned(in->beta, 4) ||
        !aligned(in->offsets, 4) || !aligned(in->initial, 4))
        return PS_ERR_ALIGNMENT;
    return PS_OK;
}

DeltaArgs delta_args(const ps_delta_input *in) {
    DeltaArgs a{};
    a.q = in->q, a.k = in->k, a.v = in->v;
    a.q_stride = in->q_stride, a.k_stride = in->k_stride, a.v_stride = in->v_stride;
    a.g = in->g, a.beta = in->beta;
    a.g_stride = in->g_stride, a.beta_stride = in->beta_stride;
    a.offsets = in->offsets;
    a.initial = in->initial;
    a.tokens = (uint32_t)in->tokens;
    a.kheads = in->kheads, a.heads = in->heads, a.key_dim = in->key_dim, a.value_dim = in->value_dim;
    a.num_seqs = in->offsets ? in->num_seqs : 1u;
    a.slots = (uint32_t)chunk_slots(in->tokens, a.num_seqs, kChunkShift);
    a.unit = in->normalize ? 1u : 0u;
    a.scale = in->scale, a.eps = in->eps;
    return a;
}

namespace {

// What a step of a walk reads: a chunk's keys, queries and values, and what was
// prepared of it.
template <class T, int W, int CT>
struct WalkTile {
    static constexpr uint32_t kCols = 64u * CT;
    RowTile<T, W> k, q;
    Prepared<T> p;
    T v[kChunk][kCols + 8u];
};
template <class T, int W, int CT>
constexpr bool kValuesFit = sizeof(WalkTile<T, W, CT>) <= kMostShared;
template <class T, int W, int CT>
constexpr size_t walk_tile_bytes() {
    return kValuesFit<T, W, CT> ? sizeof(WalkTile<T, W, CT>) : sizeof(WalkTile<T, W, CT>) - sizeof(WalkTile<T, W, CT>::v);
}

// Four waves walk over a sequence's chunks, each with 16 CT columns of a
// head's state; four feed them, loading a chunk while the one before is worked
// on and leaving it in the tile of the two that is not in use (or, where shared
// memory has room for one, after a barrier in that one).
template <class T, int W, int CT, bool E>
__global__ __launch_bounds__(512) void delta_walk_kernel(DeltaArgs a, uint32_t first, const Prepared<T> *__restrict__ prepared,
                                                         T *__restrict__ out, float *__restrict__ final,
                                                         float *__restrict__ states, float *__restrict__ rhos) {
    typedef typename Form<T>::Mid Mid;
    typedef WalkTile<T, W, CT> Tile;
    constexpr uint32_t kTiles = W / 16, kCols = Tile::kCols;
    constexpr bool kTwo = 2u * sizeof(Tile) <= kMostShared, kV = kValuesFit<T, W, CT>;
    __shared__ __attribute__((aligned(16))) char memory[kTwo ? 2u * sizeof(Tile) : walk_tile_bytes<T, W, CT>()];
    const uint32_t blocks = (a.value_dim + kCols - 1u) / kCols, b = first + blockIdx.x;
    const uint32_t head = b / blocks % a.heads, seq = b / blocks / a.heads, khead = head / (a.heads / a.kheads);
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u, m = lane & 15u, q = lane >> 4;
    const uint32_t block0 = (b % blocks) * kCols;
    const Rows r = sequence_rows(a.offsets, a.tokens, seq, kChunkShift);
    const uint32_t chunks = (r.hi - r.lo + kChunk - 1u) / kChunk;
    const T *values = static_cast<const T *>(a.v) + (uint64_t)head * a.value_dim;
    auto tile = [&](uint32_t i) { return reinterpret_cast<Tile *>(memory + (kTwo && (i & 1u) ? sizeof(Tile) : 0u)); };
    if (wave >= 4u) {
        // the feeding waves
        constexpr uint32_t kKeys = (W + 31) / 32, kVals = kCols / 32u;
        constexpr uint32_t kWords = (sizeof(Prepared<T>) + 4095u) / 4096u;
        const uint32_t thread = threadIdx.x - 256u, row = thread >> 2, part = (thread & 3u) * 8u;
        Pack<T, 8> ks[kKeys], qs[kKeys], vs[kVals];
        u32x4 ps[kWords];
        auto fetch = [&](uint32_t i) {
            const int64_t lo = r.lo + i * kChunk;
            const bool is = lo + row < r.hi;
            const T *k0 = static_cast<const T *>(a.k) + lo * a.k_stride + (uint64_t)khead * a.key_dim;
            const T *q0 = static_cast<const T *>(a.q) + lo * a.q_stride + (uint64_t)khead * a.key_dim;
#pragma unroll
            for (uint32_t c = 0; c < kKeys; ++c) {
                ks[c] = raw8<E, T>(k0 + row * a.k_stride, k0, is, part + 32u * c, a.key_dim);
                qs[c] = raw8<E, T>(q0 + row * a.q_stride, q0, is, part + 32u * c, a.key_dim);
            }
            if constexpr (kV) {
                const T *v0 = values + lo * a.v_stride;
#pragma unroll
                for (uint32_t c = 0; c < kVals; ++c)
                    vs[c] = raw8<E, T>(v0 + row * a.v_stride, v0, is, block0 + part + 32u * c, a.value_dim);
            }
            const u32x4 *p = reinterpret_cast<const u32x4 *>(&prepared[(uint64_t)(r.base + i) * a.heads + head]);
#pragma unroll
            for (uint32_t c = 0; c < kWords; ++c) {
                const uint32_t at = thread + 256u * c;
                if (at < sizeof(Prepared<T>) / 16u) ps[c] = p[at];
            }
        };
        auto leave = [&](uint32_t i) {
            Tile *to = tile(i);
#pragma unroll
            for (uint32_t c = 0; c < kKeys; ++c) {
                float v[8];
                values_of<T>(v, ks[c]);
                to->k.put(row, part + 32u * c, v);
                values_of<T>(v, qs[c]);
                to->q.put(row, part + 32u * c, v);
            }
            if constexpr (kV) {
#pragma unroll
                for (uint32_t c = 0; c < kVals; ++c) *reinterpret_cast<Pack<T, 8> *>(&to->v[row][part + 32u * c]) = vs[c];
            }
#pragma unroll
            for (uint32_t c = 0; c < kWords; ++c) {
                const uint32_t at = thread + 256u * c;
                if (at < sizeof(Prepared<T>) / 16u) reinterpret_cast<u32x4 *>(&to->p)[at] = ps[c];
            }
        };
        if (chunks) fetch(0u), leave(0u);
        __syncthreads();
        for (uint32_t i = 0; i < chunks; ++i) {
            const bool more = i + 1u < chunks;
            if (more) fetch(i + 1u);
            if (!kTwo) __syncthreads();
            if (more) leave(i + 1u);
            __syncthreads();
        }
        return;
    }
    const uint32_t col0 = block0 + wave * 16u * CT, here = wave * 16u * CT;
    const uint64_t cells = (uint64_t)a.key_dim * a.value_dim;
    f32x4 S[CT][kTiles];
    load_states<E>(S, a.initial ? a.initial + ((uint64_t)seq * a.heads + head) * cells : nullptr, a, col0, lane);
    __syncthreads();
    for (uint32_t c = 0; c < chunks; ++c) {
        const uint32_t lo = r.lo + c * kChunk, rows = r.hi - lo < kChunk ? r.hi - lo : kChunk;
        const Tile &in = *tile(c);
        if (col0 < a.value_dim) {
            if (states) store_states<E>(states + ((uint64_t)(r.base + c) * a.heads + head) * cells, S, a, col0, lane);
            f32x4 x[CT][4], o[CT][4], y[CT][4];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int t = 0; t < 4; ++t) x[ct][t] = o[ct][t] = y[ct][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            // K S, and (Q S)^T: the operands' sides are the other way round, which
            // leaves a row of out in a lane and neighbouring columns in its registers
#pragma unroll
            for (uint32_t s = 0; s < kTiles / 2u; ++s) {
                Mid h[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) h[ct] = operand_of<Mid>(S[ct][2u * s], S[ct][2u * s + 1u]);
#pragma unroll
                for (uint32_t t = 0; t < 4u; ++t) {
                    const auto ka = in.k.along(16u * t + m, 32u * s + 8u * q), qa = in.q.along(16u * t + m, 32u * s + 8u * q);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        mma(x[ct][t], ka, h[ct]);
                        mma(o[ct][t], h[ct], qa);
                    }
                }
            }
            auto numbers = [&](uint32_t which, uint32_t t) {
                return *reinterpret_cast<const f32x4 *>(&in.p.row[which + 16u * t + 4u * q]);
            };
            __builtin_amdgcn_sched_barrier(0);
            // R = V - e K S
#pragma unroll
            for (uint32_t t = 0; t < 4u; ++t) {
                const f32x4 e = numbers(kRowE, t);
#pragma unroll
                for (uint32_t ct = 0; ct < (uint32_t)CT; ++ct) {
                    f32x4 v;
                    if constexpr (kV && sizeof(T) == 2) {
                        const uint32_t at = here + (CT == 1 ? 4u * (m & 3u) : 8u * (m & 3u) + 4u * ct);
                        const i16x4 raw = read_transposed(
                            reinterpret_cast<const uint16_t *>(&in.v[16u * t + 4u * q + (m >> 2)][at]));
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = (float)__builtin_bit_cast(T, (uint16_t)raw[i]);
                    } else if constexpr (kV) {
#pragma unroll
                        for (uint32_t i = 0; i < 4u; ++i) v[i] = (float)in.v[16u * t + 4u * q + i][here + column<CT>(ct, m)];
                    } else {
                        const uint32_t col = col0 + column<CT>(ct, m);
#pragma unroll
                        for (uint32_t i = 0; i < 4u; ++i) {
                            const uint32_t row = 16u * t + 4u * q + i;
                            v[i] = row < rows && col < a.value_dim ? (float)values[(int64_t)(lo + row) * a.v_stride + col] : 0.0f;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[ct][t][i] = __builtin_fmaf(-e[i], x[ct][t][i], v[i]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            // rho
#pragma unroll
            for (uint32_t s = 0; s < 2u; ++s) {
                Mid h[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) h[ct] = operand_of<Mid>(x[ct][2u * s], x[ct][2u * s + 1u]);
#pragma unroll
                for (uint32_t t = 2u * s; t < 4u; ++t) {
                    const Mid inverse = in.p.inverse[lower_at(t, s)][lane];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) mma(y[ct][t], inverse, h[ct]);
                }
            }
            if (rhos)
                store_rows<E>(rhos + ((uint64_t)lo * a.heads + head) * a.value_dim, (uint64_t)a.heads * a.value_dim, y, rows,
                              col0, a.value_dim, lane);
            __builtin_amdgcn_sched_barrier(0);
            // out^T = scale e (Q S)^T + U^T P^T
#pragma unroll
            for (uint32_t t = 0; t < 4u; ++t) {
                const f32x4 beta = numbers(kRowBeta, t);
                const float e = in.p.row[kRowQ + 16u * t + m];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) y[ct][t] *= beta, o[ct][t] *= e;
            }
#pragma unroll
            for (uint32_t s = 0; s < 2u; ++s) {
                Mid h[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) h[ct] = operand_of<Mid>(y[ct][2u * s], y[ct][2u * s + 1u]);
#pragma unroll
                for (uint32_t t = 2u * s; t < 4u; ++t) {
                    const Mid scores = in.p.scores[lower_at(t, s)][lane];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) mma(o[ct][t], h[ct], scores);
                }
            }
#pragma unroll
            for (uint32_t t = 0; t < 4u; ++t) {
                const uint32_t row = 16u * t + m, col = col0 + 4u * CT * q;
                if (row < rows && col < a.value_dim) {
                    T *to = out + ((uint64_t)(lo + row) * a.heads + head) * a.value_dim + col;
                    Pack<T, 4 * CT> w;
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int i = 0; i < 4; ++i) w.v[4 * ct + i] = (T)o[ct][t][i];
                    if (E || col + 4u * CT <= a.value_dim) {
                        *reinterpret_cast<Pack<T, 4 * CT> *>(to) = w;
                    } else {
#pragma unroll
                        for (uint32_t i = 0; i < 4u * CT; ++i)
                            if (col + i < a.value_dim) to[i] = w.v[i];
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            // S = e_C S + K^T diag(exp(G_C - G)) U
            const float whole = in.p.row[kRowWhole];
#pragma unroll
            for (uint32_t t = 0; t < 4u; ++t) {
                const f32x4 tail = numbers(kRowTail, t);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) y[ct][t] *= tail;
            }
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (uint32_t t = 0; t < kTiles; ++t) S[ct][t] *= whole;
#pragma unroll
            for (uint32_t s = 0; s < 2u; ++s) {
                Mid h[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) h[ct] = operand_of<Mid>(y[ct][2u * s], y[ct][2u * s + 1u]);
#pragma unroll
                for (uint32_t t = 0; t < kTiles; ++t) {
                    const auto ka = in.k.across(s, t, lane);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) mma(S[ct][t], ka, h[ct]);
                }
            }
        }
        if (!kTwo) __syncthreads();
        __syncthreads();
    }
    if (final && col0 < a.value_dim) store_states<E>(final + ((uint64_t)seq * a.heads + head) * cells, S, a, col0, lane);
}

// ---------------------------------------------------------------------------
// single tokens
// ---------------------------------------------------------------------------
// A workgroup has `cols` columns of one head's state, four a thread and up to
// kStepRows rows of them: the state is read once, held in registers, and
// written once.  out = scale (e S^T q + (k q) u) needs no second sum over the
// new state.
constexpr uint32_t kStepRows = 16u;

template <class T>
__global__ __launch_bounds__(1024) void delta_step_kernel(DeltaArgs a, uint32_t first, uint32_t groups, const float *state,
                                                          float *new_state, const int32_t *__restrict__ slots,
                                                          uint32_t pool, T *__restrict__ out) {
    __shared__ float key[PS_DELTA_MAX_DIM], query[PS_DELTA_MAX_DIM];
    __shared__ float part[2][4096];
    const uint32_t cols = groups * 4u, blocks = (a.value_dim + cols - 1u) / cols;
    const uint32_t b = first + blockIdx.x, head = b / blocks % a.heads, row = b / blocks / a.heads;
    const uint32_t khead = head / (a.heads / a.kheads), lane = threadIdx.x & 63u;
    const uint32_t mine = threadIdx.x % groups, band = threadIdx.x / groups, bands = blockDim.x / groups;
    const uint32_t col = (b % blocks) * cols + mine * 4u, have = col < a.value_dim ? a.value_dim - col : 0u;
    const int32_t slot = slots ? slots[row] : (int32_t)row;
    const bool held = slot >= 0 && (uint32_t)slot < pool;
    const uint64_t cells = (uint64_t)a.key_dim * a.value_dim;
    const uint64_t at = held ? ((uint64_t)slot * a.heads + head) * cells + col : 0u;
    float S[kStepRows][4];
#pragma unroll
    for (uint32_t i = 0; i < kStepRows; ++i) {
        const uint32_t d = band + i * bands;
        const float *p = state + at + (uint64_t)d * a.value_dim;
        if (held && d < a.key_dim && have >= 4u) {
            const Pack<float, 4> w = *reinterpret_cast<const Pack<float, 4> *>(p);
#pragma unroll
            for (uint32_t j = 0; j < 4u; ++j) S[i][j] = w.v[j];
        } else {
#pragma unroll
            for (uint32_t j = 0; j < 4u; ++j) S[i][j] = held && d < a.key_dim && j < have ? p[j] : 0.0f;
        }
    }
    const T *k = static_cast<const T *>(a.k) + (int64_t)row * a.k_stride + (uint64_t)khead * a.key_dim;
    const T *q = static_cast<const T *>(a.q) + (int64_t)row * a.q_stride + (uint64_t)khead * a.key_dim;
    float kk = 0.0f, qq = 0.0f, kq = 0.0f;
    for (uint32_t d = lane; d < PS_DELTA_MAX_DIM; d += 64u) {
        const float kd = d < a.key_dim ? (float)k[d] : 0.0f, qd = d < a.key_dim ? (float)q[d] : 0.0f;
        kk = __builtin_fmaf(kd, kd, kk);
        qq = __builtin_fmaf(qd, qd, qq);
        kq = __builtin_fmaf(kd, qd, kq);
        if (threadIdx.x < 64u) key[d] = kd, query[d] = qd;
    }
    kk = wave_total(kk), qq = wave_total(qq), kq = wave_total(kq);
    const float nu = a.unit ? 1.0f / __builtin_sqrtf(kk + a.eps) : 1.0f, mu = a.unit ? 1.0f / __builtin_sqrtf(qq + a.eps) : 1.0f;
    float g = a.g[(int64_t)row * a.g_stride + head];
    const float beta = a.beta[(int64_t)row * a.beta_stride + head];
    const float e = exp_hw(g);
    __syncthreads();
    float ks[4] = {}, qs[4] = {};
#pragma unroll
    for (uint32_t i = 0; i < kStepRows; ++i) {
        const uint32_t d = band + i * bands;
        const float kd = d < a.key_dim ? key[d] : 0.0f, qd = d < a.key_dim ? query[d] : 0.0f;
#pragma unroll
        for (uint32_t j = 0; j < 4u; ++j) {
            ks[j] = __builtin_fmaf(kd, S[i][j], ks[j]);
            qs[j] = __builtin_fmaf(qd, S[i][j], qs[j]);
        }
    }
#pragma unroll
    for (uint32_t j = 0; j < 4u; ++j) {
        part[0][band * cols + mine * 4u + j] = ks[j];
        part[1][band * cols + mine * 4u + j] = qs[j];
    }
    __syncthreads();
#pragma unroll
    for (uint32_t j = 0; j < 4u; ++j) ks[j] = qs[j] = 0.0f;
    for (uint32_t i = 0; i < bands; ++i)
#pragma unroll
        for (uint32_t j = 0; j < 4u; ++j) {
            ks[j] += part[0][i * cols + mine * 4u + j];
            qs[j] += part[1][i * cols + mine * 4u + j];
        }
    const T *v = static_cast<const T *>(a.v) + (int64_t)row * a.v_stride + (uint64_t)head * a.value_dim + col;
    float u[4], o[4];
#pragma unroll
    for (uint32_t j = 0; j < 4u; ++j) {
        const float value = j < have ? (float)v[j] : 0.0f;
        u[j] = beta * __builtin_fmaf(-e * nu, ks[j], value);
        o[j] = a.scale * mu * __builtin_fmaf(e, qs[j], kq * nu * u[j]);
    }
    if (band == 0u) {
        T *to = out + ((uint64_t)row * a.heads + head) * a.value_dim + col;
#pragma unroll
        for (uint32_t j = 0; j < 4u; ++j)
            if (j < have) to[j] = (T)o[j];
    }
    if (!held) return;
#pragma unroll
    for (uint32_t i = 0; i < kStepRows; ++i) {
        const uint32_t d = band + i * bands;
        if (d >= a.key_dim) continue;
        const float kd = key[d] * nu;
        float *p = new_state + at + (uint64_t)d * a.value_dim;
        Pack<float, 4> w;
#pragma unroll
        for (uint32_t j = 0; j < 4u; ++j) w.v[j] = __builtin_fmaf(kd, u[j], e * S[i][j]);
        if (have >= 4u) *reinterpret_cast<Pack<float, 4> *>(p) = w;
        else
#pragma unroll
            for (uint32_t j = 0; j < 4u; ++j)
                if (j < have) p[j] = w.v[j];
    }
}

}  // namespace
}  // namespace dwps

using namespace dwps;

extern "C" uint64_t ps_gated_delta_checkpoint_floats(uint64_t tokens, uint32_t num_seqs, uint32_t heads, uint32_t key_dim,
                                                     uint32_t value_dim) {
    return chunk_slots(tokens, num_seqs, kChunkShift) * heads * key_dim * value_dim + tokens * heads * value_dim;
}

extern "C" ps_status ps_gated_delta(void *ws, size_t *ws_bytes, const ps_delta_input *in, void *out, float *final,
                                    float *checkpoints, void *stream) {
    ps_status st = delta_sizes(in);
    if (st != PS_OK) return st;
    const DeltaArgs a = delta_args(in);
    return with_type(in->dtype, [&](auto zero) {
        using T = decltype(zero);
        PlainWs plan;
        const size_t prepared_at = plan.take((size_t)a.slots * a.heads * sizeof(Prepared<T>));
        bool query = false;
        ps_status st = workspace_protocol(ws, ws_bytes, plan.at, &query);
        if (st != PS_OK || query) return st;
        if ((st = delta_pointers(in)) != PS_OK) return st;
        if (in->tokens && !out) return PS_ERR_NULL;
        if (!aligned(ws, 16) || !aligned(out, sizeof(T)) || !aligned(final, 4) || !aligned(checkpoints, 4))
            return PS_ERR_ALIGNMENT;
        const DeltaBytes n(in);
        const size_t kept = ps_gated_delta_checkpoint_floats(in->tokens, a.num_seqs, a.heads, a.key_dim, a.value_dim) * 4u;
        if (outputs_overlap({{out, n.values}, {final, n.states}, {checkpoints, kept}},
                            {{in->q, n.q}, {in->k, n.k}, {in->v, n.v}, {in->g, n.g}, {in->beta, n.beta},
                             {in->offsets, n.offsets}, {in->initial, n.states}}))
            return PS_ERR_ALIAS;
        if (!a.num_seqs) return PS_OK;
        hipStream_t s = static_cast<hipStream_t>(stream);
        Prepared<T> *prepared = ws_at<Prepared<T>>(ws, prepared_at);
        float *rhos = checkpoints ? checkpoints + (uint64_t)a.slots * a.heads * a.key_dim * a.value_dim : nullptr;
        return with_key_width(a.key_dim, [&](auto w) {
            constexpr int W = decltype(w)::value;
            timing_begin(s);
            launch_in_parts((uint64_t)a.slots * a.kheads, 1u, 256u, [&](uint32_t first, uint32_t grid) {
                hipLaunchKernelGGL((delta_prepare_kernel<T, W, false>), dim3(grid), dim3(256), 0, s, a, first, prepared,
                                   ws_counter(ws), plan.words());
            });
            // 32 columns a wave where there are more than 64, and registers for their states
            auto walk = [&](auto ct, auto eights) {
                constexpr int CT = decltype(ct)::value;
                constexpr bool E = decltype(eights)::value;
                const uint64_t groups = (uint64_t)a.num_seqs * a.heads * ceil_div(a.value_dim, 64u * CT);
                launch_in_parts(groups, 1u, 512u, [&](uint32_t first, uint32_t grid) {
                    hipLaunchKernelGGL((delta_walk_kernel<T, W, CT, E>), dim3(grid), dim3(512), 0, s, a, first, prepared,
                                       static_cast<T *>(out), final, checkpoints, rhos);
                });
            };
            const bool eights = a.key_dim % 8u == 0u && a.value_dim % 8u == 0u;
            auto shape = [&](auto e) {
                if (W <= 128 && a.value_dim > 64u) walk(std::integral_constant<int, W <= 128 ? 2 : 1>(), e);
                else walk(std::integral_constant<int, 1>(), e);
            };
            if (eights) shape(std::true_type());
            else shape(std::false_type());
            timing_end(s);
            return launch_status();
        });
    });
}

extern "C" ps_status ps_gated_delta_step(const ps_delta_input *in, const float *state, float *new_state,
                                         const int32_t *slots, uint32_t pool, void *out, void *stream) {
    ps_delta_input one;
    if (!in) return PS_ERR_NULL;
    one = *in;
    one.offsets = nullptr, one.initial = nullptr, one.num_seqs = 1u;
    in = &one;
    ps_status st = delta_sizes(in);
    if (st != PS_OK) return st;
    if (!slots && in->tokens > pool) return PS_ERR_SIZE;
    if ((st = delta_pointers(in)) != PS_OK) return st;
    if (!in->tokens) return PS_OK;
    if (!out || (pool && (!state || !new_state))) return PS_ERR_NULL;
    if (!aligned(out, dtype_bytes(in->dtype)) || !aligned(state, 4) || !aligned(new_state, 4) || !aligned(slots, 4))
        return PS_ERR_ALIGNMENT;
    const DeltaBytes n(in);
    const size_t states = (size_t)pool * in->heads * in->key_dim * in->value_dim * 4u;
    const Bytes before = {new_state == state ? nullptr : state, states};
    if (outputs_overlap({{out, n.values}, {new_state, states}},
                        {{in->q, n.q}, {in->k, n.k}, {in->v, n.v}, {in->g, n.g}, {in->beta, n.beta},
                         {slots, slots ? in->tokens * 4u : 0u}, before}))
        return PS_ERR_ALIAS;
    const DeltaArgs a = delta_args(in);
    hipStream_t s = static_cast<hipStream_t>(stream);
    return with_type(in->dtype, [&](auto zero) {
        using T = decltype(zero);
        uint32_t groups = 4u;
        while (groups * 4u < a.value_dim) groups *= 2u;
        uint32_t bands = 1u;
        while (bands * kStepRows < a.key_dim || bands * groups < 64u) bands *= 2u;
        const uint64_t work = (uint64_t)a.tokens * a.heads * ceil_div(a.value_dim, groups * 4u);
        timing_begin(s);
        launch_in_parts(work, 1u, groups * bands, [&](uint32_t first, uint32_t grid) {
            hipLaunchKernelGGL((delta_step_kernel<T>), dim3(grid), dim3(groups * bands), 0, s, a, first, groups, state,
                               new_state, slots, pool, static_cast<T *>(out));
        });
        timing_end(s);
        return launch_status();
    });
}
