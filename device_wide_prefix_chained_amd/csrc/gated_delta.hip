// gated_delta.hip -- the gated delta rule over packed sequences, and for
// single tokens.
//
//   S' = exp(g) S,  u = beta (v - S'^T k),  S = S' + k u^T,  out = scale S^T q
//
// Packed sequences are in delta_walk.hpp.
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
    // what one launch counts, and a workgroup's number: chunks and heads
    if (chunk_slots(in->tokens, in->offsets ? in->num_seqs : 1u, kChunkShift) * (uint64_t)h >= 1ull << 31) return PS_ERR_SIZE;
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

// ---------------------------------------------------------------------------
// single tokens
// ---------------------------------------------------------------------------
// A workgroup has `cols` columns of one head's state, four a thread and up to
// kStepRows rows of them: the state is read once, held in registers, and
// written once.  out = scale (e S^T q + (k q) u) needs no second sum over the
// new state.  Bound by memory, the state's 8 bytes an element: 256 rows of 16
// heads, 128 x 128, 115 us, 4.7 TB/s (129 with the gates, keys and values asked
// for after the state, 154 also with 64 columns a workgroup).  A row of 16 heads 7.2,
// and 6.8 with 16 x 16 states: the launch and one wave's chain of loads, sums and
// barriers, not the state's bytes (8.2 where they come from HBM).
constexpr uint32_t kStepRows = 16u, kStepThreads = 512u, kStepKeys = PS_DELTA_MAX_DIM / 64u;

template <class T>
__global__ __launch_bounds__(kStepThreads) void delta_step_kernel(DeltaArgs a, uint32_t first, uint32_t groups, const float *state,
                                                          float *new_state, const int32_t *__restrict__ slots,
                                                          uint32_t pool, T *__restrict__ out) {
    __shared__ float key[PS_DELTA_MAX_DIM], query[PS_DELTA_MAX_DIM];
    __shared__ float part[2][2048];
    const uint32_t cols = groups * 4u, blocks = (a.value_dim + cols - 1u) / cols;
    const uint32_t item = first + blockIdx.x / blocks, head = item % a.heads, row = item / a.heads;
    const uint32_t khead = head / (a.heads / a.kheads), lane = threadIdx.x & 63u;
    const uint32_t mine = threadIdx.x % groups, band = threadIdx.x / groups, bands = blockDim.x / groups;
    const uint32_t col = (blockIdx.x % blocks) * cols + mine * 4u, have = col < a.value_dim ? a.value_dim - col : 0u;
    const int32_t slot = slots ? slots[row] : (int32_t)row;
    // what does not hang on the slot is on its way before the state
    const T *k = static_cast<const T *>(a.k) + (int64_t)row * a.k_stride + (uint64_t)khead * a.key_dim;
    const T *q = static_cast<const T *>(a.q) + (int64_t)row * a.q_stride + (uint64_t)khead * a.key_dim;
    const T *v = static_cast<const T *>(a.v) + (int64_t)row * a.v_stride + (uint64_t)head * a.value_dim + col;
    const float g = a.g[(int64_t)row * a.g_stride + head], beta = a.beta[(int64_t)row * a.beta_stride + head];
    T ks_in[kStepKeys], qs_in[kStepKeys], value[4];
#pragma unroll
    for (uint32_t i = 0; i < kStepKeys; ++i) {
        const uint32_t d = lane + 64u * i;
        ks_in[i] = d < a.key_dim ? k[d] : (T)0.0f, qs_in[i] = d < a.key_dim ? q[d] : (T)0.0f;
    }
#pragma unroll
    for (uint32_t j = 0; j < 4u; ++j) value[j] = j < have ? v[j] : (T)0.0f;
    const bool held = slot >= 0 && (uint32_t)slot < pool;
    const uint64_t cells = (uint64_t)a.key_dim * a.value_dim;
    const uint64_t at = held ? ((uint64_t)slot * a.heads + head) * cells : 0u;
    const float *from = state + at;
    float *into = new_state + at;
    float S[kStepRows][4];
#pragma unroll
    for (uint32_t i = 0; i < kStepRows; ++i) {
        const uint32_t d = band + i * bands;
        const float *p = from + (d * a.value_dim + col);
        if (held && d < a.key_dim && have >= 4u) {
            const Pack<float, 4> w = *reinterpret_cast<const Pack<float, 4> *>(p);
#pragma unroll
            for (uint32_t j = 0; j < 4u; ++j) S[i][j] = w.v[j];
        } else {
#pragma unroll
            for (uint32_t j = 0; j < 4u; ++j) S[i][j] = held && d < a.key_dim && j < have ? p[j] : 0.0f;
        }
    }
    float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < kStepKeys; ++i) {
        const float kd = (float)ks_in[i], qd = (float)qs_in[i];
        kk = __builtin_fmaf(kd, kd, kk);
        qq = __builtin_fmaf(qd, qd, qq);
        kq = __builtin_fmaf(kd, qd, kq);
        if (threadIdx.x < 64u) key[lane + 64u * i] = kd, query[lane + 64u * i] = qd;
    }
    kk = wave_total(kk), qq = wave_total(qq), kq = wave_total(kq);
    const float nu = a.unit ? 1.0f / __builtin_sqrtf(kk + a.eps) : 1.0f, mu = a.unit ? 1.0f / __builtin_sqrtf(qq + a.eps) : 1.0f;
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
    float u[4], o[4];
#pragma unroll
    for (uint32_t j = 0; j < 4u; ++j) {
        u[j] = beta * __builtin_fmaf(-e * nu, ks[j], (float)value[j]);
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
        float *p = into + (d * a.value_dim + col);
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
    // no offsets may come with no number of sequences: all rows are one
    return chunk_slots(tokens, num_seqs ? num_seqs : 1u, kChunkShift) * heads * ((uint64_t)(key_dim + kChunk) * value_dim + kSizes);
}

extern "C" ps_status ps_gated_delta(void *ws, size_t *ws_bytes, const ps_delta_input *in, void *out, float *final,
                                    float *checkpoints, void *stream) {
    ps_status st = delta_sizes(in);
    if (st != PS_OK) return st;
    return with_type(in->dtype, [&](auto zero) {
        return delta_forward<decltype(zero)>(ws, ws_bytes, in, out, final, checkpoints, static_cast<hipStream_t>(stream));
    });
}

extern "C" ps_status ps_gated_delta_bwd(void *ws, size_t *ws_bytes, const ps_delta_input *in, const void *dout,
                                        const float *dfinal, const float *checkpoints, const ps_delta_grads *grads,
                                        void *stream) {
    ps_status st = delta_sizes(in);
    if (st != PS_OK) return st;
    return with_type(in->dtype, [&](auto zero) {
        return delta_backward<decltype(zero)>(ws, ws_bytes, in, dout, dfinal, checkpoints, grads, static_cast<hipStream_t>(stream));
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
    if ((!slots && in->tokens > pool) || in->tokens * in->heads >= 1ull << 31) return PS_ERR_SIZE;
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
        // up to 128 columns a workgroup; fewer while they leave CUs without one
        uint32_t groups = 4u;
        while (groups < 32u && groups * 4u < a.value_dim) groups *= 2u;
        while (groups > 4u && (uint64_t)a.tokens * a.heads * ceil_div(a.value_dim, groups * 4u) < 256u) groups /= 2u;
        uint32_t bands = 1u;
        while (bands * kStepRows < a.key_dim || bands * groups < 64u) bands *= 2u;
        const uint64_t blocks = ceil_div(a.value_dim, groups * 4u);
        timing_begin(s);
        launch_in_parts((uint64_t)a.tokens * a.heads, blocks, groups * bands, [&](uint32_t first, uint32_t grid) {
            hipLaunchKernelGGL((delta_step_kernel<T>), dim3(grid), dim3(groups * bands), 0, s, a, first, groups, state,
                               new_state, slots, pool, static_cast<T *>(out));
        });
        timing_end(s);
        return launch_status();
    });
}
