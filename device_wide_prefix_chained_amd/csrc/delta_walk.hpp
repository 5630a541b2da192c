// delta_walk.hpp -- the gated delta rule over packed sequences: kernels that walk
// over chunks, and their launches.  One type of activations a source file.
//
// Every chunk of 64 rows is prepared by itself (delta_block.hpp).  Then a
// workgroup walks over a sequence's chunks with 64 columns of a head's state in its
// registers; long sequences in segments side by side, for which
// two walks and a link first find the states that enter them.
#pragma once

#include "delta_block.hpp"

namespace dwps {
namespace {

// Waves of a workgroup that walk, with 16 columns each; four more feed them.  With
// eight, a chunk's keys are read once for 128 columns, but the eight wait for one
// another at more barriers: 453 us in place of 422 for 16384 rows of 16 heads, 128
// x 128, bf16, 869 in place of 849 for a training step of 8192.
constexpr int kWalkWaves = 4;

// What a step of a walk reads: a chunk's keys, queries and values, and what was
// prepared of it.
template <class T, int W>
struct WalkTile {
    static constexpr uint32_t kCols = 16u * kWalkWaves;
    KeyTile<T, W> k, q;
    Prepared<T> p;
    T v[kChunk][kCols + 8u];
};
template <class T, int W>
constexpr bool kValuesFit = sizeof(WalkTile<T, W>) <= kMostShared;
template <class T, int W>
constexpr size_t walk_tile_bytes() {
    return kValuesFit<T, W> ? sizeof(WalkTile<T, W>) : sizeof(WalkTile<T, W>) - sizeof(WalkTile<T, W>::v);
}

// Rows 16 t + 4 q + i of column `here` + m of a tile of values.
template <class T, uint32_t STRIDE>
__device__ __forceinline__ f32x4 value_rows(const T (&tile)[kChunk][STRIDE], uint32_t t, uint32_t q, uint32_t m, uint32_t here) {
    f32x4 v;
    if constexpr (sizeof(T) == 2) {
        const i16x4 raw = read_transposed(
            reinterpret_cast<const uint16_t *>(&tile[16u * t + 4u * q + (m >> 2)][here + 4u * (m & 3u)]));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = finite_or_nan((float)__builtin_bit_cast(T, (uint16_t)raw[i]));
    } else {
#pragma unroll
        for (uint32_t i = 0; i < 4u; ++i) v[i] = finite_or_nan((float)tile[16u * t + 4u * q + i][here + m]);
    }
    return v;
}

// Where a sequence is walked over in segments of 2^shift rows side by side: a
// state that enters a segment leaves it as M S + N, whose columns are walks of
// their own, M's from the unit matrix without values and N's from zero.
// `shift` 31: whole sequences, one segment each.
struct Segments {
    uint32_t shift;
    void *m;   // [segment numbers, heads] of SegmentMatrix
    float *n;  // [segment numbers, heads, key_dim, value_dim]: N, then the states that enter
};
// M as operands: rows place(t, lane & 15), columns 32 c + 8 (lane >> 4) .., each
// operand with what takes its scale back.
template <class T, int W>
struct SegmentMatrix {
    typename Form<T>::Mid m[W / 16][W / 32][64];
    float back[W / 16][W / 32];
};
// Columns of M that four waves hold, into operands, by way of shared memory;
// all eight waves, `walks`: those that hold them.  The block with the last of the
// `keys` columns leaves zeros for the blocks after it, which have no walk (129 to
// 192 keys of W 256): the link reads all W columns.
template <class T, int W>
__device__ __forceinline__ void store_matrix(SegmentMatrix<T, W> &to, float *shared, const f32x4 (*S)[W / 16], float by,
                                             uint32_t block0, uint32_t keys, uint32_t wave, uint32_t lane, bool walks) {
    constexpr uint32_t kCols = 16u * kWalkWaves, kRow = kCols + 4u;
    static_assert(W * kRow * 4u <= kMostShared, "a block of M fits shared memory");
    const uint32_t m = lane & 15u, q = lane >> 4;
    if (walks) {
#pragma unroll
        for (uint32_t t = 0; t < W / 16u; ++t)
#pragma unroll
            for (uint32_t i = 0; i < 4u; ++i) shared[place(t, 4u * q + i) * kRow + wave * 16u + m] = (*S)[t][i] * by;
    }
    __syncthreads();
    for (uint32_t i = wave; i < W / 16u * (kCols / 32u); i += kWalkWaves + 4u) {
        const uint32_t t = i / (kCols / 32u), c = i % (kCols / 32u);
        if (block0 + 32u * c >= (uint32_t)W) continue;
        const float *p = shared + place(t, m) * kRow + 32u * c + 8u * q;
        float v[8], most = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = p[j], most = __builtin_fmaxf(most, __builtin_fabsf(v[j]));
        const Scale of = scale_of<Form<T>::scaled>(Form<T>::scaled ? wave_largest(most) : 0.0f);
        operand_of(to.m[t][block0 / 32u + c][lane], v, of.by);
        if (lane == 0u) to.back[t][block0 / 32u + c] = of.back;
    }
    const uint32_t next = block0 + kCols;
    if (next < keys || next >= (uint32_t)W) return;
    const uint32_t rest = ((uint32_t)W - next) / 32u;
    for (uint32_t i = wave; i < W / 16u * rest; i += kWalkWaves + 4u) {
        const uint32_t t = i / rest, c = next / 32u + i % rest;
        const float zeros[8] = {};
        operand_of(to.m[t][c][lane], zeros);
        if (lane == 0u) to.back[t][c] = 0.0f;
    }
}
struct WalkResults {
    void *out;
    float *final;
    float *states, *rhos;  // [chunk numbers, heads, key_dim | kChunk, value_dim]
    float *sizes;  // [chunk numbers, heads, kSizes]: the largest of `states` and of `rhos`, by wave of columns
};

// The feeding waves of a walk: keys, queries, values and what was prepared of
// each chunk, from memory into registers, a whole chunk's work before they are
// waited for, then into the tile.
template <class T, int W, bool E>
struct DeltaFeed {
    typedef WalkTile<T, W> Tile;
    const DeltaArgs &a;
    const Prepared<T> *prepared;
    Chunk r;
    uint32_t base, head, khead, block0;  // of the first chunk; the head and its keys'; the block's first column
    const T *values;                     // of the head
    int64_t values_stride;

    // LEAD: no queries and no scores.  order(i): the i-th chunk to come.
    template <bool LEAD, class F, class O>
    __device__ __forceinline__ void run(uint32_t chunks, bool with_values, F tile, O order) const {
        constexpr bool kTwo = 2u * sizeof(Tile) <= kMostShared, kV = kValuesFit<T, W>;
        constexpr uint32_t kKeys = W / 32, kVals = Tile::kCols / 32u;
        constexpr uint32_t kBytes = LEAD ? offsetof(Prepared<T>, scores) : sizeof(Prepared<T>), kWords = (kBytes + 4095u) / 4096u;
        const uint32_t thread = threadIdx.x - 64u * kWalkWaves, row = thread >> 2, part = (thread & 3u) * 8u;
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
                if (!LEAD) qs[c] = raw8<E, T>(q0 + row * a.q_stride, q0, is, part + 32u * c, a.key_dim);
            }
            if constexpr (kV) {
                const T *v0 = values + lo * values_stride;
#pragma unroll
                for (uint32_t c = 0; c < kVals; ++c)
                    vs[c] = raw8<E, T>(v0 + row * values_stride, v0, is && with_values, block0 + part + 32u * c, a.value_dim);
            }
            const u32x4 *p = reinterpret_cast<const u32x4 *>(&prepared[(uint64_t)(base + i) * a.heads + head]);
#pragma unroll
            for (uint32_t c = 0; c < kWords; ++c) {
                const uint32_t at = thread + 256u * c;
                if (at < kBytes / 16u) ps[c] = p[at];
            }
        };
        auto leave = [&](Tile *to) {
            auto put = [&](KeyTile<T, W> &tile, const Pack<T, 8>(&from)[kKeys]) {
                float v[kKeys][8];
#pragma unroll
                for (uint32_t c = 0; c < kKeys; ++c) values_of<T>(v[c], from[c]);
                const Scale by = row_scale<T, 4>(v);
#pragma unroll
                for (uint32_t c = 0; c < kKeys; ++c) tile.put(row, part + 32u * c, v[c], by.by);
            };
            put(to->k, ks);
            if (!LEAD) put(to->q, qs);
            if constexpr (kV) {
#pragma unroll
                for (uint32_t c = 0; c < kVals; ++c) *reinterpret_cast<Pack<T, 8> *>(&to->v[row][part + 32u * c]) = vs[c];
            }
#pragma unroll
            for (uint32_t c = 0; c < kWords; ++c) {
                const uint32_t at = thread + 256u * c;
                if (at < kBytes / 16u) reinterpret_cast<u32x4 *>(&to->p)[at] = ps[c];
            }
        };
        if (chunks) fetch(order(0u)), leave(tile(0u));
        if (chunks > 1u) fetch(order(1u));
        __syncthreads();
        for (uint32_t i = 0; i < chunks; ++i) {
            if (!kTwo) __syncthreads();
            if (i + 1u < chunks) leave(tile(i + 1u));
            if (i + 2u < chunks) fetch(order(i + 2u));
            __syncthreads();
        }
    }
};

// A column of the unit matrix.
template <int TILES>
__device__ __forceinline__ void unit_states(f32x4 (&S)[TILES], uint32_t col, uint32_t q) {
#pragma unroll
    for (uint32_t t = 0; t < (uint32_t)TILES; ++t)
#pragma unroll
        for (uint32_t i = 0; i < 4u; ++i) S[t][i] = place(t, 4u * q + i) == col ? 1.0f : 0.0f;
}
// The operands of one triangle, and four numbers of each of a chunk's rows.
template <class M>
struct Triangle {
    M of[kTriangle];
    __device__ __forceinline__ void load(const M (&from)[kTriangle][64], uint32_t lane) {
#pragma unroll
        for (uint32_t i = 0; i < kTriangle; ++i) of[i] = from[i][lane];
    }
};
struct RowNumbers {
    f32x4 of[4];
    __device__ __forceinline__ void load(const float *row, uint32_t q) {
#pragma unroll
        for (uint32_t t = 0; t < 4u; ++t) of[t] = *reinterpret_cast<const f32x4 *>(row + 16u * t + 4u * q);
    }
};
// y += T h for the lower triangle's tiles (upper: the upper one's) of 32 places s.
template <class M, class H>
__device__ __forceinline__ void mma_lower(f32x4 (&y)[4], const Triangle<M> &t, const H (&h)[2]) {
    mma_rows(y, {t.of[lower_at(0, 0)], t.of[lower_at(1, 0)], t.of[lower_at(2, 0)], t.of[lower_at(3, 0)]}, h[0]);
    f32x4 low[2] = {y[2], y[3]};
    mma_rows(low, {t.of[lower_at(2, 1)], t.of[lower_at(3, 1)]}, h[1]);
    y[2] = low[0], y[3] = low[1];
}
template <class M, class H>
__device__ __forceinline__ void mma_upper(f32x4 (&y)[4], const Triangle<M> &t, const H (&h)[2]) {
    mma_rows(y, {t.of[upper_at(0, 1)], t.of[upper_at(1, 1)], t.of[upper_at(2, 1)], t.of[upper_at(3, 1)]}, h[1]);
    f32x4 high[2] = {y[0], y[1]};
    mma_rows(high, {t.of[upper_at(0, 0)], t.of[upper_at(1, 0)]}, h[0]);
    y[0] = high[0], y[1] = high[1];
}
// S += K^T h, four tiles of keys at a time.
template <int TILES, class Tile, class M>
__device__ __forceinline__ void mma_keys(f32x4 (&S)[TILES], const Tile &k, uint32_t s, const M &h, uint32_t lane) {
    constexpr int G = TILES < 4 ? TILES : 4;
#pragma unroll
    for (int g = 0; g < TILES; g += G) {
        decltype(k.across(0u, 0u, 0u)) a[G];
        f32x4 acc[G];
#pragma unroll
        for (int t = 0; t < G; ++t) a[t] = k.across(s, g + t, lane), acc[t] = S[g + t];
        mma_rows(acc, a, h);
#pragma unroll
        for (int t = 0; t < G; ++t) S[g + t] = acc[t];
    }
}

// kWalkWaves waves walk over a segment's chunks, each with 16 columns of a head's state;
// four feed them, leaving a chunk in the tile of the two that is not in use while
// the one before is worked on (or, where shared memory has room for one, after a
// barrier in that one).  LEAD: the walks for M and N, of segments that another
// follows.
// Bound by the chain of a step, K S, the inverse, U and the state, each of which
// waits for the one before: 3.1 us with one wave, 4.3 with the four that share the
// CU's matrix units and shared memory.  8192 rows of 16 heads, 128 x 128, bf16, in
// one sequence: 75 us, and 90 for M and N.  16 columns a wave: with 32 the states
// took the registers that the operands of the next product wait in.
template <class T, int W, bool E, bool LEAD>
__global__ __launch_bounds__(64 * (kWalkWaves + 4)) void delta_walk_kernel(DeltaArgs a, uint32_t first, const Prepared<T> *__restrict__ prepared,
                                                         Segments seg, WalkResults to) {
    typedef typename Form<T>::Mid Mid;
    typedef typename Form<T>::In In;
    typedef WalkTile<T, W> Tile;
    constexpr uint32_t kTiles = W / 16, kCols = Tile::kCols;
    constexpr bool kTwo = 2u * sizeof(Tile) <= kMostShared, kV = kValuesFit<T, W>;
    __shared__ __attribute__((aligned(16))) char memory[kTwo ? 2u * sizeof(Tile) : walk_tile_bytes<T, W>()];
    const uint32_t value_blocks = (a.value_dim + kCols - 1u) / kCols, key_blocks = LEAD ? (a.key_dim + kCols - 1u) / kCols : 0u;
    const uint32_t blocks = value_blocks + key_blocks, block = blockIdx.x % blocks, item = first + blockIdx.x / blocks;
    const uint32_t head = item % a.heads, number = item / a.heads, khead = head / (a.heads / a.kheads);
    const uint32_t wave = wave_number(), lane = threadIdx.x & 63u, m = lane & 15u, q = lane >> 4;
    const bool unit = block < key_blocks;  // columns of M
    const uint32_t block0 = (block - (unit ? 0u : key_blocks)) * kCols, width = unit ? a.key_dim : a.value_dim;
    const Chunk r = find_chunk(a.offsets, a.num_seqs, a.tokens, seg.shift, number);
    const Rows seq = sequence_rows(a.offsets, a.tokens, r.seq, kChunkShift);
    if (r.index == kNoChunk || (r.lo == r.hi && r.index != 0u) || (LEAD && r.hi == seq.hi)) return;
    const uint32_t chunks = (r.hi - r.lo + kChunk - 1u) / kChunk;
    const uint32_t base = seq.base + ((r.lo - seq.lo) >> kChunkShift);  // its first chunk's number
    const T *values = static_cast<const T *>(a.v) + (uint64_t)head * a.value_dim;
    auto tile = [&](uint32_t i) { return reinterpret_cast<Tile *>(memory + (kTwo && (i & 1u) ? sizeof(Tile) : 0u)); };
    const DeltaFeed<T, W, E> feed = {a, prepared, r, base, head, khead, block0, values, a.v_stride};
    if (wave >= (uint32_t)kWalkWaves) {
        feed.template run<LEAD>(chunks, !unit, tile, [](uint32_t i) { return i; });
        if (LEAD && unit)
            store_matrix<T, W>(static_cast<SegmentMatrix<T, W> *>(seg.m)[(uint64_t)number * a.heads + head],
                                   reinterpret_cast<float *>(memory), nullptr, 1.0f, block0, a.key_dim, wave, lane, false);
        return;
    }
    const uint32_t here = wave * 16u, col0 = block0 + here, col = col0 + m;
    const uint64_t cells = (uint64_t)a.key_dim * a.value_dim;
    constexpr bool kScaled = Form<T>::scaled;
    f32x4 S[kTiles];  // times `unit_of`, the states
    float unit_of = 1.0f;
    {
        const float *from = nullptr;
        if (!LEAD && r.index) from = seg.n + ((uint64_t)number * a.heads + head) * cells;
        else if (!LEAD && a.initial) from = a.initial + ((uint64_t)r.seq * a.heads + head) * cells;
        load_states<E>(S, from, a.key_dim, a.value_dim, col, q);
        if (unit) unit_states(S, col, q);
    }
    __syncthreads();
    for (uint32_t c = 0; c < chunks; ++c) {
        const uint32_t lo = r.lo + c * kChunk, rows = r.hi - lo < kChunk ? r.hi - lo : kChunk;
        const Tile &in = *tile(c);
        if (col0 < width) {
            if (!LEAD && to.states)
                store_states<E>(to.states + ((uint64_t)(base + c) * a.heads + head) * cells, S, unit_of, a.key_dim, a.value_dim,
                                col, q);
            const float most = kScaled ? wave_largest(largest(S)) : 0.0f;
            const Scale of_s = scale_of<kScaled>(most);
            f32x4 x[4], o[4], y[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = o[t] = y[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            // K S, and (Q S)^T: the operands' sides are the other way round, which
            // leaves a row of out in a lane and neighbouring columns in its registers
            In ka[4], qa[4];
            auto keys = [&](uint32_t s) {
#pragma unroll
                for (uint32_t t = 0; t < 4u; ++t) {
                    ka[t] = in.k.along(16u * t + m, 32u * s + 8u * q);
                    if (!LEAD) qa[t] = in.q.along(16u * t + m, 32u * s + 8u * q);
                }
            };
            keys(0u);
#pragma unroll
            for (uint32_t s = 0; s < kTiles / 2u; ++s) {
                const Mid h = operand_of<Mid>(S[2u * s], S[2u * s + 1u], of_s.by);
                mma_rows(x, ka, h);
                if (!LEAD) mma_columns(o, h, qa);
                if (s + 1u < kTiles / 2u) keys(s + 1u);
            }
            // R = V - e K S
            RowNumbers e;
            e.load(in.p.row + kRowE, q);
            f32x4 v[4];
            if constexpr (kV) {
#pragma unroll
                for (uint32_t t = 0; t < 4u; ++t) v[t] = value_rows<T>(in.v, t, q, m, here);
            } else {
#pragma unroll
                for (uint32_t t = 0; t < 4u; ++t)
#pragma unroll
                    for (uint32_t i = 0; i < 4u; ++i) {
                        const uint32_t row = 16u * t + 4u * q + i;
                        v[t][i] = row < rows && col < a.value_dim && !unit
                                      ? finite_or_nan((float)values[(int64_t)(lo + row) * a.v_stride + col])
                                      : 0.0f;
                    }
            }
            Triangle<Mid> tri;
            tri.load(in.p.inverse, lane);
            const float inverse_back = in.p.row[kRowInverse];
            __builtin_amdgcn_sched_barrier(0);
            const float from_s = of_s.back * unit_of;
#pragma unroll
            for (uint32_t t = 0; t < 4u; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[t][i] = __builtin_fmaf(-from_s * e.of[t][i], x[t][i], v[t][i]);
            // rho
            const Scale of_x = scale_of<kScaled>(kScaled ? wave_largest(largest(x)) : 0.0f);
            const float from_x = kScaled ? of_x.back * inverse_back : 1.0f;
            {
                const Mid h[2] = {operand_of<Mid>(x[0], x[1], of_x.by), operand_of<Mid>(x[2], x[3], of_x.by)};
                mma_lower(y, tri, h);
            }
            if (!LEAD && to.rhos) {
                if (kScaled) {
                    const float of_y = wave_largest(largest(y)) * from_x;
                    float *sizes = to.sizes + ((uint64_t)(base + c) * a.heads + head) * kSizes + col0 / 16u;
                    if (lane == 0u) sizes[0] = most * unit_of, sizes[kSizeWaves] = of_y;
                }
                if (col < a.value_dim)
                    store_rows(to.rhos + ((uint64_t)(base + c) * a.heads + head) * kChunk * a.value_dim, a.value_dim, y, from_x, col, q);
            }
            __builtin_amdgcn_sched_barrier(0);
            // U, and out^T = scale e (Q S)^T + U^T P^T
            RowNumbers beta, tail;
            float eq[4];
            beta.load(in.p.row + kRowBeta, q);
            if (!LEAD) {
                tri.load(in.p.scores, lane);
#pragma unroll
                for (uint32_t t = 0; t < 4u; ++t) eq[t] = in.p.row[kRowQ + 16u * t + m];
            }
            const float kept = unit_of * in.p.row[kRowWhole], scores_back = in.p.row[kRowScores];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (uint32_t t = 0; t < 4u; ++t) y[t] *= beta.of[t] * from_x;
            tail.load(in.p.row + kRowTail, q);
            if constexpr (!LEAD) {
                const Scale of_u = scale_of<kScaled>(kScaled ? wave_largest(largest(y)) : 0.0f);
                const float from_o = kScaled ? of_u.back * scores_back : 1.0f;
                // the two parts of out are summed at the end, each by its own scale: where U
                // and the scores are zero or small, theirs would take the states' part past
                // fp32's range
                f32x4 pu[4];
#pragma unroll
                for (uint32_t t = 0; t < 4u; ++t) pu[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f}, o[t] *= eq[t] * from_s;
                const Mid h[2] = {operand_of<Mid>(y[0], y[1], of_u.by), operand_of<Mid>(y[2], y[3], of_u.by)};
                mma_columns(pu, h[0], {tri.of[lower_at(0, 0)], tri.of[lower_at(1, 0)], tri.of[lower_at(2, 0)], tri.of[lower_at(3, 0)]});
                f32x4 low[2] = {pu[2], pu[3]};
                mma_columns(low, h[1], {tri.of[lower_at(2, 1)], tri.of[lower_at(3, 1)]});
                pu[2] = low[0], pu[3] = low[1];
#pragma unroll
                for (uint32_t t = 0; t < 4u; ++t) {
                    const uint32_t row = 16u * t + m, at = col0 + 4u * q;
                    if (row < rows && at < a.value_dim) {
                        T *p = static_cast<T *>(to.out) + ((uint64_t)(lo + row) * a.heads + head) * a.value_dim + at;
                        Pack<T, 4> w;
#pragma unroll
                        for (int i = 0; i < 4; ++i) w.v[i] = (T)__builtin_fmaf(pu[t][i], from_o, o[t][i]);
                        if (E || at + 4u <= a.value_dim) {
                            *reinterpret_cast<Pack<T, 4> *>(p) = w;
                        } else {
#pragma unroll
                            for (uint32_t i = 0; i < 4u; ++i)
                                if (at + i < a.value_dim) p[i] = w.v[i];
                        }
                    }
                }
            }
            // S = e_C S + K^T diag(exp(G_C - G)) U
#pragma unroll
            for (uint32_t t = 0; t < 4u; ++t) y[t] *= tail.of[t];
            const Scale of_u = scale_of_sum<kScaled>(kScaled ? wave_largest(largest(y)) : 0.0f, most * kept);
#pragma unroll
            for (uint32_t t = 0; t < kTiles; ++t) S[t] *= kept * of_u.by;
            unit_of = of_u.back;
            mma_keys(S, in.k, 0u, operand_of<Mid>(y[0], y[1], of_u.by), lane);
            mma_keys(S, in.k, 1u, operand_of<Mid>(y[2], y[3], of_u.by), lane);
        }
        if (!kTwo) __syncthreads();
        __syncthreads();
    }
    const uint64_t place_of = (uint64_t)number * a.heads + head;
    if (LEAD && unit) {
        store_matrix<T, W>(static_cast<SegmentMatrix<T, W> *>(seg.m)[place_of], reinterpret_cast<float *>(memory), &S, unit_of,
                               block0, a.key_dim, wave, lane, true);
        return;
    }
    if (col0 >= width) return;
    if (LEAD) store_states<E>(seg.n + place_of * cells, S, unit_of, a.key_dim, a.value_dim, col, q);
    else if (to.final && r.hi == seq.hi)
        store_states<E>(to.final + ((uint64_t)r.seq * a.heads + head) * cells, S, unit_of, a.key_dim, a.value_dim, col, q);
}

// The states that enter a sequence's segments after the first, S <- M S + N,
// in the places of N.  BACK: the gradients that enter from the segment after,
// from the last to the first; `start` holds what enters the sequence, or is
// NULL.  A wave has 32 keys of a workgroup's columns, so that a step is short: every
// wave leaves its keys as operands in shared memory, and multiplies its rows of M,
// which are on their way kAhead groups of 32 columns before they are used.
// Bound by a step's chain of loads, products and a barrier, 2.4 to 2.9 us: 15 steps
// of 16 heads, 128 x 128, 36 to 44 us; with a wave for all keys of 16 columns 85 us,
// and M as rows of numbers 138 us.  Nothing is done to N as it arrives, or the
// step before would wait for it (80 us).
// More than 128 keys: eight waves, 16 columns a workgroup and half of M ahead, which
// 200 registers hold; 3 steps of 16 heads, 256 x 256, 25 us (fp32 31).  Four waves
// with twice the keys and all of M ahead spilled 580 registers, took 126 us, and in
// fp32 came out wrong: the compiler (ROCm 7.2) lost one of the four registers of a
// tile of N that it had moved to accumulation registers and to scratch in part.
template <int W>
struct Link {
    static constexpr uint32_t kKeys = W / 32, kAhead = kKeys < 4 ? kKeys : 4, kColumns = W > 128 ? 16 : 32;
    static constexpr int kThreads = kKeys < 4 ? 256 : 64 * kKeys;
};
template <class T, int W, bool BACK>
__global__ __launch_bounds__(Link<W>::kThreads) void delta_link_kernel(DeltaArgs a, uint32_t first, Segments seg, const float *start) {
    typedef typename Form<T>::Mid Mid;
    constexpr uint32_t kKeys = Link<W>::kKeys, kAhead = Link<W>::kAhead, CT = Link<W>::kColumns / 16;
    constexpr bool kScaled = Form<T>::scaled;
    __shared__ Mid operands[2][kKeys][CT][64];
    __shared__ float backs[2][kKeys];
    const uint32_t blocks = (a.value_dim + 16u * CT - 1u) / (16u * CT), item = first + blockIdx.x / blocks, head = item % a.heads;
    const uint32_t wave = wave_number(), lane = threadIdx.x & 63u, m = lane & 15u, q = lane >> 4;
    const uint32_t col0 = blockIdx.x % blocks * 16u * CT, s = item / a.heads;
    const Rows r = sequence_rows(a.offsets, a.tokens, s, seg.shift);
    const uint64_t cells = (uint64_t)a.key_dim * a.value_dim;
    const uint32_t segments = (uint32_t)(((uint64_t)(r.hi - r.lo) + (1ull << seg.shift) - 1u) >> seg.shift);
    if (segments < 2u) return;
    const bool works = wave < kKeys;
    auto number = [&](uint32_t i) { return (uint64_t)(r.base + (BACK ? segments - 1u - i : i)) * a.heads + head; };
    auto each = [&](auto f) {  // f(columns, half, row of the four, whether it is there, offset)
#pragma unroll
        for (uint32_t ct = 0; ct < CT; ++ct)
#pragma unroll
            for (uint32_t h = 0; h < 2u; ++h)
#pragma unroll
                for (uint32_t i = 0; i < 4u; ++i) {
                    const uint32_t row = place(2u * wave + h, 4u * q + i), col = col0 + 16u * ct + m;
                    const bool is = works && row < a.key_dim && col < a.value_dim;
                    f(ct, h, i, is, row * a.value_dim + col);
                }
    };
    f32x4 S[CT][2], N[CT][2];
    auto load = [&](f32x4 (&to)[CT][2], const float *from) {
        each([&](uint32_t ct, uint32_t h, uint32_t i, bool is, uint32_t at) { to[ct][h][i] = from && is ? from[at] : 0.0f; });
    };
    Mid mat[2][kAhead];
    float back[2][kAhead];
    auto fetch = [&](uint32_t i, uint32_t h, uint32_t c) {
        const SegmentMatrix<T, W> &from = static_cast<const SegmentMatrix<T, W> *>(seg.m)[number(i)];
        const uint32_t t = 2u * wave + h;
        mat[h][c % kAhead] = from.m[t][c][lane];
        back[h][c % kAhead] = kScaled ? from.back[t][c] : 1.0f;
    };
    load(S, start ? start + ((uint64_t)s * a.heads + head) * cells : nullptr);
    each([&](uint32_t ct, uint32_t h, uint32_t i, bool, uint32_t) { S[ct][h][i] = finite_or_nan(S[ct][h][i]); });
    load(N, seg.n + number(0u) * cells);
    if (works)
#pragma unroll
        for (uint32_t c = 0; c < kAhead; ++c) fetch(0u, 0u, c), fetch(0u, 1u, c);
    for (uint32_t i = 0; i + 1u < segments; ++i) {
        const uint32_t b = i & 1u;
        if (works) {
            float most = 0.0f;
            if (kScaled)
#pragma unroll
                for (uint32_t ct = 0; ct < CT; ++ct) most = __builtin_fmaxf(most, largest(S[ct]));
            const Scale of = scale_of<kScaled>(kScaled ? wave_largest(most) : 0.0f);
#pragma unroll
            for (uint32_t ct = 0; ct < CT; ++ct) operands[b][wave][ct][lane] = operand_of<Mid>(S[ct][0], S[ct][1], of.by);
            if (lane == 0u) backs[b][wave] = of.back;
        }
        __syncthreads();  // two sets of operands: those of the step before may still be read
        if (works) {
#pragma unroll
            for (uint32_t ct = 0; ct < CT; ++ct) S[ct][0] = N[ct][0], S[ct][1] = N[ct][1];
#pragma unroll
            for (uint32_t c = 0; c < kKeys; ++c) {
                const float from = backs[b][c];
#pragma unroll
                for (uint32_t ct = 0; ct < CT; ++ct) {
                    const Mid h = operands[b][c][ct][lane];
#pragma unroll
                    for (uint32_t t = 0; t < 2u; ++t) {
                        f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma(sum, mat[t][c % kAhead], h);
                        S[ct][t] += sum * (back[t][c % kAhead] * from);
                    }
                }
                if (c + kAhead < kKeys) fetch(i, 0u, c + kAhead), fetch(i, 1u, c + kAhead);
                else if (i + 2u < segments) fetch(i + 1u, 0u, c + kAhead - kKeys), fetch(i + 1u, 1u, c + kAhead - kKeys);
            }
            float *n = seg.n + number(i + 1u) * cells;
            if (i + 2u < segments) load(N, n);
            each([&](uint32_t ct, uint32_t h, uint32_t j, bool is, uint32_t at) {
                if (is) n[at] = S[ct][h][j];
            });
        }
    }
}

// Bytes of a segment's M.
template <class T>
inline size_t matrix_bytes(uint32_t key_dim) {
    size_t n = 0;
    with_key_width(key_dim, [&](auto w) {
        n = sizeof(SegmentMatrix<T, decltype(w)::value>);
        return PS_OK;
    });
    return n;
}

// Rows of a segment, as a shift: as many as take the least time by what the
// parts of a call were measured to take (us; bf16, 128 keys and columns, where 256
// workgroups run at once): a step of a walk 4.3, of the walks for M and N 2.7,
// the start of either 7, a link 2.2.  Other types and widths take other times in
// about the same proportions: with each shift tried, the chosen one was within 4% of
// the best, in us for 8191 rows of 16 heads in one sequence (in brackets walked
// whole): 128 x 128 219 (460), fp32 476 (1275); 64 x 64 137 (352), fp32 202 (709);
// 256 x 256 616 (871), fp32 2030 (3113); 16384 rows in four sequences, 128 x 128,
// fp32 737 (809).
// A call knows how many rows and sequences it has, not where they are cut, which is on
// the device: they are reckoned to be cut at random, and the longest of n is then
// the mean times 1 + 1/2 + ... + 1/n.  One long sequence among many short ones may be
// walked whole for that: 12000 of 16384 rows, 19 others, 16 heads, 128 x 128, bf16,
// 768 us, where segments of 1024 rows would take 415.
uint32_t segment_shift(const DeltaArgs &a) {
    constexpr uint32_t cols = 16u * kWalkWaves;
    const double chunks = (double)ceil_div(a.tokens, kChunk), heads = a.heads, n = a.num_seqs;
    const double value_blocks = (double)ceil_div(a.value_dim, cols), key_blocks = (double)ceil_div(a.key_dim, cols);
    double longest = 0.0;
    for (uint32_t i = 1; i <= a.num_seqs && i <= 64u; ++i) longest += 1.0 / i;
    longest *= chunks / n;
    longest = longest > chunks ? chunks : longest;
    auto rounds = [](double groups) { return groups > 256.0 ? groups / 256.0 : 1.0; };
    const double work = (chunks + 0.5 * (n - 1.0)) * heads * value_blocks / 256.0;
    double best = 7.0 + 4.3 * (longest > work ? longest : work);
    uint32_t shift = 31u;
    for (uint32_t by = 2u; by <= 7u; ++by) {
        const double rows = (double)(1u << by), segments = __builtin_ceil(chunks / rows) + 0.5 * (n - 1.0);
        if (longest < 2.0 * rows) break;
        const double led = segments > n ? segments - n : 1.0;
        const double cost = rounds(segments * heads * value_blocks) * (7.0 + 4.3 * rows) +
                            rounds(led * heads * (value_blocks + key_blocks)) * (7.0 + 2.7 * rows) + 2.2 * longest / rows + 6.0;
        if (cost < best) best = cost, shift = kChunkShift + by;
    }
    return shift;
}

}  // namespace

template <class T>
ps_status delta_forward(void *ws, size_t *ws_bytes, const ps_delta_input *in, void *out, float *final, float *checkpoints,
                        hipStream_t s) {
    const DeltaArgs a = delta_args(in);
    PlainWs plan;
    const size_t prepared_at = plan.take((size_t)a.slots * a.heads * sizeof(Prepared<T>));
    Segments seg{};
    seg.shift = segment_shift(a);
    const uint64_t segments = chunk_slots(a.tokens, a.num_seqs, seg.shift), cells = (uint64_t)a.key_dim * a.value_dim;
    const uint64_t linked = seg.shift < 31u ? segments * a.heads : 0u;
    const size_t m_at = plan.take(linked * matrix_bytes<T>(a.key_dim)), n_at = plan.take(linked * cells * 4u);
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
    Prepared<T> *prepared = ws_at<Prepared<T>>(ws, prepared_at);
    float *rhos = checkpoints ? checkpoints + (uint64_t)a.slots * a.heads * cells : nullptr;
    float *sizes = checkpoints ? rhos + (uint64_t)a.slots * a.heads * kChunk * a.value_dim : nullptr;
    return with_key_width(a.key_dim, [&](auto w) {
        constexpr int W = decltype(w)::value;
        timing_begin(s);
        launch_in_parts((uint64_t)a.slots * a.kheads, 1u, 256u, [&](uint32_t first, uint32_t grid) {
            hipLaunchKernelGGL((delta_prepare_kernel<T, W, false>), dim3(grid), dim3(256), 0, s, a, first, prepared,
                               ws_counter(ws), plan.words());
        });
        seg.m = ws_at<void *>(ws, m_at), seg.n = ws_at<float>(ws, n_at);
        const WalkResults to = {out, final, checkpoints, rhos, sizes};
        auto walk = [&](auto eights) {
            constexpr bool E = decltype(eights)::value;
            const uint64_t blocks = ceil_div(a.value_dim, 16u * kWalkWaves), all = blocks + ceil_div(a.key_dim, 16u * kWalkWaves);
            if (linked) {
                launch_in_parts(segments * a.heads, all, 64u * (kWalkWaves + 4), [&](uint32_t first, uint32_t grid) {
                    hipLaunchKernelGGL((delta_walk_kernel<T, W, E, true>), dim3(grid), dim3(64 * (kWalkWaves + 4)), 0, s, a,
                                       first, prepared, seg, to);
                });
                const uint64_t columns = ceil_div(a.value_dim, Link<W>::kColumns);
                launch_in_parts((uint64_t)a.num_seqs * a.heads, columns, Link<W>::kThreads, [&](uint32_t first, uint32_t grid) {
                    hipLaunchKernelGGL((delta_link_kernel<T, W, false>), dim3(grid), dim3(Link<W>::kThreads), 0, s, a, first, seg,
                                       a.initial);
                });
            }
            launch_in_parts(segments * a.heads, blocks, 64u * (kWalkWaves + 4), [&](uint32_t first, uint32_t grid) {
                hipLaunchKernelGGL((delta_walk_kernel<T, W, E, false>), dim3(grid), dim3(64 * (kWalkWaves + 4)), 0, s, a,
                                   first, prepared, seg, to);
            });
        };
        // rows of whole vectors of 8 have no bounds within one: 8192 rows of 16 heads,
        // 128 keys, bf16, with checkpoints 285 us for 128 columns, 396 for 124 (more
        // than 128 keys in 16 bits, not whole vectors: 62 spilled registers, 65 backwards)
        const bool eights = a.key_dim % 8u == 0u && a.value_dim % 8u == 0u;
        if (eights) walk(std::true_type());
        else walk(std::false_type());
        timing_end(s);
        return launch_status();
    });
}

}  // namespace dwps
