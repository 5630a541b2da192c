// delta_back.hpp -- gradients of the gated delta rule over packed sequences.  One
// type of activations a source file.
//
// With D the gradient of the state that leaves a chunk (delta_block.hpp names
// the rest), backwards over the chunks
//   dU = P^T dO + diag(exp(G_C - G)) K D,  omega = (1 + diag(beta) a)^-T dU
//   dR = beta omega = dV
//   D <- e_C D + Q^T diag(scale e) dO - K^T diag(e) dR
// is a walk like the forward one, with the same segments.  It leaves D and
// omega, from which every chunk finds its own gradients:
//   dbeta = rho omega (summed over columns)
//   dqk_ij = scale exp(G_i - G_j) dO_i U_j (j <= i),  dkk_ij = -exp(G_i - G_j) dR_i U_j (j < i)
//   dQ = scale e dO S^T + dqk K
//   dK = -e dR S^T + exp(G_C - G) U D^T + dkk K + dqk^T Q + dkk^T K
// Every exp(G_i - G_j) holds the g of the rows t with j < t <= i, e_i those up to
// i, exp(G_C - G_j) those after j, so with z_ij = dqk_ij q_i k_j + dkk_ij k_i k_j
//   dg_t = sum_{j < t <= i} z_ij + sum_{i >= t} e_i (scale q_i S dO_i - k_i S dR_i)
//        + sum_{j < t} exp(G_C - G_j) k_j D u_j + e_C <S, D>
// as they stand: no term is added that another takes away.
#pragma once

#include "delta_walk.hpp"

namespace dwps {
namespace {

struct BackResults {
    const float *dfinal;  // [num_seqs, heads, key_dim, value_dim] or NULL
    float *dinitial;      // the same, or NULL
    float *dstates;       // [chunk numbers, heads, key_dim, value_dim]: D
    float *omega;         // [chunk numbers, heads, kChunk, value_dim]
    float *sizes;         // [chunk numbers, heads, kBackSizes]: the largest of `dstates`, `omega` and dout
};
constexpr uint32_t kBackSizes = 3u * kSizeWaves;

// The walk backwards.  lead: the walks for M and N of segments that are not a
// sequence's first, which keep nothing but their end.  Bound like the walk
// forwards: 8192 rows of 16 heads, 128 x 128, bf16, in four sequences, 98 us, and
// as much for M and N.
template <class T, int W, bool E>
__global__ __launch_bounds__(64 * (kWalkWaves + 4)) void delta_walk_back_kernel(DeltaArgs a, uint32_t first, const Prepared<T> *__restrict__ prepared,
                                                              Segments seg, const T *__restrict__ dout, bool lead, BackResults to) {
    typedef typename Form<T>::Mid Mid;
    typedef typename Form<T>::In In;
    typedef WalkTile<T, W> Tile;
    constexpr uint32_t kTiles = W / 16, kCols = Tile::kCols;
    constexpr bool kTwo = 2u * sizeof(Tile) <= kMostShared, kV = kValuesFit<T, W>;
    __shared__ __attribute__((aligned(16))) char memory[kTwo ? 2u * sizeof(Tile) : walk_tile_bytes<T, W>()];
    const uint32_t value_blocks = (a.value_dim + kCols - 1u) / kCols, key_blocks = lead ? (a.key_dim + kCols - 1u) / kCols : 0u;
    const uint32_t blocks = value_blocks + key_blocks, block = blockIdx.x % blocks, item = first + blockIdx.x / blocks;
    const uint32_t head = item % a.heads, number = item / a.heads, khead = head / (a.heads / a.kheads);
    const uint32_t wave = wave_number(), lane = threadIdx.x & 63u, m = lane & 15u, q = lane >> 4;
    const bool unit = block < key_blocks;  // columns of M
    const uint32_t block0 = (block - (unit ? 0u : key_blocks)) * kCols, width = unit ? a.key_dim : a.value_dim;
    const Chunk r = find_chunk(a.offsets, a.num_seqs, a.tokens, seg.shift, number);
    const Rows seq = sequence_rows(a.offsets, a.tokens, r.seq, kChunkShift);
    if (r.index == kNoChunk || (r.lo == r.hi && r.index != 0u) || (lead && r.lo == seq.lo)) return;
    const uint32_t chunks = (r.hi - r.lo + kChunk - 1u) / kChunk;
    const uint32_t base = seq.base + ((r.lo - seq.lo) >> kChunkShift);
    const T *grads = dout + (uint64_t)head * a.value_dim;
    const int64_t grads_stride = (int64_t)a.heads * a.value_dim;
    const DeltaFeed<T, W, E> feed = {a, prepared, r, base, head, khead, block0, grads, grads_stride};
    auto tile = [&](uint32_t i) { return reinterpret_cast<Tile *>(memory + (kTwo && (i & 1u) ? sizeof(Tile) : 0u)); };
    if (wave >= (uint32_t)kWalkWaves) {
        feed.template run<false>(chunks, !unit, tile, [&](uint32_t i) { return chunks - 1u - i; });
        if (unit)
            store_matrix<T, W>(static_cast<SegmentMatrix<T, W> *>(seg.m)[(uint64_t)number * a.heads + head],
                                   reinterpret_cast<float *>(memory), nullptr, 1.0f, block0, a.key_dim, wave, lane, false);
        return;
    }
    const uint32_t here = wave * 16u, col0 = block0 + here, col = col0 + m;
    const uint64_t cells = (uint64_t)a.key_dim * a.value_dim;
    constexpr bool kScaled = Form<T>::scaled;
    f32x4 D[kTiles];  // times `unit_of`, the gradients of the states
    float unit_of = 1.0f;
    {
        const float *from = nullptr;
        if (!lead && r.hi != seq.hi) from = seg.n + ((uint64_t)number * a.heads + head) * cells;
        else if (!lead && to.dfinal) from = to.dfinal + ((uint64_t)r.seq * a.heads + head) * cells;
        load_states<E>(D, from, a.key_dim, a.value_dim, col, q);
        if (unit) unit_states(D, col, q);
    }
    __syncthreads();
    for (uint32_t i = 0; i < chunks; ++i) {
        const uint32_t c = chunks - 1u - i, lo = r.lo + c * kChunk, rows = r.hi - lo < kChunk ? r.hi - lo : kChunk;
        const Tile &in = *tile(i);
        if (col0 < width) {
            if (!lead)
                store_states<E>(to.dstates + ((uint64_t)(base + c) * a.heads + head) * cells, D, unit_of, a.key_dim, a.value_dim,
                                col, q);
            const float most = kScaled ? wave_largest(largest(D)) : 0.0f;
            const Scale of_d = scale_of<kScaled>(most);
            f32x4 x[4], y[4], o[4];  // o: dO
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = y[t] = o[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            // dU = exp(G_C - G) K D + P^T dO
            In ka[4];
            auto keys = [&](uint32_t s) {
#pragma unroll
                for (uint32_t t = 0; t < 4u; ++t) ka[t] = in.k.along(16u * t + m, 32u * s + 8u * q);
            };
            keys(0u);
#pragma unroll
            for (uint32_t s = 0; s < kTiles / 2u; ++s) {
                mma_rows(x, ka, operand_of<Mid>(D[2u * s], D[2u * s + 1u], of_d.by));
                if (s + 1u < kTiles / 2u) keys(s + 1u);
            }
            RowNumbers tail;
            tail.load(in.p.row + kRowTail, q);
            Triangle<Mid> tri;
            if (!unit) {
                if constexpr (kV) {
#pragma unroll
                    for (uint32_t t = 0; t < 4u; ++t) o[t] = value_rows<T>(in.v, t, q, m, here);
                } else {
#pragma unroll
                    for (uint32_t t = 0; t < 4u; ++t)
#pragma unroll
                        for (uint32_t j = 0; j < 4u; ++j) {
                            const uint32_t row = 16u * t + 4u * q + j;
                            o[t][j] = row < rows && col < a.value_dim ? finite_or_nan((float)grads[(int64_t)(lo + row) * grads_stride + col]) : 0.0f;
                        }
                }
                tri.load(in.p.scores, lane);
            }
            __builtin_amdgcn_sched_barrier(0);
            const float most_o = kScaled ? wave_largest(largest(o)) : 0.0f;
            const Scale of_o = scale_of<kScaled>(most_o);
            // K D and P^T dO are summed with their scales taken back: where dO and the
            // scores are zero or small, theirs would take K D past fp32's range
            const float from_p = kScaled ? of_o.back * in.p.row[kRowScores] : 1.0f, from_d = of_d.back * unit_of;
#pragma unroll
            for (uint32_t t = 0; t < 4u; ++t) x[t] *= tail.of[t] * from_d;
            if (!unit) {
                f32x4 p[4];
#pragma unroll
                for (uint32_t t = 0; t < 4u; ++t) p[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                const In h[2] = {operand_of<In>(o[0], o[1], of_o.by), operand_of<In>(o[2], o[3], of_o.by)};
                mma_upper(p, tri, h);
#pragma unroll
                for (uint32_t t = 0; t < 4u; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[t][j] = __builtin_fmaf(p[t][j], from_p, x[t][j]);
            }
            tri.load(in.p.inverse, lane);
            const float inverse_back = in.p.row[kRowInverse], kept = unit_of * in.p.row[kRowWhole];
            __builtin_amdgcn_sched_barrier(0);
            // omega
            const Scale of_x = scale_of<kScaled>(kScaled ? wave_largest(largest(x)) : 0.0f);
            const float from_y = kScaled ? of_x.back * inverse_back : 1.0f;
            {
                const Mid h[2] = {operand_of<Mid>(x[0], x[1], of_x.by), operand_of<Mid>(x[2], x[3], of_x.by)};
                mma_upper(y, tri, h);
            }
            if (!lead) {
                if (kScaled) {
                    const float of_y = wave_largest(largest(y)) * from_y;
                    float *sizes = to.sizes + ((uint64_t)(base + c) * a.heads + head) * kBackSizes + col0 / 16u;
                    if (lane == 0u) sizes[0] = most * unit_of, sizes[kSizeWaves] = of_y, sizes[2u * kSizeWaves] = most_o;
                }
                if (col < a.value_dim)
                    store_rows(to.omega + ((uint64_t)(base + c) * a.heads + head) * kChunk * a.value_dim, a.value_dim, y, from_y, col, q);
            }
            // D = e_C D + Q^T diag(scale e) dO - K^T diag(e) beta omega
            __builtin_amdgcn_sched_barrier(0);
            RowNumbers e, eq;
            e.load(in.p.row + kRowE, q);
            eq.load(in.p.row + kRowQ, q);
#pragma unroll
            for (uint32_t t = 0; t < 4u; ++t) {
                y[t] *= e.of[t] * -from_y;
                o[t] *= eq.of[t];
            }
            const Scale of_y = scale_of_sum<kScaled>(
                kScaled ? wave_largest(__builtin_fmaxf(largest(y), largest(o))) : 0.0f, most * kept);
#pragma unroll
            for (uint32_t t = 0; t < kTiles; ++t) D[t] *= kept * of_y.by;
            unit_of = of_y.back;
            mma_keys(D, in.k, 0u, operand_of<Mid>(y[0], y[1], of_y.by), lane);
            mma_keys(D, in.k, 1u, operand_of<Mid>(y[2], y[3], of_y.by), lane);
            if (!unit) {
                mma_keys(D, in.q, 0u, operand_of<Mid>(o[0], o[1], of_y.by), lane);
                mma_keys(D, in.q, 1u, operand_of<Mid>(o[2], o[3], of_y.by), lane);
            }
        }
        if (!kTwo) __syncthreads();
        __syncthreads();
    }
    const uint64_t place_of = (uint64_t)number * a.heads + head;
    if (unit) {
        store_matrix<T, W>(static_cast<SegmentMatrix<T, W> *>(seg.m)[place_of], reinterpret_cast<float *>(memory), &D, unit_of,
                               block0, a.key_dim, wave, lane, true);
        return;
    }
    if (col0 >= width) return;
    if (lead) store_states<E>(seg.n + place_of * cells, D, unit_of, a.key_dim, a.value_dim, col, q);
    else if (to.dinitial && r.lo == seq.lo)
        store_states<E>(to.dinitial + ((uint64_t)r.seq * a.heads + head) * cells, D, unit_of, a.key_dim, a.value_dim, col, q);
}

// ---------------------------------------------------------------------------
// a chunk's own gradients
// ---------------------------------------------------------------------------
struct DeltaGradPtrs {
    void *dq, *dk, *dv;
    float *dg, *dbeta;
};

__device__ __forceinline__ double shuffle(double v, uint32_t from) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute((int)(from * 4u), (int)(uint32_t)b);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_bpermute((int)(from * 4u), (int)(uint32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float shuffle(float v, uint32_t from) {
    return __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute((int)(from * 4u), __builtin_bit_cast(int, v)));
}
// The sum over the four lanes of a column, in every one of them.
__device__ __forceinline__ float column_total(float v) {
    float w = v;
    swap_rows(v, w);
    v += w;
    w = v;
    swap_halves(v, w);
    return v + w;
}

// 32 columns of a chunk's rows.
template <class T>
struct GradColumns {
    RowTile<typename Form<T>::In, 32> dout;
    RowTile<typename Form<T>::Mid, 32> rho, omega;
};
// Sums over keys of a chunk's rows, by wave.
struct GradSums {
    float query[8][kChunk], key[8][kChunk], end[8][kChunk], pair[8][kChunk];
};
template <class T, int W>
struct GradShared {
    static constexpr size_t kFixed = 2u * sizeof(KeyTile<T, W>) + 2048u;
    // two sets of columns, and the sums in memory of their own, where there is room
    static constexpr bool kTwo = kFixed + 2u * sizeof(GradColumns<T>) + sizeof(GradSums) <= kMostShared;
    static constexpr bool kApart = kTwo;
    KeyTile<T, W> k, q;
    union {
        GradColumns<T> in[kTwo ? 2 : 1];
        typename Form<T>::Mid triangle[2][kTriangle][64];
        GradSums within;
    };
    GradSums apart[kApart ? 1 : 0];
    double sum[kChunk];
    float beta[kChunk], nu[kChunk], mu[kChunk], dot[8], most[8];
    __device__ __forceinline__ GradSums &part() {
        if constexpr (kApart) return apart[0];
        else return within;
    }
};

// One workgroup a chunk and head of keys; it takes the heads of values that
// share them in turn and adds their gradients in registers.  A wave has DT tiles
// of 16 keys for TT tiles of 16 rows, a row in a lane and its keys in the
// registers.  Of the 64 x 64 products waves 0 to 3 have dO rho^T, waves 4 to 7
// omega rho^T: wave w the columns of tile w & 3 of the lower triangle as it is
// (five, slots up to w: rows j, columns i) and transposed (slots above: rows
// i, columns j), so that both are operands as they come.
// Bound by latency: 108 KB of shared memory and 240 registers leave a CU one
// workgroup, whose parts wait for one another.  8192 rows of 16 heads, 128 x 128,
// bf16: 300 us for 364 MB, of which start and end 80, the sums over columns 136,
// the triangles 83; in half the registers it spills (596 us).  SOLO, heads that
// share no keys, adds up nothing over heads (27 us more with the sums, which spill 13
// to 29 registers at 128 keys).  More than 128 keys spill 76 to 285.
template <class T, int W, bool E, bool SOLO>
__global__ __launch_bounds__(512) void delta_grads_kernel(DeltaArgs a, uint32_t first, const T *__restrict__ dout,
                                                          const float *__restrict__ states, const float *__restrict__ rhos,
                                                          const float *__restrict__ sizes, const float *__restrict__ dstates,
                                                          const float *__restrict__ omega, const float *__restrict__ back_sizes,
                                                          uint32_t size_waves, DeltaGradPtrs to) {
    typedef typename Form<T>::Mid Mid;
    constexpr bool kScaled = Form<T>::scaled;
    constexpr uint32_t DT = W > 128 ? W / 128 : 1, TT = W >= 128 ? 4 : W / 32, kTiles = W / 16;
    __shared__ GradShared<T, W> sh;
    const uint32_t item = first + blockIdx.x, slot = item / a.kheads, khead = item % a.kheads;
    const Chunk c = find_chunk(a.offsets, a.num_seqs, a.tokens, kChunkShift, slot);
    const uint32_t rows = c.hi - c.lo;
    if (rows == 0u) return;
    const uint32_t wave = wave_number();
    uint32_t lane = threadIdx.x & 63u, n = lane & 15u, q = lane >> 4;
    const uint32_t tile0 = W >= 128 ? wave * DT : wave % kTiles, t0 = W >= 128 ? 0u : wave / kTiles * TT;
    const uint32_t own_tile = wave & 3u;
    uint32_t own = 16u * own_tile + n;
    const bool keys_side = wave >= 4u;  // omega rho^T and k k^T, not dO rho^T and q k^T
    uint32_t row = threadIdx.x >> 3, part = (threadIdx.x & 7u) * 4u;
    const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
    float raw_nu, raw_mu;
    {
        const float own_nu = fill_rows<T, 8, W>(sh.k, a.k, a.k_stride, khead, c.lo, rows, a, &raw_nu);
        const float own_mu = fill_rows<T, 8, W>(sh.q, a.q, a.q_stride, khead, c.lo, rows, a, &raw_mu);
        if ((threadIdx.x & 7u) == 0u) sh.nu[row] = own_nu, sh.mu[row] = own_mu;
    }
    __syncthreads();
    f32x4 dq[DT][TT], dk[DT][TT];  // with respect to the keys and queries of length 1
    if (!SOLO)
#pragma unroll
        for (uint32_t d = 0; d < DT; ++d)
#pragma unroll
            for (uint32_t t = 0; t < TT; ++t) dq[d][t] = dk[d][t] = none;
    const uint32_t per = SOLO ? 1u : a.heads / a.kheads;
    const uint64_t cells = (uint64_t)a.key_dim * a.value_dim;
    for (uint32_t j = 0; j < per; ++j) {
        const uint32_t head = khead * per + j;
        // what follows from a lane's number is found anew for each head: kept over
        // the heads it takes the registers that the sums need
        asm volatile("" : "+v"(n), "+v"(q), "+v"(own), "+v"(lane), "+v"(row), "+v"(part));
        const uint64_t of_head = (uint64_t)slot * a.heads + head, at_row = ((uint64_t)(c.lo + row) * a.heads + head) * a.value_dim;
        const float *state = states + of_head * cells, *dstate = dstates + of_head * cells;
        // the next 32 columns of the rows, on their way while some are worked on
        f32x4 next_rho, next_omega, next_dout;
        float next_s[DT][8], next_d[DT][8];
        auto fetch = [&](uint32_t v0) {
#pragma unroll
            for (uint32_t d = 0; d < DT; ++d) {
                const uint32_t key = 16u * (tile0 + d) + n, col = v0 + 8u * q;
                const bool there = key < a.key_dim && col < a.value_dim;
                const uint32_t at = there ? key * a.value_dim + col : 0u;
                if (E || (there && col + 8u <= a.value_dim)) {
                    const Pack<float, 8> ps = *reinterpret_cast<const Pack<float, 8> *>(state + at);
                    const Pack<float, 8> pg = *reinterpret_cast<const Pack<float, 8> *>(dstate + at);
#pragma unroll
                    for (int i = 0; i < 8; ++i) next_s[d][i] = there ? ps.v[i] : 0.0f, next_d[d][i] = there ? pg.v[i] : 0.0f;
                } else {
#pragma unroll
                    for (uint32_t i = 0; i < 8u; ++i) {
                        const bool is = there && col + i < a.value_dim;
                        next_s[d][i] = is ? state[at + i] : 0.0f;
                        next_d[d][i] = is ? dstate[at + i] : 0.0f;
                    }
                }
            }
            const bool there = row < rows && v0 + part < a.value_dim;
            const uint64_t at = there ? at_row + v0 + part : ((uint64_t)c.lo * a.heads + head) * a.value_dim;
            const uint64_t kept = of_head * kChunk * a.value_dim + (there ? row * a.value_dim + v0 + part : 0u);
            if (E || (there && v0 + part + 4u <= a.value_dim)) {
                next_rho = __builtin_bit_cast(f32x4, *reinterpret_cast<const Pack<float, 4> *>(rhos + kept));
                next_omega = __builtin_bit_cast(f32x4, *reinterpret_cast<const Pack<float, 4> *>(omega + kept));
                const Pack<T, 4> o = *reinterpret_cast<const Pack<T, 4> *>(dout + at);
#pragma unroll
                for (int i = 0; i < 4; ++i) next_dout[i] = (float)o.v[i];
                if (!there) next_rho = next_omega = next_dout = none;
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 4u; ++i) {
                    const bool is = there && v0 + part + i < a.value_dim;
                    next_rho[i] = is ? rhos[kept + i] : 0.0f;
                    next_omega[i] = is ? omega[kept + i] : 0.0f;
                    next_dout[i] = is ? (float)dout[at + i] : 0.0f;
                }
            }
        };
        fetch(0u);
        const double sums = running_decay(a, head, c.lo, rows, lane);
        const float own_beta = row < rows ? a.beta[(int64_t)(c.lo + row) * a.beta_stride + head] : 0.0f;
        Scale of_s = {1.0f, 1.0f}, of_d = of_s, of_rho = of_s, of_omega = of_s, of_o = of_s;
        if constexpr (kScaled) {
            const bool has = lane < size_waves;
            const float *f = sizes + of_head * kSizes + lane, *b = back_sizes + of_head * kBackSizes + lane;
            of_s = scale_of<true>(wave_largest(has ? f[0] : 0.0f));
            of_rho = scale_of<true>(wave_largest(has ? f[kSizeWaves] : 0.0f));
            of_d = scale_of<true>(wave_largest(has ? b[0] : 0.0f));
            of_omega = scale_of<true>(wave_largest(has ? b[kSizeWaves] : 0.0f));
            of_o = scale_of<true>(wave_largest(has ? b[2u * kSizeWaves] : 0.0f));
        }
        __syncthreads();  // the head before is done with
        if (wave == 0u) sh.sum[lane] = sums;
        if ((threadIdx.x & 7u) == 0u) sh.beta[row] = own_beta;
        f32x4 qs[DT][TT], rs[DT][TT], ends[DT][TT], e[5];
#pragma unroll
        for (uint32_t d = 0; d < DT; ++d)
#pragma unroll
            for (uint32_t t = 0; t < TT; ++t) qs[d][t] = rs[d][t] = ends[d][t] = none;
#pragma unroll
        for (int t = 0; t < 5; ++t) e[t] = none;
        float dot = 0.0f, dbeta = 0.0f;
        for (uint32_t v0 = 0; v0 < a.value_dim; v0 += 32u) {
            if (!GradShared<T, W>::kTwo && v0) __syncthreads();  // the columns before are read
            GradColumns<T> &in = sh.in[GradShared<T, W>::kTwo ? v0 >> 5 & 1u : 0u];
#pragma unroll
            for (int i = 0; i < 4; ++i) dbeta = __builtin_fmaf(next_rho[i], next_omega[i], dbeta);
            if (row < rows) {
                T *p = static_cast<T *>(to.dv) + at_row + v0 + part;
                Pack<T, 4> w;
#pragma unroll
                for (int i = 0; i < 4; ++i) w.v[i] = (T)(own_beta * next_omega[i]);
                if (E ? v0 + part < a.value_dim : v0 + part + 4u <= a.value_dim) {
                    *reinterpret_cast<Pack<T, 4> *>(p) = w;
                } else if (!E) {
#pragma unroll
                    for (uint32_t i = 0; i < 4u; ++i)
                        if (v0 + part + i < a.value_dim) p[i] = w.v[i];
                }
            }
            in.dout.put(row, part, next_dout, of_o.by);
            in.rho.put(row, part, next_rho, of_rho.by);
            in.omega.put(row, part, next_omega, of_omega.by);
            Mid S[DT], D[DT];
#pragma unroll
            for (uint32_t d = 0; d < DT; ++d) {
                if (t0 == 0u)
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(next_s[d][i], next_d[d][i], dot);
                operand_of(S[d], next_s[d], of_s.by);
                operand_of(D[d], next_d[d], of_d.by);
            }
            if (v0 + 32u < a.value_dim) fetch(v0 + 32u);
            __syncthreads();
#pragma unroll
            for (uint32_t t = 0; t < TT; ++t) {
                const uint32_t at = 16u * (t0 + t) + n;
                const auto o = in.dout.along(at, 8u * q);
                const auto w = in.omega.along(at, 8u * q), r = in.rho.along(at, 8u * q);
#pragma unroll
                for (uint32_t d = 0; d < DT; ++d) {
                    mma(rs[d][t], S[d], w);
                    mma(ends[d][t], D[d], r);
                    mma(qs[d][t], S[d], o);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            const auto own_r = in.rho.along(own, 8u * q);
            if (keys_side) {
                const auto own_w = in.omega.along(own, 8u * q);
#pragma unroll
                for (uint32_t t = 0; t < 4u; ++t) {
                    if (t <= own_tile) mma(e[t], in.rho.along(16u * t + n, 8u * q), own_w);
                    if (t >= own_tile) mma(e[t + 1], in.omega.along(16u * t + n, 8u * q), own_r);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                const auto own_o = in.dout.along(own, 8u * q);
#pragma unroll
                for (uint32_t t = 0; t < 4u; ++t) {
                    if (t <= own_tile) mma(e[t], in.rho.along(16u * t + n, 8u * q), own_o);
                    if (t >= own_tile) mma(e[t + 1], in.dout.along(16u * t + n, 8u * q), own_r);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        dbeta = neighbours_sum<8>(dbeta);
        if (row < rows && (threadIdx.x & 7u) == 0u) to.dbeta[(uint64_t)(c.lo + row) * a.heads + head] = dbeta;
        dot = wave_total(dot);
        __syncthreads();  // the last columns are read
        if (lane == 0u) sh.dot[wave] = dot;
        const double all = sh.sum[kChunk - 1u];
        // the parts that a state has, their factors, and their sums with q and k
#pragma unroll
        for (uint32_t t = 0; t < 4u; ++t) {
            const uint32_t at = 16u * t + n;
            float query = 0.0f, key = 0.0f, end = 0.0f;
            if (t >= t0 && t < t0 + TT) {
                const double G = sh.sum[at];
                const float grow = exp_hw((float)G), tail = exp_hw((float)(all - G)), be = sh.beta[at];
                const float by_q = a.scale * grow * (of_s.back * of_o.back), by_r = grow * be * (of_s.back * of_omega.back);
                const float by_e = tail * be * (of_d.back * of_rho.back);
#pragma unroll
                for (uint32_t tt = 0; tt < TT; ++tt) {
                    if (t0 + tt != t) continue;
#pragma unroll
                    for (uint32_t d = 0; d < DT; ++d) {
                        const uint32_t col = 16u * (tile0 + d) + 4u * q;
                        const f32x4 kv = sh.k.four(at, col), qv = sh.q.four(at, col);
                        const f32x4 x = qs[d][tt] * by_q, y = rs[d][tt] * by_r, z = ends[d][tt] * by_e;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            query = __builtin_fmaf(qv[i], x[i], query);
                            key = __builtin_fmaf(kv[i], y[i], key);
                            end = __builtin_fmaf(kv[i], z[i], end);
                        }
                        dq[d][tt] = SOLO ? x : dq[d][tt] + x;
                        dk[d][tt] = SOLO ? z - y : dk[d][tt] + (z - y);
                    }
                }
            }
            query = column_total(query), key = column_total(key), end = column_total(end);
            if (q == 0u) {
                sh.part().query[wave][at] = query * sh.mu[at];
                sh.part().key[wave][at] = key * sh.nu[at];
                sh.part().end[wave][at] = end * sh.nu[at];
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // k_j k_i or k_j q_i, rows j in the registers, i = own in the lane
        f32x4 kk[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) kk[t] = none;
#pragma unroll
        for (uint32_t col = 0; col < (uint32_t)W; col += 32u) {
            const auto b = keys_side ? sh.k.along(own, col + 8u * q) : sh.q.along(own, col + 8u * q);
#pragma unroll
            for (uint32_t t = 0; t < 4u; ++t)
                if (t <= own_tile) mma(kk[t], sh.k.along(16u * t + n, col + 8u * q), b);
        }
        // the triangles become dqk or dkk with the factors of what they meet, and
        // the pairs' sums of z
        const double G_own = sh.sum[own];
        const float beta_own = sh.beta[own], with_own = keys_side ? -beta_own * sh.nu[own] : a.scale * sh.mu[own];
        const float back = of_rho.back * (keys_side ? of_omega.back : of_o.back), by_own = back * (keys_side ? -beta_own : a.scale);
        float pairs[16], before = 0.0f;
#pragma unroll
        for (uint32_t t = 0; t < 4u; ++t) {
            float z[4] = {};
            if (t <= own_tile) {
#pragma unroll
                for (uint32_t i = 0; i < 4u; ++i) {
                    const uint32_t at = 16u * t + 4u * q + i;  // j; the lane has i
                    const bool is = keys_side ? at < own : at <= own;
                    const float f = is ? exp_hw((float)(G_own - sh.sum[at])) * sh.beta[at] * sh.nu[at] : 0.0f;
                    z[i] = f * e[t][i] * back * kk[t][i] * with_own;
                    e[t][i] *= f * by_own;
                }
            }
            // sums over the rows before each, this tile's and those of the tiles before
            float upto = 0.0f;
            const float four = (z[0] + z[1]) + (z[2] + z[3]);
#pragma unroll
            for (uint32_t p = 0; p < 3u; ++p) {
                const float v = shuffle(four, n + 16u * p);
                if (q > p) upto += v;
            }
            upto += before;
#pragma unroll
            for (uint32_t i = 0; i < 4u; ++i) {
                pairs[4 * t + i] = 16u * t + 4u * q + i <= own ? upto : 0.0f;
                upto += z[i];
            }
            before += column_total(four);
            __builtin_amdgcn_sched_barrier(0);
        }
        const float pair = row_sums(pairs, lane);  // lane n of quarter q: tile n >> 2, row 4 q + (n & 3)
        sh.part().pair[wave][16u * (n >> 2) + 4u * q + (n & 3u)] = pair;
        const float into_own = back * beta_own * (keys_side ? -1.0f : a.scale);
#pragma unroll
        for (uint32_t t = 0; t < 4u; ++t) {
            if (t < own_tile) continue;
#pragma unroll
            for (uint32_t i = 0; i < 4u; ++i) {
                const uint32_t at = 16u * t + 4u * q + i;  // i; the lane has j
                const bool is = keys_side ? at > own : at >= own;
                const float f = is ? exp_hw((float)(sh.sum[at] - G_own)) : 0.0f;
                e[t + 1][i] *= f * into_own * (keys_side ? sh.beta[at] * sh.nu[at] : sh.mu[at]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kScaled) {
            float m = 0.0f;
#pragma unroll
            for (int t = 0; t < 5; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(e[t][i]));
            m = wave_largest(m);
            if (lane == 0u) sh.most[wave] = m;
        }
        __syncthreads();
        // dqk has a scale of its own for dq, and dkk's too where they meet in dk
        Scale of_e = {1.0f, 1.0f}, of_q = of_e;
        if constexpr (kScaled) {
            auto four = [&](int w) {
                return __builtin_fmaxf(__builtin_fmaxf(sh.most[w], sh.most[w + 1]), __builtin_fmaxf(sh.most[w + 2], sh.most[w + 3]));
            };
            const float m = four(0);
            of_q = scale_of<true, -30>(m);
            of_e = scale_of<true, -30>(__builtin_fmaxf(m, four(4)));
        }
        // the log decays' gradients, from the sums that all waves have left
        auto decays = [&]() {
            if (wave != 0u) return;
            auto sum_of = [&](const float(&p)[8][kChunk]) {
                return ((p[0][lane] + p[1][lane]) + (p[2][lane] + p[3][lane])) + ((p[4][lane] + p[5][lane]) + (p[6][lane] + p[7][lane]));
            };
            double after = (double)sum_of(sh.part().query) - (double)sum_of(sh.part().key), ends_before = sum_of(sh.part().end);
#pragma unroll
            for (uint32_t by = 1u; by < 64u; by *= 2u) {
                const double up = shuffle(after, lane + by), down = shuffle(ends_before, lane - by);
                if (lane + by < 64u) after += up;
                if (lane >= by) ends_before += down;
            }
            float whole = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) whole += sh.dot[w];
            double prior = shuffle(ends_before, lane - 1u);  // up to the row before
            if (lane == 0u) prior = 0.0;
            if (lane < rows)
                to.dg[(uint64_t)(c.lo + lane) * a.heads + head] =
                    (float)(sum_of(sh.part().pair) + after + prior + (double)(exp_hw((float)all) * whole));
        };
        if (!GradShared<T, W>::kApart) decays();
        // dqk K and dkk K, then dqk^T Q and dkk^T K, two triangles in shared memory at a time
        if (kScaled) {
#pragma unroll
            for (uint32_t d = 0; d < DT; ++d)
#pragma unroll
                for (uint32_t t = 0; t < TT; ++t) dq[d][t] *= of_q.by, dk[d][t] *= of_e.by;
        }
#pragma unroll
        for (uint32_t upper = 0; upper < 2u; ++upper) {
            __syncthreads();
#pragma unroll
            for (uint32_t s = 0; s < 2u; ++s) {
                if (upper ? s < (own_tile >> 1) : s > (own_tile >> 1)) continue;
                f32x4 two[2];
#pragma unroll
                for (uint32_t h = 0; h < 2u; ++h) {
                    const uint32_t t = 2u * s + h;
                    const bool there = upper ? t >= own_tile : t <= own_tile;
                    two[h] = there ? e[t + upper] : none;
                }
                sh.triangle[keys_side ? 1 : 0][upper ? upper_at(own_tile, s) : lower_at(own_tile, s)][lane] =
                    operand_of<Mid>(two[0], two[1], upper || keys_side ? of_e.by : of_q.by);
            }
            __syncthreads();
#pragma unroll
            for (uint32_t s = 0; s < 2u; ++s)
#pragma unroll
                for (uint32_t d = 0; d < DT; ++d) {
                    const auto keys = sh.k.columns(s, 16u * (tile0 + d), 4u, lane);
                    const auto queries = upper ? sh.q.columns(s, 16u * (tile0 + d), 4u, lane) : keys;
#pragma unroll
                    for (uint32_t t = 0; t < TT; ++t) {
                        const uint32_t tile = t0 + t;
                        if (upper ? s < (tile >> 1) : s > (tile >> 1)) continue;
                        const uint32_t at = upper ? upper_at(tile, s) : lower_at(tile, s);
                        mma(upper ? dk[d][t] : dq[d][t], queries, sh.triangle[0][at][lane]);
                        mma(dk[d][t], keys, sh.triangle[1][at][lane]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
        }
        if (kScaled) {
#pragma unroll
            for (uint32_t d = 0; d < DT; ++d)
#pragma unroll
                for (uint32_t t = 0; t < TT; ++t) dq[d][t] *= of_q.back, dk[d][t] *= of_e.back;
        }
        if (GradShared<T, W>::kApart) decays();
    }
    __syncthreads();
    if ((threadIdx.x & 7u) == 0u) sh.beta[row] = raw_mu, sh.sum[row] = raw_nu;
    if (a.unit) {
        // dq = mu (dq - q (q dq)) of q by its length
#pragma unroll
        for (uint32_t t = 0; t < 4u; ++t) {
            const uint32_t at = 16u * t + n;
            float query = 0.0f, key = 0.0f;
#pragma unroll
            for (uint32_t tt = 0; tt < TT; ++tt) {
                if (t0 + tt != t) continue;
#pragma unroll
                for (uint32_t d = 0; d < DT; ++d) {
                    const uint32_t col = 16u * (tile0 + d) + 4u * q;
                    const f32x4 kv = sh.k.four(at, col), qv = sh.q.four(at, col);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        query = __builtin_fmaf(qv[i], dq[d][tt][i], query);
                        key = __builtin_fmaf(kv[i], dk[d][tt][i], key);
                    }
                }
            }
            query = column_total(query), key = column_total(key);
            if (q == 0u) sh.part().query[wave][at] = query, sh.part().key[wave][at] = key;
        }
    }
    __syncthreads();
#pragma unroll
    for (uint32_t t = 0; t < TT; ++t) {
        const uint32_t at = 16u * (t0 + t) + n;
        float query = 0.0f, key = 0.0f;
        const float nu = sh.nu[at], mu = sh.mu[at], by_q = sh.beta[at], by_k = (float)sh.sum[at];
        if (a.unit) {
            auto sum_of = [&](const float(&p)[8][kChunk]) {
                return ((p[0][at] + p[1][at]) + (p[2][at] + p[3][at])) + ((p[4][at] + p[5][at]) + (p[6][at] + p[7][at]));
            };
            query = sum_of(sh.part().query) * mu * mu, key = sum_of(sh.part().key) * nu * nu;
        }
        if (at >= rows) continue;
#pragma unroll
        for (uint32_t d = 0; d < DT; ++d) {
            const uint32_t col = 16u * (tile0 + d) + 4u * q;
            if (col >= a.key_dim) continue;
            const f32x4 kv = sh.k.four(at, col), qv = sh.q.four(at, col);
            const uint64_t to_row = ((uint64_t)(c.lo + at) * a.kheads + khead) * a.key_dim + col;
            Pack<T, 4> wq, wk;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wq.v[i] = (T)(by_q * __builtin_fmaf(-qv[i], query, dq[d][t][i]));
                wk.v[i] = (T)(by_k * __builtin_fmaf(-kv[i], key, dk[d][t][i]));
            }
            T *pq = static_cast<T *>(to.dq) + to_row, *pk = static_cast<T *>(to.dk) + to_row;
            if (E || col + 4u <= a.key_dim) {
                *reinterpret_cast<Pack<T, 4> *>(pq) = wq;
                *reinterpret_cast<Pack<T, 4> *>(pk) = wk;
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 4u; ++i)
                    if (col + i < a.key_dim) pq[i] = wq.v[i], pk[i] = wk.v[i];
            }
        }
    }
}

}  // namespace

template <class T>
ps_status delta_backward(void *ws, size_t *ws_bytes, const ps_delta_input *in, const void *dout, const float *dfinal,
                         const float *checkpoints, const ps_delta_grads *grads, hipStream_t s) {
    const DeltaArgs a = delta_args(in);
    PlainWs plan;
    const size_t prepared_at = plan.take((size_t)a.slots * a.heads * sizeof(Prepared<T>));
    Segments seg{};
    seg.shift = segment_shift(a);
    const uint64_t segments = chunk_slots(a.tokens, a.num_seqs, seg.shift), cells = (uint64_t)a.key_dim * a.value_dim;
    const uint64_t linked = seg.shift < 31u ? segments * a.heads : 0u, state_floats = (uint64_t)a.slots * a.heads * cells;
    const size_t m_at = plan.take(linked * matrix_bytes<T>(a.key_dim)), n_at = plan.take(linked * cells * 4u);
    const size_t sizes_at = plan.take((size_t)a.slots * a.heads * kBackSizes * 4u);
    const size_t d_at = plan.take(state_floats * 4u), omega_at = plan.take((size_t)a.slots * a.heads * kChunk * a.value_dim * 4u);
    bool query = false;
    ps_status st = workspace_protocol(ws, ws_bytes, plan.at, &query);
    if (st != PS_OK || query) return st;
    if ((st = delta_pointers(in)) != PS_OK) return st;
    if (!grads) return PS_ERR_NULL;
    if (in->tokens && (!dout || !checkpoints || !grads->dq || !grads->dk || !grads->dv || !grads->dg || !grads->dbeta))
        return PS_ERR_NULL;
    if (!aligned(ws, 16) || !aligned(dout, sizeof(T)) || !aligned(dfinal, 4) || !aligned(checkpoints, 4) ||
        !aligned(grads->dq, sizeof(T)) || !aligned(grads->dk, sizeof(T)) || !aligned(grads->dv, sizeof(T)) ||
        !aligned(grads->dg, 4) || !aligned(grads->dbeta, 4) || !aligned(grads->dinitial, 4))
        return PS_ERR_ALIGNMENT;
    const DeltaBytes n(in);
    const size_t kept = ps_gated_delta_checkpoint_floats(in->tokens, a.num_seqs, a.heads, a.key_dim, a.value_dim) * 4u;
    if (outputs_overlap({{grads->dq, n.keys}, {grads->dk, n.keys}, {grads->dv, n.values}, {grads->dg, n.gates},
                         {grads->dbeta, n.gates}, {grads->dinitial, n.states}},
                        {{in->q, n.q}, {in->k, n.k}, {in->v, n.v}, {in->g, n.g}, {in->beta, n.beta}, {in->offsets, n.offsets},
                         {in->initial, n.states}, {dout, n.values}, {dfinal, n.states}, {checkpoints, kept}}))
        return PS_ERR_ALIAS;
    if (!a.num_seqs) return PS_OK;
    Prepared<T> *prepared = ws_at<Prepared<T>>(ws, prepared_at);
    seg.m = ws_at<void *>(ws, m_at), seg.n = ws_at<float>(ws, n_at);
    float *dstates = ws_at<float>(ws, d_at), *omega = ws_at<float>(ws, omega_at);
    const T *g = static_cast<const T *>(dout);
    float *back_sizes = ws_at<float>(ws, sizes_at);
    const float *rhos = checkpoints + state_floats, *sizes = rhos + (uint64_t)a.slots * a.heads * kChunk * a.value_dim;
    const BackResults to = {dfinal, grads->dinitial, dstates, omega, back_sizes};
    const DeltaGradPtrs out = {grads->dq, grads->dk, grads->dv, grads->dg, grads->dbeta};
    return with_key_width(a.key_dim, [&](auto w) {
        constexpr int W = decltype(w)::value;
        timing_begin(s);
        launch_in_parts((uint64_t)a.slots * a.kheads, 1u, 256u, [&](uint32_t first, uint32_t grid) {
            hipLaunchKernelGGL((delta_prepare_kernel<T, W, true>), dim3(grid), dim3(256), 0, s, a, first, prepared,
                               ws_counter(ws), plan.words());
        });
        auto walk = [&](auto eights) {
            constexpr bool E = decltype(eights)::value;
            const uint64_t blocks = ceil_div(a.value_dim, 16u * kWalkWaves), all = blocks + ceil_div(a.key_dim, 16u * kWalkWaves);
            if (linked) {
                launch_in_parts(segments * a.heads, all, 64u * (kWalkWaves + 4), [&](uint32_t first, uint32_t grid) {
                    hipLaunchKernelGGL((delta_walk_back_kernel<T, W, E>), dim3(grid), dim3(64 * (kWalkWaves + 4)), 0, s, a, first, prepared,
                                       seg, g, true, to);
                });
                const uint64_t columns = ceil_div(a.value_dim, Link<W>::kColumns);
                launch_in_parts((uint64_t)a.num_seqs * a.heads, columns, Link<W>::kThreads, [&](uint32_t first, uint32_t grid) {
                    hipLaunchKernelGGL((delta_link_kernel<T, W, true>), dim3(grid), dim3(Link<W>::kThreads), 0, s, a, first, seg, dfinal);
                });
            }
            launch_in_parts(segments * a.heads, blocks, 64u * (kWalkWaves + 4), [&](uint32_t first, uint32_t grid) {
                hipLaunchKernelGGL((delta_walk_back_kernel<T, W, E>), dim3(grid), dim3(64 * (kWalkWaves + 4)), 0, s, a, first, prepared, seg,
                                   g, false, to);
            });
            launch_in_parts((uint64_t)a.slots * a.kheads, 1u, 512u, [&](uint32_t first, uint32_t grid) {
                auto launch = [&](auto solo) {
                    hipLaunchKernelGGL((delta_grads_kernel<T, W, E, decltype(solo)::value>), dim3(grid), dim3(512), 0, s, a, first, g,
                                       checkpoints, rhos, sizes, dstates, omega, back_sizes,
                                       (uint32_t)ceil_div(a.value_dim, 16u), out);
                };
                if (a.heads == a.kheads) launch(std::true_type());
                else launch(std::false_type());
            });
        };
        const bool eights = a.key_dim % 8u == 0u && a.value_dim % 8u == 0u;
        if (eights) walk(std::true_type());
        else walk(std::false_type());
        timing_end(s);
        return launch_status();
    });
}

}  // namespace dwps
