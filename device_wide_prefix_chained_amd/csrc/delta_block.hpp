// delta_block.hpp -- parts shared by the gated delta rule's kernels: operands
// of the matrix instructions, the tile of a chunk's keys or queries in shared
// memory, and the kernel that prepares a chunk.
//
// A chunk is 64 rows of one sequence, S the state that enters it, G the running
// sum of g in it, e = exp(G), k and q with their factors nu and mu of length 1
// (or 1), and
//   a_ij = exp(G_i - G_j) k_i k_j (j < i),  P_ij = scale exp(G_i - G_j) q_i k_j (j <= i)
//   rho  = (1 + a diag(beta))^-1 (V - e K S),  U = beta rho
//   out  = scale e Q S + P U,  S' = e_C S + K^T diag(exp(G_C - G)) U
// which is the rule S' = exp(g) S, u = beta (v - S'^T k), S = S' + k u^T of one
// row after another, with 64 of the rows' corrections solved for at once.
//
// Operands.  A product's result has a column in a lane (l & 15) and four
// neighbouring rows in its registers (4 (l >> 4) + r); the next product takes
// its right operand with a column in a lane and eight places of the summed
// index, 8 (l >> 4) + j.  The order of the summed index is free as long as both
// operands have the same, so the eight places of a lane are its four rows of
// each of two result tiles, and states, corrections and values never leave the
// registers.  For rows of a chunk that means places in the order of token_at();
// keys are laid over a pair of tiles by place() instead, so that a lane's eight
// keys are neighbours.
//
// Precision.  16-bit activations use the fp16 matrix instruction.  A row of
// keys or queries is one fp16 plane times a power of two that brings its largest
// near 2^15 (whole for fp16 and, down to 2^-21 of the row's largest, for bf16); dout
// is one plane too, by the largest of a wave's columns or of a chunk.
// fp32 numbers that a chunk computes (states, corrections, inverses) are two
// fp16 planes of a common power of two for a wave's tiles, a rounding and the
// rounding of what is left: off by 2^-22 of the number or 2^-39 of the largest,
// against 2^-11 of one plane, for which a product takes 2 or 3 instructions (the
// planes' largest products).  Two planes of bf16 would need no powers of two but
// hold 16 bits: states came out 2 to 3e-6 off (norms; now 2e-7).  All sums are
// fp32, and so is everything kept from chunk to chunk.  fp32 activations use the
// fp32 matrix instruction throughout (a sixteenth of the rate).
#pragma once

#include "block_device.hpp"
#include "chunks.hpp"

namespace dwps {

constexpr uint32_t kChunk = 64u, kChunkShift = 6u;
constexpr size_t kMostShared = 160u * 1024u;  // of a workgroup

typedef f16_t f16x8 __attribute__((ext_vector_type(8)));
typedef f16_t f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint64_t uint64x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ i16x4 read_transposed(const uint16_t *shared) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) i16x4 *)(uintptr_t)(const __attribute__((address_space(3))) uint16_t *)shared);
}

struct DeltaArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const float *g, *beta;
    int64_t g_stride, beta_stride;
    const uint32_t *offsets;
    const float *initial;
    uint32_t tokens, kheads, heads, key_dim, value_dim, num_seqs;
    uint32_t slots;  // numbers of chunks
    uint32_t unit;   // q and k by their lengths
    float scale, eps;
};

// The wave's number in its workgroup, in a scalar register: what depends on it
// is a branch of the wave, not a mask of its lanes.
__device__ __forceinline__ uint32_t wave_number() {
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

// Eight places of an operand: N fp16 planes, or the numbers themselves.
template <int N>
struct Planes {
    f16x8 p[N];
};
struct Wide {
    float p[8];
};

// The operand of eight numbers times `by`: each plane is the rounding of what
// the ones before leave.
template <int N>
__device__ __forceinline__ void operand_of(Planes<N> &o, const float (&v)[8], float by = 1.0f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        o.p[0][j] = (f16_t)(v[j] * by);
        if (N > 1) o.p[N - 1][j] = (f16_t)__builtin_fmaf(v[j], by, -(float)o.p[0][j]);
    }
}
__device__ __forceinline__ void operand_of(Wide &o, const float (&v)[8], float = 1.0f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o.p[j] = v[j];
}
// The operand of two tiles of a result: rows 4 q + r of the first and of the second.
template <class M>
__device__ __forceinline__ M operand_of(const f32x4 &a, const f32x4 &b, float by = 1.0f) {
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    M o;
    operand_of(o, v, by);
    return o;
}

// acc += A B over 32 places: the products of planes i and j with i + j below
// the larger number of planes, smallest first.
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4 &acc, const Planes<NA> &a, const Planes<NB> &b) {
    constexpr int most = NA > NB ? NA : NB;
#pragma unroll
    for (int sum = most - 1; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (sum - i >= 0 && sum - i < NB)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.p[i], b.p[sum - i], acc, 0, 0, 0);
}
// The same for N sums with one left operand or one right operand each: product
// by product over all sums, so that no instruction waits for the one before.
template <int N, int NA, int NB>
__device__ __forceinline__ void mma_rows(f32x4 (&acc)[N], const Planes<NA> (&a)[N], const Planes<NB> &b) {
    constexpr int most = NA > NB ? NA : NB;
#pragma unroll
    for (int sum = most - 1; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (sum - i >= 0 && sum - i < NB)
#pragma unroll
                for (int t = 0; t < N; ++t)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[t].p[i], b.p[sum - i], acc[t], 0, 0, 0);
}
template <int N, int NA, int NB>
__device__ __forceinline__ void mma_columns(f32x4 (&acc)[N], const Planes<NA> &a, const Planes<NB> (&b)[N]) {
    constexpr int most = NA > NB ? NA : NB;
#pragma unroll
    for (int sum = most - 1; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (sum - i >= 0 && sum - i < NB)
#pragma unroll
                for (int t = 0; t < N; ++t)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.p[i], b[t].p[sum - i], acc[t], 0, 0, 0);
}
template <int N>
__device__ __forceinline__ void mma_rows(f32x4 (&acc)[N], const Wide (&a)[N], const Wide &b) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int t = 0; t < N; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[t].p[j], b.p[j], acc[t], 0, 0, 0);
}
template <int N>
__device__ __forceinline__ void mma_columns(f32x4 (&acc)[N], const Wide &a, const Wide (&b)[N]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int t = 0; t < N; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(a.p[j], b[t].p[j], acc[t], 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4 &acc, const Wide &a, const Wide &b) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.p[j], b.p[j], acc, 0, 0, 0);
}

// How activations of type T are held in shared memory and become operands; Mid:
// operands made of computed numbers.
template <class T>
struct Form {
    typedef uint16_t Word;
    static constexpr bool scaled = true;
    typedef Planes<1> In;
    typedef Planes<2> Mid;
};
template <>
struct Form<float> {
    typedef float Word;
    static constexpr bool scaled = false;
    typedef Wide In;
    typedef Wide Mid;
};

// A power of two that brings numbers up to `most` to 2^14 .. 2^15, and its
// reciprocal.  Numbers below 2^least are left small: a product's scale is that
// of both operands, and what is added to it has to stay in fp32's range (least
// -60 for one and -20 for the other leave it 2^17).  Of numbers with an infinity
// among them no power of two keeps the others: the scale is NaN, and so are they.
struct Scale {
    float by, back;
};
template <bool scaled, int least = -60>
__device__ __forceinline__ Scale scale_of(float most) {
    if (!scaled) return {1.0f, 1.0f};
    // exponents as they stand in the words: 2^14 over the largest's
    const uint32_t e = __builtin_bit_cast(uint32_t, __builtin_fmaxf(most, __builtin_ldexpf(1.0f, least))) & 0x7F800000u;
    const uint32_t by = e == 0x7F800000u ? 0x7FC00000u : (268u << 23) - e;
    return {__builtin_bit_cast(float, by), __builtin_bit_cast(float, e - (14u << 23))};
}
// NaN for an infinity: a column that holds one has no finite result, and its
// neighbours, which share its scale, keep theirs.
__device__ __forceinline__ float finite_or_nan(float v) { return __builtin_fmaf(v, 0.0f, v); }
// The same for terms that are added to numbers up to `held`, which take the
// scale with them and must not leave fp32's range for small terms.
template <bool scaled>
__device__ __forceinline__ Scale scale_of_sum(float most, float held) {
    return scale_of<scaled>(__builtin_fmaxf(most, held * 0x1p-24f));
}
// The largest of a lane's tiles.
template <int N>
__device__ __forceinline__ float largest(const f32x4 (&v)[N]) {
    float m[4] = {};
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = __builtin_fmaxf(m[i], __builtin_fabsf(v[t][i]));
    return __builtin_fmaxf(__builtin_fmaxf(m[0], m[1]), __builtin_fmaxf(m[2], m[3]));
}
__device__ __forceinline__ float wave_largest(float v) {
    v = __builtin_fmaxf(v, dpp<kRowMirror>(v));
    v = __builtin_fmaxf(v, dpp<kRowHalfMirror>(v));
    v = __builtin_fmaxf(v, dpp<kQuadSwap2>(v));
    v = __builtin_fmaxf(v, dpp<kQuadSwap1>(v));
    float w = v;
    swap_rows(v, w);
    v = __builtin_fmaxf(v, w);
    w = v;
    swap_halves(v, w);
    return __builtin_fmaxf(v, w);
}

// The key in row m of a state's tile: the 32 keys of a pair of tiles, eight to
// each quarter of the lanes, four of them in each tile.
__device__ __forceinline__ uint32_t place(uint32_t tile, uint32_t m) {
    return 32u * (tile >> 1) + 8u * (m >> 2) + 4u * (tile & 1u) + (m & 3u);
}

// The row of a chunk at place j of lanes 16 q .. of the s-th 32 places: rows
// 4 q + i of tiles 2 s and 2 s + 1.
__device__ __forceinline__ uint32_t token_at(uint32_t s, uint32_t q, uint32_t j) {
    return 32u * s + 16u * (j >> 2) + 4u * q + (j & 3u);
}

// kChunk rows of `W` columns in shared memory, as operands O (one or two planes
// of words, or numbers).  A column of a tile of keys is read across the rows
// with the transposing read, which gives lane m of 16 the m & 3'rd of the four
// words that lanes (m >> 2) + 4 j point at.
template <class O, int W>
struct RowTile;
template <int N, int W>
struct RowTile<Planes<N>, W> {
    static constexpr int kStride = W + 16;  // 32 bytes: the transposing reads of 16 rows meet no bank twice
    uint16_t w[N][kChunk][kStride];
    __device__ __forceinline__ void put(uint32_t row, uint32_t col, const float (&v)[8], float by) {
        Planes<N> o;
        operand_of(o, v, by);
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<f16x8 *>(&w[i][row][col]) = o.p[i];
    }
    __device__ __forceinline__ void put(uint32_t row, uint32_t col, const f32x4 &v, float by) {
        f16x4 hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[i] = (f16_t)(v[i] * by);
            lo[i] = (f16_t)__builtin_fmaf(v[i], by, -(float)hi[i]);
        }
        *reinterpret_cast<f16x4 *>(&w[0][row][col]) = hi;
        if (N > 1) *reinterpret_cast<f16x4 *>(&w[N - 1][row][col]) = lo;
    }
    // Eight columns of a row; four of them as numbers (of the first plane).
    __device__ __forceinline__ Planes<N> along(uint32_t row, uint32_t col) const {
        Planes<N> o;
#pragma unroll
        for (int i = 0; i < N; ++i) o.p[i] = *reinterpret_cast<const f16x8 *>(&w[i][row][col]);
        return o;
    }
    __device__ __forceinline__ f32x4 four(uint32_t row, uint32_t col) const {
        const f16x4 r = *reinterpret_cast<const f16x4 *>(&w[0][row][col]);
        return f32x4{(float)r[0], (float)r[1], (float)r[2], (float)r[3]};
    }
    // Columns col0 + step (m >> 2) + (m & 3) at the places token_at(s, q, 0..7).
    __device__ __forceinline__ Planes<N> columns(uint32_t s, uint32_t col0, uint32_t step, uint32_t lane) const {
        const uint32_t i = lane & 15u, row = 32u * s + 4u * (lane >> 4) + (i >> 2), col = col0 + step * (i & 3u);
        Planes<N> o;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint64_t a = __builtin_bit_cast(uint64_t, read_transposed(&w[n][row][col]));
            const uint64_t b = __builtin_bit_cast(uint64_t, read_transposed(&w[n][row + 16u][col]));
            o.p[n] = __builtin_bit_cast(f16x8, uint64x2{a, b});
        }
        return o;
    }
    __device__ __forceinline__ Planes<N> across(uint32_t s, uint32_t tile, uint32_t lane) const {
        return columns(s, place(tile, 0u), 8u, lane);
    }
};
template <int W>
struct RowTile<Wide, W> {
    static constexpr int kStride = W + 4;
    float w[1][kChunk][kStride];
    __device__ __forceinline__ void put(uint32_t row, uint32_t col, const float (&v)[8], float) {
        *reinterpret_cast<f32x4 *>(&w[0][row][col]) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4 *>(&w[0][row][col + 4]) = f32x4{v[4], v[5], v[6], v[7]};
    }
    __device__ __forceinline__ void put(uint32_t row, uint32_t col, const f32x4 &v, float) {
        *reinterpret_cast<f32x4 *>(&w[0][row][col]) = v;
    }
    __device__ __forceinline__ Wide along(uint32_t row, uint32_t col) const {
        const f32x4 a = four(row, col), b = four(row, col + 4u);
        Wide o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o.p[i] = a[i], o.p[4 + i] = b[i];
        return o;
    }
    __device__ __forceinline__ f32x4 four(uint32_t row, uint32_t col) const {
        return *reinterpret_cast<const f32x4 *>(&w[0][row][col]);
    }
    __device__ __forceinline__ Wide columns(uint32_t s, uint32_t col0, uint32_t step, uint32_t lane) const {
        const uint32_t m = lane & 15u;
        Wide o;
#pragma unroll
        for (uint32_t j = 0; j < 8u; ++j) o.p[j] = w[0][token_at(s, lane >> 4, j)][col0 + step * (m >> 2) + (m & 3u)];
        return o;
    }
    __device__ __forceinline__ Wide across(uint32_t s, uint32_t tile, uint32_t lane) const {
        return columns(s, place(tile, 0u), 8u, lane);
    }
};
template <class T, int W>
using KeyTile = RowTile<typename Form<T>::In, W>;

// Eight activations of a row from column c of `width`, zeros past its end.
template <class T>
__device__ __forceinline__ void load8(float (&v)[8], const T *row, uint32_t c, uint32_t width) {
    if (c + 8u <= width) {
        const Pack<T, 8> r = *reinterpret_cast<const Pack<T, 8> *>(row + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (float)r.v[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c + j < width ? (float)row[c + j] : 0.0f;
    }
}

// Eight activations as they are in memory, held until they are written on:
// columns c .. c + 8 of a row of `width`, zeros past it or where !is.  E: the
// width is a multiple of 8.  `any` is a row that exists.
template <bool E, class T>
__device__ __forceinline__ Pack<T, 8> raw8(const T *row, const T *any, bool is, uint32_t c, uint32_t width) {
    Pack<T, 8> r;
    if (E) {
        const bool there = is && c < width;
        r = *reinterpret_cast<const Pack<T, 8> *>(there ? row + c : any);
        if (!there)
#pragma unroll
            for (int j = 0; j < 8; ++j) r.v[j] = (T)0.0f;
    } else if (is && c + 8u <= width) {
        r = *reinterpret_cast<const Pack<T, 8> *>(row + c);
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 8u; ++j) r.v[j] = is && c + j < width ? row[c + j] : (T)0.0f;
    }
    return r;
}
template <class T>
__device__ __forceinline__ void values_of(float (&v)[8], const Pack<T, 8> &r) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)r.v[j];
}

// Sum or largest of a row's numbers over its PER = 4 or 8 neighbouring threads.
template <int PER>
__device__ __forceinline__ float neighbours_sum(float v) {
    v += dpp<kQuadSwap2>(v);
    v += dpp<kQuadSwap1>(v);
    return PER == 8 ? v + dpp<kRowHalfMirror>(v) : v;
}
template <int PER>
__device__ __forceinline__ float neighbours_largest(float m) {
    m = __builtin_fmaxf(m, dpp<kQuadSwap2>(m));
    m = __builtin_fmaxf(m, dpp<kQuadSwap1>(m));
    return PER == 8 ? __builtin_fmaxf(m, dpp<kRowHalfMirror>(m)) : m;
}
// The scale of a row of keys or queries that PER neighbouring threads hold.
template <class T, int PER, int N>
__device__ __forceinline__ Scale row_scale(const float (&v)[N][8]) {
    if (!Form<T>::scaled) return {1.0f, 1.0f};
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < N; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = __builtin_fmaxf(m, __builtin_fabsf(v[c][j]));
    return scale_of<true>(neighbours_largest<PER>(m));
}

// Rows lo .. lo + rows of a head's keys or queries into a tile, zeros after
// them, PER threads a row.  Returns the factor of the thread's row (threadIdx.x
// / PER) in a product with the tile: 1 by its length or 1, and what takes the
// tile's power of two back; `raw`: without the latter.
template <class T, int PER, int W>
__device__ __forceinline__ float fill_rows(KeyTile<T, W> &tile, const void *from, int64_t stride, uint32_t head,
                                           uint32_t lo, uint32_t rows, const DeltaArgs &a, float *raw = nullptr) {
    constexpr uint32_t kStep = 8u * PER, kVecs = (W + kStep - 1u) / kStep;
    const uint32_t row = threadIdx.x / PER, part = (threadIdx.x % PER) * 8u;
    const T *p = static_cast<const T *>(from) + (int64_t)(lo + row) * stride + (int64_t)head * a.key_dim;
    float v[kVecs][8] = {}, sum = 0.0f;
#pragma unroll
    for (uint32_t c = 0; c < kVecs; ++c) {
        if (row < rows) load8<T>(v[c], p, part + kStep * c, a.key_dim);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(v[c][j], v[c][j], sum);
    }
    const Scale s = row_scale<T, PER>(v);
#pragma unroll
    for (uint32_t c = 0; c < kVecs; ++c)
        if (part + kStep * c < (uint32_t)W) tile.put(row, part + kStep * c, v[c], s.by);
    const float squares = neighbours_sum<PER>(sum);
    // 1 for a row that is not there, also where eps is 0
    const float by = a.unit && row < rows ? 1.0f / __builtin_sqrtf(squares + a.eps) : 1.0f;
    if (raw) *raw = by;
    return by * s.back;
}

// A wave's 16 columns of a matrix [rows, width], a head's state as a rule: tile
// t's register i is row place(t, 4 q + i) of column col.  E: both dimensions are
// multiples of 8, so a lane's four rows are all there or none.
template <bool E, int TILES>
__device__ __forceinline__ void load_states(f32x4 (&S)[TILES], const float *from, uint32_t rows, uint32_t width, uint32_t col,
                                            uint32_t q) {
#pragma unroll
    for (uint32_t t = 0; t < (uint32_t)TILES; ++t) {
        const uint32_t row = place(t, 4u * q);
        S[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (!from || row >= rows || col >= width) continue;
#pragma unroll
        for (uint32_t i = 0; i < 4u; ++i)
            if (E || row + i < rows) S[t][i] = finite_or_nan(from[(row + i) * width + col]);
    }
}
// The width is hidden from the compiler where it stores: it would keep the
// addresses of every row over a whole walk, in registers that the walk needs.
template <bool E, int TILES>
__device__ __forceinline__ void store_states(float *to, const f32x4 (&S)[TILES], float by, uint32_t rows, uint32_t width,
                                             uint32_t col, uint32_t q) {
    asm volatile("" : "+s"(width));
    if (col >= width) return;
#pragma unroll
    for (uint32_t t = 0; t < (uint32_t)TILES; ++t) {
        const uint32_t row = place(t, 4u * q);
        if (row >= rows) continue;
        float *p = to + (row * width + col);
#pragma unroll
        for (uint32_t i = 0; i < 4u; ++i)
            if (E || row + i < rows) p[i * width] = S[t][i] * by;
    }
}
// A result's tiles over all of a chunk's rows into packed rows of `width`.
__device__ __forceinline__ void store_rows(float *to, uint32_t width, const f32x4 (&y)[4], float by, uint32_t col, uint32_t q) {
    asm volatile("" : "+s"(width));
#pragma unroll
    for (uint32_t t = 0; t < 4u; ++t) {
        float *p = to + ((16u * t + 4u * q) * width + col);
#pragma unroll
        for (uint32_t i = 0; i < 4u; ++i) p[i * width] = y[t][i] * by;
    }
}

// ---------------------------------------------------------------------------
// what a chunk's preparation leaves in the workspace for each head
// ---------------------------------------------------------------------------
// Numbers for each row: e nu (backwards times beta), scale e mu, beta, exp(G_C -
// G) nu (nu and mu with what takes the keys' and queries' powers of two back);
// then exp(G_C) and what takes the triangles' scales back, the inverse's and the
// scores'.
constexpr uint32_t kRowE = 0u, kRowQ = 64u, kRowBeta = 128u, kRowTail = 192u, kRowWhole = 256u, kRowInverse = 257u,
                   kRowScores = 258u, kRowFloats = 320u;
// Two triangles as operands in the order that the lanes read them: rows of tile
// t and the places of token_at(s, ..); six of the eight hold something.
constexpr uint32_t kTriangle = 6u;
__host__ __device__ constexpr uint32_t lower_at(uint32_t t, uint32_t s) { return t < 2u ? t : 2u * t - 2u + s; }
__host__ __device__ constexpr uint32_t upper_at(uint32_t t, uint32_t s) { return t < 2u ? 2u * t + s : 2u + t; }

template <class T>
struct Prepared {
    typedef typename Form<T>::Mid Mid;
    float row[kRowFloats];
    Mid inverse[kTriangle][64];
    Mid scores[kTriangle][64];
};

__device__ __forceinline__ double shuffle_up(double v, uint32_t by, uint32_t lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const int from = (int)(lane - by) * 4;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)(uint32_t)b);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)(uint32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Running sums of a chunk's log decays, in 64 bits: what passes between two
// rows is the difference of two sums, which may be much smaller than they are.
// A log decay below -512 counts as that, so that minus infinity, a state that
// starts again, stays a number; exp of any sum with it is zero.
__device__ __forceinline__ double running_decay(const DeltaArgs &a, uint32_t head, uint32_t lo, uint32_t rows,
                                                uint32_t lane) {
    float g = lane < rows ? a.g[(int64_t)(lo + lane) * a.g_stride + head] : 0.0f;
    g = g < -512.0f ? -512.0f : g;
    double G = g;
#pragma unroll
    for (uint32_t by = 1u; by < 64u; by *= 2u) {
        const double below = shuffle_up(G, by, lane);
        if (lane >= by) G += below;
    }
    return G;
}
__device__ __forceinline__ float exp_hw(float v) { return exp2_hw(v * kLog2e); }

// A chunk's sums of g and its beta, held by every wave for itself.
struct ChunkGates {
    double sum[kChunk];
    float beta[kChunk];
};

// One 16 x 16 x 16 product in fp32: rows of `a`, columns from `col`; the right
// operand's tile as a result leaves it.
__device__ __forceinline__ f32x4 block_product(const float *a, uint32_t stride, const f32x4 &b, uint32_t lane, f32x4 acc) {
    const f32x4 v = *reinterpret_cast<const f32x4 *>(a + (lane & 15u) * stride + 4u * (lane >> 4));
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(v[i], b[i], acc, 0, 0, 0);
    return acc;
}

// The inverse of one plus a strict triangle, 256 threads.  Backwards a lower
// triangle A is inverted by columns: wave w has block column w in x, tiles of
// rows, by forward substitution in blocks of 16,
//   x_w = (1 + A_ww)^-1,  x_i = -(1 + A_ii)^-1 sum_{w <= l < i} A_il x_l.
// Forwards the rows of the inverse are wanted in the lanes, which is the same
// of the transpose, an upper triangle, from the last block up.  `tri` is the
// triangle, row after row, complete before the call.  Every wave inverts a
// block of the diagonal (a column in a lane) for all; the rest of its blocks
// it has in its own registers.  Nothing is squared or summed over powers, so a
// triangle of large entries loses no more than the substitution itself.
constexpr uint32_t kTriStride = 68u, kDiagonal = 20u;  // words from row to row
template <bool BACK>
__device__ __forceinline__ void unit_inverse(const float *tri, float (*diagonal)[16 * kDiagonal], uint32_t wave, uint32_t lane,
                                             f32x4 (&x)[4]) {
    const uint32_t n = lane & 15u, q = lane >> 4;
    const float *block = tri + 16u * wave * (kTriStride + 1u);
    float c[16];
#pragma unroll
    for (uint32_t k = 0; k < 16u; ++k) {
        const uint32_t i = BACK ? k : 15u - k;
        float s = i == n ? 1.0f : 0.0f;
#pragma unroll
        for (uint32_t l = 0; l < 16u; ++l)
            if (BACK ? l < i : l > i) s = __builtin_fmaf(-block[i * kTriStride + l], c[l], s);
        c[i] = s;
    }
    f32x4 own;
#pragma unroll
    for (uint32_t i = 0; i < 4u; ++i) {
        own[i] = q == 0u ? c[i] : q == 1u ? c[4u + i] : q == 2u ? c[8u + i] : c[12u + i];
        diagonal[wave][(4u * q + i) * kDiagonal + n] = own[i];
    }
    __syncthreads();
    const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (uint32_t k = 0; k < 4u; ++k) x[k] = k == wave ? own : none;
#pragma unroll
    for (uint32_t k = 1; k < 4u; ++k) {
        const uint32_t i = BACK ? k : 3u - k;
        if (BACK ? i > wave : i < wave) {
            f32x4 sum = none;
#pragma unroll
            for (uint32_t l = 0; l < 4u; ++l)  // tiles not yet there are zero
                if (BACK ? l < i : l > i) sum = block_product(tri + 16u * (i * kTriStride + l), kTriStride, x[l], lane, sum);
            x[i] = block_product(diagonal[i], kDiagonal, -sum, lane, none);
        }
    }
}

// A chunk's numbers for the kernels that walk over chunks.  One workgroup a
// chunk and head of keys: the two products are shared by the heads of values.
// Forwards the inverse of 1 + a diag(beta) and the scores P, backwards the
// transposes of (1 + diag(beta) a)^-1 and P.  Wave w has what operands of row
// tile w hold: all tiles are computed with their summed index in the registers
// and are operands as they come.
// Bound by vector issue (a wave's 1960 operations: rows to planes, 64 x 64
// exponentials, the substitution) and the 240 MB that it moves: 16384 rows of 16
// heads, 128 keys, bf16, 113 us.
template <class T, int W, bool BACK>
__global__ __launch_bounds__(256, 3) void delta_prepare_kernel(DeltaArgs a, uint32_t first, Prepared<T> *__restrict__ to,
                                                               uint32_t *hdr, uint32_t words) {
    typedef typename Form<T>::Mid Mid;
    union Shared {
        struct {
            KeyTile<T, W> k, q;
        } in;
        float tri[kChunk * kTriStride];
    };
    __shared__ Shared sh;
    __shared__ float diagonal[4][16 * kDiagonal];
    __shared__ ChunkGates gates[4];
    __shared__ float nu[kChunk], mu[kChunk], most[2][4];
    const uint32_t b = first + blockIdx.x;
    if (b == 0u && threadIdx.x == 0u) mark_plain(hdr, words);
    const uint32_t slot = b / a.kheads, khead = b % a.kheads;
    const Chunk c = find_chunk(a.offsets, a.num_seqs, a.tokens, kChunkShift, slot);
    const uint32_t rows = c.hi - c.lo;
    if (rows == 0u) return;
    const uint32_t wave = wave_number(), lane = threadIdx.x & 63u, n = lane & 15u, q = lane >> 4;
    const float own_nu = fill_rows<T, 4, W>(sh.in.k, a.k, a.k_stride, khead, c.lo, rows, a);
    const float own_mu = fill_rows<T, 4, W>(sh.in.q, a.q, a.q_stride, khead, c.lo, rows, a);
    if ((threadIdx.x & 3u) == 0u) nu[threadIdx.x >> 2] = own_nu, mu[threadIdx.x >> 2] = own_mu;
    __syncthreads();
    // kk: rows k_l, columns k of tile `wave`; qk: forwards rows k_j, columns q of
    // the tile, backwards rows q_i, columns k.  l > column or l < column.
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) kk[t] = qk[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (uint32_t col = 0; col < (uint32_t)W; col += 32u) {
        const auto kb = sh.in.k.along(16u * wave + n, col + 8u * q);
        const auto qb = sh.in.q.along(16u * wave + n, col + 8u * q);
#pragma unroll
        for (uint32_t t = 0; t < 4u; ++t) {
            const bool below = t <= wave, above = t >= wave;
            if (BACK ? below : above) mma(kk[t], sh.in.k.along(16u * t + n, col + 8u * q), kb);
            if (BACK && above) mma(qk[t], sh.in.q.along(16u * t + n, col + 8u * q), kb);
            if (!BACK && below) mma(qk[t], sh.in.k.along(16u * t + n, col + 8u * q), qb);
        }
    }
    const uint32_t per = a.heads / a.kheads;
    ChunkGates &gate = gates[wave];
    for (uint32_t j = 0; j < per; ++j) {
        const uint32_t head = khead * per + j;
        Prepared<T> &out = to[(uint64_t)slot * a.heads + head];
        const double sum = running_decay(a, head, c.lo, rows, lane);
        const float beta = lane < rows ? a.beta[(int64_t)(c.lo + lane) * a.beta_stride + head] : 0.0f;
        gate.sum[lane] = sum;
        gate.beta[lane] = beta;
        if (wave == 0u) {
            const uint64_t bits = __builtin_bit_cast(uint64_t, sum);
            const double all = __builtin_bit_cast(
                double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(bits >> 32), 63) << 32 |
                            (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)bits, 63));
            const float e = exp_hw((float)sum);
            out.row[kRowE + lane] = e * nu[lane] * (BACK ? beta : 1.0f);
            out.row[kRowQ + lane] = a.scale * e * mu[lane];
            out.row[kRowBeta + lane] = beta;
            out.row[kRowTail + lane] = exp_hw((float)(all - sum)) * nu[lane];
            if (lane == 0u) out.row[kRowWhole] = exp_hw((float)all);
        }
        const uint32_t col = 16u * wave + n;
        const double here = gate.sum[col];
        const float beta_here = gate.beta[col], nu_here = nu[col], mu_here = mu[col];
        f32x4 p[4], x[4];
        __syncthreads();  // the products, or the triangle of the head before, are read
#pragma unroll
        for (uint32_t t = 0; t < 4u; ++t) {
            f32x4 tri;
#pragma unroll
            for (uint32_t i = 0; i < 4u; ++i) {
                const uint32_t row = 16u * t + 4u * q + i;
                const float apart = (float)(gate.sum[row] - here);  // from the column's row to this one
                const float forth = exp_hw(row >= col ? apart : -apart);
                const float both = forth * nu[row];
                // forwards a_lj beta_j for l > j, the transpose's row j; backwards beta_i a_il
                tri[i] = (BACK ? row < col : row > col) ? both * nu_here * beta_here * kk[t][i] : 0.0f;
                const float along = BACK ? forth * mu[row] * nu_here : both * mu_here;
                p[t][i] = (BACK ? row >= col : row <= col) ? a.scale * along * qk[t][i] : 0.0f;
            }
            *reinterpret_cast<f32x4 *>(&sh.tri[col * kTriStride + 16u * t + 4u * q]) = tri;
        }
        __syncthreads();
        unit_inverse<BACK>(sh.tri, diagonal, wave, lane, x);
        Scale inverse = {1.0f, 1.0f}, scores = {1.0f, 1.0f};
        if constexpr (Form<T>::scaled) {
            const float mx = wave_largest(largest(x)), mp = wave_largest(largest(p));
            if (lane == 0u) most[0][wave] = mx, most[1][wave] = mp;
            __syncthreads();
            auto all = [&](const float(&m)[4]) { return __builtin_fmaxf(__builtin_fmaxf(m[0], m[1]), __builtin_fmaxf(m[2], m[3])); };
            inverse = scale_of<true, -20>(all(most[0]));
            scores = scale_of<true, -20>(all(most[1]));
        }
        if (threadIdx.x == 0u) {
            out.row[kRowInverse] = inverse.back;
            out.row[kRowScores] = scores.back;
        }
#pragma unroll
        for (uint32_t s = 0; s < 2u; ++s) {
            if (BACK ? s < (wave >> 1) : s > (wave >> 1)) continue;
            const uint32_t at = BACK ? upper_at(wave, s) : lower_at(wave, s);
            out.inverse[at][lane] = operand_of<Mid>(x[2u * s], x[2u * s + 1u], inverse.by);
            out.scores[at][lane] = operand_of<Mid>(p[2u * s], p[2u * s + 1u], scores.by);
        }
    }
}

// Sizes of a chunk's states and corrections that a walk leaves for the gradients:
// the largest of each, by wave of columns.
constexpr uint32_t kSizeWaves = 16u, kSizes = 2u * kSizeWaves;

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
ps_status delta_sizes(const ps_delta_input *in);
ps_status delta_pointers(const ps_delta_input *in);
DeltaArgs delta_args(const ps_delta_input *in);

// ps_gated_delta of one type, after delta_sizes.
template <class T>
ps_status delta_forward(void *ws, size_t *ws_bytes, const ps_delta_input *in, void *out, float *final, float *checkpoints,
                        hipStream_t stream);

// Bytes of a call's arrays; keys and values: packed rows of activations.
struct DeltaBytes {
    size_t q, k, v, g, beta, offsets, states, keys, values, gates;
    explicit DeltaBytes(const ps_delta_input *in) {
        const size_t e = dtype_bytes(in->dtype), kd = (size_t)in->kheads * in->key_dim, vd = (size_t)in->heads * in->value_dim;
        q = rows_bytes(in->tokens, in->q_stride, kd, e);
        k = rows_bytes(in->tokens, in->k_stride, kd, e);
        v = rows_bytes(in->tokens, in->v_stride, vd, e);
        g = rows_bytes(in->tokens, in->g_stride, in->heads, 4u);
        beta = rows_bytes(in->tokens, in->beta_stride, in->heads, 4u);
        offsets = in->offsets ? ((size_t)in->num_seqs + 1u) * 4u : 0u;
        states = (size_t)(in->offsets ? in->num_seqs : 1u) * in->heads * in->key_dim * in->value_dim * 4u;
        keys = in->tokens * kd * e;
        values = in->tokens * vd * e;
        gates = in->tokens * in->heads * 4u;
    }
};

// ps_gated_delta_bwd of one type, after delta_sizes.
template <class T>
ps_status delta_backward(void *ws, size_t *ws_bytes, const ps_delta_input *in, const void *dout, const float *dfinal,
                         const float *checkpoints, const ps_delta_grads *grads, hipStream_t stream);

// Calls f with the padded number of keys as a constant.
template <class F>
inline ps_status with_key_width(uint32_t key_dim, F f) {
    if (key_dim <= 32u) return f(std::integral_constant<int, 32>());
    if (key_dim <= 64u) return f(std::integral_constant<int, 64>());
    if (key_dim <= 128u) return f(std::integral_constant<int, 128>());
    return f(std::integral_constant<int, 256>());
}

}  // namespace dwps
