// block_device.hpp -- parts shared by the state space block's kernels:
// activation types, the scalar functions, pieces of packed sequences and
// sums across a row of 16 lanes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>
#include <type_traits>
#include <utility>

#include "dwps.h"
#include "host_common.hpp"
#include "launch_parts.hpp"
#include "pieces.hpp"

namespace dwps {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

constexpr float kLog2e = 1.4426950408889634f;

// exp2, log2 and reciprocal as the hardware's instructions (1 ulp; results
// below 2^-126 flush to zero, far under anything the sums here can see).
__device__ __forceinline__ float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float rcp_hw(float v) { return __builtin_amdgcn_rcpf(v); }

// 1 / (1 + e^-v); e^-v = inf gives 0.
__device__ __forceinline__ float sigmoid(float v) { return rcp_hw(1.0f + exp2_hw(v * -kLog2e)); }

// softplus(v) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1].  log1p by the
// series of the inverse hyperbolic tangent: with q = e / (2 + e) <= 1/3,
// log(1 + e) = 2 (q + q^3/3 + q^5/5 + ...); the terms left out, from q^15/15
// on, are below 2^-26 of the sum (at v = 0; a quarter of a rounding), so
// small steps (v << 0) keep full precision, which log(1 + e) itself would lose.
__device__ __forceinline__ float softplus(float v) {
    const float e = exp2_hw(__builtin_fabsf(v) * -kLog2e);
    const float q = e * rcp_hw(2.0f + e);
    const float s = q * q;
    float p = __builtin_fmaf(s, 1.0f / 13.0f, 1.0f / 11.0f);
    p = __builtin_fmaf(s, p, 1.0f / 9.0f);
    p = __builtin_fmaf(s, p, 1.0f / 7.0f);
    p = __builtin_fmaf(s, p, 1.0f / 5.0f);
    p = __builtin_fmaf(s, p, 1.0f / 3.0f);
    const float tail = q * s * p;
    return __builtin_fmaxf(v, 0.0f) + 2.0f * (q + tail);  // NaN through q
}

// An argument whose softplus is exactly 0.
constexpr float kNoStep = -256.0f;

// d silu(v) / dv from s = sigmoid(v).
__device__ __forceinline__ float dsilu(float v, float s) { return s * __builtin_fmaf(v, 1.0f - s, 1.0f); }
__device__ __forceinline__ float silu(float v) {
    const float s = sigmoid(v);
    return v * s;
}

// `n` activations of type T at p, unaligned to more than one element.
template <class T, int n>
struct __attribute__((packed, aligned(sizeof(T)))) Pack {
    T v[n];
};

// ---------------------------------------------------------------------------
// rows of 16 lanes
// ---------------------------------------------------------------------------
template <int ctrl>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl, 0xF, 0xF, true));
}
// Lane j of each row, in every lane of the row.
template <int j>
__device__ __forceinline__ float row_lane(float v) {
    return dpp<0x150 + j>(v);
}
constexpr int kRowRotate8 = 0x128, kRowMirror = 0x140, kRowHalfMirror = 0x141, kQuadSwap2 = 0x4E, kQuadSwap1 = 0xB1;

// Sixteen sums across each row of 16 lanes at once: lane l gets the sum over
// its row of v[l].  Every level adds to a lane's half of the values their
// mirror images (mirrored row, mirrored half) or neighbours (two lanes on,
// one lane on; together the partners are the 16 lanes), so the values halve
// from level to level.  The first two levels take whole banks of four lanes:
// the lower half's sum is formed in every lane, then the upper half's in its
// banks alone (a DPP bank mask, in assembly: the compiler has no way to say
// it), 24 additions for 12 values; then 9 operations in the quads.
#define DPP_ADD4(what, mask)                                                                                  \
    "v_add_f32_dpp %0, %4, %4 " what " row_mask:0xf bank_mask:" mask "\n\t"                                   \
    "v_add_f32_dpp %1, %5, %5 " what " row_mask:0xf bank_mask:" mask "\n\t"                                   \
    "v_add_f32_dpp %2, %6, %6 " what " row_mask:0xf bank_mask:" mask "\n\t"                                   \
    "v_add_f32_dpp %3, %7, %7 " what " row_mask:0xf bank_mask:" mask
struct Four {
    float v[4];
};
// The first level for four pairs (lower half: lo, upper half: hi).
__device__ __forceinline__ Four row_fold8(const Four &lo, const Four &hi) {
#pragma clang fp contract(off)  // a product fused into the first addition would cost a move for its partner
    Four a;
#pragma unroll
    for (int j = 0; j < 4; ++j) a.v[j] = lo.v[j] + dpp<kRowMirror>(lo.v[j]);
    // s_nop: two wait states between a VALU write and a DPP read of it
    asm("s_nop 1\n\t" DPP_ADD4("row_mirror", "0xc")
        : "+v"(a.v[0]), "+v"(a.v[1]), "+v"(a.v[2]), "+v"(a.v[3])
        : "v"(hi.v[0]), "v"(hi.v[1]), "v"(hi.v[2]), "v"(hi.v[3]));
    return a;
}
// The other levels: a holds values 0-3 and 8-11, b values 4-7 and 12-15.
__device__ __forceinline__ float row_fold(const Four &a, const Four &b, uint32_t lane) {
    const bool b2 = lane & 2u, b1 = lane & 1u;
    float q[4], c[2];
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = a.v[j] + dpp<kRowHalfMirror>(a.v[j]);
    asm("s_nop 1\n\t" DPP_ADD4("row_half_mirror", "0xa")
        : "+v"(q[0]), "+v"(q[1]), "+v"(q[2]), "+v"(q[3])
        : "v"(b.v[0]), "v"(b.v[1]), "v"(b.v[2]), "v"(b.v[3]));
#pragma unroll
    for (int j = 0; j < 2; ++j) c[j] = (b2 ? q[j + 2] : q[j]) + dpp<kQuadSwap2>(b2 ? q[j] : q[j + 2]);
    return (b1 ? c[1] : c[0]) + dpp<kQuadSwap1>(b1 ? c[0] : c[1]);
}
__device__ __forceinline__ float row_sums(const float (&v)[16], uint32_t lane) {
    const Four a = row_fold8({{v[0], v[1], v[2], v[3]}}, {{v[8], v[9], v[10], v[11]}});
    const Four b = row_fold8({{v[4], v[5], v[6], v[7]}}, {{v[12], v[13], v[14], v[15]}});
    return row_fold(a, b, lane);
}
#undef DPP_ADD4

// The sum over each row of 16 lanes, in every lane.
__device__ __forceinline__ float row_total(float v) {
    v += dpp<kRowMirror>(v);
    v += dpp<kRowHalfMirror>(v);
    v += dpp<kQuadSwap2>(v);
    return v + dpp<kQuadSwap1>(v);
}

// a = (a's lower half, b's lower half), b = (a's upper half, b's upper half);
// for 16: the same of each pair of rows.  In assembly, for the builtin of ROCm
// 7.2 gives its first result in place of both.  The wait states cover a VALU
// write of the operands just before, which the compiler cannot see inside.
__device__ __forceinline__ void swap_halves(float &a, float &b) {
    asm("s_nop 4\n\tv_permlane32_swap_b32 %0, %1" : "+v"(a), "+v"(b));
}
__device__ __forceinline__ void swap_rows(float &a, float &b) {
    asm("s_nop 4\n\tv_permlane16_swap_b32 %0, %1" : "+v"(a), "+v"(b));
}

// The sum over a wave, in every lane.
__device__ __forceinline__ float wave_total(float v) {
    v = row_total(v);
    float w = v;
    swap_rows(v, w);
    v += w;
    w = v;
    swap_halves(v, w);
    return v + w;
}

// f(0), f(1), ... with the index as a constant.
template <class F, int... i>
__device__ __forceinline__ void for_each_index(F f, std::integer_sequence<int, i...>) {
    (f(std::integral_constant<int, i>()), ...);
}

// p[first * stride] + p[(first + step) * stride] + ... up to `rows`, eight
// loads at a time on their way, in a fixed order.
__device__ __forceinline__ float column_sum(const float *p, uint32_t first, uint32_t step, uint32_t rows, uint64_t stride) {
    float v[8] = {};
    uint32_t r = first;
    for (; r + 7u * step < rows; r += 8u * step) {
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] += p[(r + u * step) * stride];
    }
    float s = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    for (; r < rows; r += step) s += p[r * stride];
    return s;
}

// Workgroups go round the 8 XCDs in turn.  Neighbouring channel blocks share
// cache lines of the token rows, so of every 8 * group workgroups each XCD
// gets `group` neighbours.
__device__ __forceinline__ uint32_t xcd_neighbours(uint32_t b, uint32_t blocks, uint32_t group) {
    const uint32_t unit = 8u * group, base = b / unit * unit;
    if (base + unit > blocks) return b;
    const uint32_t i = b - base;
    return base + (i & 7u) * group + (i >> 3);
}

// Marks the words of a workspace that a call uses as plain memory dirty, for
// the scans that may use it next (ws_state.hpp).  One thread of one launch.
__device__ __forceinline__ void mark_plain(uint32_t *hdr, uint32_t words) {
    if (hdr[kHdrMagic] != kWsMagic) return;  // not prepared: preparing it marks everything
    uint32_t lo = hdr[kHdrDirtyLo], hi = hdr[kHdrDirtyHi];
    ws_mark_dirty(lo, hi, 0u, words < hdr[kHdrCapacity] ? words : hdr[kHdrCapacity]);
    hdr[kHdrDirtyLo] = lo;
    hdr[kHdrDirtyHi] = hi;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline size_t dtype_bytes(ps_dtype t) { return t == PS_F32 ? 4u : t == PS_BF16 || t == PS_F16 ? 2u : 0u; }

constexpr uint64_t kBlockMaxTokens = (1ull << 31) - 1u;
constexpr uint32_t kBlockMaxChannels = 1u << 24;
constexpr uint32_t kBlockMaxSeqs = (1u << 24) - 1u;
// Offsets within 32 rows of a token array are 32-bit byte counts.
constexpr int64_t kBlockMaxStride = 1 << 24;

// Bytes from the first to past the last element of `rows` rows.
inline size_t rows_bytes(uint64_t rows, int64_t stride, uint64_t row, size_t elem) {
    return rows ? ((rows - 1u) * (uint64_t)stride + row) * elem : 0u;
}

// An array of a call; NULL or 0 bytes: not there.
struct Bytes {
    const void *at;
    size_t n;
};
// Whether an output overlaps an input or another output.
inline bool outputs_overlap(std::initializer_list<Bytes> outs, std::initializer_list<Bytes> ins) {
    auto meet = [](const Bytes &a, const Bytes &b) { return a.at && b.at && ranges_overlap(a.at, a.n, b.at, b.n); };
    for (const Bytes *o = outs.begin(); o != outs.end(); ++o) {
        for (const Bytes &i : ins)
            if (meet(*o, i)) return true;
        for (const Bytes *p = outs.begin(); p != o; ++p)
            if (meet(*o, *p)) return true;
    }
    return false;
}

// Plain memory of a workspace, handed out in pieces of whole 256 bytes after
// the header.
struct PlainWs {
    size_t at = kWsHeader;
    size_t take(size_t bytes) {
        const size_t here = at;
        at += round_up(bytes, 256);
        return here;
    }
    uint32_t words() const {
        const size_t w = (at - kWsHeader) / 8u;
        return w > 0xFFFFFFFFull ? 0xFFFFFFFFu : (uint32_t)w;
    }
};
template <class T>
inline T *ws_at(void *ws, size_t at) {
    return reinterpret_cast<T *>(static_cast<char *>(ws) + at);
}

// Calls f with a value of the activations' type.
template <class F>
inline ps_status with_type(ps_dtype t, F f) {
    switch (t) {
    case PS_F32: return f(float());
    case PS_BF16: return f(bf16_t());
    case PS_F16: return f(f16_t());
    default: return PS_ERR_UNSUPPORTED;
    }
}

}  // namespace dwps
