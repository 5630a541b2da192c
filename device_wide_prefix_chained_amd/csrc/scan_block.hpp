// scan_block.hpp -- parts shared by the selective scan's kernels
// (selective_scan.hip, selective_scan_bwd.hip).
//
// Layout of the walking kernels: a row of 16 lanes owns one channel, lane n
// its states n, n + 16, ...; a workgroup of 4 waves owns 16 channels of one
// group, so that a token row's 16 channels are one 32-byte (16-bit types) or
// 64-byte load and B and C are staged once for all of them.  Tokens are
// staged 32 at a time, aligned to 32 packed rows; rows of the block outside
// the piece have step = 0 and zero inputs, which leaves the states as they
// are.
#pragma once

#include "block_device.hpp"
#include "scan_shape.hpp"

namespace dwps {

constexpr uint32_t kScanCellShift = 5;            // rows between checkpoints
constexpr uint32_t kScanCell = 1u << kScanCellShift;
constexpr int kScanTile = 32;                     // tokens staged at a time
constexpr int kScanThreads = 256;
// Floats from one staged channel (or state) to the next: a multiple of 4 for
// 16-byte reads, and 36 mod 64 = 36 spreads pairs of channels over the banks.
constexpr int kScanPad = kScanTile + 4;

struct ScanArgs {
    const void *x, *dt, *z, *B, *C;
    const float *A, *D, *bias, *initial;
    const uint32_t *offsets;
    int64_t x_stride, dt_stride, z_stride, b_stride, c_stride;
    uint32_t tokens, channels, groups, states, num_seqs;
    uint32_t first;            // piece (rows' share, for single tokens) of the launch's first workgroup
    uint32_t shift;            // log2 of the rows of a piece; 32: whole sequences
    uint32_t group_channels;   // channels / groups
    uint32_t group_blocks;     // workgroups of 16 channels in a group
    uint32_t col_blocks;       // groups * group_blocks
};

// What a workgroup works on.
struct ScanPlace {
    Piece q;
    uint32_t p;         // piece number
    uint32_t group;
    uint32_t ch0;       // first channel
    uint32_t have;      // channels, up to 16
};

__device__ __forceinline__ ScanPlace scan_place(const ScanArgs &a, uint32_t b) {
    ScanPlace w;
    w.p = a.first + b / a.col_blocks;
    const uint32_t cb = b % a.col_blocks;
    w.group = cb / a.group_blocks;
    const uint32_t in_group = cb % a.group_blocks * kScanChannels;
    w.ch0 = w.group * a.group_channels + in_group;
    w.have = a.group_channels - in_group < (uint32_t)kScanChannels ? a.group_channels - in_group : kScanChannels;
    w.q = find_piece(a.offsets, a.num_seqs, a.tokens, a.shift, w.p);
    return w;
}

// Two neighbouring elements of a token's row as they were loaded.  FULL: both
// exist, one load (kept as the 32 bits it is: split into elements, the
// compiler would wait for it long before its use).  Otherwise each has an
// offset of its own that stays inside the row (the second of a pair that ends
// the row, or both of a pair past it, repeat an element), and values() drops
// what is not `in`.  No load is under a branch, so all of a block's are on
// their way at once.
template <class T, bool FULL>
struct RawPair {
    T e0, e1;
    __device__ __forceinline__ void load(const char *base, uint32_t byte0, uint32_t byte1) {
        e0 = *reinterpret_cast<const T *>(base + byte0);
        e1 = *reinterpret_cast<const T *>(base + (FULL ? byte0 + (uint32_t)sizeof(T) : byte1));
    }
    __device__ __forceinline__ void values(float (&v)[2], bool in0, bool in1) const {
        v[0] = in0 ? (float)e0 : 0.0f;
        v[1] = in1 ? (float)e1 : 0.0f;
    }
};
typedef uint32_t __attribute__((aligned(2), may_alias)) word_at_2;
template <>
struct RawPair<bf16_t, true> {
    uint32_t w;
    __device__ __forceinline__ void load(const char *base, uint32_t byte0, uint32_t) {
        w = *reinterpret_cast<const word_at_2 *>(base + byte0);
    }
    __device__ __forceinline__ void values(float (&v)[2], bool in0, bool in1) const {
        v[0] = in0 ? __builtin_bit_cast(float, w << 16) : 0.0f;
        v[1] = in1 ? __builtin_bit_cast(float, w & 0xFFFF0000u) : 0.0f;
    }
};
template <>
struct RawPair<f16_t, true> {
    uint32_t w;
    __device__ __forceinline__ void load(const char *base, uint32_t byte0, uint32_t) {
        w = *reinterpret_cast<const word_at_2 *>(base + byte0);
    }
    __device__ __forceinline__ void values(float (&v)[2], bool in0, bool in1) const {
        v[0] = in0 ? (float)__builtin_bit_cast(f16_t, (uint16_t)w) : 0.0f;
        v[1] = in1 ? (float)__builtin_bit_cast(f16_t, (uint16_t)(w >> 16)) : 0.0f;
    }
};
// One token array as a thread of the staging sees it: its pair's place in 32
// rows (32 bits, so that a load is one instruction on the block's address in
// scalar registers).
template <class T, bool FULL>
struct PairRows {
    const T *base;
    int64_t stride;
    uint32_t byte0, byte1;
    __device__ __forceinline__ void place(uint32_t row, uint32_t e0, uint32_t e1) {
        byte0 = (row * (uint32_t)stride + e0) * (uint32_t)sizeof(T);
        byte1 = FULL ? 0u : (row * (uint32_t)stride + e1) * (uint32_t)sizeof(T);
    }
    __device__ __forceinline__ void load(RawPair<T, FULL> &r, uint32_t first_row) const {
        r.load(reinterpret_cast<const char *>(base + (int64_t)first_row * stride), byte0, byte1);
    }
};
// Offset of element c of `have`, kept inside.
__device__ __forceinline__ uint32_t inside(uint32_t c, uint32_t have) { return c < have ? c : have - 1u; }

// How far each carry reaches: row 0 unused.
enum ScanLink : uint32_t { kLinkNone = 0, kLinkStart = 1, kLinkChain = 2 };

// Workgroups side by side for one piece, so that a piece fits a launch.
constexpr uint64_t kScanMaxBlocks = (1u << 23) - 1u;
static_assert(kScanMaxBlocks <= kLaunchMostItems / (2 * kScanThreads), "a piece fits a launch");

ScanArgs scan_args(const ps_scan_input *in, uint32_t shift);
ps_status scan_sizes(const ps_scan_input *in, bool packed);
ps_status scan_pointers(const ps_scan_input *in);
// Bytes of a call's arrays; cells and bc: packed rows of x's and B's shape,
// edge: initial, final and dinitial.
struct ScanBytes {
    size_t x, dt, z, B, C, cells, bc, A, channel, offsets, edge, marks;
    explicit ScanBytes(const ps_scan_input *in) {
        const size_t e = dtype_bytes(in->dtype), c = in->channels, gn = (size_t)in->groups * in->states;
        x = rows_bytes(in->tokens, in->x_stride, c, e);
        dt = rows_bytes(in->tokens, in->dt_stride, c, e);
        z = rows_bytes(in->tokens, in->z_stride, c, e);
        B = rows_bytes(in->tokens, in->b_stride, gn, e);
        C = rows_bytes(in->tokens, in->c_stride, gn, e);
        cells = in->tokens * c * e;
        bc = in->tokens * gn * e;
        A = c * in->states * 4u;
        channel = c * 4u;
        offsets = ((size_t)in->num_seqs + 1u) * 4u;
        edge = (in->offsets ? in->num_seqs : 1u) * A;
        marks = ceil_div(in->tokens, kScanCell) * A;
    }
};

// Carries from cell to cell (forward: entering each cell from the left, in
// increasing order; backward: from the right): carry[c] = part[c] +
// exp(A steps[c]) carry[c -+ 1], or part[c] alone where the chain starts.
void launch_scan_link(const ScanArgs &a, float *carry, const float *steps, const uint32_t *links, uint32_t cells,
                      bool backward, hipStream_t s);

// Calls f(true) if a kernel with per_lane states in a lane has no place without
// a state or a channel (pairs are then loaded whole).
template <class F>
inline ps_status with_full(const ps_scan_input *in, uint32_t per_lane, F f) {
    if (scan_whole(in->channels / in->groups, in->states, per_lane)) return f(std::true_type());
    return f(std::false_type());
}

// Calls f with the states of a lane.
template <class F>
inline ps_status with_states(uint32_t states, F f) {
    switch (scan_states_per_lane(states)) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    default: return f(std::integral_constant<int, 16>());
    }
}

}  // namespace dwps
