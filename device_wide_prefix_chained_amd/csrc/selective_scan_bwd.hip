// selective_scan_bwd.hip -- gradients of the selective scan.
//
// With g = dout * silu(z) (the gradient of C . h + D x), a = exp(step A) and
// dh[t] the gradient of h[t]:
//   dh[t]  = C[t] g[t] + a[t + 1] dh[t + 1]            (backwards in time)
//   flow   = a[t] dh[t] h[t - 1]                       (gradient of step A)
//   dx     = D g + step (sum_n dh B)
//   dstep  = sum_n flow A + x (sum_n dh B),   ddt = dstep sigmoid(dt + bias)
//   dB     = sum_d dh step x,   dC = sum_d g h,   dA = sum_t flow step
//   dz     = dout (C . h + D x) silu'(z),   dD = sum_t g x,   dinitial = a dh
//            of a sequence's first row.
// Every piece of a sequence in a cell of 32 rows is worked on by itself.  A
// first pass walks back over each to find what it adds to a dh where it
// crosses to the cell before, these are linked from cell to cell (carry), and
// the main pass starts from the checkpoint that the forward pass left at the
// cell's first row and from the carry at its last.
// Sums over channels and over pieces go to partial sums that a last launch
// adds up in a fixed order.
#include <hip/hip_runtime.h>

#include "scan_block.hpp"

namespace dwps {
namespace {

// Nothing read from shared memory moves across this, so that values are read
// where they are used and do not push others out of the registers.
__device__ __forceinline__ void read_later() { asm volatile("" ::: "memory"); }

// No instruction moves across this: the reads before it are on their way
// while the arithmetic after it runs.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

typedef float f4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ f4 four(const float *p) { return *reinterpret_cast<const f4 *>(p); }

// What each piece that starts its cell inside a sequence adds to the carry
// out of the cell (carry[cell], from no carry in), the sum of its steps, and
// how its cell's carry follows from the next cell's (links).  One piece and a
// range of channel blocks; four waves feed the four that walk.  A walk needs
// exp2 and 3 operations for every state, about as much as the steps and gated
// gradients that feed it, so the feeding waves are the other half of the work.
// 8192 x 2048 x 16 states, bf16: 69 us; walking whole sequences took 307 us.
template <class T, int S, bool FULL>
__global__ __launch_bounds__(2 * kScanThreads) void scan_back_kernel(ScanArgs a, const T *__restrict__ dout,
                                                                     float *__restrict__ carry, float *__restrict__ steps,
                                                                     uint32_t *__restrict__ links, uint32_t ranges,
                                                                     uint32_t per_range) {
    constexpr int kPlane = kScanChannels * kScanPad;
    __shared__ __attribute__((aligned(16))) float sStep[2][kPlane], sGrad[2][kPlane], sC[16 * S * kScanPad];
    const uint32_t p = a.first + blockIdx.x / (a.groups * ranges), rg = blockIdx.x % (a.groups * ranges);
    const uint32_t group = rg / ranges, range = rg % ranges;
    const Piece q = find_piece(a.offsets, a.num_seqs, a.tokens, a.shift, p);
    if (!q.any || q.lo != (uint64_t)q.cell << a.shift) return;  // starts inside its cell: nothing enters another
    const bool on = q.lo > q.seq_lo;
    if (rg == 0u && threadIdx.x == 0)
        links[q.cell] = !on ? kLinkNone
                        : (uint64_t)q.seq_hi > ((uint64_t)(q.cell + 1u) << a.shift) ? kLinkChain : kLinkStart;
    if (!on) return;
    const uint32_t cb0 = range * per_range;
    const uint32_t cb1 = cb0 + per_range < a.group_blocks ? cb0 + per_range : a.group_blocks;
    const uint32_t N = a.states, blk = q.lo;
    const int64_t DN = (int64_t)a.channels * N;
    auto have_of = [&](uint32_t cb) {
        const uint32_t left = a.group_channels - cb * kScanChannels;
        return FULL || left >= (uint32_t)kScanChannels ? (uint32_t)kScanChannels : left;
    };
    if (__builtin_amdgcn_readfirstlane(threadIdx.x) < (uint32_t)kScanThreads) {
        const uint32_t c2 = (threadIdx.x & 7u) * 2u, row = threadIdx.x >> 3;
        const bool live = blk + row < q.hi;
        // rows past the last repeat it; staging drops them
        const uint32_t rt = row < a.tokens - 1u - blk ? row : a.tokens - 1u - blk;
        struct Raw {
            RawPair<T, FULL> dt, dy, z;
            float bias[2];
        } raw[2];
        PairRows<T, FULL> rdt{static_cast<const T *>(a.dt), a.dt_stride}, rdy{dout, a.channels};
        PairRows<T, FULL> rz{static_cast<const T *>(a.z ? a.z : a.dt), a.z ? a.z_stride : a.dt_stride};
        auto fetch = [&](Raw &r, uint32_t cb) {
            if (cb >= cb1) cb = cb1 - 1u;
            const uint32_t have = have_of(cb), ch0 = group * a.group_channels + cb * kScanChannels;
            const uint32_t e0 = FULL ? c2 : inside(c2, have), e1 = FULL ? c2 + 1u : inside(c2 + 1u, have);
            auto pair = [&](RawPair<T, FULL> &to, PairRows<T, FULL> rows) {
                rows.place(rt, e0, e1);
                rows.base += ch0;
                rows.load(to, blk);
            };
            pair(r.dt, rdt);
            pair(r.dy, rdy);
            pair(r.z, rz);
            r.bias[0] = a.bias ? a.bias[ch0 + e0] : 0.0f, r.bias[1] = a.bias ? a.bias[ch0 + e1] : 0.0f;
        };
        auto stage = [&](Raw &r, uint32_t cb, int half) {
            const uint32_t have = cb < cb1 ? have_of(cb) : 0u;
            const bool in0 = live && c2 < have, in1 = live && c2 + 1u < have;
            float v[2], z[2];
            r.dy.values(v, true, true);
            r.z.values(z, true, true);
            if (a.z) v[0] *= silu(z[0]), v[1] *= silu(z[1]);
            sGrad[half][c2 * kScanPad + row] = in0 ? v[0] : 0.0f;
            sGrad[half][(c2 + 1) * kScanPad + row] = in1 ? v[1] : 0.0f;
            r.dt.values(v, true, true);
            sStep[half][c2 * kScanPad + row] = softplus(in0 ? v[0] + r.bias[0] : kNoStep);
            sStep[half][(c2 + 1) * kScanPad + row] = softplus(in1 ? v[1] + r.bias[1] : kNoStep);
            fetch(r, cb + 2u);
        };
        fetch(raw[0], cb0);
        fetch(raw[1], cb0 + 1u);
        PairRows<T, FULL> rC{static_cast<const T *>(a.C) + (int64_t)group * N, a.c_stride};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const uint32_t m = s * 16 + c2, n0 = FULL ? m : inside(m, N), n1 = FULL ? m + 1u : inside(m + 1u, N);
            RawPair<T, FULL> vC;
            float v[2];
            rC.place(rt, n0, n1);
            rC.load(vC, blk);
            vC.values(v, live && (FULL || m < N), live && (FULL || m + 1u < N));
            sC[m * kScanPad + row] = v[0];
            sC[(m + 1) * kScanPad + row] = v[1];
        }
        stage(raw[0], cb0, 0);
        __syncthreads();
        for (uint32_t cb = cb0; cb < cb1; cb += 2u) {
            stage(raw[1], cb + 1u, 1);  // past the range: dropped
            __syncthreads();
            if (cb + 1u < cb1) {
                stage(raw[0], cb + 2u, 0);
                __syncthreads();
            }
        }
        return;
    }
    const uint32_t lane = threadIdx.x & 63u, l = lane & 15u;
    const uint32_t cw = ((threadIdx.x - kScanThreads) >> 6) * 4u + (lane >> 4);
    __builtin_amdgcn_s_setprio(2);
    float next[S];
    auto fetch = [&](uint32_t cb) {
        if (cb >= cb1) cb = cb1 - 1u;
        const uint32_t d = group * a.group_channels + cb * kScanChannels + (FULL ? cw : inside(cw, have_of(cb)));
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const uint32_t n = s * 16 + l;
            next[s] = a.A[(int64_t)d * N + (FULL || n < N ? n : N - 1u)];
        }
    };
    fetch(cb0);
    __syncthreads();
    for (uint32_t cb = cb0; cb < cb1; ++cb) {
        const uint32_t half = (cb - cb0) & 1u, d = group * a.group_channels + cb * kScanChannels + cw;
        const float *pS = sStep[half] + cw * kScanPad, *pG = sGrad[half] + cw * kScanPad;
        float A2[S], back[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            A2[s] = FULL || (cw < have_of(cb) && s * 16 + l < N) ? next[s] * kLog2e : 0.0f;
            back[s] = 0.0f;
        }
        fetch(cb + 1u);
        const float total = row_total(pS[l] + pS[16 + l]);
#pragma unroll
        for (int k0 = kScanTile - 4; k0 >= 0; k0 -= 4) {
            const f4 S4 = four(pS + k0), G4 = four(pG + k0);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const f4 C4 = four(sC + (s * 16 + l) * kScanPad + k0);
#pragma unroll
                for (int i = 3; i >= 0; --i) back[s] = exp2_hw(S4[i] * A2[s]) * __builtin_fmaf(G4[i], C4[i], back[s]);
            }
            if (S > 1 && k0 % 8 == 0) read_later();
        }
        if (FULL || cw < have_of(cb)) {
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (FULL || s * 16 + l < N) carry[(int64_t)q.cell * DN + (int64_t)d * N + s * 16 + l] = back[s];
            if (l == 0u) steps[(int64_t)q.cell * a.channels + d] = total;
        }
        __syncthreads();
    }
}

struct BackOut {
    void *dx, *ddt, *dz;
    float *dinitial;
    float *part_A;     // [pieces][channels][states]
    float *part_D;     // [pieces][channels], then ddt_bias' the same
    float *part_bias;
    float *part_B;     // [ranges][tokens][groups][states]
    float *part_C;
    uint32_t ranges;   // of a group's channel blocks
    uint32_t per_range;
    uint32_t blocks;   // groups * ranges
};

// Adds v over the four rows of a wave and spreads 32 values over them: row r
// gets v[r * 8 .. r * 8 + 7].
__device__ __forceinline__ void fold_rows(float (&o)[8], float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        swap_halves(v[j], v[j + 16]);
        v[j] += v[j + 16];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        swap_rows(v[j], v[j + 8]);
        o[j] = v[j] + v[j + 8];
    }
}

// One piece of a cell, a range of channel blocks.  States 16 at a time
// (outer loop), channels 16 at a time (inner loop): a lane sums dB and dC of
// its state over the inner loop in registers, token by token, and keeps a
// and h of the piece's 32 rows between the walk forward and the walk back.
// With more than 16 states the three sums over states wait in shared memory
// for the last 16.
//
// As in the forward walk, four waves feed (they load, stage and, a block
// later, form the block's outputs) and four walk.  Bound by arithmetic: for
// every state 5 operations and exp2 forwards, 8 backwards and 99 / 16 for the
// three sums over states.  The 64 sums, 32 states and 32 decays of a walking
// lane and four tokens' values on their way from shared memory take 200 of the
// 256 registers that two waves per SIMD leave it; what it starts from and
// leaves goes through shared memory too, since with those loads of its own it
// spilled and waited for memory in every block (350 to 510 us).
// 8192 x 2048 x 16 states, bf16: 292 us, 70% of the vector issue slots taken.
template <class T, bool FULL, bool MANY>
__global__ __launch_bounds__(2 * kScanThreads, 2) void scan_grad_kernel(ScanArgs a, const T *__restrict__ dout,
                                                                        const float *__restrict__ marks,
                                                                        const float *__restrict__ carry, BackOut o,
                                                                        uint32_t *hdr, uint32_t words) {
    constexpr int kPlane = kScanChannels * kScanPad;
    __shared__ __attribute__((aligned(16))) float sStep[2][kPlane], sDrive[2][kPlane], sGrad[2][kPlane], sB[kPlane],
        sC[kPlane];
    __shared__ float sFold[2][4][8][64];
    // for each walking lane A, the states and the carry that enter its piece; its dA and the carry that leaves
    __shared__ float sEnter[2][3][kScanThreads], sLeave[2][2][kScanThreads];
    __shared__ float sSum[2][4][4][8];  // [half][wave][dD of two channels, ddt_bias of two][pair]
    extern __shared__ float sCell[];    // [channel blocks of the range, or 2][3][kPlane]
    if (blockIdx.x == 0 && threadIdx.x == 0) mark_plain(hdr, words);
    // piece by piece of one range, the shorter last ranges at the end
    const uint32_t pieces = gridDim.x / o.blocks, p = a.first + blockIdx.x % pieces, rg = blockIdx.x / pieces;
    const uint32_t group = rg % a.groups, range = rg / a.groups;
    const Piece q = find_piece(a.offsets, a.num_seqs, a.tokens, a.shift, p);
    const uint32_t cb0 = range * o.per_range;
    const uint32_t cb1 = cb0 + o.per_range < a.group_blocks ? cb0 + o.per_range : a.group_blocks;
    const uint32_t N = a.states;
    const int64_t DN = (int64_t)a.channels * N;
    if (!q.any || q.lo == q.hi) {  // no rows: sums of nothing, an empty sequence's dinitial
        const uint32_t c_lo = group * a.group_channels + cb0 * kScanChannels;
        uint32_t c_hi = group * a.group_channels + cb1 * kScanChannels;
        if (c_hi > (group + 1u) * a.group_channels) c_hi = (group + 1u) * a.group_channels;
        for (int64_t i = (int64_t)c_lo * N + threadIdx.x; i < (int64_t)c_hi * N; i += 2 * kScanThreads) {
            o.part_A[p * DN + i] = 0.0f;
            if (q.any && o.dinitial) o.dinitial[q.seq * DN + i] = 0.0f;
        }
        for (uint32_t c = c_lo + threadIdx.x; c < c_hi; c += 2 * kScanThreads) {
            o.part_D[(int64_t)p * a.channels + c] = 0.0f;
            o.part_bias[(int64_t)p * a.channels + c] = 0.0f;
        }
        return;
    }
    const uint32_t blk = q.cell << kScanCellShift;
    const uint32_t state_blocks = MANY ? (N + 15u) / 16u : 1u;
    const bool feeds = __builtin_amdgcn_readfirstlane(threadIdx.x) < (uint32_t)kScanThreads;
    const uint32_t lane = threadIdx.x & 63u, l = lane & 15u, wave = (threadIdx.x >> 6) & 3u;
    auto have_of = [&](uint32_t cb) {
        const uint32_t left = a.group_channels - cb * kScanChannels;
        return FULL || left >= (uint32_t)kScanChannels ? (uint32_t)kScanChannels : left;
    };
    // the sums over states of block cb
    auto cell_of = [&](uint32_t cb) {
        return sCell + (MANY ? cb - cb0 : (cb - cb0) & 1u) * 3u * kPlane;
    };
    // dB, dC over the range's channels: the last sums over the waves
    auto write_parts = [&](uint32_t sb) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t j = threadIdx.x >> 6, ln = threadIdx.x & 63u;
            const float v = ((sFold[r][0][j][ln] + sFold[r][1][j][ln]) + sFold[r][2][j][ln]) + sFold[r][3][j][ln];
            const uint32_t tk = blk + (ln >> 4) * 8u + j, nn = sb * 16u + (ln & 15u);
            if (tk >= q.lo && tk < q.hi && nn < N)
                (r ? o.part_C : o.part_B)[(((int64_t)range * a.tokens + tk) * a.groups + group) * N + nn] = v;
        }
    };
    if (feeds) {
        const uint32_t c2 = (threadIdx.x & 7u) * 2u, row = threadIdx.x >> 3, t = blk + row;
        const bool live = t >= q.lo && t < q.hi;
        // rows past the last repeat it; staging drops them
        const uint32_t rt = row < a.tokens - 1u - blk ? row : a.tokens - 1u - blk;
        struct Raw {
            RawPair<T, FULL> x, dt, dy, z;
            float bias[2], skip[2];
            float A, h, back;  // of the walking lane with this thread's place
        } raw;
        const uint32_t cw = wave * 4u + (lane >> 4);
        const bool on = (uint64_t)q.seq_hi > (uint64_t)blk + kScanCell, starts = q.lo == q.seq_lo;
        // the states that enter the piece: a checkpoint, initial ones or zeros (then any address does)
        const float *enter = !starts ? marks + (int64_t)q.cell * DN : a.initial ? a.initial + (int64_t)q.seq * DN : a.A;
        const float *enter_back = on ? carry + (int64_t)(q.cell + 1u) * DN : a.A;
        // this lane's place among 16 channels' states, in bytes from the block's first
        auto lane_byte = [&](uint32_t have, uint32_t sb) {
            const uint32_t n = sb * 16u + l;
            return ((FULL ? cw : inside(cw, have)) * N + (FULL || n < N ? n : N - 1u)) * 4u;
        };
        auto of_lane = [](auto *base, int64_t first, uint32_t byte) {
            return reinterpret_cast<decltype(base)>((uintptr_t)(base + first) + byte);
        };
        const bool has_enter = !starts || a.initial;
        // what the outputs of a block need of its inputs, one block long
        struct Kept {
            RawPair<T, FULL> x, dy, z;
            float raw[2], st[2], skip[2], sz[2];
        } kept, next;
        PairRows<T, FULL> rx{static_cast<const T *>(a.x), a.x_stride}, rdt{static_cast<const T *>(a.dt), a.dt_stride};
        PairRows<T, FULL> rdy{dout, a.channels}, rz{static_cast<const T *>(a.z ? a.z : a.x), a.z ? a.z_stride : a.x_stride};
        auto place = [&](uint32_t e0, uint32_t e1) {
            rx.place(rt, e0, e1);
            rdt.place(rt, e0, e1);
            rdy.place(rt, e0, e1);
            rz.place(rt, e0, e1);
        };
        place(c2, c2 + 1u);
        if (MANY) {  // the sums over states start from zero: the walk adds to them without a branch
            for (uint32_t i = threadIdx.x; i < (cb1 - cb0) * 3u * kPlane; i += kScanThreads) sCell[i] = 0.0f;
        }
        auto fetch = [&](uint32_t cb, uint32_t sb) {
            if (cb >= cb1) cb = cb1 - 1u;
            const uint32_t have = have_of(cb), ch0 = group * a.group_channels + cb * kScanChannels;
            const uint32_t e0 = FULL ? c2 : inside(c2, have), e1 = FULL ? c2 + 1u : inside(c2 + 1u, have);
            if (!FULL) place(e0, e1);
            {   // lanes without a channel or state read one that exists; staging drops it
                const uint32_t byte = lane_byte(have, sb);
                const int64_t first = (int64_t)ch0 * N;
                raw.A = *of_lane(a.A, first, byte);
                raw.h = *of_lane(enter, first, byte);
                raw.back = *of_lane(enter_back, first, byte);
            }
            auto pair = [&](RawPair<T, FULL> &to, PairRows<T, FULL> rows) {
                rows.base += ch0;
                rows.load(to, blk);
            };
            pair(raw.x, rx);
            pair(raw.dt, rdt);
            pair(raw.dy, rdy);
            pair(raw.z, rz);
            raw.bias[0] = a.bias ? a.bias[ch0 + e0] : 0.0f, raw.bias[1] = a.bias ? a.bias[ch0 + e1] : 0.0f;
            raw.skip[0] = a.D ? a.D[ch0 + e0] : 0.0f, raw.skip[1] = a.D ? a.D[ch0 + e1] : 0.0f;
        };
        auto stage = [&](uint32_t cb, uint32_t sb) {
            const uint32_t half = (cb - cb0) & 1u, have = cb < cb1 ? have_of(cb) : 0u;
            const bool in0 = live && c2 < have, in1 = live && c2 + 1u < have;
            const bool walks = FULL || (cw < have && sb * 16u + l < N);
            sEnter[half][0][threadIdx.x] = walks ? raw.A : 0.0f;
            sEnter[half][1][threadIdx.x] = walks && has_enter ? raw.h : 0.0f;
            sEnter[half][2][threadIdx.x] = walks && on ? raw.back : 0.0f;
            float x[2], v[2], z[2];
            raw.x.values(x, in0, in1);
            raw.dy.values(v, in0, in1);
            raw.z.values(z, true, true);
            next.sz[0] = next.sz[1] = 1.0f;
            if (a.z) {
                next.sz[0] = sigmoid(z[0]), next.sz[1] = sigmoid(z[1]);
                v[0] *= z[0] * next.sz[0], v[1] *= z[1] * next.sz[1];
            }
            sGrad[half][c2 * kScanPad + row] = in0 ? v[0] : 0.0f;
            sGrad[half][(c2 + 1) * kScanPad + row] = in1 ? v[1] : 0.0f;
            raw.dt.values(v, true, true);
            next.x = raw.x, next.dy = raw.dy, next.z = raw.z;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                next.raw[i] = v[i] + raw.bias[i];
                next.skip[i] = raw.skip[i];
                next.st[i] = softplus((i ? in1 : in0) ? next.raw[i] : kNoStep);
                sStep[half][(c2 + i) * kScanPad + row] = next.st[i];
                sDrive[half][(c2 + i) * kScanPad + row] = next.st[i] * x[i];
            }
            // the next block, or the first with the next states
            if (cb + 1u < cb1) fetch(cb + 1u, sb);
            else fetch(cb0, sb + 1u < state_blocks ? sb + 1u : sb);
        };
        // a walking lane's dA and dinitial
        auto leave = [&](uint32_t cb, uint32_t sb) {
            const uint32_t half = (cb - cb0) & 1u, have = have_of(cb), byte = lane_byte(have, sb);
            const int64_t first = (int64_t)(group * a.group_channels + cb * kScanChannels) * N;
            if (FULL || (cw < have && sb * 16u + l < N)) {
                *of_lane(o.part_A, p * DN + first, byte) = sLeave[half][0][threadIdx.x];
                if (o.dinitial && starts) *of_lane(o.dinitial, (int64_t)q.seq * DN + first, byte) = sLeave[half][1][threadIdx.x];
            }
        };
        const uint32_t out_byte = (row * a.channels + c2) * (uint32_t)sizeof(T);
        auto outputs = [&](uint32_t cb) {
            const uint32_t have = have_of(cb), ch0 = group * a.group_channels + cb * kScanChannels;
            float x[2], dy[2], z[2], sx[2], sd[2];
            const bool in0 = c2 < have, in1 = c2 + 1u < have;
            kept.x.values(x, true, true);
            kept.dy.values(dy, true, true);
            kept.z.values(z, true, true);
            const float *c = cell_of(cb) + c2 * kScanPad + row;
            T vx[2], vd[2], vz[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float inner = c[i * kScanPad], along = c[kPlane + i * kScanPad], flow = c[2 * kPlane + i * kScanPad];
                const float sz = kept.sz[i];
                const float g = a.z ? dy[i] * (z[i] * sz) : dy[i];
                const float ddt = __builtin_fmaf(x[i], along, flow) * sigmoid(kept.raw[i]);
                vx[i] = (T)__builtin_fmaf(kept.skip[i], g, kept.st[i] * along);
                vd[i] = (T)ddt;
                vz[i] = (T)(dy[i] * __builtin_fmaf(kept.skip[i], x[i], inner) * dsilu(z[i], sz));
                sx[i] = live ? g * x[i] : 0.0f;
                sd[i] = live ? ddt : 0.0f;
            }
            if (live) {
                const int64_t first = (int64_t)blk * a.channels + ch0;
                T *dx = of_lane(static_cast<T *>(o.dx), first, out_byte), *dd = of_lane(static_cast<T *>(o.ddt), first, out_byte);
                T *dz = o.dz ? of_lane(static_cast<T *>(o.dz), first, out_byte) : nullptr;
                if (FULL) {
                    *reinterpret_cast<Pack<T, 2> *>(dx) = Pack<T, 2>{{vx[0], vx[1]}};
                    *reinterpret_cast<Pack<T, 2> *>(dd) = Pack<T, 2>{{vd[0], vd[1]}};
                    if (dz) *reinterpret_cast<Pack<T, 2> *>(dz) = Pack<T, 2>{{vz[0], vz[1]}};
                } else {
                    if (in0) dx[0] = vx[0], dd[0] = vd[0];
                    if (in1) dx[1] = vx[1], dd[1] = vd[1];
                    if (in0 && dz) dz[0] = vz[0];
                    if (in1 && dz) dz[1] = vz[1];
                }
            }
            // over the wave's 8 tokens: rows of lanes end up with one sum each
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sx[i] += dpp<kRowRotate8>(sx[i]);
                sd[i] += dpp<kRowRotate8>(sd[i]);
            }
            swap_rows(sx[0], sx[1]);
            swap_rows(sd[0], sd[1]);
            float ux = sx[0] + sx[1], ud = sd[0] + sd[1];
            swap_halves(ux, ud);
            if (l < 8u) sSum[(cb - cb0) & 1u][wave][lane >> 4][l] = ux + ud;
        };
        // and, a barrier later, over the 4 waves
        auto totals = [&](uint32_t cb) {
            if (threadIdx.x >= 32u) return;
            const uint32_t which = threadIdx.x >> 3, pair = threadIdx.x & 7u, c = pair * 2u + (which & 1u);
            const float(*v)[4][8] = sSum[(cb - cb0) & 1u];
            if (c < have_of(cb))
                (which >= 2u ? o.part_bias : o.part_D)[(int64_t)p * a.channels + group * a.group_channels + cb * kScanChannels + c] =
                    ((v[0][which][pair] + v[1][which][pair]) + v[2][which][pair]) + v[3][which][pair];
        };
        PairRows<T, FULL> rB{static_cast<const T *>(a.B) + (int64_t)group * N, a.b_stride};
        PairRows<T, FULL> rC{static_cast<const T *>(a.C) + (int64_t)group * N, a.c_stride};
        RawPair<T, FULL> vB, vC;
        auto fetch_states = [&](uint32_t sb) {
            const uint32_t m = sb * 16u + c2, n0 = FULL ? m : inside(m, N), n1 = FULL ? m + 1u : inside(m + 1u, N);
            rB.place(rt, n0, n1);
            rC.place(rt, n0, n1);
            rB.load(vB, blk);
            rC.load(vC, blk);
        };
        fetch(cb0, 0u);
        fetch_states(0u);
        for (uint32_t sb = 0; sb < state_blocks; ++sb) {
            const bool last = sb + 1u == state_blocks;
            {
                const uint32_t m = sb * 16u + c2;
                float v[2];
                vB.values(v, live && (FULL || m < N), live && (FULL || m + 1u < N));
                sB[c2 * kScanPad + row] = v[0];
                sB[(c2 + 1) * kScanPad + row] = v[1];
                vC.values(v, live && (FULL || m < N), live && (FULL || m + 1u < N));
                sC[c2 * kScanPad + row] = v[0];
                sC[(c2 + 1) * kScanPad + row] = v[1];
                if (!last) fetch_states(sb + 1u);
            }
            stage(cb0, sb);
            __syncthreads();
            for (uint32_t cb = cb0; cb < cb1; ++cb) {
                if (last && cb > cb0 + 1u) totals(cb - 2u);
                if (cb > cb0) leave(cb - 1u, sb);
                if (last && cb > cb0) outputs(cb - 1u);
                kept = next;
                stage(cb + 1u, sb);  // past the range: dropped
                __syncthreads();
            }
            leave(cb1 - 1u, sb);
            if (last && cb1 > cb0 + 1u) totals(cb1 - 2u);
            if (last) outputs(cb1 - 1u);
            __syncthreads();
            if (last) totals(cb1 - 1u);
            write_parts(sb);
            __syncthreads();
        }
        return;
    }
    const uint32_t cw = wave * 4u + (lane >> 4), place = threadIdx.x - kScanThreads;
    __builtin_amdgcn_s_setprio(2);  // the feeding waves fill the gaps
    for (uint32_t sb = 0; sb < state_blocks; ++sb) {
        float accB[32], accC[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) accB[j] = accC[j] = 0.0f;
        const float *pB = sB + l * kScanPad, *pC = sC + l * kScanPad;
        auto add_to = [&](float *to, float v) { *to = MANY ? *to + v : v; };
        __syncthreads();
        for (uint32_t cb = cb0; cb < cb1; ++cb) {
            const uint32_t half = (cb - cb0) & 1u;
            const float A = sEnter[half][0][place], A2 = A * kLog2e, h0 = sEnter[half][1][place];
            float back = sEnter[half][2][place];
            float *cell = cell_of(cb) + cw * kScanPad + l;
            const float *pS = sStep[half] + cw * kScanPad, *pD = sDrive[half] + cw * kScanPad, *pG = sGrad[half] + cw * kScanPad;
            float h[32];
            f4 decay[8];
            float run = h0;
            const float stv[2] = {pS[l], pS[16 + l]}, drv[2] = {pD[l], pD[16 + l]};
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                Four y[4];
                auto quad = [&](auto jc) {
                    constexpr int q0 = decltype(jc)::value;
                    const f4 B4 = four(pB + sub * 16 + q0 * 4), C4 = four(pC + sub * 16 + q0 * 4);
                    f4 e;
                    auto token = [&](auto ic) {
                        constexpr int i = decltype(ic)::value;
                        const int k = sub * 16 + q0 * 4 + i;
                        e[i] = exp2_hw(row_lane<q0 * 4 + i>(stv[sub]) * A2);
                        run = __builtin_fmaf(e[i], run, row_lane<q0 * 4 + i>(drv[sub]) * B4[i]);
                        h[k] = run;
                        y[q0].v[i] = run * C4[i];
                    };
                    for_each_index(token, std::make_integer_sequence<int, 4>());
                    decay[sub * 4 + q0] = e;
                    if constexpr (q0 >= 2) y[q0 - 2] = row_fold8(y[q0 - 2], y[q0]);
                };
                for_each_index(quad, std::make_integer_sequence<int, 4>());
                add_to(cell + sub * 16, row_fold(y[0], y[1], lane));
            }
            read_later();
            float sumA = 0.0f;
            f4 uB = four(pB + 28), uC = four(pC + 28), uS = four(pS + 28), uD = four(pD + 28), uG = four(pG + 28);
#pragma unroll
            for (int sub = 1; sub >= 0; --sub) {
                Four along[4], flowA[4];
                auto quad = [&](auto jc) {
                    constexpr int q0 = 3 - decltype(jc)::value;
                    const int k0 = sub * 16 + q0 * 4;
                    const f4 B4 = uB, C4 = uC, S4 = uS, D4 = uD, G4 = uG, E4 = decay[k0 / 4];
                    if (k0) {
                        uB = four(pB + k0 - 4), uC = four(pC + k0 - 4), uS = four(pS + k0 - 4);
                        uD = four(pD + k0 - 4), uG = four(pG + k0 - 4);
                    }
                    in_order();
#pragma unroll
                    for (int i = 3; i >= 0; --i) {
                        const int k = k0 + i;
                        const float dh = __builtin_fmaf(G4[i], C4[i], back);
                        accC[k] = __builtin_fmaf(G4[i], h[k], accC[k]);
                        accB[k] = __builtin_fmaf(D4[i], dh, accB[k]);
                        back = E4[i] * dh;
                        const float flow = back * (k ? h[k ? k - 1 : 0] : h0);
                        sumA = __builtin_fmaf(S4[i], flow, sumA);
                        along[q0].v[i] = dh * B4[i];
                        flowA[q0].v[i] = flow * A;
                    }
                    // the upper half's values wait for the lower half's
                    if constexpr (q0 < 2) {
                        along[q0] = row_fold8(along[q0], along[q0 + 2]);
                        flowA[q0] = row_fold8(flowA[q0], flowA[q0 + 2]);
                    }
                };
                for_each_index(quad, std::make_integer_sequence<int, 4>());
                float *to = cell + kPlane + sub * 16;
                add_to(to, row_fold(along[0], along[1], lane));
                add_to(to + kPlane, row_fold(flowA[0], flowA[1], lane));
            }
            sLeave[half][0][place] = sumA;
            sLeave[half][1][place] = back;
            __syncthreads();
        }
        // dB, dC over the range's channels: rows of a wave, then the waves
        float f[8];
        fold_rows(f, accB);
#pragma unroll
        for (int j = 0; j < 8; ++j) sFold[0][wave][j][lane] = f[j];
        fold_rows(f, accC);
#pragma unroll
        for (int j = 0; j < 8; ++j) sFold[1][wave][j][lane] = f[j];
        __syncthreads();
        write_parts(sb);
        __syncthreads();
    }
}

// The last launch: column sums of partial sums, several at once.
struct SumJob {
    const float *part;
    void *out;
    uint64_t cols;
    uint32_t rows;
    uint64_t first;   // workgroup
    uint32_t typed;   // the activations' type, not fp32
    uint32_t guard;   // rows of tokens outside every sequence stay unwritten
};
struct SumJobs {
    SumJob job[5];
    uint32_t count;
};

template <class T>
__global__ __launch_bounds__(256) void scan_sums_kernel(SumJobs jobs, ScanArgs a) {  // a.first: workgroups before these
    __shared__ float s[4][64];
    uint32_t k = 0;
    const uint64_t b = (uint64_t)a.first + blockIdx.x;
    while (k + 1u < jobs.count && b >= jobs.job[k + 1u].first) ++k;
    const SumJob j = jobs.job[k];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint64_t col = (b - j.first) * 64u + lane;
    float v = col < j.cols ? column_sum(j.part + col, wave, 4u, j.rows, j.cols) : 0.0f;
    s[wave][lane] = v;
    __syncthreads();
    if (wave != 0u || col >= j.cols) return;
    if (j.guard && a.offsets) {
        const uint32_t t = (uint32_t)(col / ((uint64_t)a.groups * a.states));
        if (t < a.offsets[0] || t >= a.offsets[a.num_seqs]) return;
    }
    v = ((s[0][lane] + s[1][lane]) + s[2][lane]) + s[3][lane];
    if (j.typed) static_cast<T *>(j.out)[col] = (T)v;
    else static_cast<float *>(j.out)[col] = v;
}

// Channel blocks that one workgroup goes through: as many as leave about 4
// rounds of the 256 workgroups that the GPU holds, 16 at most (the sums of dB
// and dC then leave a workgroup once in 256 channels).  Two rounds, and 4
// blocks at most, with more than 16 states, whose sums wait in shared memory.
// Several ranges are cut so that the last is about half as long: run last, it
// fills the gaps that whole rounds leave (8192 x 2048, 16 states: 308 us with 8
// equal ranges, 293 with 8 and a half).
uint32_t grad_range(const ScanArgs &a, uint64_t pieces) {
    const uint64_t fit = pieces * a.groups * a.group_blocks / (a.states > 16u ? 512u : 1024u);
    const uint64_t most = a.states > 16u ? 4u : 16u;
    const uint64_t per = fit < 1u ? 1u : fit > most ? most : fit;
    if (per >= a.group_blocks) return a.group_blocks;
    const uint64_t ranges = ceil_div(a.group_blocks, per) + 1u, cut = 2u * a.group_blocks / (2u * ranges - 1u);
    return (uint32_t)(cut < 1u ? 1u : cut);
}

}  // namespace
}  // namespace dwps

using namespace dwps;

extern "C" ps_status ps_selective_scan_bwd(void *ws, size_t *ws_bytes, const ps_scan_input *in, const void *dout,
                                           const float *checkpoints, const ps_scan_grads *grads, void *stream) {
    ps_status st = scan_sizes(in, true);
    if (st != PS_OK) return st;
    const size_t e = dtype_bytes(in->dtype);
    const uint64_t DN = (uint64_t)in->channels * in->states, GN = (uint64_t)in->groups * in->states;
    ScanArgs a = scan_args(in, kScanCellShift);
    const uint64_t cells = ceil_div(in->tokens, kScanCell);
    const uint64_t pieces = piece_count(in->tokens, a.num_seqs, in->offsets != nullptr, a.shift);
    const uint32_t per_range = grad_range(a, pieces);
    BackOut o{};
    o.per_range = per_range;
    o.ranges = (uint32_t)ceil_div(a.group_blocks, per_range);
    o.blocks = o.ranges * in->groups;
    PlainWs plan;
    const size_t carry_at = plan.take((cells + 1u) * DN * 4u), steps_at = plan.take((cells + 1u) * in->channels * 4u),
                 links_at = plan.take((cells + 1u) * 4u), pA_at = plan.take(pieces * DN * 4u),
                 pD_at = plan.take(pieces * in->channels * 4u), pb_at = plan.take(pieces * in->channels * 4u),
                 pB_at = plan.take(o.ranges * in->tokens * GN * 4u), pC_at = plan.take(o.ranges * in->tokens * GN * 4u);
    bool query = false;
    st = workspace_protocol(ws, ws_bytes, plan.at, &query);
    if (st != PS_OK || query) return st;
    if ((st = scan_pointers(in)) != PS_OK) return st;
    if (!grads || !grads->dA || (in->tokens && (!dout || !checkpoints || !grads->dx || !grads->ddt || !grads->dB || !grads->dC)))
        return PS_ERR_NULL;
    if (!aligned(ws, 16) || !aligned(dout, e) || !aligned(checkpoints, 4) || !aligned(grads->dx, e) ||
        !aligned(grads->ddt, e) || !aligned(grads->dz, e) || !aligned(grads->dB, e) || !aligned(grads->dC, e) ||
        !aligned(grads->dA, 4) || !aligned(grads->dD, 4) || !aligned(grads->ddt_bias, 4) || !aligned(grads->dinitial, 4))
        return PS_ERR_ALIGNMENT;
    const ScanBytes n(in);
    if (outputs_overlap({{grads->dx, n.cells}, {grads->ddt, n.cells}, {in->z ? grads->dz : nullptr, n.cells},
                         {grads->dB, n.bc}, {grads->dC, n.bc}, {grads->dA, n.A}, {grads->dD, n.channel},
                         {grads->ddt_bias, n.channel}, {grads->dinitial, n.edge}},
                        {{in->x, n.x}, {in->dt, n.dt}, {in->z, n.z}, {in->B, n.B}, {in->C, n.C}, {in->A, n.A},
                         {in->D, n.channel}, {in->dt_bias, n.channel}, {in->offsets, n.offsets}, {in->initial, n.edge},
                         {dout, n.cells}, {checkpoints, n.marks}}))
        return PS_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    o.dx = grads->dx, o.ddt = grads->ddt, o.dz = in->z ? grads->dz : nullptr, o.dinitial = grads->dinitial;
    o.part_A = ws_at<float>(ws, pA_at), o.part_D = ws_at<float>(ws, pD_at), o.part_bias = ws_at<float>(ws, pb_at);
    o.part_B = ws_at<float>(ws, pB_at), o.part_C = ws_at<float>(ws, pC_at);
    SumJobs jobs{};
    uint64_t at = 0;
    auto add = [&](const float *part, void *out, uint64_t cols, uint64_t rows, bool typed, bool guard) {
        if (!out || !cols) return;
        jobs.job[jobs.count++] = SumJob{part, out, cols, (uint32_t)rows, at, typed ? 1u : 0u, guard ? 1u : 0u};
        at += ceil_div(cols, 64);
    };
    add(o.part_A, grads->dA, DN, pieces, false, false);
    add(o.part_D, grads->dD, in->channels, pieces, false, false);
    add(o.part_bias, grads->ddt_bias, in->channels, pieces, false, false);
    if (a.num_seqs) {
        add(o.part_B, grads->dB, in->tokens * GN, o.ranges, true, true);
        add(o.part_C, grads->dC, in->tokens * GN, o.ranges, true, true);
    }
    return with_type(in->dtype, [&](auto zero) {
        using T = decltype(zero);
        float *carry = ws_at<float>(ws, carry_at), *steps = ws_at<float>(ws, steps_at);
        uint32_t *links = ws_at<uint32_t>(ws, links_at);
        timing_begin(s);
        if (pieces && cells > 1u) {
            with_states(in->states, [&](auto sc) {
                return with_full(in, decltype(sc)::value, [&](auto full) {
                    launch_in_parts(pieces, o.blocks, 2 * kScanThreads, [&](uint32_t first, uint32_t grid) {
                        a.first = first;
                        hipLaunchKernelGGL((scan_back_kernel<T, decltype(sc)::value, decltype(full)::value>), dim3(grid),
                                           dim3(2 * kScanThreads), 0, s, a, static_cast<const T *>(dout), carry, steps,
                                           links, o.ranges, o.per_range);
                    });
                    return PS_OK;
                });
            });
            launch_scan_link(a, carry, steps, links, (uint32_t)cells, true, s);
        }
        const uint32_t held = in->states > 16u ? per_range : 2u;
        // this kernel takes the states 16 at a time
        with_full(in, (uint32_t)ceil_div(in->states, kScanLanes), [&](auto full) {
            auto launch = [&](auto many) {
                launch_in_parts(pieces, o.blocks, 2 * kScanThreads, [&](uint32_t first, uint32_t grid) {
                    a.first = first;
                    hipLaunchKernelGGL((scan_grad_kernel<T, decltype(full)::value, decltype(many)::value>), dim3(grid),
                                       dim3(2 * kScanThreads), held * 3u * kScanChannels * kScanPad * 4u, s, a,
                                       static_cast<const T *>(dout), checkpoints, carry, o, ws_counter(ws), plan.words());
                });
            };
            if (in->states > 16u) launch(std::true_type());
            else launch(std::false_type());
            return PS_OK;
        });
        launch_in_parts(at, 1u, 256u, [&](uint32_t first, uint32_t grid) {
            a.first = first;
            hipLaunchKernelGGL(scan_sums_kernel<T>, dim3(grid), dim3(256), 0, s, jobs, a);
        });
        timing_end(s);
        return launch_status();
    });
}
