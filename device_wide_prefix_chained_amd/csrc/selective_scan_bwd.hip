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
// Two passes: the first walks backwards and stores a dh where it crosses from
// one cell of 32 rows to the one before (carry); then every piece of a
// sequence in a cell is worked on by itself, from the checkpoint that the
// forward pass left at the cell's first row and from the carry at its last.
// Sums over channels and over pieces go to partial sums that a last launch
// adds up in a fixed order.
#include <hip/hip_runtime.h>

#include "scan_block.hpp"

namespace dwps {
namespace {

// Two neighbouring elements, or zeros where they are not `in`.
template <class T>
__device__ __forceinline__ void load_pair(float (&v)[2], const T *p, bool in0, bool in1) {
    v[0] = in0 ? (float)p[0] : 0.0f;
    v[1] = in1 ? (float)p[1] : 0.0f;
}

// Walks backwards over a piece (a whole sequence, or its rows in one cell).
// WHOLE: stores the carry at every cell it crosses.  Otherwise stores what
// the piece adds to the carry out of its cell, and the sum of its steps.
template <class T, int S, bool WHOLE>
__global__ __launch_bounds__(kScanThreads) void scan_back_kernel(ScanArgs a, const T *__restrict__ dout,
                                                                 float *__restrict__ carry, float *__restrict__ steps,
                                                                 uint32_t *__restrict__ links) {
    __shared__ __attribute__((aligned(16))) float sStep[kScanChannels * kScanPad], sGrad[kScanChannels * kScanPad],
        sC[16 * S * kScanPad];
    const ScanPlace w = scan_place(a, xcd_neighbours(blockIdx.x, gridDim.x, sizeof(T) == 2 ? 4u : 2u));
    const Piece &q = w.q;
    if (!q.any) return;
    const uint32_t N = a.states;
    const int64_t DN = (int64_t)a.channels * N;
    if (!WHOLE) {
        if (q.lo != (uint64_t)q.cell << a.shift) return;  // starts inside its cell: nothing enters another
        const bool on = q.lo > q.seq_lo;
        if (w.ch0 == 0u && threadIdx.x == 0)
            links[q.cell] = !on ? kLinkNone
                            : (uint64_t)q.seq_hi > ((uint64_t)(q.cell + 1u) << a.shift) ? kLinkChain : kLinkStart;
        if (!on) return;
    }
    const uint32_t c2 = (threadIdx.x & 7u) * 2u, row = threadIdx.x >> 3;
    const bool in0 = c2 < w.have, in1 = c2 + 1u < w.have;
    const uint32_t cs = w.ch0 + c2;
    const float bias0 = a.bias && in0 ? a.bias[cs] : 0.0f, bias1 = a.bias && in1 ? a.bias[cs + 1] : 0.0f;
    const uint32_t lane = threadIdx.x & 63u, l = lane & 15u;
    const uint32_t cw = (threadIdx.x >> 6) * 4u + (lane >> 4);
    const uint32_t d = w.ch0 + cw;
    float A2[S], back[S], total = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const uint32_t n = s * 16 + l;
        A2[s] = cw < w.have && n < N ? a.A[(int64_t)d * N + n] * kLog2e : 0.0f;
        back[s] = 0.0f;
    }
    const uint32_t first = q.lo & ~(uint32_t)(kScanTile - 1);
    // a sequence's first cell sends nothing on
    const uint32_t stop = WHOLE ? (q.lo | (kScanCell - 1u)) + 1u : first;
    for (uint32_t end = (q.hi + kScanTile - 1u) & ~(uint32_t)(kScanTile - 1); end > stop; end -= kScanTile) {
        const uint32_t blk = end - kScanTile, t = blk + row;
        const bool live = t >= q.lo && t < q.hi;
        float dt[2], g[2], z[2];
        load_pair<T>(dt, static_cast<const T *>(a.dt) + (int64_t)t * a.dt_stride + cs, live && in0, live && in1);
        load_pair<T>(g, dout + (int64_t)t * a.channels + cs, live && in0, live && in1);
        if (a.z) {
            load_pair<T>(z, static_cast<const T *>(a.z) + (int64_t)t * a.z_stride + cs, live && in0, live && in1);
            g[0] *= silu(z[0]);
            g[1] *= silu(z[1]);
        }
        sStep[c2 * kScanPad + row] = live ? softplus(dt[0] + bias0) : 0.0f;
        sStep[(c2 + 1) * kScanPad + row] = live ? softplus(dt[1] + bias1) : 0.0f;
        sGrad[c2 * kScanPad + row] = g[0];
        sGrad[(c2 + 1) * kScanPad + row] = g[1];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const uint32_t n = s * 16 + c2;
            float v[2];
            load_pair<T>(v, static_cast<const T *>(a.C) + (int64_t)t * a.c_stride + w.group * N + n, live && n < N,
                         live && n + 1 < N);
            sC[n * kScanPad + row] = v[0];
            sC[(n + 1) * kScanPad + row] = v[1];
        }
        __syncthreads();
#pragma unroll
        for (int sub = kScanTile / 16 - 1; sub >= 0; --sub) {
            const float st = sStep[cw * kScanPad + sub * 16 + l], gr = sGrad[cw * kScanPad + sub * 16 + l];
            if (!WHOLE) total += st;
            auto token = [&](auto jc) {
                constexpr int j = 15 - decltype(jc)::value;
                const float stj = row_lane<j>(st), gj = row_lane<j>(gr);
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const float e = exp2_hw(stj * A2[s]);
                    back[s] = e * __builtin_fmaf(gj, sC[(s * 16 + l) * kScanPad + sub * 16 + j], back[s]);
                }
            };
            for_each_index(token, std::make_integer_sequence<int, 16>());
        }
        if (WHOLE && cw < w.have) {
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (s * 16 + l < N)
                    carry[(int64_t)(blk >> kScanCellShift) * DN + (int64_t)d * N + s * 16 + l] = back[s];
        }
        __syncthreads();
    }
    if (!WHOLE && cw < w.have) {
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (s * 16 + l < N) carry[(int64_t)q.cell * DN + (int64_t)d * N + s * 16 + l] = back[s];
        total = row_total(total);
        if (l == 0u) steps[(int64_t)q.cell * a.channels + d] = total;
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
// and h of the piece's 32 rows in registers between the walk forward and the
// walk back.  With more than 16 states the three sums over states wait in
// shared memory for the last 16.
template <class T>
__global__ __launch_bounds__(kScanThreads) void scan_grad_kernel(ScanArgs a, const T *__restrict__ dout,
                                                                 const float *__restrict__ marks,
                                                                 const float *__restrict__ carry, BackOut o,
                                                                 uint32_t *hdr, uint32_t words) {
    constexpr int kPlane = kScanChannels * kScanPad;
    __shared__ __attribute__((aligned(16))) float sStep[kPlane], sDrive[kPlane], sGrad[kPlane], sB[kPlane], sC[kPlane];
    __shared__ float sFold[4][8][64];
    __shared__ float sSum[4][2][kScanChannels];
    extern __shared__ float sCell[];  // [channel blocks of the range or 1][3][kPlane]
    if (blockIdx.x == 0 && threadIdx.x == 0) mark_plain(hdr, words);
    const uint32_t p = blockIdx.x / o.blocks, rg = blockIdx.x % o.blocks;
    const uint32_t group = rg / o.ranges, range = rg % o.ranges;
    const Piece q = find_piece(a.offsets, a.num_seqs, a.tokens, a.shift, p);
    const uint32_t cb0 = range * o.per_range;
    const uint32_t cb1 = cb0 + o.per_range < a.group_blocks ? cb0 + o.per_range : a.group_blocks;
    const uint32_t N = a.states;
    const int64_t DN = (int64_t)a.channels * N;
    const uint32_t c2 = (threadIdx.x & 7u) * 2u, row = threadIdx.x >> 3;
    const uint32_t lane = threadIdx.x & 63u, l = lane & 15u, wave = threadIdx.x >> 6;
    const uint32_t cw = wave * 4u + (lane >> 4);
    if (!q.any || q.lo == q.hi) {  // no rows: sums of nothing, an empty sequence's dinitial
        const uint32_t c_lo = group * a.group_channels + cb0 * kScanChannels;
        uint32_t c_hi = group * a.group_channels + cb1 * kScanChannels;
        if (c_hi > (group + 1u) * a.group_channels) c_hi = (group + 1u) * a.group_channels;
        for (int64_t i = (int64_t)c_lo * N + threadIdx.x; i < (int64_t)c_hi * N; i += kScanThreads) {
            o.part_A[p * DN + i] = 0.0f;
            if (q.any && o.dinitial) o.dinitial[q.seq * DN + i] = 0.0f;
        }
        for (uint32_t c = c_lo + threadIdx.x; c < c_hi; c += kScanThreads) {
            o.part_D[(int64_t)p * a.channels + c] = 0.0f;
            o.part_bias[(int64_t)p * a.channels + c] = 0.0f;
        }
        return;
    }
    const uint32_t blk = q.cell << kScanCellShift, t = blk + row;
    const bool live = t >= q.lo && t < q.hi;
    const bool on = (uint64_t)q.seq_hi > (uint64_t)blk + kScanCell;
    const uint32_t state_blocks = (N + 15u) / 16u;
    for (uint32_t sb = 0; sb < state_blocks; ++sb) {
        const bool last = sb + 1u == state_blocks;
        {
            const uint32_t n = sb * 16u + c2;
            float v[2];
            load_pair<T>(v, static_cast<const T *>(a.B) + (int64_t)t * a.b_stride + group * N + n, live && n < N,
                         live && n + 1 < N);
            sB[c2 * kScanPad + row] = v[0];
            sB[(c2 + 1) * kScanPad + row] = v[1];
            load_pair<T>(v, static_cast<const T *>(a.C) + (int64_t)t * a.c_stride + group * N + n, live && n < N,
                         live && n + 1 < N);
            sC[c2 * kScanPad + row] = v[0];
            sC[(c2 + 1) * kScanPad + row] = v[1];
        }
        const uint32_t n = sb * 16u + l;
        float accB[32], accC[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) accB[j] = accC[j] = 0.0f;
        for (uint32_t cb = cb0; cb < cb1; ++cb) {
            float *cell = sCell + (state_blocks > 1u ? (cb - cb0) * 3u * kPlane : 0u);
            const uint32_t ch0 = group * a.group_channels + cb * kScanChannels;
            const uint32_t left = a.group_channels - cb * kScanChannels;
            const uint32_t have = left < (uint32_t)kScanChannels ? left : kScanChannels;
            const bool in0 = c2 < have, in1 = c2 + 1u < have;
            const uint32_t cs = ch0 + c2;
            float x[2], raw[2], dy[2], z[2] = {0.0f, 0.0f}, g[2], st[2];
            load_pair<T>(x, static_cast<const T *>(a.x) + (int64_t)t * a.x_stride + cs, live && in0, live && in1);
            load_pair<T>(raw, static_cast<const T *>(a.dt) + (int64_t)t * a.dt_stride + cs, live && in0, live && in1);
            load_pair<T>(dy, dout + (int64_t)t * a.channels + cs, live && in0, live && in1);
            if (a.z)
                load_pair<T>(z, static_cast<const T *>(a.z) + (int64_t)t * a.z_stride + cs, live && in0, live && in1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool in = i ? in1 : in0;
                raw[i] += a.bias && in ? a.bias[cs + i] : 0.0f;
                st[i] = live ? softplus(raw[i]) : 0.0f;
                g[i] = a.z ? dy[i] * silu(z[i]) : dy[i];
                sStep[(c2 + i) * kScanPad + row] = st[i];
                sDrive[(c2 + i) * kScanPad + row] = st[i] * x[i];
                sGrad[(c2 + i) * kScanPad + row] = g[i];
            }
            const uint32_t d = ch0 + cw;
            const bool in = cw < have && n < N;
            const int64_t at = (int64_t)d * N + n;
            const float A = in ? a.A[at] : 0.0f, A2 = A * kLog2e;
            float h0 = 0.0f, back = 0.0f;
            if (in) {
                if (q.lo > q.seq_lo) h0 = marks[(int64_t)q.cell * DN + at];
                else if (a.initial) h0 = a.initial[(int64_t)q.seq * DN + at];
                if (on) back = carry[(int64_t)(q.cell + 1u) * DN + at];
            }
            __syncthreads();
            float e[32], h[32], y[16];
            float stv[2], drv[2], grv[2];
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                stv[sub] = sStep[cw * kScanPad + sub * 16 + l];
                drv[sub] = sDrive[cw * kScanPad + sub * 16 + l];
                grv[sub] = sGrad[cw * kScanPad + sub * 16 + l];
            }
            float run = h0;
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                auto token = [&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    const int k = sub * 16 + j;
                    e[k] = exp2_hw(row_lane<j>(stv[sub]) * A2);
                    run = __builtin_fmaf(e[k], run, row_lane<j>(drv[sub]) * sB[l * kScanPad + k]);
                    h[k] = run;
                    y[j] = run * sC[l * kScanPad + k];
                };
                for_each_index(token, std::make_integer_sequence<int, 16>());
                const float v = row_sums(y, lane);
                float *to = cell + cw * kScanPad + sub * 16 + l;
                *to = sb ? *to + v : v;
            }
            float sumA = 0.0f;
#pragma unroll
            for (int sub = 1; sub >= 0; --sub) {
                float along[16], flowA[16];
                auto token = [&](auto jc) {
                    constexpr int j = 15 - decltype(jc)::value;
                    const int k = sub * 16 + j;
                    const float gj = row_lane<j>(grv[sub]);
                    const float dh = __builtin_fmaf(gj, sC[l * kScanPad + k], back);
                    accC[k] = __builtin_fmaf(gj, h[k], accC[k]);
                    accB[k] = __builtin_fmaf(row_lane<j>(drv[sub]), dh, accB[k]);
                    back = e[k] * dh;
                    const float flow = back * (k ? h[k ? k - 1 : 0] : h0);
                    sumA = __builtin_fmaf(flow, row_lane<j>(stv[sub]), sumA);
                    along[j] = dh * sB[l * kScanPad + k];
                    flowA[j] = flow * A;
                };
                for_each_index(token, std::make_integer_sequence<int, 16>());
                const float va = row_sums(along, lane), vf = row_sums(flowA, lane);
                float *to = cell + kPlane + cw * kScanPad + sub * 16 + l;
                to[0] = sb ? to[0] + va : va;
                to[kPlane] = sb ? to[kPlane] + vf : vf;
            }
            if (in) {
                o.part_A[p * DN + at] = sumA;
                if (o.dinitial && q.lo == q.seq_lo) o.dinitial[(int64_t)q.seq * DN + at] = back;
            }
            __syncthreads();
            if (last) {
                float sx[2], sd[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool have_c = i ? in1 : in0;
                    const float skip = a.D && have_c ? a.D[cs + i] : 0.0f;
                    const float *c = cell + (c2 + i) * kScanPad + row;
                    const float ddt = __builtin_fmaf(x[i], c[kPlane], c[2 * kPlane]) * sigmoid(raw[i]);
                    sx[i] = live ? g[i] * x[i] : 0.0f;
                    sd[i] = live ? ddt : 0.0f;
                    if (live && have_c) {
                        const int64_t to = (int64_t)t * a.channels + cs + i;
                        static_cast<T *>(o.dx)[to] = (T)__builtin_fmaf(skip, g[i], st[i] * c[kPlane]);
                        static_cast<T *>(o.ddt)[to] = (T)ddt;
                        if (o.dz)
                            static_cast<T *>(o.dz)[to] =
                                (T)(dy[i] * __builtin_fmaf(skip, x[i], c[0]) * dsilu(z[i], sigmoid(z[i])));
                    }
                }
                // over the wave's 8 tokens, then the 4 waves
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int m = 8; m < 64; m *= 2) {
                        sx[i] += __shfl_xor(sx[i], m);
                        sd[i] += __shfl_xor(sd[i], m);
                    }
                    if (lane < 8u) {
                        sSum[wave][0][c2 + i] = sx[i];
                        sSum[wave][1][c2 + i] = sd[i];
                    }
                }
                __syncthreads();
                if (threadIdx.x < 32u) {
                    const uint32_t which = threadIdx.x >> 4, c = threadIdx.x & 15u;
                    if (c < have) {
                        const float v = ((sSum[0][which][c] + sSum[1][which][c]) + sSum[2][which][c]) + sSum[3][which][c];
                        (which ? o.part_bias : o.part_D)[(int64_t)p * a.channels + ch0 + c] = v;
                    }
                }
            }
        }
        // dB, dC over the range's channels: rows of a wave, then the waves
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float f[8];
            if (which) fold_rows(f, accC);
            else fold_rows(f, accB);
#pragma unroll
            for (int j = 0; j < 8; ++j) sFold[wave][j][lane] = f[j];
            __syncthreads();
            float *part = which ? o.part_C : o.part_B;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t i = r * 256u + threadIdx.x, j = i >> 6, ln = i & 63u;
                const float v = ((sFold[0][j][ln] + sFold[1][j][ln]) + sFold[2][j][ln]) + sFold[3][j][ln];
                const uint32_t tk = blk + (ln >> 4) * 8u + j, nn = sb * 16u + (ln & 15u);
                if (tk >= q.lo && tk < q.hi && nn < N)
                    part[(((int64_t)range * a.tokens + tk) * a.groups + group) * N + nn] = v;
            }
            __syncthreads();
        }
    }
}

// The last launch: column sums of partial sums, several at once.
struct SumJob {
    const float *part;
    void *out;
    uint64_t cols;
    uint32_t rows;
    uint32_t first;   // workgroup
    uint32_t typed;   // the activations' type, not fp32
    uint32_t guard;   // rows of tokens outside every sequence stay unwritten
};
struct SumJobs {
    SumJob job[5];
    uint32_t count;
};

template <class T>
__global__ __launch_bounds__(256) void scan_sums_kernel(SumJobs jobs, ScanArgs a) {
    __shared__ float s[4][64];
    uint32_t k = 0;
    while (k + 1u < jobs.count && blockIdx.x >= jobs.job[k + 1u].first) ++k;
    const SumJob j = jobs.job[k];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint64_t col = (uint64_t)(blockIdx.x - j.first) * 64u + lane;
    float v = 0.0f;
    if (col < j.cols)
        for (uint32_t r = wave; r < j.rows; r += 4u) v += j.part[r * j.cols + col];
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

bool back_split(const ps_scan_input *) { return false; }

}  // namespace
}  // namespace dwps

using namespace dwps;

extern "C" ps_status ps_selective_scan_bwd(void *ws, size_t *ws_bytes, const ps_scan_input *in, const void *dout,
                                           const float *checkpoints, const ps_scan_grads *grads, void *stream) {
    ps_status st = scan_sizes(in, true);
    if (st != PS_OK) return st;
    const size_t e = dtype_bytes(in->dtype);
    const uint64_t DN = (uint64_t)in->channels * in->states, GN = (uint64_t)in->groups * in->states;
    const bool split = back_split(in);
    const ScanArgs a = scan_args(in, kScanCellShift);
    const uint64_t cells = ceil_div(in->tokens, kScanCell);
    const uint64_t pieces = piece_count(in->tokens, a.num_seqs, in->offsets != nullptr, a.shift);
    const uint32_t per_range = a.group_blocks < 4u ? a.group_blocks : 4u;
    BackOut o{};
    o.per_range = per_range;
    o.ranges = (uint32_t)ceil_div(a.group_blocks, per_range);
    o.blocks = o.ranges * in->groups;
    PlainWs plan;
    const size_t carry_at = plan.take((cells + 1u) * DN * 4u), steps_at = plan.take((cells + 1u) * in->channels * 4u),
                 links_at = plan.take((cells + 1u) * 4u), pA_at = plan.take(pieces * DN * 4u),
                 pD_at = plan.take(pieces * in->channels * 4u), pb_at = plan.take(pieces * in->channels * 4u),
                 pB_at = plan.take(o.ranges * in->tokens * GN * 4u), pC_at = plan.take(o.ranges * in->tokens * GN * 4u);
    const uint64_t grid = pieces * o.blocks;
    const ScanArgs wa = scan_args(in, split ? kScanCellShift : 32u);
    const uint64_t back_grid = piece_count(in->tokens, a.num_seqs, in->offsets != nullptr, wa.shift) * wa.col_blocks;
    if (grid > kScanMaxGrid || back_grid > kScanMaxGrid) return PS_ERR_SIZE;
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
    const size_t cell_bytes = in->tokens * in->channels * e, bc_bytes = in->tokens * GN * e;
    for (const void *p : {grads->dx, grads->ddt, grads->dz})
        if (scan_overlaps(in, p, cell_bytes) || (p && ranges_overlap(p, cell_bytes, dout, cell_bytes))) return PS_ERR_ALIAS;
    for (const void *p : {grads->dB, grads->dC})
        if (scan_overlaps(in, p, bc_bytes) || (p && ranges_overlap(p, bc_bytes, dout, cell_bytes))) return PS_ERR_ALIAS;
    hipStream_t s = static_cast<hipStream_t>(stream);
    o.dx = grads->dx, o.ddt = grads->ddt, o.dz = in->z ? grads->dz : nullptr, o.dinitial = grads->dinitial;
    o.part_A = ws_at<float>(ws, pA_at), o.part_D = ws_at<float>(ws, pD_at), o.part_bias = ws_at<float>(ws, pb_at);
    o.part_B = ws_at<float>(ws, pB_at), o.part_C = ws_at<float>(ws, pC_at);
    SumJobs jobs{};
    uint64_t at = 0;
    auto add = [&](const float *part, void *out, uint64_t cols, uint64_t rows, bool typed, bool guard) {
        if (!out || !cols) return;
        jobs.job[jobs.count++] = SumJob{part, out, cols, (uint32_t)rows, (uint32_t)at, typed ? 1u : 0u, guard ? 1u : 0u};
        at += ceil_div(cols, 64);
    };
    add(o.part_A, grads->dA, DN, pieces, false, false);
    add(o.part_D, grads->dD, in->channels, pieces, false, false);
    add(o.part_bias, grads->ddt_bias, in->channels, pieces, false, false);
    if (a.num_seqs) {
        add(o.part_B, grads->dB, in->tokens * GN, o.ranges, true, true);
        add(o.part_C, grads->dC, in->tokens * GN, o.ranges, true, true);
    }
    if (at > kScanMaxGrid) return PS_ERR_SIZE;
    return with_type(in->dtype, [&](auto zero) {
        using T = decltype(zero);
        float *carry = ws_at<float>(ws, carry_at), *steps = ws_at<float>(ws, steps_at);
        uint32_t *links = ws_at<uint32_t>(ws, links_at);
        timing_begin(s);
        if (back_grid && in->tokens) {
            with_states(in->states, [&](auto sc) {
                constexpr int S = decltype(sc)::value;
                if (split) {
                    hipLaunchKernelGGL((scan_back_kernel<T, S, false>), dim3((uint32_t)back_grid), dim3(kScanThreads), 0,
                                       s, wa, static_cast<const T *>(dout), carry, steps, links);
                    launch_scan_link(wa, carry, steps, links, (uint32_t)cells, true, s);
                } else {
                    hipLaunchKernelGGL((scan_back_kernel<T, S, true>), dim3((uint32_t)back_grid), dim3(kScanThreads), 0,
                                       s, wa, static_cast<const T *>(dout), carry, steps, links);
                }
                return PS_OK;
            });
        }
        if (grid) {
            const uint32_t held = in->states > 16u ? per_range : 1u;
            hipLaunchKernelGGL(scan_grad_kernel<T>, dim3((uint32_t)grid), dim3(kScanThreads),
                               held * 3u * kScanChannels * kScanPad * 4u, s, a, static_cast<const T *>(dout), checkpoints,
                               carry, o, ws_counter(ws), plan.words());
        }
        hipLaunchKernelGGL(scan_sums_kernel<T>, dim3((uint32_t)at), dim3(256), 0, s, jobs, a);
        timing_end(s);
        return launch_status();
    });
}
