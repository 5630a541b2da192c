// selective_scan.hip -- the selective scan of a state space block: forward
// over packed sequences and the form for single tokens.
//
//   step = softplus(dt + bias),  a = exp(step A),  h <- a h + step B x
//   out = (C . h + D x) * silu(z)
#include <hip/hip_runtime.h>

#include "scan_block.hpp"

namespace dwps {
namespace {

// One walk over a piece.  OUT: outputs, final states and checkpoints, from
// the initial states or from carry[cell].  Otherwise: only what the piece
// adds to the states that enter the next cell (carry[cell + 1]) and the sum
// of its steps, for pieces that go on there.
//
// Four waves walk and four feed them.  A feeding thread loads its pair of a
// block of 32 tokens kAhead blocks before its turn, writes step, step x, B
// and C as fp32 into one half of shared memory while the walking waves work
// on the other, and gates and stores the outputs of the block before; one
// barrier a block.  The walk is bound by arithmetic: for every state exp2
// (two issue slots) and 4 more operations (the broadcasts of step and step x
// are part of the products), and 33 for 16 sums over states.  8191 x 4096 x 16
// states, bf16, one sequence (a walking wave for each SIMD): 191 to 207 us, 77%
// of the vector issue slots taken; without waves that feed 289 us, without the
// walking waves' priority 215 us.
template <class T, int S, bool OUT, bool FULL>
__global__ __launch_bounds__(2 * kScanThreads) void scan_walk_kernel(ScanArgs a, T *__restrict__ out,
                                                                     float *__restrict__ fin, float *__restrict__ marks,
                                                                     float *__restrict__ carry, float *__restrict__ steps,
                                                                     uint32_t *__restrict__ links, uint32_t *hdr,
                                                                     uint32_t words) {
    constexpr int kPlane = kScanChannels * kScanPad;
    constexpr int kAhead = S <= 4 ? 4 : 2;  // even: the halves of shared memory go round with it
    __shared__ __attribute__((aligned(16))) float sStep[2][kPlane], sDrive[2][kPlane], sY[2][OUT ? kPlane : 1],
        sB[2][16 * S * kScanPad], sC[2][OUT ? 16 * S * kScanPad : 1];
    if (!OUT && blockIdx.x == 0 && threadIdx.x == 0) mark_plain(hdr, words);
    const ScanPlace w = scan_place(a, xcd_neighbours(blockIdx.x, gridDim.x, sizeof(T) == 2 ? 4u : 2u));
    const Piece &q = w.q;
    if (!q.any) return;
    const uint32_t N = a.states;
    const int64_t DN = (int64_t)a.channels * N;
    if (!OUT) {
        const uint64_t cell_end = (uint64_t)(q.cell + 1u) << a.shift;
        if (q.hi != cell_end) return;  // reaches no further cell
        const bool on = q.seq_hi > q.hi;
        if (w.ch0 == 0u && threadIdx.x == 0)
            links[q.cell + 1u] = !on ? kLinkNone : q.lo == q.seq_lo ? kLinkStart : kLinkChain;
        if (!on) return;
    }
    const uint32_t first = q.lo & ~(uint32_t)(kScanTile - 1);
    const uint32_t blocks = q.lo < q.hi ? (q.hi - first + kScanTile - 1u) / kScanTile : 0u;
    const bool feeds = __builtin_amdgcn_readfirstlane(threadIdx.x) < (uint32_t)kScanThreads;
    if (feeds) {
        if (blocks == 0u) return;
        // two channels (and two states of each 16) of one token
        const uint32_t c2 = (threadIdx.x & 7u) * 2u, row = threadIdx.x >> 3;
        const bool in0 = FULL || c2 < w.have, in1 = FULL || c2 + 1u < w.have;
        const uint32_t o0 = FULL ? c2 : inside(c2, w.have), o1 = FULL ? c2 + 1u : inside(c2 + 1u, w.have);
        const uint32_t cs = w.ch0 + c2;
        const float bias0 = a.bias && in0 ? a.bias[cs] : 0.0f, bias1 = a.bias && in1 ? a.bias[cs + 1] : 0.0f;
        const float skip0 = OUT && a.D && in0 ? a.D[cs] : 0.0f, skip1 = OUT && a.D && in1 ? a.D[cs + 1] : 0.0f;
        const bool gated = OUT && a.z;
        struct Raw {
            RawPair<T, FULL> x, dt, z, B[S], C[OUT ? S : 1];
        };
        PairRows<T, FULL> rx{static_cast<const T *>(a.x) + w.ch0, a.x_stride};
        PairRows<T, FULL> rdt{static_cast<const T *>(a.dt) + w.ch0, a.dt_stride};
        // without a gate: any row, not used
        PairRows<T, FULL> rz{static_cast<const T *>(gated ? a.z : a.x) + w.ch0, gated ? a.z_stride : a.x_stride};
        PairRows<T, FULL> rB[S], rC[OUT ? S : 1];
        auto place = [&](uint32_t r) {
            rx.place(r, o0, o1);
            rdt.place(r, o0, o1);
            if (OUT) rz.place(r, o0, o1);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const uint32_t n = s * 16 + c2, n0 = FULL ? n : inside(n, N), n1 = FULL ? n + 1u : inside(n + 1u, N);
                rB[s] = {static_cast<const T *>(a.B) + (int64_t)w.group * N, a.b_stride};
                rB[s].place(r, n0, n1);
                if (OUT) {
                    rC[s] = {static_cast<const T *>(a.C) + (int64_t)w.group * N, a.c_stride};
                    rC[s].place(r, n0, n1);
                }
            }
        };
        place(row);
        auto load = [&](Raw &r, uint32_t k) {
            uint32_t blk = first + k * kScanTile;
            if (blk + kScanTile > a.tokens) {  // rows past the last repeat it; staging drops them
                if (blk >= a.tokens) blk = a.tokens - 1u;
                place(row < a.tokens - 1u - blk ? row : a.tokens - 1u - blk);
            }
            rx.load(r.x, blk);
            rdt.load(r.dt, blk);
            if (OUT) rz.load(r.z, blk);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                rB[s].load(r.B[s], blk);
                if (OUT) rC[s].load(r.C[s], blk);
            }
        };
        RawPair<T, FULL> kept_x[2], kept_z[2];
        const uint32_t out_byte = (row * a.channels + c2) * (uint32_t)sizeof(T);
        auto stage = [&](Raw &r, uint32_t k, int half) {
            const uint32_t t = first + k * kScanTile + row;
            const bool live = t >= q.lo && t < q.hi;
            float x[2], v[2];
            r.x.values(x, live && in0, live && in1);
            r.dt.values(v, true, true);
            const float st0 = softplus(live && in0 ? v[0] + bias0 : kNoStep);
            const float st1 = softplus(live && in1 ? v[1] + bias1 : kNoStep);
            sStep[half][c2 * kScanPad + row] = st0;
            sStep[half][(c2 + 1) * kScanPad + row] = st1;
            sDrive[half][c2 * kScanPad + row] = st0 * x[0];
            sDrive[half][(c2 + 1) * kScanPad + row] = st1 * x[1];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const uint32_t n = s * 16 + c2;
                r.B[s].values(v, live && (FULL || n < N), live && (FULL || n + 1u < N));
                sB[half][n * kScanPad + row] = v[0];
                sB[half][(n + 1) * kScanPad + row] = v[1];
                if (OUT) {
                    r.C[s].values(v, live && (FULL || n < N), live && (FULL || n + 1u < N));
                    sC[half][n * kScanPad + row] = v[0];
                    sC[half][(n + 1) * kScanPad + row] = v[1];
                }
            }
            if (OUT) kept_x[half] = r.x, kept_z[half] = r.z;
            load(r, k + kAhead);
        };
        auto store = [&](uint32_t k, int half) {
            const uint32_t blk = first + k * kScanTile, t = blk + row;
            if (t < q.lo || t >= q.hi) return;
            float x[2], z[2];
            kept_x[half].values(x, true, true);
            float y0 = __builtin_fmaf(skip0, x[0], sY[half][c2 * kScanPad + row]);
            float y1 = __builtin_fmaf(skip1, x[1], sY[half][(c2 + 1) * kScanPad + row]);
            if (gated) {
                kept_z[half].values(z, true, true);
                y0 *= silu(z[0]);
                y1 *= silu(z[1]);
            }
            T *o = reinterpret_cast<T *>(reinterpret_cast<char *>(out + (int64_t)blk * a.channels + w.ch0) + out_byte);
            if (FULL) {
                *reinterpret_cast<Pack<T, 2> *>(o) = Pack<T, 2>{{(T)y0, (T)y1}};
            } else {
                if (in0) o[0] = (T)y0;
                if (in1) o[1] = (T)y1;
            }
        };
        Raw raw[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(raw[i], i);
        stage(raw[0], 0u, 0);
        __syncthreads();
        auto turn = [&](uint32_t k, int i) {
            if (OUT && k > 0u) store(k - 1u, (i + 1) & 1);
            stage(raw[(i + 1) % kAhead], k + 1u, (i + 1) & 1);
            __syncthreads();
        };
        // Whole rounds of the ring without a branch around any load: only
        // then does the compiler wait for the oldest loads alone.  Past the
        // last block there are only dropped rows to stage.
        uint32_t k = 0;
        for (; k + kAhead <= blocks; k += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) turn(k + i, i);
        }
#pragma unroll
        for (int i = 0; i < kAhead - 1; ++i)
            if (k + i < blocks) turn(k + i, i);
        if (OUT && (blocks & 1u)) store(blocks - 1u, 0);
        if (OUT && !(blocks & 1u)) store(blocks - 1u, 1);
        return;
    }
    // walking: one channel of a row of lanes
    const uint32_t lane = threadIdx.x & 63u, l = lane & 15u;
    const uint32_t cw = ((threadIdx.x - kScanThreads) >> 6) * 4u + (lane >> 4);
    const uint32_t d = w.ch0 + cw;
    float A2[S], h[S], total = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const uint32_t n = s * 16 + l;
        const bool in = cw < w.have && n < N;
        A2[s] = in ? a.A[(int64_t)d * N + n] * kLog2e : 0.0f;
        h[s] = 0.0f;
        if (in) {
            if (q.lo == q.seq_lo) h[s] = a.initial ? a.initial[(int64_t)q.seq * DN + (int64_t)d * N + n] : 0.0f;
            else if (OUT) h[s] = carry[(int64_t)q.cell * DN + (int64_t)d * N + n];
        }
    }
    auto walk = [&](uint32_t k, int half) {
        const uint32_t blk = first + k * kScanTile;
        if (OUT && marks && blk > q.seq_lo && (blk & (kScanCell - 1u)) == 0u && cw < w.have) {
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (s * 16 + l < N) marks[(int64_t)(blk >> kScanCellShift) * DN + (int64_t)d * N + s * 16 + l] = h[s];
        }
#pragma unroll
        for (int sub = 0; sub < kScanTile / 16; ++sub) {
            const float st = sStep[half][cw * kScanPad + sub * 16 + l], dr = sDrive[half][cw * kScanPad + sub * 16 + l];
            if (!OUT) total += st;
            float y[16];
            auto token = [&](auto jc) {
                constexpr int j = decltype(jc)::value;
                const float stj = row_lane<j>(st), drj = row_lane<j>(dr);
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const float e = exp2_hw(stj * A2[s]);
                    h[s] = __builtin_fmaf(e, h[s], drj * sB[half][(s * 16 + l) * kScanPad + sub * 16 + j]);
                    if (OUT) {
                        const float c = sC[half][(s * 16 + l) * kScanPad + sub * 16 + j];
                        y[j] = s ? __builtin_fmaf(h[s], c, y[j]) : h[s] * c;
                    }
                }
            };
            for_each_index(token, std::make_integer_sequence<int, 16>());
            if (OUT) sY[half][cw * kScanPad + sub * 16 + l] = row_sums(y, lane);
        }
    };
    __builtin_amdgcn_s_setprio(2);  // the feeding waves fill the gaps
    if (blocks) __syncthreads();
    for (uint32_t k = 0; k < blocks; k += 2u) {
        walk(k, 0);
        __syncthreads();
        if (k + 1u < blocks) {
            walk(k + 1u, 1);
            __syncthreads();
        }
    }
    if (OUT) {
        if (fin && q.hi == q.seq_hi && cw < w.have) {
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (s * 16 + l < N) fin[(int64_t)q.seq * DN + (int64_t)d * N + s * 16 + l] = h[s];
        }
    } else if (cw < w.have) {
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (s * 16 + l < N) carry[(int64_t)(q.cell + 1u) * DN + (int64_t)d * N + s * 16 + l] = h[s];
        total = row_total(total);
        if (l == 0u) steps[(int64_t)(q.cell + 1u) * a.channels + d] = total;
    }
}

// One (channel, state) per lane, from cell to cell; 256 cells of 2048 x 16 take
// 23 us (2.9 TB/s, each load 256 bytes of a row of its own).  The loads of 32
// cells are on their way at once (64 take all registers, for 7% less).
__global__ __launch_bounds__(64) void scan_link_kernel(ScanArgs a, float *__restrict__ carry,
                                                        const float *__restrict__ steps,
                                                        const uint32_t *__restrict__ links, uint32_t cells,
                                                        int backward) {
    const int64_t i = (int64_t)(a.first + blockIdx.x) * 64 + threadIdx.x;
    const int64_t DN = (int64_t)a.channels * a.states;
    if (i >= DN) return;
    const uint32_t d = (uint32_t)(i / a.states);
    const float A2 = a.A[i] * kLog2e;
    float h = 0.0f;
    auto batch = [&](uint32_t k0, auto count) {
        constexpr int U = decltype(count)::value;
        float v[U], keep[U];
        uint32_t link[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t c = backward ? cells - (k0 + u) : k0 + u;
            v[u] = carry[c * DN + i];
            keep[u] = steps[(int64_t)c * a.channels + d];
            link[u] = links[c];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t c = backward ? cells - (k0 + u) : k0 + u;
            // a chain starts anew where nothing enters (steps are not written there)
            h = link[u] == kLinkChain ? __builtin_fmaf(exp2_hw(A2 * keep[u]), h, v[u]) : v[u];
            carry[c * DN + i] = h;
        }
    };
    uint32_t k = 1;
    for (; k + 32u <= cells; k += 32u) batch(k, std::integral_constant<int, 32>());
    for (; k + 8u <= cells; k += 8u) batch(k, std::integral_constant<int, 8>());
    for (; k < cells; ++k) batch(k, std::integral_constant<int, 1>());
}

// One token for each row.  A lane holds 4 states of one channel (16 bytes of
// the state, where VEC: the states are a multiple of 4), a power of two
// `lanes` of them a channel, and a workgroup takes `each` rows: A, as large as
// a row's states, is read once for them.  Bound by memory, the states once in
// and once out; the next row's are on their way while one is worked on.
// 384 rows x 4096 x 16 states: 46 us (4.7 TB/s); one row of 1536 channels: 3 us.
template <class T, bool VEC>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanArgs a, const float *state, float *new_state,
                                                        const int32_t *__restrict__ slots, uint32_t pool,
                                                        T *__restrict__ out, uint32_t lanes, uint32_t blocks,
                                                        uint32_t each) {
    const uint32_t at = blockIdx.x % blocks * 256u + threadIdx.x;
    const uint32_t i0 = (a.first + blockIdx.x / blocks) * each, i1 = i0 + each < a.tokens ? i0 + each : a.tokens;
    const uint32_t N = a.states, own = at / lanes, n = at % lanes * 4u;
    // lanes past the last channel or state work on one that exists and store nothing
    const uint32_t d = own < a.channels ? own : a.channels - 1u;
    const bool in = own < a.channels && n < N;
    const uint32_t n0 = n < N ? n : VEC ? N - 4u : N - 1u;
    const uint32_t g = d / a.group_channels;
    uint32_t off[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) off[k] = VEC || n0 + k < N ? k : 0u;
    struct Row {
        float h[4], x, dt, z;
        T b[4], c[4];
        int64_t slot;
    };
    auto fetch = [&](Row &r, uint32_t i) {
        if (i >= i1) i = i1 - 1u;
        const int64_t slot = slots ? (int64_t)slots[i] : (int64_t)i;
        r.slot = slot >= 0 && slot < (int64_t)pool ? slot : -1;
        const T *b = static_cast<const T *>(a.B) + (int64_t)i * a.b_stride + g * N + n0;
        const T *c = static_cast<const T *>(a.C) + (int64_t)i * a.c_stride + g * N + n0;
        // padding reads a slot that exists and drops it (any floats where there is none)
        const float *h = (pool ? state + ((r.slot < 0 ? 0 : r.slot) * a.channels + d) * (int64_t)N : a.A + (int64_t)d * N) + n0;
        if (VEC) {
            const Pack<float, 4> hv = *reinterpret_cast<const Pack<float, 4> *>(h);
            const Pack<T, 4> bv = *reinterpret_cast<const Pack<T, 4> *>(b), cv = *reinterpret_cast<const Pack<T, 4> *>(c);
#pragma unroll
            for (int k = 0; k < 4; ++k) r.h[k] = hv.v[k], r.b[k] = bv.v[k], r.c[k] = cv.v[k];
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) r.h[k] = h[off[k]], r.b[k] = b[off[k]], r.c[k] = c[off[k]];
        }
        r.x = (float)static_cast<const T *>(a.x)[(int64_t)i * a.x_stride + d];
        r.dt = (float)static_cast<const T *>(a.dt)[(int64_t)i * a.dt_stride + d];
        r.z = a.z ? (float)static_cast<const T *>(a.z)[(int64_t)i * a.z_stride + d] : 0.0f;
    };
    Row next;
    fetch(next, i0);
    float A2[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) A2[k] = a.A[(int64_t)d * N + n0 + off[k]] * kLog2e;
    const float bias = a.bias ? a.bias[d] : 0.0f, skip = a.D ? a.D[d] : 0.0f;
    for (uint32_t i = i0; i < i1; ++i) {
        const Row r = next;
        if (i + 1u < i1) fetch(next, i + 1u);
        const float step = softplus(r.dt + bias), drive = step * r.x;
        float h[4], sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = __builtin_fmaf(exp2_hw(step * A2[k]), r.slot < 0 ? 0.0f : r.h[k], drive * (float)r.b[k]);
            if (n < N && (VEC || n + k < N)) sum = __builtin_fmaf(h[k], (float)r.c[k], sum);
        }
        if (in && r.slot >= 0) {
            float *to = new_state + (r.slot * a.channels + d) * (int64_t)N + n;
            if (VEC) {
                *reinterpret_cast<Pack<float, 4> *>(to) = Pack<float, 4>{{h[0], h[1], h[2], h[3]}};
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (n + k < N) to[k] = h[k];
            }
        }
        for (uint32_t m = lanes / 2u; m; m /= 2u) sum += __shfl_xor(sum, (int)m);
        if (in && n == 0u) {
            const float y = __builtin_fmaf(skip, r.x, sum);
            out[(int64_t)i * a.channels + d] = (T)(a.z ? y * silu(r.z) : y);
        }
    }
}

// Rows of a piece, as a power of two: 32 for whole sequences, or less where
// those leave too much of the GPU idle.  Then cells of sequences are walked
// side by side, after a first walk for the states that enter them, which
// computes every decay twice.  Counted in turns (32 tokens of 16 channels on
// one of 256 CUs, 0.75 us): whole sequences take the longer of the longest
// sequence (random cuts: (1 + ln seqs) / seqs of the rows) and an even share;
// cells 1.75 shares and about 30 turns for two more launches, and the link of
// 32 cells about 4.  Cells are as long as leaves four workgroups for a CU.
// The lengths are on the device and not looked at: one long sequence among many
// short ones is walked whole (16384 rows of 512 channels in 41 sequences, one
// of 16000 rows: 367 us).
// Both sides in us, bf16, 16 states, one sequence, whole / cells: 16384 rows
// of 64 channels 358 / 46, 512: 359 / 88, 1024: 361 / 151, 2048: 364 / 273
// (4096: 387 whole); 256 channels of 4096 rows 91 / 33, 2048: 48 / 29 (1024:
// 26 whole).
uint32_t scan_shift(const ps_scan_input *in) {
    const ScanArgs a = scan_args(in, 32u);
    const double blocks = (double)ceil_div(in->tokens, kScanTile), share = blocks * a.col_blocks / 256.0;
    const uint32_t seqs = a.num_seqs ? a.num_seqs : 1u;
    const double longest = blocks * (1.0 + 0.6931 * (31 - __builtin_clz(seqs))) / seqs;
    const double whole = longest > share ? longest : share;
    uint32_t shift = kScanCellShift;
    while (shift < 9u && ceil_div(in->tokens, 2ull << shift) * a.col_blocks >= 1024u) ++shift;
    const double cells = (double)ceil_div(in->tokens, 1ull << shift);
    return 1.75 * share + 30.0 + cells / 8.0 < whole ? shift : 32u;
}

}  // namespace

ScanArgs scan_args(const ps_scan_input *in, uint32_t shift) {
    ScanArgs a{};
    a.x = in->x, a.dt = in->dt, a.z = in->z, a.B = in->B, a.C = in->C;
    a.A = in->A, a.D = in->D, a.bias = in->dt_bias, a.initial = in->initial;
    a.offsets = in->offsets;
    a.x_stride = in->x_stride, a.dt_stride = in->dt_stride, a.z_stride = in->z_stride;
    a.b_stride = in->b_stride, a.c_stride = in->c_stride;
    a.tokens = (uint32_t)in->tokens, a.channels = in->channels, a.groups = in->groups, a.states = in->states;
    a.num_seqs = in->offsets ? in->num_seqs : 1u;
    a.shift = shift;
    a.group_channels = in->channels / in->groups;
    a.group_blocks = (uint32_t)ceil_div(a.group_channels, kScanChannels);
    a.col_blocks = in->groups * a.group_blocks;
    return a;
}

ps_status scan_sizes(const ps_scan_input *in, bool packed) {
    if (!in) return PS_ERR_NULL;
    if (!dtype_bytes(in->dtype)) return PS_ERR_UNSUPPORTED;
    const int64_t c = in->channels, gn = (int64_t)in->groups * in->states;
    if (in->tokens > kBlockMaxTokens || in->channels == 0u || in->channels > kBlockMaxChannels || in->groups == 0u ||
        in->groups > in->channels || in->channels % in->groups || in->states == 0u || in->states > PS_SCAN_MAX_STATES ||
        in->num_seqs > kBlockMaxSeqs || in->x_stride < c || in->dt_stride < c || (in->z && in->z_stride < c) ||
        in->b_stride < gn || in->c_stride < gn || in->x_stride > kBlockMaxStride || in->dt_stride > kBlockMaxStride ||
        (in->z && in->z_stride > kBlockMaxStride) || in->b_stride > kBlockMaxStride || in->c_stride > kBlockMaxStride)
        return PS_ERR_SIZE;
    if ((uint64_t)in->groups * ceil_div(in->channels / in->groups, kScanChannels) > kScanMaxBlocks) return PS_ERR_SIZE;
    if (packed && !in->offsets && in->num_seqs > 1u) return PS_ERR_SIZE;
    return PS_OK;
}

ps_status scan_pointers(const ps_scan_input *in) {
    const size_t e = dtype_bytes(in->dtype);
    if (!in->A || (in->tokens && (!in->x || !in->dt || !in->B || !in->C))) return PS_ERR_NULL;
    if (!aligned(in->x, e) || !aligned(in->dt, e) || !aligned(in->z, e) || !aligned(in->B, e) || !aligned(in->C, e) ||
        !aligned(in->A, 4) || !aligned(in->D, 4) || !aligned(in->dt_bias, 4) || !aligned(in->offsets, 4) ||
        !aligned(in->initial, 4))
        return PS_ERR_ALIGNMENT;
    return PS_OK;
}

void launch_scan_link(const ScanArgs &a, float *carry, const float *steps, const uint32_t *links, uint32_t cells,
                      bool backward, hipStream_t s) {
    launch_in_parts(ceil_div((uint64_t)a.channels * a.states, 64), 1u, 64u, [&](uint32_t first, uint32_t grid) {
        ScanArgs part = a;
        part.first = first;
        hipLaunchKernelGGL(scan_link_kernel, dim3(grid), dim3(64), 0, s, part, carry, steps, links, cells, backward ? 1 : 0);
    });
}

}  // namespace dwps

using namespace dwps;

extern "C" uint64_t ps_selective_scan_checkpoint_rows(uint64_t tokens, uint32_t states) {
    (void)states;  // the same spacing for every number of states
    return ceil_div(tokens, kScanCell);
}

extern "C" ps_status ps_selective_scan(void *ws, size_t *ws_bytes, const ps_scan_input *in, void *out, float *final,
                                       float *checkpoints, void *stream) {
    ps_status st = scan_sizes(in, true);
    if (st != PS_OK) return st;
    const size_t e = dtype_bytes(in->dtype);
    const uint64_t DN = (uint64_t)in->channels * in->states;
    ScanArgs a = scan_args(in, scan_shift(in));
    const bool split = a.shift < 32u;
    const uint64_t cells = split ? ceil_div(in->tokens, 1ull << a.shift) : 0u;
    PlainWs plan;
    size_t carry_at = 0, steps_at = 0, links_at = 0;
    if (split) {
        carry_at = plan.take((cells + 1u) * DN * 4u);
        steps_at = plan.take((cells + 1u) * in->channels * 4u);
        links_at = plan.take((cells + 1u) * 4u);
    }
    bool query = false;
    st = workspace_protocol(ws, ws_bytes, plan.at, &query);
    if (st != PS_OK || query) return st;
    if ((st = scan_pointers(in)) != PS_OK) return st;
    if (in->tokens && !out) return PS_ERR_NULL;
    if (!aligned(ws, 16) || !aligned(out, e) || !aligned(final, 4) || !aligned(checkpoints, 4)) return PS_ERR_ALIGNMENT;
    const ScanBytes n(in);
    if (outputs_overlap({{out, n.cells}, {final, n.edge}, {checkpoints, n.marks}},
                        {{in->x, n.x}, {in->dt, n.dt}, {in->z, n.z}, {in->B, n.B}, {in->C, n.C}, {in->A, n.A},
                         {in->D, n.channel}, {in->dt_bias, n.channel}, {in->offsets, n.offsets}, {in->initial, n.edge}}))
        return PS_ERR_ALIAS;
    const uint64_t pieces = piece_count(in->tokens, a.num_seqs, in->offsets != nullptr, a.shift);
    if (!pieces) return PS_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return with_type(in->dtype, [&](auto zero) {
        using T = decltype(zero);
        return with_states(in->states, [&](auto sc) {
            constexpr int S = decltype(sc)::value;
            float *carry = split ? ws_at<float>(ws, carry_at) : nullptr;
            float *steps = split ? ws_at<float>(ws, steps_at) : nullptr;
            uint32_t *links = split ? ws_at<uint32_t>(ws, links_at) : nullptr;
            return with_full(in, S, [&](auto full) {
                constexpr bool FULL = decltype(full)::value;
                timing_begin(s);
                if (split) {
                    launch_in_parts(pieces, a.col_blocks, 2 * kScanThreads, [&](uint32_t first, uint32_t grid) {
                        a.first = first;
                        hipLaunchKernelGGL((scan_walk_kernel<T, S, false, FULL>), dim3(grid), dim3(2 * kScanThreads), 0, s, a,
                                           (T *)nullptr, (float *)nullptr, (float *)nullptr, carry, steps, links,
                                           ws_counter(ws), plan.words());
                    });
                    launch_scan_link(a, carry, steps, links, (uint32_t)cells, false, s);
                }
                launch_in_parts(pieces, a.col_blocks, 2 * kScanThreads, [&](uint32_t first, uint32_t grid) {
                    a.first = first;
                    hipLaunchKernelGGL((scan_walk_kernel<T, S, true, FULL>), dim3(grid), dim3(2 * kScanThreads), 0, s, a,
                                       static_cast<T *>(out), final, checkpoints, carry, steps, links, (uint32_t *)nullptr, 0u);
                });
                timing_end(s);
                return launch_status();
            });
        });
    });
}

extern "C" ps_status ps_selective_scan_step(const ps_scan_input *in, const float *state, float *new_state,
                                            const int32_t *slots, uint32_t pool, void *out, void *stream) {
    ps_status st = scan_sizes(in, false);
    if (st != PS_OK) return st;
    if ((st = scan_pointers(in)) != PS_OK) return st;
    const size_t e = dtype_bytes(in->dtype);
    if (in->tokens && (!out || (pool && (!state || !new_state)))) return PS_ERR_NULL;
    if (!aligned(out, e) || !aligned(state, 4) || !aligned(new_state, 4) || !aligned(slots, 4)) return PS_ERR_ALIGNMENT;
    if (!slots && in->tokens > pool) return PS_ERR_SIZE;
    const ScanBytes n(in);
    const size_t state_bytes = pool * n.A;
    if (outputs_overlap({{out, n.cells}, {new_state, state_bytes}},
                        {{in->x, n.x}, {in->dt, n.dt}, {in->z, n.z}, {in->B, n.B}, {in->C, n.C}, {in->A, n.A},
                         {in->D, n.channel}, {in->dt_bias, n.channel}, {slots, in->tokens * 4u},
                         {state != new_state ? state : nullptr, state_bytes}}))
        return PS_ERR_ALIAS;
    if (!in->tokens) return PS_OK;
    uint32_t lanes = 1u;
    while (lanes < 64u && lanes * 4u < in->states) lanes *= 2u;
    const uint64_t blocks = ceil_div((uint64_t)in->channels * lanes, 256);
    // up to 8 rows a workgroup, while 4 workgroups are left for each CU
    const uint64_t share = in->tokens * blocks / 1024u;
    const uint32_t each = share < 1u ? 1u : share > 8u ? 8u : (uint32_t)share;
    hipStream_t s = static_cast<hipStream_t>(stream);
    ScanArgs a = scan_args(in, 32u);
    return with_type(in->dtype, [&](auto zero) {
        using T = decltype(zero);
        timing_begin(s);
        auto launch = [&](auto vec) {
            launch_in_parts(ceil_div(in->tokens, each), blocks, 256u, [&](uint32_t first, uint32_t grid) {
                a.first = first;
                hipLaunchKernelGGL((scan_step_kernel<T, decltype(vec)::value>), dim3(grid), dim3(256), 0, s, a, state,
                                   new_state, slots, pool, static_cast<T *>(out), lanes, (uint32_t)blocks, each);
            });
        };
        if (in->states % 4u == 0u) launch(std::true_type());
        else launch(std::false_type());
        timing_end(s);
        return launch_status();
    });
}
