// pieces.hpp -- how packed sequences are cut into pieces for the state space
// block's kernels.  Pure integer rules, compiled for the device and, in
// tests/c/pieces_model.cpp, for the host.
#pragma once

#include <stdint.h>

#ifndef DWPS_HD
#ifdef __HIPCC__
#define DWPS_HD __host__ __device__
#else
#define DWPS_HD
#endif
#endif

namespace dwps {

// A piece of one sequence: rows [lo, hi), which lie in one cell of 2^shift
// packed rows, of the sequence's rows [seq_lo, seq_hi).  Piece p is the part
// of sequence s in cell c with c + s = p: along the packed rows either the
// cell or the sequence goes up by at least one from piece to piece, so every
// part has a number of its own below cells + num_seqs, a sequence's first
// cell is told by its first row alone, and an empty sequence has a piece too
// (lo == hi == seq_lo).  shift == 32: a cell holds everything, piece p is
// sequence p.
struct Piece {
    uint32_t seq, cell;
    uint32_t lo, hi, seq_lo, seq_hi;
    bool any;  // some sequence has this piece
};

DWPS_HD inline uint32_t cell_of(uint32_t row, uint32_t shift) { return shift >= 32u ? 0u : row >> shift; }

DWPS_HD inline Piece find_piece(const uint32_t *offsets, uint32_t num_seqs, uint32_t tokens,
                                            uint32_t shift, uint32_t p) {
    Piece q;
    q.any = true;
    if (!offsets) {
        q.seq = 0u;
        q.seq_lo = 0u;
        q.seq_hi = tokens;
        q.cell = p;
    } else {
        uint32_t s = p;
        if (shift < 32u) {
            uint32_t lo = 0u, hi = num_seqs;  // the last s with cell(offsets[s]) + s <= p lies in [lo, hi)
            while (hi - lo > 1u) {
                const uint32_t mid = lo + (hi - lo) / 2u;
                const uint32_t o = offsets[mid] < tokens ? offsets[mid] : tokens;
                if ((o >> shift) + mid <= p) lo = mid;
                else hi = mid;
            }
            s = lo;
        }
        const uint32_t a = offsets[s], b = offsets[s + 1u];
        q.seq = s;
        q.seq_lo = a < tokens ? a : tokens;
        q.seq_hi = b < tokens ? b : tokens;
        if (q.seq_hi < q.seq_lo) q.seq_hi = q.seq_lo;
        q.cell = p - s;
        if (p < s || q.cell < cell_of(q.seq_lo, shift)) q.any = false;
    }
    const uint64_t c0 = shift >= 32u ? 0ull : (uint64_t)q.cell << shift;
    const uint64_t c1 = shift >= 32u ? (uint64_t)tokens : (uint64_t)(q.cell + 1u) << shift;
    q.lo = q.seq_lo > c0 ? q.seq_lo : (uint32_t)(c0 < tokens ? c0 : tokens);
    q.hi = q.seq_hi < c1 ? q.seq_hi : (uint32_t)c1;
    if (q.hi < q.lo) q.hi = q.lo;
    // past the sequence's last row there is a piece only if it is the first
    if (q.lo >= q.seq_hi && !(q.seq_lo == q.seq_hi && q.cell == cell_of(q.seq_lo, shift))) q.any = false;
    return q;
}

// Pieces of the rows at a cell size (an upper bound: some numbers have none).
inline uint64_t piece_count(uint64_t tokens, uint32_t num_seqs, bool has_offsets, uint32_t shift) {
    if (has_offsets && num_seqs == 0u) return 0u;
    if (!has_offsets) return shift >= 32u ? 1u : (tokens >> shift) + 1u;
    return shift >= 32u ? num_seqs : (tokens >> shift) + 1u + num_seqs;
}

}  // namespace dwps
