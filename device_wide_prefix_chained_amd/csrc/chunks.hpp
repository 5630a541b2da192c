// chunks.hpp -- how packed sequences are cut into chunks of 2^shift rows that
// begin at each sequence's first row.  Pure integer rules, compiled for the
// device and, in tests/c/chunks_model.cpp, for the host.
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

// A sequence's rows [lo, hi) and the number of its first chunk.  Chunk c of
// sequence s has the number (lo >> shift) + s + c: floor(x) + floor(y) + 1 is
// at least ceil(x + y) less one for whole lo + length, so the numbers of a
// sequence end before the next one's begin, and all lie below chunk_slots
// (also where offsets break their contract: (lo >> shift) + ((hi - 1 - lo) >>
// shift) <= (tokens - 1) >> shift).
struct Rows {
    uint32_t lo, hi;
    uint32_t base;
};

DWPS_HD inline uint32_t rows_before(const uint32_t *offsets, uint32_t s, uint32_t tokens) {
    const uint32_t o = offsets[s];
    return o < tokens ? o : tokens;
}

DWPS_HD inline Rows sequence_rows(const uint32_t *offsets, uint32_t tokens, uint32_t s, uint32_t shift) {
    Rows r;
    r.lo = offsets ? rows_before(offsets, s, tokens) : 0u;
    r.hi = offsets ? rows_before(offsets, s + 1u, tokens) : tokens;
    if (r.hi < r.lo) r.hi = r.lo;
    r.base = (r.lo >> shift) + s;
    return r;
}

// The chunk with number p: rows [lo, hi), which are none where no chunk has
// the number; `index` counts the sequence's chunks.  Each sequence's first
// number is found with index 0, also that of an empty one; a number before the
// first sequence's has the index kNoChunk.
constexpr uint32_t kNoChunk = 0xFFFFFFFFu;
struct Chunk {
    uint32_t seq, index;
    uint32_t lo, hi;
};

DWPS_HD inline Chunk find_chunk(const uint32_t *offsets, uint32_t num_seqs, uint32_t tokens, uint32_t shift,
                                uint32_t p) {
    uint32_t s = 0u;
    if (offsets) {
        uint32_t hi = num_seqs;  // the last s whose first chunk's number is at most p lies in [s, hi)
        while (hi - s > 1u) {
            const uint32_t mid = s + (hi - s) / 2u;
            if ((rows_before(offsets, mid, tokens) >> shift) + mid <= p) s = mid;
            else hi = mid;
        }
    }
    const Rows r = sequence_rows(offsets, tokens, s, shift);
    Chunk c;
    c.seq = s;
    c.index = p < r.base ? kNoChunk : p - r.base;
    const uint64_t at = r.lo + ((uint64_t)c.index << shift);
    c.lo = at < r.hi ? (uint32_t)at : r.hi;
    c.hi = r.hi - c.lo > (1u << shift) ? c.lo + (1u << shift) : r.hi;
    return c;
}

// Numbers of chunks (an upper bound: some numbers have none).
inline uint64_t chunk_slots(uint64_t tokens, uint32_t num_seqs, uint32_t shift) {
    return num_seqs ? (tokens >> shift) + num_seqs : 0u;
}

}  // namespace dwps
