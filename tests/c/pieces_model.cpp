// Pieces of packed sequences (csrc/pieces.hpp) on the CPU: with offsets that
// keep the contract, the pieces of every numbering hold each row of each
// sequence exactly once, stay inside one cell, start a sequence at its first
// row, and give each empty sequence one empty piece; with offsets that break
// it, every piece stays inside the rows.
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <random>
#include <vector>

#include "pieces.hpp"

using namespace dwps;

static long violations = 0;
static void check(bool ok, const char *what) {
    if (!ok) {
        if (violations < 10) printf("violation: %s\n", what);
        ++violations;
    }
}

int main() {
    std::mt19937 rng(12345);
    long cases = 0;
    for (int round = 0; round < 6000; ++round) {
        const uint32_t tokens = rng() % 5 == 0 ? rng() % 4 : rng() % 400;
        const uint32_t seqs = rng() % 12;
        const bool broken = round % 3 == 2, whole = rng() % 4 == 0, none = rng() % 8 == 0;
        const uint32_t shift = whole ? 32u : 1u + rng() % 7;
        std::vector<uint32_t> off(seqs + 1);
        for (auto &o : off) o = broken ? (rng() % 3 ? rng() % 500 : rng()) : rng() % (tokens + 1);
        if (!broken) std::sort(off.begin(), off.end());
        const uint32_t n_seqs = none ? 1u : seqs;
        const uint64_t pieces = piece_count(tokens, n_seqs, !none, shift);
        std::vector<int> held(tokens, 0), starts(n_seqs, 0), empties(n_seqs, 0);
        for (uint64_t p = 0; p < pieces; ++p) {
            const Piece q = find_piece(none ? nullptr : off.data(), n_seqs, tokens, shift, (uint32_t)p);
            if (!q.any) continue;
            check(q.seq < n_seqs, "sequence number");
            check(q.lo <= q.hi && q.hi <= tokens && q.seq_hi <= tokens, "rows in bounds");
            check(q.seq_lo <= q.lo && q.hi <= q.seq_hi, "rows of the sequence");
            if (q.lo < q.hi && !whole)
                check((q.lo >> shift) == q.cell && ((q.hi - 1u) >> shift) == q.cell, "one cell");
            if (!(q.seq < n_seqs && q.hi <= tokens)) continue;
            for (uint32_t t = q.lo; t < q.hi; ++t) ++held[t];
            if (q.lo == q.seq_lo) ++starts[q.seq];
            if (q.lo == q.hi) ++empties[q.seq];
        }
        if (!broken) {
            for (uint32_t t = 0; t < tokens; ++t) {
                const bool in = none || (seqs && t >= off[0] && t < off[seqs]);
                check(held[t] == (in ? 1 : 0), "each row once");
            }
            for (uint32_t s = 0; s < n_seqs; ++s) {
                const bool empty = none ? tokens == 0 : off[s] == off[s + 1];
                check(starts[s] == 1, "one first piece for each sequence");
                check(empties[s] == (empty ? 1 : 0), "empty pieces");
            }
        }
        ++cases;
    }
    printf("%ld cases, %ld violations\n", cases, violations);
    return violations ? 1 : 0;
}
