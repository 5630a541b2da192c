// Chunks of packed sequences (csrc/chunks.hpp) on the CPU: with offsets that
// keep the contract, every chunk number belongs to at most one chunk, the
// chunks found by number are those that a walk over the sequences meets, and
// they hold each row of each sequence exactly once; with offsets that break
// it, every chunk stays inside the rows and every number below the slots.
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <random>
#include <vector>

#include "chunks.hpp"

using namespace dwps;

static long violations = 0;
static void check(bool ok, const char *what) {
    if (!ok) {
        if (violations < 10) printf("violation: %s\n", what);
        ++violations;
    }
}

int main() {
    std::mt19937 rng(4321);
    long cases = 0;
    for (int round = 0; round < 8000; ++round) {
        const uint32_t tokens = rng() % 5 == 0 ? rng() % 4 : rng() % 700;
        const uint32_t seqs = rng() % 12, shift = rng() % 6 ? 1u + rng() % 10 : 31u;
        const bool broken = round % 3 == 2, none = rng() % 8 == 0;
        std::vector<uint32_t> off(seqs + 1);
        for (auto &o : off) o = broken ? (rng() % 3 ? rng() % 900 : rng()) : rng() % (tokens + 1);
        if (!broken) std::sort(off.begin(), off.end());
        const uint32_t *o = none ? nullptr : off.data();
        const uint32_t n = none ? 1u : seqs;
        const uint64_t slots = chunk_slots(tokens, n, shift);
        std::vector<int> held(tokens, 0), walked(slots, 0), firsts(n, 0);
        for (uint32_t s = 0; s < n; ++s) {
            const Rows r = sequence_rows(o, tokens, s, shift);
            check(r.lo <= r.hi && r.hi <= tokens, "rows of a sequence");
            for (uint32_t at = r.lo, c = 0; at < r.hi; at += std::min(r.hi - at, 1u << shift), ++c) {
                check(r.base + c < slots, "number below the slots");
                if (r.base + c >= slots) continue;
                ++walked[r.base + c];
                if (broken) continue;
                const Chunk f = find_chunk(o, n, tokens, shift, r.base + c);
                check(f.seq == s && f.index == c && f.lo == at && f.hi == std::min(r.hi, at + (1u << shift)), "the chunk walked to");
            }
        }
        for (uint64_t p = 0; p < slots; ++p) {
            const Chunk c = find_chunk(o, n, tokens, shift, (uint32_t)p);
            check(c.seq < n && c.lo <= c.hi && c.hi <= tokens && c.hi - c.lo <= (1u << shift), "chunk in bounds");
            if (broken || !(c.hi <= tokens)) continue;
            check(c.index != kNoChunk || c.lo == c.hi, "no chunk before the first");
            if (c.index == 0u) ++firsts[c.seq];
            check((c.lo < c.hi) == (walked[p] == 1) && walked[p] <= 1, "one chunk for a number");
            for (uint32_t t = c.lo; t < c.hi; ++t) ++held[t];
        }
        if (!broken)
            for (uint32_t s = 0; s < n; ++s) check(firsts[s] == 1, "one first number for each sequence");
        if (!broken)
            for (uint32_t t = 0; t < tokens; ++t)
                check(held[t] == ((none || (seqs && t >= off[0] && t < off[seqs])) ? 1 : 0), "each row once");
        ++cases;
    }
    printf("%ld cases, %ld violations\n", cases, violations);
    return violations ? 1 : 0;
}
