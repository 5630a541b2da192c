// launch_in_parts (csrc/launch_parts.hpp) on the CPU: every workgroup of every
// item is launched once and in order, and no launch holds more work items or
// workgroups than a dispatch can count, at sizes that the entry points take.
#include <stdint.h>
#include <stdio.h>

#include <random>

#include "launch_parts.hpp"

using namespace dwps;

static long violations = 0, cases = 0, split = 0;
static void check(bool ok, const char *what, uint64_t count, uint64_t each, uint32_t threads) {
    if (!ok) {
        if (violations < 10) printf("violation: %s (%llu items of %llu workgroups of %u threads)\n", what,
                                    (unsigned long long)count, (unsigned long long)each, threads);
        ++violations;
    }
}

static void one(uint64_t count, uint64_t each, uint32_t threads) {
    uint64_t next = 0, launches = 0;
    launch_in_parts(count, each, threads, [&](uint32_t first, uint32_t grid) {
        check(first == next, "the first item follows the last launch's", count, each, threads);
        check(grid > 0 && grid % each == 0, "whole items", count, each, threads);
        check((uint64_t)grid * threads < (1ull << 32), "work items of a launch", count, each, threads);
        check(grid < (1u << 31), "workgroups of a launch", count, each, threads);
        next += grid / each;
        ++launches;
    });
    check(next == count, "every item", count, each, threads);
    const bool fits = (__uint128_t)count * each * threads < ((__uint128_t)1 << 32) && count * each < (1ull << 31);
    check(!fits || launches == (count ? 1u : 0u), "one launch where it holds all", count, each, threads);
    split += launches > 1;
    ++cases;
}

int main() {
    one(0, 1, 64);
    one(1, (1u << 23) - 1u, 512);             // the widest scan
    one(40000, 256, 512);                     // sequences of 4096 channels
    one(65536, 128, 512);                     // 2^32 work items exactly
    one((1u << 23) + 77u, 1, 512);
    one((1u << 26) + 5u, 1, 64);              // rows of a norm
    one((1u << 31) - 1u, 1, 64);
    one((1u << 24) - 1u, 1u << 18, 64);       // one-token sequences of 2^24 channels
    one((1u << 24) + (1u << 26), 1u << 20, 512);
    std::mt19937_64 rng(4);
    for (int i = 0; i < 3000; ++i) {
        const uint32_t threads = 64u << rng() % 5;
        const uint64_t widest = kLaunchMostItems / threads;
        const uint64_t each = 1u + rng() % (1ull << rng() % 23);
        const uint64_t count = rng() % (1ull << rng() % 32);
        if (each <= widest && count / (widest / each) < 100000u) one(count, each, threads);
    }
    check(split > 100, "cases of several launches", 0, 0, 0);
    printf("%ld cases, %ld violations\n", cases, violations);
    return violations ? 1 : 0;
}
