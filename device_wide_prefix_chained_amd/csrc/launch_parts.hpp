// launch_parts.hpp -- launches of more work than one launch may hold.  Pure
// integer rules, compiled for the library's host side and for the test in
// tests/c/launch_parts_model.cpp.
#pragma once

#include <stdint.h>

namespace dwps {

// A dispatch counts work items in 32 bits and workgroups in 31.
constexpr uint64_t kLaunchMostItems = 0xFFFFFFFFull;
constexpr uint64_t kLaunchMostGroups = 0x7FFFFFFFull;

// Launches `count` items of `groups_each` workgroups with `threads` threads:
// f(first item, workgroups) for as many whole items as a launch holds, in
// order, until all are launched.  An item has to fit a launch.
template <class F>
inline void launch_in_parts(uint64_t count, uint64_t groups_each, uint32_t threads, F f) {
    const uint64_t by_items = kLaunchMostItems / threads;
    const uint64_t most = (by_items < kLaunchMostGroups ? by_items : kLaunchMostGroups) / groups_each;
    for (uint64_t first = 0u; first < count; first += most) {
        const uint64_t here = count - first < most ? count - first : most;
        f((uint32_t)first, (uint32_t)(here * groups_each));
    }
}

}  // namespace dwps
