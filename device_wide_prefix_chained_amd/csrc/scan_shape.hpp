// scan_shape.hpp -- how a channel's states are laid over the 16 lanes of the
// selective scan's kernels, and when a kernel may leave out its bounds.
// Pure integer rules, compiled for the device and, in
// tests/c/scan_shape_model.cpp, for the host.
#pragma once

#include <stdint.h>

namespace dwps {

constexpr int kScanLanes = 16;     // lanes of a channel
constexpr int kScanChannels = 16;  // channels of a workgroup

// States of a lane in the kernels that hold all of a channel's at once: lane l
// has the states l, l + 16, ...; a power of two, so a channel of 48 states
// has 64 places of which 16 hold none.
inline uint32_t scan_states_per_lane(uint32_t states) {
    uint32_t s = 1u;
    while (s * (uint32_t)kScanLanes < states) s *= 2u;
    return s;
}

// Whether every one of `per_lane` places of a lane holds a state and every
// row of lanes a channel.  Only then may a kernel load, add up and store
// without asking whether the state or the channel exists: a place past the
// last state lies in the next channel's, group's or token's row, or past the
// end of the array.
inline bool scan_whole(uint32_t group_channels, uint32_t states, uint32_t per_lane) {
    return group_channels % (uint32_t)kScanChannels == 0u && states == per_lane * (uint32_t)kScanLanes;
}

}  // namespace dwps
