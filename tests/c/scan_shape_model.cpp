// The selective scan's layout rules (csrc/scan_shape.hpp) on the CPU: for
// every number of states and of channels in a group, the places of a channel's
// lanes hold each state exactly once, and a kernel that leaves out its bounds
// (scan_whole) has no place past the last state or the last channel.
#include <stdint.h>
#include <stdio.h>

#include <vector>

#include "scan_shape.hpp"

using namespace dwps;

static long violations = 0;
static void check(bool ok, const char *what, uint32_t states, uint32_t channels) {
    if (!ok) {
        if (violations < 10) printf("violation: %s (%u states, %u channels)\n", what, states, channels);
        ++violations;
    }
}

static void places(uint32_t states, uint32_t channels, uint32_t per_lane) {
    const bool whole = scan_whole(channels, states, per_lane);
    std::vector<int> held(states, 0);
    for (uint32_t s = 0; s < per_lane; ++s)
        for (uint32_t l = 0; l < (uint32_t)kScanLanes; ++l) {
            const uint32_t n = s * kScanLanes + l;
            if (n < states) ++held[n];
            else check(!whole, "a place without a state in a kernel without bounds", states, channels);
        }
    for (uint32_t n = 0; n < states; ++n) check(held[n] == 1, "each state in one place", states, channels);
    const uint32_t blocks = (channels + kScanChannels - 1u) / kScanChannels;
    if (whole) check(blocks * kScanChannels == channels, "a row of lanes without a channel in a kernel without bounds", states, channels);
}

int main() {
    long cases = 0, whole = 0;
    for (uint32_t states = 1; states <= 256; ++states)
        for (uint32_t channels = 1; channels <= 80; ++channels) {
            const uint32_t s = scan_states_per_lane(states);
            check(s == 1 || s == 2 || s == 4 || s == 8 || s == 16, "states of a lane", states, channels);
            places(states, channels, s);                     // all of a channel's states at once
            places(states, channels, (states + 15u) / 16u);  // 16 at a time
            whole += scan_whole(channels, states, s);
            ++cases;
        }
    check(whole == 5 * 5, "kernels without bounds for 16, 32, 64, 128 and 256 states", 0, 0);
    printf("%ld cases, %ld violations\n", cases, violations);
    return violations ? 1 : 0;
}
