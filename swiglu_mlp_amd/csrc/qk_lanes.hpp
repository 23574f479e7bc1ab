// qk_lanes.hpp -- which channels of a head each lane of a team holds in
// qk_norm_rope_kernel, and which it turns them with.  Plain C++, so that every
// index of every lane is checked on the host (tests/test_host_headers.py).
#pragma once
#include <cstdint>

namespace ck {
namespace qkn {

struct Lane {
    bool live;         // has channels at all
    bool turns;        // and they are among the first rot
    bool upper;        // half pairing: the second channels of their pairs
    uint32_t c;        // its first of 8 channels; 0 in a lane without any
    uint32_t other;    // the lane with the pairs' other channels: itself but for the half pairing
    uint32_t other_c;  // and its first channel
    uint32_t table;    // its first of 8 (half) or 4 (interleaved) entries of a row of the tables
};

// Lane `lane` of a team of at least d / 8 lanes; d a multiple of 8, rot <= d a
// multiple of 16 (half) or 8 (interleaved).
constexpr Lane lane_of(uint32_t lane, uint32_t d, uint32_t rot, bool half)
{
    Lane l{};
    l.live = lane * 8 < d;
    l.c = lane * 8 < d ? lane * 8 : 0;
    // without the first condition a lane past d would turn channel 0, and read its
    // partner's weights rot / 2 channels past its own place, behind the weights' end
    l.turns = l.live && l.c < rot;
    l.upper = l.c >= rot / 2;
    l.other = !half || !l.turns ? lane : l.upper ? lane - rot / 16 : lane + rot / 16;
    l.other_c = half && l.turns ? l.other * 8 : l.c;
    l.table = !half ? l.c / 2 : l.upper ? l.c - rot / 2 : l.c;
    return l;
}

}  // namespace qkn
}  // namespace ck
