// How the scored routing of many tokens is dealt to CTAs: contiguous chunks of tokens, one CTA each, in one
// round (so never more than the device has SMs: a CTA takes one whole).
#pragma once

#include <cstdint>

namespace mx {

constexpr int kRouteMaxChunks = 148;   // what the joining of the chunks' counts is laid out for
constexpr int kRouteMinChunk = 8;      // tokens that share a CTA's set-up, a warp each (4 and 16 differ by 0.5 us, 32 takes 1 to 2 more)

constexpr int64_t route_max_chunks(int sm_count) { return sm_count < kRouteMaxChunks ? sm_count : kRouteMaxChunks; }

// Tokens of a chunk: kRouteMinChunk while the SMs last, then what fills one CTA per SM.
constexpr int64_t route_chunk(int64_t T, int sm_count) {
    const int64_t most = route_max_chunks(sm_count), n = (T + most - 1) / most;
    return n < kRouteMinChunk ? kRouteMinChunk : n;
}

constexpr int64_t route_chunks(int64_t T, int sm_count) {
    const int64_t c = route_chunk(T, sm_count);
    return (T + c - 1) / c;
}

}  // namespace mx
