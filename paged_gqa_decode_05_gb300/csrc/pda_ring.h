// pda_ring.h -- how the shared-prefix kernel (pda_prefix.cuh) splits its work over
// CTAs and takes its slots, for the kernel and for a simulation of its loaders and
// streams on the host.
#pragma once

#include <math.h>

#include "pda_plan.h"

#if defined(__CUDACC__)
#define PDA_UNROLL_1 _Pragma("unroll 1")
#else
#define PDA_UNROLL_1
#endif

namespace pda {

// CTAs that W positions of `units` units are split over: none without a position,
// and no more pieces of a unit than the join takes for the tiles they save, as
// many for every unit where there are CTAs enough (one that walks into a second
// unit loads q rows and writes a state twice).  3 sqrt(W units): 16000 tokens of
// one kv head of 128 in 19.1 us, 29.3 over the whole grid, 5586 of four of 256
// 36.8 and 48.2, 8000 of four of 64 in e4m3 21.1 and 26.4; at 2.5 sqrt 19.6, 36.4
// and 22.6, at 4 sqrt 19.3, 47.6, 26.4.  Units cut alike: 16 units of 16384 tokens
// in e4m3 112.6 us for 115.2.
PDA_HD int64_t prefix_ctas(int64_t W, int64_t units, int64_t grid) {
    const int64_t best = (int64_t)(3.f * sqrtf((float)W * (float)units)), some = best > 1 ? best : 1;
    const int64_t most = W < grid ? W : grid, P = some < most ? some : most;
    return units < P ? P / units * units : P;
}

// The ring of slots.  Two q tiles, or one stream: both streams use every slot, all
// slots in a ring.  One q tile for two streams: a stream's tiles have half of the
// slots for a ring of their own.  So whoever waits for a slot's phase has seen the
// phase before it, without which a parity does not say which phase it is (with one
// ring for alternate tiles a stream that ran ahead took a slot that was still to be
// filled for the other one).  Uses of a ring are numbered in the order in which the
// products take them: K of tiles 0 and 1, then V of tile i and K of tile i + 2 in
// turn, then the last V.  A loader that fills every second use or so of a ring knows
// from the last one it filled that the phase before the one it waits for is over; at a
// segment's start, where rings begin anew and may change, it waits for all products of
// the segment before, and the streams do by their q rows.
template <int SLOTS, bool TWO>
struct PrefixRing {
    uint32_t parity = 0;  // of every slot's uses in the segments before
    static PDA_HD int k_use(int i) { return i + (i > 1 ? i - 1 : 0); }
    static PDA_HD int v_use(int i, int items) { return i + (i + 2 < items ? i + 2 : items); }
    // The slot of a use, and the parity of its phase.
    PDA_HD uint32_t slot(bool shared, int st, int use, uint32_t& phase) const {
        uint32_t at = (uint32_t)use % SLOTS, round = (uint32_t)use / SLOTS;
        if (TWO && !shared) {
            at = (uint32_t)use % (SLOTS / 2) + st * (SLOTS / 2);
            round = (uint32_t)use / (SLOTS / 2);
        }
        phase = ((parity >> at) ^ round) & 1u;
        return at;
    }
    // Past a segment of n tiles.
    PDA_HD void next(bool shared, int n) {
        PDA_UNROLL_1
        for (int at = 0; at < SLOTS; ++at) {
            int uses = 2 * n, size = SLOTS, i = at;
            if (TWO && !shared) {
                size = SLOTS / 2;
                if (at >= 2 * size) break;
                const int st = at >= size;
                i = at - st * size;
                uses = (n - st + 1) / 2 * 2;
            }
            if (uses > i) parity ^= (uint32_t)(((uses - i + size - 1) / size) & 1) << at;
        }
    }
};

}  // namespace pda
