// How the two warps that hold the halves of the same rows swap a value per row, where either may leave early
// (device; the host compiles it for its test).
//
// A swap meets the other warp at a barrier, which by itself waits without limit, and the waits around the swaps
// can run out in one warp and not in the other.  So a warp that leaves puts a mark in the place of its next value and
// arrives without waiting: the other's next swap, if there is one, ends at once and finds the mark.  Each of a warp's swaps has
// its place by parity, so the mark overwrites nothing that is still to be read: that of two swaps before was read
// before the other came to the last one.
#pragma once

#include <stdint.h>
#include <string.h>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

// A NaN that no arithmetic gives (it gives the positive quiet one without a payload).
constexpr uint32_t kLeftMark = 0xFFFACADEu;

// Meet: sync() waits for the other warp's sync() or arrive(), arrive() does not wait; both order the places' reads and writes.
template <class Meet>
struct PairExchange {
    uint32_t* at;        // this lane's places: [parity][half], `lanes` apart
    int lanes, half;
    uint32_t swaps;
    Meet meet;

    // x: this half's value, then the other's.  False if the other warp has left (x is then of no use).
    MOE_HD bool swap(float& x) {
        uint32_t* place = at + 2 * lanes * (swaps++ & 1);
        uint32_t bits;
        memcpy(&bits, &x, 4);
        place[lanes * half] = bits;
        meet.sync();
        bits = place[lanes * (half ^ 1)];
        memcpy(&x, &bits, 4);
        return bits != kLeftMark;
    }
    // Once, by a warp that leaves, whatever the other does or has done.
    MOE_HD void leave() {
        at[2 * lanes * (swaps & 1) + lanes * half] = kLeftMark;
        meet.arrive();
    }
};

}  // namespace moe
