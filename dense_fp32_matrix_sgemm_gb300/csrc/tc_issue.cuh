// What the tensor kernels' issuing threads (TMA producer, MMA issuer) share:
// election of the thread, waits, ring positions.
#pragma once

#include <cstdint>

#include "tc_utils.cuh"

namespace sgemm {
namespace tc {

// True in one lane of a converged warp.  The producer's and the MMA issuer's
// loops run in such a lane: elect.sync tells the compiler that a single thread
// is active, so descriptors and coordinates stay in uniform registers.  In the
// same loops under "lane == 0" an M256 N256 K16 MMA took about 226 clocks to
// issue, against the 128 that it runs (a 4096 x 8192 x 4096 bf16 product: 224
// us, 160 elected).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Bounded wait that polls before it reads the clock or the abort word: a
// stage is handed over every 512 clocks, and those two reads in front of each
// poll alone held the pair kernel at 157 us where this takes 140.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity, abort);
}

// Position in a ring of N stages: the stage, the parity of its current round,
// and how many stages have been used so far (up to N).
template <int N>
struct Ring {
    int s = 0, parity = 0, used = 0;
    __device__ __forceinline__ void next() {
        if (used < N) ++used;
        if (++s == N) {
            s = 0;
            parity ^= 1;
        }
    }
};

// Waits (bounded) until the latest fill of every used stage has landed: a CTA
// that gave up does not leave with copies in flight.
template <int N>
__device__ __forceinline__ void drain_ring(const Ring<N> &r, uint32_t full0) {
    for (int s = 0; s < r.used; ++s) {
        const int parity = s < r.s ? r.parity : r.parity ^ 1;
        const long long t0 = clock64();
        while (!mbar_try_wait(full0 + 8 * s, parity) &&
               clock64() - t0 < kWaitLimitCycles) {
        }
    }
}

}  // namespace tc
}  // namespace sgemm
