// The workspace header, bounded waits on barriers, and rings of slots.
#pragma once
#include "fp8_ptx.cuh"

namespace gct {
namespace fp8 {

constexpr int DEV_TIMEOUT = 1;

// where-codes recorded when a bounded wait gives up
enum : int {
    WAIT_EMPTY = 101,
    WAIT_FULL = 102,
    WAIT_FULL_B = 103,
    WAIT_ACC_EMPTY = 104,
    WAIT_ACC_FULL = 105,
    WAIT_RAW = 106,
    WAIT_A_EMPTY = 107,
    WAIT_PARTS = 108,
    WAIT_TAIL = 109,
    WAIT_FACTOR = 110,
    WAIT_FACTOR_EMPTY = 111,
    WAIT_DRAIN_TMA = 120,  // from here on: teardown
    WAIT_DRAIN_MMA = 121,
};

// The library's workspace header (same layout for every op).
struct WsHeader {
    uint32_t epoch;        // epoch of the last completed launch
    uint32_t ctr[2];       // queue heads of other ops; zero between launches
    uint32_t done_ctr;     // CTAs finished in this launch
    int status;            // sticky first device error (0 = none)
    uint32_t abort_epoch;  // == current epoch while the launch is stopping
    int err_where;
    int err_index;
    uint32_t pad[56];
};
static_assert(sizeof(WsHeader) == 256, "workspace header is 256 bytes");

struct Ctl {
    WsHeader* ws;
    uint32_t epoch;
    unsigned long long limit;
    int rank;  // in the cluster: the half of a pair's tile, or the part of the contraction
};

__device__ __forceinline__ bool launch_aborted(const Ctl& c) {
    return *reinterpret_cast<volatile uint32_t*>(&c.ws->abort_epoch) == c.epoch;
}
__device__ __forceinline__ void raise_timeout(const Ctl& c, int where, int index) {
    if (atomicCAS(&c.ws->status, 0, DEV_TIMEOUT) == 0) {
        c.ws->err_where = where;
        c.ws->err_index = index;
    }
    __threadfence();
    atomicExch(&c.ws->abort_epoch, c.epoch);
}
// Bounded wait for a phase of a barrier; false = gave up, here or elsewhere.
__device__ __forceinline__ bool wait_bar(const Ctl& c, uint32_t bar, uint32_t parity, int where) {
    if (bar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        if (bar_try_wait(bar, parity)) return true;
        if ((i & 15) == 0) {
            // teardown waits are for work already issued: they go on while the launch stops
            if (where < WAIT_DRAIN_TMA && launch_aborted(c)) return false;
            if (global_timer_ns() - t0 > c.limit) {
                raise_timeout(c, where, -1);
                return false;
            }
        }
    }
}
// for barriers that other CTAs' promotion warps arrive on after writing shared
// memory that this one reads
__device__ __forceinline__ bool wait_bar_cluster(const Ctl& c, uint32_t bar, uint32_t parity, int where) {
    if (!wait_bar(c, bar, parity, where)) return false;
    return bar_try_wait_cluster(bar, parity);  // the phase is over: this only acquires at cluster scope
}

// Position in a ring of N slots.
template <int N>
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1;
        }
    }
};
// A producer's record of its fills: bit s of `filled` is the phase of slot s's
// last one.
struct Fills {
    uint32_t used = 0, filled = 0;
    __device__ __forceinline__ void add(uint32_t slot, uint32_t phase) {
        filled = (filled & ~(1u << slot)) | phase << slot;
        used |= 1u << slot;
    }
    // every load has landed before the CTA leaves
    __device__ __forceinline__ void drain(const Ctl& ctl, uint32_t bars, int n) const {
        for (int s = 0; s < n; ++s)
            if ((used & (1u << s)) && !wait_bar(ctl, bars + 8 * s, filled >> s & 1u, WAIT_DRAIN_TMA)) return;
    }
};

}  // namespace fp8
}  // namespace gct
