// warp.cuh -- what a whole warp does together: electing a lane, waiting on mbarriers
// with a bound, and arriving at them.
#pragma once
#include "tc.cuh"

namespace rc {
namespace tc {

// One lane of a warp that is here as a whole; what it issues takes its operands from
// uniform registers when the code around it is the same for all lanes.
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// A value that is the same in every lane, in a form the compiler knows to be so.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Every lane waits; the same answer in all.  (A wait by one lane, handed on by a
// shuffle, costs the warp over 100 clocks more: the softmax warps waiting that way
// made a 16384-token prompt 11 % slower.)  With a second barrier of the same parity
// both are asked for before either answer is looked at.  CLUSTER: acquire at cluster
// scope, of both (what they announce lies in another CTA, or was sent from there).
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, const Abort &ab, int where, uint32_t also = 0)
{
    uint64_t t0 = 0;
    auto one = [&](uint32_t b) { return CLUSTER ? mbar_try_wait_cluster(b, parity) : mbar_try_wait(b, parity); };
    auto passed = [&] {
        const bool first = one(bar);
        return also ? first & one(also) : first;
    };
    for (uint32_t it = 0; !__all_sync(0xFFFFFFFFu, passed()); ++it) {
        if ((it & 63u) != 63u) continue;
        bool over = *(volatile int *)ab.flag != 0;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (!over && now - t0 > ab.timeout_ns) {
            record_timeout(ab, where);
            over = true;
        }
        if (__any_sync(0xFFFFFFFFu, over)) return false;
    }
    return true;
}

// One arrival by a warp whose lanes are all here (no branch around it).
__device__ __forceinline__ void arrive_warp(uint32_t bar, int lane)
{
    __syncwarp();
    asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar), "r"(lane) : "memory");
}

// The same for a warp in no hurry: asleep between polls, which would take issue
// slots from the warps that share its scheduler.
__device__ __forceinline__ bool wait_idle(uint32_t bar, uint32_t parity, const Abort &ab, int where)
{
    uint64_t t0 = 0;
    while (!__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) {
        __nanosleep(64);
        bool over = *(volatile int *)ab.flag != 0;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (!over && now - t0 > ab.timeout_ns) {
            record_timeout(ab, where);
            over = true;
        }
        if (__any_sync(0xFFFFFFFFu, over)) return false;
    }
    return true;
}

} // namespace tc
} // namespace rc
