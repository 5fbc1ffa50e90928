// Joining an item's parts in the kernel that made them.  Kernels for many rows do: a part is up to 130 KB, and a second
// kernel would read them all again (prompts in chunks over 9000 keys: 171 us for 189; 7 short prompts: 23 us for 28; 256 rows over
// 65536 keys, one item in 256 parts: 62 us for 106).  Kernels for few rows leave it to a second one, whose workgroups read an
// item's many small parts at once (a token over 4097 keys: 13.4 us for 15.9).
#pragma once

#include "cf_attn_plan.h"

namespace cf {
namespace {

// Two floats of a part, for another workgroup of the same launch, maybe on another XCD: written past this XCD's L2 and
// read past it, so that no cache has to be written back or emptied (a fence does that to the whole L2: calls of 40 us
// took 160).
__device__ __forceinline__ void store_far(float* y, float a, float b) {
    const uint64_t bits = static_cast<uint64_t>(__float_as_uint(b)) << 32 | __float_as_uint(a);
    __hip_atomic_store(reinterpret_cast<uint64_t*>(y), bits, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 load_far(const float* y) {
    const uint64_t bits = __hip_atomic_load(reinterpret_cast<const uint64_t*>(y), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return float2{__uint_as_float(static_cast<uint32_t>(bits)), __uint_as_float(static_cast<uint32_t>(bits >> 32))};
}

// All that the wave has stored so is where every XCD sees it.
__device__ __forceinline__ void wait_far() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Run that a place in the work is in.
__device__ __forceinline__ int run_of(int64_t at, int64_t chunk) {
    if ((at | chunk) >> 31 == 0) return uniform(static_cast<int>(static_cast<uint32_t>(at) / static_cast<uint32_t>(chunk)));
    return uniform(static_cast<int>(at / chunk));
}

// For a workgroup that has units [a, z) of an item's count, where w.at is behind them.  An item's parts are joined in
// pairs, those in pairs, and so on: the first of a pair's two to come leaves what it has, its mark, and the item; the
// second takes that to its own.  So nobody waits, and a part is written and read once.  Whoever is second adds the
// same two numbers.  A mark is the call's own 64-bit number: nothing that lies in the workspace before the call is taken
// for one.  The second takes it away again, so that the same call, replayed, finds none.
// leave(slot) writes the workgroup's results to that part, join(slot) takes the part to them.  True: they are the item's.
template <typename LEAVE, typename JOIN>
__device__ __forceinline__ bool join_parts(const AttnRows& p, const Place& w, int z, int count, LEAVE leave, JOIN join) {
    __shared__ int found[2];
    const int64_t end = w.at + count - z;
    const int first = run_of(end - count, w.chunk), parts = run_of(end - 1, w.chunk) + 1 - first;
    const auto slot = [&](int i) { return 2 * int64_t(first + i) + (i == 0); };
    int mine = w.me - first;  // the first of the parts that the workgroup has
    for (int step = 1; step < parts; step <<= 1) {
        const int other = mine ^ step, right = mine | step;
        if (right >= parts) continue;
        uint64_t* const mark = p.marks + first + right;  // each part but the first is one pair's right one
        if (threadIdx.x == 0) found[0] = __hip_atomic_load(mark, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.call;
        __syncthreads();
        if (!found[0]) {
            leave(slot(mine));
            wait_far();
            __syncthreads();
            if (threadIdx.x == 0) found[1] = __hip_atomic_exchange(mark, p.call, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.call;
            __syncthreads();
            if (!found[1]) return false;
        }
        if (threadIdx.x == 0) __hip_atomic_store(mark, uint64_t(0), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        join(slot(other));
        mine &= ~step;
        __syncthreads();  // found has been read
    }
    return true;
}

// A kernel of shape S, and the join behind it where it does not join by itself.
template <typename S, typename A, typename K>
hipError_t launch_attn(A& p, K kernel, int64_t max_rows, void* workspace, hipStream_t stream) {
    p.groups = plan_of<S>(S::kDim).groups;
    p.joins = static_cast<int32_t*>(workspace);
    p.part = reinterpret_cast<float*>(p.joins + kJoin * p.groups);
    if constexpr (S::kJoins) p.marks = static_cast<uint64_t*>(workspace), p.call = call_number();
    kernel<<<p.groups, S::kGroup, 0, stream>>>(p);
    if (hipError_t e = hipGetLastError()) return e;
    if constexpr (S::kJoins) return hipSuccess;
    return launch_join<S>(p, max_rows, stream);
}

}  // namespace
}  // namespace cf
