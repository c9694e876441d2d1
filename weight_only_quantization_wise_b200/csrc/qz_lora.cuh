// qz_lora.cuh -- which adapters a call's tokens use, found by each warp from the
// M <= 64 indices on the device.  Internal; not installed.
#pragma once

#include <stdint.h>

namespace qz {
namespace lora {

// Adapter of token m, -1 for none (a negative index, or one out of range).
__device__ __forceinline__ int adapter_of(const int32_t *ids, int adapters, int m) {
    const int id = ids[m];
    return id >= 0 && id < adapters ? id : -1;
}

// Walks the adapters in use, in the order of their first tokens: after next()
// returned true, `id` is one and `tokens` its tokens as a bit mask.  All lanes
// of a warp together; every lane takes part in every exchange.
struct Groups {
    int a, b;                  // adapters of tokens lane and lane + 32
    uint64_t firsts;           // first tokens still to come
    int id = -1;
    uint64_t tokens = 0;

    __device__ __forceinline__ Groups(const int32_t *ids, int M, int adapters, int lane) {
        a = lane < M ? adapter_of(ids, adapters, lane) : -1;
        b = lane + 32 < M ? adapter_of(ids, adapters, lane + 32) : -1;
        const uint32_t same_a = __match_any_sync(0xFFFFFFFFu, a);
        const bool first_a = a >= 0 && __ffs(same_a) - 1 == lane;
        const uint32_t fa = __ballot_sync(0xFFFFFFFFu, first_a);
        uint32_t fb = 0;
        if (M > 32) {
            const uint32_t same_b = __match_any_sync(0xFFFFFFFFu, b);
            bool first_b = b >= 0 && __ffs(same_b) - 1 == lane;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int other = __shfl_sync(0xFFFFFFFFu, a, i);
                if (other == b) first_b = false;
            }
            fb = __ballot_sync(0xFFFFFFFFu, first_b);
        }
        firsts = (uint64_t)fb << 32 | fa;
    }
    // Leaves out the next n adapters.
    __device__ __forceinline__ void skip(int n) {
        for (; n > 0 && firsts; --n) firsts &= firsts - 1;
    }
    __device__ __forceinline__ bool next() {
        if (!firsts) return false;
        const int m = __ffsll((long long)firsts) - 1;
        firsts &= firsts - 1;
        const int ia = __shfl_sync(0xFFFFFFFFu, a, m & 31), ib = __shfl_sync(0xFFFFFFFFu, b, m & 31);
        id = m < 32 ? ia : ib;
        const uint32_t ta = __ballot_sync(0xFFFFFFFFu, a == id), tb = __ballot_sync(0xFFFFFFFFu, b == id);
        tokens = (uint64_t)tb << 32 | ta;
        return true;
    }
};

}  // namespace lora
}  // namespace qz
