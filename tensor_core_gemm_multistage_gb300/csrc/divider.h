// divider.h - division of non-negative ints by a divisor that the host knows.
#pragma once

#include <cstdint>

namespace gsr {

// n / d for 0 <= n < 2^31: with 2^s >= d and m = ceil(2^(31 + s) / d), n m / 2^(31 + s) exceeds n / d
// by less than n / 2^31 / d, too little to reach the next integer.
struct Divider {
    uint32_t d, s;
    uint64_t m;
    explicit Divider(uint32_t div) : d(div), s(0) {
        while ((1ull << s) < d) ++s;
        m = ((1ull << (31 + s)) + d - 1) / d;
    }
    __host__ __device__ __forceinline__ int operator()(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> (31 + s)); }
};

}  // namespace gsr
