// Division of a number below 2^31 by a divisor known at launch.
#pragma once
#include <cstdint>

namespace atc_gb300 {

// With 2^s >= d > 2^(s - 1) and mul = floor(2^(31 + s) / d) + 1, mul * d exceeds 2^(31 + s) by at most d <= 2^s,
// so for n < 2^31 the product n * mul / 2^(31 + s) exceeds n / d by less than 1 / d: its floor is n / d.
struct FastDiv {
    uint32_t d = 1, mul = 0x80000001u;
    int shift = 31;

    FastDiv() = default;
    explicit FastDiv(uint32_t divisor) : d(divisor)
    {
        int s = 0;
        while ((1ULL << s) < d) ++s;
        shift = 31 + s;
        mul = static_cast<uint32_t>((1ULL << shift) / d + 1);
    }
    __device__ __forceinline__ int div(int n) const { return static_cast<int>((static_cast<unsigned long long>(static_cast<uint32_t>(n)) * mul) >> shift); }
    // rounded up; n + d may pass 2^31
    __device__ __forceinline__ int up(int n) const
    {
        const int q = div(n);
        return q + (n - q * static_cast<int>(d) != 0 ? 1 : 0);
    }
};

}  // namespace atc_gb300
