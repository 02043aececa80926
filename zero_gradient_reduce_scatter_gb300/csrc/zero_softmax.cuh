// Device pieces shared by the kernels that take log-probabilities over a vocabulary: element
// types, the running maximum and sums of a softmax, and how two of them are joined.
//
// For a row x and C = log2(e) / temperature, a part of the row is held as its maximum m (in x
// itself, exact) and, with d_j = (x_j - m) C <= 0, the sums s = sum 2^d_j and
// q = sum 2^d_j d_j. The difference is taken before the product: rows of any magnitude, of the
// type's lowest value among others, keep their differences, and nothing overflows. Then
//   logp_y = (x_y - m) / temperature - log2 s ln 2,   lse = m / temperature + log2 s ln 2,
//   entropy = (log2 s - q / s) ln 2.
#pragma once

#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace zg {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
__device__ __forceinline__ float widen(float x) { return x; }
template <class T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half narrow<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }

// 2^x, subnormal results flushed to 0 (they are below 2^-126 of a row's largest term).
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// C in two parts, c a little below it and lo > 0 the rest. C rounded to one fp32 number would
// shift every d_j the same way, and the log-probabilities of a sequence with it: 6e-8 each at
// temperature 1, which outgrows their own roundings once a few dozen are added up. With both
// parts positive a difference of -inf stays -inf.
struct Scale {
    float c, lo;
};
inline Scale make_scale(double temperature) {
    const double C = 1.4426950408889634074 / temperature;
    Scale k;
    k.c = (float)C;
    if ((double)k.c > C) k.c = nextafterf(k.c, 0.0f);
    k.lo = fmaxf((float)(C - (double)k.c), 1e-30f);
    return k;
}
__device__ __forceinline__ float scaled(float x, Scale k) { return fmaf(x, k.lo, x * k.c); }

// A maximum as it is subtracted: 0 for a part that has no value above -inf, so that its terms
// are 2^-inf = 0 and not 2^(inf - inf).
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

// Differences below this have 2^d = 0; the sum q takes them as this, so that 0 is not multiplied
// by -inf.
constexpr float kFar = -1000.0f;

struct RowStat {
    float m, s, q;
};

__device__ __forceinline__ RowStat empty_stat() { return {-INFINITY, 0.0f, 0.0f}; }

// The sums of `a` taken to the base `m` (base_of a maximum that is at least a.m).
template <bool ENTROPY>
__device__ __forceinline__ void rebase(RowStat& a, float m, Scale k) {
    const float shift = scaled(a.m - m, k), f = pow2(shift);
    if (ENTROPY) a.q = f * fmaf(a.s, fmaxf(shift, kFar), a.q);
    a.s *= f;
}

template <bool ENTROPY>
__device__ __forceinline__ RowStat join(RowStat a, RowStat b, Scale k) {
    const float m = fmaxf(a.m, b.m), base = base_of(m);
    rebase<ENTROPY>(a, base, k);
    rebase<ENTROPY>(b, base, k);
    return {m, a.s + b.s, ENTROPY ? a.q + b.q : 0.0f};
}

// One term over the base m.
template <bool ENTROPY>
__device__ __forceinline__ void add_term(RowStat& a, float x, Scale k, float m) {
    const float d = scaled(x - m, k), e = pow2(d);
    a.s += e;
    if (ENTROPY) a.q = fmaf(e, fmaxf(d, kFar), a.q);
}

// Joins the parts of all threads of a CTA, in a fixed order; the result is valid everywhere.
template <bool ENTROPY, int THREADS>
__device__ __forceinline__ RowStat cta_join(RowStat a, Scale k, RowStat* sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        RowStat b;
        b.m = __shfl_xor_sync(~0u, a.m, o);
        b.s = __shfl_xor_sync(~0u, a.s, o);
        b.q = ENTROPY ? __shfl_xor_sync(~0u, a.q, o) : 0.0f;
        a = join<ENTROPY>(a, b, k);
    }
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = a;
    __syncthreads();
    a = sm[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w) a = join<ENTROPY>(a, sm[w], k);
    __syncthreads();
    return a;
}

struct RowResult {
    float logp, lse, entropy;
};

// pow2 errs low by this share on average (measured over 2^24 arguments), and so does a sum of many
// terms, all but its largest, which is 2^0 = 1 exactly. A log-probability's own rounding hides it,
// a sequence's sum of them would not.
constexpr double kPow2Low = 4.9e-8;

// A row's results from its sums, rounded once; x_y is the target's logit.
__device__ __forceinline__ RowResult finish_row(const RowStat& a, float x_y, double inv_t) {
    RowResult r;
    if (a.s == 0.0f) {  // nothing but -inf
        r.logp = r.lse = -INFINITY;
        r.entropy = 0.0f;
        return r;
    }
    const double s = (double)a.s, l = log(s) + kPow2Low * (1.0 - 1.0 / s);
    r.logp = (float)(((double)x_y - (double)a.m) * inv_t - l);
    r.lse = (float)((double)a.m * inv_t + l);
    r.entropy = (float)(l - (double)a.q / s * 0.69314718055994530942);
    return r;
}

}  // namespace zg
