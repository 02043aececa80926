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

// For kernels launched with launch_linked. A call's last kernel lets the next one start only after
// its own wait, or not at all: what follows the call may be a kernel that does not wait itself
// (ZERO_OVERLAP_BUCKETS), and must not start before all that preceded the call is complete.
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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

// C in two parts, c and the rest lo. C rounded to one fp32 number would shift every d_j the same
// way, and the log-probabilities of a sequence with it: 6e-8 each at temperature 1, which outgrows
// their own roundings once a few dozen are added up. Where q is formed, it gives the shift back at
// the end (log2 s moves by lo / c times q / s); elsewhere every d_j is formed with both parts,
// which are both positive, so that a difference of -inf stays -inf.
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
template <bool ENTROPY>
__device__ __forceinline__ float scaled(float x, Scale k) { return ENTROPY ? x * k.c : fmaf(x, k.lo, x * k.c); }

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
    const float shift = scaled<ENTROPY>(a.m - m, k), f = pow2(shift);
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

// ---- two fp32 numbers in one instruction -------------------------------------------------
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// 16 bytes that this kernel reads once and does not write, past L1.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

// ---- 16 bytes of a row ---------------------------------------------------------------------
template <class T>
constexpr int kVec = 16 / (int)sizeof(T);

// Elements 2i and 2i + 1 as fp32.
template <class T>
__device__ __forceinline__ uint64_t widen2(const uint4& v, int i);
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
template <>
__device__ __forceinline__ uint64_t widen2<__nv_bfloat16>(const uint4& v, int i) {
    const uint32_t w = word(v, i);
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ uint64_t widen2<__half>(const uint4& v, int i) {
    const uint32_t w = word(v, i);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pack2(f.x, f.y);
}
template <>
__device__ __forceinline__ uint64_t widen2<float>(const uint4& v, int i) {
    return pack2(__uint_as_float(word(v, 2 * i)), __uint_as_float(word(v, 2 * i + 1)));
}
// The largest element; a NaN beside numbers is passed over (its term makes the sum NaN).
template <class T>
__device__ __forceinline__ float max_of(const uint4& v);
template <>
__device__ __forceinline__ float max_of<__nv_bfloat16>(const uint4& v) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
}
template <>
__device__ __forceinline__ float max_of<__half>(const uint4& v) {
    const __half2* h = reinterpret_cast<const __half2*>(&v);
    const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
}
template <>
__device__ __forceinline__ float max_of<float>(const uint4& v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
}
// Two fp32 numbers rounded to the row's type, for word i of 16 bytes.
template <class T>
__device__ __forceinline__ void narrow2(uint4& v, int i, float2 f);
__device__ __forceinline__ void set_word(uint4& v, int i, uint32_t w) {
    if (i == 0) v.x = w;
    else if (i == 1) v.y = w;
    else if (i == 2) v.z = w;
    else v.w = w;
}
template <>
__device__ __forceinline__ void narrow2<__nv_bfloat16>(uint4& v, int i, float2 f) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    set_word(v, i, *reinterpret_cast<const uint32_t*>(&h));
}
template <>
__device__ __forceinline__ void narrow2<__half>(uint4& v, int i, float2 f) {
    const __half2 h = __floats2half2_rn(f.x, f.y);
    set_word(v, i, *reinterpret_cast<const uint32_t*>(&h));
}
template <>
__device__ __forceinline__ void narrow2<float>(uint4& v, int i, float2 f) {
    set_word(v, 2 * i, __float_as_uint(f.x));
    set_word(v, 2 * i + 1, __float_as_uint(f.y));
}

// One thread's sums over a row.
// Not CHECKED: over a base that is given and stays, usually the target's logit: no comparing, no
// rescaling, and the parts of a row are plain sums. The sums are floating-point, so a base well
// below the maximum is as good, until 2^60. An entropy is the difference of log s and q / s, which
// are both as large as the distance of the row's mass from its base, and so are the roundings of q:
// off by 4e-7 (root mean square) where the target is the likely token, as in any fp32 form, by 2e-6
// where it is 2^30 times less likely, and by 4e-6, past the bound of a row's other roundings, at
// 2^60; so with ENTROPY until 2^30. And its sum meets 0 times -inf at a logit of -inf. All of these
// show in the result, and the row is then taken again, CHECKED: the base follows the
// maximum (only once a value exceeds it by 2^40: comparing costs less than rescaling) and
// differences are kept finite.
// pow2 errs low below 0 and high above it, by 5e-8 and 3e-8 on average: over a base that is not the
// maximum the errors of a row's terms would depend on where its mass lies. So without CHECKED the
// terms are 2^(d_j - kDown), below 1 for all but rows whose target is 2^kDown times less likely
// than another token, and the sums are taken back up in the end; the base's own term stays exact.
constexpr float kDown = 20.0f;

template <class T, bool ENTROPY, bool CHECKED>
struct Sums {
    float m, limit;  // base, and the largest value that is taken over it
    uint64_t base;   // -m, twice
    uint64_t s[2], q[2];
    const uint64_t c, lo;  // the scale's parts, twice each
    const Scale k;

    __device__ __forceinline__ Sums(Scale k, float from) : c(pack2(k.c, k.c)), lo(pack2(k.lo, k.lo)), k(k) {
        m = CHECKED ? -INFINITY : base_of(from);
        limit = -INFINITY;
        base = CHECKED ? pack2(0.0f, 0.0f) : pack2(-m, -m);
        s[0] = s[1] = q[0] = q[1] = pack2(0.0f, 0.0f);
    }
    __device__ __forceinline__ void raise(float top) {
        const float to = base_of(top), shift = scaled<ENTROPY>(m - to, k), f = pow2(shift);
        const uint64_t f2 = pack2(f, f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (ENTROPY) {
                const float d = fmaxf(shift, kFar);
                q[i] = mul2(f2, fma2(s[i], pack2(d, d), q[i]));
            }
            s[i] = mul2(s[i], f2);
        }
        m = top;
        base = pack2(-to, -to);
        limit = top + 40.0f / k.c;
    }
    __device__ __forceinline__ void term(int i, uint64_t x) {
        // d_j for the sum q, and the exponent that is taken, kDown lower
        const uint64_t t = add2(x, base), down = pack2(-kDown, -kDown), d = mul2(t, c);
        const uint64_t z = CHECKED ? (ENTROPY ? d : fma2(t, lo, d)) : ENTROPY ? add2(d, down) : fma2(t, lo, fma2(t, c, down));
        const float2 zf = unpack2(z);
        const uint64_t e = pack2(pow2(zf.x), pow2(zf.y));
        s[i] = add2(s[i], e);
        if (ENTROPY) q[i] = fma2(e, CHECKED ? pack2(fmaxf(zf.x, kFar), fmaxf(zf.y, kFar)) : d, q[i]);
    }
    __device__ __forceinline__ void add(const uint4& v) {
        if (CHECKED) {
            const float top = max_of<T>(v);
            if (top > limit) raise(top);
        }
#pragma unroll
        for (int i = 0; i < kVec<T> / 2; ++i) term(i & 1, widen2<T>(v, i));
    }
    __device__ __forceinline__ void add_one(float x) {
        if (CHECKED && x > limit) raise(x);
        const float t = x - base_of(m), down = CHECKED ? 0.0f : -kDown, d = t * k.c;
        const float e = pow2(ENTROPY ? d + down : fmaf(t, k.lo, CHECKED ? d : fmaf(t, k.c, down)));
        s[0] = add2(s[0], pack2(e, 0.0f));
        if (ENTROPY) q[0] = fma2(pack2(e, 0.0f), pack2(CHECKED ? fmaxf(d, kFar) : d, 0.0f), q[0]);
    }
    __device__ __forceinline__ RowStat stat() const {
        const float2 a = unpack2(add2(s[0], s[1])), b = unpack2(add2(q[0], q[1]));
        const float up = CHECKED ? 1.0f : 0x1p20f, sum = a.x + a.y;
        static_assert(kDown == 20.0f, "2^kDown");
        return {m, sum * up, ENTROPY ? (b.x + b.y) * up : 0.0f};
    }
};

// Whether sums that were not CHECKED are good.
template <bool ENTROPY>
__device__ __forceinline__ bool good_sums(const RowStat& a) {
    return ENTROPY ? a.s < 0x1p30f && a.q == a.q : a.s < 0x1p60f;
}

// Joins the parts of a warp's lanes (the first N of them) in a fixed order; valid in every lane.
// One rescaling each: the common base first, then plain sums.
// CHECKED as in Sums: else all bases are equal.
template <bool ENTROPY, bool CHECKED, int N = 32>
__device__ __forceinline__ RowStat warp_join(RowStat a, Scale k) {
    if (CHECKED) {
        float m = a.m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < N) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        rebase<ENTROPY>(a, base_of(m), k);
        a.m = m;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (o >= N) continue;
        a.s += __shfl_xor_sync(~0u, a.s, o);
        if (ENTROPY) a.q += __shfl_xor_sync(~0u, a.q, o);
    }
    return a;
}

// Joins the parts of all threads of a group of WARPS warps (at most 16) that meet at the named
// barrier `id`; valid in all of them. sm[0 .. WARPS) may be written again after the group's next
// barrier.
template <bool ENTROPY, bool CHECKED, int WARPS>
__device__ __forceinline__ RowStat group_join(RowStat a, Scale k, RowStat* sm, int id) {
    a = warp_join<ENTROPY, CHECKED>(a, k);
    const int lane = threadIdx.x & 31;
    if (lane == 0) sm[threadIdx.x >> 5] = a;
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 * WARPS) : "memory");
    const RowStat none = {CHECKED ? -INFINITY : a.m, 0.0f, 0.0f};
    a = (lane & 15) < WARPS ? sm[lane & 15] : none;
    return warp_join<ENTROPY, CHECKED, 16>(a, k);
}

struct RowResult {
    float logp, lse, entropy;
    float low;  // what logp was short of before it was rounded
};

// pow2 errs low by this share on average (measured over 2^24 arguments below 0), and so does a sum
// of many terms, all but the base's own, whose argument is an integer. A log-probability's own
// rounding hides it, a sequence's sum of them would not.
constexpr float kPow2Low = 5.0e-8f;

// A row's results from its sums; x_y is the target's logit. ENTROPY says how the sums were formed.
// log s and what is added to it is held in two fp32 numbers until the last sum: with s = 2^n f,
// hi = n times ln 2's first 12 bits, which is exact, and lo, below 1, all the rest (Cody and
// Waite's reduction). fp64 would do the same in a few microseconds, a third of a row's time.
template <bool ENTROPY>
__device__ __forceinline__ RowResult finish_row(const RowStat& a, float x_y, Scale k, float inv_t) {
    RowResult r;
    if (a.s == 0.0f) {  // nothing but -inf
        r.logp = r.lse = -INFINITY;
        r.entropy = r.low = 0.0f;
        return r;
    }
    constexpr float kLn2Hi = 2839.0f / 4096.0f, kLn2Lo = 3.1946184945309e-5f;
    const uint32_t bits = __float_as_uint(a.s);
    const bool plain = a.s >= 0x1p-126f && a.s < INFINITY;  // else (tiny, infinite, NaN) as it is
    const float n = plain ? (float)((int)(bits >> 23) - 127) : 0.0f;
    const float f = plain ? __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u) : a.s;
    const float mean = ENTROPY ? a.q / a.s * kLn2 : 0.0f, low = k.lo / k.c;
    const float hi = n * kLn2Hi, lo = logf(f) + fmaf(n, kLn2Lo, fmaf(low, mean, kPow2Low * (1.0f - 1.0f / a.s)));
    const float base = base_of(a.m);
    const float top = (x_y - base) * inv_t - hi;
    r.logp = __fsub_rn(top, lo);
    const float z = __fsub_rn(r.logp, top);
    r.low = __fsub_rn(__fsub_rn(top, __fsub_rn(r.logp, z)), __fadd_rn(lo, z));
    if (!(fabsf(r.logp) < INFINITY)) r.low = 0.0f;
    r.lse = fmaf(base, inv_t, hi) + lo;
    r.entropy = hi - fmaf(mean, low, mean) + lo;
    return r;
}

// log s as hi + lo (finish_row's reduction), hi exact; `share` of it are terms whose pow2 errs low.
__device__ __forceinline__ float2 log_parts(float s, float share = 1.0f) {
    constexpr float kLn2Hi = 2839.0f / 4096.0f, kLn2Lo = 3.1946184945309e-5f;
    const uint32_t bits = __float_as_uint(s);
    const bool plain = s >= 0x1p-126f && s < INFINITY;
    const float n = plain ? (float)((int)(bits >> 23) - 127) : 0.0f, f = plain ? __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u) : s;
    return make_float2(n * kLn2Hi, logf(f) + fmaf(n, kLn2Lo, kPow2Low * share));
}

// 1 / temperature in two numbers.
__device__ __forceinline__ float2 inverse(double inv_t) { return make_float2((float)inv_t, (float)(inv_t - (double)(float)inv_t)); }

// (x - base) / temperature in two numbers, for what is a small difference of log-probabilities near 10, whose own roundings
// would be 1e-6 of it. Past fp32 (logits at the type's lowest value, a temperature below 1) it is infinite, with nothing beside it.
__device__ __forceinline__ float2 over_base(float x, float base, float2 inv_t) {
    const float d = __fsub_rn(x, base), z = __fsub_rn(d, x), lost = __fsub_rn(__fsub_rn(x, __fsub_rn(d, z)), __fadd_rn(base, z));
    const float hi = __fmul_rn(d, inv_t.x);
    return make_float2(hi, fabsf(hi) < INFINITY ? __fmaf_rn(d, inv_t.x, -hi) + __fmaf_rn(d, inv_t.y, lost * inv_t.x) : 0.0f);
}

}  // namespace zg
