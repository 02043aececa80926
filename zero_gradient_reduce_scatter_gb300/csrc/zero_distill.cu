// zero_distill.cu -- the divergence of a student's logits from a teacher's most likely tokens, with its
// gradient on the logits, for sm_103a.
//
// Bound by reading [rows, vocab] logits and writing their gradient. A token's list S (at most 512 places)
// and the rest of the vocabulary as one more entry are a small distribution of their own; the row itself
// is needed for two things: the rest's sum over the softmax, and the gradient, which outside S is
// q_j times one number. With z = x / temperature, q = softmax(z), an entry's r = log p - log q, and c its
// part of dD / d log q:
//   forward  D = sum p r              c = -p
//   reverse  D = -sum q r             c = -q r                       (up to a constant that cancels)
//   js       D = b sum p (log p - log m) + (1 - b) sum q (log q - log m),  m = b p + (1 - b) q
//                                     c = (1 - b) q (log q - log m)
//   dD / dz_j = c_j - q_j C in S, q_j (c_rest / q_rest - C) outside, C = the sum of all c.
// The rest's sum is formed over the rest alone, never as 1 - sum q: a student that is nearly sure of S
// still has its rest to full precision, and the places of S are left out by a bitmap of the vocabulary
// in shared memory, 16 bytes of the row to a byte of it.

#include <cfloat>

#include <type_traits>

#include "zero_rows.cuh"

namespace zg {
namespace {

constexpr int kListMost = 512;              // longest list
constexpr int64_t kDistillVocab = 1 << 20;  // a bitmap of 128 KB

struct DistillTokens : TokenWeights {
    static constexpr bool kClips = false;
    const int64_t* index;  // [rows][k]
    const float *teacher, *teacher_rest;
    float *kl, *logp;      // [rows]
    float *out_loss, *out_kl;
    float* clipped = nullptr;
    float* out_clip = nullptr;
    int k;
    float mix, student, kl_coef, ce_coef;  // shares of a mixture: neither is 0
    int32_t kind, tail;

    __device__ __forceinline__ void spread(int64_t, int64_t) const {}
};

// What a CTA holds of a token's list in shared memory: a bitmap of the vocabulary, and the entries.
struct List {
    uint32_t* bits;
    float *x, *lp;  // the student's logit, later the gradient; the teacher's log-probability
    int* place;     // kNotThere, or kPastVocab
    int k;

    __device__ __forceinline__ List(uint8_t* smem, int words, int k, int buffer = 0) : k(k) {
        bits = reinterpret_cast<uint32_t*>(smem);
        x = reinterpret_cast<float*>(bits + words) + 3 * k * buffer;
        lp = x + k;
        place = reinterpret_cast<int*>(lp + k);
    }
};
constexpr int kNotThere = -1, kPastVocab = -2;
__host__ __device__ constexpr int bitmap_words(int64_t vocab) { return (int)((vocab + 8 + 31) / 32); }

// Whether place j is in the list. Bits begin `shift` before the vocabulary, so that a vector's are neighbours in a byte.
__device__ __forceinline__ bool listed(const uint32_t* bits, int j, int shift) { return bits[(j + shift) >> 5] >> ((j + shift) & 31) & 1; }

// The bits of the vector that begins at place `at`.
template <class T>
__device__ __forceinline__ uint32_t vector_bits(const uint32_t* bits, int at, int shift) {
    const uint32_t b = reinterpret_cast<const uint8_t*>(bits)[(at + shift) >> 3];
    return sizeof(T) == 2 ? b : b >> ((at + shift) & 4) & 15u;
}

// -inf in the marked places of a vector.
template <class T>
__device__ __forceinline__ void strike(uint4& v, uint32_t marks) {
#pragma unroll
    for (int i = 0; i < kVec<T> / 2; ++i) {
        float2 x = unpack2(widen2<T>(v, i));
        if (marks >> (2 * i) & 1) x.x = -INFINITY;
        if (marks >> (2 * i + 1) & 1) x.y = -INFINITY;
        narrow2<T>(v, i, x);
    }
}

// log p - log q, log p = lp - shift, log q = z - log s, with z in two numbers (over_base).
__device__ __forceinline__ float log_ratio(float lp, float shift, float2 z, float2 log_s) {
    const float d = __fsub_rn(lp, z.x), w = __fsub_rn(d, lp), lost = __fsub_rn(__fsub_rn(lp, __fsub_rn(d, w)), __fadd_rn(z.x, w));
    return fabsf(d) < INFINITY ? __fadd_rn(__fadd_rn(d, log_s.x), ((lost + log_s.y) - z.y) - shift) : d;
}

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// An entry's part of D and of C.
struct Part {
    float d, c;
};
// b: the teacher's share of a mixture, s the student's, 1 - b.
__device__ __forceinline__ Part entry_part(int kind, float b, float s, float p, float q, float r) {
    if (kind == ZERO_DISTILL_FORWARD) return {p > 0.0f || p != p ? p * r : 0.0f, -p};
    if (kind == ZERO_DISTILL_REVERSE) {
        const float d = q > 0.0f || q != q ? -q * r : 0.0f;
        return {d, d};
    }
    // log p - log m and log q - log m from r alone: the logarithm of the mixture in units of the larger side, that of a small sum where
    // 1 - s or 1 - b would have lost it
    const float x = r > 0.0f ? s * expm1f(-r) : b * expm1f(r);
    const float m = x < -0.5f ? logf(r > 0.0f ? fmaf(s, expf(-r), b) : fmaf(b, expf(r), s)) : log1pf(x);
    const float pm = r > 0.0f ? -m : r - m, qm = r > 0.0f ? -(r + m) : -m;
    const float c = q > 0.0f || q != q ? s * q * qm : 0.0f;
    return {(p > 0.0f || p != p ? b * p * pm : 0.0f) + c, c};
}

// A row's gradient outside its list: 2^((x_j - base) c) * factor; beside it the target's own part, and the
// target's entry where it is outside the list.
struct DistillRow {
    float base, factor;
    float target;  // the target's gradient
    bool target_listed;
    bool zero;     // no loss: a row of zeros
};

// e^x, 1 at most, in units of 2^-48, off by 2^-39 of itself and a unit: x = n ln 2 + r with ln 2 in three parts (Cody and Waite),
// u = e^(r / 64) - 1 by its Taylor terms, the first two of them in two numbers, and six times u -> 2u + u^2.
__device__ __forceinline__ uint64_t fixed_exp(float x) {
    if (!(x > -80.0f)) return 0;
    if (x >= 0.0f) return 1ull << 48;
    constexpr float kLn2[3] = {2839.0f / 4096.0f, 3.19461832987e-5f, 1.64659497e-12f};
    const float n = rintf(x * kLog2e), r = __fmaf_rn(-n, kLn2[0], x), d = __fmul_rn(-n, kLn2[1]), z = __fadd_rn(r, d), e = __fsub_rn(z, r);
    const float lost = __fadd_rn(__fsub_rn(r, __fsub_rn(z, e)), __fsub_rn(d, e));
    const float m = z * 0x1p-6f, m_lo = (lost + __fmaf_rn(-n, kLn2[1], -d) - n * kLn2[2]) * 0x1p-6f;
    const float half = 0.5f * m, q = __fmul_rn(half, m), cube = m * m * m * fmaf(m, fmaf(m, 1.0f / 120.0f, 1.0f / 24.0f), 1.0f / 6.0f);
    float u = __fadd_rn(m, q), u_lo = __fsub_rn(q, __fsub_rn(u, m)) + (cube + __fmaf_rn(half, m, -q) + fmaf(m, m_lo, m_lo));
#pragma unroll
    for (int i = 0; i < 6; ++i) {
        const float p = __fmul_rn(u, u), p_lo = fmaf(2.0f * u, u_lo, __fmaf_rn(u, u, -p)), two = 2.0f * u;
        u = __fadd_rn(two, p);
        u_lo = __fsub_rn(p, __fsub_rn(u, two)) + (p_lo + 2.0f * u_lo);
    }
    const float up = __int_as_float(((int)n + 127 + 48) << 23);
    return (uint64_t)(__float2ll_rn(up) + __float2ll_rn(u * up) + __float2ll_rn(u_lo * up));
}

// What the teacher's log-probability of the rest is formed from: the number that is given, or what the list leaves of 1, in units of
// 2^-48. Whole numbers lose nothing and have no order: the reverse form weighs this logarithm by the student's own rest, and from
// a sum of expf it was off by 9% at a rest of 1e-6.
constexpr unsigned long long kWhole = 1ull << 48;
struct TeacherRest {
    unsigned long long left;  // kWhole before its row
    float given;
};
// By the warps that have no part in sum_list first. logp(i): entry i's, -inf where it is not there.
template <int THREADS, class F>
__device__ __forceinline__ void take_rest(const DistillTokens& p, int64_t t, TeacherRest& rest, F logp) {
    const int at = THREADS - 1 - threadIdx.x;
    if ((at & ~31) >= p.k || p.tail != ZERO_TAIL_REST) return;
    if (p.teacher_rest) {
        if (at == 0) rest.given = p.teacher_rest[t];
        return;
    }
    uint64_t mass = 0;
    for (int i = at; i < p.k; i += THREADS) mass += fixed_exp(logp(i));
    const uint32_t low = (uint32_t)mass & 0x3FFFFFFu, high = (uint32_t)(mass >> 26);  // of 8 entries: 32 of either are below 2^32
    mass = ((uint64_t)__reduce_add_sync(~0u, high) << 26) + __reduce_add_sync(~0u, low);
    if ((at & 31) == 0) atomicAdd(&rest.left, 0ull - mass);
}
__device__ __forceinline__ float its_logp(const DistillTokens& p, const TeacherRest& rest) {
    return p.teacher_rest ? rest.given : logf(fmaxf(__ll2float_rn((int64_t)rest.left) * 0x1p-48f, 0x1p-24f));
}

// A warp's share of a list: its largest logit, the sum of 2^((x - it) C), the teacher's mass, and how many entries there
// are, 1024 more where the target is one. Before the barrier that finish_list's threads pass.
template <int THREADS>
__device__ __forceinline__ void sum_list(const List& list, Scale k, int64_t y, float4* shares) {
    float top = -INFINITY, mass = 0.0f, sum = 0.0f;
    int count = 0;
    bool target = false;
    for (int i = threadIdx.x; i < list.k; i += THREADS) {
        if (list.place[i] < 0) continue;
        ++count;
        target = target || list.place[i] == y;
        top = fmaxf(top, list.x[i]);
        mass += expf(list.lp[i]);
    }
    if ((threadIdx.x & ~31) < list.k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        for (int i = threadIdx.x; i < list.k; i += THREADS)
            if (list.place[i] >= 0) sum += pow2(scaled<false>(list.x[i] - base_of(top), k));
        sum = warp_add(sum);
        mass = warp_add(mass);
        count = __reduce_add_sync(~0u, count) + (__any_sync(~0u, target) ? 1024 : 0);
    }
    if ((threadIdx.x & 31) == 0) shares[threadIdx.x >> 5] = make_float4(top, sum, mass, __int_as_float(count));
}

// What log p is formed with where the list is renormalised, log p = lp - base - shift, for lists whose sum fp32 does not hold
// (unnormalised logits, a distribution's far tail): over the largest lp. Each warp for itself, once the list is in shared memory.
__device__ __forceinline__ float2 far_mass(const float* lp, const int* place, int k) {
    const int lane = threadIdx.x & 31;
    float base = -INFINITY, sum = 0.0f;
#pragma unroll 1
    for (int i = lane; i < k; i += 32)
        if (place[i] >= 0) base = fmaxf(base, lp[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) base = fmaxf(base, __shfl_xor_sync(~0u, base, o));
#pragma unroll 1
    for (int i = lane; i < k; i += 32)
        if (place[i] >= 0) sum += expf(lp[i] - base);
    return make_float2(base, logf(warp_add(sum)));
}

// What the row's sums and its list come to. rest: the sums outside the list. Writes the token's results (`first`: this CTA
// does) and the gradients of this thread's entries over list.x. Valid in all threads.
template <int THREADS, class S>
__device__ __forceinline__ DistillRow finish_list(const DistillTokens& a, const List& list, const RowStat& rest, bool bad, int64_t t, int64_t y,
                                                  float x_y, int64_t vocab, Scale k, float2 inv_t, bool first, const float4* shares,
                                                  const TeacherRest& teacher, float2* parts, S sync) {
    constexpr int kWarps = THREADS / 32;
    const float w = a.w[t];
    float top = rest.s != 0.0f ? rest.m : -INFINITY, mass = 0.0f, total = 0.0f;
    int count = 0;
    const int warps = min(kWarps, (list.k + 31) / 32);
    for (int i = 0; i < warps; ++i) {
        const float4 v = shares[i];
        top = fmaxf(top, v.x);
        mass += v.z;
        count += __float_as_int(v.w);
    }
    DistillRow r;
    r.target_listed = count >= 1024;  // more often where it is listed twice, which is bad
    count &= 1023;
    const float base = base_of(top), rest_base = base_of(rest.m), up = pow2(scaled<false>(rest_base - base, k));
    for (int i = 0; i < warps; ++i) total += shares[i].y != 0.0f ? shares[i].y * pow2(scaled<false>(base_of(shares[i].x) - base, k)) : 0.0f;
    if (rest.s != 0.0f) total += rest.s * up;
    if (bad || y >= vocab) total = NAN;
    const bool nothing = total == 0.0f;  // -inf alone
    const float over = nothing ? 0.0f : 1.0f / total;
    const float2 all = log_parts(total, 1.0f - over);
    const bool with_rest = a.tail == ZERO_TAIL_REST && count < vocab;
    float lp_base = 0.0f, shift = 0.0f;  // log p = lp - lp_base - shift
    if (a.tail == ZERO_TAIL_RENORMALISE && count > 0) {
        shift = logf(mass);
        if (!(mass > 0x1p-90f && mass < 0x1p90f)) {
            const float2 far = far_mass(list.lp, list.place, list.k);
            lp_base = far.x;
            shift = far.y;
        }
    }
    auto ratio = [&](float lp, float x) { return nothing ? INFINITY : log_ratio(lp, shift, over_base(x, base, inv_t), all); };
    float d = 0.0f, c = 0.0f;
    if ((threadIdx.x & ~31) < list.k) {
        for (int i = threadIdx.x; i < list.k; i += THREADS) {
            if (list.place[i] < 0) continue;
            const float x = list.x[i], lp = list.lp[i] - lp_base, q = pow2(scaled<false>(x - base, k)) * over;
            const Part part = entry_part(a.kind, a.mix, a.student, expf(lp - shift), q, ratio(lp, x));
            d += part.d;
            c += part.c;
        }
        d = warp_add(d);
        c = warp_add(c);
    }
    if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = make_float2(d, c);
    sync();
    d = c = 0.0f;
    for (int i = 0; i < warps; ++i) {
        d += parts[i].x;
        c += parts[i].y;
    }
    Part outside = {0.0f, 0.0f};
    if (with_rest) {
        const float lp = its_logp(a, teacher);
        const float2 own = log_parts(rest.s);
        const bool none = nothing || rest.s == 0.0f;  // no q
        const float q = none ? 0.0f : rest.s * up * over, p = mass == mass ? expf(lp) : NAN;
        const float r_rest = none ? INFINITY : log_ratio(lp, 0.0f, over_base(rest_base, base, inv_t), make_float2(all.x - own.x, all.y - own.y));
        if (!(lp == -INFINITY && none)) outside = entry_part(a.kind, a.mix, a.student, p, q, r_rest);
        d += outside.d;
        c += outside.c;
    }
    // a coefficient of 0 leaves its term out, also where that is infinite
    const float g = w * a.kl_coef * inv_t.x, h = w * a.ce_coef * inv_t.x;
    const float share = (a.ce_coef != 0.0f ? h : 0.0f) - (a.kl_coef != 0.0f ? g * c : 0.0f);
    r.base = rest_base;
    r.factor = 0.0f;  // outside the list there is nothing above -inf
    if (rest.s != 0.0f) {
        r.factor = share * up * over;
        if (with_rest && a.kl_coef != 0.0f) r.factor += g * outside.c / rest.s;
    }
    if (total != total) r.factor = NAN;
    for (int i = threadIdx.x; i < list.k; i += THREADS) {
        if (list.place[i] < 0) continue;
        const float x = list.x[i], lp = list.lp[i] - lp_base, q = pow2(scaled<false>(x - base, k)) * over;
        float v = share * q;
        if (a.kl_coef != 0.0f) v += g * entry_part(a.kind, a.mix, a.student, expf(lp - shift), q, ratio(lp, x)).c;
        if (list.place[i] == y) v -= h;
        list.x[i] = nothing ? 0.0f : v;
    }
    r.zero = w == 0.0f || nothing;
    r.target = nothing ? 0.0f : fmaf(pow2(scaled<false>(x_y - rest_base, k)), r.factor, -h);
    if (first && threadIdx.x == 0) {
        const float2 z = over_base(x_y, base, inv_t);
        const float logp = y >= vocab ? NAN : nothing || x_y == -INFINITY ? -INFINITY : __fsub_rn(z.x, all.x) + (z.y - all.y);
        float loss = 0.0f;
        if (a.kl_coef != 0.0f) loss += a.kl_coef * d;
        if (a.ce_coef != 0.0f) loss -= a.ce_coef * logp;
        if (total != total) loss = d = NAN;
        a.loss[t] = w != 0.0f ? loss * w : 0.0f;
        a.kl[t] = w != 0.0f ? d : 0.0f;
        a.logp[t] = w != 0.0f ? logp : 0.0f;
    }
    return r;
}

// The rest's sum over a base that is given and stays, the list's largest logit: near the row's mass, so that exponents and
// their roundings are small (over the target's logit, as elsewhere, an unlikely target cost 7e-7 of a divergence). Where the
// rest is not good_rest, the sum is formed once more over its own maximum (Sums, CHECKED).
template <class T>
struct RestSums {
    const float m;
    const uint64_t base, c, lo;
    uint64_t s[2];
    const Scale k;

    __device__ __forceinline__ RestSums(Scale k, float m) : m(m), base(pack2(-m, -m)), c(pack2(k.c, k.c)), lo(pack2(k.lo, k.lo)), k(k) {
        s[0] = s[1] = pack2(0.0f, 0.0f);
    }
    __device__ __forceinline__ void add(const uint4& v) {
#pragma unroll
        for (int i = 0; i < kVec<T> / 2; ++i) {
            const uint64_t t = add2(widen2<T>(v, i), base);
            const float2 z = unpack2(fma2(t, lo, mul2(t, c)));
            s[i & 1] = add2(s[i & 1], pack2(pow2(z.x), pow2(z.y)));
        }
    }
    __device__ __forceinline__ void add_one(float x) { s[0] = add2(s[0], pack2(pow2(scaled<false>(x - m, k)), 0.0f)); }
    __device__ __forceinline__ RowStat stat() const {
        const float2 f = unpack2(add2(s[0], s[1]));
        return {m, f.x + f.y, 0.0f};
    }
};
template <class T, bool CHECKED>
using SumsOf = std::conditional_t<CHECKED, Sums<T, false, true>, RestSums<T>>;

// The list's largest logit (sum_list), after a barrier.
template <int THREADS>
__device__ __forceinline__ float list_top(const float4* shares, int k) {
    float top = -INFINITY;
    for (int i = 0; i < min(THREADS / 32, (k + 31) / 32); ++i) top = fmaxf(top, shares[i].x);
    return top;
}

// Whether sums that were not CHECKED are good: the rest may be any share of the base's term.
__device__ __forceinline__ bool good_rest(const RowStat& a) { return a.s > 0x1p-60f && a.s < 0x1p60f; }

// The list's gradients and the target's over what the vectors left there, by the CTA that wrote their places.
template <class T, int THREADS>
__device__ __forceinline__ void write_entries(const List& list, const DistillRow& r, const Slice<T>& s, T* out, int64_t y, int64_t vocab) {
    auto ours = [&](int64_t j) {
        return (j >= s.first && j < s.first + s.n * kVec<T>) || (s.head && j < s.head) || (s.tail && j >= s.tail_at);
    };
    for (int i = threadIdx.x; i < list.k; i += THREADS)
        if (list.place[i] >= 0 && ours(list.place[i])) out[list.place[i]] = narrow<T>(r.factor == r.factor ? list.x[i] : NAN);
    if (threadIdx.x == 0 && !r.target_listed && y < vocab && ours(y)) out[y] = narrow<T>(r.target);
}

// Entry i of token t's list into shared memory.
template <class T>
__device__ __forceinline__ void take_entry(const DistillTokens& p, const List& list, const T* x, int64_t vocab, int64_t t, int i) {
    const int64_t j = p.index[t * p.k + i];
    const float lp = p.teacher[t * p.k + i];
    const bool there = j >= 0 && lp != -INFINITY, past = j >= vocab;
    if (there && !past) list.x[i] = widen(x[j]);
    list.lp[i] = lp;
    list.place[i] = !there ? kNotThere : past ? kPastVocab : (int)j;
}
// Its bit into the bitmap. False: it names a place twice or past the vocabulary.
__device__ __forceinline__ bool mark_entry(const List& list, int i, int shift) {
    const int j = list.place[i];
    if (j < 0) return j != kPastVocab;
    const uint32_t bit = 1u << ((j + shift) & 31);
    return !(atomicOr(list.bits + ((j + shift) >> 5), bit) & bit);
}

// Any row: read once for the rest's sum and again for the gradient, by `size` CTAs (a cluster). Bound by HBM where rows are wide:
// 2039 x 151936 bf16, lists of 128, 263 us, 78% of the copy peak on the three passes' 1.4 GB (61% on two). With 512 threads and two
// CTAs an SM, so that L2 could hold the rows until the second reading, 296.
template <class T, int THREADS>
__global__ void __launch_bounds__(THREADS) k_distill_rows(const Rows<T> a, const DistillTokens p, int size, T* dx, int64_t dstride) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ RowStat sm[THREADS / 32], mine;
    __shared__ float4 shares[THREADS / 32];
    __shared__ float2 sums_of[THREADS / 32];
    __shared__ int shared_bad;
    __shared__ TeacherRest teacher;
    wait_for_kernel_before();
    let_next_kernel_start();
    const int64_t t = blockIdx.x / size;
    const int rank = (int)(blockIdx.x % size), id = threadIdx.x;
    const int64_t y = a.targets[t];
    const T* x = a.x + t * a.stride;
    T* out = dx + t * dstride;
    if (y < 0 || p.w[t] == 0.0f) {
        zero_row<T, THREADS>(out, a.vocab, rank, size);
        if (rank == 0 && id == 0) p.loss[t] = p.kl[t] = p.logp[t] = 0.0f;
        return;
    }
    const Slice<T> s(x, a.vocab, rank, size);
    auto load = [&](int i) { return s.v[i]; };
    const RowStart<T, THREADS> start(s, x, load);
    const int words = bitmap_words(a.vocab);
    const List list(smem, words, p.k);
    for (int i = id; i < words; i += THREADS) list.bits[i] = 0;
    if (id == 0) {
        shared_bad = 0;
        teacher.left = kWhole;
    }
    __syncthreads();
    const float x_y = y < a.vocab ? widen(x[y]) : NAN;
    const int shift = (kVec<T> - (s.tail_at % kVec<T>)) % kVec<T>;
    for (int i = id; i < p.k; i += THREADS) {
        take_entry(p, list, x, a.vocab, t, i);
        if (!mark_entry(list, i, shift)) shared_bad = 1;
    }
    sum_list<THREADS>(list, a.k, y, shares);
    take_rest<THREADS>(p, t, teacher, [&](int i) { return p.index[t * p.k + i] >= 0 ? p.teacher[t * p.k + i] : -INFINITY; });
    __syncthreads();
    const float listed_top = list_top<THREADS>(shares, p.k);
    auto sums = [&](auto checked) {
        constexpr bool kChecked = decltype(checked)::value;
        SumsOf<T, kChecked> run(a.k, listed_top);
        auto use = [&](int i, uint4 q) {
            const uint32_t marks = vector_bits<T>(list.bits, s.first + i * kVec<T>, shift);
            if (marks) strike<T>(q, marks);
            run.add(q);
        };
        if (kChecked) for_vectors<THREADS>(s.n, load, use);
        else start.vectors(s.n, load, use);
        if (id < s.head && !listed(list.bits, id, shift)) run.add_one(widen(start.head));
        if (id < s.tail && !listed(list.bits, s.tail_at + id, shift)) run.add_one(widen(start.tail));
        return group_join<false, kChecked, THREADS / 32>(run.stat(), a.k, sm, 0);
    };
    RowStat st;
    bool good = false;
    if (fabsf(listed_top) < INFINITY) {
        st = sums(std::false_type());
        good = good_rest(st);
        if (!good) __syncthreads();
    }
    if (!good) st = sums(std::true_type());
    st = cluster_join<false>(st, size, a.k, &mine);
    const DistillRow r = finish_list<THREADS>(p, list, st, shared_bad != 0, t, y, x_y, a.vocab, a.k, inverse(a.inv_t), rank == 0, shares,
                                              teacher, sums_of, [] { __syncthreads(); });
    const GradRow grad = {0.0f, -r.factor, 0.0f, r.base, 0.0f};
    if (same_alignment(x, out)) {
        const GradVector<T, false> vector(grad, a.c);
        uint4* to = reinterpret_cast<uint4*>(out + s.first);
        for_vectors<THREADS>(s.n, load, [&](int i, const uint4& q) { __stcs(to + i, vector(q)); });
    } else {
        for (int j = s.first + id; j < s.first + s.n * kVec<T>; j += THREADS) out[j] = narrow<T>(grad_term<false>(grad, widen(x[j]), a.c, false));
    }
    if (id < s.head) out[id] = narrow<T>(grad_term<false>(grad, widen(start.head), a.c, false));
    if (id < s.tail) out[s.tail_at + id] = narrow<T>(grad_term<false>(grad, widen(start.tail), a.c, false));
    __syncthreads();
    write_entries<T, THREADS>(list, r, s, out, y, a.vocab);
    if (size > 1) cg::this_cluster().sync();  // no CTA leaves while another reads its sums
}

// Forward and backward in one pass over each row, as k_policy_rows takes it: the row's slice comes to shared memory by bulk
// copies, is read for the rest's sum as it arrives, and again for the gradient; a producer warp refills each part with the
// next row's as soon as it has been read. It reads the list too, a row ahead, and looks for places that are named twice; the
// list's places in shared memory then become -inf, so that the sum over the row is the rest's. 8192 x 50257 bf16 in lists of 64,
// a quarter masked: 280 us, 76% of the copy peak on 1.45 GB (the same rows read twice: 304; policy_loss, which has no list to
// look at between its two readings, 232). A bitmap tested for every 16 bytes instead of -inf in place: 286.
template <class T, int WARPS>
__global__ void __launch_bounds__(32 * WARPS + 32, fused_ctas(WARPS))
    k_distill_fused(const Rows<T> a, const DistillTokens p, int size, int per, int slots, T* dx, int64_t dstride) {
    constexpr int kThreads = 32 * WARPS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ RowStat sm[WARPS], mine[2];
    __shared__ float4 shares[WARPS];
    __shared__ float2 sums_of[WARPS];
    __shared__ uint32_t end_listed[16];  // elements that no vector holds: the number of the row whose list has them
    __shared__ int shared_bad[2];
    __shared__ int64_t row_at[2], row_y[2];
    __shared__ float row_x[2];  // the target's logit
    __shared__ TeacherRest teacher[2];  // a row's, and the next one's
    __shared__ uint64_t bars[2 * kSlots + 4];
    __shared__ int gave_up;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kSlots, row_full = empty + 8 * kSlots, row_empty = row_full + 16;
    const int rank = (int)(blockIdx.x % size), lane = threadIdx.x & 31, words = bitmap_words(a.vocab);
    const int64_t first = blockIdx.x / size, clusters = gridDim.x / size;
    uint8_t* const lists = smem + (size_t)16 * slots * per;
    uint32_t* const bits = reinterpret_cast<uint32_t*>(lists);
    if (threadIdx.x == 0) {
        gave_up = 0;
        shared_bad[0] = shared_bad[1] = 0;
        teacher[0].left = teacher[1].left = kWhole;
        for (int i = 0; i < 16; ++i) end_listed[i] = 0;
        for (int i = 0; i < slots; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, WARPS);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(row_full + 8 * i, 1);
            mbar_init(row_empty + 8 * i, WARPS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = threadIdx.x; i < words; i += kThreads + 32) bits[i] = 0;
    __syncthreads();

    // As in k_policy_rows: what the caller gives may be read at once, the weights after the kernel before this one.
    let_next_kernel_start();
    int64_t n = 0;  // rows taken
    if (threadIdx.x >= kThreads) {
        Slot slot;
        bool ok = true;
        // The next row and its target; its list is read a row ahead, behind this row's copies.
        int64_t t = -1, y = -1;
        auto next = [&](int64_t i) {
            t = first + i * clusters;
            if (size == 1 && i > 0) {
                if (i == 1) wait_for_kernel_before();
                if (lane == 0) t = (int64_t)gridDim.x + (int64_t)atomicAdd(p.ticket, 1u);
                t = __shfl_sync(~0u, t, 0);
            }
            if (t >= a.rows) t = -1;
            ok = ok && mbar_wait(row_empty + 8 * (i & 1), ((uint32_t)(i >> 1) & 1) ^ 1, &gave_up);
            ok = __all_sync(~0u, ok);
            if (!ok) t = -1;
            y = t >= 0 ? a.targets[t] : -1;
            if (y < 0) return;
            const List list(lists, words, p.k, i & 1);
            const T* x = a.x + t * a.stride;
#pragma unroll 4
            for (int e = lane; e < p.k; e += 32) take_entry(p, list, x, a.vocab, t, e);
            __syncwarp();
            bool bad = false;
            for (int e = lane; e < p.k; e += 32) bad = !mark_entry(list, e, 0) || bad;
            __syncwarp();
            for (int e = lane; e < p.k; e += 32)
                if (list.place[e] >= 0) list.bits[list.place[e] >> 5] = 0;
            bad = __any_sync(~0u, bad);
            if (lane == 0) shared_bad[i & 1] = bad;
            __syncwarp();
        };
        for (next(0);; ++n) {
            const int64_t y_now = y;
            const T* x = a.x + t * a.stride;
            if (lane == 0) {
                row_at[n & 1] = t;
                row_y[n & 1] = y;
                row_x[n & 1] = y >= 0 && y < a.vocab ? widen(x[y]) : NAN;
                mbar_arrive(row_full + 8 * (n & 1));
            }
            if (t < 0) break;
            if (y >= 0 && lane == 0) {
                const Slice<T> s(x, a.vocab, rank, size);
                for (int i = 0; i < kChunks; ++i) {
                    ok = ok && mbar_wait(empty + 8 * slot.at, slot.phase ^ 1, &gave_up);
                    const int at = min(s.n, i * per), bytes = 16 * (min(s.n, at + per) - at);
                    mbar_expect(full + 8 * slot.at, ok ? bytes : 0);
                    if (ok && bytes) bulk_load(smem_addr(smem) + 16 * slot.at * per, s.v + at, bytes, full + 8 * slot.at);
                    slot.next(slots);
                }
            }
            __syncwarp();
            // the consumers' cluster_join, which does not wait for the list
            if (size > 1 && y_now >= 0) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
            next(n + 1);
            if (size > 1 && y_now >= 0) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        }
    } else {
        uint32_t taken = 0;
        Slot begin;  // of the row at hand
        const uint4* parts = reinterpret_cast<const uint4*>(smem);
        for (;; ++n) {
            // Not left early where another wait gave up (k_policy_rows)
            bool got = mbar_try(row_full + 8 * (n & 1), (uint32_t)(n >> 1) & 1);
            for (int i = 0; i < 4 * kWaitLimit && !got; ++i) got = mbar_try(row_full + 8 * (n & 1), (uint32_t)(n >> 1) & 1);
            const int64_t t = got ? row_at[n & 1] : -1, y = row_y[n & 1];
            const float x_y = row_x[n & 1];
            auto release = [&] {  // this warp has done with the row's numbers and its list
                __syncwarp();
                if (lane == 0) mbar_arrive(row_empty + 8 * (n & 1));
            };
            if (t < 0) break;
            T* out = dx + t * dstride;
            if (n == 0) wait_for_kernel_before();
            if (y < 0) {
                zero_row<T, kThreads>(out, a.vocab, rank, size);
                if (threadIdx.x == 0 && rank == 0) p.loss[t] = p.kl[t] = p.logp[t] = 0.0f;
                release();
                continue;
            }
            const T* x = a.x + t * a.stride;
            const Slice<T> s(x, a.vocab, rank, size);
            const List list(lists, words, p.k, n & 1);
            const float x_head = threadIdx.x < s.head ? widen(x[threadIdx.x]) : 0.0f;
            const float x_tail = threadIdx.x < s.tail ? widen(x[s.tail_at + threadIdx.x]) : 0.0f;
            sum_list<kThreads>(list, a.k, y, shares);
            take_rest<kThreads>(p, t, teacher[taken & 1], [&](int i) { return list.place[i] != kNotThere ? list.lp[i] : -INFINITY; });
            for (int i = threadIdx.x; i < p.k; i += kThreads) {
                const int j = list.place[i];
                if (j >= 0 && j < s.head) end_listed[j] = taken + 1;
                if (j >= s.tail_at && s.tail) end_listed[8 + j - s.tail_at] = taken + 1;
            }
            bool ok = true, struck = false;
            // -inf in the places of the list that part i of the slice has, once it is there
            auto strike_list = [&](int i, const Slot& slot) {
                ok = ok && mbar_wait(full + 8 * slot.at, slot.phase, &gave_up);
                const int at = min(s.n, i * per), from = s.first + at * kVec<T>, m = (min(s.n, at + per) - at) * kVec<T>;
                T* v = reinterpret_cast<T*>(smem) + (size_t)slot.at * per * kVec<T>;
                for (int e = threadIdx.x; e < p.k; e += kThreads) {
                    const int j = list.place[e] - from;
                    if (list.place[e] >= 0 && j >= 0 && j < m) v[j] = narrow<T>(-INFINITY);
                }
                consumers_sync<kThreads>();
            };
            strike_list(0, begin);
            const float listed_top = list_top<kThreads>(shares, p.k);
            auto sums = [&](auto checked) {
                constexpr bool kChecked = decltype(checked)::value;
                SumsOf<T, kChecked> run(a.k, listed_top);
                Slot slot = begin;
                for (int i = 0; i < kChunks; ++i, slot.next(slots)) {
                    if (i > 0 && !struck) strike_list(i, slot);
                    const int at = min(s.n, i * per);
                    const uint4* v = parts + slot.at * per;
                    for_vectors<kThreads>(min(s.n, at + per) - at, [&](int j) { return v[j]; }, [&](int, const uint4& q) { run.add(q); });
                }
                if (threadIdx.x < s.head && end_listed[threadIdx.x] != taken + 1) run.add_one(x_head);
                if (threadIdx.x < s.tail && end_listed[8 + threadIdx.x] != taken + 1) run.add_one(x_tail);
                struck = true;
                return group_join<false, kChecked, WARPS>(run.stat(), a.k, sm, 1);
            };
            RowStat st;
            bool good = false;
            if (fabsf(listed_top) < INFINITY) {
                st = sums(std::false_type());
                good = good_rest(st);
                if (!good) consumers_sync<kThreads>();
            }
            if (!good) st = sums(std::true_type());
            if (!ok || *(volatile int*)&gave_up) st.s = NAN;  // a copy did not come: no result
            st = cluster_join<false>(st, size, a.k, mine + (taken & 1));
            const DistillRow r = finish_list<kThreads>(p, list, st, shared_bad[n & 1] != 0, t, y, x_y, a.vocab, a.k, inverse(a.inv_t), rank == 0, shares,
                                                       teacher[taken & 1], sums_of, [] { consumers_sync<kThreads>(); });
            const GradRow grad = {0.0f, -r.factor, 0.0f, r.base, 0.0f};
            const bool fast = same_alignment(x, out);
            if (r.zero) {
                zero_row<T, kThreads>(out, a.vocab, rank, size);
            } else {
                if (threadIdx.x < s.head) out[threadIdx.x] = narrow<T>(grad_term<false>(grad, x_head, a.c, false));
                if (threadIdx.x < s.tail) out[s.tail_at + threadIdx.x] = narrow<T>(grad_term<false>(grad, x_tail, a.c, false));
            }
            const GradVector<T, false> vector(grad, a.c);
            for (int i = 0; i < kChunks; ++i, begin.next(slots)) {
                const int at = min(s.n, i * per), m = min(s.n, at + per) - at;
                const uint4* v = parts + begin.at * per;
                const int from = s.first + at * kVec<T>;  // the chunk's first element
                if (!r.zero && fast) {
                    uint4* to = reinterpret_cast<uint4*>(out + from);
                    for_vectors<kThreads>(m, [&](int j) { return v[j]; }, [&](int j, const uint4& q) { __stcs(to + j, vector(q)); });
                } else if (!r.zero) {
                    const T* e = reinterpret_cast<const T*>(v);
                    for (int j = threadIdx.x; j < m * kVec<T>; j += kThreads) out[from + j] = narrow<T>(grad_term<false>(grad, widen(e[j]), a.c, false));
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // -inf was written to it
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + 8 * begin.at);  // this warp has done with the part
            }
            consumers_sync<kThreads>();
            if (threadIdx.x == 0) teacher[taken & 1].left = kWhole;  // it is not wanted before the next row's barriers
            if (!r.zero) write_entries<T, kThreads>(list, r, s, out, y, a.vocab);
            release();
            ++taken;
        }
    }
    __syncwarp();
    if (*(volatile int*)&gave_up)  // leave no copy in flight behind: they take microseconds, this a millisecond
        for (int j = 0; j < 1000; ++j) __nanosleep(1000);
    if (size > 1) {
        // after giving up: keep in step with the other CTAs, which get no sums from this one
        for (; first + n * clusters < a.rows; ++n) {
            if (a.targets[first + n * clusters] < 0) continue;
            if (threadIdx.x == 0) mine[0].s = mine[1].s = NAN;
            __syncwarp();
            cg::this_cluster().sync();
        }
        cg::this_cluster().sync();  // no CTA leaves while another reads its sums
    }
}

constexpr int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

// Rows of up to this many bytes are read twice, by small CTAs: 8192 x 4000 bf16 54 us by 64 threads, 77 by 256.
constexpr int64_t kDistillShort = 16384;
constexpr int64_t kDistillSpare = 2048;  // two CTAs of an SM have this much more than k_policy_rows takes

template <class T, int THREADS>
int launch_distill_rows(const Rows<T>& rows, int size, const DistillTokens& a, const zero_distill* p, size_t smem, cudaStream_t s) {
    auto* kernel = k_distill_rows<T, THREADS>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * bitmap_words(kDistillVocab) + 24 * kListMost + 16);
    if (e != cudaSuccess) return record_cuda_error(e);
    return launch_linked(kernel, (unsigned)(rows.rows * size), THREADS, smem, size, s, rows, a, size, (T*)p->dlogits, p->dstride);
}

template <class T, int WARPS>
int launch_distill_fused(const Rows<T>& rows, const FusedPlan& f, const DistillTokens& a, const zero_distill* p, size_t extra, int sms, cudaStream_t s) {
    auto* kernel = k_distill_fused<T, WARPS>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(fused_room(WARPS) + kDistillSpare));
    if (e != cudaSuccess) return record_cuda_error(e);
    const int64_t clusters = std::min<int64_t>(rows.rows, fused_ctas(WARPS) * sms / f.size);
    return launch_linked(kernel, (unsigned)(clusters * f.size), 32 * WARPS + 32, (size_t)16 * f.slots * f.part + extra, f.size, s, rows, a, f.size, f.part,
                         f.slots, (T*)p->dlogits, p->dstride);
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" int64_t zero_distill_workspace(int64_t rows) {
    if (rows < 0 || rows > INT64_MAX / 64) return -1;
    return 3 * 4 * round_up(rows, 4) + 64;
}

extern "C" int zero_distill_loss(const zero_logits* x, const zero_distill* p, void* workspace, int64_t workspace_bytes, void* stream) {
    int rc = check_logits(x);
    if (!rc && (!p || p->k < 1 || p->k > kListMost || p->k > x->vocab || x->vocab > kDistillVocab || p->kind < ZERO_DISTILL_FORWARD ||
                p->kind > ZERO_DISTILL_JS || p->tail < ZERO_TAIL_REST || p->tail > ZERO_TAIL_RENORMALISE ||
                (p->kind != ZERO_DISTILL_FORWARD && p->tail != ZERO_TAIL_REST) || !(p->mix > 0.0 && p->mix < 1.0) ||
                !std::isfinite((float)p->kl_coef) || !std::isfinite((float)p->ce_coef) || p->reduce < ZERO_REDUCE_TOKEN ||
                p->reduce > ZERO_REDUCE_SUM))
        rc = ZERO_ERR_INVALID_ARG;
    if (!rc && (p->offsets ? p->seqs < 0 : p->reduce == ZERO_REDUCE_SEQUENCE)) rc = ZERO_ERR_INVALID_ARG;
    if (!rc) rc = check_dlogits(x, p->dlogits, p->dstride);
    if (rc) return rc;
    if (workspace_bytes < zero_distill_workspace(x->rows)) return ZERO_ERR_SIZE_MISMATCH;
    CallDevice d(p->loss, stream);
    if (x->rows > 0) {
        need_logits(d, x);
        d.need(p->index, 8);
        d.need(p->teacher_logp, 4);
        d.optional(p->teacher_rest, 4);
        d.need(p->token_kl, 4);
        d.need(p->logp, 4);
        d.need(p->dlogits, type_size(x->type));
    }
    d.optional(p->offsets, 8);
    d.need(p->loss, 4);
    d.need(p->kl, 4);
    d.need(workspace, 16);
    if (d.rc) return d.rc;
    cudaStream_t s = (cudaStream_t)stream;
    float* f = (float*)workspace;
    const int64_t n = round_up(x->rows, 4);
    DistillTokens a;
    a.targets = x->targets;
    a.offsets = p->offsets;
    a.w = f;
    a.loss = f + n;
    a.of = (uint32_t*)(f + 2 * n);
    a.ticket = (uint32_t*)(f + 3 * n);
    a.rows = x->rows;
    a.seqs = p->seqs;
    a.reduce = p->reduce;
    a.index = p->index;
    a.teacher = p->teacher_logp;
    a.teacher_rest = p->teacher_rest;
    a.kl = p->token_kl;
    a.logp = p->logp;
    a.out_loss = p->loss;
    a.out_kl = p->kl;
    a.k = (int)p->k;
    a.mix = std::max((float)p->mix, FLT_MIN);
    a.student = (float)(1.0 - p->mix);
    a.kl_coef = (float)p->kl_coef;
    a.ce_coef = (float)p->ce_coef;
    a.kind = p->kind;
    a.tail = p->tail;
    const int sms = d.sm_count(), ctas = token_ctas(x->rows);
    if (x->rows > 0) {
        if ((rc = launch_linked(k_token_setup<DistillTokens>, (unsigned)ctas, kSetupThreads, 0, ctas, s, a))) return rc;
        const size_t extra = (size_t)up16(4 * (int64_t)bitmap_words(x->vocab) + 24 * (int64_t)a.k);
        const FusedPlan f = x->vocab * type_size(x->type) > kDistillShort ? fused_plan(x, sms, (int64_t)extra, kDistillSpare) : FusedPlan();
        rc = by_type(x->type, [&](auto tag) {
            using T = decltype(tag);
            const Rows<T> rows = rows_of<T>(x, nullptr);
            if (f.size)
                return f.warps == kFusedWarps ? launch_distill_fused<T, kFusedWarps>(rows, f, a, p, extra, sms, s)
                                              : launch_distill_fused<T, kFusedWarpsSmall>(rows, f, a, p, extra, sms, s);
            if (x->vocab * type_size(x->type) <= kDistillShort && x->rows >= 8 * (int64_t)sms) return launch_distill_rows<T, 64>(rows, 1, a, p, extra, s);
            return launch_distill_rows<T, kRowThreads>(rows, ctas_per_row(x, sms, extra > 16384 ? 4 : kRowCtas / 2), a, p, extra, s);
        });
        if (rc) return rc;
    }
    return launch_linked(k_token_finish<DistillTokens>, (unsigned)ctas, kSetupThreads, 0, ctas, s, a);
}
