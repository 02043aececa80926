// zero_top.cu -- the k largest logits of every token with their log-probabilities, for sm_103a.
//
// Bound by reading [rows, vocab] logits once, beside the sums of a softmax (zero_softmax.cuh). A row is
// read as a stream without a barrier: every thread leaves the largest value and the sum of each segment
// of a few vectors of its own. The largest values give a threshold that more than k values of the row
// reach, and hardly more; the few segments that reach it are read again (from L2), their values above it
// become candidates, and their sums are formed once more without those. So the probability outside the k
// is a sum of its own, not a difference. The candidates are sorted: by value, the lower place first among
// equal ones. Rows that this does not fit (floods of equal values, nothing but -inf, values too far
// apart for one base) are taken again chunk by chunk, in a way that holds for all (TopRow::chunk).

#include <climits>
#include <type_traits>

#include "zero_rows.cuh"

namespace zg {
namespace {

constexpr int kTopMost = 512;  // largest k

// fp32 values as whole numbers in the same order, and back. 0 and -0 are equal; NaN does not occur.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ ((uint32_t)((int32_t)~key >> 31) | 0x80000000u));
}
constexpr uint32_t kKeyLow = 0x007FFFFFu;  // -inf

// A candidate: its value's key above, and below it the complement of its place, so that a larger one is the
// better and no two are equal.
__device__ __forceinline__ uint64_t candidate(float x, int place) { return (uint64_t)key_of(x) << 32 | (uint32_t)~place; }

// What the THREADS that share a row (a CTA's, or a warp's) hold in shared memory, and behind it the largest value and the
// sum of every thread's segments, [segments][THREADS] each.
constexpr int kSegments = 16, kShortSegments = 32;
template <int THREADS, int CAP>
struct TopSpace {
    // segments that reach the threshold: about as many as values, which are k + k / 4 and some more
    static constexpr int kHot = THREADS == 32 ? 160 : CAP == 512 ? 384 : CAP == 1024 ? 512 : 1024;
    alignas(16) uint64_t cand[CAP];
    int n;                   // candidates; counts on past CAP where they did not fit
    int hots;
    uint32_t hot[kHot];      // segment * THREADS + thread
    uint32_t keys[2 * THREADS];  // of every thread's largest values, of half its vectors each
    int sums[2][THREADS / 32];
    float2 floats[THREADS / 32];
    float bases[THREADS / 32];
    unsigned long long gone[THREADS / 32];
    uint32_t key;            // the threshold's
    // for the cluster's first CTA
    int kept;
    float low, rest;

    __device__ __forceinline__ float* largest() { return reinterpret_cast<float*>(this + 1); }
};

// Candidates to which they are cut back.
__host__ __device__ constexpr int top_few(int k) { return k + k / 8 + 16; }

// What a row has come to: candidates, the threshold, and this thread's sum over it as a base.
struct Taken {
    int n;
    float low, sum;
};

template <class T, int THREADS, int CAP>
struct TopRow {
    using Space = TopSpace<THREADS, CAP>;
    static constexpr int kRanked = THREADS == 32 ? 128 : CAP <= 1024 ? 2 * THREADS : 0;  // so many candidates are ranked by counting
    static constexpr int kRoom = CAP - 16;  // the ends of a row always fit
    Space& sm;
    const Scale scale;
    const int k, id;
    int turn = 0;           // of sm.sums
    int n = 0;              // candidates
    bool have = false;      // whether there is a threshold: at least k candidates are not below it
    float low = -INFINITY;  // the threshold, and the base of the sum
    uint64_t s[2];          // sum of 2^((x - low) C) over what is no candidate
    uint64_t base, c2, lo2;

    __device__ __forceinline__ TopRow(Space& sm, Scale scale, int k) : sm(sm), scale(scale), k(k), id(place_in_group<THREADS>()) {
        s[0] = s[1] = base = pack2(0.0f, 0.0f);
        c2 = pack2(scale.c, scale.c);
        lo2 = pack2(scale.lo, scale.lo);
        sync();
        if (id == 0) sm.n = sm.hots = 0;
        sync();
    }
    // What has been taken of a row.
    __device__ __forceinline__ TopRow(Space& sm, Scale scale, int k, const Taken& t) : sm(sm), scale(scale), k(k), id(place_in_group<THREADS>()) {
        s[0] = pack2(t.sum, 0.0f);
        s[1] = pack2(0.0f, 0.0f);
        base = pack2(-base_of(t.low), -base_of(t.low));
        c2 = pack2(scale.c, scale.c);
        lo2 = pack2(scale.lo, scale.lo);
        n = t.n;
        low = t.low;
        have = n >= k;
    }
    __device__ __forceinline__ Taken taken() const {
        const float2 f = unpack2(add2(s[0], s[1]));
        return {n, low, f.x + f.y};
    }
    static __device__ __forceinline__ void sync() {
        if (THREADS == 32) __syncwarp();
        else __syncthreads();
    }
    // The sum over the group, in all of its threads. Also a barrier.
    __device__ __forceinline__ int total(int x) {
        x = __reduce_add_sync(~0u, x);
        if (THREADS == 32) {
            __syncwarp();
            return x;
        }
        int* a = sm.sums[turn];
        turn ^= 1;
        if ((id & 31) == 0) a[id >> 5] = x;
        __syncthreads();
        x = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) x += a[w];
        return x;
    }
    __device__ __forceinline__ uint32_t largest(uint32_t x) {
        x = __reduce_max_sync(~0u, x);
        if (THREADS == 32) return x;
        int* a = sm.sums[turn];
        turn ^= 1;
        if ((id & 31) == 0) a[id >> 5] = (int)x;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) x = max(x, (uint32_t)a[w]);
        return x;
    }

    // A key that at least k of a set reach, and at most `most` where keys alone can do that: else the
    // k-th largest. count(v): this thread's members that are not below v. At least k reach lo, fewer
    // than k reach hi; n: how many reach the result, INT_MAX if that was not counted.
    template <class F>
    __device__ __forceinline__ uint32_t cut(F count, uint32_t lo, uint32_t hi, int most, int& reach) {
        while (reach > most && hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            const int c = total(count(value_of(mid)));
            if (c >= k) {
                lo = mid;
                reach = c;
            } else {
                hi = mid;
            }
        }
        return lo;
    }
    // The last place of the first `need` members of a set; count(p): this thread's members up to place p.
    template <class F>
    __device__ __forceinline__ int cut_places(F count, int need) {
        int lo = -1, hi = 1 << 30;  // fewer than `need` up to lo, at least as many up to hi: a vocabulary's places are below
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            if (total(count(mid)) >= need) hi = mid;
            else lo = mid;
        }
        return hi;
    }

    // The sum taken to a higher base.
    __device__ __forceinline__ void raise_base(float to) {
        const float f = pow2(scaled<false>(low - base_of(to), scale));
        s[0] = mul2(s[0], pack2(f, f));
        s[1] = mul2(s[1], pack2(f, f));
        low = to;
        base = pack2(-base_of(to), -base_of(to));
    }
    __device__ __forceinline__ void add_one(float x) {
        s[0] = add2(s[0], pack2(pow2(scaled<false>(x - base_of(low), scale)), 0.0f));
    }
    __device__ __forceinline__ void add(const uint4& v) {
#pragma unroll
        for (int i = 0; i < kVec<T> / 2; ++i) {
            const uint64_t t = add2(widen2<T>(v, i), base);
            const float2 z = unpack2(fma2(t, lo2, mul2(t, c2)));
            s[i & 1] = add2(s[i & 1], pack2(pow2(z.x), pow2(z.y)));
        }
    }
    __device__ __forceinline__ void keep(float x, int place) {
        const int at = atomicAdd(&sm.n, 1);
        if (at < CAP) sm.cand[at] = candidate(x, place);
    }

    // Cuts the candidates back to at most top_few(k), the k best among them.
    __device__ __forceinline__ void cut_back() {
        constexpr int kMine = CAP / THREADS;
        const int few = top_few(k);
        if (n <= few) return;
        uint64_t mine[kMine];
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            mine[i] = id + i * THREADS < n ? sm.cand[id + i * THREADS] : 0;
            best = max(best, (uint32_t)(mine[i] >> 32));
        }
        best = largest(best);
        auto reaches = [&](float v) {
            const uint32_t key = key_of(v);
            int c = 0;
#pragma unroll
            for (int i = 0; i < kMine; ++i) c += (uint32_t)(mine[i] >> 32) >= key;
            return c;
        };
        int reach = n;
        const uint32_t key = cut(reaches, have ? max(key_of(low), kKeyLow) : kKeyLow, best + 1, few, reach);
        int last = INT_MAX;  // among those of the key itself
        if (reach > few) {
            int above = 0;
#pragma unroll
            for (int i = 0; i < kMine; ++i) above += (uint32_t)(mine[i] >> 32) > key;
            above = total(above);
            last = cut_places(
                [&](int p) {
                    int c = 0;
#pragma unroll
                    for (int i = 0; i < kMine; ++i) c += (uint32_t)(mine[i] >> 32) == key && (int)~(uint32_t)mine[i] <= p;
                    return c;
                },
                k - above);
        }
        raise_base(value_of(key));
        have = true;
        sync();
        if (id == 0) sm.n = 0;
        sync();
        int kept = 0;
        // Candidates lie in no fixed order: what is dropped is added up in whole numbers, of 2^-44 of the
        // threshold's own term, so that equal calls give equal bits.
        unsigned long long gone = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            if (mine[i] == 0) continue;
            const uint32_t its = (uint32_t)(mine[i] >> 32);
            if (its > key || (its == key && (int)~(uint32_t)mine[i] <= last)) {
                sm.cand[atomicAdd(&sm.n, 1)] = mine[i];
                ++kept;
            } else {
                gone += __float2ull_rn(pow2(scaled<false>(value_of(its) - base_of(low), scale)) * 0x1p44f);
            }
        }
        const unsigned high = __reduce_add_sync(~0u, (unsigned)(gone >> 22)), rest = __reduce_add_sync(~0u, (unsigned)gone & 0x3FFFFFu);
        gone = ((unsigned long long)high << 22) + rest;
        if (THREADS > 32 && (id & 31) == 0) sm.gone[id >> 5] = gone;
        n = total(kept);
        if (id == 0) {
            if (THREADS > 32) {
                gone = 0;
                for (int w = 0; w < THREADS / 32; ++w) gone += sm.gone[w];
            }
            s[0] = add2(s[0], pack2(__ull2float_rn(gone) * 0x1p-44f, 0.0f));
        }
    }

    // ---- the usual way -----------------------------------------------------------------
    // A segment is `vectors` vectors of a thread, THREADS apart; the row's are numbered through. 2^(x C - from),
    // with the product inside the fused operation, so that differences of any large values are kept.
    __device__ __forceinline__ void term(uint64_t (&sum)[2], int i, uint64_t x, uint64_t from) const {
        const float2 z = unpack2(fma2(x, lo2, fma2(x, c2, from)));
        sum[i & 1] = add2(sum[i & 1], pack2(pow2(z.x), pow2(z.y)));
    }

    // A key that at least k of the threads' keys reach and at most four more, or more that equal it. By a warp.
    __device__ __forceinline__ uint32_t few_reach() const {
        constexpr int kEach = 2 * THREADS / 32;
        uint32_t mine[kEach], lo = ~0u, hi = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            mine[i] = sm.keys[id + 32 * i];
            lo = min(lo, mine[i]);
            hi = max(hi, mine[i]);
        }
        lo = __reduce_min_sync(~0u, lo);
        hi = __reduce_max_sync(~0u, hi) + 1;
        int reach = 2 * THREADS;
        while (reach > k + 4 && hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            int c = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) c += mine[i] >= mid;
            c = __reduce_add_sync(~0u, c);
            if (c >= k) {
                lo = mid;
                reach = c;
            } else {
                hi = mid;
            }
        }
        return lo;
    }

    // A whole row, or a CTA's share of it, of which each thread has a vector. False: it has to be taken the other way.
    __device__ __forceinline__ bool fast(const Slice<T>& part, const T* x, int vectors) {
        const int per = vectors * THREADS, segments = (part.n + per - 1) / per;
        float* const tops = sm.largest();
        float* const segs = tops + segments * THREADS;
        float halves[2] = {-INFINITY, -INFINITY}, base_c = 0.0f;
        T head, tail;  // read before they are wanted
        if (id < part.head) head = x[id];
        if (id < part.tail) tail = x[part.tail_at + id];
        uint64_t from = 0;
        float least = INFINITY;  // of the segments' largest values
        float top = -INFINITY;
        uint64_t sum[2] = {pack2(0.0f, 0.0f), pack2(0.0f, 0.0f)};
        constexpr int kStep = kUnroll * THREADS;
        const int steps = (part.n + kStep - 1) / kStep;
        int left = vectors;  // of the segment at hand
        float* its_top = tops + id;
        float* its_sum = segs + id;
        auto load = [&](uint4* q, int c) {
            const uint4* v = part.v + c * kStep + id;
            if ((c + 1) * kStep <= part.n) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) q[u] = THREADS == 32 ? __ldg(v + u * THREADS) : load_once(v + u * THREADS);
            } else {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    q[u] = lowest();
                    if (c * kStep + id + u * THREADS < part.n) q[u] = THREADS == 32 ? __ldg(v + u * THREADS) : load_once(v + u * THREADS);
                }
            }
        };
        auto use = [&](const uint4* q, int c) {
            const float half = largest_of(q), other = largest_of(q + kUnroll / 2), its = fmaxf(half, other);
            halves[0] = fmaxf(halves[0], half);
            halves[1] = fmaxf(halves[1], other);
            top = fmaxf(top, its);
            if (c == 0) {  // the base: the least of the warp's largest first values
                float low = its;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) low = fminf(low, __shfl_xor_sync(~0u, low, o));
                base_c = low * scale.c;
                from = pack2(-base_c, -base_c);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
                for (int i = 0; i < kVec<T> / 2; ++i) term(sum, i, widen2<T>(q[u], i), from);
                if (THREADS == 32) {  // a segment each
                    const int at = (c * kUnroll + u) * THREADS;
                    if (at < part.n) {
                        const float2 f = unpack2(add2(sum[0], sum[1]));
                        const float largest = fmaxf(-INFINITY, max_of<T>(q[u]));
                        tops[at + id] = largest;
                        segs[at + id] = f.x + f.y;
                        if (at + id < part.n) least = fminf(least, largest);
                    }
                    sum[0] = sum[1] = pack2(0.0f, 0.0f);
                }
            }
            if (THREADS > 32) {
                left -= kUnroll;
                if (left == 0 || c == steps - 1) {
                    const float2 f = unpack2(add2(sum[0], sum[1]));
                    *its_top = top;
                    *its_sum = f.x + f.y;
                    its_top += THREADS;
                    its_sum += THREADS;
                    if ((c / (vectors / kUnroll)) * per + id < part.n) least = fminf(least, top);
                    sum[0] = sum[1] = pack2(0.0f, 0.0f);
                    top = -INFINITY;
                    left = vectors;
                }
            }
        };
        {
            uint4 a[kUnroll], b[kUnroll];
            load(a, 0);
            for (int c = 0;;) {  // the next vectors are on their way beside these
                if (c + 1 < steps) load(b, c + 1);
                use(a, c);
                if (++c >= steps) break;
                if (c + 1 < steps) load(a, c + 1);
                use(b, c);
                if (++c >= steps) break;
            }
        }
        if ((id & 31) == 0) sm.bases[id >> 5] = base_c;
        if (THREADS == 32) __syncwarp();  // a warp's threshold may take no other barrier (equal maxima in all lanes)

        // the threshold
        const float most = fmaxf(halves[0], halves[1]);
        float limit;
        if (kRanked > 0 && THREADS > 32) {  // by the threads' largest values, which one warp looks through
            sm.keys[id] = key_of(halves[0]);
            sm.keys[THREADS + id] = key_of(halves[1]);
            sync();
            if (id < 32) {
                const uint32_t key = few_reach();
                if (id == 0) sm.key = key;
            }
            sync();
            limit = value_of(sm.key);
        } else {  // by the segments' largest values
            const int groups = THREADS == 32 ? part.n : (segments - 1) * THREADS + min(THREADS, part.n - (segments - 1) * per);
            if (groups < 2 * k) return false;
            const uint32_t best = largest(key_of(most)), lo = ~largest(~key_of(k <= THREADS ? most : least));
            int reach = INT_MAX;
            const uint32_t key = cut(
                [&](float v) {
                    int c = 0;
                    for (int g = 0; g < segments; ++g) c += tops[g * THREADS + id] >= v;
                    return c;
                },
                lo, best + 1, k + k / 4 + 8, reach);
            limit = value_of(key);
        }
        // not -inf, and no base so far above it that its terms are too small to count, or so far below that they overflow
        bool good = limit > -INFINITY;
        float gap = 0.0f;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            const float its = base_of_rest(limit, sm.bases[w]);
            good = good && fabsf(its) <= 80.0f;
            if (w == id >> 5) gap = its;
        }
        if (!good) return false;
        low = limit;
        have = true;

        // the segments that reach it: one place on the list for all of a thread's
        uint32_t marks = 0;
#pragma unroll 4
        for (int g = 0; g < segments; ++g) marks |= (uint32_t)(tops[g * THREADS + id] >= limit) << g;
        if (marks) {
            int to = atomicAdd(&sm.hots, __popc(marks));
            for (; marks; marks &= marks - 1, ++to)
                if (to < Space::kHot) sm.hot[to] = (__ffs(marks) - 1) * THREADS + id;
        }
        sync();
        const int hots = sm.hots;
        if (hots > Space::kHot) return false;
        for (int h = id; h < hots; h += THREADS) {
            const int its = sm.hot[h], g = its / THREADS, who = its % THREADS;
            const float its_base = sm.bases[who >> 5];
            const uint64_t its_from = pack2(-its_base, -its_base);
            uint64_t sum[2] = {pack2(0.0f, 0.0f), pack2(0.0f, 0.0f)};
            for (int at = g * per + who, end = min(part.n, (g + 1) * per); at < end; at += kUnroll * THREADS) {
                uint4 q[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    q[u] = lowest();
                    if (at + u * THREADS < end) q[u] = __ldg(part.v + at + u * THREADS);
                }
                // the candidates' bits, and the sum with -inf in their place: a branch for each would run for each
                uint32_t marks = 0;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
                    for (int i = 0; i < kVec<T> / 2; ++i) {
                        float2 e = unpack2(widen2<T>(q[u], i));
                        if (e.x >= limit) {
                            marks |= 1u << (u * kVec<T> + 2 * i);
                            e.x = -INFINITY;
                        }
                        if (e.y >= limit) {
                            marks |= 1u << (u * kVec<T> + 2 * i + 1);
                            e.y = -INFINITY;
                        }
                        term(sum, i, pack2(e.x, e.y), its_from);
                    }
                }
                while (marks) {
                    const int bit = __ffs(marks) - 1, place = part.first + (at + bit / kVec<T> * THREADS) * kVec<T> + bit % kVec<T>;
                    marks &= marks - 1;
                    keep(widen(x[place]), place);
                }
            }
            const float2 f = unpack2(add2(sum[0], sum[1]));
            segs[its] = f.x + f.y;
        }
        sync();
        float mass = 0.0f;
        for (int g = 0; g < segments; ++g) mass += segs[g * THREADS + id];
        s[0] = pack2(mass * pow2(gap), 0.0f);
        s[1] = pack2(0.0f, 0.0f);
        base = pack2(-low, -low);
        // the ends of the row
        if (id < part.head) {
            const float e = widen(head);
            if (e >= low) keep(e, id);
            else add_one(e);
        }
        if (id < part.tail) {
            const float e = widen(tail);
            if (e >= low) keep(e, part.tail_at + id);
            else add_one(e);
        }
        sync();
        n = sm.n;
        if (n > CAP) return false;
        if (n > kRanked) cut_back();
        return true;
    }
    // The exponent that takes sums over a base to the base `to`.
    __device__ __forceinline__ float base_of_rest(float to, float base_c) const { return -fmaf(to, scale.lo, fmaf(to, scale.c, -base_c)); }
    // The largest value of two vectors; NaN beside numbers is passed over.
    static __device__ __forceinline__ float largest_of(const uint4* q) {
        if constexpr (sizeof(T) == 4) {
            return fmaxf(max_of<T>(q[0]), max_of<T>(q[1]));
        } else {
            using P = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
            const P* h = reinterpret_cast<const P*>(q);
            const P m = __hmax2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])), __hmax2(__hmax2(h[4], h[5]), __hmax2(h[6], h[7])));
            return fmaxf(widen(m.x), widen(m.y));
        }
    }
    static __device__ __forceinline__ uint4 lowest() {
        uint4 v;
#pragma unroll
        for (int i = 0; i < kVec<T> / 2; ++i) narrow2<T>(v, i, make_float2(-INFINITY, -INFINITY));
        return v;
    }

    // ---- the way that holds for all rows -----------------------------------------------
    // Takes a chunk: `present` says which of this thread's vectors there are, vector u begins at place at + u * step.
    // full: all threads have all of theirs.
    __device__ __forceinline__ void chunk(uint4* q, const bool* present, int at, int step, bool full) {
        if (have && n > CAP / 2) cut_back();
        float limit = low;  // kept: values above it ..
        int last = -1;      // .. and equal ones up to this place
        const int before = n;
        bool done = false;
        if (have) {
            int mine = 0;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (present[u] && max_of<T>(q[u]) > limit) mine += push(q[u], at + u * step, limit, last);
            n += total(mine);
            done = n <= kRoom;
        } else {
            int there = 0;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) there += present[u] ? kVec<T> : 0;
            if (total(there) <= kRoom - n) {  // all of it fits
                limit = -INFINITY;
                last = INT_MAX;
            } else {
                limit = first_limit(q, present, full);
                last = INT_MAX;
            }
            int mine = 0;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (present[u]) mine += push(q[u], at + u * step, limit, last);
            n += total(mine);
            done = n <= kRoom;
        }
        if (!done) {  // more than fit: the chunk's own k best, and the candidates cut back
            sync();
            if (id == 0) sm.n = before;
            n = before;
            sync();
            cut_back();
            pick(q, present, at, step, limit, last);
            int mine = 0;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (present[u]) mine += push(q[u], at + u * step, limit, last);
            n += total(mine);
        }
        if (limit > low || !have) {
            if (n - before >= k || have) {
                // at least k candidates are not below the limit
                if (limit > low) raise_base(limit);
                have = have || n - before >= k;
            }
        }
        if (have) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (!present[u]) continue;
                if (!(max_of<T>(q[u]) < limit)) strike(q[u], at + u * step, limit, last);
                add(q[u]);
            }
        } else {  // no threshold yet: everything but NaN was kept
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (present[u]) add_missing(q[u]);
        }
    }

private:
    static __device__ __forceinline__ bool kept(float x, int place, float limit, int last) { return x > limit || (x == limit && place <= last); }

    __device__ __forceinline__ int push(const uint4& v, int at, float limit, int last) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < kVec<T> / 2; ++i) {
            const float2 x = unpack2(widen2<T>(v, i));
            if (kept(x.x, at + 2 * i, limit, last)) {
                keep(x.x, at + 2 * i);
                ++c;
            }
            if (kept(x.y, at + 2 * i + 1, limit, last)) {
                keep(x.y, at + 2 * i + 1);
                ++c;
            }
        }
        return c;
    }
    // -inf in the place of what was kept.
    __device__ __forceinline__ void strike(uint4& v, int at, float limit, int last) {
#pragma unroll
        for (int i = 0; i < kVec<T> / 2; ++i) {
            float2 x = unpack2(widen2<T>(v, i));
            if (kept(x.x, at + 2 * i, limit, last)) x.x = -INFINITY;
            if (kept(x.y, at + 2 * i + 1, limit, last)) x.y = -INFINITY;
            narrow2<T>(v, i, x);
        }
    }
    __device__ __forceinline__ void add_missing(const uint4& v) {
#pragma unroll
        for (int i = 0; i < kVec<T> / 2; ++i) {
            const float2 x = unpack2(widen2<T>(v, i));
            if (x.x != x.x || x.y != x.y) s[0] = pack2(NAN, NAN);
        }
    }

    // A value that at least k of the chunk reach, and not many more: by the maxima of groups of four.
    __device__ __forceinline__ float first_limit(const uint4* q, const bool* present, bool full) {
        constexpr int kGroups = kVec<T> / 4;
        float top[kUnroll * kGroups];
        float most = -INFINITY, least = INFINITY;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const float2 a = unpack2(widen2<T>(q[u], 2 * g)), b = unpack2(widen2<T>(q[u], 2 * g + 1));
                const float m = fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y));  // a NaN is passed over
                top[u * kGroups + g] = present[u] && m == m ? m : -INFINITY;
                most = fmaxf(most, top[u * kGroups + g]);
                least = fminf(least, top[u * kGroups + g]);
            }
        }
        const uint32_t best = largest(key_of(most));
        // each thread has a group that reaches the least of all threads' largest
        uint32_t lo = kKeyLow;
        if (full) lo = ~largest(~key_of(k <= THREADS ? most : least));
        int reach = INT_MAX;
        const uint32_t key = cut(
            [&](float v) {
                int c = 0;
#pragma unroll
                for (int i = 0; i < kUnroll * kGroups; ++i) c += top[i] >= v;
                return c;
            },
            lo, best + 1, k + k / 4 + 8, reach);
        return value_of(key);
    }

    // The limit that the chunk's k best are kept by. At least k values are above (limit, last), or fewer and all fit.
    __device__ __forceinline__ void pick(const uint4* q, const bool* present, int at, int step, float& limit, int& last) {
        auto members = [&](auto is) {
            int c = 0;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (!present[u]) continue;
#pragma unroll
                for (int i = 0; i < kVec<T> / 2; ++i) {
                    const float2 x = unpack2(widen2<T>(q[u], i));
                    c += is(x.x, at + u * step + 2 * i) + is(x.y, at + u * step + 2 * i + 1);
                }
            }
            return c;
        };
        if (have) {  // the candidates' threshold may have risen
            limit = low;
            last = -1;
        }
        const int few = min(top_few(k), kRoom - n);
        int reach = total(members([&](float x, int p) { return (int)kept(x, p, limit, last); }));
        if (reach <= few) return;
        uint32_t best = 0;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (!present[u]) continue;
            const float m = max_of<T>(q[u]);
            if (m == m) best = max(best, key_of(m));
        }
        best = largest(best);
        const uint32_t from = last < 0 ? key_of(limit) + 1 : max(key_of(limit), kKeyLow);
        const uint32_t key = cut([&](float v) { return members([&](float x, int) { return (int)(x >= v); }); }, from, best + 1, few, reach);
        limit = value_of(key);
        last = INT_MAX;
        if (reach > few) {
            const float v = limit;
            const int above = total(members([&](float x, int) { return (int)(x > v); }));
            last = cut_places([&](int most) { return members([&](float x, int p) { return (int)(x == v && p <= most); }); }, k - above);
        }
    }
};

// A row, or a CTA's share of it, chunk by chunk (TopRow::chunk).
template <class T, int THREADS, int CAP>
__device__ __noinline__ Taken top_slow(TopSpace<THREADS, CAP>& sm, const Slice<T> part, const T* x, Scale scale, int k) {
    TopRow<T, THREADS, CAP> row(sm, scale, k);
    const int id = row.id;
    if (part.head) {
        int mine = 0;
        if (id < part.head) {
            const float v = widen(x[id]);
            if (v == v) {
                row.keep(v, id);
                mine = 1;
            } else {
                row.s[0] = pack2(NAN, NAN);
            }
        }
        row.n += row.total(mine);
    }
    for (int from = 0; from < part.n; from += kUnroll * THREADS) {
        uint4 v[kUnroll];
        bool present[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = from + id + u * THREADS;
            present[u] = i < part.n;
            if (present[u]) v[u] = __ldg(part.v + i);
        }
        row.chunk(v, present, part.first + (from + id) * kVec<T>, THREADS * kVec<T>, from + kUnroll * THREADS <= part.n);
    }
    if (part.tail) {
        int mine = 0;
        if (id < part.tail) {
            const float v = widen(x[part.tail_at + id]);
            if (row.have ? v > row.low : v == v) {
                row.keep(v, part.tail_at + id);
                mine = 1;
            } else if (row.have || v != v) {
                row.add_one(v);
            }
        }
        row.n += row.total(mine);
    }
    row.cut_back();
    return row.taken();
}

// Sorts a list of n <= MOST numbers, all different, the largest first: each thread counts what is larger than its own.
// With more than one warp's threads that takes a quarter of the time that one warp's sorting network does.
template <int THREADS, int MOST, class S>
__device__ __forceinline__ void rank_all(uint64_t* list, int n, S sync) {
    constexpr int kMine = MOST / THREADS;
    const int id = place_in_group<THREADS>();
    uint64_t mine[kMine];
    int rank[kMine];
#pragma unroll
    for (int r = 0; r < kMine; ++r) {
        mine[r] = id + r * THREADS < n ? list[id + r * THREADS] : ~0ull;
        rank[r] = 0;
    }
    if ((THREADS == 32 ? 0 : id & ~31) < n) {
        const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(list);
        auto count = [&](auto each) {  // numbers of this thread
#pragma unroll 4
            for (int j = 0; j < n / 2; ++j) {
                const ulonglong2 p = pairs[j];
#pragma unroll
                for (int r = 0; r < decltype(each)::value; ++r) rank[r] += (p.x > mine[r]) + (p.y > mine[r]);
            }
            if (n & 1)
#pragma unroll
                for (int r = 0; r < decltype(each)::value; ++r) rank[r] += list[n - 1] > mine[r];
        };
        if (n <= THREADS) count(std::integral_constant<int, 1>());
        else if (n <= 2 * THREADS) count(std::integral_constant<int, kMine < 2 ? kMine : 2>());
        else count(std::integral_constant<int, kMine>());
    }
    sync();
#pragma unroll
    for (int r = 0; r < kMine; ++r)
        if (id + r * THREADS < n) list[rank[r]] = mine[r];
    sync();
}

// Sorts a longer list, of n <= size_all, a power of two; 0 fills up, and is smaller than any candidate.
template <int THREADS>
__device__ __forceinline__ void sort_in_place(uint64_t* list, int n, int size_all) {
    for (int i = n + threadIdx.x; i < size_all; i += THREADS) list[i] = 0;
    __syncthreads();
    for (int size = 2; size <= size_all; size *= 2) {
        for (int stride = size / 2; stride > 0; stride /= 2) {
            for (int p = threadIdx.x; p < size_all / 2; p += THREADS) {
                const int i = 2 * p - (p & (stride - 1)), j = i + stride;
                const uint64_t a = list[i], b = list[j];
                if ((a < b) == ((i & size) == 0)) {
                    list[i] = b;
                    list[j] = a;
                }
            }
            __syncthreads();
        }
    }
}

struct TopOut {
    int64_t* index;
    float *logp, *lse, *rest;
};

// A CTA of 128 threads per row (256 for k > 128), several per short batch's row, or a warp per short row. 8192 x 50257 bf16 with a
// quarter masked, k = 64: 142 us, 65% of the copy peak on 624 MB; k = 8 unmasked 143 us, 85%. The stream alone keeps up with
// HBM; what a row does after it (threshold, segments read again, ranking) is a chain of latencies of 9 us, behind which eight
// CTAs of an SM hide three quarters: with four of 256 threads 206 us. Loads run a step ahead of the sums (170 us without).
template <class T, int THREADS, int CAP>
__global__ void __launch_bounds__(THREADS == 32 ? kRowThreads : THREADS, THREADS == 32 ? 3 : 1024 / THREADS) k_top_rows(const Rows<T> a, int k, int size, int vectors, int space, const TopOut out) {
    using Row = TopRow<T, THREADS, CAP>;
    extern __shared__ __align__(16) uint8_t smem[];
    typename Row::Space& sm = *reinterpret_cast<typename Row::Space*>(smem + (THREADS == 32 ? (threadIdx.x >> 5) * space : 0));
    wait_for_kernel_before();
    let_next_kernel_start();
    const int64_t t = row_of<THREADS>(size);
    if (THREADS == 32 && t >= a.rows) return;
    const int rank = THREADS == 32 ? 0 : (int)(blockIdx.x % size), id = place_in_group<THREADS>();
    if (a.targets && a.targets[t] < 0) {
        if (rank == 0) {
            for (int i = id; i < k; i += THREADS) {
                out.index[t * k + i] = -1;
                out.logp[t * k + i] = 0.0f;
            }
            if (id == 0) out.lse[t] = out.rest[t] = 0.0f;
        }
        return;
    }
    const T* x = a.x + t * a.stride;
    const Slice<T> part(x, a.vocab, rank, size);
    Taken taken;
    bool done = false;
    if (part.n >= THREADS) {  // each thread has a vector
        Row fast(sm, a.k, k + 1);  // one more: the largest of the rest, the base of its sum
        done = fast.fast(part, x, vectors);
        taken = fast.taken();
    }
    if (!done) taken = top_slow<T, THREADS, CAP>(sm, part, x, a.k, k + 1);
    Row row(sm, a.k, k + 1, taken);

    // The sum of what is no candidate, and the other CTAs' candidates and sums.
    auto group_sum = [&](float2 v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(~0u, v.x, o);
            v.y += __shfl_xor_sync(~0u, v.y, o);
        }
        if (THREADS == 32) return v;
        Row::sync();
        if ((id & 31) == 0) sm.floats[id >> 5] = v;
        Row::sync();
        v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            v.x += sm.floats[w].x;
            v.y += sm.floats[w].y;
        }
        return v;
    };
    float lows[8], rests[8];
    if (THREADS != 32 && size > 1) {
        cg::cluster_group cl = cg::this_cluster();
        const float2 s2 = unpack2(add2(row.s[0], row.s[1]));
        const float mine = group_sum(make_float2(s2.x + s2.y, 0.0f)).x;
        if (id == 0) {
            sm.kept = row.n;
            sm.low = row.low;
            sm.rest = mine;
        }
        cl.sync();
        if (rank == 0) {
            for (int r = 1; r < size; ++r) {
                const typename Row::Space* other = cl.map_shared_rank(&sm, r);
                const int more = other->kept;
                if (row.n + more > Row::kRoom) row.cut_back();
                for (int i = id; i < more; i += THREADS) sm.cand[row.n + i] = other->cand[i];
                row.n += more;
                Row::sync();
                if (id == 0) sm.n = row.n;
                Row::sync();
            }
            row.cut_back();
        }
#pragma unroll
        for (int r = 1; r < 8; ++r) {
            lows[r] = -INFINITY;
            rests[r] = 0.0f;
            if (rank == 0 && r < size) {
                const typename Row::Space* other = cl.map_shared_rank(&sm, r);
                lows[r] = other->low;
                rests[r] = other->rest;
            }
        }
        cl.sync();  // the others may leave
        if (rank != 0) return;
    }
    Row::sync();
    const int n = row.n;
    if constexpr (Row::kRanked > 0) {
        rank_all<THREADS, Row::kRanked>(sm.cand, n, [] { Row::sync(); });
    } else {
        int all = 256;
        while (all < n) all *= 2;
        sort_in_place<THREADS>(sm.cand, n, all);
    }
    // The rest over a base that none of its terms exceeds, and all over the row's maximum.
    const float top = n > 0 ? value_of((uint32_t)(sm.cand[0] >> 32)) : -INFINITY;
    // (its largest: every CTA's threshold is one that k + 1 candidates reach)
    const float under = n > k ? value_of((uint32_t)(sm.cand[k] >> 32)) : row.low;
    const float top_base = base_of(top), under_base = base_of(under);
    row.raise_base(under);
    const float2 s2 = unpack2(add2(row.s[0], row.s[1]));
    float rest = s2.x + s2.y, sel = 0.0f;
    for (int i = id; i < n; i += THREADS) {
        const float v = value_of((uint32_t)(sm.cand[i] >> 32));
        if (i < k) sel += pow2(scaled<false>(v - top_base, a.k));
        else rest += pow2(scaled<false>(v - under_base, a.k));
    }
    const float2 sums = group_sum(make_float2(rest, sel));
    rest = sums.x;
    sel = sums.y;
    if (THREADS != 32 && size > 1) {
#pragma unroll
        for (int r = 1; r < 8; ++r) rest += r < size ? rests[r] * pow2(scaled<false>(lows[r] - under_base, a.k)) : 0.0f;
    }
    if (id >= k) return;  // no result of this thread's
    const float2 inv_t = inverse(a.inv_t);
    const float total = sel + rest * pow2(scaled<false>(under_base - top_base, a.k));
    const float2 all = log_parts(total, 1.0f - 1.0f / total), outside = log_parts(rest);
    const bool nothing = total == 0.0f;  // -inf alone
    for (int i = id; i < k; i += THREADS) {
        const uint64_t its = i < n ? sm.cand[i] : 0;
        const float v = value_of((uint32_t)(its >> 32));
        out.index[t * k + i] = i < n ? (int64_t)(int)~(uint32_t)its : -1;
        const float2 z = over_base(v, top_base, inv_t);
        // a row that holds NaN or +inf (total is NaN) has no results, also where -inf is listed
        out.logp[t * k + i] = i >= n || total != total ? NAN : nothing || v == -INFINITY ? -INFINITY : __fsub_rn(z.x, all.x) + (z.y - all.y);
    }
    if (id == 0) {
        const float2 z = over_base(under_base, top_base, inv_t);
        out.lse[t] = nothing ? -INFINITY : fmaf(top_base, inv_t.x, all.x) + fmaf(top_base, inv_t.y, all.y);
        // from the smaller of the two probabilities
        out.rest[t] = rest == 0.0f && total == total ? -INFINITY
                      : sel < 0.5f * total           ? log1pf(-sel / total)
                                                     : __fadd_rn(z.x, outside.x - all.x) + (z.y + (outside.y - all.y));
    }
}

// Rows of up to this many bytes, enough of them for every SM and short lists: a warp each. 8192 x 4000 bf16, k = 20: 30 us.
constexpr int64_t kTopShort = 16384;
constexpr int kTopShortMost = 64;

template <class T, int THREADS, int CAP>
int launch_top(const zero_logits* x, int k, int size, const TopOut& out, unsigned grid, cudaStream_t s) {
    // a segment: one vector of a warp's short row, else four, or as many as leave kSegments
    constexpr int kMost = THREADS == 32 ? kShortSegments : kSegments;
    static_assert(kTopShort <= 16 * 32 * kShortSegments, "a warp's row has a segment for every vector");
    const int64_t vecs = (x->vocab * type_size(x->type) / 16 + size - 1) / size;
    int vectors = THREADS == 32 ? 1 : kUnroll;
    while (vecs > (int64_t)kMost * vectors * THREADS) vectors += kUnroll;
    const int segments = (int)((vecs + vectors * THREADS - 1) / (vectors * THREADS));
    const int space = (int)(sizeof(TopSpace<THREADS, CAP>) + 8 * (size_t)segments * THREADS);
    const size_t bytes = (size_t)space * (THREADS == 32 ? kRowThreads / 32 : 1);
    auto* kernel = k_top_rows<T, THREADS, CAP>;
    constexpr size_t kBytes = (sizeof(TopSpace<THREADS, CAP>) + 8 * (size_t)THREADS * kMost) * (THREADS == 32 ? kRowThreads / 32 : 1);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kBytes);
    if (e != cudaSuccess) return record_cuda_error(e);
    return launch_linked(kernel, grid, THREADS == 32 ? kRowThreads : THREADS, bytes, size, s, rows_of<T>(x, nullptr), k, size, vectors, space, out);
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" int zero_top_logits(const zero_logits* x, int64_t k, int64_t* index, float* logp, float* lse, float* rest, void* stream) {
    int rc = check_logits(x);
    if (!rc && (k < 1 || k > kTopMost || k > x->vocab)) rc = ZERO_ERR_INVALID_ARG;
    if (rc || x->rows == 0) return rc;
    CallDevice d(x->logits, stream);
    d.need(x->logits, type_size(x->type));
    d.optional(x->targets, 8);
    d.need(index, 8);
    d.need(logp, 4);
    d.need(lse, 4);
    d.need(rest, 4);
    if (d.rc) return d.rc;
    const int sms = d.sm_count(), most = (int)k;
    const TopOut out = {index, logp, lse, rest};
    cudaStream_t s = (cudaStream_t)stream;
    return by_type(x->type, [&](auto tag) {
        using T = decltype(tag);
        if (x->vocab * type_size(x->type) <= kTopShort && most <= kTopShortMost && x->rows >= 8 * (int64_t)sms)
            return launch_top<T, 32, 256>(x, most, 1, out, (unsigned)((x->rows + kRowThreads / 32 - 1) / (kRowThreads / 32)), s);
        const int size = ctas_per_row(x, sms);
        const unsigned grid = (unsigned)(x->rows * size);
        if (most <= 128) return launch_top<T, 128, 512>(x, most, size, out, grid, s);
        return most <= 256 ? launch_top<T, 256, 1024>(x, most, size, out, grid, s) : launch_top<T, 256, 2048>(x, most, size, out, grid, s);
    });
}
