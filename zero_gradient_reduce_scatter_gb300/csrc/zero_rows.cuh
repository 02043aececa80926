// Rows of logits as the kernels over a vocabulary take them: a row's 16-byte vectors and its ends, how a
// CTA, a warp or a cluster shares it, the weights of a batch's tokens and the means of their losses,
// and the host's checks and launch shapes.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cooperative_groups.h>

#include "zero_host.h"
#include "zero_softmax.cuh"
#include "zero_sum.cuh"
#include "zero_tcgen05.cuh"

namespace zg {
namespace {

namespace cg = cooperative_groups;

constexpr int kRowThreads = 256;
constexpr int kRowCtas = 12;  // CTAs of an SM up to which short batches cut their rows
constexpr int kUnroll = 4;  // 16-byte loads of a thread on their way at a time

// Logits as the kernels take them.
template <class T>
struct Rows {
    const T* x;
    const int64_t* targets;
    const float* weight;  // nullptr, or 0 for rows that carry no loss
    int64_t rows, vocab, stride;
    Scale k;              // log2(e) / temperature
    float c;              // the same in one number, for gradients
    double inv_t;         // 1 / temperature
};

template <class T>
__device__ __forceinline__ int64_t live_target(const Rows<T>& a, int64_t t) {
    return a.weight && a.weight[t] == 0.0f ? -1 : a.targets[t];
}

// A row as the CTAs of a cluster share it: up to 7 elements before the first 16-byte boundary
// (the first CTA's), `n` whole vectors of each CTA from element `first` on, and up to 7 elements
// behind the last (the last CTA's). A row of an odd vocabulary starts at any even address.
template <class T>
struct Slice {
    int head, n, first, tail_at, tail;
    const uint4* v;  // this CTA's vectors

    __device__ __forceinline__ Slice(const T* x, int64_t vocab, int rank, int size) {
        const int len = (int)vocab, to = (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T);
        const int before = min(to, len), vecs = (len - before) / kVec<T>, per = (vecs + size - 1) / size;
        const int lo = min(per * rank, vecs);
        n = min(per, vecs - lo);
        first = before + lo * kVec<T>;
        tail_at = before + vecs * kVec<T>;
        head = rank == 0 ? before : 0;
        tail = rank == size - 1 ? len - tail_at : 0;
        v = reinterpret_cast<const uint4*>(x + first);
    }
};

// A thread's place among the THREADS that share a row: those of a CTA, or of a warp.
template <int THREADS>
__device__ __forceinline__ int place_in_group() { return THREADS == 32 ? threadIdx.x & 31 : threadIdx.x; }

// This thread's vectors of n, from its place `i` on, kUnroll at a time: `load` first for all of them,
// then `use`.
template <int THREADS, class L, class U>
__device__ __forceinline__ void for_vectors(int n, L load, U use, int i = place_in_group<THREADS>()) {
    for (; i + (kUnroll - 1) * THREADS < n; i += kUnroll * THREADS) {
        uint4 q[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) q[u] = load(i + u * THREADS);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) use(i + u * THREADS, q[u]);
    }
    if (i < n) {
        uint4 q[kUnroll - 1];
#pragma unroll
        for (int u = 0; u < kUnroll - 1; ++u)
            if (i + u * THREADS < n) q[u] = load(i + u * THREADS);
#pragma unroll
        for (int u = 0; u < kUnroll - 1; ++u)
            if (i + u * THREADS < n) use(i + u * THREADS, q[u]);
    }
}

// The part of a row that a thread reads first: its first vectors and its elements at the row's ends,
// on their way at once with whatever else the row waits for.
template <class T, int THREADS>
struct RowStart {
    uint4 q[kUnroll];
    T head, tail;

    template <class L>
    __device__ __forceinline__ RowStart(const Slice<T>& s, const T* x, L load) {
        const int id = place_in_group<THREADS>();
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (id + u * THREADS < s.n) q[u] = load(id + u * THREADS);
        if (id < s.head) head = x[id];
        if (id < s.tail) tail = x[s.tail_at + id];
    }
    // for_vectors over all of the thread's vectors
    template <class L, class U>
    __device__ __forceinline__ void vectors(int n, L load, U use) const {
        const int id = place_in_group<THREADS>();
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (id + u * THREADS < n) use(id + u * THREADS, q[u]);
        for_vectors<THREADS>(n, load, use, id + kUnroll * THREADS);
    }
};

// The sums of all CTAs of a cluster (at most 8), joined in a fixed order; valid everywhere. `mine` is
// shared memory of this CTA, which stays as it is until the cluster's next barrier. A lane reads a
// CTA's sums, so that their latencies are one.
template <bool ENTROPY>
__device__ __forceinline__ RowStat cluster_join(RowStat a, int size, Scale k, RowStat* mine) {
    if (size == 1) return a;
    cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x == 0) *mine = a;
    cl.sync();
    const int lane = threadIdx.x & 7;
    a = lane < size ? *cl.map_shared_rank(mine, lane) : empty_stat();
    return warp_join<ENTROPY, true, 8>(a, k);
}

// The row and the part of it that this thread works on: `size` CTAs per row, or (THREADS = 32) a
// warp each.
template <int THREADS>
__device__ __forceinline__ int64_t row_of(int size) {
    return THREADS == 32 ? (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5) : blockIdx.x / size;
}

// dx_j = g [j = y] - 2^d_j (ka + kb d_j) with d_j = (x_j - base) c - off, so that 2^d_j is p_j or
// a multiple of it that ka and kb make up for.
struct GradRow {
    float g, ka, kb, base, off;
};

// One element, in the very operations of GradVector: the bits do not depend on alignment. CLAMP:
// the row may hold -inf, whose term 2^d (ka + kb d) is 0 times -inf.
template <bool H, bool CLAMP = H>
__device__ __forceinline__ float grad_term(const GradRow& r, float x, float c, bool target) {
    const float d = fmaf(x - r.base, c, -r.off);
    const float f = __fmul_rn(pow2(d), H ? fmaf(-r.kb, CLAMP ? fmaxf(d, kFar) : d, -r.ka) : -r.ka);
    return target ? __fadd_rn(f, r.g) : f;
}

// The same for 16 bytes of a row that do not hold the target, or before it is set right.
template <class T, bool H, bool CLAMP = H>
struct GradVector {
    const uint64_t base, c, off, ka, kb;  // twice each

    __device__ __forceinline__ GradVector(const GradRow& r, float c)
        : base(pack2(-r.base, -r.base)), c(pack2(c, c)), off(pack2(-r.off, -r.off)), ka(pack2(-r.ka, -r.ka)), kb(pack2(-r.kb, -r.kb)) {}

    __device__ __forceinline__ uint4 operator()(const uint4& x) const {
        uint4 out;
#pragma unroll
        for (int i = 0; i < kVec<T> / 2; ++i) {
            const uint64_t d = fma2(add2(widen2<T>(x, i), base), c, off);
            const float2 df = unpack2(d);
            const uint64_t e = pack2(pow2(df.x), pow2(df.y));
            const uint64_t b = CLAMP ? pack2(fmaxf(df.x, kFar), fmaxf(df.y, kFar)) : d;
            narrow2<T>(out, i, unpack2(mul2(e, H ? fma2(kb, b, ka) : ka)));
        }
        return out;
    }
};

// Zeros into this CTA's share of a row.
template <class T, int THREADS>
__device__ __forceinline__ void zero_row(T* out, int64_t vocab, int rank, int size) {
    const Slice<T> s(out, vocab, rank, size);
    const int id = place_in_group<THREADS>();
    uint4* v = const_cast<uint4*>(s.v);
    for (int i = id; i < s.n; i += THREADS) __stcs(v + i, make_uint4(0, 0, 0, 0));
    if (id < s.head) out[id] = narrow<T>(0.0f);
    if (id < s.tail) out[s.tail_at + id] = narrow<T>(0.0f);
}

template <class T>
__device__ __forceinline__ bool same_alignment(const T* a, const T* b) {
    return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

__device__ __forceinline__ int64_t clamp_offset(int64_t o, int64_t lo, int64_t hi) {
    return o < lo ? lo : (o > hi ? hi : o);
}

// ---- one pass over rows that stay in shared memory ------------------------------------------
// What kernels share that bring a row's slice to shared memory by bulk copies, sum over it as it arrives,
// and read it again for the gradient, while a producer warp brings the next row in behind it.
constexpr int kChunks = 2, kSlots = 8;  // parts of a slice; most parts that shared memory holds
// Computing warps of a CTA, and how many CTAs an SM then holds, by registers and shared memory.
constexpr int kFusedWarps = 7, kFusedWarpsSmall = 3;
constexpr int fused_ctas(int warps) { return warps == kFusedWarps ? 2 : 4; }
constexpr int64_t fused_room(int warps) { return warps == kFusedWarps ? 110 * 1024 : 54 * 1024; }

template <int THREADS>
__device__ __forceinline__ void consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// Place and phase in a ring of a number of slots.
struct Slot {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int slots) {
        if (++at == slots) {
            at = 0;
            phase ^= 1;
        }
    }
};

// The weights of a batch's tokens in a loss that is a weighted sum over them.
struct TokenWeights {
    const int64_t* targets;
    const int64_t* offsets;  // sequences, or nullptr
    float* w;                // [rows] 0: no loss
    float* loss;             // [rows] weighted
    uint32_t* of;            // [rows] a sequence's targets, at its first token
    uint32_t* ticket;        // the next row of a kernel that hands rows out
    int64_t rows, seqs;
    int32_t reduce;
};

// The kernels over tokens alone: one cluster of token_ctas(rows) CTAs.
constexpr int kSetupThreads = 1024;

// The sequence that token t lies in, -1 in front of the first, `seqs` behind the last: the last one
// that begins at or before it.
__device__ __forceinline__ int64_t sequence_of(const int64_t* offsets, int64_t seqs, int64_t t) {
    int64_t lo = 0, hi = seqs + 1;  // offsets below lo are at most t, those from hi on are more
    while (lo < hi) {
        const int64_t mid = lo + (hi - lo) / 2;
        if (offsets[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo - 1;
}

// Weights of all tokens, and what else the loss spreads over them: targets are counted, in all and by sequence, then spread. A
// thread finds its token's sequence by bisection, so that one sequence of all tokens takes no longer
// than many: 32768 tokens in one sequence took a warp of its own 700 us.
template <class A>
__global__ void __launch_bounds__(kSetupThreads) k_token_setup(const A a) {
    __shared__ uint32_t counted[2], all[2];  // tokens with a target, sequences that have one: added up in the first CTA's; everyone's copy
    const cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31;
    const int64_t first = (int64_t)blockIdx.x * kSetupThreads + threadIdx.x, step = (int64_t)gridDim.x * kSetupThreads;
    const bool by_sequence = a.reduce == ZERO_REDUCE_SEQUENCE;
    uint32_t* of = a.of;
    wait_for_kernel_before();
    let_next_kernel_start();
    if (threadIdx.x < 2) counted[threadIdx.x] = 0;
    if (first == 0) *a.ticket = 0;
    if (by_sequence)
        for (int64_t t = first; t < a.rows; t += step) of[t] = 0;
    cl.sync();
    uint32_t* sums = cl.map_shared_rank(counted, 0);
    uint32_t targets = 0, filled = 0;
    for (int64_t t0 = first - lane; t0 < a.rows; t0 += step) {
        const int64_t t = t0 + lane;
        const bool target = t < a.rows && a.targets[t] >= 0;
        const int64_t s = a.offsets && target ? sequence_of(a.offsets, a.seqs, t) : 0;
        const bool live = target && (!a.offsets || (s >= 0 && s < a.seqs));
        targets += live;
        const unsigned lives = __ballot_sync(~0u, live);
        if (!by_sequence || !lives) continue;
        // a warp's tokens are most often of one sequence
        const int64_t b = live ? clamp_offset(a.offsets[s], 0, a.rows - 1) : 0, b0 = __shfl_sync(~0u, b, __ffs(lives) - 1);
        if (__all_sync(~0u, !live || b == b0)) {
            if (lane == 0) filled += atomicAdd(of + b0, (uint32_t)__popc(lives)) == 0;
        } else if (live) {
            filled += atomicAdd(of + b, 1u) == 0;
        }
    }
    targets = __reduce_add_sync(~0u, targets);
    filled = __reduce_add_sync(~0u, filled);
    if (lane == 0 && targets) atomicAdd(sums, targets);
    if (lane == 0 && filled) atomicAdd(sums + 1, filled);
    cl.sync();
    if (threadIdx.x < 2) all[threadIdx.x] = sums[threadIdx.x];
    __syncthreads();
    const float tokens = (float)max(all[0], 1u), sequences = (float)max(all[1], 1u);
    const float same = a.reduce == ZERO_REDUCE_TOKEN ? 1.0f / tokens : 1.0f;
    for (int64_t t = first; t < a.rows; t += step) {
        const int64_t s = a.offsets ? sequence_of(a.offsets, a.seqs, t) : 0;
        if (a.offsets && (s < 0 || s >= a.seqs)) {  // in front of the first sequence or behind the last
            a.w[t] = 0.0f;
            continue;
        }
        float w = a.targets[t] >= 0 ? same : 0.0f;
        if (by_sequence && w != 0.0f) w = 1.0f / (float)__ldcg(of + clamp_offset(a.offsets[s], 0, a.rows - 1)) / sequences;
        a.w[t] = w;
        a.spread(t, s);
        a.loss[t] = NAN;  // until its row is done
    }
    cl.sync();  // no CTA leaves while another reads its sums
}

// The means, in a fixed order. A::kClips: the loss counts the tokens that it clips.
template <class A>
__global__ void __launch_bounds__(kSetupThreads) k_token_finish(const A a) {
    __shared__ Sum sm[kSetupThreads / 32];
    __shared__ struct {
        float loss[2], kl[2];
        uint32_t targets, clipped;
    } mine;
    const cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x == 0) mine.targets = mine.clipped = 0;
    wait_for_kernel_before();
    Sum loss, kl;
    uint32_t clipped = 0, n = 0;
#pragma unroll 4
    for (int64_t t = (int64_t)blockIdx.x * kSetupThreads + threadIdx.x; t < a.rows; t += (int64_t)gridDim.x * kSetupThreads) {
        loss.add(a.w[t] != 0.0f ? a.loss[t] : 0.0f);
        kl.add(a.kl[t]);
        if (A::kClips) clipped += a.clipped[t] != 0.0f;
        n += a.w[t] != 0.0f;
    }
    loss = cta_sum<kSetupThreads>(loss, sm);
    kl = cta_sum<kSetupThreads>(kl, sm);
    clipped = __reduce_add_sync(~0u, clipped);
    n = __reduce_add_sync(~0u, n);
    if ((threadIdx.x & 31) == 0) {
        atomicAdd(&mine.targets, n);
        atomicAdd(&mine.clipped, clipped);
    }
    if (threadIdx.x == 0) {
        mine.loss[0] = loss.hi;
        mine.loss[1] = loss.lo;
        mine.kl[0] = kl.hi;
        mine.kl[1] = kl.lo;
    }
    cl.sync();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        n = mine.targets;
        clipped = mine.clipped;
#pragma unroll 1
        for (unsigned i = 1; i < gridDim.x; ++i) {
            const auto* other = cl.map_shared_rank(&mine, i);
            loss.add(Sum{other->loss[0], other->loss[1]});
            kl.add(Sum{other->kl[0], other->kl[1]});
            n += other->targets;
            clipped += other->clipped;
        }
        const double tokens = n ? (double)n : 1.0;
        *a.out_loss = (float)loss.value();
        *a.out_kl = (float)(kl.value() / tokens);
        if (A::kClips) *a.out_clip = (float)((double)clipped / tokens);
    }
    cl.sync();  // no CTA leaves while the first reads its sums
}

// ---------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------
inline int check_logits(const zero_logits* x) {
    if (!x || x->rows < 0 || x->rows > INT32_MAX || x->vocab < 1 || x->vocab > (1 << 30) || x->stride < x->vocab || !type_ok(x->type)) return ZERO_ERR_INVALID_ARG;
    if (!temperature_ok(x->temperature)) return ZERO_ERR_INVALID_ARG;
    if (x->rows > 0 && x->stride > INT64_MAX / 8 / x->rows) return ZERO_ERR_INVALID_ARG;
    return ZERO_OK;
}

inline void need_logits(CallDevice& d, const zero_logits* x) {
    d.need(x->logits, type_size(x->type));
    d.need(x->targets, 8);
}

template <class T>
Rows<T> rows_of(const zero_logits* x, const float* weight) {
    Rows<T> a;
    a.x = (const T*)x->logits;
    a.targets = x->targets;
    a.weight = weight;
    a.rows = x->rows;
    a.vocab = x->vocab;
    a.stride = x->stride;
    a.k = make_scale(x->temperature);
    a.c = (float)(1.4426950408889634 / x->temperature);
    a.inv_t = 1.0 / x->temperature;
    return a;
}

template <class F>
int by_type(int32_t type, F f) {
    if (type == ZERO_T_BF16) return f(__nv_bfloat16());
    if (type == ZERO_T_FP16) return f(__half());
    return f(float());
}

// CTAs per row: 1 where the rows fill the GPU, else the row is cut (into at most 8, of 4 KB at
// least), while every SM has at most `per_sm`.
inline int ctas_per_row(const zero_logits* x, int sms, int per_sm = kRowCtas) {
    int size = 1;
    while (size < 8 && 2 * size * x->rows <= per_sm * (int64_t)sms && x->vocab * type_size(x->type) / (2 * size) >= 4096) size *= 2;
    return size;
}

// How the one-pass kernel takes a row.
struct FusedPlan {
    int size = 0;      // CTAs per row; 0: two passes over the row instead
    int warps = 0;
    int part = 0;      // vectors of one part of a CTA's slice
    int slots = 0;     // parts in shared memory: with more than a row's, the next row's copies begin earlier
};

// CTAs per row as ctas_per_row for few rows, else one, or two where a slice would not fit: four CTAs
// per row wait for each other longer than a second pass takes (2709 rows of 151936 bf16: 414 us
// against 347). Rows of half the room go to smaller CTAs, twice as many.
// `reserve`: bytes of shared memory that a kernel needs beside the slices; `spare`: what its larger CTAs may take over the room.
inline FusedPlan fused_plan(const zero_logits* x, int sms, int64_t reserve = 0, int64_t spare = 0) {
    FusedPlan f;
    const int64_t vecs = x->vocab * type_size(x->type) / 16;
    const int few = ctas_per_row(x, sms, 2);
    for (int size = few; size <= std::max(few, 2); size *= 2) {
        const int64_t part = std::max<int64_t>(1, ((vecs + size - 1) / size + kChunks - 1) / kChunks);
        if (16 * kChunks * part > fused_room(kFusedWarps) + spare - reserve) continue;
        f.size = size;
        f.warps = size == 1 && 16 * kChunks * part <= fused_room(kFusedWarpsSmall) - reserve ? kFusedWarpsSmall : kFusedWarps;
        f.part = (int)part;
        f.slots = (int)std::min<int64_t>(kSlots, (fused_room(f.warps) + (f.warps == kFusedWarps ? spare : 0) - reserve) / (16 * part));
        return f;
    }
    return f;
}

// CTAs of the kernels over tokens alone: a cluster of eight begins 3 us later than one CTA, which
// it has made up at 2048 tokens (4096 of 50257 in 123 us against 129).
inline int token_ctas(int64_t rows) { return rows <= 2048 ? 1 : 8; }

inline int check_dlogits(const zero_logits* x, const void* dx, int64_t dstride) {
    if (dstride < x->vocab || (x->rows > 0 && dstride > INT64_MAX / 8 / x->rows)) return ZERO_ERR_INVALID_ARG;
    if (dx == x->logits && x->rows > 0 && dstride != x->stride) return ZERO_ERR_INVALID_ARG;
    return ZERO_OK;
}

inline int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

}  // namespace
}  // namespace zg
