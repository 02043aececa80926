// zero_logits.cu -- token log-probabilities over a vocabulary and their gradient, and the
// preference and policy losses on them, for sm_103a.
//
// All of it is bound by reading and writing [rows, vocab] logits; the arithmetic on them is a
// softmax, so every row is read with its sums carried along (zero_softmax.cuh). An element costs
// about six instructions forward and six back, the most of them two to an instruction, which
// leaves an SM's issue slots half free at HBM's rate. Figures below: one GB300, HBM copy peak
// 6,673 GB/s, a vocabulary of 50257 (rows at any even address), calls replayed from a graph.

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "zero_rows.cuh"

namespace zg {
namespace {

// Whether a row is taken without CHECKED (Sums) first: its target's logit is a base, and a vocabulary
// padded with -inf or the type's lowest value, at its end or start, does not make an entropy's sum
// fail anyway. -inf elsewhere in the vocabulary shows in the sum only, and the row is then taken twice:
// with an entropy, 4096 x 50257 bf16 token_logp 65 us without a mask, 70 with one at the end, 122 with one
// in the middle, policy_loss 140, 160 and 212; 8192 x 4000 token_logp 16, 19 and 26, policy_loss 34, 37 and
// 45. A function of the row alone, so that its bits are too.
template <bool ENTROPY, class T>
__device__ __forceinline__ bool fast_row(const T* x, int64_t vocab, float x_y, Scale k) {
    if (ENTROPY && fminf(widen(x[0]) - x_y, widen(x[vocab - 1]) - x_y) * k.c == -INFINITY) return false;
    return fabsf(x_y) < INFINITY;
}

// The sums of a row, or of a CTA's share of it, by the THREADS that take it: a CTA's (joined through
// sm, THREADS / 32 entries), or one warp's, which takes the whole row and needs no sm. WRITTEN: the
// kernel writes the row afterwards (a gradient in place), so not through the read-only path.
template <int THREADS, bool ENTROPY, bool WRITTEN, class T>
__device__ __forceinline__ RowStat row_sums(const T* x, int64_t vocab, int64_t y, float* x_target, Scale k, int rank, int size, RowStat* sm) {
    const Slice<T> s(x, vocab, rank, size);
    const int id = place_in_group<THREADS>();
    auto load = [&](int i) { return WRITTEN ? s.v[i] : THREADS == 32 ? __ldg(s.v + i) : load_once(s.v + i); };
    const RowStart<T, THREADS> start(s, x, load);
    const float x_y = *x_target = y < vocab ? widen(x[y]) : NAN;
    auto sums = [&](auto checked) {
        constexpr bool kChecked = decltype(checked)::value;
        Sums<T, ENTROPY, kChecked> run(k, x_y);
        auto use = [&](int, const uint4& q) { run.add(q); };
        if (kChecked) for_vectors<THREADS>(s.n, load, use);
        else start.vectors(s.n, load, use);
        if (id < s.head) run.add_one(widen(start.head));
        if (id < s.tail) run.add_one(widen(start.tail));
        if constexpr (THREADS == 32) return warp_join<ENTROPY, kChecked>(run.stat(), k);
        else return group_join<ENTROPY, kChecked, THREADS / 32>(run.stat(), k, sm, 0);
    };
    if (fast_row<ENTROPY>(x, vocab, x_y, k)) {
        const RowStat st = sums(std::false_type());
        if (good_sums<ENTROPY>(st)) return st;
        if (THREADS > 32) __syncthreads();
    }
    return sums(std::true_type());
}

// Forward, bound by reading the logits once: `size` CTAs per row (a cluster; several where there
// are few rows), each thread kUnroll vectors at a time. 4096 fp16 tokens, a quarter of them masked:
// 50.4 us, 309 MB, 92% of the copy peak (128 or 512 threads and 2 or 6 vectors lie within 5%); one
// token 3.3 us, over eight CTAs. Rows of up to kShortRowRead bytes go to a warp each: a CTA's joining
// would take longer than their reading.
template <class T, bool ENTROPY, int THREADS>
__global__ void __launch_bounds__(kRowThreads, 5)
    k_token_logp(const Rows<T> a, int size, float* logp, float* lse, float* entropy, float* low, float* cleared, uint32_t* counter) {
    __shared__ RowStat sm[kRowThreads / 32], mine;
    wait_for_kernel_before();
    let_next_kernel_start();
    const int64_t t = row_of<THREADS>(size);
    if (THREADS == 32 && t >= a.rows) return;
    const int rank = THREADS == 32 ? 0 : (int)(blockIdx.x % size);
    const int64_t y = live_target(a, t);
    RowResult r = {0.0f, 0.0f, 0.0f, 0.0f};
    const bool first = place_in_group<THREADS>() == 0 && rank == 0;
    if (y >= 0) {
        const T* x = a.x + t * a.stride;
        float x_y;
        RowStat st = row_sums<THREADS, ENTROPY, false>(x, a.vocab, y, &x_y, a.k, rank, size, sm);
        if (THREADS != 32) st = cluster_join<ENTROPY>(st, size, a.k, &mine);
        if (first) {
            r = finish_row<ENTROPY>(st, x_y, a.k, (float)a.inv_t);
            if (y >= a.vocab) r.logp = NAN;
        }
    }
    if (first) {
        logp[t] = r.logp;
        lse[t] = r.lse;
        if (ENTROPY) entropy[t] = r.entropy;
        if (low) low[t] = r.low;
        if (cleared) cleared[t] = 0.0f;
        if (counter && t == 0) *counter = 0;
    }
    if (THREADS != 32 && size > 1 && y >= 0) cg::this_cluster().sync();  // no CTA leaves while another reads its sums
}

// From what zero_token_logp gave. log p is rebuilt from whichever is the smaller number and so
// the more exact in fp32: the target's log-probability (base = its logit) or lse.
__device__ __forceinline__ GradRow grad_row(float g, float h, float x_y, float logp, float lse, float entropy, double inv_t) {
    GradRow r;
    const float i = (float)inv_t;
    if (fabsf(logp) <= fabsf(lse)) {
        r.base = x_y;
        r.off = -logp * kLog2e;
    } else {
        r.base = lse / i;
        r.off = (float)(((double)lse - (double)r.base * inv_t) * 1.4426950408889634);
    }
    r.g = g * i;
    r.ka = i * (h == 0.0f ? g : fmaf(h, entropy, g));
    r.kb = i * h * kLn2;
    return r;
}

// From a row's sums: 2^d_j = s p_j, and log p_j = (d_j - log2 s) ln 2.
__device__ __forceinline__ GradRow grad_row(float g, float h, const RowStat& a, float entropy, double inv_t) {
    const float i = (float)inv_t, f = i / a.s;
    return {g * i, f * (h == 0.0f ? g : fmaf(h, entropy - log2f(a.s) * kLn2, g)), f * h * kLn2, base_of(a.m), 0.0f};
}

// The target's place in a row that has it, or a place that no slice reaches.
__device__ __forceinline__ int place_of(int64_t y, int64_t vocab) { return y < vocab ? (int)y : -1; }

// The elements of a row that no vector holds.
template <class T, bool H, bool CLAMP = H>
__device__ __forceinline__ void write_ends(const Slice<T>& s, const GradRow& r, int i, float x_head, float x_tail, T* out, float c, int y) {
    if (i < s.head) out[i] = narrow<T>(grad_term<H, CLAMP>(r, x_head, c, i == y));
    if (i < s.tail) out[s.tail_at + i] = narrow<T>(grad_term<H, CLAMP>(r, x_tail, c, s.tail_at + i == y));
}

// Backward, bound by reading the logits and writing their gradient: 2048 bf16 rows in 63.5 us, 412
// MB, 97% of the copy peak (8192 in 245 us, 101%). Where the gradient's rows have another alignment than the logits',
// elements are taken one at a time.
template <int THREADS, bool H, class T, class L>
__device__ __forceinline__ void write_grad(float c, const GradRow& r, const Slice<T>& s, const RowStart<T, THREADS>& start, const T* x, T* out, L load,
                                           int y, float x_y) {
    const int id = place_in_group<THREADS>();
    if (same_alignment(x, out)) {
        const GradVector<T, H> grad(r, c);
        uint4* to = reinterpret_cast<uint4*>(out + s.first);
        start.vectors(s.n, load, [&](int i, const uint4& q) { __stcs(to + i, grad(q)); });
        // the thread that wrote the target's vector sets the target right
        const int at = y - s.first;
        if (at >= 0 && at < s.n * kVec<T> && at / kVec<T> % THREADS == id) out[y] = narrow<T>(grad_term<H>(r, x_y, c, true));
    } else {
        for (int j = s.first + id; j < s.first + s.n * kVec<T>; j += THREADS)
            out[j] = narrow<T>(grad_term<H>(r, widen(x[j]), c, j == y));
    }
    write_ends<T, H>(s, r, id, id < s.head ? widen(start.head) : 0.0f, id < s.tail ? widen(start.tail) : 0.0f, out, c, y);
}

// The CTAs of an SM are bounded for fp32, whose rows bring few bytes per register: 40 registers for a
// CTA's rows are 174 us for 2039 of 50257 with their forward pass, 32 are 171; 16-bit rows are the
// faster with all that the compiler takes.
template <class T, bool H, int THREADS>
__global__ void __launch_bounds__(kRowThreads, sizeof(T) == 4 ? (THREADS == 32 ? 5 : 8) : 1)
    k_token_grad(const Rows<T> a, int size, const float* logp, const float* lse, const float* entropy, const float* dlogp,
                 const float* dentropy, T* dx, int64_t dstride) {
    wait_for_kernel_before();
    let_next_kernel_start();
    // From the last row: what a forward pass read last may still be in L2.
    const int64_t t = a.rows - 1 - row_of<THREADS>(size);
    if (THREADS == 32 && t < 0) return;
    const int rank = THREADS == 32 ? 0 : (int)(blockIdx.x % size);
    const int64_t y = live_target(a, t);
    const float row_logp = logp[t], row_lse = lse[t], row_entropy = H ? entropy[t] : 0.0f, row_g = dlogp[t], row_h = H ? dentropy[t] : 0.0f;
    const float g = y < 0 ? 0.0f : row_g, h = y < 0 ? 0.0f : row_h;
    T* out = dx + t * dstride;
    if ((g == 0.0f && h == 0.0f) || row_lse == -INFINITY) {
        zero_row<T, THREADS>(out, a.vocab, rank, size);
        return;
    }
    const T* x = a.x + t * a.stride;
    const Slice<T> s(x, a.vocab, rank, size);
    auto load = [&](int i) { return __ldcs(s.v + i); };
    const RowStart<T, THREADS> start(s, x, load);
    const float x_y = y < a.vocab ? widen(x[y]) : NAN;
    const GradRow r = grad_row(y < a.vocab ? g : NAN, h, x_y, row_logp, row_lse, h != 0.0f ? row_entropy : 0.0f, a.inv_t);
    if (out == x) {  // the target's logit is read before any thread writes it
        if (THREADS == 32) __syncwarp();
        else if (size > 1) cg::this_cluster().sync();
        else __syncthreads();
    }
    write_grad<THREADS, H>(a.c, r, s, start, x, out, load, place_of(y, a.vocab), x_y);
}

// ---------------------------------------------------------------------------------------
// Preference loss, between the forward kernel and the gradient's: a CTA per pair sums its two
// sequences and spreads the gradient over their tokens. g holds 0 for the tokens of no pair
// (written before). Sequences sum what their log-probabilities were before they were rounded to
// fp32 (low): a reward is the small difference of such sums, and 100 roundings of numbers near 10
// are 3e-6 of it. The loss of a pair needs all of its rows, so the logits are read twice: 8192
// tokens in 16 pairs, a quarter masked, take 320 us, 96% of the copy peak on their 2.06 GB. One
// kernel that follows each pair's forward rows with its gradient rows, to read them from L2, took
// 450 us and more: the L2 gave back 6%, handing out rows cost 20%.
// ---------------------------------------------------------------------------------------
struct PairArgs {
    const int64_t* targets;
    const int64_t* offsets;
    const float *logp, *low;
    const float* ref;
    float* g;
    float *pair_loss, *chosen, *rejected, *loss;
    uint32_t* done;  // CTAs that have ended; 0 before
    int64_t rows, pairs;
    double beta, half_over_beta, smoothing;
    int32_t kind, average;
};

// log(1 + e^x) without overflow; a NaN stays
__device__ __forceinline__ float softplus(float x) { return (x < 0.0f ? 0.0f : x) + log1pf(expf(-fabsf(x))); }

__global__ void __launch_bounds__(kRowThreads) k_pairs(const PairArgs a) {
    constexpr int kWarps = kRowThreads / 32, kHalf = kRowThreads / 2;  // half of the CTA per sequence
    __shared__ Sum sm[kWarps];
    __shared__ int counts[kWarps];
    __shared__ float g_side[2];
    let_next_kernel_start();
    wait_for_kernel_before();
    const int warp = threadIdx.x >> 5, side = threadIdx.x / kHalf, id = threadIdx.x % kHalf;
    for (int64_t i = blockIdx.x; i < a.pairs; i += gridDim.x) {
        const int64_t lo = clamp_offset(a.offsets[2 * i + side], 0, a.rows), hi = clamp_offset(a.offsets[2 * i + side + 1], lo, a.rows);
        Sum sum;
        int targets = 0;
#pragma unroll 4
        for (int64_t t = lo + id; t < hi; t += kHalf) {
            const float lp = a.logp[t], low = a.low[t], ref = a.ref ? a.ref[t] : 0.0f;
            if (a.targets[t] < 0) continue;
            sum.add(lp);
            sum.lo += low;
            if (a.ref) sum.add(-ref);
            ++targets;
        }
        sum = warp_sum(sum);
        targets = __reduce_add_sync(~0u, targets);
        if ((threadIdx.x & 31) == 0) {
            sm[warp] = sum;
            counts[warp] = targets;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            double d[2];
            float n[2];
            for (int k = 0; k < 2; ++k) {
                Sum all = sm[k * kWarps / 2];
                int count = counts[k * kWarps / 2];
                for (int w = 1; w < kWarps / 2; ++w) {
                    all.add(sm[k * kWarps / 2 + w]);
                    count += counts[k * kWarps / 2 + w];
                }
                n[k] = a.average && count ? (float)count : 1.0f;
                d[k] = all.value();
                if (a.average && count) d[k] /= (double)count;
            }
            // the margin in fp64 (it may cancel), what follows from it in fp32
            const double m = d[0] - d[1];
            const float b = (float)a.beta, e = (float)a.smoothing, s = (float)(a.beta * m);
            float loss, dm;
            if (a.kind == ZERO_PREF_SIGMOID) {
                loss = (1.0f - e) * softplus(-s);
                if (e != 0.0f) loss += e * softplus(s);  // not 0 times an infinite margin
                // sigmoid(s) - (1 - e), each half formed without cancellation
                dm = b * (e / (1.0f + expf(-s)) - (1.0f - e) / (1.0f + expf(s)));
            } else if (a.kind == ZERO_PREF_HINGE) {
                const float gap = (float)(1.0 - a.beta * m);
                loss = gap > 0.0f || gap != gap ? gap : 0.0f;
                dm = gap > 0.0f ? -b : gap == gap ? 0.0f : gap;
            } else {
                const float gap = (float)(m - a.half_over_beta);
                loss = gap * gap;
                dm = 2.0f * gap;
            }
            a.pair_loss[i] = loss;
            a.chosen[i] = (float)(a.beta * d[0]);
            a.rejected[i] = (float)(a.beta * d[1]);
            g_side[0] = dm / (n[0] * (float)a.pairs);
            g_side[1] = -dm / (n[1] * (float)a.pairs);
        }
        __syncthreads();
        for (int64_t t = lo + id; t < hi; t += kHalf) a.g[t] = g_side[side];
        __syncthreads();
    }
    // the CTA that ends last takes the mean, in the pairs' order
    __shared__ bool last;
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(a.done, 1u) == gridDim.x - 1;
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
    Sum s;
    for (int64_t i = threadIdx.x; i < a.pairs; i += kRowThreads) s.add(__ldcg(a.pair_loss + i));
    s = cta_sum<kRowThreads>(s, sm);
    if (threadIdx.x == 0) *a.loss = (float)(s.value() / (double)a.pairs);
}

// ---------------------------------------------------------------------------------------
// Policy loss.
// ---------------------------------------------------------------------------------------
// What a token's loss needs beside its row: its weight (0: no loss) and its advantage.
struct PolicyTokens : TokenWeights {
    static constexpr bool kClips = true;
    const float* advantages;
    const float *old_logp, *ref_logp;
    float* adv;            // [rows]
    float *lse, *g, *h;    // [rows]
    float *kl, *clipped;   // [rows]
    float *out_loss, *out_clip, *out_kl;
    float lo, hi, dual, kl_coef, entropy_coef;
    int32_t kl_kind, per_sequence;

    __device__ __forceinline__ void spread(int64_t t, int64_t s) const { adv[t] = advantages[per_sequence ? s : t]; }
};

// What a token's loss takes, read ahead of its row's sums.
struct TokenIn {
    float w, adv, old, ref;
    __device__ __forceinline__ TokenIn(const PolicyTokens& a, int64_t t)
        : w(a.w[t]), adv(a.adv[t]), old(a.old_logp ? a.old_logp[t] : 0.0f), ref(a.ref_logp ? a.ref_logp[t] : 0.0f) {}
};

struct TokenLoss {
    float loss, kl, clipped, g, h;  // loss and the gradients on logp and entropy, weighted
};

__device__ __forceinline__ TokenLoss policy_token(const PolicyTokens& a, const TokenIn& in, float logp, float entropy) {
    TokenLoss r;
    // without old_logp the ratio is 1, of a log-probability of -inf too; a NaN stays
    const float w = in.w, A = in.adv, ratio = a.old_logp ? expf(logp - in.old) : logp == logp ? 1.0f : logp;
    // a ratio past fp32 times an advantage of 0 is 0
    const float plain = A == 0.0f && ratio == INFINITY ? 0.0f : -ratio * A, clip = -fminf(fmaxf(ratio, a.lo), a.hi) * A;
    float loss = !(plain < clip) ? plain : clip;  // a NaN stays
    bool off = (A > 0.0f && ratio > a.hi) || (A < 0.0f && ratio < a.lo);
    if (a.dual > 0.0f && A < 0.0f && ratio > a.dual) {
        off = true;
        loss = -a.dual * A;
    }
    float g = off ? 0.0f : plain;
    r.kl = 0.0f;
    if (a.ref_logp) {
        const float d = in.ref - logp;
        float dkl;
        if (a.kl_kind == ZERO_KL_K1) {
            r.kl = -d;
            dkl = 1.0f;
        } else if (a.kl_kind == ZERO_KL_K2) {
            r.kl = 0.5f * d * d;
            dkl = -d;
        } else {
            const float e = expm1f(d);
            r.kl = e < INFINITY ? e - d : e;  // not inf - inf where the target has no probability
            dkl = -e;
        }
        if (a.kl_coef != 0.0f) {
            loss = fmaf(a.kl_coef, r.kl, loss);
            g = fmaf(a.kl_coef, dkl, g);
        }
    }
    if (a.entropy_coef != 0.0f) loss = fmaf(-a.entropy_coef, entropy, loss);
    r.loss = loss * w;
    r.clipped = off ? 1.0f : 0.0f;
    r.g = g * w;
    r.h = -a.entropy_coef * w;
    return r;
}

// Forward and backward in one pass over each row: its slice is brought to shared memory by bulk
// copies, read for the sums as it arrives, joined over the cluster, and read again for the
// gradient. So the logits cross HBM once each way, where a second pass over them would read them
// again. Two CTAs per SM, each with one slice: a producer warp refills a part of it with the next
// row as soon as the gradient of this one has been taken from it, so that copies run beside
// everything else. Rows are handed out one by one (some carry no loss and cost half). 8192 bf16
// tokens, a quarter masked, with entropy bonus: 232 us the whole call, 1.44 GB, 93% of the copy peak
// (two passes over the logits: 383 us). Seven warps compute: with ten, and four parts to a slice,
// 252 us, since registers then spill; with fifteen 325.
// H: entropies are formed, for the loss or only for the caller, who may want them beside a coefficient
// of 0.
template <class T, bool H, int WARPS>
__global__ void __launch_bounds__(32 * WARPS + 32, fused_ctas(WARPS))
    k_policy_rows(const Rows<T> a, const PolicyTokens p, int size, int per, int slots, float* logp, float* entropy, T* dx, int64_t dstride) {
    constexpr int kThreads = 32 * WARPS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ RowStat sm[WARPS], mine[2];
    __shared__ GradRow shared_row;
    __shared__ bool shared_zero;
    __shared__ int64_t row_at[2], row_y[2];
    __shared__ float row_x[2];  // the target's logit
    __shared__ bool row_fast[2];
    __shared__ uint64_t bars[2 * kSlots + 4];
    __shared__ int gave_up;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kSlots, row_full = empty + 8 * kSlots, row_empty = row_full + 16;
    const int rank = (int)(blockIdx.x % size), lane = threadIdx.x & 31;
    const int64_t first = blockIdx.x / size, clusters = gridDim.x / size;
    if (threadIdx.x == 0) {
        gave_up = 0;
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
    __syncthreads();

    // The kernel before this one sets up the weights; it lets this one start once it has waited for
    // the logits' producer, so logits and targets may be read at once, and the rest after it.
    let_next_kernel_start();
    int64_t n = 0;  // rows taken
    if (threadIdx.x >= kThreads) {
        Slot slot;
        bool ok = true;
        for (;; ++n) {
            int64_t t = first + n * clusters;
            if (size == 1 && n > 0) {
                if (n == 1) wait_for_kernel_before();
                if (lane == 0) t = (int64_t)gridDim.x + (int64_t)atomicAdd(p.ticket, 1u);
                t = __shfl_sync(~0u, t, 0);
            }
            if (t >= a.rows) t = -1;
            ok = ok && mbar_wait(row_empty + 8 * (n & 1), ((uint32_t)(n >> 1) & 1) ^ 1, &gave_up);
            ok = __all_sync(~0u, ok);
            if (!ok) t = -1;
            const int64_t y = t >= 0 ? a.targets[t] : -1;
            const T* x = a.x + t * a.stride;
            if (lane == 0) {
                row_at[n & 1] = t;
                row_y[n & 1] = y;
                const float x_y = y >= 0 && y < a.vocab ? widen(x[y]) : NAN;
                row_x[n & 1] = x_y;
                row_fast[n & 1] = y >= 0 && fast_row<H>(x, a.vocab, x_y, a.k);
                mbar_arrive(row_full + 8 * (n & 1));
            }
            if (t < 0) break;
            if (y < 0) continue;
            if (lane == 0) {
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
            if (size > 1) cg::this_cluster().sync();  // the consumers' cluster_join
        }
    } else {
        uint32_t taken = 0;
        Slot begin;  // of the row at hand
        const uint4* parts = reinterpret_cast<const uint4*>(smem);
        for (;; ++n) {
            // Not left early where another wait gave up: the producer announces an end even then, and
            // all warps have to take the same rows.
            bool got = mbar_try(row_full + 8 * (n & 1), (uint32_t)(n >> 1) & 1);
            for (int i = 0; i < 4 * kWaitLimit && !got; ++i) got = mbar_try(row_full + 8 * (n & 1), (uint32_t)(n >> 1) & 1);
            const int64_t t = got ? row_at[n & 1] : -1, y = row_y[n & 1];
            const float x_y = row_x[n & 1];
            const bool try_fast = row_fast[n & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(row_empty + 8 * (n & 1));
            if (t < 0) break;
            T* out = dx + t * dstride;
            if (n == 0) wait_for_kernel_before();
            if (y < 0) {
                zero_row<T, kThreads>(out, a.vocab, rank, size);
                if (threadIdx.x == 0 && rank == 0) {
                    logp[t] = p.loss[t] = p.kl[t] = p.clipped[t] = 0.0f;
                    if (entropy) entropy[t] = 0.0f;
                }
                continue;
            }
            const T* x = a.x + t * a.stride;
            const Slice<T> s(x, a.vocab, rank, size);
            // read ahead: the token's numbers and the elements that no vector holds
            const TokenIn in(p, t);
            const float x_head = threadIdx.x < s.head ? widen(x[threadIdx.x]) : 0.0f;
            const float x_tail = threadIdx.x < s.tail ? widen(x[s.tail_at + threadIdx.x]) : 0.0f;
            bool ok = true;
            auto sums = [&](auto checked) {
                constexpr bool kChecked = decltype(checked)::value;
                Sums<T, H, kChecked> run(a.k, x_y);
                Slot slot = begin;
                for (int i = 0; i < kChunks; ++i, slot.next(slots)) {
                    ok = ok && mbar_wait(full + 8 * slot.at, slot.phase, &gave_up);
                    const int at = min(s.n, i * per);
                    const uint4* v = parts + slot.at * per;
                    for_vectors<kThreads>(min(s.n, at + per) - at, [&](int j) { return v[j]; }, [&](int, const uint4& q) { run.add(q); });
                }
                if (threadIdx.x < s.head) run.add_one(x_head);
                if (threadIdx.x < s.tail) run.add_one(x_tail);
                return group_join<H, kChecked, WARPS>(run.stat(), a.k, sm, 1);
            };
            RowStat st;
            bool good = false;
            if (try_fast) {
                st = sums(std::false_type());
                good = good_sums<H>(st);
                if (!good) consumers_sync<kThreads>();
            }
            if (!good) st = sums(std::true_type());
            if (!ok || *(volatile int*)&gave_up) st.s = NAN;  // a copy did not come: no result
            st = cluster_join<H>(st, size, a.k, mine + (taken & 1));
            if (threadIdx.x == 0) {
                RowResult r = {0.0f, 0.0f, 0.0f, 0.0f};
                TokenLoss l = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                if (in.w != 0.0f) {
                    r = finish_row<H>(st, x_y, a.k, (float)a.inv_t);
                    if (y >= a.vocab) r.logp = NAN;
                    l = policy_token(p, in, r.logp, r.entropy);
                }
                shared_zero = (l.g == 0.0f && l.h == 0.0f) || st.s == 0.0f;
                shared_row = grad_row(l.g, l.h, st, r.entropy, a.inv_t);
                if (rank == 0) {
                    logp[t] = r.logp;
                    if (entropy) entropy[t] = r.entropy;
                    p.loss[t] = l.loss;
                    p.kl[t] = l.kl;
                    p.clipped[t] = l.clipped;
                }
            }
            consumers_sync<kThreads>();
            const GradRow r = shared_row;
            const bool zero = shared_zero;
            const int place = place_of(y, a.vocab);
            const bool fast = same_alignment(x, out);
            const float c = H ? a.k.c : a.c;  // as in the sums
            auto write = [&](auto clamp) {
                constexpr bool kClamp = decltype(clamp)::value;
                const GradVector<T, H, kClamp> grad(r, c);
                if (zero) zero_row<T, kThreads>(out, a.vocab, rank, size);
                else write_ends<T, H, kClamp>(s, r, threadIdx.x, x_head, x_tail, out, c, place);
                for (int i = 0; i < kChunks; ++i, begin.next(slots)) {
                    const int at = min(s.n, i * per), m = min(s.n, at + per) - at;
                    const uint4* v = parts + begin.at * per;
                    const int from = s.first + at * kVec<T>;  // the chunk's first element
                    if (!zero && fast) {
                        uint4* to = reinterpret_cast<uint4*>(out + from);
                        for_vectors<kThreads>(m, [&](int j) { return v[j]; }, [&](int j, const uint4& q) { __stcs(to + j, grad(q)); });
                        // the thread that wrote the target's vector sets the target right
                        const int dy = place - from;
                        if (dy >= 0 && dy < m * kVec<T> && dy / kVec<T> % kThreads == threadIdx.x)
                            out[place] = narrow<T>(grad_term<H, kClamp>(r, x_y, c, true));
                    } else if (!zero) {
                        const T* e = reinterpret_cast<const T*>(v);
                        for (int j = threadIdx.x; j < m * kVec<T>; j += kThreads)
                            out[from + j] = narrow<T>(grad_term<H, kClamp>(r, widen(e[j]), c, from + j == place));
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(empty + 8 * begin.at);  // this warp has done with the part
                }
            };
            // -inf in this slice, or a base that another CTA's slice raised far above this one's values
            if (H && !(good && st.m == base_of(x_y))) write(std::true_type());
            else write(std::false_type());
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

// The same for rows of up to kShortRow bytes, a warp each, which reads its row twice, the second
// time from L1 or L2.
template <class T, bool H>
__global__ void __launch_bounds__(kRowThreads)
    k_policy_short(const Rows<T> a, const PolicyTokens p, float* logp, float* entropy, T* dx, int64_t dstride) {
    let_next_kernel_start();
    const int64_t t = row_of<32>(1);
    if (t >= a.rows) return;
    const int lane = threadIdx.x & 31;
    const int64_t y = a.targets[t];  // these and the logits may be read at once, as in k_policy_rows
    T* out = dx + t * dstride;
    const T* x = a.x + t * a.stride;
    RowResult r = {0.0f, 0.0f, 0.0f, 0.0f};
    TokenLoss l = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    RowStat st = empty_stat();
    float x_y = NAN;
    if (y >= 0) st = row_sums<32, H, true>(x, a.vocab, y, &x_y, a.k, 0, 1, nullptr);
    wait_for_kernel_before();
    const TokenIn in(p, t);
    if (in.w != 0.0f) {
        r = finish_row<H>(st, x_y, a.k, (float)a.inv_t);
        if (y >= a.vocab) r.logp = NAN;
        l = policy_token(p, in, r.logp, r.entropy);
    }
    if (lane == 0) {
        logp[t] = r.logp;
        if (entropy) entropy[t] = r.entropy;
        p.loss[t] = l.loss;
        p.kl[t] = l.kl;
        p.clipped[t] = l.clipped;
    }
    if ((l.g == 0.0f && l.h == 0.0f) || st.s == 0.0f) {
        zero_row<T, 32>(out, a.vocab, 0, 1);
        return;
    }
    const GradRow grad = grad_row(l.g, l.h, st, r.entropy, a.inv_t);
    const Slice<T> s(x, a.vocab, 0, 1);
    auto load = [&](int i) { return __ldcs(s.v + i); };
    const RowStart<T, 32> start(s, x, load);
    __syncwarp();  // the row's ends and its target are read before any lane writes
    write_grad<32, H>(H ? a.k.c : a.c, grad, s, start, x, out, load, place_of(y, a.vocab), x_y);
}

__global__ void __launch_bounds__(kRowThreads) k_policy_tokens(const PolicyTokens a, const float* logp, const float* entropy) {
    for (int64_t t = blockIdx.x * (int64_t)kRowThreads + threadIdx.x; t < a.rows; t += (int64_t)gridDim.x * kRowThreads) {
        const TokenIn in(a, t);
        TokenLoss r = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (in.w != 0.0f) r = policy_token(a, in, logp[t], entropy ? entropy[t] : 0.0f);
        a.loss[t] = r.loss;
        a.kl[t] = r.kl;
        a.clipped[t] = r.clipped;
        a.g[t] = r.g;
        a.h[t] = r.h;
    }
}

// ---------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------
// Whether each row goes to a warp: short rows, enough of them for every SM. 8192 bf16 rows, a warp each
// against a CTA each: of 16 KB 25.8 us against 30.4 forward, 57 against 63 for the policy loss, the same
// for the gradient alone; of 32 KB 45.2 against 49.6 forward, but 113 against 83 for the policy loss
// and 83 against 78 for the gradient; of 64 KB 86 against 80 forward. 2048 rows of 32 KB are the same
// either way.
constexpr int64_t kShortRow = 16384, kShortRowRead = 32768;
bool short_rows(const zero_logits* x, int sms, int64_t most = kShortRow) {
    const int64_t bytes = x->vocab * type_size(x->type);
    return bytes <= most && x->rows >= (bytes > kShortRow ? 16 : 8) * (int64_t)sms;
}
unsigned short_grid(const zero_logits* x) { return (unsigned)((x->rows + kRowThreads / 32 - 1) / (kRowThreads / 32)); }

int launch_finish(const PolicyTokens& p, cudaStream_t s) {
    return launch_linked(k_token_finish<PolicyTokens>, (unsigned)token_ctas(p.rows), kSetupThreads, 0, token_ctas(p.rows), s, p);
}

int launch_token_logp(const zero_logits* x, const float* weight, float* logp, float* lse, float* entropy, float* low,
                      float* cleared, uint32_t* counter, int sms, cudaStream_t s) {
    if (x->rows == 0) return ZERO_OK;
    return by_type(x->type, [&](auto tag) {
        using T = decltype(tag);
        const Rows<T> a = rows_of<T>(x, weight);
        if (short_rows(x, sms, kShortRowRead))
            return launch_linked(entropy ? k_token_logp<T, true, 32> : k_token_logp<T, false, 32>, short_grid(x), kRowThreads, 0, 1, s, a, 1,
                                 logp, lse, entropy, low, cleared, counter);
        const int size = ctas_per_row(x, sms);
        return launch_linked(entropy ? k_token_logp<T, true, kRowThreads> : k_token_logp<T, false, kRowThreads>, (unsigned)(x->rows * size),
                             kRowThreads, 0, size, s, a, size, logp, lse, entropy, low, cleared, counter);
    });
}

int launch_token_grad(const zero_logits* x, const float* weight, const float* logp, const float* lse, const float* entropy,
                      const float* g, const float* h, void* dx, int64_t dstride, int sms, cudaStream_t s) {
    if (x->rows == 0) return ZERO_OK;
    return by_type(x->type, [&](auto tag) {
        using T = decltype(tag);
        const Rows<T> a = rows_of<T>(x, weight);
        if (short_rows(x, sms))
            return launch_linked(h ? k_token_grad<T, true, 32> : k_token_grad<T, false, 32>, short_grid(x), kRowThreads, 0, 1, s, a, 1, logp,
                                 lse, entropy, g, h, (T*)dx, dstride);
        const int size = ctas_per_row(x, sms);
        return launch_linked(h ? k_token_grad<T, true, kRowThreads> : k_token_grad<T, false, kRowThreads>, (unsigned)(x->rows * size),
                             kRowThreads, 0, size, s, a, size, logp, lse, entropy, g, h, (T*)dx, dstride);
    });
}

template <class T, int WARPS>
int launch_fused(const zero_logits* x, const FusedPlan& f, const PolicyTokens& p, const zero_policy* q, int sms, cudaStream_t s) {
    auto* kernel = q->entropy ? k_policy_rows<T, true, WARPS> : k_policy_rows<T, false, WARPS>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)fused_room(WARPS));
    if (e != cudaSuccess) return record_cuda_error(e);
    const int64_t clusters = std::min<int64_t>(x->rows, fused_ctas(WARPS) * sms / f.size);
    return launch_linked(kernel, (unsigned)(clusters * f.size), 32 * WARPS + 32, (size_t)16 * f.slots * f.part, f.size, s, rows_of<T>(x, nullptr),
                         p, f.size, f.part, f.slots, q->logp, q->entropy, (T*)q->dlogits, q->dstride);
}

int launch_policy_rows(const zero_logits* x, const FusedPlan& f, const PolicyTokens& p, const zero_policy* q, int sms, cudaStream_t s) {
    const int rc = by_type(x->type, [&](auto tag) {
        using T = decltype(tag);
        if (short_rows(x, sms))
            return launch_linked(q->entropy ? k_policy_short<T, true> : k_policy_short<T, false>, short_grid(x), kRowThreads, 0, 1, s,
                                 rows_of<T>(x, nullptr), p, q->logp, q->entropy, (T*)q->dlogits, q->dstride);
        return f.warps == kFusedWarps ? launch_fused<T, kFusedWarps>(x, f, p, q, sms, s) : launch_fused<T, kFusedWarpsSmall>(x, f, p, q, sms, s);
    });
    if (rc) return rc;
    return launch_finish(p, s);
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" int zero_token_logp(const zero_logits* x, float* logp, float* lse, float* entropy, void* stream) {
    int rc = check_logits(x);
    if (rc || x->rows == 0) return rc;
    CallDevice d(x->logits, stream);
    need_logits(d, x);
    d.need(logp, 4);
    d.need(lse, 4);
    d.optional(entropy, 4);
    if (d.rc) return d.rc;
    return launch_token_logp(x, nullptr, logp, lse, entropy, nullptr, nullptr, nullptr, d.sm_count(), (cudaStream_t)stream);
}

extern "C" int zero_token_logp_backward(const zero_logits* x, const float* logp, const float* lse, const float* entropy,
                                        const float* dlogp, const float* dentropy, void* dlogits, int64_t dstride, void* stream) {
    int rc = check_logits(x);
    if (!rc) rc = check_dlogits(x, dlogits, dstride);
    if (!rc && dentropy && !entropy) rc = ZERO_ERR_INVALID_ARG;
    if (rc || x->rows == 0) return rc;
    CallDevice d(x->logits, stream);
    need_logits(d, x);
    d.need(logp, 4);
    d.need(lse, 4);
    d.optional(entropy, 4);
    d.need(dlogp, 4);
    d.optional(dentropy, 4);
    d.need(dlogits, type_size(x->type));
    if (d.rc) return d.rc;
    return launch_token_grad(x, nullptr, logp, lse, entropy, dlogp, dentropy, dlogits, dstride, d.sm_count(), (cudaStream_t)stream);
}

extern "C" int64_t zero_preference_workspace(int64_t rows) {
    if (rows < 0 || rows > INT64_MAX / 64) return -1;
    return 3 * 4 * round_up(rows, 4) + 64;
}

extern "C" int zero_preference_loss(const zero_logits* x, const zero_preference* p, void* workspace, int64_t workspace_bytes,
                                    void* stream) {
    int rc = check_logits(x);
    if (!rc && (!p || p->pairs < 1 || p->pairs > INT32_MAX / 2 || !(p->beta > 0.0) || !std::isfinite(p->beta) ||
                !(p->label_smoothing >= 0.0 && p->label_smoothing <= 0.5) || p->kind < ZERO_PREF_SIGMOID ||
                p->kind > ZERO_PREF_IPO || p->average < 0 || p->average > 1))
        rc = ZERO_ERR_INVALID_ARG;
    if (!rc) rc = check_dlogits(x, p->dlogits, p->dstride);
    if (rc) return rc;
    if (workspace_bytes < zero_preference_workspace(x->rows)) return ZERO_ERR_SIZE_MISMATCH;
    CallDevice d(p->loss, stream);
    if (x->rows > 0) {
        need_logits(d, x);
        d.optional(p->ref_logp, 4);
        d.need(p->logp, 4);
        d.need(p->dlogits, type_size(x->type));
    }
    d.need(p->offsets, 8);
    d.need(p->loss, 4);
    d.need(p->pair_loss, 4);
    d.need(p->chosen_reward, 4);
    d.need(p->rejected_reward, 4);
    d.need(workspace, 16);
    if (d.rc) return d.rc;
    cudaStream_t s = (cudaStream_t)stream;
    float* lse = (float*)workspace;
    float* g = lse + round_up(x->rows, 4);
    float* low = g + round_up(x->rows, 4);
    uint32_t* done = (uint32_t*)(low + round_up(x->rows, 4));
    const int sms = d.sm_count();
    const PairArgs a = {x->targets, p->offsets, p->logp, low, p->ref_logp, g, p->pair_loss, p->chosen_reward, p->rejected_reward, p->loss, done,
                        x->rows, p->pairs, p->beta, 0.5 / p->beta, p->kind == ZERO_PREF_SIGMOID ? p->label_smoothing : 0.0, p->kind, p->average};
    if (x->rows == 0) {  // no forward kernel that clears the counter
        const cudaError_t e = cudaMemsetAsync(done, 0, 4, s);
        if (e != cudaSuccess) return record_cuda_error(e);
    }
    if ((rc = launch_token_logp(x, nullptr, p->logp, lse, nullptr, low, g, done, sms, s))) return rc;
    if ((rc = launch_linked(k_pairs, (unsigned)std::min<int64_t>(p->pairs, 1 << 20), kRowThreads, 0, 1, s, a))) return rc;
    return launch_token_grad(x, nullptr, p->logp, lse, nullptr, g, nullptr, p->dlogits, p->dstride, sms, s);
}

extern "C" int64_t zero_policy_workspace(int64_t rows) {
    if (rows < 0 || rows > INT64_MAX / 64) return -1;
    return 8 * 4 * round_up(rows, 4) + 64;
}

extern "C" int zero_policy_loss(const zero_logits* x, const zero_policy* p, void* workspace, int64_t workspace_bytes, void* stream) {
    int rc = check_logits(x);
    if (!rc && (!p || !(p->clip_low >= 0.0 && p->clip_low <= 1.0) || !(p->clip_high >= 0.0) || !std::isfinite(p->clip_high) ||
                !(p->dual_clip == 0.0 || p->dual_clip > 1.0) || !std::isfinite(p->dual_clip) || !std::isfinite(p->kl_coef) ||
                !std::isfinite(p->entropy_coef) || p->kl < ZERO_KL_K1 || p->kl > ZERO_KL_K3 || p->reduce < ZERO_REDUCE_TOKEN ||
                p->reduce > ZERO_REDUCE_SUM || p->per_sequence < 0 || p->per_sequence > 1))
        rc = ZERO_ERR_INVALID_ARG;
    if (!rc && (p->offsets ? p->seqs < 0 : p->per_sequence || p->reduce == ZERO_REDUCE_SEQUENCE)) rc = ZERO_ERR_INVALID_ARG;
    if (!rc && x->rows > 0 && ((p->kl_coef != 0.0 && !p->ref_logp) || (p->entropy_coef != 0.0 && !p->entropy))) rc = ZERO_ERR_INVALID_ARG;
    if (!rc) rc = check_dlogits(x, p->dlogits, p->dstride);
    if (rc) return rc;
    if (workspace_bytes < zero_policy_workspace(x->rows)) return ZERO_ERR_SIZE_MISMATCH;
    CallDevice d(p->loss, stream);
    if (x->rows > 0) {
        need_logits(d, x);
        if (!p->per_sequence || p->seqs > 0) d.need(p->advantages, 4);
        d.optional(p->old_logp, 4);
        d.optional(p->ref_logp, 4);
        d.need(p->logp, 4);
        d.optional(p->entropy, 4);
        d.need(p->dlogits, type_size(x->type));
    }
    d.optional(p->offsets, 8);
    d.need(p->loss, 4);
    d.need(p->clip_fraction, 4);
    d.need(p->kl_mean, 4);
    d.need(workspace, 16);
    if (d.rc) return d.rc;
    cudaStream_t s = (cudaStream_t)stream;
    float* f = (float*)workspace;
    const int64_t n = round_up(x->rows, 4);
    PolicyTokens a;
    a.targets = x->targets;
    a.offsets = p->offsets;
    a.advantages = p->advantages;
    a.old_logp = p->old_logp;
    a.ref_logp = p->ref_logp;
    a.w = f;
    a.adv = f + n;
    a.lse = f + 2 * n;
    a.g = f + 3 * n;
    a.h = f + 4 * n;
    a.of = (uint32_t*)a.h;  // free until the rows
    a.loss = f + 5 * n;
    a.kl = f + 6 * n;
    a.clipped = f + 7 * n;
    a.ticket = (uint32_t*)(f + 8 * n);
    a.out_loss = p->loss;
    a.out_clip = p->clip_fraction;
    a.out_kl = p->kl_mean;
    a.rows = x->rows;
    a.seqs = p->seqs;
    a.lo = (float)(1.0 - p->clip_low);
    a.hi = (float)(1.0 + p->clip_high);
    a.dual = (float)p->dual_clip;
    a.kl_coef = (float)p->kl_coef;
    a.entropy_coef = (float)p->entropy_coef;
    a.kl_kind = p->kl;
    a.reduce = p->reduce;
    a.per_sequence = p->per_sequence;
    const int sms = d.sm_count();
    if (x->rows > 0) {
        if ((rc = launch_linked(k_token_setup<PolicyTokens>, (unsigned)token_ctas(x->rows), kSetupThreads, 0, token_ctas(x->rows), s, a))) return rc;
        const FusedPlan f = fused_plan(x, sms);
        if (f.size) return launch_policy_rows(x, f, a, p, sms, s);
        if ((rc = launch_token_logp(x, a.w, p->logp, a.lse, p->entropy, nullptr, nullptr, nullptr, sms, s))) return rc;
        k_policy_tokens<<<(int)std::min<int64_t>((x->rows + kRowThreads - 1) / kRowThreads, 1024), kRowThreads, 0, s>>>(a, p->logp, p->entropy);
        if ((rc = launched())) return rc;
        rc = launch_token_grad(x, a.w, p->logp, a.lse, p->entropy, a.g, a.entropy_coef != 0.0f ? a.h : nullptr, p->dlogits, p->dstride, sms, s);
        if (rc) return rc;
    }
    return launch_finish(a, s);
}
