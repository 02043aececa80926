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

#include <climits>

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
    float mix, kl_coef, ce_coef;
    int32_t kind, tail;

    __device__ __forceinline__ void spread(int64_t, int64_t) const {}
};

// What a CTA holds of a token's list in shared memory: the bitmap, then the entries.
struct List {
    uint32_t* bits;
    float *x, *lp;  // the student's logit, the teacher's log-probability; later x: the gradient
    int* place;     // -1: not there
    int k;

    __device__ __forceinline__ List(uint8_t* smem, int words, int k) : k(k) {
        bits = reinterpret_cast<uint32_t*>(smem);
        x = reinterpret_cast<float*>(bits + words);
        lp = x + k;
        place = reinterpret_cast<int*>(lp + k);
    }
};
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

// log s as hi + lo (finish_row's reduction), hi exact.
__device__ __forceinline__ float2 log_parts(float s) {
    constexpr float kLn2Hi = 2839.0f / 4096.0f, kLn2Lo = 3.1946184945309e-5f;
    const uint32_t bits = __float_as_uint(s);
    const bool plain = s >= 0x1p-126f && s < INFINITY;
    const float n = plain ? (float)((int)(bits >> 23) - 127) : 0.0f, f = plain ? __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u) : s;
    return make_float2(n * kLn2Hi, logf(f) + fmaf(n, kLn2Lo, kPow2Low));
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
__device__ __forceinline__ Part entry_part(int kind, float b, float p, float q, float r) {
    if (kind == ZERO_DISTILL_FORWARD) return {p > 0.0f || p != p ? p * r : 0.0f, -p};
    if (kind == ZERO_DISTILL_REVERSE) {
        const float d = q > 0.0f || q != q ? -q * r : 0.0f;
        return {d, d};
    }
    // log p - log m and log q - log m from r alone
    float pm, qm;
    if (r > 0.0f) {
        const float m = logf(fmaf(1.0f - b, expf(-r), b));
        pm = -m;
        qm = -(r + m);
    } else {
        const float m = logf(fmaf(b, expf(r), 1.0f - b));
        pm = r - m;
        qm = -m;
    }
    const float c = q > 0.0f || q != q ? (1.0f - b) * q * qm : 0.0f;
    return {(p > 0.0f || p != p ? b * p * pm : 0.0f) + c, c};
}

// A row's gradient outside its list: 2^((x_j - base) c) * factor; beside it the target's own part, and the
// target's entry where it is outside the list.
struct DistillRow {
    float base, factor;
    float target;  // the target's gradient
    bool target_listed;
};

// What the row's sums and its list come to, by one warp. rest: the sums outside the list. Writes the token's
// results (`first`: this CTA does) and the list's gradients over list.x.
__device__ __forceinline__ DistillRow finish_list(const DistillTokens& a, const List& list, const RowStat& rest, bool bad, int64_t t, int64_t y,
                                                  float x_y, int64_t vocab, Scale k, float inv_t, bool first) {
    const int lane = threadIdx.x & 31;
    const float w = a.w[t];
    // the row's maximum, and the list's sums
    float top = rest.s != 0.0f ? rest.m : -INFINITY;
    int count = 0;
    float mass = 0.0f;
    for (int i = lane; i < list.k; i += 32) {
        if (list.place[i] < 0) continue;
        ++count;
        top = fmaxf(top, list.x[i]);
        mass += expf(list.lp[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    count = __reduce_add_sync(~0u, count);
    mass = warp_add(mass);
    const float base = base_of(top), rest_base = base_of(rest.m), up = pow2(scaled<false>(rest_base - base, k));
    float total = 0.0f;
    for (int i = lane; i < list.k; i += 32)
        if (list.place[i] >= 0) total += pow2(scaled<false>(list.x[i] - base, k));
    total = warp_add(total) + (rest.s != 0.0f ? rest.s * up : 0.0f);
    if (bad || y >= vocab) total = NAN;
    const bool nothing = total == 0.0f;  // -inf alone
    const float2 all = log_parts(total);
    const bool with_rest = a.tail == ZERO_TAIL_REST && count < vocab;
    const float shift = a.tail == ZERO_TAIL_RENORMALISE && count > 0 ? logf(mass) : 0.0f;
    auto logq = [&](float x) { return nothing ? -INFINITY : ((x - base) * inv_t - all.x) - all.y; };
    float d = 0.0f, c = 0.0f;
    for (int i = lane; i < list.k; i += 32) {
        if (list.place[i] < 0) continue;
        const float x = list.x[i], lp = list.lp[i] - shift, lq = logq(x);
        const float q = nothing ? 0.0f : pow2(scaled<false>(x - base, k)) / total;
        const Part part = entry_part(a.kind, a.mix, expf(lp), q, lp - lq);
        d += part.d;
        c += part.c;
    }
    d = warp_add(d);
    c = warp_add(c);
    Part outside = {0.0f, 0.0f};
    if (with_rest) {
        const float lp = a.teacher_rest ? a.teacher_rest[t] : logf(fmaxf(1.0f - mass, 0x1p-24f));
        const float2 own = log_parts(rest.s);
        const float lq = nothing || rest.s == 0.0f ? -INFINITY : ((rest_base - base) * inv_t + (own.x - all.x)) + (own.y - all.y);
        const float q = nothing ? 0.0f : rest.s != 0.0f ? rest.s * up / total : 0.0f;
        const float p = mass == mass ? expf(lp) : NAN;
        if (!(lp == -INFINITY && lq == -INFINITY)) outside = entry_part(a.kind, a.mix, p, q, lp - lq);
        d += outside.d;
        c += outside.c;
    }
    const float logp = y < vocab ? logq(x_y) : NAN;
    // a coefficient of 0 leaves its term out, also where that is infinite
    const float g = w * a.kl_coef * inv_t, h = w * a.ce_coef * inv_t;
    const float share = (a.ce_coef != 0.0f ? h : 0.0f) - (a.kl_coef != 0.0f ? g * c : 0.0f);
    DistillRow r;
    r.base = rest_base;
    r.factor = 0.0f;  // outside the list there is nothing above -inf
    if (rest.s != 0.0f) {
        r.factor = share * up / total;
        if (with_rest && a.kl_coef != 0.0f) r.factor += g * outside.c / rest.s;
    }
    if (total != total) r.factor = NAN;
    r.target_listed = false;
    for (int i = lane; i < list.k; i += 32) {
        if (list.place[i] < 0) continue;
        const float x = list.x[i], lp = list.lp[i] - shift;
        const float q = nothing ? 0.0f : pow2(scaled<false>(x - base, k)) / total;
        float v = share * q;
        if (a.kl_coef != 0.0f) v += g * entry_part(a.kind, a.mix, expf(lp), q, lp - logq(x)).c;
        if (list.place[i] == y) {
            v -= h;
            r.target_listed = true;
        }
        list.x[i] = nothing ? 0.0f : v;
    }
    r.target_listed = __any_sync(~0u, r.target_listed);
    r.target = nothing ? 0.0f : fmaf(pow2(scaled<false>(x_y - rest_base, k)), r.factor, -h);
    if (first && lane == 0) {
        float loss = 0.0f;
        if (a.kl_coef != 0.0f) loss += a.kl_coef * d;
        if (a.ce_coef != 0.0f) loss -= a.ce_coef * logp;
        if (total != total) loss = d = NAN;
        a.loss[t] = loss * w;
        a.kl[t] = d;
        a.logp[t] = logp;
    }
    return r;
}

// Any row: read once for the rest's sum and again for the gradient, by `size` CTAs (a cluster).
template <class T, int THREADS>
__global__ void __launch_bounds__(THREADS) k_distill_rows(const Rows<T> a, const DistillTokens p, int size, T* dx, int64_t dstride) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ RowStat sm[THREADS / 32], mine;
    __shared__ DistillRow shared_row;
    __shared__ int shared_bad;
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
    if (id == 0) shared_bad = 0;
    __syncthreads();
    const float x_y = y < a.vocab ? widen(x[y]) : NAN;
    const int shift = (kVec<T> - (s.tail_at % kVec<T>)) % kVec<T>;
    for (int i = id; i < p.k; i += THREADS) {
        const int64_t j = p.index[t * p.k + i];
        const float lp = p.teacher[t * p.k + i];
        int place = -1;
        if (j >= 0 && lp != -INFINITY) {
            if (j >= a.vocab) {
                shared_bad = 1;
            } else {
                place = (int)j;
                const uint32_t bit = 1u << ((place + shift) & 31);
                if (atomicOr(list.bits + ((place + shift) >> 5), bit) & bit) shared_bad = 1;  // twice in the list
                list.x[i] = widen(x[j]);
                list.lp[i] = lp;
            }
        }
        list.place[i] = place;
    }
    __syncthreads();
    auto sums = [&](auto checked) {
        constexpr bool kChecked = decltype(checked)::value;
        Sums<T, false, kChecked> run(a.k, x_y);
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
    if (fabsf(x_y) < INFINITY) {
        st = sums(std::false_type());
        good = st.s > 0x1p-60f && st.s < 0x1p60f;
        if (!good) __syncthreads();
    }
    if (!good) st = sums(std::true_type());
    st = cluster_join<false>(st, size, a.k, &mine);
    if (id < 32) {
        const DistillRow r = finish_list(p, list, st, shared_bad != 0, t, y, x_y, a.vocab, a.k, (float)a.inv_t, rank == 0);
        if (id == 0) shared_row = r;
    }
    __syncthreads();
    const DistillRow r = shared_row;
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
    // the list's entries and the target, by the CTA that wrote their places
    auto ours = [&](int64_t j) {
        return (j >= s.first && j < s.first + s.n * kVec<T>) || (s.head && j < s.head) || (s.tail && j >= s.tail_at);
    };
    for (int i = id; i < p.k; i += THREADS)
        if (list.place[i] >= 0 && ours(list.place[i])) out[list.place[i]] = narrow<T>(r.factor == r.factor ? list.x[i] : NAN);
    if (id == 0 && !r.target_listed && y < a.vocab && ours(y)) out[y] = narrow<T>(r.target);
    if (size > 1) cg::this_cluster().sync();  // no CTA leaves while another reads its sums
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
    a.mix = (float)p->mix;
    a.kl_coef = (float)p->kl_coef;
    a.ce_coef = (float)p->ce_coef;
    a.kind = p->kind;
    a.tail = p->tail;
    const int sms = d.sm_count(), ctas = token_ctas(x->rows);
    if (x->rows > 0) {
        if ((rc = launch_linked(k_token_setup<DistillTokens>, (unsigned)ctas, kSetupThreads, 0, ctas, s, a))) return rc;
        rc = by_type(x->type, [&](auto tag) {
            using T = decltype(tag);
            auto* kernel = k_distill_rows<T, kRowThreads>;
            const size_t smem = (size_t)4 * bitmap_words(x->vocab) + 12 * (size_t)a.k;
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(4 * bitmap_words(kDistillVocab) + 12 * kListMost));
            if (e != cudaSuccess) return record_cuda_error(e);
            const int size = ctas_per_row(x, sms, smem > 16384 ? 4 : kRowCtas / 2);
            return launch_linked(kernel, (unsigned)(x->rows * size), kRowThreads, smem, size, s, rows_of<T>(x, nullptr), a, size, (T*)p->dlogits,
                                 p->dstride);
        });
        if (rc) return rc;
    }
    return launch_linked(k_token_finish<DistillTokens>, (unsigned)ctas, kSetupThreads, 0, ctas, s, a);
}
