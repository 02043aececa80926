// zero_grads.cu -- the global L2 norm over many separate tensors, and clipping, for sm_103a.
//
// The tensors are laid end to end in units of 2 source bytes, each starting at a multiple of
// 128 bytes of that line, and the line is cut into one range per CTA, so that every CTA reads
// the same number of bytes whatever the tensors' sizes and types. A CTA's part of a tensor has
// a slot of its own (CTA index + tensor index: along the line one of the two always grows), and
// slots and totals are added in a fixed order: the sums do not depend on which CTA ends first.
// Two launches: the sums of squares, and the scaled copy, each CTA over the same range. The norm
// has to be known before anything is written, so the gradients are read twice. On one GB300 (copy
// peak 6,673 GB/s), replayed from a graph: 1.3B bf16 into bf16 1.24 ms, 7.86 GB in three passes,
// 95% of the peak; 124M fp32 into bf16 201 us, 92%; 26 vectors of 768 11.2 us, two launches' worth.

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <new>
#include <unordered_set>
#include <vector>

#include "zero_host.h"
#include "zero_softmax.cuh"
#include "zero_sum.cuh"

struct zero_grads {
    int64_t n, units, per;  // tensors; 2-byte units of the line, and of one CTA
    int grid;
    char* workspace;
};

namespace zg {
namespace {

constexpr int kGradThreads = 512, kGradWarps = kGradThreads / 32;
constexpr int kGradMaxGrid = 1024;
constexpr int64_t kGradAlign = 64;  // units: 128 bytes of source
constexpr int kBatch = 64;          // tensors whose rows a CTA holds at a time
constexpr int kSmallSpan = 4096;    // elements of a tensor up to which one warp takes it alone

// One tensor of the line.
struct GradRow {
    const void* src;
    void* dst;
    int64_t numel;
    int64_t start;  // its first unit
    int32_t src_type, dst_type;
};
static_assert(sizeof(GradRow) == 40, "table row is 40 bytes");

struct GradArgs {
    const GradRow* rows;
    const int32_t* first;  // [grid] the tensor that holds a CTA's first unit
    double* slots;     // [n + grid] one per CTA's part of a tensor
    double* totals;    // [grid] of a CTA's whole range
    int64_t n, units, per;  // units of a CTA
    int32_t grid;      // CTAs of the line
    float *norm, *scale, *norms;
    double max_norm;
};

// Elements of tensor r that lie in units [u0, u1).
struct Span {
    int64_t b, e;
};
__device__ __forceinline__ Span span_of(const GradRow& r, int64_t u0, int64_t u1) {
    const int w = r.src_type == ZERO_T_FP32 ? 1 : 0;  // units per element: 2 or 1
    int64_t b = (u0 - r.start) >> w, e = (u1 - r.start) >> w;
    b = b < 0 ? 0 : b;
    e = e > r.numel ? r.numel : e;
    return {b, e < b ? b : e};
}

// Calls `whole(i, row, span)` with all threads for this CTA's part of each large tensor and
// `alone(i, row, span)` with one warp for each small one; i is the tensor. The rows of up to kBatch
// tensors are fetched at once: thousands of small tensors would wait for each other's otherwise.
template <class W, class A>
__device__ __forceinline__ void for_tensors(const GradArgs& a, int64_t u0, int64_t u1, GradRow* batch, W whole, A alone) {
    if (u0 >= u1) return;
    const int warp = threadIdx.x >> 5;
    for (int64_t t0 = a.first[blockIdx.x];; t0 += kBatch) {
        const int64_t t = t0 + threadIdx.x;
        if (threadIdx.x < kBatch) {
            batch[threadIdx.x].start = INT64_MAX;
            if (t < a.n) batch[threadIdx.x] = a.rows[t];
        }
        __syncthreads();
        for (int i = 0; i < kBatch && batch[i].start < u1; ++i) {
            const Span sp = span_of(batch[i], u0, u1);
            if (sp.e - sp.b > kSmallSpan) whole(t0 + i, batch[i], sp);
        }
        for (int i = warp; i < kBatch && batch[i].start < u1; i += kGradWarps) {
            const Span sp = span_of(batch[i], u0, u1);
            if (sp.e - sp.b <= kSmallSpan) alone(t0 + i, batch[i], sp);
        }
        const bool more = batch[kBatch - 1].start < u1;
        __syncthreads();
        if (!more) return;
    }
}

// A sum of squares whose terms may leave fp32 either way. The squares of up to 32 values are added
// in fp32; where that sum is no usable number (over 2^80, or under 2^-100: values of 2^-50 and
// less, or none but zeros), each value goes into the sum of its own size, scaled so that 2^31 of
// the largest still fit.
struct Squares {
    Sum mid, big, small;  // big: times 2^-180, small: times 2^150
    __device__ __forceinline__ void one_by_one(float x) {
        const float y = fabsf(x);
        if (y > 0x1p40f) big.add((x * 0x1p-90f) * (x * 0x1p-90f));
        else if (y < 0x1p-60f) small.add((x * 0x1p75f) * (x * 0x1p75f));
        else mid.add(x * x);
    }
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N]) {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < N; ++i) s[i & 3] = fmaf(x[i], x[i], s[i & 3]);
        const float p = (s[0] + s[1]) + (s[2] + s[3]);
        if (p >= 0x1p-100f && p < 0x1p80f) {
            mid.add(p);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) one_by_one(x[i]);
        }
    }
    __device__ __forceinline__ void over_warp() {
        mid = warp_sum(mid);
        if (__any_sync(~0u, big.hi != 0.0f)) big = warp_sum(big);
        if (__any_sync(~0u, small.hi != 0.0f)) small = warp_sum(small);
    }
    __device__ __forceinline__ double value() const { return mid.value() + big.value() * 0x1p180 + small.value() * 0x1p-150; }
};

// Eight elements of type T from p (aligned for 16-byte loads where ALIGNED). LAST: nothing reads
// them again; they may be written by this kernel, so not through the read-only path.
template <class T, bool ALIGNED, bool LAST>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    if constexpr (!ALIGNED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = widen(p[i]);
    } else {
        constexpr int kVecs = 8 / kVec<T>;
        uint4 v[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const uint4* q = reinterpret_cast<const uint4*>(p) + i;
            v[i] = LAST ? __ldcs(q) : load_once(q);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(widen2<T>(v[i / (kVec<T> / 2)], i % (kVec<T> / 2)));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
    constexpr int kVecs = 8 / kVec<T>;
    uint4 v[kVecs];
#pragma unroll
    for (int i = 0; i < 4; ++i) narrow2<T>(v[i / (kVec<T> / 2)], i % (kVec<T> / 2), make_float2(x[2 * i], x[2 * i + 1]));
#pragma unroll
    for (int i = 0; i < kVecs; ++i) __stcs(reinterpret_cast<uint4*>(p) + i, v[i]);
}

// Elements before the first 16-byte boundary of p.
template <class T>
__device__ __forceinline__ int64_t to_boundary(const T* p) {
    return (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int64_t)sizeof(T);
}

// Squares of src[b, e) as threads `id` of `count` take them, 32 elements at a time.
template <class T>
__device__ __forceinline__ void sum_span(const T* src, Span sp, int id, int count, Squares& sq) {
    const T* p = src + sp.b;
    const int64_t n = sp.e - sp.b;
    int64_t head = to_boundary(p);
    head = head < n ? head : n;
    const int64_t groups = (n - head) / 8, tail = head + groups * 8;
    p += head;
    int64_t i = id;
    for (; i + 3 * (int64_t)count < groups; i += 4 * (int64_t)count) {
        float x[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) load8<T, true, false>(p + (i + u * (int64_t)count) * 8, x[u]);
        sq.add(reinterpret_cast<float(&)[32]>(x));
    }
    for (; i < groups; i += count) {
        float x[8];
        load8<T, true, false>(p + i * 8, x);
        sq.add(x);
    }
    p -= head;
    if (id < head) sq.one_by_one(widen(p[id]));
    if (id < n - tail) sq.one_by_one(widen(p[tail + id]));
}
__device__ __forceinline__ void sum_any(const GradRow& r, Span sp, int id, int count, Squares& sq) {
    if (r.src_type == ZERO_T_BF16) sum_span((const __nv_bfloat16*)r.src, sp, id, count, sq);
    else if (r.src_type == ZERO_T_FP16) sum_span((const __half*)r.src, sp, id, count, sq);
    else sum_span((const float*)r.src, sp, id, count, sq);
}

// Bound by reading the gradients once.
__global__ void __launch_bounds__(kGradThreads, 2) k_grads_sumsq(const GradArgs a) {
    __shared__ GradRow batch[kBatch];
    __shared__ double sm[kGradWarps], small_totals[kGradWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    let_next_kernel_start();
    wait_for_kernel_before();
    const int64_t u0 = min(a.units, a.per * blockIdx.x), u1 = min(a.units, u0 + a.per);
    double total = 0.0, alone_total = 0.0;  // in thread 0; in lane 0 of each warp
    for_tensors(
        a, u0, u1, batch,
        [&](int64_t t, const GradRow& r, Span sp) {
            Squares sq;
            sum_any(r, sp, threadIdx.x, kGradThreads, sq);
            sq.over_warp();
            if (lane == 0) sm[warp] = sq.value();
            __syncthreads();
            if (threadIdx.x == 0) {
                double s = 0.0;
                for (int w = 0; w < kGradWarps; ++w) s += sm[w];
                a.slots[blockIdx.x + t] = s;
                total += s;
            }
            __syncthreads();
        },
        [&](int64_t t, const GradRow& r, Span sp) {
            Squares sq;
            sum_any(r, sp, lane, 32, sq);
            sq.over_warp();
            if (lane == 0) {
                const double s = sq.value();
                a.slots[blockIdx.x + t] = s;
                alone_total += s;
            }
        });
    if (lane == 0) small_totals[warp] = alone_total;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 0; w < kGradWarps; ++w) total += small_totals[w];
        a.totals[blockIdx.x] = total;
    }
}

// dst[b, e) = src[b, e) * f as threads `id` of `count` take them, from the end: what the sum of
// squares read last may still be in L2. Groups of eight lie at dst's 16-byte boundaries; src's are
// loaded one by one (through L1) where its alignment differs: the whole call on 124M values into bf16,
// from fp32 213 us where dst begins at an odd element and 197 where it is aligned, from bf16 148 and 126.
template <class S, class D, bool ALIGNED>
__device__ __forceinline__ void scale_groups(const S* s, D* d, int64_t groups, int id, int count, float f) {
    const int64_t last = (groups - 1 - id) / count;  // this thread's last round; negative rounds to 0
    if (id >= groups) return;
    int64_t k = last;
    for (; k >= 3; k -= 4) {
        float x[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) load8<S, ALIGNED, true>(s + (id + (k - u) * count) * 8, x[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[u][j] *= f;
            store8(d + (id + (k - u) * count) * 8, x[u]);
        }
    }
    for (; k >= 0; --k) {
        float x[8];
        load8<S, ALIGNED, true>(s + (id + k * count) * 8, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= f;
        store8(d + (id + k * count) * 8, x);
    }
}
template <class S, class D>
__device__ __forceinline__ void scale_span(const S* src, D* dst, Span sp, int id, int count, float f) {
    const S* s = src + sp.b;
    D* d = dst + sp.b;
    const int64_t n = sp.e - sp.b;
    int64_t head = to_boundary(d);
    head = head < n ? head : n;
    const int64_t groups = (n - head) / 8, tail = head + groups * 8;
    if (to_boundary(s + head) == 0) scale_groups<S, D, true>(s + head, d + head, groups, id, count, f);
    else scale_groups<S, D, false>(s + head, d + head, groups, id, count, f);
    if (id < head) d[id] = narrow<D>(widen(s[id]) * f);
    if (id < n - tail) d[tail + id] = narrow<D>(widen(s[tail + id]) * f);
}
template <class S>
__device__ __forceinline__ void scale_to(const GradRow& r, Span sp, int id, int count, float f) {
    if (r.dst_type == ZERO_T_BF16) scale_span((const S*)r.src, (__nv_bfloat16*)r.dst, sp, id, count, f);
    else if (r.dst_type == ZERO_T_FP16) scale_span((const S*)r.src, (__half*)r.dst, sp, id, count, f);
    else scale_span((const S*)r.src, (float*)r.dst, sp, id, count, f);
}
__device__ __forceinline__ void scale_any(const GradRow& r, Span sp, int id, int count, float f) {
    if (!r.dst || (r.dst == r.src && f == 1.0f)) return;
    if (r.src_type == ZERO_T_BF16) scale_to<__nv_bfloat16>(r, sp, id, count, f);
    else if (r.src_type == ZERO_T_FP16) scale_to<__half>(r, sp, id, count, f);
    else scale_to<float>(r, sp, id, count, f);
}

// Bound by reading the gradients again and writing them. Every CTA adds the totals of all in the
// same order (a warp, a few hundred numbers from L2), which is cheaper than a kernel between.
__global__ void __launch_bounds__(kGradThreads, 2) k_grads_scale(const GradArgs a) {
    __shared__ GradRow batch[kBatch];
    __shared__ float factor;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    wait_for_kernel_before();
    if (warp == 0) {
        double s = 0.0;
        for (int i = lane; i < a.grid; i += 32) s += a.totals[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        if (lane == 0) {
            const double norm = sqrt(s);
            const float rounded = (float)norm;
            factor = isfinite(rounded) && norm > a.max_norm ? (float)(a.max_norm / norm) : 1.0f;
            if (blockIdx.x == 0) {
                *a.norm = rounded;
                *a.scale = factor;
            }
        }
    }
    __syncthreads();
    // every tensor's own norm, a warp each
    if (a.norms)
        for (int64_t t = (int64_t)blockIdx.x * kGradWarps + warp; t < a.n; t += (int64_t)gridDim.x * kGradWarps) {
            const GradRow r = a.rows[t];
            const int64_t len = r.src_type == ZERO_T_FP32 ? 2 * r.numel : r.numel;
            double s = 0.0;
            if (len > 0)
                for (int64_t b = r.start / a.per + lane; b <= (r.start + len - 1) / a.per; b += 32) s += a.slots[b + t];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
            if (lane == 0) a.norms[t] = (float)sqrt(s);
        }
    const float f = factor;
    const int64_t u0 = min(a.units, a.per * blockIdx.x), u1 = min(a.units, u0 + a.per);
    for_tensors(
        a, u0, u1, batch, [&](int64_t, const GradRow& r, Span sp) { scale_any(r, sp, threadIdx.x, kGradThreads, f); },
        [&](int64_t, const GradRow& r, Span sp) { scale_any(r, sp, lane, 32, f); });
}

std::mutex g_plans_mu;
std::unordered_set<const zero_grads*> g_plans;  // plans not yet destroyed

int64_t table_bytes(int64_t n) { return (n * (int64_t)sizeof(GradRow) + 255) / 256 * 256; }

// A plan's workspace: the table, slots, totals, and the CTAs' first tensors.
double* slots_of(void* workspace, int64_t n) { return (double*)((char*)workspace + table_bytes(n)); }
int32_t* first_of(void* workspace, int64_t n) { return (int32_t*)(slots_of(workspace, n) + n + 2 * kGradMaxGrid); }

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" int64_t zero_grads_workspace(int64_t n) {
    if (n < 1 || n > INT32_MAX) return -1;
    return table_bytes(n) + (n + 2 * kGradMaxGrid) * 8 + kGradMaxGrid * 4;
}

extern "C" int zero_grads_init(zero_grads** out, const zero_grad_tensor* tensors, int64_t n, void* workspace,
                               int64_t workspace_bytes, void* stream) {
    if (out) *out = nullptr;
    if (!out || !tensors || n < 1 || n > INT32_MAX) return ZERO_ERR_INVALID_ARG;
    if (workspace_bytes < zero_grads_workspace(n)) return ZERO_ERR_SIZE_MISMATCH;
    CallDevice d(workspace, stream);
    d.need(workspace, 256);
    std::vector<GradRow> rows;
    try {
        rows.resize((size_t)n);
    } catch (...) {
        return ZERO_ERR_INVALID_ARG;
    }
    int64_t at = 0;
    for (int64_t i = 0; i < n && !d.rc; ++i) {
        const zero_grad_tensor& t = tensors[i];
        if (t.numel < 0 || t.numel > (INT64_C(1) << 44) || !type_ok(t.src_type) || (t.dst && !type_ok(t.dst_type))) return ZERO_ERR_INVALID_ARG;
        if (t.dst && t.dst == t.src && t.dst_type != t.src_type) return ZERO_ERR_INVALID_ARG;
        if (t.numel > 0) {
            d.need(t.src, type_size(t.src_type));
            if (t.dst) d.need(t.dst, type_size(t.dst_type));
        }
        rows[(size_t)i] = GradRow{t.src, t.numel > 0 ? t.dst : nullptr, t.numel, at, t.src_type, t.dst_type};
        const int64_t units = t.numel * (type_size(t.src_type) / 2);
        at += (units + kGradAlign - 1) / kGradAlign * kGradAlign;
        if (at > (INT64_C(1) << 46)) return ZERO_ERR_INVALID_ARG;
    }
    if (d.rc) return d.rc;
    const int64_t want = at / (32 * kGradAlign) + 1;  // at least 4 KB of source a CTA
    const int64_t most = std::min<int64_t>(std::min<int64_t>(want, 2 * d.sm_count()), kGradMaxGrid);
    const int64_t per = std::max<int64_t>(1, (at / kGradAlign + most - 1) / most) * kGradAlign;
    const int grid = (int)std::max<int64_t>(1, (at + per - 1) / per);
    int32_t first[kGradMaxGrid] = {};
    for (int64_t b = 0, t = 0; b < grid; ++b) {  // the last tensor that starts at or before the CTA's range
        while (t + 1 < n && rows[(size_t)t + 1].start <= b * per) ++t;
        first[b] = (int32_t)t;
    }
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = cudaMemcpyAsync(workspace, rows.data(), (size_t)n * sizeof(GradRow), cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaMemcpyAsync(first_of(workspace, n), first, sizeof first, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return record_cuda_error(e);
    zero_grads* p = new (std::nothrow) zero_grads{n, at, per, grid, (char*)workspace};
    if (!p) return ZERO_ERR_INVALID_ARG;
    try {
        std::lock_guard<std::mutex> lk(g_plans_mu);
        g_plans.insert(p);
    } catch (...) {
        delete p;
        return ZERO_ERR_INVALID_ARG;
    }
    *out = p;
    return ZERO_OK;
}

extern "C" int zero_grads_clip(zero_grads* p, double max_norm, float* norm, float* scale, float* tensor_norms, void* stream) {
    {
        std::lock_guard<std::mutex> lk(g_plans_mu);
        if (!p || !g_plans.count(p)) return ZERO_ERR_BAD_CONTEXT;
    }
    if (!(max_norm > 0.0)) return ZERO_ERR_INVALID_ARG;
    CallDevice d(p->workspace, stream);
    d.need(norm, 4);
    d.need(scale, 4);
    d.optional(tensor_norms, 4);
    if (d.rc) return d.rc;
    cudaStream_t s = (cudaStream_t)stream;
    GradArgs a;
    a.rows = (const GradRow*)p->workspace;
    a.first = first_of(p->workspace, p->n);
    a.slots = slots_of(p->workspace, p->n);
    a.totals = a.slots + p->n + kGradMaxGrid;
    a.n = p->n;
    a.units = p->units;
    a.per = p->per;
    a.grid = p->grid;
    a.norm = norm;
    a.scale = scale;
    a.norms = tensor_norms;
    a.max_norm = max_norm;
    const int rc = launch_linked(k_grads_sumsq, (unsigned)p->grid, kGradThreads, 0, 1, s, a);
    return rc ? rc : launch_linked(k_grads_scale, (unsigned)p->grid, kGradThreads, 0, 1, s, a);
}

extern "C" int zero_grads_destroy(zero_grads* p) {
    std::lock_guard<std::mutex> lk(g_plans_mu);
    if (!p || !g_plans.erase(p)) return ZERO_ERR_BAD_CONTEXT;
    delete p;
    return ZERO_OK;
}
