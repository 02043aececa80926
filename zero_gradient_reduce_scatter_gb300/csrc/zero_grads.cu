// zero_grads.cu -- the global L2 norm over many separate tensors, and clipping, for sm_103a.
//
// The tensors are laid end to end in units of 2 source bytes, each starting at a multiple of
// 128 bytes of that line, and the line is cut into one range per CTA, so that every CTA reads
// the same number of bytes whatever the tensors' sizes and types. A CTA's part of a tensor has
// a slot of its own (CTA index + tensor index: along the line one of the two always grows), and
// the slots of a tensor are added in order: the sums do not depend on which CTA ends first.

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <new>
#include <unordered_set>
#include <vector>

#include "zero_host.h"
#include "zero_softmax.cuh"

struct zero_grads {
    int device;
    int64_t n;
    int64_t units;
    int grid;
    bool has_dst;
    char* workspace;
};

namespace zg {
namespace {

constexpr int kGradThreads = 512;
constexpr int kGradMaxGrid = 1024;
constexpr int64_t kGradAlign = 64;  // units: 128 bytes of source

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
    double* slots;   // [n + grid]
    int64_t n, units;
    float *norm, *scale, *norms;
    double max_norm;
};

__host__ __device__ __forceinline__ int64_t range_start(int64_t units, int grid, int b) {
    const int64_t per = (units / kGradAlign + grid - 1) / grid * kGradAlign;
    const int64_t u = per * b;
    return u < units ? u : units;
}

// The tensor that holds unit u: the last one that starts at or before it.
__device__ __forceinline__ int64_t tensor_of(const GradRow* rows, int64_t n, int64_t u) {
    int64_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (rows[mid].start <= u) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Elements of tensor r that lie in units [u0, u1).
struct Span {
    int64_t b, e;
};
__device__ __forceinline__ Span span_of(const GradRow& r, int64_t u0, int64_t u1) {
    const int w = r.src_type == ZERO_T_FP32 ? 1 : 0;  // units per element: 2 or 1
    int64_t b = (u0 - r.start) >> w, e = (u1 - r.start) >> w;
    b = b < 0 ? 0 : b;
    e = e > r.numel ? r.numel : e;
    return {b, e};
}

__device__ __forceinline__ float load_any(const void* p, int32_t type, int64_t i) {
    if (type == ZERO_T_BF16) return widen(((const __nv_bfloat16*)p)[i]);
    if (type == ZERO_T_FP16) return widen(((const __half*)p)[i]);
    return ((const float*)p)[i];
}
__device__ __forceinline__ void store_any(void* p, int32_t type, int64_t i, float x) {
    if (type == ZERO_T_BF16) ((__nv_bfloat16*)p)[i] = narrow<__nv_bfloat16>(x);
    else if (type == ZERO_T_FP16) ((__half*)p)[i] = narrow<__half>(x);
    else ((float*)p)[i] = x;
}

__device__ __forceinline__ double block_sum(double x, double* sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    double t = 0.0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += sm[w];
    __syncthreads();
    return t;
}

__global__ void __launch_bounds__(kGradThreads) k_grads_sumsq(const GradArgs a) {
    __shared__ double sm[kGradThreads / 32];
    const int64_t u0 = range_start(a.units, gridDim.x, blockIdx.x), u1 = range_start(a.units, gridDim.x, blockIdx.x + 1);
    if (u0 >= u1) return;
    for (int64_t t = tensor_of(a.rows, a.n, u0); t < a.n && a.rows[t].start < u1; ++t) {
        const GradRow r = a.rows[t];
        const Span sp = span_of(r, u0, u1);
        double s = 0.0;
        for (int64_t i = sp.b + threadIdx.x; i < sp.e; i += kGradThreads) {
            const double x = load_any(r.src, r.src_type, i);
            s += x * x;
        }
        s = block_sum(s, sm);
        if (threadIdx.x == 0) a.slots[blockIdx.x + t] = s;
    }
}

// One warp per tensor adds its slots; then the tensors' sums are added in order.
__global__ void __launch_bounds__(1024) k_grads_finish(const GradArgs a, int grid) {
    __shared__ double sm[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t per = (a.units / kGradAlign + grid - 1) / grid * kGradAlign;
    double total = 0.0;
    for (int64_t t = warp; t < a.n; t += 32) {
        const GradRow r = a.rows[t];
        const int64_t len = r.src_type == ZERO_T_FP32 ? 2 * r.numel : r.numel;
        double s = 0.0;
        if (len > 0) {
            const int64_t b0 = r.start / per, b1 = (r.start + len - 1) / per;
            for (int64_t b = b0 + lane; b <= b1; b += 32) s += a.slots[b + t];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        if (lane == 0) {
            total += s;
            if (a.norms) a.norms[t] = (float)sqrt(s);
        }
    }
    const double norm = sqrt(block_sum(total, sm));
    if (threadIdx.x == 0) {
        *a.norm = (float)norm;
        *a.scale = isfinite(norm) && norm > a.max_norm ? (float)(a.max_norm / norm) : 1.0f;
    }
}

__global__ void __launch_bounds__(kGradThreads) k_grads_scale(const GradArgs a) {
    const float f = *a.scale;
    const int64_t u0 = range_start(a.units, gridDim.x, blockIdx.x), u1 = range_start(a.units, gridDim.x, blockIdx.x + 1);
    if (u0 >= u1) return;
    for (int64_t t = tensor_of(a.rows, a.n, u0); t < a.n && a.rows[t].start < u1; ++t) {
        const GradRow r = a.rows[t];
        if (!r.dst || (r.dst == r.src && f == 1.0f)) continue;
        const Span sp = span_of(r, u0, u1);
        for (int64_t i = sp.b + threadIdx.x; i < sp.e; i += kGradThreads)
            store_any(r.dst, r.dst_type, i, load_any(r.src, r.src_type, i) * f);
    }
}

std::mutex g_plans_mu;
std::unordered_set<const zero_grads*> g_plans;  // plans not yet destroyed

int64_t table_bytes(int64_t n) { return (n * (int64_t)sizeof(GradRow) + 255) / 256 * 256; }

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" int64_t zero_grads_workspace(int64_t n) {
    if (n < 1 || n > INT32_MAX) return -1;
    return table_bytes(n) + (n + kGradMaxGrid) * 8;
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
    bool has_dst = false;
    for (int64_t i = 0; i < n && !d.rc; ++i) {
        const zero_grad_tensor& t = tensors[i];
        if (t.numel < 0 || t.numel > (INT64_C(1) << 44) || !type_ok(t.src_type) || (t.dst && !type_ok(t.dst_type))) return ZERO_ERR_INVALID_ARG;
        if (t.dst && t.dst == t.src && t.dst_type != t.src_type) return ZERO_ERR_INVALID_ARG;
        if (t.numel > 0) {
            d.need(t.src, type_size(t.src_type));
            if (t.dst) d.need(t.dst, type_size(t.dst_type));
            has_dst |= t.dst != nullptr;
        }
        rows[(size_t)i] = GradRow{t.src, t.numel > 0 ? t.dst : nullptr, t.numel, at, t.src_type, t.dst_type};
        const int64_t units = t.numel * (type_size(t.src_type) / 2);
        at += (units + kGradAlign - 1) / kGradAlign * kGradAlign;
        if (at > (INT64_C(1) << 46)) return ZERO_ERR_INVALID_ARG;
    }
    if (d.rc) return d.rc;
    const int64_t want = at / (16 * kGradAlign) + 1;  // at least 2 KB of source a CTA
    const int grid = (int)std::min<int64_t>(std::min<int64_t>(want, 4 * d.sm_count()), kGradMaxGrid);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = cudaMemcpyAsync(workspace, rows.data(), (size_t)n * sizeof(GradRow), cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return record_cuda_error(e);
    zero_grads* p = new (std::nothrow) zero_grads{d.device(), n, at, grid, has_dst, (char*)workspace};
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
    a.slots = (double*)(p->workspace + table_bytes(p->n));
    a.n = p->n;
    a.units = p->units;
    a.norm = norm;
    a.scale = scale;
    a.norms = tensor_norms;
    a.max_norm = max_norm;
    int rc = ZERO_OK;
    if (p->units > 0) {
        k_grads_sumsq<<<p->grid, kGradThreads, 0, s>>>(a);
        if ((rc = launched())) return rc;
    }
    k_grads_finish<<<1, 1024, 0, s>>>(a, p->grid);
    if ((rc = launched())) return rc;
    if (p->units > 0 && p->has_dst) {
        k_grads_scale<<<p->grid, kGradThreads, 0, s>>>(a);
        rc = launched();
    }
    return rc;
}

extern "C" int zero_grads_destroy(zero_grads* p) {
    std::lock_guard<std::mutex> lk(g_plans_mu);
    if (!p || !g_plans.erase(p)) return ZERO_ERR_BAD_CONTEXT;
    delete p;
    return ZERO_OK;
}
