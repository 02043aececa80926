// zero_embed.cu -- the rows of a vocabulary matrix for a batch's tokens, and their gradient, for sm_103a.
//
// Forward: out[t] = scale * weight[token[t]]. Backward: dweight[v] = scale * sum of dhidden[t] over the
// tokens t that are v, in the order of t, added to what is there or written; rows of no token are zeros.
// Both are bound by memory: the forward reads the batch's different rows once and writes one row a
// token, the backward reads one row a token and writes the matrix (or, adding, reads and writes the
// batch's different rows).

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "zero_host.h"
#include "zero_softmax.cuh"

namespace zg {
namespace {

constexpr int kEmbedThreads = 256;

// A row's slice of 32 lanes with 16 bytes of T each: lane's elements are kVec<T> neighbours (VEC: the
// addresses are aligned for it) or every 32nd.
template <class T, bool VEC>
__device__ __forceinline__ int64_t element(int64_t slice, int lane, int i) {
    constexpr int P = kVec<T>;
    return VEC ? (slice * 32 + lane) * P + i : slice * 32 * P + 32 * i + lane;
}

// This lane's elements of a row, as fp32; 0 past its end. A row is read once: past L1.
template <class T, bool VEC>
struct LaneRow {
    uint4 v;
    T e[VEC ? 1 : kVec<T>];

    __device__ __forceinline__ void load(const T* row, int64_t slice, int lane, int64_t dim) {
        if (VEC) {
            v = make_uint4(0, 0, 0, 0);
            const int64_t at = element<T, VEC>(slice, lane, 0);
            if (at < dim) v = load_once(reinterpret_cast<const uint4*>(row + at));
        } else {
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) {
                const int64_t at = element<T, VEC>(slice, lane, i);
                e[VEC ? 0 : i] = at < dim ? row[at] : narrow<T>(0.0f);
            }
        }
    }
    __device__ __forceinline__ void to(float* f) const {
#pragma unroll
        for (int i = 0; i < kVec<T>; i += 2) {
            if (VEC) {
                const float2 x = unpack2(widen2<T>(v, i / 2));
                f[i] = x.x;
                f[i + 1] = x.y;
            } else {
                f[i] = widen(e[VEC ? 0 : i]);
                f[i + 1] = widen(e[VEC ? 0 : i + 1]);
            }
        }
    }
};

// kVec<T> numbers of this lane to and from a row of another type.
template <class T, class O, bool VEC>
__device__ __forceinline__ void lane_store(O* row, int64_t slice, int lane, int64_t dim, const float* f) {
    constexpr int P = kVec<T>;
    if constexpr (VEC) {
        const int64_t at = element<T, VEC>(slice, lane, 0);
        if (at >= dim) return;
        struct alignas(P * sizeof(O) < 16 ? P * sizeof(O) : 16) Out {
            O o[P];
        } out;
#pragma unroll
        for (int i = 0; i < P; ++i) out.o[i] = narrow<O>(f[i]);
        *reinterpret_cast<Out*>(row + at) = out;
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t at = element<T, VEC>(slice, lane, i);
            if (at < dim) row[at] = narrow<O>(f[i]);
        }
    }
}
template <class T, class O, bool VEC>
__device__ __forceinline__ void lane_load(const O* row, int64_t slice, int lane, int64_t dim, float* f) {
    constexpr int P = kVec<T>;
    if constexpr (VEC) {
        const int64_t at = element<T, VEC>(slice, lane, 0);
        if (at >= dim) return;
        struct alignas(P * sizeof(O) < 16 ? P * sizeof(O) : 16) In {
            O o[P];
        };
        const In in = *reinterpret_cast<const In*>(row + at);
#pragma unroll
        for (int i = 0; i < P; ++i) f[i] = widen(in.o[i]);
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t at = element<T, VEC>(slice, lane, i);
            if (at < dim) f[i] = widen(row[at]);
        }
    }
}

// ---------------------------------------------------------------------------------------
// Forward: a warp per kRowSlices slices of a token's row.
// ---------------------------------------------------------------------------------------
constexpr int kRowSlices = 4;

template <class T, bool VEC>
__global__ void __launch_bounds__(kEmbedThreads)
    k_embed(const T* weight, int64_t ldw, const int64_t* tokens, int64_t rows, int64_t vocab, int64_t dim, float scale, T* out, int64_t ldo,
            int64_t parts) {
    wait_for_kernel_before();
    let_next_kernel_start();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kEmbedThreads / 32);
    for (int64_t unit = (int64_t)blockIdx.x * (kEmbedThreads / 32) + (threadIdx.x >> 5); unit < rows * parts; unit += step) {
        const int64_t t = unit / parts, first = unit % parts * kRowSlices;
        const int64_t y = tokens[t];
        const bool there = y >= 0 && y < vocab;
        LaneRow<T, VEC> r[kRowSlices];
#pragma unroll
        for (int u = 0; u < kRowSlices; ++u) r[u].load(weight + (there ? y * ldw : 0), first + u, lane, there ? dim : 0);
#pragma unroll
        for (int u = 0; u < kRowSlices; ++u) {
            float f[kVec<T>];
            r[u].to(f);
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) f[i] = there ? f[i] * scale : y < 0 ? 0.0f : NAN;
            lane_store<T, T, VEC>(out + t * ldo, first + u, lane, dim, f);
        }
    }
}

// ---------------------------------------------------------------------------------------
// Backward, first kernel: positions in the order of their tokens. CTA c owns the tokens
// [c * width, (c + 1) * width) and reads all positions twice (from L2 but for the first CTA): once to
// count its own tokens and those below them, which is where its part of the order begins, and once
// to write its positions there. A warp takes a contiguous share of the positions with counters of its
// own, and lanes of one token rank themselves, so the order is that of the positions: no CTA waits
// for another, and equal calls give equal bits. Rows of no token are zeroed by their owner meanwhile.
// ---------------------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortWidth = 1024;  // most tokens of a CTA: a thread each

struct SortArgs {
    const int64_t* tokens;
    int64_t rows, vocab;
    int width;
    int32_t *position, *token;  // [rows] in order
    int32_t *begin, *count;     // [vocab] of tokens that there are: a token's place and number in the order
    int64_t* live;              // [1] length of the order
    uint32_t* counters;         // to be zeroed
    int64_t n_counters;
    uint8_t* zero;              // the matrix where its rows of no token are zeroed, or nullptr
    int64_t row_bytes, stride_bytes;
    int element;                // bytes
};

__device__ __forceinline__ void zero_bytes(uint8_t* p, int64_t bytes, int element, int lane) {
    const int64_t head = min((int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15), bytes), vecs = (bytes - head) / 16;
    auto one = [&](int64_t at) {
        if (element == 2) *reinterpret_cast<uint16_t*>(p + at) = 0;
        else *reinterpret_cast<uint32_t*>(p + at) = 0;
    };
    if (lane * element < head) one(lane * element);
    for (int64_t i = lane; i < vecs; i += 32) __stcs(reinterpret_cast<uint4*>(p + head) + i, make_uint4(0, 0, 0, 0));
    if (head + 16 * vecs + lane * element < bytes) one(head + 16 * vecs + lane * element);
}

__global__ void __launch_bounds__(kSortThreads) k_embed_sort(const SortArgs a) {
    extern __shared__ int32_t counts[];  // [kSortWarps][width]
    __shared__ int32_t warp_sum[kSortWarps];
    __shared__ unsigned long long below_all;
    __shared__ int32_t total[kSortWidth];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t lo = (int64_t)blockIdx.x * a.width, hi = min(lo + a.width, a.vocab);
    int32_t* mine = counts + warp * a.width;
    for (int b = lane; b < a.width; b += 32) mine[b] = 0;
    if (threadIdx.x == 0) below_all = 0;
    wait_for_kernel_before();
    let_next_kernel_start();
    for (int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; i < a.n_counters; i += (int64_t)gridDim.x * kSortThreads) a.counters[i] = 0;
    __syncthreads();

    const int64_t share = ((a.rows + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int64_t from = min(share * warp, a.rows), to = min(from + share, a.rows);
    unsigned below = 0;
#pragma unroll 4
    for (int64_t t = from + lane; t < to; t += 32) {
        const int64_t y = a.tokens[t];
        below += y >= 0 && y < lo;
        if (y >= lo && y < hi) atomicAdd(mine + (y - lo), 1);
    }
    below = __reduce_add_sync(~0u, below);
    if (lane == 0 && below) atomicAdd(&below_all, (unsigned long long)below);
    __syncthreads();

    // thread b: token lo + b. Its number, its place among this CTA's, and every warp's place in it
    const int b = threadIdx.x;
    int32_t n = 0;
    if (b < a.width)
        for (int w = 0; w < kSortWarps; ++w) n += counts[w * a.width + b];
    int32_t scan = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(~0u, scan, o);
        if (lane >= o) scan += x;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    int32_t before = lane < warp ? warp_sum[lane] : 0;
    before = __reduce_add_sync(~0u, before);
    int32_t at = (int32_t)below_all + before + scan - n;
    total[b] = n;
    if (b < a.width) {
        if (n > 0) {
            a.begin[lo + b] = at;
            a.count[lo + b] = n;
        }
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t c = counts[w * a.width + b];
            counts[w * a.width + b] = at;
            at += c;
        }
    }
    if (blockIdx.x == gridDim.x - 1 && b == kSortThreads - 1) *a.live = at;
    __syncthreads();

#pragma unroll 4
    for (int64_t t0 = from; t0 < to; t0 += 32) {
        const int64_t t = t0 + lane, y = t < to ? a.tokens[t] : -1;
        const bool in = y >= lo && y < hi;
        const unsigned ours = __ballot_sync(~0u, in);
        if (!ours) continue;
        if (in) {
            const unsigned same = __match_any_sync(ours, (int)(y - lo));
            const int32_t place = mine[y - lo] + __popc(same & ((1u << lane) - 1));
            __syncwarp(ours);
            if ((same >> lane) == 1) mine[y - lo] = place + 1;  // the last of them
            a.position[place] = (int32_t)t;
            a.token[place] = (int32_t)y;
        }
        __syncwarp();
    }
    if (a.zero)
        for (int64_t v = lo + warp; v < hi; v += kSortWarps)
            if (total[v - lo] == 0) zero_bytes(a.zero + v * a.stride_bytes, a.row_bytes, a.element, lane);
}

// ---------------------------------------------------------------------------------------
// Backward, second kernel: the order is cut into blocks of `block` positions; a warp adds up one slice of
// a block's rows, run by run. A token's run that lies in one block is written at once; one that
// goes on in others leaves its part in the workspace, and the warp that ends last adds the parts up, in
// their order: first those within kGroup blocks, then the groups'. So a token that is all of the batch
// is as well spread over the GPU as one that occurs twice.
// ---------------------------------------------------------------------------------------
constexpr int kGroup = 32;  // blocks
constexpr int kAhead = 8;   // rows of a warp on their way at a time

struct SumArgs {
    const int32_t *position, *token, *begin, *count;
    const int64_t* live;
    float *part, *group;                   // [2 * blocks][width], [2 * groups][width]
    uint32_t *part_done, *group_done;      // [2 * blocks][slices], [2 * groups][slices]
    int64_t dim, width, ldh, ldw, slices, units;
    int block;
    float scale;
    int accumulate;
};

// The lane's numbers of one part.
template <class T, bool VEC>
__device__ __forceinline__ void put_part(float* row, int64_t slice, int lane, int64_t dim, const float* f) {
    lane_store<T, float, VEC>(row, slice, lane, dim, f);
}

// The sum of parts: first, then every other from `next` on, `n` in all, each `step` floats behind the last.
template <class T, bool VEC>
__device__ __forceinline__ void add_parts(const float* first, const float* next, int64_t n, int64_t step, int64_t slice, int lane, int64_t dim,
                                          float* f) {
    constexpr int P = kVec<T>;
#pragma unroll
    for (int i = 0; i < P; ++i) f[i] = 0.0f;
    for (int64_t k = 0; k < n; k += 4) {
        float x[4][P];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t at = element<T, VEC>(slice, lane, i);
                x[u][i] = k + u < n && at < dim ? __ldcg((k + u == 0 ? first : next + (k + u - 1) * step) + at) : 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] += x[u][i];
    }
}

// Counts this warp among those that have written their part; true for the last of n, to which all
// parts are then visible.
__device__ __forceinline__ bool last_of(uint32_t* done, uint32_t n, int lane) {
    __threadfence();
    __syncwarp();
    uint32_t before = 0;
    if (lane == 0) before = atomicAdd(done, 1u);
    before = __shfl_sync(~0u, before, 0);
    __threadfence();
    return before == n - 1;
}

template <class T, class O, bool VEC>
__global__ void __launch_bounds__(kEmbedThreads) k_embed_sums(const SumArgs a, const T* dh, O* dw) {
    constexpr int P = kVec<T>;
    wait_for_kernel_before();
    let_next_kernel_start();
    const int lane = threadIdx.x & 31;
    const int64_t live = *a.live, step = (int64_t)gridDim.x * (kEmbedThreads / 32);
    auto write = [&](int64_t v, int64_t slice, float* f) {
#pragma unroll
        for (int i = 0; i < P; ++i) f[i] *= a.scale;
        O* row = dw + v * a.ldw;
        if (a.accumulate) {
            float old[P];
            lane_load<T, O, VEC>(row, slice, lane, a.dim, old);
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] += old[i];
        }
        lane_store<T, O, VEC>(row, slice, lane, a.dim, f);
    };
    for (int64_t unit = (int64_t)blockIdx.x * (kEmbedThreads / 32) + (threadIdx.x >> 5); unit < a.units; unit += step) {
        const int64_t b = unit / a.slices, slice = unit % a.slices, first = b * a.block;
        if (first >= live) return;
        const int n = (int)min((int64_t)a.block, live - first);
        const int32_t pos = lane < n ? a.position[first + lane] : 0, tok = lane < n ? a.token[first + lane] : -1;
        const int32_t left = first > 0 ? a.token[first - 1] : -1, right = first + n < live ? a.token[first + n] : -1;
        float sum[P];
        int run = 0;  // where the run at hand begins
#pragma unroll
        for (int i = 0; i < P; ++i) sum[i] = 0.0f;
        for (int k = 0; k < n; k += kAhead) {
            LaneRow<T, VEC> r[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int32_t p = __shfl_sync(~0u, pos, (k + u) & 31);
                if (k + u < n) r[u].load(dh + p * a.ldh, slice, lane, a.dim);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int32_t y = __shfl_sync(~0u, tok, (k + u) & 31), after = __shfl_sync(~0u, tok, (k + u + 1) & 31);
                if (k + u >= n) continue;
                float f[P];
                r[u].to(f);
#pragma unroll
                for (int i = 0; i < P; ++i) sum[i] += f[i];
                const bool ends = k + u == n - 1;
                if (!ends && after == y) continue;
                const bool from_left = run == 0 && left == y, to_right = ends && right == y;
                if (!from_left && !to_right) {
                    write(y, slice, sum);
                } else {
                    put_part<T, VEC>(a.part + (2 * b + (from_left ? 0 : 1)) * a.width, slice, lane, a.dim, sum);
                    // the blocks of this run, all of them and those of this block's group
                    const int64_t begin = a.begin[y], b0 = begin / a.block, b1 = (begin + a.count[y] - 1) / a.block;
                    const int64_t g = b / kGroup, from = max(b0, g * kGroup), to = min(b1, (g + 1) * kGroup - 1);
                    const int64_t slot = 2 * from + (from == b0 ? 1 : 0);
                    if (last_of(a.part_done + slot * a.slices + slice, (uint32_t)(to - from + 1), lane)) {
                        add_parts<T, VEC>(a.part + slot * a.width, a.part + 2 * (from + 1) * a.width, to - from + 1, 2 * a.width, slice, lane, a.dim,
                                          sum);
                        const int64_t g0 = b0 / kGroup, g1 = b1 / kGroup;
                        if (g0 == g1) {
                            write(y, slice, sum);
                        } else {
                            put_part<T, VEC>(a.group + (2 * g + (g == g0 ? 1 : 0)) * a.width, slice, lane, a.dim, sum);
                            if (last_of(a.group_done + (2 * g0 + 1) * a.slices + slice, (uint32_t)(g1 - g0 + 1), lane)) {
                                add_parts<T, VEC>(a.group + (2 * g0 + 1) * a.width, a.group + 2 * (g0 + 1) * a.width, g1 - g0 + 1, 2 * a.width, slice,
                                                  lane, a.dim, sum);
                                write(y, slice, sum);
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < P; ++i) sum[i] = 0.0f;
                run = k + u + 1;
            }
        }
    }
}

// ---------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------
constexpr int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

template <class F>
int by_type(int32_t type, F f) {
    if (type == ZERO_T_BF16) return f(__nv_bfloat16());
    if (type == ZERO_T_FP16) return f(__half());
    return f(float());
}

// Whether rows of `ld` elements at p may be read and written 16 bytes of T (P elements) at a time.
bool vector_rows(const void* p, int64_t ld, int64_t dim, int32_t type, int64_t elements) {
    const int64_t bytes = std::min<int64_t>(16, elements * type_size(type));
    return dim % elements == 0 && aligned(p, bytes) && ld * type_size(type) % bytes == 0;
}

bool matrix_ok(int64_t rows, int64_t dim, int64_t ld) {
    return dim >= 1 && dim <= (1 << 30) && ld >= dim && ld <= INT64_MAX / 8 / std::max<int64_t>(rows, 1);
}

int check_embed(int64_t rows, int64_t vocab, double scale) {
    return rows < 0 || rows > INT32_MAX || vocab < 1 || vocab > (1 << 30) || !std::isfinite((float)scale) ? ZERO_ERR_INVALID_ARG : ZERO_OK;
}

// Positions of a block: 32, or 8 where so few blocks would not fill the GPU. Of 768 bf16 numbers (three
// slices) 512 positions are 48 warps in blocks of 32 and 192 in blocks of 8.
int block_of(int64_t rows) { return rows <= 4096 ? 8 : 32; }

// The backward's workspace.
struct EmbedSpace {
    int64_t blocks, groups, slices, width;
    int64_t live, position, token, begin, count, counters, n_counters, part, group, bytes;

    EmbedSpace(int64_t rows, int64_t vocab, int64_t dim, int64_t element) {
        blocks = (rows + block_of(rows) - 1) / block_of(rows);
        groups = (blocks + kGroup - 1) / kGroup;
        const int64_t per = 32 * (16 / element);
        slices = (dim + per - 1) / per;
        width = up(dim, 8);
        int64_t at = 16;
        live = 0;
        auto take = [&](int64_t n) {
            const int64_t here = at;
            at += up(n, 16);
            return here;
        };
        position = take(4 * rows);
        token = take(4 * rows);
        begin = take(4 * vocab);
        count = take(4 * vocab);
        n_counters = 2 * (blocks + groups) * slices;
        counters = take(4 * n_counters);
        part = take(4 * 2 * blocks * width);
        group = take(4 * 2 * groups * width);
        bytes = at;
    }
};

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" int zero_embedding(const zero_embed* x, void* out, int64_t ld_out, void* stream) {
    if (!x || !type_ok(x->type) || check_embed(x->rows, x->vocab, x->scale) || !matrix_ok(x->vocab, x->dim, x->ld_weight) ||
        !matrix_ok(x->rows, x->dim, ld_out))
        return ZERO_ERR_INVALID_ARG;
    if (x->rows == 0) return ZERO_OK;
    CallDevice d(out, stream);
    d.need(x->weight, type_size(x->type));
    d.need(x->tokens, 8);
    d.need(out, type_size(x->type));
    if (d.rc) return d.rc;
    const int sms = d.sm_count();
    return by_type(x->type, [&](auto tag) {
        using T = decltype(tag);
        constexpr int P = kVec<T>;
        const int64_t slices = (x->dim + 32 * P - 1) / (32 * P), parts = (slices + kRowSlices - 1) / kRowSlices;
        const bool vec = vector_rows(x->weight, x->ld_weight, x->dim, x->type, P) && vector_rows(out, ld_out, x->dim, x->type, P);
        const int64_t ctas = std::min((x->rows * parts + kEmbedThreads / 32 - 1) / (kEmbedThreads / 32), (int64_t)sms * 1024);
        return launch_linked(vec ? k_embed<T, true> : k_embed<T, false>, (unsigned)ctas, kEmbedThreads, 0, 1, (cudaStream_t)stream, (const T*)x->weight,
                             x->ld_weight, x->tokens, x->rows, x->vocab, x->dim, (float)x->scale, (T*)out, ld_out, parts);
    });
}

extern "C" int64_t zero_embedding_backward_workspace(int64_t rows, int64_t vocab, int64_t dim, int32_t type) {
    if (check_embed(rows, vocab, 1.0) || !type_ok(type) || !matrix_ok(std::max(rows, vocab), dim, dim)) return -1;
    return EmbedSpace(rows, vocab, dim, type_size(type)).bytes;
}

extern "C" int zero_embedding_backward(const zero_embed_grad* x, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!x || !type_ok(x->type) || !type_ok(x->out_type) || check_embed(x->rows, x->vocab, x->scale) || x->accumulate < 0 || x->accumulate > 1 ||
        !matrix_ok(x->rows, x->dim, x->ld_hidden) || !matrix_ok(std::max(x->rows, x->vocab), x->dim, x->dim) ||
        !matrix_ok(x->vocab, x->dim, x->ld_weight))
        return ZERO_ERR_INVALID_ARG;
    const EmbedSpace s(x->rows, x->vocab, x->dim, type_size(x->type));
    if (workspace_bytes < s.bytes) return ZERO_ERR_SIZE_MISMATCH;
    if (x->rows == 0 && x->accumulate) return ZERO_OK;
    CallDevice d(x->dweight, stream);
    d.need(x->dweight, type_size(x->out_type));
    d.need(workspace, 16);
    if (x->rows > 0) {
        d.need(x->tokens, 8);
        d.need(x->dhidden, type_size(x->type));
    }
    if (d.rc) return d.rc;
    const int sms = d.sm_count();
    uint8_t* ws = (uint8_t*)workspace;
    SortArgs a;
    a.tokens = x->tokens;
    a.rows = x->rows;
    a.vocab = x->vocab;
    const int64_t owners = std::max<int64_t>(sms, (x->vocab + kSortWidth - 1) / kSortWidth);
    a.width = (int)((x->vocab + owners - 1) / owners);
    a.position = (int32_t*)(ws + s.position);
    a.token = (int32_t*)(ws + s.token);
    a.begin = (int32_t*)(ws + s.begin);
    a.count = (int32_t*)(ws + s.count);
    a.live = (int64_t*)(ws + s.live);
    a.counters = (uint32_t*)(ws + s.counters);
    a.n_counters = s.n_counters;
    a.zero = x->accumulate ? nullptr : (uint8_t*)x->dweight;
    a.element = (int)type_size(x->out_type);
    a.row_bytes = x->dim * a.element;
    a.stride_bytes = x->ld_weight * a.element;
    const size_t smem = (size_t)4 * kSortWarps * a.width;
    const cudaError_t e = cudaFuncSetAttribute(k_embed_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kSortWarps * kSortWidth);
    if (e != cudaSuccess) return record_cuda_error(e);
    cudaStream_t st = (cudaStream_t)stream;
    const int64_t grid = (x->vocab + a.width - 1) / a.width;
    int rc = launch_linked(k_embed_sort, (unsigned)grid, kSortThreads, smem, 1, st, a);
    if (rc || x->rows == 0) return rc;
    SumArgs u;
    u.position = a.position;
    u.token = a.token;
    u.begin = a.begin;
    u.count = a.count;
    u.live = a.live;
    u.part = (float*)(ws + s.part);
    u.group = (float*)(ws + s.group);
    u.part_done = a.counters;
    u.group_done = a.counters + 2 * s.blocks * s.slices;
    u.dim = x->dim;
    u.width = s.width;
    u.ldh = x->ld_hidden;
    u.ldw = x->ld_weight;
    u.slices = s.slices;
    u.units = s.blocks * s.slices;
    u.block = block_of(x->rows);
    u.scale = (float)x->scale;
    u.accumulate = x->accumulate;
    const int64_t ctas = std::min((u.units + kEmbedThreads / 32 - 1) / (kEmbedThreads / 32), (int64_t)sms * 1024);
    return by_type(x->type, [&](auto tag) {
        using T = decltype(tag);
        return by_type(x->out_type, [&](auto out) {
            using O = decltype(out);
            const bool vec = vector_rows(x->dhidden, x->ld_hidden, x->dim, x->type, kVec<T>) &&
                             vector_rows(x->dweight, x->ld_weight, x->dim, x->out_type, kVec<T>);
            return launch_linked(vec ? k_embed_sums<T, O, true> : k_embed_sums<T, O, false>, (unsigned)ctas, kEmbedThreads, 0, 1, st, u,
                                 (const T*)x->dhidden, (O*)x->dweight);
        });
    });
}
