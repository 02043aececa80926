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

#include <cooperative_groups.h>

#include "zero_host.h"
#include "zero_softmax.cuh"

namespace zg {
namespace {

namespace cg = cooperative_groups;

constexpr int kEmbedThreads = 256;

// A row's slice of 32 lanes with 16 bytes of T each: lane's elements are kVec<T> neighbours (VEC: the
// addresses are aligned for it) or every 32nd.
template <class T, bool VEC>
__device__ __forceinline__ int64_t element(int64_t slice, int lane, int i) {
    constexpr int P = kVec<T>;
    return VEC ? (slice * 32 + lane) * P + i : slice * 32 * P + 32 * i + lane;
}

// This lane's elements of a row; 0 past its end, which is `left` elements from its first one. A row is read once: past L1.
template <class T, bool VEC>
struct LaneRow {
    uint4 v;
    T e[VEC ? 1 : kVec<T>];

    __device__ __forceinline__ void load(const T* mine, bool there, int64_t left) {
        if (VEC) {
            v = make_uint4(0, 0, 0, 0);
            if (there) v = load_once(reinterpret_cast<const uint4*>(mine));
        } else {
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) e[VEC ? 0 : i] = 32 * i < left ? mine[32 * i] : narrow<T>(0.0f);
        }
    }
    // Elements 2i and 2i + 1 as fp32.
    __device__ __forceinline__ uint64_t two(int i) const {
        return VEC ? widen2<T>(v, i) : pack2(widen(e[VEC ? 0 : 2 * i]), widen(e[VEC ? 0 : 2 * i + 1]));
    }
};

// kVec<T> numbers of this lane to a row of another type, and what such a row holds.
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
struct LaneOld {
    static constexpr int P = kVec<T>;
    alignas(P * sizeof(O) < 16 ? P * sizeof(O) : 16) O o[P];

    __device__ __forceinline__ void load(const O* mine, bool there, int64_t left) {
        if constexpr (VEC) {
            if (there) *this = *reinterpret_cast<const LaneOld*>(mine);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (32 * i < left) o[i] = mine[32 * i];
        }
    }
};

// ---------------------------------------------------------------------------------------
// Forward: a warp per kRowSlices slices of a token's row. 16384 x 2048 bf16 11.6 us, bound by memory (12.8 us from HBM alone; the
// matrix' frequent rows stay in L2); one token 1.8 us.
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
        for (int u = 0; u < kRowSlices; ++u) {
            const int64_t at = element<T, VEC>(first + u, lane, 0);
            r[u].load(weight + (there ? y * ldw : 0) + at, there && at < dim, there ? dim - at : 0);
        }
#pragma unroll
        for (int u = 0; u < kRowSlices; ++u) {
            float f[kVec<T>];
#pragma unroll
            for (int i = 0; i < kVec<T>; i += 2) {
                const float2 x = unpack2(r[u].two(i / 2));
                f[i] = there ? x.x * scale : y < 0 ? 0.0f : NAN;
                f[i + 1] = there ? x.y * scale : y < 0 ? 0.0f : NAN;
            }
            lane_store<T, T, VEC>(out + t * ldo, first + u, lane, dim, f);
        }
    }
}

// ---------------------------------------------------------------------------------------
// Backward, first kernel: positions in the order of their tokens. A cluster owns the tokens
// [c * width, (c + 1) * width) and reads all positions twice (from L2 but for the first one), its CTAs a
// share each: once to count its own tokens and those below them, which is where its part of the order
// begins, and once to write its positions there. A warp takes a contiguous share of the positions with
// counters of its own, and lanes of one token rank themselves, so the order is that of the positions, and
// equal calls give equal bits. 65536 positions take 18 us, a chain of latencies: 33 clusters read 35 MB of positions from L2, which
// would be 3 us at its rate, between rounds over 32 counters a token and their barriers; each CTA for itself 31.
// ---------------------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortWidth = 1600;  // most tokens of a cluster: 205 KB of counters

struct SortArgs {
    const int64_t* tokens;
    int64_t rows, vocab;
    int width, size;            // tokens and CTAs of a cluster
    int32_t *position, *token;  // [rows] in order
    int32_t *begin, *count;     // [vocab] a token's place and number in the order
    int64_t* live;              // [1] length of the order
    uint32_t* counters;         // to be zeroed
    int64_t n_counters;
};

__global__ void __launch_bounds__(kSortThreads) k_embed_sort(const SortArgs a) {
    extern __shared__ int32_t counts[];  // [kSortWarps][width]
    __shared__ int32_t warp_sum[kSortWarps];
    __shared__ int32_t mine_of[kSortWidth];  // of the CTA's share
    __shared__ uint32_t below_mine;
    cg::cluster_group cl = cg::this_cluster();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = (int)(blockIdx.x % a.size);
    const int64_t lo = (int64_t)(blockIdx.x / a.size) * a.width, hi = min(lo + a.width, a.vocab);
    int32_t* mine = counts + warp * a.width;
    for (int b = lane; b < a.width; b += 32) mine[b] = 0;
    if (threadIdx.x == 0) below_mine = 0;
    wait_for_kernel_before();
    let_next_kernel_start();
    for (int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; i < a.n_counters; i += (int64_t)gridDim.x * kSortThreads) a.counters[i] = 0;
    __syncthreads();

    const int64_t share = ((a.rows + kSortWarps * a.size - 1) / (kSortWarps * a.size) + 31) / 32 * 32;
    const int64_t from = min(share * (rank * kSortWarps + warp), a.rows), to = min(from + share, a.rows);
    uint32_t below = 0;
#pragma unroll 8
    for (int64_t t = from + lane; t < to; t += 32) {
        const int64_t y = a.tokens[t];
        below += y >= 0 && y < lo;
        if (y >= lo && y < hi) atomicAdd(mine + (y - lo), 1);
    }
    below = __reduce_add_sync(~0u, below);
    if (lane == 0 && below) atomicAdd(&below_mine, below);
    __syncthreads();
    for (int b = threadIdx.x; b < a.width; b += kSortThreads) {
        int32_t n = 0;
        for (int w = 0; w < kSortWarps; ++w) n += counts[w * a.width + b];
        mine_of[b] = n;
    }
    if (a.size > 1) cl.sync();
    else __syncthreads();

    // Thread b: tokens lo + 2b and the next. Their number, their places in the order, and every warp's in those.
    uint32_t below_all = 0;
    for (int r = 0; r < a.size; ++r) below_all += r == rank ? below_mine : *cl.map_shared_rank(&below_mine, r);
    int32_t n[2] = {0, 0}, before[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int b = 2 * threadIdx.x + i;
        if (b >= a.width) continue;
        for (int r = 0; r < a.size; ++r) {
            const int32_t x = r == rank ? mine_of[b] : cl.map_shared_rank(mine_of, r)[b];
            n[i] += x;
            if (r < rank) before[i] += x;
        }
    }
    int32_t scan = n[0] + n[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(~0u, scan, o);
        if (lane >= o) scan += x;
    }
    if (lane == 31) warp_sum[warp] = scan;
    if (a.size > 1) cl.sync();  // no CTA leaves or goes on while another reads its counts
    else __syncthreads();
    int32_t at = __reduce_add_sync(~0u, lane < warp ? warp_sum[lane] : 0) + (int32_t)below_all + scan - n[0] - n[1];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int b = 2 * threadIdx.x + i;
        if (b < a.width) {
            if (rank == 0 && lo + b < hi) {
                a.begin[lo + b] = at;
                a.count[lo + b] = n[i];
            }
            int32_t place = at + before[i];
            for (int w = 0; w < kSortWarps; ++w) {
                const int32_t c = counts[w * a.width + b];
                counts[w * a.width + b] = place;
                place += c;
            }
        }
        at += n[i];
    }
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == kSortThreads - 1) *a.live = at;
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
}

// ---------------------------------------------------------------------------------------
// Backward, second kernel: the order is cut into blocks of `block` positions; a warp adds up one slice of
// a block's rows, run by run. A token's run that lies in one block is written at once; one that
// goes on in others leaves its part in the workspace, and the warp that ends last adds the parts up, in
// their order: first those within kGroup blocks, then the groups'. So a token that is all of the batch
// is as well spread over the GPU as one that occurs twice. 65536 rows of 2048 bf16, tokens as text has them, added to a matrix:
// 97 us with the sort, 60% of the copy peak on 398 MB; rows in registers, eight ahead and then none, 140. The rest is the warps'
// first rows and the joins of runs. Rows of no token are zeroed by warps beside these: 16384 rows of 2048 fp32 into 412 MB 89 us with
// the sort, 85% of the copy peak; zeroed beside the sort 98.
// ---------------------------------------------------------------------------------------
constexpr int kGroup = 32;  // blocks
constexpr int kAhead = 8;        // rows of a warp on their way at a time
constexpr int kLoose = 4;        // the same where they are loaded element by element
constexpr int kBlockMost = 128;  // positions of a block
constexpr int kChain = 32;       // of which so many are added one to another
constexpr int64_t kZeroBytes = 16384;  // of the rows of no token that a warp looks after

struct SumArgs {
    const int32_t *position, *token, *begin, *count;
    const int64_t* live;
    float *part, *group;                   // [2 * blocks][width], [2 * groups][width]
    uint32_t *part_done, *group_done;      // [2 * blocks][slices], [2 * groups][slices]
    int64_t dim, width, ldh, ldw, slices, units;
    int block;
    float scale;
    // the rows of no token, `zero_rows` to a unit behind the blocks' units
    uint8_t* zero;  // the matrix, or nullptr where it is added to
    int64_t vocab, zero_units, row_bytes, stride_bytes;
    int zero_rows, element;
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
// Zeros into those of a unit's rows that have no token.
__device__ __forceinline__ void zero_unit(const SumArgs& a, int64_t unit, int lane) {
    const int64_t first = unit * a.zero_rows;
    unsigned none = __ballot_sync(~0u, lane < a.zero_rows && first + lane < a.vocab && a.count[first + lane] == 0);
    for (; none; none &= none - 1) zero_bytes(a.zero + (first + __ffs(none) - 1) * a.stride_bytes, a.row_bytes, a.element, lane);
}

// The lane's numbers of one part.
template <class T, bool VEC>
__device__ __forceinline__ void put_part(float* row, int64_t slice, int lane, int64_t dim, const uint64_t* sum) {
    float f[kVec<T>];
#pragma unroll
    for (int i = 0; i < kVec<T>; i += 2) {
        const float2 x = unpack2(sum[i / 2]);
        f[i] = x.x;
        f[i + 1] = x.y;
    }
    lane_store<T, float, VEC>(row, slice, lane, dim, f);
}

// The sum of parts: first, then every other from `next` on, `n` in all, each `step` floats behind the last.
template <class T, bool VEC>
__device__ __forceinline__ void add_parts(const float* first, const float* next, int64_t n, int64_t step, int64_t slice, int lane, int64_t dim,
                                          uint64_t* f) {
    constexpr int P = kVec<T>, kParts = 4;
#pragma unroll
    for (int i = 0; i < P / 2; ++i) f[i] = 0;
    for (int64_t k = 0; k < n; k += kParts) {
        float x[kParts][P];
#pragma unroll
        for (int u = 0; u < kParts; ++u) {
            const float* p = k + u == 0 ? first : next + (k + u - 1) * step;
            if constexpr (VEC) {
                const int64_t at = element<T, VEC>(slice, lane, 0);
#pragma unroll
                for (int i = 0; i < P; i += 4) {
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (k + u < n && at < dim) v = __ldcg(reinterpret_cast<const float4*>(p + at + i));
                    x[u][i] = v.x;
                    x[u][i + 1] = v.y;
                    x[u][i + 2] = v.z;
                    x[u][i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const int64_t at = element<T, VEC>(slice, lane, i);
                    x[u][i] = k + u < n && at < dim ? __ldcg(p + at) : 0.0f;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kParts; ++u)
#pragma unroll
            for (int i = 0; i < P; i += 2) f[i / 2] = add2(f[i / 2], pack2(x[u][i], x[u][i + 1]));
    }
}

// Counts this warp among those that have written their part; true for the last of n, to which all
// parts are then visible (read past L1).
__device__ __forceinline__ bool last_of(uint32_t* done, uint32_t n, int lane) {
    __syncwarp();
    uint32_t before = 0;
    if (lane == 0) asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(done) : "memory");
    before = __shfl_sync(~0u, before, 0);
    __syncwarp();
    return before == n - 1;
}

// A lane's sums of a run's earlier chains in a block. In shared memory, where registers for them would cost an SM one of its CTAs
// (16384 x 767 fp32 55 us against 51); in registers, where shared memory would (65536 x 2048 bf16 added to fp32 142 against 126).
template <int N, bool SHARED>
struct Chains {
    struct Room {
        uint64_t at[N][32];
    };
    uint64_t (*const at)[32];
    __device__ __forceinline__ Chains(Room* of) : at(of[threadIdx.x >> 5].at) {}
    __device__ __forceinline__ uint64_t& operator[](int i) { return at[i][threadIdx.x & 31]; }
};
template <int N>
struct Chains<N, false> {
    struct Room {};
    uint64_t v[N];
    __device__ __forceinline__ Chains(Room*) {}
    __device__ __forceinline__ uint64_t& operator[](int i) { return v[i]; }
};
template <class T, bool VEC, bool ADD>
using ChainsOf = Chains<kVec<T> / 2, !(VEC && ADD)>;

// One warp's work on the runs of a block: what both kernels below do with the rows that they bring.
template <class T, class O, bool VEC, bool ADD>
struct Runs {
    static constexpr int P = kVec<T>;
    const SumArgs& a;
    O* const dw;
    const int lane;
    int64_t b, slice, first;
    int n;
    int32_t left;
    uint64_t sum[P / 2];
    ChainsOf<T, VEC, ADD> chains;
    bool chained;           // whether they hold anything
    bool started, carried;  // a run has ended in this block; one that came from the left has
    int32_t last;           // the token of a run that goes on to the right

    __device__ __forceinline__ Runs(const SumArgs& a, O* dw, typename ChainsOf<T, VEC, ADD>::Room* room) : a(a), dw(dw), lane(threadIdx.x & 31), chains(room) {}

    // False: no such block. Rows of `live` positions.
    __device__ __forceinline__ bool begin(int64_t unit, int64_t live) {
        b = unit / a.slices;
        slice = unit % a.slices;
        first = b * a.block;
        if (first >= live) return false;
        n = (int)min((int64_t)a.block, live - first);
        left = first > 0 ? a.token[first - 1] : -1;
        started = carried = chained = false;
        last = -1;
        clear();
        return true;
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < P / 2; ++i) sum[i] = 0;
    }
    // Every kChain positions: roundings grow with the additions that a sum goes through.
    __device__ __forceinline__ void end_chain() {
#pragma unroll
        for (int i = 0; i < P / 2; ++i) chains[i] = chained ? add2(chains[i], sum[i]) : sum[i];
        chained = true;
        clear();
    }
    // Before the few rows among which the run ends.
    __device__ __forceinline__ void add_chains(bool ends) {
        if (!chained || !ends) return;
        chained = false;
#pragma unroll
        for (int i = 0; i < P / 2; ++i) sum[i] = add2(chains[i], sum[i]);
    }
    __device__ __forceinline__ O* at(int64_t v) const { return dw + v * a.ldw + element<T, VEC>(slice, lane, 0); }
    __device__ __forceinline__ int64_t in_row() const { return a.dim - element<T, VEC>(slice, lane, 0); }
    __device__ __forceinline__ void write(int64_t v, const uint64_t* total, const LaneOld<T, O, VEC>& old) const {
        float f[P];
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            const float2 x = unpack2(total[i / 2]);
            f[i] = ADD ? fmaf(x.x, a.scale, widen(old.o[i])) : x.x * a.scale;
            f[i + 1] = ADD ? fmaf(x.y, a.scale, widen(old.o[i + 1])) : x.y * a.scale;
        }
        lane_store<T, O, VEC>(dw + v * a.ldw, slice, lane, a.dim, f);
    }
    // The run of token y ends here.
    __device__ __forceinline__ void end(int32_t y, const LaneOld<T, O, VEC>& old) {
        if (!started && left == y) {
            carried = true;
            put_part<T, VEC>(a.part + 2 * b * a.width, slice, lane, a.dim, sum);
        } else {
            write(y, sum, old);
        }
        started = true;
        clear();
    }
    // What goes on in other blocks: a run that came from the left, then one that goes on to the right.
    __device__ __forceinline__ void finish() {
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
            if (side == 0 ? !carried : last < 0) continue;
            const int32_t y = side == 0 ? left : last;
            const int64_t part = 2 * b + (side == 0 || (!started && left == y) ? 0 : 1);
            if (side == 1) {
                add_chains(true);
                put_part<T, VEC>(a.part + part * a.width, slice, lane, a.dim, sum);
            }
            // the blocks of this run, all of them and those of this block's group
            const int64_t begin = a.begin[y], b0 = begin / a.block, b1 = (begin + a.count[y] - 1) / a.block;
            const int64_t g = b / kGroup, from = max(b0, g * kGroup), to = min(b1, (g + 1) * kGroup - 1);
            const int64_t slot = 2 * from + (from == b0 ? 1 : 0);
            if (!last_of(a.part_done + slot * a.slices + slice, (uint32_t)(to - from + 1), lane)) continue;
            uint64_t all[P / 2];
            add_parts<T, VEC>(a.part + slot * a.width, a.part + 2 * (from + 1) * a.width, to - from + 1, 2 * a.width, slice, lane, a.dim, all);
            const int64_t g0 = b0 / kGroup, g1 = b1 / kGroup;
            if (g0 != g1) {
                put_part<T, VEC>(a.group + (2 * g + (g == g0 ? 1 : 0)) * a.width, slice, lane, a.dim, all);
                if (!last_of(a.group_done + (2 * g0 + 1) * a.slices + slice, (uint32_t)(g1 - g0 + 1), lane)) continue;
                add_parts<T, VEC>(a.group + (2 * g0 + 1) * a.width, a.group + 2 * (g0 + 1) * a.width, g1 - g0 + 1, 2 * a.width, slice, lane, a.dim, all);
            }
            LaneOld<T, O, VEC> old;
            if (ADD) old.load(at(y), in_row() > 0, in_row());
            write(y, all, old);
        }
    }
};

__device__ __forceinline__ void copy_16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_8(void* to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

// Rows that can be read 16 bytes at a time: a ring in shared memory keeps kAhead of them on their way, and with them what the
// runs that end are added to. A lane reads what it has copied itself, so no warp waits for another.
template <class T, class O, bool ADD>
struct EmbedRing {
    uint4 row[kAhead][32];
    LaneOld<T, O, true> old[ADD ? kAhead : 1][32];
    int64_t offset[kBlockMost + kAhead];  // of the rows; behind the last one that one again
    int32_t token[kBlockMost];
    uint32_t ends[kBlockMost / 32 + 2];   // whether a run ends there
};

template <class T, class O, bool ADD>
__global__ void __launch_bounds__(kEmbedThreads, !ADD && sizeof(T) == 4 ? 4 : 0) k_embed_sums(const SumArgs a, const T* dh, O* dw) {
    extern __shared__ __align__(16) uint8_t smem[];
    using Ring = EmbedRing<T, O, ADD>;
    using Old = LaneOld<T, O, true>;
    Ring& ring = reinterpret_cast<Ring*>(smem)[threadIdx.x >> 5];
    wait_for_kernel_before();
    let_next_kernel_start();
    __shared__ typename ChainsOf<T, true, ADD>::Room room[kEmbedThreads / 32];
    Runs<T, O, true, ADD> run(a, dw, room);
    const int lane = run.lane;
    const int64_t live = *a.live, step = (int64_t)gridDim.x * (kEmbedThreads / 32);
    for (int64_t unit = (int64_t)blockIdx.x * (kEmbedThreads / 32) + (threadIdx.x >> 5); unit < a.units + a.zero_units; unit += step) {
        if (unit >= a.units) {
            zero_unit(a, unit - a.units, lane);
            continue;
        }
        if (!run.begin(unit, live)) continue;
        const int n = run.n;
        for (int i0 = 0; i0 < n + kAhead; i0 += 32) {
            const int i = i0 + lane;
            int32_t tok = -1, after = -1;
            if (i < n + kAhead) ring.offset[i] = a.position[run.first + min(i, n - 1)] * a.ldh;
            if (i < n) {
                ring.token[i] = tok = a.token[run.first + i];
                if (run.first + i + 1 < live) after = a.token[run.first + i + 1];
            }
            const unsigned ends = __ballot_sync(~0u, i < n && after != tok);
            if (lane == 0) {
                ring.ends[i0 / 32] = ends;
                ring.ends[i0 / 32 + 1] = 0;
            }
            if (i == n - 1) run.last = after == tok ? tok : -1;
        }
        run.last = __shfl_sync(~0u, run.last, (n - 1) & 31);
        __syncwarp();
        const bool there = run.in_row() > 0;
        const T* mine = dh + (there ? element<T, true>(run.slice, lane, 0) : 0);  // a lane past the row's end brings its first numbers
        auto bring = [&](int e, int slot, bool ends) {
            copy_16(&ring.row[slot][lane], mine + ring.offset[e]);
            if (ADD && ends && there) {
                uint8_t* to = reinterpret_cast<uint8_t*>(&ring.old[ADD ? slot : 0][lane]);
                const uint8_t* from = reinterpret_cast<const uint8_t*>(run.at(ring.token[e]));
                if (sizeof(Old) == 8) copy_8(to, from);
#pragma unroll
                for (int i = 0; i + 16 <= (int)sizeof(Old); i += 16) copy_16(to + i, from + i);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        static_assert(kAhead == 8, "a power of two that divides 32");
#pragma unroll
        for (int e = 0; e < kAhead - 1; ++e) bring(e, e, ring.ends[0] >> e & 1);
        for (int e0 = 0; e0 < n; e0 += kAhead) {
            if (e0 > 0 && e0 % kChain == 0) run.end_chain();
            const unsigned ends = __funnelshift_r(ring.ends[e0 / 32], ring.ends[e0 / 32 + 1], e0 & 31);
            run.add_chains(ends & ((1u << kAhead) - 1));
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (e0 + u >= n) break;
                bring(e0 + u + kAhead - 1, (u + kAhead - 1) % kAhead, ends >> (u + kAhead - 1) & 1);
                asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
                const uint4 v = ring.row[u][lane];
#pragma unroll
                for (int i = 0; i < kVec<T> / 2; ++i) run.sum[i] = add2(run.sum[i], widen2<T>(v, i));
                if (ends >> u & 1) run.end(ring.token[e0 + u], ring.old[ADD ? u : 0][lane]);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        run.finish();
        __syncwarp();  // the positions are read
    }
}

// Rows of any alignment, kLoose at a time in registers.
template <class T, class O, bool ADD>
__global__ void __launch_bounds__(kEmbedThreads, 2) k_embed_sums_loose(const SumArgs a, const T* dh, O* dw) {
    wait_for_kernel_before();
    let_next_kernel_start();
    __shared__ typename ChainsOf<T, false, ADD>::Room room[kEmbedThreads / 32];
    Runs<T, O, false, ADD> run(a, dw, room);
    const int lane = run.lane;
    const int64_t live = *a.live, step = (int64_t)gridDim.x * (kEmbedThreads / 32);
    for (int64_t unit = (int64_t)blockIdx.x * (kEmbedThreads / 32) + (threadIdx.x >> 5); unit < a.units + a.zero_units; unit += step) {
        if (unit >= a.units) {
            zero_unit(a, unit - a.units, lane);
            continue;
        }
        if (!run.begin(unit, live)) continue;
        const T* mine = dh + element<T, false>(run.slice, lane, 0);
        for (int k0 = 0; k0 < run.n; k0 += kChain) {
            if (k0 > 0) run.end_chain();
            const int m = min(32, run.n - k0);
            const int64_t at = run.first + k0 + lane;
            const int32_t pos = lane < m ? a.position[at] : 0, tok = lane < m ? a.token[at] : -1;
            const int32_t after = lane < m && at + 1 < live ? a.token[at + 1] : -1;
            const unsigned ends = __ballot_sync(~0u, lane < m && after != tok);
            run.last = __shfl_sync(~0u, tok, m - 1);
            if (ends >> (m - 1) & 1) run.last = -1;
            for (int k = 0; k < m; k += kLoose) {
                LaneRow<T, false> r[kLoose];
#pragma unroll
                for (int u = 0; u < kLoose; ++u)  // past the last row the first of all, which is not used
                    r[u].load(mine + __shfl_sync(~0u, pos, k + u) * a.ldh, true, run.in_row());
                run.add_chains(ends >> k & ((1u << kLoose) - 1));
#pragma unroll
                for (int u = 0; u < kLoose; ++u) {
                    if (k + u >= m) break;
#pragma unroll
                    for (int i = 0; i < kVec<T> / 2; ++i) run.sum[i] = add2(run.sum[i], r[u].two(i));
                    if (!(ends >> (k + u) & 1)) continue;
                    const int32_t y = __shfl_sync(~0u, tok, k + u);
                    LaneOld<T, O, false> old;
                    if (ADD) old.load(run.at(y), true, run.in_row());
                    run.end(y, old);
                }
            }
        }
        run.finish();
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

// Positions of a block: as many as leave 4096 warps, 8 to 128. Fewer leave SMs without work, and with more blocks more runs
// are cut: 65536 positions of 2048 bf16 numbers 97 us in blocks of 128 or 64, 104 of 32.
int block_of(int64_t rows, int64_t slices) {
    int block = 8;
    while (block < kBlockMost && rows * slices / (2 * block) >= 4096) block *= 2;
    return block;
}
// Batches from here on have their positions read by a cluster of four CTAs instead of by each (k_embed_sort): 16384 rows of 768 bf16
// 36.3 us against 37.5, 8192 34.5 against 32.6.
constexpr int64_t kSortShared = 16384;

// The backward's workspace.
struct EmbedSpace {
    int block;
    int64_t blocks, groups, slices, width;
    int64_t live, position, token, begin, count, counters, n_counters, part, group, bytes;

    EmbedSpace(int64_t rows, int64_t vocab, int64_t dim, int64_t element) {
        const int64_t per = 32 * (16 / element);
        slices = (dim + per - 1) / per;
        block = block_of(rows, slices);
        blocks = (rows + block - 1) / block;
        groups = (blocks + kGroup - 1) / kGroup;
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
    a.size = x->rows >= kSortShared ? 4 : 1;
    // clusters leave SMs over where a GPU's parts hold no whole one
    const int64_t owners = std::max<int64_t>(a.size > 1 ? sms * 7 / 8 / a.size : sms, (x->vocab + kSortWidth - 1) / kSortWidth);
    a.width = (int)((x->vocab + owners - 1) / owners);
    a.position = (int32_t*)(ws + s.position);
    a.token = (int32_t*)(ws + s.token);
    a.begin = (int32_t*)(ws + s.begin);
    a.count = (int32_t*)(ws + s.count);
    a.live = (int64_t*)(ws + s.live);
    a.counters = (uint32_t*)(ws + s.counters);
    a.n_counters = s.n_counters;
    const size_t smem = (size_t)4 * kSortWarps * a.width;
    const cudaError_t e = cudaFuncSetAttribute(k_embed_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kSortWarps * kSortWidth);
    if (e != cudaSuccess) return record_cuda_error(e);
    cudaStream_t st = (cudaStream_t)stream;
    const int64_t grid = (x->vocab + a.width - 1) / a.width * a.size;
    int rc = launch_linked(k_embed_sort, (unsigned)grid, kSortThreads, smem, a.size, st, a);
    if (rc) return rc;
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
    u.block = s.block;
    u.scale = (float)x->scale;
    u.element = (int)type_size(x->out_type);
    u.row_bytes = x->dim * u.element;
    u.stride_bytes = x->ld_weight * u.element;
    u.zero = x->accumulate ? nullptr : (uint8_t*)x->dweight;
    u.vocab = x->vocab;
    u.zero_rows = (int)std::max<int64_t>(1, std::min<int64_t>(32, kZeroBytes / u.row_bytes));
    u.zero_units = x->accumulate ? 0 : (x->vocab + u.zero_rows - 1) / u.zero_rows;
    const int64_t ctas = std::min((u.units + u.zero_units + kEmbedThreads / 32 - 1) / (kEmbedThreads / 32), (int64_t)sms * 1024);
    return by_type(x->type, [&](auto tag) {
        using T = decltype(tag);
        return by_type(x->out_type, [&](auto out) {
            using O = decltype(out);
            const bool vec = vector_rows(x->dhidden, x->ld_hidden, x->dim, x->type, kVec<T>) &&
                             vector_rows(x->dweight, x->ld_weight, x->dim, x->out_type, kVec<T>);
            if (!vec)
                return launch_linked(x->accumulate ? k_embed_sums_loose<T, O, true> : k_embed_sums_loose<T, O, false>, (unsigned)ctas, kEmbedThreads, 0,
                                     1, st, u, (const T*)x->dhidden, (O*)x->dweight);
            auto* kernel = x->accumulate ? k_embed_sums<T, O, true> : k_embed_sums<T, O, false>;
            const size_t ring = (kEmbedThreads / 32) * (x->accumulate ? sizeof(EmbedRing<T, O, true>) : sizeof(EmbedRing<T, O, false>));
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ring);
            if (e != cudaSuccess) return record_cuda_error(e);
            return launch_linked(kernel, (unsigned)ctas, kEmbedThreads, ring, 1, st, u, (const T*)x->dhidden, (O*)x->dweight);
        });
    });
}
