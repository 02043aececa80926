// zero_linear.cu -- token log-probabilities from hidden states and the vocabulary matrix, with
// no logits in memory, for sm_103a.
//
// logits = hidden weight^T is formed tile by tile by tcgen05 and stays in TMEM; a tile's part
// of each row's softmax sums (zero_softmax.cuh) goes to the workspace, and a second kernel joins
// the parts of a row in their order. Row tiles without a target are left out.

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "zero_host.h"
#include "zero_softmax.cuh"
#include "zero_tcgen05.cuh"

namespace zg {
namespace {

constexpr int kRowsTile = 128;    // tokens of a CTA's tile: the lanes of TMEM
constexpr int kDepth = 64;         // elements of the inner dimension per stage: 128 bytes
constexpr int kEpilogueWarps = 8;  // two for each quarter of the lanes
constexpr int kLinearThreads = 128 + 32 * kEpilogueWarps;
// 384 threads launch with 168 registers each, 64,512 in all: the first warpgroup gives back what
// the two of the epilogue take (128 (56 + 2 x 224) = 64,512).
constexpr int kFewRegisters = 56, kManyRegisters = 224;
static_assert(128 * (kFewRegisters + 2 * kManyRegisters) <= kLinearThreads * 168, "the register split fits the launch");

struct LinearArgs {
    const int64_t* targets;
    float *m, *s, *q;  // [parts, rows]
    float* zy;         // [rows] the target's logit
    int32_t* status;   // [grid of the product] set where a wait gave up
    int32_t* tiles;    // [0]: how many row tiles hold a target, [4...]: those tiles; nullptr: one tile, taken as it is
    int64_t rows, vocab, dim;
    int32_t tile_rows, row_tiles, tile_cols, col_tiles, group, grid;
    int32_t load_rows;  // tokens of a CTA's tile that are loaded: all, or the multiple of 8 that holds the few there are
    Scale k;       // log2(e) / temperature
    float inv_t;   // 1 / temperature
};

// Row tiles with at least one target, in order. One CTA, a warp per tile.
__global__ void __launch_bounds__(1024) k_linear_tiles(const LinearArgs a) {
    __shared__ int32_t any[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    let_next_kernel_start();
    wait_for_kernel_before();
    int32_t n = 0;  // kept by warp 0
    for (int32_t t0 = 0; t0 < a.row_tiles; t0 += 32) {
        const int32_t t = t0 + warp;
        bool mine = false;
        if (t < a.row_tiles)
            for (int i = lane; i < a.tile_rows; i += 32) {
                const int64_t r = (int64_t)t * a.tile_rows + i;
                mine |= r < a.rows && a.targets[r] >= 0;
            }
        mine = __any_sync(~0u, mine);
        if (lane == 0) any[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const unsigned ballot = __ballot_sync(~0u, any[lane] != 0);
            if (any[lane]) a.tiles[4 + n + __popc(ballot & ((1u << lane) - 1))] = t0 + lane;
            n += __popc(ballot);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) a.tiles[0] = n;
}

// Tile `i` of the run: groups of row tiles that stay in L2 while the vocabulary passes by, and
// within a group the row tiles fastest, so that CTAs working side by side share their columns.
__device__ __forceinline__ void tile_of(const LinearArgs& a, int32_t live, int64_t i, int32_t* row, int32_t* col) {
    const int64_t per = (int64_t)a.group * a.col_tiles;
    const int32_t g = (int32_t)(i / per), first = g * a.group;
    const int32_t size = min(a.group, live - first);
    const int64_t in = i - (int64_t)g * per;
    *col = (int32_t)(in / size);
    *row = a.tiles ? a.tiles[4 + first + (int32_t)(in % size)] : 0;
}

// N logits of one row: their sums, in four chains of two numbers to an instruction.
template <bool ENTROPY, int N>
__device__ __forceinline__ RowStat sum_of(const float (&v)[N], Scale k) {
    float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int j = 4; j < N; ++j) top[j & 3] = fmaxf(top[j & 3], v[j]);
    const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    const uint64_t base = pack2(-base_of(m), -base_of(m)), c = pack2(k.c, k.c), lo = pack2(k.lo, k.lo);
    uint64_t s[4], q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = q[i] = pack2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
        const uint64_t t = add2(pack2(v[2 * j], v[2 * j + 1]), base), p = mul2(t, c);
        const float2 d = unpack2(ENTROPY ? p : fma2(t, lo, p));
        const uint64_t e = pack2(pow2(d.x), pow2(d.y));
        s[j & 3] = add2(s[j & 3], e);
        if (ENTROPY) q[j & 3] = fma2(e, pack2(fmaxf(d.x, kFar), fmaxf(d.y, kFar)), q[j & 3]);
    }
    const float2 a = unpack2(add2(add2(s[0], s[1]), add2(s[2], s[3]))), b = unpack2(add2(add2(q[0], q[1]), add2(q[2], q[3])));
    return {m, a.x + a.y, b.x + b.y};
}

// One CTA per SM walks over tiles of 128 tokens by tile_cols (at most BN) columns of the
// vocabulary, or (CG = 2) a pair of CTAs over tiles of 256 by tile_cols, each CTA loading its own
// tokens and half of the columns.
// Warp 0 keeps kStages pairs of operand tiles on their way by TMA, one thread of warp 1 (of the
// pair's first CTA) issues the MMAs into one of two accumulators in TMEM, and eight warps read the
// other, one row per thread, half of the columns per warpgroup. The tensor core drops the low
// bits of each sum it forms, always towards zero, so an accumulator takes kChunk stages (512
// products) only; the epilogue adds the accumulators of a tile in registers, rounded to nearest,
// and then forms the softmax sums while the next tile's products run. In whole sums of 2048
// products log-probabilities were off by 1.7e-6 of themselves, in these by 3.8e-7, as the fp32
// product is; it costs 3%.
// 8192 tokens x 50257 x 2048, a quarter masked: 657 us for 1.26e12 operations, 1.93 PFLOP/s, 102% of
// the rate measured for the library's bf16 product (741 us under the power cap of a long run); bound
// by the tensor cores. 16 tokens x 50257 x 768: 21.4 us, half of the rate of reading the matrix (77 MB),
// the rest a first load's latency, the last tile's sums and the join.
constexpr int kChunk = 8;

template <int CG, int BN>
struct LinearShape {
    static constexpr int kBRows = BN / CG;
    static constexpr int kA = kRowsTile * 128, kB = kBRows * 128, kStage = kA + kB;
    static constexpr int kStages = 196608 / kStage;
    static constexpr int kSmem = kStages * kStage + 1024;
};

template <int TYPE, int CG, int BN, bool ENTROPY>
__global__ void __launch_bounds__(kLinearThreads, 1)
    k_linear_mma(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const LinearArgs a) {
    using S = LinearShape<CG, BN>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * S::kStages + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    const uint32_t tiles = (smem_addr(raw) + 1023) & ~1023u;
    const uint32_t full = smem_addr(bars), empty = full + 8 * S::kStages, acc_full = empty + 8 * S::kStages,
                   acc_empty = acc_full + 16, drained = acc_empty + 16;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, CG * kEpilogueWarps);
        }
        mbar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<CG>(smem_addr(&tmem_slot), 2 * BN);
    tcgen05_before_sync();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tcgen05_after_sync();
    const uint32_t tmem = tmem_slot;
    let_next_kernel_start();
    wait_for_kernel_before();
    const int32_t live = a.tiles ? a.tiles[0] : 1;
    const int64_t total = (int64_t)live * a.col_tiles;
    const int steps = (int)((a.dim + kDepth - 1) / kDepth);

    if (warp < 4) {
        fewer_registers<kFewRegisters>();
        if (warp == 0 && lane == 0) {
            Ring<S::kStages> ring;
            int filled = 0;  // stages in use, up to all of them
            bool ok = true;
            for (int64_t i = blockIdx.x / CG; i < total && ok; i += gridDim.x / CG) {
                int32_t row, col;
                tile_of(a, live, i, &row, &col);
                for (int k = 0; k < steps; ++k) {
                    if (!(ok = mbar_wait(empty + 8 * ring.at, ring.phase ^ 1, &gave_up))) break;
                    const uint32_t at = tiles + ring.at * S::kStage;
                    // both CTAs' bytes count on the first one's barrier
                    if (rank == 0) mbar_expect(full + 8 * ring.at, CG * a.load_rows * 128 + a.tile_cols * 128);
                    const uint32_t bar = CG == 2 ? smem_of(full + 8 * ring.at, 0) : full + 8 * ring.at;
                    tma_load<CG>(at, &map_a, bar, k * kDepth, (row * CG + (int)rank) * kRowsTile);
                    tma_load<CG>(at + S::kA, &map_b, bar, k * kDepth, col * a.tile_cols + (int)rank * (a.tile_cols / CG));
                    ring.next();
                    filled += filled < S::kStages;
                }
            }
            // the last stages' releases have arrived before the barriers go away
            for (int k = 0; k < filled && ok; ++k) {
                // back over the ring: stage at - 1 - k, in the phase it was filled in
                const int st = ring.at - 1 - k < 0 ? ring.at - 1 - k + S::kStages : ring.at - 1 - k;
                ok = mbar_wait(empty + 8 * st, ring.at - 1 - k < 0 ? ring.phase ^ 1 : ring.phase, &gave_up);
            }
            if (!ok) {  // leave no copy in flight behind: they take microseconds, this a millisecond
                for (int j = 0; j < 1000; ++j) __nanosleep(1000);
            }
        } else if (warp == 1 && lane == 0 && rank == 0) {
            const uint32_t idesc = instr_desc(CG * kRowsTile, a.tile_cols, TYPE == ZERO_T_BF16 ? 1 : 0);
            const uint64_t desc_a = smem_desc(tiles), desc_b = smem_desc(tiles + S::kA);
            Ring<S::kStages> ring;
            Ring<2> acc;
            bool ok = true;
            for (int64_t i = blockIdx.x / CG; i < total && ok; i += gridDim.x / CG) {
                for (int k0 = 0; k0 < steps && ok; k0 += kChunk) {
                    if (!(ok = mbar_wait(acc_empty + 8 * acc.at, acc.phase ^ 1, &gave_up))) break;
                    tcgen05_after_sync();
                    const uint32_t d = tmem + acc.at * BN;
                    const int n = min(kChunk, steps - k0);
                    for (int k = 0; k < n; ++k) {
                        if (!(ok = mbar_wait(full + 8 * ring.at, ring.phase, &gave_up))) break;
                        tcgen05_after_sync();
                        const uint64_t at = (uint64_t)(ring.at * (S::kStage >> 4));
#pragma unroll
                        for (int j = 0; j < kDepth / 16; ++j)  // 16 elements: 32 bytes further in the swizzled rows
                            mma_f16<CG>(d, desc_a + at + 2 * j, desc_b + at + 2 * j, idesc, k > 0 || j > 0);
                        mma_commit<CG>(empty + 8 * ring.at);
                        ring.next();
                    }
                    if (ok) mma_commit<CG>(acc_full + 8 * acc.at);
                    acc.next();
                }
            }
            if (!ok) {
                mma_commit<CG>(drained);
                for (int j = 0; j < kWaitLimit && !mbar_try(drained, 0); ++j) {}
            }
        }
    } else {
        more_registers<kManyRegisters>();
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const int cols = a.tile_cols / 2;  // of this thread's part of a row
        const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16) + half * cols;
        Ring<2> acc;
        bool ok = true;
        for (int64_t i = blockIdx.x / CG; i < total && ok; i += gridDim.x / CG) {
            int32_t row, col;
            tile_of(a, live, i, &row, &col);
            const int64_t r = ((int64_t)row * CG + rank) * kRowsTile + quarter * 32 + lane;
            const int64_t col0 = (int64_t)col * a.tile_cols + half * cols;
            const int n = (int)min((int64_t)cols, a.vocab - col0);  // may be 0 or less
            const int64_t y = r < a.rows ? a.targets[r] - col0 : -1;
            float v[BN / 2];
            auto take = [&](auto add) {
                if (!(ok = __all_sync(~0u, mbar_wait(acc_full + 8 * acc.at, acc.phase, &gave_up)))) return;
                tcgen05_after_sync();
#pragma unroll
                for (int j = 0; j < BN / 2; j += 64) {
                    float u[64];
                    tmem_load64(mine + acc.at * BN + j, u);
#pragma unroll
                    for (int n = 0; n < 64; ++n) v[j + n] = decltype(add)::value ? v[j + n] + u[n] : u[n];
                }
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2) mbar_arrive_at(smem_of(acc_empty + 8 * acc.at, 0));
                    else mbar_arrive(acc_empty + 8 * acc.at);
                }
                acc.next();
            };
            take(std::false_type());
            for (int k = kChunk; k < steps && ok; k += kChunk) take(std::true_type());
            if (!ok) break;
            if (n < BN / 2) {
#pragma unroll
                for (int j = 0; j < BN / 2; ++j)
                    if (j >= n) v[j] = -INFINITY;
            }
            if (__any_sync(~0u, y >= 0 && y < n)) {
#pragma unroll
                for (int j = 0; j < BN / 2; ++j)
                    if (y == j && j < n) a.zy[r] = v[j];
            }
            const RowStat st = sum_of<ENTROPY>(v, a.k);
            if (r < a.rows) {
                const int64_t o = ((int64_t)col * 2 + half) * a.rows + r;
                a.m[o] = st.m;
                a.s[o] = st.s;
                if (ENTROPY) a.q[o] = st.q;
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (CG == 2) cluster_sync();  // neither CTA leaves while the other's MMAs or arrivals use its memory
    if (warp == 1) {
        tcgen05_after_sync();
        tmem_free<CG>(tmem, 2 * BN);
    }
    if (threadIdx.x == 0) a.status[blockIdx.x] = gave_up;
}

// A row's results from its joined sums, by one thread.
template <bool ENTROPY>
__device__ __forceinline__ void finish(const LinearArgs& a, int64_t t, int64_t y, const RowStat& s, bool gave_up, float* logp, float* lse,
                                       float* entropy) {
    RowResult r = {0.0f, 0.0f, 0.0f, 0.0f};
    if (y >= 0) {
        r = finish_row<ENTROPY>(s, y < a.vocab ? a.zy[t] : NAN, a.k, a.inv_t);
        if (y >= a.vocab) r.logp = NAN;
    }
    if (gave_up) r.logp = r.lse = r.entropy = NAN;  // no result
    logp[t] = r.logp;
    lse[t] = r.lse;
    if (ENTROPY) entropy[t] = r.entropy;
}

// Whether a wait of the product gave up, seen by all threads.
__device__ __forceinline__ bool any_gave_up(const LinearArgs& a) {
    bool gave_up = false;
    for (int i = threadIdx.x; i < a.grid; i += blockDim.x) gave_up |= a.status[i] != 0;
    return __syncthreads_or(gave_up);
}

// Many rows: 32 rows (lanes, so that loads are whole lines) by 16 slices of their parts, four
// parts on their way at a time; the slices are joined in order.
constexpr int kJoinSlices = 16;

template <bool ENTROPY>
__global__ void __launch_bounds__(32 * kJoinSlices) k_linear_join(const LinearArgs a, int parts, float* logp, float* lse, float* entropy) {
    __shared__ RowStat sm[kJoinSlices][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_kernel_before();
    const int64_t t = (int64_t)blockIdx.x * 32 + lane;
    RowStat s = empty_stat();
    const int64_t y = t < a.rows ? a.targets[t] : -1;
    if (y >= 0)  // parts of rows without a target may not have been written
        for (int p0 = warp; p0 < parts; p0 += 4 * kJoinSlices) {
            RowStat b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t p = p0 + i * kJoinSlices;
                b[i] = empty_stat();
                if (p < parts) b[i] = {a.m[p * a.rows + t], a.s[p * a.rows + t], ENTROPY ? a.q[p * a.rows + t] : 0.0f};
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s = join<ENTROPY>(s, b[i], a.k);
        }
    sm[warp][lane] = s;
    const bool gave_up = any_gave_up(a);
    if (warp != 0 || t >= a.rows) return;
    for (int w = 1; w < kJoinSlices; ++w) s = join<ENTROPY>(s, sm[w][lane], a.k);
    finish<ENTROPY>(a, t, y, s, gave_up, logp, lse, entropy);
}

// Few rows: a CTA each, a thread per part. The other form would have one CTA go through all parts
// of 32 rows, one latency after the other (14 us for 16 rows of 898 parts). The whole call with either
// form, 50257 x 64: 16 rows 12.5 against 16.4 us, 1024 rows 40.0 against 41.4, 2048 rows 55.6 against
// 53.4, 4096 rows 103 against 89; 8000 x 64 crosses between 1024 and 2048 as well.
constexpr int kJoinThreads = 256;
constexpr int64_t kJoinFewRows = 1024;

template <bool ENTROPY>
__global__ void __launch_bounds__(kJoinThreads) k_linear_join_few(const LinearArgs a, int parts, float* logp, float* lse, float* entropy) {
    __shared__ RowStat sm[kJoinThreads / 32];
    wait_for_kernel_before();
    const int64_t t = blockIdx.x, y = a.targets[t];
    RowStat s = empty_stat();
    if (y >= 0)
        for (int64_t p = threadIdx.x; p < parts; p += kJoinThreads) {
            const RowStat b = {a.m[p * a.rows + t], a.s[p * a.rows + t], ENTROPY ? a.q[p * a.rows + t] : 0.0f};
            s = join<ENTROPY>(s, b, a.k);
        }
    s = group_join<ENTROPY, true, kJoinThreads / 32>(s, a.k, sm, 0);
    const bool gave_up = any_gave_up(a);
    if (threadIdx.x == 0) finish<ENTROPY>(a, t, y, s, gave_up, logp, lse, entropy);
}

constexpr int kMaxGrid = 1024;

// How a call is cut up, and where things lie in its workspace.
struct LinearPlan {
    bool pairs;
    int32_t tile_rows, row_tiles, tile_cols, col_tiles;
    int64_t parts, parts_bytes, bytes;
};

// Up to 128 tokens: single CTAs on narrow tiles. Beyond: pairs of CTAs on tiles of 256 tokens, or
// single CTAs on tiles of 128, whichever has the busiest CTA go through fewer columns; single CTAs
// count for 8% more, since each loads all of its columns itself (300 tokens x 50257 x 2048: three
// tiles of 128 in 62 us, two of 256 in 74; 500 tokens: 82 and 75). Of 130 to 3000 tokens by 50257 x 768,
// 50257 x 2048, 32000 x 1024 and 130000 x 1024, 40 shapes, this takes the faster form or one within 1%
// of it. The width of a tile is likewise the one, of those that
// an MMA takes, with the fewest columns for the busiest CTA: 50257 columns over 152 CTAs are three
// tiles of 112 each rather than one or two of 256. Tiles narrower than 192 would slow the MMAs
// where these are what bounds.
LinearPlan linear_plan(int64_t rows, int64_t vocab, int sms) {
    LinearPlan l = {};
    double least = 1e300;
    auto consider = [&](bool pairs, int widest, int narrowest, int step, double weight) {
        const int tile_rows = pairs ? 2 * kRowsTile : kRowsTile, workers = std::max(1, pairs ? sms / 2 : sms);
        const int64_t row_tiles = (rows + tile_rows - 1) / tile_rows;
        for (int cols = widest; cols >= narrowest; cols -= step) {
            const int64_t tiles = (vocab + cols - 1) / cols * row_tiles;
            const double most = (double)((tiles + workers - 1) / workers) * cols * weight;
            if (most >= least) continue;
            least = most;
            l.pairs = pairs;
            l.tile_rows = tile_rows;
            l.row_tiles = (int32_t)row_tiles;
            l.tile_cols = cols;
        }
    };
    if (rows <= kRowsTile) {
        consider(false, 128, 64, 16, 1.0);
    } else {
        consider(true, 256, 224, 32, 1.0);
        consider(false, 256, 192, 16, 1.08);
    }
    l.col_tiles = (int32_t)((vocab + l.tile_cols - 1) / l.tile_cols);
    l.parts = 2 * (int64_t)l.col_tiles;
    l.parts_bytes = (12 * l.parts * rows + 4 * rows + 15) / 16 * 16;
    l.bytes = l.parts_bytes + 4 * (kMaxGrid + 4 + (int64_t)l.row_tiles);
    return l;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library is not linked against the driver).
EncodeTiled encoder() {
    static const EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return (EncodeTiled)p;
    }();
    return f;
}

// [rows, dim] of 16-bit elements, ld apart, in boxes of `box` rows by 64 elements; what lies
// outside reads as 0.
bool encode(CUtensorMap* map, int32_t type, const void* p, int64_t rows, int64_t dim, int64_t ld, int box) {
    const cuuint64_t dims[2] = {(cuuint64_t)dim, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t boxes[2] = {kDepth, (cuuint32_t)box}, steps[2] = {1, 1};
    return encoder()(map, type == ZERO_T_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, (void*)p, dims,
                     strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int TYPE, int CG, int BN, bool ENTROPY>
int launch_product(const zero_linear* x, const LinearArgs& a, cudaStream_t s) {
    using S = LinearShape<CG, BN>;
    CUtensorMap ma, mb;
    if (!encode(&ma, x->type, x->hidden, x->rows, x->dim, x->ld_hidden, a.load_rows) ||
        !encode(&mb, x->type, x->weight, x->vocab, x->dim, x->ld_weight, a.tile_cols / CG))
        return record_cuda_error(cudaErrorInvalidValue);
    const cudaError_t e = cudaFuncSetAttribute(k_linear_mma<TYPE, CG, BN, ENTROPY>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return record_cuda_error(e);
    return launch_linked(k_linear_mma<TYPE, CG, BN, ENTROPY>, a.grid, kLinearThreads, S::kSmem, CG, s, ma, mb, a);
}

template <bool ENTROPY>
int run_linear(const zero_linear* x, const LinearArgs& a, const LinearPlan& l, float* logp, float* lse, float* entropy, cudaStream_t s) {
    int rc = a.tiles ? launch_linked(k_linear_tiles, 1, 1024, 0, 1, s, a) : ZERO_OK;
    if (rc) return rc;
    const bool bf16 = x->type == ZERO_T_BF16;
    if (l.pairs) rc = bf16 ? launch_product<ZERO_T_BF16, 2, 256, ENTROPY>(x, a, s) : launch_product<ZERO_T_FP16, 2, 256, ENTROPY>(x, a, s);
    else if (l.tile_cols > 128) rc = bf16 ? launch_product<ZERO_T_BF16, 1, 256, ENTROPY>(x, a, s) : launch_product<ZERO_T_FP16, 1, 256, ENTROPY>(x, a, s);
    else rc = bf16 ? launch_product<ZERO_T_BF16, 1, 128, ENTROPY>(x, a, s) : launch_product<ZERO_T_FP16, 1, 128, ENTROPY>(x, a, s);
    if (rc) return rc;
    if (x->rows <= kJoinFewRows)
        return launch_linked(k_linear_join_few<ENTROPY>, (unsigned)x->rows, kJoinThreads, 0, 1, s, a, (int)l.parts, logp, lse, entropy);
    return launch_linked(k_linear_join<ENTROPY>, (unsigned)((x->rows + 31) / 32), 32 * kJoinSlices, 0, 1, s, a, (int)l.parts, logp, lse, entropy);
}

// The workspace of any number of SMs.
int64_t most_bytes(int64_t rows, int64_t vocab) {
    const int64_t narrowest = rows > kRowsTile ? 192 : 64;
    return 12 * 2 * ((vocab + narrowest - 1) / narrowest) * rows + 4 * rows + 16 + 4 * (kMaxGrid + 4 + rows / kRowsTile + 1);
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" int64_t zero_linear_logp_workspace(int64_t rows, int64_t vocab) {
    if (rows < 0 || vocab < 1 || vocab > INT32_MAX || rows > INT32_MAX) return -1;
    return most_bytes(rows, vocab);
}

extern "C" int zero_linear_logp(const zero_linear* x, float* logp, float* lse, float* entropy, void* workspace,
                                int64_t workspace_bytes, void* stream) {
    if (!x || x->rows < 0 || x->rows > INT32_MAX || x->vocab < 1 || x->vocab > INT32_MAX || x->dim < 1 || x->dim > INT32_MAX ||
        x->ld_hidden < x->dim || x->ld_weight < x->dim || (x->type != ZERO_T_BF16 && x->type != ZERO_T_FP16) ||
        !temperature_ok(x->temperature))
        return ZERO_ERR_INVALID_ARG;
    if (x->ld_hidden > (INT64_C(1) << 36) || x->ld_weight > (INT64_C(1) << 36)) return ZERO_ERR_INVALID_ARG;
    if (x->ld_hidden % 8 || x->ld_weight % 8) return ZERO_ERR_MISALIGNED;
    if (x->rows == 0) return ZERO_OK;
    if (workspace_bytes < zero_linear_logp_workspace(x->rows, x->vocab)) return ZERO_ERR_SIZE_MISMATCH;
    CallDevice d(x->hidden, stream);
    d.need(x->hidden, 16);
    d.need(x->weight, 16);
    d.need(x->targets, 8);
    d.need(logp, 4);
    d.need(lse, 4);
    d.optional(entropy, 4);
    d.need(workspace, 16);
    if (d.rc) return d.rc;
    if (!encoder()) return record_cuda_error(cudaErrorNotSupported);
    cudaStream_t s = (cudaStream_t)stream;
    const int sms = d.sm_count();
    const LinearPlan l = linear_plan(x->rows, x->vocab, sms);
    LinearArgs a;
    a.targets = x->targets;
    a.m = (float*)workspace;
    a.s = a.m + l.parts * x->rows;
    a.q = a.s + l.parts * x->rows;
    a.zy = a.q + l.parts * x->rows;
    a.status = (int32_t*)((char*)workspace + l.parts_bytes);
    a.tiles = l.row_tiles > 1 ? a.status + kMaxGrid : nullptr;
    a.rows = x->rows;
    a.vocab = x->vocab;
    a.dim = x->dim;
    a.tile_rows = l.tile_rows;
    a.row_tiles = l.row_tiles;
    // the MMA's other rows then hold whatever the stage held: no row of a product sees another
    a.load_rows = (int32_t)std::min<int64_t>(kRowsTile, (x->rows + 7) / 8 * 8);
    a.tile_cols = l.tile_cols;
    a.col_tiles = l.col_tiles;
    // row tiles of 32 MB of hidden states at most stay in L2 together
    a.group = (int32_t)std::max<int64_t>(1, std::min<int64_t>(8192 / a.tile_rows, (INT64_C(32) << 20) / (a.tile_rows * 2 * x->dim)));
    const int width = l.pairs ? 2 : 1;
    a.grid = (int32_t)(std::min<int64_t>((int64_t)l.row_tiles * l.col_tiles, std::min(sms, kMaxGrid) / width) * width);
    a.k = make_scale(x->temperature);
    a.inv_t = (float)(1.0 / x->temperature);
    return entropy ? run_linear<true>(x, a, l, logp, lse, entropy, s) : run_linear<false>(x, a, l, logp, lse, entropy, s);
}
