// zero_linear.cu -- token log-probabilities from hidden states and the vocabulary matrix, with
// no logits in memory, for sm_103a.
//
// logits = hidden weight^T is formed tile by tile by tcgen05 and stays in TMEM; a tile's part
// of each row's softmax sums (zero_softmax.cuh) goes to the workspace, and a second kernel joins
// the parts of a row in their order. Row tiles without a target are left out.

#include <algorithm>
#include <cmath>
#include <cstdint>

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
    int32_t* tiles;    // [0]: how many row tiles hold a target, [1]: set when a wait gave up, [4...]: those tiles
    int64_t rows, vocab, dim;
    int32_t tile_rows, row_tiles, col_tiles, group;
    Scale k;       // log2(e) / temperature
    double inv_t;  // 1 / temperature
};

// Row tiles with at least one target, in order. One CTA.
__global__ void __launch_bounds__(1024) k_linear_tiles(const LinearArgs a) {
    __shared__ int32_t base, sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) base = 0;
    __syncthreads();
    for (int32_t t0 = 0; t0 < a.row_tiles; t0 += 32) {
        // a warp per tile looks at its rows
        const int32_t t = t0 + warp;
        bool any = false;
        if (t < a.row_tiles)
            for (int i = lane; i < a.tile_rows; i += 32) {
                const int64_t r = (int64_t)t * a.tile_rows + i;
                any |= r < a.rows && a.targets[r] >= 0;
            }
        any = __any_sync(~0u, any);
        if (lane == 0) sums[warp] = any;
        __syncthreads();
        if (warp == 0) {
            const bool mine = sums[lane] != 0;
            const unsigned ballot = __ballot_sync(~0u, mine);
            const int32_t at = base;
            if (mine) a.tiles[4 + at + __popc(ballot & ((1u << lane) - 1))] = t0 + lane;
            __syncwarp();
            if (lane == 0) base = at + __popc(ballot);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        a.tiles[0] = base;
        a.tiles[1] = 0;
    }
}

// Tile `i` of the run: groups of row tiles that stay in L2 while the vocabulary passes by, and
// within a group the row tiles fastest, so that CTAs working side by side share their columns.
__device__ __forceinline__ void tile_of(const LinearArgs& a, int32_t live, int64_t i, int32_t* row, int32_t* col) {
    const int64_t per = (int64_t)a.group * a.col_tiles;
    const int32_t g = (int32_t)(i / per), first = g * a.group;
    const int32_t size = min(a.group, live - first);
    const int64_t in = i - (int64_t)g * per;
    *col = (int32_t)(in / size);
    *row = a.tiles[4 + first + (int32_t)(in % size)];
}

// N logits of one row: their sums, in four chains.
template <int N>
__device__ __forceinline__ RowStat sum_of(const float (&v)[N], Scale k) {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < N; ++j) m = fmaxf(m, v[j]);
    const float base = base_of(m);
    RowStat part[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) part[i] = {m, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < N; ++j) add_term<true>(part[j & 3], v[j], k, base);
    return {m, (part[0].s + part[1].s) + (part[2].s + part[3].s), (part[0].q + part[1].q) + (part[2].q + part[3].q)};
}

// One CTA per SM walks over tiles of 128 tokens by BN columns of the vocabulary, or (CG = 2) a
// pair of CTAs over tiles of 256 by BN, each CTA loading its own tokens and half of the columns.
// Warp 0 keeps kStages pairs of operand tiles on their way by TMA, one thread of warp 1 (of the
// pair's first CTA) issues the MMAs into one of two accumulators in TMEM, and eight warps read the
// other, one row per thread, half of the columns per warpgroup. The tensor core drops the low
// bits of each sum it forms, always towards zero, so an accumulator takes kChunk stages (512
// products) only; the epilogue adds the accumulators of a tile in registers, rounded to nearest,
// and then forms the softmax sums while the next tile's products run.
constexpr int kChunk = 8;

template <int CG, int BN>
struct LinearShape {
    static constexpr int kBRows = BN / CG;
    static constexpr int kA = kRowsTile * 128, kB = kBRows * 128, kStage = kA + kB;
    static constexpr int kStages = 196608 / kStage;
    static constexpr int kSmem = kStages * kStage + 1024;
};

template <int TYPE, int CG, int BN>
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
    const int32_t live = a.tiles[0];
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
                    if (rank == 0) mbar_expect(full + 8 * ring.at, CG * S::kStage);
                    const uint32_t bar = CG == 2 ? smem_of(full + 8 * ring.at, 0) : full + 8 * ring.at;
                    tma_load<CG>(at, &map_a, bar, k * kDepth, (row * CG + (int)rank) * kRowsTile);
                    tma_load<CG>(at + S::kA, &map_b, bar, k * kDepth, col * BN + (int)rank * S::kBRows);
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
            constexpr uint32_t idesc = instr_desc(CG * kRowsTile, BN, TYPE == ZERO_T_BF16 ? 1 : 0);
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
        const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16) + half * (BN / 2);
        Ring<2> acc;
        bool ok = true;
        for (int64_t i = blockIdx.x / CG; i < total && ok; i += gridDim.x / CG) {
            int32_t row, col;
            tile_of(a, live, i, &row, &col);
            const int64_t r = ((int64_t)row * CG + rank) * kRowsTile + quarter * 32 + lane;
            const int64_t col0 = (int64_t)col * BN + half * (BN / 2);
            const int64_t y = r < a.rows ? a.targets[r] - col0 : -1;
            float v[BN / 2];
#pragma unroll
            for (int j = 0; j < BN / 2; ++j) v[j] = 0.0f;
            for (int k = 0; k < steps; k += kChunk, acc.next()) {
                if (!(ok = __all_sync(~0u, mbar_wait(acc_full + 8 * acc.at, acc.phase, &gave_up)))) break;
                tcgen05_after_sync();
#pragma unroll
                for (int j = 0; j < BN / 2; j += 64) {
                    float u[64];
                    tmem_load64(mine + acc.at * BN + j, u);
#pragma unroll
                    for (int n = 0; n < 64; ++n) v[j + n] += u[n];
                }
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2) mbar_arrive_at(smem_of(acc_empty + 8 * acc.at, 0));
                    else mbar_arrive(acc_empty + 8 * acc.at);
                }
            }
            if (!ok) break;
            if (col0 + BN / 2 > a.vocab) {
#pragma unroll
                for (int j = 0; j < BN / 2; ++j)
                    if (col0 + j >= a.vocab) v[j] = -INFINITY;
            }
            if (__any_sync(~0u, y >= 0 && y < BN / 2)) {
#pragma unroll
                for (int j = 0; j < BN / 2; ++j)
                    if (y == j && col0 + y < a.vocab) a.zy[r] = v[j];
            }
            const RowStat st = sum_of(v, a.k);
            if (r < a.rows) {
                const int64_t o = ((int64_t)col * 2 + half) * a.rows + r;
                a.m[o] = st.m;
                a.s[o] = st.s;
                a.q[o] = st.q;
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
    if (threadIdx.x == 0 && gave_up) a.tiles[1] = 1;
}

// 32 rows by 32 slices of their parts; the slices are joined in order.
__global__ void __launch_bounds__(1024) k_linear_join(const LinearArgs a, int64_t parts, float* logp, float* lse, float* entropy) {
    __shared__ RowStat sm[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * 32 + lane;
    RowStat s = empty_stat();
    const int64_t y = t < a.rows ? a.targets[t] : -1;
    if (y >= 0)  // parts of rows without a target may not have been written
        for (int64_t p = warp; p < parts; p += 32) {
            const RowStat b = {a.m[p * a.rows + t], a.s[p * a.rows + t], a.q[p * a.rows + t]};
            s = join<true>(s, b, a.k);
        }
    sm[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || t >= a.rows) return;
    for (int w = 1; w < 32; ++w) s = join<true>(s, sm[w][lane], a.k);
    RowResult r = {0.0f, 0.0f, 0.0f};
    if (y >= 0) {
        r = finish_row(s, y < a.vocab ? a.zy[t] : NAN, a.inv_t);
        if (y >= a.vocab) r.logp = NAN;
    }
    if (a.tiles[1]) r.logp = r.lse = r.entropy = NAN;  // a wait of the product gave up: no result
    logp[t] = r.logp;
    lse[t] = r.lse;
    if (entropy) entropy[t] = r.entropy;
}

// Pairs of CTAs once there are tokens for more than one CTA's tile.
bool linear_pairs(int64_t rows) { return rows > kRowsTile; }

// Where the parts, the targets' logits and the list of row tiles lie in the workspace.
struct LinearLayout {
    int64_t row_tiles, parts, parts_bytes, bytes;
};
LinearLayout linear_layout(int64_t rows, int64_t vocab, int tile_rows, int bn) {
    LinearLayout l;
    l.row_tiles = (rows + tile_rows - 1) / tile_rows;
    l.parts = (vocab + bn - 1) / bn * 2;
    l.parts_bytes = (12 * l.parts * rows + 4 * rows + 15) / 16 * 16;
    l.bytes = l.parts_bytes + 4 * (4 + l.row_tiles);
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

template <int TYPE, int CG, int BN>
int launch_linear(const zero_linear* x, const LinearArgs& a, int sms, cudaStream_t s) {
    using S = LinearShape<CG, BN>;
    CUtensorMap ma, mb;
    if (!encode(&ma, x->type, x->hidden, x->rows, x->dim, x->ld_hidden, kRowsTile) ||
        !encode(&mb, x->type, x->weight, x->vocab, x->dim, x->ld_weight, S::kBRows))
        return record_cuda_error(cudaErrorInvalidValue);
    cudaError_t e = cudaFuncSetAttribute(k_linear_mma<TYPE, CG, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return record_cuda_error(e);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(std::min<int64_t>((int64_t)a.row_tiles * a.col_tiles, sms / CG) * CG));
    cfg.blockDim = dim3(kLinearThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = CG == 2 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, k_linear_mma<TYPE, CG, BN>, ma, mb, a);
    return e == cudaSuccess ? ZERO_OK : record_cuda_error(e);
}

template <int CG, int BN>
int run_linear(const zero_linear* x, const LinearArgs& a, int sms, cudaStream_t s) {
    k_linear_tiles<<<1, 1024, 0, s>>>(a);
    const int rc = launched();
    if (rc) return rc;
    return x->type == ZERO_T_BF16 ? launch_linear<ZERO_T_BF16, CG, BN>(x, a, sms, s) : launch_linear<ZERO_T_FP16, CG, BN>(x, a, sms, s);
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" int64_t zero_linear_logp_workspace(int64_t rows, int64_t vocab) {
    if (rows < 0 || vocab < 1 || vocab > INT32_MAX || rows > INT32_MAX) return -1;
    return linear_layout(rows, vocab, linear_pairs(rows) ? 2 * kRowsTile : kRowsTile, 256).bytes;
}

extern "C" int zero_linear_logp(const zero_linear* x, float* logp, float* lse, float* entropy, void* workspace,
                                int64_t workspace_bytes, void* stream) {
    if (!x || x->rows < 0 || x->rows > INT32_MAX || x->vocab < 1 || x->vocab > INT32_MAX || x->dim < 1 || x->dim > INT32_MAX ||
        x->ld_hidden < x->dim || x->ld_weight < x->dim || (x->type != ZERO_T_BF16 && x->type != ZERO_T_FP16) ||
        !(x->temperature > 0.0) || !std::isfinite(x->temperature))
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
    const bool pairs = linear_pairs(x->rows);
    const LinearLayout l = linear_layout(x->rows, x->vocab, pairs ? 2 * kRowsTile : kRowsTile, 256);
    LinearArgs a;
    a.targets = x->targets;
    a.m = (float*)workspace;
    a.s = a.m + l.parts * x->rows;
    a.q = a.s + l.parts * x->rows;
    a.zy = a.q + l.parts * x->rows;
    a.tiles = (int32_t*)((char*)workspace + l.parts_bytes);
    a.rows = x->rows;
    a.vocab = x->vocab;
    a.dim = x->dim;
    a.tile_rows = (int32_t)(pairs ? 2 * kRowsTile : kRowsTile);
    a.row_tiles = (int32_t)l.row_tiles;
    a.col_tiles = (int32_t)(l.parts / 2);
    a.group = (int32_t)std::max<int64_t>(1, std::min<int64_t>(8192 / a.tile_rows, (INT64_C(32) << 20) / (a.tile_rows * 2 * x->dim)));
    a.k = make_scale(x->temperature);
    a.inv_t = 1.0 / x->temperature;
    const int sms = d.sm_count();
    int rc = pairs ? run_linear<2, 256>(x, a, sms, s) : run_linear<1, 256>(x, a, sms, s);
    if (rc) return rc;
    k_linear_join<<<(unsigned)((x->rows + 31) / 32), 1024, 0, s>>>(a, l.parts, logp, lse, entropy);
    return launched();
}
