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

constexpr int kRowsTile = 128;    // tokens of a tile: the lanes of TMEM
constexpr int kDepth = 64;         // elements of the inner dimension per stage: 128 bytes
constexpr int kEpilogueWarps = 8;  // two for each quarter of the lanes
constexpr int kLinearThreads = 64 + 32 * kEpilogueWarps;

struct LinearArgs {
    const int64_t* targets;
    float *m, *s, *q;  // [parts, rows]
    float* zy;         // [rows] the target's logit
    int32_t* tiles;    // [0]: how many row tiles hold a target, [1]: set when a wait gave up, [4...]: those tiles
    int64_t rows, vocab, dim;
    int32_t row_tiles, col_tiles, group;
    float c, inv_t;  // log2(e) / temperature, 1 / temperature
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
            for (int i = lane; i < kRowsTile; i += 32) {
                const int64_t r = (int64_t)t * kRowsTile + i;
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

// 32 logits of one row into its sums.
__device__ __forceinline__ void add32(RowStat& st, const float (&v)[32], float c) {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < 32; ++j) m = fmaxf(m, v[j]);
    m = fmaxf(m, st.m);
    const float base = base_of(m);
    rebase<true>(st, base, c);
    st.m = m;
#pragma unroll
    for (int j = 0; j < 32; ++j) add_term<true>(st, v[j], c, base);
}

// One CTA per SM walks over tiles of 128 tokens by BN columns of the vocabulary. Warp 0 keeps
// kStages pairs of operand tiles on their way by TMA, one thread of warp 1 issues the MMAs into
// one of two accumulators in TMEM, and eight warps take the other's logits through the softmax
// sums meanwhile, one row per thread, half of the columns per warpgroup.
template <int BN>
struct LinearShape {
    static constexpr int kA = kRowsTile * 128, kB = BN * 128, kStage = kA + kB;
    static constexpr int kStages = 196608 / kStage;
    static constexpr int kSmem = kStages * kStage + 1024;
};

template <int TYPE, int BN>
__global__ void __launch_bounds__(kLinearThreads, 1)
    k_linear_mma(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const LinearArgs a) {
    using S = LinearShape<BN>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * S::kStages + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    const uint32_t tiles = (smem_addr(raw) + 1023) & ~1023u;
    const uint32_t full = smem_addr(bars), empty = full + 8 * S::kStages, acc_full = empty + 8 * S::kStages,
                   acc_empty = acc_full + 16, drained = acc_empty + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, kEpilogueWarps);
        }
        mbar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(smem_addr(&tmem_slot), 2 * BN);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = tmem_slot;
    const int32_t live = a.tiles[0];
    const int64_t total = (int64_t)live * a.col_tiles;
    const int steps = (int)((a.dim + kDepth - 1) / kDepth);

    if (warp == 0) {
        if (lane == 0) {
            int64_t n = 0;  // stages filled so far
            bool ok = true;
            for (int64_t i = blockIdx.x; i < total && ok; i += gridDim.x) {
                int32_t row, col;
                tile_of(a, live, i, &row, &col);
                for (int k = 0; k < steps; ++k, ++n) {
                    const int st = (int)(n % S::kStages);
                    const uint32_t turn = (uint32_t)(n / S::kStages);
                    if (!(ok = mbar_wait(empty + 8 * st, (turn & 1) ^ 1, &gave_up))) break;
                    const uint32_t at = tiles + st * S::kStage;
                    mbar_expect(full + 8 * st, S::kStage);
                    tma_load(at, &map_a, full + 8 * st, k * kDepth, row * kRowsTile);
                    tma_load(at + S::kA, &map_b, full + 8 * st, k * kDepth, col * BN);
                }
            }
            if (!ok)  // leave no copy in flight behind
                for (int64_t k = n > S::kStages ? n - S::kStages : 0; k < n; ++k)
                    for (int j = 0; j < kWaitLimit && !mbar_try(full + 8 * (int)(k % S::kStages), (uint32_t)(k / S::kStages) & 1); ++j) {}
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = instr_desc(kRowsTile, BN, TYPE == ZERO_T_BF16 ? 1 : 0);
            int64_t n = 0, it = 0;
            bool ok = true;
            for (int64_t i = blockIdx.x; i < total && ok; i += gridDim.x, ++it) {
                const int acc = (int)(it & 1);
                if (!(ok = mbar_wait(acc_empty + 8 * acc, ((uint32_t)(it >> 1) & 1) ^ 1, &gave_up))) break;
                tcgen05_after_sync();
                for (int k = 0; k < steps; ++k, ++n) {
                    const int st = (int)(n % S::kStages);
                    if (!(ok = mbar_wait(full + 8 * st, (uint32_t)(n / S::kStages) & 1, &gave_up))) break;
                    tcgen05_after_sync();
                    const uint64_t da = smem_desc(tiles + st * S::kStage), db = smem_desc(tiles + st * S::kStage + S::kA);
#pragma unroll
                    for (int j = 0; j < kDepth / 16; ++j)  // 16 elements: 32 bytes further in the swizzled rows
                        mma_f16(tmem + acc * BN, da + 2 * j, db + 2 * j, idesc, k > 0 || j > 0);
                    mma_commit(empty + 8 * st);
                }
                if (ok) mma_commit(acc_full + 8 * acc);
            }
            if (!ok) {
                mma_commit(drained);
                for (int j = 0; j < kWaitLimit && !mbar_try(drained, 0); ++j) {}
            }
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        int64_t it = 0;
        for (int64_t i = blockIdx.x; i < total; i += gridDim.x, ++it) {
            int32_t row, col;
            tile_of(a, live, i, &row, &col);
            const int acc = (int)(it & 1);
            const int64_t r = (int64_t)row * kRowsTile + quarter * 32 + lane;
            const int64_t col0 = (int64_t)col * BN + half * (BN / 2);
            const int64_t y = r < a.rows ? a.targets[r] - col0 : -1;
            if (!__all_sync(~0u, mbar_wait(acc_full + 8 * acc, (uint32_t)(it >> 1) & 1, &gave_up))) break;
            tcgen05_after_sync();
            RowStat st = empty_stat();
#pragma unroll 1
            for (int j = 0; j < BN / 2; j += 32) {
                float v[32];
                tmem_load32(tmem + ((uint32_t)(quarter * 32) << 16) + acc * BN + half * (BN / 2) + j, v);
                if (col0 + j + 32 > a.vocab) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (col0 + j + k >= a.vocab) v[k] = -INFINITY;
                }
                if (__any_sync(~0u, y >= j && y < j + 32)) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (y == j + k && col0 + y < a.vocab) a.zy[r] = v[k];
                }
                add32(st, v, a.c);
            }
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + 8 * acc);
            if (r < a.rows) {
                const int64_t o = ((int64_t)col * 2 + half) * a.rows + r;
                a.m[o] = st.m;
                a.s[o] = st.s;
                a.q[o] = st.q;
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        tcgen05_after_sync();
        tmem_free(tmem, 2 * BN);
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
            s = join<true>(s, b, a.c);
        }
    sm[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || t >= a.rows) return;
    for (int w = 1; w < 32; ++w) s = join<true>(s, sm[w][lane], a.c);
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

constexpr int kMaxBN = 256;

// Where the parts, the targets' logits and the list of row tiles lie in the workspace.
struct LinearLayout {
    int64_t row_tiles, parts, parts_bytes, bytes;
};
LinearLayout linear_layout(int64_t rows, int64_t vocab, int bn) {
    LinearLayout l;
    l.row_tiles = (rows + kRowsTile - 1) / kRowsTile;
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

template <int TYPE, int BN>
int launch_linear(const zero_linear* x, LinearArgs a, int sms, cudaStream_t s) {
    CUtensorMap ma, mb;
    if (!encode(&ma, x->type, x->hidden, x->rows, x->dim, x->ld_hidden, kRowsTile) ||
        !encode(&mb, x->type, x->weight, x->vocab, x->dim, x->ld_weight, BN))
        return record_cuda_error(cudaErrorInvalidValue);
    const cudaError_t e = cudaFuncSetAttribute(k_linear_mma<TYPE, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, LinearShape<BN>::kSmem);
    if (e != cudaSuccess) return record_cuda_error(e);
    const int64_t tiles = (int64_t)a.row_tiles * a.col_tiles;
    k_linear_mma<TYPE, BN><<<(unsigned)std::min<int64_t>(tiles, sms), kLinearThreads, LinearShape<BN>::kSmem, s>>>(ma, mb, a);
    return launched();
}

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" int64_t zero_linear_logp_workspace(int64_t rows, int64_t vocab) {
    if (rows < 0 || vocab < 1 || vocab > INT32_MAX || rows > INT32_MAX) return -1;
    return linear_layout(rows, vocab, kMaxBN).bytes;
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
    const LinearLayout l = linear_layout(x->rows, x->vocab, kMaxBN);
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
    a.row_tiles = (int32_t)l.row_tiles;
    a.col_tiles = (int32_t)(l.parts / 2);
    a.group = (int32_t)std::max<int64_t>(1, std::min<int64_t>(64, (INT64_C(32) << 20) / (kRowsTile * 2 * x->dim)));
    a.c = (float)(1.4426950408889634 / x->temperature);
    a.inv_t = (float)(1.0 / x->temperature);
    k_linear_tiles<<<1, 1024, 0, s>>>(a);
    int rc = launched();
    if (rc) return rc;
    const int sms = d.sm_count();
    rc = x->type == ZERO_T_BF16 ? launch_linear<ZERO_T_BF16, 256>(x, a, sms, s) : launch_linear<ZERO_T_FP16, 256>(x, a, sms, s);
    if (rc) return rc;
    k_linear_join<<<(unsigned)((x->rows + 31) / 32), 1024, 0, s>>>(a, l.parts, logp, lse, entropy);
    return launched();
}
