// zero_linear.cu -- token log-probabilities from hidden states and the vocabulary matrix, with
// no logits in memory, for sm_103a.
//
// logits = hidden weight^T is formed tile by tile; a tile's part of each row's softmax sums
// (zero_softmax.cuh) goes to the workspace, and a second kernel joins the parts of a row in
// their order.

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "zero_host.h"
#include "zero_softmax.cuh"

namespace zg {
namespace {

constexpr int kPartCols = 128;  // vocabulary columns of one part of a row

struct LinearArgs {
    const int64_t* targets;
    float *m, *s, *q;  // [parts, rows]
    float* zy;         // [rows] the target's logit
    int64_t rows, vocab, dim, ld_hidden, ld_weight;
    float c, inv_t;  // log2(e) / temperature, 1 / temperature
};

template <class T>
__global__ void __launch_bounds__(256) k_linear_tile(const LinearArgs a, const T* hidden, const T* weight) {
    constexpr int kM = 64, kN = kPartCols, kK = 16;
    __shared__ float sa[kK][kM + 4], sb[kK][kN + 4];
    __shared__ RowStat st[16][kM];
    const int64_t row0 = (int64_t)blockIdx.y * kM, col0 = (int64_t)blockIdx.x * kN;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][8] = {};
    for (int64_t k0 = 0; k0 < a.dim; k0 += kK) {
        for (int i = threadIdx.x; i < kM * kK; i += 256) {
            const int64_t r = row0 + i / kK, k = k0 + i % kK;
            sa[i % kK][i / kK] = r < a.rows && k < a.dim ? widen(hidden[r * a.ld_hidden + k]) : 0.0f;
        }
        for (int i = threadIdx.x; i < kN * kK; i += 256) {
            const int64_t r = col0 + i / kK, k = k0 + i % kK;
            sb[i % kK][i / kK] = r < a.vocab && k < a.dim ? widen(weight[r * a.ld_weight + k]) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kK; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 8 + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const int64_t r = row0 + ty * 4 + i;
        const int64_t y = r < a.rows ? a.targets[r] : -1;
        RowStat s = empty_stat();
        for (int j = 0; j < 8; ++j)
            if (col0 + tx * 8 + j < a.vocab) s.m = fmaxf(s.m, acc[i][j]);
        const float base = base_of(s.m);
        for (int j = 0; j < 8; ++j) {
            const int64_t col = col0 + tx * 8 + j;
            if (col >= a.vocab) break;
            add_term<true>(s, acc[i][j], a.c, base);
            if (col == y) a.zy[r] = acc[i][j];
        }
        st[tx][ty * 4 + i] = s;
    }
    __syncthreads();
    if (threadIdx.x < kM && row0 + threadIdx.x < a.rows) {
        RowStat s = st[0][threadIdx.x];
        for (int i = 1; i < 16; ++i) s = join<true>(s, st[i][threadIdx.x], a.c);
        const int64_t o = (int64_t)blockIdx.x * a.rows + row0 + threadIdx.x;
        a.m[o] = s.m;
        a.s[o] = s.s;
        a.q[o] = s.q;
    }
}

// 32 rows by 32 slices of their parts; the slices are joined in order.
__global__ void __launch_bounds__(1024) k_linear_join(const LinearArgs a, int64_t parts, float* logp, float* lse, float* entropy) {
    __shared__ RowStat sm[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * 32 + lane;
    RowStat s = empty_stat();
    if (t < a.rows)
        for (int64_t p = warp; p < parts; p += 32) {
            const RowStat b = {a.m[p * a.rows + t], a.s[p * a.rows + t], a.q[p * a.rows + t]};
            s = join<true>(s, b, a.c);
        }
    sm[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || t >= a.rows) return;
    for (int w = 1; w < 32; ++w) s = join<true>(s, sm[w][lane], a.c);
    const int64_t y = a.targets[t];
    RowResult r = {0.0f, 0.0f, 0.0f};
    if (y >= 0) {
        r = finish_row(s, y < a.vocab ? a.zy[t] : NAN, a.inv_t);
        if (y >= a.vocab) r.logp = NAN;
    }
    logp[t] = r.logp;
    lse[t] = r.lse;
    if (entropy) entropy[t] = r.entropy;
}

int64_t parts_of(int64_t vocab) { return (vocab + kPartCols - 1) / kPartCols; }

}  // namespace
}  // namespace zg

using namespace zg;

extern "C" int64_t zero_linear_logp_workspace(int64_t rows, int64_t vocab) {
    if (rows < 0 || vocab < 1 || vocab > INT32_MAX || rows > INT32_MAX) return -1;
    return 12 * parts_of(vocab) * rows + 4 * rows + 16;
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
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t parts = parts_of(x->vocab);
    LinearArgs a;
    a.targets = x->targets;
    a.m = (float*)workspace;
    a.s = a.m + parts * x->rows;
    a.q = a.s + parts * x->rows;
    a.zy = a.q + parts * x->rows;
    a.rows = x->rows;
    a.vocab = x->vocab;
    a.dim = x->dim;
    a.ld_hidden = x->ld_hidden;
    a.ld_weight = x->ld_weight;
    a.c = (float)(1.4426950408889634 / x->temperature);
    a.inv_t = (float)(1.0 / x->temperature);
    // rows in the grid's second dimension, 65535 tiles of 64 at a time
    const dim3 grid((unsigned)parts, (unsigned)((x->rows + 63) / 64));
    if (grid.y > 65535) return ZERO_ERR_TOO_LARGE;
    if (x->type == ZERO_T_BF16)
        k_linear_tile<<<grid, 256, 0, s>>>(a, (const __nv_bfloat16*)x->hidden, (const __nv_bfloat16*)x->weight);
    else
        k_linear_tile<<<grid, 256, 0, s>>>(a, (const __half*)x->hidden, (const __half*)x->weight);
    int rc = launched();
    if (rc) return rc;
    k_linear_join<<<(unsigned)((x->rows + 31) / 32), 1024, 0, s>>>(a, parts, logp, lse, entropy);
    return launched();
}
