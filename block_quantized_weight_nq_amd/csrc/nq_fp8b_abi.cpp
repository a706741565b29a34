// nq_fp8b_abi.cpp -- the C ABI of the E4M3 block operators and of the experts' rows: argument checks (the launch plan is
// nq_fp8b.h's).
#include "../../include/nq.h"
#include "nq_fp8b.h"

#define NQ_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr int64_t MOST = 1ll << 30;        // rows, pairs, N, and scales of rows
constexpr int64_t MOST_K = 1ll << 23;
constexpr int64_t MOST_EXPERTS = 1024, MOST_TOP = 1024;
constexpr int64_t THREADS = (1ll << 32) - 1;  // of a grid along an axis

int64_t element_size(int32_t dtype) { return dtype == NQ_F32 ? 4 : 2; }
bool bad_dtype(int32_t dtype) { return dtype != NQ_F32 && dtype != NQ_F16 && dtype != NQ_BF16; }

// Rows `stride` elements apart that are only read: they may overlap (a gradient that is one row for all).
int check_stride(int64_t stride, int64_t rows) {
    if (stride < 0) return NQ_ERR_BAD_DIM;
    if (rows > 0 && stride > (1ll << 60) / rows) return NQ_ERR_OVERFLOW;
    return NQ_OK;
}

// What quantizing and its inverse share.
int check_blocks(int32_t dtype, int64_t matrices, int64_t rows, int64_t cols, int32_t tile) {
    if (bad_dtype(dtype)) return NQ_ERR_BAD_DTYPE;
    if (matrices < 0 || rows < 0 || cols < 0 || (tile != 1 && tile != nq::FB)) return NQ_ERR_BAD_DIM;
    if (cols % nq::FB != 0) return NQ_ERR_NOT_BLOCK_ALIGNED;
    if (matrices > MOST || rows > MOST || cols > MOST) return NQ_ERR_OVERFLOW;
    if (rows > 0 && matrices > (1ll << 60) / rows) return NQ_ERR_OVERFLOW;
    if (cols > 0 && matrices * rows > (1ll << 59) / cols) return NQ_ERR_OVERFLOW;
    return NQ_OK;
}

int check_plan(const nq_moe_plan *p) {
    if (!p) return NQ_ERR_NULL_ARG;
    if (p->tokens < 0 || p->top < 1 || p->experts < 1) return NQ_ERR_BAD_DIM;
    if (p->top > MOST_TOP || p->tokens > MOST / p->top || p->experts > MOST_EXPERTS) return NQ_ERR_OVERFLOW;
    if (!p->offsets || (p->tokens > 0 && (!p->order || !p->places))) return NQ_ERR_NULL_ARG;
    if (((uintptr_t)p->order | (uintptr_t)p->places | (uintptr_t)p->offsets) % 4) return NQ_ERR_MISALIGNED;
    return NQ_OK;
}

// The checks that the product and its workspace share, and its plan.
int check_gemm(const nq_fp8_block_args *x, const nq_moe_plan *plan, nq::Fp8Plan *p) {
    if (!x) return NQ_ERR_NULL_ARG;
    const bool codes = x->x_scales != nullptr;
    if ((!codes && bad_dtype(x->x_dtype)) || bad_dtype(x->out_dtype)) return NQ_ERR_BAD_DTYPE;
    if (x->rows < 0 || x->N < 1 || x->K < 1 || (x->gated != 0 && x->gated != 1) || (x->sorted != 0 && x->sorted != 1))
        return NQ_ERR_BAD_DIM;
    if (x->K % nq::FB != 0 || (x->gated && x->N % (2 * nq::FB) != 0)) return NQ_ERR_NOT_BLOCK_ALIGNED;
    if (x->rows > MOST || x->N > MOST || x->K > MOST_K || x->rows > MOST / (x->K / nq::FB)) return NQ_ERR_OVERFLOW;
    int64_t out_rows = x->rows, experts = 0;
    if (plan) {
        const int st = check_plan(plan);
        if (st != NQ_OK) return st;
        out_rows = plan->tokens * plan->top;
        experts = plan->experts;
        if (x->rows != (x->sorted ? out_rows : plan->tokens)) return NQ_ERR_BAD_DIM;
    } else if (x->sorted) {
        return NQ_ERR_BAD_DIM;
    }
    const int st = check_stride(x->x_row_stride, x->rows);
    if (st != NQ_OK) return st;
    if (out_rows > 0 && x->N > (1ll << 55) / out_rows) return NQ_ERR_OVERFLOW;
    const int64_t esz = codes ? 1 : element_size(x->x_dtype);
    if (codes && x->x_row_stride % 16 != 0) return NQ_ERR_MISALIGNED;
    const bool raw = (uintptr_t)x->x % 16 == 0 && x->x_row_stride * esz % 16 == 0;
    *p = nq::fb_plan(x->rows, out_rows, experts, x->N, x->K, x->gated != 0, codes, raw, x->out_dtype == NQ_F32,
                     x->rows > 0 && (x->rows - 1) * x->x_row_stride + x->K > 1ll << 32, nq::device_compute_units());
    if (p->few) {
        const int64_t groups = nq::fb_ceil(x->gated ? x->N / 2 : x->N, nq::fb_few_cols(p->weight_tiles, x->gated != 0));
        if (groups > THREADS / (64 * p->waves) || p->tiles_m > 65535) return NQ_ERR_OVERFLOW;
    } else {
        const nq::Fp8Config &c = nq::fb_configs[p->config];
        const int64_t most = THREADS / c.threads - nq::FB_XCDS * nq::FB_MOST_SPAN;  // (the grid is whole turns of the XCDs)
        if (nq::fb_ceil(x->N, c.cols) > most / (p->tiles_m > 0 ? p->tiles_m : 1)) return NQ_ERR_OVERFLOW;
    }
    return NQ_OK;
}

int check_rows(const nq_moe_plan *plan, int32_t dtype, int64_t cols) {
    if (bad_dtype(dtype)) return NQ_ERR_BAD_DTYPE;
    if (cols < 0) return NQ_ERR_BAD_DIM;
    if (cols > MOST) return NQ_ERR_OVERFLOW;
    return check_plan(plan);
}

void take_plan(const nq_moe_plan *p, nq::MoeRowsLaunch *L) {
    L->places = p->places;
    L->offsets = p->offsets;
    L->tokens = p->tokens;
    L->pairs = p->tokens * p->top;
    L->top = (int32_t)p->top;
    L->experts = (int32_t)p->experts;
}

}  // namespace

NQ_API int nq_quantize_fp8_block(const void *x, int32_t in_dtype, int64_t matrices, int64_t rows, int64_t cols,
                                 int64_t row_stride, int32_t tile, void *codes, float *scales, hipStream_t stream) {
    int st = check_blocks(in_dtype, matrices, rows, cols, tile);
    if (st != NQ_OK) return st;
    if ((st = check_stride(row_stride, matrices * rows)) != NQ_OK) return st;
    if (matrices * rows * cols == 0) return NQ_OK;
    if (!x || !codes || !scales) return NQ_ERR_NULL_ARG;
    if ((uintptr_t)x % element_size(in_dtype) || (uintptr_t)codes % 16 || (uintptr_t)scales % 4) return NQ_ERR_MISALIGNED;
    nq::Fp8QuantLaunch L = {};
    L.x = x;
    L.row_stride = row_stride;
    L.rows = rows, L.cols = cols, L.matrices = matrices;
    L.codes = (uint8_t *)codes;
    L.scales = scales;
    L.in_dtype = in_dtype, L.tile = tile;
    return nq::launch_fp8_quantize(L, stream);
}

NQ_API int nq_dequantize_fp8_block(const void *codes, const float *scales, int64_t matrices, int64_t rows, int64_t cols,
                                   int32_t tile, int32_t out_dtype, void *out, hipStream_t stream) {
    const int st = check_blocks(out_dtype, matrices, rows, cols, tile);
    if (st != NQ_OK) return st;
    if (matrices * rows * cols == 0) return NQ_OK;
    if (!codes || !scales || !out) return NQ_ERR_NULL_ARG;
    if ((uintptr_t)codes % 16 || (uintptr_t)scales % 4 || (uintptr_t)out % 16) return NQ_ERR_MISALIGNED;
    nq::Fp8ValuesLaunch L = {};
    L.codes = (const uint8_t *)codes;
    L.scales = scales;
    L.out = out;
    L.rows = rows, L.cols = cols, L.matrices = matrices;
    L.out_dtype = out_dtype, L.tile = tile;
    return nq::launch_fp8_values(L, stream);
}

NQ_API int nq_gemm_fp8_block_workspace(const nq_fp8_block_args *args, const nq_moe_plan *plan, uint64_t *bytes) {
    if (!bytes) return NQ_ERR_NULL_ARG;
    *bytes = 0;
    nq::Fp8Plan p = {};
    const int st = check_gemm(args, plan, &p);
    if (st != NQ_OK) return st;
    *bytes = p.codes_bytes + p.scales_bytes + p.part_bytes;
    return NQ_OK;
}

NQ_API int nq_gemm_fp8_block(const nq_fp8_block_args *args, const nq_moe_plan *plan, void *workspace,
                             uint64_t workspace_bytes, hipStream_t stream) {
    nq::Fp8Plan p = {};
    const int st = check_gemm(args, plan, &p);
    if (st != NQ_OK) return st;
    const nq_fp8_block_args &x = *args;
    const bool codes = x.x_scales != nullptr;
    if (!x.weight || !x.weight_scales || (x.rows > 0 && (!x.x || !x.out))) return NQ_ERR_NULL_ARG;
    const uintptr_t esz = codes ? 16 : (uintptr_t)element_size(x.x_dtype);
    if ((uintptr_t)x.x % esz || (uintptr_t)x.weight % 16 || (uintptr_t)x.out % 16 || (uintptr_t)workspace % 16 ||
        ((uintptr_t)x.x_scales | (uintptr_t)x.weight_scales) % 4)
        return NQ_ERR_MISALIGNED;
    const uint64_t need = p.codes_bytes + p.scales_bytes + p.part_bytes;
    if (need > 0 && (!workspace || workspace_bytes < need)) return NQ_ERR_SCRATCH;
    if (x.rows == 0) return NQ_OK;
    nq::Fp8GemmLaunch L = {};
    L.x = x.x;
    L.x_stride = x.x_row_stride;
    L.x_scales = x.x_scales;
    L.x_type = codes ? nq::FB_CODES : x.x_dtype;
    L.w = (const uint8_t *)x.weight;
    L.w_scales = x.weight_scales;
    L.out = x.out;
    L.x_rows = x.rows;
    L.out_rows = plan ? plan->tokens * plan->top : x.rows;
    L.N = (int32_t)x.N, L.K = (int32_t)x.K;
    if (plan) {
        L.experts = (int32_t)plan->experts, L.top = (int32_t)plan->top;
        L.order = x.sorted ? nullptr : plan->order;
        L.offsets = plan->offsets;
    }
    L.out_dtype = x.out_dtype, L.gated = x.gated;
    L.tiles_m = p.tiles_m, L.waves = p.waves, L.splits = p.splits, L.per_split = p.per_split;
    L.part = (float *)((uint8_t *)workspace + p.codes_bytes + p.scales_bytes);
    if (p.quantize) {
        nq::Fp8QuantLaunch q = {};
        q.x = x.x;
        q.row_stride = x.x_row_stride;
        q.rows = x.rows, q.cols = x.K, q.matrices = 1;
        q.codes = (uint8_t *)workspace;
        q.scales = (float *)((uint8_t *)workspace + p.codes_bytes);
        q.in_dtype = x.x_dtype, q.tile = 1;
        const int qs = nq::launch_fp8_quantize(q, stream);
        if (qs != NQ_OK) return qs;
        L.x = q.codes, L.x_stride = x.K, L.x_type = nq::FB_CODES;
        L.x_scales = q.scales;
    }
    return p.few ? nq::launch_fp8_few(L, p.weight_tiles, stream) : nq::launch_fp8_rows(L, p.config, stream);
}

NQ_API int nq_moe_sort_workspace(int64_t tokens, int64_t top, int64_t experts, uint64_t *bytes) {
    if (!bytes) return NQ_ERR_NULL_ARG;
    *bytes = 0;
    if (tokens < 0 || top < 1 || experts < 1) return NQ_ERR_BAD_DIM;
    if (top > MOST_TOP || tokens > MOST / top || experts > MOST_EXPERTS) return NQ_ERR_OVERFLOW;
    const int64_t chunks = nq::fb_ceil(tokens * top, nq::moe_chunk(tokens * top));
    if (chunks > 1) *bytes = (uint64_t)chunks * experts * 4;
    return NQ_OK;
}

NQ_API int nq_moe_sort(const void *ids, int32_t wide, int64_t tokens, int64_t top, int64_t experts, int32_t *order,
                       int32_t *places, int32_t *offsets, void *workspace, uint64_t workspace_bytes, hipStream_t stream) {
    uint64_t need = 0;
    const int st = nq_moe_sort_workspace(tokens, top, experts, &need);
    if (st != NQ_OK) return st;
    if (wide != 0 && wide != 1) return NQ_ERR_BAD_DTYPE;
    if (!offsets || (tokens > 0 && (!ids || !order || !places))) return NQ_ERR_NULL_ARG;
    if ((uintptr_t)ids % (wide ? 8 : 4) || ((uintptr_t)order | (uintptr_t)places | (uintptr_t)offsets | (uintptr_t)workspace) % 4)
        return NQ_ERR_MISALIGNED;
    if (need > 0 && (!workspace || workspace_bytes < need)) return NQ_ERR_SCRATCH;
    nq::MoeSortLaunch L = {};
    L.ids = ids;
    L.order = order, L.places = places, L.offsets = offsets;
    L.counts = (int32_t *)workspace;
    L.pairs = tokens * top;
    L.experts = (int32_t)experts, L.wide = wide;
    L.chunk = nq::moe_chunk(L.pairs);
    L.chunks = need > 0 ? (int32_t)nq::fb_ceil(L.pairs, L.chunk) : 1;
    return nq::launch_moe_sort(L, stream);
}

NQ_API int nq_moe_gather(const nq_moe_plan *plan, const void *x, int64_t row_bytes, int64_t row_stride_bytes, void *out,
                         hipStream_t stream) {
    int st = check_plan(plan);
    if (st != NQ_OK) return st;
    if (row_bytes < 0) return NQ_ERR_BAD_DIM;
    if (row_bytes > 4 * MOST) return NQ_ERR_OVERFLOW;
    if ((st = check_stride(row_stride_bytes, plan->tokens)) != NQ_OK) return st;
    if (plan->tokens == 0 || row_bytes == 0) return NQ_OK;
    if (!x || !out) return NQ_ERR_NULL_ARG;
    nq::MoeRowsLaunch L = {};
    take_plan(plan, &L);
    L.x = x, L.x_stride = row_stride_bytes;
    L.cols = row_bytes;
    L.out = out;
    return nq::launch_moe_gather(L, stream);
}

NQ_API int nq_moe_combine(const nq_moe_plan *plan, const void *rows, int64_t row_stride, int32_t dtype, int64_t cols,
                          const float *weights, void *out, hipStream_t stream) {
    int st = check_rows(plan, dtype, cols);
    if (st != NQ_OK) return st;
    if ((st = check_stride(row_stride, plan->tokens * plan->top)) != NQ_OK) return st;
    if (plan->tokens == 0 || cols == 0) return NQ_OK;
    if (!rows || !out) return NQ_ERR_NULL_ARG;
    const int64_t esz = element_size(dtype);
    if (((uintptr_t)rows | (uintptr_t)out) % esz || (uintptr_t)weights % 4) return NQ_ERR_MISALIGNED;
    nq::MoeRowsLaunch L = {};
    take_plan(plan, &L);
    L.rows = rows, L.rows_stride = row_stride;
    L.weights = weights;
    L.out = out;
    L.cols = cols, L.dtype = dtype;
    L.vec = ((uintptr_t)rows | (uintptr_t)out) % 16 == 0 && row_stride * esz % 16 == 0 && cols % 8 == 0;
    return nq::launch_moe_combine(L, stream);
}

NQ_API int nq_moe_combine_grad(const nq_moe_plan *plan, const void *grad, int64_t grad_stride, const void *rows,
                               int64_t row_stride, int32_t dtype, int64_t cols, const float *weights, void *grad_rows,
                               float *grad_weights, hipStream_t stream) {
    int st = check_rows(plan, dtype, cols);
    if (st != NQ_OK) return st;
    if ((st = check_stride(grad_stride, plan->tokens)) != NQ_OK) return st;
    if ((st = check_stride(row_stride, plan->tokens * plan->top)) != NQ_OK) return st;
    if (plan->tokens == 0) return NQ_OK;
    if (cols > 0 && (!grad || !grad_rows || (grad_weights && !rows))) return NQ_ERR_NULL_ARG;
    const int64_t esz = element_size(dtype);
    if (((uintptr_t)grad | (uintptr_t)rows | (uintptr_t)grad_rows) % esz || ((uintptr_t)weights | (uintptr_t)grad_weights) % 4)
        return NQ_ERR_MISALIGNED;
    nq::MoeRowsLaunch L = {};
    take_plan(plan, &L);
    L.x = grad, L.x_stride = grad_stride;
    L.rows = rows, L.rows_stride = row_stride;
    L.weights = weights;
    L.out = grad_rows;
    L.out_weights = grad_weights;
    L.cols = cols, L.dtype = dtype;
    L.vec = ((uintptr_t)grad | (uintptr_t)rows | (uintptr_t)grad_rows) % 16 == 0 && grad_stride * esz % 16 == 0 &&
            row_stride * esz % 16 == 0 && cols % 8 == 0;
    return nq::launch_moe_combine_grad(L, stream);
}
