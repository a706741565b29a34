// nq_fp8b.h -- E4M3 codes with one binary32 scale for each block of 128, and
// rows sorted by expert: what the kernels take, the launch plan and the index
// rules that host and device share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nq {

constexpr int FB = 128;                      // values of a block along a row
constexpr float FB_TINY = 1.17549435e-38f;   // 2^-126, the least scale
constexpr int FB_CODES = 3;                  // x_type of rows that are codes already; 0 to 2 as nq_dtype

struct Fp8QuantLaunch {
    const void *x;      // element (i, r, c) at (i * rows + r) * row_stride + c
    int64_t row_stride;
    int64_t rows, cols, matrices;
    uint8_t *codes;
    float *scales;      // [matrices, ceil(rows / tile), cols / 128]
    int32_t in_dtype, tile;
};

struct Fp8ValuesLaunch {
    const uint8_t *codes;
    const float *scales;
    void *out;
    int64_t rows, cols, matrices;
    int32_t out_dtype, tile;
};

struct Fp8GemmLaunch {
    const void *x;
    int64_t x_stride;                // elements
    const float *x_scales;           // [x_rows, K / 128]
    const uint8_t *w;                // [experts,] N, K
    const float *w_scales;           // [experts,] ceil(N / 128), K / 128
    void *out;                       // [out_rows, N], gated: [out_rows, N / 2]
    float *part;                     // [splits, out_rows, N] sums, where K is split
    const int32_t *order, *offsets;  // experts: the plan; order NULL where rows are sorted
    int64_t x_rows, out_rows;
    int64_t tiles_m;                 // row tiles, the most there can be
    int32_t N, K, experts, top;      // experts 0: one weight for all rows
    int32_t x_type, out_dtype, gated;
    int32_t waves, splits, per_split;  // few rows: waves of a workgroup; many rows: pieces of K and blocks of each
    int32_t span;                      // many rows: consecutive tiles of an XCD
};

// What the host decides from the sizes alone.
struct Fp8Plan {
    int32_t few;        // 1: the kernel for few rows of a weight, 16 * row_tiles of them a workgroup
    int32_t row_tiles;
    int32_t config;     // many rows: 0 is 64, 1 is 128, 2 is 256 rows a workgroup; 3 is 128, and x takes more than 32 bits
    int32_t waves, splits, per_split;
    int32_t quantize;   // 1: a launch of its own makes codes of the rows first
    int64_t tiles_m;
    uint64_t codes_bytes, scales_bytes, part_bytes;  // of the workspace, in this order, each a multiple of 256
};

constexpr int fb_config_rows[4] = {64, 128, 256, 128};     // rows (tokens) of a workgroup's tile
constexpr int fb_config_cols[4] = {128, 128, 256, 128};    // weight rows of it

__host__ __device__ inline int64_t fb_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles that `rows` rows of `experts` segments (and the rows behind the last) can need: a segment of n rows has
// ceil(n / bm) of them.
inline int64_t fb_row_tiles(int64_t rows, int64_t experts, int64_t bm) {
    if (experts == 0) return fb_ceil(rows, bm);
    const int64_t most = rows / bm + experts + 1;
    return rows < most ? rows : most;
}

// The segment and rows of row tile `t` of `bm` rows: expert -1 is what lies behind the last expert's rows (they get 0),
// count 0 that there is no such tile.  `at(i)` reads offset i; whatever it holds, first and count stay within rows.
struct Fp8Tile {
    int32_t expert;
    int64_t first;
    int32_t count;
};

__host__ __device__ inline int64_t fb_clamp(int64_t v, int64_t hi) { return v < 0 ? 0 : v > hi ? hi : v; }

template <typename At>
inline Fp8Tile fb_find_tile_host(At at, int32_t experts, int64_t rows, int32_t bm, int64_t t) {
    for (int32_t e = 0; e <= experts; e++) {
        const int64_t lo = fb_clamp(at(e), rows), hi = e < experts ? fb_clamp(at(e + 1), rows) : rows;
        const int64_t n = hi > lo ? fb_ceil(hi - lo, bm) : 0;
        if (t < n) {
            const int64_t first = lo + t * bm;
            return {e < experts ? e : -1, first, (int32_t)(hi - first < bm ? hi - first : bm)};
        }
        t -= n;
    }
    return {-1, 0, 0};
}

constexpr int64_t FB_FEW_ROWS = 64;  // most rows of a tile of the few-rows kernel

// The launch of a product.  `rows`: output rows; `raw`: the rows of x are values that the few-rows kernel can read 16
// bytes at a time; `wide`: binary32 outputs; `far`: codes that are given
// lie further than 32 bits from the first.
inline Fp8Plan fb_plan(int64_t x_rows, int64_t rows, int64_t experts, int64_t N, int64_t K, bool gated, bool codes, bool raw,
                       bool wide, bool far, int64_t cus) {
    Fp8Plan p = {};
    const int64_t KB = K / FB;
    const int64_t each = experts > 0 ? fb_ceil(rows, experts) : rows;  // rows of a weight, if all have the same
    p.splits = 1, p.per_split = (int32_t)KB;
    if (each <= FB_FEW_ROWS) {
        p.few = 1;
        p.row_tiles = each <= 16 ? 1 : each <= 32 ? 2 : 4;
        p.tiles_m = fb_row_tiles(rows, experts, 16 * p.row_tiles);
        const int64_t groups = fb_ceil(gated ? N / 2 : N, gated ? 16 : 32) * (experts > 0 ? (rows < experts ? rows : experts) : p.tiles_m);
        p.waves = 2;
        while (p.waves < 8 && p.waves < KB && groups * p.waves < cus * 12) p.waves *= 2;
        p.quantize = !codes && (!raw || p.row_tiles > 1);
    } else {
        p.config = each <= 64 ? 0 : each <= 256 ? 1 : 2;
        const int64_t wgs = fb_ceil(N, fb_config_cols[2]) * fb_row_tiles(rows, experts, 256);
        if (p.config == 2 && (wide || wgs < cus)) p.config = 1;
        if (codes ? far : x_rows * K >= 1ll << 32) p.config = 3;
        p.tiles_m = fb_row_tiles(rows, experts, fb_config_rows[p.config]);
        if (experts == 0) {
            const int64_t groups = fb_ceil(N, fb_config_cols[p.config]) * p.tiles_m;
            while (groups * p.splits < cus && KB / (2 * p.splits) >= 4 && p.splits < 16) p.splits *= 2;
            p.per_split = (int32_t)fb_ceil(KB, p.splits);
            p.splits = (int32_t)fb_ceil(KB, p.per_split);
        }
        p.quantize = !codes;
    }
    const auto room = [](uint64_t n) { return (n + 255) / 256 * 256; };
    if (p.quantize) {
        p.codes_bytes = room((uint64_t)x_rows * K);
        p.scales_bytes = room((uint64_t)x_rows * KB * 4);
    }
    if (p.splits > 1) p.part_bytes = room((uint64_t)p.splits * rows * N * 4);
    return p;
}

struct MoeSortLaunch {
    const void *ids;
    int32_t *order, *places, *offsets, *counts;  // counts: [chunks, experts], where there is more than one chunk
    int64_t pairs;
    int32_t experts, wide, chunks;               // wide: ids of 64 bits
};

constexpr int64_t MOE_CHUNK = 4096;  // pairs of a workgroup of the sort

struct MoeRowsLaunch {
    const void *x;        // gather: [tokens], gradient: [tokens] gradients of the tokens, combine: sorted rows
    int64_t x_stride;     // elements (gather: bytes)
    const void *rows;     // gradient: sorted rows, stride `rows_stride`
    int64_t rows_stride;
    const float *weights;
    const int32_t *places, *offsets;
    void *out;            // gather and gradient: [pairs, cols]; combine: [tokens, cols]
    float *out_weights;
    int64_t tokens, cols, pairs;
    int32_t top, experts, dtype, vec;
};

uint32_t device_compute_units();
int launch_fp8_quantize(const Fp8QuantLaunch &L, hipStream_t s);
int launch_fp8_values(const Fp8ValuesLaunch &L, hipStream_t s);
int launch_fp8_few(const Fp8GemmLaunch &L, int row_tiles, hipStream_t s);
int launch_fp8_rows(const Fp8GemmLaunch &L, int config, hipStream_t s);
int launch_moe_sort(const MoeSortLaunch &L, hipStream_t s);
int launch_moe_gather(const MoeRowsLaunch &L, hipStream_t s);
int launch_moe_combine(const MoeRowsLaunch &L, hipStream_t s);
int launch_moe_combine_grad(const MoeRowsLaunch &L, hipStream_t s);

}  // namespace nq
