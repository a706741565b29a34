// nq_fp8b.h -- E4M3 codes with one binary32 scale for each block of 128, and
// rows sorted by expert: what the kernels take, the launch plan and the index
// rules that host and device share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nq {

constexpr int FB = 128;                      // values of a block along a row
constexpr float FB_TINY = 1.17549435e-38f;   // 2^-126, the least scale
constexpr float FB_MOST = 3.40282347e+38f;   // the largest binary32 number
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
    int32_t chunk;                     // few rows: blocks whose codes are in LDS at a time
};

// What the host decides from the sizes alone.
struct Fp8Plan {
    int32_t few;           // 1: the kernel for few rows of a weight, 16 of them a workgroup
    int32_t weight_tiles;  // few rows: tiles of 16 weight rows of a workgroup
    int32_t config;        // many rows: the tile (fb_configs)
    int32_t waves, splits, per_split;
    int32_t quantize;   // 1: a launch of its own makes codes of the rows first
    int64_t tiles_m;
    uint64_t codes_bytes, scales_bytes, part_bytes;  // of the workspace, in this order, each a multiple of 256
};

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
// A wave searches, a lane looks at one expert: `Wave` has numbers of its lanes (Lanes, 32 bits, whose sums wrap) and what
// a wave does with them, each(f) of f(lane), scan, the mask of those above a number, and one lane's.
struct Fp8Tile {
    int32_t expert;
    int64_t first;
    int32_t count;
};

__host__ __device__ inline int64_t fb_clamp(int64_t v, int64_t hi) { return v < 0 ? 0 : v > hi ? hi : v; }

template <typename Wave, typename At>
__host__ __device__ inline Fp8Tile fb_find_tile_by(At at, int32_t experts, int64_t rows, int32_t bm, int32_t t) {
    const int32_t most = (int32_t)rows;  // (at most 2^30)
    uint32_t left = (uint32_t)t;
    for (int32_t e0 = 0; e0 <= experts; e0 += 64) {
        // (two loads that no condition keeps apart)
        const auto lo = Wave::each([&](int lane) {
            const int32_t e = e0 + lane, v = (int32_t)fb_clamp(at(e < experts ? e : experts), most);
            return e <= experts ? v : 0;
        });
        const auto hi = Wave::each([&](int lane) {
            const int32_t e = e0 + lane, v = (int32_t)fb_clamp(at(e < experts ? e + 1 : experts), most);
            return e < experts ? v : e == experts ? most : 0;
        });
        const auto n = Wave::each([&](int lane) {
            const int32_t rows_of = Wave::own(hi, lane) - Wave::own(lo, lane);
            return rows_of > 0 ? (int32_t)((uint32_t)(rows_of + bm - 1) / (uint32_t)bm) : 0;
        });
        const auto sum = Wave::scan(n);
        const uint64_t past = Wave::above(sum, (int32_t)left);
        if (past) {
            const int i = __builtin_ctzll(past);
            const int32_t from = Wave::lane(lo, i), end = Wave::lane(hi, i);
            const int32_t before = (int32_t)((uint32_t)Wave::lane(sum, i) - (uint32_t)Wave::lane(n, i));
            const int64_t first = from + (int64_t)(int32_t)(left - (uint32_t)before) * bm;
            if (first < from || first >= end) break;  // offsets that no sort gives: their sum may have left 32 bits
            return {e0 + i < experts ? e0 + i : -1, first, (int32_t)(end - first < bm ? end - first : bm)};
        }
        left -= (uint32_t)Wave::lane(sum, 63);
    }
    return {-1, 0, 0};
}

// The tiles of the many-rows kernel: rows of x and of the weight, workgroups that a compute unit holds, their threads, and
// the time of one block of 128 columns in us, where compute units have few workgroups and where they have all (measured at
// K = 4096, 1024 to 28672 weight rows, 48 to 8192 rows; times 1.6 for binary32 outputs).  The first and the fourth keep
// three blocks on their way instead of one, which is what calls of few tiles wait for: 77 rows of [4096, 14336] 21.4 us
// with the fourth, 26.0 with the second; 1024 rows of [28672, 4096] 173 and 151 (119 with the third).  The fifth has more
// workgroups at a time, for many experts of few rows (1800 rows of 64 [2048, 1408] 43 us, 51 with the first).  The last is
// the second for x beyond 32 bits.
//
// The model takes the mean load of the compute units, while the one with the most workgroups decides: where tiles are a few
// more than there are units, it is a fifth to a quarter low (1536 rows of gated [2816, 10496], 264 tiles of 82 blocks: 72 us
// for the blocks, while the eight units with two tiles take 94, and the call 93).
struct Fp8Config {
    int32_t rows, cols, held, threads;
    float alone, full;
};
constexpr Fp8Config fb_configs[6] = {{64, 64, 2, 256, 0.30f, 0.42f}, {128, 128, 2, 256, 0.6f, 1.15f}, {256, 256, 1, 512, 1.4f, 1.84f},
                                     {128, 128, 1, 512, 0.34f, 0.55f}, {64, 64, 4, 256, 0.42f, 1.0f}, {128, 128, 2, 256, 0.6f, 1.15f}};
constexpr int FB_WIDEST = 2, FB_FAR = 5;
constexpr int FB_DEEP_BLOCKS = 32;  // most blocks of a piece of K for the first and the fourth: their scales are loaded once

// Most rows of a weight, on average, that the few-rows kernel takes.  One weight: 17 rows are two workgroups' tiles, each of
// which reads it.  Experts whose pairs fall at random (few-rows kernel / many-rows kernel, us; 8 choices): 64 gated
// [2816, 2048] 77 / 78 at 8 rows, 73 / 79 at 12, 91 / 79 at 16, 108 / 80 at 20; 64 [2048, 1408] 42 / 44 at 4, 50 / 44 at 14,
// 55 / 44 at 16; 256 gated [512, 2048] 55 / 62 at 4, 64 / 64 at 14, 71 / 65 at 16.  From 5 to 13 on,
// by the weight, the many-rows kernel is faster: experts with more than 16 rows are read twice.  The border is also where exact
// products end, and is the same for one weight.
constexpr int64_t FB_FEW_ROWS = 16;
constexpr int64_t FB_RAW_VALUES = 16384;  // most values of them that its workgroups make codes of, each for itself

// Workgroup b's tile in the many-rows kernel.  Workgroups go to the eight XCDs in turn; `span` consecutive tiles stay on
// one, and run along FB_GM row tiles first, so that an XCD's L2 has few weight rows and rows of x at a time.  A grid of
// whole turns (FB_XCDS * span) has every tile once; *m is tiles_m where there is none.
constexpr uint32_t FB_XCDS = 8, FB_MOST_SPAN = 32, FB_GM = 8;
inline uint32_t fb_span(int64_t tiles) {
    const int64_t part = tiles / (4 * FB_XCDS);
    return part < 1 ? 1 : part > FB_MOST_SPAN ? FB_MOST_SPAN : (uint32_t)part;
}
__host__ __device__ inline void fb_place_tile(uint32_t b, uint32_t span, uint32_t tiles_m, uint32_t tiles_n, uint32_t *m, uint32_t *n) {
    const uint32_t turn = b / FB_XCDS, q = turn / span, t = (q * FB_XCDS + b % FB_XCDS) * span + (turn - q * span);
    const uint32_t band = t / (FB_GM * tiles_n), in = t - band * FB_GM * tiles_n, first = band * FB_GM;
    const uint32_t high = first >= tiles_m ? 0 : tiles_m - first < FB_GM ? tiles_m - first : FB_GM;
    *n = high > 0 ? in / high : 0;
    *m = high > 0 && *n < tiles_n ? first + in - *n * high : tiles_m;
}

// Blocks of a wave of the few-rows kernel that are on their way, and blocks whose codes its workgroups make at a time: a
// turn of all waves, and all of them where few rows leave room in 16 KB.
__host__ __device__ constexpr int32_t fb_few_depth(int32_t weight_tiles) { return weight_tiles > 2 ? 2 : 3; }
inline int32_t fb_few_chunk(int64_t rows, int32_t waves, int32_t weight_tiles) {
    const int32_t most = rows < 16 ? (int32_t)rows : 16, turn = fb_few_depth(weight_tiles) * waves, fit = 16384 / FB / most;
    return fit > turn ? fit / turn * turn : turn;
}

// Output columns of a workgroup of the few-rows kernel.
inline int64_t fb_few_cols(int32_t weight_tiles, bool gated) { return gated ? 8 * weight_tiles : 16 * weight_tiles; }

// The launch of a product.  `rows`: output rows; `raw`: the rows of x are values that the few-rows kernel can read 16
// bytes at a time; `wide`: binary32 outputs; `far`: codes that are given lie further than 32 bits from the first.
inline Fp8Plan fb_plan(int64_t x_rows, int64_t rows, int64_t experts, int64_t N, int64_t K, bool gated, bool codes, bool raw,
                       bool wide, bool far, int64_t cus) {
    Fp8Plan p = {};
    const int64_t KB = K / FB;
    const int64_t busy = experts > 0 ? (rows < experts ? rows : experts) : 1;  // weights that have rows, at most
    const int64_t each = busy > 0 ? fb_ceil(rows, busy) : 0;                   // rows of a weight, if all have the same
    p.splits = 1, p.per_split = (int32_t)KB;
    if ((experts > 0 ? fb_ceil(rows, experts) : rows) <= FB_FEW_ROWS) {
        p.few = 1;
        p.tiles_m = fb_row_tiles(rows, experts, 16);
        // weight rows of a workgroup: few where more would leave compute units idle ([4096, 14336]: 14.8 us with 16, 18.9
        // with 32), many where there are enough workgroups (gated [28672, 4096]: 26.0 us with 64, 27.4 with 32)
        const int64_t cols = gated ? N / 2 : N;
        p.weight_tiles = 2;
        if (!gated && fb_ceil(cols, 16) * busy <= cus) p.weight_tiles = 1;
        if (gated && fb_ceil(cols, 32) * busy >= cus + cus / 2) p.weight_tiles = 4;
        const int64_t groups = fb_ceil(cols, fb_few_cols(p.weight_tiles, gated)) * busy;
        // waves that share K (one row, us with 2, 4 and 8): [4096, 14336], 256 workgroups, 26.8, 17.7, 15.0; [14336, 4096],
        // 448, 15.1, 14.5, 17.3; gated [28672, 4096], 448, 28.8, 25.8, 32.5; [28672, 4096], 896, 27.0, 27.9, 31.1; gated
        // [57344, 4096], 896, 51.0, 48.4, 58.2.  (Just above a workgroup a unit eight are late: [9216, 4096], 288, 12.2,
        // 11.8, 14.8.)
        p.waves = 4 * groups <= 5 * cus ? 8 : groups <= 3 * cus ? 4 : 2;
        while (p.waves > 1 && p.waves > KB) p.waves /= 2;
        // one row of [28672, 4096] 27.1 us with codes made in each workgroup, 28.7 with a launch before; four rows of
        // [4096, 14336] 20.7 and 17.2
        p.quantize = !codes && (!raw || each * K > FB_RAW_VALUES);
    } else {
        // the least of: rounds of workgroups, with the time of a block between that of few workgroups and of full compute
        // units; half of the weight's bytes, which these times do not have; where K is split, a launch more and each
        // piece's sums written and read
        float least = 0.0f;
        const bool beyond = codes ? far : x_rows * K > 1ll << 32;
        for (int c = 0; c <= FB_FAR; c++) {
            if (beyond ? c != FB_FAR : c == FB_FAR || (wide && c == FB_WIDEST)) continue;
            const Fp8Config &f = fb_configs[c];
            const int64_t tiles = fb_ceil(N, f.cols) * (experts > 0 ? busy * fb_ceil(2 * each + f.rows, 2 * f.rows) : fb_ceil(rows, f.rows));
            for (int s = 1; s <= 16; s *= 2) {
                if (s > 1 && (experts > 0 || KB / s < 4)) break;
                if ((c == 0 || c == 3) && fb_ceil(KB, s) > FB_DEEP_BLOCKS) continue;
                const int64_t slots = cus * f.held, rounds = fb_ceil(tiles * s, slots);
                const float load = (float)(tiles * s) / (float)(rounds * slots);
                float t = (float)(rounds * fb_ceil(KB, s)) * (f.alone + (f.full - f.alone) * load) * (wide ? 1.6f : 1.0f) + 2.5f * (float)rounds;
                t += (float)(busy * N) * (float)K / 9.6e6f;
                if (s > 1) t += 3.5f + (float)(s * rows) * (float)N * 8.0f / 5e6f;
                if (least == 0.0f || t < least) {
                    least = t;
                    p.config = c;
                    p.splits = s;
                }
            }
        }
        p.tiles_m = fb_row_tiles(rows, experts, fb_configs[p.config].rows);
        p.per_split = (int32_t)fb_ceil(KB, p.splits);
        p.splits = (int32_t)fb_ceil(KB, p.per_split);
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
    int64_t pairs, chunk;                        // chunk: pairs of a workgroup
    int32_t experts, wide, chunks;               // wide: ids of 64 bits
};

// Pairs of a workgroup of the sort: MOE_CHUNK, and a multiple of it where there would be more than MOE_CHUNKS workgroups,
// each of which reads the counts of all.
constexpr int64_t MOE_CHUNK = 4096, MOE_CHUNKS = 512;
inline int64_t moe_chunk(int64_t pairs) {
    const int64_t times = fb_ceil(pairs, MOE_CHUNK * MOE_CHUNKS);
    return MOE_CHUNK * (times > 1 ? times : 1);
}

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
int launch_fp8_few(const Fp8GemmLaunch &L, int weight_tiles, hipStream_t s);
int launch_fp8_rows(const Fp8GemmLaunch &L, int config, hipStream_t s);
int launch_moe_sort(const MoeSortLaunch &L, hipStream_t s);
int launch_moe_gather(const MoeRowsLaunch &L, hipStream_t s);
int launch_moe_combine(const MoeRowsLaunch &L, hipStream_t s);
int launch_moe_combine_grad(const MoeRowsLaunch &L, hipStream_t s);

}  // namespace nq
