// nq_fp8_emu.hip -- host run of the E4M3 products' plan, of their tiles' places and of the experts' tile rule (test
// infrastructure).  Built host-only.
#include "../../block_quantized_weight_nq_amd/csrc/nq_fp8b.h"

#define EMU_API extern "C" __attribute__((visibility("default")))

// The row tiles of a launch: hits and expert of each row; returns the tiles that leave the rows.
EMU_API int64_t nq_fp8_emu_tiles(const int32_t *offsets, int experts, int64_t rows, int bm, int32_t *hits, int32_t *expert) {
    int64_t bad = 0;
    const int64_t n = nq::fb_row_tiles(rows, experts, bm);
    for (int64_t t = 0; t < n + 3; t++) {
        const nq::Fp8Tile x = nq::fb_find_tile_host([&](int i) { return (int64_t)offsets[i]; }, experts, rows, bm, t);
        if (x.count == 0) continue;
        if (x.count < 0 || x.count > bm || x.first < 0 || x.first + x.count > rows || x.expert >= experts || x.expert < -1) {
            bad++;
            continue;
        }
        for (int64_t r = x.first; r < x.first + x.count; r++) {
            if (t < n) hits[r]++;
            expert[r] = x.expert;
        }
    }
    return bad;
}

// The plan's numbers, in the order of the test's names.
EMU_API void nq_fp8_emu_plan(int64_t x_rows, int64_t rows, int64_t experts, int64_t N, int64_t K, int gated, int codes, int raw,
                             int wide, int far, int64_t cus, int64_t *out) {
    const nq::Fp8Plan p = nq::fb_plan(x_rows, rows, experts, N, K, gated, codes, raw, wide, far, cus);
    const int64_t v[] = {p.few, p.weight_tiles, p.config, p.waves, p.splits, p.per_split, p.quantize, p.tiles_m,
                         (int64_t)p.codes_bytes, (int64_t)p.scales_bytes, (int64_t)p.part_bytes,
                         p.few ? nq::fb_few_chunk(rows, p.waves, p.weight_tiles) : 0, p.few ? nq::fb_few_depth(p.weight_tiles) : 0};
    for (int i = 0; i < 13; i++) out[i] = v[i];
}

// How often a grid of the many-rows kernel has each tile [tiles_m, tiles_n]; returns the workgroups outside.
EMU_API int64_t nq_fp8_emu_grid(int64_t tiles_m, int64_t tiles_n, int32_t *hits) {
    const uint32_t span = nq::fb_span(tiles_m * tiles_n);
    const int64_t round = (int64_t)nq::FB_XCDS * span, grid = nq::fb_ceil(tiles_m * tiles_n, round) * round;
    int64_t bad = 0;
    for (int64_t b = 0; b < grid; b++) {
        uint32_t m, n;
        nq::fb_place_tile((uint32_t)b, span, (uint32_t)tiles_m, (uint32_t)tiles_n, &m, &n);
        if (m >= tiles_m) continue;
        if (n >= tiles_n)
            bad++;
        else
            hits[(int64_t)m * tiles_n + n]++;
    }
    return bad;
}
