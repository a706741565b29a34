// nq_fp8_emu.hip -- host run of the E4M3 products' plan, of their tiles' places and of the experts' tile rule (test
// infrastructure).  Built host-only.
#include "../../block_quantized_weight_nq_amd/csrc/nq_fp8b.h"

#define EMU_API extern "C" __attribute__((visibility("default")))

namespace nq {

// The tile rule one expert after another: the oracle of the wave's search.
template <typename At>
static Fp8Tile fb_find_tile_host(At at, int32_t experts, int64_t rows, int32_t bm, int64_t t) {
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

// Sixty-four lanes in a loop: what the kernels' wave does in fb_find_tile_by.
struct HostWave {
    struct Lanes {
        int32_t v[64];
    };
    template <typename F>
    static Lanes each(F f) {
        Lanes l;
        for (int i = 0; i < 64; i++) l.v[i] = f(i);
        return l;
    }
    static int32_t own(const Lanes &l, int i) { return l.v[i]; }
    static Lanes scan(const Lanes &l) {
        Lanes s;
        uint32_t sum = 0;
        for (int i = 0; i < 64; i++) s.v[i] = (int32_t)(sum += (uint32_t)l.v[i]);
        return s;
    }
    static uint64_t above(const Lanes &l, int32_t t) {
        uint64_t m = 0;
        for (int i = 0; i < 64; i++) m |= (uint64_t)(l.v[i] > t) << i;
        return m;
    }
    static int32_t lane(const Lanes &l, int i) { return l.v[i]; }
};

}  // namespace nq

// The kernels' search for one tile: expert, first, count; and the rule's.
EMU_API void nq_fp8_emu_search(const int32_t *offsets, int experts, int64_t rows, int bm, int32_t t, int64_t *found, int64_t *rule) {
    const auto at = [&](int i) { return (int64_t)offsets[i]; };
    const nq::Fp8Tile x = nq::fb_find_tile_by<nq::HostWave>(at, experts, rows, bm, t), y = nq::fb_find_tile_host(at, experts, rows, bm, t);
    found[0] = x.expert, found[1] = x.first, found[2] = x.count;
    rule[0] = y.expert, rule[1] = y.first, rule[2] = y.count;
}

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
