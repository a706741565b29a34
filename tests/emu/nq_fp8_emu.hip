// nq_fp8_emu.hip -- host run of the experts' tile rule (test infrastructure).  Built host-only.
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
