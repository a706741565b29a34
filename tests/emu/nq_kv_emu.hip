// nq_kv_emu.hip -- host run of the key/value cache kernels' index rules (test infrastructure).
//
// Walks every workgroup, wave, key tile and lane of a launch with the rules
// of nq_kv.h that the kernels use, and checks each address against the pool.
// Built host-only.
#include <vector>

#include "../../block_quantized_weight_nq_amd/csrc/nq_kv.h"

#define EMU_API extern "C" __attribute__((visibility("default")))

namespace {
struct HostTable {
    const int32_t *row;
    int width;
    long *bad;
    int operator()(int i) const {
        if (i < 0 || i >= width) {
            ++*bad;
            return -1;
        }
        return row[i];
    }
};

int page_of(const HostTable &tab, int key, const nq::KvTile &t, int bsh, int64_t blocks) {
    return nq::kv_named(tab(nq::kv_entry(key, t, (uint32_t)bsh)), key, t, (uint32_t)bsh, blocks);
}
}  // namespace

// How often each token is stored: the units of a store launch over starts
// [requests + 1] with first-token offsets off0.  Returns units outside a request's tokens.
EMU_API long nq_kv_emu_units(const int32_t *starts, int requests, const int32_t *off0, int bsh, int64_t tokens,
                             int32_t *hits) {
    long bad = 0;
    const int64_t units = nq::kv_unit_first(tokens, requests, (uint32_t)bsh);
    for (int64_t u = 0; u < units; u++) {
        int r = -1;
        for (int i = 0; i < requests; i++) r += nq::kv_unit_first(starts[i], i, (uint32_t)bsh) <= u;
        if (r < 0) continue;
        const int64_t s0 = starts[r], s1 = starts[r + 1] < tokens ? starts[r + 1] : tokens;
        if (s0 < 0 || s0 >= s1) continue;
        int64_t lo, hi;
        nq::kv_unit_tokens(s0, s1, u - nq::kv_unit_first(s0, r, (uint32_t)bsh), off0[r], (uint32_t)bsh, &lo, &hi);
        for (int64_t t = lo; t < hi; t++) {
            if (t < s0 || t >= s1)
                bad++;
            else
                hits[t]++;
        }
    }
    return bad;
}

// The addresses of a request and key head in the few-rows attention kernel (key tiles of KT): bytes against the
// pool, table entries against its width.  visits[key] counts the tile-0 visits of every key.
EMU_API long nq_kv_emu_attention(int added, int length, int cap, int group, int window, int chunk, int max_splits,
                                 const int32_t *table, int width, int bsh, int dim, int KT, int heads, int64_t blocks,
                                 int32_t *visits) {
    nq::KvPool c = {};
    c.blocks = blocks;
    c.heads = (uint32_t)heads;
    c.dim = (uint32_t)dim;
    c.bsh = (uint32_t)bsh;
    const int64_t pool = blocks * heads * (int64_t)dim << bsh;
    const int KPG = KT / 4;
    long bad = 0;
    const HostTable tab = {table, width, &bad};
    for (int tile = 0; tile * 16 < added * group; tile++) {
        const nq::KvTile t = nq::kv_tile(added, length, cap, group, tile, 16, window, chunk);
        bad += t.nsplit > max_splits;
        for (int split = 0; split < t.nsplit; split++) {
            const int k0 = t.kbeg + split * chunk, k1 = t.kend - k0 > chunk ? k0 + chunk : t.kend;
            for (int wave = 0; wave < 4; wave++)
                for (int key0 = k0 + wave * KT; key0 < k1; key0 += 4 * KT)
                    for (int lane = 0; lane < 64; lane++)
                        for (int head = 0; head < heads; head += heads > 1 ? heads - 1 : 1) {
                            const int r = lane & 15, g = lane >> 4;
                            const int kp = page_of(tab, key0 + KPG * (r >> 2), t, bsh, blocks);
                            const int64_t k = nq::kv_k_at(c, kp, (uint32_t)head, key0 + KPG * (r >> 2) + (r & 3)) + 16 * g;
                            const int64_t kl = k + 4 * (KT / 16 - 1) * dim + 64 * (dim / 64 - 1) + 16;
                            bad += k < 0 || kl > pool;
                            const int kv0 = key0 + KPG * g;
                            const int vp = page_of(tab, kv0, t, bsh, blocks);
                            const int64_t v = nq::kv_v_at(c, vp, (uint32_t)head, r, kv0);
                            bad += v < 0 || v + ((int64_t)(dim / 16 - 1) << (bsh + 4)) + KPG > pool;
                            bad += vp >= 0 && (kv0 & ((1 << bsh) - 1)) + KPG > (1 << bsh);
                            if (tile == 0 && head == 0 && r == 0 && vp >= 0)
                                for (int i = 0; i < KPG; i++)
                                    if (kv0 + i < t.kend && kv0 + i >= t.kb) visits[kv0 + i]++;
                        }
        }
    }
    return bad;
}
