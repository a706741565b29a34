// nq_kv_plan_emu.hip -- host run of the key/value cache kernels' searches, plans and places (test infrastructure).
// Built host-only.
#include <vector>

#include "../../block_quantized_weight_nq_amd/csrc/nq_kv.h"

#define EMU_API extern "C" __attribute__((visibility("default")))

// The request that a store workgroup of `threads` threads finds for unit u, or -1, by the kernel's rounds; *bad counts
// reads of starts outside its requests + 1 entries, *rounds the rounds before the last.
EMU_API int nq_kv_emu_request(const int32_t *starts, int requests, int64_t u, int bsh, int threads, int32_t *bad,
                              int32_t *rounds) {
    int32_t from = 0, left = requests;
    *bad = *rounds = 0;
    while (left > threads) {
        const int32_t step = nq::kv_probe_step(left, threads);
        int32_t hits = 0;
        for (int32_t tid = 0; tid < threads; tid++) {
            if (tid * step >= left) continue;
            const int32_t i = from + tid * step;
            if (i < 0 || i >= requests)
                ++*bad;
            else
                hits += nq::kv_unit_first(starts[i], i, (uint32_t)bsh) <= u;
        }
        if (hits == 0) return -1;
        nq::kv_narrow(&from, &left, step, hits);
        ++*rounds;
    }
    int found = -1;
    for (int32_t tid = 0; tid < threads && tid < left; tid++) {
        const int32_t i = from + tid;
        if (i < 0 || i >= requests)
            ++*bad;
        else if (nq::kv_unit_first(starts[i], i, (uint32_t)bsh) <= u && u < nq::kv_unit_first(starts[i + 1], i + 1, (uint32_t)bsh))
            found = i;
    }
    return found;
}

namespace {
struct Walk {
    const nq::KvAttnLaunch &a;
    int width;        // entries of a table row
    int64_t pool;     // bytes of either code pool
    uint8_t *places;  // [many-rows pieces, few-rows pieces]: how often each is written
    long bad = 0;

    int entry(int req, int key, const nq::KvTile &t) {
        const int i = nq::kv_entry(key, t, a.c.bsh);
        if (i < 0 || i >= width) {
            bad++;
            return -1;
        }
        return a.table[req * a.table_stride + i];
    }

    void wrote(bool few, int64_t row, int split) {
        const int64_t splits = few ? a.splits_few : a.splits, base = few ? (int64_t)nq::kv_part_rows(a) * a.splits : 0;
        const int64_t rows = (int64_t)(few ? nq::kv_few_part_rows(a) : nq::kv_part_rows(a));
        if (row < 0 || row >= rows || split >= splits)
            bad++;
        else
            bad += places[base + row * splits + split]++ != 0;
    }

    // The rows of a tile whose output goes to the workspace.
    void rows_of(const nq::KvReq &q, const nq::KvTile &t, int req, int tile, int ROWS, bool few, int kv_head) {
        bad += t.nsplit > (few ? a.splits_few : a.splits);
        if (t.nsplit == 1) return;
        for (int row = tile * ROWS; row < t.rows && row < (tile + 1) * ROWS; row++) {
            const int tok = row / a.group, head = kv_head * a.group + row % a.group;
            const int64_t at = few ? nq::kv_few_row(a, req, q.s0, tok, head) : (int64_t)(q.s0 + tok) * a.q_heads + head;
            for (int s = 0; s < t.nsplit; s++) wrote(few, at, s);
        }
    }

    // What a many-rows workgroup's waves stage: every code of each tile's keys once, from its own place.
    template <int DIM, int NW>
    void stage(const nq::KvTile &t, int req, int head, int k0, int k1) {
        using C = nq::KvRows<DIM, NW>;
        const uint32_t bsh = a.c.bsh;
        const int nt = (k1 - k0 + C::KT - 1) / C::KT;
        if (nt <= 0) return;
        for (int j = 0; j < nt + 3; j++) {  // keys are fetched three tiles past the one in work, values two
            const int key0 = k0 + j * C::KT;
            std::vector<uint8_t> kseen(C::K_ELEMS), vseen(C::V_ELEMS);
            for (int wave = 0; wave < NW; wave++) {
                const int sub = wave / C::PER, part = wave % C::PER, key = key0 + 16 * sub;
                const int page = nq::kv_named(entry(req, key, t), key, t, bsh, a.c.blocks);
                for (int lane = 0; lane < 64; lane++)
                    for (int n = 0; n < C::NL; n++) {
                        const int64_t kat = (int64_t)head * (DIM << bsh) + C::k_from(part, lane, 0) + (int64_t)C::block_at(a.c, page) +
                                            C::k_at(key, bsh) + C::k_from(0, 0, n);
                        const int64_t vat = (int64_t)head * (DIM << bsh) + C::v_from(part, lane, 0, bsh) + (int64_t)C::block_at(a.c, page) +
                                            C::v_at(key, bsh) + C::v_from(0, 0, n, bsh);
                        bad += kat < 0 || kat + 16 > pool || vat < 0 || vat + 16 > pool || kat % 16 || vat % 16;
                        const int kput = C::k_put(sub, part, lane, 0) + C::k_put(0, 0, 0, n);
                        const int vput = C::v_put(sub, part, lane, 0) + C::v_put(0, 0, 0, n);
                        if (kput < 0 || kput + 16 > C::K_ELEMS || vput < 0 || vput + 16 > C::V_ELEMS) {
                            bad++;
                            continue;
                        }
                        // the place says which key and channel are meant: the address has to be theirs
                        const int kk = kput / C::KS, kc = kput % C::KS, vc = vput / C::VS, vk = vput % C::VS;
                        bad += kc + 16 > DIM || vk + 16 > C::KT;
                        bad += kat != nq::kv_k_at(a.c, page, (uint32_t)head, key0 + kk) + kc;
                        bad += vat != nq::kv_v_at(a.c, page, (uint32_t)head, vc, key0 + vk);
                        bad += key0 + kk < key || key0 + kk >= key + 16 || key0 + vk != key;
                        for (int i = 0; i < 16; i++) bad += kseen[kput + i]++ + vseen[vput + i]++;
                    }
            }
            for (int k = 0; k < C::KT; k++)
                for (int c = 0; c < DIM; c++) bad += kseen[k * C::KS + c] != 1 || vseen[c * C::VS + k] != 1;
        }
    }
};
}  // namespace

// A call of nq_kv_attention on the host: its plan, the requests' rows, the pieces' places in the workspace (each
// written at most once, and inside) and the many-rows kernel's staging.  Returns what was wrong; rows[t] counts how
// often the row of token t (and the first query head) is computed.
EMU_API long nq_kv_emu_call(const int32_t *starts, const int32_t *lengths, int requests, int tokens, int heads, int group,
                            int dim, int bsh, int dtype, int window, int max_new, int max_length, const int32_t *table,
                            int width, int64_t blocks, int cus, int32_t *rows, int32_t *cuts) {
    nq::KvAttnLaunch L = {};
    L.c.blocks = blocks;
    L.c.heads = (uint32_t)heads;
    L.c.dim = (uint32_t)dim;
    L.c.bsh = (uint32_t)bsh;
    L.starts = starts;
    L.lengths = lengths;
    L.table = table;
    L.table_stride = width;
    L.tokens = tokens;
    L.requests = requests;
    L.q_heads = heads * group;
    L.group = group;
    L.cap = max_length < width << bsh ? max_length : width << bsh;
    L.max_new = max_new < tokens ? max_new : tokens;
    L.window = window;
    L.dtype = dtype;
    nq::kv_attn_plan(L, (uint32_t)cus);
    cuts[0] = L.splits;
    cuts[1] = L.splits_few;
    cuts[2] = L.few_tokens;
    std::vector<uint8_t> places((size_t)(nq::kv_part_rows(L) * (uint64_t)L.splits + nq::kv_few_part_rows(L) * (uint64_t)L.splits_few));
    Walk w{L, width, blocks * heads * ((int64_t)dim << bsh), places.data()};
    for (int req = 0; req < requests; req++) {
        const nq::KvReq q = nq::kv_request(L, req);
        w.bad += q.s0 < 0 || q.s1 < q.s0 || q.end < q.s1 || q.end > tokens || q.s1 - q.s0 > L.max_new;
        const int n = (q.s1 - q.s0) * group;
        if (n == 0) continue;
        const bool few = n <= L.few;
        const int ROWS = few ? 16 : 32 * L.waves, tiles = (n + ROWS - 1) / ROWS;
        w.bad += !few && L.waves == 0;
        w.bad += tiles > (few ? L.tiles_few : L.tiles);
        if (w.bad) return w.bad;
        for (int tile = 0; tile < tiles; tile++) {
            const nq::KvTile t = nq::kv_tile(q.s1 - q.s0, q.len, L.cap, group, tile, ROWS, window, few ? L.chunk_few : L.chunk);
            for (int row = tile * ROWS; row < t.rows && row < (tile + 1) * ROWS; row++)
                if (row % group == 0) rows[q.s0 + row / group]++;
            for (int head = 0; head < heads; head++) {
                w.rows_of(q, t, req, tile, ROWS, few, head);
                if (few || (head > 0 && head < heads - 1)) continue;
                for (int s = 0; s < t.nsplit; s++) {
                    const int k0 = t.kbeg + s * L.chunk, k1 = t.kend - k0 > L.chunk ? k0 + L.chunk : t.kend;
                    if (dim == 64)
                        w.stage<64, 4>(t, req, head, k0, k1);
                    else if (dim == 128)
                        w.stage<128, 8>(t, req, head, k0, k1);
                    else
                        w.stage<256, 4>(t, req, head, k0, k1);
                }
            }
        }
    }
    return w.bad;
}
