// nq_kv.h -- the 8-bit key/value cache: layouts, host-checkable index rules and launch arguments.
//
// A cache is a pool of blocks of T tokens (T = 16, 32, 64 or 128).  A block
// holds, for each of H key/value heads, T x D key codes ([T][D], a token's
// codes contiguous) and D x T value codes ([D][T], a channel's tokens
// contiguous), one binary32 scale for its keys and one for its values.  A
// code c stands for RN32(c * scale); c is a signed byte in -127..127 or an
// E4M3FN word.  The two layouts are the ones the attention's matrix
// instructions read without a transpose: scores contract over the channels of
// a key, outputs over the tokens of a channel.
//
// The functions marked NQ_HD decide which bytes a kernel touches; a host
// build runs them to check every address against the buffers.
#pragma once

#include "nq_decode.h"

namespace nq {

constexpr int KV_Q8 = 0, KV_E4M3 = 1;
constexpr float KV_TINY = 1.17549435082228750797e-38f;  // 2^-126, the least scale

// Status bits the kernels set.
constexpr uint32_t KV_ST_NOT_FINITE = 1u, KV_ST_BAD_SLOT = 2u;                     // store
constexpr uint32_t KV_ST_NO_BLOCKS = 1u, KV_ST_BAD_LENGTH = 2u, KV_ST_TOKENS = 4u, KV_ST_RING = 8u;  // tables

struct KvPool {
    uint8_t *k, *v;
    float *ks, *vs;
    int64_t blocks;
    uint32_t heads, dim, bsh;  // T = 1 << bsh
};

// Byte offset of (block, head) in either code pool.
NQ_HD int64_t kv_tile_at(const KvPool &c, int64_t block, uint32_t head) {
    return (block * (int64_t)c.heads + (int64_t)head) * (int64_t)((uint64_t)c.dim << c.bsh);
}

// ---------------------------------------------------------------------------
// Store: which tokens a workgroup writes
// ---------------------------------------------------------------------------
// A request's tokens are consecutive positions, so the blocks they fall into
// follow from the offset of its first token.  n tokens touch at most
// floor(n / T) + 2 blocks, so request r owns the units floor(s_r / T) + 2 r
// up to those of request r + 1: the launch needs no host copy of the starts.
NQ_HD int64_t kv_unit_first(int64_t start, int64_t r, uint32_t bsh) { return (start >> bsh) + 2 * r; }

// The request of a unit, among requests [lo, lo + n), by a workgroup: its threads look at every step-th of them; `hits`
// have a first unit at or before this one (the starts are sorted, so these are the first), and the request is the last of
// them or one of those up to the next that was looked at.  Whatever the starts are, [lo, lo + n) stays inside itself.
NQ_HD int32_t kv_probe_step(int32_t n, int32_t threads) { return (n - 1) / threads + 1; }
NQ_HD void kv_narrow(int32_t *lo, int32_t *n, int32_t step, int32_t hits) {
    const int32_t skip = (hits - 1) * step;
    *lo += skip;
    *n = *n - skip < step ? *n - skip : step;
}

// Tokens [lo, hi) of unit j of a request whose tokens are [s0, s1) and whose
// first one sits at offset off0 of its block.
NQ_HD void kv_unit_tokens(int64_t s0, int64_t s1, int64_t j, int64_t off0, uint32_t bsh, int64_t *lo, int64_t *hi) {
    const int64_t T = (int64_t)1 << bsh;
    const int64_t a = s0 + j * T - off0, b = a + T;
    *lo = a > s0 ? a : s0;
    *hi = b < s1 ? b : s1;
}

// ---------------------------------------------------------------------------
// Attention: which keys a row tile reads
// ---------------------------------------------------------------------------
// The rows of a request and key head are its new tokens times the query heads
// that share the key head, token-major; a tile is ROWS of them.
struct KvTile {
    int rows;         // rows of the request (all tiles)
    int base;         // position of the request's first new token (negative if it has fewer keys than new tokens)
    int live;         // keys the request has
    int first, last;  // the tile's first and last new token
    int kb;           // first key that some row sees
    int kbeg, kend;   // keys the tile reads: kbeg is kb rounded down to a multiple of 64
    int nsplit;       // pieces of `chunk` keys, at least 1
};

NQ_HD KvTile kv_tile(int added, int length, int cap, int group, int tile, int ROWS, int window, int chunk) {
    KvTile t;
    t.rows = added * group;
    t.base = length - added;
    t.live = length < cap ? length : cap;
    if (t.live < 0) t.live = 0;
    const int row0 = tile * ROWS;
    const int rowl = (row0 + ROWS < t.rows ? row0 + ROWS : t.rows) - 1;
    t.first = row0 / group;
    t.last = rowl / group;
    int kend = t.base + t.last + 1;
    if (kend > t.live) kend = t.live;
    t.kend = kend < 0 ? 0 : kend;
    int kb = window > 0 ? t.base + t.first - window + 1 : 0;
    if (kb > t.kend) kb = t.kend;
    t.kb = kb < 0 ? 0 : kb;
    t.kbeg = t.kb & ~63;
    t.nsplit = (t.kend - t.kbeg + chunk - 1) / chunk;
    if (t.nsplit < 1) t.nsplit = 1;
    return t;
}

// The table entry that names the block of key position `key`, kept inside the
// entries of the tile's keys, and the block it names, or -1 where the tile
// must not look: past its keys, before its window, or where the table names no
// block of the pool.  Two steps, so that a kernel can have entries on their
// way while it works on others.
NQ_HD int kv_entry(int key, const KvTile &t, uint32_t bsh) {
    const int last = (t.kend - 1) >> bsh, i = key >> bsh;
    return i < last ? i : last < 0 ? 0 : last;
}
NQ_HD int kv_named(int entry, int key, const KvTile &t, uint32_t bsh, int64_t blocks) {
    if (key >= t.kend || (((key >> bsh) + 1) << bsh) <= t.kb) return -1;
    return entry >= 0 && (int64_t)entry < blocks ? entry : -1;
}

// Byte offsets of a key's codes and of a channel's codes from token `key` on,
// in the block `page` that kv_named named (block 0 stands in for -1: what is
// read there is masked).
NQ_HD int64_t kv_k_at(const KvPool &c, int page, uint32_t head, int key) {
    return kv_tile_at(c, page < 0 ? 0 : page, head) + (int64_t)(key & ((1 << c.bsh) - 1)) * c.dim;
}
NQ_HD int64_t kv_v_at(const KvPool &c, int page, uint32_t head, int channel, int key) {
    return kv_tile_at(c, page < 0 ? 0 : page, head) + ((int64_t)channel << c.bsh) + (key & ((1 << c.bsh) - 1));
}

// ---------------------------------------------------------------------------
// Attention for many rows: who stages what
// ---------------------------------------------------------------------------
// NW waves stage the codes of 64 keys.  All pieces of a wave lie in the same
// 16 keys (its `sub`, shared by PER waves, of which it is `part`), so a tile
// takes it one table entry.  A piece of the keys is 1 KB in a row (KL keys),
// one of the values 16 keys of 64 channels; 16 bytes of it are a lane's.
template <int DIM, int NW>
struct KvRows {
    static constexpr int KT = 64, ROWS = 32 * NW;
    static constexpr int PER = NW / 4;                      // waves that stage 16 keys
    static constexpr int KL = 1024 / DIM;                   // keys of a 1 KB piece
    static constexpr int NL = 16 / (PER * KL);              // a wave's pieces of the keys, and of the values
    static constexpr int KS = DIM + 8, VS = KT + 8;         // row strides in LDS, binary16 elements
    static constexpr int K_ELEMS = KT * KS, V_ELEMS = DIM * VS;
    static constexpr int SC = 20;                           // floats of a buffer's scales
    static constexpr int LDS_BYTES = 2 * (K_ELEMS + V_ELEMS) * 2 + 2 * SC * 4;
    static_assert(NL >= 1 && NL * PER * KL == 16 && NL * PER * 64 == DIM, "the waves share 16 keys evenly");

    // byte offsets of a lane's part of piece n: in the codes of 16 keys, and in those of DIM channels from a key on
    NQ_HD static uint32_t k_from(int part, int lane, int n) { return (uint32_t)((part * NL + n) * 1024 + 16 * lane); }
    NQ_HD static uint32_t v_from(int part, int lane, int n, uint32_t bsh) { return (uint32_t)(64 * (part * NL + n) + lane) << bsh; }
    // its places in the LDS buffers, in elements
    NQ_HD static int k_put(int sub, int part, int lane, int n) {
        return (16 * sub + (part * NL + n) * KL + lane / (DIM / 16)) * KS + 16 * (lane % (DIM / 16));
    }
    NQ_HD static int v_put(int sub, int part, int lane, int n) { return (64 * (part * NL + n) + lane) * VS + 16 * sub; }
    // the block that kv_named named (block 0 for none), and a key's codes in a block
    NQ_HD static uint64_t block_at(const KvPool &c, int page) {
        return (uint64_t)(uint32_t)(page < 0 ? 0 : page) * (c.heads * ((uint32_t)DIM << c.bsh));  // 2^16 * 2^15 at most
    }
    NQ_HD static uint32_t k_at(int key, uint32_t bsh) { return (uint32_t)(key & ((1 << bsh) - 1)) * DIM; }
    NQ_HD static uint32_t v_at(int key, uint32_t bsh) { return (uint32_t)(key & ((1 << bsh) - 1)); }
};

// ---------------------------------------------------------------------------
// Launch arguments
// ---------------------------------------------------------------------------
struct KvTablesLaunch {
    const int32_t *lengths, *added;
    int32_t *table, *ring;
    const int32_t *state;
    int32_t *lengths_out, *starts;
    int64_t *slots;
    int32_t *state_out;
    uint32_t *status;
    int64_t table_stride, tokens;
    int32_t requests, width, ring_size;
    uint32_t bsh;
};
int launch_kv_tables(const KvTablesLaunch &L, hipStream_t s);

struct KvStoreLaunch {
    KvPool c;
    const void *x[2];           // new keys, new values
    int64_t ts[2], hs[2];       // their token and head strides in elements
    const int64_t *slots;
    const int32_t *starts;
    uint32_t *status;
    int64_t tokens;
    int32_t requests, code, in_dtype;
};
int launch_kv_store(const KvStoreLaunch &L, hipStream_t s);

struct KvLoadLaunch {
    KvPool c;
    const int32_t *ids;
    void *out[2];
    int64_t n;
    int32_t code, out_dtype;
    int32_t group;  // heads of a workgroup
};
int launch_kv_load(const KvLoadLaunch &L, hipStream_t s);

struct KvAttnLaunch {
    KvPool c;
    const void *q;
    int64_t q_ts, q_hs;  // token and head strides of q in elements
    const int32_t *starts, *lengths, *table;
    int64_t table_stride;
    void *out;           // [tokens, q_heads, dim], contiguous
    float *lse;          // [tokens, q_heads] or NULL
    float *part;         // normalized outputs of the many-rows kernel's pieces, [tokens, q_heads, splits, dim]
    float *part_lse;     // their base-2 logarithms of the sums, [tokens, q_heads, splits]
    float *few_part;     // likewise of the few-rows kernel, rows as kv_few_row has them, splits_few
    float *few_part_lse;
    int32_t tokens, requests, q_heads, group;
    int32_t cap;         // keys a request can have: max_length, and what its table row can name
    int32_t max_new, window;
    int32_t code, dtype;
    bool q_vec;          // rows of q start on 16-byte boundaries
    float scale;
    // the plan
    int32_t few;         // requests of at most this many rows go to the few-rows kernel
    int32_t waves;       // of a many-rows workgroup, 32 rows each; 0 without such a launch
    int32_t tiles, tiles_few;    // tiles of a request and key head, at most
    int32_t chunk, chunk_few;    // keys of a piece
    int32_t splits, splits_few;  // pieces of a tile, at most
    int32_t few_tokens;  // new tokens of a request that the few-rows kernel can have, or 0: see kv_few_row
};

// A request's token range and length, made safe: starts inside [0, tokens].  Of more than max_new new tokens the first
// max_new are computed, [s0, s1); without the others, up to `end`, the request is one that ends there (len), so the
// positions stay what they are.
struct KvReq {
    int s0, s1, end, len;
};
NQ_HD KvReq kv_request(const KvAttnLaunch &a, int r) {
    KvReq q;
    q.s0 = a.starts[r];
    int s1 = a.starts[r + 1];
    q.len = a.lengths[r];
    q.s0 = q.s0 < 0 ? 0 : q.s0 > a.tokens ? a.tokens : q.s0;
    s1 = s1 < q.s0 ? q.s0 : s1 > 1 << 30 ? 1 << 30 : s1;  // 2^30 tokens at most: no sum below leaves 32 bits
    if (q.len < 0) q.len = 0;
    q.end = s1 > a.tokens ? a.tokens : s1;
    q.s1 = q.end - q.s0 > a.max_new ? q.s0 + a.max_new : q.end;
    q.len -= s1 - q.s1;
    return q;
}

// The place of a row's pieces among the few-rows kernel's: every request has few_tokens * q_heads places, where that
// is less than one for each row of the call (a prompt's rows take none), or (few_tokens = 0) its own rows' places.
NQ_HD int64_t kv_few_row(const KvAttnLaunch &a, int req, int start, int tok, int head) {
    const int64_t at = a.few_tokens > 0 ? (int64_t)req * a.few_tokens : (int64_t)start;
    return (at + tok) * a.q_heads + head;
}
NQ_HD uint64_t kv_part_rows(const KvAttnLaunch &a) { return a.splits > 1 ? (uint64_t)a.tokens * (uint64_t)a.q_heads : 0u; }
NQ_HD uint64_t kv_few_part_rows(const KvAttnLaunch &a) {
    if (a.splits_few <= 1) return 0;
    return (a.few_tokens > 0 ? (uint64_t)a.requests * (uint64_t)a.few_tokens : (uint64_t)a.tokens) * (uint64_t)a.q_heads;
}

// How the work of an attention call is cut: the host knows the bounds
// max_new and max_length, not the lengths themselves (reading those would
// wait for the stream), so every request gets the workgroups of the longest
// one and those past its own end return at once.
//
// Requests of at most `few` rows go to the kernel for few rows, the others to
// the one for many: measured at 32 requests of 2000 to 4000 keys, few against
// many at 64 and 128 rows 84 / 105 and 98 / 131 us (64 channels), 119 / 194
// and 166 / 198 us (128), at 32 and 48 rows 267 / 341 and 358 / 318 us (256).
// Binary32 queries stay with few rows: their second terms cost the other
// kernel its second wave a SIMD.  Built for them too, it measured, few against
// many at 256 rows of such requests, 152 / 199 us (64 channels) and 256 / 386
// us (128), and at 2048 tokens of one request 228 / 231 and 554 / 485 us.
//
// A piece is `chunk` keys: several pieces a row let few rows fill the card,
// each costs a workgroup's start and end and a partial output.  Measured for
// few rows at pieces of 256, 512, 1024, 2048 and 4096 keys: 128 ragged
// requests of up to 8200 keys 127, 99, 86, 82 and 88 us; two of 131001 and
// about 90000 keys 153, 114, 97, 95 and 92 us; 32 requests with 5 tokens and a
// window of 2049 keys 37, 33, 32, 38 and 33 us.  Many rows are cut only where
// the tiles leave compute units idle.
inline void kv_attn_plan(KvAttnLaunch &L, uint32_t cus) {
    const int64_t rows = (int64_t)L.max_new * L.group;
    auto span_of = [&](int64_t tile_rows) {
        const int64_t seen = (int64_t)L.window + tile_rows / L.group + 2 + 63;
        const int64_t span = L.window > 0 && seen < L.cap ? seen : L.cap;
        return span < 1 ? 1 : span;
    };
    auto cut = [](int64_t span, int64_t pieces, int64_t least, int32_t *chunk, int32_t *splits) {
        if (pieces > 65535) pieces = 65535;
        int64_t c = ((span + pieces - 1) / pieces + 63) / 64 * 64;
        if (c < least) c = least;
        *chunk = (int32_t)c;
        *splits = (int32_t)((span + c - 1) / c);
    };
    L.few = L.c.dim == 256 ? 32 : 128;
    L.waves = 0;
    L.tiles = L.splits = 0;
    L.chunk = 256;
    if (L.dtype == 0) L.few = 1 << 30;  // binary32: two terms a row
    if (rows > L.few) {
        L.waves = L.c.dim == 128 ? 8 : 4;
        const int64_t tr = 32 * L.waves;
        const int64_t tiles = (rows + tr - 1) / tr;
        L.tiles = (int32_t)tiles;
        // tiles that have rows, at most
        int64_t busy = (int64_t)L.tokens * L.group / tr + L.requests;
        if (busy > L.requests * tiles) busy = L.requests * tiles;
        busy *= L.c.heads;
        const int64_t want = L.c.dim == 64 ? 2 * cus : cus;  // workgroups that the card holds
        cut(span_of(tr), busy >= want ? 1 : (want + busy - 1) / busy, 512, &L.chunk, &L.splits);
    }
    const int64_t few_rows = rows < L.few ? rows : L.few;
    L.tiles_few = (int32_t)((few_rows + 15) / 16);
    const int64_t span = span_of(16);
    int64_t busy = (int64_t)L.tokens * L.group / 16 + L.requests;
    if (busy > (int64_t)L.requests * L.tiles_few) busy = (int64_t)L.requests * L.tiles_few;
    busy *= L.c.heads;
    // six workgroups a compute unit, and no piece above 2048 keys where lengths differ
    int64_t pieces = busy > 0 ? (6ll * cus + busy - 1) / busy : 1;
    if (L.tiles_few <= 4 && pieces < (span + 2047) / 2048) pieces = (span + 2047) / 2048;
    cut(span, pieces, 512, &L.chunk_few, &L.splits_few);
    const int64_t most = L.few / L.group < L.max_new ? L.few / L.group : L.max_new;
    if (most == 0) L.splits_few = 1;  // a single token has more rows than the few-rows kernel takes
    L.few_tokens = most * L.requests < L.tokens ? (int32_t)most : 0;
}

}  // namespace nq
