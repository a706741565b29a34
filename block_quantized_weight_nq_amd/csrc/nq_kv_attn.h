// nq_kv_attn.h -- attention over the 8-bit key/value cache.
//
// For a new token at position p of its request, query head h and key head
// h / group, over the keys j <= p of the request (and j > p - window):
//   s_j = scale * ks_j * sum_c q_c kc_jc,  out = sum_j softmax(s)_j * vs_j * vc_j,
//   lse = ln sum_j exp(s_j),
// with ks, vs the block scales and kc, vc the codes.  A row that sees no key
// gives out = 0 and lse = -inf.
//
// Arithmetic.  A code is exact in binary16, so the products run on
// the binary16 matrix instructions with binary32 accumulation:
//   * a query row is multiplied by a power of two that brings its largest
//     element to [2^14, 2^15) and rounded to binary16, whose least step is
//     2^-24: binary16 queries stay exact (but for subnormals beside elements
//     of 2^15), bfloat16 ones down to 2^-31 of the largest element; a
//     binary32 query is the sum of two terms, off by 2^-22 of an element.
//     What is smaller is off by at most 2^-39 of the largest;
//   * exp(s_j - m) vs_j / vref, at most 1, times 2^14 is rounded to binary16
//     (2^-11 of its value), or to two terms for binary32 queries (2^-22).
//     Weights too small for that precision (below 2^-28 of 1; a wave sees
//     whether its tile has any) are multiplied up and
//     added by products of their own: a channel in which the dominant keys
//     are 0 keeps the relative precision of what is left;
//   * maxima, sums, outputs and the block scales stay in binary32, the
//     running maximum m in base-2 logarithms.
// vref is the largest value scale met so far; like m, it is a factor of the
// running output and is corrected when it grows.
#pragma once

#include "nq_kv_codes.h"

namespace nq {

constexpr float KV_LOG2E = 1.44269504088896340736f, KV_LN2 = 0.69314718055994530942f;
constexpr float KV_PSCALE = 16384.0f;  // 2^14

// Weights (times 2^14) below KV_LEAST lose precision in binary16; KV_UP brings
// the next level to just below 2^14.  A second term is kept times KV_SECOND,
// with a sum of its own, so that it keeps its precision as long as the first.
constexpr float KV_LEAST = 0x1p-14f, KV_UP = 0x1p28f, KV_SECOND = 2048.0f;

struct KvAttnArgs {
    KvAttnLaunch L;
};

// 2^x, v_exp_f32 (1 ulp; results below 2^-126 are 0)
__device__ __forceinline__ float kv_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// The power of two that brings amax to [2^14, 2^15) (1 where amax is 0, infinite or NaN).
__device__ __forceinline__ float kv_row_scale(float amax) {
    const uint32_t e = (__builtin_bit_cast(uint32_t, amax) >> 23) & 0xFFu;
    if (e == 255u || amax == 0.0f) return 1.0f;
    const int s = 127 + 14 + 127 - (int)e;  // e = 0: a subnormal row stays below 2^14
    return bits_f32((uint32_t)(s > 250 ? 250 : s) << 23);
}

// A score's factor (row scale times key scale) kept finite: a query row whose channels of 2^127 meet keys of 0 only
// has scores of 0, not NaN.
constexpr float KV_MOST = 3.40282346638528859812e38f;
__device__ __forceinline__ float kv_finite(float x) { return __builtin_amdgcn_fmed3f(x, -KV_MOST, KV_MOST); }

__device__ __forceinline__ float kv_xor_max(float x, int d) { return fmaxf(x, __shfl_xor(x, d, 64)); }
__device__ __forceinline__ float kv_xor_add(float x, int d) { return x + __shfl_xor(x, d, 64); }

// A request's row of the table.
struct KvTableRow {
    const int32_t *row;
    __device__ __forceinline__ int operator()(int i) const { return row[i]; }
};

// ---------------------------------------------------------------------------
// Few rows: one wave per run of keys
// ---------------------------------------------------------------------------
// A tile is 16 rows (the matrix instruction's width).  A workgroup has four
// waves; wave w takes the key tiles w, w + 4, ... of its piece, keeps its own
// maximum, sum and output, and the four are joined at the end.  Codes go from
// memory to registers in the operands' own order, 16 bytes a lane: nothing is
// staged, so nothing waits but the loads.  Per KT keys (64; 32 for 256
// channels, and for 128 in two terms) with lane = 16 g + r:
//   scores  A = keys [16][32 channels]: row r of key tile t is key KT/4 * (r/4)
//           + 4 t + r%4, channels 64 a + 16 g + 8 b ..+7 for step 2 a + b;
//           the result gives lane (r = query row, g) the keys KT/4 * g + 4 t + i;
//   output  A = values [16 channels][32 keys]: channel 16 dt + r, keys
//           KT/4 * g + 8 b ..+7: just those of the lane's own scores, so the
//           probabilities are the B operand where they are.
// The keys of a lane lie in one block, so its scales are two registers.
template <int CODE, int DIM, int IN, int TERMS>
struct KvDec {
    static constexpr int KT = DIM > 128 || (DIM == 128 && TERMS == 2) ? 32 : 64;  // keys of a tile (32: fewer registers)
    static constexpr int KPG = KT / 4;              // keys of a lane
    static constexpr int NT = KT / 16;              // score tiles
    static constexpr int NA = DIM / 64;             // 16-byte loads of a key
    static constexpr int ND = DIM / 16;             // output tiles
    static constexpr int NB = KT / 32;              // steps of the output product
    static constexpr int OS = DIM + 4;              // row stride of the joined output in LDS
    static constexpr int LDS_FLOATS = 4 * 16 * OS + 2 * 64 + 4;
};

template <int CODE, int DIM, int IN, int TERMS>
__global__ __launch_bounds__(256, DIM > 128 ? 1 : 2) void k_kv_attn_dec(KvAttnArgs args) {
    using C = KvDec<CODE, DIM, IN, TERMS>;
    constexpr int KT = C::KT, KPG = C::KPG, NT = C::NT, NA = C::NA, ND = C::ND, NB = C::NB;
    extern __shared__ float lds[];
    const KvAttnLaunch &a = args.L;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
    const uint32_t head = blockIdx.x % a.c.heads;
    const int tile = (int)(blockIdx.x / a.c.heads), split = (int)blockIdx.y, req = (int)blockIdx.z;
    const int group = a.group;

    auto zeros = [&](int64_t from, int64_t to) {  // outputs of rows that are not computed
        for (int64_t tok = from + tile; tok < to; tok += a.tiles_few)
            for (int i = tid; i < group * DIM; i += 256) {
                const int64_t row = tok * a.q_heads + (int64_t)head * group + i / DIM;
                if constexpr (IN == 0)
                    ((float *)a.out)[row * DIM + i % DIM] = 0.0f;
                else
                    ((uint16_t *)a.out)[row * DIM + i % DIM] = 0;
                if (a.lse && i % DIM == 0) a.lse[row] = -__builtin_inff();
            }
    };
    if (req == a.requests) {  // tokens of no request
        if (split != 0) return;
        const int s = a.starts[a.requests];
        zeros(s < 0 ? 0 : s, a.tokens);
        return;
    }
    const KvReq q = kv_request(a, req);
    if (split == 0 && q.end > q.s1) zeros(q.s1, q.end);
    const int rows = (q.s1 - q.s0) * group;
    if (rows > a.few || tile * 16 >= rows) return;
    const KvTile t = kv_tile(q.s1 - q.s0, q.len, a.cap, group, tile, 16, a.window, a.chunk_few);
    if (split >= t.nsplit) return;
    const int k0 = t.kbeg + split * a.chunk_few;
    const int k1 = t.kend - k0 > a.chunk_few ? k0 + a.chunk_few : t.kend;

    // this lane's query row (as the column of the score tiles); the last row stands in for those past it
    const int row = tile * 16 + r < t.rows ? tile * 16 + r : t.rows - 1, tok = row / group;
    const int p = t.base + tok;
    const int hi = p + 1 < t.live ? p + 1 : t.live;
    const int lo = a.window > 0 && p - a.window + 1 > 0 ? p - a.window + 1 : 0;
    const int all_hi = t.base + t.first + 1 < t.live ? t.base + t.first + 1 : t.live;
    const int all_lo = a.window > 0 ? t.base + t.last - a.window + 1 : 0;
    const KvTableRow table = {a.table + (int64_t)req * a.table_stride};
    const uint32_t bsh = a.c.bsh;
    const int kr = KPG * (r >> 2) + (r & 3);  // key of row r in score tile 0

    kv_u4 K[NT][NA];
    kv_u2 V[ND][NB];
    kv_f4 O[ND];
#pragma unroll
    for (int d = 0; d < ND; d++) O[d] = kv_f4{0, 0, 0, 0};
    float m = -__builtin_inff(), l = 0.0f, vref = KV_TINY;

    // Table entries are read a tile ahead of the codes that they lead to.
    int ek = 0, ev = 0;
    auto find = [&](int key0) {
        ek = table(kv_entry(key0 + KPG * (r >> 2), t, bsh));
        ev = table(kv_entry(key0 + KPG * g, t, bsh));
    };
    auto load_k = [&](int key0) {
        const int pg = kv_named(ek, key0 + KPG * (r >> 2), t, bsh, a.c.blocks);
        const uint8_t *src = a.c.k + kv_k_at(a.c, pg, head, key0 + kr) + 16 * g;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int i = 0; i < NA; i++) K[n][i] = *(const kv_u4 *)(src + 4 * n * DIM + 64 * i);
    };

    int key0 = k0 + wave * KT, at_v = 0;
    if (key0 < k1) find(key0);
    // the row's loads and the table's first, the keys' next, then the row's conversion
    float f[NA][16];
    const int64_t qat = (int64_t)(q.s0 + tok) * a.q_ts + ((int64_t)head * group + row % group) * a.q_hs;
#pragma unroll
    for (int i = 0; i < NA; i++) {
        if (a.q_vec)
            kv_read16<IN, true>(a.q, qat + 64 * i + 16 * g, f[i]);
        else
            kv_read16<IN, false>(a.q, qat + 64 * i + 16 * g, f[i]);
    }
    if (key0 < k1) {
        load_k(key0);
        at_v = ev;
        find(key0 + 4 * KT);
    }
    kv_h8 Q[TERMS][2 * NA];
    float qscale;
    {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < NA; i++)
#pragma unroll
            for (int k = 0; k < 16; k++) amax = fmaxf(amax, fabsf(f[i][k]));
        amax = kv_xor_max(kv_xor_max(amax, 16), 32);
        const float up = kv_row_scale(amax);
        qscale = a.scale * KV_LOG2E / up;
#pragma unroll
        for (int i = 0; i < NA; i++)
#pragma unroll
            for (int k = 0; k < 16; k++) {
                const float x = f[i][k] * up;
                const _Float16 h = (_Float16)x;
                Q[0][2 * i + (k >> 3)][k & 7] = h;
                if constexpr (TERMS == 2) Q[1][2 * i + (k >> 3)][k & 7] = (_Float16)(x - (float)h);
            }
    }
    for (; key0 < k1; key0 += 4 * KT) {
        // values and scales of the lane's own keys
        const int kv0 = key0 + KPG * g;
        const int pg = kv_named(at_v, kv0, t, bsh, a.c.blocks);
        const int64_t sc_at = (int64_t)(pg < 0 ? 0 : pg) * a.c.heads + head;
        float ks = a.c.ks[sc_at], vs = a.c.vs[sc_at];
        if (pg < 0) ks = vs = 0.0f;
        {
            const uint8_t *src = a.c.v + kv_v_at(a.c, pg, head, r, kv0);
#pragma unroll
            for (int d = 0; d < ND; d++) {
                if constexpr (NB == 2) {
                    const kv_u4 w = *(const kv_u4 *)(src + ((int64_t)d << (bsh + 4)));
                    V[d][0] = kv_u2{w[0], w[1]};
                    V[d][NB - 1] = kv_u2{w[2], w[3]};
                } else {
                    V[d][0] = *(const kv_u2 *)(src + ((int64_t)d << (bsh + 4)));
                }
            }
        }
        kv_f4 S[NT];
#pragma unroll
        for (int n = 0; n < NT; n++) {
            S[n] = kv_f4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < NA; i++)
#pragma unroll
                for (int b = 0; b < 2; b++) {
                    const kv_h8 kk = kv_codes8_f16<CODE>(kv_u2{K[n][i][2 * b], K[n][i][2 * b + 1]});
#pragma unroll
                    for (int e = 0; e < TERMS; e++)
                        S[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kk, Q[e][2 * i + b], S[n], 0, 0, 0);
                }
        }
        if (key0 + 4 * KT < k1) load_k(key0 + 4 * KT);
        at_v = ev;
        find(key0 + 8 * KT);

        const float cf = kv_finite(qscale * ks);
        const bool dead = pg < 0;
        const bool edge = key0 < all_lo || key0 + KT > all_hi || __ballot(dead) != 0;
        float top = -__builtin_inff();
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int i = 0; i < 4; i++) S[n][i] *= cf;
        if (edge) {
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int key = kv0 + 4 * n + i;
                    if (dead || key < lo || key >= hi) S[n][i] = -__builtin_inff();
                }
            // codes of places that hold no key may be anything: E4M3's NaN among them
#pragma unroll
            for (int d = 0; d < ND; d++)
#pragma unroll
                for (int b = 0; b < NB; b++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        uint32_t keep = 0;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const int key = kv0 + 8 * b + 4 * h + i;
                            if (!dead && key >= t.kb && key < t.kend) keep |= 0xFFu << (8 * i);
                        }
                        V[d][b][h] &= keep;
                    }
        }
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int i = 0; i < 4; i++) top = fmaxf(top, S[n][i]);
        top = kv_xor_max(kv_xor_max(top, 16), 32);
        const float m1 = fmaxf(m, top), safe = m1 == -__builtin_inff() ? 0.0f : m1;
        const float vr1 = fmaxf(vref, kv_xor_max(kv_xor_max(fabsf(vs), 16), 32));
        const float alpha = kv_exp2(m - safe), beta = alpha * (vref / vr1);
        const float pv = vs / vr1 * KV_PSCALE;
        m = m1;
        vref = vr1;
        l *= alpha;
        float x[NT][4], least = KV_PSCALE;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float e = kv_exp2(S[n][i] - safe);
                l += e;
                x[n][i] = e * pv;
                least = fminf(least, fabsf(x[n][i]));
            }
        // O = O * fo + values * weights * ft: all weights at once, or level by level where some are small
        float fo = beta, ft = 1.0f;
        for (bool slow = __ballot(least < KV_LEAST) != 0;;) {
            float rest[NT][4];
            bool more = false;
            if (slow) {
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        rest[n][i] = fabsf(x[n][i]) < KV_LEAST ? x[n][i] : 0.0f;
                        more |= rest[n][i] != 0.0f;
                        x[n][i] -= rest[n][i];
                    }
            }
            kv_h8 P[TERMS][NB];
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const _Float16 h = (_Float16)x[n][i];
                    P[0][n >> 1][4 * (n & 1) + i] = h;
                    if constexpr (TERMS == 2) P[1][n >> 1][4 * (n & 1) + i] = (_Float16)((x[n][i] - (float)h) * KV_SECOND);
                }
#pragma unroll
            for (int d = 0; d < ND; d++) {
                kv_f4 acc = {0, 0, 0, 0}, acc2 = {0, 0, 0, 0};
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    // keeps the conversion in this loop: hoisted, the values would hold twice the registers
                    asm volatile("" : "+v"(V[d][b]));
                    const kv_h8 vv = kv_codes8_f16<CODE>(V[d][b]);
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, P[0][b], acc, 0, 0, 0);
                    if constexpr (TERMS == 2) acc2 = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, P[1][b], acc2, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float sum = TERMS == 2 ? __builtin_fmaf(acc2[i], 1.0f / KV_SECOND, acc[i]) : acc[i];
                    O[d][i] = __builtin_fmaf(O[d][i], fo, sum * ft);
                }
            }
            if (!slow || !__ballot(more)) break;  // weights are multiples of 2^-149: at most 10 rounds
            fo = 1.0f;
            ft *= 1.0f / KV_UP;
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int i = 0; i < 4; i++) x[n][i] = rest[n][i] * KV_UP;
        }
    }
    l = kv_xor_add(kv_xor_add(l, 16), 32);

    // Join the four waves.
    float *so = lds + wave * 16 * C::OS, *sm = lds + 4 * 16 * C::OS, *sl = sm + 64, *sv = sl + 64;
#pragma unroll
    for (int d = 0; d < ND; d++) *(kv_f4 *)(so + r * C::OS + 16 * d + 4 * g) = O[d];
    if (g == 0) {
        sm[wave * 16 + r] = m;
        sl[wave * 16 + r] = l;
    }
    if (lane == 0) sv[wave] = vref;
    __syncthreads();
    const int orow = tid >> 4, c0 = (tid & 15) * ND;
    if (tile * 16 + orow >= t.rows) return;
    float mm = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < 4; w++) mm = fmaxf(mm, sm[w * 16 + orow]);
    const float safe = mm == -__builtin_inff() ? 0.0f : mm;
    float sum = 0.0f, fw[4], vmax = sv[0];
#pragma unroll
    for (int w = 1; w < 4; w++) vmax = fmaxf(vmax, sv[w]);
#pragma unroll
    for (int w = 0; w < 4; w++) {
        const float e = kv_exp2(sm[w * 16 + orow] - safe);
        sum += e * sl[w * 16 + orow];
        fw[w] = e;
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int w = 0; w < 4; w++) fw[w] = fw[w] * inv * (sv[w] / vmax);  // vmax itself may be near 2^-126: the sum's factor
    const float lse2 = sum == 0.0f ? -__builtin_inff() : safe + __builtin_amdgcn_logf(sum);
    const int otok = (tile * 16 + orow) / group, oh = (int)head * group + (tile * 16 + orow) % group;
    const int64_t oat = (int64_t)(q.s0 + otok) * a.q_heads + oh;
    float res[ND];
#pragma unroll
    for (int i = 0; i < ND; i++) {
        res[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; w++) res[i] += lds[w * 16 * C::OS + orow * C::OS + c0 + i] * fw[w];
        res[i] = res[i] * (1.0f / KV_PSCALE) * vmax;
    }
    if (t.nsplit == 1) {
#pragma unroll
        for (int i = 0; i < ND; i += 4) {
            const float f[4] = {res[i], res[i + 1], res[i + 2], res[i + 3]};
            kv_write4<IN>(a.out, oat * DIM + c0 + i, f);
        }
        if (a.lse && c0 == 0) a.lse[oat] = lse2 * KV_LN2;
    } else {
        const int64_t pat = kv_few_row(a, req, q.s0, otok, oh) * a.splits_few + split;
#pragma unroll
        for (int i = 0; i < ND; i++) a.few_part[pat * DIM + c0 + i] = res[i];
        if (c0 == 0) a.few_part_lse[pat] = lse2;
    }
}

// ---------------------------------------------------------------------------
// Joining the pieces of a row
// ---------------------------------------------------------------------------
// out = sum_s 2^(lse_s - max) out_s / sum_s 2^(lse_s - max) for every new token
// and query head that has more than one piece.  WAVES waves share a row: one
// where there are at most 16 pieces (many short rows: 4096 workgroups took 8 us
// for 128 requests, a quarter of them ended at once), four beyond.
template <int DIM, int IN, int WAVES>
__global__ __launch_bounds__(256) void k_kv_attn_join(KvAttnArgs args) {
    constexpr int PL = DIM / 64;
    __shared__ float so[4][DIM], ssum[4];
    const KvAttnLaunch &a = args.L;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = wave % WAVES, tok = (int)blockIdx.x, req = (int)blockIdx.z;
    const int h = (int)blockIdx.y * (4 / WAVES) + wave / WAVES;
    const KvReq q = kv_request(a, req);
    if (tok >= q.s1 - q.s0 || h >= a.q_heads) return;
    const int row = tok * a.group + h % a.group;
    const bool few = (q.s1 - q.s0) * a.group <= a.few;
    const int ROWS = few ? 16 : 32 * a.waves;
    const KvTile t = kv_tile(q.s1 - q.s0, q.len, a.cap, a.group, row / ROWS, ROWS, a.window, few ? a.chunk_few : a.chunk);
    if (t.nsplit == 1) return;
    const int64_t at = (int64_t)(q.s0 + tok) * a.q_heads + h;
    const int64_t pat = few ? kv_few_row(a, req, q.s0, tok, h) * a.splits_few : at * a.splits;
    const float *pl = (few ? a.few_part_lse : a.part_lse) + pat;
    const float *po = (few ? a.few_part : a.part) + pat * DIM;
    float mm = -__builtin_inff();
    for (int s = lane; s < t.nsplit; s += 64) mm = fmaxf(mm, pl[s]);
    for (int d = 1; d < 64; d <<= 1) mm = kv_xor_max(mm, d);
    const float safe = mm == -__builtin_inff() ? 0.0f : mm;
    float o[PL], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PL; i++) o[i] = 0.0f;
    for (int s0 = part; s0 < t.nsplit; s0 += 8 * WAVES) {  // eight pieces of this wave on their way at a time
        float w[8], x[8][PL];
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const int s = s0 + WAVES * k < t.nsplit ? s0 + WAVES * k : t.nsplit - 1;
            w[k] = pl[s];
#pragma unroll
            for (int i = 0; i < PL; i++) x[k][i] = po[(int64_t)s * DIM + lane + 64 * i];
        }
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const float e = s0 + WAVES * k < t.nsplit ? kv_exp2(w[k] - safe) : 0.0f;
            sum += e;
#pragma unroll
            for (int i = 0; i < PL; i++) o[i] += e * x[k][i];
        }
    }
    if constexpr (WAVES > 1) {
#pragma unroll
        for (int i = 0; i < PL; i++) so[wave][lane + 64 * i] = o[i];
        if (lane == 0) ssum[wave] = sum;
        __syncthreads();  // the whole workgroup has this row
        if (wave != 0) return;
        sum = ssum[0] + ssum[1] + ssum[2] + ssum[3];
#pragma unroll
        for (int i = 0; i < PL; i++) o[i] = so[0][lane + 64 * i] + so[1][lane + 64 * i] + so[2][lane + 64 * i] + so[3][lane + 64 * i];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < PL; i++) {
        const int64_t c = at * DIM + lane + 64 * i;
        const float y = o[i] * inv;
        if constexpr (IN == 0)
            ((float *)a.out)[c] = y;
        else if constexpr (IN == 1)
            ((_Float16 *)a.out)[c] = (_Float16)y;
        else
            ((__bf16 *)a.out)[c] = (__bf16)y;
    }
    if (lane == 0 && a.lse) a.lse[at] = (sum == 0.0f ? -__builtin_inff() : safe + __builtin_amdgcn_logf(sum)) * KV_LN2;
}

}  // namespace nq
