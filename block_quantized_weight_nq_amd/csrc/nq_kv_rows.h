// nq_kv_rows.h -- attention over the 8-bit key/value cache for many rows (prompts, chunks of prompts) of 16-bit queries.
//
// The formulas and the arithmetic are nq_kv_attn.h's.  With many rows the
// matrix instructions and the softmax bound the work, so a key's codes are
// converted to binary16 once for 32 * NW rows: a workgroup of NW waves stages
// 64 keys at a time in LDS, and each wave holds 32 rows, whose queries and
// outputs stay in registers.  With lane = 32 h + r:
//   scores  A = keys [32][16 channels], B = the queries: the result gives lane
//           (r = query row, h) the keys 32 kt + 8 j + 4 h + i;
//   output  A = values [32 channels][16 keys], B = the weights, which are
//           where the scores were: the values of 16 keys are laid out in LDS as
//           0-3 8-11 4-7 12-15, so that a lane's eight are contiguous.
// Rows of the LDS tiles are padded by 16 bytes: 16 lanes' reads then fall into
// different banks.
//
// A wave alone issues a vector instruction every 8 cycles or so, and a SIMD
// has only two of these waves, so each wave mixes its own work: the scores of
// tile i + 1 are multiplied while the weights of tile i are formed, and the
// codes of the tiles after are converted while its output is multiplied.
// Keys are staged two tiles ahead and values one, in two buffers each; one
// barrier a tile.
#pragma once

#include "nq_kv_attn.h"

namespace nq {

typedef float kv_f16x __attribute__((ext_vector_type(16)));
typedef __bf16 kv_b8 __attribute__((ext_vector_type(8)));

// Weights are times 2^14: a row's maximum in use may lag behind by 2^KV_LAG
// before its output is multiplied down (binary16 holds up to 2^16).
constexpr float KV_LAG = 1.5f;
// vref is at least KV_VREF_MIN.  The sum l is in units of 2^14 / vref and, where every value is 0 (block scales of
// 2^-126), stays in those of KV_VREF_MIN: 2^30 keys whose weights lag by KV_LAG make it 2^125.5.
constexpr float KV_VREF_MIN = 0x1p-80f, KV_LUNIT_MAX = 94.0f;  // and log2(2^14 / KV_VREF_MIN)

// Codes of keys outside [lo, hi), or of no block, become 0: what lies there may be E4M3's NaN.
__device__ __forceinline__ void kv_mask16(kv_u4 &w, int key, int lo, int hi, bool dead) {
    if (!dead && key >= lo && key + 16 <= hi) return;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        uint32_t keep = 0;
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (!dead && key + 4 * j + i >= lo && key + 4 * j + i < hi) keep |= 0xFFu << (8 * i);
        w[j] &= keep;
    }
}

// The upper halves of two binary32 values: bfloat16, cut off.
__device__ __forceinline__ uint32_t kv_two_high(float a, float b) {
    return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u);
}

// The larger of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float kv_max_halves(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
}

// A lane's half of its query row (the 16-channel steps' channels 8 h..+7, at element `at` of q) as binary16 with the
// row's power of two; returns what a product with a key's codes is multiplied by, times the scale and log2(e).
template <int IN, int NS>
__device__ __forceinline__ float kv_load_rows(const KvAttnLaunch &a, int64_t at, kv_h8 (&Q)[NS]) {
    float amax = 0.0f;
    float f[NS][8];
#pragma unroll
    for (int s = 0; s < NS; s++) {
        if (a.q_vec) {
            kv_read4<IN, true>(a.q, at + 16 * s, *(float(*)[4])&f[s][0]);
            kv_read4<IN, true>(a.q, at + 16 * s + 4, *(float(*)[4])&f[s][4]);
        } else {
            kv_read4<IN, false>(a.q, at + 16 * s, *(float(*)[4])&f[s][0]);
            kv_read4<IN, false>(a.q, at + 16 * s + 4, *(float(*)[4])&f[s][4]);
        }
#pragma unroll
        for (int i = 0; i < 8; i++) amax = fmaxf(amax, fabsf(f[s][i]));
    }
    const float up = kv_row_scale(kv_max_halves(amax));
#pragma unroll
    for (int s = 0; s < NS; s++)
#pragma unroll
        for (int i = 0; i < 8; i++) Q[s][i] = (_Float16)(f[s][i] * up);
    return a.scale * KV_LOG2E / up;
}

// The scales of 16 keys for the weights (their place in the kernels' sc).
__device__ __forceinline__ void kv_put_scales(float *s, float ks, float vs, bool dead) {
    const bool odd = !(ks > 0.0f && vs > 0.0f && vs < __builtin_inff());
    s[0] = dead ? 1.0f : ks;  // a block that is not there: its keys are masked, any scale will do
    s[4] = dead ? KV_VREF_MIN : vs;
    s[8] = __builtin_amdgcn_logf(dead ? KV_VREF_MIN : vs);
    s[12] = __builtin_amdgcn_rcpf(dead ? KV_VREF_MIN : vs);  // 1 ulp
    ((int *)s)[16] = dead ? 3 : odd ? 2 : 0;
}

// The request with the z-th largest length (of equal ones the first): the
// longest requests' workgroups start first, so that none of them is left at
// the end (24 requests, a third of them with chunks: 213 us without, 202 with).
// TB threads of one workgroup, KV_RANKED requests at most; more keep their
// order.  The few-rows kernel keeps it too: its workgroups are short, and their
// ranking took longer than it saved (128 requests: 82 us without, 120 with).
constexpr int KV_RANKED = 256;
template <int TB>
__device__ __forceinline__ int kv_ranked(const KvAttnLaunch &a, int z) {
    __shared__ int len[KV_RANKED], rank[KV_RANKED], found;
    const int R = a.requests, tid = threadIdx.x;
    if (R > KV_RANKED || R == 1) return z;
    for (int i = tid; i < R; i += TB) {
        len[i] = a.lengths[i];
        rank[i] = 0;
    }
    __syncthreads();
    // pairs (i, j): TB / R threads share a request's comparisons
    const int per = TB / R > 0 ? TB / R : 1, i = tid / per, part = tid % per;
    if (i < R) {
        const int mine = len[i];
        int above = 0;
        for (int j = part; j < R; j += per) above += len[j] > mine || (len[j] == mine && j < i);
        if (per == 1)
            rank[i] = above;
        else if (above)
            atomicAdd(&rank[i], above);
    }
    __syncthreads();
    for (int k = tid; k < R; k += TB)
        if (rank[k] == z) found = k;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(found);
}

template <int CODE, int DIM, int IN, int NW>
__global__ __launch_bounds__(64 * NW, DIM > 128 ? 1 : 2) void k_kv_attn_rows(KvAttnArgs args) {
    using C = KvRows<DIM, NW>;
    constexpr int KT = C::KT, NL = C::NL, KS = C::KS, VS = C::VS, SC = C::SC;
    constexpr int NS = DIM / 16;  // channel steps of a score
    constexpr int ND = DIM / 32;  // output tiles
    extern __shared__ __align__(16) uint8_t lds_raw[];
    _Float16 *const kbuf = (_Float16 *)lds_raw, *const vbuf = kbuf + 2 * C::K_ELEMS;
    // of 16 keys each: [0-3] key scales, [4-7] value scales, [8-11] their base-2 logarithms, [12-15] their
    // inverses, [16-19] flags: 1 no block, 2 a scale that is not positive
    float *const sc = (float *)(vbuf + 2 * C::V_ELEMS);
    const KvAttnLaunch &a = args.L;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t head = blockIdx.x % a.c.heads;
    const int tile = a.tiles - 1 - (int)(blockIdx.x / a.c.heads);  // the longest rows first
    const int split = (int)blockIdx.y, req = kv_ranked<64 * NW>(a, (int)blockIdx.z), group = a.group;
    const KvReq q = kv_request(a, req);
    const int rows = (q.s1 - q.s0) * group;
    if (rows <= a.few || tile * C::ROWS >= rows) return;
    const KvTile t = kv_tile(q.s1 - q.s0, q.len, a.cap, group, tile, C::ROWS, a.window, a.chunk);
    if (split >= t.nsplit) return;
    const int k0 = t.kbeg + split * a.chunk;
    const int k1 = t.kend - k0 > a.chunk ? k0 + a.chunk : t.kend;

    // this lane's query row; the last row stands in for those past it
    const int row_at = tile * C::ROWS + wave * 32 + r;
    const int row = row_at < t.rows ? row_at : t.rows - 1, tok = row / group;
    const int p = t.base + tok;
    const int hi = p + 1 < t.live ? p + 1 : t.live;
    const int lo = a.window > 0 && p - a.window + 1 > 0 ? p - a.window + 1 : 0;
    // of the wave's rows: the fewest keys' end and the last beginning
    const int w0 = (tile * C::ROWS + wave * 32 < t.rows ? tile * C::ROWS + wave * 32 : t.rows - 1) / group;
    const int w1 = (tile * C::ROWS + wave * 32 + 31 < t.rows ? tile * C::ROWS + wave * 32 + 31 : t.rows - 1) / group;
    const int all_hi = t.base + w0 + 1 < t.live ? t.base + w0 + 1 : t.live;
    const int all_lo = a.window > 0 ? t.base + w1 - a.window + 1 : 0;

    kv_h8 Q[NS];
    const float qscale = kv_load_rows<IN, NS>(a, (int64_t)(q.s0 + tok) * a.q_ts + ((int64_t)head * group + row % group) * a.q_hs + 8 * h, Q);

    // Staging.  What lies past the last tile is fetched and staged as if it were there (from block 0): nothing reads it.
    const int sub = wave / C::PER, part = wave % C::PER;
    const int32_t *const table = a.table + (int64_t)req * a.table_stride;
    const uint32_t bsh = a.c.bsh, tile_bytes = (uint32_t)DIM << bsh;
    const uint8_t *const kbase = a.c.k + (uint64_t)head * tile_bytes + C::k_from(part, lane, 0);
    const uint8_t *const vbase = a.c.v + (uint64_t)head * tile_bytes + C::v_from(part, lane, 0, bsh);
    _Float16 *const kput = kbuf + C::k_put(sub, part, lane, 0);
    _Float16 *const vput = vbuf + C::v_put(sub, part, lane, 0);
    kv_u4 rk[NL], rv[NL];
    int entry = 0, page = -1, was = -1;  // the table entry on its way, the block of the keys and of the values fetched last
    float rks = 0.0f, rvs = 0.0f;
    // Vector loads, though the address is the wave's: scalar ones share the LDS reads' counter and complete out of
    // order, so that every wait for an LDS read would wait for memory.
    int none = 0;
    asm volatile("" : "+v"(none));
    auto find = [&](int key0) { entry = table[kv_entry(key0 + 16 * sub, t, bsh) + none]; };
    auto fetch_k = [&](int key0) {
        page = kv_named(__builtin_amdgcn_readfirstlane(entry), key0 + 16 * sub, t, bsh, a.c.blocks);
        const uint8_t *const src = kbase + C::block_at(a.c, page) + C::k_at(key0 + 16 * sub, bsh);
#pragma unroll
        for (int n = 0; n < NL; n++) rk[n] = *(const kv_u4 *)(src + C::k_from(0, 0, n));
    };
    auto fetch_v = [&](int key0, int block) {
        was = block;
        const uint8_t *const src = vbase + C::block_at(a.c, block) + C::v_at(key0 + 16 * sub, bsh);
#pragma unroll
        for (int n = 0; n < NL; n++) rv[n] = *(const kv_u4 *)(src + C::v_from(0, 0, n, bsh));
        if (part == 0) {
            const uint64_t s = (uint64_t)(block < 0 ? 0 : (uint32_t)block) * a.c.heads + head + none;
            rks = a.c.ks[s];
            rvs = a.c.vs[s];
        }
    };
    auto clean_v = [&](int key0) {  // signed bytes are finite whatever they are, and their weights 0
        if constexpr (CODE == KV_E4M3)
#pragma unroll
            for (int n = 0; n < NL; n++) kv_mask16(rv[n], key0 + 16 * sub, t.kb, t.kend, was < 0);
    };
    auto stage_k = [&](int b) {
#pragma unroll
        for (int n = 0; n < NL; n++) {
            _Float16 *const d = kput + b * C::K_ELEMS + C::k_put(0, 0, 0, n);
            *(kv_h8 *)d = kv_codes8_f16<CODE>(kv_u2{rk[n][0], rk[n][1]});
            *(kv_h8 *)(d + 8) = kv_codes8_f16<CODE>(kv_u2{rk[n][2], rk[n][3]});
        }
    };
    auto stage_v = [&](int b) {
#pragma unroll
        for (int n = 0; n < NL; n++) {
            _Float16 *const d = vput + b * C::V_ELEMS + C::v_put(0, 0, 0, n);
            *(kv_h8 *)d = kv_codes8_f16<CODE>(kv_u2{rv[n][0], rv[n][2]});
            *(kv_h8 *)(d + 8) = kv_codes8_f16<CODE>(kv_u2{rv[n][1], rv[n][3]});
        }
    };
    auto stage_scales = [&](int b) {
        if (part == 0 && lane == 0) kv_put_scales(sc + SC * b + sub, rks, rvs, was < 0);
    };

    // O and l are in units of 2^14 / vref: O sums x codes and l sums x / vs, x = 2^(score - m) vs 2^14 / vref.
    kv_f16x O[ND];
#pragma unroll
    for (int d = 0; d < ND; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) O[d][i] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;
    float vref = KV_VREF_MIN, unit = KV_PSCALE / KV_VREF_MIN, lunit = KV_LUNIT_MAX;  // and log2(unit)

    auto scores = [&](int b, kv_f16x (&S)[2]) {
        const _Float16 *const K = kbuf + b * C::K_ELEMS + r * KS + 8 * h;
#pragma unroll
        for (int kt = 0; kt < 2; kt++)
#pragma unroll
            for (int i = 0; i < 16; i++) S[kt][i] = 0.0f;
        // two sums in turn: a matrix instruction does not wait for the one before it
#pragma unroll
        for (int s = 0; s < NS; s++)
#pragma unroll
            for (int kt = 0; kt < 2; kt++)
                S[kt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(*(const kv_h8 *)(K + 32 * kt * KS + 16 * s), Q[s], S[kt], 0, 0, 0);
    };

    // Tile i (keys from key0 on): its scores are in S; next gets those of tile i + 1.  b = i mod 2.
    auto step = [&](int key0, int b, kv_f16x (&S)[2], kv_f16x (&next)[2]) {
        const float *const s4 = sc + SC * b;
        const kv_f4 ks = *(const kv_f4 *)s4, vs = *(const kv_f4 *)(s4 + 4), lv = *(const kv_f4 *)(s4 + 8);
        const kv_f4 iv = *(const kv_f4 *)(s4 + 12);
        const kv_u4 fl = *(const kv_u4 *)(s4 + 16);
        const int flags = __builtin_amdgcn_readfirstlane((int)(fl[0] | fl[1] | fl[2] | fl[3]));
        const float most = fmaxf(fmaxf(fabsf(vs[0]), fabsf(vs[1])), fmaxf(fabsf(vs[2]), fabsf(vs[3])));
        const float fewest = fminf(fminf(vs[0], vs[1]), fminf(vs[2], vs[3]));
        const float vr1 = fmaxf(vref, most);
        // scores in base-2 logarithms are S * cf.  Scales that are not positive, and value scales far below vref
        // (whose weights would leave binary32's range where l divides by the scale), take the plain order.
        const bool odd = (flags & 2) || !(a.scale > 0.0f) || __ballot(fewest * 0x1p20f < vr1);
        // Otherwise the factor multiplies masked scores of -inf too and has to be positive: one that is too small for
        // binary32 (keys of zero and a small query row) is taken as 2^-126: S is below 2^32, so no score is off by 2^-94.
        // One that is too large must not turn a score of 0 into NaN (kv_finite).
        float cf[4];
#pragma unroll
        for (int g = 0; g < 4; g++) cf[g] = qscale * ks[g];
        if (odd) {
#pragma unroll
            for (int g = 0; g < 4; g++) {
                cf[g] = kv_finite(cf[g]);
#pragma unroll
                for (int i = 0; i < 8; i++) S[g >> 1][8 * (g & 1) + i] *= cf[g];
                cf[g] = 1.0f;
            }
        } else {
#pragma unroll
            for (int g = 0; g < 4; g++) cf[g] = __builtin_amdgcn_fmed3f(cf[g], KV_TINY, KV_MOST);
        }
        if (key0 < all_lo || key0 + KT > all_hi || (flags & 1)) {
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const bool dead = fl[g] & 1;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const int key = key0 + 16 * g + 8 * (i >> 2) + 4 * h + (i & 3);
                    if (dead || key < lo || key >= hi) S[g >> 1][8 * (g & 1) + i] = -__builtin_inff();
                }
            }
        }
        float top = -__builtin_inff(), low[4];
#pragma unroll
        for (int g = 0; g < 4; g++) {
            float high = S[g >> 1][8 * (g & 1)];
            low[g] = high;
#pragma unroll
            for (int i = 1; i < 8; i++) {
                high = fmaxf(high, S[g >> 1][8 * (g & 1) + i]);
                low[g] = fminf(low[g], S[g >> 1][8 * (g & 1) + i]);
            }
            top = fmaxf(top, high * cf[g]);
        }
        top = kv_max_halves(top);
        // the maximum in use may be lower than the true one by KV_LAG
        if (__ballot(top > m + KV_LAG || vr1 > vref)) {
            const float m1 = fmaxf(m, top);
            const float fo = kv_exp2(m - (m1 == -__builtin_inff() ? 0.0f : m1)) * (vref / vr1);
            l *= fo;
#pragma unroll
            for (int d = 0; d < ND; d++)
#pragma unroll
                for (int i = 0; i < 16; i++) O[d][i] *= fo;
            m = m1;
            vref = vr1;
            unit = KV_PSCALE / vref;
            lunit = __builtin_amdgcn_logf(unit);
        }
        const float safe = m == -__builtin_inff() ? 0.0f : m;
        clean_v(key0 + KT);
        const _Float16 *const V = vbuf + b * C::V_ELEMS + r * VS + 8 * h;
        kv_h8 P[4];
        float at[4], least = 0.0f;  // and the logarithm of the smallest weight
#pragma unroll
        for (int g = 0; g < 4; g++) {
            at[g] = lv[g] + lunit - safe;
            least = fminf(least, __builtin_fmaf(low[g], cf[g], at[g]));
        }
        if (!odd && !__ballot(!(least >= -14.0f))) {
            scores(b ^ 1, next);
#pragma unroll
            for (int g = 0; g < 4; g++) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float x = kv_exp2(__builtin_fmaf(S[g >> 1][8 * (g & 1) + i], cf[g], at[g]));
                    sum += x;
                    P[g][i] = (_Float16)x;
                }
                l = __builtin_fmaf(sum, iv[g], l);
            }
        } else {
            asm volatile("" ::: "memory");
            // Any scales; small weights by themselves as two bfloat16 terms, cut off to 15 bits or more, fewer only
            // where a term falls below 2^-126, times the codes, which are exact in bfloat16 too.  A tile with such
            // weights costs about twice another; as binary16 times a power of two a row and 16 keys, in sums of their
            // own, they cost 8% more: 4096 of 8192 tokens 865 against 936 us where every tile has some, 629 against
            // 672 with scores of one to three nats' deviation by block, 455 against 458 without any.
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const float w = vs[g] * unit;
                float x[8], sum = 0.0f, big = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float e = kv_exp2(__builtin_fmaf(S[g >> 1][8 * (g & 1) + i], cf[g], -safe));
                    x[i] = e * w;
                    sum += e;
                    P[g][i] = (_Float16)x[i];
                    big = fmaxf(big, fabsf(x[i]) < KV_LEAST ? fabsf(x[i]) : 0.0f);
                }
                l = __builtin_fmaf(sum, unit, l);
                if (__ballot(big > 0.0f)) {
                    uint32_t hi[4], mid[4];
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const bool is = fabsf(x[i]) < KV_LEAST;
                        P[g][i] = is ? (_Float16)0.0f : P[g][i];
                        x[i] = is ? x[i] : 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        hi[i] = kv_two_high(x[2 * i], x[2 * i + 1]);
                        mid[i] = kv_two_high(x[2 * i] - bits_f32(hi[i] << 16), x[2 * i + 1] - bits_f32(hi[i] & 0xFFFF0000u));
                    }
                    const kv_b8 W0 = __builtin_bit_cast(kv_b8, (kv_u4){hi[0], hi[1], hi[2], hi[3]});
                    const kv_b8 W1 = __builtin_bit_cast(kv_b8, (kv_u4){mid[0], mid[1], mid[2], mid[3]});
#pragma unroll
                    for (int d = 0; d < ND; d++) {
                        const kv_h8 c = *(const kv_h8 *)(V + 32 * d * VS + 16 * g);
                        kv_u4 v;
#pragma unroll
                        for (int i = 0; i < 4; i++) v[i] = kv_two_high((float)c[2 * i], (float)c[2 * i + 1]);
                        O[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(kv_b8, v), W0, O[d], 0, 0, 0);
                        O[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(kv_b8, v), W1, O[d], 0, 0, 0);
                    }
                }
                asm volatile("" ::: "memory");  // the values are read again, not held meanwhile
            }
            scores(b ^ 1, next);
        }
#pragma unroll
        for (int g = 0; g < 4; g++)
#pragma unroll
            for (int d = 0; d < ND; d++)
                O[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(*(const kv_h8 *)(V + 32 * d * VS + 16 * g), P[g], O[d], 0, 0, 0);
        stage_k(b);
        stage_v(b ^ 1);
        stage_scales(b ^ 1);
        const int block = page;  // of the keys of tile i + 2
        fetch_k(key0 + 3 * KT);
        fetch_v(key0 + 2 * KT, block);
        find(key0 + 4 * KT);
        __syncthreads();
    };

    const int nt = (k1 - k0 + KT - 1) / KT;
    if (nt > 0) {
        // keys of tiles 0 and 1 and values of tile 0 into LDS; those of tiles 2 and 1 on their way
        find(k0);
        fetch_k(k0);
        find(k0 + KT);
        fetch_v(k0, page);
        stage_k(0);
        clean_v(k0);
        stage_v(0);
        stage_scales(0);
        fetch_k(k0 + KT);
        find(k0 + 2 * KT);
        fetch_v(k0 + KT, page);
        stage_k(1);
        fetch_k(k0 + 2 * KT);
        find(k0 + 3 * KT);
        __syncthreads();
        kv_f16x S0[2], S1[2];
        scores(0, S0);
        __syncthreads();  // tile 0 is read before tile 2 is staged in its place
        for (int i = 0; i < nt; i += 2) {
            step(k0 + i * KT, 0, S0, S1);
            if (i + 1 < nt) step(k0 + (i + 1) * KT, 1, S1, S0);
        }
    }

    l += __shfl_xor(l, 32, 64);
    if (row_at >= t.rows) return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const float lse2 = l == 0.0f ? -__builtin_inff() : (m == -__builtin_inff() ? 0.0f : m) + __builtin_amdgcn_logf(l / unit);
    const int64_t oat = (int64_t)(q.s0 + tok) * a.q_heads + (int64_t)head * group + row % group;
    const int64_t pat = oat * a.splits + split;
#pragma unroll
    for (int d = 0; d < ND; d++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float f[4] = {O[d][4 * j] * inv, O[d][4 * j + 1] * inv, O[d][4 * j + 2] * inv, O[d][4 * j + 3] * inv};
            const int c = 32 * d + 8 * j + 4 * h;
            if (t.nsplit == 1)
                kv_write4<IN>(a.out, oat * DIM + c, f);
            else
                *(kv_f4 *)(a.part + pat * DIM + c) = kv_f4{f[0], f[1], f[2], f[3]};
        }
    if (h == 0) {
        if (t.nsplit > 1)
            a.part_lse[pat] = lse2;
        else if (a.lse)
            a.lse[oat] = lse2 * KV_LN2;
    }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
template <int CODE, int DIM, int IN>
int launch_kv_attn_dim(const KvAttnLaunch &L, hipStream_t s) {
    constexpr int TERMS = IN == 0 ? 2 : 1;
    KvAttnArgs a{L};
    if constexpr (TERMS == 1) {
        const dim3 grid(L.c.heads * (uint32_t)L.tiles, (uint32_t)L.splits, (uint32_t)L.requests);
        if (L.waves > 0) {
            constexpr int NW = DIM == 128 ? 8 : 4;
            hipLaunchKernelGGL((k_kv_attn_rows<CODE, DIM, IN, NW>), grid, dim3(64 * NW), (KvRows<DIM, NW>::LDS_BYTES), s, a);
            if (hipGetLastError() != hipSuccess) return 9;  // NQ_ERR_HIP
        }
    }
    const dim3 grid(L.c.heads * (uint32_t)L.tiles_few, (uint32_t)L.splits_few, (uint32_t)L.requests + 1);
    constexpr uint32_t lds = KvDec<CODE, DIM, IN, TERMS>::LDS_FLOATS * 4;
    hipLaunchKernelGGL((k_kv_attn_dec<CODE, DIM, IN, TERMS>), grid, dim3(256), lds, s, a);
    if (hipGetLastError() != hipSuccess) return 9;  // NQ_ERR_HIP
    const int32_t most_splits = L.splits > L.splits_few ? L.splits : L.splits_few;
    if (most_splits > 1) {
        // new tokens of a request that can have several pieces
        const int32_t most = L.splits > 1 || L.few / L.group >= L.max_new ? L.max_new : L.few / L.group;
        const uint32_t tokens = (uint32_t)(most < 1 ? 1 : most), heads = (uint32_t)L.q_heads, reqs = (uint32_t)L.requests;
        if (most_splits <= 16)
            hipLaunchKernelGGL((k_kv_attn_join<DIM, IN, 1>), dim3(tokens, (heads + 3) / 4, reqs), dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_kv_attn_join<DIM, IN, 4>), dim3(tokens, heads, reqs), dim3(256), 0, s, a);
        if (hipGetLastError() != hipSuccess) return 9;  // NQ_ERR_HIP
    }
    return 0;
}

template <int CODE>
int launch_kv_attn_code(const KvAttnLaunch &L, hipStream_t s) {
    switch ((L.c.dim == 64 ? 0 : L.c.dim == 128 ? 3 : 6) + L.dtype) {
    case 0: return launch_kv_attn_dim<CODE, 64, 0>(L, s);
    case 1: return launch_kv_attn_dim<CODE, 64, 1>(L, s);
    case 2: return launch_kv_attn_dim<CODE, 64, 2>(L, s);
    case 3: return launch_kv_attn_dim<CODE, 128, 0>(L, s);
    case 4: return launch_kv_attn_dim<CODE, 128, 1>(L, s);
    case 5: return launch_kv_attn_dim<CODE, 128, 2>(L, s);
    case 6: return launch_kv_attn_dim<CODE, 256, 0>(L, s);
    case 7: return launch_kv_attn_dim<CODE, 256, 1>(L, s);
    default: return launch_kv_attn_dim<CODE, 256, 2>(L, s);
    }
}

}  // namespace nq
