// nq_kv_rows.h -- attention over the 8-bit key/value cache for many rows (prompts, chunks of prompts) of 16-bit queries.
//
// The formulas and the arithmetic are nq_kv_attn.h's.  With many rows the
// matrix instructions bound the work, so a key's codes are converted to
// binary16 once for 32 * NW rows: a workgroup of NW waves stages 64 keys at a
// time in LDS (two buffers, one barrier a tile; the codes of the next tile
// but one are on their way to registers), and each wave holds 32 rows: their
// queries and outputs stay in registers.  With lane = 32 h + r:
//   scores  A = keys [32][16 channels], B = the queries: the result gives lane
//           (r = query row, h) the keys 32 kt + 8 j + 4 h + i;
//   output  A = values [32 channels][16 keys], B = the weights, which are
//           where the scores were: the values of 16 keys are laid out in LDS as
//           0-3 8-11 4-7 12-15, so that a lane's eight are contiguous.
// Rows of the LDS tiles are padded by 16 bytes: 16 lanes' reads then fall into
// different banks.
#pragma once

#include "nq_kv_attn.h"

namespace nq {

typedef float kv_f16x __attribute__((ext_vector_type(16)));

template <int DIM, int NW>
struct KvRows {
    static constexpr int KT = 64, ROWS = 32 * NW, TB = 64 * NW;
    static constexpr int UNITS = KT * DIM / 16;             // 16-byte pieces of a tile's keys, and of its values
    static constexpr int NL = UNITS / TB;                   // a thread's
    static constexpr int KS = DIM + 8, VS = KT + 8;         // row strides in LDS, binary16 elements
    static constexpr int K_ELEMS = KT * KS, V_ELEMS = DIM * VS;
    static constexpr int BUF = K_ELEMS + V_ELEMS;           // elements of a buffer
    static constexpr int LDS_BYTES = 2 * BUF * 2 + 2 * 8 * 4;
    static_assert(NL >= 1 && NL * TB == UNITS, "every thread stages the same number of pieces");
};

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

// The larger of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float kv_max_halves(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
}

template <int CODE, int DIM, int IN, int NW>
__global__ __launch_bounds__(64 * NW, DIM > 128 ? 1 : 2) void k_kv_attn_rows(KvAttnArgs args) {
    using C = KvRows<DIM, NW>;
    constexpr int KT = C::KT, NL = C::NL, KS = C::KS, VS = C::VS, TB = C::TB;
    constexpr int NS = DIM / 16;  // channel steps of a score
    constexpr int ND = DIM / 32;  // output tiles
    extern __shared__ __align__(16) uint8_t lds_raw[];
    _Float16 *const buf = (_Float16 *)lds_raw;
    float *const sc = (float *)(lds_raw + 2 * C::BUF * 2);  // [2][8]: key scales, value scales of 16 keys
    const KvAttnLaunch &a = args.L;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 31, h = lane >> 5;
    const uint32_t head = blockIdx.x % a.c.heads;
    const int tile = a.tiles - 1 - (int)(blockIdx.x / a.c.heads);  // the longest rows first
    const int split = (int)blockIdx.y, req = (int)blockIdx.z, group = a.group;
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
    float qscale;
    {
        const int64_t at = (int64_t)(q.s0 + tok) * a.q_ts + ((int64_t)head * group + row % group) * a.q_hs + 8 * h;
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
        amax = kv_max_halves(amax);
        const float up = kv_row_scale(amax);
        qscale = a.scale * KV_LOG2E / up;
#pragma unroll
        for (int s = 0; s < NS; s++)
#pragma unroll
            for (int i = 0; i < 8; i++) Q[s][i] = (_Float16)(f[s][i] * up);
    }

    // Staging: a thread's pieces of a tile's keys (16 channels of a key) and values (16 keys of a channel).
    const KvTableRow table = {a.table + (int64_t)req * a.table_stride};
    const uint32_t bsh = a.c.bsh;
    kv_u4 rk[NL], rv[NL];
    int pk[NL], pv[NL];  // blocks of the pieces
    float rks = 0.0f, rvs = 0.0f;
    auto find = [&](int key0) {
#pragma unroll
        for (int n = 0; n < NL; n++) {
            const int u = tid + n * TB;
            pk[n] = kv_page(table, key0 + u / (DIM / 16), t, bsh, a.c.blocks);
            pv[n] = kv_page(table, key0 + 16 * (u & 3), t, bsh, a.c.blocks);
        }
    };
    auto fetch = [&](int key0) {
#pragma unroll
        for (int n = 0; n < NL; n++) {
            const int u = tid + n * TB;
            rk[n] = *(const kv_u4 *)(a.c.k + kv_k_at(a.c, pk[n], head, key0 + u / (DIM / 16)) + 16 * (u % (DIM / 16)));
            rv[n] = *(const kv_u4 *)(a.c.v + kv_v_at(a.c, pv[n], head, u >> 2, key0 + 16 * (u & 3)));
        }
        if (tid < 4) {
            const int64_t at = (int64_t)(pv[0] < 0 ? 0 : pv[0]) * a.c.heads + head;
            rks = a.c.ks[at];
            rvs = a.c.vs[at];
        }
    };
    // dead: the pieces' blocks when they were fetched
    auto stage = [&](int key0, int b, const int (&was)[NL]) {
        _Float16 *const K = buf + b * C::BUF, *const V = K + C::K_ELEMS;
#pragma unroll
        for (int n = 0; n < NL; n++) {
            const int u = tid + n * TB;
            _Float16 *const dk = K + (u / (DIM / 16)) * KS + 16 * (u % (DIM / 16));
            *(kv_h8 *)dk = kv_codes8_f16<CODE>(kv_u2{rk[n][0], rk[n][1]});
            *(kv_h8 *)(dk + 8) = kv_codes8_f16<CODE>(kv_u2{rk[n][2], rk[n][3]});
            kv_mask16(rv[n], key0 + 16 * (u & 3), t.kb, t.kend, was[n] < 0);
            _Float16 *const dv = V + (u >> 2) * VS + 16 * (u & 3);
            *(kv_h8 *)dv = kv_codes8_f16<CODE>(kv_u2{rv[n][0], rv[n][2]});
            *(kv_h8 *)(dv + 8) = kv_codes8_f16<CODE>(kv_u2{rv[n][1], rv[n][3]});
        }
        if (tid < 4) {
            // a block that is not there: its keys are masked, any scale will do
            sc[8 * b + tid] = was[0] < 0 ? 0.0f : rks;
            sc[8 * b + 4 + tid] = was[0] < 0 ? 0.0f : rvs;
        }
    };

    kv_f16x O[ND];
#pragma unroll
    for (int d = 0; d < ND; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) O[d][i] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f, vref = KV_TINY;

    int was[NL];
    if (k0 < k1) {
        find(k0);
        fetch(k0);
#pragma unroll
        for (int n = 0; n < NL; n++) was[n] = pv[n];
        find(k0 + KT);
        stage(k0, 0, was);
        if (k0 + KT < k1) fetch(k0 + KT);
#pragma unroll
        for (int n = 0; n < NL; n++) was[n] = pv[n];
        find(k0 + 2 * KT);
    }
    __syncthreads();
    int b = 0;
    for (int key0 = k0; key0 < k1; key0 += KT, b ^= 1) {
        const _Float16 *const K = buf + b * C::BUF, *const V = K + C::K_ELEMS;
        kv_f16x S[2];
#pragma unroll
        for (int kt = 0; kt < 2; kt++) {
#pragma unroll
            for (int i = 0; i < 16; i++) S[kt][i] = 0.0f;
#pragma unroll
            for (int s = 0; s < NS; s++) {
                const kv_h8 kk = *(const kv_h8 *)(K + (32 * kt + r) * KS + 16 * s + 8 * h);
                S[kt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kk, Q[s], S[kt], 0, 0, 0);
            }
        }
        float ks[4], vs[4];
#pragma unroll
        for (int g = 0; g < 4; g++) {
            ks[g] = sc[8 * b + g];
            vs[g] = sc[8 * b + 4 + g];
        }
        if (key0 + KT < k1) {
            stage(key0 + KT, b ^ 1, was);
            if (key0 + 2 * KT < k1) fetch(key0 + 2 * KT);
#pragma unroll
            for (int n = 0; n < NL; n++) was[n] = pv[n];
            find(key0 + 3 * KT);
        }
        // scores in base-2 logarithms
        float cf[4];
        bool odd = false;
#pragma unroll
        for (int g = 0; g < 4; g++) {
            cf[g] = qscale * ks[g];
            odd |= !(cf[g] > 0.0f);
        }
        if (__ballot(odd)) {  // negative, zero or NaN scales, blocks that are not there
#pragma unroll
            for (int g = 0; g < 4; g++) {
#pragma unroll
                for (int i = 0; i < 8; i++) S[g >> 1][8 * (g & 1) + i] *= cf[g];
                cf[g] = 1.0f;
            }
        }
        bool gone = false;
#pragma unroll
        for (int g = 0; g < 4; g++) gone |= ks[g] == 0.0f && vs[g] == 0.0f;
        if (key0 < all_lo || key0 + KT > all_hi || __ballot(gone)) {
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const bool dead = kv_page(table, key0 + 16 * g, t, bsh, a.c.blocks) < 0;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const int key = key0 + 16 * g + 8 * (i >> 2) + 4 * h + (i & 3);
                    if (dead || key < lo || key >= hi) S[g >> 1][8 * (g & 1) + i] = -__builtin_inff();
                }
            }
        }
        float top = -__builtin_inff(), vr1 = vref;
#pragma unroll
        for (int g = 0; g < 4; g++) {
            float x = S[g >> 1][8 * (g & 1)];
#pragma unroll
            for (int i = 1; i < 8; i++) x = fmaxf(x, S[g >> 1][8 * (g & 1) + i]);
            top = fmaxf(top, x * cf[g]);
            vr1 = fmaxf(vr1, fabsf(vs[g]));
        }
        top = kv_max_halves(top);
        const float m1 = fmaxf(m, top), safe = m1 == -__builtin_inff() ? 0.0f : m1;
        float fo = 1.0f;
        if (__ballot(m1 > m || vr1 > vref)) {
            const float alpha = kv_exp2(m - safe);
            l *= alpha;
            fo = alpha * (vref / vr1);
#pragma unroll
            for (int d = 0; d < ND; d++)
#pragma unroll
                for (int i = 0; i < 16; i++) O[d][i] *= fo;
            m = m1;
            vref = vr1;
        }
        float least = KV_PSCALE;
        const float unit = KV_PSCALE / vref;
#pragma unroll
        for (int g = 0; g < 4; g++) {
            const float w = vs[g] * unit;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float e = kv_exp2(__builtin_fmaf(S[g >> 1][8 * (g & 1) + i], cf[g], -safe));
                const float x = e * w;
                sum += e;
                S[g >> 1][8 * (g & 1) + i] = x;
                least = fminf(least, fabsf(x));
            }
            l += sum;
        }
        // O += values * weights.  Where some weights are small, those once more by themselves, multiplied by the
        // power of two that brings the row's largest of them to [2^13, 2^14).
        const bool slow = __ballot(least < KvLevel<1>::LEAST) != 0;
        float up = 1.0f;
        kv_h8 P[4], P2[4];
#pragma unroll
        for (int g = 0; g < 4; g++)
#pragma unroll
            for (int i = 0; i < 8; i++) P[g][i] = (_Float16)S[g >> 1][8 * (g & 1) + i];
        if (slow) {
            float most = 0.0f;
#pragma unroll
            for (int g = 0; g < 4; g++)
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float x = fabsf(S[g >> 1][8 * (g & 1) + i]);
                    most = fmaxf(most, x < KvLevel<1>::LEAST ? x : 0.0f);
                }
            // |O| <= 2^14 * 448 * 2 max(l): up stops where their product would pass 2^127
            const int e = (int)(__builtin_bit_cast(uint32_t, kv_max_halves(most)) >> 23) - 127;
            const int el = (int)(__builtin_bit_cast(uint32_t, kv_max_halves(l)) >> 23) - 127;
            const int room = el > 0 ? 100 - el : 100;
            up = bits_f32((uint32_t)(127 + (13 - e < room ? 13 - e : room)) << 23);
#pragma unroll
            for (int g = 0; g < 4; g++)
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float x = S[g >> 1][8 * (g & 1) + i];
                    const bool small = fabsf(x) < KvLevel<1>::LEAST;
                    P[g][i] = small ? (_Float16)0.0f : P[g][i];
                    P2[g][i] = (_Float16)(small ? x * up : 0.0f);
                }
        }
#pragma unroll
        for (int d = 0; d < ND; d++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const kv_h8 vv = *(const kv_h8 *)(V + (32 * d + r) * VS + 16 * g + 8 * h);
                O[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, P[g], O[d], 0, 0, 0);
            }
        if (slow) {
#pragma unroll
            for (int d = 0; d < ND; d++) {
#pragma unroll
                for (int i = 0; i < 16; i++) O[d][i] *= up;
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    const kv_h8 vv = *(const kv_h8 *)(V + (32 * d + r) * VS + 16 * g + 8 * h);
                    O[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, P2[g], O[d], 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 16; i++) O[d][i] *= 1.0f / up;
            }
        }
        __syncthreads();
    }

    l += __shfl_xor(l, 32, 64);
    if (row_at >= t.rows) return;
    const float inv = l == 0.0f ? 0.0f : vref * (1.0f / KV_PSCALE) / l;
    const float lse2 = l == 0.0f ? -__builtin_inff() : (m == -__builtin_inff() ? 0.0f : m) + __builtin_amdgcn_logf(l);
    const int64_t oat = (int64_t)(q.s0 + tok) * a.q_heads + (int64_t)head * group + row % group;
    const int64_t pat = oat * a.max_splits + split;
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
        if (L.waves == 4) {
            hipLaunchKernelGGL((k_kv_attn_rows<CODE, DIM, IN, 4>), grid, dim3(256), (KvRows<DIM, 4>::LDS_BYTES), s, a);
            if (hipGetLastError() != hipSuccess) return 9;  // NQ_ERR_HIP
        }
        if constexpr (DIM == 128) {
            if (L.waves == 8) {
                hipLaunchKernelGGL((k_kv_attn_rows<CODE, DIM, IN, 8>), grid, dim3(512), (KvRows<DIM, 8>::LDS_BYTES), s, a);
                if (hipGetLastError() != hipSuccess) return 9;  // NQ_ERR_HIP
            }
        }
    }
    const dim3 grid(L.c.heads * (uint32_t)L.tiles_few, (uint32_t)L.splits_few, (uint32_t)L.requests + 1);
    constexpr uint32_t lds = KvDec<CODE, DIM, IN, TERMS>::LDS_FLOATS * 4;
    hipLaunchKernelGGL((k_kv_attn_dec<CODE, DIM, IN, TERMS>), grid, dim3(256), lds, s, a);
    if (hipGetLastError() != hipSuccess) return 9;  // NQ_ERR_HIP
    if (L.max_splits > 1) {
        // new tokens of a request that can have several pieces
        const int32_t most = L.splits > 1 || L.few / L.group >= L.max_new ? L.max_new : L.few / L.group;
        const dim3 jgrid((uint32_t)(most < 1 ? 1 : most), (uint32_t)L.q_heads, (uint32_t)L.requests);
        hipLaunchKernelGGL((k_kv_attn_join<DIM, IN>), jgrid, dim3(256), 0, s, a);
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
