// nq_fp8b_codes.h -- device helpers of the E4M3 block operators.
#pragma once

#include "nq_fp8b.h"
#include "nq_kv_codes.h"

namespace nq {

// Eight consecutive elements of type IN as binary32; VEC: the address is a multiple of 16 bytes.
template <int IN, bool VEC>
__device__ __forceinline__ void fb_read8(const void *x, int64_t i, float (&f)[8]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] = kv_read<IN>(x, i + j);
    } else if constexpr (IN == 0) {
#pragma unroll
        for (int v = 0; v < 2; v++) {
            const kv_f4 w = *(const kv_f4 *)((const float *)x + i + 4 * v);
#pragma unroll
            for (int j = 0; j < 4; j++) f[4 * v + j] = w[j];
        }
    } else {
        const kv_u4 w = *(const kv_u4 *)((const uint16_t *)x + i);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const uint32_t h = (w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
            f[j] = IN == 1 ? f16(h) : bits_f32(h << 16);
        }
    }
}

// The largest magnitude of N values and m, as words: integers in the same order, infinities and NaN above all.
template <int N>
__device__ __forceinline__ uint32_t fb_amax(const float (&f)[N], uint32_t m) {
#pragma unroll
    for (int i = 0; i < N; i++) {
        const uint32_t x = __builtin_bit_cast(uint32_t, f[i]) & 0x7FFFFFFFu;
        m = x > m ? x : m;
    }
    return m;
}
template <int N>
__device__ __forceinline__ uint32_t fb_amax_finite(const float (&f)[N], uint32_t m) {
#pragma unroll
    for (int i = 0; i < N; i++) {
        const uint32_t x = __builtin_bit_cast(uint32_t, f[i]) & 0x7FFFFFFFu;
        m = x > m && x < 0x7F800000u ? x : m;
    }
    return m;
}
__device__ __forceinline__ uint32_t fb_amax8(const float (&f)[8], uint32_t m) { return fb_amax<8>(f, m); }
__device__ __forceinline__ uint32_t fb_amax8_finite(const float (&f)[8], uint32_t m) { return fb_amax_finite<8>(f, m); }

// Infinities become NaN, so that their codes are.
template <int N>
__device__ __forceinline__ void fb_mark_not_finite(float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; i++)
        if ((__builtin_bit_cast(uint32_t, f[i]) & 0x7FFFFFFFu) >= 0x7F800000u) f[i] = bits_f32(0x7FC00000u);
}

// The largest of four lanes' words, in each of them.
__device__ __forceinline__ uint32_t fb_max4(uint32_t m) {
    uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true);  // lane ^ 1
    m = o > m ? o : m;
    o = (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true);  // lane ^ 2
    return o > m ? o : m;
}

// The largest of sixteen lanes' words, in each of them.
__device__ __forceinline__ uint32_t fb_max16(uint32_t m) {
    m = fb_max4(m);
    const auto other = [&](uint32_t o) { m = o > m ? o : m; };
    other((uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, true));  // mirrored in eight
    other((uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xF, 0xF, true));  // mirrored in sixteen
    return m;
}

__device__ __forceinline__ uint32_t fb_codes4(float a, float b, float c, float d) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Eight codes of RN32(f * inv).
__device__ __forceinline__ kv_u2 fb_codes8(const float (&f)[8], float inv) {
    kv_u2 w = {fb_codes4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
               fb_codes4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv)};
    return w;
}

// Two dwords of codes as eight binary16 numbers (exact).
__device__ __forceinline__ kv_h8 fb_half8(uint32_t lo, uint32_t hi) {
    kv_u2 w = {lo, hi};
    return kv_codes8_f16<KV_E4M3>(w);
}

// The sum of the lanes' numbers up to each.
__device__ __forceinline__ int32_t fb_scan(int32_t v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // from 1, 2, 4 and 8 lanes before, in rows of sixteen
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // the end of a row to the next, of rows 0 and 2
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // the end of row 1 to rows 2 and 3
    return v;
}

// The row tile of a workgroup (fb_find_tile_host's rule), by a wave: a lane looks at one expert.
__device__ __forceinline__ Fp8Tile fb_find_tile(const int32_t *offsets, int32_t experts, int64_t rows, int32_t bm, int32_t t) {
    const int lane = threadIdx.x & 63;
    const int32_t most = (int32_t)rows;  // (at most 2^30)
    for (int32_t e0 = 0; e0 <= experts; e0 += 64) {
        const int32_t e = e0 + lane;
        int32_t lo = 0, hi = 0;
        if (e <= experts) {
            lo = (int32_t)fb_clamp(offsets[e], most);
            hi = e < experts ? (int32_t)fb_clamp(offsets[e + 1], most) : most;
        }
        const int32_t n = hi > lo ? (int32_t)((uint32_t)(hi - lo + bm - 1) / (uint32_t)bm) : 0, sum = fb_scan(n);
        const uint64_t past = __ballot(sum > t);
        if (past) {
            const int at = __builtin_ctzll(past);
            const int32_t from = __builtin_amdgcn_readlane(lo, at), end = __builtin_amdgcn_readlane(hi, at);
            const int64_t first = from + (int64_t)(t - (__builtin_amdgcn_readlane(sum, at) - __builtin_amdgcn_readlane(n, at))) * bm;
            if (first < from || first >= end) break;  // offsets that no sort gives: their sum may have left 32 bits
            return {e0 + at < experts ? e0 + at : -1, first, (int32_t)(end - first < bm ? end - first : bm)};
        }
        t -= __builtin_amdgcn_readlane(sum, 63);
    }
    return {-1, 0, 0};
}

// The row of x that output row p takes.
__device__ __forceinline__ int64_t fb_source_row(const Fp8GemmLaunch &a, int64_t p) {
    if (!a.order) return p;
    const int32_t o = a.order[p];
    const int64_t r = o < 0 ? 0 : o / a.top;
    return r < a.x_rows ? r : a.x_rows - 1;
}

// g / (1 + e^-g).  For 16-bit outputs the hardware's exponential and reciprocal, each within 1 ulp of binary32; the
// argument's rounding makes the exponential off by |g| * 2^-24 of itself at most, 2^-17 at the ends of binary32.
template <int OT>
__device__ __forceinline__ float fb_silu(float g) {
    if constexpr (OT == 0)
        return g / (1.0f + expf(-g));
    else
        return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f));
}

// One value of type ot.
__device__ __forceinline__ void fb_write1(void *y, int64_t i, float f, int32_t ot) {
    if (ot == 0)
        ((float *)y)[i] = f;
    else if (ot == 1)
        ((_Float16 *)y)[i] = (_Float16)f;
    else
        ((__bf16 *)y)[i] = (__bf16)f;
}

// Four consecutive values of type ot, the address a multiple of their bytes.
__device__ __forceinline__ void fb_write4(void *y, int64_t i, const float (&f)[4], int32_t ot) {
    if (ot == 0)
        kv_write4<0>(y, i, f);
    else if (ot == 1)
        kv_write4<1>(y, i, f);
    else
        kv_write4<2>(y, i, f);
}

}  // namespace nq
