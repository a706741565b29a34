// nq_fp8b_codes.h -- device helpers of the E4M3 block operators.
#pragma once

#include "nq_fp8b.h"
#include "nq_kv_codes.h"

namespace nq {

// Eight consecutive elements of type IN as binary32, the address a multiple of 16 bytes.
template <int IN>
__device__ __forceinline__ void fb_read8(const void *x, int64_t i, float (&f)[8]) {
    if constexpr (IN == 0) {
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

// Eight consecutive elements as they are.
template <int IN>
struct FbRaw {
    uint32_t w[IN == 0 ? 8 : 4];
};

template <int IN, bool VEC>
__device__ __forceinline__ FbRaw<IN> fb_raw8(const void *x, int64_t i) {
    FbRaw<IN> r;
    if constexpr (VEC) {
#pragma unroll
        for (int v = 0; v < (IN == 0 ? 2 : 1); v++) {
            const kv_u4 w = ((const kv_u4 *)((const uint8_t *)x + i * (IN == 0 ? 4 : 2)))[v];
#pragma unroll
            for (int j = 0; j < 4; j++) r.w[4 * v + j] = w[j];
        }
    } else if constexpr (IN == 0) {
#pragma unroll
        for (int j = 0; j < 8; j++) r.w[j] = ((const uint32_t *)x)[i + j];
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) r.w[j] = ((const uint16_t *)x)[i + 2 * j] | (uint32_t)((const uint16_t *)x)[i + 2 * j + 1] << 16;
    }
    return r;
}

template <int IN>
__device__ __forceinline__ float fb_value(const FbRaw<IN> &r, int j) {
    if constexpr (IN == 0) return __builtin_bit_cast(float, r.w[j]);
    const uint32_t w = r.w[j >> 1];
    if constexpr (IN == 1) return f16(j & 1 ? w >> 16 : w & 0xFFFFu);
    return bits_f32(j & 1 ? w & 0xFFFF0000u : w << 16);
}

// The largest magnitude of eight elements and m, in the type's own words (two 16-bit ones side by side): integers in the
// same order, infinities and NaN above all.
template <int IN>
__device__ __forceinline__ uint32_t fb_amax8(const FbRaw<IN> &r, uint32_t m) {
    if constexpr (IN == 0) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t x = r.w[i] & 0x7FFFFFFFu;
            m = x > m ? x : m;
        }
        return m;
    } else {
        typedef uint16_t u2 __attribute__((ext_vector_type(2)));
        u2 t = __builtin_bit_cast(u2, m);
#pragma unroll
        for (int i = 0; i < 4; i++) t = __builtin_elementwise_max(t, __builtin_bit_cast(u2, r.w[i] & 0x7FFF7FFFu));
        return __builtin_bit_cast(uint32_t, t);
    }
}
// ... as a binary32 word, what is not finite above all that is.
template <int IN>
__device__ __forceinline__ uint32_t fb_amax_word(uint32_t m) {
    if constexpr (IN == 0) return m;
    const uint32_t h = (m >> 16) > (m & 0xFFFFu) ? m >> 16 : m & 0xFFFFu;
    if constexpr (IN == 2) return h << 16;
    return h >= 0x7C00u ? 0x7F800000u : __builtin_bit_cast(uint32_t, f16(h));
}
// The largest finite magnitude of eight elements and m, as a binary32 word.
template <int IN>
__device__ __forceinline__ uint32_t fb_amax8_finite(const FbRaw<IN> &r, uint32_t m) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t x = __builtin_bit_cast(uint32_t, fb_value<IN>(r, i)) & 0x7FFFFFFFu;
        m = x > m && x < 0x7F800000u ? x : m;
    }
    return m;
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

// Eight codes of RN32(x * inv); BAD: some may not be finite, and become NaN.
template <int IN, bool BAD>
__device__ __forceinline__ kv_u2 fb_codes8(const FbRaw<IN> &r, float inv) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float v = fb_value<IN>(r, i);
        f[i] = v * inv;
        if (BAD && !(v - v == 0.0f)) f[i] = bits_f32(0x7FC00000u);
    }
    kv_u2 w = {fb_codes4(f[0], f[1], f[2], f[3]), fb_codes4(f[4], f[5], f[6], f[7])};
    return w;
}

// The scale of a block whose largest magnitude is the binary32 word `top`.
__device__ __forceinline__ float fb_scale(uint32_t top) { return fmaxf(__builtin_bit_cast(float, top) / 448.0f, FB_TINY); }

// Two dwords of codes as eight binary16 numbers (exact).
__device__ __forceinline__ kv_h8 fb_half8(uint32_t lo, uint32_t hi) {
    kv_u2 w = {lo, hi};
    return kv_codes8_f16<KV_E4M3>(w);
}

// The sum of the lanes' numbers up to each.
__device__ __forceinline__ int32_t fb_scan(int32_t v) {
    uint32_t s = (uint32_t)v;  // (sums wrap)
    s += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, 0x111, 0xF, 0xF, false);  // from 1, 2, 4 and 8 lanes before, in rows of sixteen
    s += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, 0x112, 0xF, 0xF, false);
    s += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, 0x114, 0xF, 0xF, false);
    s += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, 0x118, 0xF, 0xF, false);
    s += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, 0x142, 0xA, 0xF, false);  // the end of a row to the next, of rows 0 and 2
    s += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)s, 0x143, 0xC, 0xF, false);  // the end of row 1 to rows 2 and 3
    return (int32_t)s;
}

// The row tile of a workgroup.
struct FbWave {
    template <typename F>
    static __device__ __forceinline__ int32_t each(F f) {
        return f((int)(threadIdx.x & 63));
    }
    static __device__ __forceinline__ int32_t own(int32_t v, int) { return v; }
    static __device__ __forceinline__ int32_t scan(int32_t v) { return fb_scan(v); }
    static __device__ __forceinline__ uint64_t above(int32_t v, int32_t t) { return __ballot(v > t); }
    static __device__ __forceinline__ int32_t lane(int32_t v, int i) { return __builtin_amdgcn_readlane(v, i); }
};
__device__ __forceinline__ Fp8Tile fb_find_tile(const int32_t *offsets, int32_t experts, int64_t rows, int32_t bm, int32_t t) {
    return fb_find_tile_by<FbWave>([=](int32_t i) { return (int64_t)offsets[i]; }, experts, rows, bm, t);
}

// The row of x that output row p takes.
__device__ __forceinline__ int64_t fb_source_row(const Fp8GemmLaunch &a, int64_t p) {
    if (!a.order) return p;
    const int32_t o = a.order[p];
    const int64_t r = o < 0 ? 0 : o / a.top;
    return r < a.x_rows ? r : a.x_rows - 1;
}

// acc + d * sx * sw for a block's sum d, s = sx * sw.  Where s leaves binary32 the value need not: a sum of zero stays
// zero, one of 2^-18 (the least product of two codes) is finite up to 2^146.  |sw| is above 1 then, so d * sx leaves
// binary32 only where the value does.
__device__ __forceinline__ float fb_scaled(float d, float sx, float sw, float s, float acc) {
    return fabsf(s) <= FB_MOST ? __builtin_fmaf(d, s, acc) : acc + d * sx * sw;
}

// g / (1 + e^-g) * u.  For 16-bit outputs the hardware's exponential and reciprocal, each within 1 ulp of binary32; the
// roundings of the argument make the exponential off by |g| * 2^-23 of itself at most.
// Below -80 (FAR: gates may be) the quotient is g * e^g (to e^-80 of itself).  e^-g leaves binary32 there (from -88.8 on),
// and the hardware's reciprocal gives no subnormal numbers (from -87.4 on), while the value with u need not be small: the
// fourth root of e^g is in range as far as u can make up for it.  u comes after the first factor, so that only the value
// itself underflows.
constexpr float FB_FAR_GATE = -80.0f;
template <int OT, bool FAR = true>
__device__ __forceinline__ float fb_gate(float g, float u) {
    if (FAR && g < FB_FAR_GATE) {
        const float h = OT == 0 ? expf(0.25f * g) : __builtin_amdgcn_exp2f(g * 0.36067376f);
        return g * h * u * h * h * h;
    }
    if constexpr (OT == 0)
        return g / (1.0f + expf(-g)) * u;
    else
        return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f)) * u;
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
