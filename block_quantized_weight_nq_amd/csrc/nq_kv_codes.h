// nq_kv_codes.h -- device conversions of the 8-bit key/value cache.
#pragma once

#include "nq_kv.h"

namespace nq {

typedef _Float16 kv_h2 __attribute__((ext_vector_type(2)));
typedef _Float16 kv_h8 __attribute__((ext_vector_type(8)));
typedef float kv_f2 __attribute__((ext_vector_type(2)));
typedef float kv_f4 __attribute__((ext_vector_type(4)));
typedef uint32_t kv_u2 __attribute__((ext_vector_type(2)));
typedef uint32_t kv_u4 __attribute__((ext_vector_type(4)));
typedef __bf16 kv_b2 __attribute__((ext_vector_type(2)));

// Four codes as binary32 (exact).
template <int CODE>
__device__ __forceinline__ void kv_codes4_f32(uint32_t w, float (&f)[4]) {
    if constexpr (CODE == KV_Q8) {
#pragma unroll
        for (int i = 0; i < 4; i++) f[i] = (float)(int)(int8_t)(w >> (8 * i));
    } else {
        const kv_f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
        const kv_f2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        f[0] = a[0], f[1] = a[1], f[2] = b[0], f[3] = b[1];
    }
}

// Four binary32 values as codes: nearest, ties to even, saturated; NaN is 0.
// FINITE: there is none.  Signed bytes round by the addition of 1.5 * 2^23,
// after which the sum's low byte is the nearest integer (ties to even).
template <int CODE, bool FINITE = false>
__device__ __forceinline__ uint32_t kv_f32_codes4(const float (&f)[4]) {
    constexpr float TOP = CODE == KV_Q8 ? 127.0f : 448.0f;
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; i++) x[i] = __builtin_amdgcn_fmed3f(FINITE || f[i] == f[i] ? f[i] : 0.0f, -TOP, TOP);
    if constexpr (CODE == KV_Q8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = __builtin_bit_cast(uint32_t, x[i] + 12582912.0f);
        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(w[3], w[2], 0x0C0C0400u),
                                     __builtin_amdgcn_perm(w[1], w[0], 0x0C0C0400u), 0x05040100u);
    } else {
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
    }
}

// Eight codes as binary16 (exact: a signed byte has 7 bits, E4M3 4).  Signed
// bytes go through 1024 + (c + 128), whose binary16 word is 0x6400 | (c + 128).
template <int CODE>
__device__ __forceinline__ kv_h8 kv_codes8_f16(kv_u2 w) {
    kv_h8 r;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        kv_h2 a, b;
        if constexpr (CODE == KV_Q8) {
            const uint32_t x = w[i] ^ 0x80808080u;
            const uint32_t lo = __builtin_amdgcn_perm(0x64646464u, x, 0x04010400u);
            const uint32_t hi = __builtin_amdgcn_perm(0x64646464u, x, 0x04030402u);
            const kv_h2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
            a = __builtin_bit_cast(kv_h2, lo) - off;
            b = __builtin_bit_cast(kv_h2, hi) - off;
        } else {
            a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w[i], 1.0f, false);
            b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w[i], 1.0f, true);
        }
        r[4 * i] = a[0], r[4 * i + 1] = a[1], r[4 * i + 2] = b[0], r[4 * i + 3] = b[1];
    }
    return r;
}

// Element i of a source of type IN (0 binary32, 1 binary16, 2 bfloat16) as binary32.
template <int IN>
__device__ __forceinline__ float kv_read(const void *x, int64_t i) {
    if constexpr (IN == 0)
        return ((const float *)x)[i];
    else if constexpr (IN == 1)
        return (float)((const _Float16 *)x)[i];
    else
        return bits_f32((uint32_t)((const uint16_t *)x)[i] << 16);
}

// Four consecutive elements; VEC: the address is a multiple of four elements' bytes.
template <int IN, bool VEC>
__device__ __forceinline__ void kv_read4(const void *x, int64_t i, float (&f)[4]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 4; j++) f[j] = kv_read<IN>(x, i + j);
    } else if constexpr (IN == 0) {
        const kv_f4 w = *(const kv_f4 *)((const float *)x + i);
#pragma unroll
        for (int j = 0; j < 4; j++) f[j] = w[j];
    } else {
        const kv_u2 w = *(const kv_u2 *)((const uint16_t *)x + i);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t h = (w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
            f[j] = IN == 1 ? f16(h) : bits_f32(h << 16);
        }
    }
}

// Sixteen consecutive elements; VEC: the address is a multiple of 16 bytes.
template <int IN, bool VEC>
__device__ __forceinline__ void kv_read16(const void *x, int64_t i, float (&f)[16]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 16; j++) f[j] = kv_read<IN>(x, i + j);
    } else if constexpr (IN == 0) {
#pragma unroll
        for (int v = 0; v < 4; v++) {
            const kv_f4 w = *(const kv_f4 *)((const float *)x + i + 4 * v);
#pragma unroll
            for (int j = 0; j < 4; j++) f[4 * v + j] = w[j];
        }
    } else {
#pragma unroll
        for (int v = 0; v < 2; v++) {
            const kv_u4 w = *(const kv_u4 *)((const uint16_t *)x + i + 8 * v);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t h = (w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
                f[8 * v + j] = IN == 1 ? f16(h) : bits_f32(h << 16);
            }
        }
    }
}

// Four consecutive elements of type OT, rounded to nearest even; the address is a multiple of their bytes.
template <int OT>
__device__ __forceinline__ void kv_write4(void *y, int64_t i, const float (&f)[4]) {
    if constexpr (OT == 0) {
        kv_f4 w = {f[0], f[1], f[2], f[3]};
        *(kv_f4 *)((float *)y + i) = w;
    } else if constexpr (OT == 1) {
        const kv_f2 a = {f[0], f[1]}, b = {f[2], f[3]};
        kv_u2 w = {__builtin_bit_cast(uint32_t, __builtin_convertvector(a, kv_h2)),
                   __builtin_bit_cast(uint32_t, __builtin_convertvector(b, kv_h2))};
        *(kv_u2 *)((uint16_t *)y + i) = w;
    } else {
        const kv_f2 a = {f[0], f[1]}, b = {f[2], f[3]};
        kv_u2 w = {__builtin_bit_cast(uint32_t, __builtin_convertvector(a, kv_b2)),
                   __builtin_bit_cast(uint32_t, __builtin_convertvector(b, kv_b2))};
        *(kv_u2 *)((uint16_t *)y + i) = w;
    }
}

}  // namespace nq
