// k_fp8b_quant.hip -- values to E4M3 codes with one binary32 scale for each block of 128 columns (of one row, or of 128
// rows), and codes back to values.
//
//   scale = max(RN32(amax / 448), 2^-126), amax over the block's finite values,
//   code  = the E4M3 value nearest to RN32(x * RN32(1 / scale)) (ties to even); a NaN word where x is not finite,
//   value = RN32(code * scale), rounded once to the output type.
//
// RN32(x * inv) is at most 448 * (1 + 2^-22), which rounds to 448: no clamp is needed.  All three kernels are bound by
// the bytes they read and write.
#include "nq_fp8b.h"
#include "nq_fp8b_codes.h"

namespace nq {

namespace {
constexpr int TB = 256;
}

// One row and 128 columns a block: sixteen lanes of eight values.
template <int IN, bool VEC>
__global__ __launch_bounds__(TB) void k_fp8_quant_rows(Fp8QuantLaunch a) {
    const int lane = threadIdx.x & 15;
    const int64_t blocks = a.cols / FB, all = a.rows * blocks, step = (int64_t)gridDim.x * (TB / 16);
    for (int64_t i = (int64_t)blockIdx.x * (TB / 16) + (threadIdx.x >> 4); i < all; i += step) {
        const int64_t r = i / blocks, b = i - r * blocks;
        float f[8];
        fb_read8<IN, VEC>(a.x, r * a.row_stride + b * FB + 8 * lane, f);
        uint32_t top = fb_amax8(f, 0);
        top = fb_max16(top);
        const bool bad = top >= 0x7F800000u;
        if (bad) {
            top = fb_max16(fb_amax8_finite(f, 0));
            fb_mark_not_finite(f);
        }
        const float scale = fmaxf(__builtin_bit_cast(float, top) / 448.0f, FB_TINY), inv = 1.0f / scale;
        *(kv_u2 *)(a.codes + r * a.cols + b * FB + 8 * lane) = fb_codes8(f, inv);
        if (lane == 0) a.scales[i] = scale;
    }
}

// 128 rows and 128 columns a block: a workgroup, each thread eight columns of every sixteenth row.
template <int IN, bool VEC>
__global__ __launch_bounds__(TB) void k_fp8_quant_tile(Fp8QuantLaunch a) {
    __shared__ uint32_t wmax[TB / 64];
    const int tid = threadIdx.x, c = 8 * (tid & 15), r0 = tid >> 4;
    const int64_t blocks = a.cols / FB, bands = fb_ceil(a.rows, FB), all = a.matrices * bands * blocks;
    for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
        const int64_t b = i % blocks, band = i / blocks, m = band / bands, rb = (band - m * bands) * FB;
        const int rows = (int)(a.rows - rb < FB ? a.rows - rb : FB);
        const int64_t row0 = m * a.rows + rb;
        float f[8][8];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const int r = r0 + 16 * k;
#pragma unroll
            for (int j = 0; j < 8; j++) f[k][j] = 0.0f;
            if (r < rows) fb_read8<IN, VEC>(a.x, (row0 + r) * a.row_stride + b * FB + c, f[k]);
        }
        const auto largest = [&](bool finite) {
            top = 0;
#pragma unroll
            for (int k = 0; k < 8; k++) top = finite ? fb_amax8_finite(f[k], top) : fb_amax8(f[k], top);
            top = fb_max16(top);
            for (int d = 16; d < 64; d <<= 1) {
                const uint32_t other = __shfl_xor(top, d, 64);
                top = other > top ? other : top;
            }
            __syncthreads();
            if ((tid & 63) == 0) wmax[tid >> 6] = top;
            __syncthreads();
            for (int w = 0; w < TB / 64; w++) top = wmax[w] > top ? wmax[w] : top;
        };
        largest(false);
        if (top >= 0x7F800000u) {
            largest(true);
#pragma unroll
            for (int k = 0; k < 8; k++) fb_mark_not_finite(f[k]);
        }
        const float scale = fmaxf(__builtin_bit_cast(float, top) / 448.0f, FB_TINY), inv = 1.0f / scale;
        if (tid == 0) a.scales[i] = scale;
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const int r = r0 + 16 * k;
            if (r < rows) *(kv_u2 *)(a.codes + (row0 + r) * a.cols + b * FB + c) = fb_codes8(f[k], inv);
        }
    }
}

// Sixteen codes a thread and turn.
template <int OT>
__global__ __launch_bounds__(TB) void k_fp8_values(Fp8ValuesLaunch a) {
    const int64_t per = a.cols / 16, blocks = a.cols / FB, bands = fb_ceil(a.rows, a.tile);
    const int64_t all = a.matrices * a.rows * per, step = (int64_t)gridDim.x * TB;
    for (int64_t i = (int64_t)blockIdx.x * TB + threadIdx.x; i < all; i += step) {
        const int64_t row = i / per, c = i - row * per;
        int64_t band = row;
        if (a.tile != 1) {
            const int64_t m = row / a.rows;
            band = m * bands + (row - m * a.rows) / FB;
        }
        const float scale = a.scales[band * blocks + c / 8];
        const kv_u4 w = *(const kv_u4 *)(a.codes + 16 * i);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            float f[4];
            kv_codes4_f32<KV_E4M3>(w[e], f);
#pragma unroll
            for (int k = 0; k < 4; k++) f[k] = f[k] * scale;
            kv_write4<OT>(a.out, 16 * i + 4 * e, f);
        }
    }
}

template <int IN>
static int quantize_in(const Fp8QuantLaunch &L, hipStream_t s) {
    constexpr int64_t ESZ = IN == 0 ? 4 : 2;
    const bool vec = (uintptr_t)L.x % 16 == 0 && L.row_stride * ESZ % 16 == 0;
    const int64_t blocks = L.cols / FB;
    const int64_t units = L.tile == 1 ? fb_ceil(L.matrices * L.rows * blocks, TB / 16) : L.matrices * fb_ceil(L.rows, FB) * blocks;
    const int64_t most = (int64_t)device_compute_units() * 32;
    const dim3 grid((uint32_t)(units < most ? units : most));
    Fp8QuantLaunch a = L;
    if (L.tile == 1) {
        a.rows *= a.matrices;
        if (vec)
            hipLaunchKernelGGL((k_fp8_quant_rows<IN, true>), grid, dim3(TB), 0, s, a);
        else
            hipLaunchKernelGGL((k_fp8_quant_rows<IN, false>), grid, dim3(TB), 0, s, a);
    } else {
        if (vec)
            hipLaunchKernelGGL((k_fp8_quant_tile<IN, true>), grid, dim3(TB), 0, s, a);
        else
            hipLaunchKernelGGL((k_fp8_quant_tile<IN, false>), grid, dim3(TB), 0, s, a);
    }
    return hipGetLastError() == hipSuccess ? 0 : 9;  // NQ_ERR_HIP
}

int launch_fp8_quantize(const Fp8QuantLaunch &L, hipStream_t s) {
    if (L.rows == 0 || L.cols == 0 || L.matrices == 0) return 0;
    switch (L.in_dtype) {
    case 0: return quantize_in<0>(L, s);
    case 1: return quantize_in<1>(L, s);
    default: return quantize_in<2>(L, s);
    }
}

int launch_fp8_values(const Fp8ValuesLaunch &L, hipStream_t s) {
    const int64_t units = fb_ceil(L.matrices * L.rows * (L.cols / 16), TB), most = (int64_t)device_compute_units() * 32;
    if (units == 0) return 0;
    const dim3 grid((uint32_t)(units < most ? units : most));
    switch (L.out_dtype) {
    case 0: hipLaunchKernelGGL((k_fp8_values<0>), grid, dim3(TB), 0, s, L); break;
    case 1: hipLaunchKernelGGL((k_fp8_values<1>), grid, dim3(TB), 0, s, L); break;
    default: hipLaunchKernelGGL((k_fp8_values<2>), grid, dim3(TB), 0, s, L); break;
    }
    return hipGetLastError() == hipSuccess ? 0 : 9;  // NQ_ERR_HIP
}

}  // namespace nq
