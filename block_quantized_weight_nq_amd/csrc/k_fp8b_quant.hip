// k_fp8b_quant.hip -- values to E4M3 codes with one binary32 scale for each block of 128 columns (of one row, or of 128
// rows), and codes back to values.
//
//   scale = max(RN32(amax / 448), 2^-126), amax over the block's finite values,
//   code  = the E4M3 value nearest to RN32(x * RN32(1 / scale)) (ties to even); a NaN word where x is not finite,
//   value = RN32(code * scale), rounded once to the output type.
//
// RN32(x * inv) is at most 448 * (1 + 2^-22), which rounds to 448: no clamp is needed.  All three kernels are bound by
// the bytes they read and write (a copy moves 5.0 TB/s): 8192 rows of 4096 bfloat16 values 21.6 us, 4.7 TB/s; tiles of
// [14336, 4096] 34 us, 5.2 TB/s; their values back 27.5 us, 6.4 TB/s (the codes are still in the last cache).  7 rows of
// 4096: 3.1 us, one load's way to memory and back, and the launch.
#include "nq_fp8b.h"
#include "nq_fp8b_codes.h"

namespace nq {

namespace {
constexpr int TB = 256;
}

// One row and 128 columns a block: sixteen lanes of eight values, whose maximum goes through the lanes' own exchange.
template <int IN, bool VEC>
__global__ __launch_bounds__(TB) void k_fp8_quant_rows(Fp8QuantLaunch a) {
    const int lane = threadIdx.x & 15;
    const int64_t blocks = a.cols / FB, all = a.rows * blocks, step = (int64_t)gridDim.x * (TB / 16);
    for (int64_t i = (int64_t)blockIdx.x * (TB / 16) + (threadIdx.x >> 4); i < all; i += step) {
        const int64_t r = i / blocks, b = i - r * blocks;
        const FbRaw<IN> v = fb_raw8<IN, VEC>(a.x, r * a.row_stride + b * FB + 8 * lane);
        uint32_t top = fb_max16(fb_amax_word<IN>(fb_amax8<IN>(v, 0)));
        const bool bad = top >= 0x7F800000u;
        if (bad) top = fb_max16(fb_amax8_finite<IN>(v, 0));
        const float scale = fb_scale(top), inv = 1.0f / scale;
        *(kv_u2 *)(a.codes + r * a.cols + b * FB + 8 * lane) = bad ? fb_codes8<IN, true>(v, inv) : fb_codes8<IN, false>(v, inv);
        if (lane == 0) a.scales[i] = scale;
    }
}

// 128 rows and 128 columns a block: a workgroup, each thread eight columns of ROWS rows, which it holds as they are (16-bit
// values in half the registers of binary32 ones; held as binary32, 56.8 us for [14336, 4096] bfloat16).
template <int IN, bool VEC>
__global__ __launch_bounds__(IN == 0 ? 2 * TB : TB) void k_fp8_quant_tile(Fp8QuantLaunch a) {
    constexpr int THREADS = IN == 0 ? 2 * TB : TB, STEP = THREADS / 16, ROWS = FB / STEP;
    __shared__ uint32_t wmax[2][THREADS / 64];
    const int tid = threadIdx.x, c = 8 * (tid & 15), r0 = tid >> 4;
    const int64_t blocks = a.cols / FB, bands = fb_ceil(a.rows, FB), all = a.matrices * bands * blocks;
    int turn = 0;
    for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
        const int64_t band = i / blocks, b = i - band * blocks, m = band / bands, rb = (band - m * bands) * FB;
        const int rows = (int)(a.rows - rb < FB ? a.rows - rb : FB);
        const int64_t row0 = m * a.rows + rb;
        FbRaw<IN> v[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; k++) {
            const int r = r0 + STEP * k;
            v[k] = fb_raw8<IN, VEC>(a.x, (row0 + (r < rows ? r : rows - 1)) * a.row_stride + b * FB + c);  // (a row twice changes no maximum)
        }
        const auto largest = [&](uint32_t top) {
            top = fb_max16(top);
            for (int d = 16; d < 64; d <<= 1) {
                const uint32_t other = __shfl_xor(top, d, 64);
                top = other > top ? other : top;
            }
            turn ^= 1;  // the words of the turn before may still be read
            if ((tid & 63) == 0) wmax[turn][tid >> 6] = top;
            __syncthreads();
            for (int w = 0; w < THREADS / 64; w++) top = wmax[turn][w] > top ? wmax[turn][w] : top;
            return top;
        };
        uint32_t words = 0;
#pragma unroll
        for (int k = 0; k < ROWS; k++) words = fb_amax8<IN>(v[k], words);
        uint32_t top = largest(fb_amax_word<IN>(words));
        const bool bad = top >= 0x7F800000u;
        if (bad) {
            top = 0;
#pragma unroll
            for (int k = 0; k < ROWS; k++) top = fb_amax8_finite<IN>(v[k], top);
            top = largest(top);
        }
        const float scale = fb_scale(top), inv = 1.0f / scale;
        if (tid == 0) a.scales[i] = scale;
#pragma unroll
        for (int k = 0; k < ROWS; k++) {
            const int r = r0 + STEP * k;
            if (r < rows)
                *(kv_u2 *)(a.codes + (row0 + r) * a.cols + b * FB + c) = bad ? fb_codes8<IN, true>(v[k], inv) : fb_codes8<IN, false>(v[k], inv);
        }
    }
}

// A thread and turn: four accesses of 16 bytes of values, side by side with its neighbours', all four on their way.
template <int OT>
__global__ __launch_bounds__(TB) void k_fp8_values(Fp8ValuesLaunch a) {
    constexpr int PER = OT == 0 ? 4 : 8, TURNS = 4;
    const int64_t per = a.cols / PER, blocks = a.cols / FB, bands = fb_ceil(a.rows, a.tile);
    const int64_t all = a.matrices * a.rows * per, step = (int64_t)gridDim.x * TB * TURNS;
    for (int64_t i0 = (int64_t)blockIdx.x * TB * TURNS + threadIdx.x; i0 < all; i0 += step) {
        uint32_t w[TURNS][PER / 4];
        float scale[TURNS];
#pragma unroll
        for (int k = 0; k < TURNS; k++) {
            const int64_t i = i0 + k * TB < all ? i0 + k * TB : i0, row = i / per, c = i - row * per;
            int64_t band = row;
            if (a.tile != 1) {
                const int64_t m = row / a.rows;
                band = m * bands + (row - m * a.rows) / FB;
            }
            scale[k] = a.scales[band * blocks + c / (FB / PER)];
#pragma unroll
            for (int e = 0; e < PER / 4; e++) w[k][e] = ((const uint32_t *)a.codes)[i * (PER / 4) + e];
        }
#pragma unroll
        for (int k = 0; k < TURNS; k++) {
            if (i0 + k * TB >= all) break;
#pragma unroll
            for (int e = 0; e < PER / 4; e++) {
                float f[4];
                kv_codes4_f32<KV_E4M3>(w[k][e], f);
#pragma unroll
                for (int j = 0; j < 4; j++) f[j] = f[j] * scale[k];
                kv_write4<OT>(a.out, (i0 + k * TB) * PER + 4 * e, f);
            }
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
        const dim3 threads(IN == 0 ? 2 * TB : TB);
        if (vec)
            hipLaunchKernelGGL((k_fp8_quant_tile<IN, true>), grid, threads, 0, s, a);
        else
            hipLaunchKernelGGL((k_fp8_quant_tile<IN, false>), grid, threads, 0, s, a);
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
    const int64_t units = fb_ceil(L.matrices * L.rows * (L.cols / (L.out_dtype == 0 ? 4 : 8)), 4 * TB), most = (int64_t)device_compute_units() * 32;
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
