// k_fp8b_rows.hip -- product of many rows with an E4M3 weight of 128 x 128 blocks, or of each expert's rows with its own.
//
//   y[m][n] = sum over blocks b of (sx[m][b] sw[n / 128][b]) * sum over k in b of cx[m][k] cw[n][k]
//
// A workgroup of WN x WM waves takes 16 WN TN weight rows by 16 WM TM rows of x, one block of 128 columns at a time.
// The weight is the matrix instruction's first operand: a lane then holds four consecutive outputs of one row of x,
// whose scale is one register, and the weight's scale is one for all lanes.
#include "nq_fp8b_codes.h"

namespace nq {

typedef int fb_i8 __attribute__((ext_vector_type(8)));

namespace {

// LDS holds rows of 128 bytes as eight pieces of 16; piece c of row r lies at c ^ (r / 2 % 8), so that sixteen lanes
// that read one piece of sixteen rows spread over all banks.
__device__ __forceinline__ uint32_t lds_at(int row, int piece) { return (uint32_t)(row * FB + ((piece ^ (row >> 1 & 7)) << 4)); }

}  // namespace

template <int WN, int WM, int TN, int TM, bool WIDE, bool GATED>
__global__ __launch_bounds__(64 * WN * WM) void k_fp8_rows(Fp8GemmLaunch a) {
    constexpr int BN = 16 * WN * TN, BM = 16 * WM * TM, THREADS = 64 * WN * WM, STAGE = (BN + BM) * 8 / THREADS;
    constexpr int H = TN / 2;  // a wave's tiles are two halves, each within one row of blocks
    __shared__ __align__(16) uint8_t lds[2 * (BN + BM) * FB];
    const int tid = threadIdx.x, lane = tid & 63, j = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wn = wave % WN, wm = wave / WN;
    const int32_t KB = a.K / FB, NO = GATED ? a.N / 2 : a.N;
    const int32_t tiles_n = (int32_t)fb_ceil(a.N, BN);
    const int64_t tile = blockIdx.x;
    const int32_t tn = (int32_t)(tile % tiles_n);
    Fp8Tile t;
    if (a.experts > 0) {
        t = fb_find_tile(a.offsets, a.experts, a.out_rows, BM, tile / tiles_n);
    } else {
        t.expert = 0;
        t.first = tile / tiles_n * BM;
        t.count = (int32_t)(a.out_rows - t.first < BM ? a.out_rows - t.first : BM);
    }
    if (t.count == 0) return;
    constexpr int OC = GATED ? BN / 2 : BN;
    const int32_t n0 = tn * OC;
    if (t.expert < 0) {
        for (int i = tid; i < t.count * OC; i += THREADS)
            if (n0 + i % OC < NO) fb_write1(a.out, (t.first + i / OC) * NO + n0 + i % OC, 0.0f, a.out_dtype);
        return;
    }
    // weight row of row r of the tile (of a wave's rows, the first half are gates and the second up, where GATED)
    const auto weight_row = [&](int r) {
        if constexpr (GATED) {
            const int v = r / (16 * TN), in = r % (16 * TN);
            return n0 + v * 16 * H + in % (16 * H) + (in >= 16 * H ? NO : 0);
        } else {
            return n0 + r;
        }
    };
    const uint8_t *const w = a.w + (int64_t)t.expert * a.N * a.K;
    const uint8_t *from[STAGE];
    uint32_t to[STAGE];
#pragma unroll
    for (int i = 0; i < STAGE; i++) {
        const int r = (tid + i * THREADS) >> 3, c = tid & 7;
        to[i] = lds_at(r, c);
        if (r < BN) {
            const int32_t n = weight_row(r);
            from[i] = w + (int64_t)(n < a.N ? n : a.N - 1) * a.K + 16 * c;
        } else {
            const int m = r - BN;
            from[i] = (const uint8_t *)a.x + fb_source_row(a, t.first + (m < t.count ? m : t.count - 1)) * a.x_stride + 16 * c;
        }
    }
    const float *xs[TM], *ws[2];
#pragma unroll
    for (int i = 0; i < TM; i++) {
        const int m = 16 * (wm * TM + i) + j;
        xs[i] = a.x_scales + fb_source_row(a, t.first + (m < t.count ? m : t.count - 1)) * a.x_scale_row;
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int32_t n = weight_row(16 * (wn * TN + h * H));
        ws[h] = a.w_scales + ((int64_t)t.expert * fb_ceil(a.N, FB) + (n < a.N ? n : a.N - 1) / FB) * KB;
    }
    const int32_t kb0 = (int32_t)blockIdx.y * a.per_split, kb1 = kb0 + a.per_split < KB ? kb0 + a.per_split : KB;

    kv_f4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; i++)
#pragma unroll
        for (int k = 0; k < TM; k++) acc[i][k] = kv_f4{0.0f, 0.0f, 0.0f, 0.0f};
    kv_u4 stage[STAGE];
    const auto read = [&](int32_t kb) {
#pragma unroll
        for (int i = 0; i < STAGE; i++) stage[i] = *(const kv_u4 *)(from[i] + (int64_t)kb * FB);
    };
    const auto put = [&](uint8_t *b) {
#pragma unroll
        for (int i = 0; i < STAGE; i++) *(kv_u4 *)(b + to[i]) = stage[i];
    };
    const auto fetch = [&](const uint8_t *b, int row, fb_i8 *v) {
        const kv_u4 lo = *(const kv_u4 *)(b + lds_at(row + j, g)), hi = *(const kv_u4 *)(b + lds_at(row + j, g + 4));
#pragma unroll
        for (int i = 0; i < 4; i++) (*v)[i] = (int)lo[i], (*v)[4 + i] = (int)hi[i];
    };
    read(kb0);
    put(lds);
    __syncthreads();
    for (int32_t kb = kb0; kb < kb1; kb++) {
        const uint8_t *const b = lds + ((kb - kb0) & 1) * (BN + BM) * FB;
        if (kb + 1 < kb1) read(kb + 1);
        float sx[TM], sw[2];
#pragma unroll
        for (int i = 0; i < TM; i++) sx[i] = xs[i][(int64_t)kb * a.x_scale_col];
        sw[0] = ws[0][kb], sw[1] = ws[1][kb];
        fb_i8 xf[TM];
#pragma unroll
        for (int i = 0; i < TM; i++) fetch(b, BN + 16 * (wm * TM + i), &xf[i]);
#pragma unroll
        for (int i = 0; i < TN; i++) {
            fb_i8 wf;
            fetch(b, 16 * (wn * TN + i), &wf);
#pragma unroll
            for (int k = 0; k < TM; k++) {
                kv_f4 d = {0.0f, 0.0f, 0.0f, 0.0f};
                if constexpr (WIDE) {
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb_half8((uint32_t)wf[2 * q], (uint32_t)wf[2 * q + 1]),
                                                                   fb_half8((uint32_t)xf[k][2 * q], (uint32_t)xf[k][2 * q + 1]), d, 0, 0, 0);
                } else {
                    d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf[k], d, 0, 0, 0, 0, 0, 0);
                }
                const float s = sx[k] * sw[i >= H];
#pragma unroll
                for (int q = 0; q < 4; q++) acc[i][k][q] = __builtin_fmaf(d[q], s, acc[i][k][q]);
            }
        }
        if (kb + 1 < kb1) put(lds + ((kb + 1 - kb0) & 1) * (BN + BM) * FB);
        __syncthreads();
    }
    // lane (j, g): outputs 4 g .. 4 g + 3 of each tile of weight rows, of row j
    const bool whole = a.splits > 1;
#pragma unroll
    for (int k = 0; k < TM; k++) {
        const int m = 16 * (wm * TM + k) + j;
        if (m >= t.count) continue;
        if (whole) {
            float *const part = a.part + ((int64_t)blockIdx.y * a.out_rows + t.first + m) * a.N;
#pragma unroll
            for (int i = 0; i < TN; i++) {
                const int32_t n = weight_row(16 * (wn * TN + i)) + 4 * g;
                if (a.N % 4 == 0 && n + 3 < a.N)
                    *(kv_f4 *)(part + n) = acc[i][k];
                else
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        if (n + q < a.N) part[n + q] = acc[i][k][q];
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < (GATED ? H : TN); i++) {
            const int32_t n = weight_row(16 * (wn * TN + i)) + 4 * g;
            float f[4];
#pragma unroll
            for (int q = 0; q < 4; q++) f[q] = GATED ? fb_silu(acc[i][k][q]) * acc[GATED ? i + H : i][k][q] : acc[i][k][q];
            const int64_t o = (t.first + m) * NO + n;
            if (NO % 4 == 0 && n + 3 < NO) {
                fb_write4(a.out, o, f, a.out_dtype);
            } else {
#pragma unroll
                for (int q = 0; q < 4; q++)
                    if (n + q < NO) fb_write1(a.out, o + q, f[q], a.out_dtype);
            }
        }
    }
}

// The pieces' sums in order, and the epilogue.
__global__ __launch_bounds__(256) void k_fp8_join(Fp8GemmLaunch a) {
    const int32_t NO = a.gated ? a.N / 2 : a.N;
    const int64_t all = a.out_rows * NO, step = (int64_t)gridDim.x * 256, piece = a.out_rows * a.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += step) {
        const int64_t m = i / NO, n = i - m * NO;
        const float *p = a.part + m * a.N + n;
        float y = p[0], up = a.gated ? p[NO] : 0.0f;
        for (int s = 1; s < a.splits; s++) {
            y += p[s * piece];
            if (a.gated) up += p[s * piece + NO];
        }
        fb_write1(a.out, i, a.gated ? fb_silu(y) * up : y, a.out_dtype);
    }
}

template <int WN, int WM, int TN, int TM, bool WIDE, bool GATED>
static int rows(const Fp8GemmLaunch &L, hipStream_t s) {
    constexpr int BN = 16 * WN * TN, BM = 16 * WM * TM;
    const dim3 grid((uint32_t)(fb_ceil(L.N, BN) * L.tiles_m), (uint32_t)L.splits);
    hipLaunchKernelGGL((k_fp8_rows<WN, WM, TN, TM, WIDE, GATED>), grid, dim3(64 * WN * WM), 0, s, L);
    if (hipGetLastError() != hipSuccess) return 9;  // NQ_ERR_HIP
    if (L.splits > 1) {
        const int64_t units = fb_ceil(L.out_rows * (GATED ? L.N / 2 : L.N), 256), most = (int64_t)device_compute_units() * 16;
        hipLaunchKernelGGL(k_fp8_join, dim3((uint32_t)(units < most ? units : most)), dim3(256), 0, s, L);
        if (hipGetLastError() != hipSuccess) return 9;
    }
    return 0;
}

template <bool WIDE, bool GATED>
static int rows_of(const Fp8GemmLaunch &L, int config, hipStream_t s) {
    switch (config) {
    case 0: return rows<4, 1, 2, 4, WIDE, GATED>(L, s);
    case 1: return rows<2, 2, 4, 4, WIDE, GATED>(L, s);
    default: return rows<2, 4, 8, 4, WIDE, GATED>(L, s);
    }
}

int launch_fp8_rows(const Fp8GemmLaunch &L, int config, hipStream_t s) {
    if (L.tiles_m == 0 || L.N == 0) return 0;
    const bool wide = L.out_dtype == 0;
    if (L.gated) return wide ? rows_of<true, true>(L, config, s) : rows_of<false, true>(L, config, s);
    return wide ? rows_of<true, false>(L, config, s) : rows_of<false, false>(L, config, s);
}

}  // namespace nq
