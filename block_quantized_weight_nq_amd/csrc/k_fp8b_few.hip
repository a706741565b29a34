// k_fp8b_few.hip -- product of up to 64 rows with an E4M3 weight of 128 x 128 blocks, and of the few rows that each of
// many experts has.
//
//   y[m][n] = sum over blocks b of (sx[m][b] sw[n / 128][b]) * sum over k in b of cx[m][k] cw[n][k]
//
// What bounds it is the weight's bytes, each of which is needed once: codes go from memory to the registers of the
// lanes that multiply with them, and nothing is staged.  A wave takes 16 * NT weight rows and every W-th block of 128
// columns; the W waves' sums join through LDS in a fixed order.  Lane (j, g) of 16 x 4 holds columns 16 g .. 16 g + 15
// and 64 + 16 g .. 64 + 16 g + 15 of a block, for weight row j and for row j of x alike, so the order in which the
// instruction takes them does not matter.
//
// The codes become binary16, which holds them exactly, and the products run on the binary16 matrix instruction: its sums
// are binary32's, whereas the 8-bit one drops what lies 2^-13 below the largest of eight products.  The conversion (16
// instructions for 2 KB of weight) hides behind memory.
//
// Rows that are not codes yet are rounded here, each wave the blocks that it multiplies (k_fp8b_quant.hip's rule):
// the four lanes of a row hold its block, so the scale takes 32 values a lane and two exchanges.
#include "nq_fp8b_codes.h"

namespace nq {

namespace {

constexpr int MAX_WAVES = 8;

// What a lane reads of one block of 128 columns of a row of x.
template <int XT>
struct XPart {
    kv_u4 v[XT == 0 ? 8 : XT == FB_CODES ? 2 : 4];
    float scale;
};

template <int XT>
__device__ __forceinline__ void read_x(const uint8_t *row, const float *scale, int32_t kb, int g, XPart<XT> &p) {
    constexpr int ESZ = XT == 0 ? 4 : XT == FB_CODES ? 1 : 2, N = 16 * ESZ / 16;
    const uint8_t *at = row + ((int64_t)kb * FB + 16 * g) * ESZ;
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
        for (int i = 0; i < N; i++) p.v[h * N + i] = ((const kv_u4 *)(at + h * 64 * ESZ))[i];
    if constexpr (XT == FB_CODES) p.scale = scale[kb];
}

// The row's scale of the block, and the lane's 32 codes of it as binary16.
template <int XT>
__device__ __forceinline__ float x_codes(const XPart<XT> &p, kv_h8 (&c)[4]) {
    if constexpr (XT == FB_CODES) {
#pragma unroll
        for (int i = 0; i < 4; i++) c[i] = fb_half8(p.v[i >> 1][2 * (i & 1)], p.v[i >> 1][2 * (i & 1) + 1]);
        return p.scale;
    } else {
        float f[32];
        if constexpr (XT == 0) {
#pragma unroll
            for (int i = 0; i < 32; i++) f[i] = __builtin_bit_cast(float, (uint32_t)p.v[i >> 2][i & 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 32; i++) {
                const uint32_t w = p.v[i >> 3][(i >> 1) & 3], h = i & 1 ? w >> 16 : w & 0xFFFFu;
                f[i] = XT == 1 ? f16(h) : i & 1 ? bits_f32(w & 0xFFFF0000u) : bits_f32(w << 16);
            }
        }
        const auto row_max = [](uint32_t m) {
            uint32_t o = __shfl_xor(m, 16, 64);
            m = o > m ? o : m;
            o = __shfl_xor(m, 32, 64);
            return o > m ? o : m;
        };
        uint32_t top = row_max(fb_amax<32>(f, 0));
        if (__any(top >= 0x7F800000u)) {
            top = row_max(fb_amax_finite<32>(f, 0));
            fb_mark_not_finite<32>(f);
        }
        const float scale = fmaxf(__builtin_bit_cast(float, top) / 448.0f, FB_TINY), inv = 1.0f / scale;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float(&q)[32] = f;
            const uint32_t lo = fb_codes4(q[8 * i] * inv, q[8 * i + 1] * inv, q[8 * i + 2] * inv, q[8 * i + 3] * inv);
            const uint32_t hi = fb_codes4(q[8 * i + 4] * inv, q[8 * i + 5] * inv, q[8 * i + 6] * inv, q[8 * i + 7] * inv);
            c[i] = fb_half8(lo, hi);
        }
        return scale;
    }
}

}  // namespace

// RT tiles of 16 rows of x, NT of 16 weight rows (GATED: half of them gate, half up).
template <int XT, int RT, int NT, bool GATED>
__global__ __launch_bounds__(64 * MAX_WAVES) void k_fp8_few(Fp8GemmLaunch a) {
    extern __shared__ kv_f4 red[];  // [wave][RT][NT][lane]
    const int tid = threadIdx.x, lane = tid & 63, j = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = a.waves;
    Fp8Tile t;
    if (a.experts > 0) {
        t = fb_find_tile(a.offsets, a.experts, a.out_rows, 16 * RT, blockIdx.y);
    } else {
        t.expert = 0;
        t.first = (int64_t)blockIdx.y * 16 * RT;
        t.count = (int32_t)(a.out_rows - t.first < 16 * RT ? a.out_rows - t.first : 16 * RT);
    }
    if (t.count == 0) return;
    constexpr int OC = GATED ? 8 * NT : 16 * NT;  // output columns of the workgroup
    const int32_t NO = GATED ? a.N / 2 : a.N, n0 = (int32_t)blockIdx.x * OC;
    if (t.expert < 0) {
        for (int i = tid; i < t.count * OC; i += 64 * waves)
            if (n0 + i % OC < NO) fb_write1(a.out, (t.first + i / OC) * NO + n0 + i % OC, 0.0f, a.out_dtype);
        return;
    }
    const int32_t KB = a.K / FB;
    const uint8_t *w[NT];
    const float *ws[NT];
    {
        const int64_t e = t.expert, nb = fb_ceil(a.N, FB);
#pragma unroll
        for (int i = 0; i < NT; i++) {
            const int32_t base = GATED ? n0 + 16 * (i % (NT / 2 ? NT / 2 : 1)) + (i >= NT / 2 ? NO : 0) : n0 + 16 * i;
            const int32_t r = base + j < a.N ? base + j : a.N - 1;
            w[i] = a.w + (e * a.N + r) * a.K + 16 * g;
            ws[i] = a.w_scales + (e * nb + (base < a.N ? base : a.N - 1) / FB) * KB;
        }
    }
    const uint8_t *x[RT];
    const float *xs[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const int m = 16 * i + j;
        const int64_t r = fb_source_row(a, t.first + (m < t.count ? m : t.count - 1));
        x[i] = (const uint8_t *)a.x + r * a.x_stride * (XT == 0 ? 4 : XT == FB_CODES ? 1 : 2);
        xs[i] = XT == FB_CODES ? a.x_scales + r * (a.K / FB) : nullptr;
    }
    kv_f4 acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int i = 0; i < NT; i++) acc[r][i] = kv_f4{0.0f, 0.0f, 0.0f, 0.0f};

    struct Part {
        kv_u4 w[NT][2];
        float ws[NT];
        XPart<XT> x[RT];
    } part[2];
    const auto read = [&](Part &p, int32_t kb) {
#pragma unroll
        for (int i = 0; i < NT; i++) {
            p.w[i][0] = *(const kv_u4 *)(w[i] + (int64_t)kb * FB);
            p.w[i][1] = *(const kv_u4 *)(w[i] + (int64_t)kb * FB + 64);
            p.ws[i] = ws[i][kb];
        }
#pragma unroll
        for (int r = 0; r < RT; r++) read_x<XT>(x[r], xs[r], kb, g, p.x[r]);
    };
    const auto multiply = [&](const Part &p) {
        kv_h8 xc[RT][4];
        float sx[RT];
#pragma unroll
        for (int r = 0; r < RT; r++) sx[r] = x_codes<XT>(p.x[r], xc[r]);
#pragma unroll
        for (int i = 0; i < NT; i++) {
            kv_h8 wc[4];
#pragma unroll
            for (int q = 0; q < 4; q++) wc[q] = fb_half8(p.w[i][q >> 1][2 * (q & 1)], p.w[i][q >> 1][2 * (q & 1) + 1]);
#pragma unroll
            for (int r = 0; r < RT; r++) {
                kv_f4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int q = 0; q < 4; q++) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(wc[q], xc[r][q], d, 0, 0, 0);
                const float s = sx[r] * p.ws[i];
#pragma unroll
                for (int k = 0; k < 4; k++) acc[r][i][k] = __builtin_fmaf(d[k], s, acc[r][i][k]);
            }
        }
    };
    if (wave < KB) {
        int32_t kb = wave;
        read(part[0], kb);
        while (true) {
            int32_t next = kb + waves;
            if (next < KB) read(part[1], next);
            multiply(part[0]);
            if (next >= KB) break;
            kb = next, next = kb + waves;
            if (next < KB) read(part[0], next);
            multiply(part[1]);
            if (next >= KB) break;
            kb = next;
        }
    }
#pragma unroll
    for (int r = 0; r < RT; r++)
#pragma unroll
        for (int i = 0; i < NT; i++) red[((wave * RT + r) * NT + i) * 64 + lane] = acc[r][i];
    __syncthreads();
    constexpr int PER = GATED ? NT / 2 : NT;
    for (int q = tid; q < RT * PER * 64; q += 64 * waves) {
        const int at = q & 63, i = (q >> 6) % PER, r = (q >> 6) / PER;
        const auto total = [&](int tile) {
            kv_f4 y = red[(r * NT + tile) * 64 + at];
            for (int v = 1; v < waves; v++) {
                const kv_f4 o = red[((v * RT + r) * NT + tile) * 64 + at];
#pragma unroll
                for (int k = 0; k < 4; k++) y[k] += o[k];
            }
            return y;
        };
        const kv_f4 y = total(i);
        float f[4] = {y[0], y[1], y[2], y[3]};
        if constexpr (GATED) {
            const kv_f4 up = total(i + PER);
#pragma unroll
            for (int k = 0; k < 4; k++) f[k] = fb_silu<0>(f[k]) * up[k];
        }
        const int m = 16 * r + (at & 15), n = n0 + 16 * i + 4 * (at >> 4);
        if (m >= t.count) continue;
        const int64_t o = (t.first + m) * NO + n;
        if (NO % 4 == 0 && n + 3 < NO) {
            fb_write4(a.out, o, f, a.out_dtype);
        } else {
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (n + k < NO) fb_write1(a.out, o + k, f[k], a.out_dtype);
        }
    }
}

template <int XT, int RT, int NT, bool GATED>
static int few(const Fp8GemmLaunch &L, hipStream_t s) {
    const int32_t oc = GATED ? 8 * NT : 16 * NT, no = GATED ? L.N / 2 : L.N;
    const dim3 grid((uint32_t)fb_ceil(no, oc), (uint32_t)L.tiles_m);
    hipLaunchKernelGGL((k_fp8_few<XT, RT, NT, GATED>), grid, dim3(64 * L.waves), (uint32_t)L.waves * RT * NT * 1024, s, L);
    return hipGetLastError() == hipSuccess ? 0 : 9;  // NQ_ERR_HIP
}

template <int XT, int RT>
static int few_form(const Fp8GemmLaunch &L, hipStream_t s) {
    return L.gated ? few<XT, RT, 2, true>(L, s) : few<XT, RT, 2, false>(L, s);
}

int launch_fp8_few(const Fp8GemmLaunch &L, int row_tiles, hipStream_t s) {
    if (L.tiles_m == 0 || L.N == 0) return 0;
    if (L.x_type == FB_CODES) {
        switch (row_tiles) {
        case 1: return few_form<FB_CODES, 1>(L, s);
        case 2: return few_form<FB_CODES, 2>(L, s);
        default: return few_form<FB_CODES, 4>(L, s);
        }
    }
    switch (L.x_type) {
    case 0: return few_form<0, 1>(L, s);
    case 1: return few_form<1, 1>(L, s);
    default: return few_form<2, 1>(L, s);
    }
}

}  // namespace nq
