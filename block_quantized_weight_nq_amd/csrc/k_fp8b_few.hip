// k_fp8b_few.hip -- product of up to 16 rows with an E4M3 weight of 128 x 128 blocks, and of the few rows that each of
// many experts has, 16 a workgroup.
//
//   y[m][n] = sum over blocks b of (sx[m][b] sw[n / 128][b]) * sum over k in b of cx[m][k] cw[n][k]
//
// What bounds it is the weight's bytes, each of which is needed once: codes go from memory to the registers of the
// lanes that multiply with them, and nothing is staged.  A wave takes 16 * NT weight rows and every W-th block of 128
// columns; the W waves' sums join through LDS in a fixed order.  Lane (j, g) of 16 x 4 holds columns 16 g .. 16 g + 15
// and 64 + 16 g .. 64 + 16 g + 15 of a block, for weight row j and for row j of x alike, so the order in which the
// instruction takes them does not matter.  One row of gated [28672, 4096]: 24.2 us, 4.9 TB/s of the 5.0 that a copy moves;
// 32 pairs on 64 experts of gated [2816, 2048], 144 MB where 25 of them are busy: 31.2 us, 4.6 TB/s.  (Loads of the weight
// that go past the L2s are slower; 32 and 64 rows a workgroup take 110 us for 33 to 64 rows of [28672, 4096], the kernel for
// many rows 32.)
//
// The codes become binary16, which holds them exactly, and the products run on the binary16 matrix instruction: its sums
// are binary32's, whereas the 8-bit one drops what lies 2^-13 below the largest of eight products.  The conversion (16
// instructions for 2 KB of weight) hides behind memory.
//
// Rows that are not codes yet are rounded here (k_fp8b_quant.hip's rule), by the whole workgroup into LDS, as many blocks
// at a time as have room; the first weight codes are on their way meanwhile.  (Each wave for itself, in the registers
// that multiply: 150 vector instructions a block of 128, which bound it at 3.5 TB/s.)
#include "nq_fp8b_codes.h"

#include <type_traits>

namespace nq {

namespace {

constexpr int MAX_WAVES = 8;

// Where 16 bytes of a block of row r lie in LDS: blocks of `rows` rows of 128 bytes, whose pieces are exchanged by the
// row's number, so that sixteen rows' pieces spread over all banks.
__device__ __forceinline__ int x_place(int block, int rows, int r, int piece) {
    return (block * rows + r) * FB + ((piece ^ (r >> 1 & 7)) << 4);
}

}  // namespace

// 16 rows of x, NT tiles of 16 weight rows (GATED: half of them gate, half up).
template <int XT, int NT, bool GATED>
__global__ __launch_bounds__(64 * MAX_WAVES) void k_fp8_few(Fp8GemmLaunch a) {
    // codes of x, a block's rows together, and their scales; in the end the waves' sums, [wave][NT][lane]
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ __align__(8) uint8_t lost[MAX_WAVES];
    const int tid = threadIdx.x, lane = tid & 63, j = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = a.waves;
    Fp8Tile t;
    if (a.experts > 0) {
        t = fb_find_tile(a.offsets, a.experts, a.out_rows, 16, (int32_t)blockIdx.y);
    } else {
        t.expert = 0;
        t.first = (int64_t)blockIdx.y * 16;
        t.count = (int32_t)(a.out_rows - t.first < 16 ? a.out_rows - t.first : 16);
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
    constexpr bool RAW = XT != FB_CODES;
    const int row = j < t.count ? j : t.count - 1;
    const uint8_t *x = nullptr;
    const float *xs = nullptr;
    if constexpr (!RAW) {
        const int64_t r = fb_source_row(a, t.first + row);
        x = (const uint8_t *)a.x + r * a.x_stride + 16 * g;
        xs = a.x_scales + r * KB;
    }
    constexpr int DEPTH = fb_few_depth(NT);
    kv_f4 acc[NT];

    struct Part {
        kv_u4 w[NT][2], x[2];
        float ws[NT], xs;
    } part[DEPTH];
    const auto read = [&](Part &p, int32_t kb) {
#pragma unroll
        for (int i = 0; i < NT; i++) {
            p.w[i][0] = *(const kv_u4 *)(w[i] + (int64_t)kb * FB);
            p.w[i][1] = *(const kv_u4 *)(w[i] + (int64_t)kb * FB + 64);
            p.ws[i] = ws[i][kb];
        }
        if constexpr (!RAW) {
            p.x[0] = *(const kv_u4 *)(x + (int64_t)kb * FB);
            p.x[1] = *(const kv_u4 *)(x + (int64_t)kb * FB + 64);
            p.xs = xs[kb];
        }
    };
    // codes of blocks from c0 on, as many as a.chunk, into LDS: four lanes take a row's block, 32 values each
    float *const scales = (float *)(lds + (int64_t)a.chunk * t.count * FB);
    const auto refill = [&](int32_t c0) {
        const int pairs = t.count * (KB - c0 < a.chunk ? KB - c0 : a.chunk), l = tid & 3;
        __syncthreads();
        for (int q = tid >> 2; q < pairs; q += 16 * waves) {
            const int b = q / t.count, m = q - b * t.count;
            const int64_t at = fb_source_row(a, t.first + m) * a.x_stride + (int64_t)(c0 + b) * FB + 32 * l;
            constexpr int IN = RAW ? XT : 0;
            FbRaw<IN> v[4];
#pragma unroll
            for (int u = 0; u < 4; u++) v[u] = fb_raw8<IN, true>(a.x, at + 8 * u);
            uint32_t words = 0;
#pragma unroll
            for (int u = 0; u < 4; u++) words = fb_amax8<IN>(v[u], words);
            uint32_t top = fb_max4(fb_amax_word<IN>(words));
            const bool bad = top >= 0x7F800000u;
            if (bad) {
                top = 0;
#pragma unroll
                for (int u = 0; u < 4; u++) top = fb_amax8_finite<IN>(v[u], top);
                top = fb_max4(top);
            }
            const float scale = fb_scale(top), inv = 1.0f / scale;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const kv_u2 lo = bad ? fb_codes8<IN, true>(v[2 * h], inv) : fb_codes8<IN, false>(v[2 * h], inv);
                const kv_u2 hi = bad ? fb_codes8<IN, true>(v[2 * h + 1], inv) : fb_codes8<IN, false>(v[2 * h + 1], inv);
                *(kv_u4 *)(lds + x_place(b, t.count, m, 2 * l + h)) = kv_u4{lo[0], lo[1], hi[0], hi[1]};
            }
            if (l == 0) scales[q] = scale;
        }
        __syncthreads();
    };
    float most = 0.0f;  // the largest sx * sw so far
    const auto multiply = [&](auto careful, const Part &p, int32_t block) {
        kv_u4 v[2];
        float sx;
        if constexpr (RAW) {
            v[0] = *(const kv_u4 *)(lds + x_place(block, t.count, row, g));
            v[1] = *(const kv_u4 *)(lds + x_place(block, t.count, row, g + 4));
            sx = scales[block * t.count + row];
        } else {
            v[0] = p.x[0], v[1] = p.x[1];
            sx = p.xs;
        }
        kv_h8 xc[4];
#pragma unroll
        for (int q = 0; q < 4; q++) xc[q] = fb_half8(v[q >> 1][2 * (q & 1)], v[q >> 1][2 * (q & 1) + 1]);
#pragma unroll
        for (int i = 0; i < NT; i++) {
            kv_f4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < 4; q++)
                d = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb_half8(p.w[i][q >> 1][2 * (q & 1)], p.w[i][q >> 1][2 * (q & 1) + 1]), xc[q], d, 0, 0, 0);
            const float s = sx * p.ws[i];
            if constexpr (!careful()) most = fmaxf(most, fabsf(s));
#pragma unroll
            for (int k = 0; k < 4; k++) acc[i][k] = careful() ? fb_scaled(d[k], sx, p.ws[i], s, acc[i][k]) : __builtin_fmaf(d[k], s, acc[i][k]);
        }
    };
    const auto blocks = [&](auto careful) {
#pragma unroll
        for (int i = 0; i < NT; i++) acc[i] = kv_f4{0.0f, 0.0f, 0.0f, 0.0f};
        // a.chunk is a multiple of DEPTH * waves
#pragma unroll
        for (int d = 0; d < DEPTH; d++)
            if (wave + d * waves < KB) read(part[d], wave + d * waves);
        for (int32_t c0 = 0; c0 < KB; c0 += a.chunk) {
            if constexpr (RAW) refill(c0);
            const int32_t end = KB - c0 < a.chunk ? KB - c0 : a.chunk;
            for (int32_t b = wave; b < end; b += DEPTH * waves) {
#pragma unroll
                for (int d = 0; d < DEPTH; d++) {
                    const int32_t now = b + d * waves, next = c0 + now + DEPTH * waves;
                    if (now < end) multiply(careful, part[d], now);
                    if (next < KB) read(part[d], next);
                }
            }
        }
        if constexpr (RAW) __syncthreads();
    };
    blocks(std::false_type());
    const bool left = __any(most > FB_MOST);
    if (lane == 0) lost[wave] = left;
    kv_f4 *const red = (kv_f4 *)lds;
#pragma unroll
    for (int i = 0; i < NT; i++) red[(wave * NT + i) * 64 + lane] = acc[i];
    __syncthreads();
    // Where some sx * sw left binary32 (fb_scaled), the workgroup does all again with care (a choice at each block: 1 us of 34
    // for 4 x 8 pairs on 64 gated [2816, 2048]).
    if (*(const uint64_t *)lost << (64 - 8 * waves)) {
        blocks(std::true_type());
#pragma unroll
        for (int i = 0; i < NT; i++) red[(wave * NT + i) * 64 + lane] = acc[i];
        __syncthreads();
    }
    constexpr int PER = GATED ? NT / 2 : NT;
    for (int q = tid; q < PER * 64; q += 64 * waves) {
        const int at = q & 63, i = q >> 6;
        const auto total = [&](int tile) {
            kv_f4 y = red[tile * 64 + at];
            for (int v = 1; v < waves; v++) {
                const kv_f4 o = red[(v * NT + tile) * 64 + at];
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
            for (int k = 0; k < 4; k++) f[k] = fb_gate<0>(f[k], up[k]);
        }
        const int m = at & 15, n = n0 + 16 * i + 4 * (at >> 4);
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

template <int XT, int NT, bool GATED>
static int few(Fp8GemmLaunch L, hipStream_t s) {
    const int32_t no = GATED ? L.N / 2 : L.N;
    const dim3 grid((uint32_t)fb_ceil(no, fb_few_cols(NT, GATED)), (uint32_t)L.tiles_m);
    uint32_t room = 0;
    L.chunk = L.K / FB;
    if (XT != FB_CODES) {
        const int32_t rows = L.out_rows < 16 ? (int32_t)L.out_rows : 16;
        L.chunk = fb_few_chunk(L.out_rows, L.waves, NT);
        room = (uint32_t)(L.chunk * rows * (FB + 4));
    }
    const uint32_t sums = (uint32_t)L.waves * NT * 1024;
    hipLaunchKernelGGL((k_fp8_few<XT, NT, GATED>), grid, dim3(64 * L.waves), room > sums ? room : sums, s, L);
    return hipGetLastError() == hipSuccess ? 0 : 9;  // NQ_ERR_HIP
}

template <int XT>
static int few_form(const Fp8GemmLaunch &L, int weight_tiles, hipStream_t s) {
    if (L.gated) return weight_tiles == 4 ? few<XT, 4, true>(L, s) : few<XT, 2, true>(L, s);
    return weight_tiles == 1 ? few<XT, 1, false>(L, s) : few<XT, 2, false>(L, s);
}

int launch_fp8_few(const Fp8GemmLaunch &L, int weight_tiles, hipStream_t s) {
    if (L.tiles_m == 0 || L.N == 0) return 0;
    switch (L.x_type) {
    case 0: return few_form<0>(L, weight_tiles, s);
    case 1: return few_form<1>(L, weight_tiles, s);
    case 2: return few_form<2>(L, weight_tiles, s);
    default: return few_form<FB_CODES>(L, weight_tiles, s);
    }
}

}  // namespace nq
