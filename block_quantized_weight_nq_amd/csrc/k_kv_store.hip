// k_kv_store.hip -- new keys and values into their cache blocks, and whole blocks back as values.
//
// Store.  For a block and head whose new tokens start at offset `first` of the block:
//   s' = max(first > 0 ? s : 0, RN32(amax / qmax), 2^-126), amax over the finite new values,
//   a new code is code(RN32(x * RN32(1 / s'))) (NaN becomes 0, infinities saturate),
//   and where s' > s the codes before `first` become code(RN32(c * RN32(s / s'))).
// So a block that fills token by token keeps one scale, and its earlier codes
// are rounded again only when a new token is larger than all before it.
//
// One workgroup per block and head, for keys and values.  A thread takes
// tiles of four tokens by four channels: a dword of four codes is then a
// token's four channels (keys) or a channel's four tokens (values) without a
// transpose.  Its first one or two tiles of each stay in registers between the search for
// amax and the writing, later ones (blocks of more than 8192 values) are read
// again.  What bounds it: the bytes of the new values for prompts, and the
// chain of dependent loads (starts, slot, values) for single tokens.
#include "nq_kv_codes.h"

#include <type_traits>

namespace nq {

namespace {

constexpr int TB = 256;

template <int CODE>
constexpr float qmax() {
    return CODE == KV_Q8 ? 127.0f : 448.0f;
}

// The larger of the magnitudes of four values and m, as words: integers in the
// same order, infinities and NaN (0x7F800000 and up) above all finite ones.
__device__ __forceinline__ uint32_t amax4(const float (&f)[4], uint32_t m) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t x = __builtin_bit_cast(uint32_t, f[i]) & 0x7FFFFFFFu;
        m = x > m ? x : m;
    }
    return m;
}

// The same over the finite ones.
__device__ __forceinline__ uint32_t amax4_finite(const float (&f)[4], uint32_t m) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t x = __builtin_bit_cast(uint32_t, f[i]) & 0x7FFFFFFFu;
        m = x > m && x < 0x7F800000u ? x : m;
    }
    return m;
}

template <int CODE>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    float f[4];
    kv_codes4_f32<CODE>(w, f);
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = f[i] * ratio;
    return kv_f32_codes4<CODE>(f);
}

}  // namespace

__global__ void k_kv_clear_status(uint32_t *status) { *status = 0u; }

// HOLD: tiles of each kind that a thread keeps, 1 for blocks of up to 4096 values (fewer registers, more workgroups at
// a time).  MANY: more than TB requests, which are searched (with the search in it, 30.6 us instead of 29.8 for 16000
// tokens of 6 requests).
template <int CODE, int IN, bool VEC, int HOLD, bool MANY>
__global__ __launch_bounds__(TB) void k_kv_store(KvStoreLaunch a) {
    __shared__ uint32_t wmax[2][TB / 64];
    __shared__ int32_t found[3];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t head = blockIdx.y;
    const int64_t u = blockIdx.x, T = (int64_t)1 << a.c.bsh, n = a.tokens;
    const int bsh = (int)a.c.bsh, q4 = (int)a.c.dim / 4, qsh = __builtin_ctz(q4);  // dim is a power of two

    // the request of this unit, among TB of them at the end
    if (tid == 0) found[0] = -1;
    int32_t from = 0, left = a.requests;
    if constexpr (MANY) {
        while (left > TB) {
            const int32_t step = kv_probe_step(left, TB), i = from + tid * step;
            const int hits = __syncthreads_count(tid * step < left && kv_unit_first(a.starts[i], i, a.c.bsh) <= u);
            if (hits == 0) return;
            kv_narrow(&from, &left, step, hits);
        }
    }
    __syncthreads();
    if (tid < left) {
        const int i = from + tid;
        const int32_t s0 = a.starts[i], s1 = a.starts[i + 1];
        if (kv_unit_first(s0, i, a.c.bsh) <= u && u < kv_unit_first(s1, i + 1, a.c.bsh)) {
            found[0] = i;
            found[1] = s0;
            found[2] = s1;
        }
    }
    __syncthreads();
    const int r = found[0];
    if (r < 0) return;
    int64_t s0 = found[1], s1 = found[2];
    const int64_t j = u - kv_unit_first(s0, r, a.c.bsh);
    if (s1 > n) s1 = n;
    if (s0 < 0 || s0 >= s1) return;
    const int64_t slot0 = a.slots[s0];
    const int64_t pool = a.c.blocks << bsh;
    int64_t lo, hi;
    kv_unit_tokens(s0, s1, j, slot0 & (T - 1), a.c.bsh, &lo, &hi);
    if (lo >= hi) return;
    // the values are on their way while the slots are checked
    const int cnt = (int)(hi - lo), first = lo > s0 ? 0 : (int)(slot0 & (T - 1)), last = first + cnt;
    const int g0 = first / 4, ng = (last + 3) / 4 - g0, tiles = ng << qsh;
    const auto place = [&](int kind, int i, int *g, int *c4) {  // lanes run along what the codes are contiguous in
        *g = g0 + (kind == 0 ? i >> qsh : i % ng);
        *c4 = kind == 0 ? i & (q4 - 1) : i / ng;
    };
    const auto read = [&](int kind, int g, int c4, float (&f)[4][4]) {  // [token][channel], 0 where there is no new token
        const int64_t x0 = (lo - first) * a.ts[kind] + head * a.hs[kind];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int tok = 4 * g + k;
            f[k][0] = f[k][1] = f[k][2] = f[k][3] = 0.0f;
            if (tok >= first && tok < last) kv_read4<IN, VEC>(a.x[kind], x0 + (int64_t)tok * a.ts[kind] + 4 * c4, f[k]);
        }
    };
    float held[2][HOLD][4][4];
    uint32_t amax[2];
#pragma unroll
    for (int kind = 0; kind < 2; kind++)
#pragma unroll
        for (int m = 0; m < HOLD; m++) {
            int g, c4;
            place(kind, tid + m * TB < tiles ? tid + m * TB : 0, &g, &c4);
            if (tid + m * TB < tiles) read(kind, g, c4, held[kind][m]);
        }
    const int64_t slot = a.slots[lo];
    bool wrong = slot < 0 || slot >= pool || (slot & (T - 1)) != first;
    if (tid < cnt) wrong |= a.slots[lo + tid] != slot + tid;
    if (__syncthreads_or(wrong)) {
        if (tid == 0 && head == 0) atomicOr(a.status, KV_ST_BAD_SLOT);
        return;
    }
    const int64_t block = slot >> bsh, tile = kv_tile_at(a.c, block, head), sat = block * a.c.heads + head;
    const float old[2] = {first > 0 ? a.c.ks[sat] : 0.0f, first > 0 ? a.c.vs[sat] : 0.0f};
    const auto largest = [&](bool finite) {
#pragma unroll
        for (int kind = 0; kind < 2; kind++) {
            uint32_t top = 0;
#pragma unroll
            for (int m = 0; m < HOLD; m++)
                if (tid + m * TB < tiles)
#pragma unroll
                    for (int k = 0; k < 4; k++) top = finite ? amax4_finite(held[kind][m][k], top) : amax4(held[kind][m][k], top);
            for (int i = tid + HOLD * TB; i < tiles; i += TB) {
                int g, c4;
                float f[4][4];
                place(kind, i, &g, &c4);
                read(kind, g, c4, f);
#pragma unroll
                for (int k = 0; k < 4; k++) top = finite ? amax4_finite(f[k], top) : amax4(f[k], top);
            }
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t other = __shfl_xor(top, d, 64);
                top = other > top ? other : top;
            }
            if (lane == 0) wmax[kind][wave] = top;
        }
        __syncthreads();
        uint32_t all[2] = {0, 0};
#pragma unroll
        for (int kind = 0; kind < 2; kind++)
            for (int w = 0; w < TB / 64; w++) all[kind] = wmax[kind][w] > all[kind] ? wmax[kind][w] : all[kind];
        amax[0] = all[0], amax[1] = all[1];
    };
    largest(false);
    const bool bad = amax[0] >= 0x7F800000u || amax[1] >= 0x7F800000u;
    if (bad) {
        if (tid == 0) atomicOr(a.status, KV_ST_NOT_FINITE);
        __syncthreads();
        largest(true);
    }
#pragma unroll
    for (int kind = 0; kind < 2; kind++) {
        const float top = __builtin_bit_cast(float, amax[kind]);
        const float now = fmaxf(fmaxf(old[kind], top / qmax<CODE>()), KV_TINY);
        const float inv = 1.0f / now, ratio = old[kind] / now;
        const bool grow = first > 0 && now > old[kind];
        if (tid == 0) (kind ? a.c.vs : a.c.ks)[sat] = now;  // every thread has the old one: they have passed a barrier since
        uint8_t *const codes = (kind ? a.c.v : a.c.k) + tile;
        const auto write = [&](int g, int c4, const float (&f)[4][4]) {
            uint32_t is_new = 0;  // bytes of a dword of four tokens
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (4 * g + k >= first && 4 * g + k < last) is_new |= 0xFFu << (8 * k);
#pragma unroll
            for (int k = 0; k < 4; k++) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; e++) y[e] = (kind == 0 ? f[k][e] : f[e][k]) * inv;
                uint32_t w = bad ? kv_f32_codes4<CODE>(y) : kv_f32_codes4<CODE, true>(y);
                if (kind == 0) {
                    if (is_new >> (8 * k) & 1u) ((uint32_t *)codes)[((4 * g + k) << qsh) + c4] = w;
                } else {
                    uint32_t *at = (uint32_t *)(codes + ((4 * c4 + k) << bsh) + 4 * g);
                    if (is_new != 0xFFFFFFFFu) {
                        const uint32_t was = *at;
                        uint32_t is_old = 0;
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (4 * g + e < first) is_old |= 0xFFu << (8 * e);
                        const uint32_t kept = grow && is_old ? (rescale4<CODE>(was, ratio) & is_old) | (was & ~is_old) : was;
                        w = (w & is_new) | (kept & ~is_new);
                    }
                    *at = w;
                }
            }
        };
#pragma unroll
        for (int m = 0; m < HOLD; m++) {
            int g, c4;
            place(kind, tid + m * TB < tiles ? tid + m * TB : 0, &g, &c4);
            if (tid + m * TB < tiles) write(g, c4, held[kind][m]);
        }
        for (int i = tid + HOLD * TB; i < tiles; i += TB) {
            int g, c4;
            float f[4][4];
            place(kind, i, &g, &c4);
            read(kind, g, c4, f);
            write(g, c4, f);
        }
        if (!grow) continue;
        // codes before the first new token, four a dword; a dword of values that has a new token is done
        const int old_dw = kind == 0 ? first << qsh : g0 << (qsh + 2);
        for (int i = tid; i < old_dw; i += TB) {
            uint32_t *w = (uint32_t *)codes + (kind == 0 ? i : (i / g0 << bsh) / 4 + i % g0);
            *w = rescale4<CODE>(*w, ratio);
        }
    }
}

template <int CODE, int IN>
static int store_in(const KvStoreLaunch &L, hipStream_t s) {
    hipLaunchKernelGGL(k_kv_clear_status, dim3(1), dim3(1), 0, s, L.status);
    if (hipGetLastError() != hipSuccess) return 9;  // NQ_ERR_HIP
    const uint64_t units = (uint64_t)kv_unit_first(L.tokens, L.requests, L.c.bsh);
    if (L.tokens == 0 || units == 0) return 0;
    constexpr int64_t ESZ = IN == 0 ? 4 : 2;
    bool vec = true;
    for (int i = 0; i < 2; i++)
        vec &= (uintptr_t)L.x[i] % (4 * ESZ) == 0 && L.ts[i] % 4 == 0 && L.hs[i] % 4 == 0;
    const dim3 grid((uint32_t)units, L.c.heads);
    const bool one = (L.c.dim << L.c.bsh) <= 16 * TB;
    const auto launch = [&](auto many) {
        if (vec && one)
            hipLaunchKernelGGL((k_kv_store<CODE, IN, true, 1, many()>), grid, dim3(TB), 0, s, L);
        else if (vec)
            hipLaunchKernelGGL((k_kv_store<CODE, IN, true, 2, many()>), grid, dim3(TB), 0, s, L);
        else
            hipLaunchKernelGGL((k_kv_store<CODE, IN, false, 2, many()>), grid, dim3(TB), 0, s, L);
    };
    if (L.requests > TB)
        launch(std::true_type());
    else
        launch(std::false_type());
    return hipGetLastError() == hipSuccess ? 0 : 9;  // NQ_ERR_HIP
}

int launch_kv_store(const KvStoreLaunch &L, hipStream_t s) {
    switch (L.code * 3 + L.in_dtype) {
    case 0: return store_in<KV_Q8, 0>(L, s);
    case 1: return store_in<KV_Q8, 1>(L, s);
    case 2: return store_in<KV_Q8, 2>(L, s);
    case 3: return store_in<KV_E4M3, 0>(L, s);
    case 4: return store_in<KV_E4M3, 1>(L, s);
    default: return store_in<KV_E4M3, 2>(L, s);
    }
}

// Load: the values RN32(c * scale) of whole blocks, [n, T, heads, D] for keys
// and for values.  A block that is not in the pool gives zeros.  A workgroup
// takes a block's kind and several heads, about 16 KB of codes; a thread writes
// eight channels (16 bytes of a 16-bit type), and value blocks turn through LDS.
template <int CODE, int OT>
__global__ __launch_bounds__(TB) void k_kv_load(KvLoadLaunch a) {
    extern __shared__ uint32_t tile[];  // [heads * D][T / 4 + 1], an odd stride in dwords
    const int tid = threadIdx.x;
    const uint32_t kind = blockIdx.z;
    const int D = (int)a.c.dim, T = 1 << a.c.bsh, q8 = D / 8;
    const int h0 = (int)blockIdx.y * a.group, nh = h0 + a.group < (int)a.c.heads ? a.group : (int)a.c.heads - h0;
    const int64_t b = blockIdx.x;
    const int64_t block = a.ids[b];
    const bool live = block >= 0 && block < a.c.blocks;
    const uint32_t *codes = (const uint32_t *)((kind ? a.c.v : a.c.k) + kv_tile_at(a.c, live ? block : 0, h0));
    const float *scales = (kind ? a.c.vs : a.c.ks) + (live ? block : 0) * a.c.heads + h0;
    const int64_t row = (int64_t)a.c.heads * D, y0 = b * T * row + (int64_t)h0 * D;
    void *y = a.out[kind];
    const int per = nh * q8;  // eights of channels of a token
    if (kind == 0) {
        for (int i = tid; i < T * per; i += TB) {
            const int t = i / per, c = i % per, h = c / q8;
            const float s = live ? scales[h] : 0.0f;
            const kv_u2 w = *(const kv_u2 *)(codes + (int64_t)(h * T + t) * (D / 4) + 2 * (c % q8));
#pragma unroll
            for (int e = 0; e < 2; e++) {
                float f[4];
                kv_codes4_f32<CODE>(live ? w[e] : 0u, f);
#pragma unroll
                for (int k = 0; k < 4; k++) f[k] = f[k] * s;
                kv_write4<OT>(y, y0 + t * row + 8 * c + 4 * e, f);
            }
        }
        return;
    }
    const int tq = T / 4, stride = tq + 1, all = nh * D * tq;
    for (int i = 4 * tid; i < all; i += 4 * TB) {  // T is at least 16: four dwords of one channel
        const kv_u4 w = *(const kv_u4 *)(codes + i);
#pragma unroll
        for (int k = 0; k < 4; k++) tile[i / tq * stride + i % tq + k] = live ? w[k] : 0u;
    }
    __syncthreads();
    for (int i = tid; i < tq * per; i += TB) {
        const int c = i % per, g = i / per;
        const float s = live ? scales[c / q8] : 0.0f;
        float f[8][4];  // [channel][token]
#pragma unroll
        for (int ch = 0; ch < 8; ch++) kv_codes4_f32<CODE>(tile[(8 * c + ch) * stride + g], f[ch]);
#pragma unroll
        for (int k = 0; k < 4; k++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                float o[4];
#pragma unroll
                for (int ch = 0; ch < 4; ch++) o[ch] = f[4 * e + ch][k] * s;
                kv_write4<OT>(y, y0 + (4 * g + k) * row + 8 * c + 4 * e, o);
            }
    }
}

template <int CODE>
static int load_code(KvLoadLaunch L, hipStream_t s) {
    // heads of a workgroup: 16 KB of codes, fewer where the blocks are too few for that (1024 workgroups)
    const int64_t one = (int64_t)L.c.dim << L.c.bsh;
    L.group = (int32_t)(one >= 16384 ? 1 : 16384 / one);
    if (L.group > (int32_t)L.c.heads) L.group = (int32_t)L.c.heads;
    while (L.group > 1 && 2 * L.n * ((L.c.heads + L.group - 1) / L.group) < 1024) L.group = (L.group + 1) / 2;
    const dim3 grid((uint32_t)L.n, (L.c.heads + L.group - 1) / L.group, 2);
    const uint32_t lds = (uint32_t)L.group * L.c.dim * ((1u << L.c.bsh) / 4 + 1) * 4;
    switch (L.out_dtype) {
    case 0: hipLaunchKernelGGL((k_kv_load<CODE, 0>), grid, dim3(TB), lds, s, L); break;
    case 1: hipLaunchKernelGGL((k_kv_load<CODE, 1>), grid, dim3(TB), lds, s, L); break;
    default: hipLaunchKernelGGL((k_kv_load<CODE, 2>), grid, dim3(TB), lds, s, L); break;
    }
    return hipGetLastError() == hipSuccess ? 0 : 9;  // NQ_ERR_HIP
}

int launch_kv_load(const KvLoadLaunch &L, hipStream_t s) {
    if (L.n == 0) return 0;
    return L.code == KV_Q8 ? load_code<KV_Q8>(L, s) : load_code<KV_E4M3>(L, s);
}

}  // namespace nq
