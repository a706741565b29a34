// k_kv_store.hip -- new keys and values into their cache blocks, and whole blocks back as values.
//
// Store.  For a block and head whose new tokens start at offset `first` of the block:
//   s' = max(first > 0 ? s : 0, RN32(amax / qmax), 2^-126), amax over the finite new values,
//   a new code is code(RN32(x * RN32(1 / s'))) (NaN becomes 0, infinities saturate),
//   and where s' > s the codes before `first` become code(RN32(c * RN32(s / s'))).
// So a block that fills token by token keeps one scale, and its earlier codes
// are rounded again only when a new token is larger than all before it.
//
// One workgroup per block, head and kind (keys or values); it reads its new
// values twice (the second time from the cache: at most 64 KB in 16 bits).
// The first pass finds amax, the second writes.  What bounds it is the
// bytes of the new values for prompts, and latency for single tokens.
#include "nq_kv_codes.h"

namespace nq {

namespace {

constexpr int TB = 256;

template <int CODE>
constexpr float qmax() {
    return CODE == KV_Q8 ? 127.0f : 448.0f;
}

// Largest magnitude among the finite ones of four values; *bad if one is not finite.
__device__ __forceinline__ float amax4(const float (&f)[4], bool *bad) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float x = fabsf(f[i]);
        const bool fin = x < __builtin_inff();
        *bad |= !fin;
        m = fmaxf(m, fin ? x : 0.0f);
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

template <int CODE, int IN, bool VEC>
__global__ __launch_bounds__(TB) void k_kv_store(KvStoreLaunch a) {
    __shared__ float wmax[TB / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t head = blockIdx.y, kind = blockIdx.z;
    const int64_t u = blockIdx.x, T = (int64_t)1 << a.c.bsh, n = a.tokens;
    const int D = (int)a.c.dim, bsh = (int)a.c.bsh;

    // the request of this unit: the last one whose first unit is not past u
    int r = -1;
    for (int b = 0; b < a.requests; b += TB) {
        const int i = b + tid;
        r += __syncthreads_count(i < a.requests && kv_unit_first(a.starts[i], i, a.c.bsh) <= u);
    }
    if (r < 0) return;
    int64_t s0 = a.starts[r], s1 = a.starts[r + 1];
    const int64_t j = u - kv_unit_first(s0, r, a.c.bsh);
    if (s1 > n) s1 = n;
    if (s0 < 0 || s0 >= s1) return;
    const int64_t slot0 = a.slots[s0];
    const int64_t pool = a.c.blocks << bsh;
    int64_t lo, hi;
    kv_unit_tokens(s0, s1, j, slot0 & (T - 1), a.c.bsh, &lo, &hi);
    if (lo >= hi) return;
    const int64_t slot = a.slots[lo];
    bool wrong = slot < 0 || slot >= pool || (lo > s0 && (slot & (T - 1)) != 0);
    const int cnt = (int)(hi - lo), first = (int)(slot & (T - 1));
    if (tid < cnt) wrong |= a.slots[lo + tid] != slot + tid;
    if (__syncthreads_or(wrong || first + cnt > (int)T)) {
        if (tid == 0) atomicOr(a.status, KV_ST_BAD_SLOT);
        return;
    }
    const int64_t block = slot >> bsh;
    uint8_t *codes = (kind ? a.c.v : a.c.k) + kv_tile_at(a.c, block, head);
    float *scale = (kind ? a.c.vs : a.c.ks) + block * a.c.heads + head;
    const void *x = a.x[kind];
    const int64_t ts = a.ts[kind], x0 = lo * ts + head * a.hs[kind];

    const int q4 = D / 4, items = cnt * q4;  // four channels of one token
    float amax = 0.0f;
    bool bad = false;
    for (int i = tid; i < items; i += TB) {
        float f[4];
        kv_read4<IN, VEC>(x, x0 + (int64_t)(i / q4) * ts + 4 * (i % q4), f);
        amax = fmaxf(amax, amax4(f, &bad));
    }
    for (int d = 1; d < 64; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d, 64));
    if (lane == 0) wmax[wave] = amax;
    if (__syncthreads_or(bad) && tid == 0) atomicOr(a.status, KV_ST_NOT_FINITE);
    for (int w = 0; w < TB / 64; w++) amax = fmaxf(amax, wmax[w]);
    const float old = first > 0 ? *scale : 0.0f;
    const float now = fmaxf(fmaxf(old, amax / qmax<CODE>()), KV_TINY);
    const float inv = 1.0f / now, ratio = old / now;
    const bool grow = first > 0 && now > old;
    __syncthreads();  // every thread has the old scale
    if (tid == 0) *scale = now;

    if (kind == 0) {
        uint32_t *row = (uint32_t *)codes + first * q4;
        for (int i = tid; i < items; i += TB) {
            float f[4];
            kv_read4<IN, VEC>(x, x0 + (int64_t)(i / q4) * ts + 4 * (i % q4), f);
#pragma unroll
            for (int k = 0; k < 4; k++) f[k] = (f[k] == f[k] ? f[k] : 0.0f) * inv;
            row[i] = kv_f32_codes4<CODE>(f);
        }
        if (grow)
            for (int i = tid; i < first * q4; i += TB) {
                uint32_t *w = (uint32_t *)codes + i;
                *w = rescale4<CODE>(*w, ratio);
            }
        return;
    }
    // Values: four channels of four tokens a thread, a dword of four tokens per channel.
    const int last = first + cnt;
    const int g0 = grow ? 0 : first / 4, g1 = (last + 3) / 4, ng = g1 - g0;
    for (int i = tid; i < ng * q4; i += TB) {
        const int g = g0 + i % ng, c4 = i / ng, t0 = 4 * g;
        float f[4][4];  // [token][channel]
#pragma unroll
        for (int k = 0; k < 4; k++) {
            if (t0 + k >= first && t0 + k < last)
                kv_read4<IN, VEC>(x, x0 + (int64_t)(t0 + k - first) * ts + 4 * c4, f[k]);
            else
                f[k][0] = f[k][1] = f[k][2] = f[k][3] = 0.0f;
        }
        uint32_t is_new = 0, is_old = 0;  // byte masks
#pragma unroll
        for (int k = 0; k < 4; k++) {
            if (t0 + k >= first && t0 + k < last) is_new |= 0xFFu << (8 * k);
            if (t0 + k < first) is_old |= 0xFFu << (8 * k);
        }
#pragma unroll
        for (int ch = 0; ch < 4; ch++) {
            uint32_t *w = (uint32_t *)(codes + ((4 * c4 + ch) << bsh) + t0);
            float g4[4];
#pragma unroll
            for (int k = 0; k < 4; k++) g4[k] = (f[k][ch] == f[k][ch] ? f[k][ch] : 0.0f) * inv;
            uint32_t res = kv_f32_codes4<CODE>(g4);
            if (is_new != 0xFFFFFFFFu) {
                const uint32_t was = *w;
                const uint32_t kept = grow && is_old ? (rescale4<CODE>(was, ratio) & is_old) | (was & ~is_old) : was;
                res = (res & is_new) | (kept & ~is_new);
            }
            *w = res;
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
    const dim3 grid((uint32_t)units, L.c.heads, 2);
    if (vec)
        hipLaunchKernelGGL((k_kv_store<CODE, IN, true>), grid, dim3(TB), 0, s, L);
    else
        hipLaunchKernelGGL((k_kv_store<CODE, IN, false>), grid, dim3(TB), 0, s, L);
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
// and for values.  A block that is not in the pool gives zeros.  One
// workgroup per block, head and kind; value blocks turn through LDS.
template <int CODE, int OT>
__global__ __launch_bounds__(TB) void k_kv_load(KvLoadLaunch a) {
    extern __shared__ uint32_t tile[];  // [D][T / 4 + 1], an odd stride in dwords
    const int tid = threadIdx.x;
    const uint32_t head = blockIdx.y, kind = blockIdx.z;
    const int D = (int)a.c.dim, T = 1 << a.c.bsh, q4 = D / 4;
    const int64_t b = blockIdx.x;
    const int64_t block = a.ids[b];
    const bool live = block >= 0 && block < a.c.blocks;
    const uint32_t *codes = (const uint32_t *)((kind ? a.c.v : a.c.k) + kv_tile_at(a.c, live ? block : 0, head));
    const float scale = live ? (kind ? a.c.vs : a.c.ks)[block * a.c.heads + head] : 0.0f;
    const int64_t row = (int64_t)a.c.heads * D;
    const int64_t y0 = b * T * row + (int64_t)head * D;
    void *y = a.out[kind];
    if (kind == 0) {
        for (int i = tid; i < T * q4; i += TB) {
            float f[4];
            kv_codes4_f32<CODE>(live ? codes[i] : 0u, f);
#pragma unroll
            for (int k = 0; k < 4; k++) f[k] = f[k] * scale;
            kv_write4<OT>(y, y0 + (i / q4) * row + 4 * (i % q4), f);
        }
        return;
    }
    const int tq = T / 4, stride = tq + 1;
    for (int i = tid; i < D * tq; i += TB) tile[(i / tq) * stride + i % tq] = live ? codes[i] : 0u;
    __syncthreads();
    for (int i = tid; i < tq * q4; i += TB) {
        const int c4 = i % q4, g = i / q4;
        float f[4][4];  // [channel][token]
#pragma unroll
        for (int ch = 0; ch < 4; ch++) kv_codes4_f32<CODE>(tile[(4 * c4 + ch) * stride + g], f[ch]);
#pragma unroll
        for (int k = 0; k < 4; k++) {
            float o[4];
#pragma unroll
            for (int ch = 0; ch < 4; ch++) o[ch] = f[ch][k] * scale;
            kv_write4<OT>(y, y0 + (4 * g + k) * row + 4 * c4, o);
        }
    }
}

template <int CODE>
static int load_code(const KvLoadLaunch &L, hipStream_t s) {
    const dim3 grid((uint32_t)L.n, L.c.heads, 2);
    const uint32_t lds = L.c.dim * ((1u << L.c.bsh) / 4 + 1) * 4;
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
