// k_moe.hip -- the (token, choice) pairs of a router in the experts' order, rows in it, and rows back to their tokens.
//
// Pair i = t * top + c of token t; a pair whose expert is not in 0 .. experts - 1 is left out.
//   order[p]   the pair at sorted place p, -1 behind the last,
//   places[i]  the place of pair i, -1 where it is left out,
//   offsets[e] the first place of expert e; offsets[experts] is the number of places.
// The sort is stable: pairs of one expert keep their order.  It is a counting sort.  A wave takes a run of consecutive
// pairs; the pairs' places follow from the expert's offset, the pairs of earlier workgroups and waves, and the rank
// among the 64 of a step, which the lanes find by comparing their experts bit by bit.  No order of atomics matters:
// they only count.
//
// Up to 4096 pairs are one launch of one workgroup (40 pairs 2.6 us), where latency is all; more are two (131072 pairs of
// 256 experts 4.9 + 9.6 us, 16 M pairs 270 us): a workgroup reads the counts of all, which is cheaper than a third launch
// between them.  The rows' kernels are bound by the bytes they move: 16384 rows of 4 KB to 131072 places 106 us (5.7 TB/s),
// 65536 rows of 4 KB back to 8192 tokens 61 us (5.0 TB/s), their gradients 119 us (4.8 TB/s).
#include "nq_fp8b_codes.h"

namespace nq {

namespace {

constexpr int MOST_EXPERTS = 1024;
// Outputs of more bytes than this go past the L2s (eight of 4 MB).  8 choices of 64 experts, 2048 bfloat16 values, us past
// them / through them, by the outputs' MB: gather 32: 7.6 / 7.8, 64: 14.8 / 12.5, 128: 26.2 / 23.8, 256: 52 / 55, 512: 104 / 125;
// gradients 16: 11.3 / 12.4, 32: 15.0 / 20.8, 64: 29.7 / 27.6, 128: 58 / 54, 256: 114 / 120, 512: 230 / 236.  Between 64 and
// 128 MB the last cache would keep them for the next call (gather and combine of 64 MB 30.0 / 25.5, of 512 MB 240 / 272).
constexpr int64_t FAR_BYTES = 32 << 20;

__device__ __forceinline__ int32_t moe_id(const MoeSortLaunch &a, int64_t i) {
    if (a.wide) {
        const int64_t e = ((const int64_t *)a.ids)[i];
        return e >= 0 && e < a.experts ? (int32_t)e : -1;
    }
    const int32_t e = ((const int32_t *)a.ids)[i];
    return e >= 0 && e < a.experts ? e : -1;
}

__device__ __forceinline__ int32_t wave_scan(int32_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(v, d, 64);
        if (lane >= d) v += o;
    }
    return v;
}

}  // namespace

// Pairs of each expert in a chunk.
__global__ __launch_bounds__(1024) void k_moe_count(MoeSortLaunch a) {
    __shared__ int32_t count[MOST_EXPERTS];
    const int tid = threadIdx.x;
    for (int e = tid; e < a.experts; e += 1024) count[e] = 0;
    __syncthreads();
    const int64_t end = ((int64_t)blockIdx.x + 1) * a.chunk;
    for (int64_t i0 = end - a.chunk; i0 < end; i0 += MOE_CHUNK) {
#pragma unroll
        for (int k = 0; k < MOE_CHUNK / 1024; k++) {
            const int64_t i = i0 + k * 1024 + tid;
            const int32_t e = i < a.pairs ? moe_id(a, i) : -1;
            if (e >= 0) atomicAdd(&count[e], 1);
        }
    }
    __syncthreads();
    for (int e = tid; e < a.experts; e += 1024) a.counts[(int64_t)blockIdx.x * a.experts + e] = count[e];
}

// WAVES: waves of a workgroup; ONE: one workgroup has all pairs, and no counts are read.
template <int WAVES, bool ONE>
__global__ __launch_bounds__(64 * WAVES) void k_moe_place(MoeSortLaunch a) {
    extern __shared__ int32_t base[];  // [WAVES][experts]: first counts, then places
    __shared__ int32_t sums[WAVES + 1];
    constexpr int TB = 64 * WAVES;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = a.experts;
    for (int i = tid; i < WAVES * E; i += TB) base[i] = 0;
    const int64_t chunk0 = ONE ? 0 : (int64_t)blockIdx.x * a.chunk;
    const int64_t chunk = ONE ? a.pairs : (a.pairs - chunk0 < a.chunk ? a.pairs - chunk0 : a.chunk);
    const int64_t per = fb_ceil(fb_ceil(chunk, WAVES), 64) * 64;
    const int64_t i0 = chunk0 + wave * per, end = chunk0 + (wave * per + per < chunk ? wave * per + per : chunk);
    __syncthreads();
    for (int64_t i = i0 + lane; i < end; i += 64) {
        const int32_t e = moe_id(a, i);
        if (e >= 0) atomicAdd(&base[wave * E + e], 1);
    }
    __syncthreads();
    // a thread's expert: pairs before this workgroup's, and of all
    int32_t run = 0;
    for (int e0 = 0; e0 < E; e0 += TB) {
        const int e = e0 + tid;
        int32_t mine = 0, before = 0, all = 0;
        if (e < E) {
            for (int w = 0; w < WAVES; w++) mine += base[w * E + e];
            all = mine;
            if constexpr (!ONE) {
                all = 0;
                for (int c0 = 0; c0 < a.chunks; c0 += 16) {  // sixteen loads on their way (one at a time: 15.4 us for 32 chunks)
                    int32_t n[16];
#pragma unroll
                    for (int k = 0; k < 16; k++) n[k] = c0 + k < a.chunks ? a.counts[(int64_t)(c0 + k) * E + e] : 0;
#pragma unroll
                    for (int k = 0; k < 16; k++) {
                        before += c0 + k < (int)blockIdx.x ? n[k] : 0;
                        all += n[k];
                    }
                }
            }
        }
        const int32_t incl = wave_scan(all);
        if (lane == 63) sums[wave] = incl;
        __syncthreads();
        int32_t first = run + incl - all;
        for (int w = 0; w < WAVES; w++) {
            first += w < wave ? sums[w] : 0;
            run += sums[w];
        }
        if (e < E) {
            if (ONE || blockIdx.x == 0) a.offsets[e] = first;
            int32_t at = first + before;
            for (int w = 0; w < WAVES; w++) {
                const int32_t n = base[w * E + e];
                base[w * E + e] = at;
                at += n;
            }
        }
        __syncthreads();
    }
    if ((ONE || blockIdx.x == 0) && tid == 0) a.offsets[E] = run;
    for (int64_t p = run + (ONE ? 0 : (int64_t)blockIdx.x * TB) + tid; p < a.pairs; p += ONE ? TB : (int64_t)gridDim.x * TB) a.order[p] = -1;
    const int bits = 32 - __builtin_clz(E);  // experts and one more for those left out
    for (int64_t s = i0; s < end; s += 64) {
        const int64_t i = s + lane;
        const bool in = i < end;
        const int32_t id = in ? moe_id(a, i) : -1;
        const uint32_t key = id >= 0 ? (uint32_t)id : (uint32_t)E;
        uint64_t same = ~0ull;
        for (int b = 0; b < bits; b++) {
            const bool bit = key >> b & 1u;
            const uint64_t set = __ballot(bit);
            same &= bit ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int32_t at = -1;
        if (id >= 0) at = base[wave * E + id] + rank;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // every lane has its place before the first of them moves it on
        __builtin_amdgcn_wave_barrier();
        if (id >= 0 && rank == 0) base[wave * E + id] = at + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (id >= 0) a.order[at] = (int32_t)i;
        if (in) a.places[i] = at;
    }
}

// (the places of each wave and expert are at most 32 KB of LDS)
template <int WAVES, bool ONE>
static int place(const MoeSortLaunch &L, hipStream_t s) {
    hipLaunchKernelGGL((k_moe_place<WAVES, ONE>), dim3((uint32_t)L.chunks), dim3(64 * WAVES), (uint32_t)L.experts * WAVES * 4, s, L);
    return hipGetLastError() == hipSuccess ? 0 : 9;  // NQ_ERR_HIP
}

int launch_moe_sort(const MoeSortLaunch &L, hipStream_t s) {
    if (L.chunks > 1) {
        hipLaunchKernelGGL(k_moe_count, dim3((uint32_t)L.chunks), dim3(1024), 0, s, L);
        if (hipGetLastError() != hipSuccess) return 9;  // NQ_ERR_HIP
        return L.experts <= 512 ? place<16, false>(L, s) : place<8, false>(L, s);
    }
    if (L.pairs <= 512) return place<4, true>(L, s);
    return L.experts <= 512 ? place<16, true>(L, s) : place<8, true>(L, s);
}

// The kernels below have G threads a row: a workgroup, a wave or a quarter of one.  Narrow rows would leave most of a
// workgroup idle, wide ones of a wave's keep less on their way (9834 tokens x 6, bfloat16, combine and gradients, threads a
// row: 136 values 56 us with 256 and 24 with 16, 512 values 60 and 40 with 64, 1024 values 94 and 89; 8192 x 8, 2048 values
// 178 and 201), and few tokens would leave compute units idle.  The gradient alone with 16, 64 and 256 threads: 16384 x 8
// pairs, 64 values 13 / 28 / 86 us, 256 values 38 / 46 / 115, 512 values 69 / 59 / 135, 1024 values 129 / 114 / 167, 2048 values
// 285 / 247 / 230; 4096 x 8, 64 values 10 / 13 / 23, 512 values 41 / 22 / 35, 2048 values 159 / 70 / 58; 1024 x 8, 512 values 26 / 11 /
// 12, 1024 values 48 / 17 / 13.  (At 4096 x 8 of 256 values the rule's 16 take 17 us, 64 would 14.)

// Rows of bytes to the places of their token's pairs: a row is read once, whatever the number of its places.  Places
// behind the last get zeros.
// FAR: more bytes than the L2s hold, which go past them (268 MB 52 us, 64 us through them).
template <typename V, int G, bool FAR>
__global__ __launch_bounds__(256) void k_moe_gather(MoeRowsLaunch a) {
    const int64_t n = a.cols / (int64_t)sizeof(V), row0 = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G, rows = (int64_t)gridDim.x * (256 / G);
    const int lane = threadIdx.x % G;
    V *const out = (V *)a.out;
    for (int64_t t = row0; t < a.tokens; t += rows) {
        const V *const x = (const V *)((const uint8_t *)a.x + t * a.x_stride);
        for (int64_t c = lane; c < n; c += G) {
            const V v = x[c];
            for (int k = 0; k < a.top; k++) {
                const int32_t p = a.places[t * a.top + k];
                if (p < 0 || p >= a.pairs) continue;
                if constexpr (FAR)
                    __builtin_nontemporal_store(v, out + (int64_t)p * n + c);
                else
                    out[(int64_t)p * n + c] = v;
            }
        }
    }
    for (int64_t p = fb_clamp(a.offsets[a.experts], a.pairs) + row0; p < a.pairs; p += rows)
        for (int64_t c = lane; c < n; c += G) out[p * n + c] = V{};
}

template <int DT, int N>
__device__ __forceinline__ void moe_read(const void *x, int64_t i, float (&f)[N]) {
    if constexpr (N == 1)
        f[0] = kv_read<DT>(x, i);
    else
        fb_read8<DT>(x, i, f);
}

// FAR: more bytes than the L2s hold, which go past them.
template <int DT, int N, bool FAR = false>
__device__ __forceinline__ void moe_write(void *y, int64_t i, const float (&f)[N]) {
    if constexpr (N == 1) {
        fb_write1(y, i, f[0], DT);
    } else {
        kv_u4 w[DT == 0 ? 2 : 1];
        const float lo[4] = {f[0], f[1], f[2], f[3]}, hi[4] = {f[4], f[5], f[6], f[7]};
        kv_write4<DT>(w, 0, lo);
        kv_write4<DT>(w, 4, hi);
        kv_u4 *const to = (kv_u4 *)((uint8_t *)y + i * (DT == 0 ? 4 : 2));
#pragma unroll
        for (int k = 0; k < (DT == 0 ? 2 : 1); k++) {
            if constexpr (FAR)
                __builtin_nontemporal_store(w[k], to + k);
            else
                to[k] = w[k];
        }
    }
}

// out[t] = sum over choices of weight * row, in their order, in binary32.  N columns a thread and turn (four
// or eight rows on their way in each thread: no faster, and slower).
template <int DT, int N, int G>
__global__ __launch_bounds__(256) void k_moe_combine(MoeRowsLaunch a) {
    for (int64_t t = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G; t < a.tokens; t += (int64_t)gridDim.x * (256 / G)) {
        for (int64_t c = (int64_t)(threadIdx.x % G) * N; c < a.cols; c += G * N) {
            float sum[N];
#pragma unroll
            for (int i = 0; i < N; i++) sum[i] = 0.0f;
            for (int k = 0; k < a.top; k++) {
                const int32_t p = a.places[t * a.top + k];
                if (p < 0 || p >= a.pairs) continue;
                const float w = a.weights ? a.weights[t * a.top + k] : 1.0f;
                float f[N];
                moe_read<DT, N>(a.rows, (int64_t)p * a.rows_stride + c, f);
#pragma unroll
                for (int i = 0; i < N; i++) sum[i] = __builtin_fmaf(w, f[i], sum[i]);
            }
            moe_write<DT, N>(a.out, t * a.cols + c, sum);
        }
    }
}

// grad_rows[p] = weight * grad[token], grad_weights = <grad[token], rows[p]>; 0 behind the last place and where a pair
// is left out.
template <int DT, int N, int G, bool FAR>
__global__ __launch_bounds__(256) void k_moe_combine_grad(MoeRowsLaunch a) {
    __shared__ float part[4];
    const int lane = threadIdx.x % G;
    const int64_t row0 = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G, rows = (int64_t)gridDim.x * (256 / G);
    for (int64_t t = row0; t < a.tokens; t += rows) {
        for (int k = 0; k < a.top; k++) {
            const int32_t p = a.places[t * a.top + k];
            const bool live = p >= 0 && p < a.pairs;
            float dot = 0.0f;
            if (live) {
                const float w = a.weights ? a.weights[t * a.top + k] : 1.0f;
                for (int64_t c = (int64_t)lane * N; c < a.cols; c += G * N) {
                    float g[N], f[N];
                    moe_read<DT, N>(a.x, t * a.x_stride + c, g);
                    if (a.out_weights) {
                        moe_read<DT, N>(a.rows, (int64_t)p * a.rows_stride + c, f);
#pragma unroll
                        for (int i = 0; i < N; i++) dot = __builtin_fmaf(g[i], f[i], dot);
                    }
#pragma unroll
                    for (int i = 0; i < N; i++) g[i] *= w;
                    moe_write<DT, N, FAR>(a.out, (int64_t)p * a.cols + c, g);
                }
            }
            if (!a.out_weights) continue;
            for (int d = 1; d < (G < 64 ? G : 64); d <<= 1) dot += __shfl_xor(dot, d, 64);
            if constexpr (G > 64) {
                if ((lane & 63) == 0) part[lane >> 6] = dot;
                __syncthreads();
                dot = part[0] + part[1] + part[2] + part[3];
                __syncthreads();
            }
            if (lane == 0) a.out_weights[t * a.top + k] = live ? dot : 0.0f;
        }
    }
    float zero[N];
#pragma unroll
    for (int i = 0; i < N; i++) zero[i] = 0.0f;
    for (int64_t p = fb_clamp(a.offsets[a.experts], a.pairs) + row0; p < a.pairs; p += rows)
        for (int64_t c = (int64_t)lane * N; c < a.cols; c += G * N) moe_write<DT, N>(a.out, p * a.cols + c, zero);
}

// Threads of a row of `units` (what a thread takes at a time), and the grid.
static int row_threads(int64_t tokens, int64_t units) {
    const int64_t cus = device_compute_units();
    if (units <= 32 && tokens >= 16 * cus) return 16;
    return units <= 128 && tokens >= 4 * cus ? 64 : 256;
}
static dim3 row_grid(const MoeRowsLaunch &L, int threads) {
    const int64_t need = fb_ceil(L.tokens, 256 / threads), most = (int64_t)device_compute_units() * 16;
    return dim3((uint32_t)(need < most ? need : most));
}

template <typename V, bool FAR>
static int gather(const MoeRowsLaunch &L, hipStream_t s) {
    const int threads = row_threads(L.tokens, L.cols / (int64_t)sizeof(V));
    const dim3 grid = row_grid(L, threads);
    switch (threads) {
    case 16: hipLaunchKernelGGL((k_moe_gather<V, 16, FAR>), grid, dim3(256), 0, s, L); break;
    case 64: hipLaunchKernelGGL((k_moe_gather<V, 64, FAR>), grid, dim3(256), 0, s, L); break;
    default: hipLaunchKernelGGL((k_moe_gather<V, 256, FAR>), grid, dim3(256), 0, s, L); break;
    }
    return hipGetLastError() == hipSuccess ? 0 : 9;  // NQ_ERR_HIP
}

int launch_moe_gather(const MoeRowsLaunch &L, hipStream_t s) {
    if (L.tokens == 0 || L.cols == 0) return 0;
    const uintptr_t all = (uintptr_t)L.x | (uintptr_t)L.out | (uintptr_t)L.x_stride | (uintptr_t)L.cols;
    if (all % 16 == 0) return L.pairs * L.cols > FAR_BYTES ? gather<kv_u4, true>(L, s) : gather<kv_u4, false>(L, s);
    return all % 4 == 0 ? gather<uint32_t, false>(L, s) : gather<uint8_t, false>(L, s);
}

template <int DT, int N>
static int combine_wide(const MoeRowsLaunch &L, hipStream_t s) {
    const int threads = row_threads(L.tokens, L.cols / N);
    const dim3 grid = row_grid(L, threads);
    switch (threads) {
    case 16: hipLaunchKernelGGL((k_moe_combine<DT, N, 16>), grid, dim3(256), 0, s, L); break;
    case 64: hipLaunchKernelGGL((k_moe_combine<DT, N, 64>), grid, dim3(256), 0, s, L); break;
    default: hipLaunchKernelGGL((k_moe_combine<DT, N, 256>), grid, dim3(256), 0, s, L); break;
    }
    return hipGetLastError() == hipSuccess ? 0 : 9;  // NQ_ERR_HIP
}

template <int DT, int N, bool FAR>
static int grad_wide(const MoeRowsLaunch &L, hipStream_t s) {
    const int threads = row_threads(L.tokens, L.cols / N);
    const dim3 grid = row_grid(L, threads);
    switch (threads) {
    case 16: hipLaunchKernelGGL((k_moe_combine_grad<DT, N, 16, FAR>), grid, dim3(256), 0, s, L); break;
    case 64: hipLaunchKernelGGL((k_moe_combine_grad<DT, N, 64, FAR>), grid, dim3(256), 0, s, L); break;
    default: hipLaunchKernelGGL((k_moe_combine_grad<DT, N, 256, FAR>), grid, dim3(256), 0, s, L); break;
    }
    return hipGetLastError() == hipSuccess ? 0 : 9;  // NQ_ERR_HIP
}

template <int DT>
static int combine_in(const MoeRowsLaunch &L, hipStream_t s) {
    return L.vec ? combine_wide<DT, 8>(L, s) : combine_wide<DT, 1>(L, s);
}

template <int DT>
static int grad_in(const MoeRowsLaunch &L, hipStream_t s) {
    if (!L.vec) return grad_wide<DT, 1, false>(L, s);
    return L.pairs * L.cols * (DT == 0 ? 4 : 2) > FAR_BYTES ? grad_wide<DT, 8, true>(L, s) : grad_wide<DT, 8, false>(L, s);
}

int launch_moe_combine(const MoeRowsLaunch &L, hipStream_t s) {
    if (L.tokens == 0 || L.cols == 0) return 0;
    return L.dtype == 0 ? combine_in<0>(L, s) : L.dtype == 1 ? combine_in<1>(L, s) : combine_in<2>(L, s);
}

int launch_moe_combine_grad(const MoeRowsLaunch &L, hipStream_t s) {
    if (L.tokens == 0) return 0;
    return L.dtype == 0 ? grad_in<0>(L, s) : L.dtype == 1 ? grad_in<1>(L, s) : grad_in<2>(L, s);
}

}  // namespace nq
