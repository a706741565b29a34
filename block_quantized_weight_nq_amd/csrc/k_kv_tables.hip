// k_kv_tables.hip -- block tables, slot map and token starts of one serving step.
//
// For request r with length len[r] and added[r] = n: n >= 0 new tokens, or -1
// when it ends.  held = ceil(len / T) blocks are in its table row, need =
// ceil((len + n) / T) - held more come from the ring of free blocks, in
// request order from its head, and the blocks of the ended requests go back
// to its tail, in request order.  Token i of request r gets slot block * T +
// offset of position len + i.
//
// One launch.  What the requests need are sums over all of them before r, and
// every workgroup forms all of these itself (a scan over the lengths: 1000
// requests are 8 KB that the L2 holds), so no workgroup waits for another:
// workgroup w fills the slots of 1024 tokens and moves the blocks of requests
// w, w + G, ...  A token's new block is read where the ring has it, not from
// the table that another workgroup is writing.  Only where the returned
// blocks would land on ring entries that this step takes (a ring shorter than
// the pool) does workgroup 0 do everything, in order.
#include "nq_kv.h"

namespace nq {

namespace {

constexpr int TOK = 1024;        // tokens a workgroup's slots cover at a time
constexpr uint32_t MAX_WG = 1024;  // workgroups of a launch

struct Sums {
    int64_t add, need, give;
};

struct Req {
    int64_t len, add, held, need, give;
    bool bad, ends;
};

__device__ __forceinline__ Req request(const KvTablesLaunch &a, int r) {
    Req q;
    q.len = a.lengths[r];
    const int64_t n = a.added[r];
    const int64_t T1 = ((int64_t)1 << a.bsh) - 1;
    q.add = n > 0 ? n : 0;
    q.held = (q.len + T1) >> a.bsh;
    q.need = ((q.len + q.add + T1) >> a.bsh) - q.held;
    q.give = n < 0 ? q.held : 0;
    q.ends = n < 0;
    q.bad = q.len < 0 || n < -1 || q.len + q.add > ((int64_t)a.width << a.bsh);
    return q;
}

__device__ __forceinline__ int64_t up64(int64_t v, int d) { return __shfl_up(v, d, 64); }

}  // namespace

// TB threads, each with its own requests: 256, or 1024 for more than 256 requests.
template <int TB>
__global__ __launch_bounds__(TB) void k_kv_tables(KvTablesLaunch a) {
    __shared__ Sums wsum[TB / 64];
    __shared__ int32_t any_bad, queued;
    __shared__ int32_t m_req[TB], m_held[TB], m_count[TB], m_first[TB];
    __shared__ int32_t owner[TOK], o_req[TOK], o_start[TOK], o_took[TOK], o_len[TOK];
    __shared__ int32_t wtop[TB / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int R = a.requests, per = (R + TB - 1) / TB;
    const int r0 = tid * per < R ? tid * per : R, r1 = r0 + per < R ? r0 + per : R;
    const int64_t head = a.state[0], count = a.state[1], ring = a.ring_size;  // on its way with the lengths
    if (tid == 0) any_bad = 0;
    const Req none = {0, 0, 0, 0, 0, false, false}, own = r0 < r1 ? request(a, r0) : none;  // read once: all of up to TB requests
    const auto req = [&](int r) { return r == r0 ? own : request(a, r); };
    __syncthreads();

    // sums over this thread's requests, then over those of the threads before it
    Sums mine = {0, 0, 0};
    bool bad = false;
    for (int r = r0; r < r1; r++) {
        const Req q = req(r);
        mine.add += q.add;
        mine.need += q.need;
        mine.give += q.give;
        bad |= q.bad;
    }
    if (bad) any_bad = 1;
    Sums inc = mine;
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t x = up64(inc.add, d), y = up64(inc.need, d), z = up64(inc.give, d);
        if (lane >= d) {
            inc.add += x;
            inc.need += y;
            inc.give += z;
        }
    }
    if (lane == 63) wsum[wave] = inc;
    __syncthreads();
    Sums before = {inc.add - mine.add, inc.need - mine.need, inc.give - mine.give}, all = {0, 0, 0};
    for (int w = 0; w < TB / 64; w++) {
        if (w < wave) {
            before.add += wsum[w].add;
            before.need += wsum[w].need;
            before.give += wsum[w].give;
        }
        all.add += wsum[w].add;
        all.need += wsum[w].need;
        all.give += wsum[w].give;
    }
    const bool no_ring = count < 0 || count > ring || head < 0 || head >= ring || count - all.need + all.give > ring;
    const uint32_t status = (all.need > count ? KV_ST_NO_BLOCKS : 0u) | (any_bad ? KV_ST_BAD_LENGTH : 0u) |
                            (all.add > a.tokens ? KV_ST_TOKENS : 0u) | (no_ring ? KV_ST_RING : 0u);
    const bool ok = status == 0;
    const bool solo = ok && count + all.give > ring;
    if (blockIdx.x == 0) {
        int64_t s = before.add;
        for (int r = r0; r < r1; r++) {
            const Req q = req(r);
            a.starts[r] = ok ? (int32_t)s : 0;
            a.lengths_out[r] = (int32_t)(!ok ? q.len : q.ends ? 0 : q.len + q.add);
            s += q.add;
        }
        if (tid == 0) {
            a.starts[R] = ok ? (int32_t)all.add : 0;
            a.state_out[0] = (int32_t)(ok ? (head + all.need) % ring : head);
            a.state_out[1] = (int32_t)(ok ? count - all.need + all.give : count);
            *a.status = status;
        }
    }
    if (!ok) {
        for (int64_t i = (int64_t)blockIdx.x * TB + tid; i < a.tokens; i += (int64_t)gridDim.x * TB) a.slots[i] = -1;
        return;
    }
    if (solo && blockIdx.x != 0) return;
    const uint32_t G = solo ? 1u : gridDim.x;

    // 32-bit ring arithmetic: ring <= 2^30, first + j < count <= ring going in and < ring coming back.
    const int64_t tail = (head + count) % ring;
    // Blocks in (pass 0) and out (pass 1).  The workgroup's requests that have any queue up in LDS, one a thread at a
    // time, and each wave moves the blocks of some.
    auto move = [&](int pass) {
        int64_t at = pass == 0 ? before.need : before.give;
        for (int k = 0; k < per; k++) {
            if (tid == 0) queued = 0;
            __syncthreads();
            const int r = r0 + k;
            if (r < r1) {
                const Req q = req(r);
                const int64_t n = pass == 0 ? q.need : q.give;
                if (n > 0 && (uint32_t)r % G == blockIdx.x) {
                    const int i = atomicAdd(&queued, 1);
                    m_req[i] = r;
                    m_held[i] = (int32_t)q.held;
                    m_count[i] = (int32_t)n;
                    m_first[i] = (int32_t)at;
                }
                at += n;
            }
            __syncthreads();
            for (int i = wave; i < queued; i += TB / 64) {
                int32_t *row = a.table + (int64_t)m_req[i] * a.table_stride;
                const int held = m_held[i], n = m_count[i], first = m_first[i];
                for (int j0 = lane; j0 < n; j0 += 512) {  // eight blocks a lane on their way
                    int32_t id[8];
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int j = j0 + 64 * e < n ? j0 + 64 * e : j0;
                        id[e] = pass == 0 ? a.ring[(uint32_t)(head + first + j) % (uint32_t)ring] : row[j];
                    }
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int j = j0 + 64 * e;
                        if (j >= n) break;
                        if (pass == 0)
                            row[held + j] = id[e];
                        else
                            a.ring[(uint32_t)(tail + first + j) % (uint32_t)ring] = id[e];
                    }
                }
            }
            __syncthreads();
        }
    };
    move(0);
    if (!solo) move(1);

    // Slots.  A request that has tokens in this range marks the place of its
    // first one there; a running maximum over the places finds each token's.
    for (int64_t t0 = (int64_t)blockIdx.x * TOK; t0 < a.tokens; t0 += (int64_t)G * TOK) {
        for (int i = tid; i < TOK; i += TB) owner[i] = -1;
        __syncthreads();
        int64_t s = before.add, took = before.need;
        for (int r = r0; r < r1; r++) {
            const Req q = req(r);
            if (q.add > 0 && s < t0 + TOK && s + q.add > t0) {
                const int p = (int)(s > t0 ? s - t0 : 0);
                owner[p] = p;
                o_req[p] = r;
                o_start[p] = (int32_t)s;
                o_took[p] = (int32_t)took;
                o_len[p] = (int32_t)q.len;
            }
            s += q.add;
            took += q.need;
        }
        __syncthreads();
        constexpr int PT = TOK / TB;
        int top[PT];
        int run = -1;
        for (int i = 0; i < PT; i++) {
            run = max(run, owner[tid * PT + i]);
            top[i] = run;
        }
        int inc_top = run;
        for (int d = 1; d < 64; d <<= 1) {
            const int x = __shfl_up(inc_top, d, 64);
            if (lane >= d) inc_top = max(inc_top, x);
        }
        if (lane == 63) wtop[wave] = inc_top;
        int prev = __shfl_up(inc_top, 1, 64);
        if (lane == 0) prev = -1;
        __syncthreads();
        for (int w = 0; w < wave; w++) prev = max(prev, wtop[w]);
        for (int i = 0; i < PT; i++) {
            const int64_t tok = t0 + tid * PT + i;
            if (tok >= a.tokens) break;
            const int p = max(prev, top[i]);
            int64_t slot = -1;
            if (tok < all.add && p >= 0) {
                const int r = o_req[p];
                const int64_t len = o_len[p];
                const int64_t held = (len + (((int64_t)1 << a.bsh) - 1)) >> a.bsh;
                const int64_t pos = len + tok - o_start[p], col = pos >> a.bsh;
                const int64_t block = col < held ? a.table[(int64_t)r * a.table_stride + col]
                                                 : a.ring[(uint32_t)(head + o_took[p] + col - held) % (uint32_t)ring];
                slot = (block << a.bsh) + (pos & (((int64_t)1 << a.bsh) - 1));
            }
            a.slots[tok] = slot;
        }
        __syncthreads();
    }
    if (solo) {
        __syncthreads();
        move(1);
    }
}

int launch_kv_tables(const KvTablesLaunch &L, hipStream_t s) {
    const uint64_t want = ((uint64_t)L.tokens + TOK - 1) / TOK;
    const uint32_t grid = want < 1 ? 1u : want > MAX_WG ? MAX_WG : (uint32_t)want;
    if (L.requests <= 256)
        hipLaunchKernelGGL(k_kv_tables<256>, dim3(grid), dim3(256), 0, s, L);
    else
        hipLaunchKernelGGL(k_kv_tables<1024>, dim3(grid), dim3(1024), 0, s, L);
    return hipGetLastError() == hipSuccess ? 0 : 9;  // NQ_ERR_HIP
}

}  // namespace nq
