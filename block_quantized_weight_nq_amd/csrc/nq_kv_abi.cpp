// nq_kv_abi.cpp -- the C ABI of the 8-bit key/value cache: argument checks (the launch plan is nq_kv.h's).
#include "../../include/nq.h"
#include "nq_kv.h"

#define NQ_API extern "C" __attribute__((visibility("default")))

namespace nq {
uint32_t device_compute_units();
int launch_kv_attn_q8(const KvAttnLaunch &L, hipStream_t s);
int launch_kv_attn_e4m3(const KvAttnLaunch &L, hipStream_t s);

}  // namespace nq

namespace {

constexpr int64_t MAX_LEN = 1ll << 30;
constexpr int64_t MAX_GROUPS = (1ll << 24) - 1;  // of 256 threads: a grid has less than 2^32 threads along an axis

int check_cache(const nq_kv_cache *c, nq::KvPool *p) {
    if (!c) return NQ_ERR_NULL_ARG;
    if (c->code != NQ_KV_Q8 && c->code != NQ_KV_E4M3) return NQ_ERR_UNKNOWN_FORMAT;
    if (c->dim != 64 && c->dim != 128 && c->dim != 256) return NQ_ERR_BAD_DIM;
    if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return NQ_ERR_BAD_DIM;
    if (c->heads < 1 || c->heads > 65535 || c->blocks < 1 || c->blocks >= (1ll << 31)) return NQ_ERR_BAD_DIM;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return NQ_ERR_NULL_ARG;
    if ((uintptr_t)c->k % 16 || (uintptr_t)c->v % 16 || (uintptr_t)c->k_scale % 4 || (uintptr_t)c->v_scale % 4)
        return NQ_ERR_MISALIGNED;
    p->k = (uint8_t *)c->k;
    p->v = (uint8_t *)c->v;
    p->ks = c->k_scale;
    p->vs = c->v_scale;
    p->blocks = c->blocks;
    p->heads = (uint32_t)c->heads;
    p->dim = (uint32_t)c->dim;
    p->bsh = c->block == 16 ? 4 : c->block == 32 ? 5 : c->block == 64 ? 6 : 7;
    return NQ_OK;
}

int64_t element_size(int32_t dtype) { return dtype == NQ_F32 ? 4 : 2; }
bool bad_dtype(int32_t dtype) { return dtype != NQ_F32 && dtype != NQ_F16 && dtype != NQ_BF16; }

// A stride of a tensor whose elements lie within 2^62 bytes of its address.
bool bad_stride(int64_t stride, int64_t count) {
    return stride < 0 || (count > 0 && stride > (1ll << 60) / count);
}

// The checks that attention and its workspace share; fills everything that the plan needs.
int check_attention(const nq_kv_cache *cache, const nq_kv_attention_args *x, nq::KvAttnLaunch *L) {
    if (!x) return NQ_ERR_NULL_ARG;
    const int st = check_cache(cache, &L->c);
    if (st != NQ_OK) return st;
    if (bad_dtype(x->dtype)) return NQ_ERR_BAD_DTYPE;
    if (x->tokens < 0 || x->requests < 1 || x->requests > 65534 || x->q_heads < 1 || x->q_heads % cache->heads != 0 ||
        x->max_new < 1 || x->max_length < 1 || x->window < 0 || x->table_width < 1)
        return NQ_ERR_BAD_DIM;
    if (x->q_heads > 65535 || x->max_new > MAX_LEN || x->max_length > MAX_LEN || x->tokens > MAX_LEN / x->q_heads || x->window > MAX_LEN ||
        x->table_width > MAX_LEN || bad_stride(x->table_stride, x->requests) || bad_stride(x->q_token_stride, x->tokens) ||
        bad_stride(x->q_head_stride, x->q_heads))
        return NQ_ERR_OVERFLOW;
    if (!(x->scale - x->scale == 0.0f)) return NQ_ERR_BAD_DIM;
    L->q_ts = x->q_token_stride;
    L->q_hs = x->q_head_stride;
    L->table_stride = x->table_stride;
    L->tokens = (int32_t)x->tokens;
    L->requests = (int32_t)x->requests;
    L->q_heads = (int32_t)x->q_heads;
    L->group = (int32_t)(x->q_heads / cache->heads);
    const int64_t named = x->table_width * cache->block;
    L->cap = (int32_t)(x->max_length < named ? x->max_length : named);
    L->max_new = (int32_t)(x->max_new < x->tokens ? x->max_new : x->tokens < 1 ? 1 : x->tokens);
    L->window = (int32_t)x->window;
    L->code = cache->code;
    L->dtype = x->dtype;
    L->scale = x->scale;
    nq::kv_attn_plan(*L, nq::device_compute_units());
    if ((int64_t)L->tiles_few * cache->heads > MAX_GROUPS || (int64_t)L->tiles * L->waves * cache->heads > 4 * MAX_GROUPS)
        return NQ_ERR_OVERFLOW;
    return NQ_OK;
}

uint64_t attention_workspace(const nq::KvAttnLaunch &L) {
    const uint64_t pieces = nq::kv_part_rows(L) * (uint64_t)L.splits + nq::kv_few_part_rows(L) * (uint64_t)L.splits_few;
    return pieces * 4 * ((uint64_t)L.c.dim + 1);
}

}  // namespace

NQ_API int nq_kv_tables(const int32_t *lengths, const int32_t *added, int64_t requests, int32_t *table,
                        int64_t table_width, int64_t table_stride, int32_t *ring, int64_t ring_size,
                        const int32_t *free_state, int32_t block, int64_t tokens, int32_t *lengths_out,
                        int32_t *token_start, int64_t *slots, int32_t *free_state_out, uint32_t *status,
                        hipStream_t stream) {
    if (block != 16 && block != 32 && block != 64 && block != 128) return NQ_ERR_BAD_DIM;
    if (requests < 1 || requests >= (1ll << 20) || table_width < 1 || ring_size < 1 || tokens < 0) return NQ_ERR_BAD_DIM;
    if (table_width > MAX_LEN || ring_size > MAX_LEN || tokens > MAX_LEN || bad_stride(table_stride, requests))
        return NQ_ERR_OVERFLOW;
    if (requests > 1 && table_stride < table_width) return NQ_ERR_BAD_DIM;
    if (!lengths || !added || !table || !ring || !free_state || !lengths_out || !token_start || !free_state_out ||
        !status || (tokens > 0 && !slots))
        return NQ_ERR_NULL_ARG;
    if (((uintptr_t)lengths | (uintptr_t)added | (uintptr_t)table | (uintptr_t)ring | (uintptr_t)free_state |
         (uintptr_t)lengths_out | (uintptr_t)token_start | (uintptr_t)free_state_out | (uintptr_t)status) % 4 ||
        (uintptr_t)slots % 8)
        return NQ_ERR_MISALIGNED;
    nq::KvTablesLaunch L;
    L.lengths = lengths;
    L.added = added;
    L.table = table;
    L.ring = ring;
    L.state = free_state;
    L.lengths_out = lengths_out;
    L.starts = token_start;
    L.slots = slots;
    L.state_out = free_state_out;
    L.status = status;
    L.table_stride = table_stride;
    L.tokens = tokens;
    L.requests = (int32_t)requests;
    L.width = (int32_t)table_width;
    L.ring_size = (int32_t)ring_size;
    L.bsh = block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7;
    return nq::launch_kv_tables(L, stream);
}

NQ_API int nq_kv_store(const nq_kv_cache *cache, const void *k, int64_t k_token_stride, int64_t k_head_stride,
                       const void *v, int64_t v_token_stride, int64_t v_head_stride, int64_t tokens, int32_t in_dtype,
                       const int64_t *slots, const int32_t *token_start, int64_t requests, uint32_t *status,
                       hipStream_t stream) {
    nq::KvStoreLaunch L;
    const int st = check_cache(cache, &L.c);
    if (st != NQ_OK) return st;
    if (bad_dtype(in_dtype)) return NQ_ERR_BAD_DTYPE;
    if (tokens < 0 || requests < 1) return NQ_ERR_BAD_DIM;
    if (tokens > MAX_LEN || requests >= (1ll << 24) || bad_stride(k_token_stride, tokens) ||
        bad_stride(v_token_stride, tokens) || bad_stride(k_head_stride, cache->heads) ||
        bad_stride(v_head_stride, cache->heads))
        return NQ_ERR_OVERFLOW;
    if (nq::kv_unit_first(tokens, requests, L.c.bsh) > MAX_GROUPS) return NQ_ERR_OVERFLOW;
    if (!status || !token_start || (tokens > 0 && (!k || !v || !slots))) return NQ_ERR_NULL_ARG;
    const uintptr_t esz = (uintptr_t)element_size(in_dtype);
    if ((uintptr_t)k % esz || (uintptr_t)v % esz || (uintptr_t)slots % 8 || (uintptr_t)token_start % 4 ||
        (uintptr_t)status % 4)
        return NQ_ERR_MISALIGNED;
    L.x[0] = k;
    L.x[1] = v;
    L.ts[0] = k_token_stride;
    L.ts[1] = v_token_stride;
    L.hs[0] = k_head_stride;
    L.hs[1] = v_head_stride;
    L.slots = slots;
    L.starts = token_start;
    L.status = status;
    L.tokens = tokens;
    L.requests = (int32_t)requests;
    L.code = cache->code;
    L.in_dtype = in_dtype;
    return nq::launch_kv_store(L, stream);
}

NQ_API int nq_kv_load(const nq_kv_cache *cache, const int32_t *ids, int64_t n, int32_t out_dtype, void *k_out,
                      void *v_out, hipStream_t stream) {
    nq::KvLoadLaunch L;
    const int st = check_cache(cache, &L.c);
    if (st != NQ_OK) return st;
    if (bad_dtype(out_dtype)) return NQ_ERR_BAD_DTYPE;
    if (n < 0) return NQ_ERR_BAD_DIM;
    if (n > MAX_GROUPS) return NQ_ERR_OVERFLOW;
    if (n == 0) return NQ_OK;
    if (!ids || !k_out || !v_out) return NQ_ERR_NULL_ARG;
    if ((uintptr_t)ids % 4 || (uintptr_t)k_out % 16 || (uintptr_t)v_out % 16) return NQ_ERR_MISALIGNED;
    L.ids = ids;
    L.out[0] = k_out;
    L.out[1] = v_out;
    L.n = n;
    L.code = cache->code;
    L.out_dtype = out_dtype;
    return nq::launch_kv_load(L, stream);
}

NQ_API int nq_kv_attention_workspace(const nq_kv_cache *cache, const nq_kv_attention_args *args, uint64_t *bytes) {
    if (!bytes) return NQ_ERR_NULL_ARG;
    *bytes = 0;
    nq::KvAttnLaunch L = {};
    const int st = check_attention(cache, args, &L);
    if (st != NQ_OK) return st;
    *bytes = attention_workspace(L);
    return NQ_OK;
}

NQ_API int nq_kv_attention(const nq_kv_cache *cache, const nq_kv_attention_args *args, void *workspace,
                           uint64_t workspace_bytes, hipStream_t stream) {
    nq::KvAttnLaunch L = {};
    const int st = check_attention(cache, args, &L);
    if (st != NQ_OK) return st;
    if (!args->token_start || !args->lengths || !args->table || (args->tokens > 0 && (!args->q || !args->out)))
        return NQ_ERR_NULL_ARG;
    const uintptr_t esz = (uintptr_t)element_size(args->dtype);
    if ((uintptr_t)args->q % esz || (uintptr_t)args->out % 16 || (uintptr_t)args->lse % 4 ||
        ((uintptr_t)args->token_start | (uintptr_t)args->lengths | (uintptr_t)args->table) % 4 ||
        (uintptr_t)workspace % 16)
        return NQ_ERR_MISALIGNED;
    const uint64_t need = attention_workspace(L);
    if (need > 0 && (!workspace || workspace_bytes < need)) return NQ_ERR_SCRATCH;
    if (args->tokens == 0) return NQ_OK;
    L.q = args->q;
    L.q_vec = (uintptr_t)args->q % 16 == 0 && args->q_token_stride * (int64_t)esz % 16 == 0 &&
              args->q_head_stride * (int64_t)esz % 16 == 0;
    L.starts = args->token_start;
    L.lengths = args->lengths;
    L.table = args->table;
    L.out = args->out;
    L.lse = args->lse;
    const uint64_t many = nq::kv_part_rows(L) * (uint64_t)L.splits, few = nq::kv_few_part_rows(L) * (uint64_t)L.splits_few;
    if (need > 0) {
        L.part = (float *)workspace;
        L.few_part = L.part + many * L.c.dim;
        L.part_lse = L.few_part + few * L.c.dim;
        L.few_part_lse = L.part_lse + many;
    }
    return L.code == NQ_KV_Q8 ? nq::launch_kv_attn_q8(L, stream) : nq::launch_kv_attn_e4m3(L, stream);
}
