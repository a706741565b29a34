// nq_kv_plan_emu.hip -- host run of the key/value cache kernels' searches, plans and places (test infrastructure).
// Built host-only.
#include "../../block_quantized_weight_nq_amd/csrc/nq_kv.h"

#define EMU_API extern "C" __attribute__((visibility("default")))

// The request that a store workgroup of `threads` threads finds for unit u, or -1, by the kernel's rounds; *bad counts
// reads of starts outside its requests + 1 entries, *rounds the rounds before the last.
EMU_API int nq_kv_emu_request(const int32_t *starts, int requests, int64_t u, int bsh, int threads, int32_t *bad,
                              int32_t *rounds) {
    int32_t from = 0, left = requests;
    *bad = *rounds = 0;
    while (left > threads) {
        const int32_t step = nq::kv_probe_step(left, threads);
        int32_t hits = 0;
        for (int32_t tid = 0; tid < threads; tid++) {
            if (tid * step >= left) continue;
            const int32_t i = from + tid * step;
            if (i < 0 || i >= requests)
                ++*bad;
            else
                hits += nq::kv_unit_first(starts[i], i, (uint32_t)bsh) <= u;
        }
        if (hits == 0) return -1;
        nq::kv_narrow(&from, &left, step, hits);
        ++*rounds;
    }
    int found = -1;
    for (int32_t tid = 0; tid < threads && tid < left; tid++) {
        const int32_t i = from + tid;
        if (i < 0 || i >= requests)
            ++*bad;
        else if (nq::kv_unit_first(starts[i], i, (uint32_t)bsh) <= u && u < nq::kv_unit_first(starts[i + 1], i + 1, (uint32_t)bsh))
            found = i;
    }
    return found;
}
