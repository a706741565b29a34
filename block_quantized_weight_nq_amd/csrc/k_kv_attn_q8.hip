// k_kv_attn_q8.hip -- attention over signed 8-bit codes.
#include "nq_kv_rows.h"

namespace nq {
int launch_kv_attn_q8(const KvAttnLaunch &L, hipStream_t s) { return launch_kv_attn_code<KV_Q8>(L, s); }
}  // namespace nq
