// k_kv_attn_e4m3.hip -- attention over E4M3 codes.
#include "nq_kv_rows.h"

namespace nq {
int launch_kv_attn_e4m3(const KvAttnLaunch &L, hipStream_t s) { return launch_kv_attn_code<KV_E4M3>(L, s); }
}  // namespace nq
