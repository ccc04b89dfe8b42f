// Attention over the 4-bit cache for a head dimension of 128.
#include "q4_kv_attn.cuh"

namespace q4kv {
Q4KV_ATTENTION(128)
}  // namespace q4kv
