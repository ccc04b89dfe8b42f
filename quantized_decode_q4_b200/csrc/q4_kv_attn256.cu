// Attention over the 4-bit cache for a head dimension of 256.
#include "q4_kv_attn.cuh"

namespace q4kv {
Q4KV_ATTENTION(256)
}  // namespace q4kv
