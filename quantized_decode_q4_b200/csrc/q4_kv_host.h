// Launches of the key/value cache kernels.
#pragma once

#include <cuda_runtime.h>

#include "q4_kv_layout.h"

namespace q4kv {
cudaError_t launch_kv_move(bool write, int dim, const MoveParams& P, cudaStream_t stream);
cudaError_t launch_kv_attention(int dim, const AttnParams& P, cudaStream_t stream);
}  // namespace q4kv
