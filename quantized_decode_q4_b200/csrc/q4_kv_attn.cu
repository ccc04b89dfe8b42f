// Decode attention over the 4-bit key/value cache.
//
// For each query token and head: s_p = scale * q . k_p over the visible positions p,
// optionally capped (cap * tanh(s / cap)) and biased (+ slope * (p - position)), then
// out = sum_p exp(s_p - m) v_p / sum_p exp(s_p - m), lse = m + log(sum).
// One warp per query row, the head dimension over its lanes; binary32 throughout, the
// running maximum and sum kept as the positions pass.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "q4_kv_layout.h"
#include "q4_kv_rows.cuh"

namespace q4kv {

namespace {

template <int DIM>
__global__ void __launch_bounds__(128) kv_attention_kernel(const AttnParams P, int64_t rows) {
    constexpr int E = DIM / 32;  // lane l holds elements l, l + 32, ... : one of each block
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int hq = (int)(row % P.q_heads), i = (int)(row / P.q_heads % P.tokens), s = (int)(row / P.q_heads / P.tokens);
    const int h = hq / (P.q_heads / P.cache.heads);
    const int len = clamp_int(P.seqs.lens[s], 0, reach(P.cache, P.seqs));
    const int nl = P.seqs.new_lens ? clamp_int(P.seqs.new_lens[s], 0, P.tokens) : P.tokens;
    const int pos = i < nl ? len - nl + i : -1;
    const int low = P.window > 0 && pos >= P.window ? pos - P.window + 1 : 0;
    const int64_t qat = row_at(P.q, s, i, hq);
    float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int b = 0; b < E; ++b) {
        const int64_t at = qat + b * 32 + lane;
        q[b] = P.q.type == Q4_F32 ? static_cast<const float*>(P.q.data)[at]
                                  : as_float(static_cast<const uint16_t*>(P.q.data)[at], P.q.type == Q4_BF16);
        o[b] = 0.0f;
    }
    const float slope = P.alibi ? P.alibi[hq] : 0.0f;
    const int byte = lane & 15, shift = lane < 16 ? 0 : 4;
    for (int p = low; p <= pos; ++p) {
        const int pg = p / P.cache.page_size, in = p - pg * P.cache.page_size;
        const int page = P.seqs.table[s * P.seqs.table_stride + pg];
        if (page < 0 || page >= P.cache.pages) {
            if (lane == 0) atomicOr(P.ws, kBadPage);
            continue;
        }
        const uint8_t* rec = P.cache.data + record_at(P.cache, DIM, page, h, in);
        const int t = in % kGroup;
        float dot = 0.0f;
#pragma unroll
        for (int b = 0; b < E; ++b) {
            const int c = rec[key_word(DIM, t, b, byte >> 2) + (byte & 3)] >> shift & 15;
            const float d = __half2float(*reinterpret_cast<const __half*>(rec + key_scale(DIM, t, b)));
            dot += d * (float)(c - 8) * q[b];
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        float x = dot * P.scale;
        if (P.softcap > 0.0f) x = P.softcap * tanhf(x / P.softcap);
        x += slope * (float)(p - pos);
        const float mn = fmaxf(m, x), a = m == mn ? 1.0f : expf(m - mn), e = expf(x - mn);
        l = l * a + e;
        m = mn;
#pragma unroll
        for (int b = 0; b < E; ++b) {
            const int c = rec[value_half(DIM, t, b, byte >> 1) + (byte & 1)] >> shift & 15;
            const float d = __half2float(*reinterpret_cast<const __half*>(rec + value_scale(DIM, t, b)));
            o[b] = o[b] * a + e * (d * (float)(c - 8));
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t oat = row_at(P.out, s, i, hq);
#pragma unroll
    for (int b = 0; b < E; ++b) {
        const int64_t at = oat + b * 32 + lane;
        const float v = o[b] * inv;
        if (P.out.type == Q4_F32)
            static_cast<float*>(P.out.data)[at] = v;
        else
            static_cast<uint16_t*>(P.out.data)[at] = (uint16_t)as_bits16(v, P.out.type == Q4_BF16);
    }
    if (P.lse && lane == 0) P.lse[row] = m + logf(l);
}

}  // namespace

cudaError_t launch_kv_attention(int dim, const AttnParams& P, cudaStream_t stream) {
    const int64_t rows = (int64_t)P.seqs.count * P.tokens * P.q_heads;
    const unsigned grid = (unsigned)((rows + 3) / 4);
    if (dim == 64)
        kv_attention_kernel<64><<<grid, 128, 0, stream>>>(P, rows);
    else if (dim == 128)
        kv_attention_kernel<128><<<grid, 128, 0, stream>>>(P, rows);
    else
        kv_attention_kernel<256><<<grid, 128, 0, stream>>>(P, rows);
    return cudaGetLastError();
}

}  // namespace q4kv
