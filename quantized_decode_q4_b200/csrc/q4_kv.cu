// Writing tokens into the 4-bit key/value cache and reading them back.
//
// Both are streaming kernels bound by memory: eight lanes own one block of 32 values,
// four neighbouring values each, so the dense side moves in coalesced 8- or 16-byte
// accesses; a warp holds the C blocks of a chunk of one (token, head) for the key and
// the value at once (two independent streams in flight). The codes follow the rule of
// q4_pack bit for bit: every binary32 step is an explicit round-to-nearest operation.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/q4.h"
#include "q4_kv_layout.h"
#include "q4_kv_rows.cuh"

namespace q4kv {

namespace {

constexpr int kThreads = 256;

// The lane's token, head and place; false when the token has none in the cache.
struct Item {
    int s, i, h, chunk, bb, i8;
};

template <int DIM>
__device__ __forceinline__ bool item_of(const MoveParams& P, Item* it) {
    constexpr int C = chunk_blocks(DIM), L = 8 * C, NCH = DIM / 32 / C;
    const uint32_t lane = threadIdx.x % L;
    const int64_t at = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
    if (at >= P.items) return false;
    uint32_t n = (uint32_t)at;
    it->chunk = (int)(n % NCH);
    n /= NCH;
    it->h = (int)(n % (uint32_t)P.cache.heads);
    n /= (uint32_t)P.cache.heads;
    it->i = (int)(n % (uint32_t)P.tokens);
    it->s = (int)(n / (uint32_t)P.tokens);
    it->bb = (int)(lane >> 3);
    it->i8 = (int)(lane & 7);
    return true;
}

// The record of position `pos` of sequence s, or nullptr outside the table or the cache.
template <int DIM>
__device__ __forceinline__ uint8_t* record(const MoveParams& P, int s, int h, int64_t pos) {
    if (pos < 0 || pos >= reach(P.cache, P.seqs)) return nullptr;
    const int p = (int)pos, pg = p / P.cache.page_size;
    const int page = P.seqs.table[s * P.seqs.table_stride + pg];
    if (page < 0 || page >= P.cache.pages) return nullptr;
    return P.cache.data + record_at(P.cache, DIM, page, h, p - pg * P.cache.page_size);
}

// Quantises the eight lanes' 32 values: *word = word i8 % 4 of the block's codes (in
// lanes i8 and i8 ^ 4), *d = its scale (in every lane). A block that holds a NaN or an
// infinity gets the scale NaN.
__device__ __forceinline__ void quantise(const float (&v)[4], int i8, uint32_t mask, uint32_t* word, uint16_t* d) {
    float m = 0.0f, amax = 0.0f;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = fabsf(v[j]);
        bad |= !(a < __int_as_float(0x7f800000));
        if (a > amax) {
            amax = a;
            m = v[j];
        }
    }
    // the lowest index wins a tie: the upper half of a pair of lanes yields to an equal one
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        const float om = __shfl_xor_sync(mask, m, off);
        const float oa = fabsf(om);
        if (oa > amax || (oa == amax && (i8 & off))) {
            amax = oa;
            m = om;
        }
    }
    const uint32_t any_bad = __ballot_sync(mask, bad);
    const uint32_t mine = 0xffu << ((threadIdx.x & 31) & ~7);
    const float dd = __fdiv_rn(m, -8.0f);
    const float inv = dd != 0.0f ? __frcp_rn(dd) : 0.0f;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float t = floorf(__fadd_rn(__fmul_rn(v[j], inv), 8.5f));
        w |= (uint32_t)(int)fminf(fmaxf(t, 0.0f), 15.0f) << (8 * j);
    }
    const uint32_t o = __shfl_xor_sync(mask, w, 4);
    *word = i8 < 4 ? w | (o << 4) : o | (w << 4);
    *d = (any_bad & mine) ? (uint16_t)0x7fffu : __half_as_ushort(__float2half_rn(dd));
}

template <int DIM>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const MoveParams P) {
    constexpr int C = chunk_blocks(DIM), L = 8 * C;
    // the lanes of one (token, head, chunk): 16 or 32, together in every shuffle
    const uint32_t mask = L == 32 ? 0xffffffffu : 0xffffu << ((threadIdx.x & 31) / L * L);
    Item it;
    if (!item_of<DIM>(P, &it)) return;
    const int len = P.seqs.lens[it.s];
    const int nl = P.seqs.new_lens ? clamp_int(P.seqs.new_lens[it.s], 0, P.tokens) : P.tokens;
    if (it.i >= nl) return;
    const int64_t pos = (int64_t)len - nl + it.i;
    uint8_t* rec = record<DIM>(P, it.s, it.h, pos);
    if (!rec) return;
    const int t = (int)pos % P.cache.page_size % kGroup;
    const int b = it.chunk * C + it.bb, x = b * 32 + 4 * it.i8;
    float kv[4], vv[4];
    load4(P.k, row_at(P.k, it.s, it.i, it.h) + x, kv);
    load4(P.v, row_at(P.v, it.s, it.i, it.h) + x, vv);
    uint32_t word;
    uint16_t d;
    quantise(kv, it.i8, mask, &word, &d);
    if (it.i8 < 4) *reinterpret_cast<uint32_t*>(rec + key_word(DIM, t, b, it.i8)) = word;
    if (it.i8 == 0) *reinterpret_cast<uint16_t*>(rec + key_scale(DIM, t, b)) = d;
    quantise(vv, it.i8, mask, &word, &d);
    // lane i8 takes half i8 of its block; the halves i8 of the chunk's blocks are neighbours
    const uint32_t from = (threadIdx.x & 31) & ~7u;
    const uint32_t w = __shfl_sync(mask, word, from + (it.i8 >> 1));
    uint32_t half = it.i8 & 1 ? w >> 16 : w & 0xffffu;
    uint32_t pair = half | (__shfl_xor_sync(mask, half, 8) << 16);
    if (C == 2) {
        if (it.bb == 0) *reinterpret_cast<uint32_t*>(rec + value_half(DIM, t, b, it.i8)) = pair;
    } else {
        const uint32_t next = __shfl_xor_sync(mask, pair, 16);
        if (it.bb == 0) *reinterpret_cast<uint2*>(rec + value_half(DIM, t, b, it.i8)) = make_uint2(pair, next);
    }
    if (it.i8 == 0) *reinterpret_cast<uint16_t*>(rec + value_scale(DIM, t, b)) = d;
}

__device__ __forceinline__ void expand(uint32_t word, int i8, uint16_t d, float (&v)[4]) {
    const uint32_t nib = i8 < 4 ? word : word >> 4;
    const float s = __half2float(__ushort_as_half(d));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __fmul_rn(s, (float)((int)((nib >> (8 * j)) & 0xfu) - 8));
}

template <int DIM>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const MoveParams P) {
    constexpr int C = chunk_blocks(DIM);
    Item it;
    if (!item_of<DIM>(P, &it)) return;
    const int64_t pos = (P.starts ? (int64_t)P.starts[it.s] : 0) + it.i;
    const uint8_t* rec = pos < P.seqs.lens[it.s] ? record<DIM>(P, it.s, it.h, pos) : nullptr;
    const int b = it.chunk * C + it.bb, x = b * 32 + 4 * it.i8;
    float kv[4] = {0.0f, 0.0f, 0.0f, 0.0f}, vv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (rec) {
        const int t = (int)pos % P.cache.page_size % kGroup, c = it.i8 & 3;
        const uint32_t kw = *reinterpret_cast<const uint32_t*>(rec + key_word(DIM, t, b, c));
        const uint32_t lo = *reinterpret_cast<const uint16_t*>(rec + value_half(DIM, t, b, 2 * c));
        const uint32_t hi = *reinterpret_cast<const uint16_t*>(rec + value_half(DIM, t, b, 2 * c + 1));
        expand(kw, it.i8, *reinterpret_cast<const uint16_t*>(rec + key_scale(DIM, t, b)), kv);
        expand(lo | (hi << 16), it.i8, *reinterpret_cast<const uint16_t*>(rec + value_scale(DIM, t, b)), vv);
    }
    store4(P.k, row_at(P.k, it.s, it.i, it.h) + x, kv);
    store4(P.v, row_at(P.v, it.s, it.i, it.h) + x, vv);
}

template <int DIM>
cudaError_t launch(bool write, const MoveParams& P, cudaStream_t stream) {
    constexpr int L = 8 * chunk_blocks(DIM);
    const unsigned grid = (unsigned)(((int64_t)P.items * L + kThreads - 1) / kThreads);
    if (write)
        kv_write_kernel<DIM><<<grid, kThreads, 0, stream>>>(P);
    else
        kv_read_kernel<DIM><<<grid, kThreads, 0, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_move(bool write, int dim, const MoveParams& P, cudaStream_t stream) {
    return dim == 64 ? launch<64>(write, P, stream) : dim == 128 ? launch<128>(write, P, stream) : launch<256>(write, P, stream);
}

}  // namespace q4kv
