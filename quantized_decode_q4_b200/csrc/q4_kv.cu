// Writing tokens into the 4-bit key/value cache and reading them back.
//
// Both move bytes and little else, so they are bound by memory once the work around a
// value is small. A warp takes a run of eight positions of one head: the page is looked up
// once a run, whose codes are contiguous in the record (by chunk, and keys and values
// apart). Eight lanes own a block of 32 values, four neighbours each, so that the dense side
// moves in coalesced 8- or 16-byte accesses. (A whole record a warp reads as fast where there
// are many, but writes 8192 tokens of 8 heads in 57 us against XXX us: too few loads in flight.) The
// codes follow the rule of q4_pack bit for bit: every binary32 step is an explicit
// round-to-nearest operation.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/q4.h"
#include "q4_kv_layout.h"
#include "q4_kv_rows.cuh"

namespace q4kv {

namespace {

constexpr int kWarps = 4;
constexpr int kUnroll = 4;  // tokens (or pairs) of a run whose loads fly together
constexpr uint32_t kFull = 0xffffffffu;

// The warp's head, sequence and how many runs its own lies behind the sequence's first;
// false behind the last task.
struct Task {
    int s, r, h;
};
__device__ __forceinline__ bool task_of(const MoveParams& P, Task* t) {
    uint32_t n = blockIdx.x * (uint32_t)kWarps + (threadIdx.x >> 5);
    if (n >= (uint32_t)P.items) return false;
    const uint32_t heads = (uint32_t)P.cache.heads, runs = (uint32_t)P.runs;
    t->h = (int)(n % heads);
    n /= heads;
    t->r = (int)(n % runs);
    t->s = (int)(n / runs);
    return true;
}

// The record of run `run` (positions 8 * run ..) of sequence s, or nullptr outside the table
// or the cache.
template <int DIM>
__device__ __forceinline__ uint8_t* record(const MoveParams& P, int s, int h, int64_t run) {
    if (run < 0 || run >= reach(P.cache, P.seqs) / kRun) return nullptr;
    const int p = (int)run * kRun, pg = p / P.cache.page_size;
    const int page = P.seqs.table[s * P.seqs.table_stride + pg];
    if (page < 0 || page >= P.cache.pages) return nullptr;
    return P.cache.data + record_at(P.cache, DIM, page, h, p - pg * P.cache.page_size);
}

// Quantises the eight lanes' 32 values: *word = word i8 % 4 of the block's codes (in
// lanes i8 and i8 ^ 4), *d = its scale (in every lane). A block that holds a NaN or an
// infinity gets the scale NaN.
__device__ __forceinline__ void quantise(const float (&v)[4], int i8, uint32_t* word, uint16_t* d) {
    float m = 0.0f;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        bad |= !(fabsf(v[j]) < __int_as_float(0x7f800000));
        if (fabsf(v[j]) > fabsf(m)) m = v[j];
    }
    // the lowest index wins a tie: the lower half of a pair of lanes keeps its own
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        const float o = __shfl_xor_sync(kFull, m, off);
        if (fabsf(o) > fabsf(m) || (fabsf(o) == fabsf(m) && (i8 & off))) m = o;
    }
    const bool any_bad = __ballot_sync(kFull, bad) >> (threadIdx.x & 24) & 0xffu;
    const float dd = __fmul_rn(m, -0.125f);  // m / -8
    const float inv = dd != 0.0f ? __frcp_rn(dd) : 0.0f;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // at or above 0.5, but for what is not a number or infinite: truncation is the floor
        const int q = (int)__fadd_rn(__fmul_rn(v[j], inv), 8.5f);
        w |= (uint32_t)min(max(q, 0), 15) << (8 * j);
    }
    const uint32_t o = __shfl_xor_sync(kFull, w, 4);
    *word = i8 < 4 ? w | (o << 4) : o | (w << 4);
    *d = any_bad ? (uint16_t)0x7fffu : __half_as_ushort(__float2half_rn(dd));
}

template <int DIM>
__global__ void __launch_bounds__(32 * kWarps) kv_write_kernel(const __grid_constant__ MoveParams P) {
    constexpr int C = chunk_blocks(DIM), NCH = DIM / 32 / C, L = 8 * C, TOK = 32 / L;  // TOK tokens at once
    Task k;
    if (!task_of(P, &k)) return;
    const int len = P.seqs.lens[k.s];
    const int nl = P.seqs.new_lens ? clamp_int(P.seqs.new_lens[k.s], 0, P.tokens) : P.tokens;
    const int64_t first = (int64_t)len - nl;  // position of the first new token
    const int64_t run = (first > 0 ? first / kRun : 0) + k.r;
    const int64_t p0 = first > run * kRun ? first : run * kRun;
    const int n = (int)((len < (run + 1) * kRun ? len : (run + 1) * kRun) - p0);
    if (n <= 0) return;
    uint8_t* const at = record<DIM>(P, k.s, k.h, run);
    if (!at) return;
    const int lane = threadIdx.x & 31, sub = lane / L, bb = lane % L / 8, i8 = lane & 7;
    const int t0 = (int)(p0 % kGroup), i0 = (int)(p0 - first);
    const int64_t ks = row_at(P.k, k.s, i0, k.h) + bb * 32 + 4 * i8, vs = row_at(P.v, k.s, i0, k.h) + bb * 32 + 4 * i8;
#pragma unroll kUnroll
    for (int base = 0; base < n; base += TOK) {
        const bool mine = base + sub < n;
        const int i = mine ? base + sub : n - 1, t = t0 + i;  // the last token twice rather than none
        float v[NCH][2][4];
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
            load4(P.k, ks + i * P.k.token + ch * 32 * C, v[ch][0]);
            load4(P.v, vs + i * P.v.token + ch * 32 * C, v[ch][1]);
        }
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
            const int b = ch * C + bb;
            uint32_t word;
            uint16_t d;
            quantise(v[ch][0], i8, &word, &d);
            if (mine && i8 < 4) *reinterpret_cast<uint32_t*>(at + key_word(DIM, t, b, i8)) = word;
            if (mine && i8 == 0) *reinterpret_cast<uint16_t*>(at + key_scale(DIM, t, b)) = d;
            quantise(v[ch][1], i8, &word, &d);
            // lane i8 takes half i8 of its block; the halves i8 of the chunk's blocks are neighbours
            const uint32_t w = __shfl_sync(kFull, word, (lane & 24) + (i8 >> 1));
            const uint32_t half = i8 & 1 ? w >> 16 : w & 0xffffu;
            const uint32_t pair = half | (__shfl_xor_sync(kFull, half, 8) << 16);
            if (C == 2) {
                if (mine && bb == 0) *reinterpret_cast<uint32_t*>(at + value_half(DIM, t, b, i8)) = pair;
            } else {
                const uint32_t next = __shfl_xor_sync(kFull, pair, 16);
                if (mine && bb == 0) *reinterpret_cast<uint2*>(at + value_half(DIM, t, b, i8)) = make_uint2(pair, next);
            }
            if (mine && i8 == 0) *reinterpret_cast<uint16_t*>(at + value_scale(DIM, t, b)) = d;
        }
    }
}

// Four values of a block: the nibbles of `word` at bits 0, 8, 16, 24, exact in binary32.
__device__ __forceinline__ void expand(uint32_t word, uint16_t d, float (&v)[4]) {
    const float s = __half2float(__ushort_as_half(d));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // 2^23 + q, less 2^23 + 8: exact
        const float f = __uint_as_float(((word >> (8 * j)) & 0xfu) | 0x4b000000u) - 8388616.0f;
        v[j] = __fmul_rn(s, f);
    }
}

template <int DIM>
__global__ void __launch_bounds__(32 * kWarps) kv_read_kernel(const __grid_constant__ MoveParams P) {
    constexpr int NB = DIM / 32, C = chunk_blocks(DIM), NCH = NB / C, L = 8 * C, TOK = 32 / L;
    constexpr int PART = 128 * C;  // bytes of a chunk of a run's keys or values
    __shared__ __align__(16) uint8_t shared[kWarps][2 * NCH * PART + 32 * NB];  // by chunk: keys, values; both scales
    Task k;
    if (!task_of(P, &k)) return;
    const int lane = threadIdx.x & 31, sub = lane / L, bb = lane % L / 8, i8 = lane & 7, c = i8 & 3;
    const int64_t first = P.starts ? P.starts[k.s] : 0;
    const int64_t run = (first >= 0 ? first / kRun : -((kRun - 1 - first) / kRun)) + k.r;
    // the run's positions that are rows of the output, and those of them that are held
    const int64_t p0 = first > run * kRun ? first : run * kRun;
    const int64_t end = first + P.tokens < (run + 1) * kRun ? first + P.tokens : (run + 1) * kRun;
    const int n = (int)(end - p0);
    if (n <= 0) return;
    const int64_t left = P.seqs.lens[k.s] - p0;
    const uint8_t* const at = left > 0 ? record<DIM>(P, k.s, k.h, run) : nullptr;
    const int held = at ? (int)(left < n ? left : n) : 0;
    uint8_t* const sm = shared[threadIdx.x >> 5];
    if (held > 0) {
        const int t = (int)(run * kRun % kGroup);
        uint4* const to = reinterpret_cast<uint4*>(sm);
#pragma unroll
        for (int i = 0; i < 2 * NCH * PART / 512; ++i) {
            // 512 bytes: a chunk's keys or values (C 4), or both (C 2)
            const int part = (i * 32 + lane) / L, ch = part / 2, in = lane % L;
            const int from = part & 1 ? value_half(DIM, t, ch * C, 0) : key_word(DIM, t, ch * C, 0);
            to[i * 32 + lane] = __ldcs(reinterpret_cast<const uint4*>(at + from) + in);
        }
        if (lane < 2 * NB) {
            const int from = lane < NB ? key_scale(DIM, t, 0) : value_scale(DIM, t, 0);
            to[2 * NCH * PART / 16 + lane] = __ldcs(reinterpret_cast<const uint4*>(at + from) + lane % NB);
        }
    }
    __syncwarp();
    const int t0 = (int)(p0 - run * kRun), i0 = (int)(p0 - first), shift = i8 < 4 ? 0 : 4;
    const int64_t ks = row_at(P.k, k.s, i0, k.h) + bb * 32 + 4 * i8, vs = row_at(P.v, k.s, i0, k.h) + bb * 32 + 4 * i8;
    const uint16_t* const scales = reinterpret_cast<const uint16_t*>(sm + 2 * NCH * PART) + bb;
#pragma unroll kUnroll
    for (int i = sub; i < n; i += TOK) {
        const int t = t0 + i;
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
            float kv[4] = {0.0f, 0.0f, 0.0f, 0.0f}, vv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (i < held) {
                const uint32_t* const keys = reinterpret_cast<const uint32_t*>(sm + 2 * ch * PART);
                const uint16_t* const values = reinterpret_cast<const uint16_t*>(sm + (2 * ch + 1) * PART);
                const int v = (t / 2 * 8 + 2 * c) * 2 + t % 2;  // half 2c of the token, the next is two behind
                const uint32_t lo = values[v * C + bb], hi = values[(v + 2) * C + bb];
                expand(keys[(t * 4 + c) * C + bb] >> shift, scales[t * NB + ch * C], kv);
                expand((lo | (hi << 16)) >> shift, scales[(kRun + t) * NB + ch * C], vv);
            }
            store4(P.k, ks + i * P.k.token + ch * 32 * C, kv);
            store4(P.v, vs + i * P.v.token + ch * 32 * C, vv);
        }
    }
}

template <int DIM>
cudaError_t launch(bool write, const MoveParams& P, cudaStream_t stream) {
    const unsigned grid = (unsigned)(((int64_t)P.items + kWarps - 1) / kWarps);
    if (write)
        kv_write_kernel<DIM><<<grid, 32 * kWarps, 0, stream>>>(P);
    else
        kv_read_kernel<DIM><<<grid, 32 * kWarps, 0, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_move(bool write, int dim, const MoveParams& P, cudaStream_t stream) {
    return dim == 64 ? launch<64>(write, P, stream) : dim == 128 ? launch<128>(write, P, stream) : launch<256>(write, P, stream);
}

}  // namespace q4kv
