// Loads and stores of four neighbouring activations of any of the library's types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/q4.h"
#include "q4_kv_layout.h"

namespace q4kv {

__device__ __forceinline__ int64_t row_at(const Rows& r, int s, int i, int h) {
    return s * r.seq + i * r.token + h * r.head;
}

__device__ __forceinline__ float as_float(uint32_t bits16, bool bf16) {
    return bf16 ? __uint_as_float(bits16 << 16) : __half2float(__ushort_as_half((unsigned short)bits16));
}

__device__ __forceinline__ uint32_t as_bits16(float v, bool bf16) {
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

// Elements at .. at + 3 (at a multiple of four from a row's start) as binary32.
__device__ __forceinline__ void load4(const Rows& r, int64_t at, float (&v)[4]) {
    if (r.type == Q4_F32) {
        const float* p = static_cast<const float*>(r.data) + at;
        if (r.vec) {
            const float4 t = *reinterpret_cast<const float4*>(p);
            v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = p[j];
        }
        return;
    }
    const uint16_t* p = static_cast<const uint16_t*>(r.data) + at;
    const bool bf = r.type == Q4_BF16;
    if (r.vec) {
        const uint2 t = *reinterpret_cast<const uint2*>(p);
        v[0] = as_float(t.x & 0xffffu, bf), v[1] = as_float(t.x >> 16, bf);
        v[2] = as_float(t.y & 0xffffu, bf), v[3] = as_float(t.y >> 16, bf);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = as_float(p[j], bf);
    }
}

// Stores v rounded once to the rows' type.
__device__ __forceinline__ void store4(const Rows& r, int64_t at, const float (&v)[4]) {
    if (r.type == Q4_F32) {
        float* p = static_cast<float*>(r.data) + at;
        if (r.vec) {
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = v[j];
        }
        return;
    }
    uint16_t* p = static_cast<uint16_t*>(r.data) + at;
    const bool bf = r.type == Q4_BF16;
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = as_bits16(v[j], bf);
    if (r.vec) {
        *reinterpret_cast<uint2*>(p) = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = (uint16_t)b[j];
    }
}

// The types of a call's rows: one of q4_dtype where all have it and four neighbours can be
// moved at once, else any, looked up at each access.
constexpr int kAnyRows = 3;
constexpr int kAnyBf16 = 4;  // bfloat16 at any alignment

template <int T>
__device__ __forceinline__ void load_four(const Rows& r, int64_t at, float (&v)[4]) {
    if constexpr (T == kAnyRows || T == kAnyBf16) {
        load4(r, at, v);
    } else if constexpr (T == Q4_F32) {
        const float4 t = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(r.data) + at));
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else {
        const uint2 t = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(r.data) + at));
        if constexpr (T == Q4_BF16) {
            v[0] = __uint_as_float(t.x << 16), v[1] = __uint_as_float(t.x & 0xffff0000u);
            v[2] = __uint_as_float(t.y << 16), v[3] = __uint_as_float(t.y & 0xffff0000u);
        } else {
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&t.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&t.y));
            v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
        }
    }
}

// Stores N = 2 or 4 neighbours rounded once to the rows' type.
template <int T, int N>
__device__ __forceinline__ void store_some(const Rows& r, int64_t at, const float (&v)[N]) {
    if constexpr (T == Q4_F32) {
        float* const p = static_cast<float*>(r.data) + at;
        if constexpr (N == 4)
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        else
            *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    } else if constexpr (T == Q4_F16 || T == Q4_BF16) {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if constexpr (T == Q4_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        uint16_t* const p = static_cast<uint16_t*>(r.data) + at;
        if constexpr (N == 4)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (r.type == Q4_F32)
                static_cast<float*>(r.data)[at + i] = v[i];
            else
                static_cast<uint16_t*>(r.data)[at + i] = (uint16_t)as_bits16(v[i], r.type == Q4_BF16);
        }
    }
}

}  // namespace q4kv
