// Decode attention over the 4-bit key/value cache.
//
// For each query token and head: x_p = scale * q . k_p over the visible positions p,
// optionally capped (cap * tanh(x / cap)) and biased (+ slope * (p - position)), then
// out = sum_p exp(x_p - m) v_p / sum_p exp(x_p - m), lse = m + log(sum).
//
// What bounds it. A token of one head is 1.125 * dim bytes for 4 * rows * dim operations
// (rows = query heads of a key/value head times new tokens): bytes at few rows, but the
// codes have to be unpacked, and at the HBM rate an SM has about three lane-instructions
// for each code. So the kernel is built around instructions per code:
//  - The products run on m16n8k16 tensor-core steps with the codes as the A operand and
//    the query rows as the eight columns of B, so that few rows waste little. A nibble
//    masked in place (bits 0-3 or 4-7 of a 16-bit half) IS the binary16 subnormal
//    q * 2^-24 or q * 2^-20, exactly: one logic operation makes two operands. The offset
//    of 8 never touches a code: it enters the scores as -8 * sum(q row) per block, in the
//    accumulator's initial value, and the outputs as -8 * sum(weights), which one
//    more tensor-core step a block sums from the very weights that the products use.
//  - The cache's layout puts each lane's operands into one 16-byte shared load (keys by
//    word, values by token pairs), a record of 32 tokens into one bulk copy.
//  - The key scale multiplies a block's accumulator in binary32; the value scale
//    multiplies the weights.
//  - Softmax keeps a reference per row instead of the exact running maximum: weights
//    are 2^(x - ref), and ref moves only when a weight times a value scale could pass
//    2^15 (the test is one vote a tile), leaving 5 bits of room.
// Rounding. binary32 and binary16 queries (and results): each query row, scaled by a power
// of two, and each weight times its scale are held as two binary16 parts (22 bits),
// neighbouring columns of B. bfloat16 queries with bfloat16 results: one part each (the
// query's 8 bits are exact; weights and their product with the scale round to binary16's
// 2^-11 twice, an eighth of the result's own last place... each).
//
// One CTA an SM; each warp streams its own tiles through its own ring of records.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "q4_device.cuh"
#include "q4_kv_host.h"
#include "q4_kv_plan.h"
#include "q4_kv_rows.cuh"

namespace q4kv {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kTimeoutFlag = 1u;
constexpr int kRoom = 5;  // bits that scores may rise after ref was set before it moves again
constexpr int kNoWindow = INT32_MAX - 64;  // positions are above -64
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int DIM_, int NT_, bool SPLIT_, bool MOD_>
struct Cfg {
    static constexpr int DIM = DIM_, NT = NT_;
    static constexpr bool SPLIT = SPLIT_, MOD = MOD_;
    static constexpr int NB = DIM / 32, C = chunk_blocks(DIM), NCH = NB / C;
    static constexpr int RPL = SPLIT ? 1 : 2;       // rows of a lane in a column tile
    static constexpr int RC = NT * RPL * 4;         // query rows of a unit
    static constexpr int VPT = 2 * RPL;             // scores of a lane in 16 tokens
    static constexpr int REC = record_bytes(DIM);
    static constexpr int STAGES = DIM == 64 ? 4 : 2;
    static constexpr int WARPS = DIM == 256 ? 8 : (DIM == 128 && NT == 2 ? 12 : 16);
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int ROW = DIM + 8;             // floats of a row of a partial result in shared memory
    static constexpr int PART = RC * ROW;
    static constexpr int WPART = RC * (DIM + 2);    // floats of one in the workspace
    // shared memory
    static constexpr int RING = STAGES * REC;
    static constexpr int OFF_PART = WARPS * RING;
    static constexpr int OFF_ML = OFF_PART + WARPS * PART * 4;
    static constexpr int OFF_ENT = OFF_ML + WARPS * 2 * 2 * RC * 4;
    static constexpr int OFF_BAR = OFF_ENT + WARPS * 2 * 32;
    static constexpr int OFF_PRE = OFF_BAR + WARPS * STAGES * 8;
    static constexpr int SMEM = OFF_PRE + (THREADS + 40) * 8;
    static_assert(PART * 4 <= RING, "a partial result fits the warp's ring");
    static_assert(SMEM <= 226 * 1024, "shared memory, with the static part");
};

// A part of a unit whose rows another warp has to see: where its sums lie.
struct Entry {
    int64_t start;  // first tile of the unit
    int32_t s, u, n;
    int32_t part;   // float offset in shared memory, -1: none
    int32_t pad[2];
};
static_assert(sizeof(Entry) == 32, "entry");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, float c0, float c1, float c2, float c3) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ uint32_t transposed(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
}

// All bits of the halves of `a` that are not zero.
__device__ __forceinline__ uint32_t nonzero_half2(uint32_t a) {
    return __hne2_mask(*reinterpret_cast<const __half2*>(&a), __floats2half2_rn(0.0f, 0.0f));
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 t = *reinterpret_cast<const uint4*>(p);
        w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
    } else if constexpr (N == 2) {
        const uint2 t = *reinterpret_cast<const uint2*>(p);
        w[0] = t.x, w[1] = t.y;
    } else {
        static_assert(N == 1);
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

__device__ __forceinline__ float half_lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))); }
__device__ __forceinline__ float half_hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }

__device__ __forceinline__ Span span_at(const AttnParams& P, int s) {
    return span_of(P.seqs.lens[s], P.seqs.new_lens ? P.seqs.new_lens[s] : P.tokens, P.tokens, P.window, reach(P.cache, P.seqs));
}

__device__ __forceinline__ void store2(const Rows& r, int64_t at, float a, float b) {
    if (r.type == Q4_F32) {
        float* p = static_cast<float*>(r.data) + at;
        if (r.vec)
            *reinterpret_cast<float2*>(p) = make_float2(a, b);
        else
            p[0] = a, p[1] = b;
        return;
    }
    uint16_t* p = static_cast<uint16_t*>(r.data) + at;
    const uint32_t x = as_bits16(a, r.type == Q4_BF16), y = as_bits16(b, r.type == Q4_BF16);
    if (r.vec)
        *reinterpret_cast<uint32_t*>(p) = x | (y << 16);
    else
        p[0] = (uint16_t)x, p[1] = (uint16_t)y;
}

// Row `row` (0 .. tokens * group - 1) of key/value head h of sequence s: its token and query
// head, and whether it has a position.
struct RowAt {
    int i, hq;
    bool real;
};
__device__ __forceinline__ RowAt row_of(const AttnParams& P, const Span& sp, int h, int group, int row) {
    RowAt r;
    r.i = row / group;
    r.hq = h * group + (row - r.i * group);
    r.real = r.i < sp.nl && sp.len - sp.nl + r.i >= 0;
    return r;
}

// Two neighbouring outputs of a row from its sums, and the row's lse with the first pair.
__device__ __forceinline__ void write_pair(const AttnParams& P, int s, const RowAt& r, int x, float a, float b, float m, float l) {
    const float inv = l == 0.0f || !r.real ? 0.0f : 1.0f / l;
    if (!r.real) a = b = 0.0f;
    store2(P.out, row_at(P.out, s, r.i, r.hq) + x, a * inv, b * inv);
    if (P.lse && x == 0)
        P.lse[((int64_t)s * P.tokens + r.i) * P.q_heads + r.hq] = l == 0.0f || !r.real ? -INFINITY : (m + log2f(l)) * kLn2;
}

// exp2(a - b) for a <= b, 1 where both are the same infinity.
__device__ __forceinline__ float weight(float a, float b) { return a == b ? 1.0f : ex2(a - b); }

// The warp's place in the work: unit u of sequence s, tile t of its span.
struct Place {
    int s, u, t;
    Span sp;
};

template <class F>
struct Warp {
    // operands of the unit's query rows
    uint32_t qb[F::NT][F::NB][4];
    float bias[F::NT][F::NB][2];
    float f[F::NT][F::RPL];      // score = f * accumulator (base-2 logarithm unless F::MOD)
    float slope[F::MOD ? F::NT : 1][F::RPL];
    int pos[F::NT][F::RPL];      // positions of the lane's rows
    int minpos, maxpos;          // over the unit's rows that have one
    // sums
    float o[F::NB][2][F::NT][4];
    float ob[F::NT][4];
    float ref[F::NT][F::RPL], l[F::NT][F::RPL];
    int E;                       // value scales are below 2^E

    __device__ __forceinline__ void start() {
#pragma unroll
        for (int nt = 0; nt < F::NT; ++nt) {
#pragma unroll
            for (int b = 0; b < F::NB; ++b)
#pragma unroll
                for (int v = 0; v < 4; ++v) o[b][0][nt][v] = o[b][1][nt][v] = 0.0f;
#pragma unroll
            for (int v = 0; v < 4; ++v) ob[nt][v] = 0.0f;
#pragma unroll
            for (int r = 0; r < F::RPL; ++r) ref[nt][r] = -INFINITY, l[nt][r] = 0.0f;
        }
        E = F::SPLIT ? -14 : 0;
    }

    // Loads the query rows of unit u of sequence s.
    __device__ __forceinline__ void load_queries(const AttnParams& P, const Place& at, int rt_count, int group, int lane) {
        const int g = lane >> 2, c = lane & 3;
        const int h = at.u / rt_count, rt = at.u - h * rt_count, rows = P.tokens * group;
        const int first = at.sp.len - at.sp.nl;
        const int last_row = min((rt + 1) * F::RC, rows) - 1;
        minpos = max(first + rt * F::RC / group, 0);
        maxpos = min(first + last_row / group, at.sp.len - 1);
#pragma unroll
        for (int nt = 0; nt < F::NT; ++nt) {
            // column g of the tile: a row, or one of its two parts
            const int row = rt * F::RC + nt * F::RPL * 4 + (F::SPLIT ? g >> 1 : g);
            float v[F::NB][8], top = 0.0f;
            if (row < rows) {
                const RowAt r = row_of(P, at.sp, h, group, row);
                const int64_t base = row_at(P.q, at.s, r.i, r.hq);
#pragma unroll
                for (int b = 0; b < F::NB; ++b) {
                    float lo[4], hi[4];
                    load4(P.q, base + 32 * b + 4 * c, lo);
                    load4(P.q, base + 32 * b + 16 + 4 * c, hi);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[b][j] = lo[j], v[b][4 + j] = hi[j];
                        top = fmaxf(top, fmaxf(fabsf(lo[j]), fabsf(hi[j])));
                    }
                }
            } else {
#pragma unroll
                for (int b = 0; b < F::NB; ++b)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[b][j] = 0.0f;
            }
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
            // a power of two that brings the row's largest element into 2^13 .. 2^14
            const int e = top == 0.0f ? 0 : clamp_int(13 - ((int)(__float_as_uint(top) >> 23) - 127), -115, 110);
            const float up = __int_as_float((e + 127) << 23), down = __int_as_float((127 - e) << 23);
#pragma unroll
            for (int b = 0; b < F::NB; ++b) {
                float w[8], sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float x = v[b][j] * up;
                    float y = __half2float(__float2half_rn(x));
                    if (F::SPLIT && (g & 1)) y = __half2float(__float2half_rn(x - y));
                    sum += y;
                    w[j] = j < 4 ? y : y * 0.0625f;  // the codes of the upper 16 are read 16 times too large
                }
                qb[nt][b][0] = pack_half2(w[0], w[2]);
                qb[nt][b][1] = pack_half2(w[4], w[6]);
                qb[nt][b][2] = pack_half2(w[1], w[3]);
                qb[nt][b][3] = pack_half2(w[5], w[7]);
                sum += __shfl_xor_sync(kFull, sum, 1);
                sum += __shfl_xor_sync(kFull, sum, 2);
                sum *= -8.0f * 0x1p-24f;
                bias[nt][b][0] = __shfl_sync(kFull, sum, 8 * c);
                bias[nt][b][1] = __shfl_sync(kFull, sum, 8 * c + 4);
            }
            const float fg = (F::MOD ? P.scale : P.scale * kLog2e) * 0x1p24f * down;
#pragma unroll
            for (int r = 0; r < F::RPL; ++r) {
                f[nt][r] = __shfl_sync(kFull, fg, 8 * c + 4 * r);
                const int mine = min(rt * F::RC + (nt * 4 + c) * F::RPL + r, rows - 1);
                const RowAt ra = row_of(P, at.sp, h, group, mine);
                pos[nt][r] = first + ra.i;
                if (F::MOD) slope[nt][r] = P.alibi ? P.alibi[ra.hq] : 0.0f;
            }
        }
    }

    // Moves the references so that the tile's scores x and value scales up to the half
    // `dmax` fit, and scales the sums with them.
    __device__ __forceinline__ void move_refs(const float (&x)[2][F::NT][F::VPT], uint32_t dmax) {
        dmax = __reduce_max_sync(kFull, dmax);
        int En = E;
        if (dmax > (uint32_t)(E + 15) << 10) En = max(E, min(16, (int)(dmax >> 10) - 14));
        const float lim = (float)(15 - En);
#pragma unroll
        for (int nt = 0; nt < F::NT; ++nt) {
            float alpha[F::RPL];
#pragma unroll
            for (int r = 0; r < F::RPL; ++r) {
                float m = -INFINITY;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int v = r; v < F::VPT; v += F::RPL) m = fmaxf(m, x[u][nt][v]);
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
                const float old = ref[nt][r], moved = old + (float)(En - E);
                ref[nt][r] = m > moved + lim ? m - (lim - (float)kRoom) : moved;
                alpha[r] = weight(old, ref[nt][r]);
                l[nt][r] *= alpha[r];
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float a = alpha[v % F::RPL];
                ob[nt][v] *= a;
#pragma unroll
                for (int b = 0; b < F::NB; ++b) o[b][0][nt][v] *= a, o[b][1][nt][v] *= a;
            }
        }
        E = En;
    }

    // One record of 32 tokens from position p0 on. EDGE: some (row, token) is masked.
    template <bool EDGE>
    __device__ __forceinline__ void tile(const AttnParams& P, const uint8_t* rec, int p0, int lane, const uint32_t (&ones)[F::NB]) {
        constexpr int NB = F::NB, C = F::C, NT = F::NT, DIM = F::DIM;
        const int g = lane >> 2, c = lane & 3;
        const int window = P.window > 0 ? P.window : kNoWindow;
        // scores
        float x[2][NT][F::VPT];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int v = 0; v < 4; ++v) s[nt][v] = 0.0f;
            uint32_t ds[2][NB / 2];
            load_words(rec + key_scale(DIM, 16 * u + g, 0), ds[0]);
            load_words(rec + key_scale(DIM, 16 * u + g + 8, 0), ds[1]);
#pragma unroll
            for (int ch = 0; ch < F::NCH; ++ch) {
                uint32_t w[2][C];
                load_words(rec + key_word(DIM, 16 * u + g, ch * C, c), w[0]);
                load_words(rec + key_word(DIM, 16 * u + g + 8, ch * C, c), w[1]);
#pragma unroll
                for (int bb = 0; bb < C; ++bb) {
                    const int b = ch * C + bb;
                    const float d0 = b & 1 ? half_hi(ds[0][b / 2]) : half_lo(ds[0][b / 2]);
                    const float d1 = b & 1 ? half_hi(ds[1][b / 2]) : half_lo(ds[1][b / 2]);
                    const uint32_t w0 = w[0][bb], w1 = w[1][bb], y0 = w0 >> 8, y1 = w1 >> 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float a[4];
                        mma(a, w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u, qb[nt][b][0], qb[nt][b][1],
                            bias[nt][b][0], bias[nt][b][1], bias[nt][b][0], bias[nt][b][1]);
                        mma(a, y0 & 0x000f000fu, y1 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x00f000f0u, qb[nt][b][2], qb[nt][b][3],
                            a[0], a[1], a[2], a[3]);
                        s[nt][0] = fmaf(d0, a[0], s[nt][0]);
                        s[nt][1] = fmaf(d0, a[1], s[nt][1]);
                        s[nt][2] = fmaf(d1, a[2], s[nt][2]);
                        s[nt][3] = fmaf(d1, a[3], s[nt][3]);
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int v = 0; v < F::VPT; ++v) {
                    const int r = v % F::RPL, key = p0 + 16 * u + g + 8 * (v / F::RPL);
                    float t = (F::SPLIT ? s[nt][2 * v] + s[nt][2 * v + 1] : s[nt][v]) * f[nt][r];
                    if (F::MOD) {
                        if (P.softcap > 0.0f) t = P.softcap * tanhf(t / P.softcap);
                        t = fmaf(slope[nt][r], (float)(key - pos[nt][r]), t) * kLog2e;
                    }
                    if (EDGE && (key > pos[nt][r] || key <= pos[nt][r] - window)) t = -INFINITY;
                    x[u][nt][v] = t;
                }
        }
        // does every weight fit?
        uint32_t dmax = 0;
        {
            uint32_t dv[NB / 2];
            load_words(rec + value_scale(DIM, lane, 0), dv);
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < NB / 2; ++i) m = __vmaxu2(m, dv[i] & 0x7fff7fffu);
            dmax = max(m & 0xffffu, m >> 16);
            if (EDGE && (p0 + lane > maxpos || p0 + lane <= minpos - window)) dmax = 0;
        }
        bool high = dmax > (uint32_t)(E + 15) << 10;
        {
            const float lim = (float)(15 - E);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int v = 0; v < F::VPT; ++v) high |= x[u][nt][v] > ref[nt][v % F::RPL] + lim;
        }
        if (__any_sync(kFull, high)) move_refs(x, dmax);
        // weights and values
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t pb[NT][NB][2];  // B operands: weights times value scales
            if constexpr (F::SPLIT) {
                uint32_t dv[2][NB / 2];
                load_words(rec + value_scale(DIM, 16 * u + g, 0), dv[0]);
                load_words(rec + value_scale(DIM, 16 * u + g + 8, 0), dv[1]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        float p = ex2(x[u][nt][v] - ref[nt][0]);
                        if (EDGE && x[u][nt][v] == -INFINITY) p = 0.0f;
                        l[nt][0] += p;
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            float y = p * (b & 1 ? half_hi(dv[v][b / 2]) : half_lo(dv[v][b / 2]));
                            if (EDGE && p == 0.0f) y = 0.0f;  // whatever the scale is
                            const float hi = __uint_as_float(__float_as_uint(y) & 0xffffe000u);
                            pb[nt][b][v] = transposed(pack_half2(hi, y - hi));
                        }
                    }
            } else {
                uint32_t dv[2][2][NB / 2];  // [8 j][token 2 c + e]
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    load_words(rec + value_scale(DIM, 16 * u + 8 * j + 2 * c, 0), dv[j][0]);
                    load_words(rec + value_scale(DIM, 16 * u + 8 * j + 2 * c + 1, 0), dv[j][1]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float p[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float t = x[u][nt][2 * j + r];
                            p[r] = ex2(t - ref[nt][r]);
                            if (EDGE && t == -INFINITY) p[r] = 0.0f;
                            l[nt][r] += p[r];
                        }
                        const uint32_t pt = transposed(pack_half2(p[0], p[1]));
                        const uint32_t keep = EDGE ? nonzero_half2(pt) : kFull;
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            pb[nt][b][j] = mul_half2(pt, __byte_perm(dv[j][0][b / 2], dv[j][1][b / 2], b & 1 ? 0x7632 : 0x5410)) & keep;
                    }
            }
#pragma unroll
            for (int ch = 0; ch < F::NCH; ++ch) {
                uint32_t w[2][C];  // token pairs 2c, 2c + 1 and 8 behind: [e][C halves]
                load_words(rec + value_half(DIM, 16 * u + 2 * c, ch * C, g), w[0]);
                load_words(rec + value_half(DIM, 16 * u + 8 + 2 * c, ch * C, g), w[1]);
#pragma unroll
                for (int bb = 0; bb < C; ++bb) {
                    const int b = ch * C + bb;
                    const uint32_t sel = bb & 1 ? 0x7632 : 0x5410;
                    const uint32_t y0 = __byte_perm(w[0][bb / 2], w[0][C / 2 + bb / 2], sel), z0 = y0 >> 8;
                    const uint32_t y1 = __byte_perm(w[1][bb / 2], w[1][C / 2 + bb / 2], sel), z1 = y1 >> 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float(&a)[4] = o[b][0][nt];
                        mma(a, y0 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x000f000fu, y1 & 0x00f000f0u, pb[nt][b][0], pb[nt][b][1], a[0], a[1], a[2], a[3]);
                        float(&z)[4] = o[b][1][nt];
                        mma(z, z0 & 0x000f000fu, z0 & 0x00f000f0u, z1 & 0x000f000fu, z1 & 0x00f000f0u, pb[nt][b][0], pb[nt][b][1], z[0], z[1], z[2], z[3]);
                        float(&n)[4] = ob[nt];
                        mma(n, ones[b], 0u, ones[b], 0u, pb[nt][b][0], pb[nt][b][1], n[0], n[1], n[2], n[3]);
                    }
                }
            }
        }
    }

    // Hands the unit's sums to `put(row of the unit, element, two neighbouring sums, ref, l)`.
    template <class Put>
    __device__ __forceinline__ void finish(int lane, Put put) {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int nt = 0; nt < F::NT; ++nt) {
            float ls[F::RPL];
#pragma unroll
            for (int r = 0; r < F::RPL; ++r) {
                ls[r] = l[nt][r];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) ls[r] += __shfl_xor_sync(kFull, ls[r], off);
            }
#pragma unroll
            for (int b = 0; b < F::NB; ++b) {
                // the block's sum of weights lies in row b of the extra accumulator
                float w[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) w[r] = 8.0f * __shfl_sync(kFull, ob[nt][r], 4 * b + c);
#pragma unroll
                for (int r = 0; r < F::RPL; ++r)
#pragma unroll
                    for (int up = 0; up < 2; ++up) {
                        const float k = up ? 0x1p20f : 0x1p24f;
                        float v[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            v[e] = fmaf(o[b][e][nt][2 * up + r], k, -w[r]);
                            if (F::SPLIT) v[e] += fmaf(o[b][e][nt][2 * up + 1], k, -w[1]);
                        }
                        put((nt * 4 + c) * F::RPL + r, 32 * b + 16 * up + 2 * g, v[0], v[1], ref[nt][r], ls[r]);
                    }
            }
        }
    }
};

// Issues the copies of the warp's tiles, one record at a time, STAGES ahead of their use.
template <class F>
struct Producer {
    Place at;
    int64_t left;         // tiles not yet issued
    int page, r;          // ordinal of the page in the sequence's table, record in the page
    int base, entry;      // lane i holds entry base + i of the table's row
    uint32_t filled;      // per stage: a copy was issued into it

    __device__ __forceinline__ void load_entries(const AttnParams& P, int lane) {
        base = page;
        const int i = base + lane;
        entry = i < P.seqs.table_pages ? P.seqs.table[at.s * P.seqs.table_stride + i] : -1;
    }
    __device__ __forceinline__ void seek(const AttnParams& P, int lane) {
        const int rpp = P.cache.page_size / kGroup, tile = at.sp.tile0 + at.t;
        page = tile / rpp;
        r = tile - page * rpp;
        load_entries(P, lane);
    }
    __device__ __forceinline__ void issue(const AttnParams& P, int units, int rt_count, uint8_t* slot, uint64_t* bar, int stage, int lane) {
        if (left <= 0) return;
        const int pg = __shfl_sync(kFull, entry, page - base);
        const bool some = !nothing(at.sp), ok = some && pg >= 0 && pg < P.cache.pages;
        filled = (filled & ~(1u << stage)) | ((uint32_t)ok << stage);
        if (lane == 0) {
            if (ok) {
                const int64_t rec = ((int64_t)pg * P.cache.heads + at.u / rt_count) * (P.cache.page_size / kGroup) + r;
                q4dev::mbar_arrive_expect_tx(bar, F::REC);
                q4dev::bulk_g2s(slot, P.cache.data + rec * F::REC, F::REC, bar);
            } else if (some) {
                atomicOr(P.ws, kBadPage);
            }
        }
        --left;
        if (++at.t < at.sp.n) {
            if (++r == P.cache.page_size / kGroup) {
                r = 0;
                ++page;
                if (page - base == 32) load_entries(P, lane);
            }
        } else if (left > 0) {
            at.t = 0;
            if (++at.u == units) {
                at.u = 0;
                at.sp = span_at(P, ++at.s);
            }
            seek(P, lane);
        }
    }
};

template <class F>
__global__ void __launch_bounds__(F::THREADS, 1) kv_attention_kernel(const AttnParams P) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float* const parts = reinterpret_cast<float*>(smem + F::OFF_PART);
    float* const ml = reinterpret_cast<float*>(smem + F::OFF_ML);  // [warp][first, last][ref, l][RC]
    Entry* const ents = reinterpret_cast<Entry*>(smem + F::OFF_ENT);
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + F::OFF_BAR) + warp * F::STAGES;
    int64_t* const pre = reinterpret_cast<int64_t*>(smem + F::OFF_PRE);
    uint8_t* const ring = smem + warp * F::RING;

    const int group = P.q_heads / P.cache.heads;
    const int rows = P.tokens * group, rt_count = (rows + F::RC - 1) / F::RC;
    const int units = P.cache.heads * rt_count;

    // tiles before each run of `run` sequences
    const int run = (P.seqs.count + F::THREADS - 1) / F::THREADS;
    int64_t total;
    {
        const int64_t s0 = (int64_t)tid * run;
        int64_t sum = 0;
        for (int i = 0; i < run && s0 + i < P.seqs.count; ++i) sum += span_at(P, (int)s0 + i).n;
        int64_t inc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(kFull, inc, off);
            if (lane >= off) inc += o;
        }
        if (lane == 31) pre[F::THREADS + warp] = inc;
        if (lane == 0) {
            for (int i = 0; i < F::STAGES; ++i) q4dev::mbar_init(bars + i, 1);
            q4dev::mbar_fence_init();
            ents[2 * warp].part = ents[2 * warp + 1].part = -1;
        }
        __syncthreads();
        int64_t before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < F::WARPS; ++w) {
            const int64_t o = pre[F::THREADS + w];
            before += w < warp ? o : 0;
            all += o;
        }
        pre[tid] = before + inc - sum;
        total = all * units;
        __syncthreads();
    }
    const int ctas = ctas_of(total, F::WARPS, gridDim.x);
    if ((int)blockIdx.x >= ctas) return;
    const int64_t a = part_begin(total, ctas, blockIdx.x), z = part_begin(total, ctas, blockIdx.x + 1);
    const int64_t wa = a + part_begin(z - a, F::WARPS, warp), wz = a + part_begin(z - a, F::WARPS, warp + 1);

    if (wa < wz) {
        // the place of tile wa
        Place at;
        int64_t start;  // first tile of the unit
        {
            const int64_t y = wa / units;
            int lo = 0, hi = F::THREADS;  // pre[lo] <= y < pre[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (pre[mid] <= y && (int64_t)mid * run < P.seqs.count)
                    lo = mid;
                else
                    hi = mid;
            }
            at.s = lo * run;
            int64_t rest = y - pre[lo];
            at.sp = span_at(P, at.s);
            while (rest >= at.sp.n) {
                rest -= at.sp.n;
                at.sp = span_at(P, ++at.s);
            }
            const int64_t off = wa - (y - rest) * units;
            at.u = (int)(off / at.sp.n);
            at.t = (int)(off - (int64_t)at.u * at.sp.n);
            start = wa - at.t;
        }
        Producer<F> prod;
        prod.at = at;
        prod.left = wz - wa;
        prod.filled = 0;
        prod.seek(P, lane);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < F::STAGES; ++i) prod.issue(P, units, rt_count, ring + i * F::REC, bars + i, i, lane);

        uint32_t ones[F::NB];
#pragma unroll
        for (int b = 0; b < F::NB; ++b) ones[b] = (lane >> 2) == b ? 0x3c003c00u : 0u;
        Warp<F> w;
        int stage = 0;
        uint32_t phases = 0;
        bool dead = false;
        int64_t cur = wa;
        while (cur < wz) {
            const int n = (int)min((int64_t)(at.sp.n - at.t), wz - cur);
            const bool whole = n == at.sp.n;
            w.load_queries(P, at, rt_count, group, lane);
            w.start();
            const int window = P.window > 0 ? P.window : kNoWindow;
            for (int i = 0; i < n; ++i) {
                if (prod.filled >> stage & 1) {
                    // after a wait that gave up nothing is issued or computed any more, and the
                    // copies in flight are still waited for
                    if (!q4dev::mbar_wait_short_bounded(bars + stage, phases >> stage & 1)) dead = true;
                    dead = __any_sync(kFull, dead);
                    phases ^= 1u << stage;
                    if (dead) {
                        prod.filled &= ~(1u << stage);
                    } else {
                        const int p0 = (at.sp.tile0 + at.t + i) * kGroup;
                        const uint8_t* rec = ring + stage * F::REC;
                        if (p0 + kGroup - 1 <= w.minpos && p0 > w.maxpos - window)
                            w.template tile<false>(P, rec, p0, lane, ones);
                        else
                            w.template tile<true>(P, rec, p0, lane, ones);
                    }
                }
                __syncwarp();
                if (!dead) prod.issue(P, units, rt_count, ring + stage * F::REC, bars + stage, stage, lane);
                stage = stage + 1 == F::STAGES ? 0 : stage + 1;
            }
            cur += n;
            if (whole) {
                const int h = at.u / rt_count, row0 = (at.u - h * rt_count) * F::RC;
                w.finish(lane, [&](int row, int x, float v0, float v1, float m, float l) {
                    if (row0 + row < rows) write_pair(P, at.s, row_of(P, at.sp, h, group, row0 + row), x, v0, v1, m, l);
                });
            } else {
                // the ring is free once the warp's last tile is done
                const bool last = cur == wz;
                float* const p = last ? reinterpret_cast<float*>(ring) : parts + warp * F::PART;
                float* const rl = ml + (warp * 2 + last) * 2 * F::RC;
                __syncwarp();
                w.finish(lane, [&](int row, int x, float v0, float v1, float m, float l) {
                    *reinterpret_cast<float2*>(p + row * F::ROW + x) = make_float2(v0, v1);
                    if (x == 0) rl[row] = m, rl[F::RC + row] = l;
                });
                if (lane == 0) {
                    Entry& e = ents[2 * warp + last];
                    e.start = start, e.s = at.s, e.u = at.u, e.n = at.sp.n;
                    e.part = (int)(p - reinterpret_cast<float*>(smem));
                }
            }
            start += at.sp.n;
            if (cur < wz) {
                at.t = 0;
                if (++at.u == units) {
                    at.u = 0;
                    at.sp = span_at(P, ++at.s);
                }
            }
        }
        if (dead && lane == 0) atomicOr(P.ws, kTimeoutFlag);
    }
    __syncthreads();

    // join the units that warps cut
    __shared__ int last_cta[2];
    __shared__ int64_t cut_start[2];
    __shared__ int cut_entry[2];
    if (tid < 2) cut_entry[tid] = -1;
    __syncthreads();
    const float* const sf = reinterpret_cast<const float*>(smem);
    for (int e0 = 0; e0 < 2 * F::WARPS;) {
        if (ents[e0].part < 0) {
            ++e0;
            continue;
        }
        int e1 = e0 + 1;
        while (e1 < 2 * F::WARPS && (ents[e1].part < 0 || ents[e1].start == ents[e0].start)) ++e1;
        const Entry en = ents[e0];
        const bool whole = en.start >= a && en.start + en.n <= z;
        const int slot = en.start > a;
        if (!whole && tid == 0) cut_start[slot] = en.start, cut_entry[slot] = e0;
        float* const wp = P.parts + ((int64_t)blockIdx.x * 2 + slot) * F::WPART;
        const int h = en.u / rt_count, row0 = (en.u - h * rt_count) * F::RC;
        const Span sp = span_at(P, en.s);
        for (int i = tid; i < F::RC * F::DIM / 2; i += F::THREADS) {
            const int row = i / (F::DIM / 2), x = 2 * (i - row * (F::DIM / 2));
            if (row0 + row >= rows) break;
            float m = -INFINITY;
            for (int e = e0; e < e1; ++e)
                if (ents[e].part >= 0) m = fmaxf(m, ml[e * 2 * F::RC + row]);
            float v0 = 0.0f, v1 = 0.0f, l = 0.0f;
            for (int e = e0; e < e1; ++e) {
                if (ents[e].part < 0) continue;
                const float k = weight(ml[e * 2 * F::RC + row], m);
                const float2 v = *reinterpret_cast<const float2*>(sf + ents[e].part + row * F::ROW + x);
                v0 = fmaf(v.x, k, v0), v1 = fmaf(v.y, k, v1), l = fmaf(ml[e * 2 * F::RC + F::RC + row], k, l);
            }
            if (whole) {
                write_pair(P, en.s, row_of(P, sp, h, group, row0 + row), x, v0, v1, m, l);
            } else {
                *reinterpret_cast<float2*>(wp + row * F::DIM + x) = make_float2(v0, v1);
                if (x == 0) wp[F::RC * F::DIM + row] = m, wp[F::RC * F::DIM + F::RC + row] = l;
            }
        }
        e0 = e1;
    }
    __threadfence();
    __syncthreads();
    // and those that CTAs cut: the last to arrive joins them in order
    if (tid < 2) {
        int join = 0;
        if (cut_entry[tid] >= 0) {
            const int64_t start = cut_start[tid];
            const int i0 = part_of(total, ctas, start), i1 = part_of(total, ctas, start + ents[cut_entry[tid]].n - 1);
            const int sh = 8 * (i0 & 3);
            uint32_t* const ticket = P.ws + 1 + (i0 >> 2);
            const uint32_t old = atomicAdd(ticket, 1u << sh);
            if ((int)(old >> sh & 255u) == i1 - i0) {
                atomicSub(ticket, (uint32_t)(i1 - i0 + 1) << sh);
                join = 1;
            }
        }
        last_cta[tid] = join;
        __threadfence();
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        if (!last_cta[k]) continue;
        const Entry en = ents[cut_entry[k]];
        const int i0 = part_of(total, ctas, en.start), i1 = part_of(total, ctas, en.start + en.n - 1);
        const int slot0 = en.start > part_begin(total, ctas, i0);
        const int h = en.u / rt_count, row0 = (en.u - h * rt_count) * F::RC;
        const Span sp = span_at(P, en.s);
        for (int i = tid; i < F::RC * F::DIM / 2; i += F::THREADS) {
            const int row = i / (F::DIM / 2), x = 2 * (i - row * (F::DIM / 2));
            if (row0 + row >= rows) break;
            float m = -INFINITY;
            for (int cta = i0; cta <= i1; ++cta)
                m = fmaxf(m, __ldcg(P.parts + ((int64_t)cta * 2 + (cta == i0 ? slot0 : 0)) * F::WPART + F::RC * F::DIM + row));
            float v0 = 0.0f, v1 = 0.0f, l = 0.0f;
            for (int cta = i0; cta <= i1; ++cta) {
                const float* const wp = P.parts + ((int64_t)cta * 2 + (cta == i0 ? slot0 : 0)) * F::WPART;
                const float q = weight(__ldcg(wp + F::RC * F::DIM + row), m);
                const float2 v = __ldcg(reinterpret_cast<const float2*>(wp + row * F::DIM + x));
                v0 = fmaf(v.x, q, v0), v1 = fmaf(v.y, q, v1), l = fmaf(__ldcg(wp + F::RC * F::DIM + F::RC + row), q, l);
            }
            write_pair(P, en.s, row_of(P, sp, h, group, row0 + row), x, v0, v1, m, l);
        }
    }
}

template <class F>
cudaError_t setup() {
    return cudaFuncSetAttribute(kv_attention_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM);
}

template <class F>
cudaError_t run(const AttnParams& P, int num_sms, cudaStream_t stream) {
    const int grid = num_sms < kMaxCtas ? num_sms : kMaxCtas;
    kv_attention_kernel<F><<<grid, F::THREADS, F::SMEM, stream>>>(P);
    return cudaGetLastError();
}

// Calls fn with the configuration of a call: the row tile that holds the unit's rows, if
// one does, and the arithmetic that the types and the scores ask for.
template <int DIM, class Fn>
cudaError_t with_dim(bool split, bool mod, int rows, Fn fn) {
    const bool one = DIM == 256 || rows <= (split ? 4 : 8);
    constexpr int WIDE = DIM == 256 ? 1 : 2;
    if (split) {
        if (mod) return one ? fn(Cfg<DIM, 1, true, true>()) : fn(Cfg<DIM, WIDE, true, true>());
        return one ? fn(Cfg<DIM, 1, true, false>()) : fn(Cfg<DIM, WIDE, true, false>());
    }
    if (mod) return one ? fn(Cfg<DIM, 1, false, true>()) : fn(Cfg<DIM, WIDE, false, true>());
    return one ? fn(Cfg<DIM, 1, false, false>()) : fn(Cfg<DIM, WIDE, false, false>());
}

}  // namespace

cudaError_t setup_kv_attention() {
    for (int i = 0; i < 8; ++i) {
        auto fn = [](auto f) { return setup<decltype(f)>(); };
        const int rows = i & 4 ? 64 : 1;
        cudaError_t e = with_dim<64>(i & 1, i & 2, rows, fn);
        if (e == cudaSuccess) e = with_dim<128>(i & 1, i & 2, rows, fn);
        if (e == cudaSuccess) e = with_dim<256>(i & 1, i & 2, rows, fn);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Floats of the partial results of any call with this head dimension: two a CTA, 16 rows.
size_t kv_attention_part_floats(int dim) { return (size_t)kMaxCtas * 2 * (dim == 256 ? 8 : 16) * (dim + 2); }

cudaError_t launch_kv_attention(int dim, const AttnParams& P, int num_sms, cudaStream_t stream) {
    const bool split = P.q.type != Q4_BF16 || P.out.type != Q4_BF16, mod = P.softcap > 0.0f || P.alibi;
    const int rows = P.tokens * (P.q_heads / P.cache.heads);
    auto fn = [&](auto f) { return run<decltype(f)>(P, num_sms, stream); };
    if (dim == 64) return with_dim<64>(split, mod, rows, fn);
    if (dim == 128) return with_dim<128>(split, mod, rows, fn);
    return with_dim<256>(split, mod, rows, fn);
}

}  // namespace q4kv
