// tps_kv.cuh -- the paged key/value cache: storing tokens (quantised where the cache holds 8-bit
// codes) and reading stored tokens back.
//
// For a (token, head) vector with a = max |x_i| (see tps_kv_format in tps.h):
//   fp8   s = 2^e, e least with a <= 448 2^e; x 2^-e is exact, so the code is e4m3 of the exact quotient
//         and code * s is exact even in bfloat16;
//   int8  s = a / 127 rounded up to bfloat16 (so |x / s| <= 127), code = rint(x / s).
// A group of L lanes handles one vector: 16 bytes of input per 8 bfloat16 components, the group's
// maximum by shuffles, one 16-byte store of codes per 16 components.  Reading is the reverse.  Both
// are one read and one write of every byte, bound by memory (by latency for a decode step's tokens): 32,749 tokens x
// 8 heads x 128 are written as int8 in 46 us and read in 42 us, 131,072 read from fp8 in 140 us (5.8 TB/s), 64 tokens
// written and read in 4.9 us.
#pragma once

#include <cstdint>

#include "tps_decode.h"
#include "tps_device.cuh"

namespace tps {

constexpr int kKvThreads = 256;
constexpr float kMinScale = 0x1p-40f;

// The bfloat16 scale of a vector whose largest magnitude has the bits b (NaN: the vector cannot be stored).
template <int kFormat>
__device__ __forceinline__ float kv_scale(uint32_t b)
{
    if (b >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    if constexpr (kFormat == TPS_KV_FP8) {
        // a = f 2^x with f in [1/2, 1) and 448 = (7/8) 2^9: e = x - 9, one more if f > 7/8.
        const int e = (int)(b >> 23) - 126 - 9 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        return __uint_as_float((uint32_t)(max(e, -40) + 127) << 23);
    } else {
        const uint32_t s = (__float_as_uint(__fdiv_rn(__uint_as_float(b), 127.f)) + 0xFFFFu) & 0xFFFF0000u;
        return fmaxf(__uint_as_float(s), kMinScale);
    }
}

// Sixteen codes of x / s, four to a word and the first in the low byte; inv = 1 / s (exact for fp8).
template <int kFormat>
__device__ __forceinline__ uint4 kv_codes(const float (&x)[16], float s, float inv)
{
    uint32_t w[4];
    if constexpr (kFormat == TPS_KV_FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("{\n\t.reg .b16 lo, hi;\n\t"
                "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
                "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
                "mov.b32 %0, {lo, hi};\n\t}"
                : "=r"(w[i])
                : "f"(x[4 * i] * inv), "f"(x[4 * i + 1] * inv), "f"(x[4 * i + 2] * inv), "f"(x[4 * i + 3] * inv));
    } else {
        // rint(x / s).  Ties are common (the quotient of two bfloat16 numbers), so the quotient has to be exact
        // there: Markstein's correction (IBM Journal of Research and Development 34, 1990) makes the correctly
        // rounded quotient of the product with the correctly rounded reciprocal, its exact remainder and one more
        // step.  Adding 1.5 * 2^23 then rounds to the nearest whole number, ties to even, and leaves it in the low
        // bits.  Four full-rate operations, where a division for each component took the write of 32,749 tokens
        // from 46 to 80 us.
        constexpr float kMagic = 12582912.f;
        uint32_t b[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float q = x[i] * inv, r = fmaf(-q, s, x[i]);
            b[i] = __float_as_uint(__fadd_rn(fmaf(r, inv, q), kMagic));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040u), __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040u), 0x5410u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Four values of a word of codes, before the scale.
template <int kFormat>
__device__ __forceinline__ void kv_decode(uint32_t w, float* x)
{
    if constexpr (kFormat == TPS_KV_FP8) {
        uint32_t lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        x[0] = p.x, x[1] = p.y, x[2] = q.x, x[3] = q.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
    }
}

// 16 components of a vector as they lie in memory (32 or 64 bytes), by 16-byte accesses where the vectors
// allow them; and their values.
template <typename T, bool kWide>
__device__ __forceinline__ void load_raw(const T* p, uint4 (&w)[sizeof(T)])
{
    if constexpr (kWide) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    } else if constexpr (sizeof(T) == 4) {
        const uint32_t* x = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
        const uint16_t* x = reinterpret_cast<const uint16_t*>(p);
        auto pair = [&](int i) { return (uint32_t)x[i] | (uint32_t)x[i + 1] << 16; };
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = make_uint4(pair(8 * i), pair(8 * i + 2), pair(8 * i + 4), pair(8 * i + 6));
    }
}
template <typename T>
__device__ __forceinline__ void values_of(const uint4 (&w)[sizeof(T)], float (&x)[16])
{
    constexpr int N = 16 / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) {
        float y[N];
        Elem<T>::unpack(w[i], y);
#pragma unroll
        for (int j = 0; j < N; ++j) x[i * N + j] = y[j];
    }
}
// The bits of the largest magnitude among them.  Magnitudes order like their bits, NaN above everything.
template <typename T>
__device__ __forceinline__ uint32_t magnitude_of(const uint4 (&w)[sizeof(T)])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = sizeof(T) == 4 ? max(m, x[j] & 0x7FFFFFFFu) : __vmaxu2(m, x[j] & 0x7FFF7FFFu);
    }
    return sizeof(T) == 4 ? m : max(m & 0xFFFF0000u, m << 16);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store16(float* p, const float (&x)[16])
{
#pragma unroll
    for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[16])
{
#pragma unroll
    for (int i = 0; i < 16; i += 8)
        *reinterpret_cast<uint4*>(p + i) = make_uint4(bf16_pair(x[i], x[i + 1]), bf16_pair(x[i + 2], x[i + 3]),
                                                      bf16_pair(x[i + 4], x[i + 5]), bf16_pair(x[i + 6], x[i + 7]));
}

// Row of slot s and head h in the code and scale arrays.
__device__ __forceinline__ int64_t kv_row(const tps_kv_cache& c, int shift, int64_t s, int h)
{
    return ((((s >> shift) * c.n_heads + h) << shift) | (s & (c.page_size - 1)));
}

// A vector of the call: j of the 2 n_heads (keys, then values) of a token; L lanes for each of them.  Going
// `stride` vectors on takes no division.
struct KvVector {
    int64_t tok;
    int j;
};
struct KvStep {
    int64_t tok;
    int j, per;
    __device__ __forceinline__ KvStep(int64_t stride, int heads) : per(2 * heads)
    {
        tok = (uint32_t)stride / (uint32_t)per;  // the grid is small: 32 bits
        j = (int)(stride - tok * per);
    }
    __device__ __forceinline__ KvVector first(int64_t i) const
    {
        const int64_t t = (uint32_t)i / (uint32_t)per;
        return KvVector{t, (int)(i - t * per)};
    }
    __device__ __forceinline__ void go(KvVector& v) const
    {
        v.tok += tok;
        v.j += j;
        if (v.j >= per) v.j -= per, ++v.tok;
    }
};

// Vectors that a group of lanes has in hand at once: a vector's slot, its data and its scale are read one
// after the other, so one vector at a time would leave the memory idle.
constexpr int kKvFlight = 4;

template <typename T, int kFormat, bool kWide>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const KvWriteArgs a, int L, int shift)
{
    constexpr int U = sizeof(T) == 2 ? kKvFlight : kKvFlight / 2;
    const tps_kv_cache& c = a.c;
    const int u = threadIdx.x & (L - 1), H = c.n_heads;
    const int64_t total = c.n_pages << shift;
    const int per = kKvThreads / L;
    const KvStep step((int64_t)gridDim.x * per, H);
    KvVector at = step.first((int64_t)blockIdx.x * per + threadIdx.x / L);
    const bool mine = u * 16 < c.head_dim;
    // whole warps go round together (the maximum needs every lane)
    for (int64_t base = (int64_t)blockIdx.x * per; base < a.T * 2 * H; base += (int64_t)gridDim.x * per * U) {
        int64_t slot[U];
        KvVector vec[U];
        uint4 raw[U][sizeof(T)];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            vec[k] = at;
            slot[k] = at.tok < a.T && mine ? a.slots[at.tok] : -1;
            step.go(at);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const bool is_v = vec[k].j >= H;
            const int h = is_v ? vec[k].j - H : vec[k].j;
            const T* src = is_v ? static_cast<const T*>(a.v) + vec[k].tok * a.v_ld + h * a.v_hd
                                : static_cast<const T*>(a.k) + vec[k].tok * a.k_ld + h * a.k_hd;
#pragma unroll
            for (int j = 0; j < (int)sizeof(T); ++j) raw[k][j] = make_uint4(0u, 0u, 0u, 0u);
            if (slot[k] >= 0 && slot[k] < total) load_raw<T, kWide>(src + u * 16, raw[k]);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const bool on = slot[k] >= 0 && slot[k] < total, is_v = vec[k].j >= H;
            const int h = is_v ? vec[k].j - H : vec[k].j;
            const int64_t row = kv_row(c, shift, slot[k], h);
            if constexpr (kFormat == TPS_KV_BF16) {
                if (!on) continue;
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? c.v : c.k) + row * c.head_dim + u * 16;
                if constexpr (sizeof(T) == 2) {
                    reinterpret_cast<uint4*>(dst)[0] = raw[k][0];
                    reinterpret_cast<uint4*>(dst)[1] = raw[k][1];
                } else {
                    float x[16];
                    values_of<T>(raw[k], x);
                    store16(dst, x);
                }
            } else {
                uint32_t m = magnitude_of<T>(raw[k]);
                for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                if (!on) continue;
                float x[16];
                values_of<T>(raw[k], x);
                const float s = kv_scale<kFormat>(m);
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (s == s) w = kv_codes<kFormat>(x, s, 1.f / s);
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(is_v ? c.v : c.k) + row * c.head_dim + u * 16) = w;
                if (u == 0) static_cast<__nv_bfloat16*>(is_v ? c.v_scale : c.k_scale)[row] = __float2bfloat16_rn(s);
            }
        }
    }
}

template <typename T, int kFormat>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvReadArgs a, int L, int shift)
{
    constexpr int U = kKvFlight;
    const tps_kv_cache& c = a.c;
    const int u = threadIdx.x & (L - 1), H = c.n_heads;
    const int64_t total = c.n_pages << shift;
    const int per = kKvThreads / L;
    const KvStep step((int64_t)gridDim.x * per, H);
    KvVector at = step.first((int64_t)blockIdx.x * per + threadIdx.x / L);
    if (u * 16 >= c.head_dim) return;
    while (at.tok < a.T) {
        int64_t slot[U];
        KvVector vec[U];
        uint4 w[U][kFormat == TPS_KV_BF16 ? 2 : 1];
        float s[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            vec[k] = at;
            slot[k] = at.tok < a.T ? a.slots[at.tok] : -1;
            step.go(at);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const bool on = slot[k] >= 0 && slot[k] < total, is_v = vec[k].j >= H;
            const int64_t row = on ? kv_row(c, shift, slot[k], is_v ? vec[k].j - H : vec[k].j) : 0;
            s[k] = 1.f;
            if constexpr (kFormat == TPS_KV_BF16) {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(is_v ? c.v : c.k) + row * c.head_dim + u * 16);
                w[k][0] = on ? src[0] : make_uint4(0u, 0u, 0u, 0u);
                w[k][1] = on ? src[1] : make_uint4(0u, 0u, 0u, 0u);
            } else {
                w[k][0] = on ? *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(is_v ? c.v : c.k) + row * c.head_dim + u * 16)
                             : make_uint4(0u, 0u, 0u, 0u);
                if (on) s[k] = __bfloat162float(static_cast<const __nv_bfloat16*>(is_v ? c.v_scale : c.k_scale)[row]);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (vec[k].tok >= a.T) break;
            float x[16];
            if constexpr (kFormat == TPS_KV_BF16) {
                float y[8];
                Elem<__nv_bfloat16>::unpack(w[k][0], y);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = y[j];
                Elem<__nv_bfloat16>::unpack(w[k][1], y);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[8 + j] = y[j];
            } else {
                kv_decode<kFormat>(w[k][0].x, x);
                kv_decode<kFormat>(w[k][0].y, x + 4);
                kv_decode<kFormat>(w[k][0].z, x + 8);
                kv_decode<kFormat>(w[k][0].w, x + 12);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] *= s[k];
            }
            const bool is_v = vec[k].j >= H;
            store16(static_cast<T*>(is_v ? a.v : a.k) + (vec[k].tok * H + (is_v ? vec[k].j - H : vec[k].j)) * c.head_dim + u * 16, x);
        }
    }
}

}  // namespace tps
