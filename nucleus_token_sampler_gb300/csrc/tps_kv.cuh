// tps_kv.cuh -- the paged key/value cache: storing tokens (quantised where the cache holds 8-bit
// codes) and reading stored tokens back.
//
// For a (token, head) vector with a = max |x_i| (see tps_kv_format in tps.h):
//   fp8   s = 2^e, e least with a <= 448 2^e; x 2^-e is exact, so the code is e4m3 of the exact quotient
//         and code * s is exact even in bfloat16;
//   int8  s = a / 127 rounded up to bfloat16 (so |x / s| <= 127), code = rint(x / s).
// A group of L lanes handles one vector: 16 bytes of input per 8 bfloat16 components, the group's
// maximum by shuffles, one 16-byte store of codes per 16 components.  Reading is the reverse.  Both
// are one read and one write of every byte, bound by memory (by latency for a decode step's tokens).
#pragma once

#include <cstdint>

#include "tps_decode.h"
#include "tps_device.cuh"

namespace tps {

constexpr int kKvThreads = 256;
constexpr float kMinScale = 0x1p-40f;

// The bfloat16 scale of a vector whose largest magnitude is a (NaN: the vector cannot be stored).
template <int kFormat>
__device__ __forceinline__ float kv_scale(float a)
{
    const uint32_t b = __float_as_uint(a);
    if (b >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    if constexpr (kFormat == TPS_KV_FP8) {
        // a = f 2^x with f in [1/2, 1) and 448 = (7/8) 2^9: e = x - 9, one more if f > 7/8.
        const int e = (int)(b >> 23) - 126 - 9 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        return __uint_as_float((uint32_t)(max(e, -40) + 127) << 23);
    } else {
        const uint32_t s = (__float_as_uint(__fdiv_rn(a, 127.f)) + 0xFFFFu) & 0xFFFF0000u;
        return fmaxf(__uint_as_float(s), kMinScale);
    }
}

// Four codes of x / s, the first in the low byte.  fp8: `inv` = 1 / s is exact.
template <int kFormat>
__device__ __forceinline__ uint32_t kv_codes(const float* x, float s, float inv)
{
    if constexpr (kFormat == TPS_KV_FP8) {
        uint32_t r;
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
            "mov.b32 %0, {lo, hi};\n\t}"
            : "=r"(r)
            : "f"(x[0] * inv), "f"(x[1] * inv), "f"(x[2] * inv), "f"(x[3] * inv));
        return r;
    } else {
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int q = max(-127, min(127, __float2int_rn(__fdiv_rn(x[i], s))));
            r |= ((uint32_t)q & 0xFFu) << (8 * i);
        }
        return r;
    }
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

// 16 components of a vector, by 16-byte accesses where the vectors allow them.
__device__ __forceinline__ void load16(const float* p, bool wide, float (&x)[16])
{
    if (wide) {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + i);
            x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = p[i];
    }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, bool wide, float (&x)[16])
{
    if (wide) {
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
            float y[8];
            Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(p + i), y);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i + j] = y[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __bfloat162float(p[i]);
    }
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

// Vectors of the call: (token, head, k or v), 2 n_heads of them for each token; each by L lanes.
template <typename T, int kFormat>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const KvWriteArgs a, int L, int shift, bool wide)
{
    const tps_kv_cache& c = a.c;
    const int u = threadIdx.x & (L - 1), H = c.n_heads;
    const int64_t n = a.T * 2 * H, total = c.n_pages << shift;
    const int64_t per = kKvThreads / L;
    for (int64_t base = blockIdx.x * per; base < n; base += gridDim.x * per) {
        const int64_t i = base + threadIdx.x / L;
        const int64_t tok = i / (2 * H);
        const int j = (int)(i - tok * 2 * H);
        const bool is_v = j >= H;
        const int h = is_v ? j - H : j;
        const int64_t slot = i < n ? a.slots[tok] : -1;
        const bool on = slot >= 0 && slot < total && u * 16 < c.head_dim;
        float x[16] = {};
        if (on) {
            const T* src = is_v ? static_cast<const T*>(a.v) + tok * a.v_ld + h * a.v_hd
                                : static_cast<const T*>(a.k) + tok * a.k_ld + h * a.k_hd;
            load16(src + u * 16, wide, x);
        }
        if constexpr (kFormat == TPS_KV_BF16) {
            if (on) {
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? c.v : c.k) + kv_row(c, shift, slot, h) * c.head_dim;
                store16(dst + u * 16, x);
            }
        } else {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) m = fmax_nan(m, fabsf(x[k]));
            for (int o = L / 2; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            if (!on) continue;
            const float s = kv_scale<kFormat>(m);
            const float inv = 1.f / s;
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = s == s ? kv_codes<kFormat>(x + 4 * k, s, inv) : 0u;
            const int64_t row = kv_row(c, shift, slot, h);
            uint8_t* dst = static_cast<uint8_t*>(is_v ? c.v : c.k) + row * c.head_dim;
            *reinterpret_cast<uint4*>(dst + u * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            if (u == 0) static_cast<__nv_bfloat16*>(is_v ? c.v_scale : c.k_scale)[row] = __float2bfloat16_rn(s);
        }
    }
}

template <typename T, int kFormat>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvReadArgs a, int L, int shift)
{
    const tps_kv_cache& c = a.c;
    const int u = threadIdx.x & (L - 1), H = c.n_heads;
    const int64_t n = a.T * 2 * H, total = c.n_pages << shift;
    const int64_t per = kKvThreads / L;
    if (u * 16 >= c.head_dim) return;
    for (int64_t i = blockIdx.x * per + threadIdx.x / L; i < n; i += gridDim.x * per) {
        const int64_t tok = i / (2 * H);
        const int j = (int)(i - tok * 2 * H);
        const bool is_v = j >= H;
        const int h = is_v ? j - H : j;
        const int64_t slot = a.slots[tok];
        float x[16] = {};
        if (slot >= 0 && slot < total) {
            const int64_t row = kv_row(c, shift, slot, h);
            if constexpr (kFormat == TPS_KV_BF16) {
                load16(static_cast<const __nv_bfloat16*>(is_v ? c.v : c.k) + row * c.head_dim + u * 16, true, x);
            } else {
                const float s = __bfloat162float(static_cast<const __nv_bfloat16*>(is_v ? c.v_scale : c.k_scale)[row]);
                const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(is_v ? c.v : c.k) +
                                                                row * c.head_dim + u * 16);
                kv_decode<kFormat>(w.x, x);
                kv_decode<kFormat>(w.y, x + 4);
                kv_decode<kFormat>(w.z, x + 8);
                kv_decode<kFormat>(w.w, x + 12);
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] *= s;
            }
        }
        store16(static_cast<T*>(is_v ? a.v : a.k) + (tok * H + h) * c.head_dim + u * 16, x);
    }
}

}  // namespace tps
