// tps_norm_rope.cuh -- root-mean-square norm of each query and key head and the rotation by the
// token's position, in one pass: y = x rsqrt(mean(x^2) + eps) w over the D components of a head, then
// (a, b) -> (a cos - b sin, b cos + a sin) on the first `rot` components.  About 8 operations for each
// element read and written: memory alone bounds it, and for a decode step's few tokens the latency of
// one read and one write.
//
// CTAs walk over the tokens.  A group of L lanes (a power of two) holds one head; a lane's unit is a pair of
// 16-byte vectors whose elements rotate with each other, so a rotation needs no other lane: for
// halves the vectors at u and rot/2 + u, for adjacent pairs two neighbours.  The cosines and sines of a
// lane's unit are the same for every head, so each lane loads them once per token and walks over the
// heads.  16,383 tokens x 40 heads x 128 in bfloat16 take 66 us (5.2 TB/s, 76% of a plain copy's rate), 8
// tokens 2.4 us.  Shapes that do not split into such units (head sizes or strides off 16 bytes) take one
// warp per head and scalar accesses.
#pragma once

#include <cstdint>
#include <type_traits>

#include "tps_decode.h"
#include "tps_device.cuh"

namespace tps {

constexpr int kNormMaxThreads = 256;

template <typename T> struct Pack;  // a 16-byte vector of T
template <> struct Pack<float> {
    static constexpr int kN = 4;
    __device__ __forceinline__ static void load(const float* p, float (&x)[kN])
    {
        const float4 v = *reinterpret_cast<const float4*>(p);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    }
    __device__ __forceinline__ static void store(float* p, const float (&x)[kN])
    {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <> struct Pack<__nv_bfloat16> {
    static constexpr int kN = 8;
    __device__ __forceinline__ static void load(const __nv_bfloat16* p, float (&x)[kN])
    {
        Elem<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4*>(p), x);
    }
    __device__ __forceinline__ static void store(__nv_bfloat16* p, const float (&x)[kN])
    {
        uint4 v;
        uint32_t* w = &v.x;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        *reinterpret_cast<uint4*>(p) = v;
    }
};

template <int N>
__device__ __forceinline__ void load_floats(const float* p, float (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + i);
        x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
    }
}

// kWhole: every component turns (rot = D), which saves the question 2% at 16,383 tokens (66.1 / 67.4 us).
template <typename T, int L, bool kInterleaved, bool kWhole, int kWalks>
__global__ void __launch_bounds__(kNormMaxThreads) norm_rope_kernel(const tps_norm_rope a)
{
    constexpr int N = Pack<T>::kN;
    const int u = threadIdx.x % L, groups = blockDim.x / L, group = threadIdx.x / L;
    const int rot = a.rot_dim, half = rot / 2, D = a.head_dim;
    const int units = D / (2 * N), turning = rot / (2 * N);
    const bool live = u < units, turn = kWhole || u < turning;
    int ia, ib;  // the unit's two vectors
    if (turn) {
        ia = kInterleaved ? u * 2 * N : u * N;
        ib = kInterleaved ? ia + N : half + u * N;
    } else {
        ia = rot + (u - turning) * 2 * N;
        ib = ia + N;
    }
    const int H = a.n_q_heads + a.n_k_heads;
    const float inv_d = 1.f / (float)D, nan = __int_as_float(0x7FC00000);
    // kWalks heads of each group at a time; the next ones (the next token's after a token's last) are asked for
    // before the present ones are worked on.
    uint4 xa[kWalks], xb[kWalks];
    auto ask = [&](int64_t tok, int h0) {
#pragma unroll
        for (int k = 0; k < kWalks; ++k) {
            const int h = h0 + k * groups + group;
            const bool is_q = h < a.n_q_heads, on = live && h < H && tok < a.T;
            const int hh = is_q ? h : h - a.n_q_heads;
            const T* src = is_q ? static_cast<const T*>(a.q) + tok * a.q_ld + hh * a.q_hd
                                : static_cast<const T*>(a.k) + tok * a.k_ld + hh * a.k_hd;
            xa[k] = on ? *reinterpret_cast<const uint4*>(src + ia) : make_uint4(0u, 0u, 0u, 0u);
            xb[k] = on ? *reinterpret_cast<const uint4*>(src + ib) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    int64_t tok = blockIdx.x;
    int pos = a.positions[tok];
    ask(tok, 0);
    for (; tok < a.T; tok += gridDim.x) {
        const int64_t next_tok = tok + gridDim.x;
        const bool known = pos >= 0 && (int64_t)pos < a.n_positions;
        if (threadIdx.x == 0 && a.out_status) a.out_status[tok] = known ? TPS_ROW_OK : TPS_ROW_BAD_PARAM;
        // halves: element j of the two vectors turns by angle u N + j; adjacent: elements 2j, 2j + 1 of the
        // pair of vectors by angle u N + j.  Either way the unit uses angles [u N, u N + N).
        float c[N], s[N];
        if (turn && live && known) {
            load_floats<N>(a.cos_sin + (int64_t)pos * rot + u * N, c);
            load_floats<N>(a.cos_sin + (int64_t)pos * rot + half + u * N, s);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) c[j] = 1.f, s[j] = 0.f;
        }
        if (next_tok < a.T) pos = a.positions[next_tok];
        for (int h0 = 0; h0 < H; h0 += groups * kWalks) {
            uint4 va[kWalks], vb[kWalks];
#pragma unroll
            for (int k = 0; k < kWalks; ++k) va[k] = xa[k], vb[k] = xb[k];
            if (h0 + groups * kWalks < H)
                ask(tok, h0 + groups * kWalks);
            else
                ask(next_tok, 0);
#pragma unroll
            for (int k = 0; k < kWalks; ++k) {
                const int h = h0 + k * groups + group;
                const bool is_q = h < a.n_q_heads;
                const int hh = is_q ? h : h - a.n_q_heads;
                float x[N], y[N];
                Elem<T>::unpack(va[k], x);
                Elem<T>::unpack(vb[k], y);
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < N; ++j) ss = fmaf(x[j], x[j], fmaf(y[j], y[j], ss));
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                if (!live || h >= H) continue;
                const float r = known ? rsqrtf(fmaf(ss, inv_d, a.eps)) : nan;
                const float* w = is_q ? a.q_weight : a.k_weight;
                if (w) {
                    float wa[N], wb[N];
                    load_floats<N>(w + ia, wa);
                    load_floats<N>(w + ib, wb);
#pragma unroll
                    for (int j = 0; j < N; ++j) x[j] *= r * wa[j], y[j] *= r * wb[j];
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) x[j] *= r, y[j] *= r;
                }
                if (!turn) {
                    // as they are: through a product with sine 0 an infinity would reach its partner as NaN
                } else if (kInterleaved) {
#pragma unroll
                    for (int j = 0; j < N; j += 2) {  // pairs inside each vector
                        const float x0 = x[j], y0 = y[j];
                        const int i = j / 2, m = N / 2 + j / 2;
                        x[j] = x0 * c[i] - x[j + 1] * s[i];
                        x[j + 1] = x[j + 1] * c[i] + x0 * s[i];
                        y[j] = y0 * c[m] - y[j + 1] * s[m];
                        y[j + 1] = y[j + 1] * c[m] + y0 * s[m];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float x0 = x[j];
                        x[j] = x0 * c[j] - y[j] * s[j];
                        y[j] = y[j] * c[j] + x0 * s[j];
                    }
                }
                T* dst = is_q ? static_cast<T*>(a.out_q) + tok * a.oq_ld + hh * a.oq_hd
                              : static_cast<T*>(a.out_k) + tok * a.ok_ld + hh * a.ok_hd;
                Pack<T>::store(dst + ia, x);
                Pack<T>::store(dst + ib, y);
            }
        }
    }
}

__device__ __forceinline__ float scalar_load(const float* p) { return *p; }
__device__ __forceinline__ float scalar_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void scalar_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void scalar_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Any head size and stride: one warp per head, a pair of components per lane and step.
template <typename T>
__global__ void __launch_bounds__(kNormMaxThreads) norm_rope_any_kernel(const tps_norm_rope a)
{
    const int64_t tok = blockIdx.x;
    const int lane = threadIdx.x & 31, H = a.n_q_heads + a.n_k_heads;
    const int rot = a.rot_dim, half = rot / 2, D = a.head_dim;
    const int pos = a.positions[tok];
    const bool known = pos >= 0 && (int64_t)pos < a.n_positions;
    if (threadIdx.x == 0 && a.out_status) a.out_status[tok] = known ? TPS_ROW_OK : TPS_ROW_BAD_PARAM;
    const float nan = __int_as_float(0x7FC00000);
    const float* cs = a.cos_sin + (known ? (int64_t)pos * rot : 0);
    for (int h = threadIdx.x >> 5; h < H; h += blockDim.x >> 5) {
        const bool is_q = h < a.n_q_heads;
        const int hh = is_q ? h : h - a.n_q_heads;
        const T* src = is_q ? static_cast<const T*>(a.q) + tok * a.q_ld + hh * a.q_hd
                            : static_cast<const T*>(a.k) + tok * a.k_ld + hh * a.k_hd;
        T* dst = is_q ? static_cast<T*>(a.out_q) + tok * a.oq_ld + hh * a.oq_hd
                      : static_cast<T*>(a.out_k) + tok * a.ok_ld + hh * a.ok_hd;
        const float* w = is_q ? a.q_weight : a.k_weight;
        float ss = 0.f;
        for (int i = lane; i < D; i += 32) {
            const float x = scalar_load(src + i);
            ss = fmaf(x, x, ss);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float r = known ? rsqrtf(ss / (float)D + a.eps) : nan;
        for (int p = lane; p < half; p += 32) {
            const int i = a.interleaved ? 2 * p : p, j = a.interleaved ? 2 * p + 1 : p + half;
            const float x = scalar_load(src + i) * r * (w ? w[i] : 1.f);
            const float y = scalar_load(src + j) * r * (w ? w[j] : 1.f);
            const float c = known ? cs[p] : nan, s = known ? cs[half + p] : nan;
            scalar_store(dst + i, x * c - y * s);
            scalar_store(dst + j, y * c + x * s);
        }
        for (int i = rot + lane; i < D; i += 32) scalar_store(dst + i, scalar_load(src + i) * r * (w ? w[i] : 1.f));
    }
}

}  // namespace tps
