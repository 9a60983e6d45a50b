// tps_attn_rows.cuh -- attention of up to 16 query rows per warp over paged keys and values, and the
// join of its parts: every sequence's own tokens, and the shared prefix where the batch has too few
// rows for the tcgen05 kernel.
//
// Mathematics.  With z_j = scale log2(e) q.k_j, one pass over the tokens holds a reference m, the sum
// l = sum 2^(z_j - m) and the output o = sum 2^(z_j - m) v_j in float32; m is raised (and l, o scaled)
// only when some z exceeds it by more than 2^kSlack, so that in most steps nothing is scaled and no
// maximum has to be agreed on between lanes.  Parts of a row (warps, CTAs, prefix and own tokens) join as
// m = max m_i, l = sum l_i 2^(m_i - m), o likewise.
// For 8-bit formats the codes go to the matrix instruction as they are (exact in float16) and the
// scales stay outside, in float32: z_j carries the key's scale, and with t_j = z_j + log2(s_j) the weight
// 2^(t_j - m) already holds the value's scale s_j; l adds 2^(t_j - m) / s_j.  The weights are float16
// with 11 bits, lifted by 2^kLift so that tokens down to 2^-(24 + kLift) of the largest still count.
//
// What bounds it: the bytes of the keys and values.  So there is no staging: each lane loads 16 bytes
// of keys and of values straight into the registers that feed mma.sync m16n8k16.  The product q.k is the
// same for any order of the D components, so a lane's 16 bytes of a key row serve as its fragments of
// consecutive k-steps as they lie, and the query fragments are loaded in the same order; likewise the
// columns of the output are renumbered so that a lane's 16 bytes of a value row are one column each of
// consecutive tiles.  Keys for the next step are requested as soon as the present ones are used, values
// likewise; four warps of a CTA take 16 tokens in turn and several CTAs share an SM.
// mma.sync rather than tcgen05: the 16 rows fill a sixteenth of a tcgen05 tile's 128 or more.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "tps_decode.h"
#include "tps_device.cuh"

namespace tps {

constexpr int kRowsThreads = 128;
constexpr int kRowsWarps = kRowsThreads / 32;
constexpr float kSlack = 8.f;  // base-2 units a score may exceed the reference by
constexpr float kLift = 7.f;   // float16 weights are lifted by 2^7: at most 2^15

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float log2_fast(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool half)
{
    if (half)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two codes to float16 (the low half first).  fp8: the two bytes of `w`'s low half.  int8: bytes that
// were already biased by 128; 0x6400 + b is the float16 1024 + b.
__device__ __forceinline__ uint32_t fp8_pair(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t int8_pair(uint32_t biased, uint32_t selector)
{
    const uint32_t p = __byte_perm(biased, 0x64646464u, selector);
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(p), "r"(0x64806480u));  // minus 1152
    return r;
}

// Bytes 0, 1 and bytes 2, 3 of a word of codes as float16 pairs.
template <int kFormat>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t& p01, uint32_t& p23)
{
    if constexpr (kFormat == TPS_KV_FP8) {
        p01 = fp8_pair(w);
        p23 = fp8_pair(w >> 16);
    } else {
        const uint32_t b = w ^ 0x80808080u;
        p01 = int8_pair(b, 0x4140u);
        p23 = int8_pair(b, 0x4342u);
    }
}

// The value's scale and the factors a token's score and weight take from it.  A stored scale is never 0;
// 0 marks a slot that was never written and counts as the smallest scale.
__device__ __forceinline__ float floor_scale(float s) { return s > 0.f || s != s ? s : 0x1p-40f; }

// Query rows of a warp: row i of the 16 is query row row0 + i of the tile's `rows`.
// Fragments hold 4 consecutive components from kstep_base(s, quad) on for k-step s.
template <int kFormat>
__device__ __forceinline__ int kstep_base(int s, int quad)
{
    return kFormat == TPS_KV_BF16 ? (s >> 1) * 32 + quad * 8 + (s & 1) * 4 : (s >> 2) * 64 + quad * 16 + (s & 3) * 4;
}

// A power of two that brings a row whose largest finite magnitude is `a` into float16's range, 1 for
// magnitudes in [2^-2, 2^15).  bfloat16 has 8 significant bits, so the components are exact in float16
// down to 2^-17; below that they are rounded to multiples of 2^-24, 2^-23 of the row's largest at most.
__device__ __forceinline__ float f16_row_scale(float a)
{
    const int e = (int)((__float_as_uint(a) >> 23) & 0xFF) - 127;
    if (e >= 128 || a == 0.f || (e <= 14 && e >= -2)) return 1.f;
    return __uint_as_float((uint32_t)min(max(127 - e, 1), 254) << 23);  // brings it to [1, 2)
}

template <int D, int kFormat> struct RowState {
    static constexpr int kSteps = D / 16;   // k-steps of q.k
    static constexpr int kTiles = D / 8;    // 8-column tiles of the output
    uint32_t q[kSteps][4];
    float o[kTiles][4];
    float m[2], l[2];  // rows g and g + 8: reference (agreed on by the quad) and this lane's part of the sum
    float unscale[2];  // what the row's float16 scaling has to be undone by, times scale log2(e)
};

// Load the fragments of the 16 query rows at `q` (row stride in elements; rows past `rows` are zero).
template <int D, int kFormat, typename RowPtr>
__device__ __forceinline__ void load_query(RowState<D, kFormat>& st, int rows, float qk_scale, RowPtr row_ptr)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = g + 8 * r;
        float amax = 0.f;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            uint2 w = make_uint2(0u, 0u);
            if (row < rows) w = *reinterpret_cast<const uint2*>(row_ptr(row) + kstep_base<kFormat>(s, quad));
            st.q[s][r] = w.x;
            st.q[s][2 + r] = w.y;
            if (kFormat != TPS_KV_BF16) {
                const float x[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                                    __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u)};
#pragma unroll
                for (int i = 0; i < 4; ++i) amax = fabsf(x[i]) < __int_as_float(0x7F800000) ? fmaxf(amax, fabsf(x[i])) : amax;
            }
        }
        st.unscale[r] = qk_scale;
        if (kFormat != TPS_KV_BF16) {
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            const float f = f16_row_scale(amax);
            st.unscale[r] = qk_scale / f;
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const uint32_t w = st.q[s][i + r];
                    const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
                    st.q[s][i + r] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
        }
        st.m[r] = -__int_as_float(0x7F800000);
        st.l[r] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < D / 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.o[t][i] = 0.f;
}

// Where the tokens lie: `pages` lists the pages of one head's tokens in order.
struct PageList {
    const int32_t* pages;
    int64_t n_pages;
    int shift, head, heads;
    // First row of the 16-token chunk that starts at token t (a multiple of 16), or -1 for a bad page.
    __device__ __forceinline__ int64_t row(int64_t t) const
    {
        const int64_t p = pages[t >> shift];
        return (p < 0 || p >= n_pages) ? -1 : ((p * heads + head) << shift) + (t & ((1 << shift) - 1));
    }
};

// Walk over the 16-token chunks first, first + step, ... below `last` tokens; row r of the warp's rows
// g and g + 8 sees the tokens below lim[r].  Returns whether every page was a page of the cache.
template <int D, int kFormat>
__device__ __forceinline__ bool attend(RowState<D, kFormat>& st, const tps_kv_cache& c, const PageList& list, int64_t first,
                                       int64_t step, int64_t last, const int64_t (&lim)[2])
{
    constexpr bool k8 = kFormat != TPS_KV_BF16;
    constexpr int kRowBytes = k8 ? D : 2 * D;
    constexpr int kKeyLoads = kRowBytes / 64;             // 16-byte loads of one key row by its quad's lane
    constexpr int kValWords = kRowBytes / 32;             // words of one value row held by a lane
    constexpr int kCols = D / 8;                          // columns of a value row held by a lane
    const int lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
    const float neg = -__int_as_float(0x7F800000);
    if (first >= last) return true;

    bool good = true;
    uint4 kreg[2][kKeyLoads];
    uint32_t vreg[4][kValWords];
    uint32_t ks[2] = {}, vs[2] = {};
    const char* kbase = static_cast<const char*>(c.k);
    const char* vbase = static_cast<const char*>(c.v);

    auto load_keys = [&](int64_t t0, int64_t row) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const bool in = t0 + n * 8 + g < last;
#pragma unroll
            for (int j = 0; j < kKeyLoads; ++j)
                kreg[n][j] = in ? *reinterpret_cast<const uint4*>(kbase + (row + n * 8 + g) * kRowBytes + j * 64 + quad * 16)
                                : make_uint4(0u, 0u, 0u, 0u);
            if (k8) {
                // the pair of tokens whose columns this lane holds; a chunk lies in one page, so both rows exist
                ks[n] = *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(c.k_scale) + row + n * 8 + quad * 2);
            }
        }
    };
    auto load_values = [&](int64_t t0, int64_t row) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = (i >> 1) * 8 + quad * 2 + (i & 1);
            const bool in = t0 + tok < last;
            const char* p = vbase + (row + tok) * kRowBytes + g * kValWords * 4;
            if (kValWords == 2) {
                const uint2 w = in ? *reinterpret_cast<const uint2*>(p) : make_uint2(0u, 0u);
                vreg[i][0] = w.x, vreg[i][1] = w.y;
            } else {
#pragma unroll
                for (int j = 0; j < kValWords; j += 4) {
                    const uint4 w = in ? *reinterpret_cast<const uint4*>(p + j * 4) : make_uint4(0u, 0u, 0u, 0u);
                    vreg[i][j] = w.x, vreg[i][(j + 1) % kValWords] = w.y, vreg[i][(j + 2) % kValWords] = w.z,
                    vreg[i][(j + 3) % kValWords] = w.w;
                }
            }
        }
        if (k8) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
                vs[n] = *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(c.v_scale) + row + n * 8 + quad * 2);
        }
    };

    int64_t row = list.row(first);
    if (row < 0) good = false, row = 0;
    load_keys(first, row);
    load_values(first, row);
    for (int64_t t0 = first; t0 < last; t0 += step) {
        const int64_t tn = t0 + step;
        int64_t next = row;
        if (tn < last) {
            next = list.row(tn);
            if (next < 0) good = false, next = 0;
        }
        float z[2][4] = {};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < kKeyLoads; ++j) {
                const uint32_t w[4] = {kreg[n][j].x, kreg[n][j].y, kreg[n][j].z, kreg[n][j].w};
                if (k8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t b0, b1;
                        code_pairs<kFormat>(w[i], b0, b1);
                        mma16816(z[n], st.q[j * 4 + i], b0, b1, true);
                    }
                } else {
                    mma16816(z[n], st.q[j * 2 % (D / 16)], w[0], w[1], false);
                    mma16816(z[n], st.q[(j * 2 + 1) % (D / 16)], w[2], w[3], false);
                }
            }
        // Scores in base-2 units, with the value's scale folded in; columns n * 8 + quad * 2 + {0, 1}.
        float inv_s[2][2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float kf = 1.f, add = 0.f;
                if (k8) {
                    kf = floor_scale(__uint_as_float(e ? ks[n] & 0xFFFF0000u : ks[n] << 16));
                    const float s = floor_scale(__uint_as_float(e ? vs[n] & 0xFFFF0000u : vs[n] << 16));
                    add = log2_fast(s);
                    inv_s[n][e] = s == s ? __fdividef(1.f, s) : 1.f;  // NaN reaches the weight through `add` where it is seen
                }
                const int64_t tok = t0 + n * 8 + quad * 2 + e;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float& x = z[n][r * 2 + e];
                    x = k8 ? fmaf(x * kf, st.unscale[r], add) : x * st.unscale[r];
                    if (tok >= lim[r]) x = neg;
                }
            }
        }
        if (tn < last) load_keys(tn, next);
        // Raise the references where a score exceeds them by more than the slack (or is the first one).
        const float top0 = fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[1][0], z[1][1]));
        const float top1 = fmaxf(fmaxf(z[0][2], z[0][3]), fmaxf(z[1][2], z[1][3]));
        if (__any_sync(0xFFFFFFFFu, top0 > st.m[0] + kSlack || top1 > st.m[1] + kSlack)) {
            const float top[2] = {top0, top1};
            float f[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float t = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 1));
                t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
                const float m = t > st.m[r] + kSlack ? t : st.m[r];
                f[r] = m == st.m[r] ? 1.f : exp2_fast(st.m[r] - m);
                st.m[r] = m;
                st.l[r] *= f[r];
            }
#pragma unroll
            for (int t = 0; t < D / 8; ++t) {
                st.o[t][0] *= f[0], st.o[t][1] *= f[0];
                st.o[t][2] *= f[1], st.o[t][3] *= f[1];
            }
        }
        uint32_t p[4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float ref = st.m[r] == neg ? 0.f : st.m[r];  // nothing seen yet: every weight is 0
                const float w0 = exp2_fast(z[n][r * 2] - ref + (k8 ? kLift : 0.f));
                const float w1 = exp2_fast(z[n][r * 2 + 1] - ref + (k8 ? kLift : 0.f));
                if (k8) {
                    st.l[r] = fmaf(w0, inv_s[n][0], fmaf(w1, inv_s[n][1], st.l[r]));
                    const __half2 h = __floats2half2_rn(w0, w1);
                    p[n * 2 + r] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    st.l[r] += w0 + w1;
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[n * 2 + r]) : "f"(w1), "f"(w0));
                }
            }
#pragma unroll
        for (int w = 0; w < kValWords; ++w) {
            if (k8) {
                // bytes of tokens (0, 1) and (2, 3) side by side: columns 4w .. 4w + 3
                uint32_t a = vreg[0][w], b = vreg[1][w], cc = vreg[2][w], d = vreg[3][w];
                if (kFormat == TPS_KV_INT8) a ^= 0x80808080u, b ^= 0x80808080u, cc ^= 0x80808080u, d ^= 0x80808080u;
                const uint32_t ab01 = __byte_perm(a, b, 0x5140u), ab23 = __byte_perm(a, b, 0x7362u);
                const uint32_t cd01 = __byte_perm(cc, d, 0x5140u), cd23 = __byte_perm(cc, d, 0x7362u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x = i < 2 ? ab01 : ab23, y = i < 2 ? cd01 : cd23;
                    uint32_t b0, b1;
                    if (kFormat == TPS_KV_FP8) {
                        b0 = fp8_pair((i & 1) ? x >> 16 : x);
                        b1 = fp8_pair((i & 1) ? y >> 16 : y);
                    } else {
                        b0 = int8_pair(x, (i & 1) ? 0x4342u : 0x4140u);
                        b1 = int8_pair(y, (i & 1) ? 0x4342u : 0x4140u);
                    }
                    mma16816(st.o[(w * 4 + i) % kCols], p, b0, b1, true);
                }
            } else {
                mma16816(st.o[(w * 2) % kCols], p, __byte_perm(vreg[0][w], vreg[1][w], 0x5410u),
                         __byte_perm(vreg[2][w], vreg[3][w], 0x5410u), false);
                mma16816(st.o[(w * 2 + 1) % kCols], p, __byte_perm(vreg[0][w], vreg[1][w], 0x7632u),
                         __byte_perm(vreg[2][w], vreg[3][w], 0x7632u), false);
            }
        }
        if (tn < last) load_values(tn, next);
        row = next;
    }
    return good;
}

// The CTA's rows after its warps have joined: unnormalised output, reference and sum.
template <int D> struct RowsShared {
    float o[kRowsWarps][16][D];
    float m[kRowsWarps][16], l[kRowsWarps][16];
    int bad;
};

// Put a warp's rows into shared memory in natural column order (a lane's columns are g_col * D/8 + tile
// for the two columns 2 quad, 2 quad + 1 of each tile).
template <int D, int kFormat>
__device__ __forceinline__ void store_rows(RowsShared<D>& sm, RowState<D, kFormat>& st)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float l = st.l[r];
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
        if (quad == 0) {
            sm.m[warp][g + 8 * r] = st.m[r];
            sm.l[warp][g + 8 * r] = l;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float* dst = &sm.o[warp][g + 8 * r][(quad * 2 + e) * (D / 8)];
#pragma unroll
            for (int t = 0; t < D / 8; t += 4)
                *reinterpret_cast<float4*>(dst + t) = make_float4(st.o[t][r * 2 + e], st.o[t + 1][r * 2 + e],
                                                                  st.o[t + 2][r * 2 + e], st.o[t + 3][r * 2 + e]);
        }
    }
}

// Weight of a part with reference m in a join whose reference is `top` (0 for a part without tokens).
__device__ __forceinline__ float join_weight(float m, float top)
{
    return m == -__int_as_float(0x7F800000) ? 0.f : exp2_fast(m - top);
}

// The shared prefix, 16 rows at a time: CTA c's part of the line of blocks (AttnPlan).
template <int D, int kFormat>
__global__ void __launch_bounds__(kRowsThreads) attn_prefix_rows_kernel(const AttnArgs a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    RowsShared<D>& sm = *reinterpret_cast<RowsShared<D>*>(raw);
    const AttnPlan& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int shift = 4;
    while ((1 << shift) < a.c.page_size) ++shift;
    const int64_t u0 = (int64_t)blockIdx.x * p.units / p.ctas, u1 = ((int64_t)blockIdx.x + 1) * p.units / p.ctas;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int64_t u = u0; u < u1;) {
        const int64_t item = u / p.nblk;
        const int64_t end = min(u1, (item + 1) * p.nblk);
        const int head = (int)(item / p.n_tiles);
        const int64_t r0 = (item - (int64_t)head * p.n_tiles) * 16;
        const int rows = (int)min((int64_t)16, p.R - r0);
        const int64_t t0 = (u - item * p.nblk) * p.block_keys;
        const int64_t t1 = min(a.a.prefix_len, (end - item * p.nblk) * (int64_t)p.block_keys);
        RowState<D, kFormat> st;
        load_query<D, kFormat>(st, rows, a.qk_scale, [&](int r) {
            const int64_t row = r0 + r, bt = row / a.G;
            return static_cast<const __nv_bfloat16*>(a.a.q) + (bt * a.a.n_q_heads + (int64_t)head * a.G + (row - bt * a.G)) * D;
        });
        const PageList list{a.a.prefix_pages, a.c.n_pages, shift, head, a.c.n_heads};
        const int64_t lim[2] = {t1, t1};
        const bool good = attend<D, kFormat>(st, a.c, list, t0 + warp * 16, kRowsWarps * 16, t1, lim);
        if (threadIdx.x == 0) sm.bad = 0;
        __syncthreads();
        store_rows<D, kFormat>(sm, st);
        if (!good && lane == 0) sm.bad = 1;
        __syncthreads();
        const int64_t piece = blockIdx.x + item;
        float* po = a.part + piece * 16 * D;
        for (int i = threadIdx.x; i < 16 * D / 4; i += kRowsThreads) {
            const int r = i / (D / 4), col = i % (D / 4) * 4;
            float top = sm.m[0][r];
#pragma unroll
            for (int w = 1; w < kRowsWarps; ++w) top = fmax_nan(top, sm.m[w][r]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f;
#pragma unroll
            for (int w = 0; w < kRowsWarps; ++w) {
                const float f = join_weight(sm.m[w][r], top);
                const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][r][col]);
                acc.x = fmaf(f, x.x, acc.x), acc.y = fmaf(f, x.y, acc.y);
                acc.z = fmaf(f, x.z, acc.z), acc.w = fmaf(f, x.w, acc.w);
                l = fmaf(f, sm.l[w][r], l);
            }
            *reinterpret_cast<float4*>(po + r * D + col) = acc;
            if (col == 0) a.ml[piece * 16 + r] = make_float2(top, sm.bad ? -1.f : l);
        }
        __syncthreads();
        u = end;
    }
}

// One sequence's own tokens for one key head (a cluster of CTAs takes them in turn), then the join with
// the pieces of the shared prefix, the division by the sum and the output.
template <int D, int kFormat>
__global__ void __launch_bounds__(kRowsThreads) attn_suffix_kernel(const AttnArgs a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    RowsShared<D>& sm = *reinterpret_cast<RowsShared<D>*>(raw);
    const AttnPlan& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    const int ncl = p.cluster, rank = (int)(blockIdx.x % ncl);
    const int64_t id = blockIdx.x / ncl;
    const int tile = (int)(id % p.suffix_tiles);
    const int64_t bh = id / p.suffix_tiles;
    const int head = (int)(bh % a.c.n_heads);
    const int64_t b = bh / a.c.n_heads;
    int shift = 4;
    while ((1 << shift) < a.c.page_size) ++shift;
    const int Tq = a.a.q_len, G = a.G, r0 = tile * 16, rows = min(16, Tq * G - r0);
    const int64_t len = a.a.suffix_len[b];
    const bool fits = len >= 0 && len <= a.a.table_width << shift;
    // Rows (t, i): query t of the sequence, head i of the group.  Its row for the key head is b Tq G + t G + i.
    auto seen = [&](int r) {  // own tokens that row r of the sequence sees
        const int64_t n = len - Tq + 1 + min(r, Tq * G - 1) / G;
        return fits && n > 0 ? n : (int64_t)0;
    };
    RowState<D, kFormat> st;
    load_query<D, kFormat>(st, rows, a.qk_scale, [&](int r) {
        const int t = (r0 + r) / G;
        return static_cast<const __nv_bfloat16*>(a.a.q) +
               ((b * Tq + t) * a.a.n_q_heads + (int64_t)head * G + (r0 + r - t * G)) * D;
    });
    const PageList list{a.a.page_table + b * a.a.table_ld, a.c.n_pages, shift, head, a.c.n_heads};
    const int64_t lim[2] = {seen(r0 + g), seen(r0 + g + 8)};
    const int64_t last = seen(r0 + rows - 1);
    const bool good =
        attend<D, kFormat>(st, a.c, list, (rank * kRowsWarps + warp) * 16, (int64_t)ncl * kRowsWarps * 16, last, lim);
    if (threadIdx.x == 0) sm.bad = fits ? 0 : 1;
    __syncthreads();
    store_rows<D, kFormat>(sm, st);
    if (!good && lane == 0) sm.bad = 1;
    if (ncl > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces of the shared prefix
    // Rank k joins every ncl-th group of four columns, from all CTAs' shared memory.
    const uint32_t base = smem_u32(raw);
    auto peer = [&](const void* p_, int who) {
        uint32_t addr = base + (uint32_t)(static_cast<const unsigned char*>(p_) - raw), out;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(addr), "r"(who));
        return out;
    };
    auto ld1 = [](uint32_t addr) {
        float x;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr));
        return x;
    };
    auto ld4 = [](uint32_t addr) {
        float4 x;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(addr));
        return x;
    };
    bool bad = false;
    for (int k = 0; k < ncl; ++k) {
        int x;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(peer(&sm.bad, k)));
        bad = bad || x != 0;
    }
    const float neg = -__int_as_float(0x7F800000);
    for (int i = threadIdx.x * ncl + rank; i < rows * (D / 4); i += kRowsThreads * ncl) {
        const int r = i / (D / 4), col = i % (D / 4) * 4;
        // the pieces of this row: CTAs c0 .. c1 of the prefix kernel
        int64_t first = 0, n_piece = 0, in_tile = 0;
        if (p.nblk > 0) {
            const int64_t row = b * Tq * G + r0 + r, item = (int64_t)head * p.n_tiles + row / p.tile_rows;
            in_tile = row % p.tile_rows;
            const int64_t c0 = ((item * p.nblk + 1) * p.ctas - 1) / p.units;
            const int64_t c1 = ((item + 1) * p.nblk * p.ctas - 1) / p.units;
            first = c0 + item;
            n_piece = c1 - c0 + 1;
        }
        float top = neg;
        for (int k = 0; k < ncl; ++k)
#pragma unroll
            for (int w = 0; w < kRowsWarps; ++w) top = fmax_nan(top, ld1(peer(&sm.m[w][r], k)));
        for (int64_t j = 0; j < n_piece; ++j) top = fmax_nan(top, a.ml[(first + j) * p.tile_rows + in_tile].x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        auto add = [&](float f, float4 x, float y) {
            acc.x = fmaf(f, x.x, acc.x), acc.y = fmaf(f, x.y, acc.y);
            acc.z = fmaf(f, x.z, acc.z), acc.w = fmaf(f, x.w, acc.w);
            l = fmaf(f, y, l);
        };
        for (int k = 0; k < ncl; ++k)
#pragma unroll
            for (int w = 0; w < kRowsWarps; ++w)
                add(join_weight(ld1(peer(&sm.m[w][r], k)), top), ld4(peer(&sm.o[w][r][col], k)), ld1(peer(&sm.l[w][r], k)));
        for (int64_t j = 0; j < n_piece; ++j) {
            const int64_t at = (first + j) * p.tile_rows + in_tile;
            const float2 ml = a.ml[at];
            if (ml.y < 0.f) bad = true;
            add(join_weight(ml.x, top), *reinterpret_cast<const float4*>(a.part + at * D + col), ml.y);
        }
        float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        if (bad) inv = __int_as_float(0x7FC00000);
        if (l == 0.f && top == neg && !bad) acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const int t = (r0 + r) / G;
        const int64_t out_row = (b * Tq + t) * a.a.n_q_heads + (int64_t)head * G + (r0 + r - t * G);
        uint2 w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(acc.y * inv), "f"(acc.x * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(acc.w * inv), "f"(acc.z * inv));
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.a.out) + out_row * D + col) = w;
        if (col == 0 && a.a.out_lse) {
            const float lift = kFormat == TPS_KV_BF16 ? 0.f : kLift;
            a.a.out_lse[out_row] = bad ? inv : (l == 0.f ? neg : (top + log2f(l) - lift) * 0.693147180559945f);
        }
        if (i == 0 && head == 0 && tile == p.suffix_tiles - 1 && a.a.out_status) a.a.out_status[b] = bad ? TPS_ROW_BAD_PARAM : TPS_ROW_OK;
    }
    if (ncl > 1) {  // no CTA may leave while others read its shared memory
        cluster_arrive();
        cluster_wait();
    }
}

}  // namespace tps
