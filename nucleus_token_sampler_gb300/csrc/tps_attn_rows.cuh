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
// What bounds it: the bytes of the keys and values, and the latency of a short sequence's few steps.  Each
// warp has a ring of its own in shared memory that bulk copies fill 16 tokens at a time, and works without
// the others: no barrier but its own.  A lane reads 16 bytes of a key row and 16 of a value row at a time;
// the product q.k is the same for any order of the D components, so they serve as its fragments of
// consecutive k-steps of mma.sync m16n8k16 as they lie (the query fragments are loaded in the same order),
// and the columns of the output are renumbered so that a lane's bytes of a value row are one column each
// of consecutive tiles.  mma.sync rather than tcgen05: the 16 rows fill an eighth of a tcgen05 tile.
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
constexpr uint64_t kAttnWaitNs = 1000000000ull;  // every wait's limit
constexpr float kPieceBadPage = -1.f, kPieceTimeout = -2.f;  // a piece's sum where it is no sum

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

// A warp's ring of 16-token chunks in shared memory: keys, values and, for 8-bit formats, their scales.
// A chunk lies in one page (pages hold 16 tokens or more), so each of them is one bulk copy.
template <int D, int kFormat> struct Chunk {
    static constexpr bool k8 = kFormat != TPS_KV_BF16;
    static constexpr int kRowBytes = k8 ? D : 2 * D;
    static constexpr int kValues = 16 * kRowBytes, kKeyScales = 32 * kRowBytes, kValueScales = kKeyScales + (k8 ? 32 : 0);
    static constexpr int kBytes = kValueScales + (k8 ? 32 : 0);
    // 12 to 16 KB for each warp: with 12 warps on an SM more bytes are on the way than the memory's latency asks for
    static constexpr int kStages = (k8 ? 4 : 2) * (D == 64 ? 2 : 1);
    static constexpr int kRing = (kStages * kBytes + 127) / 128 * 128;
};

template <int D, int kFormat> struct RowsShared {
    unsigned char ring[kRowsWarps][Chunk<D, kFormat>::kRing];  // and a warp's 16 rows of output, once its tokens are done
    uint64_t full[kRowsWarps][Chunk<D, kFormat>::kStages];
    float m[kRowsWarps][16], l[kRowsWarps][16];
    int bad;  // 1: a bad page or length, 2: a wait ran out
};

// Where the tokens lie: `pages` lists the pages of one head's tokens in order.
struct PageList {
    const int32_t* pages;
    int64_t n_pages;
    int shift, head, heads;
    // First row of the 16-token chunk that starts at token t (a multiple of 16), or -1 for a bad page.
    __device__ __forceinline__ int64_t row(int t) const
    {
        const int p = pages[t >> shift];
        return (p < 0 || p >= n_pages) ? -1 : (((int64_t)p * heads + head) << shift) + (t & ((1 << shift) - 1));
    }
};

// A warp's walk over the 16-token chunks first, first + step, ... below `last` tokens.
template <int D, int kFormat> struct Walk {
    using C = Chunk<D, kFormat>;
    const tps_kv_cache& c;
    const PageList& list;
    unsigned char* ring;
    uint64_t* full;
    uint32_t fills;  // copies into the ring so far, over the life of the kernel (parity of the barriers)

    // Ask for the chunk at `row` (its first cache row): one lane for each of the copies.
    __device__ __forceinline__ void request(int64_t row)
    {
        const int lane = threadIdx.x & 31, stage = (int)(fills % C::kStages);
        unsigned char* dst = ring + stage * C::kBytes;
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], C::kBytes);
        __syncwarp();
        if (lane == 0) bulk_g2s(dst, static_cast<const char*>(c.k) + row * C::kRowBytes, 16 * C::kRowBytes, &full[stage]);
        if (lane == 1) bulk_g2s(dst + C::kValues, static_cast<const char*>(c.v) + row * C::kRowBytes, 16 * C::kRowBytes, &full[stage]);
        if (C::k8 && lane == 2) bulk_g2s(dst + C::kKeyScales, static_cast<const char*>(c.k_scale) + row * 2, 32, &full[stage]);
        if (C::k8 && lane == 3) bulk_g2s(dst + C::kValueScales, static_cast<const char*>(c.v_scale) + row * 2, 32, &full[stage]);
        ++fills;
    }
};

// Attend to the chunks first, first + step, ... below `last` tokens; the warp's rows g and g + 8 see the tokens
// below lim[0], lim[1].  Returns 0, or 1 after a page that is not the cache's, 2 after a wait that ran out.
template <int D, int kFormat>
__device__ __forceinline__ int attend(RowState<D, kFormat>& st, Walk<D, kFormat>& walk, int first, int step, int last,
                                      const int (&lim)[2])
{
    using C = Chunk<D, kFormat>;
    constexpr bool k8 = C::k8;
    constexpr int kKeyLoads = C::kRowBytes / 64;  // 16-byte pieces of one key row held by its quad's lane
    constexpr int kValWords = C::kRowBytes / 32;  // words of one value row held by a lane
    constexpr int kCols = D / 8;                  // columns of a value row held by a lane
    const int lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
    const float neg = -__int_as_float(0x7F800000);
    if (first >= last) return 0;

    int fault = 0;
    // `ahead` is the next chunk to ask for; its page number is read one request early.
    int ahead = first;
    int64_t row = walk.list.row(first);
    auto request = [&]() {
        if (row < 0) fault = 1, row = 0;
        walk.request(row);
        ahead += step;
        if (ahead < last) row = walk.list.row(ahead);
    };
    uint32_t at = walk.fills;  // the fill that is used next
#pragma unroll
    for (int i = 0; i < C::kStages; ++i)
        if (ahead < last) request();
    for (int t0 = first; t0 < last; t0 += step, ++at) {
        const int stage = (int)(at % C::kStages);
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&walk.full[stage], (at / C::kStages) & 1, kAttnWaitNs))) {
            for (; at != walk.fills; ++at)  // what is on the way lands before the warp goes on (bounded again)
                mbar_wait_bounded(&walk.full[at % C::kStages], (at / C::kStages) & 1, kAttnWaitNs);
            return 2;
        }
        const unsigned char* buf = walk.ring + stage * C::kBytes;
        const bool partial = t0 + 16 > last;
        float z[2][4] = {};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < kKeyLoads; ++j) {
                const uint4 x = *reinterpret_cast<const uint4*>(buf + (n * 8 + g) * C::kRowBytes + j * 64 + quad * 16);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
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
        uint32_t vreg[4][kValWords];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = (i >> 1) * 8 + quad * 2 + (i & 1);
            const unsigned char* p = buf + C::kValues + tok * C::kRowBytes + g * kValWords * 4;
            if (kValWords == 2) {
                const uint2 w = *reinterpret_cast<const uint2*>(p);
                vreg[i][0] = w.x, vreg[i][1] = w.y;
            } else {
#pragma unroll
                for (int j = 0; j < kValWords; j += 4) {
                    const uint4 w = *reinterpret_cast<const uint4*>(p + j * 4);
                    vreg[i][j] = w.x, vreg[i][(j + 1) % kValWords] = w.y, vreg[i][(j + 2) % kValWords] = w.z,
                    vreg[i][(j + 3) % kValWords] = w.w;
                }
            }
            if (partial && t0 + tok >= last) {  // rows past the end hold anything, and 0 * NaN is NaN
#pragma unroll
                for (int j = 0; j < kValWords; ++j) vreg[i][j] = 0u;
            }
        }
        // Scores in base-2 units, with the value's scale folded in; columns n * 8 + quad * 2 + {0, 1}.
        float inv_s[2][2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            uint32_t ks = 0, vs = 0;
            if (k8) {
                ks = *reinterpret_cast<const uint32_t*>(buf + C::kKeyScales + n * 16 + quad * 4);
                vs = *reinterpret_cast<const uint32_t*>(buf + C::kValueScales + n * 16 + quad * 4);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float kf = 1.f, add = 0.f;
                if (k8) {
                    kf = floor_scale(__uint_as_float(e ? ks & 0xFFFF0000u : ks << 16));
                    const float s = floor_scale(__uint_as_float(e ? vs & 0xFFFF0000u : vs << 16));
                    add = log2_fast(s);
                    inv_s[n][e] = s == s ? __fdividef(1.f, s) : 1.f;  // NaN reaches the weight through `add` where it is seen
                }
                const int tok = t0 + n * 8 + quad * 2 + e;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float& x = z[n][r * 2 + e];
                    x = k8 ? fmaf(x * kf, st.unscale[r], add) : x * st.unscale[r];
                    if (tok >= lim[r]) x = neg;
                }
            }
        }
        __syncwarp();  // every lane has read the stage
        if (ahead < last) request();
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
    }
    return fault;
}

// This lane's part of the sums becomes the row's.
template <int D, int kFormat>
__device__ __forceinline__ void finish_sums(RowState<D, kFormat>& st)
{
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        st.l[r] += __shfl_xor_sync(0xFFFFFFFFu, st.l[r], 1);
        st.l[r] += __shfl_xor_sync(0xFFFFFFFFu, st.l[r], 2);
    }
}

// Put a warp's first `rows` rows into its part of shared memory in natural column order (a lane's columns are
// (2 quad + e) D/8 + tile).
template <int D, int kFormat>
__device__ __forceinline__ void store_rows(RowsShared<D, kFormat>& sm, RowState<D, kFormat>& st, int rows)
{
    static_assert(sizeof(sm.ring[0]) >= 16 * D * sizeof(float), "the ring holds 16 rows of output");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
    float* o = reinterpret_cast<float*>(sm.ring[warp]);
    finish_sums(st);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = g + 8 * r;
        if (row >= rows) continue;
        if (quad == 0) {
            sm.m[warp][row] = st.m[r];
            sm.l[warp][row] = st.l[r];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float* dst = o + row * D + (quad * 2 + e) * (D / 8);
#pragma unroll
            for (int t = 0; t < D / 8; t += 4)
                *reinterpret_cast<float4*>(dst + t) = make_float4(st.o[t][r * 2 + e], st.o[t + 1][r * 2 + e],
                                                                  st.o[t + 2][r * 2 + e], st.o[t + 3][r * 2 + e]);
        }
    }
}

template <int D, int kFormat>
__device__ __forceinline__ void init_rings(RowsShared<D, kFormat>& sm)
{
    if (threadIdx.x == 0) {
        for (int w = 0; w < kRowsWarps; ++w)
            for (int i = 0; i < Chunk<D, kFormat>::kStages; ++i) mbar_init(&sm.full[w][i], 1);
        sm.bad = 0;
        fence_proxy_async();
    }
    __syncthreads();
}

// Weight of a part with reference m in a join whose reference is `top` (0 for a part without tokens).
__device__ __forceinline__ float join_weight(float m, float top)
{
    return m == -__int_as_float(0x7F800000) ? 0.f : exp2_fast(m - top);
}

// A join of the parts of one row.
struct Joined {
    float top, l;
    float4 acc;
    __device__ __forceinline__ void add(float m, float4 x, float y)
    {
        const float f = join_weight(m, top);
        acc.x = fmaf(f, x.x, acc.x), acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z), acc.w = fmaf(f, x.w, acc.w);
        l = fmaf(f, y, l);
    }
};

// The shared prefix, 16 rows at a time: CTA c's part of the line of blocks (AttnPlan).
template <int D, int kFormat>
__global__ void __launch_bounds__(kRowsThreads, 3) attn_prefix_rows_kernel(const AttnArgs a)
{
    extern __shared__ __align__(128) unsigned char raw[];
    RowsShared<D, kFormat>& sm = *reinterpret_cast<RowsShared<D, kFormat>*>(raw);
    const AttnPlan& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t u0 = (int64_t)blockIdx.x * p.units / p.ctas, u1 = ((int64_t)blockIdx.x + 1) * p.units / p.ctas;
    init_rings(sm);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    PageList list{a.a.prefix_pages, a.c.n_pages, a.page_shift, 0, a.c.n_heads};
    Walk<D, kFormat> walk{a.c, list, sm.ring[warp], sm.full[warp], 0u};
    for (int64_t u = u0; u < u1;) {
        const int64_t item = u / p.nblk;
        const int64_t end = min(u1, (item + 1) * p.nblk);
        const int head = (int)(item / p.n_tiles);
        const int64_t r0 = (item - (int64_t)head * p.n_tiles) * 16;
        const int rows = (int)min((int64_t)16, p.R - r0);
        const int t0 = (int)(u - item * p.nblk) * p.block_keys;
        const int t1 = (int)min(a.a.prefix_len, (end - item * p.nblk) * (int64_t)p.block_keys);
        RowState<D, kFormat> st;
        load_query<D, kFormat>(st, rows, a.qk_scale, [&](int r) {
            const int64_t row = r0 + r, bt = row / a.G;
            return static_cast<const __nv_bfloat16*>(a.a.q) + (bt * a.a.n_q_heads + (int64_t)head * a.G + (row - bt * a.G)) * D;
        });
        list.head = head;
        const int lim[2] = {t1, t1};
        const int fault = attend<D, kFormat>(st, walk, t0 + warp * 16, kRowsWarps * 16, t1, lim);
        store_rows<D, kFormat>(sm, st, 16);
        if (fault && lane == 0) atomicMax(&sm.bad, fault);
        __syncthreads();
        const int64_t piece = blockIdx.x + item;
        float* po = a.part + piece * 16 * D;
        for (int i = threadIdx.x; i < 16 * D / 4; i += kRowsThreads) {
            const int r = i & 15, col = (i >> 4) * 4;
            Joined j{sm.m[0][r], 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
            for (int w = 1; w < kRowsWarps; ++w) j.top = fmax_nan(j.top, sm.m[w][r]);
#pragma unroll
            for (int w = 0; w < kRowsWarps; ++w)
                j.add(sm.m[w][r], *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.ring[w]) + r * D + col), sm.l[w][r]);
            *reinterpret_cast<float4*>(po + (col / 4 * 16 + r) * 4) = j.acc;
            if (col == 0) a.ml[piece * 16 + r] = make_float2(j.top, sm.bad == 2 ? kPieceTimeout : (sm.bad ? kPieceBadPage : j.l));
        }
        __syncthreads();
        // The rings held output: order those accesses before the next copies into them.
        fence_proxy_async();
        if (sm.bad == 2) {  // give up: every later piece says so (uniform: nothing writes it here)
            for (u = end; u < u1; u = min(u1, (u / p.nblk + 1) * p.nblk))
                if (threadIdx.x < 16) a.ml[(blockIdx.x + u / p.nblk) * 16 + threadIdx.x] = make_float2(0.f, kPieceTimeout);
            break;
        }
        u = end;
    }
}

// The pieces of the shared prefix that hold a row's item: piece `first` on, `count` of them.
struct Pieces {
    int64_t first;
    int count;
};
__device__ __forceinline__ Pieces pieces_of(const AttnPlan& p, int64_t item)
{
    if (p.nblk == 0) return Pieces{0, 0};
    const int64_t c0 = ((item * p.nblk + 1) * p.ctas - 1) / p.units, c1 = ((item + 1) * p.nblk * p.ctas - 1) / p.units;
    return Pieces{c0 + item, (int)(c1 - c0 + 1)};
}

// 1 / sum as the output takes it: 0 where no token was seen, NaN where something was bad.
__device__ __forceinline__ float inverse_sum(float l, bool bad)
{
    if (bad) return __int_as_float(0x7FC00000);
    return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
}

template <int kFormat>
__device__ __forceinline__ float log_sum(float top, float l, bool bad)
{
    const float lift = kFormat == TPS_KV_BF16 ? 0.f : kLift;
    if (bad) return __int_as_float(0x7FC00000);
    return l == 0.f ? -__int_as_float(0x7F800000) : (top + log2f(l) - lift) * 0.693147180559945f;
}

// One sequence's own tokens for one key head, then the join with the pieces of the shared prefix, the
// division by the sum and the output.  With many sequences each warp has one for itself, and joins in
// registers; else the four warps of a CTA, or of a cluster of CTAs, take its chunks in turn and join
// through (distributed) shared memory.
template <int D, int kFormat, bool kOneWarp>
__global__ void __launch_bounds__(kRowsThreads, 3) attn_suffix_kernel(const AttnArgs a)
{
    extern __shared__ __align__(128) unsigned char raw[];
    RowsShared<D, kFormat>& sm = *reinterpret_cast<RowsShared<D, kFormat>*>(raw);
    const AttnPlan& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
    const int ncl = kOneWarp ? 1 : p.cluster, rank = kOneWarp ? 0 : (int)(blockIdx.x % ncl);
    const uint32_t id = kOneWarp ? blockIdx.x * kRowsWarps + warp : blockIdx.x / ncl;
    init_rings(sm);
    const uint32_t bh = id / (uint32_t)p.suffix_tiles;
    const int tile = (int)(id - bh * p.suffix_tiles);
    const int64_t b = bh / (uint32_t)a.c.n_heads;
    const int head = (int)(bh - (uint32_t)b * a.c.n_heads);
    if (kOneWarp && b >= a.a.B) return;  // the last CTA's spare warps
    const int Tq = a.a.q_len, G = a.G, r0 = tile * 16, rows = min(16, Tq * G - r0);
    const int len = a.a.suffix_len[b];
    const bool fits = len >= 0 && len <= a.a.table_width << a.page_shift;
    // Row r of the sequence is query r / G, head r % G of the group: own tokens that it sees.
    auto seen = [&](int r) {
        const int n = len - Tq + 1 + min(r, Tq * G - 1) / G;
        return fits && n > 0 ? n : 0;
    };
    auto out_row = [&](int r) {
        const int t = (r0 + r) / G;
        return (b * Tq + t) * a.a.n_q_heads + (int64_t)head * G + (r0 + r - t * G);
    };
    RowState<D, kFormat> st;
    load_query<D, kFormat>(st, rows, a.qk_scale, [&](int r) { return static_cast<const __nv_bfloat16*>(a.a.q) + out_row(r) * D; });
    const PageList list{a.a.page_table + b * a.a.table_ld, a.c.n_pages, a.page_shift, head, a.c.n_heads};
    Walk<D, kFormat> walk{a.c, list, sm.ring[warp], sm.full[warp], 0u};
    const int lim[2] = {seen(r0 + g), seen(r0 + g + 8)};
    const int last = seen(r0 + rows - 1);
    const int fault = attend<D, kFormat>(st, walk, kOneWarp ? 0 : (rank * kRowsWarps + warp) * 16, kOneWarp ? 16 : ncl * kRowsWarps * 16,
                                         last, lim);
    const float neg = -__int_as_float(0x7F800000);
    const int64_t row0 = b * Tq * G + r0;  // the tile's first row among the key head's R

    if (kOneWarp) {
        finish_sums(st);
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces of the shared prefix
        const Pieces pc = pieces_of(p, (int64_t)head * p.n_tiles + row0 / p.tile_rows);
        const int in0 = (int)(row0 % p.tile_rows);
        bool any_bad = false, any_late = fault == 2;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r;
            if (row >= rows) continue;
            // A tile of the prefix may end inside these rows: its next one is the next item.
            Pieces mine = pc;
            int in_tile = in0 + row;
            if (in_tile >= p.tile_rows) in_tile -= p.tile_rows, mine = pieces_of(p, (int64_t)head * p.n_tiles + row0 / p.tile_rows + 1);
            const float2* ml = a.ml + mine.first * p.tile_rows + in_tile;
            float top = st.m[r];
#pragma unroll 4
            for (int j = 0; j < mine.count; ++j) top = fmax_nan(top, ml[(int64_t)j * p.tile_rows].x);
            const float f0 = join_weight(st.m[r], top);
            float l = st.l[r] * f0;
            bool bad = fault || !fits, late = fault == 2;
#pragma unroll
            for (int t = 0; t < D / 8; ++t) st.o[t][2 * r] *= f0, st.o[t][2 * r + 1] *= f0;
            const float4* part = reinterpret_cast<const float4*>(a.part) + mine.first * p.tile_rows * (D / 4) + in_tile;
#pragma unroll 2
            for (int j = 0; j < mine.count; ++j) {
                const float2 x = ml[(int64_t)j * p.tile_rows];
                const float f = join_weight(x.x, top);
                bad = bad || x.y < 0.f;
                late = late || x.y == kPieceTimeout;
                l = fmaf(f, x.y, l);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int t = 0; t < D / 8; t += 4) {
                        const float4 y = part[((int64_t)j * (D / 4) + ((quad * 2 + e) * (D / 8) + t) / 4) * p.tile_rows];
                        st.o[t][2 * r + e] = fmaf(f, y.x, st.o[t][2 * r + e]);
                        st.o[t + 1][2 * r + e] = fmaf(f, y.y, st.o[t + 1][2 * r + e]);
                        st.o[t + 2][2 * r + e] = fmaf(f, y.z, st.o[t + 2][2 * r + e]);
                        st.o[t + 3][2 * r + e] = fmaf(f, y.w, st.o[t + 3][2 * r + e]);
                    }
            }
            const float inv = inverse_sum(l, bad);
            const int64_t orow = out_row(row);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t w[D / 16];
#pragma unroll
                for (int t = 0; t < D / 8; t += 2)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[t / 2]) : "f"(st.o[t + 1][2 * r + e] * inv), "f"(st.o[t][2 * r + e] * inv));
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.a.out) + orow * D + (quad * 2 + e) * (D / 8));
#pragma unroll
                for (int i = 0; i < D / 64; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
            if (quad == 0 && a.a.out_lse) a.a.out_lse[orow] = log_sum<kFormat>(top, l, bad);
            any_bad = any_bad || bad;
            any_late = any_late || late;
        }
        any_bad = __any_sync(0xFFFFFFFFu, any_bad);
        any_late = __any_sync(0xFFFFFFFFu, any_late);
        if (lane == 0 && head == 0 && tile == p.suffix_tiles - 1 && a.a.out_status)
            a.a.out_status[b] = any_late ? TPS_ROW_TIMEOUT : (any_bad ? TPS_ROW_BAD_PARAM : TPS_ROW_OK);
    } else {
        store_rows<D, kFormat>(sm, st, rows);
        if (lane == 0 && (fault || !fits)) atomicMax(&sm.bad, max(fault, 1));
        if (ncl > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
        // Rank k joins every ncl-th group of four columns, from all CTAs' shared memory.
        const uint32_t base = smem_u32(raw);
        auto peer = [&](const void* x, int who) {
            const uint32_t addr = base + (uint32_t)(static_cast<const unsigned char*>(x) - raw);
            uint32_t out;
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
        int own_bad = 0;
        for (int k = 0; k < ncl; ++k) {
            int x;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(peer(&sm.bad, k)));
            own_bad = max(own_bad, x);
        }
        for (int i = threadIdx.x * ncl + rank; i < rows * (D / 4); i += kRowsThreads * ncl) {
            const int r = i / (D / 4), col = i % (D / 4) * 4;
            const int64_t row = row0 + r;
            const Pieces mine = pieces_of(p, (int64_t)head * p.n_tiles + row / p.tile_rows);
            const int in_tile = (int)(row % p.tile_rows);
            const float2* ml = a.ml + mine.first * p.tile_rows + in_tile;
            Joined j{neg, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
            for (int k = 0; k < ncl; ++k)
#pragma unroll
                for (int w = 0; w < kRowsWarps; ++w) j.top = fmax_nan(j.top, ld1(peer(&sm.m[w][r], k)));
#pragma unroll 4
            for (int n = 0; n < mine.count; ++n) j.top = fmax_nan(j.top, ml[(int64_t)n * p.tile_rows].x);
            for (int k = 0; k < ncl; ++k)
#pragma unroll
                for (int w = 0; w < kRowsWarps; ++w)
                    j.add(ld1(peer(&sm.m[w][r], k)), ld4(peer(reinterpret_cast<const float*>(sm.ring[w]) + r * D + col, k)),
                          ld1(peer(&sm.l[w][r], k)));
            bool bad = own_bad != 0, late = own_bad == 2;
            const float4* part = reinterpret_cast<const float4*>(a.part) + (mine.first * (D / 4) + col / 4) * p.tile_rows + in_tile;
#pragma unroll 8
            for (int n = 0; n < mine.count; ++n) {
                const float2 x = ml[(int64_t)n * p.tile_rows];
                bad = bad || x.y < 0.f;
                late = late || x.y == kPieceTimeout;
                j.add(x.x, part[(int64_t)n * (D / 4) * p.tile_rows], x.y);
            }
            const float inv = inverse_sum(j.l, bad);
            const int64_t orow = out_row(r);
            uint2 w;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(j.acc.y * inv), "f"(j.acc.x * inv));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(j.acc.w * inv), "f"(j.acc.z * inv));
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.a.out) + orow * D + col) = w;
            if (col == 0 && a.a.out_lse) a.a.out_lse[orow] = log_sum<kFormat>(j.top, j.l, bad);
            if (i == 0 && head == 0 && tile == p.suffix_tiles - 1 && a.a.out_status)
                a.a.out_status[b] = late ? TPS_ROW_TIMEOUT : (bad ? TPS_ROW_BAD_PARAM : TPS_ROW_OK);
        }
        if (ncl > 1) {  // no CTA may leave while others read its shared memory
            cluster_arrive();
            cluster_wait();
        }
    }
}

}  // namespace tps
