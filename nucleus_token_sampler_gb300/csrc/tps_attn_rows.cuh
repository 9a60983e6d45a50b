// tps_attn_rows.cuh -- attention of up to 16 query rows per warp over paged keys and values, and the
// join of its parts: every sequence's own tokens, and the prefix of a call too small to share its work; also
// (kTree) trees of few rows, whose masks are looked up where drafted tokens are.
//
// Mathematics.  With z_j = scale log2(e) q.k_j, one pass over the tokens holds a reference m, the sum
// l = sum 2^(z_j - m) and the output o = sum 2^(z_j - m) v_j in float32; m is raised (and l, o scaled)
// only when some z exceeds it by more than kSlack, so that in most steps nothing is scaled and no
// maximum has to be agreed on between lanes.  Parts of a row (warps, CTAs, prefix and own tokens) join as
// m = max m_i, l = sum l_i 2^(m_i - m), o likewise.
// For 8-bit formats the codes go to the matrix instruction as they are (exact in float16) and the
// scales stay outside, in float32: z_j carries the key's scale, and with t_j = z_j + log2(s_j) the weight
// 2^(t_j - m) already holds the value's scale s_j; l adds 2^(t_j - m) / s_j.  The weights are float16
// with 11 bits, lifted by 2^kLift so that tokens down to 2^-(24 + kLift) of the largest still count.  Next to a
// bfloat16 cache they are bfloat16 with 8: both factors of a product have one type, and float16 would not hold
// every value.  Against 64 bits such outputs are off by 0.0023 of their size (root mean square; their own
// rounding alone makes 0.0016), those of 8-bit caches by 0.0017.
//
// What bounds it: the bytes of the keys and values, and the latency of a short sequence's few steps.  Each
// warp has a ring of its own in shared memory that bulk copies fill 16 tokens at a time, and works without
// the others: no barrier but its own.  The products are taken transposed, K Q^T and V^T P^T, with the
// tokens (and then the D components) as the 16 rows of mma.sync m16n8k16 and the query rows as its 8
// columns: the 4 to 8 query heads of a key head fill an 8-wide tile where they would leave a 16-wide one
// half empty, in matrix instructions, in exponentials and in registers.  The product q.k is the same for any
// order of the D components, so a lane's 16 bytes of a key row serve as its fragments of consecutive
// k-steps as they lie (the query fragments are loaded in the same order); a lane's 16 bytes of a value row
// become rows g and g + 8 of consecutive tiles.  mma.sync rather than tcgen05: 8 or 16 rows fill a
// sixteenth or an eighth of a tcgen05 tile.  Measured: 16 sequences of up to 16,000 own tokens, 4 key heads of 128 in
// bfloat16, 65 us with the prefix and the join (4.1 TB/s); 8 sequences on 1,000 shared and 40 tokens of their own 10.0 us,
// the launch of the shared part and the join with it.
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

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, bool half)
{
    if (half)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit numbers held as a fragment.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
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

// A value's scale goes into its weight as a power and out of the sum again: w / s. A stored scale is at least 2^-40; what
// lies below 2^-80 (0 of a slot never written, what stands in rows past the end, whose weight is 0) counts as that, so
// that a sum of 2^31 weights up to 2^15, each over its scale, is finite.
constexpr float kLeastScale = 0x1p-80f;
__device__ __forceinline__ float floor_scale(float s) { return s >= kLeastScale || s != s ? s : kLeastScale; }

// Components of a head that a lane holds for k-step s: 4 consecutive ones from here on.
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
    const bool usual = (e >= -2 && e <= 14) || e >= 128 || a == 0.f;
    const uint32_t f = (uint32_t)min(max(127 - e, 1), 254) << 23;  // brings it to [1, 2)
    return __uint_as_float(usual ? 0x3F800000u : f);
}

// A warp's work on 8 N query rows.  Lane (g, quad) = (lane / 4, lane % 4) holds, of rows 8 n + 2 quad + e, the
// reference and its part of the sum, and the output's components g D/8 + 2 t + h in o[n][t][2 h + e].
template <int D, int N> struct RowState {
    static constexpr int kSteps = D / 16;   // k-steps of q.k
    static constexpr int kTiles = D / 16;   // 16-component tiles of the output
    uint32_t q[N][kSteps][2];               // row 8 n + g
    float o[N][kTiles][4];
    float m[N][2], l[N][2];
    float unscale[N][2];  // scale log2(e), over the power of two of the row's float16 form
};

// Ask for the query rows (those from `rows` on are zero); ready_query makes them what the products take.
template <int D, int kFormat, int N, typename RowPtr>
__device__ __forceinline__ void load_query(RowState<D, N>& st, int rows, RowPtr row_ptr)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int row = 8 * n + g;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            uint2 w = make_uint2(0u, 0u);
            if (row < rows) w = *reinterpret_cast<const uint2*>(row_ptr(row) + kstep_base<kFormat>(s, quad));
            st.q[n][s][0] = w.x;
            st.q[n][s][1] = w.y;
        }
    }
}
template <int D, int kFormat, int N>
__device__ __forceinline__ void ready_query(RowState<D, N>& st, float qk_scale)
{
    const int quad = threadIdx.x & 3;
    const float inf = __int_as_float(0x7F800000);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        float amax = 0.f, f = 1.f;
        if (kFormat != TPS_KV_BF16) {
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                const uint2 w = make_uint2(st.q[n][s][0], st.q[n][s][1]);
                const float x[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                                    __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u)};
#pragma unroll
                for (int i = 0; i < 4; ++i) amax = fabsf(x[i]) < inf ? fmaxf(amax, fabsf(x[i])) : amax;
            }
        }
        if (kFormat != TPS_KV_BF16) {
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            f = f16_row_scale(amax);
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t w = st.q[n][s][i];
                    const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
                    st.q[n][s][i] = *reinterpret_cast<const uint32_t*>(&h);
                }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // lane 4 r holds row r's factor
            st.unscale[n][e] = kFormat != TPS_KV_BF16 ? qk_scale / __shfl_sync(0xFFFFFFFFu, f, (2 * quad + e) * 4) : qk_scale;
            st.m[n][e] = -inf;
            st.l[n][e] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[n][t][i] = 0.f;
    }
}

// A warp's ring of 16-token chunks in shared memory: keys, values and, for 8-bit formats, their scales.
// A chunk lies in one page (pages hold 16 tokens or more), so each of them is one bulk copy.
template <int D, int kFormat> struct Chunk {
    static constexpr bool k8 = kFormat != TPS_KV_BF16;
    static constexpr int kRowBytes = k8 ? D : 2 * D;
    static constexpr int kValues = 16 * kRowBytes, kKeyScales = 32 * kRowBytes, kValueScales = kKeyScales + (k8 ? 32 : 0);
    static constexpr int kBytes = kValueScales + (k8 ? 32 : 0);
    // 12 to 16 KB for each warp: with 12 to 16 warps on an SM more bytes are on the way than the latency asks for
    static constexpr int kStages = (k8 ? 3 : 2) * (D == 64 ? 2 : 1);
    static constexpr int kRing = (kStages * kBytes + 127) / 128 * 128;
};

template <int D, int kFormat> struct RowsShared {
    unsigned char ring[kRowsWarps][Chunk<D, kFormat>::kRing];  // and a warp's 16 rows of output, once its tokens are done
    uint64_t full[kRowsWarps][Chunk<D, kFormat>::kStages];
    float m[kRowsWarps][16], l[kRowsWarps][16];
    int bad;  // 1: a bad page or length, 2: a wait ran out
};

// A warp's walk over the 16-token chunks first, first + step, ... below `last` tokens; `pages` lists the pages
// of one head's tokens in order.
template <int D, int kFormat> struct Walk {
    using C = Chunk<D, kFormat>;
    const AttnArgs& a;
    int head;
    unsigned char* ring;
    uint64_t* full;
    const int32_t* pages;
    uint32_t fills;  // copies into the ring so far, over the life of the kernel (parity of the barriers)
    int first, step, last, ahead;  // `ahead`: the next chunk to ask for
    int page;                      // its page, read one request early and not looked at before the next one
    int fault;                     // 1: a page that is not the cache's; 4: values taken out of a product (add_not_finite)

    // The page of the chunk at `first`, if the list reaches as far as `tokens`: may be called before the number of
    // tokens is known, so that this read does not wait for that one.
    __device__ __forceinline__ void look(const int32_t* pages_, int first_, int64_t tokens)
    {
        pages = pages_;
        page = first_ < tokens ? pages[first_ >> a.page_shift] : 0;
    }
    // Ask for the next chunk: one lane for each of its copies.
    __device__ __forceinline__ void request()
    {
        const int lane = threadIdx.x & 31, stage = (int)(fills % C::kStages), shift = a.page_shift;
        const tps_kv_cache& c = a.c;
        int id = page;
        if (id < 0 || id >= c.n_pages) fault |= 1, id = 0;
        const int64_t row = (((int64_t)id * c.n_heads + head) << shift) + (ahead & ((1 << shift) - 1));
        ahead += step;
        if (ahead < last) page = pages[ahead >> shift];
        unsigned char* dst = ring + stage * C::kBytes;
        ++fills;
        if (head == a.stall_head) return;
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], C::kBytes);
        __syncwarp();
        if (lane == 0) bulk_g2s(dst, static_cast<const char*>(c.k) + row * C::kRowBytes, 16 * C::kRowBytes, &full[stage]);
        if (lane == 1) bulk_g2s(dst + C::kValues, static_cast<const char*>(c.v) + row * C::kRowBytes, 16 * C::kRowBytes, &full[stage]);
        if (C::k8 && lane == 2) bulk_g2s(dst + C::kKeyScales, static_cast<const char*>(c.k_scale) + row * 2, 32, &full[stage]);
        if (C::k8 && lane == 3) bulk_g2s(dst + C::kValueScales, static_cast<const char*>(c.v_scale) + row * 2, 32, &full[stage]);
    }
    // Begin, after look(): the first chunks are on their way when this returns (the ring holds nothing still used).
    __device__ __forceinline__ void start(int first_, int step_, int last_)
    {
        first = ahead = first_, step = step_, last = last_;
#pragma unroll
        for (int i = 0; i < C::kStages; ++i)
            if (ahead < last) request();
    }
};

// Of a call on trees (tps_tree_attention with few rows): a sequence's tokens, the drafted ones among them, the last; none of either
// where the lengths are not possible.
struct TreeTokens {
    int len, nodes;
    bool fits;
};
__device__ __forceinline__ TreeTokens tree_tokens(const AttnArgs& a, int64_t b)
{
    const int len = a.a.suffix_len[b], nodes = a.tree_len ? a.tree_len[b] : a.a.q_len;
    const bool fits = len >= 0 && nodes >= 0 && nodes <= a.a.q_len && nodes <= len && len <= a.a.table_width << a.page_shift;
    return fits ? TreeTokens{len, nodes, true} : TreeTokens{0, 0, false};
}
// Whether row r of the sequence sees drafted token j (from 0 on).
__device__ __forceinline__ bool tree_sees(const AttnArgs& a, int64_t b, const TreeTokens& t, int r, int j)
{
    const int node = min(r / a.G, a.a.q_len - 1);
    return j < t.nodes && node < t.nodes && (a.tree[b * a.tree_ld + node] >> j & 1);
}

// How many of the first drafted tokens all rows see that are not padding (whose sums are cleared); a warp's rows begin at r0.  A
// decode step masks nothing, and a tree nothing up to its first fork.
template <int N> __device__ __forceinline__ int all_nodes_see(const AttnArgs& a, int64_t b, int r0, const TreeTokens& t)
{
    uint64_t bits = ~0ull;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int node = (r0 + 8 * n + 2 * ((int)threadIdx.x & 3) + e) / a.G;
            if (node < t.nodes) bits &= a.tree[b * a.tree_ld + node];
        }
    const uint32_t low = __reduce_and_sync(0xFFFFFFFFu, (uint32_t)bits), high = __reduce_and_sync(0xFFFFFFFFu, (uint32_t)(bits >> 32));
    const int first = low != ~0u ? __ffs(~low) - 1 : high != ~0u ? 31 + __ffs(~high) : 64;  // that one of them does not see
    return min(first, t.nodes);
}

// bfloat16 values of tokens that not every row sees: the product would bring a hidden token's NaN or infinity to every row
// (0 * NaN), so attend() takes those components out of it, and the rows that see the token get them here.
__device__ __forceinline__ uint32_t not_finite(uint32_t w)  // the halves that are not, else 0
{
    return ((w & 0x7F80u) == 0x7F80u ? w & 0xFFFFu : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? w & 0xFFFF0000u : 0u);
}
template <int D, int kFormat, int N, bool kTree>
__device__ __forceinline__ void add_not_finite(RowState<D, N>& st, const Walk<D, kFormat>& walk, const int (&lim)[N][2], int all_see, int64_t b,
                                               int r0, const TreeTokens& tree)
{
    const int g = (threadIdx.x & 31) >> 2, quad = threadIdx.x & 3, shift = walk.a.page_shift;
#pragma unroll 1
    for (int t0 = walk.first; t0 < walk.last; t0 += walk.step)
#pragma unroll 1
        for (int t = max(t0, all_see); t < min(t0 + 16, walk.last); ++t) {
            const int id = walk.pages[t >> shift];
            if (id < 0 || id >= walk.a.c.n_pages) continue;
            const int64_t row = (((int64_t)id * walk.a.c.n_heads + walk.head) << shift) + (t & ((1 << shift) - 1));
            const uint32_t* v = static_cast<const uint32_t*>(walk.a.c.v) + (row * D + g * (D / 8)) / 2;
            const int j = kTree ? t - (tree.len - tree.nodes) : -1;  // a drafted token
            bool sees[N][2];
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    sees[n][e] = t < lim[n][e] && (!kTree || j < 0 || tree_sees(walk.a, b, tree, r0 + 8 * n + 2 * quad + e, j));
#pragma unroll
            for (int w = 0; w < D / 16; ++w) {
                const uint32_t x = not_finite(v[w]);
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (sees[n][e]) {
                            st.o[n][w][e] += __uint_as_float(x << 16);
                            st.o[n][w][2 + e] += __uint_as_float(x & 0xFFFF0000u);
                        }
            }
        }
}

// Attend to the chunks of a walk that has been started; row 8 n + 2 quad + e sees the tokens below
// lim[n][e].  Returns 0, or 1 after a page that is not the cache's, 2 after a wait that ran out.
// kTree: of the sequence's drafted tokens, which begin at `tree`, a row sees those that its mask names; its first row is r0.
template <int D, int kFormat, int N, bool kTree = false>
__device__ __forceinline__ int attend(RowState<D, N>& st, Walk<D, kFormat>& walk, const int (&lim)[N][2], int64_t b = 0, int r0 = 0,
                                      const TreeTokens tree = {})
{
    using C = Chunk<D, kFormat>;
    constexpr bool k8 = C::k8;
    constexpr int kKeyLoads = C::kRowBytes / 64;  // 16-byte pieces of one key row held by its quad's lane
    constexpr int kValWords = C::kRowBytes / 32;  // words of one value row held by a lane
    constexpr int kTiles = D / 16;
    const int lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
    const float neg = -__int_as_float(0x7F800000);
    const int last = walk.last;
    if (walk.first >= last) return walk.fault & 1;
    int all_see = last;  // tokens that every row sees
#pragma unroll
    for (int n = 0; n < N; ++n) all_see = min(all_see, min(lim[n][0], lim[n][1]));
    all_see = (int)__reduce_min_sync(0xFFFFFFFFu, (uint32_t)all_see);
    if (kTree) all_see = min(all_see, tree.len - tree.nodes + all_nodes_see<N>(walk.a, b, r0, tree));
    const uint32_t chunks = (uint32_t)((last - walk.first + walk.step - 1) / walk.step);
    uint32_t at = walk.fills - min(chunks, (uint32_t)C::kStages);  // the fill that is used next
    for (int t0 = walk.first; t0 < last; t0 += walk.step, ++at) {
        const int stage = (int)(at % C::kStages);
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&walk.full[stage], (at / C::kStages) & 1, walk.a.wait_ns))) {
            for (; at != walk.fills && walk.head != walk.a.stall_head; ++at)  // what is on the way lands before the warp goes on (bounded again)
                mbar_wait_bounded(&walk.full[at % C::kStages], (at / C::kStages) & 1, kAttnWaitNs);
            return 2;
        }
        unsigned char* buf = walk.ring + stage * C::kBytes;
        if (!k8 && all_see < last && t0 + 16 > all_see) {
            uint4* v = reinterpret_cast<uint4*>(buf + C::kValues);
#pragma unroll 1
            for (int i = lane; i < C::kRowBytes; i += 32) {  // 16-byte pieces of 16 rows
                const int t = t0 + i / (C::kRowBytes / 16);
                if (t < all_see || t >= last) continue;
                const uint4 x = v[i], y = make_uint4(not_finite(x.x), not_finite(x.y), not_finite(x.z), not_finite(x.w));
                if (y.x | y.y | y.z | y.w) walk.fault |= 4;
                v[i] = make_uint4(x.x ^ y.x, x.y ^ y.y, x.z ^ y.z, x.w ^ y.w);
            }
            __syncwarp();
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
        }
        // tokens g (0, 1) and g + 8 (2, 3), rows 2 quad + {0, 1}; every other k-step in a chain of its own
        float z[N][4] = {}, z_odd[N][4] = {};
#pragma unroll
        for (int j = 0; j < kKeyLoads; ++j) {
            const uint4 x = *reinterpret_cast<const uint4*>(buf + g * C::kRowBytes + j * 64 + quad * 16);
            const uint4 y = *reinterpret_cast<const uint4*>(buf + (g + 8) * C::kRowBytes + j * 64 + quad * 16);
            const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
            if (k8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t x0, x1, y0, y1;
                    code_pairs<kFormat>(wx[i], x0, x1);
                    code_pairs<kFormat>(wy[i], y0, y1);
#pragma unroll
                    for (int n = 0; n < N; ++n) mma16816(i & 1 ? z_odd[n] : z[n], x0, y0, x1, y1, st.q[n][j * 4 + i][0], st.q[n][j * 4 + i][1], true);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < N; ++n)
                        mma16816(i & 1 ? z_odd[n] : z[n], wx[2 * i], wy[2 * i], wx[2 * i + 1], wy[2 * i + 1], st.q[n][(j * 2 + i) % (D / 16)][0],
                                 st.q[n][(j * 2 + i) % (D / 16)][1], false);
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[n][i] += z_odd[n][i];
        // Scores in base-2 units, with the value's scale folded in.
        float add[2] = {0.f, 0.f}, inv_s[2] = {1.f, 1.f};
        if (k8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t ks = *reinterpret_cast<const uint16_t*>(buf + C::kKeyScales + (g + 8 * h) * 2);
                const uint32_t vs = *reinterpret_cast<const uint16_t*>(buf + C::kValueScales + (g + 8 * h) * 2);
                const float kf = __uint_as_float(ks << 16), s = floor_scale(__uint_as_float(vs << 16));
                add[h] = log2_fast(s);
                inv_s[h] = s == s ? __fdividef(1.f, s) : 1.f;  // NaN reaches the weight through `add` where it is seen
#pragma unroll
                for (int n = 0; n < N; ++n) z[n][2 * h] *= kf, z[n][2 * h + 1] *= kf;
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[n][i] = fmaf(z[n][i], st.unscale[n][i & 1], add[i >> 1]);
        if (t0 + 16 > all_see) {
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (t0 + g + 8 * (i >> 1) >= lim[n][i & 1]) z[n][i] = neg;
            if (kTree) {
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = t0 + g + 8 * (i >> 1) - (tree.len - tree.nodes);
                        if (j >= 0 && !tree_sees(walk.a, b, tree, r0 + 8 * n + 2 * quad + (i & 1), j)) z[n][i] = neg;
                    }
            }
            if (t0 + 16 > last) {  // rows past the end hold anything, and 0 * NaN is NaN
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (t0 + (i >> 1) * 8 + quad * 2 + (i & 1) >= last) {
#pragma unroll
                        for (int j = 0; j < kValWords; ++j) vreg[i][j] = 0u;
                    }
            }
        }
        // Every lane has read the stage, values included, before a copy may write there: to the compiler the copy's
        // writes are no stores, so without the fence it may move the loads of the values past the request.
        fence_proxy_async();
        __syncwarp();
        if (walk.ahead < last) walk.request();
        // Raise the references where a score exceeds them by more than the slack (or is the first one).
        bool over = false;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) over = over || fmaxf(z[n][e], z[n][2 + e]) > st.m[n][e] + kSlack;
        if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float t = fmaxf(z[n][e], z[n][2 + e]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
                    const float m = t > st.m[n][e] + kSlack ? t : st.m[n][e];
                    f[e] = m == st.m[n][e] ? 1.f : exp2_fast(st.m[n][e] - m);
                    st.m[n][e] = m;
                    st.l[n][e] *= f[e];
                }
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) st.o[n][t][i] *= f[i & 1];
            }
        }
        uint32_t p[N][2];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float m = st.m[n][i & 1];  // -inf: nothing seen yet, every weight is 0
                w[i] = exp2_fast(z[n][i] - (m == neg ? 0.f : m) + (k8 ? kLift : 0.f));
                st.l[n][i & 1] = k8 ? fmaf(w[i], inv_s[i >> 1], st.l[n][i & 1]) : st.l[n][i & 1] + w[i];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t x;
                if (k8) {
                    const __half2 y = __floats2half2_rn(w[2 * h], w[2 * h + 1]);
                    x = *reinterpret_cast<const uint32_t*>(&y);
                } else {
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(w[2 * h + 1]), "f"(w[2 * h]));
                }
                p[n][h] = transpose8(x);  // tokens 8 h + 2 quad + {0, 1} of row g
            }
        }
#pragma unroll
        for (int w = 0; w < kValWords; ++w) {
            if (k8) {
                // bytes of tokens (0, 1) and (2, 3) side by side: components 4w .. 4w + 3, two tiles
                uint32_t a = vreg[0][w], b = vreg[1][w], cc = vreg[2][w], d = vreg[3][w];
                if (kFormat == TPS_KV_INT8) a ^= 0x80808080u, b ^= 0x80808080u, cc ^= 0x80808080u, d ^= 0x80808080u;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t ab = __byte_perm(a, b, half ? 0x7362u : 0x5140u), cd = __byte_perm(cc, d, half ? 0x7362u : 0x5140u);
                    uint32_t a0, a1, a2, a3;
                    if (kFormat == TPS_KV_FP8) {
                        a0 = fp8_pair(ab), a1 = fp8_pair(ab >> 16), a2 = fp8_pair(cd), a3 = fp8_pair(cd >> 16);
                    } else {
                        a0 = int8_pair(ab, 0x4140u), a1 = int8_pair(ab, 0x4342u);
                        a2 = int8_pair(cd, 0x4140u), a3 = int8_pair(cd, 0x4342u);
                    }
#pragma unroll
                    for (int n = 0; n < N; ++n)
                        mma16816(st.o[n][(w * 2 + half) % kTiles], a0, a1, a2, a3, p[n][0], p[n][1], true);
                }
            } else {
                const uint32_t a0 = __byte_perm(vreg[0][w], vreg[1][w], 0x5410u), a1 = __byte_perm(vreg[0][w], vreg[1][w], 0x7632u);
                const uint32_t a2 = __byte_perm(vreg[2][w], vreg[3][w], 0x5410u), a3 = __byte_perm(vreg[2][w], vreg[3][w], 0x7632u);
#pragma unroll
                for (int n = 0; n < N; ++n) mma16816(st.o[n][w % kTiles], a0, a1, a2, a3, p[n][0], p[n][1], false);
            }
        }
    }
    if (!k8 && __any_sync(0xFFFFFFFFu, walk.fault & 4)) add_not_finite<D, kFormat, N, kTree>(st, walk, lim, all_see, b, r0, tree);
    walk.fault &= 1;
    return walk.fault;
}

// This lane's part of the sums becomes the row's.
template <int D, int N>
__device__ __forceinline__ void finish_sums(RowState<D, N>& st)
{
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) st.l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, st.l[n][e], o);
}

// Put a warp's first `rows` rows into its part of shared memory.
template <int D, int kFormat, int N>
__device__ __forceinline__ void store_rows(RowsShared<D, kFormat>& sm, RowState<D, N>& st, int rows)
{
    static_assert(sizeof(sm.ring[0]) >= 16 * D * sizeof(float), "the ring holds 16 rows of output");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, quad = lane & 3;
    float* o = reinterpret_cast<float*>(sm.ring[warp]);
    finish_sums(st);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = 8 * n + 2 * quad + e;
            if (row >= rows) continue;
            if (g == 0) {
                sm.m[warp][row] = st.m[n][e];
                sm.l[warp][row] = st.l[n][e];
            }
            float* dst = o + row * D + g * (D / 8);
#pragma unroll
            for (int t = 0; t < D / 16; t += 2)
                *reinterpret_cast<float4*>(dst + 2 * t) =
                    make_float4(st.o[n][t][e], st.o[n][t][2 + e], st.o[n][t + 1][e], st.o[n][t + 1][2 + e]);
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

// The join of the CTA's warps becomes piece `piece` (their rows are in shared memory, after a barrier).
template <int D, int kFormat, int N>
__device__ __forceinline__ void write_piece(const RowsShared<D, kFormat>& sm, float* part, float2* ml, int64_t piece)
{
    constexpr int kRows = 8 * N;
    float* po = part + piece * kRows * D;
    for (int i = threadIdx.x; i < kRows * D / 4; i += kRowsThreads) {
        const int r = i % kRows, col = i / kRows * 4;
        Joined j{sm.m[0][r], 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
        for (int w = 1; w < kRowsWarps; ++w) j.top = fmax_nan(j.top, sm.m[w][r]);
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w)
            j.add(sm.m[w][r], *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.ring[w]) + r * D + col), sm.l[w][r]);
        *reinterpret_cast<float4*>(po + (col / 4 * kRows + r) * 4) = j.acc;
        if (col == 0) ml[piece * kRows + r] = make_float2(j.top, sm.bad == 2 ? kPieceTimeout : (sm.bad ? kPieceBadPage : j.l));
    }
}

// The pieces of the shared prefix that hold a row's item: piece `first` on, `count` of them.
struct Pieces {
    int64_t first;
    int count;
};
__device__ __forceinline__ Pieces pieces_of(const AttnPlan& p, int64_t item)
{
    const int first = (int)item * p.nblk, c0 = first / p.share, c1 = (first + p.nblk - 1) / p.share;
    return Pieces{c0 + item, c1 - c0 + 1};
}

// 1 / sum as the output takes it: 0 where no token was seen, NaN where something was bad.
__device__ __forceinline__ float inverse_sum(float l, bool bad)
{
    if (bad) return __int_as_float(0x7FC00000);
    return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
}

// The join of many parts of a few rows by a CTA.  The parts' (maximum, sum) come in parallel, 64 at a time; a warp
// for each row turns them into weights in shared memory; then every thread adds up its float4 columns with many loads
// on the way at once, the first sixteen since before the weights were known.  The loops are short on purpose: this
// code runs once for a CTA, and instructions that are fetched for one use cost more than they do.
constexpr int kJoinChunk = 64, kFlight = 16, kNearFlight = 8;
template <int kRows> struct JoinShared {
    float2 ml[kRows][kJoinChunk];  // then (weight, -)
    float scale[kRows], top[kRows], l[kRows];
    int state[kRows];  // 1: a bad page, 2: a wait that ran out
};

struct NoPart {
    static constexpr int count = 0;
    __device__ __forceinline__ NoPart operator()(int) const { return *this; }
    __device__ __forceinline__ operator float2() const { return make_float2(0.f, 0.f); }
    __device__ __forceinline__ operator float4() const { return make_float4(0.f, 0.f, 0.f, 0.f); }
};

// Parts of one row (and column) that lie a constant distance apart in memory.
struct PartRow {
    const float2* at;
    int64_t stride;
    int count;
    __device__ __forceinline__ float2 operator()(int j) const { return at[j * stride]; }
};
struct PartCell {
    const float4* at;
    int64_t stride;
    int count;
    __device__ __forceinline__ float4 operator()(int j) const { return at[j * stride]; }
};

// The outputs of a join, by number: `columns` float4 (a power of two) from `first` on of each of `rows` rows.  Parts in
// memory hold a column's values of neighbouring rows side by side: four rows to four lanes (shift 2) use the 32 bytes
// of a sector whole (64 x (8,191 + 60), fp8: 41.2 -> 30.1 us).  In shared memory those would meet in one bank: shift 0
// where there are no pieces of the prefix (8 x 1,000: 10.8 instead of 11.1 us).
struct JoinOut {
    int rows, first, columns, shift;
    __device__ __forceinline__ int row(int i) const { return ((i >> shift) / columns << shift) + (i & ((1 << shift) - 1)); }
    __device__ __forceinline__ int column(int i) const { return first + (i >> shift) % columns; }
    __device__ __forceinline__ bool in(int i) const { return row(i) < rows; }
};

// Join two groups of parts, at most n_near and n_far of any row.  row(r): the (maximum, sum) of row r's parts of the
// group; cell(r, column): their values; both with the row's count.  kMost: outputs of a thread, at most.
template <int kRows, int kMost, typename NearRow, typename NearCell, typename FarRow, typename FarCell>
__device__ __forceinline__ void join_parts(JoinShared<kRows>& sm, const JoinOut& out, float4 (&acc)[kMost], int n_near, NearRow near_row,
                                           NearCell near_cell, int n_far, FarRow far_row, FarCell far_cell)
{
    constexpr int kPerRow = kRowsThreads / kRows, kEach = kJoinChunk / kPerRow;  // threads that fetch a row's (maximum, sum), of each
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rows = out.rows;
    const float neg = -__int_as_float(0x7F800000);
    if (threadIdx.x < kRows) {
        sm.top[threadIdx.x] = neg;
        sm.l[threadIdx.x] = 0.f;
        sm.state[threadIdx.x] = 0;
    }
#pragma unroll
    for (int k = 0; k < kMost; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; c0 < n_near + n_far; c0 += kJoinChunk) {
        __syncthreads();
        const int far0 = max(c0 - n_near, 0);  // the chunk's first far part
        float2 ml[kEach];
        if (threadIdx.x / kPerRow < rows) {
            const int r = threadIdx.x / kPerRow;
            const auto near = near_row(r);
            const auto far = far_row(r);
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int j = c0 + threadIdx.x % kPerRow + k * kPerRow;
                ml[k] = make_float2(neg, 0.f);
                if (j < n_near) {
                    if (j < near.count) ml[k] = near(j);
                } else if (j - n_near < far.count) {
                    ml[k] = far(j - n_near);
                }
            }
        }
        float4 x[kFlight];
        auto fetch = [&](const auto& value, int j, int n) {
#pragma unroll
            for (int t = 0; t < kFlight; ++t) x[t] = value(min(j + t, n - 1));  // past the end: the last one again
        };
        if (out.in(threadIdx.x)) {
            const auto value = far_cell(out.row(threadIdx.x), out.column(threadIdx.x));
            const int n = min(value.count, c0 + kJoinChunk - n_near);
            if (far0 < n) fetch(value, far0, n);
        }
        if (threadIdx.x / kPerRow < rows)
#pragma unroll
            for (int k = 0; k < kEach; ++k) sm.ml[threadIdx.x / kPerRow][threadIdx.x % kPerRow + k * kPerRow] = ml[k];
        __syncthreads();
#pragma unroll 1
        for (int r = warp; r < rows; r += kRowsWarps) {
            float2 x[kJoinChunk / 32];
            const float was = sm.top[r];
            float top = was;
#pragma unroll
            for (int k = 0; k < kJoinChunk / 32; ++k) {
                x[k] = sm.ml[r][lane + 32 * k];
                top = fmax_nan(top, x[k].x);
            }
            top = warp_max_nan(top);
            float l = 0.f;
            int state = 0;
#pragma unroll
            for (int k = 0; k < kJoinChunk / 32; ++k) {
                const float w = join_weight(x[k].x, top);
                state = max(state, x[k].y < 0.f ? (x[k].y == kPieceTimeout ? 2 : 1) : 0);
                l = fmaf(w, x[k].y, l);
                sm.ml[r][lane + 32 * k].x = w;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
            state = (int)warp_max_u32((uint32_t)state);
            if (lane == 0) {
                const float f = join_weight(was, top);
                sm.scale[r] = f;
                sm.top[r] = top;
                sm.l[r] = fmaf(sm.l[r], f, l);
                sm.state[r] = max(sm.state[r], state);
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
            const int i = threadIdx.x + k * kRowsThreads;
            if (!out.in(i)) continue;
            const int r = out.row(i);
            const float f = sm.scale[r];
            float4 y = make_float4(acc[k].x * f, acc[k].y * f, acc[k].z * f, acc[k].w * f);
            auto add = [&](float w, const float4& v) {
                y.x = fmaf(w, v.x, y.x), y.y = fmaf(w, v.y, y.y);
                y.z = fmaf(w, v.z, y.z), y.w = fmaf(w, v.w, y.w);
            };
            const auto near = near_cell(r, out.column(i));
            const int near_n = min(near.count, c0 + kJoinChunk);
#pragma unroll 1
            for (int j = c0; j < near_n; j += kNearFlight) {
                float4 v[kNearFlight];
#pragma unroll
                for (int t = 0; t < kNearFlight; ++t) v[t] = near(min(j + t, near_n - 1));
#pragma unroll
                for (int t = 0; t < kNearFlight; ++t)
                    if (j + t < near_n) add(sm.ml[r][j + t - c0].x, v[t]);
            }
            const auto far = far_cell(r, out.column(i));
            const int n = min(far.count, c0 + kJoinChunk - n_near);
#pragma unroll 1
            for (int j = far0; j < n; j += kFlight) {
                if (k > 0 || j > far0) fetch(far, j, n);
#pragma unroll
                for (int t = 0; t < kFlight; ++t)
                    if (j + t < n) add(sm.ml[r][j + t + n_near - c0].x, x[t]);
            }
            acc[k] = y;
        }
    }
    __syncthreads();
}

// The prefix's pieces for the rows of one tile of a sequence: a tile of the prefix may end inside them.
struct PrefixPieces {
    Pieces mine, next;
    int in0, tile_rows;
    __device__ __forceinline__ PrefixPieces(const AttnPlan& p, int head, int64_t row0, int rows)
        : mine{0, 0}, next{0, 0}, in0(0), tile_rows(p.tile_rows)
    {
        if (!p.shared) return;
        const int t = row0 <= 0x7FFFFFFF ? (int)((uint32_t)row0 / (uint32_t)p.tile_rows) : (int)(row0 / p.tile_rows);
        in0 = (int)(row0 - (int64_t)t * p.tile_rows);
        mine = pieces_of(p, head * p.n_tiles + t);
        if (in0 + rows > p.tile_rows) next = pieces_of(p, head * p.n_tiles + t + 1);
    }
    __device__ __forceinline__ int most() const { return max(mine.count, next.count); }
    __device__ __forceinline__ const Pieces& of(int r) const { return in0 + r >= tile_rows ? next : mine; }
    __device__ __forceinline__ int in_tile(int r) const { return in0 + r >= tile_rows ? in0 + r - tile_rows : in0 + r; }
    __device__ __forceinline__ PartRow row(const AttnArgs& a, int r) const
    {
        return PartRow{a.ml + of(r).first * tile_rows + in_tile(r), tile_rows, of(r).count};
    }
    __device__ __forceinline__ PartCell cell(const AttnArgs& a, int D, int r, int col) const
    {
        return PartCell{reinterpret_cast<const float4*>(a.part) + (of(r).first * (D / 4) + col) * tile_rows + in_tile(r),
                       (int64_t)(D / 4) * tile_rows, of(r).count};
    }
};

// A sequence's status: the worst of what its heads and row tiles met (state 1: a bad page or length, 2: a wait that
// ran out, which concerns one CTA and so maybe a single head).  The call's first kernel clears it, and the joins raise
// it after their wait for that kernel; a call that is one kernel has a small one ahead for this alone (8 x 300: 9.4 us
// without a status array, 10.1 with one).
static_assert(TPS_ROW_TIMEOUT > TPS_ROW_BAD_PARAM && TPS_ROW_BAD_PARAM > TPS_ROW_OK && TPS_ROW_OK == 0, "the worst is the largest");
__device__ __forceinline__ void report_row(const AttnArgs& a, int64_t b, int state)
{
    if (a.a.out_status) atomicMax(&a.a.out_status[b], state == 2 ? TPS_ROW_TIMEOUT : TPS_ROW_BAD_PARAM);
}

__device__ __forceinline__ void clear_status(const AttnArgs& a)
{
    if (a.a.out_status)
        for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < a.a.B; i += (int64_t)gridDim.x * blockDim.x)
            a.a.out_status[i] = TPS_ROW_OK;
}

template <int kFormat>
__device__ __forceinline__ float log_sum(float top, float l, bool bad)
{
    const float lift = kFormat == TPS_KV_BF16 ? 0.f : kLift;
    if (bad) return __int_as_float(0x7FC00000);
    return l == 0.f ? -__int_as_float(0x7F800000) : (top + log2f(l) - lift) * 0.693147180559945f;
}

// Rows from `past` of the sequence on are padding's: they have seen nothing.
template <int D, int N> __device__ __forceinline__ void clear_padding(RowState<D, N>& st, int r0, int past)
{
    const int quad = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (r0 + 8 * n + 2 * quad + e >= past) {
                st.m[n][e] = -__int_as_float(0x7F800000), st.l[n][e] = 0.f;
#pragma unroll
                for (int t = 0; t < D / 16; ++t) st.o[n][t][e] = st.o[n][t][2 + e] = 0.f;
            }
}

// One sequence's own tokens for one key head, then the join with the pieces of the shared prefix, the
// division by the sum and the output.  With many sequences each warp has one for itself, and joins in
// registers; else the four warps of a CTA, or of a cluster of CTAs, take its chunks in turn and join
// through (distributed) shared memory.  A small call has no pieces: every sequence walks over the prefix
// itself (AttnPlan::shared).
template <int D, int kFormat, int N, bool kOneWarp, bool kTree>
__global__ void __launch_bounds__(kRowsThreads, N == 1 ? 4 : 3) attn_suffix_kernel(const AttnArgs a)
{
    constexpr int kRows = 8 * N;
    extern __shared__ __align__(128) unsigned char raw[];
    RowsShared<D, kFormat>& sm = *reinterpret_cast<RowsShared<D, kFormat>*>(raw);
    JoinShared<kRows>& js = *reinterpret_cast<JoinShared<kRows>*>(raw + (sizeof(sm) + 15) / 16 * 16);  // not there where kOneWarp
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
    const int Tq = a.a.q_len, G = a.G, r0 = tile * kRows, rows = min(kRows, Tq * G - r0);
    TreeTokens tree = {};
    if constexpr (kTree) tree = tree_tokens(a, b);
    const int len = kTree ? tree.len : a.a.suffix_len[b];
    const bool fits = kTree ? tree.fits : len >= 0 && len <= a.a.table_width << a.page_shift;
    // Row r of the sequence is query r / G, head r % G of the group: own tokens that it sees.
    auto seen = [&](int r) {
        if constexpr (kTree) return len;
        const int n = len - Tq + 1 + (Tq == 1 ? 0 : min(r, Tq * G - 1) / G);
        return fits && n > 0 ? n : 0;
    };
    auto out_row = [&](int r) {
        const int t = Tq == 1 ? 0 : (r0 + r) / G;
        return (b * Tq + t) * a.a.n_q_heads + (int64_t)head * G + (r0 + r - t * G);
    };
    const int first = kOneWarp ? 0 : (rank * kRowsWarps + warp) * 16, step = kOneWarp ? 16 : ncl * kRowsWarps * 16;
    const bool own_prefix = !p.shared && a.a.prefix_len;
    const int32_t* own_pages = a.a.page_table + b * a.a.table_ld;
    const int64_t capacity = a.a.table_width << a.page_shift;
    Walk<D, kFormat> walk{a, head, sm.ring[warp], sm.full[warp]};
    walk.look(own_prefix ? a.a.prefix_pages : own_pages, first, own_prefix ? a.a.prefix_len : capacity);
    RowState<D, N> st;
    load_query<D, kFormat, N>(st, rows, [&](int r) { return static_cast<const __nv_bfloat16*>(a.a.q) + out_row(r) * D; });
    walk.start(first, step, own_prefix ? (int)a.a.prefix_len : seen(r0 + rows - 1));
    ready_query<D, kFormat, N>(st, a.qk_scale);
    int lim[N][2];
    int fault = 0;
    if (own_prefix) {
#pragma unroll
        for (int n = 0; n < N; ++n) lim[n][0] = lim[n][1] = (int)a.a.prefix_len;
        const int own_first = own_pages && first < capacity ? own_pages[first >> a.page_shift] : 0;  // on its way meanwhile
        fault = attend<D, kFormat, N>(st, walk, lim);
        walk.pages = own_pages, walk.page = own_first;
        walk.start(first, step, fault == 2 ? 0 : seen(r0 + rows - 1));
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) lim[n][e] = seen(r0 + 8 * n + 2 * quad + e);
    fault = max(fault, attend<D, kFormat, N, kTree>(st, walk, lim, b, r0, tree));
    if constexpr (kTree) clear_padding(st, r0, tree.nodes * G);
    const float neg = -__int_as_float(0x7F800000);
    const int64_t row0 = b * Tq * G + r0;  // the tile's first row among the key head's R

    if (kOneWarp) {
        finish_sums(st);
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces of the shared prefix
        const PrefixPieces pieces(p, head, row0, rows);
        bool any_bad = false, any_late = fault == 2;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * n + 2 * quad + e;
                if (row >= rows) continue;
                const Pieces mine = pieces.of(row);
                const int in_tile = pieces.in_tile(row);
                const float2* ml = a.ml + mine.first * p.tile_rows + in_tile;
                float top = st.m[n][e];
                for (int j = 0; j < mine.count; j += 4) {  // four at a time, past the end the last one again
                    float m[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) m[t] = ml[(int64_t)min(j + t, mine.count - 1) * p.tile_rows].x;
#pragma unroll
                    for (int t = 0; t < 4; ++t) top = fmax_nan(top, m[t]);
                }
                const float f0 = join_weight(st.m[n][e], top);
                float l = st.l[n][e] * f0;
                bool bad = fault || !fits, late = fault == 2;
                float acc[D / 8];
#pragma unroll
                for (int t = 0; t < D / 16; ++t) acc[2 * t] = st.o[n][t][e] * f0, acc[2 * t + 1] = st.o[n][t][2 + e] * f0;
                const float4* part = reinterpret_cast<const float4*>(a.part) + (mine.first * (D / 4) + g * (D / 32)) * p.tile_rows + in_tile;
                for (int j = 0; j < mine.count; j += 2) {  // two at a time, past the end with weight 0
                    const int next = min(j + 1, mine.count - 1);
                    const float2 x[2] = {ml[(int64_t)j * p.tile_rows], ml[(int64_t)next * p.tile_rows]};
                    float4 y[2][D / 32];
#pragma unroll
                    for (int t = 0; t < D / 32; ++t) {
                        y[0][t] = part[((int64_t)j * (D / 4) + t) * p.tile_rows];
                        y[1][t] = part[((int64_t)next * (D / 4) + t) * p.tile_rows];
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (k && j + 1 >= mine.count) break;
                        const float f = join_weight(x[k].x, top);
                        bad = bad || x[k].y < 0.f;
                        late = late || x[k].y == kPieceTimeout;
                        l = fmaf(f, x[k].y, l);
#pragma unroll
                        for (int t = 0; t < D / 32; ++t) {
                            acc[4 * t] = fmaf(f, y[k][t].x, acc[4 * t]), acc[4 * t + 1] = fmaf(f, y[k][t].y, acc[4 * t + 1]);
                            acc[4 * t + 2] = fmaf(f, y[k][t].z, acc[4 * t + 2]), acc[4 * t + 3] = fmaf(f, y[k][t].w, acc[4 * t + 3]);
                        }
                    }
                }
                const float inv = inverse_sum(l, bad);
                const int64_t orow = out_row(row);
                uint32_t w[D / 16];
#pragma unroll
                for (int t = 0; t < D / 16; ++t)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[t]) : "f"(acc[2 * t + 1] * inv), "f"(acc[2 * t] * inv));
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.a.out) + orow * D + g * (D / 8));
#pragma unroll
                for (int i = 0; i < D / 64; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                if (g == 0 && a.a.out_lse) a.a.out_lse[orow] = log_sum<kFormat>(top, l, bad);
                any_bad = any_bad || bad;
                any_late = any_late || late;
            }
        any_bad = __any_sync(0xFFFFFFFFu, any_bad);
        any_late = __any_sync(0xFFFFFFFFu, any_late);
        if (lane == 0 && any_bad) report_row(a, b, any_late ? 2 : 1);
    } else {
        store_rows<D, kFormat, N>(sm, st, rows);
        if (lane == 0 && (fault || !fits)) atomicMax(&sm.bad, max(fault, 1));
        if (ncl > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        // Every rank joins a D / ncl columns wide strip, from all CTAs' shared memory and from the pieces.
        const uint32_t base = smem_u32(raw);
        auto peer = [&](const void* x, int who) {
            const uint32_t addr = base + (uint32_t)(static_cast<const unsigned char*>(x) - raw);
            uint32_t out;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(addr), "r"(who));
            return out;
        };
        const PrefixPieces pieces(p, head, row0, rows);
        const int own = ncl * kRowsWarps, columns = D / 4 / ncl;
        const JoinOut out{rows, rank * columns, columns, p.shared ? 2 : 0};
        struct NearRow {
            uint32_t m, l;  // of this CTA's warp 0
            int count;
            __device__ __forceinline__ float2 operator()(int j) const
            {
                float2 x;
                uint32_t at_m, at_l;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at_m) : "r"(m + (j % kRowsWarps) * 64u), "r"(j / kRowsWarps));
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at_l) : "r"(l + (j % kRowsWarps) * 64u), "r"(j / kRowsWarps));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x.x) : "r"(at_m));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x.y) : "r"(at_l));
                return x;
            }
        };
        struct NearCell {
            uint32_t o;
            int count;
            __device__ __forceinline__ float4 operator()(int j) const
            {
                float4 x;
                uint32_t at;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(o + (j % kRowsWarps) * (uint32_t)sizeof(sm.ring[0])), "r"(j / kRowsWarps));
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(at));
                return x;
            }
        };
        static_assert(sizeof(sm.m[0]) == 64 && sizeof(sm.l[0]) == 64, "a warp's sixteen rows");
        constexpr int kMost = (kRows * D / 4 + kRowsThreads - 1) / kRowsThreads;
        float4 acc[kMost];
        int own_bad = 0;
        if (lane < ncl) asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(own_bad) : "r"(peer(&sm.bad, lane)));
        own_bad = (int)warp_max_u32((uint32_t)own_bad);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        auto own_row = [&](int r) { return NearRow{smem_u32(&sm.m[0][r]), smem_u32(&sm.l[0][r]), own}; };
        auto own_cell = [&](int r, int col) { return NearCell{smem_u32(sm.ring[0]) + (uint32_t)(r * D + col * 4) * 4u, own}; };
        if (p.shared)
            join_parts(
                js, out, acc, own, own_row, own_cell, pieces.most(), [&](int r) { return pieces.row(a, r); },
                [&](int r, int col) { return pieces.cell(a, D, r, col); });
        else  // the loads in the wider of the two ways
            join_parts(js, out, acc, 0, [](int) { return NoPart{}; }, [](int, int) { return NoPart{}; }, own, own_row, own_cell);
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
            const int i = threadIdx.x + k * kRowsThreads;
            if (!out.in(i)) continue;
            const int r = out.row(i), col = out.column(i);
            const int state = max(js.state[r], own_bad);
            const float inv = inverse_sum(js.l[r], state != 0);
            const int64_t orow = out_row(r);
            uint2 w;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(acc[k].y * inv), "f"(acc[k].x * inv));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(acc[k].w * inv), "f"(acc[k].z * inv));
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.a.out) + orow * D + col * 4) = w;
            if (col == 0 && a.a.out_lse) a.a.out_lse[orow] = log_sum<kFormat>(js.top[r], js.l[r], state != 0);
            if (col == 0 && state) report_row(a, b, state);
        }
        if (ncl > 1) {  // no CTA may leave while others read its shared memory
            cluster_arrive();
            cluster_wait();
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Few sequences with many tokens of their own: their lengths differ, so the tokens are cut evenly instead.
// The 64-token blocks of all (sequence, row tile, key head) items form one line, whose length only the
// device knows: every CTA adds up the sequences' blocks, then takes its share of the line and leaves a
// piece for each item it meets, as for the prefix; a last kernel joins the pieces.  Where the prefix is
// not shared, its blocks come first in each item.
// ---------------------------------------------------------------------------------------------
constexpr int kLineMax = 1024;  // (sequence, row tile) pairs that a CTA adds up
constexpr int kLineBlock = kRowsWarps * 16;

// Tokens of its own that the last row of a tile sees (0 where the length is bad), and whether it is not.
struct OwnTokens {
    int seen;
    bool fits;
};
template <bool kTree> __device__ __forceinline__ OwnTokens own_tokens(const AttnArgs& a, int64_t b, int row)
{
    if constexpr (kTree) {
        const TreeTokens t = tree_tokens(a, b);
        return OwnTokens{t.len, t.fits};
    }
    const int len = a.a.suffix_len[b], Tq = a.a.q_len;
    const bool fits = len >= 0 && len <= a.a.table_width << a.page_shift;
    const int n = len - Tq + 1 + (Tq == 1 ? 0 : min(row, Tq * a.G - 1) / a.G);
    return OwnTokens{fits && n > 0 ? n : 0, fits};
}

// Blocks of the pairs before each one, before[pairs] and on: all of them.  8 consecutive pairs for each thread.
struct LineSums {
    int64_t before[kLineMax + 1], warp_sum[kRowsWarps];
};
template <bool kTree> __device__ __forceinline__ void line_sums(LineSums& sm, const AttnArgs& a, int tile_rows)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pairs = (int)(a.a.B * a.p.suffix_tiles), rows = a.a.q_len * a.G;
    const int shared_blocks = a.p.shared ? 0 : ((int)a.a.prefix_len + kLineBlock - 1) / kLineBlock;
    constexpr int kEach = kLineMax / kRowsThreads;
    int64_t mine[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int bt = threadIdx.x * kEach + i;
        mine[i] = sum;
        if (bt < pairs) {
            const int b = bt / a.p.suffix_tiles, tile = bt - b * a.p.suffix_tiles;
            sum += shared_blocks + (own_tokens<kTree>(a, b, min(rows, (tile + 1) * tile_rows) - 1).seen + kLineBlock - 1) / kLineBlock;
        }
    }
    int64_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) sm.warp_sum[warp] = upto;
    __syncthreads();
    int64_t base = upto - sum;
    for (int w = 0; w < warp; ++w) base += sm.warp_sum[w];
#pragma unroll
    for (int i = 0; i < kEach; ++i) sm.before[threadIdx.x * kEach + i] = base + mine[i];
    if (threadIdx.x == kRowsThreads - 1) sm.before[kLineMax] = base + sum;
    __syncthreads();
}

template <int D, int kFormat, int N, bool kTree>
__global__ void __launch_bounds__(kRowsThreads, N == 1 ? 4 : 3) attn_line_kernel(const AttnArgs a)
{
    constexpr int kRows = 8 * N;
    extern __shared__ __align__(128) unsigned char raw[];
    RowsShared<D, kFormat>& sm = *reinterpret_cast<RowsShared<D, kFormat>*>(raw);
    LineSums& sums = *reinterpret_cast<LineSums*>(raw + (sizeof(sm) + 15) / 16 * 16);
    const AttnPlan& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane & 3;
    const int heads = a.c.n_heads, pairs = (int)(a.a.B * p.suffix_tiles), Tq = a.a.q_len, G = a.G;
    init_rings(sm);
    if (!p.shared) clear_status(a);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int shared_len = p.shared ? 0 : (int)a.a.prefix_len, shared_blocks = (shared_len + kLineBlock - 1) / kLineBlock;
    line_sums<kTree>(sums, a, kRows);
    const int64_t* before = sums.before;
    const int64_t total = before[kLineMax] * heads;

    Walk<D, kFormat> walk{a, 0, sm.ring[warp], sm.full[warp]};
    const int64_t share = (total + p.line_ctas - 1) / p.line_ctas, u0 = blockIdx.x * share, u1 = min(u0 + share, total);
    bool gave_up = false;
    for (int64_t u = u0; u < u1;) {
        // The pair whose blocks, once for each head, hold block u of the line.
        int lo = 0, hi = pairs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before[mid] * heads <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int bt = lo, b = bt / p.suffix_tiles, tile = bt - b * p.suffix_tiles;
        const int64_t blocks = (bt + 1 < pairs ? before[bt + 1] : before[kLineMax]) - before[bt];
        const int head = (int)((u - before[bt] * heads) / blocks);
        const int64_t start = before[bt] * heads + head * blocks, end = min(u1, start + blocks);
        const int r0 = tile * kRows, rows = min(kRows, Tq * G - r0);
        const int first = (int)(u - start), past = (int)(end - start);  // blocks of the item
        if (!gave_up) {
            // Its blocks of the prefix (where each sequence walks over it itself), then its own.
            const int p0 = min(first, shared_blocks) * kLineBlock, p1 = min(min(past, shared_blocks) * kLineBlock, shared_len);
            const int seen = own_tokens<kTree>(a, b, r0 + rows - 1).seen;
            const int t0 = max(first - shared_blocks, 0) * kLineBlock, t1 = min(max(past - shared_blocks, 0) * kLineBlock, seen);
            const int32_t* own_pages = a.a.page_table + b * a.a.table_ld;
            walk.head = head;
            walk.look(p0 < p1 ? a.a.prefix_pages : own_pages, (p0 < p1 ? p0 : t0) + warp * 16, p0 < p1 ? p1 : t1);
            RowState<D, N> st;
            load_query<D, kFormat, N>(st, rows, [&](int r) {
                const int t = Tq == 1 ? 0 : (r0 + r) / G;
                return static_cast<const __nv_bfloat16*>(a.a.q) +
                       (((int64_t)b * Tq + t) * a.a.n_q_heads + (int64_t)head * G + (r0 + r - t * G)) * D;
            });
            walk.start((p0 < p1 ? p0 : t0) + warp * 16, kRowsWarps * 16, p0 < p1 ? p1 : t1);
            ready_query<D, kFormat, N>(st, a.qk_scale);
            int lim[N][2];
            int fault = 0;
            if (p0 < p1) {
#pragma unroll
                for (int n = 0; n < N; ++n) lim[n][0] = lim[n][1] = p1;
                fault = attend<D, kFormat, N>(st, walk, lim);
                walk.look(own_pages, t0 + warp * 16, t1);
                walk.start(t0 + warp * 16, kRowsWarps * 16, fault == 2 ? 0 : t1);
            }
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) lim[n][e] = min(t1, own_tokens<kTree>(a, b, r0 + 8 * n + 2 * quad + e).seen);
            TreeTokens tree = {};
            if constexpr (kTree) tree = tree_tokens(a, b);
            fault = max(fault, attend<D, kFormat, N, kTree>(st, walk, lim, b, r0, tree));
            if constexpr (kTree) clear_padding(st, r0, tree.nodes * G);
            store_rows<D, kFormat, N>(sm, st, kRows);
            if (fault && lane == 0) atomicMax(&sm.bad, fault);
        }
        __syncthreads();
        gave_up = sm.bad == 2;
        write_piece<D, kFormat, N>(sm, a.line_part, a.line_ml, blockIdx.x + (int64_t)bt * heads + head);
        __syncthreads();
        if (threadIdx.x == 0 && !gave_up) sm.bad = 0;  // a bad page is this item's alone
        walk.fault = 0;
        fence_proxy_async();  // the rings held output: those accesses come before the next copies into them
        __syncthreads();
        u = end;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // this grid ends after the prefix's, so the join need wait for this one only
}

// The join: a CTA for each item and strip of 32 columns.
constexpr int kStrip = 32;
template <int D, int kFormat, bool kTree>
__global__ void __launch_bounds__(kRowsThreads) attn_join_kernel(const AttnArgs a)
{
    __shared__ JoinShared<16> js;
    __shared__ LineSums sums;
    const AttnPlan& p = a.p;
    const int heads = a.c.n_heads, Tq = a.a.q_len, G = a.G;
    const uint32_t bt = blockIdx.x / (uint32_t)heads;
    const int head = (int)(blockIdx.x - bt * heads);
    const int64_t b = bt / (uint32_t)p.suffix_tiles;
    const int tile = (int)(bt - (uint32_t)b * p.suffix_tiles);
    const int r0 = tile * p.suffix_rows, rows = min(p.suffix_rows, Tq * G - r0);
    const int64_t row0 = b * Tq * G + r0;
    const bool fits = own_tokens<kTree>(a, b, 0).fits;
    Pieces own{0, 0};
    const PrefixPieces pieces(p, head, row0, rows);
    line_sums<kTree>(sums, a, p.suffix_rows);  // while the line is still at work
    const int64_t total = sums.before[kLineMax] * heads, before = sums.before[bt];
    const int64_t blocks = ((int64_t)bt + 1 < a.a.B * p.suffix_tiles ? sums.before[bt + 1] : sums.before[kLineMax]) - before;
    if (blocks) {
        const int64_t start = before * heads + head * blocks;
        const int64_t share = (total + p.line_ctas - 1) / p.line_ctas, c0 = start / share, c1 = (start + blocks - 1) / share;
        own = Pieces{c0 + (int64_t)bt * heads + head, (int)(c1 - c0 + 1)};
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kMost = 16 * (kStrip / 4) / kRowsThreads, kColumns = kStrip / 4;
    float4 acc[kMost];
    const JoinOut out{rows, (int)blockIdx.y * kColumns, kColumns, 2};
    join_parts(
        js, out, acc, pieces.most(), [&](int r) { return pieces.row(a, r); },
        [&](int r, int col) { return pieces.cell(a, D, r, col); }, own.count,
        [&](int r) { return PartRow{a.line_ml + own.first * p.suffix_rows + r, p.suffix_rows, own.count}; },
        [&](int r, int col) {
            return PartCell{reinterpret_cast<const float4*>(a.line_part) + (own.first * (D / 4) + col) * p.suffix_rows + r,
                            (int64_t)(D / 4) * p.suffix_rows, own.count};
        });
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
        const int i = threadIdx.x + k * kRowsThreads;
        if (!out.in(i)) continue;
        const int r = out.row(i), col = out.column(i), state = max(js.state[r], fits ? 0 : 1);
        const float inv = inverse_sum(js.l[r], state != 0);
        const int t = (r0 + r) / G;
        const int64_t orow = (b * Tq + t) * a.a.n_q_heads + (int64_t)head * G + (r0 + r - t * G);
        uint2 w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(acc[k].y * inv), "f"(acc[k].x * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(acc[k].w * inv), "f"(acc[k].z * inv));
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.a.out) + orow * D + col * 4) = w;
        if (col == 0 && a.a.out_lse) a.a.out_lse[orow] = log_sum<kFormat>(js.top[r], js.l[r], state != 0);
        if (col == 0 && state) report_row(a, b, state);
    }
}

}  // namespace tps
