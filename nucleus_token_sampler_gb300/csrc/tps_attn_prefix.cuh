// tps_attn_prefix.cuh -- the shared part of tps_prefix_attention on the tcgen05 matrix unit: all query
// rows of one key head (R = B Tq G of them) against the keys and values that every sequence shares.
//
// Mathematics.  As in tps_attn_rows.cuh: weights 2^(z - m) with a reference m per row that is raised only
// when a score exceeds it by more than kSlack; m is a whole number here, so that raising it scales what
// was already computed by an exact power of two.  8-bit formats become float16 on the way to the matrix
// unit.  For every block of 128 tokens the scales are taken in the block's unit, a power of two: nk for keys and
// nv for values.  Codes of fp8 are multiplied by their scale in that unit.  Codes of int8 stay whole numbers (7 bits
// times a scale's 8 would be rounded to float16's 11): the scores take the keys' scales, and a weight takes its
// value's scale in float32, before its one rounding.  The block's units stay scalars outside: z = (q.k') nk, and the
// weights take log2(nv) in their exponent (the row sum divides by nv again).
//
// float16 holds a scale in its block's unit only so far: a token may attract all the weight with values 2^-20 of its
// neighbours' (whose small weights, in the same unit, keep few bits), and next to a key 2^26 times the others' those
// would vanish.  A block whose scales lie further apart than 2^kSpread (or, in fp8, are no powers of two) is wide: its
// codes stay as they are, each score takes its key's scale and each weight's exponent its value's, as for own tokens,
// and the sum takes that out again.  A cache of nothing but wide blocks takes 49 us instead of 35 (64 x 8,191 in fp8) or
// 711 instead of 298 (1,024 x 16,384); that the softmax can do so costs the other blocks registers and instructions
// (33.5 and 290 us without it, 143 and 146 in int8 for 48 x 5 x 20,011).
//
// What bounds it: with R of some hundreds, the matrix unit (512 clocks per 128 x 128 tile at D = 128) and
// next to it the exponentials (one for each of its 16,384 weights) and the conversion of 8-bit codes; with
// fewer rows, the bytes of the cache.  One CTA per SM; the blocks of all items form one line that is
// cut evenly (AttnPlan).  A CTA holds one or two tiles of 128 query rows: with two, one tile's softmax
// runs while the other's products do, and each block of keys and values is loaded and converted once
// for 256 rows.  Measured with 8 key heads of 128: 1,024 x 4 rows on 16,384 tokens take 169 us in bfloat16 (1.62
// PFLOP/s, the matrix unit 53% busy at half that length under a profiler) and 223 us in fp8 (1.23 PFLOP/s; the conversion
// and the softmax share the issue slots); 48 x 25 rows of 64 on 20,011 tokens 114 us in int8 (0.43 PFLOP/s: half the
// products for the same weights; 95 us where the values' scales were rounded into the codes, which cost a second
// 2^-11); 4 x 4 rows on 16,384 tokens 26 us with the join (2.6 TB/s).  A third score buffer, so that scores run ahead of
// the softmax, helped D = 64 (92.1 -> 88.8 us in bfloat16) and cost D = 128 more (125.5 -> 132.9 us): each tile has
// one.  Roles:
//   warps 0 .. 4 kTiles - 1   softmax, one thread per query row: scores from TMEM, weights back to
//                             TMEM over them, where they are the first operand of the second product
//   the next warp             issues every product
//   one warp                  loads tiles: bf16 by TMA into place, 8-bit codes by bulk copies
//   8-bit: one warp           brings the tokens' scales to a tile's unit
//   8-bit: eight warps        convert code tiles to float16 ones
// Shared memory: the query tiles and a ring of 128-token tiles (keys, values, keys, ...), in the 128-byte
// swizzle, and a ring of code tiles; TMEM: scores and outputs of each tile.  Every wait is bounded: a wait that runs
// out makes all roles leave, and the pieces say so.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include "tps_attn_rows.cuh"
#include "tps_decode.h"
#include "tps_tcgen05.cuh"

namespace tps {

constexpr int kScalars = 8;         // blocks whose scale factors are kept
constexpr int kSpread = 8;          // down to 2^-8 of its block's unit a scale times any code is exact (fp8), and small weights keep their bits

template <int D, int kFormat, int kTiles> struct PrefixShape {
    static constexpr bool k8 = kFormat != TPS_KV_BF16;
    static constexpr int kMmaWarp = 4 * kTiles, kLoadWarp = kMmaWarp + 1, kScaleWarp = kMmaWarp + 2;
    static constexpr int kConvertWarp = kMmaWarp + 4, kConvertWarps = 8;
    static constexpr int kThreads = (kConvertWarp + (k8 ? kConvertWarps : 0)) * 32;
    // Registers where the roles share them out: 640 threads at 96 at launch, 2 x 144 + 3 x 64 = 5 x 96 (fp8, whose
    // conversion needs fewer: 2 x 152 + 3 x 56), or 512 threads at 128, 200 + 3 x 104 = 4 x 128.
    static constexpr bool kSplitRegs = kFormat == TPS_KV_INT8 || (k8 && kTiles == 2);
    static constexpr bool kFp8 = kFormat == TPS_KV_FP8;
    static constexpr int kRegsLaunch = kTiles == 2 ? 96 : 128, kRegsSoftmax = kTiles == 2 ? (kFp8 ? 152 : 144) : 200,
                         kRegsOthers = kTiles == 2 ? (kFp8 ? 56 : 64) : 104;
    static_assert(kTiles * kRegsSoftmax + 3 * kRegsOthers <= (kTiles + 3) * kRegsLaunch, "no more than the launch gave");
    static constexpr int kTileBytes = 128 * D * 2;         // a query, key or value tile
    static constexpr int kRing = k8 && D == 128 && kTiles == 2 ? 3 : 4;  // key and value tiles in shared memory
    static constexpr int kRaw = D == 128 ? 3 : 4;          // tiles of 8-bit codes
    static constexpr int kRawBytes = 128 * D + 128 * 2;    // codes and scales of a tile
    static constexpr int kTmemCols = kTiles == 2 ? 512 : 256;
    static constexpr int kScoreCol = 0, kOutCol = 128 * kTiles;  // tile m: scores at 128 m, outputs at kOutCol + D m
    struct Control {
        uint64_t q_full, full[kRing], empty[kRing], s_full[kTiles], p_full[kTiles], o_full[kTiles], drain;
        uint64_t tail[kRing];  // bf16: the rows past the prefix of the value tile in this slot are zero
        uint64_t raw_full[kRaw], factor_full[kRaw], raw_empty[kRaw], scalar_full[kScalars];
        uint32_t tmem;
        int abort, bad;
        float key_unit[kScalars], value_exp[kScalars];
        int wide[kScalars];  // 1: the block's keys, 2: its values
        // Of the block's tokens: keys' scales (int8, or wide), values' in the block's unit, at most 1 (int8), or one over
        // them and their base-2 logarithms (wide).
        alignas(16) float key_scale[k8 ? kScalars : 1][128], value_scale[k8 ? kScalars : 1][128], value_log[k8 ? kScalars : 1][128];
        alignas(16) __half factor[kFormat == TPS_KV_FP8 ? kRaw : 1][128];  // fp8: of the tokens of a code tile
    };
    static constexpr size_t kSmem =
        (size_t)(kTiles + kRing) * kTileBytes + (k8 ? (size_t)kRaw * kRawBytes : 0) + sizeof(Control) + 1024;
    static_assert(kSmem <= 232448, "fits one CTA's shared memory");
};

// Byte of 16-byte chunk c of row r in a tile: 64-element column blocks of 128 rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_byte(int r, int c)
{
    return (uint32_t)((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// A CTA's way along the line of blocks, item by item.
struct Way {
    int item, head, tile, block, left;  // tile: row tile of the head; block: of the item; left: blocks of the CTA from here on
    __device__ __forceinline__ explicit Way(const AttnPlan& p)
    {
        const int u0 = (int)blockIdx.x * p.share;
        left = min(p.share, p.units - u0);
        item = u0 / p.nblk;
        block = u0 - item * p.nblk;
        head = item / p.n_tiles;
        tile = item - head * p.n_tiles;
    }
    __device__ __forceinline__ int blocks(const AttnPlan& p) const { return min(left, p.nblk - block); }  // of this item
    __device__ __forceinline__ void next(const AttnPlan& p)
    {
        left -= blocks(p);
        block = 0;
        ++item;
        if (++tile == p.n_tiles) tile = 0, ++head;
    }
    __device__ __forceinline__ void step(const AttnPlan& p)  // one block on
    {
        --left;
        if (++block == p.nblk) {
            block = 0;
            ++item;
            if (++tile == p.n_tiles) tile = 0, ++head;
        }
    }
};

// A place in a ring of barriers: which one, and the parity of its present phase.
template <int kSlots> struct Turn {
    int slot = 0;
    uint32_t parity;
    __device__ __forceinline__ explicit Turn(uint32_t parity_) : parity(parity_) {}
    __device__ __forceinline__ void next()
    {
        if (++slot == kSlots) slot = 0, parity ^= 1;
    }
};

template <int D, int kFormat, int kTiles>
__global__ void __launch_bounds__(PrefixShape<D, kFormat, kTiles>::kThreads, 1)
    attn_prefix_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using Shape = PrefixShape<D, kFormat, kTiles>;
    using Control = typename Shape::Control;
    constexpr bool k8 = Shape::k8;
    constexpr int kRing = Shape::kRing, kRaw = Shape::kRaw;
    extern __shared__ unsigned char raw_smem[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    unsigned char* q_tile = smem;
    unsigned char* ring = smem + kTiles * Shape::kTileBytes;
    unsigned char* raw_ring = ring + kRing * Shape::kTileBytes;
    Control& ctl = *reinterpret_cast<Control*>(raw_ring + (k8 ? kRaw * Shape::kRawBytes : 0));

    const AttnPlan& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int prefix = (int)a.a.prefix_len;

    if (threadIdx.x == 0) {
        mbar_init(&ctl.q_full, 4 * kTiles);
        for (int i = 0; i < kRing; ++i) mbar_init(&ctl.full[i], k8 ? Shape::kConvertWarps : 1), mbar_init(&ctl.empty[i], 1), mbar_init(&ctl.tail[i], 1);
        for (int i = 0; i < kTiles; ++i) mbar_init(&ctl.s_full[i], 1), mbar_init(&ctl.p_full[i], 128), mbar_init(&ctl.o_full[i], 1);
        for (int i = 0; i < kScalars; ++i) mbar_init(&ctl.scalar_full[i], 1);
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(&ctl.raw_full[i], 1);
            mbar_init(&ctl.factor_full[i], 1);
            mbar_init(&ctl.raw_empty[i], Shape::kConvertWarps);
        }
        mbar_init(&ctl.drain, 1);
        ctl.abort = 0;
        ctl.bad = 0;
        fence_proxy_async();
    }
    if (warp == Shape::kMmaWarp) tmem_alloc(&ctl.tmem, Shape::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    clear_status(a);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    volatile int* abort_flag = &ctl.abort;
    // Wait for a phase; false once any role has given up (this one after a.wait_ns).
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        for (;;) {
            if (mbar_try_wait(bar, parity, 20000u)) return true;  // suspended, not spinning
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > a.wait_ns) {
                *abort_flag = 1;
                return false;
            }
        }
    };
    // The same for a whole warp, whose lanes go on or give up together.
    auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0; };
    bool alive = true;
    if constexpr (Shape::kSplitRegs) {
        if (warp < 4 * kTiles)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Shape::kRegsSoftmax));
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Shape::kRegsOthers));
    }

    if (warp < 4 * kTiles) {
        // ---------------------------------------------------------------------------- softmax
        const int m = warp >> 2;
        const int in_tile = (int)threadIdx.x;  // row of the CTA's kTiles * 128
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lanes + Shape::kScoreCol + 128 * m, o_addr = tmem + lanes + Shape::kOutCol + D * m;
        const float neg = -__int_as_float(0x7F800000);
        unsigned char* my_q = q_tile + m * Shape::kTileBytes;
        uint32_t s_parity = 0, o_parity = 0;
        Turn<kScalars> scalar(0);
        const uint32_t sign = a.qk_scale < 0.f ? 0x80008000u : 0u;
        const float unit = fabsf(a.qk_scale);
        Way way(p);
        for (; way.left > 0 && alive; way.next(p)) {
            // The warp's 32 query rows, D / 8 lanes to a row: as they are (bf16) or brought into float16's range.
            float row_unit = unit;
            {
                constexpr int kLanes = D / 8, kRows = 32 / kLanes, kSteps = 32 / kRows;  // lanes of a row, rows at a time
                const int piece = lane % kLanes, sub = lane / kLanes;
                const int64_t first = (int64_t)way.tile * (128 * kTiles) + warp * 32 + sub, row_elems = (int64_t)a.a.n_q_heads * D;
                // row = bt G + gi lies at bt * row_elems + (head G + gi) D; kRows rows on without a division
                const int64_t bt = first <= 0x7FFFFFFF ? (uint32_t)first / (uint32_t)a.G : first / a.G;
                int gi = (int)(first - bt * a.G);
                const int wraps = kRows / a.G, rem = kRows - wraps * a.G;
                const __nv_bfloat16* src =
                    static_cast<const __nv_bfloat16*>(a.a.q) + bt * row_elems + ((int64_t)way.head * a.G + gi) * D + piece * 8;
                // All on their way at once, straight to their places; loops and not unrolled code, whose instructions
                // would be fetched for this one use.
                auto place = [&](int i) { return my_q + tile_byte((warp & 3) * 32 + i * kRows + sub, piece); };
#pragma unroll 2
                for (int i = 0; i < kSteps; ++i) {
                    const bool in = first + i * kRows < p.R;  // else zeros
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(place(i))),
                                 "l"(in ? static_cast<const void*>(src) : a.a.q), "r"(in ? 16 : 0)
                                 : "memory");
                    const bool over = gi + rem >= a.G;
                    src += (wraps + over) * row_elems + (rem - (over ? a.G : 0)) * D;
                    gi += rem - (over ? a.G : 0);
                }
                asm volatile("cp.async.wait_all;" ::: "memory");  // each lane goes on with what it copied itself
                float row_f = 1.f;                                // of this lane's row, row `lane` of the warp
                if (k8 || sign) {
                    constexpr int kAtOnce = 4;
#pragma unroll 1
                    for (int i0 = 0; i0 < kSteps; i0 += kAtOnce) {
                        uint32_t x[kAtOnce][4], most[kAtOnce];
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) {
                            const uint4 w = *reinterpret_cast<const uint4*>(place(i0 + i));
                            x[i][0] = w.x ^ sign, x[i][1] = w.y ^ sign, x[i][2] = w.z ^ sign, x[i][3] = w.w ^ sign;
                            // magnitudes order like their bits (a NaN or an infinity leaves the row as it is)
                            most[i] = 0;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                most[i] = max(most[i], x[i][k] & 0x7FFF0000u);
                                most[i] = max(most[i], x[i][k] << 16 & 0x7FFF0000u);
                            }
                        }
                        if (k8) {
#pragma unroll
                            for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
                                for (int i = 0; i < kAtOnce; ++i) most[i] = max(most[i], __shfl_xor_sync(0xFFFFFFFFu, most[i], o));
#pragma unroll
                            for (int i = 0; i < kAtOnce; ++i) {
                                const float f = f16_row_scale(__uint_as_float(most[i]));
                                const float other = __shfl_sync(0xFFFFFFFFu, f, (lane % kRows) * kLanes);  // row i kRows + lane % kRows
                                if (lane / kRows == i0 + i) row_f = other;
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const __half2 h =
                                        __floats2half2_rn(__uint_as_float(x[i][k] << 16) * f, __uint_as_float(x[i][k] & 0xFFFF0000u) * f);
                                    x[i][k] = *reinterpret_cast<const uint32_t*>(&h);
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i)
                            *reinterpret_cast<uint4*>(place(i0 + i)) = make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
                    }
                }
                row_unit = unit / row_f;
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.q_full);
            }
            float ref = neg, sum = 0.f;
            const int blocks = way.blocks(p);
            for (int v = 0; v < blocks; ++v) {
                if (!(alive = wait_all(&ctl.s_full[m], s_parity))) break;
                s_parity ^= 1;
                tc_fence_after();
                float c = row_unit, add = 0.f, inv = 1.f;
                int wide = 0;
                const int scales = scalar.slot;
                if (k8) {
                    if (!(alive = wait_all(&ctl.scalar_full[scalar.slot], scalar.parity))) break;
                    c *= ctl.key_unit[scalar.slot];
                    add = ctl.value_exp[scalar.slot];
                    inv = exp2_fast(-add);
                    wide = ctl.wide[scalar.slot];
                    scalar.next();
                }
                c = fmaxf(c, 0x1p-126f);  // never 0: a masked score, -inf, times it stays -inf (any other times that is nothing)
                const int left = prefix - (way.block + v) * kBlockKeys;
                float2 total = make_float2(0.f, 0.f);
                // int8: a score's key scale (the codes are in the tile as they are).  Scores past the prefix become -inf.
                auto ready = [&](float (&s)[32], int ch) {
                    if constexpr (kFormat == TPS_KV_INT8) {
                        const float4* f = reinterpret_cast<const float4*>(ctl.key_scale[scales] + ch * 32);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 x = f[i];
                            const float2 y = mul2(make_float2(s[4 * i], s[4 * i + 1]), make_float2(x.x, x.y));
                            const float2 z = mul2(make_float2(s[4 * i + 2], s[4 * i + 3]), make_float2(x.z, x.w));
                            s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = z.x, s[4 * i + 3] = z.y;
                        }
                    }
                    if (left < ch * 32 + 32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (ch * 32 + i >= left) s[i] = neg;
                    }
                };
                auto largest = [&](const float (&s)[32]) {
                    float t = s[0];
#pragma unroll
                    for (int i = 1; i < 32; ++i) t = fmaxf(t, s[i]);
                    return t;
                };
                // Raise the reference of a row that needs it (the warp's others go along with factor 1, so that no row's
                // bits depend on its neighbours): scale the sum, the output and the weights of chunks 0 .. done - 1.
                auto raise = [&](bool need, float top, int done) {
                    const float to = need && top > ref ? ceilf(top) : ref;
                    const float f = to == ref ? 1.f : exp2_fast(ref - to);
                    ref = to;
                    sum *= f;
                    total.x *= f, total.y *= f;
                    if (v > 0) {
#pragma unroll 1
                        for (int i = 0; i < D; i += 16) {
                            uint32_t o[16];
                            tmem_ld16(o_addr + i, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st16(o_addr + i, o);
                        }
                    }
#pragma unroll 1
                    for (int i = 0; i < done; ++i) {
                        uint32_t w[16];
                        tmem_wait_st();
                        tmem_ld16(s_addr + i * 16, w);
                        tmem_wait_ld(w);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (k8) {
                                const __half2 h = __hmul2(*reinterpret_cast<__half2*>(&w[j]), __float2half2_rn(f));
                                w[j] = *reinterpret_cast<const uint32_t*>(&h);
                            } else {
                                const __nv_bfloat162 h = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&w[j]), __float2bfloat162_rn(f));
                                w[j] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                        }
                        tmem_st16(s_addr + i * 16, w);
                    }
                };
                // Weights of 32 scores, to columns [16 ch, 16 ch + 16), whose scores have been read; their sum.
                auto weigh = [&](const float (&s)[32], int ch, float b) {
                    float2 part[2];
                    uint32_t w[16];
                    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float2 x = fma2(make_float2(s[i], s[i + 1]), make_float2(c, c), make_float2(b, b));
                        x.x = exp2_fast(x.x), x.y = exp2_fast(x.y);
                        part[(i >> 1) & 1] = i < 4 ? x : add2(part[(i >> 1) & 1], x);
                        if constexpr (kFormat == TPS_KV_INT8) {  // the value's scale, after the sum and before the rounding
                            if (i % 4 == 0) f = reinterpret_cast<const float4*>(ctl.value_scale[scales] + ch * 32)[i / 4];
                            x = mul2(x, i % 4 == 0 ? make_float2(f.x, f.y) : make_float2(f.z, f.w));
                        }
                        if (k8) {
                            const __half2 h = __floats2half2_rn(x.x, x.y);
                            w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
                        } else {
                            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i / 2]) : "f"(x.y), "f"(x.x));
                        }
                    }
                    tmem_st16(s_addr + ch * 16, w);
                    return add2(part[0], part[1]);
                };
                // 32 scores of a wide block, against their largest: the exponents take the scales, and the sum adds up the
                // weights without their values' scales.
                auto weigh_wide = [&](float (&s)[32], int ch) {
                    const bool keys = kFormat == TPS_KV_FP8 && (wide & 1), values = wide & 2;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        float4 l = reinterpret_cast<const float4*>(ctl.value_log[scales] + ch * 32)[i / 4];
                        if (!values) l = make_float4(add, add, add, add);
                        const float ll[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float y = keys ? s[i + j] * ctl.key_scale[scales][ch * 32 + i + j] : s[i + j];
                            s[i + j] = s[i + j] == neg ? neg : fmaf(y, c, ll[j]);
                        }
                    }
                    const float top = largest(s);
                    const bool need = top > ref + kSlack;
                    if (__any_sync(0xFFFFFFFFu, need)) raise(need, top, ch);
                    const float b = (ref == neg ? 0.f : -ref) + kLift;
                    float2 t = make_float2(0.f, 0.f);
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 x = make_float2(exp2_fast(s[i] + b), exp2_fast(s[i + 1] + b));
                        const float2 inv_s = reinterpret_cast<const float2*>(ctl.value_scale[scales] + ch * 32)[i / 2];
                        t = fma2(x, values ? inv_s : make_float2(1.f, 1.f), t);
                        const __half2 h = __floats2half2_rn(x.x, x.y);
                        w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    tmem_wait_st();
                    tmem_st16(s_addr + ch * 16, w);
                    return t;
                };
                // 64 scores at a time, first weighed against the reference as it stands: a weight above 2^kSlack
                // (times the lift) shows in their sum, so the usual step looks for no maximum at all.
                constexpr float kMost = k8 ? 32768.f : 256.f;  // 2^(kSlack + kLift), 2^kSlack
#pragma unroll
                for (int ch = 0; ch < 4; ch += 2) {
                    float sa[32], sb[32];
                    tmem_ld32(s_addr + ch * 32, sa);
                    tmem_ld32(s_addr + ch * 32 + 32, sb);
                    tmem_wait_ld(sa);
                    tmem_wait_ld(sb);
                    ready(sa, ch);
                    ready(sb, ch + 1);
                    float b = add - (ref == neg ? 0.f : ref) + (k8 ? kLift : 0.f);
                    float2 x = add2(weigh(sa, ch, b), weigh(sb, ch + 1, b));
                    const bool need = !(x.x + x.y <= kMost) || ref == neg;
                    if (__any_sync(0xFFFFFFFFu, need || wide)) {  // a wide block comes this way every time
                        if (!k8 || !wide) {
                            raise(need, fmaf(fmaxf(largest(sa), largest(sb)), c, add), ch);
                            b = add - (ref == neg ? 0.f : ref) + (k8 ? kLift : 0.f);
                            tmem_wait_st();
                            x = add2(weigh(sa, ch, b), weigh(sb, ch + 1, b));
                        } else {
                            x = weigh_wide(sa, ch);  // may scale the total, so not inside its sum
                            total = add2(total, x);
                            x = weigh_wide(sb, ch + 1);
                        }
                    }
                    total = add2(total, x);
                }
                sum = fmaf(total.x + total.y, inv, sum);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&ctl.p_full[m]);
            }
            if (alive) alive = wait_all(&ctl.o_full[m], o_parity);
            o_parity ^= 1;
            const int64_t piece = (int64_t)blockIdx.x + way.item;
            if (alive) {
                tc_fence_after();
                float4* dst = reinterpret_cast<float4*>(a.part + piece * p.tile_rows * D) + in_tile;
#pragma unroll 1
                for (int i = 0; i < D; i += 32) {
                    float o[32];
                    tmem_ld32(o_addr + i, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        dst[(i + j) / 4 * p.tile_rows] = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
                tc_fence_before();
            }
            a.ml[piece * p.tile_rows + in_tile] = make_float2(ref, !alive ? kPieceTimeout : (*(volatile int*)&ctl.bad ? kPieceBadPage : sum));
        }
        if (!alive)  // the pieces of the items that were not reached
            for (Way rest(p); rest.left > 0; rest.next(p))
                a.ml[((int64_t)blockIdx.x + rest.item) * p.tile_rows + in_tile] = make_float2(neg, kPieceTimeout);
    } else if (warp == Shape::kMmaWarp) {
        // ---------------------------------------------------------------------------- products
        // The whole warp walks along and one lane issues: a hand-over costs a few instructions, and the
        // descriptors are constants added to three bases.
        constexpr uint32_t kScoreDesc = mma_desc(128, 128, !k8, false), kOutDesc = mma_desc(128, D, !k8, true);
        const uint64_t q_desc = smem_desc(smem_u32(q_tile), 16), k_desc = smem_desc(smem_u32(ring), 16);
        const uint64_t v_desc = smem_desc(smem_u32(ring), 128 * 128);
        const bool leader = elect_one();
        uint32_t q_parity = 0, p_parity = 0, tail_parity = 0;  // of the tail: a bit for each slot
        Turn<kRing> turn(0);
        auto take = [&]() {  // wait for the ring's next tile; its slot
            alive = wait_all(&ctl.full[turn.slot], turn.parity);
            const int slot = turn.slot;
            turn.next();
            return slot;
        };
        auto scores = [&](int m, int slot) {
            if (leader) {
                const uint64_t qd = q_desc + (uint64_t)(m * (Shape::kTileBytes >> 4)), kd = k_desc + (uint64_t)(slot * (Shape::kTileBytes >> 4));
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint64_t off = (uint64_t)(((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4);
                    mma_ss(tmem + Shape::kScoreCol + 128 * m, qd + off, kd + off, kScoreDesc, s > 0);
                }
                tc_commit(&ctl.s_full[m]);
            }
        };
        Way way(p);
        for (; way.left > 0 && alive; way.next(p)) {
            const int blocks = way.blocks(p);
            if (!(alive = wait_all(&ctl.q_full, q_parity))) break;
            q_parity ^= 1;
            int kslot = take();
            if (!alive) break;
            tc_fence_after();
#pragma unroll
            for (int m = 0; m < kTiles; ++m) scores(m, kslot);
            if (leader) tc_commit(&ctl.empty[kslot]);
            for (int v = 0; v < blocks && alive; ++v) {
                const int vslot = take();
                if (!alive) break;
                if (!k8 && prefix < (way.block + v + 1) * kBlockKeys) {  // its rows past the prefix are zeroed
                    if (!(alive = wait_all(&ctl.tail[vslot], tail_parity >> vslot & 1))) break;
                    tail_parity ^= 1u << vslot;
                }
#pragma unroll
                for (int m = 0; m < kTiles; ++m) {
                    if (!(alive = wait_all(&ctl.p_full[m], p_parity))) break;
                    tc_fence_after();
                    if (leader) {
                        const uint64_t vd = v_desc + (uint64_t)(vslot * (Shape::kTileBytes >> 4));
#pragma unroll
                        for (int s = 0; s < kBlockKeys / 16; ++s)
                            mma_ts(tmem + Shape::kOutCol + D * m, tmem + Shape::kScoreCol + 128 * m + s * 8, vd + (uint64_t)(s * (2048 >> 4)),
                                   kOutDesc, s > 0 || v > 0);
                        if (v + 1 == blocks) tc_commit(&ctl.o_full[m]);
                    }
                    if (v + 1 < blocks) {
                        if (m == 0) {
                            kslot = take();
                            if (!alive) break;
                            tc_fence_after();
                        }
                        scores(m, kslot);
                    }
                }
                if (!alive) break;
                p_parity ^= 1;
                if (leader) {
                    tc_commit(&ctl.empty[vslot]);
                    if (v + 1 < blocks) tc_commit(&ctl.empty[kslot]);
                }
            }
        }
        // Products in flight end before the tensor memory is given back (bounded, as every wait).
        if (leader) tc_commit(&ctl.drain);
        mbar_wait_bounded(&ctl.drain, 0, kAttnWaitNs);
        __syncwarp();
    } else if (warp == Shape::kLoadWarp) {
        // ---------------------------------------------------------------------------- loads
        // A lane for each box: the tokens of one page within a block, up to 128 of them.
        constexpr int kSlots = k8 ? kRaw : kRing;
        uint64_t* filled = k8 ? ctl.raw_full : ctl.full;
        uint64_t* freed = k8 ? ctl.raw_empty : ctl.empty;
        const int box = min(a.c.page_size, kBlockKeys), boxes = kBlockKeys / box;
        auto page_of = [&](int token) { return lane < boxes && token < prefix ? a.a.prefix_pages[token >> a.page_shift] : 0; };
        Way way(p);
        int page = page_of(way.block * kBlockKeys + lane * box);
        Turn<kSlots> turn(1);  // a slot's first fill waits for nothing: the phase before its first
        int fills = 0;
        while (way.left > 0 && alive && way.head != a.stall_head) {
            const int head = way.head, token = way.block * kBlockKeys, left = prefix - token;
            const int live = min(boxes, (left + box - 1) / box);
            const int row = (token + lane * box) & (a.c.page_size - 1);
            int id = page;
            if (id < 0 || id >= a.c.n_pages) {
                *(volatile int*)&ctl.bad = 1;
                id = 0;
            }
            way.step(p);
            if (way.left > 0) page = page_of(way.block * kBlockKeys + lane * box);  // the next block's, not looked at before it is needed
            for (int kv = 0; kv < 2; ++kv) {
                if (!(alive = wait_all(&freed[turn.slot], turn.parity))) break;
                unsigned char* dst = k8 ? raw_ring + turn.slot * Shape::kRawBytes : ring + turn.slot * Shape::kTileBytes;
                uint64_t* bar = &filled[turn.slot];
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(live * box) * (k8 ? D + 2 : 2 * D));
                __syncwarp();
                if (lane < live) {
                    if (k8) {
                        const int64_t at = (((int64_t)id * a.c.n_heads + head) << a.page_shift) + row;
                        bulk_g2s(dst + lane * box * D, static_cast<const char*>(kv ? a.c.v : a.c.k) + at * D, (uint32_t)(box * D), bar);
                        bulk_g2s(dst + 128 * D + lane * box * 2, static_cast<const char*>(kv ? a.c.v_scale : a.c.k_scale) + at * 2,
                                 (uint32_t)(box * 2), bar);
                    } else {
                        for (int cb = 0; cb < D / 64; ++cb)
                            tma_load4(dst + cb * (128 * 128) + lane * box * 128, kv ? &vmap : &kmap, cb * 64, row, head, id, bar);
                    }
                }
                const uint32_t parity = turn.parity ^ 1;  // of this fill
                const int slot = turn.slot;
                turn.next();
                ++fills;
                if (!k8 && kv && left < kBlockKeys) {
                    // Rows past the prefix hold anything (0 * NaN is NaN): zero them once the copy has landed.  Each slot has
                    // a signal of its own: its next one comes after the slot was given back, so after this one's wait.  One
                    // signal for all could complete two phases before the first was waited for, where items are one block long.
                    if (!(alive = wait_all(bar, parity))) break;
                    for (int i = lane; i < (kBlockKeys - left) * (D / 8); i += 32)
                        *reinterpret_cast<uint4*>(dst + tile_byte(left + i / (D / 8), i % (D / 8))) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.tail[slot]);
                }
            }
        }
        // Copies in flight land before the CTA leaves: the last fill of every slot.
        for (int i = 1; i <= min(fills, kSlots); ++i)
            mbar_wait_bounded(&filled[(fills - i) % kSlots], (uint32_t)((fills - i) / kSlots) & 1, kAttnWaitNs);
    } else if (k8 && warp == Shape::kScaleWarp) {
        // ---------------------------------------------------------------------------- scales
        // A tile's unit is a power of two next to its largest scale, the one below for fp8 and the one above for int8,
        // whose weights (up to 2^15) are multiplied by the scales; 1 if there is none.  fp8: a token's scale in that
        // unit is the factor of its codes.  int8: the scores and the weights take the scales.  A unit is at least 2^-80
        // (kLeastScale), so that the sum, which is divided by the values', stays finite.  One warp for every tile in
        // turn: a barrier's phase may only be waited for by a role that sees each of its phases.
        Way way(p);
        Turn<kRaw> raw_turn(0);
        Turn<kScalars> scalar(0);
        for (; way.left > 0 && alive; way.step(p), scalar.next()) {
            const int left = prefix - way.block * kBlockKeys;
            int wide = 0;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, raw_turn.next()) {
                const int rs = raw_turn.slot;
                if (!(alive = wait_all(&ctl.raw_full[rs], raw_turn.parity))) break;
                uint2 w = *reinterpret_cast<const uint2*>(raw_ring + rs * Shape::kRawBytes + 128 * D + lane * 8);
                if (left < kBlockKeys) {  // past the prefix: anything
                    const int in = left - lane * 4;
                    w.x = in >= 2 ? w.x : (in == 1 ? w.x & 0xFFFFu : 0u);
                    w.y = in >= 4 ? w.y : (in == 3 ? w.y & 0xFFFFu : 0u);
                }
                const float s[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                                    __uint_as_float(w.y & 0xFFFF0000u)};
                if (kFormat == TPS_KV_INT8 && !kv) {
                    *reinterpret_cast<float4*>(&ctl.key_scale[scalar.slot][lane * 4]) = make_float4(s[0], s[1], s[2], s[3]);
                    if (lane == 0) ctl.key_unit[scalar.slot] = 1.f;
                } else {
                    // The largest scale and the smallest that is not 0, by their bits (0 counts as 2^16).
                    const uint32_t high = __vmaxu2(w.x, w.y), low = __vminu2(__vsub2(w.x, 0x10001u), __vsub2(w.y, 0x10001u));
                    const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, max(high >> 16, high & 0xFFFFu));
                    const bool odd = kFormat == TPS_KV_FP8 && ((w.x | w.y) & 0x7F007Fu) != 0;  // not a power of two
                    const uint32_t least = __reduce_min_sync(0xFFFFFFFFu, odd ? 0u : min(low >> 16, low & 0xFFFFu)) + 1;
                    const int e = most ? max(-80, min((int)((most + (kFormat == TPS_KV_INT8 ? 0x7Fu : 0u)) >> 7) - 127, 126)) : 0;
                    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
                    const bool far = least < (uint32_t)(e + 127 - kSpread) << 7;
                    float f[4];  // in the block's unit
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = s[i] * inv;
                    if (far) {
                        wide |= 1 << kv;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (kv) {
                                const float y = floor_scale(s[i]);
                                ctl.value_log[scalar.slot][lane * 4 + i] = log2_fast(y);
                                ctl.value_scale[scalar.slot][lane * 4 + i] = y == y ? 1.f / y : 1.f;  // NaN comes by its logarithm
                            } else {
                                ctl.key_scale[scalar.slot][lane * 4 + i] = s[i];
                            }
                            f[i] = 1.f;
                        }
                    } else if (kFormat == TPS_KV_INT8) {
                        *reinterpret_cast<float4*>(&ctl.value_scale[scalar.slot][lane * 4]) = make_float4(f[0], f[1], f[2], f[3]);
                    }
                    if constexpr (kFormat == TPS_KV_FP8) {
                        const __half2 lo = __floats2half2_rn(f[0], f[1]), hi = __floats2half2_rn(f[2], f[3]);
                        *reinterpret_cast<uint2*>(&ctl.factor[rs][lane * 4]) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                    }
                    if (lane == 0) {
                        if (kv)
                            ctl.value_exp[scalar.slot] = far ? 0.f : (float)e, ctl.wide[scalar.slot] = wide;
                        else
                            ctl.key_unit[scalar.slot] = far ? 1.f : __uint_as_float((uint32_t)(127 + e) << 23);
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&ctl.factor_full[rs]);
                    if (kv) mbar_arrive(&ctl.scalar_full[scalar.slot]);
                }
            }
        }
    } else if (k8 && warp >= Shape::kConvertWarp) {
        // ---------------------------------------------------------------------------- 8-bit codes to float16
        constexpr int kPieces = D / 16;                           // 16-byte pieces of a code row
        constexpr int kThreadsConv = Shape::kConvertWarps * 32;
        constexpr int kSteps = 128 * kPieces / kThreadsConv, kRowsPerStep = kThreadsConv / kPieces;
        const int t = (int)threadIdx.x - Shape::kConvertWarp * 32;
        // Eight lanes at a time read 16 bytes each and write two 16-byte chunks each.  At D = 128 they are the first half
        // of one code row and the second half of the next: then both the reads and, by the swizzle, the writes of
        // the eight hit different banks.
        const int piece = kPieces == 8 ? (t & 3) + 4 * ((t >> 2 ^ t >> 3) & 1) : t % kPieces;
        const int sub = kPieces == 8 ? (t >> 5) * 4 + (t >> 4 & 1) * 2 + (t >> 2 & 1) : t / kPieces;
        Way way(p);
        Turn<kRaw> raw_turn(0);
        Turn<kRing> turn(1);
        for (; way.left > 0 && alive; way.step(p)) {
            const int left = prefix - way.block * kBlockKeys;
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv, raw_turn.next(), turn.next()) {
                const int rs = raw_turn.slot;
                const unsigned char* raw = raw_ring + rs * Shape::kRawBytes;
                if (!(alive = wait_all(&ctl.factor_full[rs], raw_turn.parity))) break;
                if (!(alive = wait_all(&ctl.raw_full[rs], raw_turn.parity))) break;
                uint4 x[kSteps];
                __half2 f[kSteps];
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const int r = i * kRowsPerStep + sub;
                    x[i] = *reinterpret_cast<const uint4*>(raw + r * D + piece * 16);
                    if constexpr (kFormat == TPS_KV_FP8) f[i] = __half2half2(ctl.factor[rs][r]);
                }
                if (left < kBlockKeys) {  // past the prefix: anything
#pragma unroll
                    for (int i = 0; i < kSteps; ++i)
                        if (i * kRowsPerStep + sub >= left) x[i] = make_uint4(0u, 0u, 0u, 0u);
                }
                if (!(alive = wait_all(&ctl.empty[turn.slot], turn.parity))) break;
                unsigned char* dst = ring + turn.slot * Shape::kTileBytes;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const int r = i * kRowsPerStep + sub;
                    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    uint32_t h[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        code_pairs<kFormat>(w[j], h[2 * j], h[2 * j + 1]);
                        if constexpr (kFormat == TPS_KV_FP8) {
#pragma unroll
                            for (int k = 2 * j; k < 2 * j + 2; ++k) {
                                const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&h[k]), f[i]);
                                h[k] = *reinterpret_cast<const uint32_t*>(&y);
                            }
                        }
                    }
                    *reinterpret_cast<uint4*>(dst + tile_byte(r, 2 * piece)) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4*>(dst + tile_byte(r, 2 * piece + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&ctl.full[turn.slot]);
                    mbar_arrive(&ctl.raw_empty[rs]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == Shape::kMmaWarp) tmem_free(tmem, Shape::kTmemCols);
}

}  // namespace tps
