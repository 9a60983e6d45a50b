// tps_attn_prompt.cuh -- causal attention of whole prompts, packed one behind another (tps_prompt_attention),
// on the tcgen05 matrix unit.
//
// Mathematics.  For a query token t of a sequence and the tokens j <= t before it: weights 2^(z_j - m) with
// z_j = scale log2(e) q.k_j and a reference m per row, a whole number that is raised only when a score exceeds
// it by more than kSlack, so that raising it scales what was already computed by an exact power of two; their sum and
// the output in float32, one pass over the keys, one division at the end.  The weights are bfloat16 for the
// second product, whose values are bfloat16 (at most 2^-8 of sum p |v|).
//
// Rows.  The query heads of one key head share its keys and values, so they are rows of the same tile: row r of a
// tile of 128 is token r / heads, head r % heads, and as many tokens as fit.  In this order one box of a tensor
// map (64 columns, the heads, the tokens) fills a tile, whatever the strides.  More than 128 heads to a key head are
// cut into equal groups.  A CTA has two such tiles, of consecutive tokens: one's softmax runs while the other's products
// do, and each block of 128 keys and values is loaded once for both.
//
// The sum.  In a sequence's first block of keys, for the tiles that do not see it whole, it takes the weights as the second product
// has them, rounded: the output is then an average of values whatever their roundings, and what sees one token has its value
// as it is.  That is where rows see few tokens, and where it counts: 2 tokens are off by 0.0018 of their size instead of 0.0023, 1 by
// nothing instead of 0.0013 (root mean square; the output's own rounding makes 0.0017).  In all blocks it would take
// 1,541 us instead of 1,420 (one prompt of 16,384) for 0.0022 instead of 0.0024.  The logarithm of the sum takes no rounding.
//
// Masks.  Only a tile's last blocks hold tokens that some row must not see; there a score past its row's limit is
// -inf.  A hidden token's value may still be NaN or infinite (also the next sequence's, or what lies behind the
// last), and 0 times that is NaN: warps of their own look through the hidden rows of those value tiles, and take what is
// not finite out of the product; a row that does see the token adds it at the end.
//
// What bounds it: for long prompts the matrix unit (a 128 x 128 tile at D = 128 takes it 634 clocks for the scores, whose operands both
// come from shared memory, and 559 for the outputs; at D = 64 378 and 367) and, under the power limit, its clock; at D = 64 the
// hand-overs between the roles (a commit is seen some 450 clocks after the product, a signal 100 after it is given), as one
// tile's softmax and its next scores wait for each other; for short prompts the 7,000 clocks or so from one item's last
// weights to the next one's.  Measured: 16,384 tokens, 32 heads on 8 of 128, 1,430 us (1.54 PFLOP/s); 4 prompts of 2,500 to 4,001, 16
// heads, 155 us (1.15); 24 of 700 to 2,011, 40 heads on 8 of 64, 384 us (0.64); 64 of 1 to 250, 32 on 8 of 128, 50 us (3.3 TB/s); one of 300
// 10.7 us.  Tried and not kept: two threads for each row (16 softmax warps; 1,531, 173, 430, 66 us where this took 1,416,
// 173, 390, 74), the outputs by way of shared memory (52 us for 49, 64 short prompts; by bulk stores 50), two pairs of query
// tiles (375 for 374 us at D = 64), a tile's next scores while the softmax still works on the present ones (D = 64: 401 us for
// 374).  One persistent CTA per SM.  Tiles of unequal length are dealt out by length,
// longest first, to and fro over the CTAs (a small kernel ahead sorts them); where all tiles fit the SMs at once each CTA finds its
// own and there is one launch.  Roles:
//   warps 0 .. 7    softmax, one thread per row: scores from TMEM, weights back over them
//   warp 8          issues every product; the next tile's first scores follow the last product of the present one
//   warp 9          loads: queries, keys, values by tensor maps
//   warps 10, 11    hidden values that are not finite
// Every wait is bounded: one that runs out makes all roles leave, and the outputs that were not reached NaN.
#pragma once

#include "tps_attn_prefix.cuh"

namespace tps {

constexpr int kPromptThreads = 384, kPromptMma = 8, kPromptLoad = 9, kPromptHidden = 10;
// Items of each tile whose marks are kept.  An item's weights come after the output of the tile's item before, the second product waits
// for them, and the loads run at most a ring of tiles ahead of it: six items, counted for each tile by itself (prompts that fit one
// tile give tile 1 nothing to do, and any number of them may go by while its softmax warps still have an output to write).
constexpr int kDirty = 8;
constexpr uint64_t kLong = 64;   // waits for what may come after the whole of a long sequence, in limits of the others

template <int D> struct PromptShape {
    static constexpr int kTileBytes = 128 * D * 2;
    static constexpr int kRing = D == 128 ? 5 : 8;  // key and value tiles in shared memory
    static constexpr int kOutCol = 256;             // TMEM: scores (and weights) of tile m at 128 m, outputs at 256 + D m
    struct Control {
        uint64_t full[kRing], empty[kRing], go[kRing], clean[kRing];
        uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], drain;
        uint32_t tmem;
        int abort;
        int dirty[2][kDirty][2];  // by tile, item of that tile and warp: values were taken out of the product
    };
    static constexpr size_t kSmem = (size_t)(2 + kRing) * kTileBytes + sizeof(Control) + 1024;
    static_assert(kSmem <= 232448, "fits one CTA's shared memory");
};

// A CTA's unit of work: up to 2 a.tile_tokens query tokens of one sequence for one group of query heads.
struct PromptItem {
    int begin, end, token, seq;  // the sequence's tokens, the first query token (absolute); -1: no such item
    int kv, head, heads;         // key head; first query head and how many
    int blocks0, blocks1, last;  // key blocks of each tile, of both
    int open;                    // blocks that all rows see whole
    __device__ __forceinline__ int blocks(int m) const { return m ? blocks1 : blocks0; }
    // Keys that tile m's row r sees.
    __device__ __forceinline__ int limit(const PromptArgs& a, int m, int r) const
    {
        return min(token + m * a.tile_tokens + r / a.group, end - 1) - begin + 1;
    }
};
__device__ __forceinline__ PromptItem prompt_item(const PromptArgs& a, const int4& e, int vh)
{
    PromptItem it;
    it.begin = e.x, it.end = e.y, it.token = e.z, it.seq = e.w;
    it.kv = vh / a.groups;
    const int first = (vh - it.kv * a.groups) * a.group;
    it.head = it.kv * a.G + first;
    it.heads = min(a.group, a.G - first);
    auto blocks = [&](int from) {
        const int to = min(from + a.tile_tokens, it.end);
        return to > from ? (to - it.begin + kBlockKeys - 1) / kBlockKeys : 0;
    };
    it.blocks0 = blocks(it.token), it.blocks1 = blocks(it.token + a.tile_tokens);
    it.last = max(it.blocks0, it.blocks1);
    it.open = (it.token - it.begin + 1) / kBlockKeys;
    return it;
}

// Sequences whose bounds are in order: not below an earlier bound, so that no two share a token.
__device__ __forceinline__ bool prompt_valid(const PromptArgs& a, int lo, int hi, int most_before)
{
    return lo >= 0 && hi >= lo && hi <= a.T && lo >= most_before;
}
__device__ __forceinline__ int prompt_tiles(const PromptArgs& a, int lo, int hi)
{
    return (hi - lo + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
}

// Tile `want` of all sequences in their order, by a whole warp: a call of few tiles needs no sorted list.
__device__ __forceinline__ int4 find_tile(const PromptArgs& a, int want)
{
    const int lane = threadIdx.x & 31;
    int before = 0, most = INT32_MIN;
    for (int64_t base = 0; base < a.B; base += 32) {
        const int64_t b = base + lane;
        const int lo = b < a.B ? a.cu_seqlens[b] : INT32_MIN, hi = b < a.B ? a.cu_seqlens[b + 1] : INT32_MIN;
        int top = lo;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xFFFFFFFFu, top, o);
            if (lane >= o) top = max(top, x);
        }
        top = max(top, most);
        const int n = prompt_valid(a, lo, hi, top) ? prompt_tiles(a, lo, hi) : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += x;
        }
        sum += before;
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, sum > want);
        if (past) {
            const int w = __ffs(past) - 1;
            const int tile = want - __shfl_sync(0xFFFFFFFFu, sum - n, w);
            const int l = __shfl_sync(0xFFFFFFFFu, lo, w), h = __shfl_sync(0xFFFFFFFFu, hi, w);
            return make_int4(l, h, l + tile * 2 * a.tile_tokens, (int)base + w);
        }
        before = __shfl_sync(0xFFFFFFFFu, sum, 31);
        most = __shfl_sync(0xFFFFFFFFu, top, 31);
    }
    return make_int4(0, 0, -1, 0);
}

// A CTA's items, in the same order for every role.
struct PromptWalk {
    const PromptArgs& a;
    int round = 0, count;  // of all CTAs' items
    int4 next;             // entry of the item after this one, read ahead
    int next_vh;
    PromptItem it;
    __device__ __forceinline__ int rank(int r) const
    {
        const int n = (int)gridDim.x, c = (int)blockIdx.x;
        return r * n + ((r & 1) ? n - 1 - c : c);
    }
    __device__ __forceinline__ void look(int r)
    {
        const int64_t at = r <= (count - 1) / (int)gridDim.x ? rank(r) : count;
        const int tile = (int)at / a.heads_v;
        next_vh = (int)at - tile * a.heads_v;
        next = at < count ? __ldcg(a.list + tile) : make_int4(0, 0, -1, 0);
    }
    __device__ __forceinline__ explicit PromptWalk(const PromptArgs& a_) : a(a_)
    {
        if (a.list) {
            count = __ldcg(a.n_tiles) * a.heads_v;
            look(0);
        } else {
            next = find_tile(a, (int)blockIdx.x / a.heads_v);
            next_vh = (int)blockIdx.x % a.heads_v;
        }
        step();
    }
    // To the next item; `next` then holds the one after it.
    __device__ __forceinline__ void step()
    {
        it = prompt_item(a, next, next_vh);
        ++round;
        if (a.list && it.token >= 0)
            look(round);
        else
            next = make_int4(0, 0, -1, 0);
    }
    __device__ __forceinline__ bool more() const { return it.token >= 0; }
};

// 32 bytes, as a whole sector where the output begins on one.
__device__ __forceinline__ void store32(const PromptArgs& a, void* p, const uint32_t* w)
{
    if (!a.sectors) {
        static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                 "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    attn_prompt_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap)
{
    using Shape = PromptShape<D>;
    using Control = typename Shape::Control;
    constexpr int kRing = Shape::kRing;
    extern __shared__ unsigned char raw_smem[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    unsigned char* q_tile = smem;
    unsigned char* ring = smem + 2 * Shape::kTileBytes;
    Control& ctl = *reinterpret_cast<Control*>(ring + kRing * Shape::kTileBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&ctl.full[i], 1), mbar_init(&ctl.empty[i], 1), mbar_init(&ctl.go[i], 1), mbar_init(&ctl.clean[i], 2);
        for (int i = 0; i < 2; ++i)
            mbar_init(&ctl.q_full[i], 1), mbar_init(&ctl.q_empty[i], 1), mbar_init(&ctl.s_full[i], 1), mbar_init(&ctl.p_full[i], 4),
                mbar_init(&ctl.o_full[i], 1);
        mbar_init(&ctl.drain, 1);
        ctl.abort = 0;
    }
    // Rows of a query tile that no box fills stay zero.
    const int used = a.tile_tokens * a.group;
    for (int i = (int)threadIdx.x; i < 2 * (128 - used) * (D / 8); i += kPromptThreads) {
        const int row = used + i / (D / 8) % (128 - used);
        *reinterpret_cast<uint4*>(q_tile + (i >= (128 - used) * (D / 8) ? Shape::kTileBytes : 0) + tile_byte(row, i % (D / 8))) =
            make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async();
    if (warp == kPromptMma) tmem_alloc(&ctl.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    if (a.list) asm volatile("griddepcontrol.wait;" ::: "memory");  // the list of tiles

    volatile int* abort_flag = &ctl.abort;
    // Wait for a phase; false once any role has given up (this one after a.wait_ns).
    auto wait = [&](uint64_t* bar, uint32_t parity, uint64_t limit) {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        for (;;) {
            if (mbar_try_wait(bar, parity, 20000u)) return true;  // suspended, not spinning
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > limit) {
                *abort_flag = 1;
                return false;
            }
        }
    };
    auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity, a.wait_ns)) != 0; };
    bool alive = true;
    PromptWalk walk(a);
    const PromptItem& it = walk.it;

    if (warp < kPromptMma) {
        // ---------------------------------------------------------------------------- softmax
        const int m = warp >> 2, row = (int)threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lanes + 128 * m, o_addr = tmem + lanes + Shape::kOutCol + D * m;
        const float neg = -__int_as_float(0x7F800000);
        const float c = fmaxf(fabsf(a.qk_scale), 0x1p-126f);  // never 0: a masked score, -inf, times it stays -inf
        uint32_t s_parity = 0, o_parity = 0;
        int item = -1;  // of the tile
        for (; walk.more(); walk.step()) {
            const int blocks = it.blocks(m);
            if (blocks == 0) continue;
            ++item;
            const int limit = it.limit(a, m, row);
            const int most = it.limit(a, m, 127);  // of any row of the tile
            // `lost`: what rounding took from the weights that `sum` has as the product has them.
            float ref = neg, sum = 0.f, lost = 0.f;
            for (int v = 0; v < blocks && alive; ++v) {
                // An item's first scores may come long after this tile's last ones: while the other tile has a long sequence's end.
                if (!(alive = __all_sync(0xFFFFFFFFu, wait(&ctl.s_full[m], s_parity, v == 0 ? a.wait_ns * kLong : a.wait_ns)))) break;
                s_parity ^= 1;
                tc_fence_after();
                const bool masked = v >= it.open;
                const int left = limit - v * kBlockKeys, wide = most - v * kBlockKeys;
                float2 total = make_float2(0.f, 0.f);
                auto hide = [&](float (&s)[32], int ch) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (ch * 32 + i >= left) s[i] = neg;
                };
                auto largest = [&](const float (&s)[32]) {
                    float t = s[0];
#pragma unroll
                    for (int i = 1; i < 32; ++i) t = fmaxf(t, s[i]);
                    return t;
                };
                // Raise the reference of a row that needs it (the warp's others go along with factor 1, so that no row's
                // bits depend on its neighbours'): scale the sum, the output and the weights of chunks 0 .. done - 1.
                auto raise = [&](bool need, float top, int done) {
                    const float to = need && top > ref ? ceilf(top) : ref;
                    const float f = to == ref ? 1.f : exp2_fast(ref - to);
                    ref = to;
                    sum *= f, lost *= f;
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
                            const __nv_bfloat162 h = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&w[j]), __float2bfloat162_rn(f));
                            w[j] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                        tmem_st16(s_addr + i * 16, w);
                    }
                };
                // Weights of 32 scores, to columns [16 ch, 16 ch + 16), whose scores have been read; their sum.
                auto weigh = [&](const float (&s)[32], int ch, float b) {
                    float2 part[2];
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float2 x = fma2(make_float2(s[i], s[i + 1]), make_float2(c, c), make_float2(b, b));
                        x.x = exp2_fast(x.x), x.y = exp2_fast(x.y);
                        part[(i >> 1) & 1] = i < 4 ? x : add2(part[(i >> 1) & 1], x);
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i / 2]) : "f"(x.y), "f"(x.x));
                    }
                    tmem_st16(s_addr + ch * 16, w);
                    return add2(part[0], part[1]);
                };
                // 64 scores at a time, first weighed against the reference as it stands (an item's first 64 have none): a weight
                // above 2^kSlack shows in their sum, so the usual step looks for no maximum at all.
#pragma unroll
                for (int ch = 0; ch < 4; ch += 2) {
                    if (ch * 32 >= wide) break;  // no row of the tile sees these: the product leaves them out, too
                    float sa[32], sb[32];
                    tmem_ld32(s_addr + ch * 32, sa);
                    tmem_ld32(s_addr + ch * 32 + 32, sb);
                    tmem_wait_ld(sa);
                    tmem_wait_ld(sb);
                    if (masked) {
                        hide(sa, ch);
                        hide(sb, ch + 1);
                    }
                    float2 x;
                    for (bool again = v == 0 && ch == 0, need = again;;) {
                        if (again) raise(need, fmaxf(largest(sa), largest(sb)) * c, ch);
                        const float b = ref == neg ? 0.f : -ref;
                        x = add2(weigh(sa, ch, b), weigh(sb, ch + 1, b));
                        if (again) break;
                        need = !(x.x + x.y <= 256.f) || ref == neg;
                        if (!__any_sync(0xFFFFFFFFu, need)) break;
                        again = true;
                        tmem_wait_st();
                    }
                    total = add2(total, x);
                }
                float mass = total.x + total.y;
                tmem_wait_st();
                if (masked && v == 0) {
                    const float rounded = weight_sum(s_addr, wide > 64 ? 4 : 2);
                    lost += mass - rounded;
                    mass = rounded;
                }
                sum += mass;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_full[m]);
            }
            if (alive) alive = wait_all(&ctl.o_full[m], o_parity);
            o_parity ^= 1;
            tc_fence_after();
            const int in_tile = row / a.group, h = row - in_tile * a.group, token = it.token + m * a.tile_tokens + in_tile;
            const bool mine = in_tile < a.tile_tokens && h < it.heads && token < it.end;
            const bool dirty = alive && (*(volatile int*)&ctl.dirty[m][item % kDirty][0] | *(volatile int*)&ctl.dirty[m][item % kDirty][1]);
            const int64_t at = (int64_t)token * a.Hq + it.head + h;
            const float inv = alive ? 1.f / sum : __int_as_float(0x7FC00000);
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at * D);
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
                float o[32];
                tmem_ld32(o_addr + i, o);
                tmem_wait_ld(o);
                if (mine) {
                    if (dirty) {  // what was taken out of the product, for a row that sees it
                        for (int j = it.token - it.begin + 1; j < limit; ++j) {
                            const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.v) +
                                                                                    (int64_t)(it.begin + j) * a.v_ld + (int64_t)it.kv * a.v_hd + i);
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const uint32_t x = not_finite(src[k]);
                                o[2 * k] += __uint_as_float(x << 16);
                                o[2 * k + 1] += __uint_as_float(x & 0xFFFF0000u);
                            }
                        }
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const __nv_bfloat162 y = __floats2bfloat162_rn(o[2 * j] * inv, o[2 * j + 1] * inv);
                        w[j] = *reinterpret_cast<const uint32_t*>(&y);
                    }
#pragma unroll
                    for (int j = 0; j < 4; j += 2) store32(a, dst + i / 8 + j, w + 4 * j);
                }
            }
            tc_fence_before();
            if (mine) {
                if (a.out_lse) a.out_lse[at] = alive ? (ref + log2f(sum + lost)) * 0.693147180559945f : __int_as_float(0x7FC00000);
                if (!alive && a.out_status) a.out_status[it.seq] = TPS_ROW_TIMEOUT;
            }
        }
    } else if (warp == kPromptMma) {
        // ---------------------------------------------------------------------------- products
        constexpr uint32_t kOutDesc = mma_desc(128, D, true, true);
        const uint32_t score_desc = mma_desc(128, 128, true, false) | (a.qk_scale < 0.f ? 1u << 13 : 0u);  // minus A
        const uint64_t q_desc = smem_desc(smem_u32(q_tile), 16), k_desc = smem_desc(smem_u32(ring), 16);
        const uint64_t v_desc = smem_desc(smem_u32(ring), 128 * 128);
        const bool leader = elect_one();
        uint32_t q_parity = 0, p_parity = 0, clean_parity = 0;  // bits: of a tile; of a slot
        Turn<kRing> turn(0);
        auto take = [&]() {  // wait for the ring's next tile; its slot
            alive = wait_all(&ctl.full[turn.slot], turn.parity);
            const int slot = turn.slot;
            turn.next();
            return slot;
        };
        auto scores = [&](int m, int slot, bool last) {
            if (leader) {
                const uint64_t qd = q_desc + (uint64_t)(m * (Shape::kTileBytes >> 4)), kd = k_desc + (uint64_t)(slot * (Shape::kTileBytes >> 4));
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint64_t off = (uint64_t)(((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4);
                    mma_ss(tmem + 128 * m, qd + off, kd + off, score_desc, s > 0);
                }
                tc_commit(&ctl.s_full[m]);
                if (last) tc_commit(&ctl.q_empty[m]);
            }
        };
        // The first scores of an item: its queries, then its first keys (taken once for both tiles).
        auto query = [&](int m) {
            alive = wait_all(&ctl.q_full[m], q_parity >> m & 1);
            q_parity ^= 1u << m;
            return alive;
        };
        int kslot = 0;
        if (walk.more()) {
            kslot = take();
            for (int m = 0; m < 2 && alive; ++m)
                if (it.blocks(m) && query(m)) {
                    tc_fence_after();
                    scores(m, kslot, it.blocks(m) == 1);
                }
            if (leader) tc_commit(&ctl.empty[kslot]);
        }
        while (walk.more() && alive) {
            const PromptItem now = walk.it;
            const int most0 = now.limit(a, 0, 127), most1 = now.limit(a, 1, 127);
            walk.step();
            const bool more = walk.more();
            for (int v = 0; v < now.last && alive; ++v) {
                const int vslot = take();
                if (!alive) break;
                if (v >= now.open) {  // its hidden rows are finite
                    if (!(alive = wait_all(&ctl.clean[vslot], clean_parity >> vslot & 1))) break;
                    clean_parity ^= 1u << vslot;
                }
                const bool end = v + 1 == now.last;
                bool taken = false;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    if (v < now.blocks(m)) {
                        if (!(alive = wait_all(&ctl.p_full[m], p_parity >> m & 1))) break;
                        p_parity ^= 1u << m;
                        tc_fence_after();
                        if (leader) {
                            const uint64_t vd = v_desc + (uint64_t)(vslot * (Shape::kTileBytes >> 4));
                            const int keys = (m ? most1 : most0) - v * kBlockKeys;  // past them every weight is 0
#pragma unroll
                            for (int s = 0; s < kBlockKeys / 16; ++s)
                                if (s * 16 < keys)
                                    mma_ts(tmem + Shape::kOutCol + D * m, tmem + 128 * m + s * 8, vd + (uint64_t)(s * (2048 >> 4)), kOutDesc,
                                           s > 0 || v > 0);
                            if (v + 1 == now.blocks(m)) tc_commit(&ctl.o_full[m]);
                        }
                    }
                    const bool same = v + 1 < now.blocks(m), other = end && more && it.blocks(m) > 0;
                    if (same || other) {
                        if (!taken) {
                            kslot = take();
                            taken = true;
                        }
                        if (!alive || (other && !query(m))) break;
                        tc_fence_after();
                        scores(m, kslot, same ? v + 2 == now.blocks(m) : it.blocks(m) == 1);
                    }
                }
                if (!alive) break;
                if (leader) {
                    tc_commit(&ctl.empty[vslot]);
                    if (taken) tc_commit(&ctl.empty[kslot]);
                }
            }
        }
        // Products in flight end before the tensor memory is given back (bounded, as every wait).
        if (leader) tc_commit(&ctl.drain);
        mbar_wait_bounded(&ctl.drain, 0, kAttnWaitNs);
        __syncwarp();
    } else if (warp == kPromptLoad) {
        // ---------------------------------------------------------------------------- loads
        const bool leader = elect_one();
        Turn<kRing> turn(1);  // a slot's first fill waits for nothing: the phase before its first
        uint32_t q_parity = 3;
        int fills = 0;
        uint32_t q_filled = 0;  // a bit for each query tile
        for (; walk.more() && alive && it.kv != a.stall_head; walk.step()) {
            auto block = [&](int v, bool values) {
                if (!(alive = wait_all(&ctl.empty[turn.slot], turn.parity))) return;
                if (leader) {
                    unsigned char* dst = ring + turn.slot * Shape::kTileBytes;
                    uint64_t* bar = &ctl.full[turn.slot];
                    mbar_arrive_expect_tx(bar, Shape::kTileBytes);
#pragma unroll
                    for (int cb = 0; cb < D / 64; ++cb)
                        tma_load3(dst + cb * (128 * 128), values ? &vmap : &kmap, cb * 64, it.kv, it.begin + v * kBlockKeys, bar);
                    if (values && v >= it.open) mbar_arrive(&ctl.go[turn.slot]);
                }
                __syncwarp();
                turn.next();
                ++fills;
            };
            auto query = [&](int m) {
                if (!it.blocks(m)) return;
                if (!(alive = wait_all(&ctl.q_empty[m], q_parity >> m & 1))) return;
                q_parity ^= 1u << m;
                if (leader) {
                    mbar_arrive_expect_tx(&ctl.q_full[m], (uint32_t)used * (D * 2));
#pragma unroll
                    for (int cb = 0; cb < D / 64; ++cb)
                        tma_load3(q_tile + m * Shape::kTileBytes + cb * (128 * 128), &qmap, cb * 64, it.head, it.token + m * a.tile_tokens,
                                  &ctl.q_full[m]);
                }
                __syncwarp();
                q_filled |= 1u << m;
            };
            block(0, false);
            if (alive) block(0, true);
            if (alive) query(0);
            if (alive) query(1);
            for (int v = 1; v < it.last && alive; ++v) {
                block(v, false);
                if (alive) block(v, true);
            }
        }
        // Copies in flight land before the CTA leaves: the last fill of every slot and of both query tiles.
        for (int i = 1; i <= min(fills, kRing); ++i)
            mbar_wait_bounded(&ctl.full[(fills - i) % kRing], (uint32_t)((fills - i) / kRing) & 1, kAttnWaitNs);
        for (int m = 0; m < 2; ++m)
            if (q_filled >> m & 1) mbar_wait_bounded(&ctl.q_full[m], q_parity >> m & 1, kAttnWaitNs);
    } else {
        // ---------------------------------------------------------------------------- hidden values that are not finite
        // A slot's signal to look into it comes with its copy and is answered before the slot is given back, so neither
        // this wait nor the one for the copy can be a phase off.
        const int half = warp - kPromptHidden;
        uint32_t go_parity = 0;
        int item0 = 0, item1 = 0;  // of each tile
        int64_t fill = 0;          // of the item's first key tile
        for (; walk.more() && alive; walk.step()) {
            bool found = false;
            auto mark = [&](int to) {
                *(volatile int*)&ctl.dirty[0][item0 % kDirty][half] = to;
                if (it.blocks1) *(volatile int*)&ctl.dirty[1][item1 % kDirty][half] = to;
            };
            if (lane == 0) mark(0);
            for (int v = min(it.open, it.last); v < it.last && alive; ++v) {
                const int64_t f = fill + 2 * v + 1;
                const int slot = (int)(f % kRing);
                // The signal comes when the copy is asked for: in a long sequence long after the item has begun.
                if (!(alive = __all_sync(0xFFFFFFFFu, wait(&ctl.go[slot], go_parity >> slot & 1, a.wait_ns * kLong)))) break;
                go_parity ^= 1u << slot;
                if (!(alive = wait_all(&ctl.full[slot], (uint32_t)(f / kRing) & 1))) break;
                unsigned char* tile = ring + slot * Shape::kTileBytes;
                const int base = v * kBlockKeys, end = it.end - it.begin - base;          // rows from here on are not the sequence's
                const int first = max(it.token - it.begin + 1 - base, 0);                 // rows from here on are hidden from some row
                const int from = first * (D / 8) + half * 32 + lane;
                // 0 times what is not finite is NaN, and stays it: one instruction for two values finds whether there is any.
                __nv_bfloat162 sum[4] = {};
                const __nv_bfloat162 zero = {};
#pragma unroll 8
                for (int i = from; i < kBlockKeys * (D / 8); i += 64) {
                    const uint4 x = *reinterpret_cast<const uint4*>(tile + tile_byte(i / (D / 8), i % (D / 8)));
                    sum[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.x), zero, sum[0]);
                    sum[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.y), zero, sum[1]);
                    sum[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.z), zero, sum[2]);
                    sum[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.w), zero, sum[3]);
                }
                sum[0] = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
                if (*reinterpret_cast<const uint32_t*>(&sum[0]) & 0x7FFF7FFFu) {
#pragma unroll 1
                    for (int i = from; i < kBlockKeys * (D / 8); i += 64) {
                        const int r = i / (D / 8);
                        uint4* p = reinterpret_cast<uint4*>(tile + tile_byte(r, i % (D / 8)));
                        const uint4 x = *p, y = make_uint4(not_finite(x.x), not_finite(x.y), not_finite(x.z), not_finite(x.w));
                        if (y.x | y.y | y.z | y.w) {
                            found |= r < end;
                            *p = make_uint4(x.x ^ y.x, x.y ^ y.y, x.z ^ y.z, x.w ^ y.w);
                        }
                    }
                    fence_proxy_async();
                }
                const bool any = __any_sync(0xFFFFFFFFu, found);
                if (lane == 0) {
                    if (any) mark(1);
                    mbar_arrive(&ctl.clean[slot]);
                }
                __syncwarp();
            }
            fill += 2 * (int64_t)it.last;
            ++item0, item1 += it.blocks1 > 0;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kPromptMma) tmem_free(tmem, 512);
}

// The tiles of all sequences, longest first, into a.list, and the sequences' statuses.  One CTA, two passes over
// the bounds; tiles of like length (kPromptLevels steps) come in any order, which no result depends on.
constexpr int kPromptLevels = 2048;
template <int kThreads>
__global__ void __launch_bounds__(kThreads) prompt_plan_kernel(const PromptArgs a, int4* list, int* n_tiles)
{
    __shared__ int count[kPromptLevels], scan[kThreads / 32], tops[kThreads / 32], top_before;
    __shared__ int3 long_ones[kThreads];  // begin, end, tiles
    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < kPromptLevels; i += kThreads) count[i] = 0;
    const int span = 2 * a.tile_tokens;
    for (int pass = 0; pass < 2; ++pass) {
        if (tid == 0) top_before = INT32_MIN;
        __syncthreads();
        for (int64_t base = 0; base < a.B; base += kThreads) {
            const int64_t b = base + tid;
            const int lo = b < a.B ? a.cu_seqlens[b] : INT32_MIN, hi = b < a.B ? a.cu_seqlens[b + 1] : INT32_MIN;
            int top = lo;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xFFFFFFFFu, top, o);
                if (lane >= o) top = max(top, x);
            }
            if (lane == 31) tops[warp] = top;
            __syncthreads();
            for (int w = 0; w < warp; ++w) top = max(top, tops[w]);
            top = max(top, top_before);
            const bool valid = prompt_valid(a, lo, hi, top);
            if (pass == 0 && a.out_status && b < a.B) a.out_status[b] = valid ? TPS_ROW_OK : TPS_ROW_BAD_PARAM;
            __syncthreads();
            if (tid == kThreads - 1) top_before = top;
            const int tiles = valid ? prompt_tiles(a, lo, hi) : 0;
            auto put = [&](int l, int h, int t, int64_t seq) {
                const int keys = (int)min((int64_t)h - l, (int64_t)(t + 1) * span);
                const int at = atomicAdd(&count[min((keys + kBlockKeys - 1) / kBlockKeys >> a.level_shift, kPromptLevels - 1)], 1);
                if (pass == 1) list[at] = make_int4(l, h, l + t * span, (int)seq);
            };
            if (!__syncthreads_or(tiles > 8)) {  // short ones: a thread each
                for (int t = 0; t < tiles; ++t) put(lo, hi, t, b);
            } else {  // long ones: a warp each, a lane for each tile
                long_ones[tid] = make_int3(lo, hi, tiles);
                __syncthreads();
                for (int i = warp; i < min(a.B - base, (int64_t)kThreads); i += kThreads / 32)
                    for (int t = lane; t < long_ones[i].z; t += 32) put(long_ones[i].x, long_ones[i].y, t, base + i);
            }
        }
        __syncthreads();
        if (pass == 0) {  // where the tiles of each level begin: those of higher levels come first
            constexpr int kEach = kPromptLevels / kThreads;
            int mine[kEach], sum = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) mine[i] = count[kPromptLevels - 1 - (tid * kEach + i)], sum += mine[i];
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += x;
            }
            if (lane == 31) scan[warp] = incl;
            __syncthreads();
            for (int w = 0; w < warp; ++w) incl += scan[w];
            if (tid == kThreads - 1) *n_tiles = incl;
            int at = incl - sum;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                count[kPromptLevels - 1 - (tid * kEach + i)] = at;
                at += mine[i];
            }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace tps
