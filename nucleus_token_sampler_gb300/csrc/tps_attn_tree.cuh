// tps_attn_tree.cuh -- attention of drafted trees over the paged cache (tps_tree_attention): what it adds to the tcgen05
// kernel of tps_attn_prefix.cuh, whose softmax, products, loads and conversions of 8-bit codes it shares, and the join.
// (Few rows go to the kernels of tps_attn_rows.cuh, by the rule in tps_api_decode.cu.)
//
// Mathematics.  A sequence's last `nodes` tokens in the cache are a tree of drafted ones; node i sees the tokens before
// them and those nodes j whose bit is set in its mask.  All (node, query head) pairs of one key head are rows of tiles of
// 128 (where they fill an odd number of those) or 256: each of the sequence's keys and values is loaded, and converted, once for each tile,
// so once for a tree of up to 128 rows, or of 129 to 256.  The tiles are those of a full tree, whatever a sequence's own number of
// nodes.  Only the blocks that hold drafted tokens are masked.
//
// Tiles of 128 rows: two groups of softmax warps take the item's blocks in turn, each with an output of its own, which are joined
// at the item's end.  While one's softmax runs, the other's products do; with one group both would wait for each other.
//
// Split.  The blocks of 128 tokens of all sequences, key heads and row tiles form one line, which is cut evenly over one
// CTA per SM: long and short sequences, few and many of them fill the SMs alike.  The lengths are on the device, so each CTA
// sums them up to find its place.  An item (sequence, key head, row tile) that lies in one CTA is finished there: at most
// two items of a CTA are not, and leave a piece each (unnormalised output, maximum and sum), which a second kernel joins: the
// workspace does not grow with the batch.
//
// What bounds it: a bfloat16 cache's bytes (256 sequences of 500 to 4,000 tokens and trees of five, 32 heads on 8 of 128: 455 us, 5.2
// TB/s); in 8-bit formats the softmax and the conversion of codes, which take a block of 128 tokens 2.1 us whatever the
// number of rows of a tile of 128 (32 sequences of 2,000 to 8,111 tokens, trees of up to 64, 40 heads on 8 of 64, int8: 377 us); for few tokens
// the launch, a chain of dependent loads (lengths, page, tokens) and the join (8 nodes on 1,000 tokens: 15.6 us; 8 trees of 16 on up to
// 4,093 in fp8: 40 us).  One group of softmax warps instead of two in turn: 20.9 and 50 us for the last two, 424 for the int8 case.
#pragma once

#include <cstdint>

#include "tps_attn_rows.cuh"
#include "tps_decode.h"
#include "tps_tcgen05.cuh"

namespace tps {

// Byte of 16-byte chunk c of row r in a tile: 64-element column blocks of 128 rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_byte(int r, int c)
{
    return (uint32_t)((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

struct TreeStart {
    int seq, head, tile, block, left;  // sequence, key head and row tile of its item, block; blocks of the CTA
    int len, nodes;                    // of the sequence, as they are
};
constexpr int kTreeMarks = 16;                   // items whose marks are kept: loads run at most a ring of single blocks ahead of the output
constexpr int kMarkBad = 1, kMarkNotFinite = 2;  // a page that is not the cache's; values taken out of the product

// A CTA's way along the line: items of sequence after sequence, each of the sequence's own number of blocks (one, where it has no tokens).
struct TreeWay {
    int seq, head, tile, block, left, ordinal;  // ordinal: of the item among the CTA's
    int len, nodes, nblk;                       // tokens of the sequence, drafted ones among them; blocks
    bool bad;                                   // lengths that are not possible: no tokens
    int next_len, next_nodes;                   // of the next sequence, read ahead
    __device__ __forceinline__ explicit TreeWay(const TreeArgs& a, const TreeStart& s)
    {
        seq = s.seq, head = s.head, tile = s.tile, block = s.block, left = s.left, ordinal = 0;
        next_len = s.len, next_nodes = s.nodes;
        enter(a);
    }
    __device__ __forceinline__ void look(const TreeArgs& a, int b)
    {
        next_len = b < a.a.B ? a.a.seq_len[b] : 0;
        next_nodes = a.a.tree_len && b < a.a.B ? a.a.tree_len[b] : a.a.n_nodes;
    }
    __device__ __forceinline__ void enter(const TreeArgs& a)
    {
        len = next_len, nodes = next_nodes;
        bad = tree_bad(a, len, nodes);
        if (bad) len = nodes = 0;
        nblk = tree_blocks(len);
        look(a, seq + 1);
    }
    static __device__ __forceinline__ bool tree_bad(const TreeArgs& a, int len, int nodes)
    {
        return len < 0 || nodes < 0 || nodes > a.a.n_nodes || nodes > len || len > a.a.table_width << a.page_shift;
    }
    static __device__ __forceinline__ int tree_blocks(int len) { return max(1, (len + kBlockKeys - 1) / kBlockKeys); }
    __device__ __forceinline__ int blocks(const TreeArgs&) const { return min(left, nblk - block); }
    __device__ __forceinline__ int tokens(const TreeArgs&) const { return len; }
    __device__ __forceinline__ int open(const TreeArgs&) const { return len - nodes; }
    __device__ __forceinline__ const int32_t* pages(const TreeArgs& a) const { return a.a.page_table + (int64_t)seq * a.a.table_ld; }
    __device__ __forceinline__ void next(const TreeArgs& a)
    {
        left -= blocks(a);
        block = 0;
        ++ordinal;
        if (++tile == a.p.n_tiles) {
            tile = 0;
            if (++head == a.c.n_heads) {
                head = 0;
                ++seq;
                enter(a);
            }
        }
    }
    __device__ __forceinline__ void step(const TreeArgs& a)
    {
        if (block + 1 == nblk)
            next(a);
        else
            --left, ++block;
    }
};

// Where a CTA's equal share of the line begins, found by all its threads.  (The host has seen to it that the line's blocks, and
// a share more, can be counted in 32 bits: divisions of 64 took 2,000 clocks at the start of every CTA.)
template <int kThreads>
__device__ __forceinline__ void tree_start(const TreeArgs& a, TreeStart& start, uint32_t (&sums)[kThreads / 32])
{
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t items = a.c.n_heads * a.p.n_tiles, B = (uint32_t)a.a.B, each = B <= kThreads ? 1 : (B + kThreads - 1) / kThreads;
    const uint32_t from = min(each * tid, B), to = min(from + each, B);
    int len = 0, nodes = 0;
    auto blocks = [&](uint32_t b) {
        len = a.a.seq_len[b], nodes = a.a.tree_len ? a.a.tree_len[b] : a.a.n_nodes;
        return (uint32_t)(TreeWay::tree_bad(a, len, nodes) ? 1 : TreeWay::tree_blocks(len));
    };
    uint32_t mine = 0;
    for (uint32_t b = from; b < to; ++b) mine += blocks(b);
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += x;
    }
    if (lane == 31) sums[warp] = sum;
    if (tid == 0) start = TreeStart{0, 0, 0, 0, 0, 0, 0};
    __syncthreads();
    uint32_t all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) sum += sums[w];
        all += sums[w];
    }
    const uint32_t units = all * items, share = (units + gridDim.x - 1) / gridDim.x, u0 = share * blockIdx.x;
    if (u0 >= (sum - mine) * items && u0 < sum * items) {
        uint32_t before = sum - mine, b = from, n = each == 1 ? mine : blocks(b);
        while (u0 >= (before + n) * items) before += n, n = blocks(++b);
        const uint32_t rest = u0 - before * items, item = rest / n, head = a.p.n_tiles == 1 ? item : item / a.p.n_tiles;
        start = TreeStart{(int)b, (int)head, (int)(item - head * a.p.n_tiles), (int)(rest - item * n), (int)min(share, units - u0), len, nodes};
    }
}

// What a row sees of its sequence's drafted tokens, and whether it is a node's at all.
struct TreeRow {
    uint64_t seen;
    bool live;
};
__device__ __forceinline__ TreeRow tree_row(const TreeArgs& a, const TreeWay& way, int in_item)
{
    const int node = in_item / a.G;
    TreeRow r = {0, in_item < a.p.R && node < way.nodes};
    if (r.live) r.seen = (uint64_t)a.a.tree[(int64_t)way.seq * a.a.tree_ld + node] & (~0ull >> (64 - way.nodes));
    return r;
}
// Of 32 tokens, the first of which is drafted token `from` (below 0: tokens before the tree, at least one of the 32 not), those that are seen.
__device__ __forceinline__ uint32_t tree_seen(uint64_t seen, int from)
{
    if (from >= 0) return from < 64 ? (uint32_t)(seen >> from) : 0u;
    return (uint32_t)(seen << -from) | ((1u << -from) - 1u);
}

// bfloat16 values of a tile's rows first .. last - 1 that are not finite leave it; true where there are any (one warp).
template <int D> __device__ __forceinline__ bool hide_not_finite(unsigned char* tile, int first, int last)
{
    bool found = false;
#pragma unroll 4
    for (int i = first * (D / 8) + (int)(threadIdx.x & 31); i < min(last, kBlockKeys) * (D / 8); i += 32) {
        uint4* p = reinterpret_cast<uint4*>(tile + tile_byte(i / (D / 8), i % (D / 8)));
        const uint4 x = *p, y = make_uint4(not_finite(x.x), not_finite(x.y), not_finite(x.z), not_finite(x.w));
        if (y.x | y.y | y.z | y.w) {
            found = true;
            *p = make_uint4(x.x ^ y.x, x.y ^ y.y, x.z ^ y.z, x.w ^ y.w);
        }
    }
    return found;
}

// The sum of a row's bfloat16 weights as the second product has them, 32 to each of `groups` 16 columns.
__device__ __forceinline__ float weight_sum(uint32_t addr, int groups)
{
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int i = 0; i < groups; ++i) {
        uint32_t w[16];
        tmem_ld16(addr + i * 16, w);
        tmem_wait_ld(w);
#pragma unroll
        for (int j = 0; j < 16; ++j) sum.x += __uint_as_float(w[j] << 16), sum.y += __uint_as_float(w[j] & 0xFFFF0000u);
    }
    return sum.x + sum.y;
}

__device__ __forceinline__ bool tree_whole(const TreeWay& way, int blocks) { return way.block == 0 && blocks == way.nblk; }
// A CTA's piece of an item that began in an earlier one, and of one that goes on in the next.
__device__ __forceinline__ int64_t tree_piece(const TreeWay& way) { return 2 * (int64_t)blockIdx.x + (way.block == 0 ? 1 : 0); }
// Row `in_item` of the call's output, in heads.
__device__ __forceinline__ int64_t tree_row_at(const TreeArgs& a, int seq, int head, int in_item)
{
    const int node = in_item / a.G;
    return ((int64_t)seq * a.a.n_nodes + node) * a.a.n_q_heads + (int64_t)head * a.G + (in_item - node * a.G);
}

// The two warps that have 32 rows in turn wait for one another.
__device__ __forceinline__ void pair_sync(int pair) { asm volatile("barrier.cta.sync.aligned %0, 64;" ::"r"(pair + 1) : "memory"); }

// The outputs of a warp's rows: finished, or a piece.  `mine_sum`: reference, sum and what rounding took from it; in turn, `other_sum` is the other group's
// part of the row, whose output lies D columns from this one's, and each group writes a half of the columns.
template <int D, int kFormat, bool kTurns>
__device__ __forceinline__ void tree_output(const TreeArgs& a, const TreeWay& way, int blocks, const TreeRow& mine, int in_tile, int in_item, int m,
                                            uint32_t out_col, uint32_t o_addr, float3 mine_sum, float3 other_sum, int marks)
{
    if (in_item - (int)(threadIdx.x & 31) >= a.p.R) return;  // none of the warp's
    const bool both = kTurns && blocks > 1, in = in_item < a.p.R, bad = marks & kMarkBad, whole = tree_whole(way, blocks);
    float ref = mine_sum.x, sum = mine_sum.y, lost = mine_sum.z, f = 1.f, g = 0.f;
    if (both) {
        ref = fmaxf(mine_sum.x, other_sum.x);
        f = mine_sum.x == ref ? 1.f : exp2_fast(mine_sum.x - ref), g = other_sum.x == ref ? 1.f : exp2_fast(other_sum.x - ref);
        sum = mine_sum.y * f + other_sum.y * g, lost = mine_sum.z * f + other_sum.z * g;
    } else if (kTurns && m == 1) {  // one block: the other group's
        ref = other_sum.x, sum = other_sum.y, lost = other_sum.z;
    }
    const bool empty = !mine.live || sum == 0.f;
    const int64_t at = tree_row_at(a, way.seq, way.head, in_item), piece = tree_piece(way);
    const float inv = bad ? __int_as_float(0x7FC00000) : (empty ? 0.f : 1.f / sum);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.a.out) + at * D);
    float4* part = reinterpret_cast<float4*>(a.part + piece * a.p.tile_rows * D) + in_tile;
    const int from = kTurns ? m * (D / 2) : 0, to = kTurns ? from + D / 2 : D;
#pragma unroll 1
    for (int i = from; i < to; i += 32) {
        float o[32];
        tmem_ld32((kTurns ? (both ? o_addr : out_col) : o_addr) + i, o);
        tmem_wait_ld(o);
        if (both) {
            float o2[32];
            tmem_ld32(out_col + D * (m ^ 1) + i, o2);
            tmem_wait_ld(o2);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = o[j] * f + o2[j] * g;
        }
        if (!in) continue;
        if (kFormat == TPS_KV_BF16 && (marks & kMarkNotFinite) && !bad) {  // what was taken out of the product, for a row that sees it
            for (uint64_t left = mine.seen; left; left &= left - 1) {
                const int token = way.len - way.nodes + __ffsll((long long)left) - 1;
                if (token < way.block * kBlockKeys || token >= (way.block + blocks) * kBlockKeys) continue;
                const int64_t id = way.pages(a)[token >> a.page_shift];
                const int64_t row = ((id * a.c.n_heads + way.head) << a.page_shift) + (token & ((1 << a.page_shift) - 1));
                const uint32_t* v = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.c.v) + row * D + i);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const uint32_t x = not_finite(v[k]);
                    o[2 * k] += __uint_as_float(x << 16);
                    o[2 * k + 1] += __uint_as_float(x & 0xFFFF0000u);
                }
            }
        }
        if (whole) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const __nv_bfloat162 y = empty && !bad ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(o[2 * j] * inv, o[2 * j + 1] * inv);
                w[j] = *reinterpret_cast<const uint32_t*>(&y);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[i / 8 + j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4) part[(i + j) / 4 * a.p.tile_rows] = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        }
    }
    if (!in || (kTurns && m == 1)) return;
    if (whole) {
        if (a.a.out_lse) a.a.out_lse[at] = log_sum<kFormat>(ref, mine.live ? sum + lost : 0.f, bad);
    } else {
        a.ml[piece * a.p.tile_rows + in_tile] = make_float2(ref, bad ? kPieceBadPage : (mine.live ? sum : 0.f));
        a.lost[piece * a.p.tile_rows + in_tile] = lost;
    }
}

// A row of an item (or of its part) that was not reached.
template <int D> __device__ __forceinline__ void tree_give_up(const TreeArgs& a, const TreeWay& way, int in_tile)
{
    const int in_item = way.tile * a.p.tile_rows + in_tile;
    if (in_item >= a.p.R) return;
    if (!tree_whole(way, way.blocks(a))) {
        a.ml[tree_piece(way) * a.p.tile_rows + in_tile] = make_float2(0.f, kPieceTimeout);
        return;
    }
    const int64_t at = tree_row_at(a, way.seq, way.head, in_item);
    const uint4 nan = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
    for (int i = 0; i < D / 8; ++i) reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.a.out) + at * D)[i] = nan;
    if (a.a.out_lse) a.a.out_lse[at] = __int_as_float(0x7FC00000);
}

}  // namespace tps
