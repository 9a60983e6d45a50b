// tps_api_decode.cu -- the C ABI of the decode-step operators declared in include/tps.h: argument
// checks, the choice of kernels and launch shapes, and the launches.  Like tps_api.cu it never
// synchronises the host and keeps no state between calls.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/tps.h"
#include "tps_decode.h"

namespace {

constexpr int kMaxHeads = 65535;
// Tokens of a prefix or of a sequence's pages: the walks over them count in 32 bits and go on by at most 512 past the
// last one, a tile's boxes by 4,096.
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - (1 << 16);

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int elem_bytes(int dtype) { return dtype == TPS_F32 ? 4 : (dtype == TPS_BF16 ? 2 : 0); }

int check_cache(const tps_kv_cache* c, bool pointers)
{
    if (!c) return TPS_ERR_ARG;
    const int ps = c->page_size;
    if (c->format < TPS_KV_BF16 || c->format > TPS_KV_INT8) return TPS_ERR_ARG;
    if (ps < 16 || ps > 256 || (ps & (ps - 1)) != 0) return TPS_ERR_ARG;
    if (c->head_dim < 16 || c->head_dim > 512 || c->head_dim % 16 != 0) return TPS_ERR_ARG;
    if (c->n_heads < 1 || c->n_heads > kMaxHeads || c->n_pages < 1 || c->n_pages > INT32_MAX) return TPS_ERR_ARG;
    if (!pointers) return TPS_OK;
    if (!c->k || !c->v) return TPS_ERR_ARG;
    if (c->format != TPS_KV_BF16 && (!c->k_scale || !c->v_scale)) return TPS_ERR_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return TPS_ERR_ALIGN;
    if (c->format != TPS_KV_BF16 && (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))) return TPS_ERR_ALIGN;
    return TPS_OK;
}

// Tokens (times triples of sequence, key head and row tile) up to which each sequence walks over the prefix
// itself: one launch instead of two, and nothing to join, for reading the prefix again from the L2 cache.
// With 8 key heads of 128, alone / shared, us: bfloat16 8 x 500 9.2 / 9.7, 5 x 1,000 11.0 / 10.0, 8 x 1,000 11.1 /
// 10.1, 2 x 2,000 14.7 / 10.5, 8 x 2,000 21.3 / 12.8; fp8 (whose shared part converts its codes) 5 x 1,000 10.9 /
// 13.3, 8 x 1,000 12.3 / 13.3, 8 x 2,000 20.6 / 16.0, 5 x 2,000 16.8 / 14.7, 2 x 4,000 16.3 / 15.9.  The product of tokens
// and triples is not all that decides: 8 x 500 in bfloat16 and 8 x 1,000 in fp8 fall on the slower side, by 0.5 and 1.0 us.
constexpr int64_t kAloneBf16 = 24576, kAlone8 = 49152;
// Sequences (times heads and row tiles) per SM from which each warp takes one for itself, and where they hold few
// tokens.  4 warps of a CTA / one warp each, on a prefix of 4,000, bfloat16, us: 768 items of up to 60 tokens 30.3 /
// 28.8, of 300 38.3 / 46.8; 1,024 items 36.4 / 29.1 and 45.6 / 48.5; 1,216 items 44.9 / 32.2 and 54.2 / 51.4.
constexpr int64_t kOneWarpItems = 8, kOneWarpShort = 5, kShortTokens = 128;
// Tokens of one sequence (at most) from which the own tokens are cut evenly over the SMs, for up to kLinePairs
// sequences times row tiles.  Clusters / even cuts, 16 sequences with 8 key heads of 128, us: bfloat16 2,000 tokens
// 36.7 / 38.0, 4,000 58.6 / 49.8; fp8 4,000 41.3 / 44.2, 9,000 69.2 / 59.6; 48 sequences: bfloat16 4,000 107 / 113,
// 8,000 196 / 171; fp8 4,000 106 / 99.  (16 x 4,000 in bfloat16 lies just below the rule, on the slower side.)  The tokens
// are those that the page table has room for; the lengths are on the device.
constexpr int64_t kLineTokens = 4096, kLinePairs = 1024;

int plan_attention(const tps_kv_cache& c, const tps_attention& a, int sms, tps::AttnPlan* out)
{
    tps::AttnPlan p = {};
    const int G = a.n_q_heads / c.n_heads;
    const int64_t own_rows = (int64_t)a.q_len * G;
    if (own_rows > (1 << 24) || a.B > (int64_t(1) << 31) / (own_rows * c.n_heads)) return TPS_ERR_ARG;
    p.R = a.B * own_rows;
    p.suffix_rows = own_rows <= 8 ? 8 : 16;
    p.suffix_tiles = (int)((own_rows + p.suffix_rows - 1) / p.suffix_rows);
    const int64_t alone = a.B * c.n_heads * p.suffix_tiles;  // (sequence, key head, tile) triples
    p.shared = a.prefix_len > 0 && a.B > 1 && alone > (c.format == TPS_KV_BF16 ? kAloneBf16 : kAlone8) / a.prefix_len;
    if (p.shared) {
        p.tile_rows = p.R <= 128 ? 128 : 256;
        const int64_t n_tiles = (p.R + p.tile_rows - 1) / p.tile_rows, items = n_tiles * c.n_heads;
        p.nblk = (int)((a.prefix_len + tps::kBlockKeys - 1) / tps::kBlockKeys);
        if (items > INT32_MAX / p.nblk) return TPS_ERR_ARG;
        p.n_tiles = (int)n_tiles;
        p.items = (int)items;
        p.units = p.items * p.nblk;
        // No more CTAs than the longest share needs: fewer pieces to join, and SMs left for the own tokens.
        p.share = (int)(((int64_t)p.units + sms - 1) / sms);
        p.ctas = (int)(((int64_t)p.units + p.share - 1) / p.share);
        p.pieces = (int64_t)p.ctas + p.items;
    }
    // Several CTAs share one sequence's tokens where there are few sequences and many tokens, as long as
    // all of them are resident at once (by the kernel's registers and shared memory).  One CTA / a cluster of 4 or 8, us:
    // 8 x (1,000 + 40) in bfloat16 17.6 / 11.2, 4 x (500 + 500) in fp8 20.0 / 10.2.
    const int64_t resident = (int64_t)sms * (p.suffix_rows == 8 && c.format != TPS_KV_BF16 ? 4 : 3);
    const int64_t tokens = a.table_width * c.page_size + (p.shared ? 0 : a.prefix_len);
    p.one_warp = alone >= (tokens <= kShortTokens ? kOneWarpShort : kOneWarpItems) * sms;
    p.line = !p.one_warp && a.B * p.suffix_tiles <= kLinePairs && tokens >= kLineTokens;
    p.cluster = 1;
    while (!p.one_warp && !p.line && p.cluster < 8 && alone * p.cluster * 2 <= resident && tokens >= (int64_t)p.cluster * 256)
        p.cluster *= 2;
    if (alone * p.cluster > INT32_MAX - 4) return TPS_ERR_ARG;
    p.off_ml = (size_t)p.pieces * p.tile_rows * c.head_dim * sizeof(float);
    p.bytes = p.off_ml + (size_t)p.pieces * p.tile_rows * sizeof(float2);
    if (p.line) {
        p.line_ctas = 3 * (int64_t)sms;  // as many as are resident
        p.line_pieces = p.line_ctas + alone;
        p.off_line_part = (p.bytes + 255) / 256 * 256;
        p.off_line_ml = p.off_line_part + (size_t)p.line_pieces * p.suffix_rows * c.head_dim * sizeof(float);
        p.bytes = p.off_line_ml + (size_t)p.line_pieces * p.suffix_rows * sizeof(float2);
    }
    *out = p;
    return TPS_OK;
}

int check_attention(const tps_kv_cache* c, const tps_attention* a, bool pointers)
{
    if (!a) return TPS_ERR_ARG;
    const int rc = check_cache(c, pointers);
    if (rc != TPS_OK) return rc;
    if (c->head_dim != 64 && c->head_dim != 128) return TPS_ERR_ARG;
    if (a->B < 0 || a->prefix_len < 0 || a->prefix_len > kMaxTokens || a->table_width < 0 || a->table_width > kMaxTokens / c->page_size ||
        a->table_ld < a->table_width || a->q_len < 1 || a->n_q_heads < 1 || a->n_q_heads % c->n_heads != 0 ||
        !std::isfinite(a->scale))
        return TPS_ERR_ARG;
    if (!pointers || a->B == 0) return TPS_OK;
    if (!a->q || !a->out || !a->suffix_len || (a->prefix_len > 0 && !a->prefix_pages) || (a->table_width > 0 && !a->page_table))
        return TPS_ERR_ARG;
    if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->out_lse, 4) || !aligned(a->prefix_pages, 4) ||
        !aligned(a->page_table, 4) || !aligned(a->suffix_len, 4) || !aligned(a->out_status, 4) || !aligned(a->workspace, 256))
        return TPS_ERR_ALIGN;
    return TPS_OK;
}

// A stride that a tensor map takes: whole 16-byte units, no two elements of the axis in one place.
bool map_stride(int64_t elements, int64_t n, int D) { return n <= 1 || (elements >= D && elements % 8 == 0 && elements < (int64_t(1) << 38)); }

// `tiles`: the most pairs of a sequence and 256 of its query rows (of one key head's group) there can be.
int check_prompt(const tps_prompt* p, tps::PromptArgs* a, int64_t* tiles)
{
    if (!p) return TPS_ERR_ARG;
    if (p->head_dim != 64 && p->head_dim != 128) return TPS_ERR_ARG;
    if (p->T < 0 || p->T > kMaxTokens || p->B < 0 || p->B > INT32_MAX || p->n_k_heads < 1 || p->n_k_heads > kMaxHeads || p->n_q_heads < 1 ||
        p->n_q_heads > kMaxHeads || p->n_q_heads % p->n_k_heads != 0 || !std::isfinite(p->scale))
        return TPS_ERR_ARG;
    if (p->B == 0) return TPS_OK;
    if (!p->cu_seqlens || (p->T > 0 && (!p->q || !p->k || !p->v || !p->out))) return TPS_ERR_ARG;
    if (!map_stride(p->q_ld, p->T, p->head_dim) || !map_stride(p->k_ld, p->T, p->head_dim) || !map_stride(p->v_ld, p->T, p->head_dim) ||
        !map_stride(p->q_hd, p->n_q_heads, p->head_dim) || !map_stride(p->k_hd, p->n_k_heads, p->head_dim) ||
        !map_stride(p->v_hd, p->n_k_heads, p->head_dim))
        return TPS_ERR_ARG;
    if (!aligned(p->q, 16) || !aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->out, 16) || !aligned(p->out_lse, 4) ||
        !aligned(p->cu_seqlens, 4) || !aligned(p->out_status, 4))
        return TPS_ERR_ALIGN;
    a->v = p->v, a->out = p->out, a->out_lse = p->out_lse, a->cu_seqlens = p->cu_seqlens, a->out_status = p->out_status;
    a->T = p->T, a->B = p->B, a->v_ld = p->v_ld, a->v_hd = p->v_hd;
    a->Hq = p->n_q_heads, a->G = p->n_q_heads / p->n_k_heads;
    a->groups = (a->G + 127) / 128;
    a->group = (a->G + a->groups - 1) / a->groups;
    a->heads_v = p->n_k_heads * a->groups;
    a->tile_tokens = 128 / a->group;
    a->sectors = aligned(p->out, 32);
    a->level_shift = 0;
    while ((p->T / tps::kBlockKeys + 1) >> a->level_shift >= 2048) ++a->level_shift;
    a->qk_scale = (float)((double)p->scale * 1.4426950408889634);
    if (!std::isfinite(a->qk_scale)) return TPS_ERR_ARG;
    *tiles = p->T / (2 * a->tile_tokens) + p->B;
    return *tiles > (INT32_MAX - 65536) / a->heads_v ? TPS_ERR_ARG : TPS_OK;
}

int check_tree(const tps_kv_cache* c, const tps_tree* t, bool pointers)
{
    if (!t) return TPS_ERR_ARG;
    const int rc = check_cache(c, pointers);
    if (rc != TPS_OK) return rc;
    if (c->head_dim != 64 && c->head_dim != 128) return TPS_ERR_ARG;
    if (t->B < 0 || t->table_width < 0 || t->table_width > kMaxTokens / c->page_size || t->table_ld < t->table_width || t->n_nodes < 1 ||
        t->n_nodes > 64 || t->n_q_heads < 1 || t->n_q_heads > kMaxHeads || t->n_q_heads % c->n_heads != 0 ||
        (t->tree_ld != 0 && t->tree_ld < t->n_nodes) || !std::isfinite((float)((double)t->scale * 1.4426950408889634)))
        return TPS_ERR_ARG;
    if (!pointers || t->B == 0) return TPS_OK;
    if (!t->q || !t->out || !t->seq_len || !t->tree || (t->table_width > 0 && !t->page_table)) return TPS_ERR_ARG;
    if (!aligned(t->q, 16) || !aligned(t->out, 16) || !aligned(t->out_lse, 4) || !aligned(t->page_table, 4) || !aligned(t->seq_len, 4) ||
        !aligned(t->tree_len, 4) || !aligned(t->tree, 8) || !aligned(t->out_status, 4) || !aligned(t->workspace, 256))
        return TPS_ERR_ALIGN;
    return TPS_OK;
}

// Rows of a sequence and key head up to which trees take the kernels of a prefix call's own tokens.  Over an 8-bit cache their products of 8
// or 16 rows convert no code twice and fill no tile of 128: less work for each token, though each 16 rows would read them again.
// tcgen05 / those, us: 8 sequences of up to 4,000 in fp8, 8 key heads of 128, 4 rows 39 / 20, 16 rows 40 / 32, 32 rows 41 / 52; 32 of up
// to 8,000 in int8, heads of 64, 5 rows 140 / 71, 15 rows 140 / 83, 30 rows 142 / 153; 256 of up to 3,000 in fp8, 8 rows 501 / 269.
constexpr int kTreeFewRows = 16;
// In bfloat16, which needs no conversion, it is a shorter chain for few tokens and a join without a second launch: where there are few
// (sequence, key head) items, and where sequences are short (by their tables: only the device knows the lengths), whose tiles of 128 rows
// cost tcgen05 some 9,000 clocks each.  Up to 8 rows, 8 heads of 128: 1 of 1,000 15.0 / 9.0, of 10,000 29.7 / 20.4, 8 of 1,000 15.7 / 12.3,
// 32 of 3,000 73 / 66, 8 of 30,000 154 / 161, 64 of 3,000 129 / 171; 64 of 1,000 58 / 67, of 500 to 1,000 56 / 50, 256 of 500 to 1,000
// 173 / 152, of 150 to 300 84 / 54, 1,000 of up to 128 218 / 77.
// 9 to 16 rows: 1 head, 1 of 300 12.0 / 13.5, of 1,000 15.1 / 15.0, of 30,000 89 / 32; 8 heads, 1 of 1,000 15.3 / 14.1, 4 of 10,000
// 42 / 49; 64 of 250 to 500 39 / 44, 256 118 / 96, 8 of up to 128 8.9 / 12.6, 1,000 of up to 128 235 / 111.
constexpr int kTreeFewRowsBf16 = 8;
constexpr int64_t kTreeFewItemsBf16 = 256, kTreeShortBf16 = 1024;
constexpr int64_t kTreeItems16Bf16 = 8, kTreeShort16Bf16 = 512, kTreeManyItemsBf16 = 1024;
bool tree_few(const tps_kv_cache& c, const tps_tree& t)
{
    const int64_t rows = (int64_t)t.n_nodes * (t.n_q_heads / c.n_heads), tokens = t.table_width * c.page_size;
    if (rows > kTreeFewRows || c.format != TPS_KV_BF16) return rows <= kTreeFewRows;
    auto most_items = [&](int64_t n) { return t.B <= n / c.n_heads; };
    if (rows <= kTreeFewRowsBf16) return most_items(kTreeFewItemsBf16) || tokens <= kTreeShortBf16;
    return tokens <= kTreeShort16Bf16 ? !most_items(kTreeManyItemsBf16 - 1) : most_items(kTreeItems16Bf16);
}
// The same call as one on own tokens alone.
tps_attention tree_as_own(const tps_tree& t)
{
    tps_attention a = {};
    a.q = t.q, a.out = t.out, a.out_lse = t.out_lse, a.page_table = t.page_table, a.suffix_len = t.seq_len, a.out_status = t.out_status;
    a.workspace = t.workspace, a.workspace_bytes = t.workspace_bytes;
    a.B = t.B, a.table_width = t.table_width, a.table_ld = t.table_ld;
    a.q_len = t.n_nodes, a.n_q_heads = t.n_q_heads, a.scale = t.scale;
    return a;
}

int plan_tree(const tps_kv_cache& c, const tps_tree& t, int sms, tps::TreePlan* out)
{
    tps::TreePlan p = {};
    const int64_t R = (int64_t)t.n_nodes * (t.n_q_heads / c.n_heads);  // at most 2^22
    p.R = (int)R;
    // Tiles of 256 rows load and convert keys and values for twice as many; those of 128 leave fewer rows unused.
    p.tile_rows = (R + 127) / 128 % 2 ? 128 : 256;
    p.n_tiles = (int)((R + p.tile_rows - 1) / p.tile_rows);
    const int64_t items = (int64_t)p.n_tiles * c.n_heads;  // of a sequence
    const int64_t most = std::max<int64_t>((t.table_width * c.page_size + tps::kBlockKeys - 1) / tps::kBlockKeys, 1) * items;
    if (most > INT32_MAX || t.B > INT32_MAX / most) return TPS_ERR_ARG;  // the kernels count the line's blocks in 32 bits
    p.ctas = (int)std::min<int64_t>(sms, most * t.B);
    p.off_ml = (size_t)2 * p.ctas * p.tile_rows * c.head_dim * sizeof(float);
    p.off_lost = p.off_ml + (size_t)2 * p.ctas * p.tile_rows * sizeof(float2);
    p.off_rec = p.off_lost + (size_t)2 * p.ctas * p.tile_rows * sizeof(float);
    p.bytes = p.off_rec + (size_t)p.ctas * sizeof(tps::TreeRecord);
    *out = p;
    return TPS_OK;
}

int check_pages(const tps_kv_pages* p, tps::PagesArgs* a)
{
    if (!p) return TPS_ERR_ARG;
    const int ps = p->page_size;
    if (ps < 16 || ps > 256 || (ps & (ps - 1)) != 0 || p->B < 0 || p->B > INT32_MAX || p->table_width < 0 ||
        p->table_width > kMaxTokens / ps || p->table_ld < p->table_width || p->n_free < 0 || p->n_free > INT32_MAX)
        return TPS_ERR_ARG;
    if (!p->free_count || (p->n_free > 0 && !p->free_pages) || (p->B > 0 && (!p->seq_len || !p->change || (p->table_width > 0 && !p->page_table))))
        return TPS_ERR_ARG;
    if (!aligned(p->page_table, 4) || !aligned(p->seq_len, 4) || !aligned(p->change, 4) || !aligned(p->free_pages, 4) ||
        !aligned(p->free_count, 4) || !aligned(p->out_status, 4))
        return TPS_ERR_ALIGN;
    a->p = *p;
    a->page_shift = 4;
    while ((1 << a->page_shift) < ps) ++a->page_shift;
    a->page_mask = ps - 1;
    return TPS_OK;
}

// The launches of a planned call (a.p, and a.tree with what belongs to it) and its workspace.
int run_attention(tps::AttnArgs& a, const tps_kv_cache& cache, const tps_attention& args, int stall_head, uint64_t wait_ns, cudaStream_t st)
{
    a.c = cache;
    a.a = args;
    a.stall_head = stall_head;
    a.wait_ns = wait_ns;
    a.G = args.n_q_heads / cache.n_heads;
    a.page_shift = 4;
    while ((1 << a.page_shift) < cache.page_size) ++a.page_shift;
    a.qk_scale = (float)((double)args.scale * 1.4426950408889634);
    unsigned char* ws = static_cast<unsigned char*>(args.workspace);
    cudaError_t e = cudaSuccess;
    if (a.p.bytes) {
        if (ws) {
            if (args.workspace_bytes < (int64_t)a.p.bytes) return TPS_ERR_SCRATCH;
        } else {
            void* mem = nullptr;
            e = tps::pool_alloc(&mem, a.p.bytes, st);
            if (e != cudaSuccess) return tps::report_cuda(e);
            ws = static_cast<unsigned char*>(mem);
        }
    }
    a.part = reinterpret_cast<float*>(ws);
    a.ml = reinterpret_cast<float2*>(ws + a.p.off_ml);
    a.line_part = reinterpret_cast<float*>(ws + a.p.off_line_part);
    a.line_ml = reinterpret_cast<float2*>(ws + a.p.off_line_ml);
    if (a.p.units) {
        e = cache.format == TPS_KV_BF16  ? tps::launch_attn_prefix_bf16(a, st)
            : cache.format == TPS_KV_FP8 ? tps::launch_attn_prefix_fp8(a, st)
                                          : tps::launch_attn_prefix_int8(a, st);
    }
    if (e == cudaSuccess) e = a.tree ? tps::launch_attn_tree_rows(a, st) : tps::launch_attn_own(a, a.p.units > 0, st);
    if (a.p.bytes && !args.workspace) {
        const cudaError_t ef = cudaFreeAsync(ws, st);
        if (e == cudaSuccess) e = ef;
    }
    return e == cudaSuccess ? TPS_OK : tps::report_cuda(e);
}

}  // namespace

extern "C" {

int tps_qk_norm_rope(const tps_norm_rope* args, void* stream)
{
    if (!args) return TPS_ERR_ARG;
    const tps_norm_rope& a = *args;
    const int es = elem_bytes(a.dtype);
    if (a.T < 0 || a.T > INT32_MAX || a.n_q_heads < 0 || a.n_q_heads > kMaxHeads || a.n_k_heads < 0 || a.n_k_heads > kMaxHeads ||
        a.head_dim < 1 || a.head_dim > 8192 || a.rot_dim < 0 || a.rot_dim > a.head_dim || a.rot_dim % 2 != 0 ||
        a.n_positions < 0 || !(a.eps >= 0.f) || std::isinf(a.eps))
        return TPS_ERR_ARG;
    if (!es) return TPS_ERR_DTYPE;
    if (a.T == 0 || a.n_q_heads + a.n_k_heads == 0) return TPS_OK;
    if ((a.n_q_heads && (!a.q || !a.out_q)) || (a.n_k_heads && (!a.k || !a.out_k)) || !a.positions ||
        (a.rot_dim && !a.cos_sin))
        return TPS_ERR_ARG;
    if ((a.n_q_heads && (!aligned(a.q, es) || !aligned(a.out_q, es))) ||
        (a.n_k_heads && (!aligned(a.k, es) || !aligned(a.out_k, es))) || !aligned(a.q_weight, 4) || !aligned(a.k_weight, 4) ||
        !aligned(a.positions, 4) || !aligned(a.cos_sin, 4) || !aligned(a.out_status, 4))
        return TPS_ERR_ALIGN;
    int sms = 0;
    if (!tps::host_sms(&sms)) return tps::report_cuda(cudaGetLastError());
    const cudaError_t e = tps::launch_norm_rope(a, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TPS_OK : tps::report_cuda(e);
}

int tps_kv_write(const tps_kv_cache* cache, const void* k, const void* v, int dtype, int64_t T, int64_t k_ld, int64_t k_hd,
                 int64_t v_ld, int64_t v_hd, const int64_t* slots, void* stream)
{
    const int rc = check_cache(cache, true);
    if (rc != TPS_OK) return rc;
    if (T < 0) return TPS_ERR_ARG;
    const int es = elem_bytes(dtype);
    if (!es) return TPS_ERR_DTYPE;
    if (T == 0) return TPS_OK;
    if (!k || !v || !slots) return TPS_ERR_ARG;
    if (!aligned(k, es) || !aligned(v, es) || !aligned(slots, 8)) return TPS_ERR_ALIGN;
    int sms = 0;
    if (!tps::host_sms(&sms)) return tps::report_cuda(cudaGetLastError());
    const tps::KvWriteArgs a{*cache, k, v, T, k_ld, k_hd, v_ld, v_hd, slots};
    const cudaError_t e = tps::launch_kv_write(a, dtype == TPS_BF16, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TPS_OK : tps::report_cuda(e);
}

int tps_kv_read(const tps_kv_cache* cache, const int64_t* slots, int64_t T, void* out_k, void* out_v, int dtype, void* stream)
{
    const int rc = check_cache(cache, true);
    if (rc != TPS_OK) return rc;
    if (T < 0) return TPS_ERR_ARG;
    if (!elem_bytes(dtype)) return TPS_ERR_DTYPE;
    if (T == 0) return TPS_OK;
    if (!slots || !out_k || !out_v) return TPS_ERR_ARG;
    if (!aligned(slots, 8) || !aligned(out_k, 16) || !aligned(out_v, 16)) return TPS_ERR_ALIGN;
    int sms = 0;
    if (!tps::host_sms(&sms)) return tps::report_cuda(cudaGetLastError());
    const tps::KvReadArgs a{*cache, slots, T, out_k, out_v};
    const cudaError_t e = tps::launch_kv_read(a, dtype == TPS_BF16, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TPS_OK : tps::report_cuda(e);
}

int64_t tps_prefix_attention_workspace(const tps_kv_cache* cache, const tps_attention* args)
{
    if (check_attention(cache, args, false) != TPS_OK) return -1;
    if (args->B == 0) return 0;
    int sms = 0;
    tps::AttnPlan p;
    if (!tps::host_sms(&sms) || plan_attention(*cache, *args, sms, &p) != TPS_OK) return -1;
    return (int64_t)p.bytes;
}

int tps_prefix_attention(const tps_kv_cache* cache, const tps_attention* args, void* stream)
{
    return tps_prefix_attention_stall_test(cache, args, -1, tps::kAttnWaitNs, stream);
}

int tps_prefix_attention_stall_test(const tps_kv_cache* cache, const tps_attention* args, int stall_head, uint64_t wait_ns,
                                    void* stream)
{
    if (wait_ns < 1 || wait_ns > tps::kAttnWaitNs) return TPS_ERR_ARG;
    int rc = check_attention(cache, args, true);
    if (rc != TPS_OK) return rc;
    if (args->B == 0) return TPS_OK;
    int sms = 0;
    if (!tps::host_sms(&sms)) return tps::report_cuda(cudaGetLastError());
    tps::AttnArgs a = {};
    rc = plan_attention(*cache, *args, sms, &a.p);
    if (rc != TPS_OK) return rc;
    return run_attention(a, *cache, *args, stall_head, wait_ns, static_cast<cudaStream_t>(stream));
}

int64_t tps_tree_attention_workspace(const tps_kv_cache* cache, const tps_tree* args)
{
    if (check_tree(cache, args, false) != TPS_OK) return -1;
    if (args->B == 0) return 0;
    int sms = 0;
    if (!tps::host_sms(&sms)) return -1;
    if (tree_few(*cache, *args)) {
        tps::AttnPlan p;
        return plan_attention(*cache, tree_as_own(*args), sms, &p) == TPS_OK ? (int64_t)p.bytes : -1;
    }
    tps::TreePlan p;
    return plan_tree(*cache, *args, sms, &p) == TPS_OK ? (int64_t)p.bytes : -1;
}

int tps_tree_attention(const tps_kv_cache* cache, const tps_tree* args, void* stream)
{
    return tps_tree_attention_stall_test(cache, args, -1, tps::kAttnWaitNs, stream);
}

int tps_tree_attention_stall_test(const tps_kv_cache* cache, const tps_tree* args, int stall_head, uint64_t wait_ns, void* stream)
{
    if (wait_ns < 1 || wait_ns > tps::kAttnWaitNs) return TPS_ERR_ARG;
    int rc = check_tree(cache, args, true);
    if (rc != TPS_OK) return rc;
    if (args->B == 0) return TPS_OK;
    int sms = 0;
    if (!tps::host_sms(&sms)) return tps::report_cuda(cudaGetLastError());
    if (tree_few(*cache, *args)) {
        tps::AttnArgs few = {};
        const tps_attention own = tree_as_own(*args);
        rc = plan_attention(*cache, own, sms, &few.p);
        if (rc != TPS_OK) return rc;
        few.tree = args->tree, few.tree_ld = args->tree_ld, few.tree_len = args->tree_len;
        return run_attention(few, *cache, own, stall_head, wait_ns, static_cast<cudaStream_t>(stream));
    }
    tps::TreeArgs a = {};
    rc = plan_tree(*cache, *args, sms, &a.p);
    if (rc != TPS_OK) return rc;
    a.c = *cache;
    a.a = *args;
    a.stall_head = stall_head;
    a.wait_ns = wait_ns;
    a.G = args->n_q_heads / cache->n_heads;
    a.page_shift = 4;
    while ((1 << a.page_shift) < cache->page_size) ++a.page_shift;
    a.qk_scale = (float)((double)args->scale * 1.4426950408889634);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(args->workspace);
    cudaError_t e = cudaSuccess;
    if (ws) {
        if (args->workspace_bytes < (int64_t)a.p.bytes) return TPS_ERR_SCRATCH;
    } else {
        void* mem = nullptr;
        e = tps::pool_alloc(&mem, a.p.bytes, st);
        if (e != cudaSuccess) return tps::report_cuda(e);
        ws = static_cast<unsigned char*>(mem);
    }
    a.part = reinterpret_cast<float*>(ws);
    a.ml = reinterpret_cast<float2*>(ws + a.p.off_ml);
    a.lost = reinterpret_cast<float*>(ws + a.p.off_lost);
    a.rec = reinterpret_cast<tps::TreeRecord*>(ws + a.p.off_rec);
    e = cache->format == TPS_KV_BF16  ? tps::launch_attn_tree_bf16(a, st)
        : cache->format == TPS_KV_FP8 ? tps::launch_attn_tree_fp8(a, st)
                                      : tps::launch_attn_tree_int8(a, st);
    if (e == cudaSuccess) e = tps::launch_tree_join(a, st);
    if (!args->workspace) {
        const cudaError_t ef = cudaFreeAsync(ws, st);
        if (e == cudaSuccess) e = ef;
    }
    return e == cudaSuccess ? TPS_OK : tps::report_cuda(e);
}

int tps_kv_extend(const tps_kv_pages* pages, int64_t tokens, int64_t* slots, int32_t* positions, int32_t* cu_seqlens, void* stream)
{
    tps::PagesArgs a = {};
    const int rc = check_pages(pages, &a);
    if (rc != TPS_OK) return rc;
    if (tokens < 0 || tokens > INT32_MAX || !cu_seqlens || (tokens > 0 && (!slots || !positions))) return TPS_ERR_ARG;
    if (!aligned(slots, 8) || !aligned(positions, 4) || !aligned(cu_seqlens, 4)) return TPS_ERR_ALIGN;
    a.tokens = tokens, a.slots = slots, a.positions = positions, a.cu_seqlens = cu_seqlens;
    const cudaError_t e = tps::launch_kv_extend(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TPS_OK : tps::report_cuda(e);
}

int tps_kv_trim(const tps_kv_pages* pages, void* stream)
{
    tps::PagesArgs a = {};
    const int rc = check_pages(pages, &a);
    if (rc != TPS_OK) return rc;
    if (pages->B == 0) return TPS_OK;
    const cudaError_t e = tps::launch_kv_trim(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TPS_OK : tps::report_cuda(e);
}

int tps_prompt_attention(const tps_prompt* args, void* stream)
{
    return tps_prompt_attention_stall_test(args, -1, tps::kAttnWaitNs, stream);
}

int tps_prompt_attention_stall_test(const tps_prompt* args, int stall_head, uint64_t wait_ns, void* stream)
{
    if (wait_ns < 1 || wait_ns > tps::kAttnWaitNs) return TPS_ERR_ARG;
    tps::PromptArgs a = {};
    int64_t tiles = 0;
    const int rc = check_prompt(args, &a, &tiles);
    if (rc != TPS_OK) return rc;
    if (args->B == 0 || (args->T == 0 && !args->out_status)) return TPS_OK;
    int sms = 0;
    if (!tps::host_sms(&sms)) return tps::report_cuda(cudaGetLastError());
    a.stall_head = stall_head;
    a.wait_ns = wait_ns;
    const cudaError_t e = tps::launch_attn_prompt(a, *args, tiles, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TPS_OK : tps::report_cuda(e);
}

}  // extern "C"
