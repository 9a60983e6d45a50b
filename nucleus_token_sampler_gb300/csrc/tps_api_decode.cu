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
    tps::AttnArgs a;
    rc = plan_attention(*cache, *args, sms, &a.p);
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
    if (a.p.bytes) {
        if (ws) {
            if (args->workspace_bytes < (int64_t)a.p.bytes) return TPS_ERR_SCRATCH;
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
        e = cache->format == TPS_KV_BF16  ? tps::launch_attn_prefix_bf16(a, st)
            : cache->format == TPS_KV_FP8 ? tps::launch_attn_prefix_fp8(a, st)
                                          : tps::launch_attn_prefix_int8(a, st);
    }
    if (e == cudaSuccess) e = tps::launch_attn_own(a, a.p.units > 0, st);
    if (a.p.bytes && !args->workspace) {
        const cudaError_t ef = cudaFreeAsync(ws, st);
        if (e == cudaSuccess) e = ef;
    }
    return e == cudaSuccess ? TPS_OK : tps::report_cuda(e);
}

}  // extern "C"
