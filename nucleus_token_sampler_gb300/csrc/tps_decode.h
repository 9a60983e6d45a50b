// tps_decode.h -- what the decode-step entry points (tps_api_decode.cu) and their kernels share: the
// launch functions, each defined in its kernel's translation unit, and the host services of
// tps_api.cu (device limits, the scratch pool, the last CUDA error).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/tps.h"

namespace tps {

// Defined in tps_api.cu.
bool host_sms(int* sms);                                                   // SMs of the current device
cudaError_t pool_alloc(void** p, size_t bytes, cudaStream_t stream);       // from the library's pool
int report_cuda(cudaError_t e);                                            // keeps e, returns TPS_ERR_CUDA

cudaError_t launch_norm_rope(const tps_norm_rope& a, int sms, cudaStream_t stream);

struct KvWriteArgs {
    tps_kv_cache c;
    const void* k;
    const void* v;
    int64_t T, k_ld, k_hd, v_ld, v_hd;
    const int64_t* slots;
};
cudaError_t launch_kv_write(const KvWriteArgs& a, bool bf16, int sms, cudaStream_t stream);

struct KvReadArgs {
    tps_kv_cache c;
    const int64_t* slots;
    int64_t T;
    void* k;
    void* v;
};
cudaError_t launch_kv_read(const KvReadArgs& a, bool bf16, int sms, cudaStream_t stream);

// The work of one prefix-attention call.  The shared part is cut along items and tokens: an item is one
// key head and `tile_rows` of its R = B Tq G query rows; its prefix is nblk blocks of `block_keys`
// tokens.  The items' blocks form one line of `units` blocks, of which CTA c of `ctas` takes
// [c units / ctas, (c + 1) units / ctas): every CTA gets the same number of blocks (give or take one)
// whatever the number of items.  A CTA's part of an item leaves one piece in the workspace, the
// unnormalised output of its rows with their maximum and sum; piece c + item is CTA c's of that item
// (going along the line either number grows, so no two share one).
struct AttnPlan {
    int64_t R;           // query rows of one key head
    int64_t items, nblk, units, ctas, pieces;
    int tile_rows, block_keys;
    int n_tiles;         // row tiles of one key head
    bool tensor;         // the tcgen05 kernel computes the shared part
    int suffix_tiles;    // 16-row tiles of one sequence's Tq G rows
    bool one_warp;       // each warp has a sequence (and head, tile) for itself
    int cluster;         // else: CTAs that share one sequence's own tokens
    size_t off_ml, bytes;  // workspace: outputs first, then (maximum, sum)
};

struct AttnArgs {
    tps_kv_cache c;
    tps_attention a;
    AttnPlan p;
    int G, page_shift;
    float qk_scale;  // scale * log2(e)
    float* part;     // [pieces][D / 4][tile_rows][4]: a warp's rows lie side by side
    float2* ml;      // [pieces, tile_rows]: maximum in base-2 units, sum (negative: a bad page id)
};

// The shared part, then the own tokens and the join.
cudaError_t launch_attn_prefix_rows(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_prefix_bf16(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_prefix_fp8(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_prefix_int8(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_suffix(const AttnArgs& a, bool after_prefix, cudaStream_t stream);

}  // namespace tps
