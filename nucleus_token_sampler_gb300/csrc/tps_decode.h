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
// key head and `tile_rows` of its R = B Tq G query rows; its prefix is nblk blocks of kBlockKeys
// tokens.  The items' blocks form one line of `units` blocks, of which each CTA takes `share` consecutive ones
// (the last CTA what is left).  A CTA's part of an item leaves one piece in the workspace, the
// unnormalised output of its rows with their maximum and sum; piece c + item is CTA c's of that item
// (going along the line either number grows, so no two share one).
constexpr int kBlockKeys = 128;
struct AttnPlan {
    int64_t R;           // query rows of one key head
    int items, nblk, units, share, ctas;
    int64_t pieces;
    int tile_rows;
    int n_tiles;         // row tiles of one key head
    bool shared;         // the prefix is computed once, into pieces (else by each sequence for itself)
    int suffix_rows;     // rows of a tile of one sequence's Tq G rows: 8 or 16
    int suffix_tiles;
    bool one_warp;       // each warp has a sequence (and head, tile) for itself
    int cluster;         // else: CTAs that share one sequence's own tokens
    bool line;           // or: the own tokens are cut evenly over `line_ctas` CTAs, which leave pieces too
    int64_t line_ctas, line_pieces;
    // workspace: outputs of the prefix's pieces, their (maximum, sum); the same of the line's
    size_t off_ml, off_line_part, off_line_ml, bytes;
};

struct AttnArgs {
    tps_kv_cache c;
    tps_attention a;
    AttnPlan p;
    int G, page_shift;
    float qk_scale;  // scale * log2(e)
    float* part;     // [pieces][D / 4][tile_rows][4]: a warp's rows lie side by side
    float2* ml;      // [pieces, tile_rows]: maximum in base-2 units, sum (negative: a bad page id)
    float* line_part;
    float2* line_ml;
    int stall_head;    // of tps_prefix_attention_stall_test, else -1
    uint64_t wait_ns;  // limit of every wait for data or for another role (copies in flight: kAttnWaitNs)
};
constexpr uint64_t kAttnWaitNs = 1000000000ull;

// The shared part, then the own tokens and the join.
cudaError_t launch_attn_prefix_bf16(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_prefix_fp8(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_prefix_int8(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attn_own(const AttnArgs& a, bool after_prefix, cudaStream_t stream);

}  // namespace tps
