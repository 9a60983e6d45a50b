// The join of the tree kernel's pieces, the sequences' statuses, and their launch.
#include "tps_attn_tree.cuh"

namespace tps {

namespace {

constexpr int kJoinThreads = 256;

// Blocks (c, y) with c below a.p.ctas: rows kTreeJoinRows y and up of the item that CTA c began and did not finish, from its piece and the
// first pieces of the CTAs after it; a lane for each row, an eighth of the columns for each warp.  The blocks after them
// tell the statuses, a warp for each sequence.
template <int D, int kFormat> __global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5, ctas = a.p.ctas, rows = a.p.tile_rows;
    if ((int)blockIdx.x >= ctas) {
        const int64_t seq = ((int64_t)(blockIdx.x - ctas) * gridDim.y + blockIdx.y) * (kJoinThreads / 32) + warp;
        if (seq >= a.a.B) return;
        const int len = a.a.seq_len[seq], nodes = a.a.tree_len ? a.a.tree_len[seq] : a.a.n_nodes;
        bool bad = TreeWay::tree_bad(a, len, nodes), late = false;
        for (int64_t i = lane; !bad && i << a.page_shift < len; i += 32) {
            const int id = a.a.page_table[seq * a.a.table_ld + i];
            if (id < 0 || id >= a.c.n_pages) bad = true;
        }
        for (int c = lane; c < ctas; c += 32) late |= a.rec[c].timeout && a.rec[c].first_seq <= seq && seq <= a.rec[c].last_seq;
        bad = __any_sync(0xFFFFFFFFu, bad), late = __any_sync(0xFFFFFFFFu, late);
        if (lane == 0) a.a.out_status[seq] = late ? TPS_ROW_TIMEOUT : (bad ? TPS_ROW_BAD_PARAM : TPS_ROW_OK);
        return;
    }
    const int cta = (int)blockIdx.x;
    const TreeRecord mine = a.rec[cta];
    if (mine.open_seq < 0) return;
    int last = cta;
    for (uint32_t ends = 0; !ends;) {  // 32 CTAs at a time
        const int c = last + 1 + lane;
        ends = __ballot_sync(0xFFFFFFFFu, c >= ctas - 1 || a.rec[c].ended);
        last += ends ? __ffs(ends) : 32;
    }
    const int n = last - cta + 1, tile = mine.open_item % a.p.n_tiles, head = mine.open_item / a.p.n_tiles;
    const int row = (int)blockIdx.y * kTreeJoinRows + lane, in_item = tile * rows + row;
    if (in_item - lane >= a.p.R) return;
    const bool in = in_item < a.p.R;
    auto piece = [&](int i) { return 2 * (int64_t)(cta + i) + (i == 0); };
    // Maxima and sums of every piece, then its factor.
    extern __shared__ float2 factor[];  // [n][32]: maximum, sum; then .x is the factor
    for (int i = warp; i < n; i += kJoinThreads / 32) factor[i * 32 + lane] = in ? a.ml[piece(i) * rows + row] : make_float2(0.f, 0.f);
    __syncthreads();
    float top = -__int_as_float(0x7F800000), sum = 0.f;
    bool bad = false;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float2 x = factor[i * 32 + lane];
        bad |= x.y < 0.f;
        if (x.y != 0.f) top = fmaxf(top, x.x);
    }
    auto weight = [&](float2 x) { return x.y == 0.f ? 0.f : (x.x == top ? 1.f : exp2_fast(x.x - top)); };
#pragma unroll 4
    for (int i = 0; i < n; ++i) sum += factor[i * 32 + lane].y * weight(factor[i * 32 + lane]);
    __syncthreads();
    for (int i = warp; i < n; i += kJoinThreads / 32) factor[i * 32 + lane].x = weight(factor[i * 32 + lane]);
    __syncthreads();
    if (!in) return;
    constexpr int kEach = D / 4 / (kJoinThreads / 32);  // columns of four of a warp
    const float4* part = reinterpret_cast<const float4*>(a.part) + row;
    float4 o[kEach] = {};
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float f = factor[i * 32 + lane].x;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const float4 y = part[(piece(i) * (D / 4) + warp * kEach + k) * rows];
            if (f != 0.f) o[k].x += y.x * f, o[k].y += y.y * f, o[k].z += y.z * f, o[k].w += y.w * f;
        }
    }
    const float inv = bad ? __int_as_float(0x7FC00000) : (sum == 0.f ? 0.f : 1.f / sum);
    const int64_t at = tree_row_at(a, mine.open_seq, head, in_item);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o[k].x * inv, o[k].y * inv), hi = __floats2bfloat162_rn(o[k].z * inv, o[k].w * inv);
        reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.a.out) + at * D)[warp * kEach + k] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    if (warp == 0 && a.a.out_lse) {
        float lost = 0.f;
        for (int i = 0; i < n; ++i) {
            const float f = factor[i * 32 + lane].x;
            if (f != 0.f) lost += f * a.lost[piece(i) * rows + row];
        }
        a.a.out_lse[at] = log_sum<kFormat>(top, sum + lost, bad);
    }
}

template <int D, int kFormat> cudaError_t join(const TreeArgs& a, cudaStream_t stream)
{
    const int64_t chunks = (a.p.tile_rows < a.p.R ? a.p.tile_rows : a.p.R) + kTreeJoinRows - 1;
    const unsigned y = (unsigned)(chunks / kTreeJoinRows);
    const int64_t each = (int64_t)y * (kJoinThreads / 32), status = a.a.out_status ? (a.a.B + each - 1) / each : 0;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.p.ctas + status), y, 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)a.p.ctas * 32 * sizeof(float2);
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<D, kFormat>, a);
}

}  // namespace

cudaError_t launch_tree_join(const TreeArgs& a, cudaStream_t stream)
{
    if (a.c.head_dim == 64) return a.c.format == TPS_KV_BF16 ? join<64, TPS_KV_BF16>(a, stream) : join<64, TPS_KV_FP8>(a, stream);
    return a.c.format == TPS_KV_BF16 ? join<128, TPS_KV_BF16>(a, stream) : join<128, TPS_KV_FP8>(a, stream);  // 8-bit formats lift alike
}

}  // namespace tps
