// The join of the tree kernel's pieces, the sequences' statuses, and their launch.
#include "tps_attn_tree.cuh"

namespace tps {

namespace {

constexpr int kJoinThreads = 256;

// Blocks (c, y) with c below a.p.ctas: rows kTreeJoinRows y and up of the item that CTA c began and did not finish, from its piece and the
// first pieces of the CTAs after it; a lane for each row, a warp for each 4 columns in turn.  The blocks after them
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
    int last = cta + 1;
    while (last + 1 < ctas && !a.rec[last].ended) ++last;
    const int tile = mine.open_item % a.p.n_tiles, head = mine.open_item / a.p.n_tiles;
    const int row = (int)blockIdx.y * kTreeJoinRows + lane, in_item = tile * rows + row;
    if (in_item - lane >= a.p.R) return;
    const bool in = in_item < a.p.R;
    const float neg = -__int_as_float(0x7F800000);
    const float2* ml = a.ml + row;
    auto piece = [&](int c) { return c == cta ? 2 * (int64_t)c + 1 : 2 * (int64_t)c; };
    float top = neg, sum = 0.f;
    bool bad = false;
    if (in) {
#pragma unroll 4
        for (int c = cta; c <= last; ++c) {
            const float2 x = ml[piece(c) * rows];
            bad |= x.y < 0.f;
            if (x.y != 0.f) top = fmaxf(top, x.x);
        }
#pragma unroll 4
        for (int c = cta; c <= last; ++c) {
            const float2 x = ml[piece(c) * rows];
            if (x.y != 0.f) sum += x.y * (x.x == top ? 1.f : exp2_fast(x.x - top));
        }
    }
    const float inv = bad ? __int_as_float(0x7FC00000) : 1.f / sum;
    const int64_t at = tree_row_at(a, mine.open_seq, head, in ? in_item : 0);
    if (!in) return;
    for (int d = warp; d < D / 4; d += kJoinThreads / 32) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int c = cta; c <= last; ++c) {
            const float2 x = ml[piece(c) * rows];
            const float4 y = *(reinterpret_cast<const float4*>(a.part + piece(c) * rows * D) + d * rows + row);
            if (x.y == 0.f) continue;
            const float f = x.x == top ? 1.f : exp2_fast(x.x - top);
            o.x += y.x * f, o.y += y.y * f, o.z += y.z * f, o.w += y.w * f;
        }
        if (sum == 0.f && !bad)
            o = make_float4(0.f, 0.f, 0.f, 0.f);
        else
            o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
        reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.a.out) + at * D)[d] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    if (warp == 0 && a.a.out_lse) a.a.out_lse[at] = log_sum<kFormat>(top, sum, bad);
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
