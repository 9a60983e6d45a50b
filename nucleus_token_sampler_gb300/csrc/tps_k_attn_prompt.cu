// The prompt attention kernels and their launch.
#include <algorithm>
#include <atomic>

#include "tps_attn_prefix_launch.cuh"
#include "tps_attn_prompt.cuh"

namespace tps {

namespace {

// A [T, heads, D] bfloat16 tensor, read 64 columns of `box_heads` heads of `box_tokens` tokens at a time.
cudaError_t encode_heads(CUtensorMap* map, const void* base, int64_t T, int heads, int D, int64_t ld, int64_t hd, int box_heads,
                         int box_tokens)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
    // the stride of an axis of one element counts for nothing
    const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? hd : D) * 2, (cuuint64_t)(T > 1 ? ld : (int64_t)heads * D) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens}, step[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch(const PromptArgs& a, const tps_prompt& p, unsigned ctas, cudaStream_t stream)
{
    using Shape = PromptShape<D>;
    auto k = attn_prompt_kernel<D>;
    static std::atomic<uint64_t> allowed{0};  // devices on which the shared memory has been asked for
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(allowed.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape::kSmem);
        if (e != cudaSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_release);
    }
    CUtensorMap qm, km, vm;
    e = encode_heads(&qm, p.q, p.T, p.n_q_heads, D, p.q_ld, p.q_hd, a.group, a.tile_tokens);
    if (e == cudaSuccess) e = encode_heads(&km, p.k, p.T, p.n_k_heads, D, p.k_ld, p.k_hd, 1, kBlockKeys);
    if (e == cudaSuccess) e = encode_heads(&vm, p.v, p.T, p.n_k_heads, D, p.v_ld, p.v_hd, 1, kBlockKeys);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(kPromptThreads, 1, 1);
    cfg.dynamicSmemBytes = Shape::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = a.list ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, a, qm, km, vm);
}

}  // namespace

cudaError_t launch_attn_prompt(const PromptArgs& args, const tps_prompt& p, int64_t tiles, int sms, cudaStream_t stream)
{
    PromptArgs a = args;
    const int64_t items = tiles * a.heads_v;
    // Every tile on an SM of its own: nothing to sort.  Statuses are the planning kernel's.
    if (items <= sms && !a.out_status && p.T > 0)
        return p.head_dim == 64 ? launch<64>(a, p, (unsigned)items, stream) : launch<128>(a, p, (unsigned)items, stream);
    void* mem = nullptr;
    cudaError_t e = pool_alloc(&mem, 16 * (size_t)(tiles + 1), stream);
    if (e != cudaSuccess) return e;
    int* n_tiles = static_cast<int*>(mem);
    int4* list = static_cast<int4*>(mem) + 1;
    constexpr int kPlanThreads = 1024;
    prompt_plan_kernel<kPlanThreads><<<1, kPlanThreads, 0, stream>>>(a, list, n_tiles);
    e = cudaGetLastError();
    a.list = list;
    a.n_tiles = n_tiles;
    if (e == cudaSuccess && p.T > 0) {
        const unsigned ctas = (unsigned)std::min<int64_t>(items, sms);
        e = p.head_dim == 64 ? launch<64>(a, p, ctas, stream) : launch<128>(a, p, ctas, stream);
    }
    const cudaError_t ef = cudaFreeAsync(mem, stream);
    return e == cudaSuccess ? ef : e;
}

}  // namespace tps
