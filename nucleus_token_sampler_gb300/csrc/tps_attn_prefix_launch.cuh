// tps_attn_prefix_launch.cuh -- launch of the tcgen05 prefix and tree kernels for one cache format (each
// format of either is a translation unit of its own).
#pragma once

#include <atomic>

#include "tps_attn_prefix.cuh"

namespace tps {

// The driver's encoder of tensor maps, looked up once.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// A bfloat16 cache tensor [pages, heads, page_size, D], read 64 columns by up to 128 rows at a time.
inline cudaError_t encode_cache(CUtensorMap* map, const tps_kv_cache& c, void* base)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.n_heads, (cuuint64_t)c.n_pages};
    const cuuint64_t row = (cuuint64_t)c.head_dim * 2;
    const cuuint64_t strides[3] = {row, row * c.page_size, row * c.page_size * c.n_heads};
    const cuuint32_t box[4] = {64, (cuuint32_t)(c.page_size < kBlockKeys ? c.page_size : kBlockKeys), 1, 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int kFormat, int kTiles, int kLine>
cudaError_t launch_prefix_shape(const typename LineOf<kLine>::Args& a, cudaStream_t stream)
{
    using Shape = PrefixShape<D, kFormat, kTiles, kLine>;
    auto k = attn_prefix_kernel<D, kFormat, kTiles, kLine>;
    static std::atomic<uint64_t> allowed{0};  // devices on which the shared memory has been asked for
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(allowed.load(std::memory_order_acquire) & bit)) {
        // The warps that ask for more registers wait for those that the others give back: the sum has to be there.
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, k);
        if (e != cudaSuccess) return e;
        if (Shape::kSplitRegs && fa.numRegs < Shape::kRegsLaunch) return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape::kSmem);
        if (e != cudaSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_release);
    }
    CUtensorMap km = {}, vm = {};
    if (kFormat == TPS_KV_BF16) {
        e = encode_cache(&km, a.c, a.c.k);
        if (e == cudaSuccess) e = encode_cache(&vm, a.c, a.c.v);
        if (e != cudaSuccess) return e;
    }
    k<<<(unsigned)a.p.ctas, Shape::kThreads, Shape::kSmem, stream>>>(a, km, vm);
    return cudaGetLastError();
}

template <int kFormat>
cudaError_t launch_prefix_format(const AttnArgs& a, cudaStream_t stream)
{
    const bool two = a.p.tile_rows == 256;
    if (a.c.head_dim == 64)
        return two ? launch_prefix_shape<64, kFormat, 2, kShared>(a, stream) : launch_prefix_shape<64, kFormat, 1, kShared>(a, stream);
    return two ? launch_prefix_shape<128, kFormat, 2, kShared>(a, stream) : launch_prefix_shape<128, kFormat, 1, kShared>(a, stream);
}

template <int kFormat>
cudaError_t launch_tree_format(const TreeArgs& a, cudaStream_t stream)
{
    const bool two = a.p.tile_rows == 256;
    if (a.c.head_dim == 64)
        return two ? launch_prefix_shape<64, kFormat, 2, kTrees>(a, stream) : launch_prefix_shape<64, kFormat, 2, kTreesInTurn>(a, stream);
    return two ? launch_prefix_shape<128, kFormat, 2, kTrees>(a, stream) : launch_prefix_shape<128, kFormat, 2, kTreesInTurn>(a, stream);
}

}  // namespace tps
