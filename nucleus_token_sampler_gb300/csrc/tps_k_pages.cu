// The page kernels and their launches.
#include "tps_pages.cuh"

namespace tps {

namespace {

// New tokens from which a second kernel over all SMs writes the slots; and from which, and sequences from which, a cluster shares
// the work of one CTA.
constexpr int64_t kSlotsAlone = 65536, kTokensShared = 4096, kSequencesShared = 64;
constexpr int kPagesCluster = 8;

template <typename Kernel> cudaError_t launch(Kernel k, const PagesArgs& a, int ctas, cudaStream_t stream)
{
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ctas;
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(kPagesThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace

cudaError_t launch_kv_extend(const PagesArgs& args, cudaStream_t stream)
{
    PagesArgs a = args;
    if (a.tokens < kSlotsAlone)
        return launch(kv_extend_kernel<true>, a, a.tokens >= kTokensShared && a.p.B <= kPagesThreads ? kPagesCluster : 1, stream);
    void* mem = nullptr;
    cudaError_t e = pool_alloc(&mem, sizeof(int2) * (size_t)(a.p.B + 1), stream);
    if (e != cudaSuccess) return e;
    a.first = static_cast<int2*>(mem);
    a.wide = reinterpret_cast<uintptr_t>(a.slots) % 16 == 0 && reinterpret_cast<uintptr_t>(a.positions) % 16 == 0;
    e = launch(kv_extend_kernel<false>, a, 1, stream);
    if (e == cudaSuccess) {
        cudaLaunchAttribute at = {};
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((a.tokens + kSlotsThreads * kSlotsEach - 1) / (kSlotsThreads * kSlotsEach)), 1, 1);
        cfg.blockDim = dim3(kSlotsThreads, 1, 1);
        cfg.stream = stream;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, kv_slots_kernel, a);
    }
    const cudaError_t ef = cudaFreeAsync(mem, stream);
    return e == cudaSuccess ? ef : e;
}

cudaError_t launch_kv_trim(const PagesArgs& a, cudaStream_t stream)
{
    return launch(kv_trim_kernel, a, a.p.B >= kSequencesShared && a.p.B <= kPagesThreads ? kPagesCluster : 1, stream);
}

}  // namespace tps
