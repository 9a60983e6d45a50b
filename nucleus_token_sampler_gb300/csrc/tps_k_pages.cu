// The page kernels and their launches.
#include "tps_pages.cuh"

namespace tps {

namespace {

// New tokens from which a second kernel over all SMs writes the slots.  One kernel / two, us, with the trim that follows: 64
// sequences of 1 token 9.5 / 10.8, of 16 10.4 / 10.3, of 64 11.1 / 10.0, of 1,024 56 / 10.5; 1,000 of 1 12.3 / 13.3, of 4 13.7 / 12.4, of 16
// 25.1 / 12.9.  (A cluster of eight CTAs in one kernel: 14.1 for the last, 14.9 for 64 of 1,024.)
constexpr int64_t kSlotsAlone = 2048;
// Places in all tables from which a trim is shared by a cluster.  One CTA / eight: 300 sequences of up to 94 of 128 pages 15 / 7.6
// us under a profiler; 1,000 of 4 of 17 pages 0.6 us less / more in a pair of calls of 71.
constexpr int64_t kTrimShared = 32768;
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
        return launch(kv_extend_kernel<true>, a, 1, stream);
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
    return launch(kv_trim_kernel, a, a.p.B <= kPagesThreads && a.p.B * a.p.table_width >= kTrimShared ? kPagesCluster : 1, stream);
}

}  // namespace tps
