// The page kernels and their launches.
#include "tps_pages.cuh"

namespace tps {

namespace {

// New tokens from which a kernel of many CTAs writes the slots.
constexpr int64_t kPagesAlone = 16384;

}  // namespace

cudaError_t launch_kv_extend(const PagesArgs& args, cudaStream_t stream)
{
    PagesArgs a = args;
    if (a.tokens < kPagesAlone) {
        kv_extend_kernel<true><<<1, kPagesThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    void* mem = nullptr;
    cudaError_t e = pool_alloc(&mem, sizeof(int32_t) * (size_t)(a.p.B > 0 ? a.p.B : 1), stream);
    if (e != cudaSuccess) return e;
    a.first = static_cast<int32_t*>(mem);
    a.wide = reinterpret_cast<uintptr_t>(a.slots) % 16 == 0 && reinterpret_cast<uintptr_t>(a.positions) % 16 == 0;
    kv_extend_kernel<false><<<1, kPagesThreads, 0, stream>>>(a);
    e = cudaGetLastError();
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
    kv_trim_kernel<<<1, kPagesThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace tps
