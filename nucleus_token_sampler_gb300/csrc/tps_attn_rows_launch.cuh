// tps_attn_rows_launch.cuh -- launches of the 8- and 16-row attention kernels: a prefix call's own tokens, and trees of few rows.
#pragma once

#include <algorithm>
#include <atomic>

#include "tps_attn_rows.cuh"

namespace tps {

// More than 48 KB of dynamic shared memory has to be asked for, once per kernel and device.
template <typename Kernel>
cudaError_t allow_smem(Kernel k, size_t bytes, std::atomic<uint64_t>& allowed)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (allowed.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) allowed.fetch_or(bit, std::memory_order_release);
    return e;
}

static __global__ void clear_status_kernel(const AttnArgs a)
{
    clear_status(a);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int D, int kFormat, int N, bool kOneWarp, bool kTree>
cudaError_t suffix_shape(const AttnArgs& a, bool after_prefix, cudaStream_t stream)
{
    static std::atomic<uint64_t> allowed{0};
    auto k = attn_suffix_kernel<D, kFormat, N, kOneWarp, kTree>;
    const size_t smem = (sizeof(RowsShared<D, kFormat>) + 15) / 16 * 16 + (kOneWarp ? 0 : sizeof(JoinShared<8 * N>));
    const cudaError_t e = allow_smem(k, smem, allowed);
    if (e != cudaSuccess) return e;
    const int64_t items = a.a.B * a.c.n_heads * a.p.suffix_tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(kOneWarp ? (items + kRowsWarps - 1) / kRowsWarps : items * a.p.cluster), 1, 1);
    cfg.blockDim = dim3(kRowsThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (a.p.cluster > 1) {  // 1 wherever kOneWarp
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)a.p.cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (after_prefix) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <int D, int kFormat, bool kTree>
cudaError_t suffix(const AttnArgs& a, bool after_prefix, cudaStream_t stream)
{
    if (a.p.suffix_rows == 8)
        return a.p.one_warp ? suffix_shape<D, kFormat, 1, true, kTree>(a, after_prefix, stream)
                            : suffix_shape<D, kFormat, 1, false, kTree>(a, after_prefix, stream);
    return a.p.one_warp ? suffix_shape<D, kFormat, 2, true, kTree>(a, after_prefix, stream)
                        : suffix_shape<D, kFormat, 2, false, kTree>(a, after_prefix, stream);
}

inline cudaLaunchAttribute dependent()
{
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    return at;
}

template <int D, int kFormat, int N, bool kTree>
cudaError_t line_shape(const AttnArgs& a, bool after_prefix, cudaStream_t stream)
{
    static std::atomic<uint64_t> allowed{0};
    auto k = attn_line_kernel<D, kFormat, N, kTree>;
    const size_t smem = (sizeof(RowsShared<D, kFormat>) + 15) / 16 * 16 + sizeof(LineSums);
    cudaError_t e = allow_smem(k, smem, allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at = dependent();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.p.line_ctas, 1, 1);
    cfg.blockDim = dim3(kRowsThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = after_prefix ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, k, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(a.a.B * a.p.suffix_tiles * a.c.n_heads), D / kStrip, 1);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D, kFormat, kTree>, a);
}

template <int D, int kFormat, bool kTree>
cudaError_t line(const AttnArgs& a, bool after_prefix, cudaStream_t stream)
{
    return a.p.suffix_rows == 8 ? line_shape<D, kFormat, 1, kTree>(a, after_prefix, stream) : line_shape<D, kFormat, 2, kTree>(a, after_prefix, stream);
}

template <int D, int kFormat, bool kTree>
cudaError_t own(const AttnArgs& a, bool after_prefix, cudaStream_t stream)
{
    if (a.p.line) return line<D, kFormat, kTree>(a, after_prefix, stream);
    if (!after_prefix && a.a.out_status) {
        clear_status_kernel<<<(unsigned)std::min<int64_t>((a.a.B + 255) / 256, 1024), 256, 0, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        after_prefix = true;
    }
    return suffix<D, kFormat, kTree>(a, after_prefix, stream);
}

}  // namespace tps
