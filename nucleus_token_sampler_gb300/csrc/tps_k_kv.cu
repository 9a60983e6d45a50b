// The cache write and read kernels for each input type and format, and their launches.
#include <cuda_fp16.h>

#include "tps_kv.cuh"

#include <algorithm>

namespace tps {

namespace {

int log2_of(int n)
{
    int s = 0;
    while ((1 << s) < n) ++s;
    return s;
}

// Lanes of a vector (a power of two holding head_dim / 16) and CTAs for n vectors.
int lanes_of(const tps_kv_cache& c) { return 1 << log2_of(c.head_dim / 16); }
unsigned grid_of(int64_t n, int L, int flight, int sms)
{
    const int64_t per = kKvThreads / L, one = (n + per - 1) / per;
    // A call too small for two CTAs on every SM takes one vector for each group of lanes, so that they spread
    // over more SMs.  One / four on the way, a write and a read of 8 key heads of 128, fp8, us: 64 tokens 4.9 / 6.1, 600
    // 6.2 / 6.8, 1,200 9.4 / 7.6, 5,000 28.4 / 19.1.
    return (unsigned)std::min<int64_t>(one <= 2 * (int64_t)sms ? one : (one + flight - 1) / flight, (int64_t)sms * 16);
}

template <typename T, bool kWide>
void write_format(const KvWriteArgs& a, unsigned grid, int L, int shift, cudaStream_t stream)
{
    switch (a.c.format) {
    case TPS_KV_BF16: kv_write_kernel<T, TPS_KV_BF16, kWide><<<grid, kKvThreads, 0, stream>>>(a, L, shift); break;
    case TPS_KV_FP8: kv_write_kernel<T, TPS_KV_FP8, kWide><<<grid, kKvThreads, 0, stream>>>(a, L, shift); break;
    default: kv_write_kernel<T, TPS_KV_INT8, kWide><<<grid, kKvThreads, 0, stream>>>(a, L, shift); break;
    }
}

template <typename T>
cudaError_t write_type(const KvWriteArgs& a, int sms, cudaStream_t stream)
{
    const int L = lanes_of(a.c), shift = log2_of(a.c.page_size), es = sizeof(T);
    const unsigned grid = grid_of(a.T * 2 * a.c.n_heads, L, sizeof(T) == 2 ? kKvFlight : kKvFlight / 2, sms);
    const bool wide = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) | (uintptr_t)(a.k_ld * es) |
                        (uintptr_t)(a.k_hd * es) | (uintptr_t)(a.v_ld * es) | (uintptr_t)(a.v_hd * es)) & 15) == 0;
    if (wide)
        write_format<T, true>(a, grid, L, shift, stream);
    else
        write_format<T, false>(a, grid, L, shift, stream);
    return cudaGetLastError();
}

template <typename T>
cudaError_t read_type(const KvReadArgs& a, int sms, cudaStream_t stream)
{
    const int L = lanes_of(a.c), shift = log2_of(a.c.page_size);
    const unsigned grid = grid_of(a.T * 2 * a.c.n_heads, L, kKvFlight, sms);
    switch (a.c.format) {
    case TPS_KV_BF16: kv_read_kernel<T, TPS_KV_BF16><<<grid, kKvThreads, 0, stream>>>(a, L, shift); break;
    case TPS_KV_FP8: kv_read_kernel<T, TPS_KV_FP8><<<grid, kKvThreads, 0, stream>>>(a, L, shift); break;
    default: kv_read_kernel<T, TPS_KV_INT8><<<grid, kKvThreads, 0, stream>>>(a, L, shift); break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteArgs& a, bool bf16, int sms, cudaStream_t stream)
{
    return bf16 ? write_type<__nv_bfloat16>(a, sms, stream) : write_type<float>(a, sms, stream);
}

cudaError_t launch_kv_read(const KvReadArgs& a, bool bf16, int sms, cudaStream_t stream)
{
    return bf16 ? read_type<__nv_bfloat16>(a, sms, stream) : read_type<float>(a, sms, stream);
}

}  // namespace tps
