// The per-head norm and rotation on float32 and bfloat16, and its launch (its own translation unit).
#include "tps_norm_rope.cuh"

#include <algorithm>

namespace tps {

namespace {

constexpr int kNormResident = 1024;  // threads of an SM that the launch fills

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

void launch_kernel(void (*kernel)(tps_norm_rope), const tps_norm_rope& a, unsigned grid, int threads, cudaStream_t stream)
{
    kernel<<<grid, threads, 0, stream>>>(a);
}

template <typename T, int L, int kWalks>
cudaError_t launch_walks(const tps_norm_rope& a, unsigned grid, int threads, cudaStream_t stream)
{
    const bool whole = a.rot_dim == a.head_dim;
    if (a.interleaved)
        whole ? launch_kernel(norm_rope_kernel<T, L, true, true, kWalks>, a, grid, threads, stream)
              : launch_kernel(norm_rope_kernel<T, L, true, false, kWalks>, a, grid, threads, stream);
    else
        whole ? launch_kernel(norm_rope_kernel<T, L, false, true, kWalks>, a, grid, threads, stream)
              : launch_kernel(norm_rope_kernel<T, L, false, false, kWalks>, a, grid, threads, stream);
    return cudaGetLastError();
}

template <typename T, int L>
cudaError_t launch_units(const tps_norm_rope& a, int sms, cudaStream_t stream)
{
    // Few tokens: a CTA for each, all of its heads at once as far as 256 threads reach.  Many: two heads for
    // each group of lanes, and no more CTAs than are resident, each walking over its tokens.  One / two heads, 40
    // heads of 128 in bfloat16 (other shapes were not swept), us: 608 tokens 3.5 / 5.1, 1,216 6.5 / 7.0, 2,700 15.7 / 14.6, 16,383 78.5 / 67.2.
    const int H = a.n_q_heads + a.n_k_heads;
    const bool two = a.T > 12 * sms && H > 1;
    const int want = two ? (H + 1) / 2 : H;                                  // groups
    const int most = kNormMaxThreads / L, walks = (want + most - 1) / most;  // rounds over the heads
    const int threads = std::min(kNormMaxThreads, ((want + walks - 1) / walks * L + 31) / 32 * 32);
    const unsigned grid = (unsigned)std::min<int64_t>(a.T, (int64_t)sms * (kNormResident / threads));
    return two ? launch_walks<T, L, 2>(a, grid, threads, stream) : launch_walks<T, L, 1>(a, grid, threads, stream);
}

template <typename T>
cudaError_t launch_type(const tps_norm_rope& a, int sms, cudaStream_t stream)
{
    constexpr int N = Pack<T>::kN;
    const int H = a.n_q_heads + a.n_k_heads, units = a.head_dim / (2 * N);
    const int64_t strides = (a.n_q_heads ? a.q_ld | a.q_hd | a.oq_ld | a.oq_hd : 0) |
                            (a.n_k_heads ? a.k_ld | a.k_hd | a.ok_ld | a.ok_hd : 0);
    const bool whole = a.head_dim % (2 * N) == 0 && a.rot_dim % (2 * N) == 0 && units <= 32 && strides % N == 0 &&
                       (!a.n_q_heads || (on16(a.q) && on16(a.out_q))) && (!a.n_k_heads || (on16(a.k) && on16(a.out_k))) &&
                       on16(a.q_weight) && on16(a.k_weight) && on16(a.cos_sin);
    if (!whole) {
        const int threads = 32 * std::min(H, kNormMaxThreads / 32);
        norm_rope_any_kernel<T><<<(unsigned)a.T, threads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    int L = 1;
    while (L < units) L *= 2;
    switch (L) {
    case 1: return launch_units<T, 1>(a, sms, stream);
    case 2: return launch_units<T, 2>(a, sms, stream);
    case 4: return launch_units<T, 4>(a, sms, stream);
    case 8: return launch_units<T, 8>(a, sms, stream);
    case 16: return launch_units<T, 16>(a, sms, stream);
    default: return launch_units<T, 32>(a, sms, stream);
    }
}

}  // namespace

cudaError_t launch_norm_rope(const tps_norm_rope& a, int sms, cudaStream_t stream)
{
    return a.dtype == TPS_BF16 ? launch_type<__nv_bfloat16>(a, sms, stream) : launch_type<float>(a, sms, stream);
}

}  // namespace tps
