// tps_pages.cuh -- the pages that sequences get from a list of free ones as they grow and give back as they shrink,
// and the cache slots of their new tokens.
//
// Formulas.  With p tokens to a page, a sequence of s tokens has ceil(s / p) pages.  One that grows by n needs
// ceil((s + n) / p) - ceil(s / p) more; they come from the end of the list, for the first sequence first: with `before` pages
// for the sequences ahead of it, its i-th new page is free[count - 1 - (before + i)].  A token at position x of its
// sequence has the slot table[x / p] p + x mod p.  Giving back is the inverse, entry for entry: a trim that undoes an
// extension leaves list and count as they were.
//
// What bounds it: the launch and a chain of few dependent loads (lengths, a scan, free pages, table entries).  One CTA
// makes the plan: sums over up to 1,024 sequences at a time in shared memory, then a thread for each new page and for each
// new token, which finds its sequence by bisection, so that long and short sequences cost alike and stores are whole
// sectors.  From kPagesAlone tokens on a second kernel, of as many CTAs as that takes, writes the slots.
#pragma once

#include "tps_decode.h"
#include "tps_device.cuh"

namespace tps {

constexpr int kPagesThreads = 1024;
constexpr int kPagesWarps = kPagesThreads / 32;
constexpr int kSlotsThreads = 256, kSlotsEach = 4;  // of the second kernel; tokens of a thread

struct PagesShared {
    int64_t parts[2][kPagesWarps];
    int pages[kPagesThreads], tokens[kPagesThreads];  // of the chunk's sequences ahead
    int length[kPagesThreads], has[kPagesThreads];    // tokens that are there (-1: nothing is done), pages
    unsigned long long moved;                         // pages that went from the list or back to it
};

// Inclusive sums of x and y over the CTA's threads, and their totals.
__device__ __forceinline__ void block_sums(PagesShared& sh, int64_t& x, int64_t& y, int64_t& all_x, int64_t& all_y)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, x, o), v = __shfl_up_sync(0xFFFFFFFFu, y, o);
        if (lane >= o) x += u, y += v;
    }
    if (lane == 31) sh.parts[0][warp] = x, sh.parts[1][warp] = y;
    __syncthreads();
    int64_t px = sh.parts[0][lane], py = sh.parts[1][lane];
    all_x = px, all_y = py;
    if (lane >= warp) px = py = 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        px += __shfl_xor_sync(0xFFFFFFFFu, px, o), py += __shfl_xor_sync(0xFFFFFFFFu, py, o);
        all_x += __shfl_xor_sync(0xFFFFFFFFu, all_x, o), all_y += __shfl_xor_sync(0xFFFFFFFFu, all_y, o);
    }
    x += px, y += py;
}

// For each x, the last of n ascending numbers that is at most x (the first one is); n is at most kPagesThreads.  Several
// at once: a step is a chain of one read.
template <int N> __device__ __forceinline__ void owners(const int* first, int n, const int (&x)[N], int (&at)[N])
{
#pragma unroll
    for (int k = 0; k < N; ++k) at[k] = 0;
#pragma unroll
    for (int step = kPagesThreads / 2; step > 0; step >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (at[k] + step < n && first[at[k] + step] <= x[k]) at[k] += step;
}

// do_one(i, the sequence that `first` gives i to) for all i below `count`, four of a thread at a time: load_one's values are on
// their way together.
template <typename Value, typename Load, typename Store>
__device__ __forceinline__ void for_each_owned(const int* first, int n, int64_t count, Load load_one, Store store_one)
{
    for (int64_t base = 0; base < count; base += 4 * kPagesThreads) {
        int x[4], at[4];
        Value v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = (int)min(base + k * kPagesThreads + (int)threadIdx.x, count - 1);
        owners(first, n, x, at);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = load_one(x[k], at[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (base + k * kPagesThreads + (int)threadIdx.x < count) store_one(x[k], at[k], v[k]);
    }
}

// Of the sequences that are served, the one most ahead: `sum` pages have gone with it.
__device__ __forceinline__ void note_moved(PagesShared& sh, bool served, int64_t sum)
{
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, served);
    if (who && (threadIdx.x & 31) == 31 - __clz(who)) atomicMax(&sh.moved, (unsigned long long)sum);
}

__device__ __forceinline__ int64_t slot_of(const PagesArgs& a, int64_t b, int at)
{
    return ((int64_t)a.p.page_table[b * a.p.table_ld + (at >> a.page_shift)] << a.page_shift) + (at & a.page_mask);
}

template <bool kSlots> __global__ void __launch_bounds__(kPagesThreads) kv_extend_kernel(const __grid_constant__ PagesArgs a)
{
    __shared__ PagesShared sh;
    const tps_kv_pages& p = a.p;
    const int tid = (int)threadIdx.x;
    const int64_t count = min((int64_t)max(*p.free_count, 0), p.n_free), room = p.table_width << a.page_shift;
    int64_t asked = 0, packed = 0, moved = 0;  // pages asked for, rows so far, pages taken from the list
    if (tid == 0) sh.moved = 0;
    for (int64_t base = 0; base < p.B; base += kPagesThreads) {
        const int64_t b = base + tid;
        const bool in = b < p.B;
        const int64_t s = in ? p.seq_len[b] : 0, n = in ? p.change[b] : 0;
        const bool valid = s >= 0 && n >= 0 && s + n <= room;
        const int64_t has = valid ? (s + a.page_mask) >> a.page_shift : 0;
        const int64_t need = valid ? ((s + n + a.page_mask) >> a.page_shift) - has : 0, rows = max(n, (int64_t)0);
        int64_t pages = need, tokens = rows, all_pages, all_tokens;
        block_sums(sh, pages, tokens, all_pages, all_tokens);
        // Once a sequence's pages or rows are too many, so are those of all that come after it and ask for any: what
        // has been taken is always a piece of the list without gaps.
        const bool fits = rows == 0 || packed + tokens <= a.tokens, there = need == 0 || asked + pages <= count, done = valid && fits && there;
        note_moved(sh, done && need > 0, asked + pages);
        sh.pages[tid] = (int)min(pages - need, (int64_t)INT32_MAX);
        sh.tokens[tid] = (int)min(tokens - rows, max(a.tokens - packed, (int64_t)0));
        sh.length[tid] = done ? (int)s : -1;
        sh.has[tid] = (int)has;
        if (in) {
            if (p.out_status) p.out_status[b] = done ? TPS_ROW_OK : (valid && fits ? TPS_ROW_NO_PAGES : TPS_ROW_BAD_PARAM);
            a.cu_seqlens[b] = (int)min(packed + tokens - rows, a.tokens);
            if (done) p.seq_len[b] = (int)(s + n);
            if (!kSlots) a.first[b] = done ? (int)s : -1;
        }
        __syncthreads();
        const int live = (int)min(p.B - base, (int64_t)kPagesThreads);
        const int64_t now = (int64_t)sh.moved;
        for_each_owned<int>(
            sh.pages, live, now - moved, [&](int i, int) { return p.free_pages[count - 1 - (moved + i)]; },
            [&](int i, int w, int page) { p.page_table[(base + w) * p.table_ld + sh.has[w] + (i - sh.pages[w])] = page; });
        if (kSlots) {
            __syncthreads();
            for_each_owned<int64_t>(
                sh.tokens, live, min(all_tokens, a.tokens - packed),
                [&](int i, int w) { return sh.length[w] >= 0 ? slot_of(a, base + w, sh.length[w] + i - sh.tokens[w]) : -1; },
                [&](int i, int w, int64_t slot) {
                    a.slots[packed + i] = slot;
                    a.positions[packed + i] = sh.length[w] >= 0 ? sh.length[w] + i - sh.tokens[w] : 0;
                });
        }
        moved = now;
        asked += all_pages;
        packed += all_tokens;
        __syncthreads();  // the chunk's numbers have been read
    }
    if (tid == 0) {
        a.cu_seqlens[p.B] = (int)min(packed, a.tokens);
        *p.free_count = (int)(count - moved);
    }
    if (kSlots)
        for (int64_t i = packed + tid; i < a.tokens; i += kPagesThreads) a.slots[i] = -1, a.positions[i] = 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The slots and positions of many tokens, kSlotsEach to a thread.
static __global__ void __launch_bounds__(kSlotsThreads) kv_slots_kernel(const __grid_constant__ PagesArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan
    const int64_t begin = (int64_t)blockIdx.x * kSlotsThreads * kSlotsEach, i0 = begin + (int64_t)threadIdx.x * kSlotsEach;
    const int total = a.cu_seqlens[a.p.B];
    // The last sequence that begins at or before the CTA's first row, and before its last: all threads count.
    int64_t low = -1, high = -1;
    for (int64_t base = 0; base < a.p.B; base += kSlotsThreads) {
        const int64_t b = base + threadIdx.x;
        const int at = b < a.p.B ? a.cu_seqlens[b] : INT32_MAX;
        low += __syncthreads_count(at <= begin);
        high += __syncthreads_count(at < begin + kSlotsThreads * kSlotsEach);
    }
    if (i0 >= a.tokens) return;
    int64_t b = low;
    while (i0 < total && high - b > 1) {
        const int64_t mid = (b + high + 1) >> 1;
        if (a.cu_seqlens[mid] <= i0)
            b = mid;
        else
            high = mid - 1;
    }
    int64_t slot[kSlotsEach];
    int position[kSlotsEach];
#pragma unroll
    for (int j = 0; j < kSlotsEach; ++j) {
        slot[j] = -1, position[j] = 0;
        if (i0 + j < total) {
            while (a.cu_seqlens[b + 1] <= i0 + j) ++b;
            const int s = a.first[b], at = s + (int)(i0 + j) - a.cu_seqlens[b];
            if (s >= 0) slot[j] = slot_of(a, b, at), position[j] = at;
        }
    }
    if (i0 + kSlotsEach <= a.tokens && a.wide) {
        reinterpret_cast<longlong2*>(a.slots + i0)[0] = make_longlong2(slot[0], slot[1]);
        reinterpret_cast<longlong2*>(a.slots + i0)[1] = make_longlong2(slot[2], slot[3]);
        *reinterpret_cast<int4*>(a.positions + i0) = make_int4(position[0], position[1], position[2], position[3]);
    } else {
        for (int j = 0; j < kSlotsEach && i0 + j < a.tokens; ++j) a.slots[i0 + j] = slot[j], a.positions[i0 + j] = position[j];
    }
}

static __global__ void __launch_bounds__(kPagesThreads) kv_trim_kernel(const __grid_constant__ PagesArgs a)
{
    __shared__ PagesShared sh;
    const tps_kv_pages& p = a.p;
    const int tid = (int)threadIdx.x;
    const int64_t count = min((int64_t)max(*p.free_count, 0), p.n_free), room = p.table_width << a.page_shift;
    if (tid == 0) sh.moved = 0;
    int64_t total = 0;
    // The list ends with the first sequence's pages, so their number has to be known before any is put down: with more
    // than one chunk of sequences a first pass counts.
    for (int pass = p.B > kPagesThreads ? 0 : 1; pass < 2; ++pass) {
        int64_t asked = 0;  // pages of the chunks before
        for (int64_t base = 0; base < p.B; base += kPagesThreads) {
            const int64_t b = base + tid;
            const bool in = b < p.B;
            const int64_t s = in ? p.seq_len[b] : 0, k = in ? p.change[b] : 0;
            const bool valid = k >= 0 && k <= s && s <= room;
            const int64_t keep = valid ? (k + a.page_mask) >> a.page_shift : 0;
            const int64_t back = valid ? ((s + a.page_mask) >> a.page_shift) - keep : 0;
            int64_t pages = back, none = 0, all_pages, all_none;
            block_sums(sh, pages, none, all_pages, all_none);
            const bool there = back == 0 || count + asked + pages <= p.n_free, done = valid && there;
            note_moved(sh, done && back > 0, asked + pages);
            if (pass == 1) {
                sh.pages[tid] = (int)min(pages - back, (int64_t)INT32_MAX);
                sh.has[tid] = (int)keep;
                if (in) {
                    if (p.out_status) p.out_status[b] = done ? TPS_ROW_OK : (valid ? TPS_ROW_NO_PAGES : TPS_ROW_BAD_PARAM);
                    if (done) p.seq_len[b] = (int)k;
                }
            }
            __syncthreads();
            if (pass == 1) {
                if (p.B <= kPagesThreads) total = (int64_t)sh.moved;
                // pages of this chunk that go back: those up to `total`
                for_each_owned<int>(
                    sh.pages, (int)min(p.B - base, (int64_t)kPagesThreads), min(all_pages, total - min(asked, total)),
                    [&](int i, int w) { return p.page_table[(base + w) * p.table_ld + sh.has[w] + (i - sh.pages[w])]; },
                    [&](int i, int, int page) { p.free_pages[count + total - 1 - (asked + i)] = page; });
            }
            asked += all_pages;
            __syncthreads();
        }
        total = (int64_t)sh.moved;
    }
    if (tid == 0) *p.free_count = (int)(count + total);
}

}  // namespace tps
