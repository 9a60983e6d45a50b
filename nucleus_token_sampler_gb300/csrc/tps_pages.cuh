// tps_pages.cuh -- the pages that sequences get from a list of free ones as they grow and give back as they shrink,
// and the cache slots of their new tokens.
//
// Formulas.  With p tokens to a page, a sequence of s tokens has ceil(s / p) pages.  One that grows by n needs
// ceil((s + n) / p) - ceil(s / p) more; they come from the end of the list, for the first sequence first: with `before` pages
// for the sequences ahead of it, its i-th new page is free[count - 1 - (before + i)].  A token at position x of its
// sequence has the slot table[x / p] p + x mod p.  Giving back is the inverse, entry for entry: a trim that undoes an
// extension leaves list and count as they were.
//
// What bounds it: the launch and a chain of few dependent loads (lengths, a scan, free pages or table entries).  Up to 1,024
// sequences at a time are summed up in shared memory; then there is a thread for each new token, which finds its sequence by
// bisection, so that long and short sequences cost alike and stores are whole sectors.  A page's first token also puts it in the
// table: the pages need no pass of their own, and no token waits for the table.  From some 2,000 tokens on they are a second
// kernel's, over all SMs; a trim of many pages is shared by a cluster of CTAs, each of which sums up for itself.
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
    for (int step = 1 << (31 - __clz(max(n - 1, 1))); step > 0; step >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (at[k] + step < n && first[at[k] + step] <= x[k]) at[k] += step;
}

// For all i below `count`, shared over the cluster's CTAs: load_one(i, the sequence that `first` gives i to), then
// store_one(i, sequence, that value); four of a thread at a time, whose loads are on their way together.
template <typename Value, typename Load, typename Store>
__device__ __forceinline__ void for_each_owned(const int* first, int n, int64_t count, Load load_one, Store store_one)
{
    for (int64_t base = (int64_t)blockIdx.x * (4 * kPagesThreads); base < count; base += (int64_t)gridDim.x * (4 * kPagesThreads)) {
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

// The page of a new token at position `at` of sequence b: one it has (`has` of them), or, of the free list, the one `from` down
// from its end and so on.
__device__ __forceinline__ int page_of(const PagesArgs& a, int64_t b, int at, int has, int64_t count, int64_t from)
{
    const int page = at >> a.page_shift;
    return *(page < has ? a.p.page_table + b * a.p.table_ld + page : a.p.free_pages + (count - 1 - (from + (page - has))));
}
// A page's first token puts it in the table, if it is new.
__device__ __forceinline__ void note_page(const PagesArgs& a, int64_t b, int at, int has, int page)
{
    if ((at & a.page_mask) == 0 && at >> a.page_shift >= has) a.p.page_table[b * a.p.table_ld + (at >> a.page_shift)] = page;
}

template <bool kSlots> __global__ void __launch_bounds__(kPagesThreads) kv_extend_kernel(const __grid_constant__ PagesArgs a)
{
    __shared__ PagesShared sh;
    const tps_kv_pages& p = a.p;
    const int tid = (int)threadIdx.x;
    const int64_t count = min((int64_t)max(*p.free_count, 0), p.n_free), room = p.table_width << a.page_shift;
    int64_t asked = 0, packed = 0;  // pages asked for, rows so far
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
        // is taken is always a piece of the list without gaps, and each sequence's pages lie as far from its end as the sum says.
        const bool fits = rows == 0 || packed + tokens <= a.tokens, there = need == 0 || asked + pages <= count, done = valid && fits && there;
        note_moved(sh, done && need > 0, asked + pages);
        sh.pages[tid] = (int)min(asked + pages - need, (int64_t)INT32_MAX);
        sh.tokens[tid] = (int)min(tokens - rows, max(a.tokens - packed, (int64_t)0));
        sh.length[tid] = done ? (int)s : -1;
        sh.has[tid] = (int)has;
        if (in) {
            if (p.out_status) p.out_status[b] = done ? TPS_ROW_OK : (valid && fits ? TPS_ROW_NO_PAGES : TPS_ROW_BAD_PARAM);
            a.cu_seqlens[b] = (int)min(packed + tokens - rows, a.tokens);
            if (!kSlots) a.first[b] = make_int2(sh.length[tid], sh.pages[tid]);
        }
        __syncthreads();
        if (kSlots)
            for_each_owned<int>(
                sh.tokens, (int)min(p.B - base, (int64_t)kPagesThreads), min(all_tokens, a.tokens - packed),
                [&](int i, int w) {
                    return sh.length[w] >= 0 ? page_of(a, base + w, sh.length[w] + i - sh.tokens[w], sh.has[w], count, sh.pages[w]) : 0;
                },
                [&](int i, int w, int page) {
                    const int at = sh.length[w] + i - sh.tokens[w];
                    const bool ok = sh.length[w] >= 0;
                    a.slots[packed + i] = ok ? ((int64_t)page << a.page_shift) + (at & a.page_mask) : -1;
                    a.positions[packed + i] = ok ? at : 0;
                    if (ok) note_page(a, base + w, at, sh.has[w], page);
                });
        if (in && done) p.seq_len[b] = (int)(s + n);
        asked += all_pages;
        packed += all_tokens;
        __syncthreads();  // the chunk's numbers have been read
    }
    if (tid == 0) {
        if (!kSlots) a.first[p.B] = make_int2((int)count, 0);
        a.cu_seqlens[p.B] = (int)min(packed, a.tokens);
        *p.free_count = (int)(count - (int64_t)sh.moved);
    }
    if (kSlots)
        for (int64_t i = packed + tid; i < a.tokens; i += kPagesThreads) a.slots[i] = -1, a.positions[i] = 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The slots, positions and new pages of many tokens, kSlotsEach tokens to a thread.  (The sequences' lengths and the count of free
// pages have been moved on: `first` holds what they were.)
static __global__ void __launch_bounds__(kSlotsThreads) kv_slots_kernel(const __grid_constant__ PagesArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan
    const int64_t begin = (int64_t)blockIdx.x * kSlotsThreads * kSlotsEach, i0 = begin + (int64_t)threadIdx.x * kSlotsEach;
    const int total = a.cu_seqlens[a.p.B];
    const int64_t count = a.first[a.p.B].x;
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
    int64_t of = -1;  // the sequence that the numbers below are of
    int2 first = {};
    int begins = 0, ends = 0, has = 0;
#pragma unroll
    for (int j = 0; j < kSlotsEach; ++j) {
        slot[j] = -1, position[j] = 0;
        if (i0 + j < total) {
            if (of < 0 || ends <= i0 + j) {
                while ((ends = a.cu_seqlens[b + 1]) <= i0 + j) ++b;
                of = b, begins = a.cu_seqlens[b], first = a.first[b], has = (first.x + a.page_mask) >> a.page_shift;
            }
            const int at = first.x + (int)(i0 + j) - begins;
            if (first.x >= 0) {
                const int page = page_of(a, b, at, has, count, first.y);
                slot[j] = ((int64_t)page << a.page_shift) + (at & a.page_mask), position[j] = at;
                note_page(a, b, at, has, page);
            }
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

// In a cluster nothing that another CTA may still read is overwritten before all have read it; it has one chunk of sequences.
__device__ __forceinline__ void all_have_read()
{
    if (gridDim.x > 1) {
        cluster_arrive();
        cluster_wait();
    }
}

static __global__ void __launch_bounds__(kPagesThreads) kv_trim_kernel(const __grid_constant__ PagesArgs a)
{
    __shared__ PagesShared sh;
    const tps_kv_pages& p = a.p;
    const int tid = (int)threadIdx.x;
    const bool first_cta = blockIdx.x == 0;
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
                if (in && first_cta && p.out_status) p.out_status[b] = done ? TPS_ROW_OK : (valid ? TPS_ROW_NO_PAGES : TPS_ROW_BAD_PARAM);
            }
            __syncthreads();
            if (pass == 1) {
                if (p.B <= kPagesThreads) total = (int64_t)sh.moved;
                // pages of this chunk that go back: those up to `total`
                for_each_owned<int>(
                    sh.pages, (int)min(p.B - base, (int64_t)kPagesThreads), min(all_pages, total - min(asked, total)),
                    [&](int i, int w) { return p.page_table[(base + w) * p.table_ld + sh.has[w] + (i - sh.pages[w])]; },
                    [&](int i, int, int page) { p.free_pages[count + total - 1 - (asked + i)] = page; });
                all_have_read();
                if (in && first_cta && done) p.seq_len[b] = (int)k;
            }
            asked += all_pages;
            __syncthreads();
        }
        total = (int64_t)sh.moved;
    }
    if (tid == 0 && first_cta) *p.free_count = (int)(count + total);
}

}  // namespace tps
