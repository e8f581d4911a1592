// The plan of a step over a paged key/value cache, made on the device from request lengths:
// which pages each request gives back or takes, where each new token's row goes, and the
// boundaries and positions the other calls read.
//
// A request holds held = seqlens[s] rows, keeps the first keep[s] of them and adds new[s]:
// after = keep + new. It had ceil(held / page) pages and needs ceil(after / page). The free
// pages are a stack: the released pages are pushed first, in the order of (request, page),
// then the pages wanted are popped in the same order, so the result does not depend on timing.
//
// One launch. Every CTA scans all lengths itself (S is small) and keeps the running sums in shared
// memory; the work after the scan is shared out. Nothing is read and written at once: pops read the
// list below free_count, pushes write it from free_count on (a popped page that this call released
// is looked up in the table it came from, not in the list), and a request that releases pages
// takes none. Only where seqlens_out is one of the inputs, or free_count_out is free_count, must every
// CTA have read them before one writes: then the CTAs are one cluster with a barrier in between, else they
// are as many as there is work for and need none. Calling again with the same seqlens and
// free_count gives the same result.
//
// Bound by latency: a launch, three dependent global reads and two block barriers. 64 requests
// 5.4 us, 1024 requests with 130000 new tokens 9.3 us. In place, where the cluster's eight CTAs do all the
// writing: 64 requests with a token each 5.7 us (5.2 with as many CTAs as there is work for), 1024 requests
// with 131072 tokens and no page moved 12.8 us (6.1).
#pragma once

#include <cooperative_groups.h>

#include "sm100_ptx.cuh"

namespace gqa {

constexpr int kPagedMaxSeqs = 8192;      // 5 ints a request of shared memory
constexpr int kPagedFewSeqs = 256;       // at most, for blocks of kPagedFewThreads
constexpr int kPagedFewThreads = 256;
// CTAs of the cluster, the portable size: with few tokens as fast as one (64 requests with a token each 5.7 us
// either way), and 64 requests with 64 tokens each 4.4 us where one CTA takes 8.1.
constexpr int kPagedCluster = 8;

struct PagedPlanParams {
    const int* held;      // [S]
    const int* keep;      // [S] or null: all held rows
    const int* added;     // [S]
    int* table;           // [S, max_pages]
    int* free_list;       // [free_capacity], a stack of free_count pages
    const int* free_count;
    int* after;           // [S]
    int* cu;              // [S + 1]
    int* positions;       // [max_tokens]
    int* slots;           // [max_tokens]
    int* free_count_out;
    int S, max_pages, page_size, num_pages, free_capacity, max_tokens;
    uint32_t* err;
};

inline size_t paged_plan_smem(int S) { return (size_t)(5 * S + 3) * sizeof(int); }

// Last s in [lo, hi) with first[s] <= x; first is non-decreasing and first[lo] <= x.
__device__ __forceinline__ int paged_find(const int* first, int lo, int hi, int x) {
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Inclusive block scans of two 64-bit values; total gets the block's sums. All threads call it.
template <int kThreads>
__device__ __forceinline__ void paged_scan(unsigned long long (&v)[2], unsigned long long (*warp_sums)[32],
                                           unsigned long long (&total)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const unsigned long long o = __shfl_up_sync(0xffffffffu, v[i], d);
            if (lane >= d) v[i] += o;
        }
    if (lane == 31) warp_sums[0][warp] = v[0], warp_sums[1][warp] = v[1];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const unsigned long long w = lane < kThreads / 32 ? warp_sums[i][lane] : 0;
        unsigned long long inc = w;
#pragma unroll
        for (int d = 1; d < kThreads / 32; d <<= 1) {
            const unsigned long long o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        total[i] = __shfl_sync(0xffffffffu, inc, kThreads / 32 - 1);
        v[i] += __shfl_sync(0xffffffffu, inc - w, warp);
    }
    __syncthreads();
}

template <int kThreads, bool kCluster>
__global__ void __launch_bounds__(kThreads, 1) gqa_paged_plan_kernel(const __grid_constant__ PagedPlanParams p) {
    namespace cg = cooperative_groups;
    extern __shared__ int paged_smem[];
    __shared__ unsigned long long warp_sums[2][32];
    int* cu = paged_smem;             // [S + 1] first token of each request
    int* first_take = cu + p.S + 1;   // [S + 1] first popped page of each request
    int* first_give = first_take + p.S + 1;  // [S + 1] first pushed page of each request
    int* keep_s = first_give + p.S + 1;      // [S]
    int* had_s = keep_s + p.S;               // [S]

    const long long capacity = (long long)p.max_pages * p.page_size;
    const int count = *p.free_count;
    bool bad = false;
    // running totals; pages: released << 32 | taken, each at most S * max_pages < 2^31 (checked on the host)
    unsigned long long tokens = 0, pages = 0;
    for (int base = 0; base < p.S; base += kThreads) {
        const int s = base + threadIdx.x;
        int held = 0, keep = 0, added = 0;
        if (s < p.S) {
            held = p.held[s];
            keep = p.keep ? p.keep[s] : held;
            added = p.added[s];
            if (held < 0 || held > capacity || keep < 0 || keep > held || added < 0 || added > p.max_tokens ||
                (long long)keep + added > capacity) {
                bad = true;
                held = keep = added = 0;
            }
        }
        const int had = (int)(((long long)held + p.page_size - 1) / p.page_size);
        const int has = (int)(((long long)keep + added + p.page_size - 1) / p.page_size);
        const unsigned long long mine =
            has > had ? (unsigned long long)(has - had) : (unsigned long long)(had - has) << 32;
        unsigned long long sums[2] = {(unsigned long long)added, mine}, all[2];
        paged_scan<kThreads>(sums, warp_sums, all);
        const unsigned long long t = tokens + sums[0] - added, g = pages + sums[1] - mine;
        tokens += all[0];
        pages += all[1];
        if (s < p.S) {
            cu[s] = (int)min(t, (unsigned long long)0x7fffffff);  // past it the call is refused below
            first_take[s] = (int)(g & 0xffffffffu);
            first_give[s] = (int)(g >> 32);
            keep_s[s] = keep;
            had_s[s] = had;
        }
    }
    const int n_take = (int)(pages & 0xffffffffu), n_give = (int)(pages >> 32);
    const int n_push = n_give - min(n_give, n_take);  // released pages that stay on the stack
    if (threadIdx.x == 0) {
        cu[p.S] = (int)min(tokens, (unsigned long long)0x7fffffff);
        first_take[p.S] = n_take;
        first_give[p.S] = n_give;
    }
    if (tokens > (unsigned long long)p.max_tokens || count < 0 || count > p.free_capacity ||
        (long long)count + n_give < n_take || (long long)count + n_push > p.free_capacity)
        bad = true;
    bad = __syncthreads_or(bad);
    if constexpr (kCluster) cg::this_cluster().sync();  // every CTA has read the lengths and the count

    // Unsigned: max_tokens and free_capacity may be 2^31 - 1, and a thread steps past them by up to the grid's
    // threads times four.
    const unsigned threads = gridDim.x * kThreads;
    const unsigned tid = blockIdx.x * kThreads + threadIdx.x;
    const unsigned n_slots = p.max_tokens;
    if (bad) {  // nothing happens to the cache; the outputs describe an empty step
        if (tid == 0) {
            atomicOr(p.err, kDevErrBadSeqlens);
            p.cu[p.S] = 0;
            if (p.free_count_out != p.free_count) *p.free_count_out = count;
        }
        for (unsigned s = tid; s < (unsigned)p.S; s += threads) {
            p.cu[s] = 0;
            if (p.after != p.held) p.after[s] = p.held[s];
        }
        for (unsigned t = tid; t < n_slots; t += threads) {
            p.positions[t] = 0;
            p.slots[t] = -1;
        }
        return;
    }

    // page i of the released ones, in push order
    const auto released = [&](int i) {
        const int s = paged_find(first_give, 0, p.S, i);
        const int has = had_s[s] - (first_give[s + 1] - first_give[s]);
        return p.table[(size_t)s * p.max_pages + has + (i - first_give[s])];
    };
    // page j of the taken ones, in pop order
    const auto taken = [&](int j) { return j < n_give ? released(n_give - 1 - j) : p.free_list[count - 1 - (j - n_give)]; };

    if (tid == 0) {
        p.cu[p.S] = cu[p.S];
        *p.free_count_out = count + (n_give - n_take);
    }
    for (unsigned s = tid; s < (unsigned)p.S; s += threads) {
        p.cu[s] = cu[s];
        p.after[s] = keep_s[s] + (cu[s + 1] - cu[s]);
    }
    // pages from the last thread down, tokens from the first up: where there are threads for both, they
    // do not wait for one another
    for (unsigned i = threads - 1 - tid; i < (unsigned)n_push; i += threads) p.free_list[count + i] = released((int)i);
    for (unsigned i = threads - 1 - tid; i < (unsigned)n_take; i += threads) {
        const int j = (int)i, s = paged_find(first_take, 0, p.S, j);
        p.table[(size_t)s * p.max_pages + had_s[s] + (j - first_take[s])] = taken(j);
    }
    // four tokens a thread, stored as one vector each; the last ones may be padding
    const int total = cu[p.S];
    for (unsigned t0 = tid * 4; t0 < n_slots; t0 += threads * 4) {
        int pos[4], slot[4];
        int s = 0, ordinal = -1, page = 0;
        for (int e = 0; e < 4; ++e) {
            pos[e] = 0;
            slot[e] = -1;
            if (t0 + e >= (unsigned)total) continue;
            const int t = (int)(t0 + e);
            if (e == 0 || t >= cu[s + 1]) {
                s = paged_find(cu, s, p.S, t);
                ordinal = -1;
            }
            pos[e] = keep_s[s] + (t - cu[s]);
            const int o = pos[e] / p.page_size;
            if (o != ordinal) {
                ordinal = o;
                // pages taken by this call are computed again: another thread writes their entries
                page = o < had_s[s] ? p.table[(size_t)s * p.max_pages + o] : taken(first_take[s] + (o - had_s[s]));
            }
            if (page >= 0 && page < p.num_pages)
                slot[e] = page * p.page_size + (pos[e] - o * p.page_size);
            else
                atomicOr(p.err, kDevErrBadSeqlens);
        }
        if (t0 + 4 <= n_slots) {
            *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
            for (int e = 0; t0 + e < n_slots; ++e) {
                p.positions[t0 + e] = pos[e];
                p.slots[t0 + e] = slot[e];
            }
        }
    }
}

}  // namespace gqa
