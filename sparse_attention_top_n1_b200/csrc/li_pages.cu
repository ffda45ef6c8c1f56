// li_pages.cu -- the pages of a PA_BSND cache: growing, forking, emptying and
// compacting rows of the block table, and copying pages.
//
// A call is two launches.  The plan kernel's first block decides everything
// that depends on an order (which free page goes to whom, which pages move):
// it scans the reference counts with all of a thread's loads in flight at once
// and ranks free or live pages by warp votes, so the result is the lowest
// pages first whatever the timing.  Its other blocks copy the counts to the
// output buffer meanwhile.  The apply kernel writes the new table, lengths and
// counts and copies page contents; it is launched programmatically, so that its
// launch is prepared beside the plan, but the plan gives no signal before its
// end and the apply's blocks start when the plan's have all exited.
//
// Bounds: the tables are a few hundred kilobytes, so small calls are bound by
// the latency of two dependent launches and one scan (5 to 7 us; one launch of a
// cluster with a barrier between the steps took 8.6 us for a reservation where
// these take 6.6); copies are bound by HBM (each page read once and written
// once, in accesses marked as used once).
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>

#include "li.h"
#include "ptx.cuh"

namespace li {
li_status report_error(li_status s, const char *msg);
void set_launch_count(int32_t n);
}  // namespace li

namespace {

using namespace li;

constexpr int kPlanThreads = 1024;
constexpr int kWarps = kPlanThreads / 32;
constexpr int kQuads = 8;                                 // int4 of counts per thread and pass
constexpr int kPassPages = kPlanThreads * 4 * kQuads;     // 32768 pages
constexpr int kApplyThreads = 256;
constexpr int kChunk = 32768;                             // bytes a block copies at a time (159 MB: 16 KB 39.6 us, 8 KB 49 us)
constexpr int kMaxPools = 64;                             // descriptors of one launch
constexpr int kFewPools = 4;                              // of a launch with short parameters
constexpr int kMaxPoolsCall = 256;

enum Op { kReserve, kFork, kFree, kCompact };

// Workspace (after a 256-byte header): claim [B] (which pair or row acts on a
// table row), old [B] (the lengths before the call, clamped), grant [B] (rank of
// the first fresh page of a row or of a pair's new row), list [num_pages] (fresh
// pages by rank; compact: holes), from [num_pages] (compact: movers), where
// [num_pages] (compact: a mover's new place, a hole's mover, else -1).
constexpr int32_t kNone = 0x7FFFFFFF;
struct Header {
    int32_t moved;       // compact: pages that move
    int32_t live;        // compact: live pages; else: fresh pages at hand
    int32_t pad[62];
};

struct PagesArgs {
    const int32_t *table, *lens, *refs;
    int32_t *table_out, *lens_out, *refs_out;
    const int32_t *arg0, *arg1;      // reserve: new lengths; fork: source rows, new rows; free: rows
    Header *hdr;
    int32_t *claim, *old, *grant, *list, *from, *where;
    int32_t *status;
    int32_t P, ps, cols, B, n;
};

template <int N>
struct Pools {
    char *base[N];
    int64_t bytes[N], stride[N];
    int32_t n;
};

__device__ __forceinline__ void flag(int32_t *status, int32_t bit)
{
    if (status) atomicOr(status, bit);
}

__device__ __forceinline__ int32_t pages_of(int32_t len, int32_t ps) { return len / ps + (len % ps != 0); }

// A row's length, clamped to what its columns hold.
__device__ __forceinline__ int32_t clamp_len(const PagesArgs &a, int32_t len)
{
    const int32_t cap = a.cols * a.ps;
    if (len < 0 || len > cap) {
        flag(a.status, LI_DEV_BAD_KLEN);
        return len < 0 ? 0 : cap;
    }
    return len;
}

// Fresh pages that a reservation of `want` tokens takes for a row of `len`.
__device__ __forceinline__ int32_t growth(const PagesArgs &a, int32_t len, int32_t want)
{
    return want > len && want <= a.cols * a.ps ? pages_of(want, a.ps) - pages_of(len, a.ps) : 0;
}

// Exclusive prefix sum of one value per thread over the block; *total receives
// the sum.
__device__ int32_t block_scan(int32_t v, int32_t *warp_sums, int32_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();                                       // warp_sums of an earlier scan have been read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int32_t w = warp_sums[lane], z = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, z, d);
            if (lane >= d) z += y;
        }
        warp_sums[lane] = z - w;
        if (lane == 31) warp_sums[32] = z;
    }
    __syncthreads();
    *total = warp_sums[32];
    return warp_sums[warp] + x - v;
}

// Ranks the pages p of [first, limit) within the pass that starts at `begin` (a
// multiple of 4) with (refs[p] == 0) == want_free in ascending order: take(rank,
// p) for the ranks below `most`, counted from rank0.
// Returns rank0 plus how many there are.  counts: [kQuads * kWarps] and
// warp_sums [33] in shared memory.
template <typename Take>
__device__ int32_t rank_pass(const PagesArgs &a, int32_t begin, int32_t first, int32_t limit, bool want_free, int32_t rank0,
                             int32_t most, int32_t *counts, int32_t *warp_sums, Take take)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t bits = 0;                                     // 4 bits per quad
    const bool wide = (reinterpret_cast<uintptr_t>(a.refs) & 15) == 0;
    int4 q[kQuads];
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
        const int32_t p = begin + (j * kPlanThreads + tid) * 4;
        if (wide && p >= first && p + 4 <= limit) {
            q[j] = *reinterpret_cast<const int4 *>(a.refs + p);
        } else {
            // outside: neither free nor live
            const int32_t none = want_free ? 1 : 0;
            q[j].x = p >= first && p < limit ? a.refs[p] : none;
            q[j].y = p + 1 >= first && p + 1 < limit ? a.refs[p + 1] : none;
            q[j].z = p + 2 >= first && p + 2 < limit ? a.refs[p + 2] : none;
            q[j].w = p + 3 >= first && p + 3 < limit ? a.refs[p + 3] : none;
        }
    }
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
        const uint32_t m = (uint32_t)((q[j].x == 0) == want_free) | (uint32_t)((q[j].y == 0) == want_free) << 1 |
                           (uint32_t)((q[j].z == 0) == want_free) << 2 | (uint32_t)((q[j].w == 0) == want_free) << 3;
        bits |= m << (4 * j);
        const int32_t c = __reduce_add_sync(0xffffffffu, __popc(m));
        if (lane == 0) counts[j * kWarps + warp] = c;
    }
    __syncthreads();
    int32_t total;
    const int32_t mine = tid < kQuads * kWarps ? counts[tid] : 0;
    const int32_t before = block_scan(mine, warp_sums, &total);
    if (tid < kQuads * kWarps) counts[tid] = before;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
        int32_t r = rank0 + counts[j * kWarps + warp];
        if (r >= most) continue;                           // uniform over the warp
        const uint32_t m = (bits >> (4 * j)) & 15u;
        int32_t x = __popc(m);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        r += x - __popc(m);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (m >> e & 1u) {
                if (r < most) take(r, begin + (j * kPlanThreads + tid) * 4 + e);
                ++r;
            }
    }
    __syncthreads();
    return rank0 + total;
}

// The moves of a compaction of at most kPassPages pages from one look at the
// counts.  With L(p) live pages below p, a free page p below the live pages' new
// end n is hole p - L(p), a live page p from n on is mover L(p) - L(n).
__device__ void compact_plan(const PagesArgs &a, int32_t *counts, int32_t *warp_sums)
{
    __shared__ int32_t below_end;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool wide = (reinterpret_cast<uintptr_t>(a.refs) & 15) == 0;
    int4 q[kQuads];
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
        const int32_t p = (j * kPlanThreads + tid) * 4;
        q[j] = make_int4(0, 0, 0, 0);
        if (wide && p + 4 <= a.P) {
            q[j] = *reinterpret_cast<const int4 *>(a.refs + p);
        } else {
            if (p < a.P) q[j].x = a.refs[p];
            if (p + 1 < a.P) q[j].y = a.refs[p + 1];
            if (p + 2 < a.P) q[j].z = a.refs[p + 2];
            if (p + 3 < a.P) q[j].w = a.refs[p + 3];
        }
    }
    uint32_t bits = 0;                                     // live pages, 4 bits per quad
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
        const uint32_t m = (uint32_t)(q[j].x != 0) | (uint32_t)(q[j].y != 0) << 1 | (uint32_t)(q[j].z != 0) << 2 |
                           (uint32_t)(q[j].w != 0) << 3;
        bits |= m << (4 * j);
        const int32_t c = __reduce_add_sync(0xffffffffu, __popc(m));
        if (lane == 0) counts[j * kWarps + warp] = c;
    }
    __syncthreads();
    int32_t live;
    const int32_t mine = tid < kQuads * kWarps ? counts[tid] : 0;
    const int32_t before = block_scan(mine, warp_sums, &live);
    if (tid < kQuads * kWarps) counts[tid] = before;
    if (tid == 0) below_end = live;                        // no page at the end: nothing moves
    __syncthreads();
    int32_t first[kQuads];                                 // L of the quad's first page
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
        const uint32_t m = (bits >> (4 * j)) & 15u;
        int32_t x = __popc(m);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        first[j] = counts[j * kWarps + warp] + x - __popc(m);
        const int32_t at = live - (j * kPlanThreads + tid) * 4;
        if (at >= 0 && at < 4) below_end = first[j] + __popc(m & ((1u << at) - 1u));
    }
    __syncthreads();
    const int32_t stay = below_end;
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
        const uint32_t m = (bits >> (4 * j)) & 15u;
        int32_t L = first[j];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int32_t p = (j * kPlanThreads + tid) * 4 + e;
            const bool is = m >> e & 1u;
            if (p < a.P) {
                if (p < live && !is) a.list[p - L] = p;
                else if (p >= live && is) a.from[L - stay] = p;
                else a.where[p] = -1;
            }
            L += is;
        }
    }
    __syncthreads();
    for (int32_t k = tid; k < live - stay; k += kPlanThreads) {
        const int32_t to = a.list[k], page = a.from[k];
        a.where[page] = to;
        a.where[to] = page;
    }
    if (tid == 0) {
        a.hdr->moved = live - stay;
        a.hdr->live = live;
    }
}

template <int OP>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PagesArgs a)
{
    if (blockIdx.x > 0) {                                  // the counts' copy (out of place only)
        for (int64_t p = (int64_t)(blockIdx.x - 1) * kPlanThreads + threadIdx.x; p < a.P;
             p += (int64_t)(gridDim.x - 1) * kPlanThreads)
            a.refs_out[p] = a.refs[p];
        return;
    }
    __shared__ int32_t counts[kQuads * kWarps];
    __shared__ int32_t warp_sums[33];
    const int tid = threadIdx.x;
    for (int32_t r = tid; r < a.B; r += kPlanThreads) {
        a.old[r] = clamp_len(a, a.lens[r]);
        a.claim[r] = kNone;
    }
    __syncthreads();
    if (OP == kCompact && a.P <= kPassPages) {
        compact_plan(a, counts, warp_sums);
        return;
    }
    if (OP == kCompact) {
        int32_t live = 0;
        for (int32_t b = 0; b < a.P; b += kPassPages)
            live = rank_pass(a, b, 0, a.P, false, live, 0, counts, warp_sums, [](int32_t, int32_t) {});
        int32_t holes = 0, movers = 0;
        for (int32_t b = 0; b < live; b += kPassPages)
            holes = rank_pass(a, b, 0, live, true, holes, a.P, counts, warp_sums,
                              [&](int32_t r, int32_t p) { a.list[r] = p; });
        for (int32_t b = live & ~3; b < a.P; b += kPassPages)
            movers = rank_pass(a, b, live, a.P, false, movers, a.P, counts, warp_sums,
                               [&](int32_t r, int32_t p) { a.from[r] = p; });
        (void)movers;
        __syncthreads();
        for (int32_t p = tid; p < a.P; p += kPlanThreads) a.where[p] = -1;
        __syncthreads();
        for (int32_t k = tid; k < holes; k += kPlanThreads) {
            a.where[a.from[k]] = a.list[k];
            a.where[a.list[k]] = a.from[k];
        }
        if (tid == 0) {
            a.hdr->moved = holes;
            a.hdr->live = live;
        }
        return;
    }
    // which argument acts on which row: the lowest one that is valid
    if (OP != kReserve) {
        for (int32_t i = tid; i < a.n; i += kPlanThreads) {
            const int32_t r = OP == kFork ? a.arg1[i] : a.arg0[i];
            bool ok = r >= 0 && r < a.B;
            if (OP == kFork && ok) {
                const int32_t src = a.arg0[i];
                ok = src >= 0 && src < a.B && a.old[r] == 0;
            }
            if (ok) atomicMin(&a.claim[r], i);
            else flag(a.status, LI_DEV_BAD_ROW);
        }
        __syncthreads();
        if (OP == kFree) {
            for (int32_t i = tid; i < a.n; i += kPlanThreads) {
                const int32_t r = a.arg0[i];
                if (r >= 0 && r < a.B && a.claim[r] != i) flag(a.status, LI_DEV_BAD_ROW);
            }
            return;
        }
    }
    // fresh pages wanted by each row (reserve) or pair (fork), in order
    const int32_t n = OP == kReserve ? a.B : a.n;
    int32_t wanted = 0;
    for (int32_t base = 0; base < n; base += kPlanThreads) {
        const int32_t i = base + tid;
        int32_t need = 0;
        if (i < n) {
            if (OP == kReserve) {
                const int32_t len = clamp_len(a, a.lens[i]), want = a.arg0[i];
                if (want < 0 || want > a.cols * a.ps) flag(a.status, LI_DEV_BAD_KLEN);
                need = growth(a, len, want);
            } else {
                const int32_t r = a.arg1[i];
                if (r >= 0 && r < a.B && a.claim[r] == i) need = clamp_len(a, a.lens[a.arg0[i]]) % a.ps != 0;
                else if (r >= 0 && r < a.B && a.claim[r] != 0x7FFFFFFF) flag(a.status, LI_DEV_BAD_ROW);
            }
        }
        int32_t total;
        // a sum beyond the pool is as good as any other such sum
        const int64_t before = (int64_t)wanted + block_scan(need, warp_sums, &total);
        if (need > 0) {
            const int32_t row = OP == kReserve ? i : a.arg1[i];
            a.grant[row] = before > a.P ? a.P + 1 : (int32_t)before;
        }
        wanted = (int64_t)wanted + total > a.P ? a.P + 1 : wanted + total;
    }
    int32_t found = 0;
    for (int32_t b = 0; b < a.P && found < wanted; b += kPassPages)
        found = rank_pass(a, b, 0, a.P, true, found, wanted < a.P ? wanted : a.P, counts, warp_sums,
                          [&](int32_t r, int32_t p) { a.list[r] = p; });
    if (tid == 0) a.hdr->live = found;                     // fresh pages that exist (those wanted, at least)
}

// The fresh pages of a row: true when they all exist.
__device__ __forceinline__ bool granted(const PagesArgs &a, int32_t row, int32_t need)
{
    return need == 0 || (int64_t)a.grant[row] + need <= a.hdr->live;
}

__device__ __forceinline__ int32_t checked_page(const PagesArgs &a, int32_t page)
{
    if (page >= 0 && page < a.P) return page;
    flag(a.status, LI_DEV_BAD_BLOCK);
    return -1;
}

// Copies `bytes` from src to dst with the threads of one block; V is the
// access type that both are aligned to.
template <typename V>
__device__ __forceinline__ void copy_run(char *dst, const char *src, int64_t bytes)
{
    const V *s = reinterpret_cast<const V *>(src);
    V *d = reinterpret_cast<V *>(dst);
    const int n = (int)(bytes / (int64_t)sizeof(V));
    int i = threadIdx.x;
    for (; i + 3 * kApplyThreads < n; i += 4 * kApplyThreads) {
        const V x0 = __ldcs(s + i), x1 = __ldcs(s + i + kApplyThreads), x2 = __ldcs(s + i + 2 * kApplyThreads),
                x3 = __ldcs(s + i + 3 * kApplyThreads);
        __stcs(d + i, x0);
        __stcs(d + i + kApplyThreads, x1);
        __stcs(d + i + 2 * kApplyThreads, x2);
        __stcs(d + i + 3 * kApplyThreads, x3);
    }
    for (; i < n; i += kApplyThreads) __stcs(d + i, __ldcs(s + i));
}

// Page contents: item = (pair, pool, chunk), dealt to the blocks in turn;
// pair(i, src, dst) names the pages, or says that there is nothing to copy.
template <int N, typename Pair>
__device__ void copy_pages(const Pools<N> &pools, int32_t pairs, Pair pair)
{
    // chunks of one pair, over all pools
    int64_t per_pair = 0;
    for (int k = 0; k < pools.n; ++k) per_pair += (pools.bytes[k] + kChunk - 1) / kChunk;
    const int64_t items = per_pair * pairs;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int32_t i = (int32_t)(it / per_pair);
        int64_t c = it - i * per_pair;
        int k = 0;
        for (;; ++k) {
            const int64_t m = (pools.bytes[k] + kChunk - 1) / kChunk;
            if (c < m) break;
            c -= m;
        }
        int32_t src, dst;
        if (!pair(i, src, dst)) continue;
        const int64_t off = c * kChunk;
        const int64_t bytes = pools.bytes[k] - off < kChunk ? pools.bytes[k] - off : kChunk;
        const char *s = pools.base[k] + src * pools.stride[k] + off;
        char *d = pools.base[k] + dst * pools.stride[k] + off;
        const uintptr_t bits = reinterpret_cast<uintptr_t>(s) | reinterpret_cast<uintptr_t>(d) | (uintptr_t)bytes;
        if ((bits & 15) == 0) copy_run<uint4>(d, s, bytes);
        else if ((bits & 3) == 0) copy_run<uint32_t>(d, s, bytes);
        else copy_run<char>(d, s, bytes);
    }
}

// TABLES: write the new table, lengths and counts (the first launch of a call
// does; further ones only copy the pools that did not fit into it).
template <int OP, bool TABLES, int N>
__global__ void __launch_bounds__(kApplyThreads) apply_kernel(const PagesArgs a, const __grid_constant__ Pools<N> pools)
{
    grid_dependency_wait();
    const int64_t t0 = (int64_t)blockIdx.x * kApplyThreads + threadIdx.x, step = (int64_t)gridDim.x * kApplyThreads;
    const bool same_table = a.table == a.table_out;
    if (TABLES) {
        const uint32_t entries = (uint32_t)(a.B * a.cols);       // < 2^31
        for (uint32_t e = (uint32_t)t0; e < entries; e += (uint32_t)step) {
            const int32_t r = (int32_t)(e / (uint32_t)a.cols), c = (int32_t)(e - (uint32_t)r * (uint32_t)a.cols);
            const int32_t len = a.old[r];
            int32_t new_len = len;
            bool write = !same_table;
            int32_t page = -1;
            if (OP == kReserve) {
                const int32_t had = pages_of(len, a.ps), want = a.arg0[r], need = growth(a, len, want);
                if (granted(a, r, need)) {
                    if (want > len && want <= a.cols * a.ps) new_len = want;
                    if (c >= had && c < had + need) {
                        page = a.list[a.grant[r] + c - had];
                        a.refs_out[page] = 1;
                        a.table_out[e] = page;
                        write = false;
                    }
                } else if (c == 0) {
                    flag(a.status, LI_DEV_NO_PAGES);
                }
            } else if (OP == kFork) {
                const int32_t i = a.claim[r];
                if (i != kNone) {
                    const int32_t src = a.arg0[i], from = a.old[src], need = from % a.ps != 0, full = from / a.ps;
                    if (granted(a, r, need)) {
                        new_len = from;
                        if (c < full) page = checked_page(a, a.table[(int64_t)src * a.cols + c]);
                        else if (c == full && need) {
                            checked_page(a, a.table[(int64_t)src * a.cols + c]);      // flagged, with or without pools
                            page = a.list[a.grant[r]];
                        }
                        if (page >= 0) atomicAdd(&a.refs_out[page], 1);
                        a.table_out[e] = page;
                        write = false;
                    } else if (c == 0) {
                        flag(a.status, LI_DEV_NO_PAGES);
                    }
                }
            } else if (OP == kFree) {
                if (a.claim[r] != kNone) {
                    new_len = 0;
                    if (c < pages_of(len, a.ps)) {
                        page = checked_page(a, a.table[e]);
                        if (page >= 0 && atomicSub(&a.refs_out[page], 1) <= 0) {
                            atomicAdd(&a.refs_out[page], 1);
                            flag(a.status, LI_DEV_BAD_BLOCK);
                        }
                    }
                    a.table_out[e] = -1;
                    write = false;
                }
            } else {
                if (c < pages_of(len, a.ps)) {
                    page = checked_page(a, a.table[e]);
                    if (page >= 0) {
                        // a live page is a mover, or below the live pages' end and no hole
                        const int32_t to = a.where[page];
                        const bool moves = page >= a.hdr->live;
                        if (moves != (to >= 0)) flag(a.status, LI_DEV_BAD_BLOCK);
                        page = moves ? to : (to >= 0 ? -1 : page);
                    }
                }
                a.table_out[e] = page;
                write = false;
            }
            if (write) a.table_out[e] = a.table[e];
            if (c == 0) a.lens_out[r] = new_len;
        }
        if (OP == kCompact) {
            const int32_t live = a.hdr->live;
            for (int64_t p = t0; p < a.P; p += step) {
                const int32_t ref = a.refs[p];
                if (p < live) {
                    if (ref == 0) {                        // a hole: its mover's count, and the mover's page is free
                        const int32_t m = a.where[p];
                        a.refs_out[p] = a.refs[m];
                        a.refs_out[m] = 0;
                    } else if (a.refs != a.refs_out) {
                        a.refs_out[p] = ref;
                    }
                } else if (ref == 0) {
                    a.refs_out[p] = 0;
                }
            }
        }
    }
    if (OP == kCompact) {
        copy_pages(pools, a.hdr->moved, [&](int32_t i, int32_t &src, int32_t &dst) {
            src = a.from[i];
            dst = a.list[i];
            return true;
        });
    } else if (OP == kFork) {
        copy_pages(pools, a.n, [&](int32_t i, int32_t &src, int32_t &dst) {
            const int32_t r = a.arg1[i];
            if (r < 0 || r >= a.B || a.claim[r] != i) return false;
            const int32_t len = a.old[a.arg0[i]];
            if (len % a.ps == 0 || !granted(a, r, 1)) return false;
            src = a.table[(int64_t)a.arg0[i] * a.cols + len / a.ps];
            dst = a.list[a.grant[r]];
            if (src < 0 || src >= a.P) {
                if (threadIdx.x == 0) flag(a.status, LI_DEV_BAD_BLOCK);
                return false;
            }
            return true;
        });
    }
}

// Pages by explicit number.
__global__ void __launch_bounds__(kApplyThreads) copy_kernel(const int32_t *src_pages, const int32_t *dst_pages,
                                                             int32_t n, int32_t P, int32_t *status,
                                                             const __grid_constant__ Pools<kMaxPools> pools)
{
    copy_pages(pools, n, [&](int32_t i, int32_t &src, int32_t &dst) {
        src = src_pages[i];
        dst = dst_pages[i];
        if (src < 0 || src >= P || dst < 0 || dst >= P) {
            if (threadIdx.x == 0) flag(status, LI_DEV_BAD_BLOCK);
            return false;
        }
        return src != dst;
    });
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

struct Carve {
    size_t claim, old, grant, list, from, where, total;
};

Carve carve(const li_pages_params &p)
{
    Carve c{};
    size_t off = sizeof(Header);
    const size_t rows = up((size_t)p.B * 4), pages = up((size_t)p.num_pages * 4);
    c.claim = off;
    c.old = off += rows;
    c.grant = off += rows;
    c.list = off += rows;
    c.from = off += pages;
    c.where = off += pages;
    c.total = off + pages;
    return c;
}

li_status bad(const char *call, li_status st, const char *what)
{
    char msg[200];
    snprintf(msg, sizeof msg, "%s: %s", call, what);
    return li::report_error(st, msg);
}

li_status check_params(const char *call, const li_pages_params *p)
{
    if (!p) return bad(call, LI_ERR_NULL, "params is NULL");
    if (p->reserved != 0) return bad(call, LI_ERR_SHAPE, "reserved must be 0");
    if (p->num_pages < 1 || p->num_pages > (1 << 26)) return bad(call, LI_ERR_SHAPE, "num_pages must be in [1, 2^26]");
    if (p->page_size < 1 || p->max_pages_per_seq < 1 || p->B < 1)
        return bad(call, LI_ERR_SHAPE, "page_size, max_pages_per_seq and B must be >= 1");
    if ((int64_t)p->max_pages_per_seq * p->page_size > 0x7FFFFFFF || (int64_t)p->B * p->max_pages_per_seq > 0x7FFFFFFF)
        return bad(call, LI_ERR_SHAPE, "max_pages_per_seq * page_size and B * max_pages_per_seq must fit int32");
    return LI_OK;
}

li_status check_pools(const char *call, const li_page_pool *pools, int32_t n)
{
    if (n < 0 || n > kMaxPoolsCall) return bad(call, LI_ERR_SHAPE, "n_pools must be in [0, 256]");
    if (n > 0 && !pools) return bad(call, LI_ERR_NULL, "pools is NULL");
    for (int k = 0; k < n; ++k) {
        if (!pools[k].base) return bad(call, LI_ERR_NULL, "a pool's base is NULL");
        if (pools[k].page_bytes < 1 || pools[k].page_bytes > ((int64_t)1 << 40) || pools[k].page_stride < pools[k].page_bytes ||
            pools[k].page_stride > ((int64_t)1 << 40))
            return bad(call, LI_ERR_SHAPE, "a pool needs 1 <= page_bytes <= page_stride");
    }
    return LI_OK;
}

template <int N>
Pools<N> some_pools(const li_page_pool *pools, int32_t from, int32_t n, int64_t *chunks)
{
    Pools<N> out{};
    out.n = n - from < N ? n - from : N;
    *chunks = 0;
    for (int k = 0; k < out.n; ++k) {
        out.base[k] = static_cast<char *>(pools[from + k].base);
        out.bytes[k] = pools[from + k].page_bytes;
        out.stride[k] = pools[from + k].page_stride;
        *chunks += (out.bytes[k] + kChunk - 1) / kChunk;
    }
    return out;
}

int sm_count()
{
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

template <int OP, int N>
cudaError_t launch_apply(const PagesArgs &a, const li_page_pool *pools, int32_t n_pools, int sms, cudaStream_t s, int *launches)
{
    cudaError_t e = cudaSuccess;
    for (int32_t from = 0; e == cudaSuccess && (from == 0 || from < n_pools); from += N) {
        int64_t chunks;
        const Pools<N> some = some_pools<N>(pools, from, n_pools, &chunks);
        int64_t blocks = from == 0 ? ((int64_t)a.B * a.cols + kApplyThreads - 1) / kApplyThreads : 1;
        if (OP == kCompact && from == 0) {
            const int64_t m = ((int64_t)a.P + kApplyThreads - 1) / kApplyThreads;
            if (blocks < m) blocks = m;
        }
        const int64_t items = chunks * (OP == kCompact ? a.P / 2 : OP == kFork ? a.n : 0);
        if (blocks < items) blocks = items;
        if (blocks > 8LL * sms) blocks = 8LL * sms;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(blocks < 1 ? 1 : blocks));
        cfg.blockDim = dim3(kApplyThreads);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = from == 0 ? cudaLaunchKernelEx(&cfg, apply_kernel<OP, true, N>, a, some)
                      : cudaLaunchKernelEx(&cfg, apply_kernel<OP, false, N>, a, some);
        ++*launches;
    }
    return e;
}

template <int OP>
cudaError_t launch(const PagesArgs &a, const li_page_pool *pools, int32_t n_pools, cudaStream_t s, int *launches)
{
    const int sms = sm_count();
    int copy_blocks = 0;
    if (OP != kCompact && a.refs != a.refs_out) {
        copy_blocks = (a.P + kPlanThreads - 1) / kPlanThreads;
        if (copy_blocks > sms - 1) copy_blocks = sms - 1;
    }
    plan_kernel<OP><<<1 + copy_blocks, kPlanThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    *launches = 1;
    if (e != cudaSuccess) return e;
    return n_pools <= kFewPools ? launch_apply<OP, kFewPools>(a, pools, n_pools, sms, s, launches)
                                : launch_apply<OP, kMaxPools>(a, pools, n_pools, sms, s, launches);
}

// Checks shared by the calls that change the state, then the launches.
template <int OP>
li_status run(const char *call, const li_pages_params *p, const li_page_pool *pools, int32_t n_pools,
              const int32_t *table, const int32_t *lens, const int32_t *refs, const int32_t *arg0, const int32_t *arg1,
              int32_t n, int32_t *table_out, int32_t *lens_out, int32_t *refs_out, int32_t *status, void *workspace,
              size_t workspace_bytes, void *stream)
{
    li::set_launch_count(0);
    li_status st = check_params(call, p);
    if (st == LI_OK) st = check_pools(call, pools, n_pools);
    if (st != LI_OK) return st;
    if (!table || !lens || !refs || !table_out || !lens_out || !refs_out)
        return bad(call, LI_ERR_NULL, "table, lens, refs and their outputs are required");
    if (n < 0) return bad(call, LI_ERR_SHAPE, "n must be >= 0");
    if ((OP == kReserve && !arg0) || ((OP == kFork || OP == kFree) && n > 0 && (!arg0 || (OP == kFork && !arg1))))
        return bad(call, LI_ERR_NULL, "the rows acted on are required");
    const uintptr_t bits = reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(lens) |
                           reinterpret_cast<uintptr_t>(refs) | reinterpret_cast<uintptr_t>(table_out) |
                           reinterpret_cast<uintptr_t>(lens_out) | reinterpret_cast<uintptr_t>(refs_out) |
                           reinterpret_cast<uintptr_t>(arg0) | reinterpret_cast<uintptr_t>(arg1) |
                           reinterpret_cast<uintptr_t>(status);
    if (bits % 4) return bad(call, LI_ERR_SHAPE, "int32 pointers must be 4-byte aligned");
    const Carve c = carve(*p);
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < c.total)
        return bad(call, LI_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or smaller than li_pages_workspace_size");
    PagesArgs a{};
    char *ws = static_cast<char *>(workspace);
    a.table = table;
    a.lens = lens;
    a.refs = refs;
    a.table_out = table_out;
    a.lens_out = lens_out;
    a.refs_out = refs_out;
    a.arg0 = arg0;
    a.arg1 = arg1;
    a.hdr = reinterpret_cast<Header *>(ws);
    a.claim = reinterpret_cast<int32_t *>(ws + c.claim);
    a.old = reinterpret_cast<int32_t *>(ws + c.old);
    a.grant = reinterpret_cast<int32_t *>(ws + c.grant);
    a.list = reinterpret_cast<int32_t *>(ws + c.list);
    a.from = reinterpret_cast<int32_t *>(ws + c.from);
    a.where = reinterpret_cast<int32_t *>(ws + c.where);
    a.status = status;
    a.P = p->num_pages;
    a.ps = p->page_size;
    a.cols = p->max_pages_per_seq;
    a.B = p->B;
    a.n = n;
    int launches = 0;
    const cudaError_t e = launch<OP>(a, pools, n_pools, static_cast<cudaStream_t>(stream), &launches);
    if (e != cudaSuccess) return bad(call, LI_ERR_CUDA, cudaGetErrorString(e));
    li::set_launch_count(launches);
    return LI_OK;
}

}  // namespace

extern "C" LI_API li_status li_pages_workspace_size(const li_pages_params *p, size_t *bytes)
{
    const li_status st = check_params("li_pages_workspace_size", p);
    if (st != LI_OK) return st;
    if (!bytes) return bad("li_pages_workspace_size", LI_ERR_NULL, "bytes is NULL");
    *bytes = carve(*p).total;
    return LI_OK;
}

extern "C" LI_API li_status li_pages_copy(const li_pages_params *p, const li_page_pool *pools, int32_t n_pools,
                                          const int32_t *src_pages, const int32_t *dst_pages, int32_t n,
                                          int32_t *status, void *stream)
{
    const char *call = "li_pages_copy";
    li::set_launch_count(0);
    li_status st = check_params(call, p);
    if (st == LI_OK) st = check_pools(call, pools, n_pools);
    if (st != LI_OK) return st;
    if (n < 0) return bad(call, LI_ERR_SHAPE, "n must be >= 0");
    if (n == 0 || n_pools == 0) return LI_OK;
    if (!src_pages || !dst_pages) return bad(call, LI_ERR_NULL, "src_pages and dst_pages are required");
    if ((reinterpret_cast<uintptr_t>(src_pages) | reinterpret_cast<uintptr_t>(dst_pages) |
         reinterpret_cast<uintptr_t>(status)) % 4)
        return bad(call, LI_ERR_SHAPE, "int32 pointers must be 4-byte aligned");
    const int sms = sm_count();
    int launches = 0;
    for (int32_t from = 0; from < n_pools; from += kMaxPools) {
        int64_t chunks;
        const Pools<kMaxPools> some = some_pools<kMaxPools>(pools, from, n_pools, &chunks);
        const int64_t items = chunks * n, blocks = items < 8LL * sms ? items : 8LL * sms;
        copy_kernel<<<(unsigned)blocks, kApplyThreads, 0, static_cast<cudaStream_t>(stream)>>>(
            src_pages, dst_pages, n, p->num_pages, status, some);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return bad(call, LI_ERR_CUDA, cudaGetErrorString(e));
        ++launches;
    }
    li::set_launch_count(launches);
    return LI_OK;
}

extern "C" LI_API li_status li_pages_reserve(const li_pages_params *p, const int32_t *table, const int32_t *lens,
                                             const int32_t *refs, const int32_t *new_lens, int32_t *table_out,
                                             int32_t *lens_out, int32_t *refs_out, int32_t *status, void *workspace,
                                             size_t workspace_bytes, void *stream)
{
    return run<kReserve>("li_pages_reserve", p, nullptr, 0, table, lens, refs, new_lens, nullptr, 0, table_out, lens_out,
                         refs_out, status, workspace, workspace_bytes, stream);
}

extern "C" LI_API li_status li_pages_fork(const li_pages_params *p, const li_page_pool *pools, int32_t n_pools,
                                          const int32_t *table, const int32_t *lens, const int32_t *refs,
                                          const int32_t *src_rows, const int32_t *dst_rows, int32_t n,
                                          int32_t *table_out, int32_t *lens_out, int32_t *refs_out, int32_t *status,
                                          void *workspace, size_t workspace_bytes, void *stream)
{
    return run<kFork>("li_pages_fork", p, pools, n_pools, table, lens, refs, src_rows, dst_rows, n, table_out, lens_out,
                      refs_out, status, workspace, workspace_bytes, stream);
}

extern "C" LI_API li_status li_pages_free(const li_pages_params *p, const int32_t *table, const int32_t *lens,
                                          const int32_t *refs, const int32_t *rows, int32_t n, int32_t *table_out,
                                          int32_t *lens_out, int32_t *refs_out, int32_t *status, void *workspace,
                                          size_t workspace_bytes, void *stream)
{
    return run<kFree>("li_pages_free", p, nullptr, 0, table, lens, refs, rows, nullptr, n, table_out, lens_out, refs_out,
                      status, workspace, workspace_bytes, stream);
}

extern "C" LI_API li_status li_pages_compact(const li_pages_params *p, const li_page_pool *pools, int32_t n_pools,
                                             const int32_t *table, const int32_t *lens, const int32_t *refs,
                                             int32_t *table_out, int32_t *lens_out, int32_t *refs_out, int32_t *status,
                                             void *workspace, size_t workspace_bytes, void *stream)
{
    return run<kCompact>("li_pages_compact", p, pools, n_pools, table, lens, refs, nullptr, nullptr, 0, table_out,
                         lens_out, refs_out, status, workspace, workspace_bytes, stream);
}
