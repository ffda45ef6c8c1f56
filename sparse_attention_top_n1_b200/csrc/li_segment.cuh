// li_segment.cuh -- geometry shared by the segment kernels (pool, select,
// attention): which batch and position a query row has, how many keys it sees,
// and where a key lies.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "li.h"

namespace li {

struct SegGeo {
    const int32_t *act_q, *act_k, *block_table;
    int32_t *status;
    int32_t layout_q, layout_kv;
    int32_t B, S1, S2, T1, T2;
    int32_t N1, N2, G;
    int32_t num_blocks, block_size, max_blocks_per_seq;
    int32_t bs_shift;                      // log2(block_size), or -1
    int32_t seg, count, init, local, max_segs, mode;
    int64_t page_stride;                   // elements between pages
    int32_t rows;
};

struct SegRow {
    int32_t b, i, Sq, Sk;
    int32_t vis;                           // keys that the row sees (0: padding row)
    int64_t k_off;                         // first key row of the batch (BSND / TND)
};

__device__ __forceinline__ int32_t seg_clamp(int64_t v, int64_t lo, int64_t hi)
{
    return (int32_t)(v < lo ? lo : (v > hi ? hi : v));
}

__device__ __forceinline__ void seg_flag(const SegGeo &g, int32_t bit)
{
    if (g.status) atomicOr(g.status, bit);
}

// Keys of batch b: their number and the first one's row.
__device__ __forceinline__ int32_t seg_keys(const SegGeo &g, int32_t b, int64_t &k_off)
{
    if (g.layout_kv == LI_BSND) {
        k_off = (int64_t)b * g.S2;
        return g.act_k ? seg_clamp(g.act_k[b], 0, g.S2) : g.S2;
    }
    if (g.layout_kv == LI_TND) {
        const int32_t start = b ? seg_clamp(g.act_k[b - 1], 0, g.T2) : 0;
        k_off = start;
        return seg_clamp(g.act_k[b], start, g.T2) - start;
    }
    k_off = 0;
    return seg_clamp(g.act_k[b], 0, (int64_t)g.max_blocks_per_seq * g.block_size);
}

__device__ __forceinline__ SegRow seg_row(const SegGeo &g, int32_t row)
{
    SegRow r;
    if (g.layout_q == LI_BSND) {
        r.b = row / g.S1;
        r.i = row - r.b * g.S1;
        r.Sq = g.act_q ? seg_clamp(g.act_q[r.b], 0, g.S1) : g.S1;
    } else {                               // prefix sums without a leading 0
        int lo = 0, hi = g.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (seg_clamp(g.act_q[mid], 0, g.T1) > row) hi = mid;
            else lo = mid + 1;
        }
        r.b = lo;
        const int32_t start = lo ? seg_clamp(g.act_q[lo - 1], 0, g.T1) : 0;
        r.i = row - start;
        r.Sq = seg_clamp(g.act_q[lo], start, g.T1) - start;
    }
    r.Sk = seg_keys(g, r.b, r.k_off);
    if (r.i < 0 || r.i >= r.Sq) r.vis = 0;
    else r.vis = g.mode == 0 ? r.Sk : seg_clamp((int64_t)r.i + 1 + r.Sk - r.Sq, 0, r.Sk);
    return r;
}

// Element offset of key t of batch b in the key and value tensors (head 0), or
// -1 (flagged) behind a bad block id.
__device__ __forceinline__ int64_t seg_key_offset(const SegGeo &g, int32_t b, int64_t k_off, int32_t t, int32_t row_elems)
{
    if (g.layout_kv != LI_PA_BSND) return (k_off + t) * row_elems;
    const int32_t pg = g.bs_shift >= 0 ? t >> g.bs_shift : t / g.block_size;
    const int32_t in = g.bs_shift >= 0 ? t & (g.block_size - 1) : t - pg * g.block_size;
    const int32_t id = g.block_table[(int64_t)b * g.max_blocks_per_seq + pg];
    if (id < 0 || id >= g.num_blocks) {
        seg_flag(g, LI_DEV_BAD_BLOCK);
        return -1;
    }
    return id * g.page_stride + (int64_t)in * row_elems;
}

// Checks the parameters that the three calls share and fills the geometry.
// `queries`: the call has query rows.  Returns LI_OK or reports `call`: reason.
li_status seg_setup(const char *call, const li_segment_params *p, bool queries, bool keys, const int32_t *act_q,
                    const int32_t *act_k, const int32_t *block_table, int32_t *status, SegGeo *g);
li_status seg_fail(const char *call, li_status st, const char *what);
// The key tensor has no elements (and, in torch, no address).
inline bool seg_no_keys(const SegGeo &g)
{
    return (g.layout_kv == LI_BSND && g.S2 == 0) || (g.layout_kv == LI_TND && g.T2 == 0);
}
int seg_sms();
// A tensor map over 16-bit elements with the 128-byte swizzle; zeros outside.
li_status tensor_map_16bit(CUtensorMap *m, const void *base, int rank, const uint64_t *dims, const uint64_t *strides_bytes,
                           const uint32_t *box, const char *what);
}  // namespace li
