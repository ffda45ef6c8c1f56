// li_segattn.cu -- attention over the selected segments.
#include <cmath>
#include <cstdio>

#include "li_segment.cuh"

namespace li {
void set_launch_count(int32_t n);
}  // namespace li

namespace {

using namespace li;

struct AttnArgs {
    SegGeo g;
    const uint16_t *q, *k, *v;
    const int32_t *idx;
    uint16_t *out;
    float *lse;
    float scale;
};

// One block per (row, query head): the threads take a key each, then a column
// each, segment by segment with a running maximum and sum.
template <int D, bool F16>
__global__ void __launch_bounds__(128) segattn_simple(const AttnArgs a)
{
    __shared__ float sq[D];
    __shared__ float sw[1024];
    __shared__ int64_t sat[1024];
    __shared__ float red[4];
    const SegGeo &g = a.g;
    const int32_t row = blockIdx.x, h = blockIdx.y, n = h / g.G, tid = threadIdx.x;
    const int32_t row_elems = g.N2 * D;
    const SegRow r = seg_row(g, row);
    auto at16 = [](const uint16_t *p, int64_t i) {
        const uint32_t w = p[i];
        return seg_lo<F16>(w);
    };
    for (int c = tid; c < D; c += 128) sq[c] = at16(a.q, ((int64_t)row * g.N1 + h) * D + c);
    __syncthreads();
    float m = -INFINITY, l = 0.f, acc = 0.f;
    int32_t last = -1;
    const int32_t segs = (int32_t)(((int64_t)r.Sk + g.seg - 1) / g.seg);
    for (int32_t e = 0; e < (r.vis > 0 ? g.count : 0); ++e) {
        const int32_t s = a.idx[((int64_t)row * g.N2 + n) * g.count + e];
        if (s == -1) continue;
        if (s < 0 || s >= segs || s <= last) {
            if (tid == 0) seg_flag(g, LI_DEV_BAD_INDEX);
            continue;
        }
        last = s;
        const int32_t t0 = s * g.seg, cnt = r.vis - t0 < g.seg ? r.vis - t0 : g.seg;
        if (cnt <= 0) continue;
        float mx = -INFINITY;
        for (int32_t t = tid; t < cnt; t += 128) {
            const int64_t at = seg_key_offset(g, r.b, r.k_off, t0 + t, row_elems);
            float x = -INFINITY;
            if (at >= 0) {
                x = 0.f;
                for (int c = 0; c < D; ++c) x = fmaf(sq[c], at16(a.k, at + n * D + c), x);
                x *= a.scale;
            }
            sw[t] = x;
            sat[t] = at;
            mx = fmaxf(mx, x);
        }
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if ((tid & 31) == 0) red[tid >> 5] = mx;
        __syncthreads();
        const float top = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        if (top > -INFINITY) {
            const float alpha = m == -INFINITY ? 0.f : expf(m - top);
            m = top;
            l *= alpha;
            acc *= alpha;
            for (int32_t t = 0; t < cnt; ++t) {
                if (sat[t] < 0) continue;
                const float w = expf(sw[t] - m);
                l += w;
                if (tid < D) acc = fmaf(w, at16(a.v, sat[t] + n * D + tid), acc);
            }
        }
        __syncthreads();
    }
    if (tid < D) {
        const float o = l == 0.f ? 0.f : acc / l;
        const int64_t at = ((int64_t)row * g.N1 + h) * D + tid;
        if constexpr (F16) a.out[at] = __half_as_ushort(__float2half_rn(o));
        else a.out[at] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
    }
    if (tid == 0 && a.lse) a.lse[(int64_t)row * g.N1 + h] = l == 0.f ? -INFINITY : m + logf(l);
}

bool off(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

}  // namespace

extern "C" LI_API li_status li_segment_attention(const li_segment_params *p, const void *query, const void *key,
                                                 const void *value, const int32_t *seg_idx, const int32_t *act_seq_q,
                                                 const int32_t *act_seq_k, const int32_t *block_table, void *out,
                                                 float *lse, int32_t *status, void *stream)
{
    const char *call = "li_segment_attention";
    AttnArgs a{};
    const li_status st = seg_setup(call, p, true, true, act_seq_q, act_seq_k, block_table, status, &a.g);
    if (st != LI_OK) return st;
    if (!query || !key || !value || !seg_idx || !out)
        return seg_fail(call, LI_ERR_NULL, "query, key, value, seg_idx and out are required");
    if (off(query, 16) || off(key, 16) || off(value, 16) || off(out, 16) || off(seg_idx, 4) || off(lse, 4))
        return seg_fail(call, LI_ERR_SHAPE, "query, key, value and out must be 16-byte aligned, seg_idx and lse 4-byte");
    if (a.g.rows == 0) return LI_OK;
    a.q = static_cast<const uint16_t *>(query);
    a.k = static_cast<const uint16_t *>(key);
    a.v = static_cast<const uint16_t *>(value);
    a.idx = seg_idx;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.scale = p->softmax_scale;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f16 = p->dtype == LI_FP16;
    const dim3 grid((unsigned)a.g.rows, (unsigned)p->N1);
    if (p->D == 128) {
        if (f16) segattn_simple<128, true><<<grid, 128, 0, s>>>(a);
        else segattn_simple<128, false><<<grid, 128, 0, s>>>(a);
    } else {
        if (f16) segattn_simple<64, true><<<grid, 128, 0, s>>>(a);
        else segattn_simple<64, false><<<grid, 128, 0, s>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return seg_fail(call, LI_ERR_CUDA, cudaGetErrorString(e));
    li::set_launch_count(1);
    return LI_OK;
}
