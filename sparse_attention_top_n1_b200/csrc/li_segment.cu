// li_segment.cu -- the cheap score of segment-sparse attention: the mean key of
// each segment (pool) and the choice of segments for each query row (select).
#include <cooperative_groups.h>

#include <cmath>
#include <cstdio>

#include "attn_common.cuh"
#include "li_segment.cuh"

namespace li {
li_status report_error(li_status s, const char *msg);
void set_launch_count(int32_t n);
cudaError_t set_max_dynamic_smem(const void *kern, int bytes);

li_status seg_fail(const char *call, li_status st, const char *what)
{
    char msg[240];
    snprintf(msg, sizeof msg, "%s: %s", call, what);
    return report_error(st, msg);
}

int seg_sms()
{
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

li_status seg_setup(const char *call, const li_segment_params *p, bool queries, bool keys, const int32_t *act_q,
                    const int32_t *act_k, const int32_t *block_table, int32_t *status, SegGeo *g)
{
    auto bad = [&](li_status st, const char *what) { return seg_fail(call, st, what); };
    set_launch_count(0);
    if (!p) return bad(LI_ERR_NULL, "params is NULL");
    if (p->reserved != 0) return bad(LI_ERR_SHAPE, "reserved must be 0");
    if (p->dtype != LI_BF16 && p->dtype != LI_FP16) return bad(LI_ERR_DTYPE, "dtype must be LI_BF16 or LI_FP16");
    if (p->layout_q != LI_BSND && p->layout_q != LI_TND) return bad(LI_ERR_LAYOUT, "layout_q must be BSND or TND");
    if (p->layout_kv != LI_PA_BSND && p->layout_kv != p->layout_q)
        return bad(LI_ERR_LAYOUT, "layout_kv must equal layout_q or be PA_BSND");
    if (p->B < 1) return bad(LI_ERR_SHAPE, "B must be >= 1");
    if (p->N2 < 1 || p->N1 < 1 || p->N1 > 1024 || p->N1 % p->N2 || p->N1 / p->N2 > 128)
        return bad(LI_ERR_SHAPE, "N2 must divide N1, N1 <= 1024 and N1/N2 <= 128");
    if (p->D != 64 && p->D != 128) return bad(LI_ERR_UNSUPPORTED, "D must be 64 or 128");
    if (p->seg_size < 16 || p->seg_size > 1024 || p->seg_size % 16)
        return bad(LI_ERR_SHAPE, "seg_size must be a multiple of 16 in [16, 1024]");
    if (p->seg_count < 1 || p->seg_count > 1024) return bad(LI_ERR_SHAPE, "seg_count must be in [1, 1024]");
    if (p->init_segs < 0 || p->local_segs < 0 || (int64_t)p->init_segs + p->local_segs > p->seg_count)
        return bad(LI_ERR_SHAPE, "init_segs and local_segs must be >= 0 and together at most seg_count");
    if (p->sparse_mode != 0 && p->sparse_mode != 3) return bad(LI_ERR_SHAPE, "sparse_mode must be 0 or 3");
    if (p->sparse_mode == 3 && p->local_segs < 1) return bad(LI_ERR_SHAPE, "sparse_mode 3 needs local_segs >= 1");
    if (p->max_segs < 1 || p->max_segs > 16384) return bad(LI_ERR_SHAPE, "max_segs must be in [1, 16384]");
    if (!(p->softmax_scale > 0.f) || !std::isfinite(p->softmax_scale))
        return bad(LI_ERR_SHAPE, "softmax_scale must be positive and finite");
    int64_t rows = 0;
    if (p->layout_q == LI_BSND) {
        if (p->S1 < 0) return bad(LI_ERR_SHAPE, "S1 must be >= 0");
        rows = (int64_t)p->B * p->S1;
    } else {
        if (p->T1 < 0) return bad(LI_ERR_SHAPE, "T1 must be >= 0");
        if (queries && !act_q) return bad(LI_ERR_NULL, "TND needs act_seq_q");
        rows = p->T1;
    }
    if (rows * p->N1 > 0x7FFFFFFF) return bad(LI_ERR_SHAPE, "query rows x heads exceed int32");
    g->page_stride = 0;
    g->bs_shift = -1;
    int64_t key_rows = 0;
    if (p->layout_kv == LI_BSND) {
        if (p->S2 < 0) return bad(LI_ERR_SHAPE, "S2 must be >= 0");
        key_rows = (int64_t)p->B * p->S2;
    } else if (p->layout_kv == LI_TND) {
        if (p->T2 < 0) return bad(LI_ERR_SHAPE, "T2 must be >= 0");
        if (!act_k) return bad(LI_ERR_NULL, "TND needs act_seq_k");
        key_rows = p->T2;
    } else {
        if (!act_k || (keys && !block_table)) return bad(LI_ERR_NULL, "PA_BSND needs act_seq_k and block_table");
        if (p->num_blocks < 1 || p->max_blocks_per_seq < 1 || p->block_size < 16 || p->block_size % 16)
            return bad(LI_ERR_SHAPE, "PA needs num_blocks, max_blocks_per_seq >= 1 and block_size a multiple of 16");
        if ((int64_t)p->max_blocks_per_seq * p->block_size > 0x7FFFFFFF)
            return bad(LI_ERR_SHAPE, "paged key capacity exceeds int32");
        const int64_t dense = (int64_t)p->block_size * p->N2 * p->D;
        g->page_stride = p->kv_block_stride ? p->kv_block_stride : dense;
        if (g->page_stride < dense || g->page_stride % 8 || g->page_stride > ((int64_t)1 << 38))
            return bad(LI_ERR_SHAPE, "kv_block_stride must be 0, or a multiple of 8 of at least one page");
        key_rows = (int64_t)p->num_blocks * p->block_size;
        if ((p->block_size & (p->block_size - 1)) == 0) {
            g->bs_shift = 0;
            while ((1 << g->bs_shift) < p->block_size) ++g->bs_shift;
        }
    }
    if (key_rows > 0x7FFFFFFF) return bad(LI_ERR_SHAPE, "more than 2^31-1 key rows");
    const uintptr_t bits = reinterpret_cast<uintptr_t>(act_q) | reinterpret_cast<uintptr_t>(act_k) |
                           reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(status);
    if (bits % 4) return bad(LI_ERR_SHAPE, "int32 pointers must be 4-byte aligned");
    g->act_q = act_q;
    g->act_k = act_k;
    g->block_table = block_table;
    g->status = status;
    g->layout_q = p->layout_q;
    g->layout_kv = p->layout_kv;
    g->B = p->B;
    g->S1 = p->S1;
    g->S2 = p->S2;
    g->T1 = p->T1;
    g->T2 = p->T2;
    g->N1 = p->N1;
    g->N2 = p->N2;
    g->G = p->N1 / p->N2;
    g->num_blocks = p->num_blocks;
    g->block_size = p->block_size;
    g->max_blocks_per_seq = p->max_blocks_per_seq;
    g->seg = p->seg_size;
    g->count = p->seg_count;
    g->init = p->init_segs;
    g->local = p->local_segs;
    g->max_segs = p->max_segs;
    g->mode = p->sparse_mode;
    g->rows = (int32_t)rows;
    return LI_OK;
}
}  // namespace li

namespace {

using namespace li;

constexpr int kPoolThreads = 256;
constexpr int kSelThreads = 256;
constexpr int kSelRows = 32;               // most query rows of one select block
constexpr int kSelSplit = 8;               // most blocks of a cluster that shares a row's segments

// ---------------------------------------------------------------------- pool

// The mean of a segment is one pass over its keys: the block's threads stand
// as tx (16 bytes of the N2*D columns) by ty (a token of every `ty_n`), sum in
// fp32 and meet in shared memory.  Bound by HBM, each key is read once: 52 MB in
// 9.7 us when they come from L2, 16.5 us from HBM (8 us at its rate; the whole is
// one wave of loads).  512 threads per block 18.5 us, loads marked as used once
// 15.7 us, which is not taken: the attention reads the keys next.
template <bool F16>
__global__ void __launch_bounds__(kPoolThreads) pool_kernel(const SegGeo g, const uint16_t *key, const int32_t *first,
                                                            float *pooled, int32_t D, int32_t tx_n)
{
    __shared__ float part[kPoolThreads * 8];
    __shared__ int32_t seen_by[kPoolThreads];
    const int32_t b = blockIdx.y, row_elems = g.N2 * D;
    const int tx = threadIdx.x % tx_n, ty = threadIdx.x / tx_n, ty_n = kPoolThreads / tx_n;
    const int32_t col = ((int)blockIdx.z * tx_n + tx) * 8;
    const bool on = ty < ty_n && col < row_elems;
    int64_t k_off;
    const int32_t Sk = seg_keys(g, b, k_off);
    int32_t segs = (int32_t)(((int64_t)Sk + g.seg - 1) / g.seg);
    if (segs > g.max_segs) {
        segs = g.max_segs;
        if (threadIdx.x == 0) seg_flag(g, LI_DEV_BAD_KLEN);
    }
    int32_t s0 = 0;
    if (first) {
        const int32_t f = first[b];
        s0 = f < 0 ? 0 : f / g.seg;
    }
    for (int32_t s = s0 + (int32_t)blockIdx.x; s < segs; s += gridDim.x) {
        const int32_t t0 = s * g.seg, n = Sk - t0 < g.seg ? Sk - t0 : g.seg;
        float acc[8] = {};
        int32_t seen = 0;
        if (on) {
#pragma unroll 8
            for (int32_t t = ty; t < n; t += ty_n) {
                const int64_t at = seg_key_offset(g, b, k_off, t0 + t, row_elems);
                if (at >= 0) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(key + at + col);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[2 * e] += unpack_lo<F16>(w[e]);
                        acc[2 * e + 1] += unpack_hi<F16>(w[e]);
                    }
                    ++seen;
                }
            }
        }
        float *mine = part + threadIdx.x * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) mine[e] = acc[e];
        seen_by[threadIdx.x] = seen;                       // keys behind a bad block id do not count
        __syncthreads();
        if (ty == 0 && on) {
            for (int y = 1; y < ty_n; ++y) {
                const float *o = part + (y * tx_n + tx) * 8;
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += o[e];
                seen += seen_by[y * tx_n + tx];
            }
            float *out = pooled + ((int64_t)b * g.max_segs + s) * row_elems + col;
            const float d = seen > 0 ? (float)seen : 1.f;
            reinterpret_cast<float4 *>(out)[0] = make_float4(acc[0] / d, acc[1] / d, acc[2] / d, acc[3] / d);
            reinterpret_cast<float4 *>(out)[1] = make_float4(acc[4] / d, acc[5] / d, acc[6] / d, acc[7] / d);
        }
        __syncthreads();
    }
}

// -------------------------------------------------------------------- select

// The choice is by comparison, so it has to be that of scores in 64 bits; but
// nearly every comparison is settled by far less.  The scores are first taken on
// the 16-bit matrix instruction from q = qh + ql and P = ph + pl (two bf16 parts
// each): qh.ph + qh.pl + ql.ph is off by at most E = 8 * 2^-16 |q| |P| (2^-16 for
// the part dropped and for the rounding of each second part; the fp32 sums, 24
// steps of 17 terms that lose 2^-23 each at the worst, 3.2 * 2^-16).  A row then bisects
// for its last chosen score; when the gap to the first one left out is above 2E,
// the choice is that of the exact scores.  Otherwise the scores within 2E of the
// border (two or three of 500, in one row of six) are computed in 64 bits and
// ranked; more than 32 of them (ties), and scores that are not finite, send the
// row to a pass in 64 bits by the whole block.
//
// A block takes R rows and one key head, its warps 16 segments at a time; when
// rows are few, a cluster of C blocks shares a row's segments and its first
// block chooses.  8192 rows over 512 segments and 4 key heads take 160 us (514 us
// with every score in 64 bits): of a block's 62000 cycles for 31 rows a quarter
// goes to reading the queries, a third to the scores (issue slots: splitting the
// means in two and their norms cost more than the products) and a third to the
// choice, ten counts of a row's scores held in registers.  64 rows over up to
// 1024 segments: 16 us (38 us).

struct SelArgs {
    SegGeo g;
    const uint16_t *q;
    const float *pooled;
    int32_t *idx;
    int32_t R, ld;                         // rows per block; scores per row
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Two numbers as their leading and following bf16 parts.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// Order of 64-bit scores as unsigned integers (NaN = -inf, -0 = +0).
__device__ __forceinline__ uint64_t order_of(double x)
{
    if (x != x) x = -INFINITY;
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ float warp_min(float x)
{
    float m;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
}
__device__ __forceinline__ float warp_max(float x)
{
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
}

// q . P[s] in 64 bits, by 32 or 8 neighbouring lanes (T).
template <int D, int T>
__device__ __forceinline__ double exact_score(const double *q, const float *P, int64_t ldp, int32_t s, int lane)
{
    double x = 0;
    const float4 *p = reinterpret_cast<const float4 *>(P + s * ldp);
#pragma unroll
    for (int c = lane % T; c < D / 4; c += T) {
        const float4 v = p[c];
        const double2 a = reinterpret_cast<const double2 *>(q)[2 * c], b = reinterpret_cast<const double2 *>(q)[2 * c + 1];
        x += (a.x * v.x + a.y * v.y) + (b.x * v.z + b.y * v.w);
    }
#pragma unroll
    for (int o = T / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What a row chooses from and where it writes.
struct SelRow {
    const float *sc;                       // approximate scores
    const double *q;
    const float *P;
    int64_t ldp;
    int32_t *out;
    int32_t ns, init, local, count;
    float err;                             // E
};

struct SelShared {
    int32_t sums[2][kSelThreads / 32];
    float lows[kSelThreads / 32], highs[kSelThreads / 32];
    int32_t band[kSelThreads / 32][32];    // segments near the border, per team
    int32_t bands[kSelThreads / 32];
    uint32_t taken[kSelThreads / 32];
};

// A team (one warp, or with WIDE the block) chooses for one row.  KR: scores per
// thread in registers (0: read again in every pass).  Returns false when the
// border cannot be settled here.
template <int D, int KR, bool WIDE>
__device__ bool choose(const SelRow &r, SelShared &sh, int team)
{
    constexpr int T = WIDE ? kSelThreads : 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = WIDE ? threadIdx.x : lane;
    auto sync = [&]() {
        if constexpr (WIDE) __syncthreads();
        else __syncwarp();
    };
    int turn = 0;
    auto sum = [&](int32_t v) {
        v = __reduce_add_sync(0xffffffffu, v);
        if constexpr (WIDE) {
            if (lane == 0) sh.sums[turn][warp] = v;
            __syncthreads();
            v = 0;
            for (int w = 0; w < kSelThreads / 32; ++w) v += sh.sums[turn][w];
            turn ^= 1;
        }
        return v;
    };
    auto least = [&](float lo) {
        lo = warp_min(lo);
        if constexpr (WIDE) {
            __syncthreads();
            if (lane == 0) sh.lows[warp] = lo;
            __syncthreads();
            for (int w = 0; w < kSelThreads / 32; ++w) lo = fminf(lo, sh.lows[w]);
        }
        return lo;
    };
    auto most = [&](float hi) {
        hi = warp_max(hi);
        if constexpr (WIDE) {
            __syncthreads();
            if (lane == 0) sh.highs[warp] = hi;
            __syncthreads();
            for (int w = 0; w < kSelThreads / 32; ++w) hi = fmaxf(hi, sh.highs[w]);
        }
        return hi;
    };
    // the free choice is from [from, to); others read as -inf
    const int32_t from = r.init, to = r.ns - r.local, need = r.count - r.init - r.local;
    auto score_at = [&](int32_t s) { return s >= from && s < to ? r.sc[s] : -INFINITY; };
    float held[KR > 0 ? KR : 1];                       // a lane's KR neighbouring segments
    // (conditions on them are written with & and as bit masks: a branch for each
    // would cost more than all the rest)
    auto bits_of = [&](int32_t lo, int32_t hi) {       // those within [lo, hi)
        lo -= t * KR;
        hi -= t * KR;
        lo = lo < 0 ? 0 : (lo > KR ? KR : lo);
        hi = hi < 0 ? 0 : (hi > KR ? KR : hi);
        return (uint32_t)((1ull << hi) - 1) & ~(uint32_t)((1ull << lo) - 1);
    };
    const uint32_t free_bits = KR > 0 ? bits_of(from, to) : 0;
    if constexpr (KR > 0) {
#pragma unroll
        for (int k = 0; k < KR; k += 4) {
            const int32_t s = t * KR + k;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s < r.ns) x = *reinterpret_cast<const float4 *>(r.sc + s);
            held[k] = free_bits >> k & 1u ? x.x : -INFINITY;
            held[k + 1] = free_bits >> (k + 1) & 1u ? x.y : -INFINITY;
            held[k + 2] = free_bits >> (k + 2) & 1u ? x.z : -INFINITY;
            held[k + 3] = free_bits >> (k + 3) & 1u ? x.w : -INFINITY;
        }
    }
    auto each = [&](auto &&f) {                        // f(segment, score), all of the row's segments
        if constexpr (KR > 0) {
#pragma unroll
            for (int k = 0; k < KR; ++k) f(t * KR + k, held[k]);
        } else {
            for (int32_t s = t; s < r.ns; s += T) f(s, score_at(s));
        }
    };
    // chosen: scores from `cut` on and above `over`; of those within [band_lo,
    // band_hi] the ones that are `taken`.  With nothing to choose, not even a score
    // that has overflowed is above `over`.
    float cut = INFINITY, over = need > 0 ? -INFINITY : INFINITY, band_lo = INFINITY, band_hi = -INFINITY;
    uint32_t taken = 0;
    int32_t ties = 0;                                  // equal scores of the cut that are chosen, lowest first (0: all)
    if (need > 0) {
        float lo = INFINITY, hi = -INFINITY;
        bool odd = false;
        if constexpr (KR > 0) {
#pragma unroll
            for (int k = 0; k < KR; ++k) {
                const bool is = free_bits >> k & 1u;
                odd |= is & !(fabsf(held[k]) < 1e38f);
                lo = fminf(lo, is ? held[k] : INFINITY);
                hi = fmaxf(hi, held[k]);
            }
        } else {
            for (int32_t s = from + t; s < to; s += T) {
                const float x = r.sc[s];
                odd |= !(fabsf(x) < 1e38f);
                lo = fminf(lo, x);
                hi = fmaxf(hi, x);
            }
        }
        odd = sum(odd) > 0;
        if (odd || !(r.err < INFINITY)) return false;
        lo = least(lo);
        hi = most(hi);
        // at least `need` scores from lo on, fewer from hi on
        hi = hi == 0.f ? 1e-45f : __int_as_float(__float_as_int(hi) + (hi > 0.f ? 1 : -1));
        bool even = false;                             // exactly `need` scores from lo on
        for (;;) {
            const float mid = 0.5f * lo + 0.5f * hi;
            if (!(mid > lo && mid < hi)) break;
            int32_t c = 0;
            if constexpr (KR > 0) {                    // four sums: adds that do not wait for one another
                int32_t c4[4] = {};
#pragma unroll
                for (int k = 0; k < KR; ++k) c4[k & 3] += held[k] >= mid;
                c = (c4[0] + c4[1]) + (c4[2] + c4[3]);
            } else {
                each([&](int32_t, float x) { c += x >= mid; });
            }
            c = sum(c);
            if (c >= need) lo = mid;
            else hi = mid;
            if (c == need) {
                even = true;
                break;
            }
        }
        // the last score chosen, and the first one left out
        float in = INFINITY, out = -INFINITY;
        each([&](int32_t, float x) {
            in = fminf(in, x >= lo ? x : INFINITY);
            out = fmaxf(out, x >= lo ? -INFINITY : x);
        });
        cut = least(in);
        if (even) {
            out = most(out);
            even = cut - out > 2.f * r.err;
        }
        if (!even) {
            if (r.err == 0.f) {                        // every score is exact (zero): only ties
                int32_t c = 0;
                each([&](int32_t, float x) { c += x > cut; });
                ties = need - sum(c);
            } else {
                band_lo = cut - 2.f * r.err;
                band_hi = cut + 2.f * r.err;
                int32_t above = 0, inside = 0;
                each([&](int32_t, float x) {
                    above += x > band_hi;
                    inside += (x >= band_lo) & (x <= band_hi);
                });
                above = sum(above);
                inside = sum(inside);
                if (inside > 32) return false;
                if (t == 0) sh.bands[team] = 0;
                sync();
                each([&](int32_t s, float x) {
                    if ((x >= band_lo) & (x <= band_hi)) sh.band[team][atomicAdd(&sh.bands[team], 1)] = s;
                });
                sync();
                if (!WIDE || warp == 0) {              // one warp ranks them: score, then the lower segment
                    double mine = 0;
                    const int32_t s = lane < inside ? sh.band[team][lane] : 0;
                    for (int i = 0; i < inside; i += 4) {
                        const int k = i + (lane >> 3);
                        const double x = exact_score<D, 8>(r.q, r.P, r.ldp, sh.band[team][k < inside ? k : inside - 1], lane);
                        const double y = __shfl_sync(0xffffffffu, x, (lane - i) * 8 & 31);
                        if (lane >= i && lane < i + 4) mine = y;
                    }
                    const uint64_t ord = order_of(mine);
                    int rank = 0;
                    for (int i = 0; i < inside; ++i) {
                        const uint64_t o = __shfl_sync(0xffffffffu, ord, i);
                        const int32_t so = __shfl_sync(0xffffffffu, s, i);
                        rank += o > ord || (o == ord && so < s);
                    }
                    const uint32_t m = __ballot_sync(0xffffffffu, lane < inside && rank < need - above);
                    if (lane == 0) sh.taken[team] = m;
                }
                sync();
                taken = sh.taken[team];
                over = band_hi;
            }
        }
    }
    // in order: the forced ones, and the chosen
    const uint32_t below = (1u << lane) - 1u;
    int32_t done = 0, tied = 0;
    if constexpr (KR > 0) {
        uint32_t mine = bits_of(0, r.ns) & ~free_bits; // bit k: segment t * KR + k
#pragma unroll
        for (int k = 0; k < KR; ++k) mine |= (held[k] >= cut) & (held[k] > over) ? 1u << k : 0u;
        for (uint32_t m = taken; m; m &= m - 1) {
            const int32_t s = sh.band[team][__ffs(m) - 1];
            if (s / KR == t) mine |= 1u << (s % KR);
        }
        auto before = [&](int32_t v) {                 // sum over the lanes below
            const int32_t own = v;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            return v - own;
        };
        if (ties > 0) {
            int32_t c = 0;
#pragma unroll
            for (int k = 0; k < KR; ++k) c += held[k] == cut;
            int32_t rank = before(c);
#pragma unroll
            for (int k = 0; k < KR; ++k)
                if (held[k] == cut && rank++ >= ties) mine &= ~(1u << k);
        }
        int32_t *out = r.out + before(__popc(mine));
        for (; mine; mine &= mine - 1) *out++ = t * KR + __ffs(mine) - 1;
        return true;
    }
    auto place = [&](bool b, int32_t base, int32_t &total) {   // rank of this thread's among the team's in order
        const uint32_t m = __ballot_sync(0xffffffffu, b);
        int32_t rank = base + __popc(m & below);
        total = __popc(m);
        if constexpr (WIDE) {
            if (lane == 0) sh.sums[turn][warp] = total;
            __syncthreads();
            total = 0;
            for (int w = 0; w < kSelThreads / 32; ++w) {
                if (w < warp) rank += sh.sums[turn][w];
                total += sh.sums[turn][w];
            }
            turn ^= 1;
        }
        return rank;
    };
    for (int32_t s0 = 0; s0 < r.ns; s0 += T) {
        const int32_t s = s0 + t;
        const float x = s < r.ns ? score_at(s) : -INFINITY;
        bool in = s < r.ns && (s < from || s >= to || (x >= cut && x > over));
        if (x >= band_lo && x <= band_hi)
            for (uint32_t m = taken; m; m &= m - 1) in |= sh.band[team][__ffs(m) - 1] == s;
        int32_t total;
        if (ties > 0) {
            const int32_t rank = place(x == cut, tied, total);
            if (x == cut && rank >= ties) in = false;
            tied += total;
        }
        const int32_t rank = place(in, done, total);
        if (in) r.out[rank] = s;
        done += total;
    }
    return true;
}

// The same from scores in 64 bits, by the whole block (x: room for ns doubles).
template <int D>
__device__ void choose_exactly(const SelRow &r, SelShared &sh, double *x)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t from = r.init, to = r.ns - r.local, need = r.count - r.init - r.local;
    __syncthreads();
    for (int32_t s = warp; s < r.ns; s += kSelThreads / 32) {
        const double v = exact_score<D, 32>(r.q, r.P, r.ldp, s, lane);
        if (lane == 0) x[s] = v;
    }
    __syncthreads();
    int turn = 0;
    auto sum = [&](int32_t v, int32_t *before) {
        v = __reduce_add_sync(0xffffffffu, v);
        if (lane == 0) sh.sums[turn][warp] = v;
        __syncthreads();
        int32_t t = 0;
        for (int w = 0; w < kSelThreads / 32; ++w) {
            if (before && w < warp) *before += sh.sums[turn][w];
            t += sh.sums[turn][w];
        }
        turn ^= 1;
        return t;
    };
    // the largest threshold that at least `need` scores reach
    uint64_t lo = 0, hi = ~0ull;
    while (lo < hi) {
        const uint64_t mid = lo + ((hi - lo) >> 1) + ((hi - lo) & 1);
        int32_t c = 0;
        for (int32_t s = from + tid; s < to; s += kSelThreads) c += order_of(x[s]) >= mid;
        if (sum(c, nullptr) >= need) lo = mid;
        else hi = mid - 1;
    }
    int32_t c = 0;
    for (int32_t s = from + tid; s < to; s += kSelThreads) c += order_of(x[s]) > lo;
    const int32_t ties = need - sum(c, nullptr);
    int32_t done = 0, tied = 0;
    for (int32_t s0 = 0; s0 < r.ns; s0 += kSelThreads) {
        const int32_t s = s0 + tid;
        bool in = s < r.ns, at = false;
        if (in && s >= from && s < to) {
            const uint64_t u = order_of(x[s]);
            in = u > lo;
            at = u == lo;
        }
        const uint32_t below = (1u << lane) - 1u;
        uint32_t m = __ballot_sync(0xffffffffu, at);
        int32_t rank = tied + __popc(m & below);
        tied += sum(at, &rank);
        in |= at && rank < ties;
        m = __ballot_sync(0xffffffffu, in);
        rank = done + __popc(m & below);
        done += sum(in, &rank);
        if (in) r.out[rank] = s;
    }
}

template <int D, bool F16, int MT, int C>
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const SelArgs a)
{
    constexpr int KS = D / 16;
    extern __shared__ double dyn[];
    const SegGeo &g = a.g;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int R = a.R;
    double *sq = dyn;                                          // [R][D + 2]: rows of a fragment fall into different banks
    uint4 *frag = reinterpret_cast<uint4 *>(sq + R * (D + 2));       // [MT][KS][2][32]: q's two parts as fragments
    float *sc = reinterpret_cast<float *>(frag + MT * KS * 64);                   // [R][ld]
    double *red = reinterpret_cast<double *>(sc + (C > 1 ? (size_t)(R > 2 ? R : 2) * a.ld : 0));   // partial sums of q
    __shared__ SegRow rows[kSelRows];
    __shared__ int32_t segs[kSelRows], most_segs;
    __shared__ float qnorm[kSelRows];
    __shared__ int32_t leader[kSelRows];                       // the first row of a row's run (of rows of one batch)
    __shared__ uint32_t pnorm[kSelRows], pbits[kSelRows];      // of a run's means: largest |P|^2, all bits; at its first row
    __shared__ int32_t unsettled[kSelRows], unsettled_n;
    __shared__ SelShared sh;
    namespace cg = cooperative_groups;
    const int rank = C > 1 ? (int)(blockIdx.x % C) : 0;
    const int32_t row0 = (int32_t)(blockIdx.x / C) * R, n = blockIdx.y;
    const int nr = g.rows - row0 < R ? g.rows - row0 : R;
    if (warp == 0) {                       // R <= 32
        SegRow r{};
        r.b = -1;
        int32_t ns = 0;
        if (lane < nr) {
            r = seg_row(g, row0 + lane);
            ns = (int32_t)(((uint32_t)r.vis + (uint32_t)g.seg - 1) / (uint32_t)g.seg);
            if (ns > g.max_segs) {
                ns = g.max_segs;
                seg_flag(g, LI_DEV_BAD_KLEN);
            }
        }
        if (lane < R) {
            rows[lane] = r;
            segs[lane] = ns;
            pnorm[lane] = pbits[lane] = 0;
        }
        const int32_t left = __shfl_up_sync(0xffffffffu, r.b, 1);
        const uint32_t starts = __ballot_sync(0xffffffffu, lane == 0 || left != r.b);
        if (lane < R) leader[lane] = 31 - __clz(starts & (0xffffffffu >> (31 - lane)));
        ns = __reduce_max_sync(0xffffffffu, ns);
        if (lane == 0) {
            most_segs = ns;
            unsettled_n = 0;
        }
    }
    __syncthreads();
    if constexpr (C > 1) cg::this_cluster().barrier_arrive();
    auto means_of = [&](int32_t b) { return a.pooled + ((int64_t)b * g.max_segs * g.N2 + n) * D; };
    const int64_t ldp = (int64_t)g.N2 * D;
    const int32_t most = most_segs;
    if (most > g.count) {
        // ---- q summed over the heads of this key head
        const int per = R * (D / 8);       // threads that cover R rows once
        const int parts = kSelThreads / per > 0 ? kSelThreads / per : 1;
        for (int base = 0; base < per; base += kSelThreads) {
            const int e = base + (parts > 1 ? tid % per : tid), part = parts > 1 ? tid / per : 0;
            const int r = e / (D / 8), c = e % (D / 8) * 8;
            double acc[8] = {};
            if (e < per && part < parts && r < nr && rows[r].vis > 0) {
                const uint16_t *src = a.q + ((int64_t)(row0 + r) * g.N1 + (int64_t)n * g.G) * D + c;
#pragma unroll 16
                for (int h = part; h < g.G; h += parts) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + (int64_t)h * D);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        acc[2 * k] += (double)unpack_lo<F16>(w[k]);
                        acc[2 * k + 1] += (double)unpack_hi<F16>(w[k]);
                    }
                }
            }
            if (e < per && part < parts) {
                double *dst = parts > 1 ? red + ((int64_t)part * R + r) * D + c : sq + r * (D + 2) + c;
#pragma unroll
                for (int k = 0; k < 8; ++k) dst[k] = acc[k];
            }
        }
        __syncthreads();
        if (parts > 1) {
            for (int e = tid; e < R * D; e += kSelThreads) {
                double acc = 0;
                for (int k = 0; k < parts; ++k) acc += red[k * R * D + e];
                sq[e / D * (D + 2) + e % D] = acc;
            }
            __syncthreads();
        }
        // ---- its fragments: lane l of step k holds columns 16k + 4(l%4) .. + 3 of
        // rows l/4 and l/4 + 8 (a dot product does not mind the order of columns)
        for (int e = tid; e < MT * KS * 32; e += kSelThreads) {
            const int l = e & 31, ks = (e >> 5) % KS, mt = (e >> 5) / KS;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int r = mt * 16 + (l >> 2) + (h & 1) * 8, c = ks * 16 + 4 * (l & 3) + (h >> 1) * 2;
                const double x = r < R ? sq[r * (D + 2) + c] : 0, y = r < R ? sq[r * (D + 2) + c + 1] : 0;
                split2((float)x, (float)y, hi[h], lo[h]);
            }
            uint4 *dst = frag + (mt * KS + ks) * 64 + l;
            dst[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            dst[32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        for (int r = warp; r < R; r += kSelThreads / 32) {
            double x = 0;
            for (int c = lane; c < D; c += 32) x = fma(sq[r * (D + 2) + c], sq[r * (D + 2) + c], x);
#pragma unroll
            for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane == 0) qnorm[r] = x > 0 ? fmaxf((float)sqrt(x) * 1.0001f, 1e-30f) : (x == 0 ? 0.f : INFINITY);
        }
        __syncthreads();
        float *there = sc;                                     // where the scores go: the cluster's first block
        if constexpr (C > 1) {
            cg::this_cluster().barrier_wait();                 // it runs
            there = cg::this_cluster().map_shared_rank(sc, 0);
        }
        // ---- scores, one run of rows of the same batch after another
        for (int r0 = 0; r0 < nr;) {
            const int32_t b = rows[r0].b;
            int r1 = r0 + 1;
            int32_t ns = segs[r0];
            while (r1 < nr && rows[r1].b == b) {
                const int32_t m = segs[r1];
                ns = m > ns ? m : ns;
                ++r1;
            }
            const float *P = means_of(b);
            float norm = 0.f;
            uint32_t bits = 0;
            for (int32_t s0 = (rank * (kSelThreads / 32) + warp) * 16; s0 < ns; s0 += C * (kSelThreads / 32) * 16) {
                float4 p[2][KS];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int32_t s = s0 + 8 * t + (lane >> 2);
                    const float4 *src = reinterpret_cast<const float4 *>(P + (s < ns ? s : ns - 1) * ldp) + (lane & 3);
#pragma unroll
                    for (int k = 0; k < KS; ++k) p[t][k] = src[4 * k];
                }
                float acc[MT][2][4] = {};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t hi[2][2], lo[2][2];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        split2(p[t][k].x, p[t][k].y, hi[t][0], lo[t][0]);
                        split2(p[t][k].z, p[t][k].w, hi[t][1], lo[t][1]);
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const uint4 qh = frag[(m * KS + k) * 64 + lane], ql = frag[(m * KS + k) * 64 + 32 + lane];
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            mma_bf16(acc[m][t], ql, hi[t][0], hi[t][1]);
                            mma_bf16(acc[m][t], qh, lo[t][0], lo[t][1]);
                            mma_bf16(acc[m][t], qh, hi[t][0], hi[t][1]);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float x = 0.f, y = 0.f;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const float4 v = p[t][k];
                        ffma2(x, y, v.x, v.y, v.x, v.y, x, y);
                        ffma2(x, y, v.z, v.w, v.z, v.w, x, y);
                        bits |= __float_as_uint(v.x) | __float_as_uint(v.y) | __float_as_uint(v.z) | __float_as_uint(v.w);
                    }
                    x += y;
                    x += __shfl_xor_sync(0xffffffffu, x, 1);
                    x += __shfl_xor_sync(0xffffffffu, x, 2);
                    norm = fmaxf(norm, x);
                    // lane: rows lane/4 and lane/4 + 8, segments s0 + 8t + 2*(lane%4) and the next
                    const int32_t c = s0 + 8 * t + 2 * (lane & 3);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int r = m * 16 + (lane >> 2) + 8 * h;
                            if (r >= r0 && r < r1) {
                                if (c < ns) there[(int64_t)r * a.ld + c] = acc[m][t][2 * h];
                                if (c + 1 < ns) there[(int64_t)r * a.ld + c + 1] = acc[m][t][2 * h + 1];
                            }
                        }
                }
            }
            const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(norm));   // (>= 0: ordered as integers)
            bits = __reduce_or_sync(0xffffffffu, bits & 0x7FFFFFFFu);
            if (lane == 0) {
                uint32_t *to_n = pnorm + r0, *to_b = pbits + r0;
                if constexpr (C > 1) {
                    to_n = cg::this_cluster().map_shared_rank(to_n, 0);
                    to_b = cg::this_cluster().map_shared_rank(to_b, 0);
                }
                atomicMax(to_n, top);
                atomicOr(to_b, bits);
            }
            r0 = r1;
        }
        if constexpr (C > 1) {
            cg::this_cluster().sync();
            if (rank != 0) return;
        }
        __syncthreads();
    } else if constexpr (C > 1) {
        cg::this_cluster().barrier_wait();
        if (rank != 0) return;
    }
    // ---- the choice
    auto row_of = [&](int r) {
        SelRow x;
        const int first = leader[r];                           // holds the norm of the run's means
        x.sc = sc + (int64_t)r * a.ld;
        x.q = sq + r * (D + 2);
        x.P = means_of(rows[r].b);
        x.ldp = ldp;
        x.out = a.idx + ((int64_t)(row0 + r) * g.N2 + n) * g.count;
        x.ns = segs[r];
        x.init = g.init;
        x.local = g.local;
        x.count = g.count;
        const float norm = __uint_as_float(pnorm[first]);
        // (squares below 1e-30 have lost bits; products below 1e-38 are lost)
        x.err = pbits[first] == 0 || qnorm[r] == 0.f ? 0.f
                : norm < 1e-30f ? INFINITY : 8.f / 65536.f * qnorm[r] * sqrtf(norm) * 1.0001f + 1e-35f;
        return x;
    };
    auto all_of = [&](int r, int t, int T) {                   // few segments: all are chosen
        int32_t *out = a.idx + ((int64_t)(row0 + r) * g.N2 + n) * g.count;
        const int32_t ns = segs[r];
        for (int32_t k = t; k < g.count; k += T) out[k] = k < ns ? k : -1;
    };
    for (int r = warp; r < nr; r += kSelThreads / 32) {
        const int32_t ns = segs[r];
        if (ns <= g.count) {
            all_of(r, lane, 32);
            continue;
        }
        if (ns > 1024) continue;
        const SelRow x = row_of(r);
        const bool ok = ns <= 256 ? choose<D, 8, false>(x, sh, warp)
                        : ns <= 512 ? choose<D, 16, false>(x, sh, warp) : choose<D, 32, false>(x, sh, warp);
        if (!ok && lane == 0) unsettled[atomicAdd(&unsettled_n, 1)] = r;
    }
    __syncthreads();
    if (most <= g.count) return;
    // rows of more segments than a warp's registers hold: the block
    for (int r = 0; r < nr; ++r) {
        if (segs[r] <= 1024 || segs[r] <= g.count) continue;
        const bool ok = choose<D, 0, true>(row_of(r), sh, 0);
        if (!ok && tid == 0) unsettled[unsettled_n++] = r;
        __syncthreads();
    }
    // (the order of these rows does not matter; the scores of the others are no longer needed)
    for (int k = 0; k < unsettled_n; ++k) choose_exactly<D>(row_of(unsettled[k]), sh, reinterpret_cast<double *>(sc));
}

bool off(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

template <int D, bool F16, int MT, int C>
cudaError_t launch_select(const SelArgs &a, size_t smem, cudaStream_t s)
{
    auto kern = select_kernel<D, F16, MT, C>;
    const cudaError_t e = li::set_max_dynamic_smem(reinterpret_cast<const void *>(kern), (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.g.rows + a.R - 1) / a.R) * C, (unsigned)a.g.N2);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D, bool F16>
cudaError_t launch_select(const SelArgs &a, int split, size_t smem, cudaStream_t s)
{
    if (split == 8) return launch_select<D, F16, 1, 8>(a, smem, s);
    if (split == 4) return launch_select<D, F16, 1, 4>(a, smem, s);
    if (split == 2) return launch_select<D, F16, 1, 2>(a, smem, s);
    return a.R > 16 ? launch_select<D, F16, 2, 1>(a, smem, s) : launch_select<D, F16, 1, 1>(a, smem, s);
}

}  // namespace

extern "C" LI_API li_status li_segment_pool(const li_segment_params *p, const void *key, const int32_t *act_seq_k,
                                            const int32_t *block_table, const int32_t *first, float *pooled,
                                            int32_t *status, void *stream)
{
    const char *call = "li_segment_pool";
    SegGeo g{};
    const li_status st = seg_setup(call, p, false, true, nullptr, act_seq_k, block_table, status, &g);
    if (st != LI_OK) return st;
    if (seg_no_keys(g)) return LI_OK;                        // no segment holds a key
    if (!key || !pooled) return seg_fail(call, LI_ERR_NULL, "key and pooled are required");
    if (off(key, 16) || off(pooled, 16) || off(first, 4))
        return seg_fail(call, LI_ERR_SHAPE, "key and pooled must be 16-byte aligned, first 4-byte");
    if (p->B > 65535) return seg_fail(call, LI_ERR_SHAPE, "B must be at most 65535");
    const int cols = p->N2 * p->D / 8;                       // 16-byte columns
    const int tx = cols < 64 ? cols : 64;
    const int z = (cols + tx - 1) / tx;
    int64_t x = (8LL * seg_sms() + (int64_t)p->B * z - 1) / ((int64_t)p->B * z);
    if (x > p->max_segs) x = p->max_segs;
    const dim3 grid((unsigned)x, (unsigned)p->B, (unsigned)z);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint16_t *k = static_cast<const uint16_t *>(key);
    if (p->dtype == LI_FP16) pool_kernel<true><<<grid, kPoolThreads, 0, s>>>(g, k, first, pooled, p->D, tx);
    else pool_kernel<false><<<grid, kPoolThreads, 0, s>>>(g, k, first, pooled, p->D, tx);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return seg_fail(call, LI_ERR_CUDA, cudaGetErrorString(e));
    li::set_launch_count(1);
    return LI_OK;
}

extern "C" LI_API li_status li_segment_select(const li_segment_params *p, const void *query, const float *pooled,
                                              const int32_t *act_seq_q, const int32_t *act_seq_k, int32_t *seg_idx,
                                              int32_t *status, void *stream)
{
    const char *call = "li_segment_select";
    SelArgs a{};
    const li_status st = seg_setup(call, p, true, false, act_seq_q, act_seq_k, nullptr, status, &a.g);
    if (st != LI_OK) return st;
    if (a.g.rows == 0) return LI_OK;                         // empty tensors have no address
    if (!query || !pooled || !seg_idx) return seg_fail(call, LI_ERR_NULL, "query, pooled and seg_idx are required");
    if (off(query, 16) || off(pooled, 16) || off(seg_idx, 4))
        return seg_fail(call, LI_ERR_SHAPE, "query and pooled must be 16-byte aligned, seg_idx 4-byte");
    a.q = static_cast<const uint16_t *>(query);
    a.pooled = pooled;
    a.idx = seg_idx;
    // rows per block: as many as stand within 110 KB (two blocks per SM), and not
    // so many that SMs stay idle
    const int sms = seg_sms(), D = p->D;
    a.ld = ((p->max_segs + 31) & ~31) + 8;               // rows of a fragment fall into different banks
    auto bytes = [&](int R, bool split) {
        const size_t sums = (size_t)kSelThreads * 8 * 8, scores = (size_t)(R > 2 ? R : 2) * a.ld * 4;
        return (size_t)R * (D + 2) * 8 + (size_t)(R > 16 ? 2 : 1) * D * 64 + (split ? scores + sums : scores > sums ? scores : sums);
    };
    int R = kSelRows;
    while (R > 1 && bytes(R, false) > 110 * 1024) --R;
    while (R > 1 && (int64_t)((a.g.rows + R - 1) / R) * p->N2 < 2 * sms) R = (R + 1) / 2;
    // the fewest rows that take as many waves (8192 rows, 4 key heads, 512 segments:
    // 28 rows, not 31, fill the last of 4)
    const int64_t blocks = (int64_t)((a.g.rows + R - 1) / R) * p->N2, waves = (blocks + 2 * sms - 1) / (2 * sms);
    const int64_t per_head = waves * 2 * sms / p->N2;
    if (per_head > 0 && (a.g.rows + per_head - 1) / per_head < R) R = (int)((a.g.rows + per_head - 1) / per_head);
    // few rows: a cluster shares a row's segments, at least 128 to a block
    int split = 1;
    if (R == 1)
        while (split < kSelSplit && (int64_t)a.g.rows * p->N2 * split * 2 <= 2LL * sms && p->max_segs >= 2 * split * 128) split *= 2;
    a.R = R;
    const size_t smem = bytes(R, split > 1);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f16 = p->dtype == LI_FP16;
    const cudaError_t e = D == 128 ? (f16 ? launch_select<128, true>(a, split, smem, s) : launch_select<128, false>(a, split, smem, s))
                                   : (f16 ? launch_select<64, true>(a, split, smem, s) : launch_select<64, false>(a, split, smem, s));
    if (e != cudaSuccess) return seg_fail(call, LI_ERR_CUDA, cudaGetErrorString(e));
    li::set_launch_count(1);
    return LI_OK;
}
