// li_segment.cu -- the cheap score of segment-sparse attention: the mean key of
// each segment (pool) and the choice of segments for each query row (select).
#include <cmath>
#include <cstdio>

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
constexpr int kSelRows = 16;               // most query rows of one select block

// ---------------------------------------------------------------------- pool

// The mean of a segment is one pass over its keys: the block's threads stand
// as tx (16 bytes of the N2*D columns) by ty (a token of every `ty_n`), sum in
// fp32 and meet in shared memory.  Bound by HBM: each key is read once.
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
                        acc[2 * e] += seg_lo<F16>(w[e]);
                        acc[2 * e + 1] += seg_hi<F16>(w[e]);
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

// A block takes R query rows and one key head.  Their scores stay in shared
// memory: q (summed over the key head's query heads) and the products are held
// in 64 bits, because the choice is by comparison and 32 bits would order
// neighbours by rounding.  The products run on the 64-bit matrix instruction
// (8 rows x 8 segments x 4 columns); a lane reads four neighbouring columns of
// a segment's mean at once and the four steps take them in that order (a dot
// product does not mind).  Then 256/R threads per row bisect for the score that
// the last chosen segment has, and write the chosen ones in order.

struct SelArgs {
    SegGeo g;
    const uint16_t *q;
    const float *pooled;
    int32_t *idx;
    int32_t R, ld;                         // rows per block; scores per row
};

__device__ __forceinline__ void mma_f64(double &d0, double &d1, double a, double b)
{
    asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0, %1}, {%2}, {%3}, {%0, %1};"
                 : "+d"(d0), "+d"(d1)
                 : "d"(a), "d"(b));
}

// Order of the scores as unsigned integers (NaN lowest, -0 = +0).
__device__ __forceinline__ uint64_t order_of(double x)
{
    if (x != x) return 0;
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ void team_sync(int team, int threads)
{
    if (threads == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

template <int D, bool F16>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelArgs a)
{
    constexpr int LDQ = D + 2;             // doubles per row: the 8 rows of a fragment hit different banks
    extern __shared__ double dyn[];
    const SegGeo &g = a.g;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int R = a.R, R8 = (R + 7) & ~7;
    double *sq = dyn;                      // [R8][LDQ]
    double *red = sq + R8 * LDQ;           // [256 / (R*D/8)][R][D] partial sums, then the scores
    double *sc = red;                      // [R][ld]
    __shared__ SegRow rows[kSelRows];
    __shared__ int32_t warp_count[2][kSelThreads / 32];
    const int32_t row0 = blockIdx.x * R, n = blockIdx.y;
    const int nr = g.rows - row0 < R ? g.rows - row0 : R;
    if (tid < R) {
        SegRow r{};
        r.b = -1;
        if (tid < nr) r = seg_row(g, row0 + tid);
        rows[tid] = r;
    }
    __syncthreads();
    auto segs_of = [&](const SegRow &r) {
        const int32_t ns = (int32_t)(((int64_t)r.vis + g.seg - 1) / g.seg);
        return ns > g.max_segs ? g.max_segs : ns;
    };
    int32_t most = 0;
    for (int r = 0; r < nr; ++r) {
        const int32_t ns = segs_of(rows[r]);
        most = ns > most ? ns : most;
        if (tid == 0 && ((int64_t)rows[r].vis + g.seg - 1) / g.seg > g.max_segs) seg_flag(g, LI_DEV_BAD_KLEN);
    }
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
#pragma unroll 4
                for (int h = part; h < g.G; h += parts) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + (int64_t)h * D);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        acc[2 * k] += (double)seg_lo<F16>(w[k]);
                        acc[2 * k + 1] += (double)seg_hi<F16>(w[k]);
                    }
                }
            }
            if (e < per && part < parts) {
                double *dst = parts > 1 ? red + ((int64_t)part * R + r) * D + c : sq + r * LDQ + c;
#pragma unroll
                for (int k = 0; k < 8; ++k) dst[k] = acc[k];
            }
        }
        __syncthreads();
        if (parts > 1) {
            for (int e = tid; e < R * D; e += kSelThreads) {
                double acc = 0;
                for (int k = 0; k < parts; ++k) acc += red[k * R * D + e];
                sq[e / D * LDQ + e % D] = acc;
            }
        }
        for (int e = R * LDQ + tid; e < R8 * LDQ; e += kSelThreads) sq[e] = 0;
        __syncthreads();
        // ---- scores, one run of rows of the same batch after another
        for (int r0 = 0; r0 < nr;) {
            const int32_t b = rows[r0].b;
            int r1 = r0 + 1;
            int32_t ns = segs_of(rows[r0]);
            while (r1 < nr && rows[r1].b == b) {
                const int32_t m = segs_of(rows[r1]);
                ns = m > ns ? m : ns;
                ++r1;
            }
            const float *P = a.pooled + ((int64_t)b * g.max_segs * g.N2 + n) * D;
            const int64_t ldp = (int64_t)g.N2 * D;
            for (int32_t s0 = warp * 8; s0 < ns; s0 += kSelThreads / 4) {
                double acc[2][2] = {};
                const int32_t s = s0 + (lane >> 2);
                const float4 *src = reinterpret_cast<const float4 *>(P + (s < ns ? s : ns - 1) * ldp) + (lane & 3);
                float4 p[D / 16];
#pragma unroll
                for (int k = 0; k < D / 16; ++k) p[k] = src[4 * k];
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const double bv[4] = {p[k].x, p[k].y, p[k].z, p[k].w};
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t * 8 >= R) break;
                        const double2 *qa = reinterpret_cast<const double2 *>(sq + (t * 8 + (lane >> 2)) * LDQ + 16 * k + 4 * (lane & 3));
                        const double2 q0 = qa[0], q1 = qa[1];
                        mma_f64(acc[t][0], acc[t][1], q0.x, bv[0]);
                        mma_f64(acc[t][0], acc[t][1], q0.y, bv[1]);
                        mma_f64(acc[t][0], acc[t][1], q1.x, bv[2]);
                        mma_f64(acc[t][0], acc[t][1], q1.y, bv[3]);
                    }
                }
                // lane: row lane/4, segments s0 + 2*(lane%4) and the next
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int r = t * 8 + (lane >> 2);
                    const int32_t c = s0 + 2 * (lane & 3);
                    if (r >= r0 && r < r1) {
                        if (c < ns) sc[(int64_t)r * a.ld + c] = acc[t][0];
                        if (c + 1 < ns) sc[(int64_t)r * a.ld + c + 1] = acc[t][1];
                    }
                }
            }
            r0 = r1;
        }
        __syncthreads();
    }
    // ---- the choice: a team of `threads` threads per row
    const int threads = R >= 8 ? 32 : kSelThreads / R;
    const int teams = kSelThreads / threads;
    const int team = tid / threads, lt = tid % threads, team_warp0 = team * (threads / 32);
    auto team_sum = [&](int32_t v, int &turn) {
        v = __reduce_add_sync(0xffffffffu, v);
        if (threads == 32) return v;
        if (lane == 0) warp_count[turn][warp] = v;
        team_sync(team, threads);
        int32_t t = 0;
        for (int w = 0; w < threads / 32; ++w) t += warp_count[turn][team_warp0 + w];
        turn ^= 1;
        return t;
    };
    int turn = 0;
    for (int r = team; r < nr; r += teams) {
        int32_t *out = a.idx + ((int64_t)(row0 + r) * g.N2 + n) * g.count;
        const int32_t ns = segs_of(rows[r]);
        if (ns <= g.count) {
            for (int32_t k = lt; k < g.count; k += threads) out[k] = k < ns ? k : -1;
            continue;
        }
        const double *mine = sc + (int64_t)r * a.ld;
        const int32_t lo_s = g.init, hi_s = ns - g.local;            // the free choice: [lo_s, hi_s)
        const int32_t need = g.count - g.init - g.local;
        // the largest threshold that at least `need` scores reach
        uint64_t lo = 0, hi = ~0ull;
        bool exact = need == 0;
        while (lo < hi && !exact) {
            const uint64_t mid = lo + ((hi - lo) >> 1) + ((hi - lo) & 1);
            int32_t c = 0;
            for (int32_t s = lo_s + lt; s < hi_s; s += threads) c += order_of(mine[s]) >= mid;
            c = team_sum(c, turn);
            if (c >= need) lo = mid;
            else hi = mid - 1;
            exact = c == need;
        }
        // `exact`: everything from lo on; else what lies above lo, and the
        // first ones at lo itself
        int32_t ties = 0;
        if (!exact) {
            int32_t c = 0;
            for (int32_t s = lo_s + lt; s < hi_s; s += threads) c += order_of(mine[s]) > lo;
            ties = need - team_sum(c, turn);
        }
        int32_t done = 0, tied = 0;
        for (int32_t base = 0; base < ns; base += threads) {
            const int32_t s = base + lt;
            bool in = false, at = false;
            if (s < ns) {
                if (s < lo_s || s >= hi_s) in = true;
                else if (need > 0) {
                    const uint64_t u = order_of(mine[s]);
                    in = exact ? u >= lo : u > lo;
                    at = !exact && u == lo;
                }
            }
            const uint32_t below = (1u << lane) - 1u;
            if (!exact) {
                // ranks among the ties, in order
                uint32_t m = __ballot_sync(0xffffffffu, at);
                int32_t rank = tied + __popc(m & below), sum = __popc(m);
                if (threads > 32) {
                    if (lane == 0) warp_count[turn][warp] = sum;
                    team_sync(team, threads);
                    sum = 0;
                    for (int w = 0; w < threads / 32; ++w) {
                        if (team_warp0 + w < warp) rank += warp_count[turn][team_warp0 + w];
                        sum += warp_count[turn][team_warp0 + w];
                    }
                    turn ^= 1;
                }
                if (at && rank < ties) in = true;
                tied += sum;
            }
            const uint32_t m = __ballot_sync(0xffffffffu, in);
            int32_t rank = done + __popc(m & below), sum = __popc(m);
            if (threads > 32) {
                if (lane == 0) warp_count[turn][warp] = sum;
                team_sync(team, threads);
                sum = 0;
                for (int w = 0; w < threads / 32; ++w) {
                    if (team_warp0 + w < warp) rank += warp_count[turn][team_warp0 + w];
                    sum += warp_count[turn][team_warp0 + w];
                }
                turn ^= 1;
            }
            if (in) out[rank] = s;
            done += sum;
        }
    }
}

bool off(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

template <int D, bool F16>
cudaError_t launch_select(SelArgs a, int R, size_t smem, cudaStream_t s)
{
    auto kern = select_kernel<D, F16>;
    const cudaError_t e = li::set_max_dynamic_smem(reinterpret_cast<const void *>(kern), (int)smem);
    if (e != cudaSuccess) return e;
    a.R = R;
    kern<<<dim3((unsigned)((a.g.rows + R - 1) / R), (unsigned)a.g.N2), kSelThreads, smem, s>>>(a);
    return cudaGetLastError();
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
    if (!query || !pooled || !seg_idx) return seg_fail(call, LI_ERR_NULL, "query, pooled and seg_idx are required");
    if (off(query, 16) || off(pooled, 16) || off(seg_idx, 4))
        return seg_fail(call, LI_ERR_SHAPE, "query and pooled must be 16-byte aligned, seg_idx 4-byte");
    if (a.g.rows == 0) return LI_OK;
    a.q = static_cast<const uint16_t *>(query);
    a.pooled = pooled;
    a.idx = seg_idx;
    // rows per block: a power of two, with the scores within 100 KB (two blocks
    // per SM) while more than one row fits, and not so many that SMs stay idle
    const int sms = seg_sms(), D = p->D;
    a.ld = (p->max_segs + 1) & ~1;
    auto bytes = [&](int R) {
        const size_t parts = (size_t)kSelThreads * 8 * 8, scores = (size_t)R * a.ld * 8;
        return (size_t)((R + 7) & ~7) * (D + 2) * 8 + (scores > parts ? scores : parts);
    };
    int R = kSelRows;
    while (R > 1 && (bytes(R) > 100 * 1024 || (int64_t)((a.g.rows + R - 1) / R) * p->N2 < 2 * sms)) R /= 2;
    const size_t smem = bytes(R);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f16 = p->dtype == LI_FP16;
    const cudaError_t e = D == 128 ? (f16 ? launch_select<128, true>(a, R, smem, s) : launch_select<128, false>(a, R, smem, s))
                                   : (f16 ? launch_select<64, true>(a, R, smem, s) : launch_select<64, false>(a, R, smem, s));
    if (e != cudaSuccess) return seg_fail(call, LI_ERR_CUDA, cudaGetErrorString(e));
    li::set_launch_count(1);
    return LI_OK;
}
