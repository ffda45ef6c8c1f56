// li_segattn.cu -- attention over the selected segments, on the 5th-generation
// tensor cores.
//
// A CTA takes one key head and R = 128 / G neighbouring query rows of one
// sequence: their R*G (row, head) pairs are the 128 tensor-core rows.  The rows
// choose their own segments, but neighbours choose alike, so the CTA walks the
// union of its rows' segments (four rows that take 32 of 256 segments each
// have a union of 57) and a row's weights are 0 where a tile is not its own: a
// warp none of whose rows takes the tile skips the softmax.  The union costs
// less than a tile per row, because the tensor core works on 128 rows whether
// they are filled or not.
//
// Planning: each round the rows' entries are marked in a table of membership
// words for a window of segments (a block with one row takes its list as it
// stands), the marked segments are listed in order, and the list is cut into
// tiles of 64 keys made of quanta (64, 32 or 16 keys that lie in one segment
// and one page).  A cluster of C CTAs takes the tiles in turn when blocks are
// few and merges its partial results through distributed shared memory.
//   warps 0-7  softmax, two threads per tensor-core row (half of the tile's keys
//              each): scores out of tensor memory, -inf where the row does not
//              take the key, weights exp2(s - m) rounded to the input type back
//              into tensor memory over the scores they came from; m moves only
//              when a tile beats it by 2^8, and only then the two threads
//              exchange their maxima and O is rescaled.  Two sums: of the weights
//              as they are rounded, which O is divided by, so that equal values
//              come out as they are (divided by the other sum they would be off
//              by up to a rounding of the largest weight), and of the weights
//              before that, so lse is an fp32 result.  (A product takes both
//              operands in one 16-bit type, so the weights are rounded as the
//              values are: the output is off by 0.0023 of its norm in bf16, where
//              its own rounding alone makes 0.0017.  The parts rounded off could
//              go through a second P V: 260 cycles more in a tile of 930.)
//   warp 8     TMA: a key and a value box per quantum; empty slots take
//              coordinates outside the tensor, which read as zeros
//   warp 9     S = Q K^T one tile ahead of O += P V (P from tensor memory)
// Two CTAs share an SM, one's softmax beside the other's products.  Bound by the
// tensor core and what stands between its products: 4096 rows of 64 heads on 2
// over 16384 keys, 2048 keys a row, take 485 us (0.57 PFLOP/s of what the rows
// ask for, 1.01 of the union's tiles; 471 us with one sum of weights), a tile of
// 64 keys 930 cycles per SM, where
// its products alone need 654 (128x64x16 with both operands in shared memory 49
// cycles, 128x128x16 with the weights in tensor memory 65).  64 decode rows of 64
// heads with 2048 keys each: 20 us, 25 us with the keys in HBM (67 MB: 10 us).
// Measured and not taken: a score buffer less and the queries in tensor memory
// (624 us); 2^x partly by a polynomial (no faster: the exponential is a third of
// a tile's latency, not the limit); at most 64 rows twice in the tensor core with
// the tiles in turn (24 us for the decode rows).
// A key that a row does not take has weight 0 in it, but 0 * inf is NaN: values
// behind the last key that the block sees are zeroed in shared memory, and a
// result that is not finite although its sum of weights is, is computed again by
// itself, key by key (never the case for finite values).  That is slow, 0.36 us
// per key and result, one after another within a block: with one infinite value
// in a segment that all of 512 rows take (32 heads, 2048 keys a row) 93 ms
// instead of 0.1.
#include <cooperative_groups.h>

#include <cmath>
#include <cstdio>

#include "attn_common.cuh"
#include "li_segment.cuh"

namespace li {
void set_launch_count(int32_t n);
cudaError_t set_max_dynamic_smem(const void *kern, int bytes);
}  // namespace li

namespace {

using namespace li;

constexpr int kM = 128;                   // tensor-core rows
constexpr int kTile = 64;                 // keys of a tile
constexpr int kSoftWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + 2);
constexpr int kWarps = kThreads / 32;
constexpr int kPlane = kTile * 128;       // bytes of 64 columns of a tile
constexpr int kMember = 1024;             // membership words, and most listed segments, of a round
constexpr int kMaxSplit = 8;
constexpr float kRescaleLog2 = 8.f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int32_t kNone = 0x7FFFFFFF;

struct AttnArgs {
    SegGeo g;
    const uint16_t *q, *k, *v;
    const int32_t *idx;
    uint16_t *out;
    float *lse;
    float scale, scale_log2;
    int32_t R;                            // query rows per block
    int32_t blocks_per_batch;             // BSND
    int32_t quantum, per;                 // keys of a quantum, quanta of a segment
    int32_t no_page;                      // a page coordinate outside the tensor
};

// Shared memory (bytes from a 1024-byte aligned base).  Key and value tiles are
// 128-byte rows in 64-column planes with the 128-byte swizzle.
template <int D>
struct Layout {
    static constexpr bool QT = D == 64;                     // queries in tensor memory; beside a 128-column O there is room
                                                            // for two score buffers only with the queries in shared memory
    static constexpr int STAGES = D == 128 ? 2 : 4;
    static constexpr int STAGE = kTile * D * 2;
    static constexpr int Q = 0;                             // [D/64][kM][128 B]
    static constexpr int K = QT ? 0 : kM * D * 2;
    static constexpr int V = K + STAGES * STAGE;
    static constexpr int MEMBER = V + STAGES * STAGE;       // uint32 [kMember]
    static constexpr int LIST = MEMBER + kMember * 4;       // int32 [kMember]
    static constexpr int VIS = LIST + kMember * 4;          // int32 [kM]
    static constexpr int CURSOR = VIS + kM * 4;             // int32 [kM]
    static constexpr int LAST = CURSOR + kM * 4;            // int32 [kM]
    static constexpr int MERGE = MEMBER;                    // float [3][kM], then [kM/C+1][C], when the tiles are done
    static constexpr int TOP = LAST + kM * 4;               // float [2][kM]: maxima, then sums, of the half rows
    static constexpr int RING = STAGES + 2;                 // tiles whose masks are held at a time
    static constexpr int MASK = TOP + 2 * kM * 4;           // uint64 [RING][kM]: the keys that a query row takes
    static constexpr int BALL = MASK + RING * kM * 8;       // uint32 [32]
    static constexpr int BARS = BALL + 32 * 4;
    static constexpr int NBARS = 4 * STAGES + 2 + 2 + 1 + 1 + 1 + RING;
    static constexpr int MISC = BARS + NBARS * 8;           // int32 [16]
    static constexpr int END = MISC + 64;
    static constexpr int BYTES = END + 1024;
    static_assert(kM * D * 4 <= MEMBER, "a CTA's partial output stands in the rings");
};

// D (+)= A B with A in tensor memory.
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Inclusive maximum over the lanes up to this one.
__device__ __forceinline__ int32_t scan_max(int32_t v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o && u > v) v = u;
    }
    return v;
}

__device__ __forceinline__ int32_t scan_add(int32_t v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Whether `p` holds in any thread of a pair of warps (64 threads on barrier `id`).
__device__ __forceinline__ bool pair_any(int id, bool p)
{
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((uint32_t)p), "r"(id)
        : "memory");
    return any != 0;
}
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// One (row, head) by the definition, key by key: the whole block works on it.
template <int D, bool F16>
__device__ void attend_plainly(const AttnArgs &a, uint8_t *smem, int32_t row, int32_t h)
{
    float *sq = reinterpret_cast<float *>(smem), *sw = sq + D, *red = sw + 1024;
    int64_t *sat = reinterpret_cast<int64_t *>(red + 32);
    const SegGeo &g = a.g;
    const int32_t n = h / g.G, tid = threadIdx.x, row_elems = g.N2 * D;
    const SegRow r = seg_row(g, row);
    __syncthreads();
    for (int c = tid; c < D; c += kThreads) sq[c] = unpack_lo<F16>(a.q[((int64_t)row * g.N1 + h) * D + c]);
    __syncthreads();
    float m = -INFINITY, l = 0.f, acc = 0.f;
    int32_t last = -1;
    const int32_t segs = (int32_t)(((int64_t)r.Sk + g.seg - 1) / g.seg);
    for (int32_t e = 0; e < (r.vis > 0 ? g.count : 0); ++e) {
        const int32_t s = a.idx[((int64_t)row * g.N2 + n) * g.count + e];
        if (s < 0 || s >= segs || s <= last) continue;
        last = s;
        const int32_t t0 = s * g.seg, cnt = r.vis - t0 < g.seg ? r.vis - t0 : g.seg;
        if (cnt <= 0) continue;
        float mx = -INFINITY;
        for (int32_t t = tid; t < cnt; t += kThreads) {
            const int64_t at = seg_key_offset(g, r.b, r.k_off, t0 + t, row_elems);
            float x = -INFINITY;
            if (at >= 0) {
                x = 0.f;
                for (int c = 0; c < D; ++c) x = fmaf(sq[c], unpack_lo<F16>(a.k[at + n * D + c]), x);
                x *= a.scale;
            }
            sw[t] = x;
            sat[t] = at;
            mx = fmaxf(mx, x);
        }
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if ((tid & 31) == 0) red[tid >> 5] = mx;
        __syncthreads();
        float top = m;
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red[w]);
        const float alpha = top == -INFINITY ? 1.f : expf(m - top);
        m = top;
        l *= alpha;
        acc *= alpha;
        for (int32_t t = 0; t < cnt; ++t) {
            if (sat[t] < 0) continue;
            const float w = sw[t] == -INFINITY ? 0.f : expf(sw[t] - m);
            l += w;
            if (tid < D) acc = fmaf(w, unpack_lo<F16>(a.v[sat[t] + n * D + tid]), acc);
        }
        __syncthreads();
    }
    if (tid < D) {
        const float o = l == 0.f ? 0.f : acc / l;
        const uint32_t w = pack2<F16>(o, o);
        a.out[((int64_t)row * g.N1 + h) * D + tid] = (uint16_t)w;
    }
}

template <int D, bool F16, int C>
__global__ void __launch_bounds__(kThreads, 2)
segattn_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v)
{
    using L = Layout<D>;
    constexpr int NS = L::STAGES;
    constexpr int kColQ = D, kColS = 128;                // tensor memory: O at 0, then the queries (D = 64), two score buffers
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint32_t *member = reinterpret_cast<uint32_t *>(base + L::MEMBER);
    int32_t *list = reinterpret_cast<int32_t *>(base + L::LIST);
    int32_t *svis = reinterpret_cast<int32_t *>(base + L::VIS);
    int32_t *cursor = reinterpret_cast<int32_t *>(base + L::CURSOR);
    int32_t *lastof = reinterpret_cast<int32_t *>(base + L::LAST);
    float *tops = reinterpret_cast<float *>(base + L::TOP);
    uint64_t *masks = reinterpret_cast<uint64_t *>(base + L::MASK);
    uint32_t *ball = reinterpret_cast<uint32_t *>(base + L::BALL);
    uint64_t *kfull = reinterpret_cast<uint64_t *>(base + L::BARS), *kempty = kfull + NS;
    uint64_t *vfull = kempty + NS, *vempty = vfull + NS;
    uint64_t *sfull = vempty + NS, *pfull = sfull + 2, *qfull = pfull + 2, *pvdone = qfull + 1, *odone = pvdone + 1,
             *mfull = odone + 1;
    int32_t *misc = reinterpret_cast<int32_t *>(base + L::MISC);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(misc);
    volatile int *abort_flag = misc + 1;
    int32_t *where = misc + 2;                           // batch, first row, rows, first row's position, Sq
    int32_t *s_next = misc + 7, *s_listed = misc + 8;
    uint32_t *bad = reinterpret_cast<uint32_t *>(misc + 9);   // [4] results to compute again

    const SegGeo &g = a.g;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int32_t blk = blockIdx.x / C, n = blockIdx.y;
    const int rank = C > 1 ? (int)(blockIdx.x % C) : 0;

    // ---- the block's rows
    if (g.layout_q == LI_BSND) {
        if (tid == 0) {
            const int32_t b = blk / a.blocks_per_batch, i0 = (blk - b * a.blocks_per_batch) * a.R;
            where[0] = b;
            where[1] = b * g.S1 + i0;
            where[2] = g.S1 - i0 < a.R ? g.S1 - i0 : a.R;
            where[3] = i0;
            where[4] = g.act_q ? seg_clamp(g.act_q[b], 0, g.S1) : g.S1;
        }
    } else if (warp == 0) {
        // blocks are counted along the sequences; entry B is the rows behind the last one
        int32_t left = blk;
        if (lane == 0) where[2] = 0;
        __syncwarp();
        for (int32_t b0 = 0; b0 <= g.B; b0 += 32) {
            const int32_t b = b0 + lane;
            int32_t start = 0, end = 0;
            if (b <= g.B) {
                start = b ? seg_clamp(g.act_q[b - 1], 0, g.T1) : 0;
                end = b < g.B ? seg_clamp(g.act_q[b], start, g.T1) : g.T1;
            }
            const int32_t mine = (end - start + a.R - 1) / a.R, upto = scan_add(mine, lane);
            const int32_t total = __shfl_sync(0xffffffffu, upto, 31);
            if (left < total) {
                if (left < upto && left >= upto - mine) {
                    const int32_t i0 = (left - (upto - mine)) * a.R;
                    where[0] = b < g.B ? b : g.B - 1;
                    where[1] = start + i0;
                    where[2] = end - start - i0 < a.R ? end - start - i0 : a.R;
                    where[3] = i0;
                    where[4] = b < g.B ? end - start : 0;
                }
                break;
            }
            left -= total;
        }
    }
    if (tid == kThreads - 1) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&kfull[s], 1);
            mbar_init(&kempty[s], 1);
            mbar_init(&vfull[s], 1);
            mbar_init(&vempty[s], 1);
        }
        mbar_init(&sfull[0], 1);
        mbar_init(&sfull[1], 1);
        // the softmax warps; one barrier per score buffer, since a warp without
        // rows may be a tile ahead of the others
        mbar_init(&pfull[0], kSoftWarps);
        mbar_init(&pfull[1], kSoftWarps);
        mbar_init(qfull, kSoftWarps);
        mbar_init(pvdone, 1);
        mbar_init(odone, 1);
        for (int s = 0; s < L::RING; ++s) mbar_init(&mfull[s], 1);
        *abort_flag = 0;
        bad[0] = bad[1] = bad[2] = bad[3] = 0;
        fence_mbarrier_init();
    }
    __syncthreads();
    const int32_t b = where[0], row0 = where[1], nr = where[2], i0 = where[3], Sq = where[4];
    if (nr <= 0) return;                                 // the whole cluster
    if (warp == kSoftWarps + 1) tmem_alloc(tslot, 256);
    int64_t k_off;
    const int32_t Sk = seg_keys(g, b, k_off);
    const int32_t segs = (int32_t)(((int64_t)Sk + g.seg - 1) / g.seg);
    auto sees = [&](int32_t i) {
        if (i >= Sq) return 0;
        return g.mode == 0 ? Sk : seg_clamp((int64_t)i + 1 + Sk - Sq, 0, Sk);
    };
    const int32_t last_row = (i0 + nr < Sq ? i0 + nr : Sq) - 1;
    const int32_t vmax = last_row >= i0 ? sees(last_row) : 0;   // keys that any row of the block sees
    if (tid < kM) {
        svis[tid] = tid < nr ? sees(i0 + tid) : 0;
        cursor[tid] = 0;
        lastof[tid] = -1;
    }
    const int32_t lanes = nr * g.G;                      // tensor-core rows in use
    const int32_t x = tid % kM, side = tid / kM;         // softmax threads: the tensor-core row, half of its columns
    const int32_t rl = x / g.G;                          // its query row
    const bool used = x < lanes;
    const uint32_t tlane = (uint32_t)((warp & 3) * 32) << 16;
    const int64_t at = (int64_t)(row0 + rl) * g.N1 + n * g.G + (x - rl * g.G);
    const bool listed_alone = nr == 1;
    const int32_t MW = (nr + 31) >> 5, W = (kMember / MW) & ~31;

    uint32_t tmem = 0;
    int32_t w0 = 0;
    uint32_t u = 0;                                      // tiles so far (every role counts alike)
    float m_run = -INFINITY, l_run = 0.f, d_run = 0.f;   // maximum; sums of the weights, exact and as they enter P V
    for (bool first = true;; first = false) {
        // ---------------------------------------------------------------- plan
        if (!listed_alone)
            for (int e = tid; e < kMember; e += kThreads) member[e] = 0;
        if (tid == 0) {
            *s_next = kNone;
            if (listed_alone) member[0] = 1;
        }
        if (first) tc_fence_before_sync();
        __syncthreads();
        if (first) {
            tc_fence_after_sync();
            tmem = __shfl_sync(0xffffffffu, *tslot, 0);
        }
        auto entries = [&](int32_t r) { return a.idx + ((int64_t)(row0 + r) * g.N2 + n) * g.count; };
        // 32 entries of a row, its last accepted one being `last`: which are accepted
        // (existing, and above all before them), the last accepted one before each,
        // and the last of all
        auto accept = [&](int32_t s, int32_t last, bool &ok, int32_t &before, int32_t &top) {
            const bool in = s >= 0 && s < segs;
            before = __shfl_up_sync(0xffffffffu, s, 1);
            if (lane == 0) before = last;
            ok = in;
            // as li_segment_select leaves them: ascending, no holes
            if (__all_sync(0xffffffffu, s == -1 || (in && s > before && (before >= 0 || lane == 0)))) {
                const uint32_t m = __ballot_sync(0xffffffffu, in);
                top = m ? __shfl_sync(0xffffffffu, s, 31 - __clz(m)) : last;
                return;
            }
            const int32_t upto = scan_max(in ? s : -1, lane);
            before = __shfl_up_sync(0xffffffffu, upto, 1);
            before = lane == 0 || before < last ? last : before;
            ok = in && s > before;
            if (s != -1 && !ok) seg_flag(g, LI_DEV_BAD_INDEX);
            top = __shfl_sync(0xffffffffu, upto, 31);
            top = top > last ? top : last;
        };
        int32_t listed = 0;
        if (listed_alone) {
            if (warp == 0) {
                const int32_t *src = entries(0), vis = svis[0];
                int32_t last = -1;
                for (int32_t e0 = 0; e0 < (vis > 0 ? g.count : 0); e0 += 32) {
                    const int32_t s = e0 + lane < g.count ? src[e0 + lane] : -1;
                    bool ok;
                    int32_t before, top;
                    accept(s, last, ok, before, top);
                    const bool use = ok && s * g.seg < vis;
                    const uint32_t m = __ballot_sync(0xffffffffu, use);
                    if (use) list[listed + __popc(m & ((1u << lane) - 1u))] = s;
                    listed += __popc(m);
                    last = top;
                }
                if (lane == 0) *s_listed = listed;
            }
            __syncthreads();
            listed = *s_listed;
        } else {
            // four rows' next entries are loaded at a time: one latency, not four
            for (int32_t r0 = warp; r0 < nr; r0 += 4 * kWarps) {
                int32_t ahead[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t r = r0 + j * kWarps;
                    ahead[j] = -1;
                    if (r < nr && svis[r] > 0 && cursor[r] + lane < g.count) ahead[j] = entries(r)[cursor[r] + lane];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t r = r0 + j * kWarps;
                    if (r >= nr || svis[r] <= 0) continue;
                    const int32_t *src = entries(r);
                    const int32_t vis = svis[r];
                    int32_t at = cursor[r], last = lastof[r], next = kNone, s = ahead[j];
                    while (at < g.count) {
                        const int32_t then = at + 32 + lane < g.count ? src[at + 32 + lane] : -1;
                        bool ok;
                        int32_t before, top;
                        accept(s, last, ok, before, top);
                        const bool use = ok && s * g.seg < vis;
                        const uint32_t later = __ballot_sync(0xffffffffu, use && s - w0 >= W);
                        const int end = later ? __ffs(later) - 1 : 32;
                        if (use && lane < end) atomicOr(&member[(s - w0) * MW + (r >> 5)], 1u << (r & 31));
                        if (later) {
                            next = __shfl_sync(0xffffffffu, s, end);
                            last = __shfl_sync(0xffffffffu, before, end);
                            at += end;
                            break;
                        }
                        last = top;
                        at += 32;
                        s = then;
                    }
                    if (lane == 0) {
                        cursor[r] = at;
                        lastof[r] = last;
                        if (next != kNone) atomicMin(s_next, next);
                    }
                }
            }
            __syncthreads();
            for (int grp = warp; grp < W / 32; grp += kWarps) {
                uint32_t any = 0;
                for (int w = 0; w < MW; ++w) any |= member[(grp * 32 + lane) * MW + w];
                const uint32_t m = __ballot_sync(0xffffffffu, any != 0);
                if (lane == 0) ball[grp] = m;
            }
            __syncthreads();
            const int32_t c = lane < W / 32 ? __popc(ball[lane]) : 0;
            const int32_t upto = scan_add(c, lane);
            listed = __shfl_sync(0xffffffffu, upto, 31);
            for (int grp = warp; grp < W / 32; grp += kWarps) {
                const uint32_t m = ball[grp];
                const int32_t before = __shfl_sync(0xffffffffu, upto - c, grp);
                if (m >> lane & 1u) list[before + __popc(m & ((1u << lane) - 1u))] = grp * 32 + lane;
            }
            __syncthreads();
        }
        const int32_t next = *s_next;
        // quanta of the round (the last listed segment may end early), tiles, and this CTA's share
        const int32_t Q = a.quantum, slots = kTile / Q;
        int32_t nq = 0, cut_at = 0;                      // cut_at: the visible keys of the last quantum, when not all
        if (listed > 0) {
            const int32_t left = vmax - (w0 + list[listed - 1]) * g.seg, tail = (left + Q - 1) / Q;
            nq = (listed - 1) * a.per + (tail < a.per ? tail : a.per);
            if (tail <= a.per) cut_at = left % Q;
        }
        const int32_t tiles = (nq + slots - 1) / slots;
        const int32_t mine = tiles > rank ? (tiles - rank + C - 1) / C : 0;
        const int32_t cut_tile = cut_at > 0 && (tiles - 1) % C == rank ? mine - 1 : -1;

        if (warp < kSoftWarps) {
            // ------------------------------------------------------------ softmax
            if (first) {
                // the queries to where the tensor core reads them, half a row per thread (rows
                // without one: zeros)
                uint4 qv[D / 16] = {};
                if (used) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + at * D + side * (D / 2));
#pragma unroll
                    for (int e = 0; e < D / 16; ++e) qv[e] = src[e];
                }
                if constexpr (L::QT) {
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[4 * e] = qv[4 * c + e].x, w[4 * e + 1] = qv[4 * c + e].y, w[4 * e + 2] = qv[4 * c + e].z,
                                  w[4 * e + 3] = qv[4 * c + e].w;
                        tmem_st16(tmem + kColQ + side * (D / 4) + 16 * c + tlane, w);
                    }
                    tmem_st_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < D / 16; ++e)
                        *reinterpret_cast<uint4 *>(base + L::Q + side * (kM * 128) + x * 128 + ((e ^ (x & 7)) << 4)) = qv[e];
                    fence_proxy_async_smem();
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(qfull);
            }
            // which of a tile's keys the row takes
            auto keys_of = [&](uint32_t t) {
                wait_phase(&mfull[t % L::RING], (t / L::RING) & 1, g.status, abort_flag);
                return used ? masks[t % L::RING * kM + rl] : 0;
            };
            uint64_t ahead = mine > 0 ? keys_of(u) : 0;
            for (int32_t k = 0; k < mine; ++k, ++u) {
                const uint32_t sb = u & 1;
                const uint32_t ts = tmem + kColS + sb * kTile + tlane;
                const uint64_t mask = ahead;
                wait_phase(&sfull[sb], (u >> 1) & 1, g.status, abort_flag);
                tc_fence_after_sync();
                if (__any_sync(0xffffffffu, mask != 0)) {        // the same for both warps of a pair
                    uint32_t sq[2][16];
                    tmem_ld16(ts + side * 32, sq[0]);
                    tmem_ld16(ts + side * 32 + 16, sq[1]);
                    tmem_ld_wait16(sq[0]);
                    tmem_ld_wait16(sq[1]);
                    auto sv = [&](int j) -> uint32_t & { return sq[j >> 4][j & 15]; };
                    const uint32_t mine_of = (uint32_t)(mask >> (32 * side));
                    if (!__all_sync(0xffffffffu, mine_of == 0xffffffffu)) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(mine_of >> j & 1u)) sv(j) = 0xff800000u;
                    }
                    float mx[11];
#pragma unroll
                    for (int j = 0; j < 10; ++j)
                        mx[j] = fmax3(__uint_as_float(sv(3 * j)), __uint_as_float(sv(3 * j + 1)),
                                      __uint_as_float(sv(3 * j + 2)));
                    mx[10] = fmaxf(__uint_as_float(sv(30)), __uint_as_float(sv(31)));
                    float mt = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                                     fmax3(fmax3(mx[6], mx[7], mx[8]), mx[9], mx[10])) * a.scale_log2;
                    // (the barrier also stands between the pair's reads of the scores and its
                    // writes of the weights over them)
                    float alpha = 1.f;
                    if (pair_any(1 + (warp & 3), mt > m_run + kRescaleLog2 || (m_run == -INFINITY && mt > -INFINITY))) {
                        tops[side * kM + x] = mt;
                        pair_sync(1 + (warp & 3));
                        mt = fmaxf(mt, tops[(side ^ 1) * kM + x]);
                        if (mt > m_run + kRescaleLog2 || (m_run == -INFINITY && mt > -INFINITY)) {
                            alpha = m_run == -INFINITY ? 0.f : ex2(m_run - mt);
                            m_run = mt;
                        }
                    }
                    const float mb = m_run == -INFINITY ? 0.f : -m_run;
                    float rs[2][2] = {}, rd[2][2] = {};
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float x0, x1;
                        ffma2(x0, x1, __uint_as_float(sv(2 * j)), __uint_as_float(sv(2 * j + 1)), a.scale_log2,
                              a.scale_log2, mb, mb);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        pk[j] = pack2<F16>(x0, x1);
                        fadd2(rs[j & 1][0], rs[j & 1][1], x0, x1);
                        fadd2(rd[j & 1][0], rd[j & 1][1], unpack_lo<F16>(pk[j]), unpack_hi<F16>(pk[j]));
                    }
                    l_run = l_run * alpha + ((rs[0][0] + rs[1][0]) + (rs[0][1] + rs[1][1]));
                    d_run = d_run * alpha + ((rd[0][0] + rd[1][0]) + (rd[0][1] + rd[1][1]));
                    tmem_st16(ts + side * 16, pk);
                    if (u > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                        wait_phase(pvdone, (u - 1) & 1, g.status, abort_flag);
                        tc_fence_after_sync();
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[16];
                            const uint32_t to = tmem + tlane + side * (D / 2) + 16 * c;
                            tmem_ld16(to, o);
                            tmem_ld_wait16(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st16(to, o);
                        }
                    }
                } else {
                    const uint32_t none[16] = {};
                    tmem_st16(ts + side * 16, none);
                }
                if (k + 1 < mine) ahead = keys_of(u + 1);       // while the weights go
                tmem_st_wait();
                if (k == cut_tile) {
                    // values behind the last visible key: zeros
                    const uint32_t vs = u % NS;
                    wait_phase(&vfull[vs], (u / NS) & 1, g.status, abort_flag);
                    const int r0 = (nq - 1) % slots * Q + cut_at, rows = Q - cut_at;
                    for (int e = tid; e < rows * (D / 8); e += 32 * kSoftWarps) {
                        const int r = r0 + e / (D / 8), ch = e % (D / 8);
                        *reinterpret_cast<uint4 *>(base + L::V + vs * L::STAGE + (ch >> 3) * kPlane + r * 128 +
                                                   (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[sb]);
            }
        } else if (warp == kSoftWarps) {
            // ------------------------------------------------------------ copies
            const bool paged = g.layout_kv == LI_PA_BSND;
            int32_t row_vis[4];                          // of rows lane, lane + 32, ...
#pragma unroll
            for (int i = 0; i < 4; ++i) row_vis[i] = svis[32 * i + lane];
            const int32_t batch = 32 / slots;            // tiles whose slots the warp's lanes hold
            int32_t mb = 0, t0 = -1, c1 = 0, c2 = a.no_page;
            // keys go a tile ahead of values, as the scores do
            auto values = [&](uint32_t t, bool my, int32_t v1, int32_t v2) {
                const uint32_t st = t % NS;
                wait_phase(&vempty[st], ((t / NS) & 1) ^ 1u, g.status, abort_flag);
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(&vfull[st], L::STAGE);
                __syncwarp();
                if (my) {
#pragma unroll
                    for (int p = 0; p < D / 64; ++p)
                        tma_load_3d(base + L::V + st * L::STAGE + p * kPlane + lane % slots * Q * 128, &map_v, &vfull[st],
                                    n * D + 64 * p, v1, v2);
                }
            };
            bool v_my = false;
            int32_t v1 = 0, v2 = 0;
            for (int32_t k = 0; k < mine; ++k, ++u) {
                const int32_t j = k % batch;
                if (j == 0) {
                    const int32_t qi = (rank + C * (k + lane / slots)) * slots + lane % slots;
                    t0 = -1, c1 = 0, c2 = a.no_page;
                    if (qi < nq && k + lane / slots < mine) {
                        const int32_t li_ = qi / a.per, at = list[li_];
                        t0 = (w0 + at) * g.seg + (qi - li_ * a.per) * Q;
                        mb = listed_alone ? 0 : at * MW;
                        if (paged) {
                            const int32_t pg = g.bs_shift >= 0 ? t0 >> g.bs_shift : t0 / g.block_size;
                            const int32_t id = g.block_table[(int64_t)b * g.max_blocks_per_seq + pg];
                            if (id >= 0 && id < g.num_blocks) {
                                c1 = t0 - pg * g.block_size;
                                c2 = id;
                            } else {
                                seg_flag(g, LI_DEV_BAD_BLOCK);
                                t0 = -1;
                            }
                        } else {
                            c1 = (int32_t)(k_off + t0);
                            c2 = 0;
                        }
                    }
                }
                const bool my = lane / slots == j;
                const int32_t slot = lane % slots;
                const uint32_t st = u % NS, ph = ((u / NS) & 1) ^ 1u;
                wait_phase(&kempty[st], ph, g.status, abort_flag);
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(&kfull[st], L::STAGE);
                __syncwarp();
                if (my) {
#pragma unroll
                    for (int p = 0; p < D / 64; ++p)
                        tma_load_3d(base + L::K + st * L::STAGE + p * kPlane + slot * Q * 128, &map_k, &kfull[st],
                                    n * D + 64 * p, c1, c2);
                }
                // the rows' masks; the entry's last reader, the softmax of tile u - RING, was
                // done before the scores that this key stage has held since were issued
                uint64_t m[4] = {};
                for (int32_t s = 0; s < slots; ++s) {
                    const int32_t from = __shfl_sync(0xffffffffu, t0, j * slots + s);
                    const int32_t at = __shfl_sync(0xffffffffu, mb, j * slots + s);
                    if (from < 0) continue;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i >= MW) break;
                        const int32_t c = row_vis[i] - from;       // keys of the quantum that the row sees
                        const int32_t cc = c < 1 ? 1 : (c < Q ? c : Q);
                        const bool takes = (c > 0) & ((member[at + i] >> lane & 1u) != 0);
                        m[i] |= takes ? ~0ull >> (64 - cc) << (s * Q) : 0ull;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < MW) masks[u % L::RING * kM + 32 * i + lane] = m[i];
                __syncwarp();
                if (lane == 0) mbar_arrive(&mfull[u % L::RING]);
                if (k > 0) values(u - 1, v_my, v1, v2);
                v_my = my, v1 = c1, v2 = c2;
            }
            if (mine > 0) values(u - 1, v_my, v1, v2);
        } else {
            // ------------------------------------------------------------ products
            // (the whole warp runs the loop and one lane issues: addresses and
            // descriptors then stay in uniform registers)
            const bool leader = elect_one();
            const uint32_t fmt = F16 ? 0u : 1u, sbase = smem_u32(base);
            const uint32_t id_s = make_idesc(fmt, fmt, kM, kTile);
            const uint32_t id_pv = make_idesc(fmt, fmt, kM, D) | (1u << 16);      // values MN-major
            const int32_t todo = __shfl_sync(0xffffffffu, mine, 0);
            if (first) wait_phase(qfull, 0, g.status, abort_flag);
            const uint64_t qd = smem_desc_sw128(sbase + L::Q);
            auto weigh = [&](uint32_t t) {               // O += P V of tile t
                const uint32_t st = t % NS, sb = t & 1;
                wait_phase(&pfull[sb], (t >> 1) & 1, g.status, abort_flag);
                wait_phase(&vfull[st], (t / NS) & 1, g.status, abort_flag);
                tc_fence_after_sync();
                __syncwarp();
                if (leader) {
                    const uint64_t vd = smem_desc_sw128_mn(sbase + L::V + st * L::STAGE, kPlane, 1024);
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        mma_f16_ta(tmem, tmem + kColS + sb * kTile + 8 * kk, vd + kk * (16 * 128 / 16), id_pv,
                                   (t > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(&vempty[st]);
                    mma_commit(pvdone);
                }
                __syncwarp();
            };
            for (int32_t k = 0; k < todo; ++k, ++u) {
                const uint32_t st = u % NS, sb = u & 1;
                wait_phase(&kfull[st], (u / NS) & 1, g.status, abort_flag);
                // the buffer's last weights have been read (before a round's first tile
                // all have: a wait for them now could take a later phase for theirs)
                if (k > 0 && u >= 2) wait_phase(pvdone, u & 1, g.status, abort_flag);
                tc_fence_after_sync();
                __syncwarp();
                if (leader) {
                    const uint64_t kd = smem_desc_sw128(sbase + L::K + st * L::STAGE);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        if constexpr (L::QT)
                            mma_f16_ta(tmem + kColS + sb * kTile, tmem + kColQ + 8 * kk, kd + kk * 2, id_s, kk != 0);
                        else
                            mma_f16(tmem + kColS + sb * kTile, qd + ((kk >> 2) * (kM * 128) + (kk & 3) * 32) / 16,
                                    kd + ((kk >> 2) * kPlane + (kk & 3) * 32) / 16, id_s, kk != 0);
                    mma_commit(&sfull[sb]);
                    mma_commit(&kempty[st]);
                }
                __syncwarp();
                if (k > 0) weigh(u - 1);
            }
            if (todo > 0) {
                if (u >= 2) wait_phase(pvdone, u & 1, g.status, abort_flag);
                __syncwarp();
                weigh(u - 1);
                wait_phase(pvdone, (u - 1) & 1, g.status, abort_flag);
            }
            // a barrier of its own for the end: whoever waits for it late must not
            // take a later phase of pvdone for an earlier one
            if (next == kNone && leader) mma_commit(odone);
        }
        __syncwarp();
        if (next == kNone) break;                        // the same for every thread, and every CTA of the cluster
        w0 = next;
        __syncthreads();
    }

    // -------------------------------------------------------------------- results
    // every role has counted this CTA's tiles in u
    if (warp < kSoftWarps) {
        if (u > 0) {
            wait_phase(odone, 0, g.status, abort_flag);
            tc_fence_after_sync();
        }
        tops[side * kM + x] = l_run;
        pair_sync(1 + (warp & 3));
        l_run += tops[(side ^ 1) * kM + x];              // (of two summands: the same in both threads)
        pair_sync(1 + (warp & 3));
        tops[side * kM + x] = d_run;
        pair_sync(1 + (warp & 3));
        d_run += tops[(side ^ 1) * kM + x];
        float *sO = reinterpret_cast<float *>(base);     // [kM][D], 16-byte chunks of row r at c ^ (r & 15)
        const float inv = d_run == 0.f ? 0.f : 1.f / d_run;
        bool odd = false;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const int col = side * (D / 2) + 16 * c;
            uint32_t o[16] = {};
            if (u > 0) {
                tmem_ld16(tmem + tlane + col, o);
                tmem_ld_wait16(o);
            }
            if constexpr (C == 1) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y0 = __uint_as_float(o[2 * e]) * inv, y1 = __uint_as_float(o[2 * e + 1]) * inv;
                    odd |= !finite(y0) || !finite(y1);
                    w[e] = pack2<F16>(y0, y1);
                }
                if (used) {
                    uint4 *dst = reinterpret_cast<uint4 *>(a.out + at * D + col);
                    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    reinterpret_cast<uint4 *>(sO)[x * (D / 4) + ((col / 4 + e) ^ (x & 15))] =
                        make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
        }
        if constexpr (C == 1) {
            const uint32_t m = __ballot_sync(0xffffffffu, used && odd && finite(l_run));
            if (lane == 0 && m) atomicOr(&bad[warp & 3], m);
            if (side == 0 && used && a.lse) a.lse[at] = l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
        } else if (side == 0) {
            float *sM = reinterpret_cast<float *>(base + L::MERGE);
            sM[x] = m_run;
            sM[kM + x] = l_run;
            sM[2 * kM + x] = d_run;
        }
    }
    if constexpr (C > 1) {
        // CTA `rank` merges its share of the tensor-core rows over the C partials
        float *sO = reinterpret_cast<float *>(base);
        float *sM = reinterpret_cast<float *>(base + L::MERGE), *sL = sM + kM, *sD = sL + kM;
        cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
        cl.sync();
        const int32_t share = (lanes + C - 1) / C, from = rank * share;
        const int32_t cnt = lanes - from < share ? (lanes > from ? lanes - from : 0) : share;
        auto out_at = [&](int32_t y) { return (int64_t)(row0 + y / g.G) * g.N1 + n * g.G + y % g.G; };
        float *sums = sD + kM;                           // weight of partial r for row x: [share][C]
        for (int e = tid; e < cnt * C; e += kThreads) {
            const int y = from + e / C, r = e % C;
            float top = -INFINITY, sum = 0.f, div = 0.f;
#pragma unroll
            for (int p = 0; p < C; ++p) top = fmaxf(top, cl.map_shared_rank(sM, p)[y]);
#pragma unroll
            for (int p = 0; p < C; ++p) {
                const float mp = cl.map_shared_rank(sM, p)[y], lp = cl.map_shared_rank(sL, p)[y];
                const float f = mp == -INFINITY ? 1.f : exp2f(mp - top);
                if (lp != 0.f) sum += lp * f, div += cl.map_shared_rank(sD, p)[y] * f;
            }
            const float mr = cl.map_shared_rank(sM, r)[y], lr = cl.map_shared_rank(sL, r)[y];
            sums[e] = lr == 0.f ? 0.f : (mr == -INFINITY ? 1.f : exp2f(mr - top)) / div;
            if (r == 0 && a.lse) a.lse[out_at(y)] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
        }
        __syncthreads();
        for (int e = tid; e < cnt * (D / 4); e += kThreads) {
            const int hl = e / (D / 4), ch = e % (D / 4), y = from + hl;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            bool whole = true;                           // every weight is finite
#pragma unroll
            for (int r = 0; r < C; ++r) {
                const float w = sums[hl * C + r];
                whole &= finite(w);
                if (w != 0.f) {
                    const float4 o = reinterpret_cast<const float4 *>(cl.map_shared_rank(sO, r))[y * (D / 4) + (ch ^ (y & 15))];
                    acc.x = fmaf(w, o.x, acc.x);
                    acc.y = fmaf(w, o.y, acc.y);
                    acc.z = fmaf(w, o.z, acc.z);
                    acc.w = fmaf(w, o.w, acc.w);
                }
            }
            if (whole && !(finite(acc.x) && finite(acc.y) && finite(acc.z) && finite(acc.w)))
                atomicOr(&bad[y >> 5], 1u << (y & 31));
            *reinterpret_cast<uint2 *>(a.out + out_at(y) * D + 4 * ch) =
                make_uint2(pack2<F16>(acc.x, acc.y), pack2<F16>(acc.z, acc.w));
        }
        cl.sync();                                       // every peer has read this CTA's partials
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kSoftWarps + 1) tmem_dealloc(tmem, 256);
    for (int w = 0; w < 4; ++w)
        for (uint32_t m = bad[w]; m; m &= m - 1) {
            const int32_t y = 32 * w + __ffs(m) - 1;
            attend_plainly<D, F16>(a, base, row0 + y / g.G, n * g.G + y % g.G);
        }
}

template <int D, bool F16, int C>
cudaError_t launch(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int64_t blocks, cudaStream_t s)
{
    auto kern = segattn_kernel<D, F16, C>;
    const int smem = Layout<D>::BYTES;
    cudaError_t e = li::set_max_dynamic_smem(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * C), (unsigned)a.g.N2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, mk, mv);
}

template <int D, bool F16>
cudaError_t launch_split(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int64_t blocks, int split,
                         cudaStream_t s)
{
    switch (split) {
    case 1: return launch<D, F16, 1>(a, mk, mv, blocks, s);
    case 2: return launch<D, F16, 2>(a, mk, mv, blocks, s);
    case 4: return launch<D, F16, 4>(a, mk, mv, blocks, s);
    case 8: return launch<D, F16, 8>(a, mk, mv, blocks, s);
    }
    return cudaErrorInvalidValue;
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
    if (a.g.rows == 0) return LI_OK;                     // empty tensors have no address
    if (seg_no_keys(a.g)) key = value = query;           // to have one: nothing is read there
    if (!query || !key || !value || !seg_idx || !out)
        return seg_fail(call, LI_ERR_NULL, "query, key, value, seg_idx and out are required");
    if (off(query, 16) || off(key, 16) || off(value, 16) || off(out, 16) || off(seg_idx, 4) || off(lse, 4))
        return seg_fail(call, LI_ERR_SHAPE, "query, key, value and out must be 16-byte aligned, seg_idx and lse 4-byte");
    a.q = static_cast<const uint16_t *>(query);
    a.k = static_cast<const uint16_t *>(key);
    a.v = static_cast<const uint16_t *>(value);
    a.idx = seg_idx;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.scale = p->softmax_scale;
    a.scale_log2 = p->softmax_scale * 1.4426950408889634f;
    const SegGeo &g = a.g;
    a.quantum = kTile;
    while (g.seg % a.quantum || (g.layout_kv == LI_PA_BSND && g.block_size % a.quantum)) a.quantum /= 2;
    a.per = g.seg / a.quantum;
    a.R = kM / g.G;
    int64_t blocks;
    if (g.layout_q == LI_BSND) {
        a.blocks_per_batch = (g.S1 + a.R - 1) / a.R;
        blocks = (int64_t)g.B * a.blocks_per_batch;
    } else {
        // the sequences' blocks and those of the rows behind them: at most one of each is not full
        blocks = ((int64_t)g.T1 + ((int64_t)g.B + 1) * (a.R - 1)) / a.R;
        if (blocks > g.T1) blocks = g.T1;
    }
    // rows of the key tensor as a box of quantum x 64 columns sees them
    const bool paged = g.layout_kv == LI_PA_BSND;
    const int64_t dense_rows = g.layout_kv == LI_BSND ? (int64_t)g.B * g.S2 : g.T2;
    const int64_t rows = paged ? g.block_size : (dense_rows > 0 ? dense_rows : 1);
    const int64_t pages = paged ? g.num_blocks : 1;
    const int64_t pitch = (int64_t)g.N2 * p->D * 2;
    a.no_page = (int32_t)pages;
    const uint64_t dims[3] = {(uint64_t)g.N2 * p->D, (uint64_t)rows, (uint64_t)pages};
    const uint64_t strides[2] = {(uint64_t)pitch, (uint64_t)(paged ? g.page_stride * 2 : pitch)};
    const uint32_t box[3] = {64, (uint32_t)a.quantum, 1};
    CUtensorMap mk, mv;
    li_status es = li::tensor_map_16bit(&mk, key, 3, dims, strides, box, "segment keys");
    if (es == LI_OK) es = li::tensor_map_16bit(&mv, value, 3, dims, strides, box, "segment values");
    if (es != LI_OK) return es;
    // CTAs per block: while the grid stays within one wave of two CTAs per SM
    // and every CTA keeps two tiles of what its rows may take
    const int64_t most = paged ? (int64_t)g.max_blocks_per_seq * g.block_size : (g.layout_kv == LI_BSND ? g.S2 : g.T2);
    // (rows that share a block take about twice what one takes; 100 rows of 6
    // segments: 14.4 us so, 16.5 us counted as one)
    const bool shared = a.R > 1 && (g.layout_q == LI_BSND ? g.S1 > 1 : g.T1 > g.B);
    const int64_t some = (int64_t)g.count * g.seg * (shared ? 2 : 1), keys = some < most ? some : most;
    const int64_t wave = 2LL * seg_sms();
    int split = 1;
    while (split < kMaxSplit && blocks * g.N2 * split * 2 <= wave && keys >= (int64_t)split * 2 * 2 * kTile) split *= 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f16 = p->dtype == LI_FP16;
    const cudaError_t e = p->D == 128 ? (f16 ? launch_split<128, true>(a, mk, mv, blocks, split, s)
                                             : launch_split<128, false>(a, mk, mv, blocks, split, s))
                                      : (f16 ? launch_split<64, true>(a, mk, mv, blocks, split, s)
                                             : launch_split<64, false>(a, mk, mv, blocks, split, s));
    if (e != cudaSuccess) return seg_fail(call, LI_ERR_CUDA, cudaGetErrorString(e));
    li::set_launch_count(1);
    return LI_OK;
}
