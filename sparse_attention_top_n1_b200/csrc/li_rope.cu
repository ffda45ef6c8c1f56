// li_rope.cu -- rotary positions of query and key heads, one launch for both.
//
// Every pair of a head is read once, turned by position * inv_freq, and
// written once: the call moves 2 * rows * (N1 + N2) * D elements and is bound
// by HBM.  What could get in its way is the angle: position * inv_freq has to
// be right to about 2^-25 of a turn at positions in the millions, which fp32
// cannot hold.  So the angle is taken in turns in 64 bits, its whole turns are
// dropped there, and only the rest (|f| <= 1/2) goes to fp32 and sincospi.
// That is one fp64 product and one sincos per (row, pair), computed once per
// block into shared memory and shared by all heads of the row.
//
// A block takes the rows of four batches of loads (with one, its start and the
// angles are not covered: 387 us for 30720 rows of 72 heads of 128, against 241),
// and loads and stores are marked as used once (186 us: 6.1 of 6.56 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>

#include "li.h"

namespace li {
li_status report_error(li_status s, const char *msg);
void set_launch_count(int32_t n);
}  // namespace li

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;              // units a thread has in flight
constexpr int kStaged = 24576;         // bytes of heads that a block turns in shared memory at a time
constexpr int kTable = 4096;           // (cos, sin) pairs of one block: 32 KB

struct Head {                          // one tensor and its output
    const void *in;
    void *out;
    int64_t row, head, out_row, out_head;   // strides in elements
};

struct RopeArgs {
    Head q, k;
    const int32_t *positions;
    const double *inv_freq;
    int32_t rows, N1, N2, D, half, off;     // half = rot_dim / 2
    int32_t row_tile, heads_per_block;
    uint32_t mul_row, mul_head, mul_half;   // ceil(2^32 / units of a row, of a head, pairs of a head) (0: divide by one)
    bool one_row;                           // (staged) blocks of one row
    float mscale, sin_sign;
    int32_t copy_rest;                      // out of place: columns outside the turned part
};

// Bytes of V elements as one register type.
template <int BYTES> struct Raw;
template <> struct Raw<16> { using T = uint4; };
template <> struct Raw<8> { using T = uint2; };
template <> struct Raw<4> { using T = uint32_t; };
template <> struct Raw<2> { using T = uint16_t; };

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// u / d with m = ceil(2^32 / d), for u * d < 2^32
__device__ __forceinline__ uint32_t quotient(uint32_t u, uint32_t m) { return m ? __umulhi(u, m) : u; }

// cos and sin of pair e % half of row row0 + e / half
__device__ __forceinline__ float2 angle(const RopeArgs &a, int64_t row0, int e)
{
    constexpr double kInvTwoPi = 0.15915494309189533576888;
    const int r = e / a.half, p = e - r * a.half;
    const double t = (double)a.positions[row0 + r] * (a.inv_freq[p] * kInvTwoPi);
    float s, c;
    sincospif(2.f * (float)(t - rint(t)), &s, &c);
    return make_float2(c * a.mscale, s * a.mscale * a.sin_sign);
}

template <typename T, int V> union Vec {
    typename Raw<sizeof(T) * V>::T raw;
    T e[V];
    __device__ Vec() {}
};

// A unit is what one thread turns at a time.  HALF: V pairs, read as V
// elements of each half.  Interleaved: V/2 pairs, V neighbouring elements (one
// pair, two elements, when V = 1).
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a)
{
    constexpr bool kTwo = HALF || V == 1;               // two accesses per unit
    constexpr int kPairs = HALF ? V : (V == 1 ? 1 : V / 2);
    extern __shared__ float2 table[];                   // [row_tile][half]
    const int tid = threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * a.row_tile;
    const int nrows = (int)(a.rows - row0 < a.row_tile ? a.rows - row0 : a.row_tile);
    const int head0 = blockIdx.y * a.heads_per_block;
    const int heads_all = a.N1 + a.N2;
    const int nheads = heads_all - head0 < a.heads_per_block ? heads_all - head0 : a.heads_per_block;
    const uint32_t per_head = (uint32_t)(a.half / kPairs);
    const uint32_t per_row = per_head * (uint32_t)nheads;
    const uint32_t units = per_row * (uint32_t)nrows;

    auto locate = [&](uint32_t r, uint32_t hl, const T *&in, T *&out) {
        const int h = head0 + (int)hl;
        const int64_t row = row0 + r;
        const Head &t = h < a.N1 ? a.q : a.k;
        const int hh = h < a.N1 ? h : h - a.N1;
        in = static_cast<const T *>(t.in) + row * t.row + hh * t.head;
        out = static_cast<T *>(t.out) + row * t.out_row + hh * t.out_head;
    };

    Vec<T, V> x[kBatch][kTwo ? 2 : 1];
    T *dst[kBatch];
    uint32_t at[kBatch];                                // table entry of the unit's first pair
    for (uint32_t base = 0; base < units; base += kThreads * kBatch) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const uint32_t u = base + j * kThreads + tid;
            if (u < units) {
                const uint32_t r = a.row_tile > 1 ? quotient(u, a.mul_row) : 0u, w = u - r * per_row;
                const uint32_t hl = quotient(w, a.mul_head), p = (w - hl * per_head) * kPairs;
                const T *in;
                locate(r, hl, in, dst[j]);
                const int c = a.off + (HALF ? (int)p : 2 * (int)p);
                dst[j] += c;
                in += c;
                at[j] = r * a.half + p;
                x[j][0].raw = __ldcs(reinterpret_cast<const typename Raw<sizeof(T) * V>::T *>(in));
                if constexpr (kTwo)
                    x[j][1].raw = __ldcs(reinterpret_cast<const typename Raw<sizeof(T) * V>::T *>(in + (HALF ? a.half : 1)));
            }
        }
        if (base == 0) {
            // the block's angles, while the first loads are under way
            for (int e = tid; e < nrows * a.half; e += kThreads) table[e] = angle(a, row0, e);
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const uint32_t u = base + j * kThreads + tid;
            if (u < units) {
#pragma unroll
                for (int e = 0; e < kPairs; ++e) {
                    T &e0 = kTwo ? x[j][0].e[HALF ? e : 0] : x[j][0].e[2 * e];
                    T &e1 = kTwo ? x[j][kTwo ? 1 : 0].e[HALF ? e : 0] : x[j][0].e[2 * e + 1];
                    const float2 cs = table[at[j] + e];
                    const float u0 = to_f<T>(e0), u1 = to_f<T>(e1);
                    e0 = from_f<T>(u0 * cs.x - u1 * cs.y);
                    e1 = from_f<T>(u1 * cs.x + u0 * cs.y);
                }
                __stcs(reinterpret_cast<typename Raw<sizeof(T) * V>::T *>(dst[j]), x[j][0].raw);
                if constexpr (kTwo)
                    __stcs(reinterpret_cast<typename Raw<sizeof(T) * V>::T *>(dst[j] + (HALF ? a.half : 1)), x[j][1].raw);
            }
        }
    }
    if (!a.copy_rest) return;
    // the columns outside the turned part, V at a time
    const uint32_t rest = (uint32_t)((a.D - 2 * a.half) / V);
    const uint32_t rest_row = rest * (uint32_t)nheads, n = rest_row * (uint32_t)nrows;
    for (uint32_t u = tid; u < n; u += kThreads) {
        const uint32_t r = u / rest_row, w = u - r * rest_row;
        const uint32_t hl = w / rest;
        int c = (int)(w - hl * rest) * V;
        if (c >= a.off) c += 2 * a.half;
        const T *in;
        T *out;
        locate(r, hl, in, out);
        *reinterpret_cast<typename Raw<sizeof(T) * V>::T *>(out + c) =
            *reinterpret_cast<const typename Raw<sizeof(T) * V>::T *>(in + c);
    }
}

// Heads whose turned part does not start or split on 16 bytes, though the heads
// themselves lie on them: whole heads come and go in 16-byte accesses, and the
// pairs are turned in shared memory, where narrow accesses cost little (20000
// rows of 72 heads of 128, 90 columns turned from column 30 on: 158 us, 404 us
// with the 4-byte accesses that the pairs allow; 64 rows 3.4 and 4.2 us).
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_staged_kernel(const RopeArgs a)
{
    constexpr int V = 16 / (int)sizeof(T);
    extern __shared__ uint4 stage[];                    // [kStaged bytes], then the angles [row_tile][half]
    float2 *table = reinterpret_cast<float2 *>(reinterpret_cast<char *>(stage) + kStaged);
    const int tid = threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * a.row_tile;
    const int nrows = (int)(a.rows - row0 < a.row_tile ? a.rows - row0 : a.row_tile);
    const int head0 = blockIdx.y * a.heads_per_block;
    const int heads_all = a.N1 + a.N2;
    const uint32_t nheads = (uint32_t)(heads_all - head0 < a.heads_per_block ? heads_all - head0 : a.heads_per_block);
    const uint32_t vecs = (uint32_t)(a.D / V), n = nheads * (uint32_t)nrows;     // vectors of a head; heads of the block
    const uint32_t most = (uint32_t)kStaged / 16 / vecs;
    for (int e = tid; e < nrows * a.half; e += kThreads) table[e] = angle(a, row0, e);
    for (uint32_t h0 = 0; h0 < n; h0 += most) {
        const uint32_t cnt = n - h0 < most ? n - h0 : most;
        auto place = [&](uint32_t e, bool in) -> uint4 * {     // vector e of these heads
            const uint32_t hr = quotient(e, a.mul_head), c = e - hr * vecs;
            const uint32_t r = a.one_row ? 0u : quotient(h0 + hr, a.mul_row);
            const int h = head0 + (int)(h0 + hr - r * nheads);
            const Head &t = h < a.N1 ? a.q : a.k;
            const int hh = h < a.N1 ? h : h - a.N1;
            const T *p = in ? static_cast<const T *>(t.in) + (row0 + r) * t.row + hh * t.head
                            : static_cast<const T *>(t.out) + (row0 + r) * t.out_row + hh * t.out_head;
            return reinterpret_cast<uint4 *>(const_cast<T *>(p)) + c;
        };
        for (uint32_t e0 = 0; e0 < cnt * vecs; e0 += kThreads * kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const uint32_t e = e0 + j * kThreads + tid;
                if (e < cnt * vecs) x[j] = __ldcs(place(e, true));
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const uint32_t e = e0 + j * kThreads + tid;
                if (e < cnt * vecs) stage[e] = x[j];
            }
        }
        __syncthreads();
        for (uint32_t u = tid; u < cnt * (uint32_t)a.half; u += kThreads) {
            const uint32_t hr = quotient(u, a.mul_half), p = u - hr * a.half;
            const uint32_t r = a.one_row ? 0u : quotient(h0 + hr, a.mul_row);
            T *head = reinterpret_cast<T *>(stage) + hr * a.D + a.off;
            T &e0 = head[HALF ? p : 2 * p], &e1 = head[HALF ? p + a.half : 2 * p + 1];
            const float2 cs = table[r * a.half + p];
            const float u0 = to_f<T>(e0), u1 = to_f<T>(e1);
            e0 = from_f<T>(u0 * cs.x - u1 * cs.y);
            e1 = from_f<T>(u1 * cs.x + u0 * cs.y);
        }
        __syncthreads();
        for (uint32_t e = tid; e < cnt * vecs; e += kThreads) __stcs(place(e, false), stage[e]);
        __syncthreads();
    }
}

uint32_t magic(uint32_t d) { return d > 1 ? 0xFFFFFFFFu / d + 1 : 0u; }

template <typename T, bool HALF>
cudaError_t launch_staged(RopeArgs a, int sms, cudaStream_t s)
{
    const int64_t heads = a.N1 + a.N2, per_row = heads * a.D * (int64_t)sizeof(T);
    int64_t tile = 2 * kStaged / per_row;               // two fillings of the stage
    if (tile > kTable / 2 / a.half) tile = kTable / 2 / a.half;
    if (tile > a.rows / (4 * sms)) tile = a.rows / (4 * sms);
    if (tile < 1) tile = 1;
    a.row_tile = (int)tile;
    int64_t grid_x = (a.rows + tile - 1) / tile, grid_y = 1;
    if (tile == 1) {
        grid_y = 2 * sms / grid_x;
        if (grid_y > heads) grid_y = heads;
        if (grid_y < 1) grid_y = 1;
    }
    a.heads_per_block = (int)((heads + grid_y - 1) / grid_y);
    grid_y = (heads + a.heads_per_block - 1) / a.heads_per_block;
    a.mul_head = magic((uint32_t)(a.D * (int)sizeof(T) / 16));
    a.mul_half = magic((uint32_t)a.half);
    // of a block's last, shorter run of heads too: rows are counted by heads_per_block
    // only when one block takes them all
    a.mul_row = tile == 1 ? 0u : magic((uint32_t)a.heads_per_block);
    a.one_row = tile == 1;
    rope_staged_kernel<T, HALF><<<dim3((unsigned)grid_x, (unsigned)grid_y), kThreads,
                                  kStaged + (size_t)tile * a.half * sizeof(float2), s>>>(a);
    return cudaGetLastError();
}

template <typename T, int V, bool HALF>
cudaError_t launch(RopeArgs a, int sms, cudaStream_t s)
{
    constexpr int kPairs = HALF ? V : (V == 1 ? 1 : V / 2);
    const int64_t heads = a.N1 + a.N2;
    const int64_t per_row = heads * (a.half / kPairs);
    // rows per block: about four batches of units, within the angle table, and
    // not so many that SMs stay idle; few rows: the heads are split instead
    int64_t tile = 4LL * kThreads * kBatch / per_row;
    if (tile > kTable / a.half) tile = kTable / a.half;
    if (tile > a.rows / (4 * sms)) tile = a.rows / (4 * sms);
    if (tile < 1) tile = 1;
    a.row_tile = (int)tile;
    int64_t grid_x = (a.rows + tile - 1) / tile, grid_y = 1;
    if (tile == 1) {
        const int64_t most = (per_row + kThreads - 1) / kThreads;       // a block's threads one unit each
        grid_y = 2 * sms / grid_x;
        if (grid_y > most) grid_y = most;
        if (grid_y > heads) grid_y = heads;
        if (grid_y < 1) grid_y = 1;
    }
    a.heads_per_block = (int)((heads + grid_y - 1) / grid_y);
    grid_y = (heads + a.heads_per_block - 1) / a.heads_per_block;
    const uint32_t head_units = (uint32_t)(a.half / kPairs), row_units = head_units * (uint32_t)a.heads_per_block;
    a.mul_row = magic(row_units);
    a.mul_head = magic(head_units);
    rope_kernel<T, V, HALF><<<dim3((unsigned)grid_x, (unsigned)grid_y), kThreads,
                              (size_t)tile * a.half * sizeof(float2), s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RopeArgs &a, bool half, int v, bool staged, int sms, cudaStream_t s)
{
    constexpr int kWide = 16 / (int)sizeof(T);
    if (v < kWide && staged) return half ? launch_staged<T, true>(a, sms, s) : launch_staged<T, false>(a, sms, s);
    if (half) {
        if (v >= kWide) return launch<T, kWide, true>(a, sms, s);
        if (v >= 2) return launch<T, 2, true>(a, sms, s);
        return launch<T, 1, true>(a, sms, s);
    }
    if (v >= kWide) return launch<T, kWide, false>(a, sms, s);
    if (v >= 2) return launch<T, 2, false>(a, sms, s);
    return launch<T, 1, false>(a, sms, s);
}

li_status bad(li_status st, const char *what)
{
    char msg[160];
    snprintf(msg, sizeof msg, "li_rope: %s", what);
    return li::report_error(st, msg);
}

}  // namespace

extern "C" LI_API li_status li_rope(const li_rope_params *p, const int32_t *positions, const double *inv_freq,
                                    const void *query, const void *key, void *query_out, void *key_out,
                                    void *stream)
{
    li::set_launch_count(0);
    if (!p) return bad(LI_ERR_NULL, "params is NULL");
    if (p->reserved != 0) return bad(LI_ERR_SHAPE, "reserved must be 0");
    if (p->dtype != LI_BF16 && p->dtype != LI_FP16 && p->dtype != LI_FP32)
        return bad(LI_ERR_DTYPE, "dtype must be LI_BF16, LI_FP16 or LI_FP32");
    if (p->pairing != LI_ROPE_HALF && p->pairing != LI_ROPE_INTERLEAVED)
        return bad(LI_ERR_LAYOUT, "pairing must be LI_ROPE_HALF or LI_ROPE_INTERLEAVED");
    if (p->inverse != 0 && p->inverse != 1) return bad(LI_ERR_SHAPE, "inverse must be 0 or 1");
    if (p->rows < 0) return bad(LI_ERR_SHAPE, "rows must be >= 0");
    if (p->N1 < 1 || p->N1 > 1024 || p->N2 < 0 || p->N2 > 1024)
        return bad(LI_ERR_SHAPE, "N1 must be in [1, 1024] and N2 in [0, 1024]");
    if (p->D < 2 || p->D > 1024) return bad(LI_ERR_SHAPE, "D must be in [2, 1024]");
    if (p->rot_dim < 2 || p->rot_dim % 2 || p->rot_offset < 0 || p->rot_dim > p->D || p->rot_offset > p->D - p->rot_dim)
        return bad(LI_ERR_SHAPE, "rot_dim must be even and rot_offset + rot_dim within the head");
    if (!(p->mscale > 0.f) || !std::isfinite(p->mscale)) return bad(LI_ERR_SHAPE, "mscale must be positive and finite");
    RopeArgs a{};
    auto head = [&](const void *in, void *out, int n, int64_t row, int64_t hd, int64_t orow, int64_t ohd, Head &t) {
        t.in = in;
        t.out = out;
        t.head = hd ? hd : p->D;
        t.out_head = ohd ? ohd : p->D;
        t.row = row ? row : (int64_t)n * p->D;
        t.out_row = orow ? orow : (int64_t)n * p->D;
        const int64_t lim = (int64_t)1 << 40;
        return t.head >= p->D && t.out_head >= p->D && t.head < lim && t.out_head < lim && t.row < lim &&
               t.out_row < lim && t.row >= (n - 1) * t.head + p->D && t.out_row >= (n - 1) * t.out_head + p->D;
    };
    if (!head(query, query_out, p->N1, p->q_row_stride, p->q_head_stride, p->q_out_row_stride, p->q_out_head_stride, a.q) ||
        (p->N2 && !head(key, key_out, p->N2, p->k_row_stride, p->k_head_stride, p->k_out_row_stride,
                        p->k_out_head_stride, a.k)))
        return bad(LI_ERR_SHAPE, "strides let heads or rows overlap");
    if (p->rows == 0) return LI_OK;                    // empty tensors have no address
    if (!positions || !inv_freq || !query || !query_out) return bad(LI_ERR_NULL, "a required pointer is NULL");
    if ((p->N2 > 0) != (key != nullptr) || (p->N2 > 0) != (key_out != nullptr))
        return bad(LI_ERR_NULL, "key and key_out go with N2 > 0");
    const bool q_in = query == query_out, k_in = p->N2 == 0 || key == key_out;
    if ((q_in && (a.q.row != a.q.out_row || a.q.head != a.q.out_head)) ||
        (p->N2 && k_in && (a.k.row != a.k.out_row || a.k.head != a.k.out_head)))
        return bad(LI_ERR_SHAPE, "in place needs the same strides for input and output");
    const uintptr_t es = p->dtype == LI_FP32 ? 4 : 2;
    uintptr_t bits = reinterpret_cast<uintptr_t>(query) | reinterpret_cast<uintptr_t>(query_out) |
                     reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(key_out);
    if (bits % es || reinterpret_cast<uintptr_t>(positions) % 4 || reinterpret_cast<uintptr_t>(inv_freq) % 8)
        return bad(LI_ERR_SHAPE, "a pointer is not aligned to its element");
    // the widest access that every address of the call is aligned to
    bits |= es * (uintptr_t)(a.q.row | a.q.head | a.q.out_row | a.q.out_head | a.k.row | a.k.head | a.k.out_row | a.k.out_head);
    bits |= es * (uintptr_t)p->D;
    const bool staged = bits % 16 == 0;                // whole heads may be read in 16-byte accesses
    bits |= es * (uintptr_t)(p->rot_offset | (p->pairing == LI_ROPE_HALF ? p->rot_dim / 2 : p->rot_dim));
    int v = 1;
    while (v * es < 16 && bits % (2 * v * es) == 0) v *= 2;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.rows = p->rows;
    a.N1 = p->N1;
    a.N2 = p->N2;
    a.D = p->D;
    a.half = p->rot_dim / 2;
    a.off = p->rot_offset;
    a.mscale = p->mscale;
    a.sin_sign = p->inverse ? -1.f : 1.f;
    a.copy_rest = p->rot_dim < p->D && !(q_in && k_in);
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool half = p->pairing == LI_ROPE_HALF;
    const cudaError_t e = p->dtype == LI_BF16   ? launch_t<__nv_bfloat16>(a, half, v, staged, sms, s)
                          : p->dtype == LI_FP16 ? launch_t<__half>(a, half, v, staged, sms, s)
                                                : launch_t<float>(a, half, v, staged, sms, s);
    if (e != cudaSuccess) return bad(LI_ERR_CUDA, cudaGetErrorString(e));
    li::set_launch_count(1);
    return LI_OK;
}

extern "C" LI_API li_status li_rope_frequencies(int32_t scaling, int32_t rot_dim, double base, double factor,
                                                int32_t original_positions, double beta_fast, double beta_slow,
                                                double *inv_freq, float *mscale)
{
    auto refuse = [](li_status st, const char *m) { return li::report_error(st, m); };
    if (!inv_freq || !mscale) return refuse(LI_ERR_NULL, "li_rope_frequencies: inv_freq and mscale are required");
    if (scaling < LI_ROPE_SCALE_NONE || scaling > LI_ROPE_SCALE_YARN)
        return refuse(LI_ERR_LAYOUT, "li_rope_frequencies: unknown scaling");
    if (rot_dim < 2 || rot_dim % 2 || rot_dim > 1024 || (scaling == LI_ROPE_SCALE_NTK && rot_dim < 4))
        return refuse(LI_ERR_SHAPE, "li_rope_frequencies: rot_dim must be even in [2, 1024] (NTK: at least 4)");
    if (!(base > 1.0) || !std::isfinite(base)) return refuse(LI_ERR_SHAPE, "li_rope_frequencies: base must be above 1");
    if (scaling == LI_ROPE_SCALE_NONE) factor = 1.0;
    if (!(factor >= 1.0) || !std::isfinite(factor))
        return refuse(LI_ERR_SHAPE, "li_rope_frequencies: factor must be at least 1");
    *mscale = 1.f;
    if (scaling == LI_ROPE_SCALE_NTK) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    double lo = 0, hi = 0;
    if (scaling == LI_ROPE_SCALE_YARN) {
        if (original_positions < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast))
            return refuse(LI_ERR_SHAPE, "li_rope_frequencies: original_positions >= 1 and beta_fast > beta_slow > 0");
        // the (fractional) pair that turns `t` times within original_positions
        auto pair_at = [&](double t) {
            return rot_dim * std::log(original_positions / (t * 2 * M_PI)) / (2 * std::log(base));
        };
        lo = std::fmax(std::floor(pair_at(beta_fast)), 0.0);
        hi = std::fmin(std::ceil(pair_at(beta_slow)), rot_dim - 1.0);
        *mscale = (float)(0.1 * std::log(factor) + 1.0);
    }
    for (int p = 0; p < rot_dim / 2; ++p) {
        const double f = std::pow(base, -2.0 * p / rot_dim);
        if (scaling == LI_ROPE_SCALE_LINEAR) {
            inv_freq[p] = f / factor;
        } else if (scaling == LI_ROPE_SCALE_YARN) {
            // (hi <= lo = 0 when even the first pair turns beta_slow times at most)
            const double keep = p >= hi ? 0.0 : 1.0 - std::fmin(std::fmax((p - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
            inv_freq[p] = f * keep + f / factor * (1.0 - keep);
        } else {
            inv_freq[p] = f;
        }
    }
    return LI_OK;
}
