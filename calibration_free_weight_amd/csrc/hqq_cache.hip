// hqq_cache.hip -- the quantized key/value cache written and read back (gfx950).
//
// Rows are one head's vector of one token. head_dim/8 lanes share a row, lane u holding
// dimensions 8u..8u+7 (one 16-byte load or store), so that a group of 32, 64 or 128
// dimensions lies in 4, 8 or 16 neighbouring lanes. A wave takes a few neighbouring tokens of
// one head at a time: their codes lie side by side in a page, the values' even interleaved
// (per four tokens), so that its narrow stores fall into the same cache lines. It goes on to
// the next heads of the same tokens, whose places it has then looked up already, with the
// loads of all of them under way.
#include "hqq_cache_internal.h"

namespace hqq {
namespace {

constexpr int kThreads = 256;

// Whether row i belongs to a sequence, and where its token lies: page (or -1), token of it.
struct Slot {
    bool mine;
    int page, t;
};
__device__ __forceinline__ Slot slot_of(const SeqView &s, int i)
{
    const int b = find_seq(s, i);
    const Rows r = rows_of(s, b);
    Slot x = {i >= r.begin && i < r.end, -1, 0};
    if (!x.mine) return x;
    const int pos = len_of(s, b) - (r.end - i);
    x.page = page_of(s, b, pos);
    x.t = pos & ((1 << s.page_shift) - 1);
    return x;
}

// The row of a lane: token i, heads h0 .. h0 + n - 1, dimensions 8u..8u+7. A wave has
// 512/head_dim tokens and up to HEADS heads.
struct Place {
    int i, h0, n, u;
};
template <int D, int HEADS>
__device__ __forceinline__ Place place_of(int heads)
{
    constexpr int kLanes = D / 8, kTokens = 64 / kLanes;
    const unsigned wave = blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned parts = (heads + HEADS - 1) / HEADS;
    const int lane = threadIdx.x & 63, h0 = (int)(wave % parts) * HEADS;
    return Place{(int)(wave / parts) * kTokens + lane / kLanes, h0, min(HEADS, heads - h0), lane % kLanes};
}

// The smallest and largest of a group: of the lane's values, then over its G/8 lanes, by
// exchanges within a row of 16 lanes (pairs, quads, halves mirrored, the row mirrored).
template <int CTRL>
__device__ __forceinline__ float other(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <int G>
__device__ __forceinline__ void group_range(float &lo, float &hi)
{
    lo = fminf(lo, other<0xb1>(lo));        // quad_perm 1, 0, 3, 2
    hi = fmaxf(hi, other<0xb1>(hi));
    lo = fminf(lo, other<0x4e>(lo));        // quad_perm 2, 3, 0, 1
    hi = fmaxf(hi, other<0x4e>(hi));
    if constexpr (G >= 64) {
        lo = fminf(lo, other<0x141>(lo));   // row_half_mirror
        hi = fmaxf(hi, other<0x141>(hi));
    }
    if constexpr (G >= 128) {
        lo = fminf(lo, other<0x140>(lo));   // row_mirror
        hi = fmaxf(hi, other<0x140>(hi));
    }
}

template <typename T>
__device__ __forceinline__ uint32_t step_up(float span, int top, double range)
{
    // The nearest number of the type to span/top is one of the two next to range/top; the
    // exact product (at most 8 + 11 bits) says whether it is the lower one.
    const float near = span * (1.0f / (float)top);
    uint32_t bits = from_f32<T>(near);
    if ((double)to_f32<T>(bits) * top < range) ++bits;
    if (Types<T>::kBf16 && range > 0 && bits < 0x0d80u) bits = 0x0d80u;   // 2^-100
    return bits;
}

// ---- write ------------------------------------------------------------------------------------
// Codes are decided exactly: a binary32 quotient errs by less than 2^-14, so only quotients
// within 2^-12 of a half take the binary64 comparison with the midpoint (about one value in
// 2000, so that one lane in 250 has one). q: the codes, as whole binary32 numbers.
template <typename T, int NB, int G>
__device__ __forceinline__ uint32_t quantize8(const uint4 raw, float (&q)[8])
{
    constexpr int kTop = (1 << NB) - 1;
    float v[8];
    unpack8<T>(raw, v);
    float lo = fminf(fminf(fminf(v[0], v[1]), fminf(v[2], v[3])), fminf(fminf(v[4], v[5]), fminf(v[6], v[7])));
    float hi = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
    group_range<G>(lo, hi);
    const uint32_t sb = step_up<T>(hi - lo, kTop, (double)hi - (double)lo);
    const float step = to_f32<T>(sb);
    const float inv = step > 0 ? 1.0f / step : 0.f;
    float y[8], most = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        y[e] = (v[e] - lo) * inv;
        q[e] = rintf(y[e]);
        most = fmaxf(most, fabsf(y[e] - q[e]));
    }
    if (most > 0.5f - 0x1p-12f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (fabsf(y[e] - q[e]) <= 0.5f - 0x1p-12f) continue;
            const float k = floorf(y[e]);
            const double twice = 2.0 * ((double)v[e] - (double)lo);
            const double mid = (2.0 * k + 1.0) * (double)step;
            q[e] = twice > mid || (twice == mid && ((int)k & 1)) ? k + 1.f : k;
        }
    }
    // the last code stays finite in binary16
    if (!Types<T>::kBf16 && fmaf((float)kTop, step, lo) >= 65520.f)
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = fminf(q[e], (float)(kTop - 1));
    return sb | (from_f32<T>(lo) << 16);
}

// Four codes as bytes, clamped to them (a number that is none becomes 0).
__device__ __forceinline__ uint32_t bytes4(float a, float b, float c, float d)
{
    uint32_t w = __builtin_amdgcn_cvt_pk_u8_f32(a, 0, 0);
    w = __builtin_amdgcn_cvt_pk_u8_f32(b, 1, w);
    w = __builtin_amdgcn_cvt_pk_u8_f32(c, 2, w);
    return __builtin_amdgcn_cvt_pk_u8_f32(d, 3, w);
}

template <typename T, int NB, int D, int G, int HEADS>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(CacheView c, SeqView s, RowPtrs p)
{
    const Place me = place_of<D, HEADS>(c.heads);
    const int i = min(me.i, s.n_tokens - 1);
    uint4 kr[HEADS], vr[HEADS];
#pragma unroll
    for (int x = 0; x < HEADS; ++x) {
        const int h = me.h0 + min(x, me.n - 1);
        kr[x] = *reinterpret_cast<const uint4 *>(p.k + i * p.k_ts + h * p.k_hs + 8 * me.u);
        vr[x] = *reinterpret_cast<const uint4 *>(p.v + i * p.v_ts + h * p.v_hs + 8 * me.u);
    }
    Slot at = slot_of(s, i);                // by all lanes: they search together
    if (me.i >= s.n_tokens || at.page < 0) return;      // whole rows leave together
    const int u = me.u;
#pragma unroll
    for (int x = 0; x < HEADS; ++x) {
        if (x >= me.n) break;
        const int64_t token = (((int64_t)at.page * c.heads + me.h0 + x) << s.page_shift);
        uint8_t *kc = c.k_codes + token * (D * NB / 8);
        uint8_t *vc = c.v_codes + token * (D * NB / 8);
        float q[8];
        const uint32_t km = quantize8<T, NB, G>(kr[x], q);
        // lane u holds unit (a, m) = (u % 4, u / 4) of the key
        uint8_t *ku = kc + k_unit_at(at.t, u & 3, u >> 2, D, NB);
        if constexpr (NB == 4)
            *reinterpret_cast<uint32_t *>(ku) = bytes4(fmaf(q[4], 16.f, q[0]), fmaf(q[5], 16.f, q[1]),
                                                       fmaf(q[6], 16.f, q[2]), fmaf(q[7], 16.f, q[3]));
        else
            *reinterpret_cast<uint2 *>(ku) = make_uint2(bytes4(q[0], q[1], q[2], q[3]), bytes4(q[4], q[5], q[6], q[7]));
        const uint32_t vm = quantize8<T, NB, G>(vr[x], q);
        if (u % (G / 8) == 0) {
            c.k_meta[(token + at.t) * (D / G) + u / (G / 8)] = km;
            c.v_meta[(token + at.t) * (D / G) + u / (G / 8)] = vm;
        }
        // and runs of G/16 codes of 128/G rows of the value
        uint32_t w[2];
        if constexpr (NB == 4)
            w[0] = w[1] = bytes4(fmaf(q[1], 16.f, q[0]), fmaf(q[3], 16.f, q[2]), fmaf(q[5], 16.f, q[4]), fmaf(q[7], 16.f, q[6]));
        else {
            w[0] = bytes4(q[0], q[1], q[2], q[3]);
            w[1] = bytes4(q[4], q[5], q[6], q[7]);
        }
        constexpr int kRun = G / 16, kBytes = kRun * NB / 8;
        uint8_t *vu = vc + v_row_at(at.t, 8 * u % G / kRun, D, NB) + 8 * u / G * kBytes;
        constexpr int kNext = D * NB / 32;  // from a row to the next
        if constexpr (kBytes == 8) *reinterpret_cast<uint2 *>(vu) = make_uint2(w[0], w[1]);
        else if constexpr (kBytes == 4) {
            *reinterpret_cast<uint32_t *>(vu) = w[0];
            if constexpr (NB == 8) *reinterpret_cast<uint32_t *>(vu + kNext) = w[1];
        } else if constexpr (kBytes == 2) {
#pragma unroll
            for (int y = 0; y < NB / 2; ++y)
                *reinterpret_cast<uint16_t *>(vu + y * kNext) = (uint16_t)(w[y / 2] >> (16 * (y & 1)));
        } else {
#pragma unroll
            for (int y = 0; y < 4; ++y) vu[y * kNext] = (uint8_t)(w[0] >> (8 * y));
        }
    }
}

// ---- read -------------------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ uint4 values8(const float (&q)[8], uint32_t meta)
{
    const float step = to_f32<T>(meta & 0xffffu), base = to_f32<T>(meta >> 16);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        w[e] = from_f32<T>(fmaf(q[2 * e], step, base)) | from_f32<T>(fmaf(q[2 * e + 1], step, base)) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float byte_of(uint32_t w, int k) { return (float)(w >> (8 * k) & 255u); }

template <typename T, int NB, int D, int G, int HEADS>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheView c, SeqView s, RowPtrs p)
{
    const Place me = place_of<D, HEADS>(c.heads);
    const int i = min(me.i, s.n_tokens - 1), u = me.u;
    const Slot at = slot_of(s, i);
    if (me.i >= s.n_tokens || !at.mine) return;         // rows of no sequence stay as they were
    constexpr int kRun = G / 16, kBytes = kRun * NB / 8, kNext = D * NB / 32;
    uint32_t kw[HEADS][NB / 4], vw[HEADS][NB / 4], km[HEADS], vm[HEADS];
#pragma unroll
    for (int x = 0; x < HEADS; ++x) {
        const int h = me.h0 + min(x, me.n - 1);
        const int64_t token = (((int64_t)max(at.page, 0) * c.heads + h) << s.page_shift);
        const uint8_t *ku = c.k_codes + token * (D * NB / 8) + k_unit_at(at.t, u & 3, u >> 2, D, NB);
        const uint8_t *vu = c.v_codes + token * (D * NB / 8) + v_row_at(at.t, 8 * u % G / kRun, D, NB) + 8 * u / G * kBytes;
        km[x] = c.k_meta[(token + at.t) * (D / G) + 8 * u / G];
        vm[x] = c.v_meta[(token + at.t) * (D / G) + 8 * u / G];
#pragma unroll
        for (int y = 0; y < NB / 4; ++y) kw[x][y] = reinterpret_cast<const uint32_t *>(ku)[y];
        if constexpr (kBytes >= 4) {
#pragma unroll
            for (int y = 0; y < NB / 4; ++y)
                vw[x][y] = *reinterpret_cast<const uint32_t *>(kBytes == 8 ? vu + 4 * y : vu + y * kNext);
        } else if constexpr (kBytes == 2) {
#pragma unroll
            for (int y = 0; y < NB / 4; ++y)
                vw[x][y] = *reinterpret_cast<const uint16_t *>(vu + 2 * y * kNext) |
                           (uint32_t)*reinterpret_cast<const uint16_t *>(vu + (2 * y + 1) * kNext) << 16;
        } else {
            vw[x][0] = vu[0] | (uint32_t)vu[kNext] << 8 | (uint32_t)vu[2 * kNext] << 16 | (uint32_t)vu[3 * kNext] << 24;
        }
    }
#pragma unroll
    for (int x = 0; x < HEADS; ++x) {
        if (x >= me.n) break;
        const int h = me.h0 + x;
        uint4 ko = {0, 0, 0, 0}, vo = {0, 0, 0, 0};
        if (at.page >= 0) {
            float kq[8], vq[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (NB == 4) {
                    kq[e] = byte_of(kw[x][0] & 0x0f0f0f0fu, e);
                    kq[e + 4] = byte_of(kw[x][0] >> 4 & 0x0f0f0f0fu, e);
                    vq[2 * e] = byte_of(vw[x][0] & 0x0f0f0f0fu, e);
                    vq[2 * e + 1] = byte_of(vw[x][0] >> 4 & 0x0f0f0f0fu, e);
                } else {
                    kq[e] = byte_of(kw[x][0], e);
                    kq[e + 4] = byte_of(kw[x][1], e);
                    vq[e] = byte_of(vw[x][0], e);
                    vq[e + 4] = byte_of(vw[x][1], e);
                }
            }
            ko = values8<T>(kq, km[x]);
            vo = values8<T>(vq, vm[x]);
        }
        *reinterpret_cast<uint4 *>(p.k + i * p.k_ts + h * p.k_hs + 8 * u) = ko;
        *reinterpret_cast<uint4 *>(p.v + i * p.v_ts + h * p.v_hs + 8 * u) = vo;
    }
}

template <typename T, int NB, int D, int G, int HEADS>
void launch_heads(bool write, const CacheView &c, const SeqView &s, const RowPtrs &p, hipStream_t stream)
{
    constexpr int kTokens = 512 / D;
    const int64_t waves = ((int64_t)s.n_tokens + kTokens - 1) / kTokens * ((c.heads + HEADS - 1) / HEADS);
    const dim3 grid((unsigned)((waves + kThreads / 64 - 1) / (kThreads / 64)));
    if (write) cache_write_kernel<T, NB, D, G, HEADS><<<grid, kThreads, 0, stream>>>(c, s, p);
    else cache_read_kernel<T, NB, D, G, HEADS><<<grid, kThreads, 0, stream>>>(c, s, p);
}

template <typename T, int NB, int D, int G>
hipError_t launch(bool write, const CacheView &c, const SeqView &s, const RowPtrs &p, hipStream_t stream)
{
    // four heads to a wave, unless that leaves the GPU's 1024 units without a few waves each
    if ((int64_t)s.n_tokens * c.heads * D >= int64_t(1) << 23) launch_heads<T, NB, D, G, 4>(write, c, s, p, stream);
    else launch_heads<T, NB, D, G, 1>(write, c, s, p, stream);
    return hipGetLastError();
}

template <typename T, int NB, int D>
hipError_t by_group(bool write, int g, const CacheView &c, const SeqView &s, const RowPtrs &p,
                    hipStream_t stream)
{
    if (g == 32) return launch<T, NB, D, 32>(write, c, s, p, stream);
    if (g == 64) return launch<T, NB, D, 64>(write, c, s, p, stream);
    if constexpr (D >= 128)
        if (g == 128) return launch<T, NB, D, 128>(write, c, s, p, stream);
    return hipErrorInvalidValue;
}

template <typename T, int NB>
hipError_t by_dim(bool write, int dim, int g, const CacheView &c, const SeqView &s,
                  const RowPtrs &p, hipStream_t stream)
{
    if (dim == 64) return by_group<T, NB, 64>(write, g, c, s, p, stream);
    if (dim == 128) return by_group<T, NB, 128>(write, g, c, s, p, stream);
    return by_group<T, NB, 256>(write, g, c, s, p, stream);
}

}  // namespace

hipError_t launch_cache_rows(bool write, const CacheView &c, const SeqView &s, const RowPtrs &p,
                             int dim, int nbits, int g, bool bf16, hipStream_t stream)
{
    if (bf16)
        return nbits == 4 ? by_dim<Bf16, 4>(write, dim, g, c, s, p, stream)
                          : by_dim<Bf16, 8>(write, dim, g, c, s, p, stream);
    return nbits == 4 ? by_dim<F16, 4>(write, dim, g, c, s, p, stream)
                      : by_dim<F16, 8>(write, dim, g, c, s, p, stream);
}

}  // namespace hqq
