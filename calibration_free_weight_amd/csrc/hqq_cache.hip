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

constexpr int kThreads = kRowThreads;

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
// 512/head_dim tokens, and a block the next waves' too, so that the cache lines that its
// tokens' grids share are filled by one block (blocks go round the eight dies, and lines that
// two of them fill in part are written twice).
struct Place {
    int i, h0, n, u;
};
template <int D, int HEADS>
__device__ __forceinline__ Place place_of(int heads)
{
    constexpr int kLanes = D / 8, kTokens = kThreads / kLanes;
    const unsigned parts = (heads + HEADS - 1) / HEADS;
    const int h0 = (int)(blockIdx.x % parts) * HEADS;
    return Place{(int)(blockIdx.x / parts) * kTokens + (int)threadIdx.x / kLanes, h0, min(HEADS, heads - h0),
                 (int)threadIdx.x % kLanes};
}

// Smallest and largest of three, of binary32 numbers or of each half of three words: NaN if one is.
__device__ __forceinline__ float smallest(float a, float b, float c)
{
    float r;
    asm("v_minimum3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float largest(float a, float b, float c)
{
    float r;
    asm("v_maximum3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ uint32_t smallest_halves(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("v_pk_minimum3_f16 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ uint32_t largest_halves(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("v_pk_maximum3_f16 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// f over the G/8 lanes of a group, by exchanges within a row of 16 lanes: pairs, quads,
// halves mirrored, the row mirrored. All of the group's lanes get it.
template <int CTRL>
__device__ __forceinline__ uint32_t other(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
template <int G, typename F>
__device__ __forceinline__ uint32_t over_group(uint32_t x, F f)
{
    x = f(x, other<0xb1>(x));               // quad_perm 1, 0, 3, 2
    x = f(x, other<0x4e>(x));               // quad_perm 2, 3, 0, 1
    if constexpr (G >= 64) x = f(x, other<0x141>(x));       // row_half_mirror
    if constexpr (G >= 128) x = f(x, other<0x140>(x));      // row_mirror
    return x;
}

// The smallest and largest of a group, of which the lane has the values v (bits raw); NaN if one
// of the group is.
template <typename T, int G>
__device__ __forceinline__ void group_range(const uint4 raw, const float (&v)[8], float &lo, float &hi)
{
    if constexpr (Types<T>::kBf16) {
        lo = smallest(smallest(smallest(v[0], v[1], v[2]), v[3], v[4]), v[5], smallest(v[6], v[7], v[7]));
        hi = largest(largest(largest(v[0], v[1], v[2]), v[3], v[4]), v[5], largest(v[6], v[7], v[7]));
        lo = __uint_as_float(over_group<G>(__float_as_uint(lo), [](uint32_t a, uint32_t b) {
            return __float_as_uint(smallest(__uint_as_float(a), __uint_as_float(b), __uint_as_float(b)));
        }));
        hi = __uint_as_float(over_group<G>(__float_as_uint(hi), [](uint32_t a, uint32_t b) {
            return __float_as_uint(largest(__uint_as_float(a), __uint_as_float(b), __uint_as_float(b)));
        }));
    } else {
        // two at a time; then the smallest, negated, and the largest in one word
        const uint32_t h = largest_halves(largest_halves(raw.x, raw.y, raw.z), raw.w, raw.w);
        const uint32_t l = smallest_halves(smallest_halves(raw.x, raw.y, raw.z), raw.w, raw.w) ^ 0x80008000u;
        const uint32_t x = __builtin_amdgcn_perm(h, l, 0x05040100u), y = __builtin_amdgcn_perm(h, l, 0x07060302u);
        const uint32_t all = over_group<G>(largest_halves(x, y, y), [](uint32_t a, uint32_t b) { return largest_halves(a, b, b); });
        lo = -to_f32<T>(all & 0xffffu);
        hi = to_f32<T>(all >> 16);
    }
}

// What a - b, rounded to `d`, leaves: a - b = d + less(a, b, d) exactly.
__device__ __forceinline__ float less(float a, float b, float d)
{
    const float x = d - a;
    return (a - (d - x)) + (-b - x);
}

// The bits of the smallest number of the type with number * top >= hi - lo. The nearest one to
// their rounded quotient is it or the one below; its product with top has at most 11 + 8 bits
// and lies next to the difference, so both the product and what it is above are exact.
template <typename T>
__device__ __forceinline__ uint32_t step_bits(float lo, float hi, int top)
{
    const float span = hi - lo;
    uint32_t bits = from_f32<T>(span * (1.0f / (float)top));
    if (to_f32<T>(bits) * (float)top - span < less(hi, lo, span)) ++bits;
    if (Types<T>::kBf16 && span > 0.f) bits = max(bits, 0x0d80u);     // 2^-100
    return bits;
}

// ---- write ------------------------------------------------------------------------------------
// Bound by neither memory nor arithmetic alone: 18060 tokens of 32 heads of 128 in 4 bits, 379 MB,
// take 105 us (3.6 TB/s; 89 when the same inputs were written just before) where their bytes take 74
// at a copy's rate, with about 100 instructions for a lane's eight values of 24 bytes in and out:
// vector instructions are issued 72% of the time, and a wave waits 45% of its own. A token of 8
// heads takes 3.4 us, the launch and a chain of loads (its sequence's row offsets, length and page;
// with many sequences two looks at the offsets first).
// Codes are decided exactly: the quotient, by a
// product with the reciprocal's estimate, errs by at most 2^(nbits - 22), so only within twice
// that of a half is it held against the midpoint, again without rounding: (2k + 1) * step has
// at most 9 + 11 bits and lies next to twice the difference. With binary16 one value in some
// thousands is a tie, so a fifth of the waves come there. q: the codes, as binary32 numbers.
template <typename T, int NB, int G>
__device__ __forceinline__ uint32_t quantize8(const uint4 raw, float (&q)[8])
{
    constexpr int kTop = (1 << NB) - 1;
    constexpr float kNear = 0.5f - (NB == 4 ? 0x1p-17f : 0x1p-13f);
    float v[8], lo, hi;
    unpack8<T>(raw, v);
    group_range<T, G>(raw, v, lo, hi);
    const uint32_t sb = step_bits<T>(lo, hi, kTop);
    const float step = to_f32<T>(sb);
    const float inv = step > 0 ? __builtin_amdgcn_rcpf(step) : 0.f;
    float y[8], most = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        y[e] = (v[e] - lo) * inv;
        q[e] = rintf(y[e]);
        most = fmaxf(most, fabsf(y[e] - q[e]));
    }
    if (most > kNear) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float k = floorf(y[e]), d = v[e] - lo, odd = fmaf(2.f, k, 1.f);
            const float above = 2.f * d - odd * step + 2.f * less(v[e], lo, d);
            const float up = above > 0.f || (above == 0.f && ((int)k & 1)) ? k + 1.f : k;
            q[e] = fabsf(y[e] - q[e]) > kNear ? up : q[e];
        }
    }
    // the last code stays finite in binary16
    if (!Types<T>::kBf16 && fmaf((float)kTop, step, lo) >= 65520.f)
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = fminf(q[e], (float)(kTop - 1));
    // A group that holds infinities or NaN reads back as NaN: step 0, which leaves what attention
    // makes of the other groups alone.
    return hi - lo < INFINITY ? sb | (from_f32<T>(lo) << 16) : Types<T>::kBf16 ? 0x7fc00000u : 0x7e000000u;
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
// Bound by memory: 65521 tokens of 8 heads of 128 in 8 bits, 407 MB, take 80 us (5.1 TB/s, a
// copy's rate). All of a lane's loads are asked for before the first is used, whatever the page.
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
    const dim3 grid((unsigned)cache_rows_blocks(write, s.n_tokens, c.heads, D));
    if (write) cache_write_kernel<T, NB, D, G, HEADS><<<grid, kThreads, 0, stream>>>(c, s, p);
    else cache_read_kernel<T, NB, D, G, HEADS><<<grid, kThreads, 0, stream>>>(c, s, p);
}

template <typename T, int NB, int D, int G>
hipError_t launch(bool write, const CacheView &c, const SeqView &s, const RowPtrs &p, hipStream_t stream)
{
    if (four_heads(write, s.n_tokens, c.heads, D)) launch_heads<T, NB, D, G, 4>(write, c, s, p, stream);
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
