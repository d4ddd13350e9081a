// hqq_cache.hip -- the quantized key/value cache written and read back (gfx950).
//
// Both kernels work on rows: one head's vector of one token. head_dim/8 lanes share a row,
// lane u holding dimensions 8u..8u+7 (one 16-byte load or store), so that a group of 32, 64
// or 128 dimensions lies in 4, 8 or 16 neighbouring lanes.
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

template <typename T>
__device__ __forceinline__ uint32_t step_up(float span, int top, double range)
{
    // The nearest number of the type to span/top is one of the two next to range/top; the
    // exact product (at most 8 + 11 bits) says whether it is the lower one.
    const float near = span / (float)top;
    uint32_t bits = from_f32<T>(near);
    if ((double)to_f32<T>(bits) * top < range) ++bits;
    if (Types<T>::kBf16 && range > 0 && bits < 0x0d80u) bits = 0x0d80u;   // 2^-100
    return bits;
}

// ---- write ------------------------------------------------------------------------------------
// Memory-bound: 2 bytes in and nbits/8 + 4/g out per value. Codes are decided exactly: a
// binary32 quotient errs by less than 2^-14, so only quotients within 2^-12 of a half take
// the binary64 comparison with the midpoint (about one value in 2000).
template <typename T, int NB, int D, int G>
__device__ __forceinline__ void quantize8(const uint4 raw, uint32_t (&q)[8], uint32_t &meta)
{
    constexpr int kTop = (1 << NB) - 1;
    float v[8];
    unpack8<T>(raw, v);
    float lo = v[0], hi = v[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        lo = fminf(lo, v[e]);
        hi = fmaxf(hi, v[e]);
    }
#pragma unroll
    for (int x = 1; x < G / 8; x <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, x));
        hi = fmaxf(hi, __shfl_xor(hi, x));
    }
    const uint32_t sb = step_up<T>(hi - lo, kTop, (double)hi - (double)lo);
    const float step = to_f32<T>(sb);
    meta = sb | (from_f32<T>(lo) << 16);
    int top = kTop;
    if (!Types<T>::kBf16 && fmaf((float)kTop, step, lo) >= 65520.f) top = kTop - 1;
    const float inv = step > 0 ? 1.0f / step : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = (v[e] - lo) * inv;
        float r = rintf(y);
        if (fabsf(y - r) > 0.5f - 0x1p-12f) {
            const float k = floorf(y);
            const double twice = 2.0 * ((double)v[e] - (double)lo);
            const double mid = (2.0 * k + 1.0) * (double)step;
            r = twice > mid || (twice == mid && ((int)k & 1)) ? k + 1.f : k;
        }
        q[e] = (uint32_t)max(0, min((int)r, top));
    }
}

template <typename T, int NB, int D, int G>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(CacheView c, SeqView s, RowPtrs p)
{
    constexpr int kLanes = D / 8;
    const int64_t row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;
    const int u = threadIdx.x % kLanes;
    const int i = (int)(row / c.heads), h = (int)(row % c.heads);
    const Slot at = slot_of(s, i);          // by all lanes: they search together
    if (!at.mine) return;                   // whole rows leave together
    const uint4 kr = *reinterpret_cast<const uint4 *>(p.k + i * p.k_ts + h * p.k_hs + 8 * u);
    const uint4 vr = *reinterpret_cast<const uint4 *>(p.v + i * p.v_ts + h * p.v_hs + 8 * u);
    uint32_t kq[8], vq[8], km, vm;
    quantize8<T, NB, D, G>(kr, kq, km);
    quantize8<T, NB, D, G>(vr, vq, vm);
    if (at.page < 0) return;
    const int64_t slice = (int64_t)at.page * c.heads + h;
    const int page = 1 << s.page_shift;
    uint8_t *kc = c.k_codes + slice * page * (D * NB / 8);
    uint8_t *vc = c.v_codes + slice * page * (D * NB / 8);
    uint32_t *kmeta = c.k_meta + (slice * page + at.t) * (D / G);
    uint32_t *vmeta = c.v_meta + (slice * page + at.t) * (D / G);
    if (u % (G / 8) == 0) {
        kmeta[u / (G / 8)] = km;
        vmeta[u / (G / 8)] = vm;
    }
    // lane u holds unit (a, m) = (u % 4, u / 4) of the key
    uint8_t *ku = kc + k_unit_at(at.t, u & 3, u >> 2, D, NB);
    if (NB == 4) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) w |= (kq[e] | kq[e + 4] << 4) << (8 * e);
        *reinterpret_cast<uint32_t *>(ku) = w;
    } else {
        uint2 w = {0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w.x |= kq[e] << (8 * e);
            w.y |= kq[e + 4] << (8 * e);
        }
        *reinterpret_cast<uint2 *>(ku) = w;
    }
    // and of the value, runs of G/16 codes of 128/G rows
    constexpr int kRun = G / 16;
    const int grp = 8 * u / G, r0 = 8 * u % G / kRun;
#pragma unroll
    for (int x = 0; x < 8 / kRun; ++x) {
        uint8_t *vu = vc + v_row_at(at.t, r0 + x, D, NB) + grp * kRun * NB / 8;
        uint64_t w = 0;
#pragma unroll
        for (int j = 0; j < kRun; ++j) w |= (uint64_t)vq[x * kRun + j] << (NB * j);
        constexpr int kBytes = kRun * NB / 8;
        if (kBytes == 1) *vu = (uint8_t)w;
        if (kBytes == 2) *reinterpret_cast<uint16_t *>(vu) = (uint16_t)w;
        if (kBytes == 4) *reinterpret_cast<uint32_t *>(vu) = (uint32_t)w;
        if (kBytes == 8) *reinterpret_cast<uint64_t *>(vu) = w;
    }
}

// ---- read -------------------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ uint4 values8(const uint32_t (&q)[8], uint32_t meta)
{
    const float step = to_f32<T>(meta & 0xffffu), base = to_f32<T>(meta >> 16);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        w[e] = from_f32<T>(fmaf((float)q[2 * e], step, base)) |
               from_f32<T>(fmaf((float)q[2 * e + 1], step, base)) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int NB, int D, int G>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheView c, SeqView s, RowPtrs p)
{
    constexpr int kLanes = D / 8;
    const int64_t row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes;
    const int u = threadIdx.x % kLanes;
    const int i = (int)(row / c.heads), h = (int)(row % c.heads);
    const Slot at = slot_of(s, i);
    if (!at.mine) return;                   // rows of no sequence stay as they were
    uint4 ko = {0, 0, 0, 0}, vo = {0, 0, 0, 0};
    if (at.page >= 0) {
        const int64_t slice = (int64_t)at.page * c.heads + h;
        const int page = 1 << s.page_shift;
        const uint8_t *kc = c.k_codes + slice * page * (D * NB / 8);
        const uint8_t *vc = c.v_codes + slice * page * (D * NB / 8);
        const uint32_t km = c.k_meta[(slice * page + at.t) * (D / G) + 8 * u / G];
        const uint32_t vm = c.v_meta[(slice * page + at.t) * (D / G) + 8 * u / G];
        const uint8_t *ku = kc + k_unit_at(at.t, u & 3, u >> 2, D, NB);
        uint32_t kq[8], vq[8];
        if (NB == 4) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(ku);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                kq[e] = w >> (8 * e) & 15;
                kq[e + 4] = w >> (8 * e + 4) & 15;
            }
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(ku);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                kq[e] = w.x >> (8 * e) & 255;
                kq[e + 4] = w.y >> (8 * e) & 255;
            }
        }
        constexpr int kRun = G / 16;
        const int grp = 8 * u / G, r0 = 8 * u % G / kRun;
#pragma unroll
        for (int x = 0; x < 8 / kRun; ++x) {
            const uint8_t *vu = vc + v_row_at(at.t, r0 + x, D, NB) + grp * kRun * NB / 8;
            constexpr int kBytes = kRun * NB / 8;
            uint64_t w = 0;
            if (kBytes == 1) w = *vu;
            if (kBytes == 2) w = *reinterpret_cast<const uint16_t *>(vu);
            if (kBytes == 4) w = *reinterpret_cast<const uint32_t *>(vu);
            if (kBytes == 8) w = *reinterpret_cast<const uint64_t *>(vu);
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                vq[x * kRun + j] = (uint32_t)(w >> (NB * j)) & ((1u << NB) - 1);
        }
        ko = values8<T>(kq, km);
        vo = values8<T>(vq, vm);
    }
    *reinterpret_cast<uint4 *>(p.k + i * p.k_ts + h * p.k_hs + 8 * u) = ko;
    *reinterpret_cast<uint4 *>(p.v + i * p.v_ts + h * p.v_hs + 8 * u) = vo;
}

template <typename T, int NB, int D, int G>
hipError_t launch(bool write, const CacheView &c, const SeqView &s, const RowPtrs &p, hipStream_t stream)
{
    const int64_t lanes = (int64_t)s.n_tokens * c.heads * (D / 8);
    const dim3 grid((unsigned)((lanes + kThreads - 1) / kThreads));
    if (write) cache_write_kernel<T, NB, D, G><<<grid, kThreads, 0, stream>>>(c, s, p);
    else cache_read_kernel<T, NB, D, G><<<grid, kThreads, 0, stream>>>(c, s, p);
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
