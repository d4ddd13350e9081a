// hqq_rotary.hip -- rotary positions: pairs of dimensions of queries and keys turned by their
// token's position (gfx950), and the frequencies that they are turned by.
//
// (a, b) -> (a cos x - b sin x, b cos x + a sin x), x = 2 pi * position * freq. Frequencies are
// turns in 64 bits behind the point, so that the product's low 64 bits are the part of a turn
// that is left, whatever the position: nothing is lost at far positions, and no range is reduced.
// Of it 32 bits are kept: 2^-33 turns, 7e-10 radians.
#include <cmath>

#include "hqq.h"
#include "hqq_cache_internal.h"
#include "hqq_internal.h"
#include "hqq_rotary.h"

namespace hqq {
namespace {

constexpr int kThreads = 256;

struct Tensor {
    const uint16_t *in;
    uint16_t *out;
    int64_t in_ts, in_hs, out_ts, out_hs;
};

struct RotaryArgs {
    Tensor x[2];
    RotaryHeads heads[2];
    const uint64_t *freqs;
    const int32_t *positions;
    float scale;
    int32_t n_tokens, pairs;    // rotary_dim / 2
    int32_t before, units;      // units of a token: the first tensor's, all
    int32_t tokens, parts;      // tokens to a block; blocks to a token
};

// Cosine and sine of a part of a turn, 2^-32 turns a step: the nearest quarter turn is taken off,
// the rest is within pi/4, where the Taylor sums below are off by 2^-26.
__device__ __forceinline__ float2 cos_sin(uint32_t part, float scale)
{
    const uint32_t quarter = (part + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(part - (quarter << 30)) * (6.283185307179586f * 0x1p-32f), y = x * x;
    float s = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(y, s, 1.f / 120.f);
    s = fmaf(y, s, -1.f / 6.f);
    s = fmaf(x * y, s, x);
    float c = fmaf(y, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(y, c, -1.f / 720.f);
    c = fmaf(y, c, 1.f / 24.f);
    c = fmaf(y, c, -0.5f);
    c = fmaf(y, c, 1.f);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return float2{((quarter + 1) & 2 ? -a : a) * scale, (quarter & 2 ? -b : b) * scale};
}

template <typename T>
__device__ __forceinline__ void turn(float a, float b, const float2 cs, uint32_t &first, uint32_t &second)
{
    first = from_f32<T>(fmaf(a, cs.x, -(b * cs.y)));
    second = from_f32<T>(fmaf(b, cs.x, a * cs.y));
}

// Eight pairs of a head, of 16 dimensions; pairs of neighbours, or of the two halves.
template <typename T, bool NEIGHBOURS>
__device__ __forceinline__ void turn8(uint4 &lo, uint4 &hi, const float2 *cs)
{
    float a[8], b[8];
    unpack8<T>(lo, a);
    unpack8<T>(hi, b);
    uint32_t x[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (NEIGHBOURS) {
            const float *p = e < 4 ? a + 2 * e : b + 2 * e - 8;
            uint32_t *to = e < 4 ? x + 2 * e : y + 2 * e - 8;
            turn<T>(p[0], p[1], cs[e], to[0], to[1]);
        } else {
            turn<T>(a[e], b[e], cs[e], x[e], y[e]);
        }
    }
    lo = uint4{x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16};
    hi = uint4{y[0] | y[1] << 16, y[2] | y[3] << 16, y[4] | y[5] << 16, y[6] | y[7] << 16};
}

// Sixteen bytes at any even address, which global memory reads and writes as it does aligned ones.
typedef uint32_t Sixteen __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ uint4 load16(const uint16_t *p)
{
    const Sixteen x = *reinterpret_cast<const Sixteen *>(p);
    return uint4{x[0], x[1], x[2], x[3]};
}
__device__ __forceinline__ void store16(uint16_t *p, uint4 x)
{
    *reinterpret_cast<Sixteen *>(p) = Sixteen{x.x, x.y, x.z, x.w};
}

struct Unit {
    const uint16_t *in;
    uint16_t *out;
    int d0, d1, pair;           // as in RotaryUnit; pair: of the token's cosines and sines
    bool wide;
};
template <bool NEIGHBOURS>
__device__ __forceinline__ Unit unit_of(const RotaryArgs &a, int t0, int j)
{
    const unsigned t = (unsigned)j / (unsigned)a.units;
    const RotaryUnit u = rotary_unit<NEIGHBOURS>(a.heads, a.pairs, a.before, j - t * a.units);
    const Tensor &x = a.x[u.tensor];
    return Unit{x.in + (t0 + (int64_t)t) * x.in_ts + u.head * x.in_hs, x.out + (t0 + (int64_t)t) * x.out_ts + u.head * x.out_hs,
                u.d0, u.d1, u.pair < 0 ? -1 : (int)(t * a.pairs) + u.pair, u.wide};
}

// A thread has one unit, whose numbers are on their way while the block makes the cosines and sines of its
// tokens (of a token with more units than a block has threads each of its blocks makes them). Bound by
// memory: 16390 tokens of 72 heads of 128, 604 MB: 101 us, 6.0 TB/s (part of it from the last level's
// cache; a copy of 4 GB reaches 5.0). 1000 tokens of 80 heads of 64: 6.8 us, 3.0 TB/s; a token 2.7 us,
// the launch and two loads that wait for each other.
template <typename T, bool NEIGHBOURS>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a)
{
    extern __shared__ float2 cs[];      // [tokens][pairs]; a unit has eight pairs at most, so 2048 of a block's
    const int t0 = (int)(blockIdx.x / (unsigned)a.parts) * a.tokens, part = (int)(blockIdx.x % (unsigned)a.parts);
    const int tokens = min(a.tokens, a.n_tokens - t0);
    const int j = part * kThreads + threadIdx.x, last = tokens * a.units - 1;
    const Unit x = unit_of<NEIGHBOURS>(a, t0, min(j, last));    // a thread without one reads the last and leaves
    uint4 lo, hi;
    if (__builtin_expect(x.wide, 1)) {
        lo = load16(x.in + x.d0);
        hi = load16(x.in + x.d1);
    } else {
        lo.x = x.in[x.d0];
        hi.x = x.in[x.d1];
    }
    for (int i = threadIdx.x; i < tokens * a.pairs; i += kThreads) {
        const unsigned t = (unsigned)i / (unsigned)a.pairs, k = i - t * a.pairs;
        const uint64_t turns = (uint64_t)(int64_t)a.positions[t0 + t] * a.freqs[k];
        cs[i] = cos_sin((uint32_t)((turns + 0x80000000u) >> 32), a.scale);
    }
    __syncthreads();
    if (j > last) return;
    if (__builtin_expect(x.wide, 1)) {
        if (x.pair >= 0) {
            turn8<T, NEIGHBOURS>(lo, hi, cs + x.pair);
            store16(x.out + x.d1, hi);
        }
        store16(x.out + x.d0, lo);
    } else {
        if (x.pair >= 0) {
            turn<T>(to_f32<T>(lo.x), to_f32<T>(hi.x), cs[x.pair], lo.x, hi.x);
            x.out[x.d1] = (uint16_t)hi.x;
        }
        x.out[x.d0] = (uint16_t)lo.x;
    }
}

template <typename T, bool NEIGHBOURS>
void launch(const RotaryArgs &a, unsigned blocks, hipStream_t stream)
{
    rotary_kernel<T, NEIGHBOURS><<<blocks, kThreads, (size_t)a.tokens * a.pairs * sizeof(float2), stream>>>(a);
}

hqq_status refuse(const char *msg)
{
    report_error(HQQ_ERR_ARG, msg);
    return HQQ_ERR_ARG;
}

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace hqq

extern "C" {

hqq_status hqq_rotary_frequencies(int rotary_dim, double theta, double factor, int64_t original_len, double low,
                                  double high, uint64_t *freqs)
{
    using namespace hqq;
    if (rotary_dim < 2 || rotary_dim > 1024 || rotary_dim % 2) return refuse("rotary_dim must be even, in [2, 1024]");
    if (!(theta >= 1.0) || !std::isfinite(theta)) return refuse("theta must be finite, at least 1");
    if (!(factor >= 1.0) || !std::isfinite(factor)) return refuse("factor must be finite, at least 1");
    if (original_len < 0) return refuse("original_len must not be negative");
    if (original_len > 0 && (!(low >= 0.0) || !(high > low) || !std::isfinite(high)))
        return refuse("low and high must be finite, with 0 <= low < high");
    if (!freqs) return refuse("freqs must be non-null");
    for (int i = 0; i < rotary_dim / 2; ++i) {
        const long double turns = std::pow((long double)theta, -2.0L * i / rotary_dim) / 6.283185307179586476925286766559L;
        long double s = 0.0L;
        if (original_len > 0) {
            s = (original_len * turns - low) / ((long double)high - low);
            s = s < 0.0L ? 0.0L : s > 1.0L ? 1.0L : s;
        }
        freqs[i] = (uint64_t)std::ldexp(turns * ((1.0L - s) / factor + s), 64);
    }
    report_error(HQQ_OK, "");
    return HQQ_OK;
}

hqq_status hqq_rotary(const uint64_t *freqs, int rotary_dim, int interleaved, float scale, const int32_t *positions,
                      int64_t n_tokens, int head_dim, int dtype, const hqq_rotary_rows *rows, int n_rows, void *stream)
{
    using namespace hqq;
    if (rotary_dim < 2 || rotary_dim % 2 || head_dim > 1024 || rotary_dim > head_dim)
        return refuse("rotary_dim must be even, 2 at least and head_dim at most, and head_dim 1024 at most");
    if (dtype != HQQ_F16 && dtype != HQQ_BF16) return refuse("dtype must be HQQ_F16 or HQQ_BF16");
    if (interleaved != 0 && interleaved != 1) return refuse("interleaved must be 0 or 1");
    if (!std::isfinite(scale)) return refuse("scale must be finite");
    if (n_tokens < 0 || n_tokens > (1 << 24)) return refuse("n_tokens must be in [0, 2^24]");
    if (n_rows < 0 || n_rows > 2 || (n_rows > 0 && !rows)) return refuse("rows must be one or two tensors");
    RotaryArgs a{};
    int n = 0;                  // tensors with something to turn
    for (int i = 0; i < n_rows; ++i) {
        const hqq_rotary_rows &r = rows[i];
        if (r.n_heads < 0 || r.n_heads > 4096) return refuse("rows: n_heads must be in [0, 4096]");
        if (r.n_heads == 0 || n_tokens == 0) continue;
        if (!r.in || !r.out) return refuse("rows: in and out must be non-null");
        if (!aligned(r.in, 2) || !aligned(r.out, 2)) return refuse("rows: in and out must be 2-byte aligned");
        const int64_t strides[] = {r.in_token_stride, r.in_head_stride, r.out_token_stride, r.out_head_stride};
        for (int64_t s : strides) {
            if (s < 0 || s > (int64_t(1) << 36)) return refuse("rows: strides must be in [0, 2^36]");
        }
        if (r.in == r.out) {
            if (strides[0] != strides[2] || strides[1] != strides[3])
                return refuse("rows: in place, the strides of in and out must be the same");
        }
        // in place, what is not turned may be shared
        if (rows_meet(n_tokens, r.n_heads, strides[2], strides[3], r.in == r.out ? rotary_dim : head_dim))
            return refuse("rows: heads and tokens of out must not overlap each other");
        if (n > 0 && r.out == a.x[0].out) return refuse("rows: the outputs must not overlap");
        a.x[n] = Tensor{static_cast<const uint16_t *>(r.in), static_cast<uint16_t *>(r.out),
                        strides[0], strides[1], strides[2], strides[3]};
        // in place, the dimensions behind those of the pairs are neither read nor written
        a.heads[n] = rotary_heads(r.n_heads, rotary_dim / 2, r.in == r.out ? 0 : head_dim - rotary_dim);
        a.units += r.n_heads * a.heads[n].per_head;
        if (n++ == 0) a.before = a.units;
    }
    if (n == 0) {
        report_error(HQQ_OK, "");
        return HQQ_OK;
    }
    if (!freqs || !positions || !aligned(freqs, 8) || !aligned(positions, 4))
        return refuse("freqs and positions must be non-null, 8- and 4-byte aligned");
    a.freqs = freqs;
    a.positions = positions;
    a.scale = scale;
    a.n_tokens = (int32_t)n_tokens;
    a.pairs = rotary_dim / 2;
    // A unit to a thread; with fewer than a block's in a token, several tokens. (Four to a thread: 16390
    // tokens of 72 heads of 128 107 us and 102 with one; 5000 of 16 heads of 256, a quarter turned, 15.9
    // and 17.3, for the angles are made more often; no difference for 4000 and fewer of the former.)
    a.tokens = kThreads / a.units > 1 ? kThreads / a.units : 1;
    if (a.tokens > a.n_tokens) a.tokens = a.n_tokens;
    a.parts = a.tokens > 1 ? 1 : (a.units + kThreads - 1) / kThreads;
    const int64_t blocks = (n_tokens + a.tokens - 1) / a.tokens * a.parts;
    if (blocks >= (1 << 24)) {
        report_error(HQQ_ERR_UNSUPPORTED, "too many rows for one call");
        return HQQ_ERR_UNSUPPORTED;
    }
    const hipStream_t str = static_cast<hipStream_t>(stream);
    if (dtype == HQQ_BF16) {
        if (interleaved) launch<Bf16, true>(a, (unsigned)blocks, str);
        else launch<Bf16, false>(a, (unsigned)blocks, str);
    } else {
        if (interleaved) launch<F16, true>(a, (unsigned)blocks, str);
        else launch<F16, false>(a, (unsigned)blocks, str);
    }
    const hipError_t e = hipGetLastError();
    const hqq_status st = e == hipSuccess ? HQQ_OK : HQQ_ERR_DEVICE;
    report_error(st, e == hipSuccess ? "" : hipGetErrorString(e));
    return st;
}

}  // extern "C"
