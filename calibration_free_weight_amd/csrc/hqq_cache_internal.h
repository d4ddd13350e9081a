// hqq_cache_internal.h -- declarations shared by the cache's translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hqq_cache.h"

namespace hqq {

struct CacheView {
    uint8_t *k_codes, *v_codes;
    uint32_t *k_meta, *v_meta;  // one word per group: step in the low half, base in the high
    int32_t heads;
};

struct RowPtrs {                // k and v rows of a write or read, strides in elements
    uint16_t *k, *v;
    int64_t k_ts, k_hs, v_ts, v_hs;
};

struct F16 {};
struct Bf16 {};

template <typename T>
struct Types;
template <>
struct Types<F16> {
    static constexpr bool kBf16 = false;
    using E = _Float16;
};
template <>
struct Types<Bf16> {
    static constexpr bool kBf16 = true;
    using E = __bf16;
};

template <typename T>
__device__ __forceinline__ float to_f32(uint32_t bits)
{
    if constexpr (Types<T>::kBf16) return __uint_as_float(bits << 16);
    else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

// Round to nearest, ties to even; the bits in the low half.
template <typename T>
__device__ __forceinline__ uint32_t from_f32(float x)
{
    return __builtin_bit_cast(uint16_t, (typename Types<T>::E)x);
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 raw, float (&v)[8])
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = to_f32<T>(w[e] & 0xffffu);
        v[2 * e + 1] = to_f32<T>(w[e] >> 16);
    }
}

// write: k and v rows into the cache; else back out of it. dim 64/128/256, nbits 4/8, g
// 32/64/128 <= dim.
hipError_t launch_cache_rows(bool write, const CacheView &c, const SeqView &s, const RowPtrs &p,
                             int dim, int nbits, int g, bool bf16, hipStream_t stream);

// ---- attention ---------------------------------------------------------------------------------
// Partial results of one side (the sequences, or the shared prefix) in the workspace. A worker
// leaves at most two pieces of split items: slot 2w for one that began before its run, 2w + 1
// for one that goes on behind it. Whole items go to the output, or with a prefix to `rows`.
struct AttnSide {
    int32_t *starts;            // [n_seqs + 1]: units before each sequence's, of one head
    float *slot_o;              // [heads][2 * workers][rows_per][dim], not divided by the sum
    float *slot_ml;             // [heads][2 * workers][rows_per][2]: maximum (base 2), sum
    float *row_o, *row_ml;      // [heads][n_tokens * per][dim], [..][2], or null
    int32_t workers;            // runs of a head's units
    int32_t tiles16;            // rows_per / 16: 1 or 2
};

struct AttnArgs {
    CacheView c;
    SeqView s;
    AttnSide side;
    const uint16_t *q;
    uint16_t *out;
    float *lse;                 // nullable
    int64_t q_ts, q_hs, o_ts, o_hs;
    int32_t per;                // query heads to a key/value head
    int32_t causal;             // rows see their own position and what is before it, else all
    float scale;                // times log2(e)
};

struct JoinArgs {
    SeqView s;                  // the call's sequences
    AttnSide side, prefix;      // prefix.starts null: none
    uint16_t *out;
    float *lse;
    int64_t o_ts, o_hs;
    int32_t per, heads, dim;
    int32_t prefix_len;
};

struct AttnShape {
    int dim, nbits, g;
    bool bf16;
};

hipError_t launch_attn(const AttnArgs &a, const AttnShape &x, hipStream_t stream);
hipError_t launch_join(const JoinArgs &a, bool bf16, hipStream_t stream);

// by type and width of the codes, one translation unit each
hipError_t launch_attn_f16_4(const AttnArgs &a, const AttnShape &x, hipStream_t stream);
hipError_t launch_attn_f16_8(const AttnArgs &a, const AttnShape &x, hipStream_t stream);
hipError_t launch_attn_bf16_4(const AttnArgs &a, const AttnShape &x, hipStream_t stream);
hipError_t launch_attn_bf16_8(const AttnArgs &a, const AttnShape &x, hipStream_t stream);

}  // namespace hqq
