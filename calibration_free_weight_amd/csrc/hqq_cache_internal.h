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

// Inclusive sum over the lanes of a wave: within rows of 16, then from row to row.
__device__ __forceinline__ int wave_sum(int x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);     // row_shr 1, 2, 4, 8
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);     // lane 15 of a row to the next one
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);     // lane 31 to the upper half
    return x;
}

// The sequence of the call's row `i`, which is the wave's first row or close behind it: the
// wave looks for the first together, 64 entries at a time, and each lane goes on from there.
// All lanes of the wave must come here.
__device__ __forceinline__ int find_seq(const SeqView &s, int i)
{
    if (!s.cu) return seq_at(s, i);
    const int lane = threadIdx.x & 63;
    const int first = __builtin_amdgcn_readfirstlane(i);
    int lo = 0, n = s.n_seqs;               // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) >> 6;
        const bool le = lane == 0 || (lane * step < n && s.cu[lo + lane * step] <= first);
        const int k = __popcll(__ballot(le)) - 1;
        n = min(step, n - k * step);
        lo += k * step;
    }
    while (lo + 1 < s.n_seqs && s.cu[lo + 1] <= i) ++lo;
    return lo;
}

// A block of a write or read has 256 * 8 / head_dim tokens of four heads at a time, whose loads
// are then under way together, or of one where four would leave the GPU's 1024 units without a
// few waves each: from 2^23 numbers on for a write (8 heads of 128, 4 bits: 4096 tokens 9.4 us
// with four and 8.1 with one, 16384 tokens both 25; 18060 tokens of 32 heads 89 and 110), 2^22
// for a read (8 heads of 128, 8 bits: 2000 tokens 4.6 and 4.7, 6000 tokens 7.9 and 9.2, 65521
// tokens 80 and 98; of 64, 4 bits: 4000 tokens 5.5 and 4.7, 12000 tokens 8.5 and 8.9).
constexpr int kRowThreads = 256;
inline bool four_heads(bool write, int64_t n_tokens, int heads, int dim)
{
    return n_tokens * heads * dim >= int64_t(1) << (write ? 23 : 22);
}
inline int64_t cache_rows_blocks(bool write, int64_t n_tokens, int heads, int dim)
{
    const int tokens = 8 * kRowThreads / dim, at_once = four_heads(write, n_tokens, heads, dim) ? 4 : 1;
    return (n_tokens + tokens - 1) / tokens * ((heads + at_once - 1) / at_once);
}

// write: k and v rows into the cache; else back out of it. dim 64/128/256, nbits 4/8, g
// 32/64/128 <= dim.
hipError_t launch_cache_rows(bool write, const CacheView &c, const SeqView &s, const RowPtrs &p,
                             int dim, int nbits, int g, bool bf16, hipStream_t stream);

// ---- accepted tokens kept -----------------------------------------------------------------------
constexpr int kKeepLayers = 64;             // of a launch: 2 KB of arguments
struct KeepArgs {
    SeqView s;
    const int32_t *kept;        // [n_seqs][max_kept]
    int32_t *lens_out;          // nullable
    int32_t max_kept, heads, groups;
    struct {
        uint8_t *part[4];       // codes of keys and of values, grids of keys and of values
    } layers[kKeepLayers];
};

hipError_t launch_keep(const KeepArgs &a, int n_layers, int dim, int nbits, hipStream_t stream);

// ---- attention ---------------------------------------------------------------------------------
// What the rows of a call attend to comes from one or two sides: the sequences, and a prefix
// that all share (one sequence with all rows of the call). A run leaves at most two pieces of
// split items in the workspace: slot 2w for one that began before the run, 2w + 1 for one that
// goes on behind it. Whole items go to the output, or with two sides to `row_o`.
struct AttnSide {
    SeqView s;
    int32_t *starts;            // [n_seqs + 2]: units before each sequence's, of one head, and
                                // their tokens; null without a joining launch, as the pieces
    float *slot_o;              // [heads][2 * workers][rows_per][dim], not divided by the sum
    float *slot_ml;             // [heads][2 * workers][rows_per][2]: maximum (base 2), sum
    float *row_o, *row_ml;      // [heads][n_tokens * per][dim], [..][2], or null
    int32_t workers;            // most runs of a head's units
    int32_t unit;               // tokens, at least
    int32_t tiles16;            // rows_per / 16: 1, 2 or 8, and 1, 2 or 4 with heads of 256
    int32_t causal;             // rows see their own position and what is before it, else all
};

struct AttnArgs {
    CacheView c;
    AttnSide side[2];           // of the same tiles16
    int32_t sides;              // in this launch
    const uint16_t *q;
    uint16_t *out;
    float *lse;                 // nullable
    int64_t q_ts, q_hs, o_ts, o_hs;
    int32_t per;                // query heads to a key/value head
    float scale;                // times log2(e)
    const uint64_t *tree;       // masks of the call's rows, tree_words each, or null
    int32_t tree_words;
};

struct JoinArgs {
    AttnSide side[2];           // the sequences; the prefix
    int32_t sides;
    uint16_t *out;
    float *lse;
    int64_t o_ts, o_hs;
    int32_t per, heads, dim;
};

struct AttnShape {
    int dim, nbits, g;
    bool bf16;
};

// Blocks of a launch that a CU holds, by the registers that the kernels' sums and codes in flight
// take: their launch bounds are made of this, and no more blocks are launched. (With 1152 or 1536
// rather than 1024 the last ones begin when the first are done, and take longer in all. Heads of 64
// in tiles of 32 rows would fit four times, with some registers in memory: 64 heads, 200 rows over
// 2000 tokens, 4 bits 94 us and 98.5, but 32 heads of 80 rows over 1000 tokens 39.6 and 33.)
constexpr int blocks_per_cu(int tiles16, int dim, int nbits)
{
    return tiles16 > 1 || dim == 256 ? 2 : nbits == 8 && dim == 128 ? 3 : 4;
}

hipError_t launch_attn(const AttnArgs &a, const AttnShape &x, hipStream_t stream);
hipError_t launch_join(const JoinArgs &a, bool bf16, hipStream_t stream);

// by type and width of the codes, one translation unit each
hipError_t launch_attn_f16_4(const AttnArgs &a, const AttnShape &x, hipStream_t stream);
hipError_t launch_attn_f16_8(const AttnArgs &a, const AttnShape &x, hipStream_t stream);
hipError_t launch_attn_bf16_4(const AttnArgs &a, const AttnShape &x, hipStream_t stream);
hipError_t launch_attn_bf16_8(const AttnArgs &a, const AttnShape &x, hipStream_t stream);
hipError_t launch_attn_tree_f16_4(const AttnArgs &a, const AttnShape &x, hipStream_t stream);
hipError_t launch_attn_tree_f16_8(const AttnArgs &a, const AttnShape &x, hipStream_t stream);
hipError_t launch_attn_tree_bf16_4(const AttnArgs &a, const AttnShape &x, hipStream_t stream);
hipError_t launch_attn_tree_bf16_8(const AttnArgs &a, const AttnShape &x, hipStream_t stream);

}  // namespace hqq
