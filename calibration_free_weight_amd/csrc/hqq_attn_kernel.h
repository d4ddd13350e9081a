// hqq_attn_kernel.h -- attention over the quantized cache on the matrix cores (gfx950);
// included by one translation unit per type and code width.
//
// A block of four waves takes a run of units (128 tokens of one sequence and key/value head)
// for a tile of 16 * RT query rows; each wave takes 32 tokens of a unit. Everything stays in
// registers: with C = A . B on 16x16x32 tiles (lane l: A row l%16, B column l%16, eight values
// of the contraction from 8*(l/16); C column l%16, rows 4*(l/16)..+3),
//   S^T = K . Q^T      A = codes of 16 tokens, B = queries: a lane gets its column's scores of
//                      tokens 4*(l/16)..+3;
//   O^T = V^T . P^T    B = weights of 32 tokens: exactly the scores the lane already has (two
//                      tiles of four tokens), the order of the contraction being free;
// so weights never cross lanes, and the running maximum and sums are per lane (the maximum
// agreed on by the four lanes of a column, and only when some column's grows by more than a
// factor of 2^6). Codes go into the products as whole numbers, and the grids are applied to
// the sums: S = step . (q, Q) + base . sum(Q) per group; V's step goes to the weights, and the
// middle of V's grid, times the weights, is summed beside. The 16 lanes of a row of lanes hold
// the grids of its four tokens, one group each, and a broadcast within the row is part of the
// multiplication that takes one (DPP), so a grid costs no register of its own and no
// conversion per use. Whatever the lengths, a token outside its sequence has grid {0, 0} and
// weight 0.
#pragma once

#include "hqq_cache_internal.h"

namespace hqq {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;

constexpr int kWaves = 4;                   // of a block for tiles of few rows
constexpr int kTile = 32;                   // tokens of a wave's step
static_assert(kTile * kWaves == kStep, "a step is a tile for each wave");

template <bool BF16>
__device__ __forceinline__ f32x4 mfma32(const u32x4 a, const u32x4 b, const f32x4 c)
{
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Lane N of each row of 16 lanes, for all of the row.
template <int N>
__device__ __forceinline__ float row_lane(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + N, 0xf, 0xf, true));
}

// acc[r] += lane N[r] of each row of 16 lanes of k[r], times x[r]: the broadcast is part of the
// instruction, which the compiler makes of a product alone. What it would keep apart for its own
// instructions is kept apart here: two wait states behind whatever wrote k and x, and `settled`,
// which reads the matrix products that x or acc come from and so comes after their last. (acc is
// written before all of k and x are read.)
template <int N0, int N1, int N2, int N3>
__device__ __forceinline__ void add_row_lanes(float (&acc)[4], const float (&k)[4], const float (&x)[4], uint32_t settled)
{
    asm("s_nop 1\n"
        "v_fmac_f32_dpp %0, %4, %8 row_newbcast:%13 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %1, %5, %9 row_newbcast:%14 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %2, %6, %10 row_newbcast:%15 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %3, %7, %11 row_newbcast:%16 row_mask:0xf bank_mask:0xf"
        : "+&v"(acc[0]), "+&v"(acc[1]), "+&v"(acc[2]), "+&v"(acc[3])
        : "v"(k[0]), "v"(k[1]), "v"(k[2]), "v"(k[3]), "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]), "v"(settled),
          "n"(N0), "n"(N1), "n"(N2), "n"(N3));
}
// The same into one number.
template <int N0, int N1, int N2, int N3>
__device__ __forceinline__ void add_row_lanes(float &acc, const float (&k)[4], const float (&x)[4])
{
    asm("s_nop 1\n"
        "v_fmac_f32_dpp %0, %1, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %0, %2, %6 row_newbcast:%10 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %0, %3, %7 row_newbcast:%11 row_mask:0xf bank_mask:0xf\n"
        "v_fmac_f32_dpp %0, %4, %8 row_newbcast:%12 row_mask:0xf bank_mask:0xf"
        : "+&v"(acc)
        : "v"(k[0]), "v"(k[1]), "v"(k[2]), "v"(k[3]), "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]),
          "n"(N0), "n"(N1), "n"(N2), "n"(N3));
}

// Two whole numbers 0..15 in neighbouring bytes (pair HI: bytes 2, 3) as two values of the
// type. A byte 0..15 read as e4m3 is that number of 2^-9: subnormal up to 7, and with
// exponent field 1 from 8 on, which has the same spacing.
template <bool BF16, bool HI>
__device__ __forceinline__ uint32_t small2(uint32_t bytes)
{
    if constexpr (BF16)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, 512.f, HI));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(bytes, 512.f, HI));
}

// Two binary32 whole numbers up to 255 as bfloat16 (their upper halves; nothing is lost).
__device__ __forceinline__ uint32_t whole_bf16x2(float a, float b)
{
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

__device__ __forceinline__ float ubyte(uint32_t w, int k) { return (float)(w >> (8 * k) & 255u); }

// The eight codes of a key's unit as a fragment of the type.
template <bool BF16, int NB>
__device__ __forceinline__ u32x4 key_frag(const uint32_t *w)
{
    u32x4 f;
    if constexpr (NB == 4) {
        const uint32_t lo = w[0] & 0x0f0f0f0fu, hi = w[0] >> 4 & 0x0f0f0f0fu;
        f[0] = small2<BF16, false>(lo);
        f[1] = small2<BF16, true>(lo);
        f[2] = small2<BF16, false>(hi);
        f[3] = small2<BF16, true>(hi);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if constexpr (BF16) {
                f[2 * k] = whole_bf16x2(ubyte(w[k], 0), ubyte(w[k], 1));
                f[2 * k + 1] = whole_bf16x2(ubyte(w[k], 2), ubyte(w[k], 3));
            } else {
                // 0x6400 | byte is 1024 + byte in binary16
                const f16x2 off = {(_Float16)1024.f, (_Float16)1024.f};
                const uint32_t a = __builtin_amdgcn_perm(0x64646464u, w[k], 0x04010400u);
                const uint32_t b = __builtin_amdgcn_perm(0x64646464u, w[k], 0x04030402u);
                f[2 * k] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) - off);
                f[2 * k + 1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, b) - off);
            }
        }
    }
    return f;
}

// Code i of a value's row for two tokens (words x, y hold it), less the middle of the codes
// (8 or 128), as binary16 numbers: exact, and half as large as the codes, so that the
// rounding of the weights they meet weighs no more than it would on the values themselves.
struct Masks {
    uint32_t low, high;         // kept in vector registers: "and" and "or" are then one instruction
};
template <int NB>
__device__ __forceinline__ uint32_t value_pair(const uint32_t *x, const uint32_t *y, int i, const Masks &masks)
{
    uint32_t w;
    float off;
    if constexpr (NB == 4) {
        // Codes 4c..4c+3 of both tokens in the halves of a word. With exponent bits over it,
        // a code in the lowest bits stands for 1024 + q, one in bits 4 to 7 for 64 + q.
        const int c = i >> 2, k = c & 1;
        uint32_t p = __builtin_amdgcn_perm(y[c >> 1], x[c >> 1], k ? 0x07060302u : 0x05040100u);
        if (i & 2) p >>= 8;
        w = i & 1 ? (p & masks.high) | 0x54005400u : (p & masks.low) | 0x64006400u;
        off = i & 1 ? 72.f : 1032.f;
    } else {
        const uint32_t p = __builtin_amdgcn_perm(y[i >> 2], x[i >> 2], i & 2 ? 0x07030602u : 0x05010400u);
        w = __builtin_amdgcn_perm(0x64646464u, p, i & 1 ? 0x04030402u : 0x04010400u);
        off = 1152.f;
    }
    const f16x2 mid = {(_Float16)off, (_Float16)off};
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, w) - mid);
}

__device__ __forceinline__ uint32_t round_pair(float a, float b)
{
    const f32x2 x = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, f16x2));
}

// Global memory from a pointer that is the same in all lanes, in scalar registers, and a
// lane's offset from it in 32 bits (an addition per load less than with a pointer per lane).
typedef const __attribute__((address_space(1))) uint8_t *Global;
__device__ __forceinline__ Global uniform(const void *p)
{
    const uint64_t x = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
    return (Global)((uint64_t)hi << 32 | lo);
}
template <typename V>
__device__ __forceinline__ V load(Global p, uint32_t offset)
{
    asm volatile("" : "+v"(offset));        // widened here, where the load can take it as it is
    return *(const __attribute__((address_space(1))) V *)(p + offset);
}

// The page of position pos (below the length) of the sequence whose pages are at `table`, or -1:
// a scalar load, for nothing writes the table while the kernel runs.
typedef const __attribute__((address_space(4))) int32_t *Constant;
__device__ __forceinline__ int page_at(const SeqView &s, const int32_t *table, int pos)
{
    const int p = ((Constant)(uint64_t)table)[pos >> s.page_shift];
    return (uint32_t)p < (uint32_t)s.n_pages ? p : -1;
}

__device__ __forceinline__ float larger3(float a, float b, float c)
{
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

template <int BYTES>
__device__ __forceinline__ void load_words(Global p, uint32_t offset, uint32_t (&w)[BYTES / 4])
{
    static_assert(BYTES == 4 || BYTES == 8 || BYTES % 16 == 0, "4, 8 or a multiple of 16");
    if constexpr (BYTES == 4) {
        w[0] = load<uint32_t>(p, offset);
    } else if constexpr (BYTES % 16 == 0) {
#pragma unroll
        for (int k = 0; k < BYTES / 16; ++k) {
            const u32x4 x = load<u32x4>(p, offset + 16 * k);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[4 * k + e] = x[e];
        }
    } else {
        const u32x2 x = load<u32x2>(p, offset);
        w[0] = x[0];
        w[1] = x[1];
    }
}

template <int I>
struct Index {
    static constexpr int value = I;
};
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(F &&f)
{
    if constexpr (I < N) {
        f(Index<I>{});
        static_for<N, I + 1>(f);
    }
}

// Largest and smallest over the lanes whose number leaves the same rest by N (1 to 8): rotations
// within rows of 16 lanes, then over the rows.
template <int N>
__device__ __forceinline__ void over_same_group(float &most, float &least)
{
    const auto with = [&](float a, float b) {
        most = fmaxf(most, a);
        least = fminf(least, b);
    };
    const auto turned = [](float x, auto by) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + by.value, 0xf, 0xf, true));
    };
    with(turned(most, Index<8>{}), turned(least, Index<8>{}));
    if constexpr (N <= 4) with(turned(most, Index<4>{}), turned(least, Index<4>{}));
    if constexpr (N <= 2) with(turned(most, Index<2>{}), turned(least, Index<2>{}));
    if constexpr (N <= 1) with(turned(most, Index<1>{}), turned(least, Index<1>{}));
    with(__shfl_xor(most, 16), __shfl_xor(least, 16));
    with(__shfl_xor(most, 32), __shfl_xor(least, 32));
}

// Sum over the four lanes of a column (16 and 32 apart).
__device__ __forceinline__ float column_sum(float x)
{
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
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

// A run's next item, or the part of it that the run has.
struct Item {
    int b;                      // sequence
    Rows rows;                  // its rows of the call
    int len, n_rows;            // tokens; query rows of this head
    int row0;                   // the item's first
    int along, u_in, count;     // units of the item, the first of this part, how many
};

// The units of a side, end to end. Up to 64 sequences each wave has them in its lanes, and
// nothing waits for another; more are summed up in LDS. Where runs would be short, units are
// made longer until there is one to a run: a run that ends one item and begins another pays
// for its start and its end twice, which is as much as several steps (16 sequences of 800 to 2900
// tokens with 5 new ones each, in tiles of 32 rows of heads of 256: 36 us, 40 with units of 128).
constexpr int kShortRun = 6;    // units

template <int ROWS, int WAVES>
struct Layout {
    const AttnSide &d;
    int per, unit, total;
    int start;                  // of sequence `lane` and its rows and length, with up to 64
    Rows rows;
    int len;
    bool falls;
    int32_t *starts, *scan;     // in LDS, with more: [n_seqs + 1], [WAVES]
    __device__ __forceinline__ bool few() const { return __builtin_expect(d.s.n_seqs <= 64, 1); }
    __device__ __forceinline__ int units(const Rows &r, int len) const
    {
        return tiles_of((r.end - r.begin) * per, ROWS) * units_along(len, unit);
    }
    // The sum of what the threads have, before the caller's (`before`) and in all.
    __device__ __forceinline__ int block_sum(int x, int &before)
    {
        const int t = threadIdx.x, upto = wave_sum(x);
        __syncthreads();
        if ((t & 63) == 63) scan[t >> 6] = upto;
        __syncthreads();
        before = upto - x;
        int all = 0;
        for (int w = 0; w < WAVES; ++w) {
            if (w < (t >> 6)) before += scan[w];
            all += scan[w];
        }
        return __builtin_amdgcn_readfirstlane(all);
    }
    // The units before the lane's sequences (`before`) and in all (none if row offsets fall), and
    // with more than 64 those of each of the thread's, to `starts`.
    __device__ __forceinline__ int count(int &before, bool keep)
    {
        if (few()) {
            const int u = (int)(threadIdx.x & 63) < d.s.n_seqs ? units(rows, len) : 0;
            const int upto = wave_sum(u);
            before = upto - u;
            return __any(falls) ? 0 : __builtin_amdgcn_readlane(upto, 63);
        }
        const int t = threadIdx.x, n = d.s.n_seqs;
        const int each = (n + 64 * WAVES - 1) / (64 * WAVES), b0 = min(t * each, n), b1 = min(b0 + each, n);
        int sum = 0;
        falls = false;
        for (int b = b0; b < b1; ++b) {
            sum += units(rows_of(d.s, b), len_of(d.s, b));
            falls = falls || falls_at(d.s, b);
        }
        const int upto = block_sum(sum, before), all = __syncthreads_or(falls) ? 0 : upto;
        if (keep) {
            int at = before;
            for (int b = b0; b < b1; ++b) {
                starts[b] = at;
                at += units(rows_of(d.s, b), len_of(d.s, b));
            }
            if (t == 0) starts[n] = all;
            __syncthreads();
        }
        return all;
    }
    __device__ __forceinline__ void read()
    {
        const int lane = threadIdx.x & 63;
        if (lane < d.s.n_seqs) {
            rows = rows_of(d.s, lane);
            len = len_of(d.s, lane);
            falls = falls_at(d.s, lane);
        }
    }

    __device__ __forceinline__ Layout(const AttnSide &side, int per, int32_t *starts, int32_t *scan)
        : d(side), per(per), unit(side.unit), start(0), rows{0, 0}, len(0), falls(false), starts(starts), scan(scan)
    {
        if (few()) read();
        total = count(start, false);
        const int longest = d.s.fixed_len >= 0 ? d.s.fixed_len : d.s.max_pages << d.s.page_shift;
        if (__builtin_expect(total > d.workers && total <= kShortRun * d.workers && unit < longest, 0)) {
            const int times = (total + d.workers - 1) / d.workers, first = unit;
            // two tries: rounding up by sequence may leave more units than runs
            for (int more = 0; more < 2; ++more) {
                unit = first * (times + more);
                total = count(start, false);
                if (total <= d.workers) break;
            }
            if (total > d.workers) {
                unit = first;
                total = count(start, false);
            }
        }
        if (!few()) count(start, true);
    }
    // Before a further item: what the lanes had is read again rather than kept in registers.
    __device__ __forceinline__ void again()
    {
        if (!few()) return;
        read();
        total = count(start, false);
    }

    // to: [n_seqs + 2] in memory, the last the unit
    __device__ __forceinline__ void put(int32_t *to) const
    {
        const int t = threadIdx.x, n = d.s.n_seqs;
        if (t == 0) to[n + 1] = unit;
        if (few()) {
            if (t < n) to[t] = start;
            if (t == 0) to[n] = total;
        } else {
            for (int b = t; b <= n; b += 64 * WAVES) to[b] = starts[b];
        }
    }

    __device__ __forceinline__ Item item(int u, int u_end) const
    {
        Item x;
        int first;
        if (few()) {
            const bool le = (int)(threadIdx.x & 63) < d.s.n_seqs && start <= u;
            x.b = __popcll(__ballot(le)) - 1;
            x.rows.begin = __builtin_amdgcn_readlane(rows.begin, x.b);
            x.rows.end = __builtin_amdgcn_readlane(rows.end, x.b);
            x.len = __builtin_amdgcn_readlane(len, x.b);
            first = __builtin_amdgcn_readlane(start, x.b);
        } else {
            x.b = 0;
            for (int hi = d.s.n_seqs; hi - x.b > 1;) {
                const int mid = (x.b + hi) >> 1;
                if (__builtin_amdgcn_readfirstlane(starts[mid]) <= u) x.b = mid; else hi = mid;
            }
            const Rows r = rows_of(d.s, x.b);
            x.rows.begin = __builtin_amdgcn_readfirstlane(r.begin);
            x.rows.end = __builtin_amdgcn_readfirstlane(r.end);
            x.len = __builtin_amdgcn_readfirstlane(len_of(d.s, x.b));
            first = __builtin_amdgcn_readfirstlane(starts[x.b]);
        }
        x.n_rows = (x.rows.end - x.rows.begin) * per;
        x.along = units_along(x.len, unit);
        const unsigned in_seq = u - first, tile = in_seq / (unsigned)x.along;
        x.row0 = (int)tile * ROWS;
        x.u_in = (int)(in_seq - tile * x.along);
        x.count = min(u_end - u, x.along - x.u_in);
        return x;
    }
};

// How far a score may lie above the maximum that weights are taken from: weights reach 2^6.
constexpr float kSlack = 6.f;
// V's steps go into the products times a power of two of the wave and group that brings them to 1
// or more and below 2^9: weight times step then stays below 2^15 in binary16, and a weight keeps 11
// bits or is off by 2^-25 at most, where a row's largest is at least 1. Tokens that do not fit in
// are left out (of the codes' part) and come behind the others, in attend_rest, where every row and
// group has a power of two of its own: however large a token's values, it has no say in rows that do
// not see it or hardly weigh it.
constexpr uint32_t kStepLow = 0x3f800000u, kStepHigh = 0x44000000u;     // bits of 1 and 2^9
// The sums of products are in units of 1/by: by is at least 2^-40, at which they hold whatever V
// can, and lose of the smallest numbers less than 2^-104 (a step of bfloat16 is 2^-100 or more);
// above that, a product of 2^60 units or more first lowers it to 2^-40.
constexpr float kLeastBy = 0x1p-40f, kMostUnits = 0x1p60f;

// What a wave keeps of its 16 * RT query rows (a lane: of its column of each 16). BASE_FRAGS: the
// bases' part of the scores is a product too, see base_query.
template <int D, int G, int RT, bool BASE_FRAGS>
struct Wave {
    static constexpr int kGroups = D / G;
    u32x4 qf[RT][D / 32];       // queries, as B fragments
    float qsum[RT][kGroups];    // their sums over each group, scaled
    int lim[RT];                // what a row sees ends here
    int lim_low, lim_high;      // for all rows, for any
    f32x4 o[RT][D / 16];
    u32x4 qb[BASE_FRAGS ? RT : 1][kGroups > 4 ? 2 : 1];      // the sums as B fragments
    // m: scores are taken from it; above: how far one may lie above before m moves (none
    // while m has not been set)
    float m[RT], above[RT], l[RT], bsum[RT][kGroups];
    float by;                   // V's steps of group lane % kGroups go in times this; 0 before there are any
    bool rest;                  // some of V's steps did not fit
};

// The bases' part of the scores as one product of bfloat16 parts: slot e of the contraction's
// quads 0, 1 and 2 has the base of group e (its first part) and the first, second and third part
// of the column's sum over that group, of quad 3 the second part of the base (none of a bfloat16
// one) and the first of the sum; slot e + base_slots() of quad 3, the second of both. What is
// left out is below 2^-23 of the product. Eight groups take two such products.
template <int GROUPS>
constexpr int base_products() { return GROUPS > 4 ? 2 : 1; }
template <int GROUPS>
constexpr int base_slots() { return GROUPS < 2 ? 2 : GROUPS / base_products<GROUPS>(); }
template <int GROUPS>
__device__ __forceinline__ u32x4 base_query(const float (&sum)[GROUPS], int product, int quad)
{
    constexpr int kSlots = base_slots<GROUPS>();
    static_assert(kSlots <= 4, "two slots for each group");
    uint32_t bits[8] = {};
#pragma unroll
    for (int g = 0; g < kSlots && g < GROUPS; ++g) {
        float x = sum[product * kSlots + g];
        const uint32_t first = from_f32<Bf16>(x);
        x -= to_f32<Bf16>(first);
        const uint32_t second = from_f32<Bf16>(x);
        x -= to_f32<Bf16>(second);
        bits[g] = quad == 1 ? second : quad == 2 ? from_f32<Bf16>(x) : first;
        bits[g + kSlots] = quad == 3 ? second : 0u;
    }
    u32x4 f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = bits[2 * e] | bits[2 * e + 1] << 16;
    return f;
}

template <typename T, int D, int G, int RT, bool BASE_FRAGS>
__device__ __forceinline__ void begin(Wave<D, G, RT, BASE_FRAGS> &w, const AttnArgs &a, bool causal, const Item &x, int h, int row0)
{
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int col = lane & 15, quad = lane >> 4;
    const unsigned per = a.per;
    // what the first and the last of the wave's rows see
    const int before = causal ? x.len - (x.rows.end - x.rows.begin) + 1 : x.len;
    const int last = min(row0 + 16 * RT, x.n_rows) - 1;
    w.lim_low = row0 <= last ? before + (causal ? (int)((unsigned)row0 / per) : 0) : 0;
    w.lim_high = row0 <= last ? before + (causal ? (int)((unsigned)last / per) : 0) : 0;
    uint4 raw[RT][D / 32];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int row = row0 + 16 * t + col;
        const bool have = row < x.n_rows;
        const int tok = have ? (int)((unsigned)row / per) : 0, hq = h * a.per + (have ? row - tok * a.per : 0);
        const uint16_t *q = a.q + (x.rows.begin + tok) * a.q_ts + hq * a.q_hs + 8 * quad;
        w.lim[t] = !have ? 0 : before + (causal ? tok : 0);
#pragma unroll
        for (int m = 0; m < D / 32; ++m) {
            raw[t][m] = uint4{0, 0, 0, 0};
            if (have) raw[t][m] = *reinterpret_cast<const uint4 *>(q + 32 * m);
        }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int g = 0; g < D / G; ++g) {
            float sum = 0.f;
#pragma unroll
            for (int m = g * G / 32; m < (g + 1) * G / 32; ++m) {
                w.qf[t][m] = u32x4{raw[t][m].x, raw[t][m].y, raw[t][m].z, raw[t][m].w};
                float v[8];
                unpack8<T>(raw[t][m], v);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += v[e];
            }
            w.qsum[t][g] = column_sum(sum) * a.scale;
            w.bsum[t][g] = 0.f;
        }
        if constexpr (BASE_FRAGS)
#pragma unroll
            for (int p = 0; p < base_products<D / G>(); ++p) w.qb[t][p] = base_query<D / G>(w.qsum[t], p, quad);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) w.o[t][j] = f32x4{0, 0, 0, 0};
        w.m[t] = 0.f;
        w.above[t] = -INFINITY;
        w.l[t] = 0.f;
    }
    w.by = 0.f;
    w.rest = false;
}

// The lanes' places for the grids of 16 tokens: quad x holds those of tokens 4x..4x+3, lane c
// of register k the one of token (c + 16 k) / kGroups of them, group (c + 16 k) % kGroups.
template <int D, int G>
struct Places {
    static constexpr int kGroups = D / G, kGrids = 4 * kGroups, kRegs = (kGrids + 15) / 16;
    static __device__ __forceinline__ int token(int k)
    {
        const int lane = threadIdx.x & 63;
        return lane / 16 * 4 + ((lane & 15 & (kGrids - 1)) + 16 * k) / kGroups;
    }
};

// Whether all of a step's 32 tokens from t0 are there, for all of the wave's rows.
template <int D, int G, int RT, bool BASE_FRAGS>
__device__ __forceinline__ bool all_there(const Wave<D, G, RT, BASE_FRAGS> &w, int t0, const int (&good)[2])
{
    return t0 + kTile <= w.lim_low && good[0] >= 16 && good[1] >= 16;
}

// The scores of 32 tokens from t0 for the wave's rows, to base 2 and less m, good[half] of each 16
// there (or more; none if negative), -infinity where a row does not see one. key_grid(half, k)
// gives {step * scale, base} of a lane's place; key(half, mm) the A fragments. after_keys() is
// called when no more keys are needed. With BASE_FRAGS base(half, p) is the A fragment of the bases
// (base_query has the other), and what key_grid says of them is not used.
template <typename T, int D, int G, int RT, bool BASE_FRAGS, typename KeyGrid, typename Base, typename Key, typename After>
__device__ __forceinline__ void scores(const Wave<D, G, RT, BASE_FRAGS> &w, int t0, const int (&good)[2], bool open,
                                       KeyGrid key_grid, Base base, Key key, After after_keys, float (&s)[RT][8])
{
    constexpr bool kBf16 = Types<T>::kBf16;
    constexpr int kGroups = D / G, kRegs = Places<D, G>::kRegs;
    const int quad = (threadIdx.x & 63) >> 4;
    static_for<2>([&](auto half) {
        f32x4 acc[RT][kGroups], from[RT];
        f32x2 kgrid[kRegs];
#pragma unroll
        for (int k = 0; k < kRegs; ++k) kgrid[k] = key_grid(half.value, k);
#pragma unroll
        for (int t = 0; t < RT; ++t) from[t] = f32x4{-w.m[t], -w.m[t], -w.m[t], -w.m[t]};
        if constexpr (BASE_FRAGS)
#pragma unroll
            for (int p = 0; p < base_products<kGroups>(); ++p) {
                const u32x4 bf = base(half.value, p);
#pragma unroll
                for (int t = 0; t < RT; ++t) from[t] = mfma32<true>(bf, w.qb[t][p], from[t]);
            }
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
#pragma unroll
            for (int t = 0; t < RT; ++t) acc[t][g] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int mm = g * G / 32; mm < (g + 1) * G / 32; ++mm) {
                const u32x4 kf = key(half.value, mm);
#pragma unroll
                for (int t = 0; t < RT; ++t) acc[t][g] = mfma32<kBf16>(kf, w.qf[t][mm], acc[t][g]);
            }
        }
        if constexpr (half.value == 1) after_keys();
        uint32_t settled = 0;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            settled |= __float_as_uint(from[t][3]);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) settled |= __float_as_uint(acc[t][g][3]);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            float sum[4] = {from[t][0], from[t][1], from[t][2], from[t][3]};
            static_for<kGroups>([&](auto g) {
                constexpr int at0 = g.value, at1 = at0 + kGroups, at2 = at1 + kGroups, at3 = at2 + kGroups;
                auto grids = [&](int e, float (&k)[4]) {
                    k[0] = kgrid[at0 / 16][e], k[1] = kgrid[at1 / 16][e], k[2] = kgrid[at2 / 16][e], k[3] = kgrid[at3 / 16][e];
                };
                float k[4];
                if constexpr (!BASE_FRAGS) {
                    const float q = w.qsum[t][g.value], all[4] = {q, q, q, q};
                    grids(1, k);
                    add_row_lanes<at0 % 16, at1 % 16, at2 % 16, at3 % 16>(sum, k, all, settled);
                }
                const f32x4 x = acc[t][g.value];
                const float each[4] = {x[0], x[1], x[2], x[3]};
                grids(0, k);
                add_row_lanes<at0 % 16, at1 % 16, at2 % 16, at3 % 16>(sum, k, each, settled);
            });
#pragma unroll
            for (int r = 0; r < 4; ++r) s[t][4 * half.value + r] = sum[r];
        }
    });
    if (__builtin_expect(!open, 0)) {
        int first = t0 + 4 * quad;
        asm volatile("" : "+v"(first));                     // a branch, not a choice in every step
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = first + 16 * (i >> 2) + (i & 3);
                if (at >= min(w.lim[t], t0 + 16 * (i >> 2) + good[i >> 2])) s[t][i] = -INFINITY;
            }
    }
}

__device__ __forceinline__ uint32_t misfit(float step) { return __float_as_uint(step) - kStepLow; }    // kMisfit or more
constexpr uint32_t kMisfit = kStepHigh - kStepLow;

// A `by` for V's steps of a step that are not all 0 and, times the one that there is, do not all
// fit. 2^8 to 2^9 for the largest, if the smallest is 1 or more then: taken at first, and when it is
// lower than what there is. At first, if they do not fit, that for the smallest: large ones are
// rarer. The same steps one after another give the same, in attend_rest again. each_step(f) calls
// f with a lane's steps, one after another.
template <int GROUPS, typename Each>
__device__ __forceinline__ float fitting(float by, Each each_step)
{
    float most = 0.f, least = INFINITY;
    each_step([&](float step) {
        most = fmaxf(most, step);
        least = fminf(least, step > 0.f ? step : INFINITY);
    });
    over_same_group<GROUPS>(most, least);
    const auto by_of = [](float step) {
        // 2^8 over the power of two at or below the step, by exponents
        return fmaxf(__uint_as_float(0x83000000u - (__float_as_uint(fmaxf(step, 0x1p-100f)) & 0x7f800000u)), kLeastBy);
    };
    const float fit = by_of(most);
    const bool fits = least * fit >= 1.f && most * fit < 0x1p9f;
    if (by == 0.f) return !(most > 0.f) ? 0.f : fits ? fit : by_of(least);
    return fits && fit < by ? fit : by;
}

// Of group g and four tokens, whose grids are v and the row's weights p: the weights times the steps.
template <int GROUPS, int REGS, typename Group>
__device__ __forceinline__ void weigh(Group g, const f32x2 (&v)[REGS], const float *p, float (&x)[4])
{
    constexpr int at0 = g.value, at1 = at0 + GROUPS, at2 = at1 + GROUPS, at3 = at2 + GROUPS;
    x[0] = row_lane<at0 % 16>(v[at0 / 16][0]) * p[0];
    x[1] = row_lane<at1 % 16>(v[at1 / 16][0]) * p[1];
    x[2] = row_lane<at2 % 16>(v[at2 / 16][0]) * p[2];
    x[3] = row_lane<at3 % 16>(v[at3 / 16][0]) * p[3];
}

// One step: 32 tokens from t0, good[half] of each 16 there. When some are not, or not for all rows,
// close() is called first, to make the grids of the missing ones {0, 0}. value_grid gives {step,
// middle} of a lane's place and value(j) the A fragments, behind after_keys(); the others are as in
// scores().
template <typename T, int D, int G, int RT, bool BASE_FRAGS, typename Close, typename KeyGrid, typename Base, typename Key,
          typename After, typename ValueGrid, typename Value>
__device__ __forceinline__ void attend_step(Wave<D, G, RT, BASE_FRAGS> &w, int t0, const int (&good)[2], Close close, KeyGrid key_grid,
                                            Base base, Key key, After after_keys, ValueGrid value_grid, Value value)
{
    constexpr int kGroups = D / G, kRegs = Places<D, G>::kRegs;
    const bool open = all_there(w, t0, good);
    if (__builtin_expect(!open, 0)) close();
    float s[RT][8];
    scores<T>(w, t0, good, open, key_grid, base, key, after_keys, s);
    float top[RT];
    bool grown = false;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        top[t] = larger3(larger3(larger3(s[t][0], s[t][1], s[t][2]), s[t][3], s[t][4]),
                         larger3(s[t][5], s[t][6], s[t][7]), s[t][7]);
        grown = grown || top[t] > w.above[t];
    }
    if (__builtin_expect(__any(grown), 0)) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            top[t] = fmaxf(top[t], __shfl_xor(top[t], 16));
            top[t] = fmaxf(top[t], __shfl_xor(top[t], 32));
            // m moves up to the largest score, or at first to it wherever it is
            const float up = top[t] > fminf(w.above[t], 0.f) ? top[t] : 0.f;
            const float f = w.above[t] < 0.f ? 1.f : __builtin_amdgcn_exp2f(-up);
            if (top[t] > -INFINITY) w.above[t] = kSlack;
            w.m[t] += up;
            w.l[t] *= f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s[t][i] -= up;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) w.bsum[t][g] *= f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) w.o[t][j] *= f;
        }
    }

    f32x2 vgrid[2][kRegs];
    uint32_t off = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int k = 0; k < kRegs; ++k) {
            vgrid[half][k] = value_grid(half, k);
            vgrid[half][k][0] *= w.by;
            off = max(off, misfit(vgrid[half][k][0]));
        }
    if (__builtin_expect(!open, 0)) {
        off = 0;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int k = 0; k < kRegs; ++k) {
                // a group that held infinities or NaN, and a weight of 0
                if (!(fabsf(vgrid[half][k][1]) < INFINITY)) vgrid[half][k][1] = 0.f;
                if (value_grid(half, k)[0] != 0.f) off = max(off, misfit(vgrid[half][k][0]));
            }
    }
    if (__builtin_expect(__any(off >= kMisfit), 0)) {       // steps of 0 too, which are no matter
        const float was = w.by;
        w.by = fitting<kGroups>(was, [&](auto f) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int k = 0; k < kRegs; ++k) f(value_grid(half, k)[0]);
        });
        const float f = was > 0.f ? w.by / was : 1.f;
        if (__any(f < 1.f))
            static_for<kGroups>([&](auto g) {
                const float fg = row_lane<g.value>(f);
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int jj = 0; jj < G / 16; ++jj) w.o[t][g.value * (G / 16) + jj] *= fg;
            });
        bool some = false;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int k = 0; k < kRegs; ++k) {
                const float step = value_grid(half, k)[0] * w.by;
                const bool out = misfit(step) >= kMisfit;
                some = some || (out && step != 0.f);
                vgrid[half][k][0] = out ? 0.f : step;
            }
        w.rest = w.rest || __any(some);
    }

#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[t][i] = __builtin_amdgcn_exp2f(s[t][i]);
            w.l[t] += s[t][i];
        }
    // weights times V's step, in binary16
    static_for<kGroups>([&](auto g) {
        u32x4 pf[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            static_for<2>([&](auto half) {
                constexpr int at0 = g.value, at1 = at0 + kGroups, at2 = at1 + kGroups, at3 = at2 + kGroups;
                const f32x2(&v)[kRegs] = vgrid[half.value];
                const float k[4] = {v[at0 / 16][1], v[at1 / 16][1], v[at2 / 16][1], v[at3 / 16][1]};
                const float p[4] = {s[t][4 * half.value], s[t][4 * half.value + 1], s[t][4 * half.value + 2], s[t][4 * half.value + 3]};
                add_row_lanes<at0 % 16, at1 % 16, at2 % 16, at3 % 16>(w.bsum[t][g.value], k, p);
                float x[4];
                weigh<kGroups>(g, v, p, x);
                pf[t][2 * half.value] = round_pair(x[0], x[1]);
                pf[t][2 * half.value + 1] = round_pair(x[2], x[3]);
            });
        }
#pragma unroll
        for (int jj = 0; jj < G / 16; ++jj) {
            const int j = g.value * (G / 16) + jj;
            const u32x4 vf = value(j);
#pragma unroll
            for (int t = 0; t < RT; ++t) w.o[t][j] = mfma32<false>(vf, pf[t], w.o[t][j]);
        }
    });
}

// What attend_step left out of 32 tokens, behind all steps of the item: the codes' part of the
// tokens whose steps of V did not fit, `by` being what it was before this step then (0 before the
// first). A row's weights go in times the power of two that brings the largest of its products in
// the group to 2^14, and its sums in units of the same meanwhile (of more where they hold 2^100 of
// these). The arguments are those of attend_step.
// Kept out of the step, where the same cost the usual path 8 to 18% (its sums were copied, or other
// values went to memory). Such tokens take about twice a step: 64 sequences of 4100 to 8190 tokens,
// 8 heads of 128, 4 bits 106 us without any, 114 with one token in 1000 and 199 with every third
// far below the others; 2 x 500 rows over 3500 to 4000 tokens, 40 heads 170, 232 and 472.
template <typename T, int D, int G, int RT, bool BASE_FRAGS, typename Close, typename KeyGrid, typename Base, typename Key,
          typename ValueGrid, typename Value>
__device__ __forceinline__ void attend_rest(Wave<D, G, RT, BASE_FRAGS> &w, float &by, int t0, const int (&good)[2], Close close,
                                            KeyGrid key_grid, Base base, Key key, ValueGrid value_grid, Value value)
{
    constexpr int kGroups = D / G, kRegs = Places<D, G>::kRegs;
    const bool open = all_there(w, t0, good);
    if (!open) close();
    f32x2 vgrid[2][kRegs];
    bool out = false, some = false;
    const auto each = [&](auto f) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int k = 0; k < kRegs; ++k) f(value_grid(half, k)[0], vgrid[half][k]);
    };
    each([&](float step, f32x2 &) { out = out || (step != 0.f && misfit(step * by) >= kMisfit); });
    if (!__any(out)) return;
    by = fitting<kGroups>(by, [&](auto f) { each([&](float step, f32x2 &) { f(step); }); });
    each([&](float step, f32x2 &v) {
        const bool left = step != 0.f && misfit(step * by) >= kMisfit;
        some = some || left;
        v = f32x2{left ? step : 0.f, 0.f};
    });
    if (!__any(some)) return;
    float s[RT][8];
    scores<T>(w, t0, good, open, key_grid, base, key, [] {}, s);
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[t][i] = __builtin_amdgcn_exp2f(s[t][i]);
    static_for<kGroups>([&](auto g) {
        u32x4 pf[RT];
        float largest[RT], unit[RT], of_group = row_lane<g.value>(w.by);
        bool many = false;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            largest[t] = 0x1p-100f;
            static_for<2>([&](auto half) {
                float x[4];
                weigh<kGroups>(g, vgrid[half.value], s[t] + 4 * half.value, x);
                largest[t] = larger3(larger3(largest[t], x[0], x[1]), x[2], x[3]);
            });
            largest[t] = fmaxf(largest[t], __shfl_xor(largest[t], 16));
            largest[t] = fmaxf(largest[t], __shfl_xor(largest[t], 32));
            many = many || largest[t] * of_group >= kMostUnits;
        }
        if (__any(many)) {
            const float f = kLeastBy / of_group;
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int jj = 0; jj < G / 16; ++jj) w.o[t][g.value * (G / 16) + jj] *= f;
            of_group = kLeastBy;
            if ((threadIdx.x & 15) % kGroups == g.value) w.by = kLeastBy;
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            float size = 0.f;
#pragma unroll
            for (int jj = 0; jj < G / 16; ++jj)
#pragma unroll
                for (int r = 0; r < 4; ++r) size = fmaxf(size, fabsf(w.o[t][g.value * (G / 16) + jj][r]));
            size = fmaxf(size, __shfl_xor(size, 16));
            size = fmaxf(size, __shfl_xor(size, 32));
            size = fmaxf(fmaxf(largest[t] * of_group * 0x1p-14f, size * 0x1p-100f), 0x1p-125f);
            unit[t] = __uint_as_float(__float_as_uint(size) & 0x7f800000u);
            const float to = of_group / unit[t], into = 1.f / unit[t];
#pragma unroll
            for (int jj = 0; jj < G / 16; ++jj) w.o[t][g.value * (G / 16) + jj] *= into;
            static_for<2>([&](auto half) {
                float x[4];
                weigh<kGroups>(g, vgrid[half.value], s[t] + 4 * half.value, x);
                pf[t][2 * half.value] = round_pair(x[0] * to, x[1] * to);
                pf[t][2 * half.value + 1] = round_pair(x[2] * to, x[3] * to);
            });
        }
#pragma unroll
        for (int jj = 0; jj < G / 16; ++jj) {
            const int j = g.value * (G / 16) + jj;
            const u32x4 vf = value(j);
#pragma unroll
            for (int t = 0; t < RT; ++t) w.o[t][j] = mfma32<false>(vf, pf[t], w.o[t][j]);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int jj = 0; jj < G / 16; ++jj) w.o[t][g.value * (G / 16) + jj] *= unit[t];
    });
}

// {step * by, base + middle * step} of a grid.
template <typename T>
__device__ __forceinline__ f32x2 open_grid(uint32_t x, float by, float middle)
{
    const float step = to_f32<T>(x & 0xffffu);
    return f32x2{step * by, fmaf(step, middle, to_f32<T>(x >> 16))};
}
template <typename T>
__device__ __forceinline__ f32x2 open_key_grid(uint32_t x, float scale) { return open_grid<T>(x, scale, 0.f); }
template <typename T, int NB>
__device__ __forceinline__ f32x2 open_value_grid(uint32_t x) { return open_grid<T>(x, 1.f, NB == 4 ? 8.f : 128.f); }

constexpr int part_dims(int dim) { return dim < 128 ? dim : 128; }      // joined over the waves at a time
constexpr int kPartPad = 4;

// Joins what TW waves found for the same rows, each on its own tokens, on the largest of their
// maxima, and writes it: waves TW * r .. TW * r + TW - 1 have rows 16 * RT * r .. of the item.
// ml: [WAVES][16 * RT][2]; part: [WAVES][16][part_dims + kPartPad]. Blocks come and leave in
// step.
template <typename T, int D, int G, int RT, int TW, int WAVES, bool BASE_FRAGS>
__device__ __forceinline__ void finish(Wave<D, G, RT, BASE_FRAGS> &w, const AttnArgs &a, const AttnSide &d, const Item &x, int h, int run,
                                       float *ml, float *part)
{
    constexpr int kGroups = D / G, kPart = part_dims(D), kStride = kPart + kPartPad;
    constexpr int kRowWaves = WAVES / TW, kRows = 16 * RT * kRowWaves;
    int thread = threadIdx.x;
    asm volatile("" : "+v"(thread));        // its places are made here, not kept through the steps
    const int lane = thread & 63, col = lane & 15, quad = lane >> 4, wave = thread >> 6;
    const float unit = w.by > 0.f ? 1.f / w.by : 0.f;
    float units[kGroups];
    static_for<kGroups>([&](auto g) { units[g.value] = row_lane<g.value>(unit); });
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        w.l[t] = column_sum(w.l[t]);
        if (quad == 0) {
            ml[(wave * 16 * RT + 16 * t + col) * 2] = w.above[t] < 0.f ? -INFINITY : w.m[t];
            ml[(wave * 16 * RT + 16 * t + col) * 2 + 1] = w.l[t];
        }
#pragma unroll
        for (int g = 0; g < kGroups; ++g) w.bsum[t][g] = column_sum(w.bsum[t][g]);
    }
    const bool whole = x.count == x.along;
    const int slot = 2 * run + (x.u_in > 0 ? 0 : 1);
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += kPart) {
            // a lane has runs of G/16 neighbouring dimensions of its column
#pragma unroll
            for (int g = d0 / G; g < (d0 + kPart) / G; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int jj = 0; jj < G / 16; ++jj)
                        part[(wave * 16 + col) * kStride + g * G - d0 + (4 * quad + i) * (G / 16) + jj] =
                            fmaf(w.o[t][g * (G / 16) + jj][i], units[g], w.bsum[t][g]);
            __syncthreads();
            for (int y = thread; y < kRowWaves * 16 * kPart / 4; y += 64 * WAVES) {
                const int r = y / (kPart / 4) % 16, first = y / (kPart / 4) / 16 * TW, e0 = d0 + y % (kPart / 4) * 4;
                const int in_item = first / TW * 16 * RT + 16 * t + r, row = x.row0 + in_item;
                if (row >= x.n_rows) break;
                float mk[TW], top = -INFINITY, all = 0.f;
#pragma unroll
                for (int k = 0; k < TW; ++k) {
                    mk[k] = ml[((first + k) * 16 * RT + 16 * t + r) * 2];
                    top = fmaxf(top, mk[k]);
                }
                f32x4 sum = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < TW; ++k) {
                    if (mk[k] == -INFINITY) continue;
                    const float f = TW == 1 ? 1.f : __builtin_amdgcn_exp2f(mk[k] - top);
                    all = fmaf(f, ml[((first + k) * 16 * RT + 16 * t + r) * 2 + 1], all);
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(part + ((first + k) * 16 + r) * kStride + e0 - d0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[e] = fmaf(f, v[e], sum[e]);
                }
                float *to_o, *to_ml;
                int64_t at;
                if (!whole) {
                    at = ((int64_t)h * 2 * d.workers + slot) * kRows + in_item;
                    to_o = d.slot_o;
                    to_ml = d.slot_ml;
                } else {
                    at = (int64_t)h * d.s.n_tokens * a.per + (int64_t)x.rows.begin * a.per + row;
                    to_o = d.row_o;
                    to_ml = d.row_ml;
                }
                if (to_o) {
                    *reinterpret_cast<f32x4 *>(to_o + at * D + e0) = sum;
                    if (e0 == 0) *reinterpret_cast<f32x2 *>(to_ml + at * 2) = f32x2{top, all};
                    continue;
                }
                const float inv = all > 0.f ? 1.f / all : 0.f;
                const int tok = x.rows.begin + row / a.per, hq = h * a.per + row % a.per;
                const uint2 packed = {from_f32<T>(sum[0] * inv) | from_f32<T>(sum[1] * inv) << 16,
                                      from_f32<T>(sum[2] * inv) | from_f32<T>(sum[3] * inv) << 16};
                *reinterpret_cast<uint2 *>(a.out + tok * a.o_ts + hq * a.o_hs + e0) = packed;
                if (a.lse && e0 == 0)
                    a.lse[(int64_t)tok * a.c.heads * a.per + hq] =
                        all > 0.f ? (top + log2f(all)) * 0.6931471805599453f : -INFINITY;
            }
            __syncthreads();
        }
}

// Where the codes and grids of 16 tokens lie, and a lane's parts of them.
template <int NB, int D, int G>
struct Spot {
    static constexpr int kRow = D * NB / 8;         // bytes of a token's codes
    static constexpr int kKeyBytes = kRow / 4;      // a lane's quarter of a token's key
    static constexpr int kValBytes = kRow / 16;     // a row of a token's value
    static constexpr int kGrids = Places<D, G>::kGrids, kRegs = Places<D, G>::kRegs;
    unsigned key_at, val_at, grid_at;
    __device__ __forceinline__ Spot()
    {
        const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
        key_at = col * kRow + quad * kKeyBytes;
        val_at = lane * 4 * kValBytes;
        grid_at = 4 * (quad * kGrids + (col & (kGrids - 1)));
    }
    // The first of the 16 tokens at position t (page `page`, any value) over all pages.
    static __device__ __forceinline__ int64_t first(const AttnArgs &a, const SeqView &s, int h, int page, int t)
    {
        const int64_t slice = (int64_t)max(page, 0) * a.c.heads + h;
        return (slice << s.page_shift) + (t & ((1 << s.page_shift) - 1));
    }
    __device__ __forceinline__ void keys(const AttnArgs &a, int64_t at, uint32_t (&w)[kKeyBytes / 4]) const
    {
        load_words<kKeyBytes>(uniform(a.c.k_codes + at * kRow), key_at, w);
    }
    __device__ __forceinline__ void values(const AttnArgs &a, int64_t at, uint32_t (&w)[kValBytes]) const
    {
        load_words<4 * kValBytes>(uniform(a.c.v_codes + at * kRow), val_at, w);
    }
    __device__ __forceinline__ void grids(const uint32_t *meta, int64_t at, uint32_t (&g)[kRegs]) const
    {
        const Global p = uniform(meta + at * (D / G));
#pragma unroll
        for (int k = 0; k < kRegs; ++k) g[k] = load<uint32_t>(p, grid_at + 64 * k);
    }
};

// Register i (0, 1) of code j's fragment: tokens 2i and 2i + 1 of a lane's four, whose rows of
// values are v.
template <int NB, int D>
__device__ __forceinline__ uint32_t value_reg(const uint32_t *v, int i, int j, const Masks &masks)
{
    constexpr int kBytes = D * NB / 128, kWords = kBytes > 4 ? kBytes / 4 : 1;
    uint32_t x[kWords], y[kWords];
    if constexpr (kBytes >= 4) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            x[k] = v[2 * i * kWords + k];
            y[k] = v[(2 * i + 1) * kWords + k];
        }
    } else {
        x[0] = v[i];
        y[0] = v[i] >> 16;
    }
    return value_pair<NB>(x, y, j, masks);
}

__device__ __forceinline__ Masks make_masks()
{
    Masks m = {0x000f000fu, 0x00f000f0u};
    asm volatile("" : "+v"(m.low), "+v"(m.high));
    return m;
}

// The side of the call that the block works on, its head and run.
struct Place {
    AttnSide d;
    int h, run;
    bool first;                 // of the side's blocks
};
__device__ __forceinline__ Place place_of(const AttnArgs &a)
{
    const unsigned blocks0 = (unsigned)a.side[0].workers * a.c.heads;
    const bool second = blockIdx.x >= blocks0;
    const unsigned block = second ? blockIdx.x - blocks0 : blockIdx.x;
    const unsigned run = block / (unsigned)a.c.heads;
    return Place{second ? a.side[1] : a.side[0], (int)(block - run * a.c.heads), (int)run, block == 0};
}

// ---- few rows, or little work: the cache is read, and little else ---------------------------
// Each wave takes 32 tokens of every 128 for all of the tile's rows, straight from memory into
// its products: no barrier but at an item's end, and a step of a third of the latency of the form
// below, which is why it takes many rows too while there is little work for each block. Codes and grids are read once and in whole lines;
// a step's 400 instructions to widen and weigh them take about as long as its bytes (4 bits,
// heads of 128), which is why grids are applied to sums and not to codes. 64 sequences of 4100 to
// 8190 tokens, 8 heads of 128, 4 bits, 455 MB: 98 us, 4.6 TB/s (a copy reaches 5.1); 131071 tokens
// of 8 bits, 277 MB: 45 us, 6.2 TB/s; 300 tokens of 32 heads: 9.8 us, four loads that wait for
// each other (lengths, pages, codes, and the instructions themselves) and three steps one after
// another.
template <typename T, int NB, int D, int G, int RT>
__global__ __launch_bounds__(64 * kWaves, blocks_per_cu(RT, D, NB) * kWaves / 4) void attn_kernel(AttnArgs a)       // waves to a SIMD
{
    constexpr int kRows = 16 * RT;
    extern __shared__ int32_t shared[];
    const Place place = place_of(a);
    const AttnSide &d = place.d;
    const int h = place.h;
    int32_t *starts = shared;                                       // [n_seqs + 1]
    int32_t *scan = shared + (((unsigned)d.s.n_seqs + 4) & ~3u);    // [8]
    float *ml = reinterpret_cast<float *>(scan + 8);
    float *part = ml + kWaves * kRows * 2;
    const Layout<kRows, kWaves> layout(d, a.per, starts, scan);
    if (place.first && d.starts) layout.put(d.starts);
    const int W = runs_of(d.workers, layout.total);
    if (place.run >= W) return;
    const int u_end = first_unit(place.run + 1, W, layout.total);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Spot<NB, D, G> spot;
    const Masks masks = make_masks();

    for (int u = first_unit(place.run, W, layout.total); u < u_end;) {
        const Item x = layout.item(u, u_end);
        u += x.count;
        Wave<D, G, RT, false> w;
        // what the last of the item's rows sees
        const int last = (int)((unsigned)(min(x.row0 + kRows, x.n_rows) - 1) / (unsigned)a.per);
        const int seen = d.causal ? x.len - (x.rows.end - x.rows.begin) + last + 1 : x.len;
        const int t_end = (int)min((int64_t)(x.u_in + x.count) * layout.unit, (int64_t)seen);
        const int32_t *table = d.s.table + (int64_t)x.b * d.s.max_pages;
        uint32_t kw[2][Spot<NB, D, G>::kKeyBytes / 4], vw[2][Spot<NB, D, G>::kValBytes];
        uint32_t kg[2][Places<D, G>::kRegs], vg[2][Places<D, G>::kRegs];
        int page[2];
        auto find = [&](int t0, int (&page)[2]) {
#pragma unroll
            for (int half = 0; half < 2; ++half) page[half] = page_at(d.s, table, min(t0 + 16 * half, x.len - 1));
        };
        auto load_keys = [&](int t0) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int64_t at = spot.first(a, d.s, h, page[half], t0 + 16 * half);
                spot.keys(a, at, kw[half]);
                spot.grids(a.c.k_meta, at, kg[half]);
            }
        };
        auto load_values = [&](int t0) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int64_t at = spot.first(a, d.s, h, page[half], t0 + 16 * half);
                spot.values(a, at, vw[half]);
                spot.grids(a.c.v_meta, at, vg[half]);
            }
        };
        const auto close = [&](const int (&good)[2]) {
            asm volatile("");
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int k = 0; k < Places<D, G>::kRegs; ++k)
                    if (Places<D, G>::token(k) >= good[half]) kg[half][k] = vg[half][k] = 0;
        };
        const auto key_grid = [&](int half, int k) { return open_key_grid<T>(kg[half][k], a.scale); };
        const auto no_base = [](int, int) { return u32x4{}; };
        const auto key = [&](int half, int mm) { return key_frag<Types<T>::kBf16, NB>(kw[half] + mm * (NB / 4)); };
        const auto value_grid = [&](int half, int k) { return open_value_grid<T, NB>(vg[half][k]); };
        const auto value = [&](int j) {
            u32x4 f;
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = value_reg<NB, D>(vw[i / 2], i % 2, j, masks);
            return f;
        };
        const int t_begin = (int)min((int64_t)x.u_in * layout.unit + wave * kTile, (int64_t)t_end);
        int t0 = t_begin;
        if (t0 < t_end) {
            find(t0, page);
            load_keys(t0);
            load_values(t0);
        }
        begin<T>(w, a, d.causal, x, h, x.row0);     // the queries, while the first codes are on their way
        for (; t0 < t_end; t0 += kStep) {
            // The next step's keys are asked for as soon as this one's are in the products,
            // its values once this one's are: both are under way during half a step, with no
            // registers but their own.
            const int next = t0 + kStep < t_end ? t0 + kStep : t0;
            int page_next[2], good[2];
            find(next, page_next);
#pragma unroll
            for (int half = 0; half < 2; ++half) good[half] = page[half] < 0 ? 0 : x.len - t0 - 16 * half;
            attend_step<T>(
                w, t0, good, [&] { close(good); }, key_grid, no_base, key,
                [&] {
                    page[0] = __builtin_amdgcn_readfirstlane(page_next[0]);
                    page[1] = __builtin_amdgcn_readfirstlane(page_next[1]);
                    load_keys(next);
                    __builtin_amdgcn_sched_barrier(0);
                },
                value_grid, value);
            load_values(next);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (__builtin_expect(w.rest, 0)) {
            float by = 0.f;
            for (t0 = t_begin; t0 < t_end; t0 += kStep) {
                int good[2];
                find(t0, page);
                load_keys(t0);
                load_values(t0);
#pragma unroll
                for (int half = 0; half < 2; ++half) good[half] = page[half] < 0 ? 0 : x.len - t0 - 16 * half;
                attend_rest<T>(w, by, t0, good, [&] { close(good); }, key_grid, no_base, key, value_grid, value);
            }
        }
        finish<T, D, G, RT, kWaves, kWaves>(w, a, d, x, h, place.run, ml, part);
    }
}

// ---- many rows over much: the arithmetic bounds it -------------------------------------------
// TW waves share each 16 rows and take turns at tiles of 32 tokens; all waves of the block meet
// the same 64 tokens a step. Together they widen the step's codes into fragments and open its
// grids, in LDS: that is paid once for the block's rows. Where LDS has room for two steps
// (heads of up to 128), the next step's are made in the other half, so that one barrier a step
// is enough; the codes of the step after that are on their way meanwhile. Eight waves of 16
// rows rather than four of 32: four waves to a SIMD hide each other's waits better than two
// that share a broadcast grid between twice the rows (84 and 87 us for the second case below).
//
// It is bound by the instructions beside the products: a wave's step of 16 rows and 32 tokens of
// heads of 128 in two groups has 18 products of 16 cycles and about 115 vector instructions of 4
// (grids, exponentials, the rounding of weights), and its share of the widening 40 more. 2 x 500
// rows over 3500 to 4000 tokens, 40 heads of 128, 4 bits: 177 us, 405 TFLOP/s; 64 x 8 rows a head
// over 16390 tokens, 8 heads: 81 us, 422 TFLOP/s, of them 16 before the first product and behind
// the last, for 33 MB of pieces. Counters of the latter: vector instructions 67% of the time, LDS
// 38%, products 23%; a wave waits 41% of its time for loads and for the block's other waves.
constexpr int kWideStep = 64, kWideTiles = kWideStep / 16;

template <int D, int G>
struct WideStep {
    u32x4 key[kWideTiles][D / 32][64];          // A fragments
    u32x4 value[kWideTiles / 2][D / 16][64];
    float key_step[kWideTiles][Places<D, G>::kRegs][64];
    uint16_t key_base[kWideTiles][2][16][D / G > 2 ? D / G : 2];    // first and second parts, of 16 tokens
    f32x2 value_grid[kWideTiles][Places<D, G>::kRegs][64];
    int good[kWideTiles];
};      // a multiple of 16 bytes
template <int D>
constexpr int wide_buffers() { return D <= 128 ? 2 : 1; }
template <int D>
constexpr int wide_waves() { return D <= 128 ? 8 : 4; }
template <int D, int G>
constexpr size_t wide_bytes()       // of the steps, or of what joins the waves in their place
{
    const size_t steps = wide_buffers<D>() * sizeof(WideStep<D, G>);
    const size_t part = 4 * (size_t)wide_waves<D>() * 16 * (part_dims(D) + kPartPad);
    return ((steps > part ? steps : part) + 15) & ~size_t(15);
}

template <typename T, int NB, int D, int G, int TW>
__global__ __launch_bounds__(64 * wide_waves<D>(), blocks_per_cu(wide_waves<D>() / TW, D, NB) * wide_waves<D>() / 4) void attn_wide_kernel(AttnArgs a)
{
    constexpr int kWide = wide_waves<D>(), kRows = 16 * (kWide / TW), kTurns = 2 / TW, kBuffers = wide_buffers<D>();
    constexpr int kRegs = Places<D, G>::kRegs, kParts = kWide / kWideTiles;
    static_assert(kParts == 1 || kParts == 2, "a wave widens 16 tokens, or half their dimensions");
    extern __shared__ u32x4 shared4[];
    const Place place = place_of(a);
    const AttnSide &d = place.d;
    const int h = place.h;
    WideStep<D, G> *steps = reinterpret_cast<WideStep<D, G> *>(shared4);
    float *part = reinterpret_cast<float *>(shared4);
    float *ml = reinterpret_cast<float *>(shared4 + wide_bytes<D, G>() / 16);
    int32_t *starts = reinterpret_cast<int32_t *>(ml + kWide * 16 * 2);
    int32_t *scan = starts + (((unsigned)d.s.n_seqs + 4) & ~3u);
    int32_t *rest = scan + 8;                   // some wave's
    Layout<kRows, kWide> layout(d, a.per, starts, scan);
    if (place.first && d.starts) layout.put(d.starts);
    const int W = runs_of(d.workers, layout.total);
    if (place.run >= W) return;
    const int u_end = first_unit(place.run + 1, W, layout.total);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int sub = wave % kWideTiles, piece = wave / kWideTiles;       // what this wave widens
    const Spot<NB, D, G> spot;
    const Masks masks = make_masks();

    for (int u = first_unit(place.run, W, layout.total); u < u_end; layout.again()) {
        const Item x = layout.item(u, u_end);
        u += x.count;
        Wave<D, G, 1, true> w;
        // what the block's rows see: the same for its waves, which go in step
        const int last = (int)((unsigned)(min(x.row0 + kRows, x.n_rows) - 1) / (unsigned)a.per);
        const int seen = d.causal ? x.len - (x.rows.end - x.rows.begin) + last + 1 : x.len;
        const int t_end = (int)min((int64_t)(x.u_in + x.count) * layout.unit, (int64_t)seen);
        const int32_t *table = d.s.table + (int64_t)x.b * d.s.max_pages;
        uint32_t kw[Spot<NB, D, G>::kKeyBytes / 4 / kParts], vw[Spot<NB, D, G>::kValBytes], kg[kRegs], vg[kRegs];
        int good;
        // this wave's 16 tokens of a step, at positions from t
        auto page_of_step = [&](int t0) { return page_at(d.s, table, min(t0 + 16 * sub, x.len - 1)); };
        auto fetch = [&](int t, int page) {
            const int64_t at = spot.first(a, d.s, h, page, t);
            load_words<Spot<NB, D, G>::kKeyBytes / kParts>(uniform(a.c.k_codes + at * spot.kRow),
                                                           spot.key_at + piece * (spot.kKeyBytes / kParts), kw);
            spot.values(a, at, vw);
            spot.grids(a.c.k_meta, at, kg);
            spot.grids(a.c.v_meta, at, vg);
            good = page < 0 ? 0 : x.len - t;
        };
        auto widen = [&](WideStep<D, G> &to) {
#pragma unroll
            for (int mm = 0; mm < D / 32 / kParts; ++mm)
                to.key[sub][piece * (D / 32 / kParts) + mm][lane] = key_frag<Types<T>::kBf16, NB>(kw + mm * (NB / 4));
            static_for<kParts>([&](auto p) {
                if (piece != p.value) return;
#pragma unroll
                for (int j = p.value * (D / 16 / kParts); j < (p.value + 1) * (D / 16 / kParts); ++j) {
                    const u32x2 f = {value_reg<NB, D>(vw, 0, j, masks), value_reg<NB, D>(vw, 1, j, masks)};
                    reinterpret_cast<u32x2 *>(&to.value[sub / 2][j][lane])[sub % 2] = f;
                }
            });
#pragma unroll
            for (int k = 0; k < kRegs; ++k) {
                const bool in = Places<D, G>::token(k) < good;
                if (piece == 0) {
                    const f32x2 grid = open_key_grid<T>(in ? kg[k] : 0u, a.scale);
                    to.key_step[sub][k][lane] = grid[0];
                    // the places of a register, once each
                    const int group = ((lane & 15) + 16 * k) % (D / G);
                    if ((lane & 15) < Places<D, G>::kGrids) {
                        const uint32_t first = from_f32<Bf16>(grid[1]);
                        to.key_base[sub][0][Places<D, G>::token(k)][group] = (uint16_t)first;
                        to.key_base[sub][1][Places<D, G>::token(k)][group] =
                            (uint16_t)from_f32<Bf16>(grid[1] - to_f32<Bf16>(first));
                    }
                }
                if (piece == kParts - 1) to.value_grid[sub][k][lane] = open_value_grid<T, NB>(in ? vg[k] : 0u);
            }
            if (lane == 0 && piece == 0) to.good[sub] = good;
        };
        // the wave's pairs of 16 tokens of a step, to do(t, good, ...) with what attend_step takes of them
        const auto turns = [&](const WideStep<D, G> &now, int t0, auto attend) {
#pragma unroll 1
            for (int turn = 0; turn < kTurns; ++turn) {
                const int pair = wave % TW + turn, t = t0 + 32 * pair;
                if (t >= min(w.lim_high, t_end)) continue;
                const int both[2] = {__builtin_amdgcn_readfirstlane(now.good[2 * pair]),
                                     __builtin_amdgcn_readfirstlane(now.good[2 * pair + 1])};
                attend(
                    t, both, [&](int half, int k) { return f32x2{now.key_step[2 * pair + half][k][lane], 0.f}; },
                    [&](int half, int p) {
                        // the same in the slots of the parts behind, which meet zeros but in quad 3
                        constexpr int kWords = base_slots<D / G>() / 2;
                        const uint16_t *b = now.key_base[2 * pair + half][lane >= 48][lane & 15] + 2 * kWords * p;
                        u32x4 f = {0, 0, 0, 0};
#pragma unroll
                        for (int e = 0; e < kWords; ++e) f[e] = f[e + kWords] = reinterpret_cast<const uint32_t *>(b)[e];
                        if (D / G == 1) f[0] = f[1] = f[0] & 0xffffu;       // the other half is not written
                        return f;
                    },
                    [&](int half, int mm) { return now.key[2 * pair + half][mm][lane]; }, [] {},
                    [&](int half, int k) { return now.value_grid[2 * pair + half][k][lane]; },
                    [&](int j) { return now.value[pair][j][lane]; });
            }
        };
        const int t_begin = (int)min((int64_t)x.u_in * layout.unit, (int64_t)t_end);
        int t0 = t_begin, page = 0, buffer = 0;
        if (threadIdx.x == 0) *rest = 0;        // before the first barrier, and behind the last item's last
        // a step that there is not is fetched like the last one, and not used
        auto within = [&](int t) { return t < t_end ? t : t0; };
        if (t0 < t_end) fetch(t0 + 16 * sub, __builtin_amdgcn_readfirstlane(page_of_step(t0)));
        begin<T>(w, a, d.causal, x, h, x.row0 + wave / TW * 16);        // while the first codes are on their way
        if (t0 < t_end) {
            if constexpr (kBuffers == 2) {
                widen(steps[0]);
                const int next = within(t0 + kWideStep);
                fetch(next + 16 * sub, __builtin_amdgcn_readfirstlane(page_of_step(next)));
                page = page_of_step(within(t0 + 2 * kWideStep));
            } else {
                page = page_of_step(within(t0 + kWideStep));
            }
        }
        for (; t0 < t_end; t0 += kWideStep) {
            __syncthreads();        // the last step's products have been made, this one's widened (two buffers)
            constexpr int kAhead = kBuffers;
            if constexpr (kBuffers == 2) {
                widen(steps[buffer ^ 1]);
            } else {
                widen(steps[0]);
                __syncthreads();
            }
            const int next = within(t0 + kAhead * kWideStep);
            fetch(next + 16 * sub, __builtin_amdgcn_readfirstlane(page));
            page = page_of_step(within(t0 + (kAhead + 1) * kWideStep));
            __builtin_amdgcn_sched_barrier(0);
            turns(steps[buffer], t0, [&](int t, const int (&good)[2], auto... parts) { attend_step<T>(w, t, good, [] {}, parts...); });
            if constexpr (kBuffers == 2) buffer ^= 1;
        }
        if (lane == 0 && w.rest) *rest = 1;
        __syncthreads();                        // `part` lies over the steps
        if (__builtin_expect(__builtin_amdgcn_readfirstlane(*rest), 0)) {
            float by = 0.f;
            for (t0 = t_begin; t0 < t_end; t0 += kWideStep) {
                __syncthreads();
                fetch(t0 + 16 * sub, __builtin_amdgcn_readfirstlane(page_of_step(t0)));
                widen(steps[0]);
                __syncthreads();
                turns(steps[0], t0, [&](int t, const int (&good)[2], auto key_grid, auto base, auto key, auto, auto value_grid, auto value) {
                    attend_rest<T>(w, by, t, good, [] {}, key_grid, base, key, value_grid, value);
                });
            }
            __syncthreads();
        }
        finish<T, D, G, 1, TW, kWide>(w, a, d, x, h, place.run, ml, part);
    }
}

// Bytes of LDS beside what the waves work in: the units before each sequence's and their scan,
// at most 16 KB, and a flag.
inline size_t starts_bytes(const AttnArgs &a)
{
    const int n = a.sides == 2 ? max(a.side[0].s.n_seqs, a.side[1].s.n_seqs) : a.side[0].s.n_seqs;
    return 4 * (((size_t)n + 4) & ~size_t(3)) + 4 * 8 + 16;
}
inline dim3 grid_of(const AttnArgs &a)
{
    const int64_t runs = a.side[0].workers + (a.sides == 2 ? a.side[1].workers : 0);
    return dim3((unsigned)(runs * a.c.heads));
}

template <typename T, int NB, int D, int G, int RT>
hipError_t launch_few(const AttnArgs &a, hipStream_t stream)
{
    const size_t lds = starts_bytes(a) + 4 * kWaves * 16 * RT * 2 + 4 * (size_t)kWaves * 16 * (part_dims(D) + kPartPad);
    attn_kernel<T, NB, D, G, RT><<<grid_of(a), 64 * kWaves, lds, stream>>>(a);
    return hipGetLastError();
}

template <typename T, int NB, int D, int G, int TW>
hipError_t launch_many(const AttnArgs &a, hipStream_t stream)
{
    const int waves = wide_waves<D>();
    const size_t lds = wide_bytes<D, G>() + 4 * waves * 16 * 2 + starts_bytes(a);
    attn_wide_kernel<T, NB, D, G, TW><<<grid_of(a), 64 * waves, lds, stream>>>(a);
    return hipGetLastError();
}

template <typename T, int NB, int D, int G>
hipError_t by_tiles(const AttnArgs &a, hipStream_t stream)
{
    // rows to a tile: 16, 32 or 128, and 16, 32 or 64 of 256-wide heads (whose sums fill the registers)
    const int n = a.side[0].tiles16;
    if (n == 1) return launch_few<T, NB, D, G, 1>(a, stream);
    if constexpr (D <= 128) {
        if (n == 2) return launch_few<T, NB, D, G, 2>(a, stream);
        if (n == 8) return launch_many<T, NB, D, G, 1>(a, stream);
    } else {
        if (n == 2) return launch_many<T, NB, D, G, 2>(a, stream);
        if (n == 4) return launch_many<T, NB, D, G, 1>(a, stream);
    }
    return hipErrorInvalidValue;
}

template <typename T, int NB, int D>
hipError_t by_group(const AttnArgs &a, int g, hipStream_t stream)
{
    if (g == 32) return by_tiles<T, NB, D, 32>(a, stream);
    if (g == 64) return by_tiles<T, NB, D, 64>(a, stream);
    if constexpr (D >= 128)
        if (g == 128) return by_tiles<T, NB, D, 128>(a, stream);
    return hipErrorInvalidValue;
}

template <typename T, int NB>
hipError_t by_dim(const AttnArgs &a, const AttnShape &x, hipStream_t stream)
{
    if (x.dim == 64) return by_group<T, NB, 64>(a, x.g, stream);
    if (x.dim == 128) return by_group<T, NB, 128>(a, x.g, stream);
    return by_group<T, NB, 256>(a, x.g, stream);
}

}  // namespace
}  // namespace hqq
