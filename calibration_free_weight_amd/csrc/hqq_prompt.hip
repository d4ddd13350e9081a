// hqq_prompt.hip -- causal attention of packed prompts over themselves on the matrix cores
// (gfx950): the kernel, its checks and its launch.
//
// A block of four waves has 128 query rows of one sequence and key/value head, a row being a token
// and one of the query heads that share the head, and goes along the sequence in tiles of keys that
// its waves share in LDS. With C = A . B on 32x32x16 tiles (lane l: A row l%32, B column l%32, eight
// values of the contraction from 8*(l/32); C column l%32, rows 8*(i/4) + 4*(l/32) + i%4),
//   S^T = K . Q^T      A = keys, B = the wave's 32 query rows: a lane has scores of its own row;
//   O^T = V^T . P^T    B = weights: the scores that the lane has, the order of the contraction being
//                      free; A = values, transposed on their way out of LDS;
// so that weights stay in registers, and maxima and sums are per lane, joined over the two lanes of
// a row. A step makes the next keys' scores while the weights of the present ones are computed, and
// then meets the values: the vector instructions of a softmax (3 and an exponential for each weight)
// take about as long as its matrix instructions and run beside them. Keys and values of the steps to
// come are in registers and in the other half of LDS meanwhile, one barrier to a step.
#include <cmath>

#include "hqq.h"
#include "hqq_cache_internal.h"
#include "hqq_internal.h"

namespace hqq {
namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(4))) short s16x4;

constexpr int kAhead = 2;         // fragments asked for before they are used
constexpr int64_t kMaxKeyStride = 1 << 22;
constexpr float kLog2e = 1.44269504088896341f;
// How far a score (to base 2) may lie above a row's maximum before what is taken off all scores moves,
// and how far below the maximum that then lies. A binary16 weight has 24 powers of two below 1 and 15
// above: from 2^7 for the largest weight, 2^15 with the slack, to 2^-25, where one is lost from the
// products that the sum counts, there are 32; from 1 there would be 25, and a long prompt's many small
// weights beside a large one went short by up to 2^-25 each. A bfloat16 weight has binary32's exponents.
constexpr float kSlack = 8.f;
template <typename T>
constexpr float kBelow = Types<T>::kBf16 ? 0.f : 7.f;

struct PromptArgs {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    float *lse;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;
    SeqView s;                  // cu, n_seqs, n_tokens
    int32_t heads, per;         // key/value heads, query heads to one
    uint64_t inv;               // 2^64 / per, rounded up; 0 with one
    float scale;                // |scale| times log2(e), or 1 where scale is 0
    uint32_t flip, keep;        // of two queries: bits that change, bits that stay
};

// row / per, of rows below 2^30 and up to 2^20 heads: what inv is too large by adds less than 2^-34.
__device__ __forceinline__ int token_of(const PromptArgs &a, int row)
{
    if (a.inv == 0) return row;
    const uint64_t high = (uint64_t)(uint32_t)row * (uint32_t)(a.inv >> 32);
    return (int)((high + __umulhi((uint32_t)row, (uint32_t)a.inv)) >> 32);
}

template <typename T>
__device__ __forceinline__ f32x16 mfma(const u32x4 a, const u32x4 b, const f32x16 c)
{
    if constexpr (Types<T>::kBf16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <typename T>
__device__ __forceinline__ uint32_t round2(float a, float b)
{
    const f32x2 x = {a, b};
    if constexpr (Types<T>::kBf16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, f16x2));
}

// NaN if one is: one instruction for two of these, where fmaxf takes two more that quiet NaN.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// x of both lanes of a row, which are 32 apart.
template <typename F>
__device__ __forceinline__ float of_row(float x, F f)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Four keys' values of a dimension each, from four rows of 16 dimensions in LDS: lane 4r + c of 16
// lanes names row r's dimensions 4c..4c+3, and gets all rows' dimension 4r + c.
__device__ __forceinline__ u32x2 read_transposed(const void *p)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p));
}

// The first n rows from p (uniform), of `dim` numbers each and `ts` apart, no more than `most`, as a
// buffer: what is read behind them is 0. (Up to 256 rows' offsets stay below 2^31.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_from(const uint16_t *p, int n, int most, int ts, int dim)
{
    const uint64_t at = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at), hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
    const int bytes = ((min(n, most) - 1) * ts + dim) * 2 & -n >> 31;      // 0 without rows, and no branch
    return __builtin_amdgcn_make_buffer_rsrc((void *)((uint64_t)hi << 32 | lo), 0, __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
// The whole offset is the lanes', which is the one that the buffer's end is held against.
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, int offset)
{
    return __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0);
}

// Whether one of two numbers is an infinity or NaN; the two with such replaced by 0.
template <typename T>
__device__ __forceinline__ bool finite2(uint32_t &w)
{
    constexpr uint32_t kExp = Types<T>::kBf16 ? 0x7f80u : 0x7c00u;
    const bool lo = (w & kExp) == kExp, hi = (w >> 16 & kExp) == kExp;
    if (lo) w &= 0xffff0000u;
    if (hi) w &= 0x0000ffffu;
    return !(lo || hi);
}

// The block's rows: of sequence rows `seq`, from row0, of n_rows.
struct Tile {
    Rows seq;
    int row0, n_rows;
};

// Sums of what the lanes of a wave, or with ALL the threads of the block have.
template <int WAVES, bool ALL>
__device__ __forceinline__ int sum_of(int x, int32_t (&scan)[2][WAVES], int &turn)
{
    x = __builtin_amdgcn_readlane(wave_sum(x), 63);
    if constexpr (ALL) {
        if ((threadIdx.x & 63) == 0) scan[turn][threadIdx.x >> 6] = x;
        __syncthreads();
        x = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) x += scan[turn][w];
        turn ^= 1;              // who is late still reads the other
    }
    return __builtin_amdgcn_readfirstlane(x);
}

// The u-th of all sequences' tiles, or none. The longest come first, those that lie furthest back in
// their sequences, for the last ones to begin to be short: behind them nothing fills the GPU. With f(k)
// tiles at place k or behind, it is at the last place where f(k) > u, which a search finds; there, the
// (u - f(k + 1))-th of the sequences that reach so far. Up to 64 sequences lie in a wave's lanes, and
// no wave waits for another.
template <int WAVES, int ROWS, bool ALL>
__device__ __forceinline__ bool find_tile(const SeqView &s, int per, int u, int32_t (&scan)[2][WAVES], int32_t (&found)[2], Tile &x)
{
    const int t = ALL ? threadIdx.x : threadIdx.x & 63, threads = ALL ? 64 * WAVES : 64;
    const int each = ALL ? (s.n_seqs + threads - 1) / threads : 1;
    const int b0 = min(t * each, s.n_seqs), b1 = min(b0 + each, s.n_seqs);
    int turn = 0;
    const auto tiles = [&](int b) {
        const Rows r = rows_of(s, b);
        return tiles_of((r.end - r.begin) * per, ROWS);
    };
    int most = 0;
    bool falls = false;
    const int own = b0 < b1 ? tiles(b0) : 0;                // with one sequence to a lane, its tiles
    for (int b = b0; b < b1; ++b) {
        most = max(most, ALL ? tiles(b) : own);
        falls = falls || falls_at(s, b);
    }
    const auto behind = [&](int k) {                        // f(k)
        int n = 0;
        for (int b = b0; b < b1; ++b) n += max(0, (ALL ? tiles(b) : own) - k);
        return sum_of<WAVES, ALL>(n, scan, turn);
    };
    // offsets that fall would count rows twice
    if (ALL ? __syncthreads_or(falls) : __any(falls)) return false;
    const int total = behind(0);
    if (u >= total) return false;
    int k = total - 1 - u, b = 0;                           // of a single sequence, from its end
    if (s.n_seqs > 1) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) most = max(most, __shfl_xor(most, d));
        if constexpr (ALL) {
            found[0] = 0;
            __syncthreads();
            if ((threadIdx.x & 63) == 0) atomicMax(&found[0], most);
            __syncthreads();
            most = found[0];
        }
        k = 0;
        for (int hi = __builtin_amdgcn_readfirstlane(most); hi - k > 1;) {      // f(k) > u >= f(hi)
            const int mid = (k + hi) >> 1;
            if (behind(mid) > u) k = mid; else hi = mid;
        }
        int which = u - behind(k + 1);
        if constexpr (ALL) {
            int mine = 0, before = 0;
            for (int c = b0; c < b1; ++c) mine += tiles(c) > k;
            const int upto = wave_sum(mine);
            if ((t & 63) == 63) scan[turn][t >> 6] = upto;
            __syncthreads();
            for (int w = 0; w < t >> 6; ++w) before += scan[turn][w];
            before += upto - mine;
            for (int c = b0; c < b1; ++c)
                if (tiles(c) > k && before++ == which) found[1] = c;
            __syncthreads();
            b = found[1];
        } else {
            uint64_t reach = __ballot(own > k);
            for (; which > 0; --which) reach &= reach - 1;
            b = __builtin_ctzll(reach);
        }
    }
    x.seq = rows_of(s, __builtin_amdgcn_readfirstlane(b));
    x.row0 = k * ROWS;
    x.n_rows = (x.seq.end - x.seq.begin) * per;
    return true;
}

template <int I>
struct Index {
    static constexpr int value = I;
};

template <typename T, int D, int DV, int WAVES, int KB>
__global__ __launch_bounds__(64 * WAVES, 2) void prompt_kernel(PromptArgs a)
{
    constexpr int kThreads = 64 * WAVES, kRows = 32 * WAVES, kKeys = 32 * KB;
    constexpr int kChunks = D / 8;                          // of 16 bytes, in a row of keys or values
    constexpr int kEach = kKeys * kChunks / kThreads;       // chunks of keys to a thread
    constexpr int kApart = kThreads / kChunks;              // rows between a thread's chunks
    constexpr int kVChunks = DV / 8, kVEach = kKeys * kVChunks / kThreads, kVApart = kThreads / kVChunks;
    static_assert(kEach * kThreads == kKeys * kChunks && kVEach * kThreads == kKeys * kVChunks, "whole chunks for each thread");
    __shared__ u32x4 keys[2][kKeys * kChunks], values[2][kKeys * kVChunks];
    __shared__ int32_t scan[2][WAVES], found[2], bad[2];    // bad: the last step whose values were not finite
    Tile x;
    const unsigned parts = a.heads * (D / DV), part = blockIdx.x % parts;
    const int h = (int)(part % (unsigned)a.heads), dv0 = (int)(part / (unsigned)a.heads) * DV;     // of the outputs
    if (threadIdx.x < 2) bad[threadIdx.x] = -1;
    const int u = (int)(blockIdx.x / parts);
    const bool has = a.s.n_seqs <= 64 ? find_tile<WAVES, kRows, false>(a.s, a.per, u, scan, found, x)
                                      : find_tile<WAVES, kRows, true>(a.s, a.per, u, scan, found, x);
    if (!has) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
    const int n = x.seq.end - x.seq.begin;
    const int wave_row = x.row0 + 32 * wave, row = wave_row + col;      // a lane's row, and its token
    const int tok = token_of(a, min(row, x.n_rows - 1)), hq = h * a.per + (row - tok * a.per);
    // tokens of the block's and the wave's first and last rows
    const int first = token_of(a, x.row0), last = min(x.row0 + kRows, x.n_rows) - 1;
    const int wave_first = token_of(a, min(wave_row, x.n_rows - 1));
    const int wave_last = token_of(a, min(wave_row + 31, x.n_rows - 1));
    const int steps = token_of(a, last) / kKeys + 1;            // of keys that some row sees

    // where a thread's chunks come from: rows and places are swapped within LDS so that no two lanes
    // that read at a time meet in a bank. Rows behind the sequence are beyond the buffer, and 0.
    const int r0 = (int)threadIdx.x / kChunks, place = (int)threadIdx.x % kChunks;
    const auto key_swap = [](int r) { return kChunks == 8 ? (r >> 1) & 7 : r & 15; };
    const auto value_swap = [](int r) { return kVChunks == 8 ? ((r >> 1) & 1) << 2 : (r & 3) << 2; };
    const int vr0 = (int)threadIdx.x / kVChunks, vplace = (int)threadIdx.x % kVChunks;
    const int k_ts = (int)a.k_ts, v_ts = (int)a.v_ts;
    const uint16_t *next_k = a.k + x.seq.begin * a.k_ts + h * a.k_hs, *next_v = a.v + x.seq.begin * a.v_ts + h * a.v_hs + dv0;
    int left_k = n, left_v = n;                             // rows from there
    u32x4 kr[kEach], vr[kVEach];
    const auto fetch_keys = [&] {
        const auto k = rows_from(next_k, left_k, kKeys, k_ts, D);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            kr[i] = load16(k, (r0 + i * kApart) * k_ts * 2 + 16 * (place ^ key_swap(r0 + i * kApart)));
        next_k += kKeys * k_ts;
        left_k -= kKeys;
    };
    const auto fetch_values = [&] {
        const auto v = rows_from(next_v, left_v, kKeys, v_ts, DV);
#pragma unroll
        for (int i = 0; i < kVEach; ++i)
            vr[i] = load16(v, (vr0 + i * kVApart) * v_ts * 2 + 16 * (vplace ^ value_swap(vr0 + i * kVApart)));
        next_v += kKeys * v_ts;
        left_v -= kKeys;
    };
    const auto put_keys = [&](int b) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) keys[b][threadIdx.x + i * kThreads] = kr[i];
    };
    const auto put_values = [&](int b) {
#pragma unroll
        for (int i = 0; i < kVEach; ++i) values[b][threadIdx.x + i * kThreads] = vr[i];
    };
    // Of a step that some rows do not see in full: values that are not finite are left out, and noted.
    const auto check_values = [&](int step) {
        if (__builtin_expect((step + 1) * kKeys - 1 <= first, 1)) return;
        bool ok = true;
#pragma unroll
        for (int i = 0; i < kVEach; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t w = vr[i][e];
                ok = finite2<T>(w) && ok;
                vr[i][e] = w;
            }
        if (!ok) bad[step & 1] = step;
    };
    u32x4 qf[D / 16];
    // Fragment d of 32 keys kb in buffer b; of the values, dimensions 32 j.. of keys 16 g..
    const auto key_frag = [&](int b, int kb, int d) { return keys[b][(32 * kb + col) * kChunks + ((2 * d + half) ^ key_swap(col))]; };
    const int vrow = 4 * half + ((lane & 15) >> 2);
    const auto value_frag = [&](int b, int g, int j) {
        const int c = (4 * j + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ value_swap(vrow);
        const char *p = reinterpret_cast<const char *>(&values[b][(16 * g + vrow) * kVChunks + c]) + 8 * (lane & 1);
        const u32x2 lo = read_transposed(p), hi = read_transposed(p + 8 * kVChunks * 16);
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    f32x16 o[DV / 32];
    float m = -INFINITY, l = 0.f;

    // The largest of a row's scores so far, and numbers e and e + 1 of them.
    const auto larger_of = [&](float top, const f32x16 (&s)[KB], int e) {
        const float p = s[e / 16][e % 16], q = s[e / 16][e % 16 + 1];
        return e == 0 ? larger(p, q) : larger(larger(top, p), q);
    };
    // Moves m, kBelow below the largest score, where the scores go beyond that by more than the slack;
    // where some row does not see some key, takes these scores out first.
    const auto look = [&](f32x16 (&s)[KB], float top, int step) {
        if (__builtin_expect((step + 1) * kKeys - 1 > wave_first, 0)) {
            int seen = tok - step * kKeys - 4 * half;
            asm volatile("" : "+v"(seen));                  // a branch, not a choice in every step
#pragma unroll
            for (int e = 0; e < 16 * KB; ++e)
                if (32 * (e / 16) + 8 * (e % 16 / 4) + e % 4 > seen) s[e / 16][e % 16] = -INFINITY;
#pragma unroll
            for (int e = 0; e < 16 * KB; e += 2) top = larger_of(top, s, e);
        }
        top = of_row(top, larger) * a.scale;
        if (__any(top > m + (kSlack + kBelow<T>))) {
            const bool up = top > m + (kSlack + kBelow<T>); // of this row: no other row's scores change it
            const float to = up ? top - kBelow<T> : m, f = up ? __builtin_amdgcn_exp2f(m - to) : 1.f;
            m = to;
            l *= f;
#pragma unroll
            for (int j = 0; j < DV / 32; ++j) o[j] *= f;
        }
    };
    // A step: its weights and their products with the values, while the next step's scores are made,
    // and what comes behind that is on its way. The order is written out, for the matrix instructions
    // to follow each other while the weights' instructions run beside them: of the pairs of weights
    // the first kBeside are made beside the scores, the others beside the first half of the products
    // with the values, and the next scores' maxima beside the second.
    const auto go = [&](auto parity, int step, f32x16 (&s)[KB], f32x16 (&next)[KB]) {
        constexpr int b = parity.value, kP = DV / 32;
        constexpr int kQ = KB * (D / 16), kV = 2 * KB * kP;                 // fragments
        constexpr int kPairs = 8 * KB, kFirst = 2;
        constexpr int kBeside = (D == 64 ? kPairs / 2 : D == 128 ? kPairs * 5 / 8 : kPairs) - kFirst;
        u32x4 pf[2 * KB], kf[kAhead + 1], vf[kAhead + 1];
        // Pairs of weights, four for 16 keys. Where it meets the values a weight has the type's bits, for a
        // matrix instruction takes one type on both sides: the rest of each in a second product would
        // be half as many matrix instructions more, of which long prompts are bound. The sum counts it
        // as it was, for lse is made of it. Errors against 64 bits, of the outputs' size: 2.3e-4 at 16 x
        // 1..1021, binary16, and 1.8e-3 at 4 x 1500..2047, bfloat16; 2.0e-4 and 1.6e-3 are the outputs' own
        // rounding.
        const auto weigh = [&](int from, int to) {
#pragma unroll
            for (int i = from; i < to; ++i) {
                const float p = __builtin_amdgcn_exp2f(fmaf(s[i / 8][i % 8 * 2], a.scale, -m));
                const float q = __builtin_amdgcn_exp2f(fmaf(s[i / 8][i % 8 * 2 + 1], a.scale, -m));
                l += p;
                l += q;
                pf[i / 4][i % 4] = round2<T>(p, q);
            }
        };
        const auto key = [&](int i) { return key_frag(b ^ 1, i % KB, i / KB); };
        const auto value = [&](int i) { return value_frag(b, i / kP, i % kP); };
        __syncthreads();
        check_values(step + 1);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) kf[i] = key(i);
        weigh(0, kFirst);               // while the first fragments are on their way
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
            f32x16 zero;
#pragma unroll
            for (int e = 0; e < 16; ++e) zero[e] = 0.f;
            next[i % KB] = mfma<T>(kf[i % (kAhead + 1)], qf[i / KB], i < KB ? zero : next[i % KB]);
            if (i + kAhead < kQ) kf[(i + kAhead) % (kAhead + 1)] = key(i + kAhead);
            else vf[(i + kAhead - kQ) % (kAhead + 1)] = value(i + kAhead - kQ);
            weigh(kFirst + i * kBeside / kQ, kFirst + (i + 1) * kBeside / kQ);
            if (i == kQ / 4) put_keys(b);                   // of step + 2
            if (i == kQ * 3 / 8) put_values(b ^ 1);         // of step + 1
            if (i == kQ / 2) fetch_keys();
            if (i == kQ * 5 / 8) fetch_values();
            __builtin_amdgcn_sched_barrier(0);
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            o[i % kP] = mfma<T>(vf[i % (kAhead + 1)], pf[i / kP], o[i % kP]);
            if (i + kAhead < kV) vf[(i + kAhead) % (kAhead + 1)] = value(i + kAhead);
            constexpr int kHalf = kV / 2, kLast = kPairs - kFirst - kBeside;
            if (i < kHalf) {
                weigh(kFirst + kBeside + i * kLast / kHalf, kFirst + kBeside + (i + 1) * kLast / kHalf);
            } else {
#pragma unroll
                for (int e = (i - kHalf) * kPairs / kHalf; e < (i - kHalf + 1) * kPairs / kHalf; ++e) top = larger_of(top, next, 2 * e);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        asm volatile("" : "+v"(top), "+v"(l));              // made here
        // values that are not finite, of keys that some rows see and others do not, were left out
        if (__builtin_expect((step + 1) * kKeys - 1 > first, 0) && bad[b] == step) {
#pragma unroll 1
            for (int j = step * kKeys; j < min((step + 1) * kKeys, wave_last + 1); ++j) {
                const uint16_t *v = a.v + (x.seq.begin + j) * a.v_ts + h * a.v_hs + dv0;
#pragma unroll
                for (int d = 0; d < DV / 32; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float y = to_f32<T>(v[32 * d + 8 * (i / 4) + 4 * half + i % 4]);
                        if (j <= tok && !(fabsf(y) < INFINITY)) o[d][i] += y;
                    }
            }
        }
        if (step + 1 < steps) look(next, top, step + 1);
    };

    fetch_keys();
    fetch_values();
    const uint16_t *q = a.q + (x.seq.begin + tok) * a.q_ts + hq * a.q_hs + 8 * half;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
        qf[d] = u32x4{0, 0, 0, 0};
        if (row < x.n_rows) qf[d] = *reinterpret_cast<const u32x4 *>(q + 16 * d);
    }
    if (__builtin_expect(a.flip != 0 || a.keep == 0, 0))
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) qf[d][e] = (qf[d][e] & a.keep) ^ a.flip;
    __syncthreads();                    // `bad` is set
    check_values(0);
    put_keys(0);
    put_values(0);
    fetch_keys();
    fetch_values();
    f32x16 s0[KB], s1[KB];
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < DV / 32; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[j][i] = 0.f;
    __syncthreads();
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
        for (int e = 0; e < 16; ++e) s0[kb][e] = 0.f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) s0[kb] = mfma<T>(key_frag(0, kb, d), qf[d], s0[kb]);
    }
#pragma unroll
    for (int e = 0; e < 16 * KB; e += 2) top = larger_of(top, s0, e);
    put_keys(1);
    fetch_keys();
    look(s0, top, 0);
    for (int step = 0;;) {
        go(Index<0>{}, step, s0, s1);
        if (++step == steps) break;
        go(Index<1>{}, step, s1, s0);
        if (++step == steps) break;
    }
    l = of_row(l, [](float p, float q) { return p + q; });
    if (row >= x.n_rows) return;
    const float inv = l > 0.f ? 1.f / l : l;
    uint16_t *to = a.out + (x.seq.begin + tok) * a.o_ts + hq * a.o_hs + dv0 + 8 * half;
#pragma unroll
    for (int j = 0; j < DV / 32; ++j)
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
            // of each sixteen dimensions the first lane of a row gets the first eight, the other the others
            const auto p = __builtin_amdgcn_permlane32_swap(round2<T>(o[j][i] * inv, o[j][i + 1] * inv),
                                                            round2<T>(o[j][i + 4] * inv, o[j][i + 5] * inv), false, false);
            const auto q = __builtin_amdgcn_permlane32_swap(round2<T>(o[j][i + 2] * inv, o[j][i + 3] * inv),
                                                            round2<T>(o[j][i + 6] * inv, o[j][i + 7] * inv), false, false);
            *reinterpret_cast<u32x4 *>(to + 32 * j + 2 * i) = u32x4{p[0], q[0], p[1], q[1]};
        }
    if (a.lse && half == 0 && dv0 == 0)
        a.lse[(int64_t)(x.seq.begin + tok) * a.heads * a.per + hq] = (m + log2f(l)) * 0.6931471805599453f;
}

template <typename T, int D, int DV, int WAVES, int KB>
hipError_t launch_tiles(const PromptArgs &a, hipStream_t stream)
{
    // no more tiles than this, however the sequences are cut
    constexpr int kRows = 32 * WAVES;
    const int64_t rows = (int64_t)a.s.n_tokens * a.per, each = rows / a.s.n_seqs;
    const int64_t tiles = a.s.cu ? rows / kRows + a.s.n_seqs : (each + kRows - 1) / kRows * a.s.n_seqs;
    prompt_kernel<T, D, DV, WAVES, KB><<<dim3((unsigned)(tiles * a.heads * (D / DV))), 64 * WAVES, 0, stream>>>(a);
    return hipGetLastError();
}

// Blocks of 128 rows that go 32 keys a step, two to a CU, or of 256 rows and with heads of 128 64 keys,
// one to a CU, which fetch a key for twice the rows and meet half as often, but begin and end alone.
// Measured in us, of 128 and of 256 rows (sequences x tokens, query heads / key heads), heads of 128:
//   1 x 8190, 64/8    1072   995      2 x 4096, 32/32   298   299      8 x 2048, 32/8    322   321
//   1 x 4096, 32/8     155   136      2 x 2048, 40/40   115   117      4 x 2048, 64/8    309   316
//   2 x 2048, 32/8      87    79      4 x 1536, 32/8     96    99      16 x 1536, 32/8   388   401
//   4 x 3000, 32/8     311   304      4 x 2048, 32/32   171   176      1 x 8190, 32/32   551   521
// and of 256:
//   1 x 8190, 16/4     739   696      1 x 4096, 16/4    209   187      2 x 3000, 16/4    221   220
//   8 x 2048, 16/4     431   434      8 x 2048, 8/8     225   238      8 x 3000, 8/8     472   484
// so the wide ones have long sequences (the rows of one head cover fewer tokens the more heads share
// it, and a tile's end wastes less) and two blocks at least to a CU. And where keys and values are more
// than the last level's cache holds, 256 MB, each block fetches them from memory, and sequences need not
// be long:
//   16 x 2048, 32/32  1048   815      64 x 512, 32/32   460   410      64 x 1024, 64/8  1857  1747
//   16 x 3000, 40/40  2724  2031      32 x 1024, 32/32  654   537      128 x 1536, 32/8 5087  3774
//   400 x 128, 32/32   534   679      200 x 300, 40/40 1058  1182      8 x 1536, 40/40   298   303 (251 MB)
//   of 256: 16 x 2048, 16/16   1165  1038      64 x 512, 16/16   498   494
// Lengths are known by their mean alone: one of 8190 among 31 of 100, 32/8, has small blocks (550 us,
// wide ones 519). (Heads of 64: 599 and 616 at 1 x 8190, 64/8.)
bool wide_blocks(const PromptArgs &a, int dim)
{
    const int64_t blocks = (int64_t)a.s.n_tokens * a.per * a.heads / 256 * (dim / 128);
    const int64_t bytes = (int64_t)a.s.n_tokens * a.heads * dim * 4;
    const int mean = a.s.n_tokens / a.s.n_seqs;
    return blocks >= 512 && (mean >= (dim == 128 && a.per >= 4 ? 2048 : 4096) || (bytes >= 1 << 28 && mean >= 512));
}

// Heads of 256 have their outputs' dimensions in two blocks, each of which makes all scores: half as
// many products more, but two waves to a SIMD where the sums of one took the registers of both (4 x
// 1500..2047, 16/4: 177 us and 201; 1 x 1000: 33 and 53; 1 x 8190: 774 and 769). Heads of 128 too while
// that leaves a CU to each block (1 x 300, 32/32: 11.6 and 13.4; 1 x 1000, 8/8: 23.9 and 27.2; 1 x 2048,
// 8/1: 40 and 45; with more, 4 x 1..1000, 32/8: 37 and 32).
bool halved(const PromptArgs &a)
{
    return ((int64_t)a.s.n_tokens * a.per / 128 + a.s.n_seqs) * a.heads <= 128;
}

template <typename T>
hipError_t launch(const PromptArgs &a, int dim, hipStream_t stream)
{
    if (dim == 64) return launch_tiles<T, 64, 64, 4, 1>(a, stream);
    const bool wide = wide_blocks(a, dim);
    if (dim == 256) return wide ? launch_tiles<T, 256, 128, 8, 1>(a, stream) : launch_tiles<T, 256, 128, 4, 1>(a, stream);
    if (halved(a)) return launch_tiles<T, 128, 64, 4, 1>(a, stream);
    return wide ? launch_tiles<T, 128, 128, 8, 2>(a, stream) : launch_tiles<T, 128, 128, 4, 1>(a, stream);
}

hqq_status refuse(const char *msg, hqq_status st = HQQ_ERR_ARG)
{
    report_error(st, msg);
    return st;
}

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace hqq

extern "C" hqq_status hqq_prompt_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
                                           int64_t k_token_stride, int64_t k_head_stride, const void *v,
                                           int64_t v_token_stride, int64_t v_head_stride, int64_t n_tokens, int n_q_heads,
                                           int n_kv_heads, int head_dim, int dtype, const int32_t *cu_tokens, int n_seqs,
                                           float scale, void *out, int64_t out_token_stride, int64_t out_head_stride,
                                           float *lse, void *stream)
{
    using namespace hqq;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return refuse("head_dim must be 64, 128 or 256");
    if (dtype != HQQ_F16 && dtype != HQQ_BF16) return refuse("dtype must be HQQ_F16 or HQQ_BF16");
    if (n_kv_heads < 1 || n_kv_heads > 1024) return refuse("n_kv_heads must be in [1, 1024]");
    if (n_q_heads < 1 || n_q_heads % n_kv_heads != 0) return refuse("n_q_heads must be a positive multiple of n_kv_heads");
    if (n_seqs < 0 || n_seqs > kMaxSeqs) return refuse("n_seqs must be in [0, 4096]");
    if (n_tokens < 0 || n_tokens > (1 << 24)) return refuse("n_tokens must be in [0, 2^24]");
    if (n_q_heads > (1 << 20) || n_tokens * n_q_heads > (1 << 30))
        return refuse("n_q_heads must be at most 2^20, and n_tokens * n_q_heads at most 2^30");
    if (!std::isfinite(scale * kLog2e)) return refuse("scale must be finite, and times log2(e) too");
    if (!aligned(cu_tokens, 4) || !aligned(lse, 4)) return refuse("cu_tokens and lse must be 4-byte aligned");
    if (n_seqs == 0 || n_tokens == 0) {
        report_error(HQQ_OK, "");
        return HQQ_OK;
    }
    if (!cu_tokens && n_tokens % n_seqs != 0) return refuse("n_tokens must be a multiple of n_seqs without cu_tokens");
    const struct {
        const void *p;
        int64_t ts, hs;
    } rows[] = {{q, q_token_stride, q_head_stride}, {k, k_token_stride, k_head_stride},
                {v, v_token_stride, v_head_stride}, {out, out_token_stride, out_head_stride}};
    for (const auto &r : rows) {
        if (!r.p) return refuse("q, k, v and out must be non-null");
        if (!aligned(r.p, 16) || r.ts < 0 || r.hs < 0 || r.ts % 8 || r.hs % 8 || r.ts > (int64_t(1) << 36) || r.hs > (int64_t(1) << 36))
            return refuse("q, k, v and out must be 16-byte aligned, with strides that are multiples of 8 in [0, 2^36]");
    }
    // offsets within a step's keys are 32 bits
    if (k_token_stride > kMaxKeyStride || v_token_stride > kMaxKeyStride)
        return refuse("the token strides of k and v must be at most 2^22");
    PromptArgs a{};
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.k_ts = k_token_stride;
    a.k_hs = k_head_stride;
    a.v_ts = v_token_stride;
    a.v_hs = v_head_stride;
    a.o_ts = out_token_stride;
    a.o_hs = out_head_stride;
    a.s.cu = cu_tokens;
    a.s.n_seqs = n_seqs;
    a.s.n_tokens = (int32_t)n_tokens;
    a.heads = n_kv_heads;
    a.per = n_q_heads / n_kv_heads;
    a.inv = a.per == 1 ? 0 : UINT64_MAX / a.per + 1;
    // the sign of scale goes to the queries, and a scale of 0 makes them 0: the largest score is then
    // the largest product, and what a row does not see stays at -infinity
    a.scale = scale == 0.f ? 1.f : std::fabs(scale) * kLog2e;
    a.flip = scale < 0.f ? 0x80008000u : 0u;
    a.keep = scale == 0.f ? 0u : 0xffffffffu;
    // blocks of the smallest tiles (a dimension of a grid has less than 2^32 threads)
    if ((n_tokens * a.per / 128 + n_seqs) * a.heads * (head_dim == 256 ? 2 : 1) >= (1 << 24)) return refuse("too many rows for one call", HQQ_ERR_UNSUPPORTED);
    const hipStream_t str = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == HQQ_BF16 ? launch<Bf16>(a, head_dim, str) : launch<F16>(a, head_dim, str);
    if (e != hipSuccess) return refuse(hipGetErrorString(e), HQQ_ERR_DEVICE);
    report_error(HQQ_OK, "");
    return HQQ_OK;
}
