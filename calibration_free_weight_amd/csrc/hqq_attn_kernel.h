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
// factor of 2^6). Codes go into the products as whole numbers, exact in either type, and the
// grids are applied to the sums: S = step . (q, Q) + base . sum(Q) per group, and
// V's step to the weights, whose product with base is summed beside. Whatever the lengths, a
// token outside its sequence has grid {0, 0} and weight 0.
#pragma once

#include "hqq_cache_internal.h"

namespace hqq {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;

constexpr int kAttnThreads = 256;
constexpr int kWaves = kAttnThreads / 64;
constexpr int kTile = 32;                   // tokens of a wave's step
static_assert(kTile * kWaves == kUnit, "a unit is one step of the block");

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

// Code i of a value's row for two tokens (words x, y hold it) as bfloat16 numbers.
template <int NB>
__device__ __forceinline__ uint32_t value_pair(const uint32_t *x, const uint32_t *y, int i)
{
    if constexpr (NB == 4) {
        // bytes 2c and 2c + 1 of both tokens, side by side: codes 4c..4c+3
        const int c = i >> 2, k = c & 1;
        const uint32_t p = __builtin_amdgcn_perm(y[c >> 1], x[c >> 1], k ? 0x07030602u : 0x05010400u);
        const uint32_t n = (i & 1 ? p >> 4 : p) & 0x0f0f0f0fu;
        return i & 2 ? small2<true, true>(n) : small2<true, false>(n);
    } else {
        return whole_bf16x2(ubyte(x[i >> 2], i & 3), ubyte(y[i >> 2], i & 3));
    }
}

// Two binary32 numbers as bfloat16 (nearest even), and what that leaves of them.
__device__ __forceinline__ uint32_t round_pair(float &a, float &b)
{
    const f32x2 x = {a, b};
    const uint32_t r = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
    a -= __uint_as_float(r << 16);
    b -= __uint_as_float(r & 0xffff0000u);
    return r;
}

template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[BYTES / 4])
{
    if constexpr (BYTES % 16 == 0) {
#pragma unroll
        for (int k = 0; k < BYTES / 16; ++k) {
            const uint4 x = reinterpret_cast<const uint4 *>(p)[k];
            w[4 * k] = x.x;
            w[4 * k + 1] = x.y;
            w[4 * k + 2] = x.z;
            w[4 * k + 3] = x.w;
        }
    } else {
        static_assert(BYTES == 8, "8 or a multiple of 16");
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x;
        w[1] = x.y;
    }
}

// Sum over the four lanes of a column (16 and 32 apart).
__device__ __forceinline__ float column_sum(float x)
{
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// The units before each sequence's, in LDS: starts[n_seqs] is their sum.
template <int ROWS>
__device__ void lay_out(const AttnArgs &a, int32_t *starts, int32_t *scan)
{
    const int t = threadIdx.x, n = a.s.n_seqs;
    const int each = (n + kAttnThreads - 1) / kAttnThreads, b0 = min(t * each, n), b1 = min(b0 + each, n);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
        const Rows r = rows_of(a.s, b);
        const int u = tiles_of((r.end - r.begin) * a.per, ROWS) * units_along(len_of(a.s, b));
        starts[b] = u;
        sum += u;
    }
    // exclusive sums over the threads: within the waves, then over them
    int run = sum;
    for (int x = 1; x < 64; x <<= 1) {
        const int y = __shfl_up(run, x);
        if ((t & 63) >= x) run += y;
    }
    if ((t & 63) == 63) scan[t >> 6] = run;
    __syncthreads();
    int before = run - sum, total = 0;
    for (int w = 0; w < kWaves; ++w) {
        if (w < (t >> 6)) before += scan[w];
        total += scan[w];
    }
    for (int b = b0; b < b1; ++b) {
        const int u = starts[b];
        starts[b] = before;
        before += u;
    }
    if (t == 0) starts[n] = total;
    __syncthreads();
}

template <typename T, int NB, int D, int G, int RT>
__global__ __launch_bounds__(kAttnThreads) void attn_kernel(AttnArgs a)
{
    constexpr bool kBf16 = Types<T>::kBf16;
    constexpr int kGroups = D / G, kRows = 16 * RT;
    constexpr int kKeyBytes = D * NB / 32;      // a lane's quarter of a token's key
    constexpr int kValBytes = D * NB / 128;     // a row of a token's value
    constexpr int kUnitWords = NB / 4;
    extern __shared__ int32_t shared[];
    int32_t *starts = shared;                                       // [n_seqs + 1]
    int32_t *scan = shared + (((unsigned)a.s.n_seqs + 4) & ~3u);    // [kWaves]
    float *ml = reinterpret_cast<float *>(scan + 4);                // [kWaves][kRows][2]
    float *sum = ml + kWaves * kRows * 2;                           // [kRows][D]

    lay_out<kRows>(a, starts, scan);
    const int h = (int)(blockIdx.x % (unsigned)a.c.heads), w = (int)(blockIdx.x / (unsigned)a.c.heads);
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b <= a.s.n_seqs; b += kAttnThreads) a.side.starts[b] = starts[b];
    const int W = a.side.workers, U = starts[a.s.n_seqs];
    const int u_end = first_unit(w + 1, W, U);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, quad = lane >> 4;

    for (int u = first_unit(w, W, U); u < u_end;) {
        // the item that unit u is of
        int b = 0;
        for (int hi = a.s.n_seqs; hi - b > 1;) {
            const int mid = (b + hi) >> 1;
            if (starts[mid] <= u) b = mid; else hi = mid;
        }
        const Rows rows = rows_of(a.s, b);
        const int len = len_of(a.s, b), n_rows = (rows.end - rows.begin) * a.per;
        const int along = units_along(len), tile = (u - starts[b]) / along, u_in = (u - starts[b]) % along;
        const int count = min(u_end - u, along - u_in);
        const int row0 = tile * kRows;
        u += count;

        // queries, as B fragments; what a column sees ends at lim
        u32x4 qf[RT][D / 32];
        float qsum[RT][kGroups];
        int lim[RT], lim_low = len, lim_high = 0;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int row = row0 + 16 * t + col;
            const bool have = row < n_rows;
            const int tok = have ? row / a.per : 0, hq = h * a.per + (have ? row % a.per : 0);
            const uint16_t *q = a.q + (rows.begin + tok) * a.q_ts + hq * a.q_hs;
            lim[t] = !have ? 0 : a.causal ? len - (rows.end - rows.begin) + tok + 1 : len;
            if (have) {
                lim_low = min(lim_low, lim[t]);
                lim_high = max(lim_high, lim[t]);
            }
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                float x = 0.f;
#pragma unroll
                for (int m = g * G / 32; m < (g + 1) * G / 32; ++m) {
                    uint4 raw = {0, 0, 0, 0};
                    if (have) raw = *reinterpret_cast<const uint4 *>(q + 32 * m + 8 * quad);
                    qf[t][m] = u32x4{raw.x, raw.y, raw.z, raw.w};
                    float v[8];
                    unpack8<T>(raw, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x += v[e];
                }
                qsum[t][g] = column_sum(x);
            }
        }
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) {
            lim_low = min(lim_low, __shfl_xor(lim_low, x));
            lim_high = max(lim_high, __shfl_xor(lim_high, x));
        }
        lim_low = __builtin_amdgcn_readfirstlane(lim_low);
        lim_high = __builtin_amdgcn_readfirstlane(lim_high);

        f32x4 o[RT][D / 16];
        float m[RT], l[RT], bsum[RT][kGroups];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            m[t] = -INFINITY;
            l[t] = 0.f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) bsum[t][g] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[t][j] = f32x4{0, 0, 0, 0};
        }

        for (int step = 0; step < count; ++step) {
            const int t0 = (u_in + step) * kUnit + wave * kTile;
            if (t0 >= lim_high) break;
            float s[RT][8];
            uint32_t vw[8][(kValBytes + 3) / 4];
            uint32_t vmeta[8][kGroups];
            int good[2];                        // tokens of each half that are in the cache
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int th = t0 + 16 * half;
                int page = th < len ? page_of(a.s, b, th) : -1;
                page = __builtin_amdgcn_readfirstlane(page);
                good[half] = page < 0 ? 0 : min(16, len - th);
                const int at = th & ((1 << a.s.page_shift) - 1);
                const int64_t slice = ((int64_t)max(page, 0) * a.c.heads + h) << a.s.page_shift;
                const uint8_t *kc = a.c.k_codes + slice * (D * NB / 8) +
                                    k_unit_at(at + col, quad, 0, D, NB);
                const uint8_t *vc = a.c.v_codes + slice * (D * NB / 8) +
                                    v_row_at(at + 4 * quad, col, D, NB);
                const uint32_t *km = a.c.k_meta + (slice + at + 4 * quad) * kGroups;
                const uint32_t *vm = a.c.v_meta + (slice + at + 4 * quad) * kGroups;
                uint32_t kw[kKeyBytes / 4], vq[kValBytes], kmeta[4][kGroups];
                load_words<kKeyBytes>(kc, kw);
                load_words<4 * kValBytes>(vc, vq);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const bool in = 4 * quad + i < good[half];
                        kmeta[i][g] = in ? km[i * kGroups + g] : 0u;
                        vmeta[4 * half + i][g] = in ? vm[i * kGroups + g] : 0u;
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (kValBytes >= 4) {
#pragma unroll
                        for (int k = 0; k < kValBytes / 4; ++k)
                            vw[4 * half + i][k] = vq[i * (kValBytes / 4) + k];
                    } else {
                        vw[4 * half + i][0] = vq[i / 2] >> (16 * (i & 1));
                    }
                }
                // scores, one group of dimensions after another
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][4 * half + i] = 0.f;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    f32x4 acc[RT];
#pragma unroll
                    for (int t = 0; t < RT; ++t) acc[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int mm = g * G / 32; mm < (g + 1) * G / 32; ++mm) {
                        const u32x4 kf = key_frag<kBf16, NB>(kw + mm * kUnitWords);
#pragma unroll
                        for (int t = 0; t < RT; ++t) acc[t] = mfma32<kBf16>(kf, qf[t][mm], acc[t]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float st = to_f32<T>(kmeta[i][g] & 0xffffu), ba = to_f32<T>(kmeta[i][g] >> 16);
#pragma unroll
                        for (int t = 0; t < RT; ++t)
                            s[t][4 * half + i] += fmaf(st, acc[t][i], ba * qsum[t][g]);
                    }
                }
            }
            const bool open = t0 + kTile <= lim_low && good[0] == 16 && good[1] == 16;
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[t][i] *= a.scale;
                    if (!open) {
                        const int at = 4 * quad + (i & 3);
                        if (t0 + 16 * (i >> 2) + at >= lim[t] || at >= good[i >> 2]) s[t][i] = -INFINITY;
                    }
                    top = fmaxf(top, s[t][i]);
                }
                // Weights are 2^(s - m) with m the largest score up to some time ago: at most
                // 2^6, which costs the sums nothing.
                if (__any(top > m[t] + 6.f)) {
                    top = fmaxf(top, __shfl_xor(top, 16));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    const float next = fmaxf(m[t], top);
                    const float f = next == m[t] ? 1.f : __builtin_amdgcn_exp2f(m[t] - next);
                    m[t] = next;
                    l[t] *= f;
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) bsum[t][g] *= f;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) o[t][j] *= f;
                }
                const float mu = m[t] == -INFINITY ? 0.f : m[t];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[t][i] = __builtin_amdgcn_exp2f(s[t][i] - mu);
                    l[t] += s[t][i];
                }
            }
            // Weights times V's step, as a bfloat16 number and what it leaves, again as one:
            // 16 bits in all, over the whole range of binary32.
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                u32x4 ph[RT], pl[RT];
#pragma unroll
                for (int t = 0; t < RT; ++t) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        float x = s[t][i] * to_f32<T>(vmeta[i][g] & 0xffffu);
                        float y = s[t][i + 1] * to_f32<T>(vmeta[i + 1][g] & 0xffffu);
                        bsum[t][g] = fmaf(s[t][i], to_f32<T>(vmeta[i][g] >> 16), bsum[t][g]);
                        bsum[t][g] = fmaf(s[t][i + 1], to_f32<T>(vmeta[i + 1][g] >> 16), bsum[t][g]);
                        ph[t][i / 2] = round_pair(x, y);
                        pl[t][i / 2] = round_pair(x, y);
                    }
                }
#pragma unroll
                for (int j = g * G / 16; j < (g + 1) * G / 16; ++j) {
                    u32x4 vf;
#pragma unroll
                    for (int i = 0; i < 4; ++i) vf[i] = value_pair<NB>(vw[2 * i], vw[2 * i + 1], j);
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        o[t][j] = mfma32<true>(vf, ph[t], o[t][j]);
                        o[t][j] = mfma32<true>(vf, pl[t], o[t][j]);
                    }
                }
            }
        }

        // The four waves' parts, on the largest of their maxima.
        __syncthreads();                        // the last piece's sums have been read
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            l[t] = column_sum(l[t]);
            if (quad == 0) {
                ml[(wave * kRows + 16 * t + col) * 2] = m[t];
                ml[(wave * kRows + 16 * t + col) * 2 + 1] = l[t];
            }
        }
        __syncthreads();
        float f[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            float top = -INFINITY;
            for (int k = 0; k < kWaves; ++k) top = fmaxf(top, ml[(k * kRows + 16 * t + col) * 2]);
            f[t] = m[t] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[t] - top);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const float base = column_sum(bsum[t][g]);
#pragma unroll
                for (int j = g * G / 16; j < (g + 1) * G / 16; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[t][j][i] = (o[t][j][i] + base) * f[t];
            }
        }
        for (int k = 0; k < kWaves; ++k) {
            if (k == wave) {
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int d = j / (G / 16) * G + (4 * quad + i) * (G / 16) + j % (G / 16);
                            float *x = sum + (16 * t + col) * D + d;
                            *x = k == 0 ? o[t][j][i] : *x + o[t][j][i];
                        }
            }
            __syncthreads();
        }
        const int rows_here = min(kRows, n_rows - row0);
        const bool whole = count == along;
        const int slot = 2 * w + (u_in > 0 ? 0 : 1);
        for (int x = threadIdx.x; x < rows_here * D; x += kAttnThreads) {
            const int r = x / D, d = x % D;
            float top = -INFINITY, all = 0.f;
            for (int k = 0; k < kWaves; ++k) top = fmaxf(top, ml[(k * kRows + r) * 2]);
            for (int k = 0; k < kWaves; ++k) {
                const float mk = ml[(k * kRows + r) * 2];
                all += mk == -INFINITY ? 0.f : ml[(k * kRows + r) * 2 + 1] * __builtin_amdgcn_exp2f(mk - top);
            }
            const int tok = rows.begin + (row0 + r) / a.per, hq = h * a.per + (row0 + r) % a.per;
            if (!whole) {
                const int64_t at = ((int64_t)h * 2 * W + slot) * kRows + r;
                a.side.slot_o[at * D + d] = sum[x];
                if (d == 0) {
                    a.side.slot_ml[at * 2] = top;
                    a.side.slot_ml[at * 2 + 1] = all;
                }
            } else if (a.side.row_o) {
                const int64_t at = (int64_t)h * a.s.n_tokens * a.per + (int64_t)rows.begin * a.per + row0 + r;
                a.side.row_o[at * D + d] = sum[x];
                if (d == 0) {
                    a.side.row_ml[at * 2] = top;
                    a.side.row_ml[at * 2 + 1] = all;
                }
            } else {
                a.out[tok * a.o_ts + hq * a.o_hs + d] = (uint16_t)from_f32<T>(all > 0.f ? sum[x] / all : 0.f);
                if (a.lse && d == 0)
                    a.lse[(int64_t)tok * a.c.heads * a.per + hq] =
                        all > 0.f ? (top + log2f(all)) * 0.6931471805599453f : -INFINITY;
            }
        }
        __syncthreads();
    }
}

template <typename T, int NB, int D, int G, int RT>
hipError_t launch_one(const AttnArgs &a, hipStream_t stream)
{
    // at most 16 KB of starts, 2 KB and 32 KB: within what any launch may ask for
    const size_t lds = 4 * (((size_t)a.s.n_seqs + 4) & ~size_t(3)) + 16 + 4 * kWaves * 16 * RT * 2 +
                       4 * (size_t)16 * RT * D;
    attn_kernel<T, NB, D, G, RT><<<dim3((unsigned)a.side.workers * a.c.heads), kAttnThreads, lds, stream>>>(a);
    return hipGetLastError();
}

template <typename T, int NB, int D, int G>
hipError_t by_tiles(const AttnArgs &a, hipStream_t stream)
{
    if (a.side.tiles16 == 1) return launch_one<T, NB, D, G, 1>(a, stream);
    if (a.side.tiles16 == 2) return launch_one<T, NB, D, G, 2>(a, stream);
    if constexpr (D <= 128)
        if (a.side.tiles16 == 4) return launch_one<T, NB, D, G, 4>(a, stream);
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
