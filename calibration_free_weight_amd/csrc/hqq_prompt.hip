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
// a row.
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

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kRows = 32 * kWaves;
constexpr float kLog2e = 1.44269504088896341f;
// How far a score (to base 2) may lie above the maximum that weights are taken from.
constexpr float kSlack = 8.f;

struct PromptArgs {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    float *lse;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;
    SeqView s;                  // cu, n_seqs, n_tokens
    int32_t heads, per;         // key/value heads, query heads to one
    float scale;                // |scale| times log2(e), or 1 where scale is 0
    uint32_t flip, keep;        // of two queries: bits that change, bits that stay
};

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

// Tile `back` from the last of all sequences (the longest tiles of each come first), or none.
// scan: [kWaves + 1] in LDS, found: [2].
__device__ __forceinline__ bool find_tile(const SeqView &s, int per, int back, int32_t *scan, int32_t *found, Tile &x)
{
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int each = (s.n_seqs + kThreads - 1) / kThreads, b0 = min(t * each, s.n_seqs), b1 = min(b0 + each, s.n_seqs);
    int sum = 0;
    bool falls = false;
    for (int b = b0; b < b1; ++b) {
        const Rows r = rows_of(s, b);
        sum += tiles_of((r.end - r.begin) * per, kRows);
        falls = falls || falls_at(s, b);
    }
    int upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(upto, d);
        if (lane >= d) upto += y;
    }
    if (lane == 63) scan[wave] = upto;
    if (__syncthreads_or(falls)) return false;      // rows would be counted twice
    int before = upto - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += scan[w];
        total += scan[w];
    }
    const int u = total - 1 - back;
    if (u < 0) return false;
    if (before <= u && u < before + sum) {
        for (int b = b0; b < b1; ++b) {
            const Rows r = rows_of(s, b);
            const int n = tiles_of((r.end - r.begin) * per, kRows);
            if (u < before + n) {
                found[0] = b;
                found[1] = u - before;
                break;
            }
            before += n;
        }
    }
    __syncthreads();
    x.seq = rows_of(s, __builtin_amdgcn_readfirstlane(found[0]));
    x.row0 = __builtin_amdgcn_readfirstlane(found[1]) * kRows;
    x.n_rows = (x.seq.end - x.seq.begin) * per;
    return true;
}

template <typename T, int D, int BN>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void prompt_kernel(PromptArgs a)
{
    constexpr int kChunks = D / 8;                          // of 16 bytes, in a row of keys or values
    constexpr int kEach = BN * kChunks / kThreads;          // chunks of keys to a thread
    constexpr int kApart = kThreads / kChunks;              // rows between a thread's chunks
    __shared__ u32x4 keys[2][BN * kChunks], values[2][BN * kChunks];
    __shared__ int32_t scan[kWaves], found[2], bad[2];      // bad: the last tile whose values were not finite
    Tile x;
    const int h = (int)(blockIdx.x % (unsigned)a.heads);
    if (threadIdx.x < 2) bad[threadIdx.x] = -1;
    if (!find_tile(a.s, a.per, (int)(blockIdx.x / (unsigned)a.heads), scan, found, x)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
    const int n = x.seq.end - x.seq.begin;
    const int row = x.row0 + 32 * wave + col;
    const bool have = row < x.n_rows;
    const int tok = (have ? row : x.n_rows - 1) / a.per, hq = h * a.per + (have ? row - tok * a.per : 0);
    // tokens of the block's and the wave's first and last rows
    const int first = x.row0 / a.per, last = min(x.row0 + kRows, x.n_rows) - 1;
    const int wave_first = min(x.row0 + 32 * wave, x.n_rows - 1) / a.per;
    const int wave_last = min(x.row0 + 32 * wave + 31, x.n_rows - 1) / a.per;
    const bool wave_has = x.row0 + 32 * wave < x.n_rows;
    const int end = last / a.per + 1;                       // keys that some row sees
    const int tiles = (end + BN - 1) / BN;

    // where a thread's chunks come from: rows and places are swapped within LDS so that no two lanes
    // that read at a time meet in a bank
    const int r0 = (int)threadIdx.x / kChunks, place = (int)threadIdx.x % kChunks;
    const auto key_swap = [](int r) { return kChunks == 8 ? (r >> 1) & 7 : r & 15; };
    const auto value_swap = [](int r) { return kChunks == 8 ? ((r >> 1) & 1) << 2 : (r & 3) << 2; };
    u32x4 kr[kEach], vr[kEach];
    const auto fetch = [&](int j0) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int r = r0 + i * kApart;
            const int64_t at = x.seq.begin + min(j0 + r, n - 1);
            kr[i] = *reinterpret_cast<const u32x4 *>(a.k + at * a.k_ts + h * a.k_hs + 8 * (place ^ key_swap(r)));
            vr[i] = *reinterpret_cast<const u32x4 *>(a.v + at * a.v_ts + h * a.v_hs + 8 * (place ^ value_swap(r)));
        }
    };
    const auto put = [&](int tile) {
        const int j0 = tile * BN, b = tile & 1;
        if (j0 + BN - 1 > first) {      // some row does not see some key
            bool ok = true;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const bool in = j0 + r0 + i * kApart < n;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (!in) vr[i][e] = 0;
                    uint32_t w = vr[i][e];
                    ok = finite2<T>(w) && ok;
                    vr[i][e] = w;
                }
            }
            if (!ok) bad[b] = tile;
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            keys[b][threadIdx.x + i * kThreads] = kr[i];
            values[b][threadIdx.x + i * kThreads] = vr[i];
        }
    };

    fetch(0);
    u32x4 qf[D / 16];
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        qf[s] = u32x4{0, 0, 0, 0};
        if (have) qf[s] = *reinterpret_cast<const u32x4 *>(a.q + (x.seq.begin + tok) * a.q_ts + hq * a.q_hs + 16 * s + 8 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) qf[s][e] = (qf[s][e] & a.keep) ^ a.flip;
    }
    put(0);
    if (tiles > 1) fetch(BN);
    f32x16 o[D / 32];
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[j][i] = 0.f;
    float m = -INFINITY, l = 0.f;

    for (int tile = 0; tile < tiles; ++tile) {
        const int j0 = tile * BN, b = tile & 1;
        __syncthreads();
        if (tile + 1 < tiles) put(tile + 1);
        if (tile + 2 < tiles) fetch(j0 + 2 * BN);
        if (j0 > wave_last || !wave_has) continue;
        f32x16 s[BN / 32];
#pragma unroll
        for (int kb = 0; kb < BN / 32; ++kb) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[kb][i] = 0.f;
            const int r = 32 * kb + col;
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
                s[kb] = mfma<T>(keys[b][r * kChunks + ((2 * d + half) ^ key_swap(r))], qf[d], s[kb]);
        }
        if (j0 + BN - 1 > wave_first)
#pragma unroll
            for (int kb = 0; kb < BN / 32; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (j0 + 32 * kb + 8 * (i / 4) + 4 * half + i % 4 > tok) s[kb][i] = -INFINITY;
        float top = s[0][0];
#pragma unroll
        for (int kb = 0; kb < BN / 32; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[kb][i]);
        top = of_row(top, [](float p, float q) { return fmaxf(p, q); }) * a.scale;
        if (__any(top > m + kSlack)) {
            const float to = fmaxf(m, top), f = m == to ? 1.f : __builtin_amdgcn_exp2f(m - to);
            m = to;
            l *= f;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) o[j] *= f;
        }
#pragma unroll
        for (int kb = 0; kb < BN / 32; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[kb][i] = __builtin_amdgcn_exp2f(fmaf(s[kb][i], a.scale, -m));
                l += s[kb][i];
            }
#pragma unroll
        for (int g = 0; g < BN / 16; ++g) {
            u32x4 pf;
#pragma unroll
            for (int e = 0; e < 4; ++e) pf[e] = round2<T>(s[g / 2][8 * (g % 2) + 2 * e], s[g / 2][8 * (g % 2) + 2 * e + 1]);
            const int r = 16 * g + 4 * half + ((lane & 15) >> 2);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const int c = (4 * j + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ value_swap(r);
                const char *p = reinterpret_cast<const char *>(&values[b][r * kChunks + c]) + 8 * (lane & 1);
                const u32x2 lo = read_transposed(p), hi = read_transposed(p + 8 * kChunks * 16);
                o[j] = mfma<T>(u32x4{lo[0], lo[1], hi[0], hi[1]}, pf, o[j]);
            }
        }
        // values that are not finite, of keys that some rows see and others do not, were left out
        if (__builtin_expect(bad[b] == tile, 0)) {
#pragma unroll 1
            for (int j = j0; j < min(j0 + BN, wave_last + 1); ++j) {
                const uint16_t *v = a.v + (x.seq.begin + j) * a.v_ts + h * a.v_hs;
#pragma unroll
                for (int d = 0; d < D / 32; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float y = to_f32<T>(v[32 * d + 8 * (i / 4) + 4 * half + i % 4]);
                        if (j <= tok && !(fabsf(y) < INFINITY)) o[d][i] += y;
                    }
            }
        }
    }
    l = of_row(l, [](float p, float q) { return p + q; });
    if (!have) return;
    const float inv = l > 0.f ? 1.f / l : l;
    uint16_t *to = a.out + (x.seq.begin + tok) * a.o_ts + hq * a.o_hs + 4 * half;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<u32x2 *>(to + 32 * j + 8 * i) = u32x2{round2<T>(o[j][4 * i] * inv, o[j][4 * i + 1] * inv),
                                                                    round2<T>(o[j][4 * i + 2] * inv, o[j][4 * i + 3] * inv)};
    if (a.lse && half == 0)
        a.lse[(int64_t)(x.seq.begin + tok) * a.heads * a.per + hq] = (m + log2f(l)) * 0.6931471805599453f;
}

template <typename T>
hipError_t launch(const PromptArgs &a, int dim, int64_t tiles, hipStream_t stream)
{
    const unsigned blocks = (unsigned)(tiles * a.heads);
    if (dim == 64) prompt_kernel<T, 64, 64><<<blocks, kThreads, 0, stream>>>(a);
    else if (dim == 128) prompt_kernel<T, 128, 64><<<blocks, kThreads, 0, stream>>>(a);
    else prompt_kernel<T, 256, 32><<<blocks, kThreads, 0, stream>>>(a);
    return hipGetLastError();
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
    // the sign of scale goes to the queries, and a scale of 0 makes them 0: the largest score is then
    // the largest product, and what a row does not see stays at -infinity
    a.scale = scale == 0.f ? 1.f : std::fabs(scale) * kLog2e;
    a.flip = scale < 0.f ? 0x80008000u : 0u;
    a.keep = scale == 0.f ? 0u : 0xffffffffu;
    // no more tiles than this, however the sequences are cut
    const int64_t each = n_tokens / n_seqs * a.per;
    const int64_t tiles = cu_tokens ? n_tokens * a.per / kRows + n_seqs : (each + kRows - 1) / kRows * n_seqs;
    if (tiles * a.heads >= (1 << 24)) return refuse("too many rows for one call", HQQ_ERR_UNSUPPORTED);
    const hipStream_t str = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == HQQ_BF16 ? launch<Bf16>(a, head_dim, tiles, str) : launch<F16>(a, head_dim, tiles, str);
    if (e != hipSuccess) return refuse(hipGetErrorString(e), HQQ_ERR_DEVICE);
    report_error(HQQ_OK, "");
    return HQQ_OK;
}
