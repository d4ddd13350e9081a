// hqq_attn.hip -- attention over the quantized cache: the choice of the kernel, and the
// joining of an item's pieces.
#include "hqq_cache_internal.h"

namespace hqq {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kJoinWaves = kJoinThreads / 64;
constexpr int kAhead = 8;       // pieces asked for at a time
// With more rows than this a block for each split item takes less time than a wave for each row,
// most of which are of whole items: 40000 rows 168 us with the attention and 192, 4096 rows 104
// both; 1280 rows 49 and 36, for the few items have many pieces then.
constexpr int64_t kManyRows = 2048;
constexpr int64_t kFewRows = 512;
constexpr int kJoinRows = 16;   // of an item, to a block
constexpr int64_t kJoinAcross = 1 << 20;        // blocks

template <int E>
struct Acc {                    // a row's result so far; a lane holds E dimensions
    float m = -INFINITY, l = 0.f;
    float o[E] = {};
};

template <int E>
struct Floats {
    float x[E];
} __attribute__((aligned(4 * E)));

// Adds up to 64 pieces (one at least): lane k has the maximum m and sum l of piece k, whose output
// is at o + off(k) * D. Of the row's WPR waves each adds every WPR-th piece's output; the first
// outputs are asked for before the maxima are looked at, which are on their way as well.
template <int E, int WPR, typename Off>
__device__ __forceinline__ void add_pieces(Acc<E> &acc, int n, float m, float l, const float *o, Off off)
{
    const int lane = threadIdx.x & 63, mine = (threadIdx.x >> 6) % WPR;
    Floats<E> x[kAhead];
    const auto load = [&](int k0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            x[j] = *reinterpret_cast<const Floats<E> *>(o + off(min(k0 + j * WPR, n - 1)) * (64 * E) + lane * E);
    };
    load(mine);
    __builtin_amdgcn_sched_barrier(0);
    float top = m;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    top = fmaxf(top, acc.m);
    if (top == -INFINITY) return;
    const float f = m == -INFINITY ? 0.f : exp2f(m - top);
    const float g = acc.m == -INFINITY ? 0.f : exp2f(acc.m - top);
    float sum = l * f;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
    acc.l = acc.l * g + sum;
    acc.m = top;
#pragma unroll
    for (int e = 0; e < E; ++e) acc.o[e] *= g;
    for (int k0 = mine; k0 < n; k0 += kAhead * WPR) {
        if (k0 != mine) load(k0);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const float fk = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), min(k0 + j * WPR, n - 1)));
            if (k0 + j * WPR < n)
#pragma unroll
                for (int e = 0; e < E; ++e) acc.o[e] = fmaf(fk, x[j].x[e], acc.o[e]);
        }
    }
}

// Adds what one side found for a row; false if the item is whole and its result elsewhere.
template <int E, int WPR>
__device__ __forceinline__ bool add_side(Acc<E> &acc, const AttnSide &d, int b, int row_in_item, int len,
                                         int h, int64_t row, int64_t rows)
{
    const int lane = threadIdx.x & 63, per = 16 * d.tiles16;
    const int U = d.starts[d.s.n_seqs], W = runs_of(d.workers, U), along = units_along(len, d.starts[d.s.n_seqs + 1]);
    if (U == 0) return false;       // row offsets that fall: there is nothing to join
    const int u0 = d.starts[b] + row_in_item / per * along;
    const int w0 = run_of(u0, W, U), w1 = run_of(u0 + along - 1, W, U);
    if (w0 == w1) {
        if (!d.row_o) return false;
        const int64_t at = h * rows + row;
        const float m = lane == 0 ? d.row_ml[at * 2] : -INFINITY, l = lane == 0 ? d.row_ml[at * 2 + 1] : 0.f;
        add_pieces<E, WPR>(acc, 1, m, l, d.row_o, [&](int) { return at; });
        return true;
    }
    // the item's first run goes on behind it, the others began before theirs
    const auto at = [&](int w) { return ((int64_t)h * 2 * d.workers + 2 * w + (w == w0)) * per + row_in_item % per; };
    for (int wb = w0; wb <= w1; wb += 64) {
        const int w = wb + lane;
        const float m = w <= w1 ? d.slot_ml[at(w) * 2] : -INFINITY, l = w <= w1 ? d.slot_ml[at(w) * 2 + 1] : 0.f;
        add_pieces<E, WPR>(acc, min(64, w1 - wb + 1), m, l, d.slot_o, [&](int k) { return at(wb + k); });
    }
    return true;
}

// WPR waves per query row: they find the pieces of its item on each side by the rule that
// dealt them out, and add them on the largest of their maxima, in order: out = sum_i 2^(m_i - m)
// o_i / sum_i 2^(m_i - m) l_i with m = max m_i. Bound by the launch and the latency of its loads:
// 5.7 us for 320 rows of 3 to 9 pieces, 12.4 us for 4096 rows of 17 (36 MB, 2.9 TB/s).
template <typename T, int D, int WPR>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(JoinArgs a)
{
    constexpr int E = D / 64;
    __shared__ float part[WPR > 1 ? kJoinWaves : 1][D];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int heads = a.heads * a.per, n_tokens = a.side[0].s.n_tokens;
    const int64_t x64 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kJoinWaves / WPR) + wave / WPR;
    if (x64 >= (int64_t)n_tokens * heads) return;   // all waves of a row together
    const int x = (int)x64, i = x / heads, hq = x % heads, h = hq / a.per;
    const int b = __builtin_amdgcn_readfirstlane(find_seq(a.side[0].s, i));
    const Rows r = rows_of(a.side[0].s, b);
    if (i < r.begin || i >= r.end) return;          // a row of no sequence stays as it was
    Acc<E> acc;
    const int64_t row = (int64_t)i * a.per + hq % a.per, rows = (int64_t)n_tokens * a.per;
    if (a.sides == 2)
        add_side<E, WPR>(acc, a.side[1], 0, (int)row, a.side[1].s.fixed_len, h, row, rows);
    if (!add_side<E, WPR>(acc, a.side[0], b, (i - r.begin) * a.per + hq % a.per,
                          len_of(a.side[0].s, b), h, row, rows))
        return;
    if constexpr (WPR > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) part[wave][lane * E + e] = acc.o[e];
        __syncthreads();
        if (wave % WPR) return;
#pragma unroll
        for (int k = 1; k < WPR; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) acc.o[e] += part[wave + k][lane * E + e];
    }
    const float inv = acc.l > 0.f ? 1.f / acc.l : 0.f;
    uint16_t *o = a.out + i * a.o_ts + hq * a.o_hs + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = (uint16_t)from_f32<T>(acc.o[e] * inv);
    if (a.lse && lane == 0)
        a.lse[x] = acc.l > 0.f ? (acc.m + log2f(acc.l)) * 0.6931471805599453f : -INFINITY;
}

// Many rows and one side: a block for each place where a run ends within an item, and head. The
// item is joined where its first run ends; other blocks have nothing to do.
template <typename T, int D>
__global__ __launch_bounds__(kJoinThreads) void join_items_kernel(JoinArgs a)
{
    constexpr int kLanes = D / 4;                   // of a row, four dimensions each
    const AttnSide &d = a.side[0];
    const int w = (int)(blockIdx.x / (unsigned)a.heads) + 1, h = (int)(blockIdx.x % (unsigned)a.heads);
    const int r0 = (int)blockIdx.y * kJoinRows;     // of the item, the block's rows
    const int U = d.starts[d.s.n_seqs], W = runs_of(d.workers, U), per = 16 * d.tiles16;
    if (w >= W) return;
    const int u = first_unit(w, W, U);
    SeqView by_unit = d.s;                          // the sequence of unit u, by the same search
    by_unit.cu = d.starts;
    const int b = __builtin_amdgcn_readfirstlane(find_seq(by_unit, u));
    const Rows rows = rows_of(d.s, b);
    const int along = units_along(len_of(d.s, b), d.starts[d.s.n_seqs + 1]), in_seq = u - d.starts[b];
    const int tile = in_seq / along, u0 = u - in_seq % along;
    if (u0 == u || run_of(u0, W, U) != w - 1) return;
    const int w1 = run_of(u0 + along - 1, W, U), row0 = tile * per;
    const int n_rows = min(min(per, r0 + kJoinRows), (rows.end - rows.begin) * a.per - row0);
    // slot 2w + 1 of the first run, 2w of the others
    const auto at = [&](int v, int r) { return ((int64_t)h * 2 * d.workers + 2 * v + (v == w - 1)) * per + r; };
    for (int r = r0 + threadIdx.x / kLanes; r < n_rows; r += kJoinThreads / kLanes) {
        const int e0 = threadIdx.x % kLanes * 4;
        float m = -INFINITY, l = 0.f;
        Floats<4> o = {};
        for (int v = w - 1; v <= w1; ++v) {
            const Floats<2> ml = *reinterpret_cast<const Floats<2> *>(d.slot_ml + at(v, r) * 2);
            const Floats<4> x = *reinterpret_cast<const Floats<4> *>(d.slot_o + at(v, r) * D + e0);
            const float top = fmaxf(m, ml.x[0]);
            const float f = m == top ? 1.f : exp2f(m - top), g = ml.x[0] == -INFINITY ? 0.f : exp2f(ml.x[0] - top);
            l = fmaf(g, ml.x[1], l * f);
            m = top;
#pragma unroll
            for (int e = 0; e < 4; ++e) o.x[e] = fmaf(g, x.x[e], o.x[e] * f);
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int tok = rows.begin + (row0 + r) / a.per, hq = h * a.per + (row0 + r) % a.per;
        const uint2 packed = {from_f32<T>(o.x[0] * inv) | from_f32<T>(o.x[1] * inv) << 16,
                              from_f32<T>(o.x[2] * inv) | from_f32<T>(o.x[3] * inv) << 16};
        *reinterpret_cast<uint2 *>(a.out + tok * a.o_ts + hq * a.o_hs + e0) = packed;
        if (a.lse && e0 == 0)
            a.lse[(int64_t)tok * a.heads * a.per + hq] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

template <typename T, int D>
void join_rows(const JoinArgs &a, hipStream_t stream)
{
    // Few rows have many pieces each: a block for each (64 rows over 131071 tokens 52 us in all, 59
    // with a wave for each; 320 rows 15.0 and 15.7; 1024 rows 25.1 and 23.9).
    const int64_t rows = (int64_t)a.side[0].s.n_tokens * a.heads * a.per;
    if (a.sides == 1 && rows > kManyRows) {
        const int ends = a.side[0].workers - 1;
        if (ends > 0) join_items_kernel<T, D><<<dim3((unsigned)(ends * a.heads), (unsigned)((16 * a.side[0].tiles16 + kJoinRows - 1) / kJoinRows)), kJoinThreads, 0, stream>>>(a);
    } else if (rows <= kFewRows)
        join_kernel<T, D, kJoinWaves><<<dim3((unsigned)rows), kJoinThreads, 0, stream>>>(a);
    else {
        // a dimension of a grid has less than 2^32 threads
        const int64_t blocks = (rows + kJoinWaves - 1) / kJoinWaves, across = blocks < kJoinAcross ? blocks : kJoinAcross;
        join_kernel<T, D, 1><<<dim3((unsigned)across, (unsigned)((blocks + across - 1) / across)), kJoinThreads, 0, stream>>>(a);
    }
}

template <typename T>
hipError_t join_typed(const JoinArgs &a, hipStream_t stream)
{
    if (a.dim == 64) join_rows<T, 64>(a, stream);
    else if (a.dim == 128) join_rows<T, 128>(a, stream);
    else join_rows<T, 256>(a, stream);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn(const AttnArgs &a, const AttnShape &x, hipStream_t stream)
{
    if (a.tree) {
        if (x.bf16) return x.nbits == 4 ? launch_attn_tree_bf16_4(a, x, stream) : launch_attn_tree_bf16_8(a, x, stream);
        return x.nbits == 4 ? launch_attn_tree_f16_4(a, x, stream) : launch_attn_tree_f16_8(a, x, stream);
    }
    if (x.bf16) return x.nbits == 4 ? launch_attn_bf16_4(a, x, stream) : launch_attn_bf16_8(a, x, stream);
    return x.nbits == 4 ? launch_attn_f16_4(a, x, stream) : launch_attn_f16_8(a, x, stream);
}

hipError_t launch_join(const JoinArgs &a, bool bf16, hipStream_t stream)
{
    return bf16 ? join_typed<Bf16>(a, stream) : join_typed<F16>(a, stream);
}

}  // namespace hqq
