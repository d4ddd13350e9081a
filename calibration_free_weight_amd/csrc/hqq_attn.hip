// hqq_attn.hip -- attention over the quantized cache: the choice of the kernel, and the
// joining of an item's pieces.
#include "hqq_cache_internal.h"

namespace hqq {
namespace {

constexpr int kJoinThreads = 256;

template <typename T, int E>
struct Acc {                    // a row's result so far; lane holds E dimensions
    float m = -INFINITY, l = 0.f, o[E] = {};
};

// Adds 64 pieces at a time: lane k has the maximum m and sum l of piece k, whose output is
// at o + off(k) * D.
template <typename T, int E, typename Off>
__device__ __forceinline__ void add_pieces(Acc<T, E> &acc, int n, float m, float l, const float *o, Off off)
{
    const int lane = threadIdx.x & 63;
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
    for (int k = 0; k < n; ++k) {
        const float fk = __shfl(f, k);
        if (fk == 0.f) continue;            // nothing was seen there, or nothing written
        const float *x = o + off(k) * (64 * E) + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) acc.o[e] = fmaf(fk, x[e], acc.o[e]);
    }
}

// Adds what one side found for a row; false if the item is whole and its result elsewhere.
template <typename T, int E>
__device__ __forceinline__ bool add_side(Acc<T, E> &acc, const AttnSide &d, int n_seqs, int b, int row_in_item,
                                         int along, int h, int64_t row, int64_t rows)
{
    const int lane = threadIdx.x & 63, per = 16 * d.tiles16;
    if (along == 0) return true;
    const int U = d.starts[n_seqs], W = d.workers;
    const int u0 = d.starts[b] + row_in_item / per * along;
    const int w0 = worker_of(u0, W, U), w1 = worker_of(u0 + along - 1, W, U);
    if (w0 == w1) {
        if (!d.row_o) return false;
        const int64_t at = h * rows + row;
        const float m = lane == 0 ? d.row_ml[at * 2] : -INFINITY, l = lane == 0 ? d.row_ml[at * 2 + 1] : 0.f;
        add_pieces<T, E>(acc, 1, m, l, d.row_o, [&](int) { return at; });
        return true;
    }
    for (int wb = w0; wb <= w1; wb += 64) {
        const int w = wb + lane;
        const auto at = [&](int v) { return ((int64_t)h * 2 * W + 2 * v + (v == w0)) * per + row_in_item % per; };
        const bool have = w <= w1 && first_unit(w, W, U) < first_unit(w + 1, W, U);
        const float m = have ? d.slot_ml[at(w) * 2] : -INFINITY, l = have ? d.slot_ml[at(w) * 2 + 1] : 0.f;
        add_pieces<T, E>(acc, min(64, w1 - wb + 1), m, l, d.slot_o, [&](int k) { return at(wb + k); });
    }
    return true;
}

// A wave per query row: finds the pieces of its item on each side by the rule that dealt them
// out, and adds them on the largest of their maxima, in order.
template <typename T, int D>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(JoinArgs a)
{
    constexpr int E = D / 64;
    const int64_t x = (int64_t)blockIdx.x * (kJoinThreads / 64) + (threadIdx.x >> 6);
    const int heads = a.heads * a.per, lane = threadIdx.x & 63;
    const int i = (int)(x / heads), hq = (int)(x % heads), h = hq / a.per;
    if (i >= a.s.n_tokens) return;
    const int b = seq_at(a.s, i);
    const Rows r = rows_of(a.s, b);
    if (i < r.begin || i >= r.end) return;          // a row of no sequence stays as it was
    Acc<T, E> acc;
    const int64_t row = (int64_t)i * a.per + hq % a.per, rows = (int64_t)a.s.n_tokens * a.per;
    if (a.prefix.starts)
        add_side<T, E>(acc, a.prefix, 1, 0, (int)row, units_along(a.prefix_len), h, row, rows);
    if (!add_side<T, E>(acc, a.side, a.s.n_seqs, b, (i - r.begin) * a.per + hq % a.per,
                        units_along(len_of(a.s, b)), h, row, rows))
        return;
    const float inv = acc.l > 0.f ? 1.f / acc.l : 0.f;
    uint16_t *o = a.out + i * a.o_ts + hq * a.o_hs + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = (uint16_t)from_f32<T>(acc.o[e] * inv);
    if (a.lse && lane == 0)
        a.lse[x] = acc.l > 0.f ? (acc.m + log2f(acc.l)) * 0.6931471805599453f : -INFINITY;
}

template <typename T>
hipError_t join_typed(const JoinArgs &a, hipStream_t stream)
{
    const int64_t rows = (int64_t)a.s.n_tokens * a.heads * a.per;
    const dim3 grid((unsigned)((rows + kJoinThreads / 64 - 1) / (kJoinThreads / 64)));
    if (a.dim == 64) join_kernel<T, 64><<<grid, kJoinThreads, 0, stream>>>(a);
    else if (a.dim == 128) join_kernel<T, 128><<<grid, kJoinThreads, 0, stream>>>(a);
    else join_kernel<T, 256><<<grid, kJoinThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn(const AttnArgs &a, const AttnShape &x, hipStream_t stream)
{
    if (x.bf16) return x.nbits == 4 ? launch_attn_bf16_4(a, x, stream) : launch_attn_bf16_8(a, x, stream);
    return x.nbits == 4 ? launch_attn_f16_4(a, x, stream) : launch_attn_f16_8(a, x, stream);
}

hipError_t launch_join(const JoinArgs &a, bool bf16, hipStream_t stream)
{
    return bf16 ? join_typed<Bf16>(a, stream) : join_typed<F16>(a, stream);
}

}  // namespace hqq
