// hqq_keep.hip -- accepted tokens moved to the places behind what a cache held before the call,
// in the caches of all layers (gfx950).
#include "hqq_cache_internal.h"

namespace hqq {
namespace {

constexpr int kThreads = 256;

// A sixteenth of a token's codes. Vectors, which stay in registers: of an array of four words the
// compiler keeps two in LDS on their way.
template <int BYTES>
struct Piece {
    typedef uint32_t Type __attribute__((ext_vector_type(BYTES / 4)));
};
template <>
struct Piece<2> {
    using Type = uint16_t;
};
template <>
struct Piece<4> {
    using Type = uint32_t;
};

// A wave has one head of one sequence in one layer. A row of 16 lanes moves a token: lane u has the
// u-th sixteenth of its key and row u of its value, lanes 0 to 7 the grids of keys, 8 to 15 those
// of values. A list ascends, so number k comes from place k or behind: four tokens at a time are
// read, then written, and no token that is still to be read lies where one has been written.
// Bound by latency: loads that wait for each other (lengths and list, pages, codes), then stores. 5 of
// 26 tokens in 32 layers of 8 heads of 128, 4 bits: 4.6 us; of 64 sequences 1 to 7 of 32, 16 layers, 8
// bits, 14 MB: 9.1 us, 1.5 TB/s (eight or sixteen tokens at a time take as long).
template <int S>                // bytes of a sixteenth of a token's codes
__global__ __launch_bounds__(kThreads) void keep_kernel(KeepArgs a)
{
    using Code = typename Piece<S>::Type;
    const int lane = threadIdx.x & 63, u = lane & 15;
    const unsigned wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + threadIdx.x / 64);
    const unsigned b = wave / (unsigned)a.heads, h = wave - b * a.heads;
    if (b >= (unsigned)a.s.n_seqs) return;
    const Rows r = rows_of(a.s, (int)b);
    const int len = len_of(a.s, (int)b), n = r.end - r.begin, first = len - n;
    const int32_t *kept = a.kept + (int64_t)b * a.max_kept;
    // how many entries ascend, from the first
    int m = 0;
    for (int k0 = 0; k0 < a.max_kept && m == k0; k0 += 64) {
        const int k = k0 + lane;
        const int j = k < a.max_kept ? kept[k] : -1, before = k > 0 && k < a.max_kept ? kept[k - 1] : -1;
        const uint64_t ok = __ballot(j > before && j < n && j >= 0);
        m += ok == ~0ull ? 64 : (int)__builtin_ctzll(~ok);
    }
    if (a.lens_out && blockIdx.y == 0 && h == 0 && lane == 0) a.lens_out[b] = max(first + m, 0);
    uint8_t *const *layer = a.layers[blockIdx.y].part;
    const auto slot = [&](int pos) {            // of a token: page and place in it, or -1
        const int p = page_of(a.s, (int)b, pos);
        return p < 0 ? -1 : (((int64_t)p * a.heads + h) << a.s.page_shift) + (pos & ((1 << a.s.page_shift) - 1));
    };
    uint32_t *meta = reinterpret_cast<uint32_t *>(layer[u < 8 ? 2 : 3]);
    const bool grid = (u & 7) < a.groups;
    const auto value_at = [&](int64_t at) { return ((at >> 2) * 64 + u * 4 + (at & 3)) * S; };
    for (int k0 = 0; k0 < m; k0 += 4) {
        const int k = k0 + lane / 16, j = k < m ? kept[k] : k;
        const int64_t from = j != k ? slot(first + j) : -1, to = j != k ? slot(first + k) : -1;
        const bool move = from >= 0 && to >= 0;
        Code key{}, value{};
        uint32_t word = 0;
        if (move) {
            key = *reinterpret_cast<const Code *>(layer[0] + (from * 16 + u) * S);
            value = *reinterpret_cast<const Code *>(layer[1] + value_at(from));
            if (grid) word = meta[from * a.groups + (u & 7)];
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");    // a place that is written may have been another lane's to read
        if (move) {
            *reinterpret_cast<Code *>(layer[0] + (to * 16 + u) * S) = key;
            *reinterpret_cast<Code *>(layer[1] + value_at(to)) = value;
            if (grid) meta[to * a.groups + (u & 7)] = word;
        }
    }
}

}  // namespace

hipError_t launch_keep(const KeepArgs &a, int n_layers, int dim, int nbits, hipStream_t stream)
{
    const int waves = kThreads / 64;
    const dim3 grid((unsigned)(((int64_t)a.s.n_seqs * a.heads + waves - 1) / waves), (unsigned)n_layers);
    const int s = dim * nbits / 128;
    if (s == 2) keep_kernel<2><<<grid, kThreads, 0, stream>>>(a);
    else if (s == 4) keep_kernel<4><<<grid, kThreads, 0, stream>>>(a);
    else if (s == 8) keep_kernel<8><<<grid, kThreads, 0, stream>>>(a);
    else keep_kernel<16><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace hqq
