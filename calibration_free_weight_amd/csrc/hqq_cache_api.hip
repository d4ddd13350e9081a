// hqq_cache_api.hip -- the C entry points of the quantized key/value cache: argument checks,
// the workspace plan of attention, and the launch sequences.
#include <cmath>

#include "hqq.h"
#include "hqq_cache_internal.h"
#include "hqq_internal.h"

namespace {

hqq_status refuse(const char *msg, hqq_status st = HQQ_ERR_ARG)
{
    hqq::report_error(st, msg);
    return st;
}

hqq_status done(hipError_t e)
{
    if (e != hipSuccess) return refuse(hipGetErrorString(e), HQQ_ERR_DEVICE);
    hqq::report_error(HQQ_OK, "");
    return HQQ_OK;
}

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

hqq_status check_cache(const hqq_cache *c)
{
    if (!c) return refuse("cache must be non-null");
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return refuse("cache: head_dim must be 64, 128 or 256");
    if (c->nbits != 4 && c->nbits != 8) return refuse("cache: nbits must be 4 or 8");
    if ((c->group_size != 32 && c->group_size != 64 && c->group_size != 128) || c->group_size > c->head_dim)
        return refuse("cache: group_size must be 32, 64 or 128 and at most head_dim");
    if (c->dtype != HQQ_F16 && c->dtype != HQQ_BF16) return refuse("cache: dtype must be HQQ_F16 or HQQ_BF16");
    if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)))
        return refuse("cache: page_size must be a power of two in [16, 4096]");
    if (c->n_heads < 1 || c->n_heads > 1024) return refuse("cache: n_heads must be in [1, 1024]");
    if (c->n_pages < 1 || c->n_pages > INT32_MAX) return refuse("cache: n_pages must be in [1, 2^31 - 1]");
    if (!c->k_codes || !c->v_codes || !c->k_meta || !c->v_meta)
        return refuse("cache: k_codes, v_codes, k_meta and v_meta must be non-null");
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_meta, 16) || !aligned(c->v_meta, 16))
        return refuse("cache: k_codes, v_codes, k_meta and v_meta must be 16-byte aligned");
    return HQQ_OK;
}

hqq_status check_seqs(const hqq_cache *c, const hqq_seqs *s)
{
    if (!s) return refuse("seqs must be non-null");
    if (s->n_seqs < 0 || s->n_seqs > hqq::kMaxSeqs) return refuse("seqs: n_seqs must be in [0, 4096]");
    if (s->n_tokens < 0 || s->n_tokens > (1 << 24)) return refuse("seqs: n_tokens must be in [0, 2^24]");
    if (s->n_tokens * c->n_heads > INT32_MAX) return refuse("seqs: n_tokens * n_heads must be below 2^31");
    if (s->max_pages < 0 || (int64_t)s->max_pages * c->page_size > (1 << 30))
        return refuse("seqs: max_pages * page_size must be in [0, 2^30]");
    if (s->n_seqs == 0 || s->n_tokens == 0) return HQQ_OK;
    if ((!s->table && s->max_pages > 0) || !s->lens) return refuse("seqs: table and lens must be non-null");
    if (!aligned(s->table, 4) || !aligned(s->lens, 4) || !aligned(s->cu_tokens, 4))
        return refuse("seqs: table, lens and cu_tokens must be 4-byte aligned");
    if (!s->cu_tokens && s->n_tokens % s->n_seqs != 0)
        return refuse("seqs: n_tokens must be a multiple of n_seqs without cu_tokens");
    return HQQ_OK;
}

// A tensor of rows: non-null, 16-byte rows.
hqq_status check_rows(const void *p, int64_t ts, int64_t hs, const char *null, const char *shape)
{
    if (!p) return refuse(null);
    if (!aligned(p, 16) || ts < 0 || hs < 0 || ts % 8 || hs % 8 || ts > (int64_t(1) << 36) ||
        hs > (int64_t(1) << 36))
        return refuse(shape);
    return HQQ_OK;
}

int log2_of(int x)
{
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

hqq::CacheView view_of(const hqq_cache *c)
{
    return hqq::CacheView{static_cast<uint8_t *>(c->k_codes), static_cast<uint8_t *>(c->v_codes),
                          static_cast<uint32_t *>(c->k_meta), static_cast<uint32_t *>(c->v_meta), c->n_heads};
}

hqq::SeqView view_of(const hqq_cache *c, const hqq_seqs *s)
{
    return hqq::SeqView{s->table,     s->lens, s->cu_tokens,         s->n_seqs,      s->max_pages, (int32_t)s->n_tokens, -1,
                        log2_of(c->page_size), (int32_t)c->n_pages};
}

hqq_status cache_rows(bool write, const hqq_cache *cache, const hqq_seqs *seqs, const void *k, int64_t k_ts,
                      int64_t k_hs, const void *v, int64_t v_ts, int64_t v_hs, void *stream)
{
    hqq_status st = check_cache(cache);
    if (st == HQQ_OK) st = check_seqs(cache, seqs);
    if (st != HQQ_OK) return st;
    if (seqs->n_seqs == 0 || seqs->n_tokens == 0) return done(hipSuccess);
    const char *null = "k and v must be non-null";
    const char *shape = "k and v must be 16-byte aligned, with strides that are multiples of 8 in [0, 2^36]";
    st = check_rows(k, k_ts, k_hs, null, shape);
    if (st == HQQ_OK) st = check_rows(v, v_ts, v_hs, null, shape);
    if (st != HQQ_OK) return st;
    // what the launch takes (a dimension of a grid has less than 2^32 threads)
    if (hqq::cache_rows_blocks(write, seqs->n_tokens, cache->n_heads, cache->head_dim) >= (1 << 24))
        return refuse("too many rows for one call", HQQ_ERR_UNSUPPORTED);
    auto rows = [](const void *p) { return static_cast<uint16_t *>(const_cast<void *>(p)); };
    const hqq::RowPtrs p{rows(k), rows(v), k_ts, k_hs, v_ts, v_hs};
    return done(hqq::launch_cache_rows(write, view_of(cache), view_of(cache, seqs), p, cache->head_dim,
                                       cache->nbits, cache->group_size, cache->dtype == HQQ_BF16,
                                       static_cast<hipStream_t>(stream)));
}

// ---- attention --------------------------------------------------------------------------------
constexpr float kLog2e = 1.44269504088896341f;

// How one side's work is cut, and where its partial results lie in the workspace.
struct SidePlan {
    int tiles16, workers, unit;
    size_t starts, slot_o, slot_ml, row_o, row_ml;      // offsets; row_* with two sides
};

struct Plan {
    SidePlan own, prefix;
    bool join;                  // pieces or two sides are put together; else no workspace
    size_t bytes;
};

// The longest side that one block takes alone: cutting it saves four steps at most, and
// joining the pieces costs a launch (sequences of 100 to 500 tokens, 64 of them: 12.0 us whole,
// 19.3 cut; one of 1000: 13.3 whole, 10.9 cut).
constexpr int64_t kWhole = 512;

// Query rows to a tile, in 16s, for `rows` rows of one head in n_seqs sequences of up to
// `longest` tokens. More rows to a tile widen the codes fewer times, and take longer for a step:
// where runs are short, smaller tiles on more of the GPU win. Measured in us with 8 heads of 128
// in 4 bits, tiles of 16, 32 and 128 rows:
//   500 rows x 4 over 500 tokens      18    19    31
//   16 x 4 over 4000                  20    22    -
//   8 x 64 x 4 over 2000              54    48    62
//   500 x 4 over 4000                 89    80    82
//   8 x 250 x 4 over 2000             189   156   128
// and with 4 heads of 256, tiles of 16, 32 and 64 rows:
//   16 x 5 x 4 over 800 to 2900       33    36    40
//   64 x 5 x 4 over 4000              184   146   180
//   500 x 4 over 500                  21    29    41
//   8 x 250 x 4 over 2000             192   185   148
// The limits are units of 128 tokens of 16 rows, to a run. (Tiles of 64 rows of heads of up to
// 128 were between the others or behind both, and are not there.) One tile for all: rows are the
// sequences' average and `longest` is the table's width, for lengths are not known here. A chunk
// among single rows, or short sequences under a wide table, get what their average would.
int tiles_for(int64_t rows, int n_seqs, int64_t longest, const hqq_cache *c)
{
    const int64_t each = (rows + n_seqs - 1) / n_seqs, few = (each + 15) / 16;
    if (few == 1) return 1;
    const int64_t units = few * n_seqs * ((longest + hqq::kStep - 1) / hqq::kStep);
    const int64_t blocks = 256 * hqq::blocks_per_cu(1, c->head_dim, c->nbits), runs = blocks / c->n_heads > 0 ? blocks / c->n_heads : 1;
    if (c->head_dim == 256) {
        // the first limit is of one tile of 32 for a sequence: smaller ones read the cache twice
        if (units <= (few == 2 ? 6 : 31) * runs) return 1;
        return few == 2 ? 2 : 4;
    }
    // sequences that are not cut are spread the better the more tiles there are
    if (units <= (longest <= kWhole ? 8 : 3) * runs) return 1;
    if (units <= 30 * runs) return 2;
    // what a step of a tile of 128 rows takes, to one of 32: 29 to 8
    return (each + 127) / 128 * 29 < (each + 31) / 32 * 8 ? 8 : 2;
}

Plan plan_of(const hqq_cache *c, const hqq_seqs *s, int n_q_heads, int64_t prefix_len)
{
    const int per = n_q_heads / c->n_heads;
    const int64_t rows = s->n_tokens * per;
    Plan p{};
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t was = at;
        at += (n + 255) / 256 * 256;
        return was;
    };
    auto cut = [&](int tiles16, int n_seqs, int64_t longest) {
        SidePlan x{};
        x.tiles16 = tiles16;
        const int64_t step = hqq::kStep;
        x.unit = (int)(longest <= kWhole ? (longest + step) / step * step : step);
        // no more than the 256 CUs hold at once (a block more would take as long again), nor than
        // the units that there can be
        const int64_t blocks = 256 * hqq::blocks_per_cu(x.tiles16, c->head_dim, c->nbits);
        const int64_t units = (rows / (16 * x.tiles16) + n_seqs) * hqq::units_along((int32_t)longest, x.unit);
        const int64_t each = blocks / c->n_heads > 0 ? blocks / c->n_heads : 1;
        x.workers = (int)(each < units ? each : units);
        return x;
    };
    auto lay = [&](SidePlan &x, int n_seqs) {
        const size_t slots = (size_t)c->n_heads * 2 * x.workers * 16 * x.tiles16;
        x.starts = take(4 * ((size_t)n_seqs + 2));
        x.slot_o = take(slots * c->head_dim * 4);
        x.slot_ml = take(slots * 8);
        if (prefix_len > 0) {
            x.row_o = take((size_t)c->n_heads * rows * c->head_dim * 4);
            x.row_ml = take((size_t)c->n_heads * rows * 8);
        }
    };
    const int64_t longest = (int64_t)s->max_pages * c->page_size;
    p.own = cut(tiles_for(rows, s->n_seqs, longest, c), s->n_seqs, longest);
    if (prefix_len > 0) {
        p.prefix = cut(tiles_for(rows, 1, prefix_len, c), 1, prefix_len);
        // Short sequences behind a prefix go in its launch, in its larger tiles, while the GPU
        // holds the blocks of both: few steps in mostly empty tiles beside the prefix's cost
        // less than a launch of their own (25 sequences of a token, 16 heads of 256, a prefix of
        // 1544: 28 us so, 37 with two).
        const SidePlan with = cut(p.prefix.tiles16, s->n_seqs, longest);
        const int64_t both = (int64_t)(with.workers + p.prefix.workers) * c->n_heads;
        if (longest <= kWhole && both <= 256 * hqq::blocks_per_cu(with.tiles16, c->head_dim, c->nbits)) p.own = with;
    }
    lay(p.own, s->n_seqs);
    if (prefix_len > 0) lay(p.prefix, 1);
    p.join = prefix_len > 0 || longest > p.own.unit;
    p.bytes = p.join ? at : 0;
    return p;
}

// Checks that the sizes allow a plan; HQQ_OK with *empty set when there is nothing to do.
hqq_status check_plan(const hqq_cache *c, const hqq_seqs *s, int n_q_heads, int64_t prefix_len, bool *empty)
{
    hqq_status st = check_cache(c);
    if (st == HQQ_OK) st = check_seqs(c, s);
    if (st != HQQ_OK) return st;
    if (n_q_heads < 1 || n_q_heads % c->n_heads != 0)
        return refuse("n_q_heads must be a positive multiple of the cache's n_heads");
    if (n_q_heads > (1 << 20) || s->n_tokens * n_q_heads > (1 << 30))
        return refuse("n_q_heads must be at most 2^20, and n_tokens * n_q_heads at most 2^30");
    if (prefix_len < 0 || prefix_len > (1 << 30)) return refuse("prefix_len must be in [0, 2^30]");
    *empty = s->n_seqs == 0 || s->n_tokens == 0;
    if (*empty) return HQQ_OK;
    // units of work are counted in 32 bits
    const int64_t tiles = s->n_tokens * (n_q_heads / c->n_heads) / 16 + s->n_seqs;
    const int64_t longest = (int64_t)s->max_pages * c->page_size;
    const int64_t far = longest > prefix_len ? longest : prefix_len;
    if (tiles > INT32_MAX / (far / hqq::kStep + 1))
        return refuse("too many rows over too long sequences for one call", HQQ_ERR_UNSUPPORTED);
    return HQQ_OK;
}

hqq::AttnSide side_at(const hqq::SeqView &s, const SidePlan &p, char *ws, bool two, bool causal)
{
    auto f = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
    return hqq::AttnSide{s, reinterpret_cast<int32_t *>(ws + p.starts), f(p.slot_o), f(p.slot_ml),
                         two ? f(p.row_o) : nullptr, two ? f(p.row_ml) : nullptr,
                         p.workers, p.unit, p.tiles16, causal};
}

}  // namespace

extern "C" {

hqq_status hqq_cache_write(const hqq_cache *cache, const hqq_seqs *seqs, const void *k, int64_t k_token_stride,
                           int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                           void *stream)
{
    return cache_rows(true, cache, seqs, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, stream);
}

hqq_status hqq_cache_read(const hqq_cache *cache, const hqq_seqs *seqs, void *k, int64_t k_token_stride,
                          int64_t k_head_stride, void *v, int64_t v_token_stride, int64_t v_head_stride,
                          void *stream)
{
    return cache_rows(false, cache, seqs, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, stream);
}

size_t hqq_cache_attention_workspace(const hqq_cache *cache, const hqq_seqs *seqs, int n_q_heads, int64_t prefix_len)
{
    bool empty;
    if (check_plan(cache, seqs, n_q_heads, prefix_len, &empty) != HQQ_OK) return 0;
    hqq::report_error(HQQ_OK, "");
    return empty ? 0 : plan_of(cache, seqs, n_q_heads, prefix_len).bytes;
}

hqq_status hqq_cache_attention_prefix(const hqq_cache *cache, const hqq_seqs *seqs, const int32_t *prefix_pages,
                                      int n_prefix_pages, int64_t prefix_len, const void *q, int64_t q_token_stride,
                                      int64_t q_head_stride, int n_q_heads, float scale, void *out,
                                      int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                                      size_t workspace_bytes, void *stream)
{
    bool empty;
    hqq_status st = check_plan(cache, seqs, n_q_heads, prefix_len, &empty);
    if (st != HQQ_OK) return st;
    if (n_prefix_pages < 0 || (int64_t)n_prefix_pages * cache->page_size > (1 << 30) ||
        prefix_len > (int64_t)n_prefix_pages * cache->page_size)
        return refuse("prefix_len must be at most n_prefix_pages * page_size, and that at most 2^30");
    if (prefix_len > 0 && (!prefix_pages || !aligned(prefix_pages, 4)))
        return refuse("prefix_pages must be non-null and 4-byte aligned");
    if (!std::isfinite(scale * kLog2e)) return refuse("scale must be finite, and times log2(e) too");
    if (empty) return done(hipSuccess);
    st = check_rows(q, q_token_stride, q_head_stride, "q must be non-null",
                    "q must be 16-byte aligned, with strides that are multiples of 8 in [0, 2^36]");
    if (st == HQQ_OK)
        st = check_rows(out, out_token_stride, out_head_stride, "out must be non-null",
                        "out must be 16-byte aligned, with strides that are multiples of 8 in [0, 2^36]");
    if (st != HQQ_OK) return st;
    if (lse && !aligned(lse, 4)) return refuse("lse must be 4-byte aligned");
    const Plan p = plan_of(cache, seqs, n_q_heads, prefix_len);
    if (p.join && (!workspace || workspace_bytes < p.bytes))
        return refuse("workspace missing or smaller than hqq_cache_attention_workspace()", HQQ_ERR_WORKSPACE);
    if (p.join && !aligned(workspace, 256)) return refuse("workspace must be 256-byte aligned");
    char *ws = static_cast<char *>(workspace);
    const bool shared = prefix_len > 0;
    const hipStream_t str = static_cast<hipStream_t>(stream);
    const hqq::AttnShape shape{cache->head_dim, cache->nbits, cache->group_size, cache->dtype == HQQ_BF16};
    hqq::AttnArgs a{};
    a.c = view_of(cache);
    a.side[0] = side_at(view_of(cache, seqs), p.own, ws, shared, true);
    if (!p.join) a.side[0].starts = nullptr;
    a.sides = 1;
    a.q = static_cast<const uint16_t *>(q);
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.o_ts = out_token_stride;
    a.o_hs = out_head_stride;
    a.per = n_q_heads / cache->n_heads;
    a.scale = scale * kLog2e;
    hqq::JoinArgs j{{a.side[0], {}}, 1, a.out, lse, a.o_ts, a.o_hs, a.per, cache->n_heads, cache->head_dim};
    hipError_t e = hipSuccess;
    if (shared) {
        // the prefix is one sequence whose rows are all rows of the call
        const hqq::SeqView all{prefix_pages, nullptr, nullptr, 1, n_prefix_pages, (int32_t)seqs->n_tokens,
                               (int32_t)prefix_len, log2_of(cache->page_size), (int32_t)cache->n_pages};
        j.side[1] = side_at(all, p.prefix, ws, true, false);
        j.sides = 2;
        if (p.own.tiles16 == p.prefix.tiles16) {
            a.side[1] = j.side[1];          // one launch for both
            a.sides = 2;
        } else {
            hqq::AttnArgs first = a;
            first.side[0] = j.side[1];
            e = hqq::launch_attn(first, shape, str);
        }
    }
    if (e == hipSuccess) e = hqq::launch_attn(a, shape, str);
    if (e == hipSuccess && p.join) e = hqq::launch_join(j, shape.bf16, str);
    return done(e);
}

hqq_status hqq_cache_attention(const hqq_cache *cache, const hqq_seqs *seqs, const void *q, int64_t q_token_stride,
                               int64_t q_head_stride, int n_q_heads, float scale, void *out,
                               int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                               size_t workspace_bytes, void *stream)
{
    return hqq_cache_attention_prefix(cache, seqs, nullptr, 0, 0, q, q_token_stride, q_head_stride, n_q_heads, scale,
                                      out, out_token_stride, out_head_stride, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
