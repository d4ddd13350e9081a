// hqq_cache.h -- the quantized key/value cache as the kernels see it: where a token's codes
// and grids lie, and which token a row of a call is. The functions here hold every index that
// comes from device arrays (page tables, lengths, row offsets) within its buffer whatever
// those arrays hold; they compile for the host too, where the tests run them on bad tables.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define HQQ_HD __host__ __device__ __forceinline__
#else
#define HQQ_HD inline
#endif

namespace hqq {

constexpr int kMaxSeqs = 4096;

// Sequences of a call (hqq_seqs), with what bounds their entries.
struct SeqView {
    const int32_t *table, *lens, *cu;
    int32_t n_seqs, max_pages;
    int32_t n_tokens;
    int32_t fixed_len;          // >= 0: every sequence has this length and `lens` is not read
    int32_t page_shift;         // log2(page_size)
    int32_t n_pages;
};

struct Rows {
    int32_t begin, end;         // rows of the call's tensors, 0 <= begin <= end <= n_tokens
};

HQQ_HD int32_t clamp_i32(int32_t x, int32_t lo, int32_t hi)
{
    return x < lo ? lo : (x > hi ? hi : x);
}

HQQ_HD Rows rows_of(const SeqView &s, int32_t b)
{
    Rows r;
    if (s.cu) {
        r.begin = clamp_i32(s.cu[b], 0, s.n_tokens);
        r.end = clamp_i32(s.cu[b + 1], r.begin, s.n_tokens);
    } else {
        const int32_t each = s.n_tokens / s.n_seqs;
        r.begin = b * each;
        r.end = r.begin + each;
    }
    return r;
}

// Whether the rows of sequence b + 1 would begin before those of b: a call where any do attends
// for none. (Else the sequences' rows are at most n_tokens together, and so is what is counted
// from them.)
HQQ_HD bool falls_at(const SeqView &s, int32_t b)
{
    return s.cu && clamp_i32(s.cu[b + 1], 0, s.n_tokens) < clamp_i32(s.cu[b], 0, s.n_tokens);
}

HQQ_HD int32_t len_of(const SeqView &s, int32_t b)
{
    // max_pages << page_shift is below 2^31 (checked by the call)
    return s.fixed_len >= 0 ? s.fixed_len
                            : clamp_i32(s.lens[b], 0, s.max_pages << s.page_shift);
}

// The page of position `pos` of sequence b, or -1 when it is not in the cache.
HQQ_HD int32_t page_of(const SeqView &s, int32_t b, int32_t pos)
{
    if (pos < 0 || (pos >> s.page_shift) >= s.max_pages) return -1;
    const int32_t p = s.table[(int64_t)b * s.max_pages + (pos >> s.page_shift)];
    return (uint32_t)p < (uint32_t)s.n_pages ? p : -1;
}

// The last sequence whose first row is at or before `row` (0 when there is none): the one
// that holds the row if any does. n_seqs >= 1.
HQQ_HD int32_t seq_at(const SeqView &s, int32_t row)
{
    if (!s.cu) {
        const int32_t each = s.n_tokens / s.n_seqs;
        return each > 0 ? clamp_i32(row / each, 0, s.n_seqs - 1) : 0;
    }
    int32_t lo = 0, hi = s.n_seqs;          // cu[lo] <= row < cu[hi], if cu ascends from 0
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (s.cu[mid] <= row) lo = mid; else hi = mid;
    }
    return lo;
}

// Byte offsets within the page of one head (row = head_dim * nbits / 8 bytes of codes).
// Keys: unit (a, m) of token t of the page. Values: row r of token t.
HQQ_HD int32_t k_unit_at(int32_t t, int32_t a, int32_t m, int32_t dim, int32_t nbits)
{
    return t * (dim * nbits / 8) + (a * (dim / 32) + m) * nbits;
}

HQQ_HD int32_t v_row_at(int32_t t, int32_t r, int32_t dim, int32_t nbits)
{
    return (((t >> 2) * 16 + r) * 4 + (t & 3)) * (dim * nbits / 128);
}

// ---- attention: units of work and who does them ---------------------------------------------
// A key/value head's work is a list of items, one per sequence and tile of query rows, each of
// ceil(length / unit) units along its sequence, one at least (an item that sees nothing still
// writes its rows). The units of all items, end to end, are dealt in equal runs to as many
// workers as there are, or as there are units: one long sequence among short ones is spread as
// evenly as a uniform batch.
constexpr int kStep = 128;      // tokens of a block's step; a unit is a multiple of it

HQQ_HD int32_t units_along(int32_t len, int32_t unit)
{
    return len <= unit ? 1 : (int32_t)(((uint32_t)len + (uint32_t)unit - 1) / (uint32_t)unit);
}

HQQ_HD int32_t tiles_of(int32_t rows, int32_t rows_per)
{
    return (int32_t)(((uint32_t)rows + (uint32_t)rows_per - 1) / (uint32_t)rows_per);
}

HQQ_HD int32_t runs_of(int32_t workers, int32_t units) { return workers < units ? workers : units; }

// First unit of run w of W over U units; run that has unit u. 1 <= W <= U: no run is empty,
// the first U % W have one unit more than the others.
HQQ_HD int32_t first_unit(int32_t w, int32_t W, int32_t U)
{
    const int32_t each = (int32_t)((uint32_t)U / (uint32_t)W), more = U - each * W;
    return w * each + (w < more ? w : more);
}

HQQ_HD int32_t run_of(int32_t u, int32_t W, int32_t U)
{
    const int32_t each = (int32_t)((uint32_t)U / (uint32_t)W), more = U - each * W;
    const int32_t longer = more * (each + 1);   // units of the longer runs; at most U
    return u < longer ? (int32_t)((uint32_t)u / (uint32_t)(each + 1))
                      : more + (int32_t)((uint32_t)(u - longer) / (uint32_t)each);
}

}  // namespace hqq
