// hqq_rotary.h -- which numbers of a call's tensors a thread of the rotary kernel has. The functions
// here compile for the host too, where the tests count what they name.
#pragma once

#include <stdint.h>

#include "hqq_cache.h"

namespace hqq {

// A unit is eight pairs, or eight dimensions that are copied; a head ends with units of one, where
// these do not go into eights.
struct RotaryHeads {            // of one tensor
    int32_t heads;
    int32_t copied;             // dimensions behind those of the pairs; none in place, where they stay
    int32_t per_head;           // units
};

HQQ_HD RotaryHeads rotary_heads(int32_t heads, int32_t pairs, int32_t copied)
{
    return RotaryHeads{heads, copied, pairs / 8 + pairs % 8 + copied / 8 + copied % 8};
}

// Where a unit lies: its first numbers, and the second of pairs.
struct RotaryUnit {
    int32_t tensor, head;
    int32_t d0, d1, pair;       // pair: the first; or -1: copied
    bool wide;
};

// The u-th unit of a token, whose first `before` units are tensor 0's.
template <bool NEIGHBOURS>
HQQ_HD RotaryUnit rotary_unit(const RotaryHeads (&x)[2], int32_t pairs, int32_t before, int32_t u)
{
    RotaryUnit r;
    r.tensor = u >= before;
    u -= r.tensor ? before : 0;
    const int32_t per_head = r.tensor ? x[1].per_head : x[0].per_head, copied = r.tensor ? x[1].copied : x[0].copied;
    r.head = (int32_t)((uint32_t)u / (uint32_t)per_head);
    u -= r.head * per_head;
    // eights that are turned and copied, then ones
    const int32_t turned8 = pairs >> 3, copied8 = copied >> 3, turned1 = pairs & 7;
    r.wide = u < turned8 + copied8;
    bool turn = u < turned8;
    int32_t first = 8 * u;                                  // pair, or dimension copied
    if (!r.wide) {
        u -= turned8 + copied8;
        turn = u < turned1;
        first = turn ? 8 * turned8 + u : 8 * copied8 + u - turned1;
    } else if (!turn) {
        first -= 8 * turned8;
    }
    if (turn) {
        r.d0 = NEIGHBOURS ? 2 * first : first;
        r.d1 = NEIGHBOURS ? r.d0 + (r.wide ? 8 : 1) : first + pairs;
        r.pair = first;
    } else {
        r.d0 = r.d1 = 2 * pairs + first;
        r.pair = -1;
    }
    return r;
}

// Whether rows of `width` numbers of n tokens and `heads` heads, these strides apart, share any.
inline bool rows_meet(int64_t n, int64_t heads, int64_t token_stride, int64_t head_stride, int64_t width)
{
    if ((n > 1 && token_stride < width) || (heads > 1 && head_stride < width)) return true;
    // in order of their tokens, or of their heads: what layouts are as a rule
    if (n <= 1 || heads <= 1 || token_stride >= (heads - 1) * head_stride + width || head_stride >= (n - 1) * token_stride + width)
        return false;
    // else a row of one token and one of another, some heads before it, the nearest two for each number of them
    const bool by_head = heads <= n;
    const int64_t few = by_head ? heads : n, many = by_head ? n : heads;
    const int64_t step = by_head ? head_stride : token_stride, other = by_head ? token_stride : head_stride;
    for (int64_t i = 1; i < few; ++i) {
        const int64_t k = i * step / other, rest = i * step - k * other;
        if ((k < many && rest < width) || (k + 1 < many && other - rest < width)) return true;
        if (k >= many) break;
    }
    return false;
}

}  // namespace hqq
