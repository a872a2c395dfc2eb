// fa_packed.cuh — what the packed attention's forward and backward share: the
// sequences of a batch, and the order in which its work is taken.
#pragma once

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

// Sequences packed one behind the other: queries cu_q[b] .. cu_q[b + 1] - 1, keys
// cu_k[b] .. (device arrays of B + 1 offsets).
struct PackedSeqs {
    const int *cu_q, *cu_k;
    int B, total_q, total_k, max_q, max_k;
};

// Sequence b: its first query and key, and their numbers. False (and an empty
// sequence) where the offsets are no valid partition or the lengths pass the
// call's bounds.
struct PackedSeq {
    int q0, n, k0, m;
};
__device__ __forceinline__ bool packed_seq(const PackedSeqs& p, int b, PackedSeq& s) {
    const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
    const bool ok = 0 <= q0 && q0 <= q1 && q1 <= p.total_q && q1 - q0 <= p.max_q && 0 <= k0 && k0 <= k1 &&
                    k1 <= p.total_k && k1 - k0 <= p.max_k;
    s.q0 = ok ? q0 : 0;
    s.n = ok ? q1 - q0 : 0;
    s.k0 = ok ? k0 : 0;
    s.m = ok ? k1 - k0 : 0;
    return ok;
}

// Sequence b has n units at levels a .. a + n - 1, one each (runs(b, a, n); n = 0:
// none); a unit's time grows with its level. Picks the unit of rank r when they are
// taken from the highest level down, so that the longest start first whatever the
// sequences' lengths and order are; by bisection over the levels, a few dozen
// instructions each, without a list in memory or a launch that makes one. Called by
// a whole warp; false where there is no such unit.
template <typename F>
__device__ __forceinline__ bool packed_pick(int B, int r, int lane, F&& runs, int& b, int& level) {
    int a0 = 0, n0 = 0;  // of the first 32 sequences; the others are read again in each round
    if (lane < B) runs(lane, a0, n0);
    auto each = [&](auto&& f) {
        f(lane, a0, n0);
        for (int c = 32; c < B; c += 32) {
            int a = 0, n = 0;
            if (c + lane < B) runs(c + lane, a, n);
            f(c + lane, a, n);
        }
    };
    int lo = 0x7fffffff, hi = -0x7fffffff, all = 0;
    each([&](int, int a, int n) {
        if (n > 0) lo = min(lo, a), hi = max(hi, a + n - 1), all += n;
    });
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    all = __reduce_add_sync(0xffffffffu, all);
    if (r >= all) return false;
    auto from = [&](int at) {  // units at this level or above
        int k = 0;
        each([&](int, int a, int n) { k += min(max(a + n - at, 0), n); });
        return __reduce_add_sync(0xffffffffu, k);
    };
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (from(mid) > r) lo = mid;
        else hi = mid - 1;
    }
    level = lo;
    int at = r - from(lo + 1);
    b = -1;
    each([&](int i, int a, int n) {
        const bool here = n > 0 && a <= lo && lo < a + n;
        const unsigned who = __ballot_sync(0xffffffffu, here);
        const unsigned mine = __ballot_sync(0xffffffffu, here && __popc(who & low_bits(lane)) == at);
        if (b < 0 && mine) b = (i - lane) + __ffs(mine) - 1;
        at -= __popc(who);
    });
    return b >= 0;
}

}  // namespace fa
