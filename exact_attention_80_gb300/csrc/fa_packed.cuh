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

// First padded row of sequence b, whose first query is q0: a multiple of 64, with room
// for its queries in whole steps of 64 before the next sequence's.
__host__ __device__ __forceinline__ long long pad_row(int q0, int b) { return (q0 & ~63) + 64ll * b; }
// Number of its first key tile among all sequences' (k0: its first key), with a number
// for each of its tiles before the next sequence's.
__host__ __device__ __forceinline__ long long tile_slot(int k0, int b) { return k0 / 128 + static_cast<long long>(b); }

constexpr int kPackedSorted = 128;  // (packed_pick)
// Unit number `lin` of `heads` heads with `all` units each: its head and its rank among
// that head's. Heads come in groups of `together`, a group's units head by head for each
// rank, all of a group's before the next group's. False: there is none.
__device__ __forceinline__ bool packed_head(long long lin, int heads, int together, int all, int& h, int& rank) {
    int first = 0, here = heads;
    if (together < heads) {
        const long long per = static_cast<long long>(all) * together;
        if (per == 0) return false;
        const int group = static_cast<int>(lin / per);
        lin -= group * per;
        first = group * together;
        if (first >= heads) return false;
        here = min(together, heads - first);
    }
    h = first + static_cast<int>(lin % here);
    rank = static_cast<int>(lin / here);
    return true;
}
// Sum over the sequences of what `units` says, by a whole warp.
template <typename F>
__device__ __forceinline__ int packed_total(int B, int lane, F&& units) {
    int n = 0;
    for (int b = lane; b < B; b += 32) n += units(b);
    return __reduce_add_sync(0xffffffffu, n);
}
// Sequence b has n units at levels a .. a + n - 1, one each (runs(b, a, n); n = 0:
// none); a unit's time grows with its level. Finds the unit of rank r: for up to 128
// sequences as they are taken from the highest level down, so that the longest start
// first whatever the sequences' lengths and order are (by bisection over the levels, a few
// dozen instructions each, without a list in memory or a launch that makes one); for more,
// where a search of this kind would read all sequences for each level, in the order of the
// sequences, each from its highest level down. (A long sequence behind more than 128 short
// ones then starts last: 16000 tokens before and behind 128 of 100, 16 heads over 4, us:
// d = 64 557 and 673, d = 128 718 and 723, backward 1954 and 1955, 2405 and 2464.) Called by
// a whole warp; false where there is no such unit.
//
// `at`: where the search begins, the first 128-sequence block that r may lie in and the
// units before it; callers whose ranks rise keep it from one call to the next.
struct PackedCursor {
    int block, before;
};
template <typename F>
__device__ __forceinline__ bool packed_pick(int B, int r, int lane, F&& runs, int& b, int& level, PackedCursor& at) {
    constexpr int CHUNKS = kPackedSorted / 32;
    int a[CHUNKS], n[CHUNKS];  // of a block of sequences, the loads of all four in flight at once
    auto load = [&](int first) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            a[c] = n[c] = 0;
            if (first + 32 * c < B && first + 32 * c + lane < B) runs(first + 32 * c + lane, a[c], n[c]);
        }
    };
    if (B > kPackedSorted) {
        for (; at.block < B; at.block += kPackedSorted) {
            load(at.block);
            int k = 0;
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) k += n[c];
            k = __reduce_add_sync(0xffffffffu, k);
            if (r < at.before + k) break;
            at.before += k;
        }
        if (at.block >= B) return false;
        int left = r - at.before;
        b = -1;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            int upto = n[c];  // units of this and the lower lanes
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            const unsigned here = __ballot_sync(0xffffffffu, left < upto);
            if (b < 0 && here) {
                const int who = __ffs(here) - 1;
                b = at.block + 32 * c + who;
                level = __shfl_sync(0xffffffffu, a[c] + upto - 1 - left, who);
            }
            left -= __shfl_sync(0xffffffffu, upto, 31);
        }
        return b >= 0;
    }
    load(0);
    int lo = 0x7fffffff, hi = -0x7fffffff, all = 0;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
        if (n[c] > 0) lo = min(lo, a[c]), hi = max(hi, a[c] + n[c] - 1), all += n[c];
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    all = __reduce_add_sync(0xffffffffu, all);
    if (r >= all) return false;
    auto from = [&](int l) {  // units at this level or above
        int k = 0;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
            if (32 * c < B) k += min(max(a[c] + n[c] - l, 0), n[c]);
        return __reduce_add_sync(0xffffffffu, k);
    };
#pragma unroll 1
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (from(mid) > r) lo = mid;
        else hi = mid - 1;
    }
    level = lo;
    int left = r - from(lo + 1);
    b = -1;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const bool here = n[c] > 0 && a[c] <= lo && lo < a[c] + n[c];
        const unsigned who = __ballot_sync(0xffffffffu, here);
        const unsigned mine = __ballot_sync(0xffffffffu, here && __popc(who & low_bits(lane)) == left);
        if (b < 0 && mine) b = 32 * c + __ffs(mine) - 1;
        left -= __popc(who);
    }
    return b >= 0;
}

}  // namespace fa
