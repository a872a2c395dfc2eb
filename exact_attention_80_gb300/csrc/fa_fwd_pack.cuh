// fa_fwd_pack.cuh — what packed sequences of different lengths with grouped heads
// change in the forward kernels: a unit's place in the batch, its query tiles, the
// end of a sequence inside a key tile, and the output rows.
//
// A query tile's 128 rows are the heads of one kv head for 128 / G tokens (G = H /
// Hkv), token by token, as one TMA box brings them from [token][H][d]: the group
// shares every K and V tile, a tile spans fewer tokens, so that less of it lies above
// the diagonal, and short sequences fill their tiles better (a prompt of 24 tokens,
// G = 4: one tile of 96 rows, not four of 24). Row r is token r / G, head r % G.
//
// Units (two tiles; one at d = 256) are taken longest first over up to 128 sequences, and
// in their order over more (packed_pick): under a causal mask a unit's time grows with its
// last position, and the last CTAs to start set the call's end.
//
// A key tile that a sequence ends in holds the next one's keys, or what lies behind
// the last one. Their scores are masked, but a weight of zero does not undo an
// infinity or a NaN in V: the producer overwrites those V rows with zeros, once per
// unit, while the unit's last scores are formed (persistent CTAs: behind the next unit's
// first loads).
//
// Persistent CTAs (d <= 128, two waves of units and more, short key lists) take one unit
// of each round, forwards and backwards in turn; an idle warp finds them a few ahead and
// hands them over in a ring, so that no other warp waits for the search (600 sequences of
// 20 tokens, 16 + 4 heads, d = 128: 93 us; 160 with a CTA and a search per unit).
#pragma once

#include "fa_fwd_win.cuh"
#include "fa_packed.cuh"

namespace fa {

struct PackUnit {
    int qbase, len_q;  // first query of the sequence, its number of queries
    int kbase, len_k;
    int token;         // the unit's first query, within the sequence
    int h;             // kv head, or -1: no more units
};
constexpr int kPackRing = 4;
struct PackRing {
    PackUnit unit[kPackRing];
};

// Reports sequences whose offsets are broken; one warp of the launch.
__device__ __forceinline__ void pack_check(const FwdParams& p, int lane) {
    const PackedSeqs s = {p.cu_q, p.cu_k, p.B, p.total_q, p.Nk, p.Nq, p.max_k};
    PackedSeq x;
    for (int b = lane; b < p.B; b += 32)
        if (!packed_seq(s, b, x)) atomicOr(p.status, kStatusBadSeqlens);
}

// Unit number `lin` (kv heads fastest), found by one warp. False: there is none.
template <int QT>
__device__ __forceinline__ bool pack_unit(const FwdParams& p, long long lin, int lane, PackUnit* u, PackedCursor& at) {
    const PackedSeqs s = {p.cu_q, p.cu_k, p.B, p.total_q, p.Nk, p.Nq, p.max_k};
    PackedSeq x;
    const int tokens = QT * p.tile_tokens;
    auto level0 = [&](const PackedSeq& y) {  // of a sequence's first unit: its offset in units, rounded down
        const int off = y.m - y.n;
        return off >= 0 ? off / tokens : -((tokens - 1 - off) / tokens);
    };
    auto runs = [&](int b, int& a, int& n) {
        PackedSeq y;
        packed_seq(s, b, y);
        a = level0(y);
        n = (y.n + tokens - 1) / tokens;
    };
    int b = 0, level = 0;
    const bool have = packed_pick(p.B, static_cast<int>(lin / p.Hkv), lane, runs, b, level, at);
    if (lane == 0) {
        x = {0, 0, 0, 0};
        if (have) packed_seq(s, b, x);
        *u = {x.q0, x.n, x.k0, x.m, have ? (level - level0(x)) * tokens : 0, have ? static_cast<int>(lin % p.Hkv) : -1};
    }
    return have;
}

// Persistent CTAs: one warp fills the ring with the CTA's units, and an end mark.
// Consumers: the producer, the issuer and the eight softmax warps.
constexpr int kPackReaders = 10;
template <int QT, typename L>
__device__ __forceinline__ void pack_feed(const FwdParams& p, PackRing* ring, uint32_t sbase, int lane,
                                          volatile uint32_t* abort_flag) {
    PackedCursor at = {0, 0};
    for (int k = 0;; ++k) {
        const int slot = k % kPackRing;
        if (k >= kPackRing &&
            !wait_phase_warp(sbase + L::BAR_OFF + 8u * (L::BAR_UEMPTY + slot), (k / kPackRing - 1) & 1, p, abort_flag,
                             kStatusWaitQ))
            return;
        const long long g = gridDim.x, c = (k & 1) ? g - 1 - blockIdx.x : blockIdx.x;
        const bool have = pack_unit<QT>(p, k * g + c, lane, &ring->unit[slot], at);
        __syncwarp();
        if (lane == 0) mbar_arrive(sbase + L::BAR_OFF + 8u * (L::BAR_UFULL + slot));
        if (!have) return;
    }
}
// The unit of a CTA that has one (an empty one where there is none).
template <int QT, int BN>
__device__ __forceinline__ void pack_work(const FwdParams& p, const PackUnit& u, WorkWin<QT>& w);
template <int QT, int BN>
__device__ __forceinline__ void pack_first(const FwdParams& p, const PackRing* ring, WorkWin<QT>& w) {
    pack_work<QT, BN>(p, ring->unit[0], w);
}
// The persistent CTA's unit number k, by a whole warp; false where there are no more (`ok`
// false: the wait for it failed).
template <int QT, int BN, typename L>
__device__ __forceinline__ bool pack_next(const FwdParams& p, PackRing* ring, uint32_t sbase, int k,
                                          volatile uint32_t* abort_flag, WorkWin<QT>& w, bool& ok) {
    const int slot = k % kPackRing;
    ok = wait_phase_warp(sbase + L::BAR_OFF + 8u * (L::BAR_UFULL + slot), (k / kPackRing) & 1, p, abort_flag,
                         kStatusWaitQ);
    if (!ok) return false;
    const PackUnit u = ring->unit[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(sbase + L::BAR_OFF + 8u * (L::BAR_UEMPTY + slot));
    if (u.h < 0) return false;
    pack_work<QT, BN>(p, u, w);
    return true;
}

// Rows that belong to no sequence (before the first one and behind the last): O = 0,
// LSE = -inf where the call asks for it. One warp of each CTA, its share of them.
template <int D>
__device__ __forceinline__ void pack_fill(const FwdParams& p, int lane) {
    if (!p.fill) return;
    const int c0 = p.cu_q[0], c1 = p.cu_q[p.B];
    if (!(0 <= c0 && c0 <= c1 && c1 <= p.total_q)) return;
    const int rest = p.total_q - (c1 - c0);
    for (long long i = blockIdx.x; i < rest; i += gridDim.x) {
        const long long token = i < c0 ? i : i + (c1 - c0);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + token * p.H * D);
        for (int e = lane; e < p.H * (D / 8); e += 32) dst[e] = make_uint4(0u, 0u, 0u, 0u);
        for (int h = lane; h < p.H; h += 32) p.lse[static_cast<long long>(h) * p.total_q + token] = -INFINITY;
    }
}

// First token of tile slot t: with two slots the later rows come first (see tile_row0).
template <int QT>
__device__ __forceinline__ int pack_tile_token(const FwdParams& p, int first, int t) {
    return first + (QT == 2 ? 1 - t : t) * p.tile_tokens;
}

template <int QT, int BN>
__device__ __forceinline__ void pack_work(const FwdParams& p, const PackUnit& u, WorkWin<QT>& w) {
    w.split = 0;
    w.bh = u.h;
    w.zq = u.h * p.group;
    w.zk = u.h;
    w.qbase = u.qbase;
    w.kbase = u.kbase;
    w.q0 = u.token;
    w.kv_tile0 = 0;
    w.kv_end = u.len_k;
    w.causal_off = u.len_k - u.len_q;
    w.rm = {0, 0, 0, u.len_q};  // (no unit: no rows, no keys)
    w.list = win_list<BN>(p, u.token + w.causal_off, min(u.token + QT * p.tile_tokens, u.len_q) - 1 + w.causal_off);
    w.nmax = w.list.n;
    w.small = QT == 2 && w.list.ns == 1 && p.sinks <= kSmallSinks;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int row0 = pack_tile_token<QT>(p, u.token, t);
        w.n[t] = w.hole[t] = w.steps[t] = 0;
        if (row0 >= u.len_q) continue;
        const int last = min(row0 + p.tile_tokens, u.len_q) - 1 + w.causal_off;
        if (last < 0) continue;
        const int end = last / BN + 1;
        const int first = p.window > 0 ? max(0, row0 + w.causal_off - p.window + 1) / BN : 0;
        w.n[t] = w.list.ns + max(0, end - w.list.lo);
        w.hole[t] = w.list.ns > 0 || w.list.lo > 0 ? max(0, min(first, end) - w.list.lo) : 0;
        w.steps[t] = w.n[t] - w.hole[t];
    }
}

// Keys of the unit's last key tile that the sequence has (BN or more: all).
template <int BN, int QT>
__device__ __forceinline__ int pack_tail(const WorkWin<QT>& w) {
    return w.kv_end - w.list.tile(w.nmax - 1) * BN;
}

// Zeros over rows `rows` .. BN - 1 of the V tile that the calling warp (the producer)
// loaded as entry number `entry` of the ring: the phase it waits for is the one in progress
// or the one just completed, since the issuer does not release the slot before the tile is
// clean. False where the wait failed.
template <typename L>
__device__ __forceinline__ bool pack_clean_v(const FwdParams& p, uint32_t sbase, int entry, int rows, uint32_t clean,
                                             volatile uint32_t* abort_flag, int lane) {
    const int slot = entry % L::STAGES;
    if (!wait_phase_warp(sbase + L::BAR_OFF + 8u * (L::BAR_KVFULL + slot), (entry / L::STAGES) & 1, p, abort_flag,
                         kStatusWaitKvFull))
        return false;
    const uint32_t tile = sbase + L::SLOT_OFF + slot * L::SLOT_BYTES;
    for (int c = 0; c < L::CHUNKS; ++c)
        for (int at = rows * 128 + lane * 16; at < L::BN * 128; at += 512)
            st_shared_v4(tile + c * (L::BN * 128) + at, 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(clean);
    return true;
}

// Output of a query tile by its 128 softmax threads (thread r = row r = TMEM lane r;
// `token` its token): O / l as bf16 staged by each warp for its own 32 rows, CHUNKS of 64
// columns at a time, `step` bytes apart from `stage` on (row r's line at r * 128, or for
// one chunk the warp's own 4 KB), then written as boxes of 32 rows or 128 bytes of a row per
// eight lanes. Rows past the sequence, or past the tile's whole tokens, are left out. n = 0:
// no key.
template <int D, int QT, bool PERSIST>
__device__ __forceinline__ void pack_store(const FwdParams& p, const WorkWin<QT>& w, int token, int r, int n, float m,
                                           float m_true, float l, float l_o, uint32_t tO, uint32_t stage) {
    constexpr int CHUNKS = PERSIST ? 1 : D / 64, STEP = kBM * 128;
    const int lane = r & 31, head = w.zq + r % p.group;
    const bool row_ok = r < p.group * p.tile_tokens && token < w.rm.len_q;
    const long long row = (static_cast<long long>(w.qbase) + token) * p.H + head;
    const RowMap rm = {row, static_cast<long long>(head) * p.total_q + w.qbase + token, 0, row_ok ? 1 : 0};
    const RowOut<D> out(p, rm, 0, 0, 0, m, m_true, l, l_o);
    // A warp whose 32 rows all exist hands them over as a box per chunk (persistent CTAs, d =
    // 128: 2500 cycles of a unit against 4900 with stores of its own; eight prompts of 2048,
    // 32 + 8 heads: 253 -> 235 us; four of 4096, 16 + 4 heads of 256, where a CTA has one unit
    // and 64 KB to hand over at its end: 446 -> 451, so not there).
    const bool box = D <= 128 && p.store_boxes && __all_sync(0xffffffffu, row_ok);
    const int token0 = __shfl_sync(0xffffffffu, token, 0);
    const uint32_t swz = static_cast<uint32_t>(r & 7);
    const uint32_t mine = stage + (PERSIST ? 0 : (r & ~31) * 128);  // the warp's 32 lines
#pragma unroll 1
    for (int c0 = 0; c0 < D / 64; c0 += CHUNKS) {
#pragma unroll 1
        for (int cc = 0; cc < CHUNKS; ++cc) {
            const int c = c0 + cc;
            uint32_t a[32], b[32];
            if (n > 0) {
                tmem_ld32(tO + c * 64, a);
                tmem_ld32(tO + c * 64 + 32, b);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) a[i] = b[i] = 0u;
            }
            if constexpr (PERSIST) {  // an earlier box may still be read
                if (lane == 0) bulk_wait_group_read0();
                __syncwarp();
            }
            const uint32_t line = mine + cc * STEP + lane * 128;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t x0 = hh ? b[2 * i] : a[2 * i];
                    const uint32_t x1 = hh ? b[2 * i + 1] : a[2 * i + 1];
                    pk[i] = pack_bf16x2(__uint_as_float(x0) * out.f, __uint_as_float(x1) * out.f);
                }
#pragma unroll
                for (int uu = 0; uu < 4; ++uu) {
                    const uint32_t u = static_cast<uint32_t>(hh * 4 + uu);
                    st_shared_v4(line + ((u ^ swz) << 4), pk[4 * uu], pk[4 * uu + 1], pk[4 * uu + 2], pk[4 * uu + 3]);
                }
            }
        }
        if (box) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
#pragma unroll
                for (int cc = 0; cc < CHUNKS; ++cc)
                    tma_store_3d(&p.tm_o, mine + cc * STEP, (c0 + cc) * 64, w.zq, w.qbase + token0);
                bulk_commit_group();
                // (Persistent CTAs wait before they write there again, and at their end.)
                if constexpr (!PERSIST) bulk_wait_group_read0();
            }
            __syncwarp();
            continue;
        }
        __syncwarp();
#pragma unroll 1
        for (int it = 0; it < 8; ++it) {
            const int rr = it * 4 + (lane >> 3), u = lane & 7;
            const bool ok = __shfl_sync(0xffffffffu, static_cast<int>(row_ok), rr) != 0;
            const long long to = __shfl_sync(0xffffffffu, row, rr);
            if (!ok) continue;
#pragma unroll
            for (int cc = 0; cc < CHUNKS; ++cc) {
                float x[4];
                ld_shared_v4f(mine + cc * STEP + rr * 128 + ((u ^ (rr & 7)) << 4), x);
                *reinterpret_cast<float4*>(static_cast<__nv_bfloat16*>(p.o) + to * D + (c0 + cc) * 64 + u * 8) =
                    make_float4(x[0], x[1], x[2], x[3]);
            }
        }
        __syncwarp();
    }
    out.finish(p);
}

}  // namespace fa
