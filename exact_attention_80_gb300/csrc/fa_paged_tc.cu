// fa_paged_tc.cu — attention over the paged e4m3 cache for many query rows
// (chunks of prompts, long drafts), on tcgen05.
//
// A CTA owns 256 rows of one (sequence, kv head): rows are (query token, head of
// the group) pairs, in two tiles of 128 that alternate on the tensor core as
// in the dense forward, and sweeps the key tiles of 128 keys they need. The
// cache stays in its 8 bits up to the operands:
//   * S = Q K^T runs as kind::f8f6f4 on K's codes as they lie in shared memory.
//     Q (bf16, eight significant bits) is split into two e4m3 terms of four
//     bits, x = hi + lo after a power-of-two scale per row, which is exact for
//     elements down to 2^-9 of the row's largest (2^-17 of it is the largest
//     error below that): twice the MMAs at twice the rate of bf16, and no
//     conversion of K.
//   * O += P V runs as kind::f16: P in f16 (relative rounding 2^-11) in TMEM
//     over its S columns, V converted from its codes (exact) by four warps of
//     their own, once per key tile for both row tiles.
// The block scales enter where fa_paged.cu has them: the K scale multiplies the
// score, log2 of the V scale adds to the exponent, and the row sum takes its
// reciprocal; scores are handled in groups of 16 keys, the smallest page.
//
// DUAL: at most 128 rows (drafts, short chunks). Both tile slots take the same
// rows, each with half of the CTA's keys, so that the two still alternate on the
// tensor core; their states meet in shared memory at the end. With at most 32
// (64) rows a slot's 128 lanes hold them four times (twice), and each copy's
// warps take their share of a tile's columns with weights of zero for the others:
// the MMAs cost the same, and four warps rather than one form a tile's
// exponentials (five drafted tokens, 20 rows, for 64 contexts of up to 32768 keys:
// 529 us, a fifth less than without shares; for one of 131072: 58).
//
// D = 256 (WIDE): O takes half of TMEM, so a CTA owns one tile of 128 rows, and S
// has two buffers: the tensor core forms S of tile j + 2 behind PV of tile j while
// the softmax (four warps) is at tile j + 1. Eight warps convert V, whose f16 form
// has one buffer: a tile is converted while S takes the tensor core (chunks of 1024
// tokens over 8192 keys, 16 + 2 heads: 197 us, 1300 TFLOP/s; 1216 us with 16 rows
// per CTA in the other kernel; 40 rows a kv head, 32 + 8 heads, over 16 contexts of
// up to 8000 keys: 114 us against 202).
//
// Roles, by warp: 0 producer (Q is written by the softmax threads; K and V pages
// by TMA into two rings), 1 issuer, 2-3 idle, 4-11 softmax (thread = row = TMEM
// lane), 12-15 converters (two warps took 2200 cycles a tile beside the
// softmax, four take 1150). Step j, per tile as its P arrives: O_t += P_t(j) V_j, then at
// once S_t(j+1) over the same columns. Every wait is bounded as in the dense
// forward.
#include <cuda_bf16.h>

#include "fa.h"
#include "fa_paged.cuh"
#include "fa_paged_phases.h"
#include "fa_rope.cuh"

namespace fa {
namespace {

// SHARES: 0 for full tiles, else the dual form and its shares.
template <int D, int SHARES>
struct TcLayout {
    static constexpr bool DUAL = SHARES > 0;
    static constexpr int BM = 128, BN = kTcKeys;
    static constexpr bool WIDE = D == 256;                // one row tile, S in two buffers
    static constexpr int ROW_BYTES = D < 128 ? D : 128;   // swizzled row of codes (D = 256: in two parts)
    static constexpr int PARTS = D / ROW_BYTES;
    static constexpr uint32_t PART = BN * ROW_BYTES;      // bytes of a part of a K or V tile (or of a term of Q)
    // Dual slots share one row tile, which leaves room for deeper rings.
    static constexpr int KSTAGES = WIDE ? 2 : D == 64 ? 6 : DUAL ? 4 : 3;
    static constexpr int VSTAGES = WIDE ? 1 : D == 64 ? 6 : DUAL ? 3 : 2;
    static constexpr int VBUFS = WIDE ? 1 : 2;            // V tiles in f16
    static constexpr int THREADS = 512;
    static constexpr int CONV_WARP0 = WIDE ? 8 : 12, CONV_WARPS = 16 - CONV_WARP0;
    static constexpr uint32_t Q_TERM = BM * D;            // one e4m3 term of a row tile
    static constexpr uint32_t Q_TILE = 2 * Q_TERM;
    static constexpr uint32_t SLOT = BN * D;              // codes of a K or V tile
    static constexpr uint32_t V16 = BN * D * 2;           // V tile in f16: 64-column chunks of 128-byte rows
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t K_OFF = Q_OFF + (DUAL || WIDE ? 1 : 2) * Q_TILE;
    static constexpr uint32_t V_OFF = K_OFF + KSTAGES * SLOT;
    static constexpr uint32_t V16_OFF = V_OFF + VSTAGES * SLOT;
    static constexpr uint32_t BAR_OFF = V16_OFF + VBUFS * V16;
    // DUAL, at the end: fp32 O of both slots' 128 lanes, then m and l.
    static constexpr uint32_t ML_OFF = 2 * BM * D * 4;
    static_assert(!DUAL || ML_OFF + 2 * 2 * BM * 4 <= BAR_OFF, "the states overwrite barriers");
    static constexpr int BAR_QFULL = 0;                    // [tile] one arrival per softmax warp with rows
    static constexpr int BAR_KFULL = 2;
    static constexpr int BAR_KEMPTY = BAR_KFULL + KSTAGES;
    static constexpr int BAR_VFULL = BAR_KEMPTY + KSTAGES;
    static constexpr int BAR_VEMPTY = BAR_VFULL + VSTAGES;   // one arrival per converter warp
    static constexpr int BAR_HFULL = BAR_VEMPTY + VSTAGES;   // [buffer] V in f16 (one arrival per converter warp)
    static constexpr int BAR_HEMPTY = BAR_HFULL + 2;         // [buffer]
    static constexpr int BAR_SFULL = BAR_HEMPTY + 2;         // [tile]
    static constexpr int BAR_PFULL = BAR_SFULL + 2;          // [tile] one arrival per softmax warp with rows
    static constexpr int BAR_OFULL = BAR_PFULL + 2;          // [tile] (WIDE: as fa_paged_phases.h says)
    static constexpr int BAR_DRAIN = BAR_OFULL + 2;
    static constexpr int NUM_BARS = BAR_DRAIN + 1;
    static constexpr uint32_t MISC_OFF = BAR_OFF + NUM_BARS * 8;
    static constexpr uint32_t BYTES = MISC_OFF + 16;
    static constexpr size_t ALLOC = BYTES + 1024;
    // TMEM columns: S_t (P_t over its first half), then O_t.
    __host__ __device__ static constexpr uint32_t S_COL(int t) { return t * BN; }
    __host__ __device__ static constexpr uint32_t O_COL(int t) { return 256 + t * D; }
    static constexpr int LAUNCH_REGS = 128, CTRL_REGS = 56, SOFTMAX_REGS = 200;
    static_assert((WIDE ? 384 : 256) * CTRL_REGS + (WIDE ? 128 : 256) * SOFTMAX_REGS <= THREADS * LAUNCH_REGS,
                  "register split");
    static_assert(ALLOC <= 232448, "shared memory over the 227 KB per-CTA limit");
    static_assert(ALLOC > 232448 / 2, "two CTAs per SM would contend for TMEM");
    static_assert(256 + (WIDE ? 1 : 2) * D <= 512, "O overflows TMEM");
    static_assert(!(WIDE && DUAL), "no room");
};

// kind::f16 with f16 operands (format code 0), fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

struct TcWork {
    NewTokens nt;
    int b, h, rows, start;
    int used;      // states that its rows leave (1: the result)
    int split;     // the state that this CTA leaves
    int row0[2];   // first row of each tile slot
    KeyList list;
    int i0[2];     // first list entry of its part
    int n[2];      // key tiles each row tile visits
    int nmax;
    int p0, p1;    // positions of the unit's first and last row
    bool live;
};

// Key tiles of a piece, the share of a CTA's two slots, where all row blocks are
// one per sequence: their lengths differ, and so the pieces are cut as long as
// makes the waves of CTAs shortest (16 sequences of five drafted tokens over 4600
// to 16200 keys, 8 kv heads: 8 % less time than with the same length for all calls
// of the shape). Called by a whole warp; every lane tries one length.
__device__ __forceinline__ int tc_piece(const PagedParams& p, int lane) {
    int n[kTcBalance / 32];
    int longest = 0;
#pragma unroll
    for (int i = 0; i < kTcBalance / 32; ++i) {
        const int b = lane + 32 * i;
        NewTokens t;
        n[i] = 0;
        if (b < p.B && new_tokens(p.cu, p.lens, b, p.total_q, p.max_q, p.max_k, t) && t.n > 0)
            n[i] = key_list<kTcKeys>(p.window, p.sinks, t.len - t.n, t.len - 1).n;
        longest = max(longest, n[i]);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    const int least = p.tiles_per_split;  // as the workspace allows
    if (longest <= least) return least;
    const int len = least + (longest - least) * lane / 31;
    const float inv = 1.f / static_cast<float>(len);
    int pieces = 0;  // (rounded about right: only the choice depends on it)
    for (int b = 0; b < p.B; ++b) {
        const int x = __shfl_sync(0xffffffffu, b < 32 ? n[0] : n[1], b & 31);
        pieces += static_cast<int>(fmaf(static_cast<float>(x), inv, 0.999f));
    }
    const int waves = (pieces * p.Hkv + kTcAtOnce - 1) / kTcAtOnce;
    const unsigned cost = static_cast<unsigned>(waves * (len + kTcStart));
    const unsigned best = __reduce_min_sync(0xffffffffu, cost);
    const int at = __ffs(__ballot_sync(0xffffffffu, cost == best)) - 1;
    return __shfl_sync(0xffffffffu, len, at);
}

template <bool DUAL, bool WIDE>
__device__ __forceinline__ void tc_work(const PagedParams& p, int piece, TcWork& w) {
    constexpr int ROWS = DUAL || WIDE ? kTcRows : 2 * kTcRows;
    const int per_unit = p.num_splits;
    unsigned lin = blockIdx.x;
    const int si = static_cast<int>(lin % per_unit);
    lin /= per_unit;
    // The last rows of a sequence see the most keys: they start first.
    const int unit = p.row_blocks - 1 - static_cast<int>(lin % p.row_blocks);
    lin /= p.row_blocks;
    w.h = static_cast<int>(lin % p.Hkv);
    w.b = static_cast<int>(lin / p.Hkv);
    w.nmax = w.n[0] = w.n[1] = 0;
    w.live = new_tokens(p.cu, p.lens, w.b, p.total_q, p.max_q, p.max_k, w.nt);
    if (!w.live) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusBadSeqlens);
        return;
    }
    w.rows = w.nt.n * p.G;
    const int r0 = unit * ROWS;
    w.live = r0 < w.rows;
    if (!w.live) return;
    w.start = w.nt.len - w.nt.n;
    w.p0 = w.start + r0 / p.G;
    w.p1 = w.start + (min(r0 + ROWS, w.rows) - 1) / p.G;
    w.list = key_list<kTcKeys>(p.window, p.sinks, w.p0, w.p1);
    if constexpr (DUAL) {
        // Pieces of equal length; the slots take a half each.
        const int pieces = min(per_unit, max(1, (w.list.n + piece - 1) / piece));
        w.used = pieces;
        w.live = si < pieces;
        if (!w.live) return;
        const int e0 = static_cast<int>(static_cast<long long>(w.list.n) * si / pieces);
        const int e1 = static_cast<int>(static_cast<long long>(w.list.n) * (si + 1) / pieces);
        const int mid = (e0 + e1 + 1) / 2;
        w.split = si;
        w.row0[0] = w.row0[1] = r0;
        w.i0[0] = e0, w.i0[1] = mid;
        w.n[0] = w.nmax = mid - e0;
        w.n[1] = e1 - mid;
        return;
    }
    w.used = max(1, (w.list.n + p.tiles_per_split - 1) / p.tiles_per_split);
    w.live = si < w.used;
    if (!w.live) return;
    w.split = si;
#pragma unroll
    for (int t = 0; t < (WIDE ? 1 : 2); ++t) {
        // Slot 0 takes the later rows, whose tile ends last: the issuer serves
        // it first.
        w.row0[t] = WIDE ? r0 : r0 + (1 - t) * kTcRows;
        w.i0[t] = si * p.tiles_per_split;
        if (w.row0[t] >= w.rows) continue;
        const int last = w.start + (min(w.row0[t] + kTcRows, w.rows) - 1) / p.G;
        const int end = w.list.ns + max(0, last / kTcKeys + 1 - w.list.lo);
        w.n[t] = max(0, min(min(w.list.n, w.i0[t] + p.tiles_per_split), end) - w.i0[t]);
        w.nmax = max(w.nmax, w.n[t]);
    }
}

__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, const PagedParams& p,
                                        volatile uint32_t* abort_flag, unsigned what, bool honor_abort = true) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long start = clock64();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (honor_abort && *abort_flag) return false;
        if (clock64() - start > p.wait_limit) {
            *abort_flag = 1u;
            atomicOr(p.status, what);
            return false;
        }
    }
}
__device__ __forceinline__ bool tc_wait_warp(uint32_t bar, uint32_t parity, const PagedParams& p,
                                             volatile uint32_t* abort_flag, unsigned what) {
    return __all_sync(0xffffffffu, tc_wait(bar, parity, p, abort_flag, what));
}

// Page of list entry i's key group at `key` (a multiple of 16), or -1 where the
// sequence has none; a bad entry is reported and taken as none.
__device__ __forceinline__ int tc_page(const PagedParams& p, const TcWork& w, const int* table, int key) {
    if (key >= w.nt.len) return -1;
    const int id = table[key >> p.log_page];
    if (id < 0 || id >= p.num_pages) {
        atomicOr(p.status, kStatusBadPage);
        return -1;
    }
    return id;
}

template <int D, int SHARES>
__global__ void __launch_bounds__(TcLayout<D, SHARES>::THREADS, 1) fa_paged_tc_kernel(const __grid_constant__ PagedParams p) {
    using L = TcLayout<D, SHARES>;
    constexpr bool DUAL = L::DUAL, WIDE = L::WIDE;
    constexpr int BN = L::BN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
    volatile uint32_t* abort_flag = misc + 1;
    auto bar = [&](int i) -> uint32_t { return sbase + L::BAR_OFF + 8u * i; };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::KSTAGES; ++s) {
            mbar_init(bar(L::BAR_KFULL + s), 1);
            mbar_init(bar(L::BAR_KEMPTY + s), 1);
        }
        for (int s = 0; s < L::VSTAGES; ++s) {
            mbar_init(bar(L::BAR_VFULL + s), 1);
            mbar_init(bar(L::BAR_VEMPTY + s), L::CONV_WARPS);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(L::BAR_HFULL + t), L::CONV_WARPS);
            mbar_init(bar(L::BAR_HEMPTY + t), 1);
            mbar_init(bar(L::BAR_QFULL + t), p.slot_warps);
            mbar_init(bar(L::BAR_SFULL + t), 1);
            mbar_init(bar(L::BAR_PFULL + t), p.slot_warps);
            mbar_init(bar(L::BAR_OFULL + t), 1);
        }
        mbar_init(bar(L::BAR_DRAIN), 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    if constexpr (DUAL) {
        if (warp == 2) {
            const int piece = p.balance ? tc_piece(p, lane) : p.tiles_per_split;
            if (lane == 0) misc[2] = piece;
        }
    }
    if (warp == 1) {
        tmem_alloc(sbase + L::MISC_OFF, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const int piece = DUAL ? static_cast<int>(misc[2]) : 0;

    if (warp < 4 || warp >= L::CONV_WARP0) {
        setmaxnreg_dec<L::CTRL_REGS>();
        TcWork w;
        tc_work<DUAL, L::WIDE>(p, piece, w);
        if (w.live && warp == 0) {
            // -------------------------------------------------------- producer
            // Entries in the issuer's order: K_0; then per step j: V_j, K_{j+1}.
            // Dual: K_0 of both slots; then per step and slot V_j, K_{j+1}. A
            // tile's pages are copied one by one; pages behind the sequence's end
            // are left out.
            const bool leader = elect_one();
            const int* table = p.page_table + static_cast<long long>(w.b) * p.max_pages;
            const int per = BN >> p.log_page;  // pages per tile (page_size <= 128)
            const uint32_t page_bytes = static_cast<uint32_t>(D) << p.log_page, part_bytes = page_bytes / L::PARTS;
            // Page ids come 32 at a time, a lane each, the next 32 on their way: a
            // tile's copies never wait for the page table. Batch q of a
            // sequence holds the pages 32 q .. of its tiles in order.
            const int log_per = __popc(per - 1);
            auto batch_of = [&](int t, int q) {
                const int page = 32 * q + lane, j = page >> log_per;
                return j < (DUAL ? w.n[t] : w.nmax)
                           ? tc_page(p, w, table, w.list.tile(w.i0[t] + j) * BN + ((page & (per - 1)) << p.log_page))
                           : -1;
            };
            auto copy = [&](const CUtensorMap* map, uint32_t dst, uint32_t full, int ids, int first) {
                // A lane per page: issued one after the other by a single lane, pages of
                // 32 tokens hold the whole CTA up (five drafted tokens for 16 contexts of
                // up to 16200 keys: 106 us against 87).
                const bool mine = ids >= 0 && lane >= first && lane < first + per;
                const unsigned here = __ballot_sync(0xffffffffu, mine);
                if (leader) mbar_arrive_expect_tx(full, __popc(here) * page_bytes);
                __syncwarp();
                if (mine) {
#pragma unroll
                    for (int c = 0; c < L::PARTS; ++c)
                        tma_load_2d(dst + c * L::PART + (lane - first) * part_bytes, map, full, c * 128,
                                    (ids * p.Hkv + w.h) << p.log_page);
                }
                __syncwarp();
            };
            int k_issued = 0, v_issued = 0;
            bool ok = true;
            auto load_k = [&](int ids, int first) -> bool {
                const int s = k_issued % L::KSTAGES;
                if (k_issued >= L::KSTAGES &&
                    !tc_wait_warp(bar(L::BAR_KEMPTY + s), (k_issued / L::KSTAGES - 1) & 1, p, abort_flag,
                                  kStatusWaitKvEmpty))
                    return false;
                copy(&p.tm_k, sbase + L::K_OFF + s * L::SLOT, bar(L::BAR_KFULL + s), ids, first);
                ++k_issued;
                return true;
            };
            auto load_v = [&](int ids, int first) -> bool {
                const int s = v_issued % L::VSTAGES;
                if (v_issued >= L::VSTAGES &&
                    !tc_wait_warp(bar(L::BAR_VEMPTY + s), (v_issued / L::VSTAGES - 1) & 1, p, abort_flag,
                                  kStatusWaitKvEmpty))
                    return false;
                copy(&p.tm_v, sbase + L::V_OFF + s * L::SLOT, bar(L::BAR_VFULL + s), ids, first);
                ++v_issued;
                return true;
            };
            if constexpr (WIDE) {
                // K runs two tiles ahead of V: pages of its own.
                int ids[2], ahead[2];  // of K, of V: the batch at hand and the next one
#pragma unroll
                for (int s = 0; s < 2; ++s) ids[s] = batch_of(0, 0), ahead[s] = batch_of(0, 1);
                auto tile = [&](int s, int j) -> bool {
                    const int first = (j << log_per) & 31;
                    if (first == 0 && j > 0) {
                        ids[s] = ahead[s];
                        ahead[s] = batch_of(0, (j << log_per >> 5) + 1);
                    }
                    return s ? load_v(ids[1], first) : load_k(ids[0], first);
                };
                for (int j = 0; j < min(2, w.nmax) && ok; ++j) ok = tile(0, j);
                for (int j = 0; j < w.nmax && ok; ++j) {
                    ok = tile(1, j);
                    if (ok && j + 2 < w.nmax) ok = tile(0, j + 2);
                }
            } else {
            constexpr int SEQS = DUAL ? 2 : 1;  // sequences of tiles
            int cur[SEQS], next[SEQS];          // the batch of the tile whose V comes next, and the one behind it
#pragma unroll
            for (int t = 0; t < SEQS; ++t) {
                cur[t] = batch_of(t, 0);
                next[t] = batch_of(t, 1);
                if (ok && (DUAL ? w.n[t] : w.nmax) > 0) ok = load_k(cur[t], 0);
            }
            for (int j = 0; j < w.nmax && ok; ++j) {
                const int first = (j << log_per) & 31;        // of tile j in its batch
                const int first_next = (first + per) & 31;    // of tile j + 1
#pragma unroll
                for (int t = 0; t < SEQS; ++t) {
                    const int n = DUAL ? w.n[t] : w.nmax;
                    if (!ok || j >= n) continue;
                    ok = load_v(cur[t], first);
                    if (first_next == 0) {
                        cur[t] = next[t];
                        next[t] = batch_of(t, ((j + 1) << log_per >> 5) + 1);
                    }
                    if (ok && j + 1 < n) ok = load_k(cur[t], first_next);
                }
            }
            }
            if (ok) {
                // No arrival may be in flight when the CTA exits.
                for (int e = max(0, k_issued - L::KSTAGES); e < k_issued && ok; ++e)
                    ok = tc_wait_warp(bar(L::BAR_KEMPTY + e % L::KSTAGES), (e / L::KSTAGES) & 1, p, abort_flag,
                                      kStatusWaitKvEmpty);
            }
            if (!ok) {
                for (int e = max(0, k_issued - L::KSTAGES); e < k_issued; ++e)
                    tc_wait(bar(L::BAR_KFULL + e % L::KSTAGES), (e / L::KSTAGES) & 1, p, abort_flag, kStatusWaitDrain,
                            false);
                for (int e = max(0, v_issued - L::VSTAGES); e < v_issued; ++e)
                    tc_wait(bar(L::BAR_VFULL + e % L::VSTAGES), (e / L::VSTAGES) & 1, p, abort_flag, kStatusWaitDrain,
                            false);
            }
        } else if (w.live && warp == 1 && w.nmax > 0) {
            // -------------------------------------------------------- MMA issuer
            const bool leader = elect_one();
            constexpr uint32_t IDESC_S = make_idesc_e4m3(128, BN, false, false);
            constexpr uint32_t IDESC_O = idesc_f16(128, D, true);
            const uint64_t kmaj0 = make_sdesc_rows<L::ROW_BYTES>(sbase, 16, 8 * L::ROW_BYTES);
            const uint64_t vmn0 = make_sdesc_sw128(sbase, BN * 128, 1024);
            const uint32_t kmaj_lo = static_cast<uint32_t>(kmaj0), kmaj_hi = static_cast<uint32_t>(kmaj0 >> 32);
            const uint32_t vmn_lo = static_cast<uint32_t>(vmn0), vmn_hi = static_cast<uint32_t>(vmn0 >> 32);
            auto desc = [](uint32_t lo, uint32_t hi, uint32_t off) -> uint64_t {
                return (static_cast<uint64_t>(hi) << 32) | (lo + (off >> 4));
            };
            auto issue_s = [&](int t, int slot) {
                const uint32_t qa = L::Q_OFF + (DUAL || WIDE ? 0 : t) * L::Q_TILE, kb = L::K_OFF + slot * L::SLOT;
#pragma unroll
                for (int term = 0; term < 2; ++term)
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk)
                        if (leader)
                            umma_ss_f8(tmem + L::S_COL(t),
                                       desc(kmaj_lo, kmaj_hi, qa + term * L::Q_TERM + (kk >> 2) * L::PART + (kk & 3) * 32),
                                       desc(kmaj_lo, kmaj_hi, kb + (kk >> 2) * L::PART + (kk & 3) * 32), IDESC_S,
                                       (term | kk) ? 1u : 0u);
                if (leader) umma_commit(bar(L::BAR_SFULL + t));
            };
            auto issue_pv = [&](int t, int buf, bool accumulate) {
                const uint32_t vb = L::V16_OFF + buf * L::V16;
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                    if (leader)
                        umma_ts(tmem + L::O_COL(WIDE ? 0 : t), tmem + L::S_COL(t) + kk * 8, desc(vmn_lo, vmn_hi, vb + kk * 2048),
                                IDESC_O, (accumulate || kk > 0) ? 1u : 0u);
            };
            int k_used = 0;  // K entries waited for
            auto wait_k = [&]() -> bool {
                const bool r = tc_wait_warp(bar(L::BAR_KFULL + k_used % L::KSTAGES), (k_used / L::KSTAGES) & 1, p,
                                            abort_flag, kStatusWaitKvFull);
                ++k_used;
                return r;
            };
            bool ok = true;
            if constexpr (WIDE) {
                // S of tile j goes to buffer j & 1, two tiles ahead of its PV: the
                // tensor core forms S_{j+2} while the softmax is at tile j + 1.
                auto next_s = [&](int j) -> bool {
                    const int slot = k_used % L::KSTAGES;
                    if (!wait_k()) return false;
                    tc_fence_after();
                    issue_s(j & 1, slot);
                    if (leader) umma_commit(bar(L::BAR_KEMPTY + slot));
                    return true;
                };
                ok = tc_wait_warp(bar(L::BAR_QFULL + 0), 0, p, abort_flag, kStatusWaitQ);
                for (int j = 0; j < min(2, w.nmax) && ok; ++j) ok = next_s(j);
                for (int j = 0; j < w.nmax && ok; ++j) {
                    ok = tc_wait_warp(bar(L::BAR_HFULL), j & 1, p, abort_flag, kStatusWaitKvFull);
                    if (ok) ok = tc_wait_warp(bar(L::BAR_PFULL + (j & 1)), (j >> 1) & 1, p, abort_flag, kStatusWaitP);
                    if (!ok) break;
                    tc_fence_after();
                    issue_pv(j & 1, 0, j > 0);
                    if (leader) {
                        umma_commit(bar(L::BAR_HEMPTY));
                        umma_commit(bar(L::BAR_OFULL + wide_pv_barrier(j, w.nmax)));
                    }
                    if (j + 2 < w.nmax) ok = next_s(j + 2);
                }
            } else if constexpr (DUAL) {
                int v_used = 0;  // V entries waited for
                // S of slot t from the next K entry.
                auto next_s = [&](int t) -> bool {
                    const int slot = k_used % L::KSTAGES;
                    if (!wait_k()) return false;
                    tc_fence_after();
                    issue_s(t, slot);
                    if (leader) umma_commit(bar(L::BAR_KEMPTY + slot));
                    return true;
                };
                ok = tc_wait_warp(bar(L::BAR_QFULL + 0), 0, p, abort_flag, kStatusWaitQ);
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (ok && w.n[t] > 0) ok = next_s(t);
                for (int j = 0; j < w.nmax && ok; ++j) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!ok || j >= w.n[t]) continue;
                        const int buf = v_used & 1;
                        ok = tc_wait_warp(bar(L::BAR_HFULL + buf), (v_used >> 1) & 1, p, abort_flag, kStatusWaitKvFull);
                        if (ok) ok = tc_wait_warp(bar(L::BAR_PFULL + t), j & 1, p, abort_flag, kStatusWaitP);
                        if (!ok) break;
                        ++v_used;
                        tc_fence_after();
                        issue_pv(t, buf, j > 0);
                        if (leader) umma_commit(bar(L::BAR_HEMPTY + buf));
                        if (j + 1 < w.n[t]) ok = next_s(t);
                        else if (leader) umma_commit(bar(L::BAR_OFULL + t));
                    }
                }
            } else {
                ok = wait_k();
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (ok && w.n[t] > 0) {
                        ok = tc_wait_warp(bar(L::BAR_QFULL + t), 0, p, abort_flag, kStatusWaitQ);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(t, 0);
                    }
                }
                if (ok && leader) umma_commit(bar(L::BAR_KEMPTY + 0));
                for (int j = 0; j < w.nmax && ok; ++j) {
                    const int buf = j & 1;
                    const bool k_next = j + 1 < w.nmax;
                    const int sk = (j + 1) % L::KSTAGES;
                    bool have_k = false, have_v = false;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!ok || j >= w.n[t]) continue;
                        if (!have_v) {
                            ok = tc_wait_warp(bar(L::BAR_HFULL + buf), (j >> 1) & 1, p, abort_flag, kStatusWaitKvFull);
                            have_v = true;
                        }
                        if (ok) ok = tc_wait_warp(bar(L::BAR_PFULL + t), j & 1, p, abort_flag, kStatusWaitP);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(t, buf, j > 0);
                        if (k_next && !have_k) {
                            ok = wait_k();
                            have_k = true;
                            if (!ok) break;
                            tc_fence_after();
                        }
                        if (j + 1 < w.n[t]) issue_s(t, sk);
                        else if (leader) umma_commit(bar(L::BAR_OFULL + t));
                    }
                    if (!ok) break;
                    if (leader) umma_commit(bar(L::BAR_HEMPTY + buf));
                    if (k_next && leader) umma_commit(bar(L::BAR_KEMPTY + sk));
                }
            }
            if (leader) umma_commit(bar(L::BAR_DRAIN));
            tc_wait(bar(L::BAR_DRAIN), 0, p, abort_flag, kStatusWaitDrain, false);
        } else if (w.live && warp >= L::CONV_WARP0) {
            // -------------------------------------------------------- converters
            // Eight rows a quarter warp apart in their swizzle, so loads and
            // stores are free of bank conflicts. A key that no row of the unit
            // sees becomes zeros: its slot may never have been written, and a
            // weight of zero does not undo a NaN.
            // A lane converts one 16-code unit u of every ROW_STEP-th key from row0
            // on: its addresses are a register and constants.
            constexpr int ROW_STEP = D == 64 ? 32 : 16, PIECES = BN / ROW_STEP;
            const int r8 = lane & 7, cw = WIDE ? warp & 3 : warp - L::CONV_WARP0;
            const int part = WIDE ? (warp - L::CONV_WARP0) >> 2 : 0;  // 128-column part of V
            const int u = D == 64 ? lane >> 3 : (cw & 1) * 4 + (lane >> 3);
            const int row0 = (D == 64 ? cw : cw >> 1) * 8 + r8;
            const uint32_t src_lane = sbase + L::V_OFF + part * L::PART + row0 * L::ROW_BYTES +
                                      ((D == 64 ? u ^ (r8 >> 1) : u ^ r8) << 4);
            const uint32_t dst_lane = sbase + L::V16_OFF + (2 * part + (u >> 2)) * (BN * 128) + row0 * 128 +
                                      (((2 * (u & 3)) ^ r8) << 4);
            const int entries = DUAL ? w.n[0] + w.n[1] : w.nmax;
            const int both = 2 * min(w.n[0], w.n[1]);  // dual: entries that alternate between the slots
            bool ok = true;
            for (int e = 0; e < entries && ok; ++e) {
                const int s = e % L::VSTAGES, buf = WIDE ? 0 : e & 1;
                if (e >= L::VBUFS)
                    ok = tc_wait_warp(bar(L::BAR_HEMPTY + buf), ((WIDE ? e : e >> 1) - 1) & 1, p, abort_flag,
                                      kStatusWaitKvEmpty);
                if (ok)
                    ok = tc_wait_warp(bar(L::BAR_VFULL + s), (e / L::VSTAGES) & 1, p, abort_flag, kStatusWaitKvFull);
                if (!ok) break;
                int at_list = w.i0[0] + e;
                if constexpr (DUAL) {
                    const int t = e < both ? e & 1 : (w.n[1] > w.n[0] ? 1 : 0);
                    const int j = e < both ? e >> 1 : e - both / 2;
                    at_list = (t ? w.i0[1] : w.i0[0]) + j;
                }
                const int key0 = w.list.tile(at_list) * BN;
                const bool whole = key0 + BN - 1 <= w.p1 && (p.window <= 0 || key0 > w.p0 - p.window || key0 + BN <= p.sinks);
                const uint32_t src = src_lane + s * L::SLOT, dst = dst_lane + buf * L::V16;
                // Four pieces' loads are in flight before the first is converted.
                static_for<PIECES / 4>([&](auto batch) {
                    constexpr int P0 = decltype(batch)::value * 4;
                    uint32_t c[4][4];
                    static_for<4>([&](auto k) { ld_shared_v4_at<(P0 + k) * ROW_STEP * L::ROW_BYTES>(c[k], src); });
                    static_for<4>([&](auto k) {
                        if (!whole) {
                            const int key = key0 + row0 + (P0 + k) * ROW_STEP;
                            const bool seen = key <= w.p1 && (p.window <= 0 || key > w.p0 - p.window || key < p.sinks);
                            if (!seen) c[k][0] = c[k][1] = c[k][2] = c[k][3] = 0u;
                        }
                        uint32_t f[8];
#pragma unroll
                        for (int e4 = 0; e4 < 4; ++e4) decode_e4m3x4_f16(c[k][e4], f[2 * e4], f[2 * e4 + 1]);
                        st_shared_v4_at<(P0 + k) * ROW_STEP * 128>(dst, f[0], f[1], f[2], f[3]);
                        st_shared_v4_at<(P0 + k) * ROW_STEP * 128>(dst ^ 16u, f[4], f[5], f[6], f[7]);
                    });
                });
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(L::BAR_HFULL + buf));
                    mbar_arrive(bar(L::BAR_VEMPTY + s));
                }
            }
            // The issuer's last releases must have arrived before the CTA exits.
            for (int e = max(0, entries - L::VBUFS); e < entries && ok; ++e)
                ok = tc_wait_warp(bar(L::BAR_HEMPTY + e % L::VBUFS), (e / L::VBUFS) & 1, p, abort_flag,
                                  kStatusWaitKvEmpty);
        }
    } else {
        // ------------------------------------------------------------ softmax
        setmaxnreg_inc<L::SOFTMAX_REGS>();
        TcWork w;
        tc_work<DUAL, L::WIDE>(p, piece, w);
        const int t = WIDE ? 0 : (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;  // TMEM lane, row of the Q tile
        // Shares: with at most 32 (64) rows, every 32 (64) lanes hold them again,
        // and each copy takes a quarter (half) of the key tile's columns.
        constexpr int shares = DUAL ? SHARES : 1;
        const int tile_row = shares == 4 ? lane : shares == 2 ? r & 63 : r;
        const int share = shares == 4 ? quarter : shares == 2 ? quarter >> 1 : 0;
        const int n = t ? w.n[1] : w.n[0];
        const int first_row = t ? w.row0[1] : w.row0[0];
        const bool part = !DUAL || n > 0;  // whether the slot has a part of the unit
        const int i0 = t ? w.i0[1] : w.i0[0];
        // A warp of a tile that no sequence of the call has rows for leaves its
        // lanes of Q, S and P as they are: those rows of O mean nothing and are
        // not read. It takes no part in the barriers either; polling them would
        // slow the others' shared-memory traffic.
        if (w.live && first_row < w.rows && part && quarter < p.slot_warps) {
            const int row = first_row + tile_row;
            const bool row_ok = row < w.rows;
            const int i = (row_ok ? row : w.rows - 1) / p.G;
            const int head = w.h * p.G + (row_ok ? row : w.rows - 1) - i * p.G;
            const int pos = w.start + i;
            const long long out_row = static_cast<long long>(w.nt.first + i) * p.H + head;
            float rowf = p.scale_log2;
            {
                // Q's two e4m3 terms into the tile's swizzled rows.
                const uint4* src = reinterpret_cast<const uint4*>(p.q + out_row * D);
                uint32_t mx = 0u;
#pragma unroll 4
                for (int u = 0; u < D / 8; ++u) {
                    float x[8];
                    unpack_bf16x8(src[u], x);
                    mx = abs_bits_max(mx, x);
                }
                float f, undo;
                query_scale(mx, f, undo);
                rowf *= undo;
                const uint32_t hi_at = sbase + L::Q_OFF + t * L::Q_TILE + r * L::ROW_BYTES;
#pragma unroll 2
                for (int u = 0; u < (DUAL && t == 1 ? 0 : D / 16); ++u) {
                    float x[16];
                    float(&x0)[8] = *reinterpret_cast<float(*)[8]>(x);
                    float(&x1)[8] = *reinterpret_cast<float(*)[8]>(x + 8);
                    unpack_bf16x8(src[2 * u], x0);
                    unpack_bf16x8(src[2 * u + 1], x1);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float y[4], z[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = x[4 * k + e] * f;
                        hi[k] = pack_e4m3x4(y[0], y[1], y[2], y[3]);
                        decode_e4m3x4(hi[k], z);
                        lo[k] = pack_e4m3x4(y[0] - z[0], y[1] - z[1], y[2] - z[2], y[3] - z[3]);
                    }
                    const uint32_t at = hi_at + (D == 64 ? (u ^ ((r >> 1) & 3)) << 4
                                                         : (u >> 3) * L::PART + (((u & 7) ^ (r & 7)) << 4));
                    st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
                    st_shared_v4(at + L::Q_TERM, lo[0], lo[1], lo[2], lo[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::BAR_QFULL + t));
            }
            const uint32_t lane_field = static_cast<uint32_t>(quarter * 32) << 16;
            const uint32_t tS0 = tmem + lane_field + L::S_COL(t);
            const uint32_t tO = tmem + lane_field + L::O_COL(t);
            const int* table = p.page_table + static_cast<long long>(w.b) * p.max_pages;
            // Scales of the next tile, 16-key group `lane & 7` per lane, loaded a
            // tile ahead; the page-table entries two tiles ahead, and looked at
            // only then (a test right behind the load would wait for it).
            auto entry_of = [&](int j) {
                const int key = j < n ? w.list.tile(i0 + j) * BN + 16 * (lane & 7) : w.nt.len;
                return key < w.nt.len ? table[key >> p.log_page] : -1;
            };
            auto scales_of = [&](int id, float& ks, float& vs) {
                // (The producer reports bad entries.)
                const bool have = id >= 0 && id < p.num_pages;
                const long long cell = static_cast<long long>(id) * p.Hkv + w.h;
                ks = have ? p.k_scale[cell] : 1.f;
                vs = have ? p.v_scale[cell] : 1.f;
            };
            float ks_next, vs_next;
            scales_of(entry_of(0), ks_next, vs_next);
            int id_next = entry_of(1);
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = 0; j < n; ++j) {
                // The groups' factors, before the wait for S: a shuffle between the
                // exponentials would hold each group up.
                const float vs = usable_scale(vs_next);
                const float ks = ks_next, lv = log2f(vs), iv = 1.f / vs;
                float kg[BN / 16], vg[BN / 16], ig[BN / 16];
                if constexpr (!DUAL) {
#pragma unroll
                    for (int g = 0; g < BN / 16; ++g) {
                        kg[g] = __shfl_sync(0xffffffffu, ks, g) * rowf;
                        vg[g] = __shfl_sync(0xffffffffu, lv, g);
                        ig[g] = __shfl_sync(0xffffffffu, iv, g);
                    }
                }
                scales_of(id_next, ks_next, vs_next);
                id_next = entry_of(j + 2);
                const int buf = WIDE ? j & 1 : t;  // S of this tile
                const uint32_t tS = WIDE ? tS0 + buf * BN : tS0;
                ok = tc_wait_warp(bar(L::BAR_SFULL + buf), (WIDE ? j >> 1 : j) & 1, p, abort_flag, kStatusWaitS);
                if (!ok) break;
                tc_fence_after();
                const int key0 = w.list.tile(i0 + j) * BN;
                const int valid = pos - key0 + 1;
                float top = -INFINITY, m_new = m, m_use = 0.f, alpha = 1.f, sum = 0.f;
                auto reference = [&] {
                    const bool move = top > m + kPSlack;
                    m_new = move ? top : m;
                    m_use = m_new == -INFINITY ? 0.f : m_new;
                    alpha = move ? ex2(m - m_use) : 1.f;
                };
                if constexpr (DUAL) {
                    // This share's columns, 32 of S at a time: read once where they
                    // are all of them, else twice (for the maximum, then for the
                    // exponentials) in loops that are not unrolled: where few warps
                    // run this code, long straight stretches of it wait for their
                    // instructions (20 rows without shares: 120 us against 140; the
                    // other way round for full tiles, 2048 and 1642 tokens over 16384
                    // and 9967 keys: 395 against 328).
                    const bool whole = __all_sync(0xffffffffu, valid >= BN && (p.window <= 0 || valid <= p.window ||
                                                                                p.sinks - key0 >= BN));
                    auto chunk = [&](int cc, float (&s)[32], float (&kc)[2], float (&vc)[2]) {
                        uint32_t raw[32];
                        tmem_ld32(tS + cc * 32, raw);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            kc[g] = __shfl_sync(0xffffffffu, ks, 2 * cc + g) * rowf;
                            vc[g] = __shfl_sync(0xffffffffu, lv, 2 * cc + g);
                        }
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[e] = __uint_as_float(raw[e]);
                        if (!whole) {
                            const int end = valid - 32 * cc, from = p.window > 0 ? end - p.window : 0;
                            const uint32_t seen =
                                low_bits(end) & (~low_bits(from) | low_bits(p.sinks - key0 - 32 * cc));
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(seen & (1u << c))) s[c] = -INFINITY;
                        }
                    };
                    auto maximum = [&](const float (&s)[32], const float (&kc)[2], const float (&vc)[2]) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            float a = max3f(s[16 * g], s[16 * g + 1], s[16 * g + 2]);
                            float b = max3f(s[16 * g + 3], s[16 * g + 4], s[16 * g + 5]);
                            a = max3f(a, s[16 * g + 6], s[16 * g + 7]);
                            b = max3f(b, s[16 * g + 8], s[16 * g + 9]);
                            a = max3f(a, s[16 * g + 10], s[16 * g + 11]);
                            b = max3f(b, s[16 * g + 12], s[16 * g + 13]);
                            a = max3f(a, s[16 * g + 14], s[16 * g + 15]);
                            top = fmaxf(top, fmaf(fmaxf(a, b), kc[g], vc[g]));
                        }
                    };
                    auto exponentials = [&](int cc, const float (&s)[32], const float (&kc)[2], const float (&vc)[2]) {
                        uint32_t pk[16];
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const float ng = vc[g] - m_use + kPShift;
                            const uint64_t k2 = f2pack(kc[g], kc[g]), n2 = f2pack(ng, ng);
                            uint64_t part[2] = {0ull, 0ull};
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int c = 16 * g + 2 * e;
                                float x0, x1;
                                f2unpack(ffma2(f2pack(s[c], s[c + 1]), k2, n2), x0, x1);
                                const float e0 = ex2(x0), e1 = ex2(x1);
                                part[e & 1] = fadd2(part[e & 1], f2pack(e0, e1));
                                pk[8 * g + e] = pack_f16x2(e0, e1);
                            }
                            float a, b;
                            f2unpack(fadd2(part[0], part[1]), a, b);
                            sum = fmaf(a + b, __shfl_sync(0xffffffffu, iv, 2 * cc + g), sum);
                        }
                        // P's 16 columns lie over S columns that have been read.
                        tmem_st16(tS + cc * 16, pk);
                    };
                    const uint32_t zero[16] = {};
                    if constexpr (shares == 4) {
                        float s[32], kc[2], vc[2];
                        chunk(share, s, kc, vc);
                        // The weights of the other shares' keys are zero for these
                        // rows.
#pragma unroll
                        for (int cc = 1; cc < 4; ++cc) tmem_st16(tS + ((share + cc) & 3) * 16, zero);
                        maximum(s, kc, vc);
                        reference();
                        exponentials(share, s, kc, vc);
                    } else {
                        const int c0 = 2 * share, c1 = shares == 2 ? c0 + 2 : BN / 32;
#pragma unroll 1
                        for (int cc = c0; cc < c1; ++cc) {
                            float s[32], kc[2], vc[2];
                            chunk(cc, s, kc, vc);
                            maximum(s, kc, vc);
                        }
                        reference();
#pragma unroll 1
                        for (int cc = c0; cc < c1; ++cc) {
                            float s[32], kc[2], vc[2];
                            chunk(cc, s, kc, vc);
                            exponentials(cc, s, kc, vc);
                        }
                        if constexpr (shares == 2) {
#pragma unroll
                            for (int cc = 0; cc < 2; ++cc) tmem_st16(tS + ((c0 ^ 2) + cc) * 16, zero);
                        }
                    }
                } else {
                    float s[BN];
#pragma unroll
                    for (int cc = 0; cc < BN / 32; ++cc) {
                        uint32_t raw[32];
                        tmem_ld32(tS + cc * 32, raw);
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[cc * 32 + e] = __uint_as_float(raw[e]);
                    }
                    tmem_wait_ld();
                    const int from = p.window > 0 ? valid - p.window : 0, sink = p.sinks - key0;
                    if (valid < BN || (from > 0 && sink < BN)) {
                        // One bit per key: half the instructions of comparisons.
#pragma unroll
                        for (int g = 0; g < BN / 32; ++g) {
                            const uint32_t seen =
                                low_bits(valid - 32 * g) & (~low_bits(from - 32 * g) | low_bits(sink - 32 * g));
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(seen & (1u << c))) s[32 * g + c] = -INFINITY;
                        }
                    }
                    __syncwarp();
                    // Row maximum of x = s (rowf ks) + log2 vs, group by group.
#pragma unroll
                    for (int g = 0; g < BN / 16; ++g) {
                        float a = max3f(s[16 * g], s[16 * g + 1], s[16 * g + 2]);
                        float b = max3f(s[16 * g + 3], s[16 * g + 4], s[16 * g + 5]);
                        a = max3f(a, s[16 * g + 6], s[16 * g + 7]);
                        b = max3f(b, s[16 * g + 8], s[16 * g + 9]);
                        a = max3f(a, s[16 * g + 10], s[16 * g + 11]);
                        b = max3f(b, s[16 * g + 12], s[16 * g + 13]);
                        a = max3f(a, s[16 * g + 14], s[16 * g + 15]);
                        top = fmaxf(top, fmaf(fmaxf(a, b), kg[g], vg[g]));
                    }
                    reference();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[32];
#pragma unroll
                        for (int gg = 0; gg < 4; ++gg) {
                            const int g = 4 * h + gg;
                            const float ng = vg[g] - m_use + kPShift;
                            const uint64_t k2 = f2pack(kg[g], kg[g]), n2 = f2pack(ng, ng);
                            uint64_t part[2] = {0ull, 0ull};
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int c = 16 * g + 2 * e;
                                float x0, x1;
                                f2unpack(ffma2(f2pack(s[c], s[c + 1]), k2, n2), x0, x1);
                                const float e0 = ex2(x0), e1 = ex2(x1);
                                part[e & 1] = fadd2(part[e & 1], f2pack(e0, e1));
                                pk[8 * gg + e] = pack_f16x2(e0, e1);
                            }
                            float a, b;
                            f2unpack(fadd2(part[0], part[1]), a, b);
                            sum = fmaf(a + b, ig[g], sum);
                        }
                        tmem_st32(tS + h * 32, pk);
                    }
                }
                if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    if constexpr (WIDE) {  // (elsewhere S_j comes behind PV_{j-1})
                        ok = tc_wait_warp(bar(L::BAR_OFULL + wide_pv_barrier(j - 1, n)), wide_pv_parity(j - 1, n), p,
                                          abort_flag, kStatusWaitO);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    const uint64_t ax2 = f2pack(alpha, alpha);
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        tmem_ld32(tO + cc * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x0, x1;
                            f2unpack(fmul2(f2pack(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), ax2), x0, x1);
                            o[2 * e] = __float_as_uint(x0);
                            o[2 * e + 1] = __float_as_uint(x1);
                        }
                        tmem_st32(tO + cc * 32, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::BAR_PFULL + buf));
                l = fmaf(l, alpha, sum);
                m = m_new;
            }
            if (ok && n > 0) {
                ok = tc_wait_warp(bar(L::BAR_OFULL + (WIDE ? wide_pv_barrier(n - 1, n) : t)),
                                  WIDE ? wide_pv_parity(n - 1, n) : 0u, p, abort_flag, kStatusWaitO);
                if (ok) tc_fence_after();
            }
            if constexpr (DUAL) {
                // The states of both slots' rows and their shares meet in shared
                // memory, which no copy or MMA of this CTA uses any more once all of
                // them have come here. (A warp that gave up comes here as well.)
                constexpr int UNITS = D / 4;  // float4 units of a row
                const int slots = w.n[1] > 0 ? 2 : 1, warps = p.slot_warps * slots;
                auto meet = [&] { asm volatile("bar.sync 1, %0;" ::"r"(32 * warps) : "memory"); };
                meet();
                float4* stage = reinterpret_cast<float4*>(smem);
                float* ml = reinterpret_cast<float*>(smem + L::ML_OFF);  // [slot][m, l][128 lanes]
                if (ok) {
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        tmem_ld32(tO + cc * 32, o);
                        tmem_wait_ld();
                        // (Units swapped row by row: no bank conflicts.)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            stage[(t * 128 + r) * UNITS + ((cc * 8 + e) ^ (lane & (UNITS - 1)))] =
                                make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                            __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                    }
                    ml[t * 256 + r] = state_ref(m, l);
                    ml[t * 256 + 128 + r] = l;
                }
                meet();
                const int here = min(kTcRows, w.rows - first_row);
                // (Warp `quarter` of slot t is t * slot_warps + quarter of them all.)
                for (int u = (t * p.slot_warps + quarter) * 32 + lane; u < here * UNITS && !*abort_flag; u += 32 * warps) {
                    const int rr = u / UNITS, c = u - rr * UNITS;
                    float mm = -INFINITY, ll = 0.f;
                    // A row's copies lie 128 / shares lanes apart.
                    for (int s = 0; s < slots; ++s)
                        for (int x = 0; x < shares; ++x) mm = fmaxf(mm, ml[s * 256 + rr + x * (128 / shares)]);
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int s = 0; s < slots; ++s)
                        for (int x = 0; x < shares; ++x) {
                            const int at = rr + x * (128 / shares);
                            const float ms = ml[s * 256 + at];
                            const float f = ms == -INFINITY ? 0.f : ex2(ms - mm);
                            const float4 y = stage[(s * 128 + at) * UNITS + (c ^ (at & 31 & (UNITS - 1)))];
                            ll = fmaf(f, ml[s * 256 + 128 + at], ll);
                            a.x = fmaf(f, y.x, a.x), a.y = fmaf(f, y.y, a.y), a.z = fmaf(f, y.z, a.z),
                            a.w = fmaf(f, y.w, a.w);
                        }
                    const int qi = (first_row + rr) / p.G, qh = w.h * p.G + (first_row + rr) - qi * p.G;
                    const long long to = static_cast<long long>(w.nt.first + qi) * p.H + qh;
                    // States that the row does not use are marked as empty for the
                    // merge.
                    if (w.split == 0 && p.num_splits > 1)
                        for (int s = (w.used == 1 ? 0 : w.used) + c; s < p.num_splits; s += UNITS)
                            p.ws_m[static_cast<long long>(s) * p.total_q * p.H + to] = -INFINITY;
                    if (w.used == 1) {
                        const float inv = ll == 0.f ? 0.f : 1.f / ll;
                        *reinterpret_cast<uint2*>(p.o + to * D + 4 * c) =
                            make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
                        if (c == 0)
                            p.lse[static_cast<long long>(qh) * p.total_q + w.nt.first + qi] = state_lse(mm, ll);
                    } else {
                        const long long at = static_cast<long long>(w.split) * p.total_q * p.H + to;
                        *reinterpret_cast<float4*>(p.ws_o + at * D + 4 * c) = a;
                        if (c == 0) {
                            p.ws_m[at] = state_ref(mm, ll);
                            p.ws_l[at] = ll;
                        }
                    }
                }
            } else if (ok) {
                const float f = w.used == 1 ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                const long long at = static_cast<long long>(w.split) * p.total_q * p.H + out_row;
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    __syncwarp();  // rows past the last one skip the stores below
                    if (n > 0) {
                        tmem_ld32(tO + cc * 32, o);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    }
                    if (!row_ok) continue;
                    if (w.used == 1) {
                        uint4* dst = reinterpret_cast<uint4*>(p.o + out_row * D + cc * 32);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t x[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                x[k] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * k]) * f,
                                                   __uint_as_float(o[8 * e + 2 * k + 1]) * f);
                            dst[e] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(p.ws_o + at * D + cc * 32);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
                if (row_ok) {
                    // States that the row does not use are marked as empty for the
                    // merge.
                    if (w.split == 0 && p.num_splits > 1)
                        for (int s = w.used == 1 ? 0 : w.used; s < p.num_splits; ++s)
                            p.ws_m[static_cast<long long>(s) * p.total_q * p.H + out_row] = -INFINITY;
                    if (w.used == 1) {
                        p.lse[static_cast<long long>(head) * p.total_q + w.nt.first + i] =
                            state_lse(m, l);
                    } else {
                        p.ws_m[at] = state_ref(m, l);
                        p.ws_l[at] = l;
                    }
                }
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D, int SHARES>
cudaError_t launch_tc(const PagedParams& p, cudaStream_t stream) {
    using L = TcLayout<D, SHARES>;
    static ContextCache<int> attr_set;
    int done = 0;
    const cudaError_t e = attr_set.get(&done, [](int* out) {
        // The setmaxnreg split is sized for exactly LAUNCH_REGS per thread.
        cudaFuncAttributes a;
        cudaError_t err = cudaFuncGetAttributes(&a, fa_paged_tc_kernel<D, SHARES>);
        if (err != cudaSuccess) return err;
        if (a.numRegs != L::LAUNCH_REGS) return cudaErrorInvalidKernelImage;
        *out = 1;
        return cudaFuncSetAttribute(fa_paged_tc_kernel<D, SHARES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(L::ALLOC));
    });
    if (e != cudaSuccess) return e;
    const long long ctas = static_cast<long long>(p.B) * p.Hkv * p.num_splits * p.row_blocks;
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    return launch_dependent(fa_paged_tc_kernel<D, SHARES>, dim3(static_cast<unsigned>(ctas)), L::THREADS, L::ALLOC,
                            stream, p);
}

}  // namespace

cudaError_t launch_paged_tc(const PagedParams& p, int d, cudaStream_t stream) {
    auto launch = [&](auto d_) {
        constexpr int D = decltype(d_)::value;
        return p.shares == 0   ? launch_tc<D, 0>(p, stream)
               : p.shares == 1 ? launch_tc<D, 1>(p, stream)
               : p.shares == 2 ? launch_tc<D, 2>(p, stream)
                               : launch_tc<D, 4>(p, stream);
    };
    if (d == 256) return launch_tc<256, 0>(p, stream);
    return d == 64 ? launch(Index<64>{}) : launch(Index<128>{});
}

}  // namespace fa
