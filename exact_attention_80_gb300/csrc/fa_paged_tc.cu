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
//     over its S columns, V converted from its codes (exact) by two warps that
//     the dense forward leaves idle, once per key tile for both row tiles.
// The block scales enter where fa_paged.cu has them: the K scale multiplies the
// score, log2 of the V scale adds to the exponent, and the row sum takes its
// reciprocal; scores are handled in groups of 16 keys, the smallest page.
//
// Roles, by warp: 0 producer (Q is written by the softmax threads; K and V pages
// by TMA into two rings), 1 issuer, 2-3 converters, 4-11 softmax (thread = row
// = TMEM lane). Step j, per tile as its P arrives: O_t += P_t(j) V_j, then at
// once S_t(j+1) over the same columns. Every wait is bounded as in the dense
// forward.
#include <cuda_bf16.h>

#include "fa.h"
#include "fa_paged.cuh"
#include "fa_rope.cuh"

namespace fa {
namespace {

template <int D>
struct TcLayout {
    static constexpr int BM = 128, BN = kTcKeys;
    static constexpr int ROW_BYTES = D < 128 ? D : 128;   // swizzled row of codes
    static constexpr int KSTAGES = D == 64 ? 4 : 3;
    static constexpr int VSTAGES = D == 64 ? 4 : 2;
    static constexpr int THREADS = 384;
    static constexpr uint32_t Q_TERM = BM * D;            // one e4m3 term of a row tile
    static constexpr uint32_t Q_TILE = 2 * Q_TERM;
    static constexpr uint32_t SLOT = BN * D;              // codes of a K or V tile
    static constexpr uint32_t V16 = BN * D * 2;           // V tile in f16: 64-column chunks of 128-byte rows
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t K_OFF = Q_OFF + 2 * Q_TILE;
    static constexpr uint32_t V_OFF = K_OFF + KSTAGES * SLOT;
    static constexpr uint32_t V16_OFF = V_OFF + VSTAGES * SLOT;
    static constexpr uint32_t BAR_OFF = V16_OFF + 2 * V16;
    static constexpr int BAR_QFULL = 0;                    // [tile] one arrival per softmax warp
    static constexpr int BAR_KFULL = 2;
    static constexpr int BAR_KEMPTY = BAR_KFULL + KSTAGES;
    static constexpr int BAR_VFULL = BAR_KEMPTY + KSTAGES;
    static constexpr int BAR_VEMPTY = BAR_VFULL + VSTAGES;   // one arrival per converter warp
    static constexpr int BAR_HFULL = BAR_VEMPTY + VSTAGES;   // [buffer] V in f16 (one arrival per converter warp)
    static constexpr int BAR_HEMPTY = BAR_HFULL + 2;         // [buffer]
    static constexpr int BAR_SFULL = BAR_HEMPTY + 2;         // [tile]
    static constexpr int BAR_PFULL = BAR_SFULL + 2;          // [tile] one arrival per softmax warp
    static constexpr int BAR_OFULL = BAR_PFULL + 2;          // [tile]
    static constexpr int BAR_DRAIN = BAR_OFULL + 2;
    static constexpr int NUM_BARS = BAR_DRAIN + 1;
    static constexpr uint32_t MISC_OFF = BAR_OFF + NUM_BARS * 8;
    static constexpr uint32_t BYTES = MISC_OFF + 16;
    static constexpr size_t ALLOC = BYTES + 1024;
    // TMEM columns: S_t (P_t over its first half), then O_t.
    __host__ __device__ static constexpr uint32_t S_COL(int t) { return t * BN; }
    __host__ __device__ static constexpr uint32_t O_COL(int t) { return 256 + t * D; }
    static constexpr int LAUNCH_REGS = 168, CTRL_REGS = 88, SOFTMAX_REGS = 208;
    static_assert(128 * CTRL_REGS + 256 * SOFTMAX_REGS == THREADS * LAUNCH_REGS, "register split");
    static_assert(ALLOC <= 232448, "shared memory over the 227 KB per-CTA limit");
    static_assert(ALLOC > 232448 / 2, "two CTAs per SM would contend for TMEM");
    static_assert(256 + 2 * D <= 512, "O overflows TMEM");
};

// kind::f16 with f16 operands (format code 0), fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

struct TcWork {
    NewTokens nt;
    int b, h, rows, start, used, split;
    int row0[2];   // first row of each tile slot
    KeyList list;
    int i0;        // first list entry of the split
    int n[2];      // key tiles each row tile visits
    int nmax;
    int p0, p1;    // positions of the unit's first and last row
    bool live;
};

__device__ __forceinline__ void tc_work(const PagedParams& p, TcWork& w) {
    unsigned lin = blockIdx.x;
    w.split = static_cast<int>(lin % p.num_splits);
    lin /= p.num_splits;
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
    const int r0 = unit * kTcRows;
    w.live = r0 < w.rows;
    if (!w.live) return;
    w.start = w.nt.len - w.nt.n;
    w.p0 = w.start + r0 / p.G;
    w.p1 = w.start + (min(r0 + kTcRows, w.rows) - 1) / p.G;
    w.list = key_list<kTcKeys>(p.window, p.sinks, w.p0, w.p1);
    w.used = max(1, (w.list.n + p.tiles_per_split - 1) / p.tiles_per_split);
    w.live = w.split < w.used;
    if (!w.live) return;
    w.i0 = w.split * p.tiles_per_split;
    const int i1 = min(w.list.n, w.i0 + p.tiles_per_split);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        // Slot 0 takes the later rows, whose tile ends last: the issuer serves
        // it first.
        w.row0[t] = r0 + (1 - t) * 128;
        if (w.row0[t] >= w.rows) continue;
        const int last = w.start + (min(w.row0[t] + 128, w.rows) - 1) / p.G;
        const int end = w.list.ns + max(0, last / kTcKeys + 1 - w.list.lo);
        w.n[t] = max(0, min(i1, end) - w.i0);
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

template <int D>
__global__ void __launch_bounds__(TcLayout<D>::THREADS, 1) fa_paged_tc_kernel(const __grid_constant__ PagedParams p) {
    using L = TcLayout<D>;
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
            mbar_init(bar(L::BAR_VEMPTY + s), 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(L::BAR_HFULL + t), 2);
            mbar_init(bar(L::BAR_HEMPTY + t), 1);
            mbar_init(bar(L::BAR_QFULL + t), 4);
            mbar_init(bar(L::BAR_SFULL + t), 1);
            mbar_init(bar(L::BAR_PFULL + t), 4);
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
    if (warp == 1) {
        tmem_alloc(sbase + L::MISC_OFF, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];

    if (warp < 4) {
        setmaxnreg_dec<L::CTRL_REGS>();
        TcWork w;
        tc_work(p, w);
        if (w.live && warp == 0) {
            // -------------------------------------------------------- producer
            // Entry e: K_0; then per step j: V_j, K_{j+1}. A tile's pages are
            // copied one by one; pages behind the sequence's end are left out.
            const bool leader = elect_one();
            const int* table = p.page_table + static_cast<long long>(w.b) * p.max_pages;
            const int per = BN >> p.log_page;  // pages per tile (page_size <= 128)
            const uint32_t page_bytes = static_cast<uint32_t>(D) << p.log_page;
            auto ids_of = [&](int j) {  // lane i: page i of the tile of step j
                return j < w.nmax && lane < per
                           ? tc_page(p, w, table, w.list.tile(w.i0 + j) * BN + (lane << p.log_page))
                           : -1;
            };
            auto copy = [&](const CUtensorMap* map, uint32_t dst, uint32_t full, int ids) {
                const unsigned here = __ballot_sync(0xffffffffu, ids >= 0);
                if (leader) mbar_arrive_expect_tx(full, __popc(here) * page_bytes);
                for (int i = 0; i < per; ++i) {
                    const int id = __shfl_sync(0xffffffffu, ids, i);
                    if (id >= 0 && leader)
                        tma_load_2d(dst + i * page_bytes, map, full, 0, (id * p.Hkv + w.h) << p.log_page);
                }
            };
            int ids_k = ids_of(0), ids_v = ids_k;
            int k_issued = 0, v_issued = 0;
            bool ok = true;
            auto load_k = [&]() -> bool {
                const int s = k_issued % L::KSTAGES;
                if (k_issued >= L::KSTAGES &&
                    !tc_wait_warp(bar(L::BAR_KEMPTY + s), (k_issued / L::KSTAGES - 1) & 1, p, abort_flag,
                                  kStatusWaitKvEmpty))
                    return false;
                copy(&p.tm_k, sbase + L::K_OFF + s * L::SLOT, bar(L::BAR_KFULL + s), ids_k);
                ++k_issued;
                return true;
            };
            if (w.nmax > 0) ok = load_k();
            for (int j = 0; j < w.nmax && ok; ++j) {
                ids_k = ids_of(j + 1);
                const int s = v_issued % L::VSTAGES;
                if (v_issued >= L::VSTAGES)
                    ok = tc_wait_warp(bar(L::BAR_VEMPTY + s), (v_issued / L::VSTAGES - 1) & 1, p, abort_flag,
                                      kStatusWaitKvEmpty);
                if (!ok) break;
                copy(&p.tm_v, sbase + L::V_OFF + s * L::SLOT, bar(L::BAR_VFULL + s), ids_v);
                ++v_issued;
                if (j + 1 < w.nmax) ok = load_k();
                ids_v = ids_k;
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
                const uint32_t qa = L::Q_OFF + t * L::Q_TILE, kb = L::K_OFF + slot * L::SLOT;
#pragma unroll
                for (int term = 0; term < 2; ++term)
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk)
                        if (leader)
                            umma_ss_f8(tmem + L::S_COL(t), desc(kmaj_lo, kmaj_hi, qa + term * L::Q_TERM + kk * 32),
                                       desc(kmaj_lo, kmaj_hi, kb + kk * 32), IDESC_S, (term | kk) ? 1u : 0u);
                if (leader) umma_commit(bar(L::BAR_SFULL + t));
            };
            auto issue_pv = [&](int t, int buf, bool accumulate) {
                const uint32_t vb = L::V16_OFF + buf * L::V16;
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                    if (leader)
                        umma_ts(tmem + L::O_COL(t), tmem + L::S_COL(t) + kk * 8, desc(vmn_lo, vmn_hi, vb + kk * 2048),
                                IDESC_O, (accumulate || kk > 0) ? 1u : 0u);
            };
            int k_used = 0;  // K entries waited for
            auto wait_k = [&]() -> bool {
                const bool r = tc_wait_warp(bar(L::BAR_KFULL + k_used % L::KSTAGES), (k_used / L::KSTAGES) & 1, p,
                                            abort_flag, kStatusWaitKvFull);
                ++k_used;
                return r;
            };
            bool ok = wait_k();
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
            if (leader) umma_commit(bar(L::BAR_DRAIN));
            tc_wait(bar(L::BAR_DRAIN), 0, p, abort_flag, kStatusWaitDrain, false);
        } else if (w.live && warp >= 2) {
            // -------------------------------------------------------- converters
            // Eight rows a quarter warp apart in their swizzle, so loads and
            // stores are free of bank conflicts. A key that no row of the unit
            // sees becomes zeros: its slot may never have been written, and a
            // weight of zero does not undo a NaN.
            constexpr int UNITS = D / 16;  // 16-code units per key
            bool ok = true;
            for (int j = 0; j < w.nmax && ok; ++j) {
                const int s = j % L::VSTAGES, buf = j & 1;
                if (j >= 2) ok = tc_wait_warp(bar(L::BAR_HEMPTY + buf), ((j >> 1) - 1) & 1, p, abort_flag, kStatusWaitKvEmpty);
                if (ok) ok = tc_wait_warp(bar(L::BAR_VFULL + s), (j / L::VSTAGES) & 1, p, abort_flag, kStatusWaitKvFull);
                if (!ok) break;
                const int key0 = w.list.tile(w.i0 + j) * BN;
                const bool whole = key0 + BN - 1 <= w.p1 && (p.window <= 0 || key0 > w.p0 - p.window || key0 + BN <= p.sinks);
                const uint32_t src = sbase + L::V_OFF + s * L::SLOT, dst = sbase + L::V16_OFF + buf * L::V16;
                const int r8 = lane & 7;
#pragma unroll 4
                for (int i = (warp - 2) * 4 + (lane >> 3); i < (BN / 8) * UNITS; i += 8) {
                    const int u = i % UNITS, r = (i / UNITS) * 8 + r8;
                    const uint32_t at = D == 64 ? src + r * 64 + ((u ^ ((r >> 1) & 3)) << 4)
                                                : src + r * 128 + ((u ^ r8) << 4);
                    uint32_t c[4];
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
                                 : "r"(at)
                                 : "memory");
                    if (!whole) {
                        const int key = key0 + r;
                        const bool seen = key <= w.p1 && (p.window <= 0 || key > w.p0 - p.window || key < p.sinks);
                        if (!seen) c[0] = c[1] = c[2] = c[3] = 0u;
                    }
                    uint32_t f[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        f[2 * k] = decode_e4m3x2_f16(static_cast<uint16_t>(c[k] & 0xffffu));
                        f[2 * k + 1] = decode_e4m3x2_f16(static_cast<uint16_t>(c[k] >> 16));
                    }
                    const uint32_t line = dst + (u >> 2) * (BN * 128) + r * 128;
                    st_shared_v4(line + (((2 * (u & 3)) ^ r8) << 4), f[0], f[1], f[2], f[3]);
                    st_shared_v4(line + (((2 * (u & 3) + 1) ^ r8) << 4), f[4], f[5], f[6], f[7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(L::BAR_HFULL + buf));
                    mbar_arrive(bar(L::BAR_VEMPTY + s));
                }
            }
            // The issuer's last releases must have arrived before the CTA exits.
            for (int j = max(0, w.nmax - 2); j < w.nmax && ok; ++j)
                ok = tc_wait_warp(bar(L::BAR_HEMPTY + (j & 1)), (j >> 1) & 1, p, abort_flag, kStatusWaitKvEmpty);
        }
    } else {
        // ------------------------------------------------------------ softmax
        setmaxnreg_inc<L::SOFTMAX_REGS>();
        TcWork w;
        tc_work(p, w);
        const int t = (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const int n = t ? w.n[1] : w.n[0];
        const int first_row = t ? w.row0[1] : w.row0[0];
        if (w.live && first_row < w.rows) {
            const int row = first_row + r;
            const bool row_ok = row < w.rows;
            const int i = (row_ok ? row : w.rows - 1) / p.G;
            const int head = w.h * p.G + (row_ok ? row : w.rows - 1) - i * p.G;
            const int pos = w.start + i;
            const long long out_row = static_cast<long long>(w.nt.first + i) * p.H + head;
            float rowf = p.scale_log2;
            {
                // Q's two e4m3 terms into the tile's swizzled rows.
                const uint4* src = reinterpret_cast<const uint4*>(p.q + out_row * D);
                float mx = 0.f;
#pragma unroll 4
                for (int u = 0; u < D / 8; ++u) {
                    float x[8];
                    unpack_bf16x8(src[u], x);
#pragma unroll
                    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(x[k]));
                }
                const int ex = mx > 0.f ? min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100), 120) : 0;
                const float f = exp2i(min(7 - ex, 120));
                rowf *= 1.f / f;
                const uint32_t hi_at = sbase + L::Q_OFF + t * L::Q_TILE + r * L::ROW_BYTES;
#pragma unroll 2
                for (int u = 0; u < D / 16; ++u) {
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
                    const uint32_t at = hi_at + (D == 64 ? (u ^ ((r >> 1) & 3)) << 4 : (u ^ (r & 7)) << 4);
                    st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
                    st_shared_v4(at + L::Q_TERM, lo[0], lo[1], lo[2], lo[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::BAR_QFULL + t));
            }
            const uint32_t lane_field = static_cast<uint32_t>(quarter * 32) << 16;
            const uint32_t tS = tmem + lane_field + L::S_COL(t);
            const uint32_t tO = tmem + lane_field + L::O_COL(t);
            const int* table = p.page_table + static_cast<long long>(w.b) * p.max_pages;
            // Scales of the next tile, 16-key group `lane & 7` per lane, loaded a
            // tile ahead; the page ids two tiles ahead.
            auto id_of = [&](int j) {
                return j < n ? tc_page(p, w, table, w.list.tile(w.i0 + j) * BN + 16 * (lane & 7)) : -1;
            };
            auto scales_of = [&](int id, float& ks, float& vs) {
                const long long cell = static_cast<long long>(id) * p.Hkv + w.h;
                ks = id >= 0 ? p.k_scale[cell] : 1.f;
                vs = id >= 0 ? p.v_scale[cell] : 1.f;
            };
            float ks_next, vs_next;
            scales_of(id_of(0), ks_next, vs_next);
            int id_next = id_of(1);
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = 0; j < n; ++j) {
                const float ks = ks_next, lv = log2f(vs_next), iv = 1.f / vs_next;
                scales_of(id_next, ks_next, vs_next);
                id_next = id_of(j + 2);
                ok = tc_wait_warp(bar(L::BAR_SFULL + t), j & 1, p, abort_flag, kStatusWaitS);
                if (!ok) break;
                tc_fence_after();
                float s[BN];
#pragma unroll
                for (int cc = 0; cc < BN / 32; ++cc) {
                    uint32_t raw[32];
                    tmem_ld32(tS + cc * 32, raw);
#pragma unroll
                    for (int e = 0; e < 32; ++e) s[cc * 32 + e] = __uint_as_float(raw[e]);
                }
                tmem_wait_ld();
                const int key0 = w.list.tile(w.i0 + j) * BN;
                const int valid = pos - key0 + 1;
                if (valid < BN) {
#pragma unroll
                    for (int c = 0; c < BN; ++c)
                        if (c >= valid) s[c] = -INFINITY;
                }
                if (p.window > 0) {
                    const int from = valid - p.window, sink = p.sinks - key0;
                    if (from > 0 && sink < BN) {
#pragma unroll
                        for (int c = 0; c < BN; ++c)
                            if (c < from && c >= sink) s[c] = -INFINITY;
                    }
                }
                __syncwarp();
                // Row maximum of x = s (rowf ks) + log2 vs, group by group.
                float top = -INFINITY;
#pragma unroll
                for (int g = 0; g < BN / 16; ++g) {
                    const float kg = __shfl_sync(0xffffffffu, ks, g) * rowf, vg = __shfl_sync(0xffffffffu, lv, g);
                    float a = max3f(s[16 * g], s[16 * g + 1], s[16 * g + 2]);
                    float b = max3f(s[16 * g + 3], s[16 * g + 4], s[16 * g + 5]);
                    a = max3f(a, s[16 * g + 6], s[16 * g + 7]);
                    b = max3f(b, s[16 * g + 8], s[16 * g + 9]);
                    a = max3f(a, s[16 * g + 10], s[16 * g + 11]);
                    b = max3f(b, s[16 * g + 12], s[16 * g + 13]);
                    a = max3f(a, s[16 * g + 14], s[16 * g + 15]);
                    top = fmaxf(top, fmaf(fmaxf(a, b), kg, vg));
                }
                const bool move = top > m + kPSlack;
                const float m_new = move ? top : m;
                const float m_use = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = move ? ex2(m - m_use) : 1.f;
                float sum = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[32];
#pragma unroll
                    for (int gg = 0; gg < 4; ++gg) {
                        const int g = 4 * h + gg;
                        const float kg = __shfl_sync(0xffffffffu, ks, g) * rowf;
                        const float ng = __shfl_sync(0xffffffffu, lv, g) - m_use + kPShift;
                        const uint64_t k2 = f2pack(kg, kg), n2 = f2pack(ng, ng);
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
                        sum = fmaf(a + b, __shfl_sync(0xffffffffu, iv, g), sum);
                    }
                    tmem_st32(tS + h * 32, pk);
                }
                if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
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
                if (lane == 0) mbar_arrive(bar(L::BAR_PFULL + t));
                l = fmaf(l, alpha, sum);
                m = m_new;
            }
            if (ok && n > 0) {
                ok = tc_wait_warp(bar(L::BAR_OFULL + t), 0, p, abort_flag, kStatusWaitO);
                if (ok) tc_fence_after();
            }
            if (ok) {
                const float f = w.used == 1 ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
                const long long at = static_cast<long long>(w.split) * p.total_q * p.H + out_row;
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
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
                    if (w.used == 1) {
                        p.lse[static_cast<long long>(head) * p.total_q + w.nt.first + i] =
                            l > 0.f ? (m - kPShift + log2f(l)) * 0.69314718055994530942f : -INFINITY;
                    } else {
                        p.ws_m[at] = l > 0.f ? m : -INFINITY;
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

template <int D>
cudaError_t launch_tc(const PagedParams& p, cudaStream_t stream) {
    using L = TcLayout<D>;
    static ContextCache<int> attr_set;
    int done = 0;
    const cudaError_t e = attr_set.get(&done, [](int* out) {
        // The setmaxnreg split is sized for exactly LAUNCH_REGS per thread.
        cudaFuncAttributes a;
        cudaError_t err = cudaFuncGetAttributes(&a, fa_paged_tc_kernel<D>);
        if (err != cudaSuccess) return err;
        if (a.numRegs != L::LAUNCH_REGS) return cudaErrorInvalidKernelImage;
        *out = 1;
        return cudaFuncSetAttribute(fa_paged_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(L::ALLOC));
    });
    if (e != cudaSuccess) return e;
    const long long ctas = static_cast<long long>(p.B) * p.Hkv * p.num_splits * p.row_blocks;
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    return launch_dependent(fa_paged_tc_kernel<D>, dim3(static_cast<unsigned>(ctas)), L::THREADS, L::ALLOC, stream, p);
}

}  // namespace

cudaError_t launch_paged_tc(const PagedParams& p, int d, cudaStream_t stream) {
    return d == 64 ? launch_tc<64>(p, stream) : launch_tc<128>(p, stream);
}

}  // namespace fa
