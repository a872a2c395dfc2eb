// fa_fwd_win.cuh — what a sliding window with sinks changes in the forward
// kernels: the list of key tiles a unit visits, and the control warps of the
// two-tile kernel.
//
// Query row i has position p = i + Nk - Nq and sees key j iff j <= p and (no
// window, or j > p - window, or j < sinks). The key tiles of a unit are then
// the tiles of the sinks and, behind a gap, the tiles from its first row's
// window to its last row's position. Step j of a unit works on one tile of
// that list; both query tiles of a CTA share the steps (and each K/V load), but
// the later rows' tile has no part in the window tiles that only the earlier
// rows see (a hole right behind the sinks), and the earlier rows' tile ends
// before the list does. Heads share kv heads in groups of H / Hkv.
#pragma once

#include "fa_fwd_common.cuh"

namespace fa {

struct WinList {
    int ns, lo, n;  // tiles 0 .. ns - 1, then tile lo on; n in all
    __device__ __forceinline__ int tile(int j) const { return j < ns ? j : lo + (j - ns); }
};

// The list of rows at positions p0 .. p1 (p0 may be negative: rows with no key).
template <int BN>
__device__ __forceinline__ WinList win_list(const FwdParams& p, int p0, int p1) {
    WinList w;
    w.ns = 0;
    w.lo = 0;
    const int end = p1 < 0 ? 0 : p1 / BN + 1;
    if (p.window > 0) {
        const int first = max(0, p0 - p.window + 1) / BN;
        const int st = min((p.sinks + BN - 1) / BN, end);
        if (first > st) {
            w.ns = st;
            w.lo = first;
        }
    }
    w.n = w.ns + max(0, end - w.lo);
    return w;
}

template <int QT>
struct WorkWin : Work<QT> {
    int zk;           // head coordinate of the K/V tensor maps
    WinList list;
    int hole[QT];     // steps ns .. ns + hole - 1 are not the tile's
    int steps[QT];    // steps the tile has a part in: n - hole
};

template <int QT, int BN>
__device__ __forceinline__ void compute_work_win(const FwdParams& p, long long lin, WorkWin<QT>& w) {
    // As compute_work (one split, dense): head groups, units heaviest first.
    const long long per_group = static_cast<long long>(p.head_group) * p.n_units;
    const int group = static_cast<int>(lin / per_group);
    const int r = static_cast<int>(lin % per_group);
    const int heads_here = min(p.head_group, p.BH - group * p.head_group);
    const int unit = p.n_units - 1 - r / heads_here;
    w.bh = group * p.head_group + r % heads_here;
    w.split = 0;
    w.zq = w.bh;
    const int b = w.bh / p.H;
    w.zk = b * p.Hkv + (w.bh - b * p.H) / p.group;
    w.qbase = 0;
    w.kbase = 0;
    w.q0 = unit * QT * kBM;
    w.kv_tile0 = 0;
    w.kv_end = p.Nk;
    w.causal_off = p.Nk - p.Nq;
    w.rm.o_base = static_cast<long long>(w.bh) * p.Nq;
    w.rm.lse_base = w.rm.o_base;
    w.rm.o_stride = 1;
    w.rm.len_q = p.Nq;
    w.list = win_list<BN>(p, w.q0 + w.causal_off, min(w.q0 + QT * kBM, p.Nq) - 1 + w.causal_off);
    w.nmax = w.list.n;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int row0 = tile_row0(p, w.q0, t);
        w.n[t] = w.hole[t] = w.steps[t] = 0;
        if (row0 >= p.Nq) continue;
        const int last = min(row0 + kBM, p.Nq) - 1 + w.causal_off;
        if (last < 0) continue;
        const int end = last / BN + 1;
        const int first = p.window > 0 ? max(0, row0 + w.causal_off - p.window + 1) / BN : 0;
        w.n[t] = w.list.ns + max(0, end - w.list.lo);
        // A list with no gap is walked from its start: its tiles before the
        // window may be sinks.
        w.hole[t] = w.list.ns > 0 || (w.list.lo > 0) ? max(0, min(first, end) - w.list.lo) : 0;
        w.steps[t] = w.n[t] - w.hole[t];
    }
}

// -inf where the row at position pos does not see key kv0 + c.
template <int BN>
__device__ __forceinline__ void win_mask(const FwdParams& p, int pos, int kv0, float (&s)[BN]) {
    const int valid = pos - kv0 + 1;
    if (valid < BN) {
#pragma unroll
        for (int c = 0; c < BN; ++c)
            if (c >= valid) s[c] = -INFINITY;
    }
    if (p.window > 0) {
        const int from = valid - p.window, sink = p.sinks - kv0;
        if (from > 0 && sink < BN) {
#pragma unroll
            for (int c = 0; c < BN; ++c)
                if (c < from && c >= sink) s[c] = -INFINITY;
        }
    }
}

// Control warps of a two-tile CTA with a window: tm_forward's producer and
// issuer with the tile list and the holes. A tile that skips step j + 1 gets no
// S there; its next S is issued in the step before its next one.
template <int D, typename L>
__device__ __forceinline__ void tm_window_control(const FwdParams& p, uint32_t sbase, uint32_t tmem,
                                                  volatile uint32_t* abort_flag, int warp) {
    constexpr int QT = L::Q_TILES;
    constexpr int BN = L::BN;
    constexpr int ST = L::STAGES;
    auto bar = [&](int i) -> uint32_t { return sbase + L::BAR_OFF + 8u * i; };
    WorkWin<QT> w;
    compute_work_win<QT, BN>(p, blockIdx.x, w);
    if (w.nmax == 0) return;
    const bool leader = elect_one();
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        auto load_q = [&](int t) {
            if (leader && w.steps[t] > 0) {
                mbar_arrive_expect_tx(bar(L::BAR_QFULL + t), L::Q_TILE_BYTES);
#pragma unroll
                for (int c = 0; c < L::CHUNKS; ++c)
                    tma_load_3d(sbase + L::Q_OFF + t * L::Q_TILE_BYTES + c * (kBM * L::ROW_BYTES), &p.tm_q,
                                bar(L::BAR_QFULL + t), L::CHUNK_ELEMS * c, tile_row0(p, w.q0, t), w.zq);
            }
        };
        load_q(0);
        const int total = 2 * w.nmax;
        RingPos<ST> pos;
        int issued = 0;
        bool ok = true;
        for (int e = 0; e < total; ++e) {
            const bool is_v = (e & 1) != 0;
            if (e >= ST) {
                ok = __all_sync(0xffffffffu, wait_phase(bar(L::BAR_KVEMPTY + pos.slot), pos.phase ^ 1u, p,
                                                        abort_flag, kStatusWaitKvEmpty));
                if (!ok) break;
            }
            if (leader) {
                mbar_arrive_expect_tx(bar(L::BAR_KVFULL + pos.slot), L::SLOT_BYTES);
                const CUtensorMap* map = is_v ? &p.tm_v : &p.tm_k;
                const int row = w.list.tile(e >> 1) * BN;
#pragma unroll
                for (int c = 0; c < L::CHUNKS; ++c)
                    tma_load_3d(sbase + L::SLOT_OFF + pos.slot * L::SLOT_BYTES + c * (BN * L::ROW_BYTES), map,
                                bar(L::BAR_KVFULL + pos.slot), L::CHUNK_ELEMS * c, row, w.zk);
            }
            issued = e + 1;
            pos.advance();
            if (e == 0) load_q(1);
        }
        if (ok) {
            for (int e = max(0, total - ST); e < total && ok; ++e)
                ok = __all_sync(0xffffffffu, wait_phase(bar(L::BAR_KVEMPTY + e % ST), (e / ST) & 1, p, abort_flag,
                                                        kStatusWaitKvEmpty));
        }
        if (!ok) {
#pragma unroll
            for (int t = 0; t < QT; ++t)
                if (w.steps[t] > 0 && issued > 0)
                    wait_phase(bar(L::BAR_QFULL + t), 0, p, abort_flag, kStatusWaitDrain, false);
            for (int e = max(0, issued - ST); e < issued; ++e)
                wait_phase(bar(L::BAR_KVFULL + e % ST), (e / ST) & 1, p, abort_flag, kStatusWaitDrain, false);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        auto wait_all = [&](uint32_t b, uint32_t parity, unsigned what) {
            return __all_sync(0xffffffffu, wait_phase(b, parity, p, abort_flag, what));
        };
        constexpr uint32_t IDESC_S = make_idesc_bf16(kBM, BN, false, false);
        constexpr uint32_t IDESC_O = make_idesc_bf16(kBM, D, false, true);
        const uint64_t kmaj0 = make_sdesc_rows<L::ROW_BYTES>(sbase, 16, 8 * L::ROW_BYTES);
        const uint64_t vmn0 = make_sdesc_rows<L::ROW_BYTES>(sbase, BN * L::ROW_BYTES, 8 * L::ROW_BYTES);
        const uint32_t kmaj_lo = static_cast<uint32_t>(kmaj0), kmaj_hi = static_cast<uint32_t>(kmaj0 >> 32);
        const uint32_t vmn_lo = static_cast<uint32_t>(vmn0), vmn_hi = static_cast<uint32_t>(vmn0 >> 32);
        auto desc = [](uint32_t lo, uint32_t hi, uint32_t off) -> uint64_t {
            return (static_cast<uint64_t>(hi) << 32) | (lo + (off >> 4));
        };
        auto issue_s = [&](int t, int slot) {
            const uint32_t qa = L::Q_OFF + t * L::Q_TILE_BYTES;
            const uint32_t kb = L::SLOT_OFF + slot * L::SLOT_BYTES;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t in_row = (kk & 3) * 32;
                if (leader)
                    umma_ss(tmem + L::S_COL(t), desc(kmaj_lo, kmaj_hi, qa + (kk >> 2) * (kBM * 128) + in_row),
                            desc(kmaj_lo, kmaj_hi, kb + (kk >> 2) * (BN * 128) + in_row), IDESC_S, kk > 0 ? 1u : 0u);
            }
            if (leader) umma_commit(bar(L::BAR_SFULL + t));
        };
        auto issue_pv = [&](int t, int slot, bool accumulate) {
            const uint32_t vb = L::SLOT_OFF + slot * L::SLOT_BYTES;
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
                if (leader)
                    umma_ts(tmem + L::O_COL(t), tmem + L::S_COL(t) + kk * 8, desc(vmn_lo, vmn_hi, vb + kk * 2048),
                            IDESC_O, (accumulate || kk > 0) ? 1u : 0u);
        };
        auto active = [&](int t, int j) {
            return j < w.n[t] && !(j >= w.list.ns && j < w.list.ns + w.hole[t]);
        };
        RingPos<ST> pos;
        int slot_v = 0, slot_k = 0;
        auto wait_kv = [&](int j) -> bool {  // V_j, then K_{j+1} if any step needs it
            slot_v = pos.slot;
            if (!wait_all(bar(L::BAR_KVFULL + pos.slot), pos.phase, kStatusWaitKvFull)) return false;
            pos.advance();
            if (j + 1 < w.nmax) {
                slot_k = pos.slot;
                if (!wait_all(bar(L::BAR_KVFULL + pos.slot), pos.phase, kStatusWaitKvFull)) return false;
                pos.advance();
            }
            return true;
        };
        int done[QT] = {};       // steps whose PV was issued
        bool q_here[QT] = {};    // Q_t landed
        // S of the tile's step j + 1, whose K is in `slot`.
        auto next_s = [&](int t, int slot) -> bool {
            if (!q_here[t]) {
                if (!wait_all(bar(L::BAR_QFULL + t), 0, kStatusWaitQ)) return false;
                q_here[t] = true;
                tc_fence_after();
            }
            issue_s(t, slot);
            return true;
        };
        bool ok = wait_all(bar(L::BAR_KVFULL + pos.slot), pos.phase, kStatusWaitKvFull);
        if (ok) {
            tc_fence_after();
#pragma unroll
            for (int t = 0; t < QT; ++t)
                if (ok && active(t, 0)) ok = next_s(t, pos.slot);
        }
        if (ok) {
            if (leader) umma_commit(bar(L::BAR_KVEMPTY + pos.slot));
            pos.advance();
            ok = wait_kv(0);
        }
        // Per step as tm_forward's issuer: the next step's K/V waits sit between
        // tile 1's PV and S at d = 128, behind tile 0's batch at d = 64.
        constexpr bool kKvWaitMid1 = (D >= 128);
        for (int j = 0; j < w.nmax && ok; ++j) {
            const int sv = slot_v, sk = slot_k;
            const bool k_next = (j + 1 < w.nmax);
#pragma unroll
            for (int t = 0; t < QT && ok; ++t) {
                const bool act = active(t, j);
                if (act) {
                    ok = wait_all(bar(L::BAR_PFULL + t), done[t] & 1, kStatusWaitP);
                    if (!ok) break;
                    tc_fence_after();
                    issue_pv(t, sv, done[t] > 0);
                    ++done[t];
                }
                if (t == QT - 1 && kKvWaitMid1 && k_next) {
                    ok = wait_kv(j + 1);
                    if (!ok) break;
                }
                if (active(t, j + 1)) {
                    ok = next_s(t, sk);
                } else if (act && j + 1 >= w.n[t]) {
                    if (leader) umma_commit(bar(L::BAR_OFULL + t));
                }
                if (t == 0 && !kKvWaitMid1 && k_next && ok) ok = wait_kv(j + 1);
            }
            if (!ok) break;
            if (leader) umma_commit(bar(L::BAR_KVEMPTY + sv));
            if (k_next && leader) umma_commit(bar(L::BAR_KVEMPTY + sk));
        }
        if (leader) umma_commit(bar(L::BAR_DRAIN));
        wait_phase(bar(L::BAR_DRAIN), 0, p, abort_flag, kStatusWaitDrain, false);
    }
}

}  // namespace fa
