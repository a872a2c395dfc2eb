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
//
// P is rounded to bf16 for its product, as in the dense forward: kind::f16 takes
// both operands in one type, and V as f16 could overflow (as bf16 P a weight is off
// by up to 2^-8; f16 would be eight times finer). Scores, sums and O are fp32.
#pragma once

#include "fa_fwd_common.cuh"

namespace fa {

constexpr int kSmallSinks = 32;

struct WinList {
    int ns, lo, n;  // tiles at .. at + ns - 1, then tile lo on; n in all
    int at;         // 0, or where a key split begins within the sinks
    __device__ __forceinline__ int tile(int j) const { return j < ns ? at + j : lo + (j - ns); }
};

// The list of rows at positions p0 .. p1 (p0 may be negative: rows with no key).
template <int BN>
__device__ __forceinline__ WinList win_list(const FwdParams& p, int p0, int p1) {
    WinList w;
    w.ns = 0;
    w.lo = 0;
    w.at = 0;
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
    // Step 0 is the sinks alone, kSmallSinks of them at most: its S and PV take
    // that many keys instead of a whole tile's.
    bool small;
};

// SPLIT: key splits (launches of persistent CTAs have none, and no registers to
// spare for them: 203 against 212 us at d = 64).
template <int QT, int BN, bool SPLIT>
__device__ __forceinline__ void compute_work_win(const FwdParams& p, long long lin, WorkWin<QT>& w) {
    // As compute_work (dense): head groups, units heaviest first, splits of a unit
    // beside one another.
    w.split = 0;
    if constexpr (SPLIT) {
        w.split = static_cast<int>(lin % p.num_splits);
        lin /= p.num_splits;
    }
    const long long per_group = static_cast<long long>(p.head_group) * p.n_units;
    const int group = static_cast<int>(lin / per_group);
    const int r = static_cast<int>(lin % per_group);
    const int heads_here = min(p.head_group, p.BH - group * p.head_group);
    const int unit = p.n_units - 1 - r / heads_here;
    w.bh = group * p.head_group + r % heads_here;
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
    // (Behind a gap no window reaches tile 0.)
    w.small = QT == 2 && w.list.ns == 1 && p.sinks <= kSmallSinks;
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
    if (SPLIT && p.num_splits > 1) {
        // This split's part of the list, entries i0 .. i1 - 1: again a run of sink
        // tiles and one of window tiles, with what is left of the holes between.
        const WinList all = w.list;
        const int each = (all.n + p.num_splits - 1) / p.num_splits;
        const int i0 = min(w.split * each, all.n), i1 = min(i0 + each, all.n);
        w.list.n = w.nmax = i1 - i0;
        w.list.ns = max(0, min(all.ns, i1) - i0);
        w.list.at = i0;
        w.list.lo = all.lo + max(0, i0 - all.ns);
        w.small = w.small && i0 == 0 && i1 > 0;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int hole0 = max(all.ns, i0), hole1 = min(all.ns + w.hole[t], i1);
            w.n[t] = max(0, min(w.n[t], i1) - i0);
            w.hole[t] = max(0, hole1 - hole0);
            // A hole up to the split's end: the tile ends before it.
            if (w.n[t] == w.list.ns + w.hole[t]) w.n[t] = w.list.ns, w.hole[t] = 0;
            w.steps[t] = w.n[t] - w.hole[t];
        }
    }
}

// -inf where the row at position pos does not see key kv0 + c. (Masking only the
// 32-key chunks that an edge crosses, and leaving out the exponentials of chunks
// that no row of the warp sees, costs more than it saves: the branches keep the
// chunks' instructions apart, 216 -> 332 us for 2 x 32 heads of 8192, window
// 1024, d = 64. One bit per key, from shifts: with a comparison per key and edge
// the same call takes 216 us against 203.)
template <int BN>
__device__ __forceinline__ void win_mask(const FwdParams& p, int pos, int kv0, float (&s)[BN]) {
    const int valid = pos - kv0 + 1;
    const int from = p.window > 0 ? valid - p.window : 0, sink = p.sinks - kv0;
    if (valid < BN || (from > 0 && sink < BN)) {
#pragma unroll
        for (int g = 0; g < BN / 32; ++g) {
            const uint32_t seen = low_bits(valid - 32 * g) & (~low_bits(from - 32 * g) | low_bits(sink - 32 * g));
#pragma unroll
            for (int c = 0; c < 32; ++c)
                if (!(seen & (1u << c))) s[32 * g + c] = -INFINITY;
        }
    }
}

// Units a CTA walks: its own, or (PERSIST) one of each round as persist_unit
// gives them; -1 where a round has none for it.
template <bool PERSIST>
__device__ __forceinline__ int win_rounds(const FwdParams& p) {
    return PERSIST ? static_cast<int>((p.total_units + gridDim.x - 1) / gridDim.x) : 1;
}
template <bool PERSIST>
__device__ __forceinline__ long long win_unit(const FwdParams& p, int k) {
    if constexpr (!PERSIST) return blockIdx.x;
    const long long g = gridDim.x;
    const long long c = (k & 1) ? g - 1 - blockIdx.x : blockIdx.x;
    const long long lin = static_cast<long long>(k) * g + c;
    return lin < p.total_units ? lin : -1;
}

// Packed sequences (fa_fwd_pack.cuh): a unit's place in the batch, a CTA's only one and a
// persistent CTA's next one as work, the token of a query tile's first row, the keys that exist in
// its last key tile, and the clearing of the others' values.
struct PackUnit;
struct PackRing;
template <int QT, int BN>
__device__ __forceinline__ void pack_first(const FwdParams& p, const PackRing* ring, WorkWin<QT>& w);
template <int QT, int BN, typename L>
__device__ __forceinline__ bool pack_next(const FwdParams& p, PackRing* ring, uint32_t sbase, int k,
                                          volatile uint32_t* abort_flag, WorkWin<QT>& w, bool& ok);
template <int QT>
__device__ __forceinline__ int pack_tile_token(const FwdParams& p, int first, int t);
template <int BN, int QT>
__device__ __forceinline__ int pack_tail(const WorkWin<QT>& w);
template <typename L>
__device__ __forceinline__ bool pack_clean_v(const FwdParams& p, uint32_t sbase, int entry, int rows, uint32_t clean,
                                             volatile uint32_t* abort_flag, int lane);

// Control warps of a two-tile CTA with a window: the producer and the issuer of
// the dense kernel with the tile list and the holes. A tile that skips step
// j + 1 gets no S there; its next S is issued in the step before its next one.
// PERSIST: the K/V ring and every barrier's phase carry over from unit to unit.
// The next unit's K_0 and Q load while the current one's last steps run (Q_t as
// soon as the unit's last S_t MMA is done, QEMPTY_t), and its first S MMAs are
// issued right behind the current unit's last PV; O_t is first overwritten by
// the unit's PV_t(0), which waits for a P that the softmax threads hand over
// only after their epilogue.
// PACK: packed sequences, whose units come through `ring`.
template <int D, typename L, bool PERSIST, bool PACK>
__device__ __forceinline__ void tm_window_control(const FwdParams& p, uint32_t sbase, uint32_t tmem,
                                                  volatile uint32_t* abort_flag, int warp, PackRing* ring) {
    constexpr int QT = L::Q_TILES;
    constexpr int BN = L::BN;
    constexpr int ST = L::STAGES;
    auto bar = [&](int i) -> uint32_t { return sbase + L::BAR_OFF + 8u * i; };
    const int rounds = PACK && PERSIST ? 0x7fffffff : win_rounds<PERSIST>(p);
    const bool leader = elect_one();
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        RingPos<ST> pos;
        int issued = 0;        // K/V entries issued, all units
        int q_loads[QT] = {};  // Q_t loads issued
        bool ok = true;
        // PACK: the last V tile of a unit whose sequence ends in it is cleared behind
        // that end once the next unit's first loads are on their way. The issuer waits for
        // one clearing at a time, so the next one is handed over when the tile before it
        // has been used: its slot was released (which the slot's next load has waited for).
        int dirty = -1, dirty_rows = 0, cleared = -1;
        auto clean = [&] {
            if constexpr (PACK) {
                if (ok && dirty >= 0) {
                    if (PERSIST && cleared >= 0 && issued <= cleared + ST)
                        ok = __all_sync(0xffffffffu, wait_phase(bar(L::BAR_KVEMPTY + cleared % ST), (cleared / ST) & 1, p,
                                                                abort_flag, kStatusWaitKvEmpty));
                    if (ok)
                        ok = pack_clean_v<L>(p, sbase, dirty, dirty_rows, bar(L::BAR_VCLEAN), abort_flag,
                                             threadIdx.x & 31);
                    cleared = dirty;
                }
                dirty = -1;
            }
        };
        auto load_q = [&](const WorkWin<QT>& w, int t) -> bool {
            if (w.steps[t] == 0) return true;
            if (PERSIST && q_loads[t] > 0 &&
                !__all_sync(0xffffffffu, wait_phase(bar(L::BAR_QEMPTY + t), (q_loads[t] - 1) & 1, p, abort_flag,
                                                    kStatusWaitQ)))
                return false;
            if (leader) {
                mbar_arrive_expect_tx(bar(L::BAR_QFULL + t), PACK ? p.q_bytes : L::Q_TILE_BYTES);
#pragma unroll
                for (int c = 0; c < L::CHUNKS; ++c)
                    tma_load_3d(sbase + L::Q_OFF + t * L::Q_TILE_BYTES + c * (kBM * L::ROW_BYTES), &p.tm_q,
                                bar(L::BAR_QFULL + t), L::CHUNK_ELEMS * c,
                                PACK ? w.zq : tile_row0(p, w.q0, t),
                                PACK ? w.qbase + pack_tile_token<QT>(p, w.q0, t) : w.zq);
            }
            ++q_loads[t];
            return true;
        };
        for (int k = 0; k < rounds && ok; ++k) {
            WorkWin<QT> w;
            if constexpr (PACK && PERSIST) {
                if (!pack_next<QT, BN, L>(p, ring, sbase, k, abort_flag, w, ok)) break;
            } else if constexpr (PACK) {
                pack_first<QT, BN>(p, ring, w);
            } else {
                const long long lin = win_unit<PERSIST>(p, k);
                if (lin < 0) continue;
                compute_work_win<QT, BN, !PERSIST>(p, lin, w);
            }
            if (w.nmax == 0) {
                clean();  // (the next unit may be given out only when the issuer has come past this one)
                continue;
            }
            if (!PERSIST) ok = load_q(w, 0);
            // Entry e: K_0; then per step j: V_j, K_{j+1}.
            for (int e = 0; e < 2 * w.nmax && ok; ++e) {
                if (issued >= ST)
                    ok = __all_sync(0xffffffffu, wait_phase(bar(L::BAR_KVEMPTY + pos.slot), pos.phase ^ 1u, p,
                                                            abort_flag, kStatusWaitKvEmpty));
                if (!ok) break;
                if (leader) {
                    mbar_arrive_expect_tx(bar(L::BAR_KVFULL + pos.slot), L::SLOT_BYTES);
                    const CUtensorMap* map = (e & 1) ? &p.tm_v : &p.tm_k;
                    const int row = (PACK ? w.kbase : 0) + w.list.tile(e >> 1) * BN;
#pragma unroll
                    for (int c = 0; c < L::CHUNKS; ++c)
                        tma_load_3d(sbase + L::SLOT_OFF + pos.slot * L::SLOT_BYTES + c * (BN * L::ROW_BYTES), map,
                                    bar(L::BAR_KVFULL + pos.slot), L::CHUNK_ELEMS * c, row, w.zk);
                }
                ++issued;
                pos.advance();
                if (e == 0) {
                    if (PERSIST) ok = load_q(w, 0);
                    if (ok) ok = load_q(w, 1);
                    clean();
                }
            }
            if constexpr (PACK) {
                dirty_rows = pack_tail<BN>(w);
                if (dirty_rows < BN) dirty = issued - 1;
            }
        }
        clean();
        if (ok) {
            // No commit arrival may be in flight when the CTA exits: the last uses
            // of the K/V slots and of the Q tiles.
            for (int e = max(0, issued - ST); e < issued && ok; ++e)
                ok = __all_sync(0xffffffffu, wait_phase(bar(L::BAR_KVEMPTY + e % ST), (e / ST) & 1, p, abort_flag,
                                                        kStatusWaitKvEmpty));
            for (int t = 0; t < QT && ok && PERSIST; ++t)
                if (q_loads[t] > 0)
                    ok = __all_sync(0xffffffffu, wait_phase(bar(L::BAR_QEMPTY + t), (q_loads[t] - 1) & 1, p,
                                                            abort_flag, kStatusWaitQ));
        }
        if (!ok) {
#pragma unroll
            for (int t = 0; t < QT; ++t)
                if (q_loads[t] > 0)
                    wait_phase(bar(L::BAR_QFULL + t), (q_loads[t] - 1) & 1, p, abort_flag, kStatusWaitDrain, false);
            for (int e = max(0, issued - ST); e < issued; ++e)
                wait_phase(bar(L::BAR_KVFULL + e % ST), (e / ST) & 1, p, abort_flag, kStatusWaitDrain, false);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        auto wait_all = [&](uint32_t b, uint32_t parity, unsigned what) {
            return __all_sync(0xffffffffu, wait_phase(b, parity, p, abort_flag, what));
        };
        constexpr uint32_t IDESC_S = make_idesc_bf16(kBM, BN, false, false);
        constexpr uint32_t IDESC_SMALL = make_idesc_bf16(kBM, kSmallSinks, false, false);
        constexpr uint32_t IDESC_O = make_idesc_bf16(kBM, D, false, true);
        const uint64_t kmaj0 = make_sdesc_rows<L::ROW_BYTES>(sbase, 16, 8 * L::ROW_BYTES);
        const uint64_t vmn0 = make_sdesc_rows<L::ROW_BYTES>(sbase, BN * L::ROW_BYTES, 8 * L::ROW_BYTES);
        const uint32_t kmaj_lo = static_cast<uint32_t>(kmaj0), kmaj_hi = static_cast<uint32_t>(kmaj0 >> 32);
        const uint32_t vmn_lo = static_cast<uint32_t>(vmn0), vmn_hi = static_cast<uint32_t>(vmn0 >> 32);
        auto desc = [](uint32_t lo, uint32_t hi, uint32_t off) -> uint64_t {
            return (static_cast<uint64_t>(hi) << 32) | (lo + (off >> 4));
        };
        auto issue_s = [&](int t, int slot, bool small) {
            const uint32_t qa = L::Q_OFF + t * L::Q_TILE_BYTES;
            const uint32_t kb = L::SLOT_OFF + slot * L::SLOT_BYTES;
            const uint32_t idesc = small ? IDESC_SMALL : IDESC_S;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t in_row = (kk & 3) * 32;
                if (leader)
                    umma_ss(tmem + L::S_COL(t), desc(kmaj_lo, kmaj_hi, qa + (kk >> 2) * (kBM * 128) + in_row),
                            desc(kmaj_lo, kmaj_hi, kb + (kk >> 2) * (BN * 128) + in_row), idesc, kk > 0 ? 1u : 0u);
            }
            if (leader) umma_commit(bar(L::BAR_SFULL + t));
        };
        auto issue_pv = [&](int t, int slot, bool accumulate, bool small) {
            const uint32_t vb = L::SLOT_OFF + slot * L::SLOT_BYTES;
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
                if (leader && (!small || kk < kSmallSinks / 16))
                    umma_ts(tmem + L::O_COL(t), tmem + L::S_COL(t) + kk * 8, desc(vmn_lo, vmn_hi, vb + kk * 2048),
                            IDESC_O, (accumulate || kk > 0) ? 1u : 0u);
        };
        RingPos<ST> pos;
        int cleaned = 0;      // PACK: cleared V tiles waited for
        int p_seen[QT] = {};  // P_t phases waited for, all units
        int q_seen[QT] = {};  // Q_t phases waited for
        bool ok = true;
        for (int k = 0; k < rounds && ok; ++k) {
            WorkWin<QT> w;
            if constexpr (PACK && PERSIST) {
                if (!pack_next<QT, BN, L>(p, ring, sbase, k, abort_flag, w, ok)) break;
            } else if constexpr (PACK) {
                pack_first<QT, BN>(p, ring, w);
            } else {
                const long long lin = win_unit<PERSIST>(p, k);
                if (lin < 0) continue;
                compute_work_win<QT, BN, !PERSIST>(p, lin, w);
            }
            if (w.nmax == 0) continue;
            auto active = [&](int t, int j) {
                return j < w.n[t] && !(j >= w.list.ns && j < w.list.ns + w.hole[t]);
            };
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
            int done[QT] = {};     // PVs issued in this unit
            int issued_s[QT] = {}; // S MMAs issued in this unit
            // S of the tile's step j, whose K is in `slot`.
            auto next_s = [&](int t, int j, int slot) -> bool {
                if (issued_s[t] == 0) {
                    if (!wait_all(bar(L::BAR_QFULL + t), q_seen[t] & 1, kStatusWaitQ)) return false;
                    ++q_seen[t];
                    tc_fence_after();
                }
                issue_s(t, slot, w.small && j == 0);
                if (++issued_s[t] == w.steps[t] && PERSIST && leader) umma_commit(bar(L::BAR_QEMPTY + t));
                return true;
            };
            ok = wait_all(bar(L::BAR_KVFULL + pos.slot), pos.phase, kStatusWaitKvFull);
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int t = 0; t < QT; ++t)
                    if (ok && active(t, 0)) ok = next_s(t, 0, pos.slot);
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
                if constexpr (PACK) {
                    if (!k_next && pack_tail<BN>(w) < BN)
                        ok = wait_all(bar(L::BAR_VCLEAN), cleaned++ & 1, kStatusWaitKvFull);
                }
#pragma unroll
                for (int t = 0; t < QT && ok; ++t) {
                    const bool act = active(t, j);
                    if (act) {
                        ok = wait_all(bar(L::BAR_PFULL + t), p_seen[t] & 1, kStatusWaitP);
                        if (!ok) break;
                        ++p_seen[t];
                        tc_fence_after();
                        issue_pv(t, sv, done[t] > 0, w.small && j == 0);
                        ++done[t];
                    }
                    if (t == QT - 1 && kKvWaitMid1 && k_next) {
                        ok = wait_kv(j + 1);
                        if (!ok) break;
                    }
                    if (active(t, j + 1)) {
                        ok = next_s(t, j + 1, sk);
                    } else if (act && j + 1 >= w.n[t]) {
                        if (leader) umma_commit(bar(L::BAR_OFULL + t));
                    }
                    if (t == 0 && !kKvWaitMid1 && k_next && ok) ok = wait_kv(j + 1);
                }
                if (!ok) break;
                if (leader) umma_commit(bar(L::BAR_KVEMPTY + sv));
                if (k_next && leader) umma_commit(bar(L::BAR_KVEMPTY + sk));
            }
        }
        // Every MMA this thread issued must finish before TMEM can be freed.
        if (leader) umma_commit(bar(L::BAR_DRAIN));
        wait_phase(bar(L::BAR_DRAIN), 0, p, abort_flag, kStatusWaitDrain, false);
    }
}

}  // namespace fa
