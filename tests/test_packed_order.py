"""The order in which packed work is taken (csrc/fa_packed.cuh), on the host: the
header's own functions, a warp's 32 lanes as coroutines that meet at every vote, shuffle
and reduction. Every unit of a batch is found exactly once, longest first where the header
says so, and padded rows and tile numbers of different sequences do not overlap. No kernel
is launched."""

import ctypes
import os
import random
import shutil
import subprocess

import numpy as np
import pytest

import exact_attention_80_gb300 as fa

CSRC = os.path.join(os.path.dirname(os.path.abspath(fa.__file__)), "csrc")

# What stands in for the header's two includes: a warp on the host.
WARP = r"""
#pragma once
#include <algorithm>
#include <cstdint>
#include <functional>
#include <ucontext.h>
#include <vector>
#define __device__
#define __host__
#define __forceinline__ inline
using std::max;
using std::min;
namespace warp {
struct Lane { ucontext_t at; std::vector<char> stack; bool done; int phase; };
inline Lane lanes[32];
inline ucontext_t home;
inline int me;
inline long long slots[2][32];
inline std::function<void(int)> body;
inline void enter() { body(me); lanes[me].done = true; swapcontext(&lanes[me].at, &home); }
inline void run(std::function<void(int)> f) {
    body = std::move(f);
    for (int l = 0; l < 32; ++l) {
        lanes[l].stack.resize(1 << 16);
        lanes[l].done = false;
        lanes[l].phase = 0;
        getcontext(&lanes[l].at);
        lanes[l].at.uc_stack.ss_sp = lanes[l].stack.data();
        lanes[l].at.uc_stack.ss_size = lanes[l].stack.size();
        makecontext(&lanes[l].at, enter, 0);
    }
    for (bool left = true; left;) {
        left = false;
        for (int l = 0; l < 32; ++l)
            if (!lanes[l].done) { me = l; swapcontext(&home, &lanes[l].at); left = left || !lanes[l].done; }
    }
}
// All lanes' values, once each has left its own.
inline const long long* meet(long long x) {
    const int l = me, p = lanes[l].phase++ & 1;
    slots[p][l] = x;
    swapcontext(&lanes[l].at, &home);
    return slots[p];
}
}  // namespace warp
inline int __reduce_add_sync(unsigned, int x) { auto v = warp::meet(x); long long s = 0; for (int l = 0; l < 32; ++l) s += v[l]; return static_cast<int>(s); }
inline int __reduce_max_sync(unsigned, int x) { auto v = warp::meet(x); return static_cast<int>(*std::max_element(v, v + 32)); }
inline int __reduce_min_sync(unsigned, int x) { auto v = warp::meet(x); return static_cast<int>(*std::min_element(v, v + 32)); }
inline unsigned __ballot_sync(unsigned, bool x) { auto v = warp::meet(x); unsigned s = 0; for (int l = 0; l < 32; ++l) s |= static_cast<unsigned>(v[l]) << l; return s; }
inline int __shfl_sync(unsigned, int x, int from) { return static_cast<int>(warp::meet(x)[from & 31]); }
inline int __shfl_up_sync(unsigned, int x, int by) { const int l = warp::me; auto v = warp::meet(x); return static_cast<int>(v[l >= by ? l - by : l]); }
inline int __ffs(unsigned x) { return __builtin_ffs(static_cast<int>(x)); }
inline int __popc(unsigned x) { return __builtin_popcount(x); }
inline uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : (1u << max(n, 0)) - 1u; }
"""

SOURCE = r"""
#include "fa_packed.cuh"
using namespace fa;
extern "C" {
// Units of the forward (fa_fwd_pack.cuh, pack_unit): `lins` are looked up one after the other, with one cursor for all
// (persistent CTAs) or one each. Out: sequence and first token, or -1.
void forward(const int* cu_q, const int* cu_k, int B, int total_q, int total_k, int max_q, int max_k, int tokens, int Hkv,
             const long long* lins, int n, int keep, int* out) {
    const PackedSeqs s = {cu_q, cu_k, B, total_q, total_k, max_q, max_k};
    auto level0 = [&](const PackedSeq& y) {
        const int off = y.m - y.n;
        return off >= 0 ? off / tokens : -((tokens - 1 - off) / tokens);
    };
    auto runs = [&](int b, int& a, int& k) {
        PackedSeq y;
        packed_seq(s, b, y);
        a = level0(y);
        k = (y.n + tokens - 1) / tokens;
    };
    std::vector<PackedCursor> cursors(32, PackedCursor{0, 0});
    for (int i = 0; i < n; ++i) {
        if (!keep) std::fill(cursors.begin(), cursors.end(), PackedCursor{0, 0});
        warp::run([&](int lane) {
            int b = 0, level = 0;
            const bool have = packed_pick(B, static_cast<int>(lins[i] / Hkv), lane, runs, b, level, cursors[lane]);
            int same[3] = {have, have ? b : 0, have ? level : 0};
            for (int x : same)
                if (__shfl_sync(~0u, x, 0) != x) std::abort();  // all lanes agree
            if (lane) return;
            PackedSeq y;
            packed_seq(s, b, y);
            out[2 * i] = have ? b : -1;
            out[2 * i + 1] = have ? (level - level0(y)) * tokens : -1;
        });
    }
}
// Units of the backward (fa_bwd.cu, bwd_pack_unit): sequence, key tile, kv head, part, or -1.
void backward(const int* cu_q, const int* cu_k, int B, int total_q, int total_k, int max_q, int max_k, int sink_tiles,
              int sink_parts, int other_parts, int Hkv, int pack_heads, long long units, int* out) {
    const PackedSeqs s = {cu_q, cu_k, B, total_q, total_k, max_q, max_k};
    auto tiles = [&](int b) {
        PackedSeq y;
        packed_seq(s, b, y);
        return (y.m + 127) / 128;
    };
    for (long long lin = 0; lin < units; ++lin)
        warp::run([&](int lane) {
            int sinks = 0, all = 0;
            if (sink_tiles > 0) sinks = sink_parts * packed_total(B, lane, [&](int b) { return min(tiles(b), sink_tiles); });
            const long long sink_units = static_cast<long long>(sinks) * Hkv;
            const bool sink = lin < sink_units;
            const int parts = sink ? sink_parts : other_parts, together = sink ? Hkv : pack_heads;
            if (together < Hkv) all = other_parts * packed_total(B, lane, [&](int b) { return max(tiles(b) - sink_tiles, 0); });
            PackedCursor first = {0, 0};
            int h = 0, at = 0;
            const bool there = packed_head(sink ? lin : lin - sink_units, Hkv, together, all, h, at);
            auto runs = [&](int b, int& a, int& n) {
                const int k = tiles(b), first = min(k, sink_tiles);
                a = sink ? k - first : 0;
                n = sink ? first : k - first;
            };
            int b = 0, level = 0;
            const bool live = there && packed_pick(B, at / parts, lane, runs, b, level, first);
            if (lane) return;
            int* o = out + 4 * lin;
            o[0] = o[1] = o[2] = o[3] = -1;
            if (live) o[0] = b, o[1] = tiles(b) - 1 - level, o[2] = h, o[3] = at % parts;
        });
}
long long pad(int q0, int b) { return pad_row(q0, b); }
long long slot(int k0, int b) { return tile_slot(k0, b); }
}
"""


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("order")
    shutil.copy(os.path.join(CSRC, "fa_packed.cuh"), at)  # (its includes are looked for beside it)
    (at / "fa_internal.h").write_text("#pragma once\n")
    (at / "sm103_ptx.cuh").write_text(WARP)
    (at / "order.cpp").write_text(SOURCE)
    lib = at / "order.so"
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-Wno-unknown-pragmas", "-shared", "-fPIC", str(at / "order.cpp"),
                    "-o", str(lib)], check=True)
    lib = ctypes.CDLL(str(lib))
    lib.pad.restype = lib.slot.restype = ctypes.c_longlong
    return lib


def ints(x):
    return np.ascontiguousarray(x, np.int32)


def ptr(x):
    return x.ctypes.data_as(ctypes.c_void_p)


def batch(rng, B, spread, first=0):
    """Lengths of queries and keys with empty sequences and with more queries than keys."""
    ns, ms = [], []
    for _ in range(B):
        n = rng.choice([0, 1, rng.randrange(spread), rng.randrange(spread)])
        ns.append(n)
        ms.append(rng.choice([n, n, 0, rng.randrange(2 * spread), n + rng.randrange(spread)]))
    cu = lambda x: ints(np.concatenate([[first], first + np.cumsum(x)]))  # noqa: E731
    return ns, ms, cu(ns), cu(ms)


BATCHES = [(1, 3000), (3, 700), (31, 300), (32, 200), (33, 200), (127, 60), (128, 60), (129, 60), (255, 40), (257, 40), (400, 9)]


def bounds(ns, ms, cu_q, cu_k):
    return int(cu_q[-1]) + 5, int(cu_k[-1]) + 5, max(1, *ns), max(1, *ms)


@pytest.mark.parametrize("B,spread", BATCHES)
def test_forward_units_come_once_and_longest_first(order, B, spread):
    rng = random.Random(B)
    for tokens in (2, 14, 64, 256):
        ns, ms, cu_q, cu_k = batch(rng, B, spread if tokens > 2 else max(2, spread // 8), rng.choice([0, 9]))
        T, S, most_q, most_k = bounds(ns, ms, cu_q, cu_k)
        live = min(B, T)
        units = min((T + live * (tokens - 1)) // tokens, live * -(-most_q // tokens))  # the grid of a kv head
        want = {(b, t) for b in range(B) for t in range(0, ns[b], tokens)}
        assert len(want) <= units
        Hkv = 3
        lins = np.arange(units, dtype=np.int64) * Hkv + rng.randrange(Hkv)
        out = np.full((units, 2), -2, np.int32)
        order.forward(ptr(cu_q), ptr(cu_k), B, T, S, most_q, most_k, tokens, Hkv, ptr(lins), units, 0, ptr(out))
        got = [tuple(x) for x in out.tolist()]
        assert set(got[: len(want)]) == want and all(x == (-1, -1) for x in got[len(want):])
        ends = [ms[b] - ns[b] + min(t + tokens, ns[b]) for b, t in got[: len(want)]]  # its last position, and one
        if B <= 128:
            levels = [(ms[b] - ns[b]) // tokens + t // tokens for b, t in got[: len(want)]]
            assert levels == sorted(levels, reverse=True)
        else:
            for (b0, _), (b1, _), e0, e1 in zip(got, got[1: len(want)], ends, ends[1:]):
                assert b0 < b1 or (b0 == b1 and e0 > e1)
        # A persistent CTA's units, with one cursor: the same.
        grid = 7
        for cta in range(grid):
            mine = [k * grid + (grid - 1 - cta if k & 1 else cta) for k in range(units * Hkv // grid + 1)]
            at = np.asarray(mine, np.int64)
            kept = np.full((len(mine), 2), -2, np.int32)
            order.forward(ptr(cu_q), ptr(cu_k), B, T, S, most_q, most_k, tokens, Hkv, ptr(at), len(mine), 1, ptr(kept))
            for lin, x in zip(mine, kept.tolist()):
                assert tuple(x) == (got[lin // Hkv] if lin // Hkv < units else (-1, -1))


@pytest.mark.parametrize("B,spread", BATCHES)
def test_backward_units_come_once(order, B, spread):
    rng = random.Random(100 + B)
    for sink_tiles, sink_parts, parts, Hkv, together in ((0, 1, 1, 1, 1), (0, 1, 3, 4, 4), (0, 1, 1, 5, 2), (0, 1, 2, 4, 1),
                                                         (1, 4, 1, 2, 2), (2, 3, 2, 1, 1)):
        ns, ms, cu_q, cu_k = batch(rng, B, max(2, spread // (1 if Hkv == 1 else 2)), rng.choice([0, 9]))
        T, S, most_q, most_k = bounds(ns, ms, cu_q, cu_k)
        live = min(B, S)
        tiles = min((S + live * 127) // 128, live * -(-most_k // 128))
        reach = min(sink_tiles, -(-most_k // 128))
        units = (min(tiles, live * reach) * sink_parts + tiles * parts) * Hkv  # the grid
        out = np.full((units, 4), -2, np.int32)
        order.backward(ptr(cu_q), ptr(cu_k), B, T, S, most_q, most_k, reach, sink_parts, parts, Hkv, together,
                       ctypes.c_longlong(units), ptr(out))
        got = [tuple(x) for x in out.tolist() if x[0] >= 0]
        want = [(b, t, h, p) for b in range(B) for t in range(-(-ms[b] // 128)) for h in range(Hkv)
                for p in range(sink_parts if t < reach else parts)]
        assert sorted(got) == want
        if together < Hkv:  # a group's units before the next one's
            heads = [h // together for _, _, h, _ in got]
            assert heads == sorted(heads)
        elif B <= 128 and reach == 0:  # a tile sees the more rows the further it lies from its sequence's end
            ends = [-(-ms[b] // 128) - 1 - t for b, t, _, _ in got]
            assert ends == sorted(ends, reverse=True)


@pytest.mark.parametrize("B,spread", BATCHES)
def test_padded_rows_and_tile_numbers_do_not_overlap(order, B, spread):
    rng = random.Random(200 + B)
    for first in (0, 1, 63, 130):
        ns, ms, cu_q, cu_k = batch(rng, B, spread, first)
        T, S = int(cu_q[-1]) + rng.randrange(3), int(cu_k[-1]) + rng.randrange(3)
        rows = slots = 0
        for b in range(B):
            at, tile = order.pad(int(cu_q[b]), b), order.slot(int(cu_k[b]), b)
            if ns[b]:
                assert at % 64 == 0 and at >= rows
                rows = at + -(-ns[b] // 64) * 64
            if ms[b]:
                assert tile >= slots
                slots = tile + -(-ms[b] // 128)
        assert rows <= -(-(T + 64 * (B + 1)) // 128) * 128 and slots <= S // 128 + B + 1


def test_broken_offsets_leave_the_others_their_units(order):
    """Sequences whose offsets are out of range have no unit; the others' come once."""
    rng = random.Random(5)
    for B in (40, 128, 150, 300):
        ns, ms, cu_q, cu_k = batch(rng, B, 50)
        ns, ms = [max(n, 1) for n in ns], [max(m, 1) for m in ms]
        cu_q, cu_k = ints(np.concatenate([[0], np.cumsum(ns)])), ints(np.concatenate([[0], np.cumsum(ms)]))
        T, S, most_q, most_k = bounds(ns, ms, cu_q, cu_k)
        bad = cu_q.copy()
        bad[7], bad[B - 3] = -5, 2 ** 31 - 1
        gone = {6, 7, B - 4, B - 3}
        tokens, units = 16, sum(-(-n // 16) for n in ns)
        lins = np.arange(units, dtype=np.int64)
        out = np.full((units, 2), -2, np.int32)
        order.forward(ptr(bad), ptr(cu_k), B, T, S, most_q, most_k, tokens, 1, ptr(lins), units, 0, ptr(out))
        want = {(b, t) for b in range(B) if b not in gone for t in range(0, ns[b], tokens)}
        got = [tuple(x) for x in out.tolist() if x[0] >= 0]
        assert len(got) == len(want) and set(got) == want
