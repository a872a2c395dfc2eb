"""Attention over packed sequences of different lengths with grouped heads, a
window and sinks, forward and backward, against the float64 oracle
(oracle/serving.py), at the lengths and masks where it can go wrong.

Tolerances, elementwise, from the roundings on the way (bf16: 2^-8 of a value),
as for the windowed calls, whose kernels these are.
 * O: its own rounding, and that of P, in the numerator and the denominator:
   2^-8 |o| + 2^-7 a, a = sum_j w_j |v_j|. LSE: fp32 scores and sums, 1e-3.
 * dV: its rounding and P's: 2^-8 |dv| + 2^-7 sum_i w_ij |dout_i|.
 * dS = P (dP - D): its rounding, P's, and D's error, which comes from the
   rounded O that the backward gets: e_ij = w_ij (2^-7 |dP - D| + dD_i),
   dD_i = sum_c |dout_ic| (2^-8 |o_ic| + 2^-7 a_ic). dQ and dK: their own
   rounding and scale times the sum of e against |k| and |q|.
And the dense path's relative L2 bound, 5e-3, over tensors of at least 1000
values.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import exact_attention_80_gb300 as fa  # noqa: E402
import oracle.serving as orc  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    fa.load_library()
    fa.fa_device_status(clear=True)


def ok():
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_OK


def f64(t):
    return t.double().cpu().numpy()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def cu_of(lengths, first=0):
    return np.concatenate([[first], first + np.cumsum(lengths)]).astype(np.int32)


def make(T, S, H, Hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    return n(T, H, d), n(S, Hkv, d), n(S, Hkv, d), n(T, H, d)


def reference(q, k, v, do, cu_q, cu_k, window, sinks):
    """Values and bounds of every output, sequence by sequence and head by head."""
    q, k, v, do = (f64(x) for x in (q, k, v, do))
    scale = fa.default_scale(q.shape[-1])
    H = q.shape[1]
    g = H // k.shape[1]
    out = {n: np.zeros(x.shape) for n, x in (("o", q), ("dq", q), ("dk", k), ("dv", v))}
    lim = {n: np.zeros(x.shape) for n, x in out.items()}
    lse = np.full((H, q.shape[0]), -np.inf)
    for b in range(len(cu_q) - 1):
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        for h in range(H):
            c = h // g
            Q, K, V, G = q[rows, h], k[keys, c], v[keys, c], do[rows, h]
            o, lse[h, rows], w = orc.attend(Q, K, V, scale, window, sinks)
            a = w @ np.abs(V)
            out["o"][rows, h], lim["o"][rows, h] = o, 2.0 ** -8 * np.abs(o) + 2.0 ** -7 * a
            dp = G @ V.T - (G * o).sum(1, keepdims=True)
            ds = w * dp
            dD = (np.abs(G) * (2.0 ** -8 * np.abs(o) + 2.0 ** -7 * a)).sum(1, keepdims=True)
            e = w * (2.0 ** -7 * np.abs(dp) + dD)
            out["dq"][rows, h], lim["dq"][rows, h] = ds @ K * scale, e @ np.abs(K) * scale
            out["dk"][keys, c] += ds.T @ Q * scale
            lim["dk"][keys, c] += e.T @ np.abs(Q) * scale
            out["dv"][keys, c] += w.T @ G
            lim["dv"][keys, c] += 2.0 ** -7 * (w.T @ np.abs(G))
    for n in ("dq", "dk", "dv"):
        lim[n] += 2.0 ** -8 * np.abs(out[n])
    return out, lim, lse


def check(got, ref, lim, what):
    got = f64(got)
    over = np.abs(got - ref) - lim - 1e-9
    assert np.all(np.isfinite(got)), what
    assert over.max() <= 0, f"{what}: {over.max():.3e} over at {np.unravel_index(over.argmax(), over.shape)}"
    if ref.size >= 1000 and np.linalg.norm(ref) > 1e-3 * np.sqrt(ref.size):
        rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert rel <= 5e-3, f"{what}: rel-L2 {rel:.3e}"


def check_lse(lse, ref):
    lse = f64(lse)
    empty = np.isneginf(ref)
    assert np.array_equal(np.isneginf(lse), empty)
    assert np.all(np.abs(lse[~empty] - ref[~empty]) <= 1e-3)


def bounds(ns, ms):
    return max(1, max(ns)), max(1, max(ms))


CASES = [
    # H, Hkv, queries, keys (None: the same), window, sinks
    (1, 1, [1], None, 0, 0),
    (4, 2, [1, 2, 1, 3], [1, 130, 128, 3], 0, 0),              # single tokens behind contexts
    (8, 2, [130, 24, 64, 1, 257], None, 0, 0),
    (3, 1, [300, 0, 41, 129], None, 0, 0),                     # three heads a group, an empty sequence
    (7, 1, [100, 37], [100, 500], 0, 0),                       # seven: tiles of 18 tokens
    (10, 2, [200, 1], [260, 1], 70, 3),
    (64, 1, [9, 33], [40, 33], 0, 0),                          # tiles of two tokens
    (128, 1, [5], [77], 0, 0),                                 # of one
    (2, 2, [513, 640], None, 0, 0),
    (4, 4, [0, 700, 5, 0], [7, 400, 0, 0], 0, 0),              # rows with no key, sequences with none
    (4, 2, [400, 130], [700, 130], 129, 4),
    (2, 1, [640, 300], [640, 1000], 200, 130),                 # sinks past a key tile
    (4, 1, [300, 200], None, 1, 0),                            # every row sees itself alone
    (2, 1, [1000], [1300], 300, 257),
    (4, 2, [5] * 40 + [200], None, 0, 0),                      # more sequences than a warp has lanes
    (2, 1, [1 + i % 7 for i in range(100)], [1 + i % 11 for i in range(100)], 0, 0),
    (1, 1, [2500], None, 0, 0),                                # one head: key tiles in parts
    (2, 1, [1500, 40], None, 200, 4),                          # the sinks' tiles in parts
]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_packed_forward_and_backward(case, d):
    H, Hkv, ns, ms, window, sinks = CASES[case]
    ms = ms or ns
    cu_q, cu_k = cu_of(ns), cu_of(ms)
    q, k, v, do = make(int(cu_q[-1]), max(1, int(cu_k[-1])), H, Hkv, d, 100 * case + d)
    out, lim, lse_ref = reference(q, k, v, do, cu_q, cu_k, window, sinks)
    gq, gk, gv, gdo = (x.cuda() for x in (q, k, v, do))
    batch = (dev(cu_q), dev(cu_k), *bounds(ns, ms), window, sinks)
    o, lse = fa.attention_packed(gq, gk, gv, *batch)
    ok()
    check(o, out["o"], lim["o"], "o")
    check_lse(lse, lse_ref)
    grads = fa.attention_packed_backward(gq, gk, gv, o, lse, gdo, *batch)
    ok()
    for n, x in zip(("dq", "dk", "dv"), grads):
        check(x, out[n], lim[n], n)


def test_parts_are_reached():
    """The batches above that are there for key tiles in parts have them: their workspace holds partial sums."""
    for case in (16, 17):
        H, Hkv, ns, _, window, sinks = CASES[case]
        for d in (64, 128, 256):
            rows = (sum(ns) + 64 * (len(ns) + 1) + 127) // 128 * 128
            n = fa.fa_bwd_packed_workspace_bytes(len(ns), sum(ns), sum(ns), max(ns), max(ns), H, Hkv, d, window, sinks)
            assert n > rows * H * (d + 2) * 4


@pytest.mark.parametrize("d", [64, 128, 256])
def test_equal_lengths_give_the_dense_result(d):
    """Sequences of one length and no window: fa_fwd_window's O and LSE, bit for bit."""
    B, H, Hkv, N, M = 3, 6, 2, 200, 333
    q, k, v, _ = make(B * N, B * M, H, Hkv, d, d)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    o, lse = fa.attention_packed(q, k, v, dev(cu_of([N] * B)), dev(cu_of([M] * B)), N, M)
    heads = lambda t: t.view(B, -1, t.shape[1], d).transpose(1, 2).contiguous()  # noqa: E731
    ow, lw = fa.attention_window(heads(q), heads(k), heads(v), 0, num_splits=1)
    ok()
    assert torch.equal(heads(o), ow) and torch.equal(lse.view(H, B, N).transpose(0, 1), lw)


@pytest.mark.parametrize("d", [64, 256])
def test_order_of_the_sequences(d):
    """A sequence's result does not depend on its neighbours, their order or its place."""
    H, Hkv, ns = 6, 2, [70, 1, 200, 129]
    q, k, v, do = make(sum(ns), sum(ns), H, Hkv, d, 3)
    q, k, v, do = (x.cuda() for x in (q, k, v, do))
    cu = cu_of(ns)
    args = lambda c: (dev(c), dev(c), 200, 200, 50, 2)  # noqa: E731
    o, lse = fa.attention_packed(q, k, v, *args(cu))
    g = fa.attention_packed_backward(q, k, v, o, lse, do, *args(cu))
    order = [2, 0, 3, 1]
    idx = torch.cat([torch.arange(cu[b], cu[b + 1]) for b in order]).cuda()
    c2 = cu_of([ns[b] for b in order])
    q2, k2, v2, do2 = (x[idx].contiguous() for x in (q, k, v, do))
    o2, l2 = fa.attention_packed(q2, k2, v2, *args(c2))
    g2 = fa.attention_packed_backward(q2, k2, v2, o2, l2, do2, *args(c2))
    ok()
    assert torch.equal(o2, o[idx]) and torch.equal(l2, lse[:, idx])
    assert torch.equal(g2[1], g[1][idx]) and torch.equal(g2[2], g[2][idx])


MANY = [
    # H, Hkv, queries, keys (None: the same), window, sinks: so many units that CTAs take several
    (32, 32, [130, 1, 0, 64, 200, 7, 0, 100, 129, 255, 256, 1, 300, 90, 33], None, 0, 0),
    (64, 32, [130, 1, 0, 64, 50, 7, 0, 100, 129, 70, 128, 1, 9, 90, 33], [130, 5, 7, 300, 0, 200, 0, 100, 10, 70, 128, 1, 9, 90, 33], 0, 0),
    (32, 16, [1 + 41 * b % 120 for b in range(34)], None, 30, 3),                       # more than 32 sequences
    (8, 4, [1 + 41 * b % 60 for b in range(150)], [1 + 31 * b % 200 for b in range(150)], 0, 0),  # than 128
    (8, 4, [b % 3 * (b % 40) for b in range(300)], [b % 50 for b in range(300)], 20, 1),          # than 256, a third with no query
    (16, 16, [700, 1500, 40, 900, 2000, 3, 1800], None, 400, 130),
    # so many tokens and heads that the backward takes some heads before the others
    (16, 16, [40, 300, 129, 1000, 1500, 0, 1000, 700, 1, 1600, 1000, 1300], None, 0, 0),
    (32, 16, [33 + b % 60 for b in range(150)], None, 0, 0),
]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_packed_batches_of_many_units(case, d):
    """Each sequence's outputs are those of a call with it alone, bit for bit; the first ones' are the oracle's."""
    H, Hkv, ns, ms, window, sinks = MANY[case]
    ms = ms or ns
    cu_q, cu_k = cu_of(ns), cu_of(ms)
    q, k, v, do = (x.cuda() for x in make(int(cu_q[-1]), max(1, int(cu_k[-1])), H, Hkv, d, 100 * case + d))
    batch = (dev(cu_q), dev(cu_k), *bounds(ns, ms), window, sinks)
    o, lse = fa.attention_packed(q, k, v, *batch)
    grads = fa.attention_packed_backward(q, k, v, o, lse, do, *batch)
    ok()
    some = [b for b in range(len(ns)) if ns[b]]
    for b in some if len(some) < 20 else some[:6] + some[-6:]:
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        kk, vv = (x[keys] if ms[b] else x[:1] for x in (k, v))
        one = (dev([0, ns[b]]), dev([0, ms[b]]), ns[b], max(1, ms[b]), window, sinks)
        o1, l1 = fa.attention_packed(q[rows], kk, vv, *one)
        g1 = fa.attention_packed_backward(q[rows], kk, vv, o1, l1, do[rows], *one)
        ok()
        assert torch.equal(o[rows], o1) and torch.equal(lse[:, rows], l1), b
        # (dQ is a sum in any order, and here dK and dV of a sequence alone may be sums of parts: a rounding apart.)
        for x, y in zip((grads[0][rows], grads[1][keys], grads[2][keys]), g1):
            if x.numel():
                assert (x.float() - y.float()).abs().max() <= 2.0 ** -7 * y.float().abs().max() + 1e-30, b
    n = min(3, len(ns))
    rows, keys = slice(0, cu_q[n]), slice(0, cu_k[n])
    out, lim, lse_ref = reference(q[rows].cpu(), k[keys].cpu(), v[keys].cpu(), do[rows].cpu(), cu_q[: n + 1], cu_k[: n + 1],
                                  window, sinks)
    check(o[rows], out["o"], lim["o"], "o")
    check_lse(lse[:, rows], lse_ref)
    for name, x, s in zip(("dq", "dk", "dv"), grads, (rows, keys, keys)):
        check(x[s], out[name], lim[name], name)


@pytest.mark.parametrize("d", [64, 128])
def test_broken_and_foreign_things_in_batches_of_many_units(d):
    """NaN in other sequences and around them, rows of no sequence, and a broken sequence, where CTAs take several units."""
    H, Hkv = 16, 4
    ns = [1 + 41 * b % 90 for b in range(140)]
    cu = cu_of(ns, 6)
    T = int(cu[-1]) + 70
    q, k, v, _ = (x.cuda() for x in make(T, T, H, Hkv, d, 2))
    o, lse = fa.attention_packed(q, k, v, dev(cu), dev(cu), max(ns), max(ns), 50, 2)
    ok()
    out = torch.ones(T, dtype=torch.bool)
    out[cu[0]: cu[-1]] = False
    assert torch.all(o[out] == 0) and torch.all(lse[:, out] == -float("inf"))
    odd = torch.zeros(T, dtype=torch.bool)
    for b in range(1, 140, 2):
        odd[cu[b]: cu[b + 1]] = True
    x = [t.clone() for t in (q, k, v)]
    for t in x:
        t[odd | out] = float("nan")
    mine = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    fa.fa_fwd_packed(*x, *mine, dev(cu), dev(cu), max(ns), max(ns), 50, 2)
    ok()
    good = ~(odd | out)
    assert torch.equal(mine[0][good], o[good]) and torch.equal(mine[1][:, good], lse[:, good])
    assert torch.all(mine[0][out] == 7.0) and torch.all(mine[1][:, out] == 7.0)
    bad = cu.copy()
    bad[71] = 2 ** 31 - 1  # sequences 70 and 71
    mine = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    fa.fa_fwd_packed(q, k, v, *mine, dev(bad), dev(cu), max(ns), max(ns), 50, 2)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_SEQLENS
    for b in (0, 1, 69, 72, 139):
        s = slice(cu[b], cu[b + 1])
        assert torch.equal(mine[0][s], o[s]) and torch.equal(mine[1][:, s], lse[:, s])
    s = slice(cu[70], cu[72])
    assert torch.all(mine[0][s] == 7.0) and torch.all(mine[1][:, s] == 7.0)


@pytest.mark.parametrize("d", [64, 128])
def test_sequences_by_the_hundred_thousand(d):
    """So many that a search for every unit would take seconds, with a long one among them: that one gets the bits of a
    call with it alone, a sequence of one token its value."""
    H, B, N = 8, 1 << 17, 9000
    ns = np.ones(B, np.int64)
    at = 70000
    ns[at] = N
    cu, T = dev(cu_of(ns)), B + N - 1
    g = torch.Generator(device="cuda").manual_seed(d)
    q, k, v = (torch.randn((T, H, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    o, lse = fa.attention_packed(q, k, v, cu, cu, N, N)
    ok()
    one, rows = dev([0, N]), slice(at, at + N)
    o1, l1 = fa.attention_packed(q[rows], k[rows], v[rows], one, one, N, N)
    ok()
    assert torch.equal(o[rows], o1) and torch.equal(lse[:, rows], l1)
    out = torch.ones(T, dtype=torch.bool, device="cuda")
    out[rows] = False
    assert torch.equal(o[out], v[out])
    want = (q.double() * k.double()).sum(-1).t() * fa.default_scale(d)
    assert ((lse - want)[:, out]).abs().max() <= 1e-3


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks,long", [(0, 0, 1), (60, 130, 1), (0, 0, 40)])
def test_falling_offsets_are_reported_and_touch_nothing_else(d, window, sinks, long):
    """Sequences that lie over one another because offsets fall: reported, and no row outside of them is written."""
    H, Hkv, T = 4, 2, 300 * long
    cu = dev([0, 100 * long, 50 * long, 200 * long, 20 * long, 120 * long])
    q, k, v, do = (x.cuda() for x in make(T, T, H, Hkv, d, 4))
    most = 150 * long
    o, lse = fa.attention_packed(q, k, v, dev([0, T]), dev([0, T]), T, T, window, sinks)
    ok()
    mine = [torch.full_like(x, 7.0) for x in (q, lse, q, k, v)]
    fa.fa_fwd_packed(q, k, v, mine[0], mine[1], cu, cu, most, most, window, sinks)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_SEQLENS
    ws = torch.zeros(fa.fa_bwd_packed_workspace_bytes(5, T, T, most, most, H, Hkv, d, window, sinks) // 4 + 1024, device="cuda")
    guard = ws[-1024:].fill_(5.0)
    fa.fa_bwd_packed(q, k, v, o, do, lse, *mine[2:], ws, cu, cu, most, most, window, sinks)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_SEQLENS
    assert torch.all(guard == 5.0)
    for x in (mine[0], mine[1].t(), *mine[2:]):
        assert torch.all(x[200 * long:] == 7.0)


def test_strided_tokens():
    """A fused projection's columns, and gradients written into one: the same bits as separate tensors."""
    H, Hkv, d, ns = 8, 2, 128, [300, 1, 77]
    T = sum(ns)
    q, k, v, do = (x.cuda() for x in make(T, T, H, Hkv, d, 5))
    fused = torch.cat([q, k, v], 1).contiguous()
    fq, fk, fv = fused[:, :H], fused[:, H: H + Hkv], fused[:, H + Hkv:]
    batch = (dev(cu_of(ns)), dev(cu_of(ns)), 300, 300)
    o, lse = fa.attention_packed(q, k, v, *batch)
    of, lf = fa.attention_packed(fq, fk, fv, *batch)
    assert torch.equal(o, of) and torch.equal(lse, lf)
    wide = torch.zeros((T, H + 3, d), dtype=torch.bfloat16, device="cuda")
    wide[:, 1: 1 + H] = do
    grads = fa.attention_packed_backward(q, k, v, o, lse, do, *batch)
    dfused = torch.full_like(fused, 9.0)
    ws = torch.empty(fa.fa_bwd_packed_workspace_bytes(len(ns), T, T, 300, 300, H, Hkv, d) // 4, device="cuda")
    fa.fa_bwd_packed(fq, fk, fv, o, wide[:, 1: 1 + H], lse, dfused[:, :H], dfused[:, H: H + Hkv], dfused[:, H + Hkv:], ws,
                     *batch)
    ok()
    assert torch.equal(dfused[:, H: H + Hkv], grads[1]) and torch.equal(dfused[:, H + Hkv:], grads[2])
    assert (dfused[:, :H].float() - grads[0].float()).abs().max() <= 2.0 ** -7 * grads[0].float().abs().max()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_tokens_behind_four_gigabytes(d):
    """Tokens so far apart that their offsets do not fit 32 bits: the bits of tokens that lie together."""
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB of device memory")
    H, Hkv, ns, window, sinks = 4, 2, [900, 1, 700], 300, 2
    T, gap = sum(ns), 2 ** 21
    q, k, v, do = (x.cuda() for x in make(T, T, H, Hkv, d, 5))
    batch = (dev(cu_of(ns)), dev(cu_of(ns)), max(ns), max(ns), window, sinks)
    o, lse = fa.attention_packed(q, k, v, *batch)
    grads = fa.attention_packed_backward(q, k, v, o, lse, do, *batch)
    wide = torch.empty((T, gap), dtype=torch.bfloat16, device="cuda")
    place = lambda i, h: wide[:, i * 2 ** 17: i * 2 ** 17 + h * d].unflatten(1, (h, d))  # noqa: E731
    far = [place(i, x.shape[1]) for i, x in enumerate((q, k, v, do, *grads))]
    assert gap * (T - 1) > 2 ** 31
    for x, y in zip(far, (q, k, v, do)):
        x.copy_(y)
    of, lf = fa.attention_packed(*far[:3], *batch)
    ws = torch.empty(fa.fa_bwd_packed_workspace_bytes(len(ns), T, T, max(ns), max(ns), H, Hkv, d, window, sinks) // 4,
                     device="cuda")
    fa.fa_bwd_packed(*far[:3], of, far[3], lf, *far[4:], ws, *batch)
    ok()
    assert torch.equal(o, of) and torch.equal(lse, lf)
    assert torch.equal(far[5], grads[1]) and torch.equal(far[6], grads[2])
    assert (far[4].float() - grads[0].float()).abs().max() <= 2.0 ** -7 * grads[0].float().abs().max()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_the_sequences_has_no_influence(d, bad):
    """Infinities and NaN in other sequences, before the first and behind the last one: the same bits."""
    H, Hkv, ns, ms = 4, 2, [70, 130, 1, 33], [70, 200, 129, 33]
    cu_q, cu_k = cu_of(ns, 5), cu_of(ms, 3)
    T, S = int(cu_q[-1]) + 140, int(cu_k[-1]) + 140
    q, k, v, do = (x.cuda() for x in make(T, S, H, Hkv, d, 7))
    batch = (dev(cu_q), dev(cu_k), 130, 200, 60, 2)
    o, lse = fa.attention_packed(q, k, v, *batch)
    g = fa.attention_packed_backward(q, k, v, o, lse, do, *batch)
    ok()
    for b in range(len(ns)):
        rows, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        x = [t.clone() for t in (q, k, v, do)]
        for t, keep in zip(x, (rows, keys, keys, rows)):
            t.fill_(bad)
        for t, s, keep in zip(x, (q, k, v, do), (rows, keys, keys, rows)):
            t[keep] = s[keep]
        o2, l2 = fa.attention_packed(*x[:3], *batch)
        # (The others' rows of O and LSE are NaN or not; the backward gets them as they are.)
        g2 = fa.attention_packed_backward(*x[:3], o2, l2, x[3], *batch)
        ok()
        assert torch.equal(o2[rows], o[rows]) and torch.equal(l2[:, rows], lse[:, rows])
        assert torch.equal(g2[1][keys], g[1][keys]) and torch.equal(g2[2][keys], g[2][keys])
        assert (g2[0][rows].float() - g[0][rows].float()).abs().max() <= 2.0 ** -7 * g[0][rows].float().abs().max() + 1e-30


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_of_no_sequence(d):
    """Before the first sequence and behind the last one: zeros and -inf in new outputs, left alone in the caller's."""
    H, Hkv, ns = 6, 2, [30, 100]
    cu = cu_of(ns, 9)
    T = int(cu[-1]) + 50
    q, k, v, do = (x.cuda() for x in make(T, T, H, Hkv, d, 8))
    batch = (dev(cu), dev(cu), 100, 100)
    out = torch.ones(T, dtype=torch.bool)
    out[cu[0]: cu[-1]] = False
    o, lse = fa.attention_packed(q, k, v, *batch)
    grads = fa.attention_packed_backward(q, k, v, o, lse, do, *batch)
    ok()
    assert torch.all(o[out] == 0) and torch.all(lse[:, out] == -float("inf")) and torch.all(torch.isfinite(lse[:, ~out]))
    for x in grads:
        assert torch.all(x[out] == 0) and torch.all(torch.isfinite(x)) and x[~out].abs().max() > 0
    mine = [torch.full_like(x, 7.0) for x in (o, lse, *grads)]
    fa.fa_fwd_packed(q, k, v, mine[0], mine[1], *batch)
    ws = torch.empty(fa.fa_bwd_packed_workspace_bytes(2, T, T, 100, 100, H, Hkv, d) // 4, device="cuda")
    fa.fa_bwd_packed(q, k, v, o, do, lse, *mine[2:], ws, *batch)
    ok()
    assert torch.all(mine[1][:, out] == 7.0)
    for x in (mine[0], *mine[2:]):
        assert torch.all(x[out] == 7.0)
    assert torch.equal(mine[0][~out], o[~out]) and torch.equal(mine[3][~out], grads[1][~out])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_sixteen_byte_alignment(d):
    """Every tensor and the workspace at a multiple of 16 bytes that is none of 32, tokens an odd number of 16 bytes
    apart: the same bits."""
    H, Hkv, ns, window, sinks = 4, 2, [130, 1, 70], 60, 2
    T = sum(ns)
    q, k, v, do = (x.cuda() for x in make(T, T, H, Hkv, d, 8))
    batch = (dev(cu_of(ns)), dev(cu_of(ns)), max(ns), max(ns), window, sinks)
    o, lse = fa.attention_packed(q, k, v, *batch)
    grads = fa.attention_packed_backward(q, k, v, o, lse, do, *batch)

    def odd(h):
        row = torch.zeros((T, h * d + 24), dtype=torch.bfloat16, device="cuda")
        x = row[:, 8: 8 + h * d].unflatten(1, (h, d))
        assert x.data_ptr() % 32 == 16 and x.stride(0) % 16 == 8
        return x

    far = [odd(h).copy_(x) for h, x in zip((H, Hkv, Hkv, H), (q, k, v, do))]
    of = torch.empty(T * H * d + 8, dtype=torch.bfloat16, device="cuda")[8:].view(T, H, d)
    lf = torch.empty(T * H + 1, device="cuda")[1:].view(H, T)
    fa.fa_fwd_packed(*far[:3], of, lf, *batch)
    assert of.data_ptr() % 32 == 16 and torch.equal(o, of) and torch.equal(lse, lf)
    out = [odd(h) for h in (H, Hkv, Hkv)]
    ws = torch.empty(fa.fa_bwd_packed_workspace_bytes(len(ns), T, T, max(ns), max(ns), H, Hkv, d, window, sinks) // 4 + 4,
                     device="cuda")[4:]
    assert ws.data_ptr() % 32 == 16
    fa.fa_bwd_packed(*far[:3], of, far[3], lf, *out, ws, *batch)
    ok()
    assert torch.equal(out[1], grads[1]) and torch.equal(out[2], grads[2])
    assert (out[0].float() - grads[0].float()).abs().max() <= 2.0 ** -7 * grads[0].float().abs().max()


def test_broken_offsets_leave_the_others_their_results():
    H, Hkv, d, ns = 4, 2, 64, [40, 50, 60]
    T = sum(ns)
    q, k, v, do = (x.cuda() for x in make(T, T, H, Hkv, d, 9))
    cu = cu_of(ns)
    o, lse = fa.attention_packed(q, k, v, dev(cu), dev(cu), 60, 60)
    grads = fa.attention_packed_backward(q, k, v, o, lse, do, dev(cu), dev(cu), 60, 60)
    ok()
    n = 2 ** 31 - 1
    # (offsets of queries, of keys, the longest, the sequences that are sound)
    for cq, ck, most, good in (([0, 40, 30, 150], cu, 60, [0]), ([0, 40, 200, 150], cu, 60, [0]),
                               (cu, [0, 40, -9, 150], 60, [0]), ([-4, 40, 90, 150], cu, 60, [1, 2]),
                               (cu, cu, 50, [0, 1]), ([0, n, 90, 150], cu, 60, [2]), (cu, [0, 40, 90, 151], 60, [0, 1]),
                               ([150, 90, 40, 0], [150, 90, 40, 0], 60, [])):
        x = [torch.full_like(t, 3.0) for t in (o, lse, *grads)]
        batch = (dev(cq), dev(ck), most, most)
        fa.fa_fwd_packed(q, k, v, x[0], x[1], *batch)
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_SEQLENS
        ws = torch.empty(fa.fa_bwd_packed_workspace_bytes(3, T, T, most, most, H, Hkv, d) // 4, device="cuda")
        fa.fa_bwd_packed(q, k, v, o, do, lse, *x[2:], ws, *batch)
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_SEQLENS
        for b in good:
            s = slice(cu[b], cu[b + 1])
            assert torch.equal(x[0][s], o[s]) and torch.equal(x[1][:, s], lse[:, s]), (cq, ck, b)
            assert torch.equal(x[3][s], grads[1][s]) and torch.equal(x[4][s], grads[2][s]), (cq, ck, b)
            assert (x[2][s].float() - grads[0][s].float()).abs().max() <= 2.0 ** -7 * grads[0][s].float().abs().max()


def test_bounds_above_the_lengths():
    """Loose bounds give the same bits."""
    H, Hkv, d, ns = 4, 1, 128, [33, 129]
    T = sum(ns)
    q, k, v, do = (x.cuda() for x in make(T, T, H, Hkv, d, 10))
    cu = dev(cu_of(ns))
    o, lse = fa.attention_packed(q, k, v, cu, cu, 129, 129)
    g = fa.attention_packed_backward(q, k, v, o, lse, do, cu, cu, 129, 129)
    o2, l2 = fa.attention_packed(q, k, v, cu, cu, T, T)
    g2 = fa.attention_packed_backward(q, k, v, o2, l2, do, cu, cu, T, T)
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, l2) and torch.equal(g[2], g2[2])


def test_gradients_against_differences():
    """The gradients' products with a direction against central differences of the oracle's forward."""
    H, Hkv, d, window, sinks, ns, ms = 4, 2, 64, 50, 3, [100, 1, 70], [130, 20, 70]
    cu_q, cu_k = cu_of(ns), cu_of(ms)
    q, k, v, do = make(sum(ns), sum(ms), H, Hkv, d, 7)
    _, lim, _ = reference(q, k, v, do, cu_q, cu_k, window, sinks)
    gq, gk, gv, gdo = (x.cuda() for x in (q, k, v, do))
    batch = (dev(cu_q), dev(cu_k), 100, 130, window, sinks)
    o, lse = fa.attention_packed(gq, gk, gv, *batch)
    grads = dict(zip(("dq", "dk", "dv"), fa.attention_packed_backward(gq, gk, gv, o, lse, gdo, *batch)))
    ok()
    rng = np.random.default_rng(0)
    scale, h = fa.default_scale(d), 1e-4
    for n, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        base = [f64(q), f64(k), f64(v)]
        step = rng.standard_normal(base[i].shape)
        f = []
        for sgn in (1, -1):
            x = [t.copy() for t in base]
            x[i] += sgn * h * step
            f.append((orc.packed_forward(*x, cu_q, cu_k, scale, window, sinks)[0] * f64(do)).sum())
        diff = (f[0] - f[1]) / (2 * h)
        assert abs(diff - (f64(grads[n]) * step).sum()) <= (lim[n] * np.abs(step)).sum() + 1e-4 * abs(diff)


def test_captured_replayed_and_on_side_streams():
    """A captured step replayed after its offsets and inputs changed; calls on two streams at once."""
    H, Hkv, d = 4, 2, 128
    T = 600
    q, k, v, do = (x.cuda() for x in make(T, T, H, Hkv, d, 3))
    lengths = [[300, 200, 100], [1, 599, 0], [200, 200, 200]]
    eager = []
    for ns in lengths:
        batch = (dev(cu_of(ns)), dev(cu_of(ns)), 600, 600, 150, 4)
        o, lse = fa.attention_packed(q, k, v, *batch)
        eager.append((o, lse, *fa.attention_packed_backward(q, k, v, o, lse, do, *batch)))
    ok()
    cu = dev(cu_of(lengths[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.attention_packed(q, k, v, cu, cu, 600, 600, 150, 4)
        outs = (o, lse, *fa.attention_packed_backward(q, k, v, o, lse, do, cu, cu, 600, 600, 150, 4))

    def same(got, want):
        for i in (0, 1, 3, 4):
            assert torch.equal(got[i], want[i])
        assert (got[2].float() - want[2].float()).abs().max() <= 2.0 ** -7 * want[2].float().abs().max()

    for i in (1, 0, 2, 1):
        cu.copy_(dev(cu_of(lengths[i])))
        for x in outs:
            x.fill_(9.0)
        graph.replay()
        ok()
        same(outs, eager[i])
    sides = [torch.cuda.Stream() for _ in range(2)]
    cus = [dev(cu_of(ns)) for ns in lengths]
    for _ in range(10):
        got = []
        for i, s in enumerate(sides):
            s.wait_stream(torch.cuda.current_stream())
            o, lse = fa.attention_packed(q, k, v, cus[i], cus[i], 600, 600, 150, 4, stream=s)
            got.append((o, lse, *fa.attention_packed_backward(q, k, v, o, lse, do, cus[i], cus[i], 600, 600, 150, 4,
                                                              stream=s)))
        for s in sides:
            torch.cuda.current_stream().wait_stream(s)
        for i in range(2):
            same(got[i], eager[i])
    ok()


def test_outliers_and_large_scores():
    """Keys eight times as large: rows dominated by one key stay exact up to their roundings."""
    H, Hkv, d, window, sinks, ns = 2, 1, 128, 130, 2, [300, 200]
    cu = cu_of(ns)
    q, k, v, do = make(500, 500, H, Hkv, d, 9)
    k[::37] *= 8
    out, lim, lse_ref = reference(q, k, v, do, cu, cu, window, sinks)
    o, lse = fa.attention_packed(q.cuda(), k.cuda(), v.cuda(), dev(cu), dev(cu), 300, 300, window, sinks)
    ok()
    check(o, out["o"], lim["o"], "o")
    assert np.all(np.abs(f64(lse) - lse_ref) <= 1e-3 + 1e-5 * np.abs(lse_ref))


def test_a_layers_pass_on_packed_documents():
    """Rotate by the positions within each document, attend, backward, rotate the gradients back."""
    H, Hkv, d, ns = 4, 2, 64, [120, 1, 75]
    T, cu = sum(ns), cu_of(ns)
    q, k, v, do = make(T, T, H, Hkv, d, 11)
    ang = np.arange(256)[:, None] * 10000.0 ** (-np.arange(0, d, 2) / d)
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pos = np.concatenate([np.arange(n) for n in ns])[None].astype(np.int32)
    gt, gp, gcu = torch.from_numpy(table).cuda(), dev(pos), dev(cu)
    gq, gk = fa.rope(q.cuda(), k.cuda(), gt, gp)
    o, lse = fa.attention_packed(gq, gk, v.cuda(), gcu, gcu, 120, 120)
    dq, dk, dv = fa.attention_packed_backward(gq, gk, v.cuda(), o, lse, do.cuda(), gcu, gcu, 120, 120)
    fa.fa_rope(dq, dk, dq, dk, gt, gp, inverse=True)
    ok()
    turn = lambda x, inverse=False: orc.rotate(x, table, pos, [d // 2], inverse=inverse)  # noqa: E731
    rq, rk, scale = turn(f64(q)), turn(f64(k)), fa.default_scale(d)
    oref = orc.packed_forward(rq, rk, f64(v), cu, cu, scale)[0]
    gref = orc.packed_backward(rq, rk, f64(v), f64(do), cu, cu, scale)
    for x, r in zip((o, dq, dk, dv), (oref, turn(gref[0], True), turn(gref[1], True), gref[2])):
        assert np.linalg.norm(f64(x) - r) <= 1e-2 * np.linalg.norm(r)  # q and k are rounded to bf16 in between
