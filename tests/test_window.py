"""Sliding-window attention with sinks and grouped heads, forward and backward,
against the float64 oracle (oracle/serving.py), at the sizes and masks where it
can go wrong.

Tolerances, elementwise, from the roundings on the way (bf16: 2^-8 of a value).
 * O: its own rounding, and that of P, in the numerator and the denominator:
   2^-8 |o| + 2^-7 a, a = sum_j w_j |v_j|. LSE: fp32 scores and sums, 1e-3 as
   the dense path.
 * dV: its rounding and P's: 2^-8 |dv| + 2^-7 sum_i w_ij |dout_i|.
 * dS = P (dP - D): its rounding, P's, and D's error, which comes from the
   rounded O the backward gets: e_ij = w_ij (2^-7 |dP - D| + dD_i),
   dD_i = sum_c |dout_ic| (2^-8 |o_ic| + 2^-7 a_ic). dQ and dK: their own
   rounding and scale times the sum of e against |k| and |q|.
And the dense path's relative L2 bound, 5e-3, over whole tensors of at least
1000 values whose rows have keys to choose from.
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


def make(B, H, Hkv, N, M, d, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    return n(B, H, N, d), n(B, Hkv, M, d), n(B, Hkv, M, d), n(B, H, N, d)


def f64(t):
    return t.double().cpu().numpy()


def reference(q, k, v, do, window, sinks):
    """Values and bounds of every output, head by head."""
    q, k, v, do = (f64(x) for x in (q, k, v, do))
    scale = fa.default_scale(q.shape[-1])
    B, H = q.shape[:2]
    g = H // k.shape[1]
    out = {n: np.zeros(x.shape) for n, x in (("o", q), ("dq", q), ("dk", k), ("dv", v))}
    lim = {n: np.zeros(x.shape) for n, x in out.items()}
    lse = np.zeros(q.shape[:3])
    for b in range(B):
        for h in range(H):
            c = h // g
            Q, K, V, G = q[b, h], k[b, c], v[b, c], do[b, h]
            o, lse[b, h], w = orc.attend(Q, K, V, scale, window, sinks)
            a = w @ np.abs(V)
            out["o"][b, h], lim["o"][b, h] = o, 2.0 ** -8 * np.abs(o) + 2.0 ** -7 * a
            dp = G @ V.T - (G * o).sum(1, keepdims=True)
            ds = w * dp
            dD = (np.abs(G) * (2.0 ** -8 * np.abs(o) + 2.0 ** -7 * a)).sum(1, keepdims=True)
            e = w * (2.0 ** -7 * np.abs(dp) + dD)
            out["dq"][b, h], lim["dq"][b, h] = ds @ K * scale, e @ np.abs(K) * scale
            out["dk"][b, c] += ds.T @ Q * scale
            lim["dk"][b, c] += e.T @ np.abs(Q) * scale
            out["dv"][b, c] += w.T @ G
            lim["dv"][b, c] += 2.0 ** -7 * (w.T @ np.abs(G))
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


CASES = [
    # B, H, Hkv, N, M, window, sinks
    (1, 1, 1, 1, 1, 1, 0),
    (1, 2, 1, 1, 300, 7, 2),          # a single token behind a cache
    (2, 4, 2, 130, 130, 1, 0),        # every row sees itself alone
    (1, 4, 1, 300, 300, 128, 0),
    (1, 2, 2, 513, 513, 100, 1),
    (2, 3, 1, 400, 700, 129, 4),
    (1, 2, 1, 700, 400, 64, 3),       # the first 300 rows see no key
    (1, 2, 2, 640, 640, 200, 130),    # sinks past a key tile
    (1, 2, 1, 1000, 1300, 300, 257),
    (1, 4, 2, 777, 777, 5000, 4),     # the window holds everything
    (1, 6, 2, 520, 600, 0, 0),        # no window
    (1, 2, 1, 129, 1000, 40, 128),
    (1, 8, 1, 1025, 1025, 96, 0),     # one kv head for all
    # more query units than SMs: persistent CTAs (d = 64, 128)
    (2, 80, 20, 513, 513, 129, 4),
    (1, 160, 160, 300, 700, 64, 40),
    (1, 200, 100, 400, 300, 0, 0),    # the first 100 rows see no key
    (1, 160, 40, 260, 900, 200, 32),
    (1, 320, 80, 256, 256, 3, 1),
    (3, 60, 20, 257, 1000, 1, 130),
]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_window_forward_and_backward(case, d):
    B, H, Hkv, N, M, window, sinks = CASES[case]
    q, k, v, do = make(B, H, Hkv, N, M, d, 100 * case + d)
    out, lim, lse_ref = reference(q, k, v, do, window, sinks)
    gq, gk, gv, gdo = (x.cuda() for x in (q, k, v, do))
    o, lse = fa.attention_window(gq, gk, gv, window, sinks)
    ok()
    check(o, out["o"], lim["o"], "o")
    empty = np.isneginf(lse_ref)
    lse_h = f64(lse)
    assert np.array_equal(np.isneginf(lse_h), empty)
    assert np.all(np.abs(lse_h[~empty] - lse_ref[~empty]) <= 1e-3)
    dq, dk, dv = fa.attention_window_backward(gq, gk, gv, o, lse, gdo, window, sinks)
    ok()
    for n, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        check(x, out[n], lim[n], n)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_no_window_equals_the_causal_forward(d):
    """One head per kv head and no window, or one that holds everything: fa_fwd's bottom-right mask, bit for bit."""
    q, k, v, _ = make(2, 3, 3, 600, 777, d, d)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    o, lse = fa.attention(q, k, v, causal="bottom_right")
    for window in (0, 777, 1 << 29):
        ow, lw = fa.attention_window(q, k, v, window)
        ok()
        assert torch.equal(o, ow) and torch.equal(lse, lw)


def test_gradients_against_differences():
    """The gradients' products with a direction against central differences of the oracle's forward."""
    B, H, Hkv, N, M, d, window, sinks = 1, 4, 2, 200, 260, 64, 50, 3
    q, k, v, do = make(B, H, Hkv, N, M, d, 7)
    out, lim, _ = reference(q, k, v, do, window, sinks)
    gq, gk, gv, gdo = (x.cuda() for x in (q, k, v, do))
    o, lse = fa.attention_window(gq, gk, gv, window, sinks)
    grads = dict(zip(("dq", "dk", "dv"), fa.attention_window_backward(gq, gk, gv, o, lse, gdo, window, sinks)))
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
            f.append((orc.window_forward(*x, scale, window, sinks)[0] * f64(do)).sum())
        diff = (f[0] - f[1]) / (2 * h)
        assert abs(diff - (f64(grads[n]) * step).sum()) <= (lim[n] * np.abs(step)).sum() + 1e-4 * abs(diff)


def test_outliers_and_large_scores():
    """Keys eight times as large: rows dominated by one key stay exact up to their roundings."""
    B, H, Hkv, N, M, d, window, sinks = 1, 2, 1, 500, 500, 128, 130, 2
    q, k, v, do = make(B, H, Hkv, N, M, d, 9)
    k[:, :, ::37] *= 8
    out, lim, lse_ref = reference(q, k, v, do, window, sinks)
    o, lse = fa.attention_window(q.cuda(), k.cuda(), v.cuda(), window, sinks)
    ok()
    check(o, out["o"], lim["o"], "o")
    assert np.all(np.abs(f64(lse) - lse_ref) <= 1e-3 + 1e-5 * np.abs(lse_ref))


def test_window_captured_replayed_and_on_a_side_stream():
    B, H, Hkv, N, M, d, window, sinks = 2, 4, 2, 700, 700, 128, 200, 4
    q, k, v, do = (x.cuda() for x in make(B, H, Hkv, N, M, d, 3))
    o, lse = fa.attention_window(q, k, v, window, sinks)
    grads = fa.attention_window_backward(q, k, v, o, lse, do, window, sinks)
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gl = fa.attention_window(q, k, v, window, sinks)
        gg = fa.attention_window_backward(q, k, v, go, gl, do, window, sinks)
    for _ in range(3):
        for x in (go, gl, *gg):
            x.fill_(9.0)
        graph.replay()
        ok()
        assert torch.equal(go, o) and torch.equal(gl, lse)
        assert torch.equal(gg[1], grads[1]) and torch.equal(gg[2], grads[2])
        assert (gg[0].float() - grads[0].float()).abs().max() <= 2.0 ** -7 * grads[0].float().abs().max()
    side = torch.cuda.Stream()
    for _ in range(10):
        x = torch.zeros_like(q)
        x.copy_(q)
        side.wait_stream(torch.cuda.current_stream())
        so, sl = fa.attention_window(x, k, v, window, sinks, stream=side)
        sg = fa.attention_window_backward(x, k, v, so, sl, do, window, sinks, stream=side)
        x.record_stream(side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(so, o) and torch.equal(sl, lse) and torch.equal(sg[1], grads[1])
    ok()


def test_rotation_window_and_gradients_together():
    """A layer's pass: rotate, attend in a window, backward, rotate the gradients back."""
    B, H, Hkv, N, d, window, sinks = 1, 4, 2, 300, 64, 90, 4
    q, k, v, do = make(B, H, Hkv, N, N, d, 11)
    inv = 10000.0 ** (-np.arange(0, d, 2) / d)
    ang = np.arange(N)[:, None] * inv
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pos = torch.arange(N, dtype=torch.int32, device="cuda").expand(B, N).contiguous()
    gt = torch.from_numpy(table).cuda()
    gq, gk = fa.rope(q.cuda(), k.cuda(), gt, pos)
    o, lse = fa.attention_window(gq, gk, v.cuda(), window, sinks)
    dq, dk, dv = fa.attention_window_backward(gq, gk, v.cuda(), o, lse, do.cuda(), window, sinks)
    fa.fa_rope(dq, dk, dq, dk, gt, pos, inverse=True)
    ok()

    def turn(x, inverse=False):
        rows = x.transpose(0, 2, 1, 3).reshape(B * N, -1, d)
        p = np.tile(np.arange(N), B)[None]
        return orc.rotate(rows, table, p, [d // 2], inverse=inverse).reshape(B, N, -1, d).transpose(0, 2, 1, 3)

    rq, rk = turn(f64(q)), turn(f64(k))
    scale = fa.default_scale(d)
    oref, _ = orc.window_forward(rq, rk, f64(v), scale, window, sinks)
    gref = orc.window_backward(rq, rk, f64(v), f64(do), scale, window, sinks)
    refs = [oref, turn(gref[0], True), turn(gref[1], True), gref[2]]
    for x, r in zip((o, dq, dk, dv), refs):  # the rotated q and k are rounded to bf16 in between: 2^-8 each
        assert np.linalg.norm(f64(x) - r) <= 1e-2 * np.linalg.norm(r)
