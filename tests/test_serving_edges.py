"""Rotary positions, the paged cache and the window in the calls around the usual
ones: several at once, replayed graphs that share a workspace, padded batches and
loose bounds, expanded inputs, offsets past 32 bits, scales of empty blocks.

Results of the same kernel on the same values are compared bit by bit; others
with the float64 oracle at the tolerances of test_serving.py: 2^-8 |o| + 2^-10
sum_j w_j |v_j|.
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


def normal(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


def cache_of(lens, page, Hkv, d, seed, max_pages=None):
    """A cache filled by the append itself, its pages in order: (codes and scales, table)."""
    need = [-(-n // page) for n in lens]
    P = sum(need)
    width = max_pages or max(need)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    c = [torch.zeros((P, Hkv, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.ones((P, Hkv), device="cuda") for _ in range(2)]
    total = sum(lens)
    cu = i32([0] + list(np.cumsum(lens)))
    fa.kv_append_fp8(None, normal((total, Hkv, d), seed), normal((total, Hkv, d), seed + 1), *c, *s, table.cuda(), cu,
                     i32(lens), max(lens))
    return c + s, table.cuda()


def paged_oracle(q, cache, table, ns, lens, window=0, sinks=0):
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    kc, vc, ks, vs = (x.cpu().numpy() for x in cache)
    return orc.paged(f64(q), kc, vc, ks, vs, table.cpu().numpy(), cu, lens, fa.default_scale(q.shape[-1]), window, sinks)


def check(o, lse, want):
    ref, ref_lse, a = want
    assert np.all(np.abs(f64(o) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * a)
    assert np.all(np.abs(f64(lse) - ref_lse) <= 5e-4)


@pytest.mark.parametrize("n", [1, 20, 150])
def test_blocks_of_zeros(n):
    """V blocks whose scale is zero (a program that never wrote one) count as zeros beside the others."""
    lens, H, Hkv, d, page = [400], 4, 2, 128, 16
    cache, table = cache_of(lens, page, Hkv, d, 1)
    zero = torch.tensor([3, 11, 24], device="cuda")
    cache[1][zero] = 0
    cache[3][zero] = 0.0
    q = normal((n, H, d), 5)
    o, lse = fa.attention_paged_fp8(q, *cache, table, i32([0, n]), i32(lens), n, 400)
    ok()
    cache[3][zero] = 2.0 ** -100
    check(o, lse, paged_oracle(q, cache, table, [n], lens))


@pytest.mark.parametrize("splits", [1, 4])
def test_loose_bounds_and_padded_batches(splits):
    """Bounds above what the batch holds, sequences with nothing new at either end, and padding rows give
    the results of the tight call."""
    lens, H, Hkv, d, page = [33, 300, 700, 5], 8, 2, 128, 16
    cache, table = cache_of(lens, page, Hkv, d, 3, max_pages=100)
    q = normal((9, H, d), 5)
    cu = i32([0, 0, 2, 3, 3])
    ns = [0, 2, 1, 0]
    o = torch.full_like(q, 9.0)
    lse = torch.full((H, 9), 9.0, device="cuda")
    ws = torch.empty(fa.fa_paged_workspace_bytes(9, H, d, max(splits, 2)) // 4, device="cuda")
    fa.fa_fwd_paged_fp8(q, *cache, o, lse, table, cu, i32(lens), 4, 1600, ws, splits)
    ok()
    check(o[:3], lse[:, :3], paged_oracle(q[:3], cache, table, ns, lens))
    assert torch.all(o[3:] == 9.0) and torch.all(lse[:, 3:] == 9.0)
    # The append with a bound of the whole batch: the same bytes as with a tight one.
    k, v = normal((9, Hkv, d), 6), normal((9, Hkv, d), 7)
    one, two = [x.clone() for x in cache], [x.clone() for x in cache]
    fa.kv_append_fp8(None, k, v, *one, table, cu, i32(lens), 2)
    fa.kv_append_fp8(None, k, v, *two, table, cu, i32(lens), 9)
    ok()
    assert all(torch.equal(x, y) for x, y in zip(one, two)) and not torch.equal(one[0], cache[0])


def test_expanded_inputs():
    """One token's k and v for every token, one head's q for every head (strides of zero)."""
    lens, Hkv, d, page = [40], 2, 64, 16
    k, v = normal((1, Hkv, d), 1).expand(40, Hkv, d), normal((1, Hkv, d), 2).expand(40, Hkv, d)
    out = []
    for a, b in ((k, v), (k.contiguous(), v.contiguous())):
        c = [torch.zeros((3, Hkv, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
        s = [torch.ones((3, Hkv), device="cuda") for _ in range(2)]
        fa.kv_append_fp8(None, a, b, *c, *s, i32([[0, 1, 2]]), i32([0, 40]), i32(lens), 40)
        out.append(c + s)
    ok()
    assert all(torch.equal(x, y) for x, y in zip(*out))
    table = torch.rand(64, d, device="cuda")
    x = normal((1, 1, 7, d), 3).expand(2, 5, 7, d)
    pos = torch.randint(0, 64, (2, 7), dtype=torch.int32, device="cuda")
    assert torch.equal(fa.rope(x, None, table, pos), fa.rope(x.contiguous(), None, table, pos))
    ok()


def test_calls_at_once():
    """Calls of every kernel on four streams at the same time, many times over: the bits of the calls alone."""
    d, page, H, Hkv = 128, 16, 8, 2
    lens = [900, 300, 2000]
    cache, table = cache_of(lens, page, Hkv, d, 1)
    jobs = []
    for ns in ([1, 1, 1], [9, 3, 7], [200, 140, 333]):  # rows, dual and full tiles
        q = normal((sum(ns), H, d), sum(ns))
        cu, ln = i32([0] + list(np.cumsum(ns))), i32(lens)
        jobs.append(lambda s, q=q, cu=cu, ln=ln, n=max(ns): fa.attention_paged_fp8(q, *cache, table, cu, ln, n, 2000,
                                                                                  num_splits=3, stream=s))
    wq, wk, wv = normal((1, H, 1000, d), 2), normal((1, Hkv, 1000, d), 3), normal((1, Hkv, 1000, d), 4)
    jobs.append(lambda s: fa.attention_window(wq, wk, wv, 200, 4, stream=s))
    table_r, pos = torch.rand(64, d, device="cuda"), torch.randint(0, 64, (1, 1000), dtype=torch.int32, device="cuda")
    jobs.append(lambda s: fa.rope(wq, wk, table_r, pos, stream=s))
    alone = []
    for job in jobs:
        alone.append(job(None))
        ok()
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        for j, job in enumerate(jobs):
            got.append((j, job(streams[(i + j) % 4])))
    ok()
    for j, out in got:
        assert all(torch.equal(x, y) for x, y in zip(out, alone[j])), j


def test_two_graphs_share_a_workspace():
    """Two captured calls of different shapes with one workspace, replayed in turns on one stream."""
    d, page, H, Hkv = 128, 16, 8, 2
    lens = [900, 300]
    cache, table = cache_of(lens, page, Hkv, d, 1)
    ws = torch.empty(fa.fa_paged_workspace_bytes(64, H, d, 8) // 4, device="cuda")
    runs = []
    for ns, splits in (([1, 1], 8), ([30, 34], 3)):
        n = sum(ns)
        q, o, lse = normal((n, H, d), n), torch.empty((n, H, d), dtype=torch.bfloat16, device="cuda"), \
            torch.empty((H, n), device="cuda")
        cu, ln = i32([0] + list(np.cumsum(ns))), i32(lens)
        args = (q, *cache, o, lse, table, cu, ln, max(ns), 900, ws, splits)
        fa.fa_fwd_paged_fp8(*args)
        ok()
        want = (o.clone(), lse.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.fa_fwd_paged_fp8(*args)
        runs.append((g, o, lse, want, args))  # (a graph does not keep its tensors)
    for _ in range(10):
        for g, o, lse, _, _ in runs:
            o.zero_()
            lse.zero_()
            g.replay()
        ok()
        for g, o, lse, want, _ in runs:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("n", [1, 40])
def test_cache_past_32_bit_offsets(n):
    """Pages whose codes lie more than 2^32 bytes into the cache."""
    d, page, H, Hkv = 128, 64, 8, 4
    pages = (5 << 30) // (Hkv * page * d)
    lens = [500]
    small, st = cache_of(lens, page, Hkv, d, 1)
    q, k, v = normal((n, H, d), 5), normal((n, Hkv, d), 6), normal((n, Hkv, d), 7)
    big = [torch.empty((pages, Hkv, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    big += [torch.empty((pages, Hkv), device="cuda") for _ in range(2)]
    table = st.clone()
    for i in range(8):
        at = pages - 1 - 2 * i
        table[0, i] = at
        for x, y in zip(big, small):
            x[at] = y[i]
    cu, ln = i32([0, n]), i32(lens)
    for cache, t in ((big, table), (small, st)):
        fa.kv_append_fp8(None, k, v, *cache, t, cu, ln, n)
    got = fa.attention_paged_fp8(q, *big, table, cu, ln, n, 500, num_splits=2)
    want = fa.attention_paged_fp8(q, *small, st, cu, ln, n, 500, num_splits=2)
    ok()
    for i in range(8):
        assert all(torch.equal(x[table[0, i]], y[i]) for x, y in zip(big, small))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rope_past_32_bit_offsets():
    N, d = 33, 64
    far = (1 << 31) + 64
    buf = torch.empty(far + 2 * N * d, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, 2, N, d), (far, N * d, d, 1))
    x.copy_(normal((2, 2, N, d), 1))
    table, pos = torch.rand(64, d, device="cuda"), torch.randint(0, 64, (2, N), dtype=torch.int32, device="cuda")
    want = fa.rope(x.contiguous(), None, table, pos)
    fa.fa_rope(x, None, x, None, table, pos)
    ok()
    assert torch.equal(x, want)


def test_window_past_32_bit_offsets():
    """2^31 query elements: the last rows of the last head, forward and backward, against the call on
    the keys and rows that they depend on alone."""
    H, Hkv, d, W = 64, 8, 128, 100
    N = (1 << 31) // (H * d) + 192
    g = torch.Generator(device="cuda").manual_seed(1)
    q, do = (torch.randn((1, H, N, d), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    k, v = (torch.randn((1, Hkv, N, d), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    o, lse = fa.attention_window(q, k, v, W)
    dq, dk, dv = fa.attention_window_backward(q, k, v, o, lse, do, W)
    ok()
    # Rows N - R and later see the last R + W - 1 keys; the last R keys are seen by
    # rows N - R and later alone.
    R = 64
    G = H // Hkv
    qs, dos = (f64(t[:, -G:, -R:]) for t in (q, do))
    ks, vs = (f64(t[:, -1:, -(R + W - 1):]) for t in (k, v))
    scale = fa.default_scale(d)
    ro, rl = orc.window_forward(qs, ks, vs, scale, W, 0)
    rq, rk, rv = orc.window_backward(qs, ks, vs, dos, scale, W, 0)
    rel = lambda x, y: np.linalg.norm(f64(x) - y) / np.linalg.norm(y)  # noqa: E731
    # Norms of errors that are independent roundings: O one rounding of P and one of O
    # (2^-9 on average, at most 2^-7); gradients a few more.
    assert rel(o[:, -G:, -R:], ro) <= 2.0 ** -7 and np.abs(f64(lse[:, -G:, -R:]) - rl).max() <= 1e-3
    assert rel(dq[:, -G:, -R:], rq) <= 2.0 ** -7
    assert rel(dk[:, -1:, -R:], rk[:, :, -R:]) <= 2.0 ** -7 and rel(dv[:, -1:, -R:], rv[:, :, -R:]) <= 2.0 ** -7


def test_compiled_calls_equal_the_python_ones():
    """The compiled form of a call and the Python one (taken on a stream that is named) give the same bits, and
    errors come from either as they should."""
    fa.load_library()
    here = torch.cuda.current_stream()
    q, k = normal((2, 4, 33, 64), 1), normal((2, 2, 33, 64), 2)
    table = torch.rand(99, 64, device="cuda")
    pos = torch.randint(0, 99, (3, 2, 33), dtype=torch.int32, device="cuda")
    fused = normal((50, 8, 128), 3)
    rows, rpos = torch.rand(99, 96, device="cuda"), torch.randint(0, 99, (1, 50), dtype=torch.int32, device="cuda")
    for a, kw in (((q, k, table, pos), dict(sections=(8, 12, 12))), ((q, None, table, pos[0]), dict(inverse=True)),
                  ((q.transpose(1, 2).contiguous().transpose(1, 2), k, table, pos), dict(sections=[8, 24, 0])),
                  ((fused[:, :6], fused[:, 6:], rows, rpos), dict(interleaved=True)),
                  ((q[:1].expand(2, 4, 33, 64), k, table, pos[1]), {})):
        assert fa._compiled.rope(*a, kw.get("sections"), kw.get("interleaved", False), kw.get("inverse", False)) is not None
        x, y = fa.rope(*a, **kw), fa.rope(*a, **kw, stream=here)
        ok()
        for u, v in zip(x if a[1] is not None else (x,), y if a[1] is not None else (y,)):
            assert torch.equal(u, v) and u.is_contiguous() and u.dtype is torch.bfloat16
    lens, d, page = [50, 20], 128, 16
    cache, pages = cache_of(lens, page, 1, d, 1)
    cu = i32([0, 3, 4])
    for qq, kw in ((fused[:4, :6], dict(table=rows)), (None, {}),
                   (fused[:4, :6], dict(table=rows, positions=rpos[0, :4].contiguous(), interleaved=True)),
                   (fused[:4, :6], dict(table=rows, positions=rpos[:, :4].repeat(2, 1).contiguous(), sections=(20, 28)))):
        got = []
        for stream in (None, here):
            c = [x.clone() for x in cache]
            got.append([fa.kv_append_fp8(qq, fused[:4, 6:7], fused[:4, 7:], *c, pages, cu, i32(lens), 3, **kw,
                                         stream=stream)] + c)
            ok()
        assert (got[0][0] is None) == (qq is None)
        assert all(x is None or torch.equal(x, y) for x, y in zip(*got))
    qd = normal((4, 6, 128), 9)
    for kw in ({}, dict(num_splits=2, window=9, sinks=2), dict(scale=0.2)):
        x, y = (fa.attention_paged_fp8(qd, *cache, pages, cu, i32(lens), 3, 60, **kw, stream=s) for s in (None, here))
        ok()
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    w = [normal(x, i, 0.5) for i, x in enumerate([(2, 4, 150, 64), (2, 2, 170, 64), (2, 2, 170, 64), (2, 4, 150, 64)])]
    for kw in (dict(sinks=3), dict(scale=0.2)):
        x, y = (fa.attention_window(*w[:3], 40, **kw, stream=s) for s in (None, here))
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
        x, y = (fa.attention_window_backward(*w[:3], *x, w[3], 40, **kw, stream=s) for s in (None, here))
        ok()
        assert torch.equal(x[1], y[1]) and torch.equal(x[2], y[2])
        # (dQ is summed by atomics: at most a rounding of bf16 apart, and of the fp32 sums.)
        assert (x[0].float() - y[0].float()).abs().max() <= 2.0 ** -7 * y[0].float().abs().max()
    # Errors: a status of the library's, and what only the Python form names.
    for bad, err in ((lambda: fa.attention_paged_fp8(qd, *cache, pages, cu, i32(lens), 3, 60, sinks=1), fa.FAError),
                     (lambda: fa.attention_paged_fp8(qd, *cache, pages, cu, i32(lens), 3, 10 ** 6), fa.FAError),
                     (lambda: fa.attention_paged_fp8(qd.float(), *cache, pages, cu, i32(lens), 3, 60), TypeError),
                     (lambda: fa.attention_paged_fp8(qd, *cache, pages.long(), cu, i32(lens), 3, 60), ValueError),
                     (lambda: fa.rope(q, k, table[:, :40].contiguous(), pos[0]), fa.FAError),
                     (lambda: fa.rope(q, k, table, pos[0], sections=(8, 8)), ValueError),
                     (lambda: fa.rope(q, k, table.cpu(), pos[0]), ValueError),
                     (lambda: fa.attention_window(*w[:3], 0, 1), fa.FAError),
                     (lambda: fa.attention_window(w[0], w[1][:, :, :9], w[2], 4), ValueError),
                     (lambda: fa.attention_window_backward(*w[:3], w[3], torch.zeros(2, 4, 149, device="cuda"), w[3], 4), ValueError),
                     (lambda: fa.attention_window_backward(*w[:3], w[3].half(), torch.zeros(2, 4, 150, device="cuda"), w[3], 4), TypeError),
                     (lambda: fa.kv_append_fp8(None, fused[:4, 6:7], fused[:4, 7:], *cache, pages, cu, i32(lens), 0), fa.FAError),
                     (lambda: fa.kv_append_fp8(None, fused[:4, 6:7], fused[:3, 7:], *cache, pages, cu, i32(lens), 3), ValueError)):
        with pytest.raises(err):
            bad()
    ok()


@pytest.mark.parametrize("case", [
    # new tokens, cache lengths, page, H, Hkv, window, sinks, splits
    ([17], [17], 16, 1, 1, 0, 0, None),
    ([20, 3], [129, 128], 128, 4, 4, 0, 0, None),
    ([40, 0, 65], [300, 9, 700], 32, 8, 2, 0, 0, 3),
    ([129], [1500], 64, 2, 1, 0, 0, 1),
    ([300, 130], [900, 2100], 16, 4, 2, 200, 3, 2),
    ([5, 8], [1300, 600], 64, 16, 2, 129, 64, None),
    ([70], [4000], 16, 4, 2, 1, 0, 4),
])
def test_wide_heads_many_rows(case):
    """d = 256 with more than 16 rows a kv head: one row tile, S in two buffers."""
    ns, lens, page, H, Hkv, window, sinks, splits = case
    d = 256
    cache, table = cache_of(lens, page, Hkv, d, 21)
    g = torch.Generator().manual_seed(4)
    grow = torch.exp2(torch.randint(-3, 4, (sum(ns), 1, 1), generator=g).float()).cuda()
    q = (normal((sum(ns), H, d), 8).float() * grow).to(torch.bfloat16)  # some rows' maxima move often
    cu = i32([0] + list(np.cumsum(ns)))
    o, lse = fa.attention_paged_fp8(q, *cache, table, cu, i32(lens), max(ns), max(lens), window=window, sinks=sinks,
                                    num_splits=splits)
    ok()
    # Rows up to eight times as large: elements of Q far below the row's largest (24 or so) are off by 2^-18 of
    # it, scores by about sqrt(256) 2^-18 24 scale = 1e-4, weights by as much beside P's 2^-11.
    ref, ref_lse, a = paged_oracle(q, cache, table, ns, lens, window, sinks)
    assert np.all(np.abs(f64(o) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * a)
    assert np.all(np.abs(f64(lse) - ref_lse) <= 2e-3)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("case", [
    # B, H, Hkv, N, M, window, sinks, splits
    (1, 2, 1, 1, 4096, 0, 0, 16), (1, 2, 1, 1, 200, 0, 0, 7), (2, 4, 2, 300, 900, 0, 0, 3),
    (1, 2, 2, 257, 2000, 700, 300, 5),   # sinks of three tiles, cut within them, and a gap
    (1, 2, 1, 512, 3000, 130, 4, 2),     # a first step of the sinks alone, and a hole behind it
    (1, 2, 1, 512, 3000, 1, 0, 4), (1, 1, 1, 400, 100, 0, 0, 2),  # rows that see no key
    (1, 2, 1, 200, 1500, 400, 129, 64),  # more splits than tiles
    (1, 3, 1, 129, 129, 60, 10, None), (1, 8, 2, 5, 3000, 0, 0, None),
])
def test_window_with_split_keys(case, d):
    """Split keys give the result of the whole: P rounded to bf16 (2^-8 of a weight) and O (2^-8)."""
    B, H, Hkv, N, M, window, sinks, splits = case
    q, k, v = normal((B, H, N, d), 1), normal((B, Hkv, M, d), 2), normal((B, Hkv, M, d), 3)
    o, lse = fa.attention_window(q, k, v, window, sinks, num_splits=splits)
    o2, lse2 = fa.attention_window(q, k, v, window, sinks, num_splits=splits, stream=torch.cuda.current_stream())
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    scale = fa.default_scale(d)
    ref, rl = orc.window_forward(f64(q), f64(k), f64(v), scale, window, sinks)
    a = orc.window_forward(f64(q), f64(k), np.abs(f64(v)), scale, window, sinks)[0]
    assert np.all(np.abs(f64(o) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.1 * 2.0 ** -8 * a)
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(f64(lse)), empty) and np.all(f64(o)[empty] == 0)
    assert np.all(np.abs(f64(lse)[~empty] - rl[~empty]) <= 1e-3)


@pytest.mark.parametrize("new,d,splits", [(1, 64, 4), (1, 256, 2), (4, 128, 8), (10, 128, 3), (20, 64, 1), (40, 128, 2),
                                          (90, 128, 2), (30, 256, 3)])
def test_broken_batches_in_every_kernel(new, d, splits):
    """Offsets, lengths and pages that are wrong: that sequence alone is left as it was and reported, whichever
    kernel takes the call (single tokens as clusters, row copies, full tiles, wide heads)."""
    page, Hkv, H = 16, 2, 8
    lens = [200, 300, 250]
    cache, table = cache_of(lens, page, Hkv, d, 31, max_pages=20)
    q = normal((3 * new, H, d), 4)
    good = [0, new, 2 * new, 3 * new]
    full = fa.attention_paged_fp8(q, *cache, table, i32(good), i32(lens), new, 320, num_splits=splits)
    ok()
    for cu, ln, at, code, broken in (([0, new, 2 * new, 3 * new + 1], lens, None, 12, [2]),
                                     (good, [200, new - 1, 250], None, 12, [1]), (good, [321, 300, 250], None, 12, [0]),
                                     ([0, new, new - 1, 3 * new], lens, None, 12, [1, 2]),
                                     (good, lens, (1, 3, 10 ** 6), 14, [1]), (good, lens, (2, 15, -7), 14, [2])):
        t = table.clone()
        if at:
            t[at[0], at[1]] = at[2]
        o = torch.full_like(q, 3.0)
        lse = torch.full((H, 3 * new), 2.0, device="cuda")
        ws = torch.empty(max(1, fa.fa_paged_workspace_bytes(3 * new, H, d, splits) // 4), device="cuda")
        fa.fa_fwd_paged_fp8(q, *cache, o, lse, t, i32(cu), i32(ln), new, 320, ws, splits)
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == code
        for b in range(3):
            rows = slice(b * new, (b + 1) * new)
            if b not in broken and cu == good:
                same = torch.equal(o[rows], full[0][rows]) and torch.equal(lse[:, rows], full[1][:, rows])
                # (The lengths of a batch also choose where its sequences are cut.)
                assert same or (o[rows].float() - full[0][rows].float()).abs().max() <= 2.0 ** -6
            elif code == 12 and b in broken and cu == good:
                assert torch.all(o[rows] == 3.0) and torch.all(lse[:, rows] == 2.0)
