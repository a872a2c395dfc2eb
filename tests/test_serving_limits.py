"""The edges of what the serving calls state in include/fa.h: elements that are not finite,
queries whose elements lie far apart, and the paths that only large batches take.

Tolerances as in test_serving.py (2^-8 |o| + 2^-10 sum_j w_j |v_j|, LSE 5e-4) unless a test
says otherwise.
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


def cache_of(lens, page, Hkv, d, seed):
    """A cache of random codes and scales in shuffled pages: [k, v, k_scale, v_scale], table."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    P = sum(need)
    ids = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at: at + n]
        at += n
    codes = [(torch.randn((P, Hkv, page, d), generator=g, device="cuda") * 90).clamp(-448, 448)
             .to(torch.float8_e4m3fn).view(torch.uint8)
             for _ in range(2)]
    scales = [torch.exp2(torch.randint(-8, -5, (P, Hkv), generator=g, device="cuda").float()) for _ in range(2)]
    return codes + scales, table


def paged_oracle(q, cache, table, ns, lens, window=0, sinks=0):
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    kc, vc, ks, vs = (x.cpu().numpy() for x in cache)
    return orc.paged(f64(q), kc, vc, ks, vs, table.cpu().numpy(), cu, lens, fa.default_scale(q.shape[-1]), window, sinks)


# 8 rows per token: the kernel for up to 16 rows (as clusters, through the workspace and
# unsplit), row copies of four and two, full tiles of one row block, several row blocks.
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,splits", [(1, 4), (2, 1), (2, 12), (4, 2), (8, 1), (15, 3), (40, 1), (40, 2)])
def test_queries_that_are_not_finite(n, d, splits):
    """A row that holds an infinity or a NaN gives NaN, also where each of its scores is minus infinity; the
    other rows keep their bits."""
    H, Hkv, page, lens = 8, 1, 16, [700, 450]
    cache, table = cache_of(lens, page, Hkv, d, 3)
    cache[0] &= 0x7F        # keys above zero
    cache[0].clamp_(8, 0x7E)
    q = normal((2 * n, H, d), n)
    args = (*cache, table, i32([0, n, 2 * n]), i32(lens), n, 700)
    want, want_lse = fa.attention_paged_fp8(q, *args, num_splits=splits)
    ok()
    bad = torch.zeros((2 * n, H), dtype=torch.bool, device="cuda")
    for i, x in enumerate((float("inf"), -float("inf"), float("nan"))):
        at, h, c = (i * 7 + 1) % (2 * n), 2 * i + 1, (i * 29 + 5) % d
        q[at, h, c] = x
        bad[at, h] = True
    q[n, 0, 3], q[n, 0, 4], bad[n, 0] = float("inf"), -float("inf"), True
    q[2 * n - 1, 6, d - 1], bad[2 * n - 1, 6] = -float("inf"), True
    o, lse = fa.attention_paged_fp8(q, *args, num_splits=splits)
    ok()
    assert torch.isnan(o[bad]).all() and torch.isnan(lse.t()[bad]).all()
    assert torch.equal(o[~bad], want[~bad]) and torch.equal(lse.t()[~bad], want_lse.t()[~bad])


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("n", [1, 3, 16, 70, 300])
def test_appended_infinities(n, rotate):
    """A new key or value that is infinite is stored as NaN, a rotated key's partner with it; its block keeps
    the scale and the codes that it has with zeros in those places."""
    d, Hkv, page = 64, 2, 64
    lens = [n + 40]
    k, v = normal((n, Hkv, d), 1), normal((n, Hkv, d), 2)
    cu, ln = i32([0, n]), i32(lens)
    pages = -(-lens[0] // page)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()[None]
    old = [torch.randint(0x20, 0x60, (pages, Hkv, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    old += [torch.full((pages, Hkv), 2.0 ** -12, device="cuda") for _ in range(2)]
    cs = None
    if rotate:
        ang = torch.rand((lens[0], d // 2), device="cuda") + 0.2
        cs = torch.cat([ang.cos(), ang.sin()], 1)
    at = torch.zeros((n, Hkv, d), dtype=torch.bool, device="cuda")
    at[0, 0, 5] = at[n // 2, 1, 17] = at[n - 1, 0, d - 1] = True
    hit = at | at.roll(d // 2, -1) if rotate else at  # pairs are half a head apart
    inf = torch.where(torch.arange(d, device="cuda") % 2 == 0, float("inf"), -float("inf")).to(torch.bfloat16).expand_as(k)
    runs = []
    for kk, vv in ((torch.where(at, inf, k), torch.where(at, inf, v)),
                   (torch.where(hit, torch.zeros_like(k), k), torch.where(at, torch.zeros_like(v), v))):
        c = [x.clone() for x in old]
        fa.kv_append_fp8(None, kk, vv, *c, table, cu, ln, n, table=cs)
        ok()
        runs.append(c)
    (kc, vc, ks, vs), (kz, vz, ksz, vsz) = runs
    assert torch.equal(ks, ksz) and torch.equal(vs, vsz)
    slot = torch.arange(40, lens[0], device="cuda")
    for got, want, places in ((kc, kz, hit), (vc, vz, at)):
        want = want.clone()
        pg = table[0].long()[slot // page]
        rows = want[pg, :, slot % page]
        want[pg, :, slot % page] = torch.where(places, torch.full_like(rows, 0x7F), rows)
        # (The sign of a NaN or of a zero is not fixed.)
        assert torch.equal(got & 0x7F, want & 0x7F)
        assert torch.equal(torch.where(got & 0x7F == 0, 0, got)[want & 0x7F != 0x7F],
                           torch.where(want & 0x7F == 0, 0, want)[want & 0x7F != 0x7F])


def test_compiled_calls_look_at_the_positions_shape():
    """The compiled calls take the shapes that the Python forms take, and leave the others to them."""
    q, table = normal((2, 4, 9, 64), 1), torch.rand(50, 64, device="cuda")
    pos = torch.randint(0, 50, (18,), dtype=torch.int32, device="cuda")
    want = fa.rope(q, None, table, pos.view(2, 9), stream=torch.cuda.current_stream())
    for shape in ((2, 9), (1, 2, 9), (18,), (1, 18)):
        assert torch.equal(fa._compiled.rope(q, None, table, pos.view(shape), None, False, False), want)
    for shape in ((9, 2), (1, 9, 2), (18, 1), (3, 6), (1, 1, 2, 9)):
        assert fa._compiled.rope(q, None, table, pos.view(shape), None, False, False) is None
        with pytest.raises(ValueError):
            fa.rope(q, None, table, pos.view(shape))
    cache, pages = cache_of([6], 16, 2, 64, 1)
    k = normal((6, 2, 64), 2)
    for shape, takes in (((6,), True), ((1, 6), True), ((6, 1), False), ((2, 3), False), ((1, 6, 1), False)):
        out = fa._compiled.append(None, k, k, *cache, pages, i32([0, 6]), i32([6]), 6, table, pos[:6].view(shape), None,
                                  False)
        assert (out is True) == takes and (takes or out is None)
    assert fa._compiled.paged(normal((6, 4, 64), 3), *cache, pages, i32([0, 6]), i32([6]), 6, 2 ** 32 + 6, 0, 0, None,
                              None) is None
    ok()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,splits", [(2, 1), (4, 2), (5, 1), (8, 3), (15, 1), (40, 1), (40, 2)])
@pytest.mark.parametrize("e", [4, 6, 10])
def test_queries_with_outlier_columns(n, splits, e, d):
    """Rows whose largest columns lie 2^e above the rest, in every kernel.

    Up to 16 rows a kv head an element of Q is off by nothing here (f16 after a power-of-two scale holds the
    eight bits of everything down to 2^-24 of the row's largest). From 17 rows on two e4m3 terms hold what is at
    least 2^-9 of the largest, and are off by at most 2^-10 where the largest lies in [2^7, 2^8): 2^-17 of it.
    A score is then off by e_j = scale sum_c |dq_c k_jc|, and by its 2 d / 32 accumulations in fp32, each by
    2^-23 of sum_c |q_c k_jc|. Weights change by a factor of at most exp(2 e), O by (exp(2 e) - 1) sum_j w_j |v_j|,
    LSE by e, e the largest e_j."""
    H, Hkv, page, lens = 8, 1, 32, [600, 333]
    cache, table = cache_of(lens, page, Hkv, d, 5)
    for s in cache[2:]:
        s *= 2.0 ** (5 - e)  # scores of about the same size for every e
    q = normal((2 * n, H, d), n + d)
    cols = torch.randperm(d, generator=torch.Generator().manual_seed(e))[:3]
    q[:, :, cols.cuda()] *= 2.0 ** e
    o, lse = fa.attention_paged_fp8(q, *cache, table, i32([0, n, 2 * n]), i32(lens), n, max(lens), num_splits=splits)
    ok()
    ref, ref_lse, a = paged_oracle(q, cache, table, [n, n], lens)
    Q, scale = np.abs(f64(q)), fa.default_scale(d)
    top = 2.0 ** np.floor(np.log2(Q.max(2, keepdims=True)))
    off = np.where(Q < 2.0 ** -9 * top, 2.0 ** -17 * top, 0.0) if n * H > 16 else np.zeros_like(Q)
    off = off + Q * (2 * d / 32) * 2.0 ** -23
    err = np.zeros((2 * n, H))
    for b in range(2):
        pages = table[b, : -(-lens[b] // page)].long()
        k = (cache[0][pages, 0].view(torch.float8_e4m3fn).double() * cache[2][pages, 0, None, None].double())
        k = np.abs(k.reshape(-1, d)[: lens[b]].cpu().numpy())
        rows = slice(b * n, (b + 1) * n)
        err[rows] = scale * (off[rows] @ k.T).max(2)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + np.expm1(2 * err))[:, :, None] * a
    assert np.all(np.abs(f64(o) - ref) <= bound)
    assert np.all(np.abs(f64(lse) - ref_lse) <= 5e-4 + err.T)


PLACES = {64: 4 * 152, 128: 3 * 152, 256: 2 * 152}  # CTAs of the 16-row kernel that run at once


def check(o, lse, want):
    ref, ref_lse, a = want
    assert np.all(np.abs(f64(o) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * a)
    assert np.all(np.abs(f64(lse) - ref_lse) <= 5e-4)


def run_paged(ns, lens, page, H, Hkv, d, splits, window=0, sinks=0, seed=7):
    assert max(ns) * H // Hkv <= 16  # the kernel for few rows
    cache, table = cache_of(lens, page, Hkv, d, seed)
    table[table < 0] = 0
    q = normal((sum(ns), H, d), seed)
    # States that no CTA fills hold NaN.
    ws = torch.full((max(1, fa.fa_paged_workspace_bytes(sum(ns), H, d, splits) // 4),), float("nan"), device="cuda")
    o, lse = torch.empty_like(q), torch.empty((H, sum(ns)), device="cuda")
    fa.fa_fwd_paged_fp8(q, *cache, o, lse, table, i32([0] + list(np.cumsum(ns))), i32(lens), max(ns), max(lens), ws, splits,
                        window, sinks)
    ok()
    check(o, lse, paged_oracle(q, cache, table, ns, lens, window, sinks))
    return ws


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ns,H,Hkv,page,splits,window,sinks", [
    ([1, 1, 1, 1, 1], 8, 2, 16, 9, 0, 0), ([1, 0, 1, 1, 1], 4, 4, 64, 16, 0, 0), ([3, 4, 1, 2, 4], 8, 2, 32, 12, 0, 0),
    ([1, 1, 2, 1, 2], 16, 2, 128, 10, 700, 40),
])
def test_few_rows_through_the_workspace(ns, H, Hkv, page, splits, window, sinks, d):
    """More splits than a cluster holds: states meet in the workspace, some sequences leave one, some all."""
    assert splits > 8
    run_paged(ns, [20, 5, 700, 5000, 2049], page, H, Hkv, d, splits, window, sinks)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("splits", [2, 5, 8])
def test_few_rows_of_more_splits_than_places(splits, d):
    """At most eight splits, but more CTAs than run at once: no clusters."""
    Hkv = 4
    B = PLACES[d] // (Hkv * splits) + 1
    assert B * Hkv * splits > PLACES[d]
    lens = np.random.default_rng(splits).integers(1, 1500, B)
    lens[:4] = 1, 16, 1500, 33
    run_paged([1] * B, [int(x) for x in lens], 16, 8, Hkv, d, splits)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("splits,length,window,sinks", [(1, 5200, 0, 0), (1, 9000, 4700, 40), (1, 8300, 8200, 3000),
                                                        (3, 14000, 0, 0), (9, 38000, 0, 0)])
def test_few_rows_over_many_tiles(splits, length, window, sinks, page, d):
    """More than 32 key tiles a warp: page ids and scales are fetched anew."""
    keys = 16 if d == 256 else 32  # of a warp's tile; four warps
    assert (min(length, window or length) // splits) > 4 * 32 * keys
    run_paged([2, 1], [length, 777], page, 8, 2, d, splits, window, sinks)


@pytest.mark.parametrize("new,d,splits", [(1, 64, 4), (1, 128, 1), (1, 256, 2), (1, 128, 12), (4, 128, 8), (10, 128, 3),
                                          (20, 64, 1), (40, 128, 2), (90, 128, 2), (30, 256, 3)])
def test_broken_offsets_leave_the_others_their_results(new, d, splits):
    """Offsets past the tokens or decreasing: the sequences whose offsets are good get their results, the rows of
    no good sequence keep what they held."""
    page, Hkv, H, lens = 16, 2, 8, [200, 300, 250]
    cache, table = cache_of(lens, page, Hkv, d, 31)
    table[table < 0] = 0
    q = normal((3 * new, H, d), 4)
    want = paged_oracle(q, cache, table, [new] * 3, lens)
    for cu, good in (([0, new, 2 * new, 3 * new + 1], 2), ([0, new, new - 1, 3 * new], 1), ([0, new, 3 * new, 3 * new], 1),
                     ([0, new, 2 * new, -1], 2)):
        o = torch.full_like(q, 3.0)
        lse = torch.full((H, 3 * new), 2.0, device="cuda")
        ws = torch.empty(max(1, fa.fa_paged_workspace_bytes(3 * new, H, d, splits) // 4), device="cuda")
        fa.fa_fwd_paged_fp8(q, *cache, o, lse, table, i32(cu), i32(lens), new, 300, ws, splits)
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_SEQLENS
        rows = good * new
        check(o[:rows], lse[:, :rows], [want[0][:rows], want[1][:, :rows], want[2][:rows]])
        assert torch.all(o[rows:] == 3.0) and torch.all(lse[:, rows:] == 2.0)


@pytest.mark.parametrize("n,H,d,window,sinks", [(1, 8, 64, 0, 0), (1, 8, 128, 500, 4), (2, 16, 256, 0, 0), (5, 8, 128, 0, 0),
                                                (40, 8, 64, 0, 0), (90, 8, 128, 300, 20), (30, 8, 256, 0, 0)])
def test_captured_steps_while_the_sequences_grow(n, H, d, window, sinks):
    """One capture of an append and the attention under a fixed bound, replayed while the batch's lengths, its
    offsets and its pages change: the results of the lengths at hand."""
    Hkv, page, bound, B = 2, 32, 4096, 3
    per = bound // page
    g = torch.Generator().manual_seed(n)
    pages = torch.randperm(B * per, generator=g).to(torch.int32).view(B, per).cuda()
    cache = [torch.zeros((B * per, Hkv, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.ones((B * per, Hkv), device="cuda") for _ in range(2)]
    # The cache holds every token already: rows behind a sequence's end are other values.
    fill = normal((B * bound, Hkv, d), 1), normal((B * bound, Hkv, d), 2)
    fa.kv_append_fp8(None, *fill, *cache, pages, i32([0, bound, 2 * bound, 3 * bound]), i32([bound] * B), bound)
    total = B * n
    q, k, v = normal((total, H, d), 3), normal((total, Hkv, d), 4), normal((total, Hkv, d), 5)
    table, cu, lens = pages.clone(), i32([0, n, 2 * n, 3 * n]), i32([n] * B)
    ang = torch.rand((bound, d // 2), generator=g).cuda()
    cs = torch.cat([ang.cos(), ang.sin()], 1)

    def step():
        qr = fa.kv_append_fp8(q, k, v, *cache, table, cu, lens, n, table=cs)
        return (qr, *fa.attention_paged_fp8(qr, *cache, table, cu, lens, n, bound, window, sinks))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr, o, lse = step()
    rng = np.random.default_rng(n)
    for i, top in enumerate((n, n + 1, 40 + n, 129 + n, 700, 2000, bound)):
        ls = [top, max(n, top // 3), int(rng.integers(n, max(n, top) + 1))]
        ns = [n, 0, max(1, n - 1)] if i % 2 else [n, n, n]
        at = [0] + [int(x) for x in np.cumsum(ns)]
        table.copy_(pages[torch.tensor([i % 3, (i + 1) % 3, (i + 2) % 3], device="cuda")])
        cu.copy_(i32(at))
        lens.copy_(i32(ls))
        o.fill_(9.0)
        lse.fill_(9.0)
        graph.replay()
        ok()
        rows = at[-1]
        check(o[:rows], lse[:, :rows], paged_oracle(qr[:rows], cache, table, ns, ls, window, sinks))
        assert torch.all(o[rows:] == 9.0) and torch.all(lse[:, rows:] == 9.0)


@pytest.mark.parametrize("n,d", [(1, 64), (2, 128), (6, 128), (50, 64), (40, 256)])
def test_sequences_that_share_pages(n, d):
    """Three sequences with the same first pages, and one named twice: the bits of the call on copies of them."""
    H, Hkv, page, lens = 8, 2, 16, [170, 300, 170, 64 + n]
    cache, table = cache_of(lens, page, Hkv, d, 9)
    shared = 64 // page
    for b in (1, 3):
        table[b, :shared] = table[0, :shared]
    table[2] = table[0]
    own = [torch.empty((sum(-(-x // page) for x in lens), *x.shape[1:]), dtype=x.dtype, device="cuda") for x in cache]
    apart, at = torch.full_like(table, -1), 0
    for b, length in enumerate(lens):
        used = -(-length // page)
        for x, y in zip(own, cache):
            x[at: at + used] = y[table[b, :used].long()]
        apart[b, :used] = torch.arange(at, at + used, device="cuda")
        at += used
    q = normal((4 * n, H, d), 2)
    batch = (i32([i * n for i in range(5)]), i32(lens), n, max(lens))
    for splits in (1, 3):
        x, y = (fa.attention_paged_fp8(q, *c, t, *batch, num_splits=splits) for c, t in ((cache, table), (own, apart)))
        ok()
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_scales_of_other_number_types():
    """A scale that float() takes gives the bits of the float."""
    q, k, v = normal((1, 4, 70, 64), 1), normal((1, 2, 90, 64), 2), normal((1, 2, 90, 64), 3)
    cache, table = cache_of([90], 16, 2, 64, 1)
    p = normal((3, 4, 64), 4)
    for scale in (np.float32(0.25), np.float64(0.25), torch.tensor(0.25)):
        for n in (20, np.int64(20)):
            for f in (lambda s, n: fa.attention_window(q, k, v, n, scale=s),
                      lambda s, n: fa.attention_paged_fp8(p, *cache, table, i32([0, 3]), i32([90]), 3, 90, n, scale=s)):
                x, y = f(scale, n), f(0.25, 20)
                ok()
                assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
