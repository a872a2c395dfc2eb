"""Rotary positions, the append to the paged e4m3 cache and attention over it,
against the float64 oracle (oracle/serving.py), at the sizes and masks where
they can go wrong.

Tolerances. A rounding to bf16 is off by at most 2^-8 of the value, to f16 by
2^-11.
 * Rotation: one bf16 rounding, and three fp32 roundings of terms no larger
   than |a| + |b|: 2^-8 |y| + 2^-22 (|a| + |b|).
 * Append: the interface fixes the fp32 operations, so codes and scales are
   equal.
 * Attention: the bf16 rounding of O, and on sum_j w_j |v_j| the f16 rounding
   of P (2^-11) and the scores' fp32 error (d products of size about one in
   fp32: below 2^-12 for these inputs): 2^-8 |o| + 2^-10 sum_j w_j |v_j|. LSE:
   the scores' error and a few fp32 roundings: 5e-4.
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
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def table_of(rows, rot):
    inv = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(rows)[:, None] * inv
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def check_rotated(y, x, ref, rot, interleaved, what=""):
    a, b = orc.pair_columns(rot, interleaved)
    size = np.zeros(x.shape)
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    assert np.all(np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * size), what
    assert np.array_equal(y[..., rot:], x[..., rot:]), what


# ----------------------------------------------------------------- rotation
ROPE = [
    # T, H, Hkv, d, rot, sections, interleaved
    (1, 1, 1, 64, 64, [32], False),
    (7, 5, 2, 64, 32, [16], True),
    (129, 8, 2, 128, 128, [64], False),
    (33, 3, 3, 128, 128, [16, 24, 24], False),
    (33, 3, 1, 128, 64, [5, 13, 14], True),      # sections that end inside a vector
    (50, 2, 2, 256, 256, [32, 96], False),
    (50, 2, 1, 256, 16, [1, 2, 0, 5], False),    # one axis with no pairs
    (1000, 4, 4, 64, 48, [24], False),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", range(len(ROPE)))
def test_rope_packed(case, inverse):
    T, H, Hkv, d, rot, sections, inter = ROPE[case]
    q, k = normal((T, H, d), 1 + case), normal((T, Hkv, d), 100 + case)
    table = table_of(2000, rot)
    pos = np.random.default_rng(case).integers(0, 2000, (len(sections), T)).astype(np.int32)
    qo, ko = fa.rope(q.cuda(), k.cuda(), torch.from_numpy(table).cuda(), torch.from_numpy(pos).cuda(),
                     sections=sections, interleaved=inter, inverse=inverse)
    ok()
    for x, y in ((q, qo), (k, ko)):
        ref = orc.rotate(f64(x), table, pos, sections, inter, inverse)
        check_rotated(f64(y), f64(x), ref, rot, inter)


@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (128, 96, True), (256, 128, False)])
def test_rope_dense_strided_in_place(d, rot, inter):
    """Head-major tensors, a fused projection's columns, and outputs in place of inputs agree."""
    B, H, Hkv, N = 2, 3, 1, 37
    q, k = normal((B, H, N, d), 5).cuda(), normal((B, Hkv, N, d), 6).cuda()
    table = torch.from_numpy(table_of(300, rot)).cuda()
    pos = torch.randint(0, 300, (B, N), dtype=torch.int32, device="cuda")
    qo, ko = fa.rope(q, k, table, pos, interleaved=inter)
    ok()
    flat = lambda t: t.transpose(1, 2).reshape(B * N, -1, d)  # noqa: E731
    fused = torch.cat([flat(q), flat(k)], 1).contiguous()
    qv, kv = fused[:, :H], fused[:, H:]
    qp, kp = fa.rope(qv, kv, table, pos.view(-1), interleaved=inter)
    assert torch.equal(qp, flat(qo)) and torch.equal(kp, flat(ko))
    fa.fa_rope(qv, kv, qv, kv, table, pos.view(-1), interleaved=inter)  # in place
    ok()
    assert torch.equal(qv, qp) and torch.equal(kv, kp)
    # token-major memory seen as [B, H, N, d]
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(fa.rope(qt, None, table, pos, interleaved=inter), qo)
    # one head shared by every batch entry (an expanded input)
    one = q[:1].expand(B, H, N, d)
    ref = fa.rope(one.contiguous(), None, table, pos, interleaved=inter)
    assert torch.equal(fa.rope(one, None, table, pos, interleaved=inter), ref)
    ok()


def test_rope_inverse_is_the_gradient():
    """<R x, g> = <x, R^-1 g> for each row, by the formula and by differences of the oracle."""
    T, H, d = 20, 2, 64
    table = table_of(50, d)
    pos = np.arange(T, dtype=np.int32)[None] * 2
    x, g = normal((T, H, d), 1), normal((T, H, d), 2)
    grad = f64(fa.rope(g.cuda(), None, torch.from_numpy(table).cuda(), torch.from_numpy(pos).cuda(), inverse=True))
    ok()
    step = normal((T, H, d), 3)
    f = lambda v: (orc.rotate(v, table, pos, [32]) * f64(g)).sum()  # noqa: E731
    diff = (f(f64(x) + 0.5 * f64(step)) - f(f64(x) - 0.5 * f64(step)))  # linear: exact for any step
    size = np.abs(orc.rotate(f64(g), table, pos, [32], inverse=True) * f64(step)).sum()
    assert abs(diff - (grad * f64(step)).sum()) <= 2.0 ** -8 * size + 1e-9


def test_rope_bad_position_reported_token_left():
    T, H, d = 5, 2, 64
    x = normal((T, H, d), 1).cuda()
    table = torch.from_numpy(table_of(10, d)).cuda()
    pos = torch.tensor([0, 10, 3, -1, 9], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 7.0)
    fa.fa_rope(x, None, out, None, table, pos)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == 15
    good = torch.tensor([0, 2, 4])
    assert torch.all(out[[1, 3]] == 7.0) and not torch.any(out[good] == 7.0)


# ------------------------------------------------------------ the paged cache
class Cache:
    """A cache with shuffled pages, its host copy and the batch's table."""

    def __init__(self, lens, page, Hkv, d, seed, fill=True, spare=3, amp=1.0):
        rng = np.random.default_rng(seed)
        self.page, self.Hkv, self.d = page, Hkv, d
        need = [-(-x // page) for x in lens]
        P = sum(need) + spare
        ids = rng.permutation(P)
        self.table = np.full((len(lens), max(max(need), 1) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at: at + n]
            at += n
        self.codes, self.scale = [], []
        for _ in range(2):
            if fill:
                x = rng.standard_normal((P, Hkv, page, d)) * amp * 2.0 ** rng.integers(-1, 2, (P, Hkv, 1, 1))
                s = np.array([[2.0 ** orc.block_exponent(np.abs(x[p, h]).max()) for h in range(Hkv)] for p in range(P)])
                self.codes.append(orc.encode_e4m3(x / s[:, :, None, None]))
            else:  # pages of earlier owners: any bytes (NaN codes among them), any scale
                self.codes.append(rng.integers(0, 256, (P, Hkv, page, d)).astype(np.uint8))
                s = 2.0 ** rng.integers(-20, 20, (P, Hkv)).astype(float)
            self.scale.append(s.astype(np.float32))

    def poison_tail(self, lens):
        """Slots behind each sequence's end hold NaN codes."""
        for b, n in enumerate(lens):
            if n % self.page:
                pg = self.table[b, n // self.page]
                for c in self.codes:
                    c[pg, :, n % self.page:] = 0x7F

    def gpu(self):
        return [torch.from_numpy(x.copy()).cuda() for x in (*self.codes, *self.scale)]


def cu_of(ns):
    return np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


APPEND = [
    # new tokens, cache lengths, page, H, Hkv, d, rot, sections, interleaved
    ([1], [1], 16, 4, 2, 64, 64, [32], False),
    ([1, 1, 1, 1], [17, 16, 5, 33], 16, 8, 2, 128, 128, [64], False),
    ([1, 0, 1], [64, 7, 200], 64, 2, 1, 256, 128, [64], True),
    ([3, 0, 5, 2], [3, 4, 20, 34], 16, 2, 2, 128, 64, [32], False),
    ([70, 1, 33], [100, 129, 33], 32, 3, 1, 64, 32, [4, 6, 6], True),
    ([300, 129], [300, 500], 128, 2, 2, 256, 256, [128], False),
    ([65, 128, 200], [70, 128, 263], 64, 4, 4, 128, 128, [16, 24, 24], False),
]


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case, strided):
    ns, lens, page, H, Hkv, d, rot, sections, inter = APPEND[case]
    T = sum(ns)
    cache = Cache(lens, page, Hkv, d, 40 + case, fill=(case % 2 == 0), amp=0.3)
    if case % 2:  # earlier tokens of the sequences are real values (no NaN codes)
        for c in cache.codes:
            c[np.isnan(orc.VALUES[c])] = 0x30
    # Tokens of very different sizes: a block's scale grows within and between appends.
    g = torch.Generator().manual_seed(case)
    grow = torch.exp2(torch.randint(-6, 7, (T, 1, 1), generator=g).float())
    fused = (torch.randn((T, H + 2 * Hkv, d), generator=g) * grow).to(torch.bfloat16)
    q, k, v = fused[:, :H], fused[:, H: H + Hkv], fused[:, H + Hkv:]
    table = table_of(1000, rot)
    pos = np.random.default_rng(case).integers(0, 1000, (len(sections), T)).astype(np.int32)
    cu = cu_of(ns)
    kc, vc, ks, vs = cache.gpu()
    f = fused.cuda()
    gq, gk, gv = f[:, :H], f[:, H: H + Hkv], f[:, H + Hkv:]
    if not strided:
        gq, gk, gv = gq.contiguous(), gk.contiguous(), gv.contiguous()
    qo = fa.kv_append_fp8(gq, gk, gv, kc, vc, ks, vs, dev(cache.table), dev(cu), dev(np.array(lens, np.int32)), max(ns),
                          table=dev(table), positions=dev(pos), sections=sections, interleaved=inter)
    ok()
    check_rotated(f64(qo), f64(q), orc.rotate(f64(q), table, pos, sections, inter), rot, inter)
    kr = orc.rotate(k.float().numpy(), table, pos, sections, inter, dtype=np.float32)
    orc.append(kr, cache.codes[0], cache.scale[0], cache.table, cu, lens, page)
    orc.append(v.float().numpy(), cache.codes[1], cache.scale[1], cache.table, cu, lens, page)
    for got, want in ((ks, cache.scale[0]), (vs, cache.scale[1]), (kc, cache.codes[0]), (vc, cache.codes[1])):
        got = got.cpu().numpy()
        if got.dtype == np.uint8:  # a zero's sign is not fixed
            got, want = np.where(got == 0x80, 0, got), np.where(want == 0x80, 0, want)
        assert np.array_equal(got, want)


def test_append_own_positions_no_rotation_no_queries():
    """positions None rotates by the cache positions; table None copies; q None is left out."""
    ns, lens, page, Hkv, d = [2, 40], [50, 41], 32, 2, 128
    T, cu = sum(ns), cu_of(ns)
    k, v, q = normal((T, Hkv, d), 1), normal((T, Hkv, d), 2), normal((T, 4, d), 3)
    table = table_of(64, d)
    own = np.concatenate([np.arange(l - n, l) for n, l in zip(ns, lens)]).astype(np.int32)[None]
    args = [dev(x) for x in (cu, np.array(lens, np.int32))]
    outs = []
    for kw in (dict(table=dev(table)), dict(table=dev(table), positions=dev(own)), dict()):
        cache = Cache(lens, page, Hkv, d, 9)
        kc, vc, ks, vs = cache.gpu()
        qo = fa.kv_append_fp8(q.cuda() if kw else None, k.cuda(), v.cuda(), kc, vc, ks, vs, dev(cache.table), *args, 40,
                              **kw)
        ok()
        x = orc.rotate(k.float().numpy(), table, own, [64], dtype=np.float32) if kw else k.float().numpy()
        orc.append(x, cache.codes[0], cache.scale[0], cache.table, cu, lens, page)
        got, want = kc.cpu().numpy(), cache.codes[0]
        assert np.array_equal(np.where(got == 0x80, 0, got), np.where(want == 0x80, 0, want))
        assert np.array_equal(ks.cpu().numpy(), cache.scale[0])
        outs.append((qo, kc, vc))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert outs[2][0] is None and torch.equal(outs[0][2], outs[2][2])


def test_append_extremes():
    """Zero blocks, the largest bf16 values, tiny ones and NaN: codes, scales, and the other tokens."""
    page, d = 16, 64
    lens, ns = [4], [4]
    cache = Cache(lens, page, 1, d, 3)
    big = float(torch.finfo(torch.bfloat16).max)
    for values, exponent in (([0.0] * 4, -100), ([big, -big, 1.0, 0.0], 120), ([1e-38, 2e-38, 0.0, 0.0], -100),
                             ([448.0, 1.0, 2.0, 3.0], 0), ([450.0, 1.0, 2.0, 3.0], 1)):
        x = torch.tensor(values).view(4, 1, 1).expand(4, 1, d).to(torch.bfloat16).contiguous()
        kc, vc, ks, vs = cache.gpu()
        fa.kv_append_fp8(None, x.cuda(), x.cuda(), kc, vc, ks, vs, dev(cache.table), dev(cu_of(ns)),
                         dev(np.array(lens, np.int32)), 4)
        ok()
        pg = cache.table[0, 0]
        assert ks[pg, 0].item() == 2.0 ** exponent == vs[pg, 0].item()
        want = orc.encode_e4m3(f64(x)[:, 0] / 2.0 ** exponent)
        assert np.array_equal(kc[pg, 0, :4].cpu().numpy() & 0x7F, want & 0x7F)
    x = torch.ones((4, 1, d), dtype=torch.bfloat16)
    x[1, 0, 3] = float("nan")
    kc, vc, ks, vs = cache.gpu()
    fa.kv_append_fp8(None, x.cuda(), x.cuda(), kc, vc, ks, vs, dev(cache.table), dev(cu_of(ns)),
                     dev(np.array(lens, np.int32)), 4)
    ok()
    got = orc.VALUES[kc[cache.table[0, 0], 0, :4].cpu().numpy()] * ks[cache.table[0, 0], 0].item()
    assert np.isnan(got[1, 3]) and np.isfinite(got).sum() == 4 * d - 1 and got[0, 0] == 1.0


def test_append_broken_batches_touch_nothing():
    page, Hkv, d = 16, 1, 64
    cache = Cache([40, 40], page, Hkv, d, 8)
    k = normal((6, Hkv, d), 1).cuda()
    t = table_of(64, d)
    cases = [
        (dict(cu=[0, 4, 2]), 12, [1]),                   # decreasing: the second is broken
        (dict(cu=[0, 3, 9]), 12, [1]),                   # past the tokens
        (dict(lens=[2, 40]), 12, [0]),                   # shorter than what it brings
        (dict(lens=[40, 4000]), 12, [1]),                # longer than its table
        (dict(table_at=(0, 2, 99)), 14, [0]),            # no such page
        (dict(table_at=(1, 2, -1)), 14, [1]),
        (dict(pos=[0, 0, 64, 0, 0, 0]), 15, [0]),        # outside the table
    ]
    for change, code, broken in cases:
        kc, vc, ks, vs = cache.gpu()
        before = [x.clone() for x in (kc, vc, ks, vs)]
        table = cache.table.copy()
        if "table_at" in change:
            b, i, x = change["table_at"]
            table[b, i] = x
        cu = np.array(change.get("cu", [0, 3, 6]), np.int32)
        lens = np.array(change.get("lens", [40, 40]), np.int32)
        pos = np.array(change.get("pos", [0] * 6), np.int32)
        fa.kv_append_fp8(None, k, k, kc, vc, ks, vs, dev(table), dev(cu), dev(lens), 4, table=dev(t),
                         positions=dev(pos))
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == code, change
        for b in broken:
            for pg in cache.table[b, :3]:
                assert torch.equal(kc[pg], before[0][pg]) and torch.equal(ks[pg], before[2][pg]), change


PAGED = [
    # new tokens, cache lengths, page, H, Hkv, d, window, sinks, splits
    ([1], [1], 16, 4, 4, 64, 0, 0, None),
    ([1, 1, 1], [31, 700, 16], 16, 8, 2, 128, 0, 0, None),
    ([1, 1, 1], [31, 700, 16], 16, 8, 2, 128, 0, 0, 5),
    ([1, 0, 1], [1000, 5, 3], 64, 16, 1, 256, 0, 0, 3),
    ([5, 3, 1], [300, 3, 129], 32, 8, 2, 64, 0, 0, None),
    ([5, 3, 1], [300, 30, 129], 128, 32, 2, 128, 40, 4, 2),
    ([1, 4], [900, 1000], 16, 6, 2, 128, 1, 0, None),
    ([1, 4], [900, 1000], 16, 6, 2, 64, 33, 100, 3),
    ([100, 70], [400, 70], 64, 4, 2, 128, 0, 0, None),
    ([130, 17], [130, 500], 16, 3, 1, 256, 64, 1, 2),
    ([200], [777], 128, 10, 2, 64, 300, 33, None),
    # many query rows: row tiles of 128, key tiles of 128
    ([300, 17, 64], [1000, 17, 500], 16, 8, 2, 128, 0, 0, 3),
    ([64, 200], [640, 200], 32, 8, 1, 64, 0, 0, 2),
    ([257, 130], [1500, 131], 64, 2, 2, 128, 0, 0, None),
    ([257, 1], [1500, 640], 64, 4, 2, 64, 130, 4, None),
    ([40, 300], [1300, 900], 16, 16, 2, 128, 200, 140, 2),
    ([513], [513], 128, 1, 1, 128, 1, 0, None),
    ([3, 3, 3], [1000, 128, 129], 128, 64, 1, 128, 0, 0, 8),
    ([20, 33], [2000, 4000], 32, 12, 4, 64, 0, 0, 16),
    ([1, 1], [2000, 300], 32, 64, 2, 128, 0, 0, None),
]


def check_paged(o, lse, ref, ref_lse, a, rows=None):
    o, lse = f64(o), f64(lse)
    err = np.abs(o - ref)
    lim = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * a
    assert np.all(err <= lim), f"worst {np.max(err - lim)} at {np.unravel_index(np.argmax(err - lim), err.shape)}"
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), empty)
    assert np.all(np.abs(lse[~empty] - ref_lse[~empty]) <= 5e-4)


@pytest.mark.parametrize("case", range(len(PAGED)))
def test_paged(case):
    ns, lens, page, H, Hkv, d, window, sinks, splits = PAGED[case]
    cache = Cache(lens, page, Hkv, d, 70 + case)
    cache.poison_tail(lens)
    q = normal((sum(ns), H, d), case)
    cu = cu_of(ns)
    kc, vc, ks, vs = cache.gpu()
    o, lse = fa.attention_paged_fp8(q.cuda(), kc, vc, ks, vs, dev(cache.table), dev(cu), dev(np.array(lens, np.int32)),
                                    max(ns), max(lens), window=window, sinks=sinks, num_splits=splits)
    ok()
    check_paged(o, lse, *orc.paged(f64(q), *cache.codes, *cache.scale, cache.table, cu, lens, fa.default_scale(d),
                                   window, sinks))


def test_paged_scales_far_apart():
    """Blocks whose scales lie 2^30 apart: each row's result follows the blocks its weights fall on."""
    page, d, H = 16, 64, 4
    lens, ns = [80], [2]
    cache = Cache(lens, page, 1, d, 5)
    for i, pg in enumerate(cache.table[0, :5]):
        cache.scale[1][pg] *= 2.0 ** (15 * (i - 2))
    q = normal((2, H, d), 3)
    kc, vc, ks, vs = cache.gpu()
    o, lse = fa.attention_paged_fp8(q.cuda(), kc, vc, ks, vs, dev(cache.table), dev(cu_of(ns)),
                                    dev(np.array(lens, np.int32)), 2, 80, num_splits=1)
    ok()
    check_paged(o, lse, *orc.paged(f64(q), *cache.codes, *cache.scale, cache.table, cu_of(ns), lens,
                                   fa.default_scale(d)))


def test_paged_other_scales():
    """Scales that are no powers of two (a cache another program filled)."""
    page, d, H = 32, 128, 8
    lens, ns = [100, 333], [1, 1]
    cache = Cache(lens, page, 2, d, 5)
    rng = np.random.default_rng(1)
    for i in range(2):
        cache.scale[i] = (cache.scale[i] * rng.uniform(0.6, 1.4, cache.scale[i].shape)).astype(np.float32)
    q = normal((2, H, d), 3)
    kc, vc, ks, vs = cache.gpu()
    o, lse = fa.attention_paged_fp8(q.cuda(), kc, vc, ks, vs, dev(cache.table), dev(cu_of(ns)),
                                    dev(np.array(lens, np.int32)), 1, 333)
    ok()
    check_paged(o, lse, *orc.paged(f64(q), *cache.codes, *cache.scale, cache.table, cu_of(ns), lens,
                                   fa.default_scale(d)))


def test_paged_large_and_small_queries():
    """Rows of very large, very small and zero queries keep their precision: each row is scaled for itself."""
    page, d, H = 16, 64, 16
    lens, ns = [64], [1]
    cache = Cache(lens, page, 1, d, 6)
    q = normal((1, H, d), 3)
    e = torch.tensor([0, 1, -3, -20, -100, -126, 0, 2] * 2).view(1, H, 1)
    q = (q.float() * torch.exp2(e.float())).to(torch.bfloat16)
    q[0, 6] = 0
    kc, vc, ks, vs = cache.gpu()
    o, lse = fa.attention_paged_fp8(q.cuda(), kc, vc, ks, vs, dev(cache.table), dev(cu_of(ns)),
                                    dev(np.array(lens, np.int32)), 1, 64)
    ok()
    check_paged(o, lse, *orc.paged(f64(q), *cache.codes, *cache.scale, cache.table, cu_of(ns), lens,
                                   fa.default_scale(d)))


def test_paged_broken_batches():
    page, Hkv, d, H = 16, 1, 64, 2
    cache = Cache([40, 40], page, Hkv, d, 8)
    q = normal((6, H, d), 1).cuda()
    kc, vc, ks, vs = cache.gpu()
    for change, code, broken in ((dict(cu=[0, 4, 2]), 12, slice(0, 0)), (dict(cu=[0, 3, 9]), 12, slice(3, 6)),
                                 (dict(lens=[2, 40]), 12, slice(0, 3)), (dict(lens=[40, 41]), 12, slice(3, 6)),
                                 (dict(cu=[0, 5, 6]), 12, slice(0, 5)), (dict(at=(0, 1, 77)), 14, slice(0, 0))):
        o = torch.full((6, H, d), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((H, 6), 2.0, device="cuda")
        table = cache.table.copy()
        if "at" in change:
            table[change["at"][:2]] = change["at"][2]
        fa.fa_fwd_paged_fp8(q, kc, vc, ks, vs, o, lse, dev(table), dev(np.array(change.get("cu", [0, 3, 6]), np.int32)),
                            dev(np.array(change.get("lens", [40, 40]), np.int32)), 4, 40)
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == code, change
        assert torch.all(o[broken] == 3.0) and torch.all(lse[:, broken] == 2.0), change


def test_rows_behind_the_last_sequence_are_left():
    page, Hkv, d, H = 16, 2, 64, 4
    cache = Cache([20, 50], page, Hkv, d, 8)
    q = normal((10, H, d), 1).cuda()
    k = normal((10, Hkv, d), 2).cuda()
    kc, vc, ks, vs = cache.gpu()
    cu, lens = dev(np.array([0, 2, 6], np.int32)), dev(np.array([20, 50], np.int32))
    q_out = torch.full_like(q, 5.0)
    fa.fa_kv_append_fp8(q, k, k, q_out, kc, vc, ks, vs, dev(cache.table), cu, lens, 4,
                        table=dev(table_of(64, d)))
    o = torch.full_like(q, 5.0)
    lse = torch.full((H, 10), 5.0, device="cuda")
    for splits in (1, 3):
        ws = torch.empty(max(1, fa.fa_paged_workspace_bytes(10, H, d, splits) // 4), device="cuda")
        fa.fa_fwd_paged_fp8(q, kc, vc, ks, vs, o, lse, dev(cache.table), cu, lens, 4, 50, ws, splits)
    ok()
    assert torch.all(q_out[6:] == 5.0) and torch.all(o[6:] == 5.0) and torch.all(lse[:, 6:] == 5.0)
    assert not torch.any(lse[:, :6] == 5.0)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 32)])
def test_prompt_then_tokens(d, page):
    """Used together: a prompt appended in two chunks, then tokens one at a time, each attended to;
    replayed from a captured graph it gives the same bits."""
    H, Hkv, B = 4, 2, 2
    steps = [[37, 20], [5, 90], [1, 1], [1, 1], [1, 0]]
    total = np.sum(steps, 0)
    cache = Cache([int(x) for x in total], page, Hkv, d, 4, fill=False)
    host = Cache([int(x) for x in total], page, Hkv, d, 4, fill=False)
    table = table_of(256, d)
    kc, vc, ks, vs = cache.gpu()
    start = [x.clone() for x in (kc, vc, ks, vs)]
    gt, gtab = dev(cache.table), dev(table)
    lens = np.zeros(B, np.int32)
    calls, wants = [], []
    for i, ns in enumerate(steps):
        lens = (lens + ns).astype(np.int32)
        cu = cu_of(ns)
        T = sum(ns)
        q, k, v = normal((T, H, d), 10 * i), normal((T, Hkv, d), 10 * i + 1), normal((T, Hkv, d), 10 * i + 2)
        calls.append([x.cuda() for x in (q, k, v)] + [dev(cu), dev(lens.copy()), max(ns), int(lens.max())])
        own = np.concatenate([np.arange(l - n, l) for n, l in zip(ns, lens)]).astype(np.int32)[None]
        orc.append(orc.rotate(k.float().numpy(), table, own, [d // 2], dtype=np.float32), host.codes[0], host.scale[0],
                   host.table, cu, lens, page)
        orc.append(v.float().numpy(), host.codes[1], host.scale[1], host.table, cu, lens, page)
        qr = torch.from_numpy(orc.rotate(q.float().numpy(), table, own, [d // 2], dtype=np.float32)).to(torch.bfloat16)
        wants.append(orc.paged(f64(qr), *host.codes, *host.scale, host.table, cu, lens, fa.default_scale(d)))

    def run():
        outs = []
        for q, k, v, cu, ln, mq, mk in calls:
            qr = fa.kv_append_fp8(q, k, v, kc, vc, ks, vs, gt, cu, ln, mq, table=gtab)
            outs.append(fa.attention_paged_fp8(qr, kc, vc, ks, vs, gt, cu, ln, mq, mk))
        return outs

    eager = run()
    ok()
    for (o, lse), want in zip(eager, wants):
        check_paged(o, lse, *want)
    for x, s in zip((kc, vc, ks, vs), start):
        x.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for _ in range(2):
        for x, s in zip((kc, vc, ks, vs), start):
            x.copy_(s)
        graph.replay()
        ok()
        for (o, lse), (eo, el) in zip(outs, eager):
            assert torch.equal(o, eo) and torch.equal(lse, el)


def test_other_stream_and_order():
    """Calls on a side stream, chained to work on the current one, give the same bits."""
    page, Hkv, d, H = 64, 2, 128, 8
    lens, ns = [500, 300], [1, 1]
    cache = Cache(lens, page, Hkv, d, 8)
    q = normal((2, H, d), 1).cuda()
    args = cache.gpu() + [dev(cache.table), dev(cu_of(ns)), dev(np.array(lens, np.int32))]
    want = fa.attention_paged_fp8(q, *args, 1, 500)
    side = torch.cuda.Stream()
    for _ in range(20):
        x = torch.zeros_like(q)
        x.copy_(q)
        side.wait_stream(torch.cuda.current_stream())
        o, lse = fa.attention_paged_fp8(x, *args, 1, 500, num_splits=4, stream=side)
        o1, lse1 = fa.attention_paged_fp8(x, *args, 1, 500, stream=side)
        x.record_stream(side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o1, want[0]) and torch.equal(lse1, want[1])
        assert (o.float() - want[0].float()).abs().max() <= 2.0 ** -7 * want[0].float().abs().max()
    ok()
