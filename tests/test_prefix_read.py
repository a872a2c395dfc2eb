"""Attention over the paged e4m3 cache for a batch that shares a prefix, and
reading the cache back, against the float64 oracle (oracle/serving.py).

Tolerances. Attention: those of the paged calls, whose kernels form both parts:
the bf16 rounding of O, and on sum_j w_j |v_j| the f16 rounding of P (2^-11) and
the scores' fp32 error: 2^-8 |o| + 2^-10 sum_j w_j |v_j|; LSE 5e-4. Reading back:
the product of a code and a power-of-two scale is exact in bf16, any other one
is rounded once, 2^-8 |x|.
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


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype)).cuda()


def cu_of(ns, first=0):
    return np.concatenate([[first], first + np.cumsum(ns)]).astype(np.int32)


class Cache:
    """A cache of real values with shuffled pages; `lens` tokens of each sequence, of which the first
    `shared` lie in the same pages. Slots behind a sequence's end hold NaN codes."""

    def __init__(self, lens, page, Hkv, d, seed, shared=0, spare=3):
        rng = np.random.default_rng(seed)
        self.page = page
        first = shared // page
        need = [max(0, -(-n // page) - first) for n in lens]
        P = first + sum(need) + spare
        ids = rng.permutation(P)
        self.table = np.full((len(lens), first + max(max(need), 1) + 1), -1, np.int32)
        at = first
        for b, n in enumerate(need):
            if lens[b] == 0:
                continue
            self.table[b, :first] = ids[:first]
            self.table[b, first: first + n] = ids[at: at + n]
            at += n
        self.codes, self.scale = [], []
        for _ in range(2):
            x = rng.standard_normal((P, Hkv, page, d)) * 2.0 ** rng.integers(-1, 2, (P, Hkv, 1, 1))
            s = np.array([[2.0 ** orc.block_exponent(np.abs(x[p, h]).max()) for h in range(Hkv)] for p in range(P)])
            self.codes.append(orc.encode_e4m3(x / s[:, :, None, None]))
            self.scale.append(s.astype(np.float32))
        for b, n in enumerate(lens):
            if n % page:
                for c in self.codes:
                    c[self.table[b, n // page], :, n % page:] = 0x7F

    def gpu(self):
        return [torch.from_numpy(x.copy()).cuda() for x in (*self.codes, *self.scale)]

    def want(self, q, cu, lens, d):
        return orc.paged(f64(q), *self.codes, *self.scale, self.table, cu, lens, fa.default_scale(d))


def check(o, lse, ref, ref_lse, a, rows=slice(None)):
    o, lse = f64(o)[rows], f64(lse)[:, rows]
    ref, ref_lse, a = ref[rows], ref_lse[:, rows], a[rows]
    over = np.abs(o - ref) - 2.0 ** -8 * np.abs(ref) - 2.0 ** -10 * a
    assert np.all(over <= 0), f"worst {over.max()} at {np.unravel_index(np.argmax(over), over.shape)}"
    assert np.all(np.abs(lse - ref_lse) <= 5e-4)


PREFIX = [
    # new tokens, tokens behind the prefix, prefix, page, H, Hkv, d, (own splits, prefix splits) or None
    ([1], [1], 16, 16, 4, 4, 64, None),
    ([1, 1, 1], [1, 40, 300], 128, 16, 8, 2, 128, None),
    ([1, 1, 1], [7, 40, 300], 1000 // 16 * 16, 16, 8, 2, 128, (3, 5)),
    ([1] * 40, [1 + 7 * b % 90 for b in range(40)], 512, 32, 8, 2, 64, None),
    ([1] * 33, [1 + 11 * b % 200 for b in range(33)], 640, 128, 14, 2, 128, (1, 1)),
    ([5, 3, 1, 8], [100, 3, 50, 8], 256, 64, 8, 2, 128, None),
    ([5] * 20, [60] * 20, 96, 32, 6, 2, 64, (2, 9)),
    ([40, 100, 1], [40, 130, 1], 448, 64, 4, 2, 128, None),       # chunks of prompts behind a shared one
    ([300, 17], [300, 500], 320, 64, 8, 2, 64, (2, 1)),
    ([1, 1], [30, 10], 208, 16, 16, 1, 256, None),
    ([1] * 20, [1 + b for b in range(20)], 384, 128, 16, 2, 256, (2, 3)),
    ([6, 30], [20, 30], 160, 32, 4, 2, 256, None),
    ([1, 0, 1, 0], [9, 5, 3, 0], 64, 16, 4, 2, 128, None),        # sequences that bring nothing
    ([0, 1, 2], [0, 77, 2], 48, 16, 3, 1, 128, (4, 2)),           # the first one brings nothing and holds nothing
    ([2] * 100, [2 + b % 50 for b in range(100)], 144, 16, 2, 1, 64, None),
    ([1, 1, 1], [7, 400, 1300], 960, 16, 8, 2, 128, (20, 25)),    # more than 32 states, and than 128
    ([1] * 12, [1 + 60 * b for b in range(12)], 2048, 64, 8, 2, 64, (40, 3)),
    ([3] * 20, [90] * 20, 1536, 32, 8, 2, 128, (3, 120)),
    ([1] * 24, [1 + 9 * b for b in range(24)], 1024, 64, 16, 2, 256, (2, 60)),
    # prefixes long enough for the tensor-core kernel: pairs of slots, whole tiles, beside few sequences and many
    ([1] * 16, [1 + 20 * b for b in range(16)], 8192, 64, 16, 4, 128, None),
    ([1] * 16, [1 + 20 * b for b in range(16)], 10240, 128, 16, 4, 64, None),
    ([1] * 24, [1 + 13 * b for b in range(24)], 6144, 64, 16, 2, 128, None),
    ([2] * 12, [2 + 13 * b for b in range(12)], 8192, 32, 16, 2, 64, None),
    ([1] * 24, [1 + 13 * b for b in range(24)], 2048, 64, 16, 2, 256, (3, 7)),
    ([int(b % 4 > 0) for b in range(120)], [1 + 29 * b % 300 for b in range(120)], 2560, 64, 8, 4, 128, None),
    ([1] * 80, [1 + 13 * b % 120 for b in range(80)], 1536, 32, 8, 4, 256, None),
    # so many sequences that each warp has a share of one for itself
    ([1] * 160, [1 + 37 * b % 150 for b in range(160)], 64, 16, 8, 4, 64, None),
    ([1] * 160, [1 + b % 3 if b != 97 else 2500 for b in range(160)], 128, 64, 4, 4, 64, None),   # one far longer
    ([1 + b % 2 for b in range(120)], [2 + 29 * b % 300 for b in range(120)], 48, 16, 8, 4, 128, None),
    ([1] * 115, [1 + 29 * b % 300 for b in range(115)], 256, 128, 28, 4, 128, (1, 1)),
    ([int(b % 5 > 0) for b in range(120)], [int(b % 5 > 0) + b % 7 for b in range(120)], 32, 16, 4, 4, 128, (3, 2)),  # some idle
    ([1] * 77, [1 + 13 * b % 120 for b in range(77)], 96, 32, 8, 4, 256, None),
    ([int(b > 70) for b in range(80)], [9 if b > 70 else 0 for b in range(80)], 16, 16, 4, 4, 256, (4, 1)),
]


@pytest.mark.parametrize("case", range(len(PREFIX)))
def test_prefix(case):
    ns, own, prefix, page, H, Hkv, d, splits = PREFIX[case]
    lens = [prefix + x if x else 0 for x in own]
    cache = Cache(lens, page, Hkv, d, 70 + case, shared=prefix)
    q, cu = normal((sum(ns), H, d), case), cu_of(ns)
    kw = {} if splits is None else dict(num_splits=splits[0], prefix_splits=splits[1])
    args = [*cache.gpu(), dev(cache.table), dev(cu), dev(lens)]
    o, lse = fa.attention_prefix_fp8(q.cuda(), *args, max(ns), max(lens), prefix, **kw)
    ok()
    want = cache.want(q, cu, lens, d)
    check(o, lse, *want)
    op, lp = fa.attention_paged_fp8(q.cuda(), *args, max(ns), max(lens)) if all(ns) else (o, lse)
    ok()
    check(op, lp, *want)


@pytest.mark.parametrize("prefix", [128, 20480])
def test_prefix_query_rows_that_are_not_finite(prefix):
    """A row with a NaN or an infinity gives NaN, the others keep their results; rows of no sequence may hold anything."""
    page, H, Hkv, d, ns, own = 16, 4, 2, 128, [1] * 24, [1 + b for b in range(24)]
    lens = [prefix + x for x in own]
    cache = Cache(lens, page, Hkv, d, 4, shared=prefix)
    q, cu = normal((30, H, d), 3).cuda(), cu_of(ns)
    args = [*cache.gpu(), dev(cache.table), dev(cu), dev(lens), 1, max(lens), prefix]
    o, lse = fa.attention_prefix_fp8(q, *args)
    q2 = q.clone()
    q2[3, 1, 5], q2[11, 0, 0], q2[24:] = float("nan"), float("inf"), float("nan")
    o2, l2 = fa.attention_prefix_fp8(q2, *args)
    ok()
    bad = torch.zeros((30, H), dtype=torch.bool)
    bad[3, 1] = bad[11, 0] = True
    bad[24:] = True
    good = ~bad
    good[24:] = False
    assert torch.equal(o2[good.cuda()], o[good.cuda()]) and torch.equal(l2.t()[good.cuda()], lse.t()[good.cuda()])
    for i, h in ((3, 1), (11, 0)):
        assert torch.all(torch.isnan(o2[i, h])) and torch.isnan(l2[h, i])


def test_prefix_broken_batches():
    """A sequence that does not hold the prefix, or is too long, is reported and not written; the others keep their
    results. Another page in the prefix, or no page of the cache, is reported."""
    prefix, page, H, Hkv, d = 64, 16, 2, 1, 64
    lens, ns = [prefix + 20, prefix + 30, prefix + 5], [2, 2, 2]
    cache = Cache(lens, page, Hkv, d, 8, shared=prefix)
    q, cu = normal((6, H, d), 1).cuda(), cu_of(ns)
    g = cache.gpu()
    most = cache.table.shape[1] * page
    want = fa.attention_prefix_fp8(q, *g, dev(cache.table), dev(cu), dev(lens), 2, most, prefix)
    ok()
    ws = torch.empty(fa.fa_paged_workspace_bytes(6, H, d, 3) // 4, device="cuda")
    for change, code, broken in ((dict(lens=[lens[0], prefix + 1, lens[2]]), 12, [1]), (dict(lens=[lens[0], 30, lens[2]]), 12, [1]),
                                 (dict(lens=[lens[0], lens[1], most + 1]), 12, [2]), (dict(cu=[0, 2, 4, 7]), 12, [2]),
                                 (dict(cu=[0, 2, -4, 6]), 12, [1, 2]), (dict(cu=[0, 3, 4, 6]), 12, [0]),
                                 (dict(at=(1, 1, 0)), 14, None), (dict(at=(2, 4, 99)), 14, None), (dict(at=(0, 0, -7)), 14, None)):
        table = cache.table.copy()
        if "at" in change:
            b, i, x = change["at"]
            table[b, i] = x if x or table[b, i] else 1
        o = torch.full((6, H, d), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((H, 6), 2.0, device="cuda")
        fa.fa_fwd_prefix_fp8(q, *g, o, lse, dev(table), dev(change.get("cu", cu)), dev(change.get("lens", lens)), 2, most,
                             prefix, ws, 1, 2)
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == code, change
        if broken is None:
            continue
        for b in range(3):
            s = slice(2 * b, 2 * b + 2)
            if b in broken:
                if "cu" not in change:
                    assert torch.all(o[s] == 3.0) and torch.all(lse[:, s] == 2.0), change
            elif "cu" not in change:
                assert (o[s].float() - want[0][s].float()).abs().max() <= 2.0 ** -6 * want[0].float().abs().max()


@pytest.mark.parametrize("prefix", [64, 4096])
def test_prefix_broken_batches_of_many(prefix):
    """As above, where each warp has a share of a sequence for itself."""
    page, H, Hkv, d, B = 16, 4, 4, 128, 130
    lens, ns = [prefix + 1 + 11 * b % 90 for b in range(B)], [1] * B
    cache = Cache(lens, page, Hkv, d, 8, shared=prefix)
    q, cu = normal((B, H, d), 1).cuda(), cu_of(ns)
    g = cache.gpu()
    most = cache.table.shape[1] * page
    want = fa.attention_prefix_fp8(q, *g, dev(cache.table), dev(cu), dev(lens), 1, most, prefix)
    ok()
    own, shared = fa.fa_prefix_num_splits(B, H, Hkv, B, 1, most, prefix, d)
    ws = torch.empty(fa.fa_paged_workspace_bytes(B, H, d, own + shared) // 4, device="cuda")
    for length, at, code, broken in ((prefix, None, 12, [77]), (3, None, 12, [77]), (most + 1, None, 12, [77]),
                                     (None, (77, 1, 0), 14, None), (None, (77, prefix // page, 99999), 14, None),
                                     (None, (0, 0, -7), 14, None)):
        table, n = cache.table.copy(), list(lens)
        if at:
            table[at[:2]] = at[2] if at[2] or table[at[:2]] else 1
        else:
            n[77] = length
        o, lse = torch.full_like(q, 3.0), torch.full((H, B), 2.0, device="cuda")
        fa.fa_fwd_prefix_fp8(q, *g, o, lse, dev(table), dev(cu), dev(n), 1, most, prefix, ws, own, shared)
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == code, (length, at)
        if broken:
            assert torch.all(o[77] == 3.0) and torch.all(lse[:, 77] == 2.0)
            keep = [b for b in range(B) if b != 77]
            assert (o[keep].float() - want[0][keep].float()).abs().max() <= 2.0 ** -6 * want[0].float().abs().max()


@pytest.mark.parametrize("prefix,page,H,Hkv,d,B", [(64, 16, 2, 1, 64, 3), (4096, 64, 8, 4, 128, 130), (1536, 32, 8, 4, 256, 24),
                                                   (8192, 64, 16, 4, 128, 16), (64, 16, 4, 4, 128, 130)])
def test_prefix_first_sequence_broken(prefix, page, H, Hkv, d, B):
    """The first sequences are rejected, for their lengths or their offsets, and their rows of the table name no page: they
    are not written, and the others keep their results."""
    lens, ns = [prefix + 3 + 11 * b % 90 for b in range(B)], [1] * B
    cache = Cache(lens, page, Hkv, d, 8, shared=prefix)
    most = cache.table.shape[1] * page
    q, cu = normal((B, H, d), 1), cu_of(ns)
    want = cache.want(q, cu, lens, d)
    args = [q.cuda(), *cache.gpu()]
    splits = fa.fa_prefix_num_splits(B, H, Hkv, B, 1, most, prefix, d)
    ws = torch.empty(fa.fa_paged_workspace_bytes(B, H, d, sum(splits)) // 4, device="cuda")
    for count, length, first in ((1, prefix, 0), (2, 1, 0), (1, most + 1, 0), (1, None, -1)):
        table, n, c = cache.table.copy(), list(lens), cu.copy()
        table[:count] = -1
        c[0] = first
        if length:
            n[:count] = [length] * count
        o, lse = torch.full((B, H, d), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((H, B), 2.0, device="cuda")
        fa.fa_fwd_prefix_fp8(*args, o, lse, dev(table), dev(c), dev(n), 1, most, prefix, ws, *splits)
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_SEQLENS, (count, length)
        assert torch.all(o[:count] == 3.0) and torch.all(lse[:, :count] == 2.0)
        check(o, lse, *want, rows=slice(count, None))


@pytest.mark.parametrize("B", [1024, 1025, 3000])
@pytest.mark.parametrize("prefix", [64, 8192])
def test_prefix_of_thousands_of_sequences(B, prefix):
    """On either side of the number up to which each warp looks through all sequences: the paged call's results, a
    sequence that brings nothing and a rejected one left as they were."""
    page, H, Hkv, d = 16, 4, 2, 64
    ns, lens = [1] * B, [prefix + 1 + 7 * b % 60 for b in range(B)]
    ns[300], ns[999] = 0, 2
    cache = Cache(lens, page, Hkv, d, 3, shared=prefix)
    q, cu = normal((sum(ns), H, d), 1), cu_of(ns)
    lens[700] = prefix
    args = [q.cuda(), *cache.gpu()]
    batch = [dev(cache.table), dev(cu), dev(lens)]
    most = cache.table.shape[1] * page
    splits = fa.fa_prefix_num_splits(B, H, Hkv, sum(ns), 2, most, prefix, d)
    ws = torch.empty(fa.fa_paged_workspace_bytes(sum(ns), H, d, sum(splits)) // 4, device="cuda")
    o, lse = torch.full_like(args[0], 3.0), torch.full((H, sum(ns)), 2.0, device="cuda")
    fa.fa_fwd_prefix_fp8(*args, o, lse, *batch, 2, most, prefix, ws, *splits)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_SEQLENS
    out = int(cu[700])
    assert torch.all(o[out] == 3.0) and torch.all(lse[:, out] == 2.0)
    op, lp = fa.attention_paged_fp8(*args, *batch, 2, most)
    ok()
    some = [int(cu[b]) for b in (0, 1, 299, 301, 699, 701, 998, 999, 1000, B - 1)] + [int(cu[999]) + 1]
    seqs = [next(b for b in range(B) if cu[b] <= i < cu[b + 1]) for i in some]
    small = type(cache).__new__(type(cache))
    small.codes, small.scale, small.table = cache.codes, cache.scale, cache.table[seqs]
    n = [lens[b] - (b == 999 and i == cu[999]) for b, i in zip(seqs, some)]
    want = small.want(q[some], cu_of([1] * len(some)), n, d)
    check(o[some], lse[:, some], *want)
    keep = [i for i in range(sum(ns)) if i != out]
    # (Each is off by 2^-8 |o| + 2^-10 a at most, and a, as |o|, is no larger than the largest |v|.)
    largest = np.nanmax(np.abs(orc.VALUES[cache.codes[1]]) * cache.scale[1][:, :, None, None])
    gap = (o[keep].float() - op[keep].float()).abs() - 2.0 ** -7 * op[keep].float().abs()
    assert gap.max() <= (2.0 ** -9 + 2.0 ** -13) * largest


@pytest.mark.parametrize("prefix,page,H,Hkv,d,B,n", [(8192, 64, 16, 4, 128, 16, 1), (4096, 64, 32, 8, 128, 64, 1), (6144, 32, 32, 8, 128, 12, 5),
                                                     (4096, 128, 16, 2, 256, 31, 1), (10240, 128, 16, 4, 64, 16, 1)])
def test_prefix_reads_what_was_just_written(prefix, page, H, Hkv, d, B, n):
    """Calls whose two launches run side by side, each right behind the copies that exchange everything they read: the
    bits of calls on tensors that lie still."""
    lens = [prefix + n + 37 * b % 500 for b in range(B)]
    states = []
    for seed, x in ((1, lens), (2, lens[::-1])):
        cache = Cache(x, page, Hkv, d, seed, shared=prefix)
        states.append([normal((B * n, H, d), seed).cuda(), *cache.gpu(), dev(cache.table), dev(x)])
    cu = dev(cu_of([n] * B))
    call = lambda *x: fa.attention_prefix_fp8(*x[:6], cu, x[6], n, max(lens), prefix)  # noqa: E731
    want = []
    for x in states:
        want.append(call(*x))
        ok()
    one = [torch.empty_like(t) for t in states[0]]
    got = []
    for i in range(40):
        for to, t in zip(one, states[i % 2]):
            to.copy_(t)
        got.append(call(*one))
    ok()
    for i, x in enumerate(got):
        assert torch.equal(x[0], want[i % 2][0]) and torch.equal(x[1], want[i % 2][1]), i


def test_prefix_rows_behind_the_last_sequence_are_left():
    prefix, page, H, Hkv, d = 32, 16, 4, 2, 64
    lens, ns = [prefix + 20, prefix + 50], [2, 4]
    cache = Cache(lens, page, Hkv, d, 8, shared=prefix)
    q = normal((10, H, d), 1).cuda()
    g = [*cache.gpu()]
    for splits in ((1, 1), (3, 2)):
        o, lse = torch.full_like(q, 5.0), torch.full((H, 10), 5.0, device="cuda")
        ws = torch.empty(fa.fa_paged_workspace_bytes(10, H, d, sum(splits)) // 4, device="cuda")
        fa.fa_fwd_prefix_fp8(q, *g, o, lse, dev(cache.table), dev(cu_of(ns)), dev(lens), 4, max(lens), prefix, ws, *splits)
        ok()
        assert torch.all(o[6:] == 5.0) and torch.all(lse[:, 6:] == 5.0) and not torch.any(lse[:, :6] == 5.0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefix_workspace_of_sixteen_byte_alignment(d):
    """The workspace at a multiple of 16 bytes that is none of 32: the same bits."""
    prefix, page, H, Hkv = 640, 32, 8, 1
    lens, ns = [prefix + 40 * b + 3 for b in range(12)], [3] * 12
    cache = Cache(lens, page, Hkv, d, 8, shared=prefix)
    q, out = normal((36, H, d), 1).cuda(), []
    args = [*cache.gpu()]
    for skip in (0, 4):
        o, lse = torch.empty_like(q), torch.empty((H, 36), device="cuda")
        ws = torch.empty(fa.fa_paged_workspace_bytes(36, H, d, 5) // 4 + 4, device="cuda")[skip:]
        assert ws.data_ptr() % 32 == 4 * skip
        fa.fa_fwd_prefix_fp8(q, *args, o, lse, dev(cache.table), dev(cu_of(ns)), dev(lens), 3, max(lens), prefix, ws, 2, 3)
        ok()
        out.append((o, lse))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_prefix_captured_replayed_and_on_a_side_stream():
    prefix, page, H, Hkv, d = 256, 32, 8, 2, 128
    ns, lens = [1] * 8, [prefix + 1 + 30 * b for b in range(8)]
    cache = Cache([prefix + 300] * 8, page, Hkv, d, 5, shared=prefix)
    q = normal((8, H, d), 2).cuda()
    args = [*cache.gpu(), dev(cache.table), dev(cu_of(ns))]
    gl = dev(lens)
    eager = []
    for extra in (0, 7):
        gl.copy_(dev([n + extra for n in lens]))
        eager.append(fa.attention_prefix_fp8(q, *args, gl, 1, prefix + 300, prefix))
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.attention_prefix_fp8(q, *args, gl, 1, prefix + 300, prefix)
    for extra, want in ((0, eager[0]), (7, eager[1]), (0, eager[0])):
        gl.copy_(dev([n + extra for n in lens]))
        o.fill_(9.0)
        graph.replay()
        ok()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    side = torch.cuda.Stream()
    for _ in range(10):
        x = torch.zeros_like(q)
        x.copy_(q)
        side.wait_stream(torch.cuda.current_stream())
        so, sl = fa.attention_prefix_fp8(x, *args, gl, 1, prefix + 300, prefix, stream=side)
        x.record_stream(side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(so, eager[0][0]) and torch.equal(sl, eager[0][1])
    ok()


# ------------------------------------------------------------------ reading back
READ = [
    # tokens read, first token, page, Hkv, d
    ([1], [0], 16, 1, 64),
    ([5, 0, 40], [3, 9, 0], 16, 2, 128),
    ([130, 77], [60, 1], 64, 8, 128),
    ([33, 300, 1], [0, 17, 255], 32, 3, 256),
    ([500], [0], 128, 5, 64),
    ([1 + b % 9 for b in range(300)], [b % 5 for b in range(300)], 16, 2, 64),  # more sequences than threads of a block
]


@pytest.mark.parametrize("case", range(len(READ)))
def test_read(case):
    ns, starts, page, Hkv, d = READ[case]
    lens = [a + b for a, b in zip(ns, starts)]
    cache = Cache(lens, page, Hkv, d, case)
    g = cache.gpu()
    k, v = fa.kv_read_fp8(*g, dev(cache.table), dev(cu_of(ns)), dev(starts), sum(ns))
    ok()
    for x, c, s in zip((k, v), cache.codes, cache.scale):
        assert np.array_equal(f64(x), orc.read(c, s, cache.table, starts, ns, page))
    if not any(starts):
        k0, v0 = fa.kv_read_fp8(*g, dev(cache.table), dev(cu_of(ns)), total=sum(ns))
        ok()
        assert torch.equal(k, k0) and torch.equal(v, v0)


def test_read_every_code_and_other_scales():
    """All 256 codes, NaN among them, under scales from the least to the largest and ones that are no powers of two."""
    page, d = 16, 64
    for scale in (1.0, 2.0 ** -100, 2.0 ** 111, 0.0, 0.7312, 3.3e-5):
        codes = np.arange(page * d).reshape(1, 1, page, d).astype(np.uint8)
        s = np.full((1, 1), scale, np.float32)
        args = [torch.from_numpy(x).cuda() for x in (codes, codes, s, s)]
        k, v = fa.kv_read_fp8(*args, dev([[0]]), dev([0, page]), None, page)
        ok()
        with np.errstate(invalid="ignore"):
            want = orc.VALUES[codes[0, 0]] * np.float64(np.float32(scale))
        got = f64(k)[:, 0]
        assert np.array_equal(np.isnan(got), np.isnan(want)) and torch.equal(k.isnan(), v.isnan())
        there = ~np.isnan(want)
        assert np.all(np.abs(got - want)[there] <= (0 if np.log2(scale or 1.0) % 1 == 0 else 2.0 ** -8) * np.abs(want)[there])


def test_read_strided_and_rows_of_no_sequence():
    """Into columns of a wider tensor; rows outside all sequences are left, or zeros where asked for."""
    ns, starts, page, Hkv, d = [20, 50], [5, 0], 16, 2, 128
    cache = Cache([25, 50], page, Hkv, d, 3)
    g, table, cu = cache.gpu(), dev(cache.table), dev(cu_of(ns, 4))
    k, v = fa.kv_read_fp8(*g, table, cu, dev(starts), 90)
    ok()
    want = [orc.read(c, s, cache.table, starts, ns, page) for c, s in zip(cache.codes, cache.scale)]
    for x, w in zip((k, v), want):
        assert np.array_equal(f64(x)[4:74], w) and torch.all(x[:4] == 0) and torch.all(x[74:] == 0)
    wide = torch.full((90, 9, d), 3.0, dtype=torch.bfloat16, device="cuda")
    fa.fa_kv_read_fp8(*g, wide[:, 1:3], wide[:, 5:7], table, cu, dev(starts))
    ok()
    assert torch.equal(wide[4:74, 1:3], k[4:74]) and torch.equal(wide[4:74, 5:7], v[4:74])
    for rows, heads in ((slice(0, 4), slice(None)), (slice(74, 90), slice(None)), (slice(None), [0, 3, 4, 7, 8])):
        assert torch.all(wide[rows, heads] == 3.0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_read_into_rows_of_sixteen_byte_alignment(d):
    """Outputs at a multiple of 16 bytes that is none of 32, and tokens an odd number of 16 bytes apart."""
    ns, starts, page, Hkv = [20, 50], [5, 0], 16, 3
    cache = Cache([25, 50], page, Hkv, d, 3)
    g, args = cache.gpu(), (dev(cache.table), dev(cu_of(ns)), dev(starts))
    k, v = fa.kv_read_fp8(*g, *args, 70)
    for skip, gap in ((8, 0), (0, 8), (8, 24)):
        out = []
        for _ in range(2):
            x = torch.zeros(70 * (Hkv * d + gap) + 8, dtype=torch.bfloat16, device="cuda")[skip:]
            out.append(x.as_strided((70, Hkv, d), (Hkv * d + gap, d, 1)))
        assert out[0].data_ptr() % 32 == 2 * skip
        fa.fa_kv_read_fp8(*g, *out, *args)
        ok()
        assert torch.equal(out[0], k) and torch.equal(out[1], v)


def test_read_broken_batches_touch_nothing():
    ns, page, Hkv, d = [20, 30, 10], 16, 1, 64
    cache = Cache([25, 30, 10], page, Hkv, d, 8)
    g, cu, starts = cache.gpu(), cu_of(ns), [5, 0, 0]
    k, v = fa.kv_read_fp8(*g, dev(cache.table), dev(cu), dev(starts), 60)
    ok()
    width = cache.table.shape[1] * page
    for change, code, broken in ((dict(cu=[0, 20, 15, 60]), 12, [1]), (dict(cu=[0, 20, 50, 61]), 12, [2]),
                                 (dict(starts=[-1, 0, 0]), 12, [0]), (dict(starts=[5, width - 29, 0]), 12, [1]),
                                 (dict(cu=[-3, 20, 50, 60]), 12, [0]), (dict(at=(2, 0, 99)), 14, [2]),
                                 (dict(at=(2, 0, -1)), 14, [2])):
        table = cache.table.copy()
        if "at" in change:
            table[change["at"][:2]] = change["at"][2]
        x = [torch.full_like(k, 3.0) for _ in range(2)]
        fa.fa_kv_read_fp8(*g, *x, dev(table), dev(change.get("cu", cu)), dev(change.get("starts", starts)), fill=True)
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == code, change
        for b in range(3):
            s = slice(cu[b], cu[b + 1])
            if b not in broken and not (change.get("cu") and b == 2):  # (a later start may overlap)
                assert torch.equal(x[0][s], k[s]) and torch.equal(x[1][s], v[s]), change
            elif b in broken and not (change.get("cu") and b != 2 and change["cu"][0] == 0):
                assert torch.all(x[0][s] == 3.0) and torch.all(x[1][s] == 3.0), change


def test_read_captured_replayed_and_on_a_side_stream():
    ns, page, Hkv, d = [20, 50], 16, 2, 128
    cache = Cache([40, 60], page, Hkv, d, 3)
    g, table, cu = cache.gpu(), dev(cache.table), dev(cu_of(ns))
    starts = dev([0, 0])
    eager = []
    for first in ([0, 10], [20, 3]):
        starts.copy_(dev(first))
        eager.append(fa.kv_read_fp8(*g, table, cu, starts, 70))
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k, v = fa.kv_read_fp8(*g, table, cu, starts, 70)
    for i in (0, 1, 0):
        starts.copy_(dev(([0, 10], [20, 3])[i]))
        k.fill_(9.0)
        graph.replay()
        ok()
        assert torch.equal(k, eager[i][0]) and torch.equal(v, eager[i][1])
    side = torch.cuda.Stream()
    for _ in range(10):
        x = [t.clone() for t in g]
        side.wait_stream(torch.cuda.current_stream())
        ks, vs = fa.kv_read_fp8(*x, table, cu, starts, 70, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(ks, eager[0][0]) and torch.equal(vs, eager[0][1])
    ok()


def test_two_graphs_of_prefix_calls_keep_their_workspaces():
    """Two captured calls, replayed in turn and on two streams at once, each with its own partials."""
    prefix, page, H, Hkv, d, B = 256, 32, 8, 2, 128, 12
    calls = []
    for i in range(2):
        lens = [prefix + 1 + (30 + 7 * i) * b for b in range(B)]
        cache = Cache(lens, page, Hkv, d, 5 + i, shared=prefix)
        q = normal((B, H, d), 2 + i).cuda()
        args = [q, *cache.gpu(), dev(cache.table), dev(cu_of([1] * B)), dev(lens), 1, max(lens), prefix, None, 4, 4]
        calls.append((args, *fa.attention_prefix_fp8(*args[:11], num_splits=4, prefix_splits=4)))
    ok()
    graphs = []
    for args, _, _ in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fa.attention_prefix_fp8(*args[:11], num_splits=4, prefix_splits=4)
        graphs.append((graph, out))
    sides = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for (graph, out), s in zip(graphs, sides):
            out[0].fill_(9.0)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                graph.replay()
        for s in sides:
            torch.cuda.current_stream().wait_stream(s)
        for (_, out), (_, o, lse) in zip(graphs, calls):
            assert torch.equal(out[0], o) and torch.equal(out[1], lse)
    ok()


def test_read_and_prefix_behind_four_gigabytes():
    """Pages, rows and strides whose offsets do not fit 32 bits: the bits of small ones."""
    page, Hkv, d, H, B, prefix = 128, 8, 256, 16, 3, 256
    P = 2 ** 31 // (Hkv * page * d) + 9 if torch.cuda.mem_get_info()[0] > 40e9 else 0
    if not P:
        pytest.skip("needs 40 GB of device memory")
    lens = [prefix + 70, prefix + 300, prefix + 1]
    cache = Cache(lens, page, Hkv, d, 5, shared=prefix, spare=0)
    small, n = cache.gpu(), cache.codes[0].shape[0]
    big = [torch.empty((P, *x.shape[1:]), dtype=x.dtype, device="cuda") for x in small]
    for x, y in zip(big, small):
        x[P - n:] = y
    far = np.where(cache.table >= 0, cache.table + P - n, -1)
    q, one = normal((B, H, d), 1).cuda(), cu_of([1] * B)
    out = []
    for g, table in ((small, cache.table), (big, far)):
        o, lse = fa.attention_prefix_fp8(q, *g, dev(table), dev(one), dev(lens), 1, max(lens), prefix)
        k, v = fa.kv_read_fp8(*g, dev(table), dev(cu_of(lens)), None, sum(lens))
        ok()
        out.append((o, lse, k, v))
    for x, y in zip(*out):
        assert torch.equal(x, y)
    wide = torch.empty((sum(lens), 2 ** 22), dtype=torch.bfloat16, device="cuda")
    k, v = (wide[:, at: at + Hkv * d].unflatten(1, (Hkv, d)) for at in (0, 2 ** 21))
    assert k.stride(0) * (k.shape[0] - 1) > 2 ** 31
    fa.fa_kv_read_fp8(*small, k, v, dev(cache.table), dev(cu_of(lens)))
    ok()
    assert torch.equal(k, out[0][2]) and torch.equal(v, out[0][3])


def test_pages_named_twice():
    """Sequences that hold the same pages, and a page that a sequence holds twice."""
    page, Hkv, d, H, prefix = 16, 2, 64, 4, 32
    cache = Cache([prefix + 50], page, Hkv, d, 5, shared=prefix)
    row = cache.table[0].copy()
    row[3] = row[2]
    cache.table = np.stack([row, cache.table[0], row])
    lens = [prefix + 45, prefix + 50, prefix + 33]
    g, table = cache.gpu(), dev(cache.table)
    q, cu = normal((3, H, d), 1), cu_of([1] * 3)
    o, lse = fa.attention_prefix_fp8(q.cuda(), *g, table, dev(cu), dev(lens), 1, max(lens), prefix)
    k, v = fa.kv_read_fp8(*g, table, dev(cu_of(lens)), None, sum(lens))
    ok()
    check(o, lse, *cache.want(q, cu, lens, d))
    for x, c, s in zip((k, v), cache.codes, cache.scale):
        assert np.array_equal(f64(x), orc.read(c, s, cache.table, [0] * 3, lens, page))


@pytest.mark.parametrize("d,H,Hkv,B,n", [(128, 32, 8, 60, 1), (128, 32, 8, 12, 5), (256, 16, 2, 31, 1), (64, 8, 8, 4, 1)])
def test_steps_that_follow_without_a_break(d, H, Hkv, B, n):
    """Tokens appended and attended to step after step, with nothing in between, and in a graph: what each step alone
    gives, launch after launch."""
    prefix, page, steps = 1280, 64, 12
    lens0 = [prefix + 1 + 23 * b % 200 for b in range(B)]
    cache = Cache([x + steps * n for x in lens0], page, Hkv, d, 7, shared=prefix)
    table, cu = dev(cache.table), dev(cu_of([n] * B))
    most = max(lens0) + steps * n
    tokens = [[normal((B * n, h, d), 3 * i + j).cuda() for j, h in enumerate((H, Hkv, Hkv))] for i in range(steps)]

    def run(pause):
        g = cache.gpu()
        lens = dev(lens0)
        q, out = torch.empty_like(tokens[0][0]), []
        for t in tokens:
            lens += n
            q.copy_(t[0])
            pause()
            fa.kv_append_fp8(None, t[1], t[2], *g, table, cu, lens, n)
            pause()
            out.append(fa.attention_prefix_fp8(q, *g, table, cu, lens, n, most, prefix))
            pause()
        return out

    want = run(torch.cuda.synchronize)
    ok()
    for _ in range(3):
        got = run(lambda: None)
        ok()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    g, lens, q = cache.gpu(), dev(lens0), torch.empty_like(tokens[0][0])
    with torch.cuda.graph(graph, stream=side):
        out = []
        for t in tokens:
            lens += n
            q.copy_(t[0])
            fa.kv_append_fp8(None, t[1], t[2], *g, table, cu, lens, n)
            out.append(fa.attention_prefix_fp8(q, *g, table, cu, lens, n, most, prefix))
    for _ in range(2):
        lens.copy_(dev(lens0))
        for x, y in zip(g, cache.gpu()):
            x.copy_(y)
        graph.replay()
        ok()
        for x, y in zip(out, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


# ---------------------------------------------------------------- used together
@pytest.mark.parametrize("d,page,H,Hkv", [(64, 16, 4, 2), (128, 64, 8, 2), (256, 32, 6, 2)])
def test_prompts_context_read_back_and_tokens_behind_a_prefix(d, page, H, Hkv):
    """A shared prompt enters the cache once; each sequence's own prompt is appended behind it; the context is read
    back and the new queries attend to it as packed sequences; then tokens are decoded over the shared prefix. All
    agree with attention over the cache, whose values they read."""
    prefix, ns = 4 * page, [page + 3, 7, 2 * page]
    B, lens = len(ns), [prefix + n for n in ns]
    cache = Cache([n + 2 for n in lens], page, Hkv, d, 2, shared=prefix)
    host = [c.copy() for c in (*cache.codes, *cache.scale)]
    g, table = cache.gpu(), dev(cache.table)
    scale = fa.default_scale(d)
    T, cu = sum(ns), cu_of(ns)
    q, k, v = (normal((T, h, d), i) for i, h in enumerate((H, Hkv, Hkv)))
    first = normal((prefix, Hkv, d), 9)
    one = dev(cache.table[:1])
    fa.kv_append_fp8(None, first.cuda(), first.cuda(), *g, one, dev([0, prefix]), dev([prefix]), prefix)
    fa.kv_append_fp8(None, k.cuda(), v.cuda(), *g, table, dev(cu), dev(lens), max(ns))
    for x, y in ((first, k), (first, v)):
        i = 0 if y is k else 1
        orc.append(x.float().numpy(), host[i], host[2 + i], cache.table[:1], [0, prefix], [prefix], page)
        orc.append(y.float().numpy(), host[i], host[2 + i], cache.table, cu, lens, page)
    kb, vb = fa.kv_read_fp8(*g, table, dev(cu_of(lens)), None, sum(lens))
    o, lse = fa.attention_packed(q.cuda(), kb, vb, dev(cu), dev(cu_of(lens)), max(ns), max(lens))
    op, lp = fa.attention_prefix_fp8(q.cuda(), *g, table, dev(cu), dev(lens), max(ns), max(lens), prefix)
    ok()
    want = orc.paged(f64(q), *host, cache.table, cu, lens, scale)
    check(op, lp, *want)
    over = np.abs(f64(o) - want[0]) - 2.0 ** -8 * np.abs(want[0]) - 2.0 ** -7 * want[2]  # P in bf16 here
    assert over.max() <= 0 and np.all(np.abs(f64(lse) - want[1]) <= 1e-3)
    for step in range(2):
        lens = [n + 1 for n in lens]
        t = [normal((B, h, d), 20 + 3 * step + i) for i, h in enumerate((H, Hkv, Hkv))]
        one_each = cu_of([1] * B)
        fa.kv_append_fp8(None, t[1].cuda(), t[2].cuda(), *g, table, dev(one_each), dev(lens), 1)
        for i in range(2):
            orc.append(t[1 + i].float().numpy(), host[i], host[2 + i], cache.table, one_each, lens, page)
        ot, lt = fa.attention_prefix_fp8(t[0].cuda(), *g, table, dev(one_each), dev(lens), 1, max(lens), prefix)
        ok()
        check(ot, lt, *orc.paged(f64(t[0]), *host, cache.table, one_each, lens, scale))
    # The context's gradients, as for a layer that is tuned on cached keys and values.
    do = normal((T, H, d), 50)
    lens = [prefix + n for n in ns]
    grads = fa.attention_packed_backward(q.cuda(), kb, vb, o, lse, do.cuda(), dev(cu), dev(cu_of(lens)), max(ns), max(lens))
    ok()
    ref = orc.packed_backward(f64(q), f64(kb), f64(vb), f64(do), cu, cu_of(lens), scale)
    for x, r in zip(grads, ref):
        assert np.linalg.norm(f64(x) - r) <= 5e-3 * np.linalg.norm(r)
