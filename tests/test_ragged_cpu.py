"""Packed attention, shared prefixes and reading the cache back on the CPU: what the
library and the binding refuse before any CUDA work, the sizes they report, and the
order in which packed work is taken. No kernel is launched."""

import ctypes

import numpy as np
import pytest

import exact_attention_80_gb300 as fa
import oracle.serving as orc

torch = pytest.importorskip("torch")

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
GROUP, WINDOW, PAGE_SIZE, STRIDE = 16, 17, 19, 20


@pytest.fixture(scope="module")
def lib():
    return fa.load_library()


# ------------------------------------------------------------ the C entry points
def _batch(cq=FAKE, ck=FAKE, B=3, total_q=40, total_k=60, max_q=20, max_k=30):
    return fa._PACKED_BATCH.pack(cq, ck, B, total_q, total_k, max_q, max_k)


def _strides(q=256, k=128, v=128, dout=256, dq=256, dk=128, dv=128):
    return fa._PACKED_STRIDES.pack(q, k, v, dout, dq, dk, dv)


def _forward(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, batch=_batch(), H=4, Hkv=2, d=64, qs=256, ks=128, vs=128,
             scale=0.125, window=0, sinks=0, fill=0)
    a.update(kw)
    return lib.fa_fwd_packed(*a.values(), 0)


def _backward(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, dout=FAKE, lse=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, batch=_batch(), H=4,
             Hkv=2, d=64, strides=_strides(), scale=0.125, window=0, sinks=0, fill=0)
    a.update(kw)
    return lib.fa_bwd_packed(*a.values(), 0)


BOTH = [
    (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(o=0), 1), (dict(lse=0), 1), (dict(batch=None), 1),
    (dict(batch=_batch(cq=0)), 1), (dict(batch=_batch(ck=0)), 1),
    (dict(q=FAKE + 8), 2), (dict(k=FAKE + 4), 2), (dict(o=FAKE + 8), 2), (dict(lse=FAKE + 2), 2),
    (dict(batch=_batch(cq=FAKE + 2)), 2), (dict(batch=_batch(ck=FAKE + 1)), 2),
    (dict(batch=_batch(B=0)), 3), (dict(batch=_batch(B=1 << 23)), 3), (dict(batch=_batch(total_q=0)), 3),
    (dict(batch=_batch(total_k=-1)), 3), (dict(batch=_batch(total_q=1 << 30)), 3), (dict(batch=_batch(max_q=0)), 3),
    (dict(batch=_batch(max_q=41)), 3), (dict(batch=_batch(max_k=61)), 3), (dict(H=0), 3), (dict(Hkv=0), 3),
    (dict(H=1 << 17), 3), (dict(d=96), 4), (dict(scale=0.0), 9), (dict(scale=float("inf")), 9),
    (dict(H=5), GROUP), (dict(H=1), GROUP), (dict(H=258, qs=258 * 64, strides=_strides(258 * 64, dout=258 * 64, dq=258 * 64)), GROUP),
    (dict(window=-1), WINDOW), (dict(sinks=1), WINDOW), (dict(window=5, sinks=-2), WINDOW), (dict(window=2 ** 30), WINDOW),
]


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(qs=255), STRIDE), (dict(ks=64), STRIDE), (dict(vs=-128), STRIDE), (dict(qs=0), STRIDE), (dict(vs=(1 << 32) + 8), STRIDE)])
def test_packed_refuses(lib, kw, code):
    kw = {k: v for k, v in kw.items() if k != "strides"}
    assert _forward(lib, **kw) == code


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(dout=0), 1), (dict(dk=0), 1), (dict(strides=None), 1), (dict(dq=FAKE + 8), 2), (dict(dv=FAKE + 2), 2),
    (dict(ws=0), 6), (dict(ws=FAKE + 4), 6), (dict(strides=_strides(q=128)), STRIDE), (dict(strides=_strides(dout=257)), STRIDE),
    (dict(strides=_strides(dq=248)), STRIDE), (dict(strides=_strides(dk=-128)), STRIDE), (dict(strides=_strides(dv=120)), STRIDE)])
def test_packed_backward_refuses(lib, kw, code):
    kw = {k: v for k, v in kw.items() if k != "qs"}
    assert _backward(lib, **kw) == code


def _many(B, tokens=1):
    return _batch(B=B, total_q=B * tokens, total_k=B * tokens, max_q=tokens, max_k=tokens)


@pytest.mark.parametrize("B", [1 << 18, 1 << 20, 1 << 22])
def test_searches_that_would_take_minutes_are_refused(lib, B):
    """Where each of very many tiles would look through very many sequences (2^22 sequences: hours)."""
    assert _forward(lib, batch=_many(B), d=256, H=8, Hkv=8, qs=2048, ks=2048, vs=2048) == 3
    wide = dict(H=8, Hkv=8, strides=_strides(*[2048] * 7))
    for d in (64, 128, 256):
        assert _backward(lib, batch=_many(B), d=d, **wide) == 3
        assert fa.fa_bwd_packed_workspace_bytes(B, B, B, 1, 1, 8, 8, d) == 0


def test_searches_of_seconds_are_not(lib):
    if torch.cuda.is_available():
        pytest.skip("would launch on fake pointers; only meaningful without a GPU")
    for B in (1 << 15, 1 << 16):
        wide = dict(H=4, Hkv=2, strides=_strides(*[1024] * 7))
        assert _forward(lib, batch=_many(B), d=256, H=4, Hkv=2, qs=1024, ks=512, vs=512) == 7
        for d in (64, 128, 256):
            assert _backward(lib, batch=_many(B), d=d, **wide) == 7
            assert fa.fa_bwd_packed_workspace_bytes(B, B, B, 1, 1, 4, 2, d) > B * 64 * 4 * d * 4
    assert _forward(lib, batch=_many(1 << 22), d=128, H=8, Hkv=8, qs=1024, ks=1024, vs=1024) == 7  # (one search a CTA)
    assert _forward(lib, batch=_many(100, 1 << 20), d=256, H=8, Hkv=8, qs=2048, ks=2048, vs=2048) == 7


def _cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=10, Hkv=2, page=16, d=64):
    return fa._PAGED_CACHE.pack(k, v, ks, vs, pages, Hkv, page, d)


def _prefix(lib, **kw):
    a = dict(q=FAKE, cache=_cache(), table=FAKE, cu=FAKE, lens=FAKE, o=FAKE, lse=FAKE, ws=FAKE, B=2, H=4, total=8, max_q=4,
             max_k=64, max_pages=4, prefix=32, scale=0.125, splits=1, prefix_splits=2)
    a.update(kw)
    return lib.fa_fwd_prefix_fp8(*a.values(), 0)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(o=0), 1), (dict(lse=0), 1), (dict(table=0), 1), (dict(cu=0), 1), (dict(cache=None), 1),
    (dict(cache=_cache(vs=0)), 1), (dict(q=FAKE + 8), 2), (dict(lse=FAKE + 1), 2), (dict(lens=FAKE + 2), 2),
    (dict(B=0), 3), (dict(total=0), 3), (dict(max_q=9), 3), (dict(max_k=65), 3), (dict(max_pages=0), 3), (dict(H=0), 3),
    (dict(prefix=0), 3), (dict(prefix=-16), 3), (dict(prefix=40), 3), (dict(prefix=64), 3), (dict(prefix=80), 3),
    (dict(cache=_cache(d=32)), 4), (dict(splits=0), 5), (dict(prefix_splits=0), 5), (dict(splits=200, prefix_splits=57), 5),
    (dict(splits=2 ** 31 - 1, prefix_splits=2 ** 31 - 1), 5), (dict(ws=0), 6), (dict(ws=FAKE + 4), 6),
    (dict(splits=1, prefix_splits=1, ws=0), 6), (dict(scale=float("nan")), 9), (dict(H=5), GROUP), (dict(H=1), GROUP),
    (dict(cache=_cache(page=24)), PAGE_SIZE)])
def test_prefix_refuses(lib, kw, code):
    assert _prefix(lib, **kw) == code


def _read(lib, **kw):
    a = dict(cache=_cache(), table=FAKE, cu=FAKE, starts=FAKE, k=FAKE, v=FAKE, B=2, total=8, max_pages=4, ks=128, vs=128, fill=0)
    a.update(kw)
    return lib.fa_kv_read_fp8(*a.values(), 0)


@pytest.mark.parametrize("kw,code", [
    (dict(cache=None), 1), (dict(cache=_cache(k=0)), 1), (dict(table=0), 1), (dict(cu=0), 1), (dict(k=0), 1), (dict(v=0), 1),
    (dict(k=FAKE + 8), 2), (dict(v=FAKE + 4), 2), (dict(starts=FAKE + 2), 2), (dict(cu=FAKE + 1), 2),
    (dict(B=0), 3), (dict(total=0), 3), (dict(total=1 << 30), 3), (dict(max_pages=0), 3), (dict(max_pages=1 << 28), 3),
    (dict(cache=_cache(pages=0)), 3), (dict(cache=_cache(d=80)), 4), (dict(cache=_cache(page=8)), PAGE_SIZE),
    (dict(ks=120), STRIDE), (dict(vs=132), STRIDE), (dict(ks=-128), STRIDE)])
def test_read_refuses(lib, kw, code):
    assert _read(lib, **kw) == code


def test_reads_whose_search_would_take_minutes_are_refused(lib):
    for B, total in ((1 << 24, 1 << 29), (1 << 28, 1 << 28), (2 ** 31 - 1, (1 << 30) - 1)):
        assert _read(lib, B=B, total=total) == 3
    if not torch.cuda.is_available():
        assert _read(lib, B=1 << 16, total=1 << 27) == 7 and _read(lib, B=1, total=(1 << 30) - 1) == 7


def test_prefix_of_more_sequences_than_can_look_for_the_first(lib):
    for B in ((1 << 19) + 1, 2 ** 31 - 1):
        assert _prefix(lib, B=B) == 3
        assert fa.fa_prefix_num_splits(B, 4, 2, 8, 4, 64, 32, 64) == (0, 0)
    assert fa.fa_prefix_num_splits(1 << 19, 4, 2, 1 << 19, 1, 64, 32, 64) != (0, 0)
    if not torch.cuda.is_available():
        assert _prefix(lib, B=1 << 19) == 7


def test_valid_calls_without_a_gpu_report_a_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("would launch on fake pointers; only meaningful without a GPU")
    assert _forward(lib) == 7 == _backward(lib) and _prefix(lib) == 7 and _read(lib) == 7 and _read(lib, starts=0) == 7


def test_sizes(lib):
    rows = (40 + 64 * 4 + 127) // 128 * 128
    assert fa.fa_bwd_packed_workspace_bytes(3, 40, 60, 20, 30, 4, 2, 64) >= rows * 4 * 66 * 4
    for bad in (dict(B=0), dict(max_q=41), dict(H=5), dict(d=96), dict(window=0, sinks=2), dict(window=-1)):
        a = dict(B=3, total_q=40, total_k=60, max_q=20, max_k=30, H=4, Hkv=2, d=64, window=0, sinks=0)
        a.update(bad)
        assert fa.fa_bwd_packed_workspace_bytes(*a.values()) == 0
    # One head of one long sequence is cut into parts, many heads are not.
    one = fa.fa_bwd_packed_workspace_bytes(1, 8192, 8192, 8192, 8192, 1, 1, 128)
    assert one > (8192 + 128) * 130 * 4
    many = fa.fa_bwd_packed_workspace_bytes(1, 8192, 8192, 8192, 8192, 64, 64, 128)
    assert many == (8192 + 128) * 64 * 130 * 4
    for args in ((1, 8, 8, 1, 1, 100, 16, 64), (64, 32, 8, 64, 1, 18000, 16384, 128), (3, 16, 2, 900, 512, 4096, 1024, 256)):
        own, shared = fa.fa_prefix_num_splits(*args)
        assert own >= 1 and shared >= 1 and own + shared <= fa.FA_MAX_SPLITS
    for args in ((1, 5, 2, 1, 1, 100, 16, 64), (1, 4, 2, 1, 1, 16, 16, 64), (1, 4, 2, 1, 1, 100, 0, 64), (1, 4, 2, 1, 1, 100, 16, 80),
                 (1, 4, 2, 1, 2, 100, 16, 64)):
        assert fa.fa_prefix_num_splits(*args) == (0, 0)
    assert lib.fa_prefix_num_splits(1, 4, 2, 1, 1, 100, 16, 64, None) == 0
    assert fa._PACKED_BATCH.size == 36 and fa._PACKED_STRIDES.size == 56


# ------------------------------------------------------------------ the binding
class _Stub:
    """Compute entry points that return FA_OK without doing anything; sizes are the library's."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith(("_bytes", "_splits", "_string")):
            return getattr(self.real, name)
        return lambda *args: (self.calls.append((name, args)), 0)[1]


@pytest.fixture
def stub(monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("CPU tensors stand in for device tensors only where no GPU exists")
    s = _Stub(fa.load_library())
    monkeypatch.setattr(fa, "load_library", lambda: s)
    monkeypatch.setattr(fa, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))
    return s


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def cache_args(pages=5, Hkv=2, page=16, d=64):
    c = torch.zeros((pages, Hkv, page, d), dtype=torch.uint8)
    return [c, c.clone(), torch.ones(pages, Hkv), torch.ones(pages, Hkv)]


def packed_args():
    q, k = bf(9, 4, 64), bf(12, 2, 64)
    return q, k, k.clone(), q.clone(), torch.zeros(4, 9), i32(4), i32(4)


def test_binding_packed(stub):
    q, k, v, o, lse, cq, ck = packed_args()
    fused = bf(9, 8, 64)
    fa.attention_packed(fused[:, :4], fused[:, 4:6], fused[:, 6:], cq, cq, 9, 9, 5, 1)
    name, args = stub.calls[-1]
    assert name == "fa_fwd_packed" and args[6:12] == (4, 2, 64, 512, 512, 512) and args[13:16] == (5, 1, 1)
    assert fa._PACKED_BATCH.unpack(args[5])[2:] == (3, 9, 9, 9, 9)
    fa.fa_fwd_packed(q, k, v, o, lse, cq, ck, 9, 12)
    assert stub.calls[-1][1][9:12] == (256, 128, 128) and stub.calls[-1][1][15] == 0
    fa.attention_packed_backward(q, k, v, o, lse, o, cq, ck, 9, 12, scale=0.25)
    name, args = stub.calls[-1]
    assert name == "fa_bwd_packed" and fa._PACKED_STRIDES.unpack(args[14]) == (256, 128, 128, 256, 256, 128, 128)
    assert args[15] == 0.25 and args[18] == 1
    ws = torch.zeros(fa.fa_bwd_packed_workspace_bytes(3, 9, 12, 9, 12, 4, 2, 64) // 4)
    grads = bf(9, 8, 64)
    fa.fa_bwd_packed(q, k, v, o, o, lse, q.clone(), k.clone(), k.clone(), ws, cq, ck, 9, 12)
    n = len(stub.calls)
    f = fa.attention_packed
    bad = [lambda: f(q.float(), k, v, cq, ck, 9, 12), lambda: f(q[0], k, v, cq, ck, 9, 12), lambda: f(q, k, v[:-1], cq, ck, 9, 12),
           lambda: f(q, bf(12, 2, 128), v, cq, ck, 9, 12), lambda: f(q, k, v, cq.long(), ck, 9, 12),
           lambda: f(q, k, v, cq, i32(5), 9, 12), lambda: f(q, k, v, i32(1), i32(1), 9, 12), lambda: f(q, k, v, i32(4, 1), ck, 9, 12),
           lambda: f(q, k, v, i32(8)[::2], ck, 9, 12), lambda: f(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, cq, ck, 9, 12),
           lambda: f(bf(9, 4, 128)[..., ::2], k, v, cq, ck, 9, 12), lambda: f(bf(0, 4, 64), k, v, cq, ck, 9, 12),
           lambda: fa.fa_fwd_packed(q, k, v, o[:-1], lse, cq, ck, 9, 12), lambda: fa.fa_fwd_packed(q, k, v, o, lse.t(), cq, ck, 9, 12),
           lambda: fa.fa_fwd_packed(q, k, v, o.float(), lse, cq, ck, 9, 12),
           lambda: fa.fa_bwd_packed(q, k, v, o, o, lse, q.clone(), k.clone(), k.clone(), ws[:-1], cq, ck, 9, 12),
           lambda: fa.fa_bwd_packed(q, k, v, o, o, lse, q.clone(), k.clone(), k.clone(), ws.double(), cq, ck, 9, 12),
           lambda: fa.fa_bwd_packed(q, k, v, o, o, lse, q.clone(), grads[:, :2], k.clone(), ws, cq, ck, 9, 12),
           lambda: fa.fa_bwd_packed(q, k, v, o, o[:, :2], lse, q.clone(), k.clone(), k.clone(), ws, cq, ck, 9, 12),
           lambda: fa.fa_bwd_packed(q, k, v, o, None, lse, q.clone(), k.clone(), k.clone(), ws, cq, ck, 9, 12)]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            call()
            pytest.fail(f"call {i} was taken")
    assert len(stub.calls) == n


def test_binding_prefix_and_read(stub):
    q, c, batch = bf(6, 4, 64), cache_args(), [i32(3, 4), i32(4), i32(3)]
    fa.attention_prefix_fp8(q, *c, *batch, 2, 60, 32)
    name, args = stub.calls[-1]
    assert name == "fa_fwd_prefix_fp8" and args[8:15] == (3, 4, 6, 2, 60, 4, 32)
    assert args[16:18] == fa.fa_prefix_num_splits(3, 4, 2, 6, 2, 60, 32, 64)
    fa.attention_prefix_fp8(q, *c, *batch, 2, 60, 32, num_splits=3, prefix_splits=2)
    assert stub.calls[-1][1][16:18] == (3, 2)
    ws = torch.zeros(fa.fa_paged_workspace_bytes(6, 4, 64, 3) // 4)
    fa.fa_fwd_prefix_fp8(q, *c, q.clone(), torch.zeros(4, 6), *batch, 2, 60, 32, ws, 1, 2)
    k, v = fa.kv_read_fp8(*c, i32(3, 4), i32(4), i32(3), 7)
    name, args = stub.calls[-1]
    assert name == "fa_kv_read_fp8" and args[6:12] == (3, 7, 4, 128, 128, 1) and args[3] != 0 and k.shape == (7, 2, 64) == v.shape
    fa.kv_read_fp8(*c, i32(3, 4), i32(4), total=7)
    assert stub.calls[-1][1][3] == 0
    wide = bf(7, 6, 64)
    fa.fa_kv_read_fp8(*c, wide[:, :2], wide[:, 2:4], i32(3, 4), i32(4))
    assert stub.calls[-1][1][9:12] == (384, 384, 0)
    n = len(stub.calls)
    bad = [lambda: fa.attention_prefix_fp8(bf(6, 4, 128), *c, *batch, 2, 60, 32), lambda: fa.attention_prefix_fp8(bf(12, 4, 64)[::2], *c, *batch, 2, 60, 32),
           lambda: fa.attention_prefix_fp8(q, *c, i32(3, 4), i32(3), i32(3), 2, 60, 32),
           lambda: fa.fa_fwd_prefix_fp8(q, *c, q.clone(), torch.zeros(4, 6), *batch, 2, 60, 32, ws, 2, 2),
           lambda: fa.fa_fwd_prefix_fp8(q, *c, None, None, *batch, 2, 60, 32, ws, 1, 2),
           lambda: fa.kv_read_fp8(*c, i32(3, 4), i32(4), i32(3)), lambda: fa.kv_read_fp8(*c, i32(3, 4), i32(4), i32(4), 7),
           lambda: fa.kv_read_fp8(*c, i32(3, 4), i32(3), i32(3), 7), lambda: fa.kv_read_fp8(*c, i32(12), i32(4), i32(3), 7),
           lambda: fa.kv_read_fp8(*c, i32(3, 4).long(), i32(4), i32(3), 7),
           lambda: fa.fa_kv_read_fp8(*c, wide[:, :2], wide[:, 2:5], i32(3, 4), i32(4)),
           lambda: fa.fa_kv_read_fp8(*c, wide[:, :2].float(), wide[:, 2:4], i32(3, 4), i32(4)),
           lambda: fa.fa_kv_read_fp8(*c, bf(7, 2, 128), bf(7, 2, 128), i32(3, 4), i32(4))]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            call()
            pytest.fail(f"call {i} was taken")
    assert len(stub.calls) == n


def test_numbers_past_32_bits_are_refused(stub):
    q, k, v, o, lse, cq, ck = packed_args()
    t, c, batch = bf(6, 4, 64), cache_args(), [i32(3, 4), i32(4), i32(3)]
    ws = torch.zeros(1 << 16)
    calls = [
        lambda n: fa.attention_packed(q, k, v, cq, ck, n, 12), lambda n: fa.attention_packed(q, k, v, cq, ck, 9, n),
        lambda n: fa.attention_packed(q, k, v, cq, ck, 9, 12, n), lambda n: fa.attention_packed(q, k, v, cq, ck, 9, 12, 4, n),
        lambda n: fa.attention_packed_backward(q, k, v, o, lse, o, cq, ck, n, 12),
        lambda n: fa.attention_packed_backward(q, k, v, o, lse, o, cq, ck, 9, 12, 4, n),
        lambda n: fa.attention_prefix_fp8(t, *c, *batch, n, 60, 32), lambda n: fa.attention_prefix_fp8(t, *c, *batch, 2, n, 32),
        lambda n: fa.attention_prefix_fp8(t, *c, *batch, 2, 60, n), lambda n: fa.attention_prefix_fp8(t, *c, *batch, 2, 60, 32, num_splits=n),
        lambda n: fa.fa_fwd_prefix_fp8(t, *c, t.clone(), torch.zeros(4, 6), *batch, 2, 60, 32, ws, 1, n),
        lambda n: fa.fa_prefix_num_splits(1, 8, 2, 1, 1, n, 16, 64), lambda n: fa.fa_bwd_packed_workspace_bytes(1, n, 5, 5, 5, 2, 2, 64),
    ]
    for i, call in enumerate(calls):
        for n in (2 ** 32 + 5, -(2 ** 32) - 5, 2 ** 31):
            with pytest.raises(OverflowError):
                call(n)
                pytest.fail(f"call {i} took {n}")
    assert not stub.calls


# ------------------------------------------------------------------- the oracle
def test_oracle_of_packed_sequences():
    """Packed sequences are the dense statement sequence by sequence; gradients against differences."""
    rng = np.random.default_rng(0)
    cu_q, cu_k = [0, 3, 3, 8], [0, 5, 6, 11]
    q, k, v, do = rng.standard_normal((8, 4, 6)), rng.standard_normal((11, 2, 6)), rng.standard_normal((11, 2, 6)), rng.standard_normal((8, 4, 6))
    o, lse, a = orc.packed_forward(q, k, v, cu_q, cu_k, 0.3, 3, 1)
    for b in range(3):
        s, t = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        x = [y.transpose(1, 0, 2)[None] for y in (q[s], k[t], v[t])]
        ob, lb = orc.window_forward(*x, 0.3, 3, 1)
        assert np.allclose(o[s].transpose(1, 0, 2), ob[0]) and np.allclose(lse[:, s], lb[0])
    assert np.all(a >= np.abs(o) - 1e-12)
    grads = orc.packed_backward(q, k, v, do, cu_q, cu_k, 0.3, 3, 1)
    for i, g in enumerate(grads):
        step, f = rng.standard_normal(g.shape), []
        for h in (1e-5, -1e-5):
            x = [q.copy(), k.copy(), v.copy()]
            x[i] += h * step
            f.append((orc.packed_forward(*x, cu_q, cu_k, 0.3, 3, 1)[0] * do).sum())
        assert abs((f[0] - f[1]) / 2e-5 - (g * step).sum()) <= 1e-6


def test_oracle_read():
    codes = np.arange(2 * 1 * 4 * 3).reshape(2, 1, 4, 3).astype(np.uint8)
    scale = np.array([[2.0], [0.5]], np.float32)
    got = orc.read(codes, scale, np.array([[1, 0], [0, -1]]), [3, 1], [2, 1], 4)
    assert np.array_equal(got[:, 0], [orc.VALUES[codes[1, 0, 3]] * 0.5, orc.VALUES[codes[0, 0, 0]] * 2, orc.VALUES[codes[0, 0, 1]] * 2])
