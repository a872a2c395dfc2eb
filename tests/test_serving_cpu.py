"""Rotary positions, the paged cache and the sliding window on the CPU: what the
library and the binding refuse before any CUDA work, the sizes they report, and
the oracle's own statements against independent ones. No kernel is launched."""

import ctypes

import numpy as np
import pytest

import exact_attention_80_gb300 as fa
import oracle
import oracle.serving as orc

torch = pytest.importorskip("torch")

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
GROUP, WINDOW, ROPE, PAGE_SIZE, STRIDE = 16, 17, 18, 19, 20


@pytest.fixture(scope="module")
def lib():
    return fa.load_library()


# ------------------------------------------------------------ the C entry points
def _rotation(table=FAKE, positions=FAKE, rot=64, axes=1, sections=(32,), max_pos=100, interleaved=0):
    return fa._ROTATION.pack(table, positions, rot, axes, *sections, *(0,) * (4 - len(sections)), max_pos, interleaved)


def _tensor(x=FAKE, y=FAKE, H=2, xs=(0, 64, 128), ys=(0, 64, 128)):
    return fa._ROPE_TENSOR.pack(x, y, H, *xs, *ys)


@pytest.mark.parametrize("q,k,rope,shape,code", [
    (_tensor(x=0), None, _rotation(), (1, 8, 64), 1), (_tensor(), _tensor(y=0), _rotation(), (1, 8, 64), 1),
    (_tensor(), None, _rotation(table=0), (1, 8, 64), 1), (_tensor(), None, _rotation(positions=0), (1, 8, 64), 1),
    (_tensor(x=FAKE + 8), None, _rotation(), (1, 8, 64), 2), (_tensor(), None, _rotation(table=FAKE + 4), (1, 8, 64), 2),
    (_tensor(), None, _rotation(positions=FAKE + 2), (1, 8, 64), 2),
    (_tensor(H=0), None, _rotation(), (1, 8, 64), 3), (_tensor(), None, _rotation(), (0, 8, 64), 3),
    (_tensor(), None, _rotation(), (1, 0, 64), 3), (_tensor(), None, _rotation(), (1 << 16, 1 << 16, 64), 3),
    (_tensor(), None, _rotation(), (1, 8, 96), 4),
    (_tensor(ys=(0, 0, 128)), None, _rotation(), (1, 8, 64), STRIDE),
    (_tensor(), None, _rotation(rot=8), (1, 8, 64), ROPE), (_tensor(), None, _rotation(rot=40), (1, 8, 64), ROPE),
    (_tensor(), None, _rotation(rot=128), (1, 8, 64), ROPE), (_tensor(), None, _rotation(axes=0), (1, 8, 64), ROPE),
    (_tensor(), None, _rotation(axes=5), (1, 8, 64), ROPE), (_tensor(), None, _rotation(max_pos=0), (1, 8, 64), ROPE),
    (_tensor(), None, _rotation(axes=2, sections=(16, 15)), (1, 8, 64), ROPE),
    (_tensor(), None, _rotation(axes=3, sections=(40, -16, 8)), (1, 8, 64), ROPE),
    (_tensor(xs=(0, 64, 100)), None, _rotation(), (1, 8, 64), STRIDE),
    (_tensor(ys=(0, -64, 128)), None, _rotation(), (1, 8, 64), STRIDE),
])
def test_rope_refuses(lib, q, k, rope, shape, code):
    assert lib.fa_rope(q, k, rope, *shape, 0, 0) == code


def _cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=10, Hkv=2, page=16, d=64):
    return fa._PAGED_CACHE.pack(k, v, ks, vs, pages, Hkv, page, d)


def _append(lib, q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, rope=None, cache=None, table=FAKE, cu=FAKE, lens=FAKE, B=2, H=4,
            total=8, max_new=4, max_pages=4, qs=256, ks=128, vs=128):
    return lib.fa_kv_append_fp8(q, k, v, q_out, rope, cache or _cache(), table, cu, lens, B, H, total, max_new,
                                max_pages, qs, ks, vs, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), 1), (dict(v=0), 1), (dict(table=0), 1), (dict(cu=0), 1), (dict(lens=0), 1), (dict(q=0), 1),
    (dict(q_out=0), 1), (dict(cache=_cache(k=0)), 1), (dict(cache=_cache(vs=0)), 1), (dict(rope=_rotation(table=0)), 1),
    (dict(k=FAKE + 8), 2), (dict(q_out=FAKE + 4), 2), (dict(table=FAKE + 2), 2), (dict(cache=_cache(v=FAKE + 8)), 2),
    (dict(cache=_cache(ks=FAKE + 2)), 2),
    (dict(B=0), 3), (dict(total=0), 3), (dict(max_new=0), 3), (dict(max_new=9), 3), (dict(max_pages=0), 3), (dict(total=2**31 - 1), 3),
    (dict(H=0), 3), (dict(cache=_cache(pages=0)), 3), (dict(cache=_cache(Hkv=0)), 3),
    (dict(cache=_cache(pages=1 << 28, Hkv=8)), 3), (dict(max_pages=1 << 30), 3),
    (dict(cache=_cache(d=96)), 4),
    (dict(cache=_cache(page=8)), PAGE_SIZE), (dict(cache=_cache(page=48)), PAGE_SIZE), (dict(cache=_cache(page=256)), PAGE_SIZE),
    (dict(rope=_rotation(rot=72)), ROPE), (dict(rope=_rotation(positions=0, axes=2, sections=(16, 16))), ROPE),
    (dict(ks=100), STRIDE), (dict(vs=-128), STRIDE), (dict(qs=12), STRIDE), (dict(qs=1 << 40), STRIDE),
])
def test_append_refuses(lib, kw, code):
    assert _append(lib, **kw) == code


def _paged(lib, q=FAKE, cache=None, table=FAKE, cu=FAKE, lens=FAKE, o=FAKE, lse=FAKE, ws=FAKE, B=2, H=4, total=8,
           max_q=4, max_k=64, max_pages=4, scale=0.125, window=0, sinks=0, splits=2):
    return lib.fa_fwd_paged_fp8(q, cache or _cache(), table, cu, lens, o, lse, ws, B, H, total, max_q, max_k, max_pages,
                                scale, window, sinks, splits, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(o=0), 1), (dict(lse=0), 1), (dict(table=0), 1), (dict(cache=_cache(ks=0)), 1),
    (dict(q=FAKE + 8), 2), (dict(o=FAKE + 8), 2), (dict(lse=FAKE + 1), 2), (dict(lens=FAKE + 2), 2),
    (dict(B=0), 3), (dict(total=0), 3), (dict(max_q=0), 3), (dict(max_q=9), 3), (dict(max_k=0), 3),
    (dict(max_k=65), 3), (dict(max_pages=1 << 28), 3), (dict(H=0), 3),
    (dict(cache=_cache(d=32)), 4), (dict(splits=0), 5), (dict(splits=257), 5), (dict(ws=0), 6), (dict(ws=FAKE + 4), 6),
    (dict(scale=0.0), 9), (dict(scale=float("nan")), 9),
    (dict(H=5), GROUP), (dict(H=1), GROUP),
    (dict(window=-1), WINDOW), (dict(sinks=4), WINDOW), (dict(window=8, sinks=-1), WINDOW),
    (dict(window=2**31 - 1), WINDOW), (dict(cache=_cache(page=100)), PAGE_SIZE),
])
def test_paged_refuses(lib, kw, code):
    assert _paged(lib, **kw) == code


def _window(lib, q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, B=1, H=4, Hkv=2, Nq=8, Nk=8, d=64, scale=0.125, window=4,
            sinks=1):
    return lib.fa_fwd_window(q, k, v, o, lse, B, H, Hkv, Nq, Nk, d, scale, window, sinks, 0)


BAD_WINDOW = [
    (dict(q=0), 1), (dict(k=0), 1), (dict(o=0), 1), (dict(lse=0), 1), (dict(v=FAKE + 8), 2), (dict(o=FAKE + 8), 2),
    (dict(lse=FAKE + 2), 2), (dict(B=0), 3), (dict(Nq=0), 3), (dict(Nk=-1), 3), (dict(Hkv=0), 3),
    (dict(Nk=2**30), 3), (dict(d=80), 4), (dict(scale=-1.0), 9), (dict(H=5), GROUP), (dict(H=1), GROUP),
    (dict(window=-4), WINDOW), (dict(sinks=-1), WINDOW), (dict(window=0, sinks=3), WINDOW), (dict(window=2**30), WINDOW),
]


@pytest.mark.parametrize("kw,code", BAD_WINDOW)
def test_window_refuses(lib, kw, code):
    assert _window(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [(k, c) for k, c in BAD_WINDOW if not {"o", "lse"} & set(k)] + [
    (dict(splits=0), 5), (dict(splits=257), 5), (dict(ws=0), 6), (dict(ws=FAKE + 8), 6)])
def test_window_splitkv_refuses(lib, kw, code):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ws=FAKE, B=1, H=4, Hkv=2, Nq=8, Nk=8, d=64, scale=0.125, window=4, sinks=1, splits=2)
    a.update(kw)
    assert lib.fa_fwd_window_splitkv(*a.values(), 0) == code


@pytest.mark.parametrize("kw,code", BAD_WINDOW + [(dict(ws=0), 6), (dict(ws=FAKE + 4), 6), (dict(dk=0), 1),
                                                 (dict(dout=FAKE + 8), 2)])
def test_window_backward_refuses(lib, kw, code):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, dout=FAKE, lse=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, B=1, H=4, Hkv=2,
             Nq=8, Nk=8, d=64, scale=0.125, window=4, sinks=1)
    a.update(kw)
    assert lib.fa_bwd_window(*a.values(), 0) == code


def test_valid_calls_without_a_gpu_report_a_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("would launch on fake pointers; only meaningful without a GPU")
    assert lib.fa_rope(_tensor(), _tensor(), _rotation(), 1, 8, 64, 0, 0) == 7
    assert _append(lib, rope=_rotation()) == 7 and _append(lib) == 7 and _append(lib, q=0, q_out=0) == 7
    assert _paged(lib) == 7 and _paged(lib, splits=1, ws=0) == 7 and _window(lib) == 7


def test_sizes(lib):
    assert fa.fa_paged_workspace_bytes(10, 8, 128, 3) == 3 * 10 * 8 * 130 * 4
    assert fa.fa_paged_workspace_bytes(10, 8, 128, 1) == 0 == fa.fa_paged_workspace_bytes(10, 8, 100, 2)
    for args in ((1, 8, 8, 1, 100, 64), (64, 32, 8, 1, 32768, 128), (2, 16, 2, 2048, 16384, 128), (3, 4, 4, 7, 1, 256)):
        assert 1 <= fa.fa_paged_num_splits(*args) <= fa.FA_MAX_SPLITS
    assert fa.fa_paged_num_splits(1, 5, 2, 1, 100, 64) == 0
    base = fa.fa_bwd_workspace_bytes(2, 4, 300, 128)
    assert fa.fa_bwd_window_workspace_bytes(2, 4, 2, 300, 300, 128, 0, 0) >= base > 0
    assert fa.fa_bwd_window_workspace_bytes(2, 4, 3, 300, 300, 128, 0, 0) == 0
    assert fa.fa_bwd_window_workspace_bytes(2, 4, 2, 300, 300, 96, 0, 0) == 0
    assert fa.fa_window_num_splits(1, 8, 2, 1, 4096, 64, 0) > 1 == fa.fa_window_num_splits(8, 32, 8, 4096, 4096, 64, 0)
    assert fa.fa_window_num_splits(1, 5, 2, 1, 4096, 64, 0) == 0 == fa.fa_window_num_splits(1, 4, 2, 1, 4096, 64, 0, 3)
    # The library's own structs are as long as the ones the binding packs.
    assert fa._ROTATION.size == 48 and fa._ROPE_TENSOR.size == 72 and fa._PAGED_CACHE.size == 48


# ------------------------------------------------------------------ the binding
class _Stub:
    """Compute entry points that return FA_OK without doing anything."""

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


def test_binding_rope(stub):
    q, k, table = bf(2, 4, 9, 64), bf(2, 2, 9, 64), torch.zeros(100, 64)
    fa.rope(q, k, table, i32(2, 9))
    fa.rope(q, None, table, i32(3, 2, 9), sections=(8, 12, 12))
    name, args = stub.calls[-1]
    assert name == "fa_rope" and args[1] is None and args[3:7] == (2, 9, 64, 0)
    packed = fa._ROPE_TENSOR.unpack(args[0])
    assert packed[2:] == (4, 4 * 9 * 64, 9 * 64, 64, 4 * 9 * 64, 9 * 64, 64)
    assert fa._ROTATION.unpack(args[2])[2:] == (64, 3, 8, 12, 12, 0, 100, 0)
    fused = bf(9, 6, 64)
    fa.rope(fused[:, :4], fused[:, 4:], table, i32(1, 9), inverse=True)
    packed = fa._ROPE_TENSOR.unpack(stub.calls[-1][1][1])
    assert packed[2:] == (2, 0, 64, 384, 0, 64, 128) and stub.calls[-1][1][6] == 1
    n = len(stub.calls)
    bad = [
        lambda: fa.rope(q.float(), k, table, i32(2, 9)), lambda: fa.rope(q, k[:, :, :8], table, i32(2, 9)),
        lambda: fa.rope(q, k, table.double(), i32(2, 9)), lambda: fa.rope(q, k, table[:, ::2], i32(2, 9)),
        lambda: fa.rope(q, k, table, i32(2, 8)), lambda: fa.rope(q, k, table, i32(2, 9).long()),
        lambda: fa.rope(q, k, table, None), lambda: fa.rope(q, k, table, i32(2, 2, 9), sections=(32,)),
        lambda: fa.rope(q.transpose(2, 3), None, table, i32(2, 9)), lambda: fa.rope(bf(2, 9), None, table, i32(2, 9)),
        lambda: fa.fa_rope(q, k, q, None, table, i32(2, 9)), lambda: fa.fa_rope(q, None, bf(2, 4, 8, 64), None, table, i32(2, 9)),
        lambda: fa.fa_rope(q, None, q, k, table, i32(2, 9)),
        lambda: fa.fa_rope(q, None, bf(1, 4, 9, 64).expand(2, 4, 9, 64), None, table, i32(2, 9)),
        lambda: fa.rope(q, k, table, i32(5, 2, 9)),
    ]
    for call in bad:
        with pytest.raises((TypeError, ValueError, fa.FAError)):
            call()
    assert len(stub.calls) == n


def _cache_args(pages=5, Hkv=2, page=16, d=64):
    c = torch.zeros((pages, Hkv, page, d), dtype=torch.uint8)
    return [c, c.clone(), torch.ones(pages, Hkv), torch.ones(pages, Hkv)]


def test_binding_append(stub):
    q, k, v = bf(6, 4, 64), bf(6, 2, 64), bf(6, 2, 64)
    batch = [i32(3, 4), i32(4), i32(3)]
    table = torch.zeros(50, 32)
    assert fa.kv_append_fp8(q, k, v, *_cache_args(), *batch, 2, table=table).shape == q.shape
    assert fa.kv_append_fp8(None, k, v, *_cache_args(), *batch, 2) is None
    fused = bf(6, 8, 64)
    fa.kv_append_fp8(fused[:, :4], fused[:, 4:6], fused[:, 6:], *_cache_args(), *batch, 2)
    assert stub.calls[-1][1][14:17] == (512, 512, 512)
    n = len(stub.calls)
    e4 = [x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x for x in _cache_args()]
    fa.kv_append_fp8(q, k, v, *e4, *batch, 2)
    n += 1
    c = _cache_args()
    bad = [
        lambda: fa.kv_append_fp8(q, k, v[:5], *c, *batch, 2), lambda: fa.kv_append_fp8(q[:5], k, v, *c, *batch, 2),
        lambda: fa.kv_append_fp8(q, bf(6, 3, 64), bf(6, 3, 64), *c, *batch, 2),
        lambda: fa.kv_append_fp8(q, k.transpose(1, 2), v, *c, *batch, 2),
        lambda: fa.kv_append_fp8(q, k, v, c[0].int(), *c[1:], *batch, 2),
        lambda: fa.kv_append_fp8(q, k, v, c[0][:4], *c[1:], *batch, 2),
        lambda: fa.kv_append_fp8(q, k, v, c[0], c[1], c[2].t(), c[3], *batch, 2),
        lambda: fa.kv_append_fp8(q, k, v, c[0], c[1], c[2].double(), c[3], *batch, 2),
        lambda: fa.kv_append_fp8(q, k, v, *c, i32(3, 4).long(), i32(4), i32(3), 2),
        lambda: fa.kv_append_fp8(q, k, v, *c, i32(3, 4), i32(3), i32(3), 2),
        lambda: fa.kv_append_fp8(q, k, v, *c, i32(2, 4), i32(4), i32(3), 2),
        lambda: fa.kv_append_fp8(q, k, v, *c, *batch, 2, positions=i32(6)),
        lambda: fa.kv_append_fp8(q, k, v, *c, *batch, 2, table=table, positions=i32(5)),
        lambda: fa.fa_kv_append_fp8(q, k, v, None, *c, *batch, 2), lambda: fa.fa_kv_append_fp8(None, k, v, q, *c, *batch, 2),
    ]
    for call in bad:
        with pytest.raises((TypeError, ValueError, AttributeError)):
            call()
    assert len(stub.calls) == n


def test_binding_paged(stub):
    q, batch = bf(6, 4, 64), [i32(3, 4), i32(4), i32(3)]
    o, lse = fa.attention_paged_fp8(q, *_cache_args(), *batch, 2, 60)
    assert o.shape == q.shape and lse.shape == (4, 6) and lse.dtype == torch.float32
    assert stub.calls[-1][1][-2] == fa.fa_paged_num_splits(3, 4, 2, 2, 60, 64)
    fa.attention_paged_fp8(q, *_cache_args(), *batch, 2, 60, num_splits=3, window=5, sinks=1)
    assert stub.calls[-1][1][-4:-1] == (5, 1, 3) and stub.calls[-1][1][7] != 0
    n, c = len(stub.calls), _cache_args()
    need = fa.fa_paged_workspace_bytes(6, 4, 64, 3) // 4
    f32 = lambda *s: torch.zeros(s)  # noqa: E731
    bad = [
        lambda: fa.attention_paged_fp8(q.half(), *c, *batch, 2, 60),
        lambda: fa.attention_paged_fp8(bf(6, 8, 64)[:, :4], *c, *batch, 2, 60),
        lambda: fa.attention_paged_fp8(bf(6, 4, 128), *c, *batch, 2, 60),
        lambda: fa.fa_fwd_paged_fp8(q, *c, bf(6, 4, 32), f32(4, 6), *batch, 2, 60),
        lambda: fa.fa_fwd_paged_fp8(q, *c, bf(6, 4, 64), f32(6, 4), *batch, 2, 60),
        lambda: fa.fa_fwd_paged_fp8(q, *c, bf(6, 4, 64), f32(4, 6), *batch, 2, 60, f32(need - 1), 3),
        lambda: fa.fa_fwd_paged_fp8(q, *c, bf(6, 4, 64), f32(4, 6), *batch, 2, 60, None, 3),
        lambda: fa.fa_fwd_paged_fp8(q, *c, None, None, *batch, 2, 60),
    ]
    for call in bad:
        with pytest.raises((TypeError, ValueError)):
            call()
    assert len(stub.calls) == n


def test_binding_window(stub):
    q, k = bf(2, 4, 9, 64), bf(2, 2, 12, 64)
    o, lse = fa.attention_window(q, k, k, 4, 1)
    dq, dk, dv = fa.attention_window_backward(q, k, k, o, lse, o, 4, 1)
    assert (dq.shape, dk.shape, dv.shape) == (q.shape, k.shape, k.shape)
    assert [c[0] for c in stub.calls] == ["fa_fwd_window", "fa_bwd_window"]
    need = fa.fa_bwd_window_workspace_bytes(2, 4, 2, 9, 12, 64, 4, 1) // 4
    ws = torch.zeros(need)
    bad = [
        lambda: fa.attention_window(q, k.float(), k, 4), lambda: fa.attention_window(q, k, k[:, :, :11], 4),
        lambda: fa.attention_window(q, k[:1], k[:1], 4), lambda: fa.attention_window(q.transpose(1, 2), k, k, 4),
        lambda: fa.fa_fwd_window(q, k, k, q, torch.zeros(2, 4, 8), 4),
        lambda: fa.fa_bwd_window(q, k, k, o, o, lse, dq, dq, dv, ws, 4, 1),
        lambda: fa.fa_bwd_window(q, k, k, o, o, lse, dq, dk, dv, ws[1:], 4, 1),
        lambda: fa.fa_bwd_window(q, k, k, o, o, lse.half(), dq, dk, dv, ws, 4, 1),
    ]
    for call in bad:
        with pytest.raises((TypeError, ValueError)):
            call()
    assert len(stub.calls) == 2


def test_the_tensors_device_is_current_during_the_call(monkeypatch):
    """A call on tensors of another device than the current one launches there, on that device's
    stream; a stream of another device is refused."""
    log = []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            log.append(("enter", self.index))

        def __exit__(self, *exc):
            log.append(("exit", self.index))

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(fa, "_raw_stream", lambda index: 100 + index)
    fn = lambda *a: log.append(a) or 0  # noqa: E731
    assert fa._on_stream(0, None, fn, 1, 2) == 0
    assert log == [(1, 2, 100)]
    log.clear()
    fa._on_stream(1, None, fn, 3)
    assert log == [("enter", 1), (3, 101), ("exit", 1)]
    log.clear()

    class Stream:
        cuda_stream = 77
        device = torch.device("cuda", 1)

    fa._on_stream(1, Stream(), fn, 4)
    assert log == [("enter", 1), (4, 77), ("exit", 1)]
    with pytest.raises(ValueError):
        fa._on_stream(0, Stream(), fn, 5)


# ------------------------------------------------------------------- the oracle
def test_oracle_e4m3_matches_torch():
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * s for s in (1e-3, 0.02, 1, 30, 100)])
    x = np.clip(np.concatenate([x, orc.VALUES[:127], (orc.VALUES[:126] + orc.VALUES[1:127]) / 2]), -448, 448)
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn)
    assert np.array_equal(orc.VALUES[orc.encode_e4m3(x)], want.double().numpy())
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(orc.VALUES, codes, equal_nan=True)


def test_oracle_scale_is_the_least_power_of_two():
    for a in (1e-3, 0.875, 7.0, 7.0000005, 448.0, 448.5, 3e38, 1e-35):
        e = orc.block_exponent(a)
        assert a <= 448.0 * 2.0 ** e and (e == orc.E_MIN or a > 448.0 * 2.0 ** (e - 1))
    assert orc.block_exponent(0.0) == orc.E_MIN


def test_oracle_window_matches_the_dense_oracle():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal(s) for s in ((1, 2, 30, 16), (1, 2, 41, 16), (1, 2, 41, 16)))
    for N in (30, 41):
        o, lse = oracle.attention_f64(q[:, :, :N], k, v, 0.25, "bottom_right")
        ow, lw = orc.window_forward(q[:, :, :N], k, v, 0.25, 0, 0)
        assert np.allclose(o, ow, atol=1e-13) and np.allclose(lse, lw, atol=1e-13)
    seen = orc.visible(7, 10, 3, 2)
    for i in range(7):
        for j in range(10):
            p = i + 3
            assert seen[i, j] == (j <= p and (p - j < 3 or j < 2))


def test_oracle_window_gradients_by_differences():
    rng = np.random.default_rng(2)
    args = [rng.standard_normal(s) for s in ((1, 4, 9, 8), (1, 2, 12, 8), (1, 2, 12, 8))]
    do = rng.standard_normal((1, 4, 9, 8))
    grads = orc.window_backward(*args, do, 0.3, 4, 2)
    f = lambda a: (orc.window_forward(*a, 0.3, 4, 2)[0] * do).sum()  # noqa: E731
    for i, g in enumerate(grads):
        step = rng.standard_normal(args[i].shape)
        lo, hi = ([x + s * 1e-5 * step if j == i else x for j, x in enumerate(args)] for s in (-1, 1))
        assert abs((f(hi) - f(lo)) / 2e-5 - (g * step).sum()) < 1e-6


def test_oracle_rotation_is_orthogonal_and_axes_agree():
    rng = np.random.default_rng(3)
    ang = rng.uniform(0, 6, (20, 16))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    x = rng.standard_normal((5, 2, 40))
    pos = rng.integers(0, 20, (3, 5))
    for inter in (False, True):
        y = orc.rotate(x, table, pos, [4, 6, 6], inter)
        assert np.allclose(orc.rotate(y, table, pos, [4, 6, 6], inter, inverse=True), x)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., 32:], x[..., 32:])
        same = np.repeat(pos[:1], 3, 0)
        assert np.array_equal(orc.rotate(x, table, same, [4, 6, 6], inter), orc.rotate(x, table, pos[:1], [16], inter))
