"""What the binding of the rotation, the paged cache and the window makes of arguments at the edge
of what it takes. CPU only: the library's compute entry points are replaced by stubs that launch
nothing, and CPU tensors stand in for device tensors."""

import pytest

import exact_attention_80_gb300 as fa

torch = pytest.importorskip("torch")


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


WIDE = 2 ** 32 + 5  # 5 in its low 32 bits


def test_numbers_past_32_bits_are_refused(stub):
    """The C interface takes 32-bit ints; a larger number is an error, not its low bits."""
    q, k = bf(1, 4, 9, 64), bf(1, 2, 12, 64)
    o, lse, dq, dk = q.clone(), torch.zeros(1, 4, 9), q.clone(), k.clone()
    ws = torch.zeros(1 << 16)
    t, c, batch = bf(6, 4, 64), cache_args(), [i32(3, 4), i32(4), i32(3)]
    kv = bf(6, 2, 64)
    to, tl = t.clone(), torch.zeros(4, 6)
    calls = [
        lambda n: fa.fa_fwd_window(q, k, k, o, lse, n), lambda n: fa.fa_fwd_window(q, k, k, o, lse, 5, n),
        lambda n: fa.attention_window(q, k, k, n), lambda n: fa.attention_window(q, k, k, 5, n),
        lambda n: fa.attention_window(q, k, k, 5, 1, num_splits=n),
        lambda n: fa.fa_fwd_window_splitkv(q, k, k, ws, n, 5), lambda n: fa.fa_fwd_window_splitkv(q, k, k, ws, 2, n),
        lambda n: fa.fa_bwd_window(q, k, k, o, o, lse, dq, dk, dk, ws, n),
        lambda n: fa.attention_window_backward(q, k, k, o, lse, o, 5, n),
        lambda n: fa.attention_paged_fp8(t, *c, *batch, n, 60), lambda n: fa.attention_paged_fp8(t, *c, *batch, 2, n),
        lambda n: fa.attention_paged_fp8(t, *c, *batch, 2, 60, n),
        lambda n: fa.attention_paged_fp8(t, *c, *batch, 2, 60, 9, n),
        lambda n: fa.attention_paged_fp8(t, *c, *batch, 2, 60, num_splits=n),
        lambda n: fa.fa_fwd_paged_fp8(t, *c, to, tl, *batch, 2, 60, ws, n),
        lambda n: fa.fa_fwd_paged_fp8(t, *c, to, tl, *batch, 2, 60, ws, 2, n),
        lambda n: fa.kv_append_fp8(t, kv, kv, *c, *batch, n), lambda n: fa.fa_kv_append_fp8(None, kv, kv, None, *c, *batch, n),
        lambda n: fa.fa_paged_num_splits(1, 8, 2, 1, n, 64), lambda n: fa.fa_paged_num_splits(1, 8, 2, 1, 99, 64, n),
        lambda n: fa.fa_paged_workspace_bytes(8, 2, 64, n), lambda n: fa.fa_window_num_splits(1, 8, 2, 1, n, 64, 5),
        lambda n: fa.fa_bwd_window_workspace_bytes(1, 8, 2, 10, 10, 64, n),
        lambda n: fa.fa_splitkv_workspace_bytes(1, 1, 1, 64, n), lambda n: fa.fa_fwd_grid_ctas(1, 1, n, 64),
        lambda n: fa.fa_bwd_workspace_bytes(1, 1, n, 64),
        lambda n: fa.fa_fwd_rows(q, q, q, o, lse, n), lambda n: fa.fa_fwd(q, q, q, o, lse, causal=n),
        lambda n: fa.fa_fwd_varlen(t, t, t, to, tl, i32(4), i32(4), n, stream=0),
        lambda n: fa.fa_fwd_splitkv_static(q, q, q, o, lse, n),
    ]
    for i, call in enumerate(calls):
        for n in (WIDE, -WIDE, 2 ** 31):
            with pytest.raises(OverflowError):
                call(n)
                pytest.fail(f"call {i} took {n}")
    assert not stub.calls


def test_positions_of_another_shape_are_refused(stub):
    """Positions belong to tokens by their shape: as many numbers in another order are an error."""
    q, k, table = bf(2, 4, 9, 64), bf(2, 2, 9, 64), torch.zeros(100, 64)
    for shape in ((2, 9), (1, 2, 9), (18,), (1, 18)):  # flat: as one axis lies in memory
        fa.rope(q, k, table, i32(*shape))
    fa.rope(q, k, table, i32(2, 2, 9), sections=(16, 16))
    t, kv, c, batch = bf(6, 4, 64), bf(6, 2, 64), cache_args(), [i32(3, 4), i32(4), i32(3)]
    for shape in ((6,), (1, 6)):
        fa.rope(t, kv, table, i32(*shape))
        fa.kv_append_fp8(t, kv, kv, *c, *batch, 2, table=table, positions=i32(*shape))
    fa.kv_append_fp8(t, kv, kv, *c, *batch, 2, table=table, positions=i32(2, 6), sections=(16, 16))
    n = len(stub.calls)
    assert n == 10
    bad = [lambda s=s: fa.rope(q, k, table, i32(*s)) for s in ((9, 2), (1, 9, 2), (18, 1), (3, 6), (1, 1, 2, 9), (6, 3))]
    bad += [lambda: fa.rope(q, k, table, i32(2, 9, 2), sections=(16, 16)),
            lambda: fa.rope(q, k, table, i32(2, 18), sections=(16, 16))]
    for s in ((2, 3), (1, 6, 1), (3, 2, 1), (1, 1, 6)):
        bad += [lambda s=s: fa.rope(t, kv, table, i32(*s)),
                lambda s=s: fa.kv_append_fp8(t, kv, kv, *c, *batch, 2, table=table, positions=i32(*s))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert len(stub.calls) == n


def test_scales_and_numbers_of_other_types(stub):
    """A scale may be any number that float() takes, as in the dense calls; an int any that is one."""
    np = pytest.importorskip("numpy")
    q, k = bf(1, 4, 9, 64), bf(1, 2, 12, 64)
    o, lse, ws = q.clone(), torch.zeros(1, 4, 9), torch.zeros(1 << 16)
    t, c, batch = bf(6, 4, 64), cache_args(), [i32(3, 4), i32(4), i32(3)]
    for scale in (0.25, np.float32(0.25), np.float64(0.25), torch.tensor(0.25), 1):
        for n in (5, np.int64(5), np.int32(5)):
            fa.fa_fwd_window(q, k, k, o, lse, n, scale=scale)
            fa.fa_fwd_window_splitkv(q, k, k, ws, 2, n, scale=scale)
            fa.attention_window(q, k, k, n, scale=scale)
            fa.attention_window_backward(q, k, k, o, lse, o, n, scale=scale)
            fa.attention_paged_fp8(t, *c, *batch, 2, 60, n, scale=scale)
        for _, args in stub.calls:
            assert sum(type(a) is float and a == float(scale) for a in args) == 1
        stub.calls.clear()
    for call in (lambda: fa.attention_window(q, k, k, 5, scale="0.25x"), lambda: fa.attention_window(q, k, k, 5, scale=[1])):
        with pytest.raises((TypeError, ValueError)):
            call()
