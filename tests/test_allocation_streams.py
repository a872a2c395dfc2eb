"""The calls that allocate their outputs, on a stream other than the current one: what they allocate may
lie in memory that the current stream still uses, and the workspace that they give back may be handed out
on the current stream while theirs still runs."""

import math

import pytest

torch = pytest.importorskip("torch")

import exact_attention_80_gb300 as fa  # noqa: E402

pytestmark = pytest.mark.gpu

B, H, Hkv, N, d = 1, 16, 4, 2048, 128


def normal(*shape, seed=1):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def calls():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    fa.load_library()
    q, k, v = normal(B, H, N, d), normal(B, Hkv, N, d, seed=2), normal(B, Hkv, N, d, seed=3)
    kf, vf = normal(B, H, N, d, seed=4), normal(B, H, N, d, seed=5)
    q8, k8, v8 = (x.to(torch.float8_e4m3fn) for x in (q, kf, vf))
    o, lse = fa.attention_window(q, k, v, 300)
    of, lf = fa.attention(q, kf, vf)
    table, pos = torch.rand(N, d, device="cuda"), torch.arange(N, dtype=torch.int32, device="cuda")[None]
    packed, pk, pv = (x[0].transpose(0, 1).contiguous() for x in (q, k, v))
    cache = [torch.zeros((N // 64, Hkv, 64, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.ones((N // 64, Hkv), device="cuda") for _ in range(2)]
    batch = (torch.arange(N // 64, dtype=torch.int32, device="cuda")[None], i32([0, N]), i32([N]))
    fa.kv_append_fp8(None, pk, pv, *cache, *batch, N)
    scratch = [x.clone() for x in cache]
    torch.cuda.synchronize()
    return {
        "rope": lambda s: fa.rope(q, k, table, pos, stream=s),
        "append": lambda s: fa.kv_append_fp8(packed, pk, pv, *scratch, *batch, N, table=table, stream=s),
        "paged": lambda s: fa.attention_paged_fp8(packed, *cache, *batch, N, N, num_splits=1, stream=s),
        "paged splits": lambda s: fa.attention_paged_fp8(packed, *cache, *batch, N, N, num_splits=3, stream=s),
        "window": lambda s: fa.attention_window(q, k, v, 300, num_splits=1, stream=s),
        "window splits": lambda s: fa.attention_window(q, k, v, 300, num_splits=3, stream=s),
        "window backward": lambda s: fa.attention_window_backward(q, k, v, o, lse, o, 300, stream=s),
        "dense": lambda s: fa.attention(q, kf, vf, stream=s),
        "dense splits": lambda s: fa.attention(q, kf, vf, num_splits=3, stream=s),
        "dense backward": lambda s: fa.attention_backward(q, kf, vf, of, lf, of, stream=s),
        "varlen": lambda s: fa.attention_varlen(packed, packed, packed, batch[1], batch[1], N, stream=s),
        "e4m3": lambda s: fa.attention_fp8(q8, k8, v8, stream=s),
        "e4m3 splits": lambda s: fa.attention_fp8(q8, k8, v8, num_splits=3, stream=s),
    }


NAMES = ["rope", "append", "paged", "paged splits", "window", "window splits", "window backward", "dense", "dense splits",
         "dense backward", "varlen", "e4m3", "e4m3 splits"]


def tensors(out):
    return [x for x in (out if isinstance(out, tuple) else (out,)) if x is not None]


def same(name, got, want):
    for i, (x, y) in enumerate(zip(tensors(got), tensors(want))):
        if "backward" in name and i == 0:  # (dQ is summed by atomics)
            assert (x.float() - y.float()).abs().max() <= 2.0 ** -7 * y.float().abs().max(), name
        else:
            assert torch.equal(x, y), name


@pytest.fixture(scope="module")
def busy():
    """Some twenty milliseconds of work on the current stream."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    a, b = normal(8192, 8192), torch.empty((8192, 8192), dtype=torch.bfloat16, device="cuda")
    a.mul_(0.01)
    torch.mm(a, a, out=b)
    torch.cuda.synchronize()

    def run():
        for _ in range(30):
            torch.mm(a, a, out=b)

    return run


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_reads(calls, busy, name, handle):
    """Tensors of the outputs' sizes are copied by the current stream later on and given back at once; the call
    on the other stream, which runs first, leaves the copies alone."""
    want = calls[name](None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    calls[name](side)  # warm-up
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full_like(x, 3.0) for x in tensors(want)]
    torch.cuda.synchronize()
    busy()
    copies = [x.clone() for x in held]
    del held
    got = calls[name](side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_OK
    for x in copies:
        assert torch.all(x == 3.0), name
    same(name, got, want)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_workspaces_last_until_their_stream_has_passed(calls, busy, name, handle):
    """The other stream is behind: memory that the call gave back is not handed out on the current stream."""
    want = calls[name](None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        busy()
    got = calls[name](side.cuda_stream if handle else side)
    junk = [torch.full((1 << n,), math.nan, device="cuda") for n in range(16, 27) for _ in range(2)]
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_OK
    same(name, got, want)
    assert all(torch.isnan(x).all() for x in junk), name


@pytest.mark.parametrize("name", NAMES)
def test_the_default_stream_by_its_handle(calls, busy, name):
    """Handle 0 is the default stream: the call's memory is that stream's, whatever the current one still reads."""
    want = calls[name](None)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        held = [torch.full_like(x, 3.0) for x in tensors(want)]
        torch.cuda.synchronize()
        busy()
        copies = [x.clone() for x in held]
        del held
        got = calls[name](0)
        with torch.cuda.stream(torch.cuda.default_stream()):
            # Memory of the default stream's that the call gave back follows it in order.
            junk = [torch.full((1 << n,), math.nan, device="cuda") for n in range(16, 27)]
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_OK
    assert all(torch.all(x == 3.0) for x in copies) and all(torch.isnan(x).all() for x in junk)
    same(name, got, want)


@pytest.mark.parametrize("name", ["rope", "paged splits", "window splits", "window backward", "dense splits"])
def test_captured_on_a_forked_stream(calls, name):
    """A capture that forks to another stream: what the call allocates there belongs to the graph."""
    want = calls[name](None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    calls[name](side)  # warm-up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = calls[name](side)
        here.wait_stream(side)
        again = calls[name](here)
    junk = [torch.full((1 << n,), math.nan, device="cuda") for n in range(16, 26)]
    for _ in range(2):
        for x in (*tensors(got), *tensors(again)):
            x.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_device_status(clear=True) == fa.FA_OK
        same(name, got, want)
        same(name, again, want)
    assert all(torch.isnan(x).all() for x in junk)
