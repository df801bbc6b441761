"""The layer drivers on a stream that is not the current one: nothing is read before it is made, and no memory is given
away while either stream still uses it.  Results are compared bit for bit with the same calls on the current stream."""
import pytest
import torch

from helpers import BF16, dev, rand_x

pytestmark = pytest.mark.gpu

sq = pytest.importorskip("w8a8_post_quantization_calib_b200")
layer = pytest.importorskip("w8a8_post_quantization_calib_b200.layer")

K, N, M = 520, 384, 40
SLEEP = 20_000_000                       # clock cycles: about 10 ms

MAKE = {
    "int8": lambda w, a, **kw: layer.QuantizedLinear.from_float(w, a, mode=sq.ACT_PER_TOKEN, **kw),
    "int8 static": lambda w, a, **kw: layer.QuantizedLinear.from_float(w, a, **kw),
    "mxfp4": lambda w, a, **kw: layer.QuantizedLinearFp4.from_float(w, a, fmt=sq.MXFP4, **kw),
    "nvfp4": lambda w, a, **kw: layer.QuantizedLinearFp4.from_float(w, a, fmt=sq.NVFP4, **kw),
}


def _k(kind):
    return 512 if kind.startswith("int8") else K            # INT8 rows are whole 16-byte vectors


def _inputs(k, seed=1):
    return dev(rand_x(seed, (N, k), BF16, 0.03), BF16), dev(rand_x(seed + 1, (200, k), BF16, 1.5, outliers=3), BF16)


def _tensors(lin):
    return {n: t for n, t in vars(lin).items() if isinstance(t, torch.Tensor)}


def _spoil(*sizes):
    """Buffers of these many bytes on the current stream, filled with NaNs' bytes."""
    return [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(6)]


def _forms(st):
    return {"stream": st, "external": torch.cuda.ExternalStream(st.cuda_stream), "address": st.cuda_stream}


@pytest.mark.parametrize("form", ["stream", "external", "address"])
@pytest.mark.parametrize("kind", MAKE)
def test_from_float(kind, form):
    k = _k(kind)
    w, x = _inputs(k)
    c = layer.Calibrator(k)
    c.add_batch(x)
    want = _tensors(MAKE[kind](w, c.act_max))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [4 * k, 4 * N, N * k, 2 * N * k, 2 * 200 * k]
    _spoil(*sizes)                                          # what new buffers hold before they are filled
    with torch.cuda.stream(st):
        _spoil(*sizes)
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)                                # the weight and the batch are made behind this
    w2, x2 = w.clone(), x.clone()
    c2 = layer.Calibrator(k)
    c2.add_batch(x2, stream=_forms(st)[form])
    got = MAKE[kind](w2, c2.act_max, stream=_forms(st)[form])
    del w2, x2, c2
    spoilt = _spoil(*sizes)
    torch.cuda.synchronize()
    assert sq.sync_status(st) == 0
    for n, t in _tensors(got).items():
        if n in ("x_sf", "w_sf"):                           # rows behind the last of a scale tile are not written
            continue
        assert torch.equal(t, want[n]), n
    y, r = got.forward(x), MAKE[kind](w, c.act_max).forward(x)
    assert sq.sync_status() == 0 and torch.equal(y, r)
    del spoilt


@pytest.mark.parametrize("form", ["stream", "external", "address"])
@pytest.mark.parametrize("kind", MAKE)
def test_forward(kind, form):
    k = _k(kind)
    w, x = _inputs(k)
    c = layer.Calibrator(k)
    c.add_batch(x)
    lin = MAKE[kind](w, c.act_max)
    x = x[:M].contiguous()
    want = lin.forward(x)
    st, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    sizes = [M * k, M * k // 2, M * k * 2, M * N * 2, 4 * M, 512 * 5, 512 * 9]
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    x2 = x.clone()
    with torch.cuda.stream(st):
        torch.cuda._sleep(4 * SLEEP)                        # the call's work is behind this
    y = lin.forward(x2, stream=_forms(st)[form])
    del x2
    spoilt = _spoil(*sizes)                                 # done before the call's work begins
    cur.wait_stream(st)
    torch.cuda._sleep(4 * SLEEP)
    z = y.clone()                                           # reads the result behind this
    del y
    with torch.cuda.stream(st):
        spoilt += _spoil(*sizes)
    torch.cuda.synchronize()
    assert sq.sync_status() == 0
    assert torch.equal(z, want)


@pytest.mark.parametrize("fmt", [sq.KV_INT8, sq.KV_FP8, sq.KV_MXFP4])
@pytest.mark.parametrize("form", ["stream", "external", "address"])
def test_cache(fmt, form):
    T, H, D, S = 30, 4, 96, 8
    k = dev(rand_x(3, (T, H, D), BF16), BF16)
    slots = torch.arange(T, device="cuda").flip(0).contiguous()
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")

    def run(stream):
        cache = layer.PagedKVCache(4, S, H, D, fmt)
        k2, s2 = k.clone(), slots.clone()
        cache.write(k2, k2, s2, stream=stream)
        del k2, s2
        ko, vo = (torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        cache.read(table.clone(), cu.clone(), ko, vo, stream=stream)
        return cache, ko, vo

    _, k_want, v_want = run(None)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    with torch.cuda.stream(st):
        torch.cuda._sleep(4 * SLEEP)
    cache, ko, vo = run(_forms(st)[form])
    spoilt = _spoil(T * H * D * 2, 8 * T, 512)
    torch.cuda.synchronize()
    assert sq.sync_status(st) == 0
    assert torch.equal(ko, k_want) and torch.equal(vo, v_want)
    del spoilt, cache


def test_a_stream_under_capture():
    """A call on a stream that captures a graph, made while another one is current, is captured."""
    T, H, D = 6, 2, 64
    cache = layer.PagedKVCache(T, 1, H, D, sq.KV_INT8)
    k = dev(rand_x(4, (T, H, D), BF16), BF16)
    slots = torch.arange(T, device="cuda")
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        graph.capture_begin()
    cache.write(k, k, slots, stream=st)
    with torch.cuda.stream(st):
        graph.capture_end()
    assert not cache.k.any()
    graph.replay()
    other = layer.PagedKVCache(T, 1, H, D, sq.KV_INT8)
    other.write(k, k, slots)
    assert sq.sync_status() == 0
    assert torch.equal(cache.k, other.k) and torch.equal(cache.v_scale, other.v_scale)


@pytest.mark.parametrize("kind", MAKE)
def test_a_stream_forked_inside_a_capture(kind):
    """Calls on a second stream while the current one captures: both end up in the graph."""
    k = _k(kind)
    w, x = _inputs(k)
    c = layer.Calibrator(k)
    c.add_batch(x)
    lin = MAKE[kind](w, c.act_max)
    a, b = x[:M].clone(), x[M:2 * M].clone()
    st, side, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    lin.forward(a)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        ya, yb = lin.forward(a), lin.forward(b, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for seed in (7, 8):
        fresh = dev(rand_x(seed, (2 * M, k), BF16, 1.5), BF16)
        a.copy_(fresh[:M])
        b.copy_(fresh[M:])
        graph.replay()
        assert torch.equal(ya, lin.forward(a)) and torch.equal(yb, lin.forward(b))
    assert sq.sync_status() == 0


@pytest.mark.parametrize("kind", MAKE)
def test_the_default_stream_from_another_one(kind):
    k = _k(kind)
    w, x = _inputs(k)
    c = layer.Calibrator(k)
    c.add_batch(x)
    lin = MAKE[kind](w, c.act_max)
    want = lin.forward(x)
    torch.cuda.synchronize()
    for stream in (0, torch.cuda.default_stream()):
        with torch.cuda.stream(torch.cuda.Stream()):
            torch.cuda._sleep(SLEEP)
            x2 = x.clone()
            y = lin.forward(x2, stream=stream)
            del x2
            spoilt = _spoil(2 * x.numel())
        torch.cuda.synchronize()
        assert sq.sync_status() == 0
        assert torch.equal(y, want)
        del spoilt


@pytest.mark.parametrize("kind", MAKE)
def test_refusals_leave_the_current_stream(kind):
    """A tensor that is not on a GPU is refused as without stream=, and the caller's stream is the current one again."""
    k = _k(kind)
    w, x = _inputs(k)
    c = layer.Calibrator(k)
    c.add_batch(x)
    lin = MAKE[kind](w, c.act_max)
    st, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    calls = [lambda: lin.forward(x.cpu(), stream=st), lambda: lin.forward(x[:, :k - 8], stream=st),
             lambda: MAKE[kind](w.cpu(), c.act_max, stream=st), lambda: c.add_batch(x.cpu(), stream=st)]
    for call in calls:
        with pytest.raises((TypeError, ValueError, sq.SQError)):
            call()
        assert torch.cuda.current_stream() == cur
    cache = layer.PagedKVCache(2, 4, 2, 64)
    kv = torch.zeros(3, 2, 64, device="cuda")
    with pytest.raises(TypeError):
        cache.write(kv, kv, torch.arange(3), stream=st)
    with pytest.raises(TypeError):
        cache.write(kv, kv, None, stream=st)
    assert torch.cuda.current_stream() == cur and sq.sync_status() == 0


def test_a_stream_of_another_device_is_refused():
    """Not made the current one: the kernels would run on its device, which cannot reach the tensors."""
    class Other(torch.cuda.Stream):
        device = torch.device("cuda", 1)

    w, x = _inputs(K)
    c = layer.Calibrator(K)
    c.add_batch(x)
    lin = MAKE["mxfp4"](w, c.act_max)
    for call in (lambda: lin.forward(x, stream=Other()), lambda: c.add_batch(x, stream=Other())):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    assert sq.sync_status() == 0
