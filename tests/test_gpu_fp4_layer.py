"""The 4-bit layer and the key/value cache as a program uses them: calibrate, quantise a fused query/key/value projection,
run tokens through it, write keys and values into pages, read the contexts back."""
import numpy as np
import pytest
import torch

import oracle
from helpers import BF16, F16, dev, host, rand_x

pytestmark = pytest.mark.gpu

sq = pytest.importorskip("w8a8_post_quantization_calib_b200")
layer = pytest.importorskip("w8a8_post_quantization_calib_b200.layer")

H, D, K = 4, 96, 520
N = 3 * H * D


def _layer(fmt, seed, bias):
    calib = [rand_x(seed + i, (200, K), BF16, 1.5, outliers=3) for i in range(2)]
    w = rand_x(seed + 9, (N, K), BF16, 0.03)
    c = layer.Calibrator(K)
    for x in calib:
        c.add_batch(dev(x, BF16))
    b = dev(rand_x(seed + 11, (N,), BF16, 0.5), BF16) if bias else None
    return layer.QuantizedLinearFp4.from_float(dev(w, BF16), c.act_max, fmt=fmt, bias=b), w, c


def _exact(lin, w, x, b):
    """y in fp64 from the oracle's codes with the layer's own factors, and the bound of the summation's error."""
    s = host(lin.s)
    ga, gw = (None, None) if lin.g_act is None else (host(lin.g_act), host(lin.g_w))
    xv = oracle.fp4_values(*oracle.quant_fp4(x, lin.fmt, s, False, ga, BF16), lin.fmt, f32=False)
    wv = oracle.fp4_values(*oracle.quant_fp4(w, lin.fmt, s, True, gw, BF16), lin.fmt, f32=False)
    f = 1.0 if ga is None else float(np.float32(ga[0] * gw[0]))
    y = xv @ wv.T * f + (0.0 if b is None else b[None, :])
    return y, f * (np.abs(xv) @ np.abs(wv).T) * K * 2.0 ** -23 + (np.abs(y) + np.abs(xv @ wv.T * f)) * 2.0 ** -23


@pytest.mark.parametrize("fmt", [sq.MXFP4, sq.NVFP4])
@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("bias", [False, True])
def test_projection_into_the_cache_and_back(fmt, T, bias):
    lin, w, c = _layer(fmt, T, bias)
    x = rand_x(77 + T, (T, K), BF16, 1.5, outliers=3)
    qkv = lin.forward(dev(x, BF16))
    assert sq.sync_status() == 0
    b = None if lin.bias is None else lin.bias.double().cpu().numpy()
    ref, calc = _exact(lin, w, x, b)
    got = qkv.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= calc + (np.abs(ref) + calc) * 2.0 ** -8)        # bf16: half a step
    for kv in (sq.KV_INT8, sq.KV_FP8, sq.KV_MXFP4):
        S, pages = 16, -(-T // 16)
        cache = layer.PagedKVCache(pages + 2, S, H, D, kv)
        order = np.random.default_rng(T).permutation(pages + 2)[:pages].astype(np.int32)
        pos = np.arange(T)
        k, v = (qkv[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (1, 2))
        cache.write(k, v, dev(order[pos // S].astype(np.int64) * S + pos % S))
        ko, vo = (torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        cache.read(dev(order[None]), dev(np.array([0, T], np.int32)), ko, vo)
        assert sq.sync_status() == 0
        for o, t in ((ko, k), (vo, v)):
            rows = t.float().cpu().numpy().reshape(T * H, D)
            want = oracle.kv_values(*oracle.kv_quant(rows, kv), kv, D).reshape(T, H, D)
            assert torch.equal(o.cpu(), torch.from_numpy(want).to(torch.bfloat16))


def test_layers_share_a_stream_and_a_graph():
    """Two layers behind one another in one graph, replayed: the bits of eager calls."""
    a, _, _ = _layer(sq.NVFP4, 5, True)
    bw = dev(rand_x(6, (K, N), F16, 0.02), F16)
    c = layer.Calibrator(N)
    x = torch.empty(17, K, dtype=torch.bfloat16, device="cuda")
    x.copy_(dev(rand_x(1, (17, K), BF16, 1.0), BF16))
    c.add_batch(a.forward(x))
    b = layer.QuantizedLinearFp4.from_float(bw, c.act_max, fmt=sq.MXFP4)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        y = b.forward(a.forward(x))
    for seed in (2, 3):
        x.copy_(dev(rand_x(seed, (17, K), BF16, 1.0), BF16))
        graph.replay()
        want = b.forward(a.forward(x))
        assert sq.sync_status() == 0
        assert torch.equal(y, want)


def test_no_tokens():
    lin, _, _ = _layer(sq.MXFP4, 3, False)
    assert lin.forward(torch.empty(0, K, dtype=torch.bfloat16, device="cuda")).shape == (0, N)
    cache = layer.PagedKVCache(2, 4, H, D, sq.KV_FP8)
    none = torch.empty(0, H, D, dtype=torch.bfloat16, device="cuda")
    cache.write(none, none, torch.empty(0, dtype=torch.int64, device="cuda"))
    cache.read(torch.empty(0, 3, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), none, none.clone())
    assert sq.sync_status() == 0
