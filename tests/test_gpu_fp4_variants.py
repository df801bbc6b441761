"""Every kernel variant of the 4-bit formats against the oracle, at the sizes of fp4_cases.py (test_fp4_plans.py checks
that each size reaches its variant).  Quantisation and values are bit-exact; products are held to test_gpu_fp4's bound."""
import numpy as np
import pytest
import torch

import fp4_cases as cases
import oracle
from helpers import BF16, F16, F32, TORCH_DT, dev, rand_x
from test_fp4_plans import linear
from test_gpu_fp4 import _buffers, _check_packed, _product, _s, _sync

pytestmark = pytest.mark.gpu

sq = pytest.importorskip("w8a8_post_quantization_calib_b200")

MX, NV = oracle.MXFP4, oracle.NVFP4


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt,rows,K,pad", [c[:4] for c in cases.QUANT])
def test_quant(dt, rows, K, pad, fmt):
    """Activations with s and g; contiguous rows as a weight as well."""
    x = rand_x(rows + K, (rows, K + pad), dt, 1.5, outliers=5)
    x[7, 3:5] = 0
    s = _s(K, rows)
    for weight in (False, True) if pad == 0 else (False,):
        top = oracle.to_f32(x[:, :K], dt) * (s if weight else 1 / s)
        g = np.array([np.abs(top).max() / 2688], np.float32)
        q, sf = _buffers(rows, K, fmt)
        if weight:
            sq.quant_weight_fp4(dev(x, dt), dev(s), fmt, q, sf, g=dev(g))
        else:
            sq.smooth_quant_act_fp4(dev(x, dt)[:, :K], dev(s), fmt, q, sf, g=dev(g))
        _sync()
        _check_packed(q, sf, *oracle.quant_fp4(x[:, :K], fmt, s, weight, g if fmt == NV else None, dt))


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt,rows,K", [c[:3] for c in cases.VALUES])
def test_values(dt, rows, K, fmt):
    r = np.random.default_rng(rows + K)
    n = -(-K // 32) * 32 // oracle.fp4_block(fmt)
    codes = r.integers(0, 16, (rows, n * oracle.fp4_block(fmt)), dtype=np.uint8)
    sb = (r.integers(100, 140, (rows, n)) if fmt == MX else r.integers(0, 127, (rows, n))).astype(np.uint8)
    sb[rows - 1, 0], sb[64, n - 1] = (255, 0) if fmt == MX else (127, 1)
    g = np.array([0.37], np.float32)
    out = torch.full((rows + 1, K), 7.0, dtype=TORCH_DT[dt], device="cuda")
    sq.dequant_fp4(dev(oracle.fp4_pack(codes)), dev(oracle.fp4_tile_scales(sb, 0xEE)), fmt, out[:rows], g=dev(g))
    _sync()
    want = torch.from_numpy(oracle.fp4_values(codes, sb, fmt, g if fmt == NV else None)[:, :K].copy()).to(TORCH_DT[dt])
    assert torch.equal(torch.nan_to_num(out[:rows].cpu(), nan=777.0), torch.nan_to_num(want, nan=777.0))
    assert torch.all(out[rows] == 7.0)


# ------------------------------------------------------------------ product
@pytest.mark.parametrize("M,N,K", [s for shapes in cases.LINEAR_SWAP.values() for s in shapes])
@pytest.mark.parametrize("fmt", [MX, NV])
def test_linear_weights_as_a(M, N, K, fmt):
    assert linear(M, N, K)[0] == 0
    _product(M, N, K, fmt, [F32, F16, BF16][(M + N + fmt) % 3], bias=(M + fmt) % 2 == 0, off=N % 2)


# every output type with and without bias; aligned rows leave by TMA stores, those off 16 bytes (odd N, or y one element
# further) by plain ones.  Which scale format a kernel is for does not enter its epilogue: the types are dealt out.
PAIR_OUTPUTS = {
    MX: [(0, BF16, True, 0), (0, F32, False, 0), (0, F16, True, 0), (0, F32, True, 1), (1, BF16, False, 0), (1, F16, True, 0)],
    NV: [(0, F16, False, 0), (0, F32, True, 0), (0, BF16, False, 0), (0, BF16, False, 1), (1, F32, True, 0), (1, F16, False, 3)],
}


@pytest.mark.parametrize("bn", cases.LINEAR_PAIRS)
@pytest.mark.parametrize("fmt,which,out_dt,bias,off", [(f, *c) for f, l in PAIR_OUTPUTS.items() for c in l])
def test_linear_pairs(bn, fmt, which, out_dt, bias, off):
    """Three tiles a CTA pair: both accumulators (that share columns at 256) and the first one again."""
    M, N, K = cases.LINEAR_PAIRS[bn][which]
    assert linear(M, N, K) == (1, bn, 2)
    _product(M, N, K, fmt, out_dt, bias, off=off)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_linear_pairs_with_rings_that_wrap_inside_a_tile(fmt):
    M, N, K = cases.LINEAR_PAIRS[256][2]
    assert linear(M, N, K) == (1, 256, 2)
    _product(M, N, K, fmt, BF16, True)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("bn", cases.LINEAR_PAIRS)
def test_linear_pairs_nan_scale_reaches_its_rows_only(bn, fmt):
    """A block with an infinity makes its token's (and its channel's) outputs NaN, and no others."""
    M, N, K = cases.LINEAR_PAIRS[bn][0]
    x, w = rand_x(1, (M, K), F32), rand_x(2, (N, K), F32)
    x[300 % M, 100], w[N - 77, K - 1], w[200, 0] = np.inf, np.nan, -np.inf
    ops = []
    for t, f in ((x, sq.smooth_quant_act_fp4), (w, sq.quant_weight_fp4)):
        q, sf = _buffers(t.shape[0], K, fmt)
        f(dev(t), None, fmt, q, sf)
        ops += [q, sf]
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    sq.linear_fp4(*ops, fmt, y)
    _sync()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[300 % M], want[:, N - 77], want[:, 200] = True, True, True
    assert torch.equal(torch.isnan(y).cpu(), want)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("M,N,K,bn", [(300, 8000, 1000, 256), (300, 7000, 300, 192), (385, 4096, 1500, 128)])
def test_withheld_stage_of_a_pair_times_out_and_context_survives(M, N, K, bn, fmt):
    """Failure detection: the bounded waits of all roles give up, the status says so once, the next product is right."""
    assert linear(M, N, K) == (1, bn, 2)
    q, sf = _buffers(M, K, fmt, 0)
    wq, wsf = _buffers(N, K, fmt, 0)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    _sync()
    sq.set_wait_timeout_ns(20_000_000)
    sq.lib().sq_debug_inject(1)
    try:
        sq.linear_fp4(q, sf, wq, wsf, fmt, y)
        assert sq.sync_status() == 5
        assert sq.sync_status() == 0
    finally:
        sq.lib().sq_debug_inject(0)
        sq.set_wait_timeout_ns(0)
    _product(M, N, K, fmt, BF16, False)


@pytest.mark.parametrize("bn,cs", [v for v in cases.LINEAR_SWAP if v[1] > 1])
def test_withheld_stage_of_a_cluster_times_out_and_context_survives(bn, cs):
    """The CTA without its stage and those that wait for its partial sums give up; the next product is right."""
    M, N, K = cases.LINEAR_SWAP[bn, cs][0]
    assert linear(M, N, K) == (0, bn, cs)
    q, sf = _buffers(M, K, NV, 0)
    wq, wsf = _buffers(N, K, NV, 0)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    _sync()
    sq.set_wait_timeout_ns(20_000_000)
    sq.lib().sq_debug_inject(1)
    try:
        sq.linear_fp4(q, sf, wq, wsf, NV, y)
        assert sq.sync_status() == 5
        assert sq.sync_status() == 0
    finally:
        sq.lib().sq_debug_inject(0)
        sq.set_wait_timeout_ns(0)
    _product(M, N, K, NV, BF16, False)


@pytest.mark.parametrize("bn", cases.LINEAR_PAIRS)
def test_linear_pairs_in_a_graph_and_on_two_streams(bn):
    """Replayed, and side by side on two streams: the bits of a call alone."""
    M, N, K = cases.LINEAR_PAIRS[bn][0]
    r = np.random.default_rng(bn)
    ops = []
    for rows in (M, N):
        ops += [dev(r.integers(0, 256, (rows, sq.fp4_code_bytes(K))).astype(np.uint8)),
                dev(r.integers(20, 60, sq.fp4_scale_bytes(NV, rows, K)).astype(np.uint8))]
    want, y = (torch.empty(M, N, device="cuda") for _ in range(2))
    sq.linear_fp4(*ops, NV, want)
    _sync()
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        sq.linear_fp4(*ops, NV, y)
    for _ in range(3):
        y.fill_(7.0)
        graph.replay()
        _sync()
        assert torch.equal(y, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty(M, N, device="cuda") for _ in range(3)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(3):
        for s, o in zip(streams, outs):
            sq.linear_fp4(*ops, NV, o[i], stream=s)
    torch.cuda.synchronize()
    _sync()
    assert all(torch.equal(o, want) for ys in outs for o in ys)
