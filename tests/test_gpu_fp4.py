"""4-bit microscaled formats on the GPU against the oracle.

Quantisation: codes and scale bytes are bit-exact.  Values: bit-exact.  Product: every product of two codes and two
block scales is exact in fp32 (at most 3 + 3 significant bits of the codes, 4 + 4 of NVFP4's scales), so y differs
from the exact fp64 product by the summation (K additions, each off by at most one unit in the last place, 2^-23 of a
partial sum that never exceeds sum |x w|) and the epilogue's roundings (the factor, the multiply-add, the output).
"""
import numpy as np
import pytest
import torch

import oracle
from helpers import BF16, F16, F32, TORCH_DT, dev, host, mismatch_report, rand_x

pytestmark = pytest.mark.gpu

sq = pytest.importorskip("w8a8_post_quantization_calib_b200")

MX, NV = oracle.MXFP4, oracle.NVFP4
HALF_STEP = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F32: 2.0 ** -149, F16: 2.0 ** -24, BF16: 2.0 ** -133}          # least step of the output type


def _sync():
    assert sq.sync_status() == 0


def _buffers(rows, K, fmt, fill=0xEE):
    return (torch.full((rows, sq.fp4_code_bytes(K)), fill, dtype=torch.uint8, device="cuda"),
            torch.full((sq.fp4_scale_bytes(fmt, rows, K),), fill, dtype=torch.uint8, device="cuda"))


def _check_packed(q, sf, codes, sb, nan=None):
    """Codes and scales on the device against the oracle's; nan: blocks whose codes are not specified."""
    got, want = host(q), oracle.fp4_pack(codes)
    if nan is not None:
        keep = np.repeat(~nan, codes.shape[1] // nan.shape[1] // 2, axis=1)
        got, want = got[keep], want[keep]
    assert np.array_equal(got, want), mismatch_report(got, want)
    rows, n = sb.shape
    t = host(sf)
    idx = oracle.fp4_scale_index(rows, -(-n // 4) * 4)
    want = oracle.fp4_tile_scales(sb)[idx]
    assert np.array_equal(t[idx], want), mismatch_report(t[idx], want)
    rest = np.ones(t.size, bool)
    rest[idx] = False
    assert np.all(t[rest] == 0xEE)                                      # rows behind the last are not written


def _s(K, seed):
    return (np.abs(np.random.default_rng(seed).standard_normal(K)) * 3 + 0.05).astype(np.float32)


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 4096), (3, 31), (7, 33), (129, 500), (300, 1000), (130, 2064), (1000, 128)])
@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("weight", [False, True])
def test_quant(rows, K, dt, fmt, weight):
    x = rand_x(rows * 7 + K + dt, (rows, K), dt, 0.02 if weight else 2.0, outliers=max(1, K // 200))
    s = _s(K, K + rows)
    top = oracle.to_f32(x, dt) * (s if weight else 1 / s)
    g = np.array([np.abs(top).max() / 2688], np.float32)
    q, sf = _buffers(rows, K, fmt)
    f = sq.quant_weight_fp4 if weight else sq.smooth_quant_act_fp4
    f(dev(x, dt), dev(s), fmt, q, sf, g=dev(g))
    _sync()
    codes, sb = oracle.quant_fp4(x, fmt, s, weight, g if fmt == NV else None, dt)
    _check_packed(q, sf, codes, sb)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("pad,off", [(24, 0), (7, 0), (5, 3), (16, 8), (1, 0), (1, 1), (2, 2), (3, 1), (4, 4), (6, 5), (9, 7)])
@pytest.mark.parametrize("rows,K", [(70, 600), (1, 517), (3, 15), (40, 1025)])
def test_quant_rows_of_a_wider_tensor(fmt, dt, pad, off, rows, K):
    """Any row stride and any start: the loads narrow to what the addresses allow; no s, no g."""
    x = rand_x(pad + off, (rows, K + pad), dt, 1.0)
    q, sf = _buffers(rows, K, fmt)
    sq.smooth_quant_act_fp4(dev(x, dt)[:, off:off + K], None, fmt, q, sf)
    _sync()
    _check_packed(q, sf, *oracle.quant_fp4(x[:, off:off + K], fmt, dt=dt))


@pytest.mark.parametrize("fmt", [MX, NV])
def test_quant_extremes(fmt):
    """Ties, zeros of both signs, subnormals, the largest finite numbers, infinities, NaN; s of 0 and of the least number."""
    K = 160
    x = np.zeros((12, K), np.float32)
    x[0] = np.tile(np.array([6, .25, -.75, 1.25, 1.75, 2.5, -3.5, 5, 0, -0.0, .5, .74, .76, 1.24, 1.26, -6], np.float32), 10)
    x[1] = np.ldexp(np.float32(1.7), np.linspace(-149, 127, K).astype(int))
    x[2] = np.finfo(np.float32).max
    x[3] = -1e-42
    x[4] = 1.0
    x[4, 37], x[4, 80] = np.inf, np.nan
    x[5] = rand_x(1, (1, K), F32, 1e-38)[0]
    x[6] = rand_x(2, (1, K), F32, 1e30)[0]
    x[7:] = rand_x(3, (5, K), F32)
    for s in (None, np.ones(K, np.float32)):
        if s is not None:
            s[3], s[40], s[41] = 0.0, 1e-45, np.float32(np.finfo(np.float32).max)
        for g in (None, np.array([1e-3], np.float32), np.array([0.0], np.float32), np.array([1e38], np.float32)):
            if g is not None and fmt == MX:
                continue
            for weight in (False, True):
                q, sf = _buffers(12, K, fmt)
                f = sq.quant_weight_fp4 if weight else sq.smooth_quant_act_fp4
                f(dev(x), None if s is None else dev(s), fmt, q, sf, g=None if g is None else dev(g))
                _sync()
                codes, sb = oracle.quant_fp4(x, fmt, s, weight, g)
                _check_packed(q, sf, codes, sb, nan=(sb == (255 if fmt == MX else 127)))


@pytest.mark.parametrize("K,alpha", [(1, 0.5), (500, 0.25), (4096, 0.5), (11008, 1.0)])
def test_smooth_scales_nvfp4(K, alpha):
    g = np.random.default_rng(K)
    am = (np.abs(g.standard_normal(K)) * 2).astype(np.float32)
    wm = (np.abs(g.standard_normal(K)) * 0.05).astype(np.float32)
    am[K // 2] = 0
    s, s2, ga, gw = (torch.empty(n, dtype=torch.float32, device="cuda") for n in (K, K, 1, 1))
    sq.smooth_scales_nvfp4(dev(am), dev(wm), alpha, s, ga, gw)
    sq.smooth_scales(dev(am), dev(wm), alpha, s2)
    _sync()
    assert torch.equal(s, s2)
    sh = host(s)
    want_a = np.float32((am * oracle.recip_finite32(sh)).astype(np.float32).max() / np.float32(2688))
    want_w = np.float32((wm * sh).astype(np.float32).max() / np.float32(2688))
    assert host(ga)[0] == want_a and host(gw)[0] == want_w


# ------------------------------------------------------------------ values
@pytest.mark.parametrize("rows,K", [(1, 1), (5, 33), (200, 500), (129, 4096), (64, 1000)])
@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("fmt", [MX, NV])
def test_dequant(rows, K, dt, fmt):
    r = np.random.default_rng(rows + K)
    n = -(-K // 32) * 32 // oracle.fp4_block(fmt)
    codes = r.integers(0, 16, (rows, n * oracle.fp4_block(fmt)))
    sb = r.integers(100, 140, (rows, n)) if fmt == MX else r.integers(0, 127, (rows, n))
    if rows > 4:
        sb[3, 0], sb[4, 0] = (255, 0) if fmt == MX else (127, 1)
    g = np.array([0.37], np.float32)
    out = torch.full((rows + 1, K), 7.0, dtype=TORCH_DT[dt], device="cuda")
    sq.dequant_fp4(dev(oracle.fp4_pack(codes)), dev(oracle.fp4_tile_scales(sb.astype(np.uint8), 0xEE)), fmt, out[:rows], g=dev(g))
    _sync()
    v = oracle.fp4_values(codes, sb, fmt, g if fmt == NV else None)[:, :K]
    want = torch.from_numpy(v.copy()).to(TORCH_DT[dt])
    assert torch.equal(torch.nan_to_num(out[:rows].cpu(), nan=777.0), torch.nan_to_num(want, nan=777.0))
    assert torch.all(out[rows] == 7.0)


@pytest.mark.parametrize("off", range(8))
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 515), (9, 1027), (5, 511), (2, 1024), (33, 17)])
@pytest.mark.parametrize("dt", [F32, F16, BF16])
def test_dequant_to_any_address(off, rows, K, dt):
    """Outputs that start and whose rows end anywhere; what lies around them stays."""
    r = np.random.default_rng(off + K)
    n = -(-K // 32) * 32 // 16
    codes, sb = r.integers(0, 16, (rows, n * 16)), r.integers(1, 100, (rows, n)).astype(np.uint8)
    full = torch.full((rows * K + 32,), 7.0, dtype=TORCH_DT[dt], device="cuda")
    sq.dequant_fp4(dev(oracle.fp4_pack(codes)), dev(oracle.fp4_tile_scales(sb, 0xEE)), NV, full[off:off + rows * K].view(rows, K))
    _sync()
    want = torch.full(full.shape, 7.0, dtype=TORCH_DT[dt])
    want[off:off + rows * K] = torch.from_numpy(oracle.fp4_values(codes, sb, NV)[:, :K].copy()).flatten().to(TORCH_DT[dt])
    assert torch.equal(full.cpu(), want)


# ------------------------------------------------------------------ product
def _product(M, N, K, fmt, out_dt, bias, seed=0, off=0, stream=None):
    r = np.random.default_rng(seed + M + 3 * N + 5 * K)
    n, B = -(-K // 32) * 32 // oracle.fp4_block(fmt), oracle.fp4_block(fmt)

    def operand(rows):
        c = r.integers(0, 16, (rows, n * B))
        c[:, K:] = 0
        sb = r.integers(122, 130, (rows, n)) if fmt == MX else r.integers(1, 100, (rows, n))
        return c, sb.astype(np.uint8)

    xc, xs = operand(M)
    wc, ws = operand(N)
    ga, gw = (np.array([v], np.float32) for v in (0.013, 0.7))
    b = rand_x(seed + N, (N,), out_dt, 3.0) if bias else None
    full = torch.full((M * N + 64 + off,), 7.0, dtype=TORCH_DT[out_dt], device="cuda")
    y = full[off:off + M * N].view(M, N)
    # rows behind the last of a scale tile hold the NaN scale: they must not reach any output
    sq.linear_fp4(dev(oracle.fp4_pack(xc)), dev(oracle.fp4_tile_scales(xs, 0xFF)), dev(oracle.fp4_pack(wc)),
                  dev(oracle.fp4_tile_scales(ws, 0xFF)), fmt, y, bias=None if b is None else dev(b, out_dt), g_act=dev(ga),
                  g_w=dev(gw), stream=stream)
    assert sq.sync_status(stream) == 0
    xv, wv = oracle.fp4_values(xc, xs, fmt, f32=False), oracle.fp4_values(wc, ws, fmt, f32=False)
    f = float(np.float32(ga[0] * gw[0])) if fmt == NV else 1.0
    acc = xv @ wv.T
    S = np.abs(xv) @ np.abs(wv).T
    ref = acc * f + (0.0 if b is None else oracle.to_f32(b, out_dt).astype(np.float64)[None, :])
    got = y.double().cpu().numpy()
    calc = f * S * K * 2.0 ** -23 + (np.abs(acc * f) + np.abs(ref)) * 2.0 ** -23
    tol = calc + (np.abs(ref) + calc) * HALF_STEP[out_dt] + TINY[out_dt]
    if out_dt == F16:                                   # beyond fp16's range the output is infinite
        fits = np.abs(ref) + tol < 65504
        got, ref, tol = got[fits], ref[fits], tol[fits]
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), mismatch_report(np.where(bad, got, 0), np.where(bad, ref, 0))
    assert torch.all(full[:off] == 7.0) and torch.all(full[off + M * N:] == 7.0)


SHAPES = [(1, 1, 1), (1, 128, 64), (1, 4096, 4096), (2, 130, 33), (16, 512, 256), (17, 300, 1000), (33, 1024, 2048),
          (64, 520, 11008), (65, 129, 500), (100, 4096, 2080), (128, 20000, 512),
          (129, 256, 256), (129, 1, 31), (200, 130, 1000), (256, 512, 4096), (300, 777, 2064), (512, 1152, 512),
          (1000, 3000, 96), (2048, 2304, 1024), (257, 8192, 160)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fmt", [MX, NV])
def test_linear(M, N, K, fmt):
    _product(M, N, K, fmt, BF16, bias=(M + N) % 2 == 0)


@pytest.mark.parametrize("M,N,K", [(5, 264, 500), (100, 1024, 1024), (300, 528, 1040), (700, 777, 512)])
@pytest.mark.parametrize("out_dt", [F32, F16, BF16])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("off", [0, 1])
def test_linear_outputs(M, N, K, out_dt, bias, off):
    """Every output type with and without bias, at aligned and odd addresses."""
    for fmt in (MX, NV):
        _product(M, N, K, fmt, out_dt, bias, off=off)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_linear_without_cluster_split(fmt):
    sq.lib().sq_debug_inject(2)
    try:
        _product(33, 512, 4096, fmt, F16, True)
        _product(7, 130, 1000, fmt, F16, True)
    finally:
        sq.lib().sq_debug_inject(0)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("M", [9, 300])
def test_linear_nan_scale_reaches_its_rows_only(M, fmt):
    """A block with an infinity makes its token's (and its channel's) outputs NaN, and no others."""
    K, N = 512, 256
    x, w = rand_x(1, (M, K), F32), rand_x(2, (N, K), F32)
    x[5, 100], w[77, 300] = np.inf, np.nan
    ops = []
    for t, f in ((x, sq.smooth_quant_act_fp4), (w, sq.quant_weight_fp4)):
        q, sf = _buffers(t.shape[0], K, fmt)
        f(dev(t), None, fmt, q, sf)
        ops += [q, sf]
    y = torch.empty(M, N, dtype=torch.float32, device="cuda")
    sq.linear_fp4(*ops, fmt, y)
    _sync()
    bad = torch.isnan(y).cpu().numpy()
    want = np.zeros((M, N), bool)
    want[5], want[:, 77] = True, True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("M,N,K", [(16, 512, 1024), (8, 8192, 512), (300, 768, 1024)])
def test_withheld_stage_times_out_and_context_survives(M, N, K):
    """Failure detection: the bounded waits give up, the status says so once, and the next product is right."""
    assert sq.sync_status() == 0
    sq.set_wait_timeout_ns(20_000_000)
    sq.lib().sq_debug_inject(1)
    try:
        q, sf = _buffers(M, K, MX, 0)
        wq, wsf = _buffers(N, K, MX, 0)
        sq.linear_fp4(q, sf, wq, wsf, MX, torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
        assert sq.sync_status() == 5
        assert sq.sync_status() == 0
    finally:
        sq.lib().sq_debug_inject(0)
        sq.set_wait_timeout_ns(0)
    _product(M, N, K, MX, BF16, False)


# ------------------------------------------------------------------ use
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("M", [4, 200])
def test_layer_in_a_graph_on_another_stream(fmt, M):
    """Quantise and multiply captured on a stream, replayed with new inputs: the same bits as eager calls."""
    K, N = 1000, 384
    w = dev(rand_x(3, (N, K), F16, 0.02), F16)
    s = dev(_s(K, 4))
    ga, gw = dev(np.array([0.01], np.float32)), dev(np.array([1e-4], np.float32))
    wq, wsf = _buffers(N, K, fmt)
    sq.quant_weight_fp4(w, s, fmt, wq, wsf, g=gw)
    x = torch.empty(M, K, dtype=torch.float16, device="cuda")
    q, sf = _buffers(M, K, fmt)
    y = torch.empty(M, N, dtype=torch.float16, device="cuda")

    def step():
        sq.smooth_quant_act_fp4(x, s, fmt, q, sf, g=ga)
        sq.linear_fp4(q, sf, wq, wsf, fmt, y, g_act=ga, g_w=gw)

    inputs = [dev(rand_x(50 + i, (M, K), F16, 2.0), F16) for i in range(3)]
    want = []
    for t in inputs:
        x.copy_(t)
        step()
        want.append(y.clone())
    _sync()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    for t, r in zip(inputs, want):
        x.copy_(t)
        y.fill_(7.0)
        graph.replay()
        _sync()
        assert torch.equal(y, r)
    # eager on a created stream: programmatic dependent launches back to back
    with torch.cuda.stream(st):
        for t, r in zip(inputs * 5, want * 5):
            x.copy_(t)
            step()
            assert torch.equal(y, r)
    _sync()


@pytest.mark.parametrize("M,N,K", [(33, 512, 8192), (100, 1024, 11008), (300, 512, 4096), (700, 4096, 1024)])
def test_two_streams_at_once_and_repeats(M, N, K):
    """Calls on two streams side by side, and again, give the bits of a call alone (sums in a fixed order)."""
    r = np.random.default_rng(M)
    ops = []
    for rows in (M, N):
        q = dev(r.integers(0, 256, (rows, K // 2)).astype(np.uint8))
        ops += [q, dev(r.integers(20, 60, sq.fp4_scale_bytes(NV, rows, K)).astype(np.uint8))]
    want = torch.empty(M, N, device="cuda")
    sq.linear_fp4(*ops, NV, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty(M, N, device="cuda") for _ in range(6)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(6):
        for st, o in zip(streams, outs):
            sq.linear_fp4(*ops, NV, o[i], stream=st)
    torch.cuda.synchronize()
    _sync()
    assert all(torch.equal(o, want) for ys in outs for o in ys)


def test_timeout_is_not_hidden_by_a_bad_index():
    """Both records of the device are kept: the timeout is reported first, then neither."""
    assert sq.sync_status() == 0
    c = torch.zeros(1, 1, 1, 16, dtype=torch.int8, device="cuda")
    s = torch.zeros(1, 1, 1, device="cuda")
    k = torch.zeros(1, 1, 16, device="cuda")
    sq.kv_cache_write(k, k, torch.tensor([5], device="cuda"), sq.KV_INT8, c, s, c.clone(), s.clone())
    sq.set_wait_timeout_ns(20_000_000)
    sq.lib().sq_debug_inject(1)
    try:
        q, sf = _buffers(4, 512, MX, 0)
        sq.linear_fp4(q, sf, q, sf, MX, torch.empty(4, 4, dtype=torch.bfloat16, device="cuda"))
        assert sq.sync_status() == 5
        assert sq.sync_status() == 0
    finally:
        sq.lib().sq_debug_inject(0)
        sq.set_wait_timeout_ns(0)


def test_python_checks():
    q, sf = _buffers(4, 64, MX)
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError):
        sq.smooth_quant_act_fp4(x, None, MX, q[:3], sf)
    with pytest.raises(ValueError):
        sq.smooth_quant_act_fp4(x, None, MX, q, sf[:100])
    with pytest.raises(TypeError):
        sq.smooth_quant_act_fp4(x, x.double()[0], MX, q, sf)
    with pytest.raises(TypeError):
        sq.smooth_quant_act_fp4(x.to(torch.int32), None, MX, q, sf)
    with pytest.raises(ValueError):
        sq.smooth_quant_act_fp4(x.cpu(), None, MX, q, sf)
    with pytest.raises(ValueError):
        sq.smooth_quant_act_fp4(x.t()[:4], None, MX, *_buffers(4, 4, MX))
    with pytest.raises(ValueError):
        sq.quant_weight_fp4(x[:, :32], None, MX, *_buffers(4, 32, MX))
    with pytest.raises(ValueError):
        sq.linear_fp4(q, sf, q, sf, MX, torch.empty(4, 5, device="cuda"))
    with pytest.raises(ValueError):
        sq.linear_fp4(q, sf, q, sf, MX, torch.empty(4, 4, device="cuda"), bias=torch.zeros(4, dtype=torch.float16, device="cuda"))
    with pytest.raises(sq.SQError):
        sq.linear_fp4(q, sf, q, torch.zeros(2048, dtype=torch.uint8, device="cuda")[1:1025], MX,
                      torch.empty(4, 4, device="cuda"))
