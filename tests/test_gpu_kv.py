"""The quantised key/value cache on the GPU against the oracle: codes, scales and values are bit-exact."""
import numpy as np
import pytest
import torch

import oracle
from helpers import BF16, F16, F32, TORCH_DT, dev, host, mismatch_report, rand_x

pytestmark = pytest.mark.gpu

sq = pytest.importorskip("w8a8_post_quantization_calib_b200")

FMTS = [oracle.KV_INT8, oracle.KV_FP8, oracle.KV_MXFP4]


def _sync():
    assert sq.sync_status() == 0


def _cache(P, S, H, D, fmt, fill=0x5A):
    """k_cache, k_scale, v_cache, v_scale full of a byte."""
    out = []
    for _ in "kv":
        c = torch.full((P, S, H, sq.kv_row_bytes(fmt, D)), fill, dtype=torch.uint8, device="cuda")
        out.append(c.view(torch.int8) if fmt == oracle.KV_INT8 else c)
        b = torch.full((P, S, H, sq.kv_scale_bytes(fmt, D)), fill, dtype=torch.uint8, device="cuda")
        out.append(b if fmt == oracle.KV_MXFP4 else b.view(torch.float32)[..., 0])
    return out


def _bytes(t):
    """A cache tensor as host bytes [slots, H, n]."""
    n = t.shape[0] * t.shape[1]
    return t.contiguous().view(torch.uint8).view(n, t.shape[2], -1).cpu().numpy()


def _oracle_rows(x, fmt, dt):
    """[T, H, D] -> cache bytes [T, H, row bytes], scale bytes [T, H, n], values fp32 [T, H, D]."""
    T, H, D = x.shape
    codes, sc = oracle.kv_quant(x.reshape(T * H, D), fmt, dt)
    v = oracle.kv_values(codes, sc, fmt, D).reshape(T, H, D)
    rb = sq.kv_row_bytes(fmt, D)
    rows = np.zeros((T * H, rb), np.uint8)
    rows[:, :codes.shape[1]] = codes.view(np.uint8)
    return rows.reshape(T, H, rb), np.ascontiguousarray(sc).view(np.uint8).reshape(T, H, -1), v


@pytest.mark.parametrize("H,D", [(1, 1), (3, 16), (2, 31), (8, 64), (5, 80), (7, 100), (8, 128), (32, 128), (1, 192), (2, 256),
                                 (3, 520), (1, 1024)])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", [F32, F16, BF16])
def test_write_and_read(H, D, fmt, dt):
    """Scattered slots of a cache, rows taken out of a fused projection; the whole cache is compared, then read back."""
    T, P, S = 37, 9, 8
    x = rand_x(H * 3 + D + fmt, (T, 3 * H * D), dt, 1.5, outliers=2)
    x[5, H * D:] = 0                                                  # an all-zero token
    xt = dev(x, dt)
    k, v = (xt[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (1, 2))
    slots = np.random.default_rng(D).permutation(P * S)[:T].astype(np.int64)
    slots[7], slots[20] = -1, -5                                      # padding
    cache = _cache(P, S, H, D, fmt)
    before = [_bytes(c) for c in cache]
    sq.kv_cache_write(k, v, dev(slots), fmt, *cache)
    _sync()
    live = slots >= 0
    vals = []
    for i in range(2):
        rows, sc, val = _oracle_rows(x[:, (i + 1) * H * D:(i + 2) * H * D].reshape(T, H, D), fmt, dt)
        for got, want, old in ((cache[2 * i], rows, before[2 * i]), (cache[2 * i + 1], sc, before[2 * i + 1])):
            full = old.copy()
            full[slots[live]] = want[live]
            got = _bytes(got)
            assert np.array_equal(got, full), mismatch_report(got, full)
        vals.append(val)
    # read each live token back as a sequence of its own, with pages of one token
    n = int(live.sum())
    one = [c.reshape(P * S, 1, *c.shape[2:]) for c in cache]
    for out_dt in (F32, F16, BF16):
        ko, vo = (torch.full((n + 2, H, D), 7.0, dtype=TORCH_DT[out_dt], device="cuda") for _ in "kv")
        sq.kv_cache_read(fmt, *one, dev(slots[live].astype(np.int32)[:, None]), dev(np.arange(n + 1, dtype=np.int32)), ko, vo)
        _sync()
        for o, val in ((ko, vals[0]), (vo, vals[1])):
            assert torch.equal(o[:n].cpu(), torch.from_numpy(val[live]).to(TORCH_DT[out_dt]))
            assert torch.all(o[n:] == 7.0)                            # rows behind the last sequence


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("S", [1, 16, 24])
@pytest.mark.parametrize("H,D", [(5, 80), (8, 128), (1, 64), (3, 31), (32, 100), (2, 512), (2, 600)])
def test_ragged_spans(fmt, S, H, D):
    """Uneven sequences, an empty one in front, amid and last; spans that start and end inside a page; rows before
    the first sequence and behind the last stay."""
    lens = [0, 1, 50, 0, 0, 33, 24, 7, 0] + [3] * 40
    starts = [0, 4, 13, 2, 0, 24, 0, 95, 1] + [5] * 40
    B = len(lens)
    T = 102
    pages = -(-T // S)
    P = pages + 3
    cache = _cache(P, S, H, D, fmt)
    x = rand_x(S + D, (T, H, D), F16)
    slots = np.random.default_rng(S).permutation(P)[:pages].astype(np.int32)
    pos = np.arange(T)
    sq.kv_cache_write(dev(x, F16), dev(x, F16), dev(slots[pos // S].astype(np.int64) * S + pos % S), fmt, *cache)
    table = np.full((B, pages + 2), 10 ** 9, np.int32)                # entries behind a sequence are never used
    table[:, :pages] = slots
    cu = (3 + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
    ko, vo = (torch.full((int(cu[-1]) + 5, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    sq.kv_cache_read(fmt, *cache, dev(table), dev(cu), ko, vo, starts=dev(np.array(starts, np.int32)))
    _sync()
    val = torch.from_numpy(_oracle_rows(x, fmt, F16)[2]).to(torch.bfloat16)
    want = torch.full(ko.shape, 7.0, dtype=torch.bfloat16)
    for b in range(B):
        want[cu[b]:cu[b + 1]] = val[starts[b]:starts[b] + lens[b]]
    assert torch.equal(ko.cpu(), want) and torch.equal(vo.cpu(), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_many_sequences(fmt):
    """The search for a row's sequence over thousands of them, most empty."""
    r = np.random.default_rng(9)
    B, S, H, D = 5000, 4, 1, 64
    lens = np.where(r.random(B) < 0.7, 0, r.integers(1, 4, B))
    P = B
    x = rand_x(4, (P * S, H, D), BF16)
    cache = _cache(P, S, H, D, fmt)
    sq.kv_cache_write(dev(x, BF16), dev(x, BF16), dev(np.arange(P * S)), fmt, *cache)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    table = r.permutation(P).astype(np.int32)[:, None]
    ko, vo = (torch.empty(int(cu[-1]), H, D, dtype=torch.float32, device="cuda") for _ in "kv")
    sq.kv_cache_read(fmt, *cache, dev(table), dev(cu), ko, vo)
    _sync()
    val = _oracle_rows(x, fmt, BF16)[2]
    idx = np.concatenate([table[b, 0] * S + np.arange(lens[b]) for b in range(B)])
    assert np.array_equal(host(ko), val[idx]) and np.array_equal(host(vo), val[idx])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", [F32, BF16])
def test_non_finite(fmt, dt):
    """A row (MXFP4: a block) with an infinity or a NaN reads back as NaN; its neighbours are untouched."""
    T, H, D = 6, 2, 96
    clean = rand_x(8, (T, H, D), F32)
    x = clean.copy()
    x[1, 0, 40], x[3, 1, 95], x[4, 0, 0] = np.inf, np.nan, -np.inf
    k = torch.from_numpy(x).cuda().to(TORCH_DT[dt])
    cache = _cache(T, 1, H, D, fmt)
    sq.kv_cache_write(k, k, dev(np.arange(T)), fmt, *cache)
    ko, vo = (torch.empty(T, H, D, dtype=torch.float32, device="cuda") for _ in "kv")
    sq.kv_cache_read(fmt, *cache, dev(np.arange(T, dtype=np.int32)[None]), dev(np.array([0, T], np.int32)), ko, vo)
    _sync()
    hit = np.zeros((T, H, D), bool)
    if fmt == oracle.KV_MXFP4:
        hit[1, 0, 32:64], hit[3, 1, 64:], hit[4, 0, :32] = True, True, True
    else:
        hit[1, 0], hit[3, 1], hit[4, 0] = True, True, True
    c = torch.from_numpy(clean).to(TORCH_DT[dt]).float().numpy()
    want = _oracle_rows(c, fmt, F32)[2]
    for o in (ko, vo):
        o = host(o)
        assert np.array_equal(np.isnan(o), hit)
        assert np.array_equal(o[~hit], want[~hit])


@pytest.mark.parametrize("fmt", FMTS)
def test_indices_outside_the_cache(fmt):
    """Neither written nor read; reported once by sync_status; every other row is right."""
    T, P, S, H, D = 5, 2, 4, 3, 64
    x = rand_x(1, (T, H, D), F16)
    cache = _cache(P, S, H, D, fmt)
    before = [_bytes(c) for c in cache]
    slots = np.array([0, P * S, 7, 1 << 40, 3], np.int64)
    sq.kv_cache_write(dev(x, F16), dev(x, F16), dev(slots), fmt, *cache)
    assert sq.sync_status() == 1
    assert sq.sync_status() == 0
    rows, sc, val = _oracle_rows(x, fmt, F16)
    for i in range(2):
        for got, want, old in ((cache[2 * i], rows, before[2 * i]), (cache[2 * i + 1], sc, before[2 * i + 1])):
            full = old.copy()
            full[[0, 7, 3]] = want[[0, 2, 4]]
            assert np.array_equal(_bytes(got), full)
    # sequence 0: page 0, then a page behind the cache; 1: a negative page; 2: a position behind the table
    table = np.array([[0, P], [-1, 1], [0, 1]], np.int32)
    cu, starts = np.array([0, 8, 10, 12], np.int32), np.array([0, 0, 7], np.int32)
    ko, vo = (torch.full((12, H, D), 7.0, dtype=torch.float32, device="cuda") for _ in "kv")
    sq.kv_cache_read(fmt, *cache, dev(table), dev(cu), ko, vo, starts=dev(starts))
    assert sq.sync_status() == 1
    assert sq.sync_status() == 0
    ko = host(ko)
    assert np.array_equal(ko[0], val[0]) and np.array_equal(ko[3], val[4]) and np.array_equal(ko[10], val[2])
    assert np.all(ko[4:8] == 0) and np.all(ko[8:10] == 0) and np.all(ko[11] == 0)


@pytest.mark.parametrize("fmt", FMTS)
def test_slot_given_twice_leaves_the_others(fmt):
    T, H, D = 64, 2, 64
    x = rand_x(2, (T, H, D), F16)
    slots = np.arange(T)
    slots[10:20] = 5
    cache = _cache(T, 1, H, D, fmt)
    sq.kv_cache_write(dev(x, F16), dev(x, F16), dev(slots), fmt, *cache)
    _sync()
    rows, sc, _ = _oracle_rows(x, fmt, F16)
    once = np.r_[0:5, 6:10, 20:T]
    assert np.array_equal(_bytes(cache[0])[once], rows[once]) and np.array_equal(_bytes(cache[1])[once], sc[once])
    assert np.all(_bytes(cache[0])[10:20] == 0x5A)


@pytest.mark.parametrize("off", [1, 8])
@pytest.mark.parametrize("fmt", FMTS)
def test_unaligned_inputs_and_outputs(fmt, off):
    """Keys and outputs that start off a 16- or 32-byte boundary, values that do not."""
    T, H, D = 20, 4, 64
    x = rand_x(off, (T * H * D + 64,), BF16)
    k = dev(x, BF16)[off:off + T * H * D].view(T, H, D)
    v = dev(x, BF16)[:T * H * D].view(T, H, D)
    cache = _cache(T, 1, H, D, fmt)
    sq.kv_cache_write(k, v, dev(np.arange(T)), fmt, *cache)
    big = [torch.full((T * H * D + 64,), 7.0, dtype=torch.float16, device="cuda") for _ in "kv"]
    ko, vo = big[0][off:off + T * H * D].view(T, H, D), big[1][:T * H * D].view(T, H, D)
    sq.kv_cache_read(fmt, *cache, dev(np.arange(T, dtype=np.int32)[None]), dev(np.array([0, T], np.int32)), ko, vo)
    _sync()
    for o, src in ((ko, x[off:off + T * H * D]), (vo, x[:T * H * D])):
        want = torch.from_numpy(_oracle_rows(src.reshape(T, H, D), fmt, BF16)[2]).to(torch.float16)
        assert torch.equal(o.cpu(), want)
    assert torch.all(big[0][:off] == 7.0) and torch.all(big[0][off + T * H * D:] == 7.0)


@pytest.mark.slow
@pytest.mark.parametrize("fmt", [oracle.KV_INT8, oracle.KV_MXFP4])
def test_offsets_behind_32_bits(fmt):
    """Slots whose bytes lie more than 4 GiB into the cache."""
    S, H, D, T = 64, 8, 128, 130
    per = H * sq.kv_row_bytes(fmt, D)
    P = (1 << 32) // (per * S) + 70
    ck = [torch.empty(P, S, H, sq.kv_row_bytes(fmt, D), dtype=torch.int8 if fmt == oracle.KV_INT8 else torch.uint8, device="cuda")
          for _ in "kv"]
    cs = [torch.empty(P, S, H, 4, dtype=torch.uint8, device="cuda") if fmt == oracle.KV_MXFP4 else
          torch.empty(P, S, H, dtype=torch.float32, device="cuda") for _ in "kv"]
    x = rand_x(7, (T, H, D), BF16)
    pages = np.array([P - 1, 3, P - 2], np.int32)
    pos = np.arange(T)
    args = (fmt, ck[0], cs[0], ck[1], cs[1])
    sq.kv_cache_write(dev(x, BF16), dev(x, BF16), dev(pages[pos // S].astype(np.int64) * S + pos % S), *args)
    ko, vo = (torch.empty(T, H, D, dtype=torch.float32, device="cuda") for _ in "kv")
    sq.kv_cache_read(*args, dev(pages[None]), dev(np.array([0, T], np.int32)), ko, vo)
    _sync()
    want = _oracle_rows(x, fmt, BF16)[2]
    assert np.array_equal(host(ko), want) and np.array_equal(host(vo), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_steps_in_a_graph(fmt):
    """A step (write one token a sequence, read the contexts back) captured once and replayed as the contexts grow."""
    B, S, H, D, steps = 3, 4, 2, 128, 9
    cache = _cache(B * 3, S, H, D, fmt)
    r = np.random.default_rng(5)
    table = r.permutation(B * 3).astype(np.int32).reshape(B, 3)
    x = rand_x(6, (steps, B, H, D), F16)
    k = torch.empty(B, H, D, dtype=torch.float16, device="cuda")
    slots = torch.empty(B, dtype=torch.int64, device="cuda")
    cu = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    ko, vo = (torch.full((B * steps, H, D), 7.0, dtype=torch.float16, device="cuda") for _ in "kv")
    tt = dev(table)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        sq.kv_cache_write(k, k, slots, fmt, *cache)
        sq.kv_cache_read(fmt, *cache, tt, cu, ko, vo)
    val = torch.from_numpy(_oracle_rows(x.reshape(steps * B, H, D), fmt, F16)[2]).to(torch.float16).view(steps, B, H, D)
    for i in range(steps):
        k.copy_(dev(x[i], F16))
        slots.copy_(dev(table[:, i // S].astype(np.int64) * S + i % S))
        cu.copy_(dev((np.arange(B + 1) * (i + 1)).astype(np.int32)))
        graph.replay()
        _sync()
        want = val[:i + 1].transpose(0, 1).reshape(B * (i + 1), H, D)
        assert torch.equal(ko[:B * (i + 1)].cpu(), want) and torch.equal(vo[:B * (i + 1)].cpu(), want)
        assert torch.all(ko[B * (i + 1):] == 7.0)


@pytest.mark.parametrize("fmt", FMTS)
def test_extremes(fmt):
    """Rows of subnormal numbers, of the least and the largest normal ones, of one element beside zeros."""
    D = 64
    x = np.zeros((9, 1, D), np.float32)
    x[0] = np.ldexp(np.float32(1.3), np.linspace(-149, -127, D).astype(int))
    x[1] = 1e-45
    x[2] = np.linspace(-190, 190, D).astype(np.float32) * np.float32(2.0 ** -149)
    x[3] = np.linspace(-1, 1, D).astype(np.float32) * np.float32(2.0 ** -121)
    x[4] = np.linspace(-1, 1, D).astype(np.float32) * np.float32(2.0 ** -126)
    x[5] = np.finfo(np.float32).max * np.linspace(-1, 1, D).astype(np.float32)
    x[6, 0, 63] = -7.25
    x[7, 0, 0], x[7, 0, 1] = -0.0, 3e38
    x[8] = np.ldexp(np.float32(-1.9), np.linspace(-149, 127, D).astype(int))
    cache = _cache(9, 1, 1, D, fmt)
    sq.kv_cache_write(dev(x), dev(x), dev(np.arange(9)), fmt, *cache)
    ko, vo = (torch.empty(9, 1, D, device="cuda") for _ in "kv")
    sq.kv_cache_read(fmt, *cache, dev(np.arange(9, dtype=np.int32)[None]), dev(np.array([0, 9], np.int32)), ko, vo)
    _sync()
    rows, sc, val = _oracle_rows(x, fmt, F32)
    assert np.array_equal(_bytes(cache[0]), rows) and np.array_equal(_bytes(cache[1]), sc)
    assert np.array_equal(host(ko), val) and np.array_equal(host(vo), val)


def test_python_checks():
    fmt = sq.KV_INT8
    c = _cache(2, 4, 3, 64, fmt)
    k = torch.zeros(5, 3, 64, device="cuda")
    slots = torch.arange(5, device="cuda")
    with pytest.raises(ValueError):
        sq.kv_cache_write(k, k[:4], slots, fmt, *c)
    with pytest.raises(ValueError):
        sq.kv_cache_write(k, k, slots.int(), fmt, *c)
    with pytest.raises(ValueError):
        sq.kv_cache_write(k, k, slots, sq.KV_MXFP4, *c)
    with pytest.raises(ValueError):
        sq.kv_cache_write(k.transpose(0, 1).contiguous().transpose(0, 1), k, slots, fmt, *c)
    with pytest.raises(ValueError):
        sq.kv_cache_write(k[:1].expand(5, 3, 64), k, slots, fmt, *c)
    with pytest.raises(ValueError):
        sq.kv_cache_write(k, k, slots.cpu(), fmt, *c)
    table, cu = torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        sq.kv_cache_read(fmt, *c, table, cu[:1], k, k.clone())
    with pytest.raises(ValueError):
        sq.kv_cache_read(fmt, *c, table.long(), cu, k, k.clone())
    with pytest.raises(ValueError):
        sq.kv_cache_read(fmt, *c, table, cu, k, k.half())
    with pytest.raises(ValueError):
        sq.kv_cache_read(fmt, *c[:2], c[2][:1], c[3], table, cu, k, k.clone())
    with pytest.raises(ValueError):
        sq.kv_row_bytes(fmt, 1025)


@pytest.mark.parametrize("fmt", FMTS)
def test_no_pages(fmt):
    """A cache without pages and a table without columns: every index is outside, padding is skipped, rows are zeros."""
    T, H, D = 3, 8, 128
    x = dev(rand_x(3, (T, H, D), F16), F16)
    none = _cache(0, 4, H, D, fmt)
    sq.kv_cache_write(x, x, dev(np.array([-1, -7, -1])), fmt, *none)
    _sync()
    sq.kv_cache_write(x, x, dev(np.array([-1, 0, -1])), fmt, *none)
    assert sq.sync_status() == 1
    some = _cache(2, 4, H, D, fmt)
    sq.kv_cache_write(x, x, dev(np.arange(T)), fmt, *some)
    _sync()
    cu = dev(np.array([1, 1, 3], np.int32))
    for cache, table in ((none, np.zeros((2, 2), np.int32)), (some, np.zeros((2, 0), np.int32)), (none, np.zeros((2, 0), np.int32))):
        ko, vo = (torch.full((5, H, D), 7.0, dtype=torch.float16, device="cuda") for _ in "kv")
        sq.kv_cache_read(fmt, *cache, dev(table), cu, ko, vo)
        assert sq.sync_status() == 1
        for o in (ko, vo):
            assert torch.all(o[1:3] == 0) and torch.all(o[:1] == 7.0) and torch.all(o[3:] == 7.0)
        ko.fill_(7.0)
        sq.kv_cache_read(fmt, *cache, dev(table), cu * 0, ko, vo)          # no rows at all
        _sync()
        assert torch.all(ko == 7.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,D", [(8, 128), (5, 80)])
def test_rows_before_the_output(fmt, H, D):
    """A first row before row 0: the sequence's first positions have no row; positions far outside the table read as zeros."""
    S, T = 4, 24
    x = rand_x(12, (T, H, D), F16)
    cache = _cache(T // S, S, H, D, fmt)
    sq.kv_cache_write(dev(x, F16), dev(x, F16), dev(np.arange(T)), fmt, *cache)
    val = _oracle_rows(x, fmt, F16)[2]
    table = dev(np.arange(T // S, dtype=np.int32)[None].repeat(2, 0))

    def read(cu, starts):
        ko, vo = (torch.full((9, H, D), 7.0, device="cuda") for _ in "kv")
        sq.kv_cache_read(fmt, *cache, table, dev(np.array(cu, np.int32)), ko, vo, starts=dev(np.array(starts, np.int32)))
        assert torch.equal(ko, vo)
        return host(ko)

    o = read([-5, 3, 8], [2, 1])
    _sync()
    assert np.array_equal(o[:3], val[7:10]) and np.array_equal(o[3:8], val[1:6]) and np.all(o[8] == 7.0)
    o = read([-2 ** 31, 2, 6], [2 ** 31 - 1, 2 ** 31 - 1])            # positions around 2^32, and around 2^31
    assert sq.sync_status() == 1
    assert np.all(o[:6] == 0) and np.all(o[6:] == 7.0)
