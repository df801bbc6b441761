"""Every kernel variant of the key/value cache against the oracle, bit for bit, at the sizes of fp4_cases.py."""
import numpy as np
import pytest
import torch

import fp4_cases as cases
import oracle
from helpers import BF16, F16, F32, TORCH_DT, dev, rand_x
from test_gpu_kv import FMTS, _bytes, _cache, _oracle_rows, _sync

pytestmark = pytest.mark.gpu

sq = pytest.importorskip("w8a8_post_quantization_calib_b200")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,H,D", [c[:3] for c in cases.KV_WRITES])
def test_write(T, H, D, dt, fmt):
    """Scattered slots, negative ones and ones behind the cache among them; the whole cache is compared."""
    S = 16
    P = -(-T // S) + 2
    r = np.random.default_rng(T + D)
    x = rand_x(T, (T, 2 * H * D + 8), dt, 1.5, outliers=2)          # keys and values in rows of a wider tensor
    x[11] = 0
    slots = r.permutation(P * S)[:T].astype(np.int64)
    out = r.permutation(T)[:60]
    slots[out[:40]], slots[out[40:]] = -1, P * S + np.arange(20)
    slots[T - 1] = -3
    k, v = (dev(x, dt)[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(2))
    cache = _cache(P, S, H, D, fmt)
    before = [_bytes(c) for c in cache]
    sq.kv_cache_write(k, v, dev(slots), fmt, *cache)
    assert sq.sync_status() == 1
    live = (slots >= 0) & (slots < P * S)
    for i in range(2):
        rows, sc, _ = _oracle_rows(np.ascontiguousarray(x[:, i * H * D:(i + 1) * H * D]).reshape(T, H, D), fmt, dt)
        for got, want, full in ((cache[2 * i], rows, before[2 * i]), (cache[2 * i + 1], sc, before[2 * i + 1])):
            full[slots[live]] = want[live]
            assert np.array_equal(_bytes(got), full)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out_dt", [F32, F16])
@pytest.mark.parametrize("rows,H,D", [c[:3] for c in cases.KV_READS])
def test_read(rows, H, D, out_dt, fmt):
    """Sequences of uneven length on scattered pages, from positions inside a page on; a page outside the cache reads
    as zeros and is reported."""
    S, B = 16, 7
    r = np.random.default_rng(rows + H + D)
    cut = np.sort(r.integers(0, rows + 1, B - 1))
    cu = np.concatenate([[0], cut, [rows]]).astype(np.int32)
    lens = np.diff(cu)
    starts = r.integers(0, 40, B).astype(np.int32)
    per = int(-(-(lens + starts).max() // S))
    T = 40 * S                                                       # a small cache: pages are shared
    x = rand_x(D, (T, H, D), F16)
    cache = _cache(40, S, H, D, fmt)
    sq.kv_cache_write(dev(x, F16), dev(x[::-1].copy(), F16), dev(np.arange(T)), fmt, *cache)
    table = r.integers(0, 40, (B, per)).astype(np.int32)
    b = int(lens.argmax())
    table[b, (starts[b] + lens[b] - 1) // S] = 40                    # its last page lies outside
    ko, vo = (torch.full((rows + 3, H, D), 7.0, dtype=TORCH_DT[out_dt], device="cuda") for _ in "kv")
    sq.kv_cache_read(fmt, *cache, dev(table), dev(cu), ko, vo, starts=dev(starts))
    assert sq.sync_status() == 1
    val = _oracle_rows(x, fmt, F16)[2]
    seq = np.repeat(np.arange(B), lens)
    pos = np.arange(rows) - cu[seq] + starts[seq]
    page = table[seq, pos // S]
    slot = np.where(page < 40, page * S + pos % S, 0)
    for o, t in ((ko, val), (vo, val[::-1])):
        want = t[slot].copy()
        want[page >= 40] = 0
        assert torch.equal(o[:rows].cpu(), torch.from_numpy(want).to(TORCH_DT[out_dt]))
        assert torch.all(o[rows:] == 7.0)
    _sync()
