"""Every kernel variant of the 4-bit formats and of the key/value cache has a case in fp4_cases.py (no GPU needed: the
rules are host arithmetic, and without a GPU they take the SM count of a B200)."""
import ctypes

import pytest

import fp4_cases as cases
from helpers import F32

sq = pytest.importorskip("w8a8_post_quantization_calib_b200")

ELT = {F32: 4}


def _plan(call, n, *args):
    plan = (ctypes.c_int * n)()
    assert getattr(sq.lib(), call)(*args, plan) == 0
    return tuple(plan)


def linear(M, N, K):
    return _plan("sq_debug_linear_fp4_plan", 3, M, N, K)


def access(dt, ld):
    return 32 if ld * ELT.get(dt, 2) % 32 == 0 else 16 if ld * ELT.get(dt, 2) % 16 == 0 else 0


def test_products_with_the_weights_as_a():
    assert set(cases.LINEAR_SWAP) == {(bn, cs) for bn in (16, 32, 64, 128) for cs in (1, 2, 4, 8)}
    for (bn, cs), shapes in cases.LINEAR_SWAP.items():
        for s in shapes:
            assert linear(*s) == (0, bn, cs), s
        if bn >= 64 and cs > 1:
            assert any(s[0] > 128 for s in shapes)


def test_products_with_cta_pairs():
    assert set(cases.LINEAR_PAIRS) == {256, 192, 128}
    for bn, shapes in cases.LINEAR_PAIRS.items():
        for M, N, K in shapes:
            assert linear(M, N, K) == (1, bn, 2), (M, N, K)
            assert -(-M // 256) * -(-N // bn) > 2 * 74              # a third tile: both accumulators, and the first again
        assert shapes[0][1] % 8 == 0 and shapes[1][1] % 8 != 0


def test_rows():
    seen = set()
    for dt, rows, K, pad, vec, per_thread, walk in cases.QUANT:
        assert access(dt, K + pad) == vec
        for fmt in (sq.MXFP4, sq.NVFP4):
            p = _plan("sq_debug_rows_fp4_plan", 2, 0, fmt, dt, vec, rows, K)
            assert p[0] == per_thread and p[1] >= walk, (dt, rows, K, p)
        seen.add((dt == F32, vec, per_thread))
    four = [c for c in cases.QUANT if c[5] == 4]
    assert seen >= {(f32, vec, 4) for f32 in (False, True) for vec in (16, 32)} | {(f32, 0, 1) for f32 in (False, True)}
    assert {c[1] % 128 for c in four} >= {0, 1, 9, 33, 127}
    seen = set()
    for dt, rows, K, vec, per_thread, walk in cases.VALUES:
        assert access(dt, K) == vec
        for fmt in (sq.MXFP4, sq.NVFP4):
            p = _plan("sq_debug_rows_fp4_plan", 2, 1, fmt, dt, vec, rows, K)
            assert p[0] == per_thread and p[1] >= walk, (dt, rows, K, p)
        seen.add((dt == F32, vec, per_thread))
    assert seen >= {(f32, vec, 4) for f32 in (False, True) for vec in (16, 32)} | {(f32, 0, 1) for f32 in (False, True)}


def test_cache():
    for T, H, D, steps, chunks in cases.KV_WRITES:
        assert _plan("sq_debug_kv_plan", 4, T, H, D)[:2] == (steps, chunks), (T, H, D)
    for rows, H, D, warps in cases.KV_READS:
        assert _plan("sq_debug_kv_plan", 4, rows, H, D)[2:] == (int(warps == 0), warps), (rows, H, D)


def test_plans_refuse_bad_sizes():
    plan = (ctypes.c_int * 4)()
    L = sq.lib()
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (-1, 1, 1)):
        assert L.sq_debug_linear_fp4_plan(*bad, plan) == 1
        assert L.sq_debug_kv_plan(*bad, plan) == 1
    for rows, K in ((0, 1), (1, 0), (-1, 1)):
        assert L.sq_debug_rows_fp4_plan(0, 0, 0, 16, rows, K, plan) == 1
    assert L.sq_debug_linear_fp4_plan(1, 1, 1, None) == 1 and L.sq_debug_kv_plan(1, 1, 1, None) == 1
    assert L.sq_debug_rows_fp4_plan(0, 2, 0, 16, 1, 1, plan) == 1 and L.sq_debug_rows_fp4_plan(0, 0, 3, 16, 1, 1, plan) == 1
    assert L.sq_debug_kv_plan(1, 1, 1025, plan) == 2
