"""The oracle of the 4-bit formats and of the quantised key/value cache, pinned by the formats' definitions (no GPU)."""
import numpy as np
import pytest
import torch

import oracle
import synth
import w8a8_post_quantization_calib_b200 as sq
from helpers import F16, F32, rand_x

EPS4 = 2.0 ** -2                      # E2M1 has one mantissa bit: half a step is a quarter of a value's power of two


def test_e2m1_nearest_ties_to_even():
    pos = oracle.E2M1_POS
    for c in range(8):
        assert oracle.e2m1_encode(np.float32(pos[c])) == c
        assert oracle.e2m1_encode(np.float32(-pos[c])) == c | 8
    for c in range(7):
        mid = np.float32((pos[c] + pos[c + 1]) / 2)
        assert oracle.e2m1_encode(mid) == (c if c % 2 == 0 else c + 1)
        assert oracle.e2m1_encode(np.nextafter(mid, np.float32(0))) == c
        assert oracle.e2m1_encode(np.nextafter(mid, np.float32(9))) == c + 1
    assert oracle.e2m1_encode(np.float32(1e30)) == 7 and oracle.e2m1_encode(np.float32(-np.inf)) == 15
    assert np.array_equal(oracle.e2m1_decode(np.arange(16)), np.concatenate([pos, -pos]))


@pytest.mark.parametrize("m,byte", [(1.0, 125), (6.0, 127), (7.9, 127), (8.0, 128), (0.0, 0), (2.0 ** -126, 0), (2.0 ** -125, 0),
                                    (2.0 ** -124, 1), (3.0e38, 252), (1e-45, 0)])
def test_mxfp4_scale_is_the_power_of_two_two_below_the_maximum(m, byte):
    """OCP Microscaling Formats v1.0: the shared exponent is floor(log2 max) - 2, held at -127."""
    x = np.zeros((1, 32), np.float32)
    x[0, 7] = m
    codes, sf = oracle.quant_fp4(x, oracle.MXFP4)
    assert sf[0, 0] == byte
    v = oracle.fp4_values(codes, sf, oracle.MXFP4)[0, 7]
    if m >= 2.0 ** -127:
        assert abs(v - np.float32(m)) <= EPS4 * m          # saturation at 6 of [4, 8) is at most a quarter too


@pytest.mark.parametrize("fmt", [oracle.MXFP4, oracle.NVFP4])
@pytest.mark.parametrize("K", [1, 31, 48, 500])
def test_quant_round_trip_error(fmt, K):
    """Half a step of E2M1 at most, and half a step of the scale: E4M3 2^-4 relative (MXFP4: saturation, a quarter)."""
    x = rand_x(K, (9, K), F32, 2.0)
    g = np.array([np.abs(x).max() / 2688], np.float32)
    codes, sf = oracle.quant_fp4(x, fmt, g=g if fmt == oracle.NVFP4 else None)
    v = oracle.fp4_values(codes, sf, fmt, g)[:, :K].astype(np.float64)
    B = oracle.fp4_block(fmt)
    pad = np.zeros((9, codes.shape[1]))
    pad[:, :K] = np.abs(x)
    m = np.repeat(pad.reshape(9, -1, B).max(axis=2), B, axis=1)[:, :K]
    # the widest step is 2 of 6 (half: a sixth of the block's maximum); with the rounded scale 6 may fall short by 2^-4
    bound = m * (0.25 if fmt == oracle.MXFP4 else 1 / 6 * (1 + 2.0 ** -4) + 2.0 ** -4)
    assert np.all(np.abs(v - x) <= bound * (1 + 1e-6))
    assert np.all(codes[:, K:] & 7 == 0)


def test_non_finite_blocks_read_back_as_nan():
    for bad in (np.inf, -np.inf, np.nan):
        for fmt in (oracle.MXFP4, oracle.NVFP4):
            x = np.ones((2, 64), np.float32)
            x[1, 40] = bad
            v = oracle.fp4_values(*oracle.quant_fp4(x, fmt), fmt)
            B = oracle.fp4_block(fmt)
            hit = np.zeros((2, 64), bool)
            hit[1, 40 // B * B:40 // B * B + B] = True
            assert np.array_equal(np.isnan(v), hit)


@pytest.mark.parametrize("fmt", [oracle.MXFP4, oracle.NVFP4])
@pytest.mark.parametrize("rows,K", [(1, 1), (128, 64), (129, 65), (300, 1000), (5, 4096)])
def test_layout_sizes_and_bijection(fmt, rows, K):
    n = -(-K // 32) * 32 // oracle.fp4_block(fmt)
    size = oracle.fp4_scale_size(rows, n)
    assert sq.fp4_scale_bytes(fmt, rows, K) == size
    assert sq.fp4_code_bytes(K) == -(-K // 32) * 16 == int(sq.lib().sq_fp4_code_bytes(K))
    i = oracle.fp4_scale_index(rows, n)
    assert len(np.unique(i)) == i.size and i.min() >= 0 and i.max() < size
    g = np.random.default_rng(rows + K)
    c = g.integers(0, 16, (rows, 2 * sq.fp4_code_bytes(K)))
    assert np.array_equal(oracle.fp4_unpack(oracle.fp4_pack(c)), c)
    sf = g.integers(0, 256, (rows, n)).astype(np.uint8)
    assert np.array_equal(oracle.fp4_tile_scales(sf)[i], sf)


@pytest.mark.parametrize("fmt", [oracle.KV_INT8, oracle.KV_FP8, oracle.KV_MXFP4])
def test_kv_round_trip_error(fmt):
    x = rand_x(3, (50, 100), F16, 1.5)
    x[7] = 0
    f = oracle.to_f32(x, F16).astype(np.float64)
    v = oracle.kv_values(*oracle.kv_quant(x, fmt, F16), fmt, 100)
    m = np.abs(f).max(axis=1, keepdims=True)
    # half a step: 1/254 of the maximum; E4M3 2^-4 relative (or half its least step); E2M1 a quarter of the block's
    tol = {oracle.KV_INT8: m / 254, oracle.KV_FP8: np.abs(f) * 2.0 ** -4 + m / 448 * 2.0 ** -10,
           oracle.KV_MXFP4: m * 0.25}[fmt] * (1 + 1e-5)
    assert np.all(np.abs(v - f) <= tol)
    assert np.all(v[7] == 0)


def test_e4m3_of_the_cache_is_torchs():
    x = rand_x(5, (4, 64), F32, 3.0)
    codes, a = oracle.kv_quant(x, oracle.KV_FP8)
    t = torch.from_numpy((x * oracle.recip_finite32(a)[:, None]).astype(np.float32)).clamp(-448, 448)
    assert np.array_equal(t.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), codes)


# ---------------------------------------------------------------- refusals, before any CUDA call
_A, _U = 16, 17


@pytest.mark.parametrize("fn,args,status", [
    ("sq_smooth_scales_nvfp4", (_A, _A, 64, 1.5, _A, _A, _A, None), 1),
    ("sq_quant_weight_fp4", (None, 1, 8, 64, _A, 0, None, _A, _A, None), 1),
    ("sq_quant_weight_fp4", (_A, 1, 8, 64, _A, 2, None, _A, _A, None), 1),            # unknown format
    ("sq_quant_weight_fp4", (_A, 5, 8, 64, _A, 0, None, _A, _A, None), 1),
    ("sq_quant_weight_fp4", (_A, 1, 8, 0, _A, 0, None, _A, _A, None), 1),
    ("sq_quant_weight_fp4", (_A, 1, 8, 64, _A, 0, None, _A, _U, None), 3),
    ("sq_quant_weight_fp4", (_U, 1, 8, 64, _A, 0, None, _A, _A, None), 3),            # off its type's alignment
    ("sq_quant_weight_fp4", (_A, 1, 0, 64, _A, 0, None, _A, _A, None), 0),
    ("sq_smooth_quant_act_fp4", (_A, 1, 4, 64, 63, _A, 0, None, _A, _A, None), 1),    # ld < K
    ("sq_smooth_quant_act_fp4", (_A, 1, -1, 64, 64, _A, 0, None, _A, _A, None), 1),
    ("sq_smooth_quant_act_fp4", (_A, 1, 4, 1 << 31, 1 << 31, _A, 0, None, _A, _A, None), 2),
    ("sq_smooth_quant_act_fp4", (_A, 1, 0, 64, 64, _A, 0, None, _A, _A, None), 0),
    ("sq_dequant_fp4", (_A, _A, 0, 4, 64, None, 3, _A, None), 1),
    ("sq_dequant_fp4", (_U, _A, 0, 4, 64, None, 1, _A, None), 3),
    ("sq_dequant_fp4", (_A, _A, 0, 0, 64, None, 1, _A, None), 0),
    ("sq_linear_fp4", (_A, _A, _A, None, 0, 4, 32, 64, None, None, None, 1, _A, None), 1),
    ("sq_linear_fp4", (_A, _A, _A, _A, 0, 4, 0, 64, None, None, None, 1, _A, None), 1),
    ("sq_linear_fp4", (_A, _A, _A, _A, 7, 4, 32, 64, None, None, None, 1, _A, None), 1),
    ("sq_linear_fp4", (_A, _U, _A, _A, 0, 4, 32, 64, None, None, None, 1, _A, None), 3),
    ("sq_linear_fp4", (_A, _A, _A, _A, 0, 4, 32, 64, None, None, _U, 1, _A, None), 3),
    ("sq_linear_fp4", (_A, _A, _A, _A, 0, 4, 32, 1 << 31, None, None, None, 1, _A, None), 2),
    ("sq_linear_fp4", (_A, _A, _A, _A, 0, 0, 32, 64, None, None, None, 1, _A, None), 0),
    ("sq_kv_cache_write", (_A, _A, 1, 4, 2, 64, 127, 128, _A, 0, 64, _A, _A, _A, _A, None), 1),     # tokens overlap
    ("sq_kv_cache_write", (_A, _A, 1, 4, 2, 64, 128, 128, _A, 3, 64, _A, _A, _A, _A, None), 1),     # unknown format
    ("sq_kv_cache_write", (_A, _A, 1, 4, 2, 1025, 4096, 4096, _A, 0, 64, _A, _A, _A, _A, None), 2),
    ("sq_kv_cache_write", (_A, _A, 1, 4, 2, 64, 128, 128, 12, 0, 64, _A, _A, _A, _A, None), 3),
    ("sq_kv_cache_write", (_A, _A, 1, 4, 2, 64, 128, 128, _A, 0, 64, _U, _A, _A, _A, None), 3),
    ("sq_kv_cache_write", (_A, _A, 1, 0, 2, 64, 128, 128, _A, 0, 64, _A, _A, _A, _A, None), 0),
    ("sq_kv_cache_read", (0, _A, _A, _A, _A, 4, 0, 2, 64, _A, 1, 4, _A, None, 8, 1, _A, _A, None), 1),    # page size 0
    ("sq_kv_cache_read", (0, _A, _A, _A, _A, 4, 16, 2, 64, None, 1, 4, _A, None, 8, 1, _A, _A, None), 1),
    ("sq_kv_cache_read", (0, _A, _A, _A, _A, 4, 16, 2, 64, _A, 1, 4, 18, None, 8, 1, _A, _A, None), 3),
    ("sq_kv_cache_read", (0, _A, _A, _A, _A, 4, 16, 2, 64, _A, 1, 4, _A, None, 1 << 31, 1, _A, _A, None), 2),
    ("sq_kv_cache_read", (0, _A, _A, _A, _A, 4, 16, 2, 64, _A, 1, 4, _A, None, 0, 1, _A, _A, None), 0),
    ("sq_kv_cache_read", (0, _A, _A, _A, _A, 4, 16, 2, 64, _A, 0, 4, _A, None, 8, 1, _A, _A, None), 0),
])
def test_entry_points_validate_before_launch(fn, args, status):
    assert getattr(sq.lib(), fn)(*args) == status


def test_sizes_of_what_cannot_be():
    lib = sq.lib()
    assert lib.sq_fp4_scale_bytes(2, 4, 64) == 0 and lib.sq_fp4_scale_bytes(0, 0, 64) == 0
    assert lib.sq_kv_row_bytes(3, 64) == 0 and lib.sq_kv_row_bytes(0, 1025) == 0 and lib.sq_kv_scale_bytes(0, 0) == 0
    assert [sq.kv_row_bytes(f, 100) for f in range(3)] == [112, 112, 64]
    assert [sq.kv_scale_bytes(f, 100) for f in range(3)] == [4, 4, 4] and sq.kv_scale_bytes(2, 128) == 4
    with pytest.raises(ValueError):
        sq.kv_row_bytes(sq.KV_INT8, 2000)


@pytest.mark.parametrize("arg,error", [(None, TypeError), (3, TypeError), (torch.zeros(4, 64), ValueError)])
def test_calls_take_cuda_tensors_only(arg, error):
    u = torch.zeros(4, 32, dtype=torch.uint8)
    for call in (lambda: sq.smooth_scales_nvfp4(arg, u, 0.5, u), lambda: sq.quant_weight_fp4(arg, None, sq.MXFP4, u, u),
                 lambda: sq.smooth_quant_act_fp4(arg, None, sq.MXFP4, u, u), lambda: sq.dequant_fp4(u, u, sq.MXFP4, arg),
                 lambda: sq.linear_fp4(u, u, u, u, sq.MXFP4, arg), lambda: sq.kv_cache_write(arg, arg, u, sq.KV_INT8, u, u, u, u),
                 lambda: sq.kv_cache_read(sq.KV_INT8, u, u, u, u, u, u, arg, arg)):
        with pytest.raises(error):
            call()
