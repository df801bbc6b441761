"""Operands of the wrong type beside another one raise TypeError (as the INT8 and FP8 calls) and ValueError."""
import pytest
import torch

pytestmark = pytest.mark.gpu

sq = pytest.importorskip("w8a8_post_quantization_calib_b200")


@pytest.mark.parametrize("error", [TypeError, ValueError])
def test_operands_of_the_wrong_type(error):
    def u8(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device="cuda")

    def f32(*shape):
        return torch.zeros(shape, device="cuda")

    q, sf = u8(4, 32), u8(512)
    with pytest.raises(error, match="bias"):
        sq.linear_fp4(q, sf, q, sf, sq.MXFP4, f32(4, 4), bias=f32(4).half())
    k, slots, c = f32(4, 2, 32), torch.arange(4, device="cuda"), [u8(1, 4, 2, 32), f32(1, 4, 2), u8(1, 4, 2, 32), f32(1, 4, 2)]
    table, cu = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(error, match="slots"):
        sq.kv_cache_write(k, k, slots.int(), sq.KV_FP8, *c)
    with pytest.raises(error, match="k_cache"):
        sq.kv_cache_write(k, k, slots, sq.KV_INT8, *c)
    with pytest.raises(error, match="v_scale"):
        sq.kv_cache_write(k, k, slots, sq.KV_FP8, *c[:3], c[3].half())
    with pytest.raises(error, match="table"):
        sq.kv_cache_read(sq.KV_FP8, *c, table.long(), cu, k, k.clone())
    with pytest.raises(error, match="cu_rows"):
        sq.kv_cache_read(sq.KV_FP8, *c, table, cu.long(), k, k.clone())
    with pytest.raises(error, match="starts"):
        sq.kv_cache_read(sq.KV_FP8, *c, table, cu, k, k.clone(), starts=cu[:1].long())
