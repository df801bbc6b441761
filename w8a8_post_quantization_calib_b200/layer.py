"""Layer-level drivers on top of the C ABI: the SmoothQuant W8A8 linear, the same
layer in 4-bit microscaled formats, and the paged key/value cache in 8 or 4 bits.

Mirrors the calibration -> offline transform -> runtime flow of the
"010. SmoothQuant Integration" design (SmoothQuantQuantizer.add_batch keeps
the per-channel max-abs; the layer holds int8 weights with per-row scales,
the per-channel smoothing factors and the activation scale).  PyTorch only
allocates device buffers; every computation is a libsq call.

Methods that take ``stream`` run whole on it (None: the current stream): their buffers belong to it, it starts behind
the work that the current stream holds at the call, and the memory of a method's arguments and results is not given to
other work before both streams are done with it.  Results are ready on that stream: wait for it before another one reads
them.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (ACT_PER_TOKEN, ACT_STATIC, KV_INT8, KV_MXFP4, MXFP4, NVFP4, calib_absmax, fp4_code_bytes,
               fp4_scale_bytes, kv_cache_read, kv_cache_write, kv_row_bytes, kv_scale_bytes, linear_fp4, linear_w8a8,
               linear_workspace_size, quant_weight, quant_weight_fp4, smooth_quant_act, smooth_quant_act_fp4,
               smooth_scales, smooth_scales_nvfp4)


class _Here:
    """A call on the current stream."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False

    def keep(self, *tensors) -> None:
        pass


_HERE = _Here()


class _Side(_Here):
    """A call on another stream, which is the current one meanwhile."""

    def __init__(self, side, caller, tensors):
        self.caller, self.side, self.tensors = caller, side, tensors
        self.context = torch.cuda.stream(side)

    def __enter__(self):
        graph = torch.cuda.is_current_stream_capturing()
        self.context.__enter__()
        try:
            # a graph under capture does not wait for work outside it: that is done, or not, when it is replayed
            if graph or not torch.cuda.is_current_stream_capturing():
                self.side.wait_stream(self.caller)
            for t in self.tensors:
                if isinstance(t, torch.Tensor) and t.is_cuda:          # others are refused by the call
                    t.record_stream(self.side)
        except BaseException:
            self.context.__exit__(None, None, None)
            raise
        return self

    def __exit__(self, *exc):
        self.context.__exit__(*exc)
        return False

    def keep(self, *tensors) -> None:
        """Tensors allocated in the call that the caller gets, for its own stream."""
        for t in tensors:
            if t is not None:
                t.record_stream(self.caller)


def _on(stream, *tensors):
    """The context of a call on `stream` (None, an object with cuda_stream, or its address) that uses the caller's
    tensors."""
    if stream is None:
        return _HERE
    caller = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream) and stream.device != caller.device:
        raise ValueError(f"the stream is on {stream.device}, the current device is {caller.device}")
    address = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if address == caller.cuda_stream:
        return _HERE
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(address) if address else torch.cuda.default_stream()
    return _Side(stream, caller, tensors)


class Calibrator:
    """Running per-channel max|X_j| over calibration batches (one layer)."""

    def __init__(self, K: int, device="cuda"):
        self.act_max = torch.zeros(K, dtype=torch.float32, device=device)

    def add_batch(self, x: torch.Tensor, stream=None) -> None:
        with _on(stream, x, self.act_max):
            calib_absmax(x.reshape(-1, x.shape[-1]), self.act_max)


@dataclass
class QuantizedLinear:
    wq: torch.Tensor          # int8 [N, K]
    w_scale: torch.Tensor     # fp32 [N]
    s: torch.Tensor           # fp32 [K]
    a_static: torch.Tensor    # fp32 [1]
    act_max: torch.Tensor     # fp32 [K]
    w_max: torch.Tensor       # fp32 [K]
    alpha: float
    mode: int = ACT_STATIC
    bias: torch.Tensor | None = None

    @property
    def N(self) -> int:
        return self.wq.shape[0]

    @property
    def K(self) -> int:
        return self.wq.shape[1]

    @classmethod
    def from_float(cls, w: torch.Tensor, act_max: torch.Tensor, alpha: float = 0.5, mode: int = ACT_STATIC,
                   bias=None, stream=None) -> "QuantizedLinear":
        N, K = w.shape
        dev = w.device
        with _on(stream, w, act_max) as call:
            w_max = torch.zeros(K, dtype=torch.float32, device=dev)
            calib_absmax(w, w_max)
            s = torch.empty(K, dtype=torch.float32, device=dev)
            a = torch.empty(1, dtype=torch.float32, device=dev)
            smooth_scales(act_max, w_max, alpha, s, a)
            wq = torch.empty(N, K, dtype=torch.int8, device=dev)
            ws = torch.empty(N, dtype=torch.float32, device=dev)
            quant_weight(w, s, wq, ws)
            call.keep(w_max, s, a, wq, ws)
        return cls(wq, ws, s, a, act_max, w_max, alpha, mode, bias)

    def quantize_input(self, x: torch.Tensor, xq=None, a_scale=None, stream=None):
        M = x.shape[0]
        with _on(stream, x, xq, a_scale, self.s, self.a_static) as call:
            if xq is None:
                xq = torch.empty(M, self.K, dtype=torch.int8, device=x.device)
            if self.mode == ACT_STATIC:
                a_scale = self.a_static
            elif a_scale is None:
                a_scale = torch.empty(M, dtype=torch.float32, device=x.device)
            smooth_quant_act(x, self.s, self.mode, a_scale, xq)
            call.keep(xq, a_scale)
        return xq, a_scale

    def workspace(self, M: int, device="cuda") -> torch.Tensor | None:
        n = linear_workspace_size(M, self.N, self.K)
        return torch.zeros(n, dtype=torch.uint8, device=device) if n else None

    def forward(self, x: torch.Tensor, out_dtype=torch.float16, y=None, workspace=None, stream=None):
        M = x.shape[0]
        with _on(stream, x, y, workspace, self.s, self.a_static, self.wq, self.w_scale, self.bias) as call:
            xq, a = self.quantize_input(x)
            if y is None:
                y = torch.empty(M, self.N, dtype=out_dtype, device=x.device)
            linear_w8a8(xq, self.wq, a, self.mode, self.w_scale, y, bias=self.bias, workspace=workspace)
            call.keep(y)
        return y


@dataclass
class QuantizedLinearFp4:
    """The smoothed layer with 4-bit weights and activations (format MXFP4 or NVFP4)."""
    wq4: torch.Tensor         # uint8 [N, fp4_code_bytes(K)]
    w_sf: torch.Tensor        # uint8, tiled block scales
    s: torch.Tensor           # fp32 [K]
    fmt: int
    K: int
    g_act: torch.Tensor | None = None      # NVFP4: tensor scales, fp32 [1]
    g_w: torch.Tensor | None = None
    bias: torch.Tensor | None = None

    @property
    def N(self) -> int:
        return self.wq4.shape[0]

    @classmethod
    def from_float(cls, w: torch.Tensor, act_max: torch.Tensor, alpha: float = 0.5, fmt: int = MXFP4, bias=None,
                   stream=None) -> "QuantizedLinearFp4":
        N, K = w.shape
        dev = w.device
        with _on(stream, w, act_max) as call:
            w_max = torch.zeros(K, dtype=torch.float32, device=dev)
            calib_absmax(w, w_max)
            s = torch.empty(K, dtype=torch.float32, device=dev)
            g_act = g_w = None
            if fmt == NVFP4:
                g_act, g_w = (torch.empty(1, dtype=torch.float32, device=dev) for _ in range(2))
            smooth_scales_nvfp4(act_max, w_max, alpha, s, g_act, g_w)
            wq4 = torch.empty(N, fp4_code_bytes(K), dtype=torch.uint8, device=dev)
            w_sf = torch.empty(fp4_scale_bytes(fmt, N, K), dtype=torch.uint8, device=dev)
            quant_weight_fp4(w, s, fmt, wq4, w_sf, g=g_w)
            call.keep(s, g_act, g_w, wq4, w_sf)
        return cls(wq4, w_sf, s, fmt, K, g_act, g_w, bias)

    def quantize_input(self, x: torch.Tensor, xq4=None, x_sf=None, stream=None):
        M = x.shape[0]
        with _on(stream, x, xq4, x_sf, self.s, self.g_act) as call:
            if xq4 is None:
                xq4 = torch.empty(M, fp4_code_bytes(self.K), dtype=torch.uint8, device=x.device)
            if x_sf is None:
                x_sf = torch.empty(fp4_scale_bytes(self.fmt, max(M, 1), self.K), dtype=torch.uint8, device=x.device)
            smooth_quant_act_fp4(x, self.s, self.fmt, xq4, x_sf, g=self.g_act)
            call.keep(xq4, x_sf)
        return xq4, x_sf

    def forward(self, x: torch.Tensor, out_dtype=torch.bfloat16, y=None, stream=None):
        with _on(stream, x, y, self.s, self.g_act, self.g_w, self.wq4, self.w_sf, self.bias) as call:
            xq4, x_sf = self.quantize_input(x)
            if y is None:
                y = torch.empty(x.shape[0], self.N, dtype=out_dtype, device=x.device)
            linear_fp4(xq4, x_sf, self.wq4, self.w_sf, self.fmt, y, bias=self.bias, g_act=self.g_act, g_w=self.g_w)
            call.keep(y)
        return y


class PagedKVCache:
    """Keys and values of H heads of D elements in num_pages pages of page_size tokens (slot = page * page_size +
    position in the page), quantised as they are written."""

    def __init__(self, num_pages: int, page_size: int, H: int, D: int, fmt: int = KV_INT8, device="cuda"):
        self.num_pages, self.page_size, self.H, self.D, self.fmt = num_pages, page_size, H, D, fmt
        codes = torch.int8 if fmt == KV_INT8 else torch.uint8
        shape = (num_pages, page_size, H)
        self.k, self.v = (torch.zeros(*shape, kv_row_bytes(fmt, D), dtype=codes, device=device) for _ in range(2))
        if fmt == KV_MXFP4:
            self.k_scale, self.v_scale = (torch.zeros(*shape, kv_scale_bytes(fmt, D), dtype=torch.uint8, device=device)
                                          for _ in range(2))
        else:
            self.k_scale, self.v_scale = (torch.zeros(shape, dtype=torch.float32, device=device) for _ in range(2))

    def write(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
        """k, v: [T, H, D]; slots: int64 [T], a negative one is skipped."""
        with _on(stream, k, v, slots, self.k, self.k_scale, self.v, self.v_scale):
            kv_cache_write(k, v, slots, self.fmt, self.k, self.k_scale, self.v, self.v_scale)

    def read(self, table: torch.Tensor, cu_rows: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor, starts=None,
             stream=None):
        """Rows cu_rows[b] .. cu_rows[b + 1] - 1 of the outputs [total, H, D] take sequence b's positions from starts[b]
        (0 without) on."""
        with _on(stream, table, cu_rows, k_out, v_out, starts, self.k, self.k_scale, self.v, self.v_scale):
            kv_cache_read(self.fmt, self.k, self.k_scale, self.v, self.v_scale, table, cu_rows, k_out, v_out, starts=starts)
        return k_out, v_out


__all__ = ["Calibrator", "QuantizedLinear", "QuantizedLinearFp4", "PagedKVCache", "ACT_STATIC", "ACT_PER_TOKEN"]
