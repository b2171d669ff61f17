"""Python binding of the 8-bit products with block scales (include/moe_gb300.h): quantisation to
e4m3 with a scale for each 128 values of a row or each 128 x 128 tile, products of such operands.

Codes are torch.float8_e4m3fn tensors, scales fp32.  Argument checks and marshalling only, as
``block``, whose conventions hold here: rows may have a stride, operands are on the current device,
work goes to ``stream`` or torch's current one.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .block import _CODE, _code, _dev, _elsewhere, _rows, _sizes, _stream, _whole, MOE_ACT_NONE, MOE_ACT_SWIGLU
from . import block as _block
from .moe import MOE_W13_UP_GATE, _check

MOE_FP8_ROWS = 0
MOE_FP8_TILES = 1
_E4M3 = torch.float8_e4m3fn


def _blocks(n):
    return -(-n // 128)


def _stack(t, name, E, N, K):
    """Row stride of matrices [E, N, K] whose rows are contiguous and evenly apart over all of them."""
    if t.dim() != 3 or t.shape[0] != E or t.shape[1] != N or t.shape[2] != K:
        raise ValueError(f"{name} must be [{E}, {N}, {K}], not {list(t.shape)}")
    per, ld, unit = t.stride()
    if N == 1:                     # the stride of a dimension of one element says nothing
        ld = per if E > 1 else K
    if (unit != 1 and K > 1) or ld < K or (per != N * ld and E > 1):
        raise ValueError(f"the rows of {name} must be contiguous and evenly apart over all matrices")
    return ld


def moe_fp8_quant(x, form=MOE_FP8_ROWS, q=None, scale=None, stream=None):
    """(q, scale): e4m3 codes of x's shape and the fp32 scales of their blocks.  MOE_FP8_ROWS: x [rows, K],
    scale [rows, ceil(K / 128)].  MOE_FP8_TILES: x [rows, K] or [E, rows, K], scale [(E,) ceil(rows / 128),
    ceil(K / 128)].  x is bf16, f16 or fp32; see moe_fp8_quant in include/moe_gb300.h."""
    dev = x.get_device()
    if dev < 0 or dev != _block._current_device():
        _elsewhere(x, "x")
    dtype = _CODE.get(x.dtype)
    if dtype is None:
        _code(x, "x")
    on = x.device
    # outputs made here need no checks
    if form == MOE_FP8_ROWS:
        if x.dim() != 2:
            raise ValueError(f"x must be [rows, K], not {list(x.shape)}")
        E, (rows, K) = 1, x.shape
        if (rows | K) >> 31:
            _sizes(rows, K)
        KB = _blocks(K)
        ldx, unit = x.stride()
        if unit != 1 or ldx < K:
            ldx = _rows(x, "x", dev, rows, K)[1]
        ldq, lds = K, KB
        if q is None:
            q = torch.empty((rows, K), dtype=_E4M3, device=on)
        else:
            ldq = _rows(q, "q", dev, rows, K, _E4M3)[1]
        if scale is None:
            scale = torch.empty((rows, KB), dtype=torch.float32, device=on)
        else:
            lds = _rows(scale, "scale", dev, rows, KB, torch.float32)[1]
    elif form == MOE_FP8_TILES:
        if x.dim() not in (2, 3):
            raise ValueError(f"x must be [rows, K] or [E, rows, K], not {list(x.shape)}")
        E, rows, K = (1, *x.shape) if x.dim() == 2 else x.shape
        if (E | rows | K) >> 31:
            _sizes(E, rows, K)
        KB, lead = _blocks(K), x.shape[:-2]
        ldx = _stack(x if lead else x.unsqueeze(0), "x", E, rows, K)
        ldq, lds = K, KB
        if q is None:
            q = torch.empty(x.shape, dtype=_E4M3, device=on)
        else:
            if q.shape != x.shape:
                raise ValueError(f"q must be {list(x.shape)}, not {list(q.shape)}")
            _dev(q, "q", dev, _E4M3)
            ldq = _stack(q if lead else q.unsqueeze(0), "q", E, rows, K)
        if scale is None:
            scale = torch.empty((*lead, _blocks(rows), KB), dtype=torch.float32, device=on)
        else:
            _whole(scale, "scale", dev, torch.float32, E * _blocks(rows) * KB)
    else:
        raise ValueError(f"form {form} is neither MOE_FP8_ROWS nor MOE_FP8_TILES")
    st = _lib.load().moe_fp8_quant(x.data_ptr(), dtype, ldx, E, rows, K, form, q.data_ptr(), ldq, scale.data_ptr(), lds,
                                   _stream(stream, dev))
    if st:
        _check(st, "moe_fp8_quant")
    return q, scale


def moe_fp8_plan(E, N, K, dtype, act, layout, limit, alpha, beta, max_rows) -> int:
    if max(E, N, K, max_rows) >> 31 > 0:
        _sizes(E, N, K, max_rows)
    out = ctypes.c_void_p()
    _check(_lib.load().moe_fp8_plan(E, N, K, dtype, act, layout, limit, alpha, beta, max_rows,
                                    ctypes.byref(out)), "moe_fp8_plan")
    return out.value


def moe_fp8_scratch_bytes(plan) -> int:
    n = ctypes.c_size_t()
    _check(_lib.load().moe_fp8_scratch_bytes(plan, ctypes.byref(n)), "moe_fp8_scratch_bytes")
    return n.value


def moe_fp8_set_wait_probe(plan, ns):
    _check(_lib.load().moe_fp8_set_wait_probe(plan, int(ns)), "moe_fp8_set_wait_probe")


def moe_fp8_get_device_error(plan, scratch, stream=None):
    """(status, code) of the device error word in `scratch`, which is cleared."""
    code = ctypes.c_int()
    dev = scratch.get_device()
    if dev < 0 or dev != _block._current_device():
        _elsewhere(scratch, "scratch")
    st = _lib.load().moe_fp8_get_device_error(plan, scratch.data_ptr(), _stream(stream, dev),
                                              ctypes.byref(code))
    return st, code.value


def moe_destroy_fp8(plan):
    _lib.load().moe_destroy_fp8(plan)


class MoEFp8:
    """Products of e4m3 operands with block scales, dense (E = 1, no offsets) or grouped by expert: the
    plan of one layer's matrices [E, N, K] and its scratch buffer on `device` (moe_fp8_plan, moe_fp8_run).
    dtype is the outputs'.  Calls that share a MoEFp8 must be stream-ordered."""

    def __init__(self, E, N, K, max_rows, dtype=torch.bfloat16, act=MOE_ACT_NONE,
                 layout=MOE_W13_UP_GATE, swiglu_limit=float("inf"), alpha=1.0, beta=0.0,
                 device="cuda"):
        self.E, self.N, self.K, self.dtype = E, N, K, dtype
        if dtype not in _CODE:
            raise ValueError(f"{dtype} is not supported")
        self.cols = N // 2 if act == MOE_ACT_SWIGLU else N
        self.blocks = _blocks(K)
        self.tall = 2 * _blocks(N // 2) if act == MOE_ACT_SWIGLU else _blocks(N)
        self.plan = moe_fp8_plan(E, N, K, _CODE[dtype], act, layout, swiglu_limit, alpha, beta, max_rows)
        self.scratch = torch.empty(moe_fp8_scratch_bytes(self.plan), dtype=torch.uint8, device=device)
        self.scratch[:4096].zero_()
        torch.cuda.current_stream(self.scratch.device).synchronize()   # calls may use any stream
        self._dev = self.scratch.get_device()
        self._fixed = (self.plan, self.scratch.data_ptr(), self.scratch.numel())

    def __call__(self, x, x_scale, w, w_scale, offsets=None, perm=None, topk=1, out=None, stream=None):
        """out[p] = act(w[e] . x[row(p)]) of the values that codes and scales stand for.  x [rows, K] and
        x_scale [rows, KB] as moe_fp8_quant gives them (MOE_FP8_ROWS); w [E, N, K], or [N, K] where E = 1,
        and w_scale [E, tile rows, KB]: tile rows = ceil(N / 128), with a SwiGLU the ceil(N / 2 / 128) of
        each half in turn.  offsets, perm and topk as for MoEGrouped; offsets may be None where E = 1."""
        dev = x.get_device()
        if dev < 0 or dev != _block._current_device():
            _elsewhere(x, "x")
        if dev != self._dev:
            raise ValueError(f"x is on cuda:{dev}, the scratch buffer on {self.scratch.device}")
        xp, ldx = _rows(x, "x", dev, None, self.K, _E4M3)
        rows = x.shape[0]
        xsp, ldxs = _rows(x_scale, "x_scale", dev, rows, self.blocks, torch.float32)
        S = rows if perm is None else perm.numel()
        if (rows | S) >> 31:
            _sizes(rows, S)
        if self.E == 1 and w.dim() == 2:
            wp, ldw = _rows(w, "w", dev, self.N, self.K, _E4M3)
        else:
            wp, ldw = _dev(w, "w", dev, _E4M3), _stack(w, "w", self.E, self.N, self.K)
        if offsets is None:
            if self.E != 1:
                raise ValueError("products of several experts need offsets")
            offsets_p = None
        else:
            offsets_p = _whole(offsets, "offsets", dev, torch.int32, self.E + 1)
        ldo = self.cols
        if out is None:
            out = torch.empty((S, ldo), dtype=self.dtype, device=x.device)
        else:
            ldo = _rows(out, "out", dev, S, ldo, self.dtype)[1]
        st = _lib.load().moe_fp8_run(
            *self._fixed, xp, ldx, rows, xsp, ldxs, wp, ldw,
            _whole(w_scale, "w_scale", dev, torch.float32, self.E * self.tall * self.blocks), offsets_p,
            None if perm is None else _whole(perm, "perm", dev, torch.int32, S), topk, out.data_ptr(), ldo, S,
            _stream(stream, dev))
        if st:
            _check(st, "moe_fp8_run")
        return out

    def device_error(self, stream=None):
        return moe_fp8_get_device_error(self.plan, self.scratch, stream)

    def close(self):
        if getattr(self, "plan", None):
            moe_destroy_fp8(self.plan)
            self.plan = None
            self._fixed = (None, 0, 0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
