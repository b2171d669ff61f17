"""Python binding of the dense gated feed-forward block (include/moe_gb300.h): forward and backward
passes.

Argument checks and marshalling only, as ``block``, whose conventions hold here: rows may have a
stride, operands are on the current device, work goes to ``stream`` or torch's current one.  Gradients
are computed by the explicit call, not recorded.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .block import _CODE, _elsewhere, _rows, _sizes, _stream, _whole
from . import block as _block
from .moe import MOE_W13_UP_GATE, _check


def moe_ff_plan(H, I, dtype, layout, limit, alpha, beta, max_rows) -> int:
    if max(H, I, max_rows) >> 31 > 0:
        _sizes(H, I, max_rows)
    out = ctypes.c_void_p()
    _check(_lib.load().moe_ff_plan(H, I, dtype, layout, limit, alpha, beta, max_rows, ctypes.byref(out)),
           "moe_ff_plan")
    return out.value


def moe_ff_scratch_bytes(plan) -> int:
    n = ctypes.c_size_t()
    _check(_lib.load().moe_ff_scratch_bytes(plan, ctypes.byref(n)), "moe_ff_scratch_bytes")
    return n.value


def moe_ff_set_wait_probe(plan, ns):
    _check(_lib.load().moe_ff_set_wait_probe(plan, int(ns)), "moe_ff_set_wait_probe")


def moe_ff_get_device_error(plan, scratch, stream=None):
    """(status, code) of the device error word in `scratch`, which is cleared."""
    code = ctypes.c_int()
    dev = scratch.get_device()
    if dev < 0 or dev != _block._current_device():
        _elsewhere(scratch, "scratch")
    st = _lib.load().moe_ff_get_device_error(plan, scratch.data_ptr(), _stream(stream, dev),
                                             ctypes.byref(code))
    return st, code.value


def moe_destroy_ff(plan):
    _lib.load().moe_destroy_ff(plan)


class MoEFeedForward:
    """Gated feed-forward block y = W2 h, h = SwiGLU(W13 x), of one layer's w13 [2 I, H] and w2 [H, I]:
    its plan and its scratch buffer on `device` (moe_ff_plan, moe_ff_forward, moe_ff_backward).  Calls that
    share a MoEFeedForward must be stream-ordered."""

    def __init__(self, H, I, max_rows, dtype=torch.bfloat16, layout=MOE_W13_UP_GATE,
                 swiglu_limit=float("inf"), alpha=1.0, beta=0.0, device="cuda"):
        self.H, self.I, self.dtype = H, I, dtype
        if dtype not in _CODE:
            raise ValueError(f"{dtype} is not supported")
        self.plan = moe_ff_plan(H, I, _CODE[dtype], layout, swiglu_limit, alpha, beta, max_rows)
        self.scratch = torch.empty(moe_ff_scratch_bytes(self.plan), dtype=torch.uint8, device=device)
        self.scratch[:4096].zero_()
        torch.cuda.current_stream(self.scratch.device).synchronize()   # calls may use any stream
        self._dev = self.scratch.get_device()
        self._fixed = (self.plan, self.scratch.data_ptr(), self.scratch.numel())

    def _here(self, t, name):
        dev = t.get_device()
        if dev < 0 or dev != _block._current_device():
            _elsewhere(t, name)
        if dev != self._dev:
            raise ValueError(f"{name} is on cuda:{dev}, the scratch buffer on {self.scratch.device}")
        return dev

    def __call__(self, x, w13, w2, out=None, stream=None):
        """y [M, H] of x [M, H]."""
        return self._forward(x, w13, w2, out, None, stream)

    def forward(self, x, w13, w2, out=None, saved=None, stream=None):
        """(y, saved): saved = (up and gate [M, 2 I] in w13's order, fp32, and h [M, I]) is what backward needs, in new
        tensors or the given ones."""
        made = None
        if saved is None:
            on, M = x.device, x.shape[0]
            saved = made = (torch.empty((M, 2 * self.I), dtype=torch.float32, device=on),
                            torch.empty((M, self.I), dtype=self.dtype, device=on))
        return self._forward(x, w13, w2, out, saved, stream, made is None), saved

    def _forward(self, x, w13, w2, out, saved, stream, given=True):
        dev = self._here(x, "x")
        H, I, dtype = self.H, self.I, self.dtype
        xp, ldx = _rows(x, "x", dev, None, H, dtype)
        M = x.shape[0]
        if M >> 31:
            _sizes(M)
        w13p, ldw13 = _rows(w13, "w13", dev, 2 * I, H, dtype)
        w2p, ldw2 = _rows(w2, "w2", dev, H, I, dtype)
        pre_p = h_p = None
        if saved is not None:
            pre, h = saved
            if given:                  # tensors made here need no checks
                _whole(pre, "saved[0]", dev, torch.float32, M * 2 * I)
                _whole(h, "saved[1]", dev, dtype, M * I)
            pre_p, h_p = pre.data_ptr(), h.data_ptr()
        ldo = H
        if out is None:
            out = torch.empty((M, H), dtype=dtype, device=x.device)
        else:
            ldo = _rows(out, "out", dev, M, H, dtype)[1]
        st = _lib.load().moe_ff_forward(*self._fixed, xp, ldx, w13p, ldw13, w2p, ldw2, pre_p, h_p,
                                        out.data_ptr(), ldo, M, _stream(stream, dev))
        if st:
            _check(st, "moe_ff_forward")
        return out

    def backward(self, dy, x, w13, w2, saved, need=(True, True, True), dx=None, dw13=None, dw2=None,
                 stream=None):
        """(dx, dw13, dw2) of forward's y at dy [M, H], in new tensors or the given ones; None for each
        that `need` leaves out.  x, w13, w2 and saved are forward's; those that no gradient of `need` takes may be
        None: x (dw13), w13 (dx), saved[1] (dw2), w2 and saved[0] (dx and dw13)."""
        dev = self._here(dy, "dy")
        H, I, dtype = self.H, self.I, self.dtype
        dyp, lddy = _rows(dy, "dy", dev, None, H, dtype)
        M = dy.shape[0]
        if M >> 31:
            _sizes(M)
        need_x, need_w13, need_w2 = need
        inner = need_x or need_w13
        pre, h = (None, None) if saved is None else saved
        for t, name, used in ((x, "x", need_w13), (w13, "w13", need_x), (w2, "w2", inner), (pre, "saved[0]", inner), (h, "saved[1]", need_w2)):
            if t is None and used:
                raise ValueError(f"{name} is needed for these gradients")
        xp, ldx = (None, H) if x is None else _rows(x, "x", dev, M, H, dtype)
        w13p, ldw13 = (None, H) if w13 is None else _rows(w13, "w13", dev, 2 * I, H, dtype)
        w2p, ldw2 = (None, I) if w2 is None else _rows(w2, "w2", dev, H, I, dtype)
        pre_p = None if pre is None else _whole(pre, "saved[0]", dev, torch.float32, M * 2 * I)
        h_p = None if h is None else _whole(h, "saved[1]", dev, dtype, M * I)
        wanted, on = [], dy.device
        for needed, t, name, rows, cols in zip(need, (dx, dw13, dw2), ("dx", "dw13", "dw2"), (M, 2 * I, H), (H, H, I)):
            if not needed:
                if t is not None:
                    raise ValueError(f"{name} is given, but need leaves it out")
                wanted.append((None, None, cols))
                continue
            if t is None:
                t = torch.empty((rows, cols), dtype=dtype, device=on)
                wanted.append((t, t.data_ptr(), cols))
            else:
                wanted.append((t, *_rows(t, name, dev, rows, cols, dtype)))
        (dx, dxp, lddx), (dw13, dw13p, lddw13), (dw2, dw2p, lddw2) = wanted
        st = _lib.load().moe_ff_backward(*self._fixed, dyp, lddy, xp, ldx, w13p, ldw13, w2p, ldw2, pre_p, h_p,
                                         dxp, lddx, dw13p, lddw13, dw2p, lddw2, M, _stream(stream, dev))
        if st:
            _check(st, "moe_ff_backward")
        return dx, dw13, dw2

    def device_error(self, stream=None):
        return moe_ff_get_device_error(self.plan, self.scratch, stream)

    def close(self):
        if getattr(self, "plan", None):
            moe_destroy_ff(self.plan)
            self.plan = None
            self._fixed = (None, 0, 0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
