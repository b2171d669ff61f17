"""Python binding of the 16-bit block's entry points (include/moe_gb300.h): router, grouping of
the slots by expert, products grouped by expert, norms around the block.

Argument checks and marshalling only, like ``moe``; the computation runs in the library's CUDA
kernels.  Matrices may have a row stride (their rows must be contiguous); everything else is
contiguous.  A call's operands are on one device, the current one (the library launches there); a
``ValueError`` says where they are not.  Work goes to ``stream``, or to torch's current stream;
tensors that are not created on that stream are the caller's to order and keep alive, as for any
stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .moe import MOE_W13_UP_GATE, _check

MOE_DTYPE_BF16 = 0
MOE_DTYPE_F16 = 1
MOE_DTYPE_F32 = 2
MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1
MOE_ACT_NONE = 0
MOE_ACT_SWIGLU = 1
MOE_NORM_RMS = 0
MOE_NORM_LAYER = 1

_CODE = {torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16, torch.float32: MOE_DTYPE_F32}


_current_device = torch._C._cuda_getDevice      # without the look at lazy initialisation: operands exist


def _stream(stream, dev):
    """Stream handle; without a stream, torch's current one on device `dev` (its raw handle: a Stream
    object costs as much as a launch)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if isinstance(stream, torch.cuda.Stream):
        if stream.device_index != dev:
            raise ValueError(f"the stream is on cuda:{stream.device_index}, the operands on cuda:{dev}")
        return stream.cuda_stream
    return int(stream)


def _elsewhere(t, name):
    """The error of a call whose first operand is not on the current device."""
    if t.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_current_device()}")


def _dev(t, name, dev, dtype=None):
    """Address of a tensor on device `dev` (of `dtype`)."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{dev}, not on {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    return t.data_ptr()


def _whole(t, name, dev, dtype, numel):
    """Address of a contiguous tensor of `numel` elements on device `dev`."""
    if t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {numel} elements")
    if t.dtype != dtype or t.get_device() != dev:
        _dev(t, name, dev, dtype)
    return t.data_ptr()


def _rows(t, name, dev, rows, cols, dtype=None):
    """(address, row stride) of a matrix [rows, cols] on device `dev` whose rows are contiguous."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name} must be [{'rows' if rows is None else rows}, {cols}], not {list(shape)}")
    step, unit = t.stride()
    if unit != 1 or step < cols:
        # the stride of a dimension of one element says nothing
        if (unit != 1 and cols > 1) or (step < cols and shape[0] > 1):
            raise ValueError(f"the rows of {name} must be contiguous and apart")
        step = max(step, cols)
    if t.get_device() != dev or (dtype is not None and t.dtype != dtype):
        _dev(t, name, dev, dtype)
    return t.data_ptr(), step


def _code(t, name):
    code = _CODE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: {t.dtype} is not supported")
    return code


# ---------------------------------------------------------------------------------- router

def moe_router(logits, topk, score=MOE_SCORE_SOFTMAX, bias=None, n_group=1, topk_group=1,
               renormalize=True, scale=1.0, ids=None, weights=None, stream=None):
    """Top-k experts and weights of every row of logits [M, E] (bf16, f16 or fp32): (ids int32
    [M, topk], weights fp32 [M, topk]); see moe_router in include/moe_gb300.h."""
    dev = logits.get_device()
    if dev < 0 or dev != _current_device():
        _elsewhere(logits, "logits")
    M, E = logits.shape
    ld, unit = logits.stride()
    dtype = _CODE.get(logits.dtype)
    if unit != 1 or ld < E or dtype is None:
        ld, dtype = _rows(logits, "logits", dev, M, E)[1], _code(logits, "logits")
    if topk < 0:
        raise ValueError("topk must not be negative")
    # outputs made here need no checks
    on = logits.device
    if ids is None:
        ids = torch.empty((M, topk), dtype=torch.int32, device=on)
    else:
        _whole(ids, "ids", dev, torch.int32, M * topk)
    if weights is None:
        weights = torch.empty((M, topk), dtype=torch.float32, device=on)
    else:
        _whole(weights, "weights", dev, torch.float32, M * topk)
    st = _lib.load().moe_router(
        logits.data_ptr(), dtype, ld, None if bias is None else _whole(bias, "bias", dev, torch.float32, E),
        M, E, topk, score, n_group, topk_group, renormalize, scale, ids.data_ptr(), weights.data_ptr(),
        _stream(stream, dev))
    if st:
        _check(st, "moe_router")
    return ids, weights


# ---------------------------------------------------------------------------------- grouping

def moe_group(topk_ids, E, first_expert=0, offsets=None, perm=None, slot_of=None, stream=None):
    """Slots of topk_ids [M, topk] (int32) grouped by expert: (offsets [E + 1], perm [M * topk],
    slot_of [M, topk]), all int32; see moe_group in include/moe_gb300.h."""
    dev = topk_ids.get_device()
    if dev < 0 or dev != _current_device():
        _elsewhere(topk_ids, "topk_ids")
    M, topk = topk_ids.shape
    n = M * topk
    ids_p = _whole(topk_ids, "topk_ids", dev, torch.int32, n)
    # outputs made here need no checks
    if offsets is None:
        offsets = torch.empty(E + 1, dtype=torch.int32, device=topk_ids.device)
    else:
        _whole(offsets, "offsets", dev, torch.int32, E + 1)
    if perm is None:
        perm = torch.empty(n, dtype=torch.int32, device=topk_ids.device)
    else:
        _whole(perm, "perm", dev, torch.int32, n)
    if slot_of is None:
        slot_of = torch.empty_like(topk_ids)
    else:
        _whole(slot_of, "slot_of", dev, torch.int32, n)
    st = _lib.load().moe_group(ids_p, M, topk, E, first_expert, offsets.data_ptr(), perm.data_ptr(),
                               slot_of.data_ptr(), _stream(stream, dev))
    if st:
        _check(st, "moe_group")
    return offsets, perm, slot_of


# ---------------------------------------------------------------------------------- grouped products

def moe_grouped_plan(E, N, K, dtype, act, layout, limit, alpha, beta, max_rows) -> int:
    out = ctypes.c_void_p()
    _check(_lib.load().moe_grouped_plan(E, N, K, dtype, act, layout, limit, alpha, beta, max_rows,
                                        ctypes.byref(out)), "moe_grouped_plan")
    return out.value


def moe_grouped_scratch_bytes(plan) -> int:
    n = ctypes.c_size_t()
    _check(_lib.load().moe_grouped_scratch_bytes(plan, ctypes.byref(n)), "moe_grouped_scratch_bytes")
    return n.value


def moe_grouped_set_wait_probe(plan, ns):
    _check(_lib.load().moe_grouped_set_wait_probe(plan, int(ns)), "moe_grouped_set_wait_probe")


def moe_grouped_get_device_error(plan, scratch, stream=None):
    """(status, code) of the device error word in `scratch`, which is cleared."""
    code = ctypes.c_int()
    dev = scratch.get_device()
    if dev < 0 or dev != _current_device():
        _elsewhere(scratch, "scratch")
    st = _lib.load().moe_grouped_get_device_error(plan, scratch.data_ptr(), _stream(stream, dev),
                                                  ctypes.byref(code))
    return st, code.value


def moe_destroy_grouped(plan):
    _lib.load().moe_destroy_grouped(plan)


class MoEGrouped:
    """Products grouped by expert with ragged sizes, 16-bit operands: the plan of one layer's
    matrices [E, N, K] and its scratch buffer on `device` (moe_grouped_plan, moe_grouped_run).  Calls
    that share a MoEGrouped must be stream-ordered."""

    def __init__(self, E, N, K, max_rows, dtype=torch.bfloat16, act=MOE_ACT_NONE,
                 layout=MOE_W13_UP_GATE, swiglu_limit=float("inf"), alpha=1.0, beta=0.0,
                 device="cuda"):
        self.E, self.N, self.K, self.dtype = E, N, K, dtype
        if dtype not in _CODE:
            raise ValueError(f"{dtype} is not supported")
        self.cols = N // 2 if act == MOE_ACT_SWIGLU else N
        self.plan = moe_grouped_plan(E, N, K, _CODE[dtype], act, layout, swiglu_limit, alpha, beta,
                                     max_rows)
        self.scratch = torch.empty(moe_grouped_scratch_bytes(self.plan), dtype=torch.uint8,
                                   device=device)
        self.scratch[:4096].zero_()
        torch.cuda.current_stream(self.scratch.device).synchronize()   # calls may use any stream
        self._dev = self.scratch.get_device()
        self._fixed = (self.plan, self.scratch.data_ptr(), self.scratch.numel())

    def __call__(self, x, w, offsets, perm=None, topk=1, out=None, stream=None):
        """out[p] = act(w[e] . x[row(p)]) for the positions p of every expert e.  offsets [E + 1]
        and perm [S] as moe_group gives them; with perm, x holds one row per token (row(p) =
        perm[p] // topk), without it one row per position."""
        dev = x.get_device()
        if dev < 0 or dev != _current_device():
            _elsewhere(x, "x")
        if dev != self._dev:
            raise ValueError(f"x is on cuda:{dev}, the scratch buffer on {self.scratch.device}")
        xp, ldx = _rows(x, "x", dev, None, self.K, self.dtype)
        S = x.shape[0] if perm is None else perm.numel()
        if w.dim() != 3 or w.shape[0] != self.E or w.shape[1] != self.N or w.shape[2] != self.K:
            raise ValueError(f"w must be [{self.E}, {self.N}, {self.K}], not {list(w.shape)}")
        per, ldw, unit = w.stride()
        if self.N == 1:                # the stride of a dimension of one element says nothing
            ldw = per if self.E > 1 else self.K
        if (unit != 1 and self.K > 1) or ldw < self.K or (per != self.N * ldw and self.E > 1):
            raise ValueError("the rows of w must be contiguous and evenly apart over all experts")
        if out is None:
            out = torch.empty((S, self.cols), dtype=self.dtype, device=x.device)
        op, ldo = _rows(out, "out", dev, S, self.cols, self.dtype)
        st = _lib.load().moe_grouped_run(
            *self._fixed, xp, ldx, x.shape[0], _dev(w, "w", dev, self.dtype), ldw,
            _whole(offsets, "offsets", dev, torch.int32, self.E + 1),
            None if perm is None else _whole(perm, "perm", dev, torch.int32, S), topk, op, ldo, S,
            _stream(stream, dev))
        if st:
            _check(st, "moe_grouped_run")
        return out

    def device_error(self, stream=None):
        return moe_grouped_get_device_error(self.plan, self.scratch, stream)

    def close(self):
        if getattr(self, "plan", None):
            moe_destroy_grouped(self.plan)
            self.plan = None
            self._fixed = (None, 0, 0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------------- norms

def moe_block_norm(residual, rows=None, slot_of=None, topk_weights=None, shared=None,
                   post_weight=None, post_bias=None, gate=None, scale=1.0, pre_weight=None,
                   pre_bias=None, eps=1e-6, kind=MOE_NORM_RMS, weight_offset=0.0, residual_out=None,
                   out=None, stream=None):
    """Norm after a block (post_weight), gate, residual scale and the norm before the next block
    (pre_weight) in one pass; with slot_of and topk_weights the rows are the experts' and their
    top-k combination is taken here too.  Returns (residual_out, out): residual_out None without
    rows, out None without pre_weight.  out is of the rows' type; without rows, and unless it is given,
    of the residual's, of pre_weight's where the residual is fp32, bf16 where both are.  gate broadcasts
    over [M, H]; weights, biases and gate are of out's type or all fp32.  See moe_block_norm in
    include/moe_gb300.h."""
    dev = residual.get_device()
    if dev < 0 or dev != _current_device():
        _elsewhere(residual, "residual")
    M, H = residual.shape
    residual_p, ld_residual = _rows(residual, "residual", dev, M, H)
    if rows is not None:
        dtype = rows.dtype
    elif out is not None:
        dtype = out.dtype
    elif residual.dtype != torch.float32:
        dtype = residual.dtype
    else:
        dtype = torch.bfloat16 if pre_weight is None or pre_weight.dtype == torch.float32 else pre_weight.dtype
    code = _CODE.get(dtype)
    if code is None:
        raise ValueError(f"rows: {dtype} is not supported")
    wt = next((t.dtype for t in (pre_weight, post_weight, gate, pre_bias, post_bias) if t is not None), dtype)
    rows_p = slot_p = weights_p = shared_p = post_p = post_b = gate_p = pre_p = pre_b = res_out_p = out_p = 0
    ld_rows = ld_shared = ld_res_out = ld_out = gate_row = gate_col = topk = n_rows = 0
    if slot_of is not None:
        if rows is None or topk_weights is None or slot_of.dim() != 2 or slot_of.shape[0] != M:
            raise ValueError("slot_of must be [M, topk], with rows and topk_weights")
        topk, n_rows = slot_of.shape[1], rows.shape[0]
        slot_p = _whole(slot_of, "slot_of", dev, torch.int32, M * topk)
        weights_p = _whole(topk_weights, "topk_weights", dev, torch.float32, M * topk)
        rows_p, ld_rows = _rows(rows, "rows", dev, None, H)
        if n_rows == 0:
            rows_p = residual_p        # an empty tensor has no address; no slot reaches it
        if shared is not None:
            shared_p, ld_shared = _rows(shared, "shared", dev, M, H, dtype)
    elif topk_weights is not None or shared is not None:
        raise ValueError("topk_weights and shared go with slot_of")
    elif rows is not None:
        rows_p, ld_rows = _rows(rows, "rows", dev, M, H)
    if post_weight is not None:
        post_p = _whole(post_weight, "post_weight", dev, wt, H)
    if post_bias is not None:
        post_b = _whole(post_bias, "post_bias", dev, wt, H)
    if gate is not None:
        gate_p = _dev(gate, "gate", dev, wt)
        shape, step = gate.shape, gate.stride()
        if len(shape) < 2:
            shape, step = (1, *(shape or (1,))), (0, *(step or (0,)))
        if len(shape) != 2 or shape[0] not in (1, M) or shape[1] not in (1, H):
            raise ValueError("gate must broadcast over [M, H]")
        gate_row = step[0] if shape[0] > 1 else 0
        gate_col = step[1] if shape[1] > 1 else 0
    if pre_weight is not None:
        pre_p = _whole(pre_weight, "pre_weight", dev, wt, H)
        if pre_bias is not None:
            pre_b = _whole(pre_bias, "pre_bias", dev, wt, H)
        if out is None:
            out = torch.empty((M, H), dtype=dtype, device=residual.device)
        out_p, ld_out = _rows(out, "out", dev, M, H, dtype)
    elif pre_bias is not None or out is not None:
        raise ValueError("pre_bias and out go with pre_weight")
    if rows is not None:
        if residual_out is None:
            residual_out = torch.empty((M, H), dtype=residual.dtype, device=residual.device)
        res_out_p, ld_res_out = _rows(residual_out, "residual_out", dev, M, H, residual.dtype)
    elif residual_out is not None:
        raise ValueError("residual_out goes with rows")
    # moe_norm_args as the compiler lays it out
    st = _lib.load().moe_block_norm(_lib.NORM_ARGS.pack(
        M, H, code, _code(residual, "residual"), _CODE.get(wt, -1), kind, eps, scale, weight_offset,
        residual_p, ld_residual, rows_p, ld_rows, slot_p, weights_p, topk, n_rows, shared_p, ld_shared,
        post_p, post_b, gate_p, gate_row, gate_col, pre_p, pre_b, res_out_p, ld_res_out, out_p, ld_out),
        _stream(stream, dev))
    if st:
        _check(st, "moe_block_norm")
    return residual_out, out


def moe_block_norm_set_wait_probe(ns):
    _check(_lib.load().moe_block_norm_set_wait_probe(int(ns)), "moe_block_norm_set_wait_probe")


def moe_block_norm_get_device_error(stream=None):
    """(status, code) of the device error word of moe_block_norm's calls on the current device, which
    is cleared."""
    code = ctypes.c_int()
    st = _lib.load().moe_block_norm_get_device_error(_stream(stream, torch.cuda.current_device()),
                                                     ctypes.byref(code))
    return st, code.value
