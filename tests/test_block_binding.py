"""The binding of the 16-bit block before it calls the library: devices of the operands.  No GPU: the tensors say that they are on one,
and the library records its arguments."""
import pytest

torch = pytest.importorskip("torch")

from serving_route_count_gb300 import _lib, block  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class On0(torch.Tensor):
    at = 0

    def get_device(self):
        return self.at


class On1(On0):
    at = 1


class FakeLibrary:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name != "moe_destroy_grouped":                   # of other tests' plans, collected here
                self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    fake = FakeLibrary()
    monkeypatch.setattr(_lib, "load", lambda: fake)
    monkeypatch.setattr(block, "_current_device", lambda: 0)
    return fake


def t(shape, dtype=BF16, on=On0):
    return torch.zeros(shape, dtype=dtype).as_subclass(on)


def grouped(on=0):
    op = block.MoEGrouped.__new__(block.MoEGrouped)
    op.E, op.N, op.K, op.cols, op.dtype, op._dev = 2, 8, 16, 8, BF16, on
    op.scratch, op.plan = t(4096, torch.uint8, On1 if on else On0), None
    op._fixed = (1, op.scratch.data_ptr(), 4096)
    return op


def operands():
    """{entry point: (its tensors by argument, other arguments)}"""
    return {
        block.moe_router: (dict(logits=t((4, 8), F32), bias=t(8, F32), ids=t((4, 2), I32), weights=t((4, 2), F32)),
                           dict(topk=2, score=block.MOE_SCORE_SIGMOID)),
        block.moe_group: (dict(topk_ids=t((4, 2), I32), offsets=t(9, I32), perm=t(8, I32), slot_of=t((4, 2), I32)), dict(E=8)),
        grouped(): (dict(x=t((4, 16)), w=t((2, 8, 16)), offsets=t(3, I32), perm=t(8, I32), out=t((8, 8))), dict(topk=2)),
        block.moe_block_norm: (dict(residual=t((4, 16)), rows=t((8, 16)), slot_of=t((4, 2), I32), topk_weights=t((4, 2), F32), shared=t((4, 16)),
                                    post_weight=t(16), post_bias=t(16), gate=t((4, 1)), pre_weight=t(16), pre_bias=t(16),
                                    residual_out=t((4, 16)), out=t((4, 16))), {}),
    }


def test_operands_of_one_device(lib):
    for call, (tensors, other) in operands().items():
        n = len(lib.calls)
        call(**tensors, **other, stream=7)
        assert len(lib.calls) == n + 1 and 7 in lib.calls[-1][1]
        for name, v in tensors.items():
            for moved in (v.as_subclass(On1), v.as_subclass(torch.Tensor)):             # another GPU; the host
                with pytest.raises(ValueError, match=name):
                    call(**{**tensors, name: moved}, **other, stream=7)
        assert len(lib.calls) == n + 1


def test_the_operands_device_is_the_current_one(lib, monkeypatch):
    for call, (tensors, other) in operands().items():
        if isinstance(call, block.MoEGrouped):
            call = grouped(1)
        elsewhere = {k: v.as_subclass(On1) for k, v in tensors.items()}
        with pytest.raises(ValueError, match="current device"):
            call(**elsewhere, **other, stream=7)
        assert not lib.calls
    monkeypatch.setattr(block, "_current_device", lambda: 1)
    for call, (tensors, other) in operands().items():
        if isinstance(call, block.MoEGrouped):
            with pytest.raises(ValueError, match="scratch"):
                call(**{k: v.as_subclass(On1) for k, v in tensors.items()}, **other, stream=7)
            call = grouped(1)
        call(**{k: v.as_subclass(On1) for k, v in tensors.items()}, **other, stream=7)
    assert len(lib.calls) == 4
    with pytest.raises(ValueError, match="current device"):
        block.moe_grouped_get_device_error(1, t(4096, torch.uint8), stream=7)


def test_the_stream_is_of_the_operands_device(monkeypatch):
    class Stream:
        cuda_stream = 77

        def __init__(self, device_index):
            self.device_index = device_index

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    assert block._stream(Stream(0), 0) == 77 and block._stream(5, 0) == 5
    with pytest.raises(ValueError, match="stream"):
        block._stream(Stream(1), 0)


@pytest.mark.parametrize("residual,weight,out", [(F32, F32, BF16), (F32, BF16, BF16), (F32, torch.float16, torch.float16), (BF16, F32, BF16),
                                                 (torch.float16, F32, torch.float16), (torch.float16, torch.float16, torch.float16)])
def test_type_of_a_norm_before_a_block(lib, monkeypatch, residual, weight, out):
    """Without rows and without out, something has to name out's 16-bit type: the residual, the weight, else bf16."""
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: empty(*a, **kw).as_subclass(On0))
    r, z = block.moe_block_norm(t((4, 16), residual), pre_weight=t(16, weight), stream=7)
    assert r is None and z.dtype == out
    code = {BF16: 0, torch.float16: 1, F32: 2}
    assert _lib.NORM_ARGS.unpack(lib.calls[0][1][0])[2:5] == (code[out], code[residual], code[weight])


@pytest.mark.parametrize("E,N,K,of,ldw", [(2, 1, 16, lambda: t((2, 24))[:, :16].unsqueeze(1), 24), (2, 1, 16, lambda: t((2, 5, 16))[:, :1], 80),
                                          (1, 1, 16, lambda: t((1, 1, 16)).as_strided((1, 1, 16), (3, 2, 1)), 16), (1, 8, 16, lambda: t((1, 8, 24))[..., :16], 24),
                                          (2, 8, 16, lambda: t((2, 8, 16)), 16)])
def test_stride_of_weight_rows(lib, E, N, K, of, ldw):
    """An expert of one row: rows are as far apart as experts are, whatever the middle dimension's stride is."""
    op = grouped()
    op.E, op.N, op.K, op.cols = E, N, K, N
    w = of()
    assert w.shape == (E, N, K)
    op(t((4, K)), w, t(E + 1, I32), out=t((4, N)), stream=7)
    assert lib.calls[0][1][7] == ldw
    if E > 1 and N > 1:
        with pytest.raises(ValueError, match="apart"):
            op(t((4, K)), t((E, N + 1, K))[:, :N], t(E + 1, I32), out=t((4, N)), stream=7)


@pytest.mark.parametrize("shape,row,col", [((), 0, 0), ((1,), 0, 0), ((16,), 0, 1), ((1, 1), 0, 0), ((1, 16), 0, 1), ((4, 1), 1, 0), ((4, 16), 16, 1)])
def test_gates_that_broadcast(lib, shape, row, col):
    """Any shape that broadcasts over [M, H], a scalar among them."""
    block.moe_block_norm(t((4, 16)), t((4, 16)), gate=t(shape), residual_out=t((4, 16)), stream=7)
    names = ("M H dtype residual_dtype weight_dtype kind eps scale weight_offset residual ld_residual rows ld_rows slot_of topk_weights topk n_rows "
             "shared ld_shared post_weight post_bias gate gate_row gate_col").split()
    args = dict(zip(names, _lib.NORM_ARGS.unpack(lib.calls[0][1][0])))
    assert args["gate"] and (args["gate_row"], args["gate_col"]) == (row, col)


@pytest.mark.parametrize("shape", [(4,), (2, 16), (4, 8), (1, 4, 16)])
def test_gates_that_do_not(lib, shape):
    with pytest.raises(ValueError, match="gate"):
        block.moe_block_norm(t((4, 16)), t((4, 16)), gate=t(shape), residual_out=t((4, 16)), stream=7)
