"""The bindings of the 8-bit products and of the feed-forward block before they call the library: devices of the operands.  No GPU: the
tensors say that they are on one, and the library records its arguments."""
import pytest

torch = pytest.importorskip("torch")

from serving_route_count_gb300 import _lib, block, feed_forward, fp8  # noqa: E402

BF16, F32, I32, E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


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
            if not name.startswith("moe_destroy"):              # of other tests' plans, collected here
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
    return torch.zeros(shape, dtype=F32).to(dtype).as_subclass(on)


def product(on=0, E=2):
    op = fp8.MoEFp8.__new__(fp8.MoEFp8)
    op.E, op.N, op.K, op.cols, op.dtype, op._dev, op.blocks, op.tall = E, 8, 144, 8, BF16, on, 2, 1
    op.scratch, op.plan = t(4096, torch.uint8, On1 if on else On0), None
    op._fixed = (1, op.scratch.data_ptr(), 4096)
    return op


def feed(on=0):
    op = feed_forward.MoEFeedForward.__new__(feed_forward.MoEFeedForward)
    op.H, op.I, op.dtype, op._dev = 16, 8, BF16, on
    op.scratch, op.plan = t(4096, torch.uint8, On1 if on else On0), None
    op._fixed = (1, op.scratch.data_ptr(), 4096)
    return op


def operands(on=0):
    """[(entry point, its tensors by argument, other arguments)]"""
    ff = dict(x=t((4, 16)), w13=t((16, 16)), w2=t((16, 8)))
    p, f = product(on), feed(on)
    return [
        (fp8.moe_fp8_quant, dict(x=t((4, 144)), q=t((4, 144), E4M3), scale=t((4, 2), F32)), {}),
        (fp8.moe_fp8_quant, dict(x=t((2, 4, 144)), q=t((2, 4, 144), E4M3), scale=t((2, 1, 2), F32)), dict(form=fp8.MOE_FP8_TILES)),
        (p, dict(x=t((4, 144), E4M3), x_scale=t((4, 2), F32), w=t((2, 8, 144), E4M3), w_scale=t((2, 1, 2), F32), offsets=t(3, I32),
                 perm=t(8, I32), out=t((8, 8))), dict(topk=2)),
        (f, dict(**ff, out=t((4, 16))), {}),
        (f.backward, dict(dy=t((4, 16)), **ff, dx=t((4, 16)), dw13=t((16, 16)), dw2=t((16, 8))), dict(saved=(t((4, 16), F32), t((4, 8))))),
    ]


def test_operands_of_one_device(lib):
    for call, tensors, other in operands():
        n = len(lib.calls)
        call(**tensors, **other, stream=7)
        assert len(lib.calls) == n + 1 and 7 in lib.calls[-1][1]
        for name, v in tensors.items():
            for moved in (v.as_subclass(On1), v.as_subclass(torch.Tensor)):             # another GPU; the host
                with pytest.raises(ValueError, match=name):
                    call(**{**tensors, name: moved}, **other, stream=7)
        assert len(lib.calls) == n + 1
    f = feed()
    good = (t((4, 16), F32), t((4, 8)))
    for i in range(2):
        bad = list(good)
        bad[i] = bad[i].as_subclass(On1)
        ff = operands()[3][1]
        with pytest.raises(ValueError, match="saved"):
            f.forward(ff["x"], ff["w13"], ff["w2"], out=ff["out"], saved=tuple(bad), stream=7)


def test_the_operands_device_is_the_current_one(lib, monkeypatch):
    for call, tensors, other in operands(1):
        other = {k: tuple(v.as_subclass(On1) for v in o) if k == "saved" else o for k, o in other.items()}
        elsewhere = {k: v.as_subclass(On1) for k, v in tensors.items()}
        with pytest.raises(ValueError, match="current device"):
            call(**elsewhere, **other, stream=7)
    assert not lib.calls
    monkeypatch.setattr(block, "_current_device", lambda: 1)
    for on in (0, 1):
        for call, tensors, other in operands(on):
            other = {k: tuple(v.as_subclass(On1) for v in o) if k == "saved" else o for k, o in other.items()}
            elsewhere = {k: v.as_subclass(On1) for k, v in tensors.items()}
            if on == 0 and call is not fp8.moe_fp8_quant:
                with pytest.raises(ValueError, match="scratch"):
                    call(**elsewhere, **other, stream=7)
            else:
                call(**elsewhere, **other, stream=7)
    assert len(lib.calls) == 2 + 5
    for get in (fp8.moe_fp8_get_device_error, feed_forward.moe_ff_get_device_error):
        with pytest.raises(ValueError, match="current device"):
            get(1, t(4096, torch.uint8), stream=7)


@pytest.mark.parametrize("w,ldw", [(lambda: t((8, 144), E4M3), 144), (lambda: t((8, 160), E4M3)[:, :144], 160), (lambda: t((1, 8, 144), E4M3), 144)])
def test_one_matrix(lib, w, ldw):
    """E = 1: weights with or without the experts' dimension, and no offsets."""
    product(E=1)(t((4, 144), E4M3), t((4, 2), F32), w(), t((1, 2), F32), out=t((4, 8)), stream=7)
    assert lib.calls[0][1][9] == ldw and lib.calls[0][1][11] is None
    with pytest.raises(ValueError, match="offsets"):
        product()(t((4, 144), E4M3), t((4, 2), F32), t((2, 8, 144), E4M3), t((2, 1, 2), F32), out=t((4, 8)), stream=7)


def large(shape, dtype=BF16):
    """A tensor with sizes alone."""
    return torch.empty(shape, dtype=dtype, device="meta").as_subclass(On0)


@pytest.mark.parametrize("rows", [1 << 31, (1 << 32) + 5])
def test_rows_past_31_bits(lib, rows):
    """The library takes 32-bit integers: more rows are refused and not cut (2^32 + 5 of them would be 5)."""
    x, xs = large((rows, 144), E4M3), large((rows, 2), F32)
    w, ws = t((2, 8, 144), E4M3), t((2, 1, 2), F32)
    ff = operands()[4][1]
    pre, h = large((rows, 16), F32), large((rows, 8))
    for call in (lambda: fp8.moe_fp8_quant(large((rows, 1)), stream=7), lambda: fp8.moe_fp8_quant(large((rows, 1)), form=fp8.MOE_FP8_TILES, stream=7),
                 lambda: fp8.moe_fp8_quant(large((1, rows)), stream=7), lambda: fp8.moe_fp8_quant(large((rows, 1, 1)), form=fp8.MOE_FP8_TILES, stream=7),
                 lambda: product()(x, xs, w, ws, offsets=t(3, I32), stream=7),
                 lambda: product()(t((4, 144), E4M3), t((4, 2), F32), w, ws, offsets=t(3, I32), perm=large(rows, I32), topk=2, stream=7),
                 lambda: feed()(large((rows, 16)), ff["w13"], ff["w2"], stream=7), lambda: feed().forward(large((rows, 16)), ff["w13"], ff["w2"], stream=7),
                 lambda: feed().backward(large((rows, 16)), large((rows, 16)), ff["w13"], ff["w2"], (pre, h), stream=7)):
        with pytest.raises(ValueError, match="below 2"):
            call()
    for E, N, K, most in ((rows, 8, 8, 8), (1, rows, 8, 8), (1, 8, rows, 8), (1, 8, 8, rows)):
        with pytest.raises(ValueError, match="below 2"):
            fp8.moe_fp8_plan(E, N, K, 0, 0, 0, 1.0, 1.0, 0.0, most)
        if E == 1:
            with pytest.raises(ValueError, match="below 2"):
                feed_forward.moe_ff_plan(N, K, 0, 0, 1.0, 1.0, 0.0, most)
    assert not lib.calls


def test_operands_that_no_gradient_takes(lib):
    """What the C call takes as NULL may be None; what a gradient needs may not."""
    _, tensors, other = operands()[4]
    pre, h = other["saved"]
    uses = dict(x=(0, 1, 0), w13=(1, 0, 0), w2=(1, 1, 0), pre=(1, 1, 0), h=(0, 0, 1))
    for need in [(a, b, c) for a in (False, True) for b in (False, True) for c in (False, True)]:
        kept = {k: v for k, v in tensors.items() if k not in ("dx", "dw13", "dw2") or need[("dx", "dw13", "dw2").index(k)]}
        have = {k: any(n and u for n, u in zip(need, use)) for k, use in uses.items()}
        kept.update({k: v if have[k] else None for k, v in kept.items() if k in uses})
        saved = (pre if have["pre"] else None, h if have["h"] else None)
        got = feed().backward(**kept, saved=saved if any(need) else None, need=need, stream=7)
        args = lib.calls[-1][1]
        assert [g is not None for g in got] == list(need)
        assert [args[i] is not None for i in (5, 7, 9, 11, 12)] == [have[k] for k in ("x", "w13", "w2", "pre", "h")]
        n = len(lib.calls)
        for k in uses:
            if have[k]:
                bad = {**kept, "saved": saved}
                if k in kept:
                    bad[k] = None
                else:
                    bad["saved"] = (None, saved[1]) if k == "pre" else (saved[0], None)
                with pytest.raises(ValueError, match="saved" if k in ("pre", "h") else k):
                    feed().backward(**bad, need=need, stream=7)
        assert len(lib.calls) == n


def test_gradients_left_out(lib):
    _, tensors, other = operands()[4]
    for need in ((True, False, False), (False, True, False), (False, False, True)):
        kept = {k: v for k, v in tensors.items() if k not in ("dx", "dw13", "dw2") or need[("dx", "dw13", "dw2").index(k)]}
        got = feed().backward(**kept, **other, need=need, stream=7)
        args = lib.calls[-1][1]
        assert [g is not None for g in got] == list(need) == [args[i] is not None for i in (13, 15, 17)]
