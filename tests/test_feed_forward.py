"""The gated feed-forward block and its gradients against their 64-bit definitions (oracle/feed_forward.py).

Tolerances, from the arithmetic.  One rounding to the operand type is within r (bf16 2^-8, f16 2^-11; f16 has half of its
smallest step, t = 2^-25, too); an fp32 sum of n terms is within n 2^-24 of the sum of their sizes.  Each stage is checked
against the 64-bit form of what it was given (the saved rows, for the later ones), so that roundings do not add up over
stages; where a product goes through rows that the call keeps to itself (du and dg), each of its terms is off by their rounding
at most, r |terms| summed."""
import math

import numpy as np
import pytest

from oracle import block as B
from oracle import feed_forward as O

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}
EPS32 = 2.0 ** -24
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from serving_route_count_gb300 import build
    build.build()
    import serving_route_count_gb300 as m
    return m


def f64(t):
    return t.detach().cpu().double().numpy()


def within(got, ref, dtype, err):
    rel, tiny = HALF[dtype]
    got = f64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got))
    off = np.abs(got - ref) - (rel * (np.abs(ref) + err) + tiny + err)
    assert off.max(initial=-1.0) <= 0, float(off.max())


# ------------------------------------------------------------------------------------ oracle pins

@pytest.mark.parametrize("limit,alpha,beta,layout", [(np.inf, 1.0, 0.0, 0), (0.8, 1.702, 1.0, 1)])
def test_oracle_gradients_by_differences(limit, alpha, beta, layout):
    rng = np.random.default_rng(3)
    M, H, I = 3, 5, 4
    args = [rng.standard_normal(s) for s in ((M, H), (2 * I, H), (H, I))]
    dy = rng.standard_normal((M, H))
    grads = O.backward(dy, *args, layout, limit, alpha, beta)
    f = lambda a: float(np.sum(dy * O.forward(*a, layout, limit, alpha, beta)[2]))  # noqa: E731
    for i, grad in enumerate(grads):
        for at in np.ndindex(*args[i].shape):
            lo, hi = [a.copy() for a in args], [a.copy() for a in args]
            lo[i][at] -= 1e-6
            hi[i][at] += 1e-6
            assert abs((f(hi) - f(lo)) / 2e-6 - grad[at]) < 1e-6


def test_oracle_by_hand():
    pre, h, y = O.forward(np.array([[2.0]]), np.array([[3.0], [0.0]]), np.array([[5.0]]))
    assert pre.tolist() == [[6.0, 0.0]] and h.tolist() == [[0.0]] and y.tolist() == [[0.0]]
    assert O.act_grad(pre, np.array([[1.0]])).tolist() == [[0.0, 3.0]]                  # dg = u sigmoid(0)
    assert O.act_grad(pre, np.array([[1.0]]), limit=5.0).tolist() == [[0.0, 2.5]]       # clamped up
    assert O.act_grad(np.array([[5.0, 5.0]]), np.array([[1.0]]), limit=5.0).all()       # the bound itself passes


# ------------------------------------------------------------------------------------ arguments, without a GPU

def test_arguments():
    import serving_route_count_gb300 as m
    from serving_route_count_gb300 import _lib, build
    build.build()
    lib = _lib.load()
    p = m.moe_ff_plan(64, 32, m.MOE_DTYPE_BF16, 0, math.inf, 1.0, 0.0, 16)
    assert m.moe_ff_scratch_bytes(p) >= 4096 + 16 * 64 * 2
    fwd = lambda plan=p, scratch=4096, size=1 << 40, x=1, ldx=64, w13=1, ld13=64, w2=1, ld2=32, pre=None, h=None, y=1, ldy=64, M=16: (  # noqa: E731
        lib.moe_ff_forward(plan, scratch, size, x, ldx, w13, ld13, w2, ld2, pre, h, y, ldy, M, None))
    assert fwd(M=0) == 0 and fwd(M=17) == 4
    for bad in (dict(plan=None), dict(M=-1), dict(scratch=None), dict(scratch=8), dict(size=4095), dict(x=None), dict(w13=None), dict(w2=None), dict(y=None),
                dict(ldx=63), dict(ld13=63), dict(ld2=31), dict(ldy=63), dict(pre=1), dict(h=1)):
        assert fwd(**bad) == 1, bad
    bwd = lambda plan=p, scratch=4096, size=1 << 40, dy=1, lddy=64, x=1, ldx=64, w13=1, ld13=64, w2=1, ld2=32, pre=1, h=1, dx=1, lddx=64, dw13=1, ldd13=64, dw2=1, ldd2=32, M=16: (  # noqa: E731
        lib.moe_ff_backward(plan, scratch, size, dy, lddy, x, ldx, w13, ld13, w2, ld2, pre, h, dx, lddx, dw13, ldd13, dw2, ldd2, M, None))
    assert bwd(M=17) == 4 and bwd(dx=None, dw13=None, dw2=None) == 0 and bwd(M=0, dw13=None, dw2=None) == 0
    for bad in (dict(plan=None), dict(M=-1), dict(scratch=None), dict(scratch=8), dict(size=4095), dict(dy=None), dict(x=None), dict(w13=None), dict(w2=None),
                dict(pre=None), dict(h=None), dict(lddy=63), dict(ldx=63), dict(ld13=63), dict(ld2=31), dict(lddx=63), dict(ldd13=63), dict(ldd2=31)):
        assert bwd(**bad) == 1, bad
    m.moe_ff_set_wait_probe(p, 1_000_000_000)
    m.moe_ff_set_wait_probe(p, 0)
    for plan, ns in ((p, 1_000_000_001), (None, 0)):
        with pytest.raises(m.MoEError) as e:
            m.moe_ff_set_wait_probe(plan, ns)
        assert e.value.status == 1
    m.moe_destroy_ff(p)
    for bad, status in (((0, 8, 0, 0, 1.0), 2), ((8, 0, 0, 0, 1.0), 2), ((8, 8, 2, 0, 1.0), 3), ((8, 8, 0, 2, 1.0), 1), ((8, 8, 0, 0, -1.0), 1),
                        ((8, 8, 0, 0, math.nan), 1), (((1 << 20) + 1, 8, 0, 0, 1.0), 2)):
        H, I, dtype, layout, limit = bad
        with pytest.raises(m.MoEError) as e:
            m.moe_ff_plan(H, I, dtype, layout, limit, 1.0, 0.0, 4)
        assert e.value.status == status, bad
    for alpha, beta in ((math.inf, 0.0), (1.0, math.nan)):
        with pytest.raises(m.MoEError):
            m.moe_ff_plan(8, 8, 0, 0, 1.0, alpha, beta, 4)


def test_scratch_bytes_by_rows():
    """A plan of a few tokens, as each layer of a decode step has one, does not hold the widest tile's pieces: 80 pairs x 2
    pieces x 2 CTAs x 128 rows in fp32 for each token of the tile, the first 4096 bytes and the rows between two products."""
    import serving_route_count_gb300 as m
    from serving_route_count_gb300 import build
    build.build()
    for max_rows, tile in ((0, 32), (1, 32), (32, 32), (33, 64), (64, 64), (65, 128), (128, 128), (129, 256), (4096, 256)):
        p = m.moe_ff_plan(7168, 1152, m.MOE_DTYPE_BF16, 0, math.inf, 1.0, 0.0, max_rows)
        need = 4096 + 80 * 2 * 2 * tile * 128 * 4 + max_rows * 2 * 1152 * 2
        assert need <= m.moe_ff_scratch_bytes(p) < need + 256
        m.moe_destroy_ff(p)


# ------------------------------------------------------------------------------------ both passes

def strided(t, ld, shift=0):
    """t with rows ld apart, `shift` elements off the allocation; NaN between them."""
    rows, cols = t.shape
    flat = torch.full((rows * (ld or cols) + shift,), math.nan, dtype=t.dtype, device="cuda")
    view = flat[shift:].view(rows, ld or cols)[:, :cols]
    view.copy_(t)
    return view


def operands(M, H, I, dtype, seed=0, ld=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda r, c, s: strided((s * torch.randn((r, c), generator=g)).to(DT[dtype]).cuda(), ld and c + ld, shift)  # noqa: E731
    return rnd(M, H, 1.0), rnd(2 * I, H, H ** -0.5), rnd(H, I, I ** -0.5), rnd(M, H, 1.0)


def check_forward(op, x, w13, w2, dtype, layout=0, limit=math.inf, alpha=1.0, beta=0.0, out=None):
    H, I = op.H, op.I
    y, (pre, h) = op.forward(x, w13, w2, out=out)
    assert op.device_error() == (0, 0)
    X, W13, W2 = f64(x), f64(w13), f64(w2)
    a = X @ W13.T
    ea = H * EPS32 * (np.abs(X) @ np.abs(W13).T)
    got = f64(pre)                                               # the sums themselves
    assert pre.dtype == torch.float32 and np.all(np.abs(got - a) <= ea)
    u, g, eu, eg = (*np.split(a, 2, 1), *np.split(ea, 2, 1)) if layout == 0 else (*np.split(a, 2, 1)[::-1], *np.split(ea, 2, 1)[::-1])
    gc, uc = np.minimum(g, limit), np.clip(u, -limit, limit) + beta
    ref = B.swiglu(u, g, limit, alpha, beta)
    # d/du = g' sigma <= |g'|; d/dg: factor at most 1 + 0.28; the second order of both; a few ulps of the fp32 formula, exp's
    # alpha |g| among them
    err = np.abs(gc) * eu + 1.3 * np.abs(uc) * eg + 2 * eu * eg + 16 * EPS32 * (np.abs(ref) + np.abs(gc * uc) * EPS32)
    err = err + 4 * EPS32 * abs(alpha) * np.abs(gc if math.isfinite(limit) else g) * np.abs(ref)
    within(h, ref, dtype, err)
    hs = f64(h)
    within(y, hs @ W2.T, dtype, I * EPS32 * (np.abs(hs) @ np.abs(W2).T))
    return y, (pre, h)


def check_backward(op, dy, x, w13, w2, saved, dtype, layout=0, limit=math.inf, alpha=1.0, beta=0.0, **kw):
    H, I, M = op.H, op.I, x.shape[0]
    dx, dw13, dw2 = op.backward(dy, x, w13, w2, saved, **kw)
    assert op.device_error() == (0, 0)
    DY, X, W13, W2, pre, h = (f64(t) for t in (dy, x, w13, w2, *saved))
    rel, tiny = HALF[dtype]
    dh = DY @ W2
    edh = H * EPS32 * (np.abs(DY) @ np.abs(W2))
    d = O.act_grad(pre, dh, layout, limit, alpha, beta)
    # relative errors of dh and of the formula's factors.  The factor of dg, s + a s (1 - s), loses up to 2^-23 of the sizes of
    # its two terms where they cancel, each within a few ulps (16, and exp's alpha |g|)
    per = np.abs(O.act_grad(pre, edh, layout, limit, alpha, beta))
    u, g = np.split(pre, 2, 1) if layout == 0 else np.split(pre, 2, 1)[::-1]
    gc, uc = np.minimum(g, limit), np.clip(u, -limit, limit) + beta
    s = B.sigmoid(alpha * gc)
    sizes = (np.abs(dh) + edh) * np.stack((np.abs(gc) * s, np.abs(uc) * (s + np.abs(alpha * gc) * s * (1 - s))))
    each = (16 + 4 * abs(alpha) * np.abs(gc)) * EPS32 * sizes
    each = np.concatenate(tuple(each) if layout == 0 else tuple(each[::-1]), axis=1)
    ed = per + each
    ed = ed + rel * (np.abs(d) + ed) + tiny                      # du and dg are rounded
    D = np.abs(d) + ed
    if dx is not None:
        within(dx, d @ W13, dtype, ed @ np.abs(W13) + 2 * I * EPS32 * (D @ np.abs(W13)))
    if dw13 is not None:
        within(dw13, d.T @ X, dtype, ed.T @ np.abs(X) + M * EPS32 * (D.T @ np.abs(X)))
    if dw2 is not None:
        within(dw2, DY.T @ h, dtype, M * EPS32 * (np.abs(DY).T @ np.abs(h)))
    return dx, dw13, dw2


def check(moe, M, H, I, dtype, seed=0, ld=0, shift=0, **kw):
    x, w13, w2, dy = operands(M, H, I, dtype, seed, ld, shift)
    names = {"limit": "swiglu_limit"}
    op = moe.MoEFeedForward(H, I, max_rows=M, dtype=DT[dtype], **{names.get(k, k): v for k, v in kw.items()})
    y, saved = check_forward(op, x, w13, w2, dtype, **kw)
    assert torch.equal(op(x, w13, w2), y)                        # without the saved rows
    grads = check_backward(op, dy, x, w13, w2, saved, dtype, **kw)
    return op, (x, w13, w2, dy), y, saved, grads


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,H,I", [(1, 64, 64), (1, 1, 1), (2, 264, 136), (17, 128, 72), (33, 520, 392), (100, 200, 600), (257, 264, 1032), (600, 136, 320),
                                   (5, 33, 7), (65, 72, 35), (70, 67, 64)])
def test_both_passes(moe, M, H, I, dtype):
    check(moe, M, H, I, dtype, seed=M + H)


@gpu
@pytest.mark.parametrize("H,I", [(128, 136), (77, 50)])          # tensor cores, CUDA cores
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("limit,alpha,beta", [(0.75, 1.0, 0.0), (0.7, 1.702, 1.0), (math.inf, -1.0, 0.5), (1e-3, 1.0, 0.0)])
def test_swiglu_options(moe, H, I, layout, limit, alpha, beta):
    """Limits that many values meet or lie next to (0.75 is a value of either type, 0.7 of neither)."""
    for dtype in ("bf16", "f16"):
        check(moe, 90, H, I, dtype, seed=layout, layout=layout, limit=limit, alpha=float(np.float32(alpha)), beta=beta)


@gpu
@pytest.mark.parametrize("ld", [16, 17])                         # tensor cores, CUDA cores
def test_sums_next_to_the_limit(moe, ld):
    """Sums just above and below a limit that both round to: x = (1, 2^-12, 0, ..) makes them from two weights.  What clamps is told
    by the sums, not by their roundings."""
    for dtype, step in (("bf16", 2.0 ** -12), ("f16", 2.0 ** -14)):
        for M in (1, 6):
            H = I = 16
            x = torch.zeros((M, H), dtype=DT[dtype])
            x[:, 0], x[:, 1] = 1, step
            w13 = torch.zeros((2 * I, H), dtype=DT[dtype])
            w13[:, 0], w13[0::2, 1], w13[1::2, 1] = 2.0, 1.0, -1.0
            w13[4:8] *= -1
            args = [strided(t.cuda(), ld) for t in (x, w13, torch.ones((H, I), dtype=DT[dtype]))]
            op = moe.MoEFeedForward(H, I, M, dtype=DT[dtype], swiglu_limit=2.0)
            y, (pre, h) = op.forward(*args)
            exact = f64(w13) @ f64(x)[0]
            assert np.array_equal(f64(pre), np.tile(exact, (M, 1)))
            _, dw13, _ = op.backward(torch.ones((M, H), dtype=DT[dtype], device="cuda"), *args, (pre, h))
            inside = np.concatenate((np.abs(exact[:I]) <= 2, exact[I:] <= 2))
            assert np.array_equal(f64(dw13)[:, 0] != 0, inside)


@gpu
@pytest.mark.parametrize("ld,shift", [(8, 0), (8, 8), (3, 0), (8, 1)])
def test_strides_and_alignment(moe, ld, shift):
    """Row strides, odd ones and bases off 16 bytes; what lies between the rows is NaN, and stays as it was in outputs."""
    M, H, I = 40, 136, 72
    x, w13, w2, dy = operands(M, H, I, "bf16", 5, ld, shift)
    op = moe.MoEFeedForward(H, I, max_rows=M)
    big = [torch.full((r, c + 5), 7.0, device="cuda").bfloat16() for r, c in ((M, H), (M, H), (2 * I, H), (H, I))]
    y, dx, dw13, dw2 = (b[:, 2:-3] for b in big)
    _, saved = check_forward(op, x, w13, w2, "bf16", out=y)
    check_backward(op, dy, x, w13, w2, saved, "bf16", dx=dx, dw13=dw13, dw2=dw2)
    for b in big:
        assert torch.all(b[:, :2] == 7) and torch.all(b[:, -3:] == 7)


@gpu
@pytest.mark.parametrize("M,H,I", [(1, 4096, 2304), (6, 7168, 576), (300, 2056, 1544), (777, 1544, 512), (1030, 1160, 2056), (2500, 520, 264)])
def test_many_units(moe, M, H, I):
    """More units than CTA pairs, units cut along K and joined, a long sum over tokens; every call gives the same bits."""
    op, (x, w13, w2, dy), y, saved, grads = check(moe, M, H, I, "bf16", seed=I, limit=1.5)
    for _ in range(20):
        y2, saved2 = op.forward(x, w13, w2)
        assert torch.equal(y2, y) and all(torch.equal(a, b) for a, b in zip(saved, saved2))
        assert all(torch.equal(a, b) for a, b in zip(grads, op.backward(dy, x, w13, w2, saved)))
    assert op.device_error() == (0, 0)


@gpu
@pytest.mark.parametrize("M,H,I", [(2, 4096, 1152), (3, 520, 2056), (4, 264, 8), (4, 8, 264), (5, 520, 136), (1, 7176, 40)])
def test_a_few_tokens(moe, M, H, I):
    """Up to four tokens and one more; a forward pass that is captured, between calls that change its input."""
    for layout in (0, 1):
        op, (x, w13, w2, dy), y, saved, grads = check(moe, M, H, I, "bf16", seed=M, layout=layout, limit=1.0)
    out = torch.empty_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op(x, w13, w2, out=out)
    keep = x.clone()
    for _ in range(3):
        x.zero_()
        graph.replay()
        assert torch.count_nonzero(out) == 0
        x.copy_(keep)
        graph.replay()
        assert torch.equal(out, y)
    assert op.device_error() == (0, 0)


@gpu
@pytest.mark.parametrize("max_rows", [1, 3, 32, 33, 64, 65, 128, 129])
@pytest.mark.parametrize("H,I", [(7168, 576), (520, 4104)])
def test_scratch_of_a_small_plan(moe, H, I, max_rows):
    """Nothing is written behind the bytes that a plan asks for, and the results are those of a plan of more tokens, bit for bit."""
    op, large = moe.MoEFeedForward(H, I, max_rows), moe.MoEFeedForward(H, I, 512)
    n = op.scratch.numel()
    buf = torch.full((n + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    buf[:4096] = 0
    op.scratch, op._fixed = buf[:n], (op.plan, buf.data_ptr(), n)
    for M in sorted({1, max_rows // 2 + 1, max_rows}):
        x, w13, w2, dy = operands(M, H, I, "bf16", M)
        y, saved = op.forward(x, w13, w2)
        want, kept = large.forward(x, w13, w2)
        assert torch.equal(y, want) and torch.equal(op(x, w13, w2), want) and all(torch.equal(a, b) for a, b in zip(saved, kept))
        for a, b in zip(op.backward(dy, x, w13, w2, saved), large.backward(dy, x, w13, w2, kept)):
            assert torch.equal(a, b)
    assert torch.all(buf[n:] == 0xA5) and op.device_error() == (0, 0)


@gpu
@pytest.mark.parametrize("H,I", [(7168, 576), (520, 1032), (100, 64)])       # 100: the first product's rows are off 16 bytes
def test_weights_written_just_before_the_call(moe, H, I):
    """The second product of one or two tokens may load its weights while the first one runs, and not before what wrote them
    is over: weights that change between calls, in the stream and in a graph."""
    op = moe.MoEFeedForward(H, I, max_rows=2)
    for M in (1, 2):
        x, w13, w2, _ = operands(M, H, I, "bf16", M)
        sets = [(w13, w2), (w13.flip(0).contiguous(), w2.flip(0).contiguous()), (-w13, 2 * w2)]
        want = [op(x, *s).clone() for s in sets]
        a, b = torch.empty_like(w13), torch.empty_like(w2)
        step = lambda s: (a.copy_(s[0]), b.copy_(s[1]), op(x, a, b))[2]  # noqa: E731
        got = [step(sets[i % 3]) for i in range(60)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, want[i % 3]) for i, g in enumerate(got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = [step(s) for s in sets]
        for _ in range(5):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert op.device_error() == (0, 0)


@gpu
@pytest.mark.parametrize("M,H,I", [(40, 4096, 256), (600, 1024, 4096)])
def test_a_wait_that_runs_out(moe, M, H, I):
    """The first CTA pair's MMA issuer gives up a wait of 2 ms in every product: both passes end with MOE_ERR_TIMEOUT in the error
    word, and the next ones give the results of a plan that never saw it."""
    op, (x, w13, w2, dy), y, saved, grads = check(moe, M, H, I, "bf16")
    moe.moe_ff_set_wait_probe(op.plan, 2_000_000)
    op(x, w13, w2)
    assert op.device_error() == (7, 2)
    op.backward(dy, x, w13, w2, saved)
    assert op.device_error() == (7, 2)
    moe.moe_ff_set_wait_probe(op.plan, 0)
    for _ in range(3):
        y2, s2 = op.forward(x, w13, w2)
        assert torch.equal(y2, y) and all(torch.equal(a, b) for a, b in zip(grads, op.backward(dy, x, w13, w2, s2)))
    assert op.device_error() == (0, 0)


@gpu
def test_gradients_by_differences(moe):
    """A step along a direction changes <dy, y> by the gradients' share: f16 rows, so that differences carry over the roundings."""
    M, H, I = 24, 64, 48
    x, w13, w2, dy = operands(M, H, I, "f16", 11)
    op = moe.MoEFeedForward(H, I, M, dtype=torch.float16)
    _, saved = op.forward(x, w13, w2)
    grads = op.backward(dy, x, w13, w2, saved)
    g = torch.Generator(device="cuda").manual_seed(2)
    args = [x, w13, w2]
    for i, grad in enumerate(grads):
        step = 0.05 * args[i].float().std() * torch.randn(args[i].shape, generator=g, device="cuda")
        hi, lo = list(args), list(args)
        hi[i], lo[i] = (args[i] + step).half(), (args[i] - step).half()
        moved = (hi[i].double() - lo[i].double())
        got = float(((op(*hi).double() - op(*lo).double()) * dy.double()).sum())
        want = float((grad.double() * moved).sum())
        # roundings of y, independent: sqrt(M H) of them of rms 2^-11 |y| / sqrt 3 times |dy|, four of each kind (h's among them);
        # the third derivative along a step of a twentieth of the values: below one percent of the gradient's norm
        noise = 8 * 2.0 ** -11 * math.sqrt(M * H)
        scale = float(grad.double().norm() * moved.norm()) / math.sqrt(moved.numel())
        assert abs(got - want) <= noise + 0.01 * max(abs(want), scale), (i, got, want)


@gpu
def test_past_32_bits(moe):
    """More than 2^31 values of x and y, and sums over as many tokens: two kinds of rows of x, so that the sums are known."""
    M, H, I = 270_001, 8192, 8
    assert M * H > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(6)
    kinds = torch.randn((2, H), generator=g, device="cuda").bfloat16()
    dkinds = torch.randn((2, H), generator=g, device="cuda").bfloat16()
    which = torch.zeros(M, dtype=torch.int64, device="cuda")
    which[-3:] = 1
    x, dy = kinds[which], torch.where(which[:, None] == 1, dkinds[1], torch.zeros_like(dkinds[0]))      # gradients of the last rows alone
    w13 = (torch.randn((2 * I, H), generator=g, device="cuda") * H ** -0.5).bfloat16()
    w2 = (torch.randn((H, I), generator=g, device="cuda") * I ** -0.5).bfloat16()
    op = moe.MoEFeedForward(H, I, max_rows=M)
    y, saved = op.forward(x, w13, w2)
    dx, dw13, dw2 = op.backward(dy, x, w13, w2, saved)
    assert op.device_error() == (0, 0)
    small = moe.MoEFeedForward(H, I, max_rows=8)
    tail = slice(M - 8, M)
    sub = [t[tail].contiguous() for t in (x, dy, *saved)]
    # rows of the tail: the same sums in whatever tiles, to a few units in the last place of their 16-bit roundings
    y8 = small(sub[0], w13, w2)
    dx8, dw138, dw28 = small.backward(sub[1], sub[0], w13, w2, (sub[2], sub[3]))
    for a, b in ((y[tail], y8), (dx[tail], dx8), (dw13, dw138), (dw2, dw28)):
        assert float((a.double() - b.double()).norm() / b.double().norm()) < 2.0 ** -7
    assert torch.count_nonzero(dx[:-3]) == 0 and torch.equal(y[0], y[M // 2])


@gpu
def test_two_at_once(moe):
    """Two plans' passes on two streams."""
    made = [operands(300, 1024, 520, "bf16", seed) for seed in (1, 2)]
    ops = [moe.MoEFeedForward(1024, 520, max_rows=300) for _ in made]

    def step(op, c):
        y, saved = op.forward(*c[:3])
        return (y, *op.backward(c[3], *c[:3], saved))

    want = [step(op, c) for op, c in zip(ops, made)]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for op, c, st in zip(ops, made, streams):
            with torch.cuda.stream(st):
                got.append(step(op, c))
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i % 2]))
    assert all(op.device_error() == (0, 0) for op in ops)


@gpu
def test_some_gradients(moe):
    op, (x, w13, w2, dy), y, saved, grads = check(moe, 30, 128, 64, "bf16")
    for need in ((True, False, False), (False, True, False), (False, False, True), (True, False, True), (False, False, False)):
        got = op.backward(dy, x, w13, w2, saved, need=need)
        for n, a, b in zip(need, got, grads):
            assert torch.equal(a, b) if n else a is None
    with pytest.raises(ValueError):
        op.backward(dy, x, w13, w2, saved, need=(False, True, True), dx=torch.empty_like(x))


@gpu
def test_some_gradients_from_what_they_take(moe):
    """A caller with frozen weights keeps neither x nor h, one with a frozen input no w13: the same bits."""
    op, (x, w13, w2, dy), y, (pre, h), (dx, dw13, dw2) = check(moe, 30, 128, 64, "bf16")
    assert torch.equal(op.backward(dy, None, w13, w2, (pre, None), need=(True, False, False))[0], dx)
    assert torch.equal(op.backward(dy, x, None, w2, (pre, None), need=(False, True, False))[1], dw13)
    assert torch.equal(op.backward(dy, None, None, None, (None, h), need=(False, False, True))[2], dw2)
    with pytest.raises(ValueError, match="w13"):
        op.backward(dy, x, None, w2, (pre, h))


@gpu
@pytest.mark.parametrize("H,I", [(64, 32), (33, 31)])
def test_no_tokens(moe, H, I):
    op = moe.MoEFeedForward(H, I, max_rows=4)
    x, w13, w2, dy = operands(0, H, I, "bf16")
    y, saved = op.forward(x, w13, w2)
    assert y.shape == (0, H) and op(x, w13, w2).shape == (0, H)
    big = torch.full((2 * I, H + 4), 7.0, device="cuda").bfloat16()
    dx, dw13, dw2 = op.backward(dy, x, w13, w2, saved, dw13=big[:, :H])
    assert dx.shape == (0, H) and torch.count_nonzero(dw13) == torch.count_nonzero(dw2) == 0 and torch.all(big[:, H:] == 7)


@gpu
@pytest.mark.parametrize("H,I", [(64, 72), (35, 72)])
def test_infinities_and_nan(moe, H, I):
    """A row of NaN or infinities stays in its own outputs and, in the gradients of the weights, spoils what sums over it."""
    x, w13, w2, dy = operands(9, H, I, "bf16", 3)
    op = moe.MoEFeedForward(H, I, max_rows=9)
    y, saved = op.forward(x, w13, w2)
    dx, _, _ = op.backward(dy, x, w13, w2, saved)
    x2, keep = x.clone(), [0, 1, 2, 4, 5, 6, 8]
    x2[3], x2[7] = math.nan, math.inf
    y2, saved2 = op.forward(x2, w13, w2)
    dx2, dw13, dw2 = op.backward(dy, x2, w13, w2, saved2)
    assert torch.equal(y2[keep], y[keep]) and torch.equal(dx2[keep], dx[keep])
    assert torch.all(torch.isnan(y2[3])) and torch.all(torch.isnan(dx2[3])) and torch.all(~torch.isfinite(y2[7]))
    assert torch.all(torch.isnan(dw13)) and torch.all(torch.isnan(dw2))


@gpu
@pytest.mark.parametrize("alpha", [1.0, -1.702])
def test_large_gates(moe, alpha):
    """Gates near the ends of the exponential's range, and of the type's."""
    g = torch.cat([torch.arange(-128, -40, 0.5), torch.arange(40, 128, 0.5), torch.tensor([0.0, -0.0, -1e30, 1e30])]).bfloat16()
    n = g.numel()
    H = 8
    x = torch.zeros((1, H), dtype=torch.bfloat16)
    x[0, 0] = 1
    w13, w2 = torch.zeros((2 * n, H), dtype=torch.bfloat16), torch.zeros((H, n), dtype=torch.bfloat16)
    w13[:n, 0], w13[n:, 0], w2[0] = 3.0, g, 1.0
    dy = torch.zeros((1, H), dtype=torch.bfloat16)
    dy[0, 0] = 1
    op = moe.MoEFeedForward(H, n, max_rows=1, alpha=alpha)
    args = [t.cuda() for t in (x, w13, w2)]
    _, saved = op.forward(*args)
    _, dw13, _ = op.backward(dy.cuda(), *args, saved)
    a = float(np.float32(alpha))
    with np.errstate(over="ignore", invalid="ignore"):
        ref = O.act_grad(np.concatenate((np.full(n, 3.0), g.double().numpy()))[None], np.ones((1, n)), alpha=a)[0]
        ref = np.where(np.isfinite(ref), ref, 0.0)               # 1e30 * 0 of the definition's second term is 0
        gd = np.abs(g.double().numpy())
        rel = np.concatenate((gd, gd)) * abs(a) * 4 * EPS32 + 40 * EPS32
        # rows of x and dy are one value each, so dW13's first column is d(up, gate) itself; a gradient below bf16's normal range
        # is within its step; the second term may lose its last places where exp is below fp32's normal range
        got = f64(dw13)[:, 0]
        tol = np.abs(ref) * (2 * 2.0 ** -8 + rel) + 3 * np.concatenate((gd, np.maximum(1, gd * abs(a)))) * 2.0 ** -126
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= tol), (np.abs(got - ref) - tol).max()


@gpu
def test_streams_and_graphs(moe):
    """Both passes on another stream and captured: the same bits."""
    op, (x, w13, w2, dy), y, saved, grads = check(moe, 130, 256, 136, "bf16")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        y2, s2 = op.forward(x, w13, w2)
        g2 = op.backward(dy, x, w13, w2, s2)
    side.synchronize()
    assert torch.equal(y2, y) and all(torch.equal(a, b) for a, b in zip(g2, grads))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, s3 = op.forward(x, w13, w2)
        g3 = op.backward(dy, x, w13, w2, s3)
    for _ in range(3):
        for t in (y3, *s3, *g3):
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y3, y) and all(torch.equal(a, b) for a, b in zip(g3, grads))
    assert op.device_error() == (0, 0)


@gpu
def test_refuses(moe):
    x, w13, w2, dy = operands(10, 64, 32, "bf16")
    op = moe.MoEFeedForward(64, 32, max_rows=10)
    y, saved = op.forward(x, w13, w2)
    for bad in ((x[:, :63], w13, w2), (x.half(), w13, w2), (x, w13[:63], w2), (x, w13.float(), w2), (x, w13, w2.t()), (x, w13, w2[:63]), (x.cpu(), w13, w2),
                (x, w13.cpu(), w2)):
        with pytest.raises(ValueError):
            op(*bad)
    with pytest.raises(ValueError):
        op.forward(x, w13, w2, saved=(saved[0][:9], saved[1]))
    for bad in (dict(dy=dy[:9]), dict(saved=(saved[0].bfloat16(), saved[1])), dict(x=x[:9]), dict(dw13=torch.empty_like(w2)), dict(dx=x.float())):
        with pytest.raises(ValueError):
            op.backward(**{**dict(dy=dy, x=x, w13=w13, w2=w2, saved=saved), **bad})
    with pytest.raises(moe.MoEError) as e:
        moe.MoEFeedForward(64, 32, max_rows=9)(x, w13, w2)
    assert e.value.status == 4
