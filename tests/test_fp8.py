"""8-bit products with block scales, and the quantisation to that form, against their definitions
(oracle/fp8.py).

Tolerances, from the arithmetic: codes and scales are equal to the fp32 quotients' (IEEE divisions, to nearest).
A product is an fp32 sum of K terms in any order, each block's sum scaled once by a product of two scales
that is rounded to fp32: within (K + 3) * 2^-24 * sum |terms|; then one rounding to the output type (bf16 2^-8,
f16 2^-11 and half of its smallest step)."""
import math

import numpy as np
import pytest

from oracle import block as B
from oracle import fp8 as F

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": (2.0 ** -8, 0.0), "f16": (2.0 ** -11, 2.0 ** -25)}
EPS32 = 2.0 ** -24
E4M3 = torch.float8_e4m3fn
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


def codes(q):
    return q.detach().cpu().contiguous().view(torch.uint8).numpy()


# ------------------------------------------------------------------------------------ oracle pins

def test_oracle_by_hand():
    x = np.zeros((2, 130), np.float32)
    x[0, :3], x[0, 129], x[1, 0] = [448.0, -1.0, 0.3], 7.0, np.nan
    q, s = F.quant_rows(x)
    assert s.tolist() == [[1.0, 2.0 ** -6], [2.0 ** -126, 2.0 ** -126]]
    assert q[0, :4].tolist() == [0x7E, 0xB8, 0x2A, 0] and q[0, 129] == 0x7E and q[1, 0] == 0x7F
    assert F.values(q, s)[0, 2] == 0.3125 and F.values(q, s)[0, 129] == 7.0
    q, s = F.quant_tiles(np.full((129, 1), 2.0, np.float32))
    assert s.shape == (2, 1) and np.all(q == 0x7E) and np.all(s == np.float32(2) / np.float32(448))
    w = F.weight_values(np.full((1, 4, 1), 0x38, np.uint8), np.array([[[2.0], [3.0]]], np.float32), True)
    assert w[0, :, 0].tolist() == [2, 2, 3, 3]


# ------------------------------------------------------------------------------------ arguments, without a GPU

def test_arguments():
    import serving_route_count_gb300 as m
    from serving_route_count_gb300 import _lib, build
    build.build()
    lib = _lib.load()
    p = m.moe_fp8_plan(2, 128, 256, m.MOE_DTYPE_BF16, 0, 0, math.inf, 1.0, 0.0, 16)
    assert m.moe_fp8_scratch_bytes(p) >= 4096
    run = lambda plan=p, scratch=4096, size=1 << 40, x=1, ldx=256, rows=16, xs=1, ldxs=2, w=1, ldw=256, ws=1, off=1, perm=None, topk=1, out=1, ldo=128, S=16: (  # noqa: E731
        lib.moe_fp8_run(plan, scratch, size, x, ldx, rows, xs, ldxs, w, ldw, ws, off, perm, topk, out, ldo, S, None))
    assert run(S=0) == 0 and run(S=17) == 4
    for bad in (dict(plan=None), dict(S=-1), dict(scratch=None), dict(scratch=8), dict(size=4095), dict(x=None), dict(xs=None), dict(w=None),
                dict(ws=None), dict(out=None), dict(ldx=255), dict(ldxs=1), dict(ldw=255), dict(ldo=127), dict(rows=15), dict(off=None),
                dict(perm=1, topk=0), dict(perm=1, rows=0)):
        assert run(**bad) == 1, bad
    m.moe_fp8_set_wait_probe(p, 1_000_000_000)
    m.moe_fp8_set_wait_probe(p, 0)
    for plan, ns in ((p, 1_000_000_001), (None, 0)):
        with pytest.raises(m.MoEError) as e:
            m.moe_fp8_set_wait_probe(plan, ns)
        assert e.value.status == 1
    m.moe_destroy_fp8(p)
    for bad, status in (((0, 8, 8, 0, 0), 2), ((1025, 8, 8, 0, 0), 2), ((1, 0, 8, 0, 0), 2), ((1, 8, 0, 0, 0), 2), ((1, 7, 8, 0, 1), 2),
                        ((1, 8, 8, 2, 0), 3), ((1, 8, 8, 0, 5), 3)):
        E, N, K, dtype, act = bad
        with pytest.raises(m.MoEError) as e:
            m.moe_fp8_plan(E, N, K, dtype, act, 0, 1.0, 1.0, 0.0, 4)
        assert e.value.status == status, bad
    for limit, alpha, beta, layout in ((0.0, 1.0, 0.0, 0), (math.nan, 1.0, 0.0, 0), (1.0, math.inf, 0.0, 0), (1.0, 1.0, math.nan, 0), (1.0, 1.0, 0.0, 2)):
        with pytest.raises(m.MoEError) as e:
            m.moe_fp8_plan(1, 8, 8, 0, 1, layout, limit, alpha, beta, 4)
        assert e.value.status == 1
    quant = lambda x=1, dtype=0, ldx=256, E=1, rows=4, K=256, form=0, q=1, ldq=256, s=1, lds=2: (  # noqa: E731
        lib.moe_fp8_quant(x, dtype, ldx, E, rows, K, form, q, ldq, s, lds, None))
    assert quant(rows=0) == 0 and quant(E=0, form=1) == 0
    for bad, status in ((dict(dtype=3), 3), (dict(form=2), 1), (dict(E=2), 2), (dict(K=0), 2), (dict(rows=-1), 1), (dict(x=None), 1),
                        (dict(q=None), 1), (dict(s=None), 1), (dict(ldx=255), 1), (dict(ldq=255), 1), (dict(lds=1), 1),
                        (dict(E=1 << 16, rows=1 << 15, form=1), 2)):
        assert quant(**bad) == status, bad


# ------------------------------------------------------------------------------------ quantisation

def check_quant(moe, x, form, **kw):
    q, s = moe.moe_fp8_quant(x, form=form, **kw)
    x = x.detach().cpu().float().numpy()
    mats, oracle = (x, F.quant_tiles) if x.ndim == 3 else (x[None], F.quant_tiles if form == moe.MOE_FP8_TILES else F.quant_rows)
    want = [oracle(m) for m in mats]
    wq, ws = (np.stack([w[i] for w in want]).reshape(t.shape) for i, t in ((0, q), (1, s)))
    got = codes(q)
    nan = (wq & 0x7F) == 0x7F
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(got[~nan], wq[~nan]) and np.all((got[nan] & 0x7F) == 0x7F)
    return q, s


def activations(shape, dtype, seed):
    """Values over several binades, with many that lie in the middle of two codes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(torch.randn(shape[-1], generator=g))
    x[..., ::3] = torch.round(x[..., ::3] * 4) / 4
    return x.to(DT[dtype]).cuda()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 7168), (3, 127), (5, 128), (2, 129), (77, 576), (33, 1001), (1000, 264), (9, 4104)])
def test_quant_rows(moe, rows, K, dtype):
    check_quant(moe, activations((rows, K), dtype, rows + K), moe.MOE_FP8_ROWS)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (129, 257), (3, 64, 100), (2, 130, 1152), (1, 300, 1000), (5, 1, 17)])
def test_quant_tiles(moe, shape, dtype):
    check_quant(moe, activations(shape, dtype, sum(shape)), moe.MOE_FP8_TILES)


@gpu
@pytest.mark.parametrize("form", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quant_extremes(moe, form, dtype):
    """Zeros of both signs, the type's smallest and largest values, infinities and NaN in some blocks."""
    fi = torch.finfo(DT[dtype])
    x = torch.randn((260, 640), generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    x[0, :128] = 0
    x[1, :128] = -0.0
    x[2, 5], x[2, 200], x[2, 300], x[2, 500] = math.nan, math.inf, -math.inf, -math.nan
    x[3, :], x[4, :] = fi.max, -fi.max
    x[5, :] = fi.smallest_normal
    x[6, :] = fi.smallest_normal * fi.eps                       # the smallest subnormal
    x[7, :] = math.nan
    check_quant(moe, x.cuda(), form)


def next_to_middles(s, seed):
    """fp32 values, 127 to a row: middles of two codes times the row's scale s, up to 2 ulps off, of both signs."""
    rng = np.random.default_rng(seed)
    mids = np.concatenate([np.arange(1, 16, 2) * 2.0 ** -10] + [(8.5 + np.arange(8)) * 2.0 ** e for e in range(-9, 6)]).astype(np.float32)
    mids = mids[mids < 448]
    x = rng.choice(mids, (len(s), 127)) * s[:, None]                            # rounded to fp32 once
    return (x.view(np.int32) + rng.integers(-2, 3, x.shape, np.int32)).view(np.float32) * rng.choice(np.float32([-1, 1]), x.shape)


@gpu
@pytest.mark.parametrize("least", [2.0 ** -8, 2.0 ** -60 * (1 - 2.0 ** -12), 2.0 ** -100, 2.0 ** 100])
def test_quant_next_to_the_middle_of_two_codes(moe, least):
    """Scales of many mantissas, on both sides of the one from which a reciprocal replaces the division; codes
    and scales are those of the IEEE quotients, bit for bit."""
    rng = np.random.default_rng(5)
    s = np.concatenate((np.float32(least) * (1 + rng.random(8192)).astype(np.float32), np.float32(least) * (1 + np.arange(-64, 8192, 2) * np.float32(2.0 ** -23))))
    top = s.astype(np.float32) * np.float32(448)                                # the largest value, whose scale is within an ulp of s
    s = top / np.float32(448)
    x = torch.from_numpy(np.concatenate((top[:, None], next_to_middles(s, 6)), axis=1)).cuda()
    q, _ = check_quant(moe, x, moe.MOE_FP8_ROWS)
    shifted = torch.empty(x.numel() + 1, device="cuda")[1:].view(x.shape)       # rows off 16 bytes: the division throughout
    q2, _ = check_quant(moe, shifted.copy_(x), moe.MOE_FP8_ROWS)
    assert np.array_equal(codes(q), codes(q2))


@gpu
def test_quant_strides_and_outputs(moe):
    """Row strides of input and outputs, bases off 16 bytes; what lies between the rows stays as it was."""
    big = activations((50, 400), "bf16", 3)
    for shift in (0, 1, 8):
        x = big[:, shift:shift + 272]
        q = torch.full((50, 300), 1.0, device="cuda").to(E4M3)
        s = torch.full((50, 7), 5.0, device="cuda")
        for qs in (0, 3):
            check_quant(moe, x, moe.MOE_FP8_ROWS, q=q[:, qs:qs + 272], scale=s[:, 2:5])
            assert torch.all(q.float()[:, qs + 272:] == 1) and torch.all(s[:, :2] == 5) and torch.all(s[:, 5:] == 5)
        w = big[:, shift:shift + 272].unflatten(0, (2, 25))
        check_quant(moe, w, moe.MOE_FP8_TILES)


@gpu
def test_quant_refuses(moe):
    x = torch.zeros((4, 256), device="cuda")
    for kw in (dict(form=2), dict(q=torch.zeros((4, 255), device="cuda").to(E4M3)), dict(q=torch.zeros((4, 256), device="cuda")),
               dict(scale=torch.zeros((4, 3), device="cuda")), dict(scale=torch.zeros((4, 2), device="cuda").bfloat16())):
        with pytest.raises(ValueError):
            moe.moe_fp8_quant(x, **kw)
    for bad in (x.double(), x[0], x.t(), x[None], x.cpu()):
        with pytest.raises(ValueError):
            moe.moe_fp8_quant(bad)
    with pytest.raises(ValueError):
        moe.moe_fp8_quant(torch.zeros((4, 8, 256), device="cuda")[:, :4], form=moe.MOE_FP8_TILES)
    q, s = moe.moe_fp8_quant(torch.zeros((0, 256), device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0, 2)


# ------------------------------------------------------------------------------------ products

def padded(t, ld, shift=0):
    """t with rows ld apart, `shift` elements off the allocation; NaN codes (fp32 NaN) between them."""
    *lead, cols = t.shape
    ld = ld or cols
    rows = int(np.prod(lead))
    raw = t.contiguous().view(torch.uint8) if t.dtype == E4M3 else t
    flat = torch.full((rows * ld + shift,), 0x7F if t.dtype == E4M3 else math.nan, dtype=raw.dtype, device="cuda")
    view = flat[shift:].view(*lead, ld)[..., :cols]
    view.copy_(raw)
    return flat.view(E4M3)[shift:].view(*lead, ld)[..., :cols] if t.dtype == E4M3 else view


def case(E, N, K, counts, gather, topk=1, act=False, seed=0, pad=0, ldx=None, ldw=None, shift=0):
    """Operands of a product: some position rows of every expert, `pad` dropped ones."""
    g = torch.Generator().manual_seed(seed)
    n, S = sum(counts), sum(counts) + pad
    rows = -(-S // topk) if gather else S
    q = lambda *shape: (100 * torch.randn(shape, generator=g)).clamp(-448, 448).to(E4M3).cuda()  # noqa: E731
    s = lambda *shape: torch.exp(0.5 * torch.randn(shape, generator=g)).cuda()  # noqa: E731
    KB, tall = -(-K // 128), 2 * -(-(N // 2) // 128) if act else -(-N // 128)
    x, xs = padded(q(max(rows, 1), K), ldx, shift), s(max(rows, 1), KB) / 100
    w, ws = padded(q(E, N, K), ldw, shift), s(E, tall, KB) * (K ** -0.5 / 100)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    perm = None
    if gather:
        perm = torch.full((S,), -1, dtype=torch.int32)
        perm[:n] = torch.randperm(S, generator=g)[:n].to(torch.int32)
        perm = perm.cuda()
    return x, xs, w, ws, off, perm, S


def check(moe, x, xs, w, ws, off, perm, S, dtype="bf16", topk=1, act=False, layout=0, limit=math.inf, alpha=1.0, beta=0.0, out=None, op=None):
    E, N, K = w.shape
    op = op or moe.MoEFp8(E, N, K, max_rows=max(S, 1), dtype=DT[dtype], act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE, layout=layout,
                          swiglu_limit=limit, alpha=alpha, beta=beta)
    got = op(x[:S] if perm is None else x, xs[:S] if perm is None else xs, w, ws, offsets=off, perm=perm, topk=topk, out=out)
    assert op.device_error() == (0, 0)
    xv, wv = F.values(codes(x), xs.cpu().numpy()), F.weight_values(codes(w), ws.cpu().numpy(), act)
    o = [0, S] if off is None else off.cpu().numpy()
    ref, mag = B.grouped(xv, wv, o, S, None if perm is None else perm.cpu().numpy(), topk)
    err = (K + 3) * EPS32 * mag
    if act:
        a, b = ref[:, :N // 2], ref[:, N // 2:]
        ea, eb = err[:, :N // 2], err[:, N // 2:]
        u, g, eu, eg = (a, b, ea, eb) if layout == 0 else (b, a, eb, ea)
        ref = B.swiglu(u, g, limit, alpha, beta)
        gc, uc = np.minimum(g, limit), np.clip(u, -limit, limit) + beta
        # d/du = g' sigma <= |g'|; d/dg = u' (sigma + alpha g sigma (1 - sigma)), factor at most 1 + 0.28; the
        # second order of both errors; a few ulps of the fp32 formula, exp's alpha |g| among them
        err = np.abs(gc) * eu + 1.3 * np.abs(uc) * eg + 2 * eu * eg + 16 * EPS32 * (np.abs(ref) + np.abs(gc * uc) * EPS32)
        err = err + 4 * EPS32 * abs(alpha) * np.abs(gc if np.isfinite(limit) else g) * np.abs(ref)
    rel, tiny = HALF[dtype]
    y = f64(got)
    assert y.shape == ref.shape and np.all(np.isfinite(y))
    off_by = np.abs(y - ref) - (rel * (np.abs(ref) + err) + tiny + err)
    assert off_by.max(initial=-1.0) <= 0, float(off_by.max())
    assert torch.count_nonzero(got[int(o[-1]):]) == 0
    return got


RAGGED = [3, 0, 1, 70, 0, 16, 129, 33]


@gpu
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("dtype,N,K", [("bf16", 256, 128), ("f16", 130, 144), ("bf16", 1, 16), ("f16", 2, 1008), ("bf16", 576, 272),
                                       ("bf16", 94, 2304), ("bf16", 33, 5), ("f16", 34, 255), ("bf16", 300, 576)])
def test_product(moe, dtype, N, K, act, gather):
    if act and N % 2:
        N += 1
    topk = 3 if gather else 1
    check(moe, *case(8, N, K, RAGGED, gather, topk, act, seed=N + K, pad=11), dtype, topk, act)


@gpu
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("S", [1, 2, 17, 32, 33, 64, 65, 128, 200, 257, 600])
def test_dense(moe, S, act):
    """One matrix and no offsets; the same with offsets and with the weights as a matrix."""
    x, xs, w, ws, off, _, _ = case(1, 392, 592, [S], False, act=act, seed=S)
    op = moe.MoEFp8(1, 392, 592, max_rows=S, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE)
    got = check(moe, x, xs, w, ws, None, None, S, act=act, op=op)
    assert torch.equal(op(x, xs, w[0], ws[0], offsets=off), got)
    perm = torch.arange(S - 1, -1, -1, dtype=torch.int32, device="cuda")
    assert torch.equal(op(x, xs, w, ws, perm=perm), got.flip(0))


@gpu
@pytest.mark.parametrize("counts", [[0, 0, 0, 0], [1, 0, 0, 0], [0, 0, 0, 1], [1, 1, 1, 1], [700, 0, 0, 2], [31, 32, 33, 64],
                                    [65, 127, 128, 129], [255, 256, 257, 513]])
def test_product_row_counts(moe, counts):
    for act in (False, True):
        check(moe, *case(4, 320, 208, counts, True, 2, act, seed=sum(counts), pad=1), "bf16", 2, act, limit=1.0)


@gpu
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("counts,N,K", [([1] * 6, 8192, 1552), ([10, 20, 0, 30, 9, 15], 8192, 1552), ([40, 3, 0, 61, 8, 64], 5888, 1808),
                                        ([700, 256, 300, 1], 8000, 1424), ([300], 5376, 4112)])
def test_product_many_units(moe, counts, N, K, act):
    """More units than CTA pairs: whole units, units cut by K steps and joined, at every token-tile width."""
    x, xs, w, ws, off, perm, S = case(len(counts), N, K, counts, True, 2, act, seed=K)
    a = check(moe, x, xs, w, ws, off, perm, S, "bf16", 2, act, limit=2.0)
    rows = perm.long() // 2
    xi, xsi = x.view(torch.uint8)[rows].view(E4M3), xs[rows].contiguous()
    check(moe, xi, xsi, w, ws, off, None, S, "bf16", act=act, limit=2.0)                # the same rows in place
    op = moe.MoEFp8(len(counts), N, K, max_rows=S, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE, swiglu_limit=2.0)
    b = op(xi, xsi, w, ws, off)
    for _ in range(30):                                     # every schedule gives the same bits, and no wait gives up
        assert torch.equal(op(x, xs, w, ws, off, perm=perm, topk=2), a)
        assert torch.equal(op(xi, xsi, w, ws, off), b)
    assert op.device_error() == (0, 0)


@gpu
@pytest.mark.parametrize("layout", [0, 1])
def test_product_swiglu_options(moe, layout):
    check(moe, *case(3, 192, 320, [5, 40, 17], False, act=True, seed=9), act=True, layout=layout, limit=0.7, alpha=1.702, beta=1.0)


@gpu
@pytest.mark.parametrize("half", [1, 15, 64, 72, 128, 130, 200, 256])
def test_halves_have_tiles_of_their_own(moe, half):
    """Up and gate of any number of rows: their tiles do not run into one another."""
    check(moe, *case(2, 2 * half, 272, [20, 7], False, act=True, seed=half), act=True)


@gpu
@pytest.mark.parametrize("ldx,ldw,shift", [(160, 176, 0), (147, 144, 0), (144, 145, 0), (144, 144, 1)])
def test_product_strides_and_alignment(moe, ldx, ldw, shift):
    """Row strides, odd ones and bases off 16 bytes; what lies between the rows is NaN."""
    x, xs, w, ws, off, perm, S = case(4, 100, 144, [9, 0, 50, 2], True, 2, ldx=ldx, ldw=ldw, shift=shift)
    big = torch.full((S, 131), 7.0, dtype=torch.float16, device="cuda")
    check(moe, x, padded(xs, 5), w, ws, off, perm, S, "f16", 2, out=big[:, 3:103])
    assert torch.all(big[:, :3] == 7) and torch.all(big[:, 103:] == 7)


@gpu
@pytest.mark.parametrize("K", [1, 3, 63, 127, 129, 250])
@pytest.mark.parametrize("gather", [False, True])
def test_product_odd_k_in_aligned_rows(moe, K, gather):
    """K of any size on the tensor cores, in rows padded (with NaN) to 16 bytes."""
    ld = (K + 15) // 16 * 16 + 16
    topk = 2 if gather else 1
    for act in (False, True):
        check(moe, *case(5, 66, K, [4, 0, 33, 1, 90], gather, topk, act, ldx=ld, ldw=ld, seed=K), "bf16", topk, act)


@gpu
def test_product_neighbours_do_not_leak(moe):
    """NaN codes and infinite scales in rows and experts that a position does not use stay out of its result."""
    x, xs, w, ws, off, _, S = case(3, 160, 144, [5, 6, 7], False, seed=4)
    op = moe.MoEFp8(3, 160, 144, max_rows=S)
    want = op(x, xs, w, ws, off)
    x2, xs2, w2, ws2 = x.view(torch.uint8).clone(), xs.clone(), w.view(torch.uint8).clone(), ws.clone()
    x2[5:11], w2[1], ws2[1], xs2[5:11] = 0x7F, 0xFF, math.inf, math.inf
    got = op(x2.view(E4M3), xs2, w2.view(E4M3), ws2, off)
    keep = [i for i in range(S) if not 5 <= i < 11]
    assert torch.equal(got[keep], want[keep]) and torch.all(torch.isnan(got[5:11]))


@gpu
def test_product_past_32_bits(moe):
    """A weight tensor of more than 2^31 elements."""
    E, N, K = 5, 21504, 20480
    assert E * N * K > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda").view(E4M3)
    w[E - 1] = (100 * torch.randn((N, K), generator=g, device="cuda")).clamp(-448, 448).to(E4M3)
    ws = torch.rand((E, N // 128, K // 128), generator=g, device="cuda") + 0.5
    x = (100 * torch.randn((5, K), generator=g, device="cuda")).clamp(-448, 448).to(E4M3)
    xs = (torch.rand((5, K // 128), generator=g, device="cuda") + 0.5) * 1e-6
    off = torch.tensor([0, 2, 2, 2, 2, 5], dtype=torch.int32, device="cuda")
    got = moe.MoEFp8(E, N, K, max_rows=5)(x, xs, w, ws, off)
    assert torch.count_nonzero(got[:2]) == 0
    wide = lambda s, n: s.double().repeat_interleave(128, 1)[:, :n]  # noqa: E731
    xv = x[2:].double() * wide(xs[2:], K)
    wv = w[E - 1].double() * wide(ws[E - 1].repeat_interleave(128, 0), K)
    ref, mag = f64(xv @ wv.t()), f64(xv.abs() @ wv.abs().t())
    err = (K + 3) * EPS32 * mag
    assert np.all(np.abs(f64(got[2:]) - ref) <= 2.0 ** -8 * (np.abs(ref) + err) + err)


@gpu
def test_rows_past_32_bits(moe):
    """Quantisation and products of more than 2^31 values of x; the last rows are theirs."""
    rows, K, N = 300_003, 7200, 24
    assert rows * K > 1 << 31
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(4))
    q, s = moe.moe_fp8_quant(x)
    last = [0, 1, rows // 2, rows - 2, rows - 1]
    wq, ws = F.quant_rows(x[last].float().cpu().numpy())
    assert np.array_equal(codes(q.view(torch.uint8)[last]), wq) and np.array_equal(s[last].cpu().numpy(), ws)
    w, wscale = moe.moe_fp8_quant(torch.randn((N, K), device="cuda"), form=moe.MOE_FP8_TILES)
    op = moe.MoEFp8(1, N, K, max_rows=rows)
    got = op(q, s, w, wscale)
    assert op.device_error() == (0, 0)
    xv, wv = F.values(wq, ws), F.weight_values(codes(w)[None], wscale.cpu().numpy()[None], False)[0]
    ref, err = xv @ wv.T, (K + 3) * EPS32 * (np.abs(xv) @ np.abs(wv).T)
    assert np.all(np.abs(f64(got[last]) - ref) <= 2.0 ** -8 * (np.abs(ref) + err) + err)


@gpu
def test_two_at_once(moe):
    """Two plans' calls on two streams, and quantisation between them: nobody waits for another kernel."""
    made = [case(4, 512, 1040, [40, 300, 0, 7], True, 1, True, seed) for seed in (1, 2)]
    ops = [moe.MoEFp8(4, 512, 1040, max_rows=347, act=moe.MOE_ACT_SWIGLU) for _ in made]
    want = [op(*c[:5], perm=c[5]) for op, c in zip(ops, made)]
    h = torch.randn((5000, 7168), device="cuda").bfloat16()
    q, s = moe.moe_fp8_quant(h)
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for op, c, st in zip(ops, made, streams):
            with torch.cuda.stream(st):
                got.append(op(*c[:5], perm=c[5]))
                got.append(moe.moe_fp8_quant(h))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        if i % 2:
            assert torch.equal(g[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(g[1], s)
        else:
            assert torch.equal(g, want[i // 2 % 2])
    assert all(op.device_error() == (0, 0) for op in ops)


@gpu
def test_product_repeats_streams_and_graphs(moe):
    """One plan over calls of other sizes and offsets, on another stream, and replayed in a graph: every call
    gives the same bits again."""
    E, N, K = 6, 512, 640
    op = moe.MoEFp8(E, N, K, max_rows=400, act=moe.MOE_ACT_SWIGLU)
    calls = []
    for seed, counts in enumerate(([1, 0, 2, 0, 0, 1], [50, 3, 0, 100, 7, 64], [0, 0, 0, 0, 0, 399])):
        x, xs, w, ws, off, perm, S = case(E, N, K, counts, True, 2, True, seed)
        calls.append(((x, xs, w, ws, off, perm, 2), check(moe, x, xs, w, ws, off, perm, S, "bf16", 2, True, op=op)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for args, want in calls:
            assert torch.equal(op(*args), want)
            with torch.cuda.stream(side):
                got = op(*args)
            side.synchronize()
            assert torch.equal(got, want)
    args, want = calls[1]
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op(*args, out=out)
    for _ in range(3):
        out.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert op.device_error() == (0, 0)


@gpu
@pytest.mark.parametrize("K", [64, 65])                          # tensor cores, CUDA cores
def test_product_reports_bad_tables(moe, K):
    """Offsets out of order and permutation entries out of range set the device error word (the kernels check
    them before they address anything)."""
    x, xs, w, ws, off, perm, S = case(3, 64, K, [4, 4, 4], True, 2)
    op = moe.MoEFp8(3, 64, K, max_rows=S)
    for bad in (10 ** 6, -7):
        p = perm.clone()
        p[5] = bad
        op(x, xs, w, ws, off, perm=p, topk=2)
        assert op.device_error() == (8, 1)
    for o in ([0, 8, 4, 12], [0, 4, 8, 13], [-1, 4, 8, 12]):
        op(x, xs, w, ws, torch.tensor(o, dtype=torch.int32, device="cuda"), perm=perm, topk=2)
        assert op.device_error() == (8, 1)
    check(moe, x, xs, w, ws, off, perm, S, "bf16", 2, op=op)


@gpu
@pytest.mark.parametrize("dtype,act", [("bf16", True), ("f16", False)])
@pytest.mark.parametrize("counts,pad", [([1] * 8, 0), ([8] + [0] * 7, 0), ([0, 3, 0, 0, 2, 0, 0, 1], 2), ([0] * 7 + [1], 0), ([0] * 8, 4),
                                        ([2, 0, 0, 0, 0, 0, 0, 3], 3), ([9] + [0] * 7, 0)])
def test_product_of_a_few_positions(moe, counts, pad, dtype, act):
    """One token's slots, several of one expert, dropped ones; K that a warp's vectors do not divide."""
    for N, K in ((130, 1040), (2, 16), (2050, 144)):
        for gather in (False, True):
            topk = 4 if gather else 1
            check(moe, *case(8, N, K, counts, gather, topk, act, seed=N, pad=pad), dtype, topk, act, limit=2.0)


@gpu
@pytest.mark.parametrize("S", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("K", [16, 128, 528, 7184])
def test_dense_of_a_few_positions(moe, S, K):
    for N, act in ((5, False), (640, False), (384, True)):
        x, xs, w, ws, off, _, _ = case(1, N, K, [S], False, act=act, seed=S)
        got = check(moe, x, xs, w, ws, None, None, S, act=act)
        op = moe.MoEFp8(1, N, K, max_rows=8, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE)
        perm = torch.tensor([2 * i for i in reversed(range(S))], dtype=torch.int32, device="cuda")
        assert torch.equal(op(x, xs, w, ws, perm=perm, topk=2), got.flip(0))


@gpu
def test_few_positions_report_bad_tables(moe):
    x, xs, w, ws, off, perm, S = case(3, 64, 64, [2, 2, 2], True, 2)
    op = moe.MoEFp8(3, 64, 64, max_rows=S)
    for bad in (10 ** 6, -7):
        p = perm.clone()
        p[5] = bad
        op(x, xs, w, ws, off, perm=p, topk=2)
        assert op.device_error() == (8, 1)
    for o in ([0, 4, 2, 6], [0, 2, 4, 7], [-1, 2, 4, 6]):
        op(x, xs, w, ws, torch.tensor(o, dtype=torch.int32, device="cuda"), perm=perm, topk=2)
        assert op.device_error() == (8, 1)
    check(moe, x, xs, w, ws, off, perm, S, "bf16", 2, op=op)


@gpu
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,N,K,act", [([9, 0, 8], 512, 4096, True),             # units cut by K steps
                                            ([40, 300, 7], 8192, 512, False),         # more units than CTA pairs, whole ones first
                                            ([20, 400, 130], 1024, 8192, True)])      # tokens as M, cut units
def test_a_wait_that_runs_out(moe, counts, N, K, act, gather):
    """The first CTA pair's MMA issuer gives up a wait of 2 ms: the call ends with MOE_ERR_TIMEOUT in the error word, and the
    next one gives the result of a plan that never saw it."""
    x, xs, w, ws, off, perm, S = case(len(counts), N, K, counts, gather, 1, act, seed=K)
    new = lambda: moe.MoEFp8(len(counts), N, K, max_rows=S, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE)  # noqa: E731
    want, op = new()(x, xs, w, ws, off, perm=perm), new()
    moe.moe_fp8_set_wait_probe(op.plan, 2_000_000)
    op(x, xs, w, ws, off, perm=perm)
    assert op.device_error() == (7, 2)
    moe.moe_fp8_set_wait_probe(op.plan, 0)
    for _ in range(3):
        assert torch.equal(op(x, xs, w, ws, off, perm=perm), want)
    assert op.device_error() == (0, 0)


@gpu
def test_product_refuses(moe):
    x, xs, w, ws, off, perm, S = case(3, 64, 64, [4, 4, 4], True, 2)
    op = moe.MoEFp8(3, 64, 64, max_rows=S)
    good = dict(x=x, x_scale=xs, w=w, w_scale=ws, offsets=off, perm=perm, topk=2)
    op(**good)
    for bad in (dict(x=x[:, :63]), dict(x=x.float()), dict(x_scale=xs[:-1]), dict(x_scale=xs.half()), dict(w=w[:2]), dict(w=w[0]),
                dict(w=w.float()), dict(w_scale=ws[:2]), dict(w_scale=ws.half()), dict(offsets=None), dict(offsets=off[:3]),
                dict(offsets=off.long()), dict(perm=perm.long()), dict(out=torch.empty((S, 63), device="cuda").bfloat16()),
                dict(out=torch.empty((S, 64), device="cuda")), dict(x=x.cpu())):
        with pytest.raises(ValueError):
            op(**{**good, **bad})
    with pytest.raises(moe.MoEError) as e:
        op(**{**good, "topk": 0})
    assert e.value.status == 1
    with pytest.raises(moe.MoEError) as e:
        moe.MoEFp8(3, 64, 64, max_rows=S - 1)(**good)
    assert e.value.status == 4
    with pytest.raises(ValueError):
        moe.MoEFp8(3, 64, 64, max_rows=S, dtype=torch.float64)


# ------------------------------------------------------------------------------------ together

@gpu
@pytest.mark.parametrize("M", [1, 37])
def test_block_of_8_bit_experts_and_a_shared_one(moe, M):
    """Router, grouping, quantised rows, 8-bit experts, a 16-bit shared expert, combine and norms: every operator takes
    what the one before it left.  Each stage is within its own roundings of the 64-bit form of what it was given."""
    E, H, I, k = 12, 512, 200, 3
    g = torch.Generator(device="cuda").manual_seed(M)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    w13, w2 = rnd(E, 2 * I, H) * H ** -0.5, rnd(E, H, I) * I ** -0.5
    halves = [moe.moe_fp8_quant(h.contiguous(), form=moe.MOE_FP8_TILES) for h in w13.chunk(2, dim=1)]
    q13 = torch.cat([h[0].view(torch.uint8) for h in halves], dim=1).view(E4M3)
    s13 = torch.cat([h[1] for h in halves], dim=1)
    q2, s2 = moe.moe_fp8_quant(w2, form=moe.MOE_FP8_TILES)
    s13w, s2w = rnd(2 * I, H).bfloat16() * H ** -0.5, rnd(H, I).bfloat16() * I ** -0.5
    r, h, post, pre = rnd(M, H).bfloat16(), rnd(M, H).bfloat16(), rnd(H).bfloat16(), rnd(H).bfloat16()
    up = moe.MoEFp8(E, 2 * I, H, M * k, act=moe.MOE_ACT_SWIGLU)
    down = moe.MoEFp8(E, H, I, M * k)
    shared = moe.MoEFeedForward(H, I, M)

    def call():
        ids, w = moe.moe_router(logits, k)
        off, perm, slot = moe.moe_group(ids, E)
        hq, hs = moe.moe_fp8_quant(h)
        u = up(hq, hs, q13, s13, off, perm=perm, topk=k)
        uq, us = moe.moe_fp8_quant(u)
        y = down(uq, us, q2, s2, off)
        z = shared(h, s13w, s2w)
        return moe.moe_block_norm(r, y, slot_of=slot, topk_weights=w, shared=z, post_weight=post, pre_weight=pre), (ids, w, off, perm, slot, u, y, z)

    logits = rnd(M, E)
    (r1, h1), (ids, w, off, perm, slot, u, y, z) = call()
    assert up.device_error() == down.device_error() == shared.device_error() == (0, 0)
    hq, hs = F.quant_rows(h.float().cpu().numpy())
    a, _ = B.grouped(F.values(hq, hs), F.weight_values(codes(q13), s13.cpu().numpy(), True), off.cpu().numpy(), M * k, perm.cpu().numpy(), k)
    near = lambda got, ref, t: np.linalg.norm(f64(got) - ref) <= t * np.linalg.norm(ref)  # noqa: E731
    assert near(u, B.swiglu(a[:, :I], a[:, I:]), 2.0 ** -8)
    uq, us = F.quant_rows(u.float().cpu().numpy())
    b, _ = B.grouped(F.values(uq, us), F.weight_values(codes(q2), s2.cpu().numpy(), False), off.cpu().numpy(), M * k)
    assert near(y, b, 2.0 ** -8)
    p = f64(h) @ f64(s13w).T
    assert near(z, B.swiglu(p[:, :I], p[:, I:]) @ f64(s2w).T, 2.0 ** -7)
    c, _ = B.combine(f64(y), slot.cpu().numpy(), f64(w), f64(z))
    ref_r = f64(r) + B.norm(c, f64(post))
    assert near(r1, ref_r, 2.0 ** -8) and near(h1, B.norm(ref_r, f64(pre)), 2.0 ** -8)
    # the same captured and replayed
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (rg, hg), _ = call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(rg, r1) and torch.equal(hg, h1)
