"""The 16-bit block around the experts against its 64-bit definitions (oracle/block.py).

Tolerances, from the arithmetic: an output rounded once to a type of p significant bits is within
2^-p of its value (bf16 2^-8, f16 2^-11; plus half of f16's smallest step, 2^-25); an fp32 sum of K
terms in any order is within K * 2^-24 * sum |terms|."""
import math

import numpy as np
import pytest

from oracle import block as B

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": (2.0 ** -8, 0.0), "f16": (2.0 ** -11, 2.0 ** -25), "f32": (2.0 ** -24, 0.0)}
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
    """|got - ref| <= rounding of ref (and of what lies within err of it) + err, element by element."""
    rel, tiny = HALF[dtype]
    got, ref, err = f64(got), np.asarray(ref), np.asarray(err)
    assert got.shape == ref.shape
    assert np.all(np.isfinite(got))
    off = np.abs(got - ref) - (rel * (np.abs(ref) + err) + tiny + err)
    assert off.max(initial=-1.0) <= 0, float(off.max())


# ------------------------------------------------------------------------------------ oracle pins

def test_oracle_router_by_hand():
    ids, w = B.router([[1.0, 3.0, 3.0, -np.inf, np.nan]], 4)
    assert ids.tolist() == [[1, 2, 0, -1]]
    e = math.exp(-2.0)
    np.testing.assert_allclose(w, [[1 / (2 + e), 1 / (2 + e), e / (2 + e), 0.0]], rtol=1e-15)
    # two runs of two, one stays: run 1 (0.5 + 0.5 + bias) beats run 0
    ids, w = B.router([[4.0, -9.0, 0.0, 0.0]], 2, score="sigmoid", bias=[0.0, 0.0, 0.3, 0.2], n_group=2,
                      topk_group=1, scale=2.0)
    assert ids.tolist() == [[2, 3]]
    np.testing.assert_allclose(w, [[1.0, 1.0]])
    ids, w = B.router([[-np.inf, np.nan]], 2)
    assert ids.tolist() == [[-1, -1]] and w.tolist() == [[0.0, 0.0]]


def test_oracle_group_by_hand():
    off, perm, slot = B.group([[5, 3], [4, 9], [3, -1]], 3, first=3)
    assert off.tolist() == [0, 2, 3, 4]
    assert perm.tolist() == [1, 4, 2, 0, -1, -1]
    assert slot.tolist() == [[3, 0], [2, -1], [1, -1]]


def test_oracle_norm_by_hand():
    np.testing.assert_allclose(B.norm(np.array([[3.0, 4.0]]), [1.0, 2.0], eps=0.0),
                               [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]])
    np.testing.assert_allclose(B.norm(np.array([[1.0, 3.0]]), [0.0, 1.0], [0.5, 0.5], "layer", 0.0, 1.0),
                               [[-0.5, 2.5]])
    y, mag = B.combine([[1.0], [10.0]], np.array([[1, -1, 0]]), np.array([[0.5, 7.0, -2.0]]))
    assert y.tolist() == [[3.0]] and mag.tolist() == [[7.0]]


def test_oracle_grouped_by_hand():
    x = [[1.0, 2.0], [3.0, 4.0]]
    w = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])
    out, _ = B.grouped(x, w, [0, 1, 3], 4, perm=[3, 0, 2, -1], topk=2)
    assert out.tolist() == [[3.0], [2.0], [4.0], [0.0]]
    assert abs(B.swiglu(np.array(9.0), np.array(8.0), 7.0, 1.0, 1.0) - 7 / (1 + math.exp(-7)) * 8) < 1e-12


# ------------------------------------------------------------------------------------ router

def sigmoid_keys(logits, bias):
    """The 32-bit keys of the formula: 1 / (1 + exp(-l)) + bias, one rounding per operation."""
    k = 1.0 / (1.0 + torch.exp(-logits.float()))
    return (k if bias is None else k + bias).cpu().numpy()


def check_router(moe, logits, topk, score, **kw):
    bias = kw.get("bias")
    ids, w = moe.moe_router(logits, topk, score=moe.MOE_SCORE_SIGMOID if score == "sigmoid" else
                            moe.MOE_SCORE_SOFTMAX, **kw)
    keys = sigmoid_keys(logits, bias) if score == "sigmoid" else f64(logits)
    kw = dict(kw, bias=None if bias is None else f64(bias))
    rids, rw = B.router(f64(logits), topk, score=score, keys=keys, **kw)
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), rids)
    # exp, a sum of at most E + topk terms (all positive) and two quotients, a few ulps each
    tol = (logits.shape[1] / 16 + 24) * EPS32
    np.testing.assert_allclose(f64(w), rw, rtol=tol, atol=1e-37)


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,topk", [(1, 1, 1), (1, 384, 6), (3, 33, 32), (5, 64, 8), (130, 100, 3), (257, 256, 8),
                                      (9, 500, 10), (7, 1024, 16), (0, 8, 2)])
def test_router(moe, score, M, E, topk):
    g = torch.Generator().manual_seed(M * 1000 + E)
    for dtype in ("f32", "bf16", "f16"):
        logits = (2 * torch.randn(M, E, generator=g)).to(DT[dtype]).cuda()
        for renorm in (True, False):
            check_router(moe, logits, topk, score, renormalize=renorm, scale=2.5)
        if score == "sigmoid":
            check_router(moe, logits, topk, score, bias=(0.2 * torch.randn(E, generator=g)).cuda())


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,keep,topk", [(256, 8, 4, 8), (24, 8, 1, 3), (32, 32, 5, 5), (384, 3, 2, 6), (1024, 16, 16, 16)])
def test_router_groups(moe, score, E, G, keep, topk):
    g = torch.Generator().manual_seed(E + G)
    logits = torch.randn(67, E, generator=g).cuda()
    bias = (0.1 * torch.randn(E, generator=g)).cuda() if score == "sigmoid" else None
    check_router(moe, logits, topk, score, bias=bias, n_group=G, topk_group=keep)


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_ties_masks_and_extremes(moe, score):
    inf, nan = math.inf, math.nan
    rows = [[0.0] * 40,                                         # all equal: lowest indices
            [0.0, -0.0] * 20,                                   # the two zeros are one value
            [-inf] * 40,                                        # nothing left
            [nan] * 40,
            [-inf] * 37 + [1.0, nan, 2.0],                      # fewer than topk left
            [1.0, inf] + [0.0] * 38,
            [-300.0] * 40,                                      # sigmoids of zero
            [88.0, -88.0] * 20,
            [3.0e38, -3.0e38] * 20]
    logits = torch.tensor(rows).cuda()
    for renorm in (True, False):
        check_router(moe, logits, 5, score, renormalize=renorm)
        check_router(moe, logits, 5, score, renormalize=renorm, n_group=4, topk_group=2)


@gpu
@pytest.mark.parametrize("E,topk", [(256, 8), (384, 16), (1000, 16), (256, 17), (512, 1)])
def test_router_many_equal_keys(moe, E, topk):
    """Rows of few values: from none to all keys equal, more of them than a warp's lanes reach the choice."""
    g = torch.Generator().manual_seed(E)
    rows = [torch.randint(0, v, (E,), generator=g).float() for v in (1, 2, 3, 8, 40, 400)]
    few = torch.full((E,), -math.inf)
    few[::61] = 1.0                                             # fewer keys than topk in some cases
    spread = torch.zeros(E)
    spread[::32] = 5.0                                          # one lane holds all the largest
    logits = torch.stack(rows + [few, spread, -spread]).cuda()
    for score in ("softmax", "sigmoid"):
        check_router(moe, logits, topk, score)


@gpu
def test_router_strided_rows_and_given_outputs(moe):
    big = torch.randn(20, 77, device="cuda")
    view = big[:, 5:69]
    ids = torch.full((20, 4), 99, dtype=torch.int32, device="cuda")
    w = torch.zeros((20, 4), device="cuda")
    a, b = moe.moe_router(view, 4, ids=ids, weights=w)
    assert a is ids and b is w
    c, d = moe.moe_router(view.contiguous(), 4)
    assert torch.equal(a, c) and torch.equal(b, d)


# ------------------------------------------------------------------------------------ grouping

@gpu
@pytest.mark.parametrize("M,topk,E,first", [(1, 1, 1, 0), (0, 3, 5, 0), (16, 6, 384, 0), (37, 6, 192, 192), (341, 6, 1024, 0),
                                            (1000, 8, 256, 64), (1025, 2, 7, 0), (2048, 5, 31, 0), (9001, 8, 256, 0), (40000, 7, 513, 100)])
def test_group(moe, M, topk, E, first):
    rng = np.random.default_rng(M + E)
    ids = rng.integers(first - 3, first + E + 3, (M, topk)).astype(np.int32)
    if M > 4:
        ids[1::5] = -1
        ids[2::7] = first + E // 2                              # one crowded expert
        ids[3, 0] = np.iinfo(np.int32).max
        ids[4, 0] = np.iinfo(np.int32).min
    off, perm, slot = moe.moe_group(torch.from_numpy(ids).cuda(), E, first_expert=first)
    roff, rperm, rslot = B.group(ids, E, first)
    assert np.array_equal(off.cpu().numpy(), roff)
    assert np.array_equal(perm.cpu().numpy(), rperm)
    assert np.array_equal(slot.cpu().numpy(), rslot)


# ------------------------------------------------------------------------------------ products

def product_case(E, N, K, counts, dtype, gather, topk=1, pad=0, seed=0, ldx=None, ldw=None, shift=0):
    """Device operands of a call whose experts have `counts` rows, `pad` dropped slots at the end."""
    g = torch.Generator().manual_seed(seed)
    S = sum(counts) + pad
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    tokens = -(-S // topk) if gather else S
    perm = torch.randperm(tokens * topk, generator=g)[:S].to(torch.int32) if gather else None
    if gather and pad:
        perm[S - pad:] = -1

    def strided(shape, ld):
        if ld is None and not shift:
            return torch.randn(shape, generator=g).to(DT[dtype]).cuda()
        ld = ld or shape[-1]
        flat = torch.full((int(np.prod(shape[:-1])) * ld + shift,), float("nan")).to(DT[dtype]).cuda()
        v = flat[shift:].view(*shape[:-1], ld)[..., :shape[-1]]
        v.copy_(torch.randn(shape, generator=g).to(DT[dtype]))
        return v

    x = strided((max(tokens, 1), K), ldx)
    w = strided((E, N, K), ldw)
    w.copy_((w.float() * K ** -0.5).to(DT[dtype]))
    return x, w, off.cuda(), None if perm is None else perm.cuda(), S


def check_product(moe, x, w, off, perm, S, dtype, topk=1, act=False, layout=0, limit=math.inf, alpha=1.0, beta=0.0,
                  op=None, out=None):
    E, N, K = w.shape
    op = op or moe.MoEGrouped(E, N, K, max_rows=max(S, 1), dtype=DT[dtype], act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE,
                              layout=layout, swiglu_limit=limit, alpha=alpha, beta=beta)
    got = op(x[:S] if perm is None else x, w, off, perm=perm, topk=topk, out=out)
    assert op.device_error() == (0, 0)
    ref, mag = B.grouped(f64(x), f64(w), off.cpu().numpy(), S, None if perm is None else perm.cpu().numpy(), topk)
    err = K * EPS32 * mag
    if act:
        a, b = ref[:, :N // 2], ref[:, N // 2:]
        ea, eb = err[:, :N // 2], err[:, N // 2:]
        u, g, eu, eg = (a, b, ea, eb) if layout == 0 else (b, a, eb, ea)
        ref = B.swiglu(u, g, limit, alpha, beta)
        gc, uc = np.minimum(g, limit), np.clip(u, -limit, limit) + beta
        # d/du = g' sigma <= |g'|; d/dg = u' (sigma + alpha g sigma (1 - sigma)), factor at most 1 + 0.28;
        # the second order of both errors, and a few ulps of the fp32 formula itself
        err = np.abs(gc) * eu + 1.3 * np.abs(uc) * eg + 2 * eu * eg + 16 * EPS32 * (np.abs(ref) + np.abs(gc * uc) * EPS32)
        if np.isfinite(limit):                       # exp(-alpha g) carries alpha |g| relative ulps
            err = err + 4 * EPS32 * abs(alpha) * np.abs(gc) * np.abs(ref)
        else:
            err = err + 4 * EPS32 * abs(alpha) * np.abs(g) * np.abs(ref)
    within(got, ref, dtype, err)
    assert torch.count_nonzero(got[int(off[-1]):]) == 0
    return got


RAGGED = [3, 0, 1, 70, 0, 16, 129, 33]


@gpu
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("dtype,N,K", [("bf16", 256, 128), ("f16", 130, 72), ("bf16", 1, 8), ("f16", 2, 1000), ("bf16", 576, 264),
                                       ("bf16", 94, 2304), ("bf16", 33, 5), ("f16", 34, 127)])
def test_product(moe, dtype, N, K, act, gather):
    if act and N % 2:
        N += 1
    x, w, off, perm, S = product_case(8, N, K, RAGGED, dtype, gather, topk=3 if gather else 1, pad=11, seed=N + K)
    check_product(moe, x, w, off, perm, S, dtype, topk=3 if gather else 1, act=act)


@gpu
@pytest.mark.parametrize("counts", [[0, 0, 0, 0], [1, 0, 0, 0], [0, 0, 0, 1], [1, 1, 1, 1], [700, 0, 0, 2], [31, 32, 33, 64],
                                    [65, 127, 128, 129], [255, 256, 257, 513]])
def test_product_row_counts(moe, counts):
    for act in (False, True):
        x, w, off, perm, S = product_case(4, 320, 200, counts, "bf16", True, topk=2, pad=1, seed=sum(counts))
        check_product(moe, x, w, off, perm, S, "bf16", topk=2, act=act, limit=1.0)


@gpu
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("counts,N,K", [([1] * 6, 8192, 1544), ([10, 20, 0, 30, 9, 15], 8192, 1544), ([40, 3, 0, 61, 8, 64], 5888, 1800),
                                        ([700, 256, 300, 1], 8000, 2888), ([513, 0, 90, 1000], 9984, 136), ([300], 5376, 5128)])
def test_product_many_units(moe, counts, N, K, act):
    """More units than CTA pairs: whole units, units cut by K steps and joined, row blocks with one of two
    accumulators, at every token-tile width."""
    x, w, off, perm, S = product_case(len(counts), N, K, counts, "bf16", True, topk=2, seed=K)
    a = check_product(moe, x, w, off, perm, S, "bf16", topk=2, act=act, limit=2.0)
    check_product(moe, x[perm.long() // 2].contiguous(), w, off, None, S, "bf16", act=act, limit=2.0)   # the same rows in place
    op = moe.MoEGrouped(len(counts), N, K, max_rows=S, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE, swiglu_limit=2.0)
    xs = x[perm.long() // 2].contiguous()
    b = op(xs, w, off)
    for _ in range(30):                                     # every schedule gives the same bits, and no wait gives up
        assert torch.equal(op(x, w, off, perm=perm, topk=2), a)
        assert torch.equal(op(xs, w, off), b)
    assert op.device_error() == (0, 0)


@gpu
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("counts,N,K", [([0, 300, 70, 513, 16, 257, 0, 70, 256], 5376, 3592), ([70, 300], 9984, 3600),
                                        ([(37 * e * e + 11) % 151 for e in range(130)], 330, 3600),
                                        ([(53 * e + 5) % 140 for e in range(513)], 34, 3584)])
def test_product_uneven_tiles(moe, counts, N, K, act):
    """Long units of uneven sizes, more of them than CTA pairs, some experts without rows, some alike: the order in which
    they are taken shows in no result."""
    assert sum(counts) > 64 * len(counts)
    x, w, off, perm, S = product_case(len(counts), N, K, counts, "f16", True, topk=2, pad=3, seed=N)
    got = check_product(moe, x, w, off, perm, S, "f16", topk=2, act=act)
    op = moe.MoEGrouped(len(counts), N, K, max_rows=S, dtype=torch.float16, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE)
    for _ in range(30):
        assert torch.equal(op(x, w, off, perm=perm, topk=2), got)
    assert op.device_error() == (0, 0)


@gpu
def test_product_past_32_bits(moe):
    """A weight tensor of more than 2^31 elements, and a K of several thousand steps' length."""
    E, N, K = 5, 21504, 20480
    assert E * N * K > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    w[E - 1] = torch.randn((N, K), generator=g, device="cuda") * K ** -0.5
    counts = [2, 0, 0, 0, 3]
    x = torch.randn((5, K), generator=g, device="cuda").bfloat16()
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    got = moe.MoEGrouped(E, N, K, max_rows=5)(x, w, off)
    assert torch.count_nonzero(got[:2]) == 0
    xs, ws = x[2:].double(), w[E - 1].double()
    mag = xs.abs() @ ws.abs().t()
    within(got[2:], f64(xs @ ws.t()), "bf16", K * EPS32 * f64(mag))


@gpu
@pytest.mark.parametrize("layout", [0, 1])
def test_product_swiglu_options(moe, layout):
    x, w, off, perm, S = product_case(3, 192, 320, [5, 40, 17], "bf16", False, seed=9)
    check_product(moe, x, w, off, perm, S, "bf16", act=True, layout=layout, limit=0.7, alpha=1.702, beta=1.0)


@gpu
@pytest.mark.parametrize("ldx,ldw,shift", [(80, 96, 0), (77, 72, 0), (72, 73, 0), (72, 72, 1)])
def test_product_strides_and_alignment(moe, ldx, ldw, shift):
    """Row strides, odd ones and bases off 16 bytes; what lies between the rows is NaN."""
    x, w, off, perm, S = product_case(4, 100, 72, [9, 0, 50, 2], "f16", True, topk=2, ldx=ldx, ldw=ldw, shift=shift)
    big = torch.full((S, 131), 7.0, dtype=torch.float16, device="cuda")
    check_product(moe, x, w, off, perm, S, "f16", topk=2, out=big[:, 3:103])
    assert torch.all(big[:, :3] == 7) and torch.all(big[:, 103:] == 7)


@gpu
@pytest.mark.parametrize("K", [1, 3, 63, 65, 129])
@pytest.mark.parametrize("gather", [False, True])
def test_product_odd_k_in_aligned_rows(moe, K, gather):
    """K of any size on the tensor cores, in rows padded (with NaN) to 16 bytes."""
    ld = (K + 7) // 8 * 8 + 8
    for act in (False, True):
        x, w, off, perm, S = product_case(5, 66, K, [4, 0, 33, 1, 90], "bf16", gather, topk=2 if gather else 1, ldx=ld, ldw=ld, seed=K)
        check_product(moe, x, w, off, perm, S, "bf16", topk=2 if gather else 1, act=act)


@gpu
def test_product_neighbours_do_not_leak(moe):
    """NaN and inf in rows of x and in experts that a position does not use stay out of its result."""
    counts = [5, 6, 7]
    x, w, off, perm, S = product_case(3, 160, 136, counts, "bf16", False, seed=4)
    op = moe.MoEGrouped(3, 160, 136, max_rows=S)
    want = op(x, w, off)
    x2, w2 = x.clone(), w.clone()
    x2[5:11] = float("nan")
    w2[1] = float("inf")
    got = op(x2, w2, off)
    keep = [i for i in range(S) if not 5 <= i < 11]
    assert torch.equal(got[keep], want[keep]) and torch.all(torch.isnan(got[5:11]))


@gpu
def test_product_repeats_streams_and_graphs(moe):
    """One plan over calls of other sizes and offsets, on another stream, and replayed in a graph:
    every call gives the same bits again."""
    E, N, K = 6, 512, 640
    op = moe.MoEGrouped(E, N, K, max_rows=400, act=moe.MOE_ACT_SWIGLU)
    calls = []
    for seed, counts in enumerate(([1, 0, 2, 0, 0, 1], [50, 3, 0, 100, 7, 64], [0, 0, 0, 0, 0, 399])):
        x, w, off, perm, S = product_case(E, N, K, counts, "bf16", True, topk=2, seed=seed)
        calls.append((x, w, off, perm, check_product(moe, x, w, off, perm, S, "bf16", topk=2, act=True, op=op)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for x, w, off, perm, want in calls:
            assert torch.equal(op(x, w, off, perm=perm, topk=2), want)
            with torch.cuda.stream(side):
                got = op(x, w, off, perm=perm, topk=2)
            side.synchronize()
            assert torch.equal(got, want)
    x, w, off, perm, want = calls[1]
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op(x, w, off, perm=perm, topk=2, out=out)
    for _ in range(3):
        out.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert op.device_error() == (0, 0)


@gpu
def test_product_reports_bad_tables(moe):
    """Offsets out of order and permutation entries out of range set the device error word (the
    kernels check them before they address anything)."""
    x, w, off, perm, S = product_case(3, 64, 64, [4, 4, 4], "bf16", True, topk=2)
    op = moe.MoEGrouped(3, 64, 64, max_rows=S)
    bad = perm.clone()
    bad[5] = 10 ** 6
    op(x, w, off, perm=bad, topk=2)
    assert op.device_error() == (8, 1)
    bad[5] = -7
    op(x, w, off, perm=bad, topk=2)
    assert op.device_error() == (8, 1)
    for o in ([0, 8, 4, 12], [0, 4, 8, 13], [-1, 4, 8, 12]):
        op(x, w, torch.tensor(o, dtype=torch.int32, device="cuda"), perm=perm, topk=2)
        assert op.device_error() == (8, 1)
    check_product(moe, x, w, off, perm, S, "bf16", topk=2, op=op)


# ------------------------------------------------------------------------------------ norms

def norm_reference(residual, rows=None, slot_of=None, topk_weights=None, shared=None, post=None, post_b=None, gate=None,
                   scale=1.0, pre=None, pre_b=None, eps=1e-6, kind="rms", offset=0.0):
    """(r, out, their fp32 error bounds).  Bounds: a combine of k terms, sums of H squares as trees of
    at most 64 levels and a handful of products and quotients: 80 ulps of the magnitudes involved."""
    u = 80 * EPS32
    r = residual
    er = u * np.abs(residual)

    def normed(v, ev, w, b):
        n = B.norm(v, w, b, kind, eps, offset)
        wa = np.abs(np.asarray(w, np.float64) + offset)
        c = v - v.mean(1, keepdims=True) if kind == "layer" else v
        inv = 1.0 / np.sqrt(np.mean(c * c, 1, keepdims=True) + eps)
        ec = ev + (ev.mean(1, keepdims=True) + u * np.abs(v).mean(1, keepdims=True) + u * np.abs(v) if kind == "layer" else 0.0)
        # d inv / inv <= inv^2 mean(|c| ec)
        rel = u + inv ** 2 * np.mean(np.abs(c) * ec, 1, keepdims=True)
        return n, wa * inv * (ec + np.abs(c) * rel) + u * (0.0 if b is None else np.abs(b))

    if rows is not None:
        if slot_of is None:
            y, mag = rows, np.abs(rows)
        else:
            y, mag = B.combine(rows, slot_of, topk_weights, shared)
        ey = u * mag
        if post is not None:
            y, ey = normed(y, ey, post, post_b)
        g = scale * (1.0 if gate is None else gate)
        r = residual + g * y
        er = er + np.abs(g) * ey + u * np.abs(g * y)
    if pre is None:
        return r, None, er, None
    z, ez = normed(r, er, pre, pre_b)
    return r, z, er, ez


def check_norm(moe, M, H, dtype="bf16", res="same", wide=False, k=0, kind="rms", post=True, gate="channel", pre=True, bias=False,
               shared=False, scale=0.5, offset=0.0, seed=0, pad=0, zero_rows=False, inplace=False):
    rng = np.random.default_rng(seed)
    dt, rt = DT[dtype], DT[dtype if res == "same" else res]
    wt = torch.float32 if wide else dt

    def t(a, ty, ld=None):
        a = torch.from_numpy(np.asarray(a, np.float32)).to(ty).cuda()
        if not pad or a.dim() != 2:
            return a
        big = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), dtype=ty, device="cuda")
        big[:, :a.shape[1]] = a
        return big[:, :a.shape[1]]

    residual = t(2 * rng.standard_normal((M, H)), rt)
    rows = t(np.zeros((max(1, M * k) if k else M, H)) if zero_rows else rng.standard_normal((max(1, M * k) if k else M, H)), dt)
    kw = {}
    ref = {"rows": f64(rows)}
    if k:
        slot = rng.permutation(M * k).reshape(M, k).astype(np.int32)
        if M > 2:
            slot[0] = -1                                        # a row without experts
            slot[1, 0] = M * k + 5                              # past the rows: dropped
        w = rng.random((M, k), np.float32)
        kw |= {"slot_of": torch.from_numpy(slot).cuda(), "topk_weights": torch.from_numpy(w).cuda()}
        ref |= {"slot_of": slot, "topk_weights": w}
        if shared:
            kw["shared"] = t(rng.standard_normal((M, H)), dt)
            ref["shared"] = f64(kw["shared"])
    if post:
        kw["post_weight"] = t(1 - offset + 0.1 * rng.standard_normal(H), wt)
        ref["post"] = f64(kw["post_weight"])
    if pre:
        kw["pre_weight"] = t(1 - offset + 0.1 * rng.standard_normal(H), wt)
        ref["pre"] = f64(kw["pre_weight"])
    if bias:
        if post:
            kw["post_bias"] = t(rng.standard_normal(H), wt)
            ref["post_b"] = f64(kw["post_bias"])
        if pre:
            kw["pre_bias"] = t(rng.standard_normal(H), wt)
            ref["pre_b"] = f64(kw["pre_bias"])
    shape = {"none": None, "channel": (H,), "token": (M, 1), "full": (M, H)}[gate]
    if shape:
        kw["gate"] = t(rng.standard_normal(shape), wt)
        ref["gate"] = f64(kw["gate"])
    r, z, er, ez = norm_reference(f64(residual), scale=scale, kind=kind, offset=offset, **ref)
    if inplace:
        kw["residual_out"] = residual
    got_r, got_z = moe.moe_block_norm(residual, rows, scale=scale, kind=moe.MOE_NORM_LAYER if kind == "layer" else moe.MOE_NORM_RMS,
                                      weight_offset=offset, **kw)
    assert moe.moe_block_norm_get_device_error() == (0, 0)
    within(got_r, r, dtype if res == "same" else res, er)
    if pre:
        within(got_z, z, dtype, ez)
    else:
        assert got_z is None


@gpu
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("k", [0, 1, 6])
@pytest.mark.parametrize("M,H", [(1, 7168), (3, 8), (5, 1), (4, 100), (2, 6144), (9, 333), (3, 12288), (2, 32768)])
def test_norm(moe, M, H, k, kind):
    check_norm(moe, M, H, k=k, kind=kind, seed=M + H)


@gpu
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("dtype,res,wide", [("bf16", "same", False), ("bf16", "f32", False), ("f16", "same", True), ("f16", "f32", True)])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_norm_types_and_parts(moe, gate, dtype, res, wide, post, pre):
    for H in (512, 515):
        check_norm(moe, 6, H, dtype=dtype, res=res, wide=wide, k=3, gate=gate, post=post, pre=pre, bias=wide, shared=wide, offset=float(wide))


@gpu
def test_norm_strides_zero_rows_and_in_place(moe):
    for pad in (8, 3):
        check_norm(moe, 5, 264, k=2, pad=pad, kind="layer", gate="full")
    check_norm(moe, 5, 264, zero_rows=True)
    check_norm(moe, 5, 264, k=2, zero_rows=True)
    check_norm(moe, 5, 264, k=2, inplace=True)
    check_norm(moe, 5, 264, res="f32", inplace=True)


@gpu
@pytest.mark.parametrize("H,res", [(4608, "same"), (7168, "f32"), (7680, "same"), (7688, "same"), (12288, "f32"), (15360, "same")])
def test_norm_many_tokens(moe, H, res):
    """More tokens than CTAs, long rows: the ring of rows wraps within and across tokens."""
    for M, k in ((700, 0), (333, 3), (310, 17)):
        if M * max(k, 1) * H < 1 << 25:
            check_norm(moe, M, H, res=res, k=k, kind="layer" if k else "rms", shared=k > 3, gate="full" if k else "token", post=k != 3)


@gpu
@pytest.mark.parametrize("M,H,k,res", [(800, 4096, 2, "same"), (1700, 2048, 1, "f32"), (3600, 1032, 2, "same"), (2500, 1544, 0, "f32")])
def test_norm_many_short_tokens(moe, M, H, k, res):
    check_norm(moe, M, H, k=k, res=res, kind="layer" if k == 1 else "rms", shared=k == 2)


@gpu
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_before_a_block_only(moe, kind):
    residual = torch.randn(7, 640, device="cuda")
    w = torch.randn(640, device="cuda").bfloat16()
    r, z = moe.moe_block_norm(residual, pre_weight=w, kind=moe.MOE_NORM_LAYER if kind == "layer" else moe.MOE_NORM_RMS)
    assert r is None and z.dtype == torch.bfloat16
    _, ref, _, e = norm_reference(f64(residual), pre=f64(w), kind=kind)
    within(z, ref, "bf16", e)


# ------------------------------------------------------------------------------------ together

@gpu
@pytest.mark.parametrize("tokens,topk", [(1, 4), (16, 4), (300, 2)])
def test_block_example(moe, tokens, topk):
    """examples/block16.py: a 16-bit block from router to the next block's norm, against 64 bits."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "block16.py")
    spec = importlib.util.spec_from_file_location("block16", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    b, layer, r0, h0, r1, h1, r2, h2 = ex.run(tokens=tokens, topk=topk)
    ids, w = b.route(h0)
    off, perm, slot = B.group(ids.cpu().numpy(), b.E)
    S = tokens * topk
    u, _ = B.grouped(f64(h0), f64(b.w13), off, S, perm, topk)
    # the 16-bit intermediate is rounded: take it from the library, checked by the product's own tests
    u16 = b.up(h0, b.w13, torch.from_numpy(off).cuda(), perm=torch.from_numpy(perm).cuda(), topk=topk)
    ref = B.swiglu(u[:, :b.I], u[:, b.I:], b.limit)
    assert np.linalg.norm(f64(u16) - ref) <= 2.0 ** -8 * np.linalg.norm(ref) + 1e-6
    y, mag = B.grouped(f64(u16), f64(b.w2), off, S)
    y16 = b.down(u16, b.w2, torch.from_numpy(off).cuda())
    within(y16, y, "bf16", b.I * EPS32 * mag)
    r, z, er, ez = norm_reference(f64(r0), f64(y16), slot, f64(w), post=f64(b.post), gate=f64(b.gate), scale=b.scale, pre=f64(b.next))
    within(r1, r, "bf16", er)
    within(h1, z, "bf16", ez)
    assert torch.isfinite(r2.float()).all() and torch.isfinite(h2.float()).all() and not torch.equal(r1, r2)
    assert b.up.device_error() == b.down.device_error() == (0, 0) and layer.device_error() == (0, 0)


# ------------------------------------------------------------------------------------ refusals

def status_of(call):
    import serving_route_count_gb300 as m
    with pytest.raises(m.MoEError) as ei:
        call()
    return ei.value.status


@pytest.fixture(scope="module")
def lib():
    from serving_route_count_gb300 import _lib, build
    build.build()
    return _lib.load()


def test_refusals_of_the_c_abi(lib):
    """Every refusal comes before any device work, so addresses that are never followed will do."""
    p = 256

    def router(M=4, E=8, k=2, score=0, groups=1, keep=1, ld=8, dtype=2, logits=p, bias=None, ids=p, w=p):
        return lib.moe_router(logits, dtype, ld, bias, M, E, k, score, groups, keep, 1, 1.0, ids, w, None)

    assert router(M=0) == 0
    assert router(M=-1) == 1 and router(dtype=3) == 1 and router(score=2) == 1
    assert router(logits=None) == 1 and router(ids=None) == 1 and router(w=None) == 1
    assert router(E=0) == 2 and router(E=1025, ld=2000) == 2 and router(k=0) == 2 and router(k=9) == 2 and router(ld=7) == 2
    assert router(groups=3) == 2 and router(groups=4, keep=5) == 2 and router(groups=4, keep=1, k=3) == 2
    assert router(E=66, ld=66, k=33) == 2 and router(bias=p) == 3

    def group(M=4, k=2, E=8, first=0, ids=p, off=p, perm=p, slot=p):
        return lib.moe_group(ids, M, k, E, first, off, perm, slot, None)

    assert group(M=-1) == 1 and group(first=-1) == 1 and group(off=None) == 1 and group(ids=None) == 1
    assert group(perm=None) == 1 and group(slot=None) == 1 and group(first=2 ** 31 - 8) == 1
    assert group(E=0) == 2 and group(E=1025) == 2 and group(k=0) == 2 and group(M=2 ** 30, k=4) == 2


def test_refusals_of_the_grouped_product(lib):
    import serving_route_count_gb300 as m
    inf = float("inf")
    plan = lambda E=4, N=8, K=16, dt=0, act=0, layout=0, limit=inf, alpha=1.0, beta=0.0, rows=32: m.moe_grouped_plan(  # noqa: E731
        E, N, K, dt, act, layout, limit, alpha, beta, rows)
    for bad, st in (({"E": 0}, 2), ({"E": 1025}, 2), ({"N": 0}, 2), ({"K": 0}, 2), ({"rows": -1}, 2), ({"N": 7, "act": 1}, 2),
                    ({"N": 2 ** 22, "K": 2 ** 20}, 2),
                    ({"E": 1, "N": 2 ** 22, "rows": 2 ** 30}, 2), ({"dt": 2}, 3), ({"act": 2}, 3), ({"layout": 2}, 1), ({"limit": 0.0}, 1),
                    ({"limit": float("nan")}, 1), ({"alpha": inf}, 1), ({"beta": float("nan")}, 1)):
        assert status_of(lambda: plan(**bad)) == st, bad
    h = plan()
    n = m.moe_grouped_scratch_bytes(h)
    p = 256

    def run(plan=h, scratch=p, size=n, x=p, ldx=16, x_rows=32, w=p, ldw=16, off=p, perm=p, topk=2, out=p, ldo=8, S=32):
        return lib.moe_grouped_run(plan, scratch, size, x, ldx, x_rows, w, ldw, off, perm, topk, out, ldo, S, None)

    assert run(S=0) == 0 and run(S=33) == 4 and run(S=-1) == 1 and run(plan=None) == 1
    for bad in ({"scratch": None}, {"scratch": 264}, {"size": n - 1}, {"x": None}, {"w": None}, {"off": None}, {"out": None},
                {"ldx": 15}, {"ldw": 15}, {"ldo": 7}, {"topk": 0}, {"x_rows": 0}, {"perm": None, "x_rows": 31}):
        assert run(**bad) == 1, bad
    m.moe_destroy_grouped(h)
    m.moe_destroy_grouped(None)
    assert lib.moe_grouped_scratch_bytes(None, None) == 1


def test_refusals_of_the_norm(lib):
    from serving_route_count_gb300 import _lib
    p = 256
    fields = ("M H dtype residual_dtype weight_dtype kind eps scale weight_offset residual ld_residual rows ld_rows slot_of topk_weights "
              "topk n_rows shared ld_shared post_weight post_bias gate gate_row gate_col pre_weight pre_bias residual_out ld_residual_out "
              "out ld_out").split()
    good = dict(M=2, H=16, eps=1e-6, scale=1.0, residual=p, ld_residual=16, rows=p, ld_rows=16, pre_weight=p, residual_out=p,
                ld_residual_out=16, out=p, ld_out=16)

    def norm(**kw):
        a = dict(good, **kw)
        return lib.moe_block_norm(_lib.NORM_ARGS.pack(*((a.get(f) or 0) for f in fields)), None)

    assert lib.moe_block_norm(None, None) == 1
    assert lib.moe_block_norm_get_device_error(None, None) == 1
    assert norm(M=0) == 0
    # the addresses of tensors without a row are 0
    gone = dict(M=0, residual=None, rows=None, residual_out=None, out=None)
    assert norm(**gone) == 0 and norm(**gone, post_weight=p, gate=p, gate_col=1) == 0
    assert norm(**gone, slot_of=None, topk_weights=None, topk=2, shared=None) == 0
    assert norm(M=0, kind=2) == 1 and norm(M=0, H=0) == 2 and norm(M=0, dtype=2) == 3
    assert norm(H=0) == 2 and norm(H=32769) == 2
    assert norm(dtype=2) == 3 and norm(residual_dtype=1) == 3 and norm(weight_dtype=1) == 3
    for bad in ({"M": -1}, {"kind": 2}, {"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}, {"residual": None}, {"rows": None},
                {"slot_of": p}, {"topk_weights": p}, {"shared": p}, {"slot_of": p, "topk_weights": p, "topk": 0},
                {"post_bias": p}, {"out": None}, {"pre_weight": None}, {"pre_weight": None, "pre_bias": p, "out": None},
                {"pre_weight": None, "out": None, "residual_out": None}, {"ld_residual": 15}, {"ld_rows": 15}, {"ld_residual_out": 15},
                {"ld_out": 15}, {"gate": p, "gate_col": 2}):
        assert norm(**bad) == 1, bad


@gpu
def test_reading_the_error_word_readies_the_scratch(moe):
    """A unit cut along K counts its pieces in the buffer's first 4096 bytes; whatever is left there is cleared."""
    x, w = (torch.randn(*s, device="cuda").bfloat16() for s in ((3, 4096), (1, 512, 4096)))
    off = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    op = moe.MoEGrouped(1, 512, 4096, max_rows=3)
    want = op(x, w, off).clone()
    op.scratch[:4096] = 1
    status, code = op.device_error()
    assert status != 0 and code == 0x01010101
    assert op.device_error() == (0, 0) and torch.equal(op(x, w, off), want)


@gpu
@pytest.mark.parametrize("combine", [False, True])
def test_a_block_without_tokens(moe, combine):
    H, dt = 64, torch.bfloat16
    none = lambda *shape, dtype=dt: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    ids, wt = moe.moe_router(none(0, 8), 2)
    offsets, perm, slot_of = moe.moe_group(ids, 8)
    assert offsets.tolist() == [0] * 9 and perm.numel() == 0 and slot_of.shape == (0, 2)
    y = moe.MoEGrouped(8, H, H, max_rows=0)(none(0, H), none(8, H, H), offsets, perm=perm, topk=2)
    args = dict(slot_of=slot_of, topk_weights=wt, shared=none(0, H)) if combine else {}
    w = torch.ones(H, dtype=dt, device="cuda")
    r, o = moe.moe_block_norm(none(0, H), y, post_weight=w, gate=none(0, 1), pre_weight=w, **args)
    assert y.shape == r.shape == o.shape == (0, H)


@gpu
@pytest.mark.parametrize("M,H,shared", [(3, 64, False), (3, 64, True), (2, 1536, True), (2, 33, True), (700, 2048, False)])
def test_norm_of_a_rank_without_expert_rows(moe, M, H, shared):
    """No slot of any token here, and rows without a row: the sum is the shared row, or zero."""
    g = torch.Generator().manual_seed(M)
    dt = torch.bfloat16
    res, sh = (torch.randn(M, H, generator=g).to(dt).cuda() for _ in range(2))
    w = torch.ones(H, dtype=dt, device="cuda")
    slot_of = torch.full((M, 2), -1, dtype=torch.int32, device="cuda")
    r, o = moe.moe_block_norm(res, res[:0], slot_of=slot_of, topk_weights=torch.full((M, 2), float("nan"), device="cuda"),
                              shared=sh if shared else None, pre_weight=w)
    r0, o0 = moe.moe_block_norm(res, sh if shared else torch.zeros_like(sh), pre_weight=w)
    assert torch.equal(r, r0) and torch.equal(o, o0)


@gpu
def test_refusals_of_the_binding(moe):
    x = torch.zeros(4, 8, device="cuda")
    for call in (lambda: moe.moe_router(x.cpu(), 2), lambda: moe.moe_router(x.double(), 2), lambda: moe.moe_router(x.t(), 2),
                 lambda: moe.moe_router(x, 2, bias=torch.zeros(7, device="cuda")), lambda: moe.moe_router(x, 2, ids=torch.zeros(4, 2, device="cuda")),
                 lambda: moe.moe_group(x, 4), lambda: moe.moe_group(torch.zeros(4, 2, dtype=torch.int32), 4),
                 lambda: moe.moe_block_norm(x, x.bfloat16(), post_weight=torch.zeros(9, device="cuda")),
                 lambda: moe.moe_block_norm(x, x.bfloat16(), topk_weights=x), lambda: moe.moe_block_norm(x, torch.zeros(3, 8, device="cuda").bfloat16()),
                 lambda: moe.moe_block_norm(x, x.bfloat16(), gate=x.bfloat16(), pre_weight=torch.zeros(8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    op = moe.MoEGrouped(2, 16, 8, max_rows=4)
    w = torch.zeros(2, 16, 8, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    xb = x.bfloat16()
    op(xb, w, off)
    for call in (lambda: op(x, w, off), lambda: op(xb, w[:1], off), lambda: op(xb, w.half(), off), lambda: op(xb, w, off[:2]), lambda: op(xb, w, off.long()),
                 lambda: op(xb, w.transpose(1, 2).contiguous().transpose(1, 2), off), lambda: op(xb, w, off, perm=torch.zeros(4, device="cuda")),
                 lambda: op(xb, w, off, out=torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")), lambda: moe.MoEGrouped(2, 16, 8, max_rows=4, dtype=torch.int8)):
        with pytest.raises(ValueError):
            call()
    assert status_of(lambda: op(torch.zeros(5, 8, dtype=torch.bfloat16, device="cuda"), w, off)) == 4
