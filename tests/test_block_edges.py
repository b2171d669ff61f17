"""Calls of the 16-bit block's operators at the edges of their ranges, against the formulas in 64 bits."""
import numpy as np
import pytest

from oracle import block as B

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from serving_route_count_gb300 import build
    build.build()
    import serving_route_count_gb300 as m
    return m


# ------------------------------------------------------------------------------------ products

@gpu
@pytest.mark.parametrize("K", [8, 7])                           # tensor cores, CUDA cores
@pytest.mark.parametrize("alpha", [1.0, 1.702, -1.0])
def test_swiglu_of_large_gates(moe, K, alpha):
    """Gates whose sigmoid is near the end of fp32's range, and of bf16's.  x = (1, 0, ..), so the products are the
    weights' first column, exactly; |u| = 3."""
    g = np.concatenate([np.arange(-128, -40, 0.5), np.arange(40, 128, 0.5), [0.0, -0.0, -1e30, 1e30, -np.inf, np.inf]])
    g = torch.from_numpy(g).bfloat16().double().numpy()
    n = g.size
    u = np.where(np.arange(n) % 2, 3.0, -3.0)
    w = torch.zeros((1, 2 * n, K), dtype=torch.bfloat16)
    w[0, :n, 0], w[0, n:, 0] = torch.from_numpy(u).bfloat16(), torch.from_numpy(g).bfloat16()
    x = torch.zeros((1, K), dtype=torch.bfloat16)
    x[0, 0] = 1
    off = torch.tensor([0, 1], dtype=torch.int32)
    finite = np.isfinite(g)                                     # 0 * inf of the row's other columns stays out: they are 0 * 0
    op = moe.MoEGrouped(1, 2 * n, K, max_rows=1, act=moe.MOE_ACT_SWIGLU, alpha=alpha)
    got = op(x.cuda(), w.cuda(), off.cuda()).double().cpu().numpy()[0]
    assert op.device_error() == (0, 0)
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.abs(np.float64(np.float32(alpha)) * g)
        ref = B.swiglu(u, g, np.inf, np.float64(np.float32(alpha)))
        # exp: 2 + 1.173 |a| ulp of 2^-23, its argument's rounding |a| 2^-24, four operations; its last place where it is below
        # fp32's normal range; then the rounding to bf16, in units of 2^-133 below its normal range
        tol = np.abs(ref) * (2.0 ** -8 + (4 + 1.7 * a) * 2.0 ** -23) + np.abs(g * u) * 2.0 ** -149 + 2.0 ** -134
        near = np.abs(got - ref) <= tol
    assert np.all(near[finite]), (g[finite & ~near], got[finite & ~near])
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    assert np.all(same[~finite])


@gpu
def test_widest_product_on_the_cuda_cores(moe):
    """N = 2^22, the most a plan takes, with rows off 16 bytes: one column tile more than a launch counts in y.  Rows past the
    last group are zeros here too."""
    N, K = 1 << 22, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((3, K), (1, N, K)))
    out = torch.full((3, N), 7.0, dtype=torch.bfloat16, device="cuda")
    op = moe.MoEGrouped(1, N, K, max_rows=3)
    op(x, w, torch.tensor([0, 2], dtype=torch.int32, device="cuda"), out=out)
    assert op.device_error() == (0, 0)
    ref, mag = x[:2].double() @ w[0].double().t(), x[:2].double().abs() @ w[0].double().abs().t()
    # rounded once to bf16, from an fp32 sum of K terms
    assert torch.all((out[:2].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2 * K * 2.0 ** -24 * mag)
    assert torch.count_nonzero(out[2]) == 0


@gpu
@pytest.mark.parametrize("ld", [24, 19])                        # tensor cores, CUDA cores
def test_experts_of_one_row(moe, ld):
    g = torch.Generator().manual_seed(2)
    w = torch.randn(3, ld, generator=g).bfloat16().cuda()[:, :16].unsqueeze(1)
    x = torch.randn(5, 16, generator=g).bfloat16().cuda()
    op = moe.MoEGrouped(3, 1, 16, max_rows=5)
    got = op(x, w, torch.tensor([0, 2, 2, 5], dtype=torch.int32, device="cuda")).double()
    e = torch.tensor([0, 0, 2, 2, 2], device="cuda")
    terms = x.double() * w[e, 0].double()
    assert torch.all((got[:, 0] - terms.sum(1)).abs() <= 2.0 ** -8 * terms.sum(1).abs() + 2 * 16 * 2.0 ** -24 * terms.abs().sum(1))


@gpu
def test_many_k_steps(moe):
    """4100 steps of 64 along K, cut among the CTA pairs.  Small whole numbers: every partial sum is exact in fp32."""
    E, N, K = 2, 40, 262400
    g = torch.Generator(device="cuda").manual_seed(4)
    x, w = (torch.randint(-1, 2, s, generator=g, device="cuda").bfloat16() for s in ((5, K), (E, N, K)))
    op = moe.MoEGrouped(E, N, K, max_rows=5)
    off = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    got = op(x, w, off)
    assert op.device_error() == (0, 0)
    ref = torch.cat([x[:3].double() @ w[0].double().t(), x[3:].double() @ w[1].double().t()])
    assert torch.equal(got, ref.bfloat16())


def test_refusals_of_the_wait_probe():
    import serving_route_count_gb300 as m
    from serving_route_count_gb300 import build
    build.build()
    h = m.moe_grouped_plan(2, 8, 16, 0, 0, 0, float("inf"), 1.0, 0.0, 4)
    m.moe_grouped_set_wait_probe(h, 1_000_000_000)
    m.moe_grouped_set_wait_probe(h, 0)
    for plan, ns in ((h, 1_000_000_001), (None, 0)):
        with pytest.raises(m.MoEError) as e:
            m.moe_grouped_set_wait_probe(plan, ns)
        assert e.value.status == 1
    m.moe_destroy_grouped(h)
    m.moe_block_norm_set_wait_probe(0)
    with pytest.raises(m.MoEError) as e:
        m.moe_block_norm_set_wait_probe(1_000_000_001)
    assert e.value.status == 1


@gpu
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,N,K,act", [([3, 0, 2], 512, 4096, True),             # units cut by K steps
                                            ([40, 300, 7], 8192, 512, False)])        # more units than CTA pairs, whole ones first
def test_a_wait_that_runs_out(moe, counts, N, K, act, gather):
    """The first CTA pair's MMA issuer gives up a wait of 2 ms: the call ends with MOE_ERR_TIMEOUT in the error word, and the
    next one gives the result of a plan that never saw it."""
    g = torch.Generator(device="cuda").manual_seed(K)
    S = sum(counts)
    x = torch.randn((S, K), generator=g, device="cuda").bfloat16()
    w = (torch.randn((len(counts), N, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    perm = torch.arange(S, dtype=torch.int32, device="cuda") if gather else None
    new = lambda: moe.MoEGrouped(len(counts), N, K, max_rows=S, act=moe.MOE_ACT_SWIGLU if act else moe.MOE_ACT_NONE)  # noqa: E731
    want, op = new()(x, w, off, perm=perm), new()
    moe.moe_grouped_set_wait_probe(op.plan, 2_000_000)
    op(x, w, off, perm=perm)
    assert op.device_error() == (7, 2)
    moe.moe_grouped_set_wait_probe(op.plan, 0)
    for _ in range(3):
        assert torch.equal(op(x, w, off, perm=perm), want)
    assert op.device_error() == (0, 0)


# ------------------------------------------------------------------------------------ norms

@gpu
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_of_an_fp32_residual_with_fp32_weights(moe, kind):
    """A norm before a block where nothing is of 16 bits: out is bf16, or of the type of the one given."""
    g = torch.Generator().manual_seed(3)
    residual, w = torch.randn(7, 640, generator=g), 1 + 0.1 * torch.randn(640, generator=g)
    k = moe.MOE_NORM_LAYER if kind == "layer" else moe.MOE_NORM_RMS
    ref = B.norm(residual.double().numpy(), w.double().numpy(), kind=kind)
    for out, rel in ((None, 2.0 ** -8), (torch.empty(7, 640, dtype=torch.float16, device="cuda"), 2.0 ** -11)):
        r, z = moe.moe_block_norm(residual.cuda(), pre_weight=w.cuda(), kind=k, out=out)
        assert r is None and z.dtype == (torch.bfloat16 if out is None else torch.float16)
        # one rounding; sums of 640 squares and a handful of operations in fp32, at most 80 ulps of the row's largest value
        assert np.all(np.abs(z.double().cpu().numpy() - ref) <= rel * np.abs(ref) + 80 * 2.0 ** -24 * np.abs(ref).max(1, keepdims=True) + 2.0 ** -25)
