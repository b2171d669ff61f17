"""The norm's kernel of many tokens, whose rows come through a ring of shared-memory buffers, in every type and part that it takes.
Each test asks which kernel its size goes to, so that none of them runs the plain-load kernel instead."""
import ctypes

import pytest

import block_shapes
from test_block_ops import DT, check_norm, f64, moe, norm_reference, within  # noqa: F401  (moe: fixture)

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    shapes = block_shapes.build(tmp_path_factory.mktemp("shapes"))

    def check(M, H, k, res):
        o = (ctypes.c_int * 3)()
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert shapes.norm_shape(M, H, 4 if res == "f32" else 2, 1, int(k > 0), sms, o) == 1, "this size takes plain loads"
        return o[2]
    return check


TYPES = [("bf16", "same", False), ("bf16", "f32", False), ("bf16", "same", True), ("bf16", "f32", True),
         ("f16", "same", False), ("f16", "f32", False), ("f16", "same", True), ("f16", "f32", True)]


@gpu
@pytest.mark.parametrize("dtype,res,wide", TYPES)
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_types_and_parts(moe, ring, dtype, res, wide, post, pre):
    """Weights held ahead (16 bits) or not (fp32), biases, an offset, one norm, both or none."""
    for M, H, k, gate, kind in ((200, 7168, 2, "full", "rms"), (1800, 2048, 3, "token", "layer"), (1800, 2048, 0, "channel", "rms")):
        ring(M, H, k, res)
        check_norm(moe, M, H, dtype=dtype, res=res, wide=wide, k=k, gate=gate, kind=kind, post=post, pre=pre, bias=wide == (k > 0), shared=k == 3,
                   offset=float(k == 2), seed=H + k)


@gpu
@pytest.mark.parametrize("res", ["same", "f32"])
@pytest.mark.parametrize("M,H,k", [(1800, 2048, 0), (1800, 2048, 2), (700, 7168, 1)])
def test_in_place(moe, ring, M, H, k, res):
    """The residual stream is written over while later tokens' rows are on their way."""
    ring(M, H, k, res)
    check_norm(moe, M, H, k=k, res=res, inplace=True)
    check_norm(moe, M, H, k=k, res=res, inplace=True, pre=False, dtype="f16")


@gpu
@pytest.mark.parametrize("dtype,res,wide", TYPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_before_a_block_only(moe, ring, kind, dtype, res, wide):
    M, H = 1800, 2048
    ring(M, H, 0, res)
    g = torch.Generator(device="cuda").manual_seed(H)
    residual = (2 * torch.randn(M, H, generator=g, device="cuda")).to(DT[dtype if res == "same" else res])
    w, b = ((c + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.float32 if wide else DT[dtype]) for c in (1, 0))
    out = torch.empty(M, H, dtype=DT[dtype], device="cuda")
    r, z = moe.moe_block_norm(residual, pre_weight=w, pre_bias=b, out=out, kind=moe.MOE_NORM_LAYER if kind == "layer" else moe.MOE_NORM_RMS)
    assert r is None and z is out and moe.moe_block_norm_get_device_error() == (0, 0)
    _, ref, _, e = norm_reference(f64(residual), pre=f64(w), pre_b=f64(b), kind=kind)
    within(z, ref, dtype, e)


@gpu
@pytest.mark.parametrize("M,H,k,res,pad", [(1800, 2048, 17, "same", 0), (200, 7168, 17, "f32", 0), (200, 15360, 17, "same", 0), (1800, 2048, 2, "f32", 8),
                                           (470, 4608, 3, "same", 24), (160, 7688, 3, "same", 0), (200, 12288, 0, "same", 0)])
def test_rows_and_strides(moe, ring, M, H, k, res, pad):
    """More rows a token than the ring has buffers, padded rows (NaN between them), both chunk counts."""
    slots = ring(M, H, k, res)
    assert k < 17 or k + 2 > slots
    check_norm(moe, M, H, k=k, res=res, pad=pad, shared=k == 17, kind="layer" if k == 3 else "rms", gate="full")


@gpu
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("M,H", [(1800, 2048), (200, 7168), (200, 15360)])
def test_no_expert_rows(moe, ring, M, H, shared):
    """Every slot was dropped, and rows has no row: buffers that hold nothing are passed on."""
    ring(M, H, 2, "same")
    g = torch.Generator(device="cuda").manual_seed(M)
    res, sh = (torch.randn(M, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    slot_of = torch.full((M, 2), -1, dtype=torch.int32, device="cuda")
    nan = torch.full((M, 2), float("nan"), device="cuda")
    r, o = moe.moe_block_norm(res, res[:0], slot_of=slot_of, topk_weights=nan, shared=sh if shared else None, pre_weight=w)
    r0, o0 = moe.moe_block_norm(res, sh if shared else torch.zeros_like(sh), pre_weight=w)
    assert moe.moe_block_norm_get_device_error() == (0, 0)
    assert torch.equal(r, r0) and torch.equal(o, o0)


@gpu
@pytest.mark.parametrize("M,H,k", [(1800, 2048, 2), (200, 7168, 0), (200, 15360, 1)])
def test_a_wait_that_runs_out(moe, ring, M, H, k):
    """The first CTA's copying warp gives up a wait of 2 ms: the call ends with MOE_ERR_TIMEOUT in the error word, other CTAs' tokens
    are right, and so is the next call."""
    ring(M, H, k, "same")
    g = torch.Generator(device="cuda").manual_seed(M)
    residual, rows = (torch.randn(n, H, generator=g, device="cuda").bfloat16() for n in (M, M * max(1, k)))
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    kw = dict(post_weight=w, pre_weight=w)
    if k:
        kw |= dict(slot_of=torch.randperm(M * k, generator=g, device="cuda").int().view(M, k), topk_weights=torch.rand(M, k, generator=g, device="cuda"))
    want = moe.moe_block_norm(residual, rows, **kw)
    try:
        moe.moe_block_norm_set_wait_probe(2_000_000)
        got = moe.moe_block_norm(residual, rows, **kw)
        assert moe.moe_block_norm_get_device_error() == (7, 2)
    finally:
        moe.moe_block_norm_set_wait_probe(0)
    assert all(torch.equal(a[1:150], b[1:150]) for a, b in zip(got, want))      # token t of the first 150 is CTA t's
    for _ in range(2):
        got = moe.moe_block_norm(residual, rows, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert moe.moe_block_norm_get_device_error() == (0, 0)
