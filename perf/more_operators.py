"""Timing cases of the 8-bit products and of the gated feed-forward block: quantisation to e4m3 with a
scale for each 128 values of a row or each 128 x 128 tile, products of such operands (dense or grouped by
expert, with an optional SwiGLU), and a dense gated feed-forward block, forward alone or as a training step.

Sizes are the layers of this repository (E=384, H=7168, I=576 or 1152, top-6; E=256, H=6144, I=512, top-8)
and generic ones around them.
"""
import math

import torch

own = False   # False: plain torch forms; True: the framework's operators

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 128
MOST = 448.0            # largest e4m3 value
LEAST = 2.0 ** -126     # least scale


def listed():
    return [
        # one token's row before an 8-bit product (latency)
        {"name": "quant_one_token", "op": "quant", "form": "rows", "E": 1, "N": 1, "K": 7168, "dtype": "bf16"},
        # the rows of a large prefill
        {"name": "quant_prefill", "op": "quant", "form": "rows", "E": 1, "N": 8192, "K": 7168, "dtype": "bf16"},
        # the 16-bit expert weights of a checkpoint, once at load
        {"name": "quant_weights", "op": "quant", "form": "tiles", "E": 24, "N": 2304, "K": 7168, "dtype": "bf16"},
        # up projections + SwiGLU of a shared expert, one token: weight streaming of a small matrix
        {"name": "fp8_shared_one_token", "op": "fp8", "M": 1, "E": 1, "k": 1, "K": 7168, "N": 2304, "act": True, "gather": False,
         "skew": 0.0, "limit": 0.0, "dtype": "bf16"},
        # up projections + SwiGLU of the routed experts in a decode step, rows gathered by permutation
        {"name": "fp8_up_decode", "op": "fp8", "M": 8, "E": 256, "k": 8, "K": 6144, "N": 1024, "act": True, "gather": True,
         "skew": 0.0, "limit": 0.0, "dtype": "bf16"},
        # down projection of a decode step: 4.5 scale blocks along K, rows already grouped
        {"name": "fp8_down_decode", "op": "fp8", "M": 16, "E": 384, "k": 6, "K": 576, "N": 7168, "act": False, "gather": False,
         "skew": 0.0, "limit": 0.0, "dtype": "bf16"},
        # the same layer's up projections in a prefill: a ragged few dozen rows an expert
        {"name": "fp8_up_prefill", "op": "fp8", "M": 2048, "E": 256, "k": 8, "K": 6144, "N": 1024, "act": True, "gather": True,
         "skew": 0.5, "limit": 7.0, "dtype": "bf16"},
        # a dense projection of a large prefill: bound by the tensor cores
        {"name": "fp8_dense_prefill", "op": "fp8", "M": 8192, "E": 1, "k": 1, "K": 7168, "N": 7168, "act": False, "gather": False,
         "skew": 0.0, "limit": 0.0, "dtype": "f16"},
        # a shared expert on one token of a decode step
        {"name": "ff_one_token", "op": "ff", "M": 1, "H": 7168, "I": 1152, "train": False, "limit": 0.0, "dtype": "bf16"},
        # a dense block of a prefill
        {"name": "ff_prefill", "op": "ff", "M": 4096, "H": 6144, "I": 4096, "train": False, "limit": 7.0, "dtype": "f16"},
        # a training step of a small shared expert over a ragged batch: output and all gradients
        {"name": "ff_train_ragged", "op": "ff", "M": 777, "H": 6144, "I": 512, "train": True, "limit": 0.0, "dtype": "bf16"},
        # a training step of a dense block
        {"name": "ff_train", "op": "ff", "M": 4096, "H": 7168, "I": 4608, "train": True, "limit": 7.0, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "fp8", "fp8", "ff", "ff"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "quant":
        form = rng.choice(["rows", "tiles"])
        E = 1 if form == "rows" else _log(rng, 1, 24)
        return {"op": op, "form": form, "E": E, "N": _log(rng, 1, 8192 if form == "rows" else 2304), "K": _log(rng, 64, 7168),
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    if op == "fp8":
        E = 1 if rng.random() < 0.4 else _log(rng, 4, 384)
        act = rng.random() < 0.5
        K = 16 * _log(rng, 8, 448)
        most = min(7168, 1_600_000_000 // (E * K))         # as many weights as the largest listed layer
        N = _log(rng, 64, max(64, most))
        N = N // 2 * 2 if act else N
        k = 1 if E == 1 else rng.randint(1, min(8, E))
        M = _log(rng, 1, max(1, min(4096, int(8e11 / (2 * N * K * k)))))
        return {"op": op, "M": M, "E": E, "k": k, "K": K, "N": N, "act": act, "gather": E > 1 and rng.random() < 0.5,
                "skew": rng.choice([0.0, 0.5]), "limit": rng.choice([0.0, 7.0]), "dtype": dtype}
    train = rng.random() < 0.6
    return {"op": op, "M": _log(rng, 1, 4096), "H": 8 * _log(rng, 8, 896), "I": 8 * _log(rng, 8, 576), "train": train,
            "limit": rng.choice([0.0, 7.0]), "dtype": dtype}


def _ids(gen, M, E, k, skew):
    """Distinct ids of every token: the k largest of random keys, over a Zipf law where it is skewed."""
    g = -torch.log(-torch.log(torch.rand((M, E), generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)))
    if skew:
        g -= skew * torch.log(1.0 + torch.randperm(E, generator=gen, device="cuda"))
    return g.topk(k, dim=1).indices


def _blocks(n):
    return -(-n // BLOCK)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)
    rnd = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    s = {"c": c, "plan": None}
    dt = DT[c["dtype"]]
    if c["op"] == "quant":
        # channels of unlike size, a few large ones among them, as activations and weights have
        channel = torch.exp(0.5 * rnd(c["K"]))
        s["x"] = torch.empty((c["E"], c["N"], c["K"]), dtype=dt, device="cuda")
        for e in range(c["E"]):
            s["x"][e] = rnd(c["N"], c["K"]) * channel
        if c["form"] == "rows":
            s["x"] = s["x"][0]
    elif c["op"] == "fp8":
        M, E, k, K, N = c["M"], c["E"], c["k"], c["K"], c["N"]
        ids = _ids(gen, M, E, k, c["skew"]) if E > 1 else torch.zeros((M, 1), dtype=torch.int64, device="cuda")
        key, perm = torch.sort(ids.reshape(-1), stable=True)
        s["perm"] = perm.to(torch.int32)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["offsets"][1:] = torch.bincount(key, minlength=E).cumsum(0)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())      # rows of the busiest expert
        # operands as a checkpoint and the quantisation before this product leave them
        rows = M if c["gather"] else M * k
        s["x"] = (90.0 * rnd(rows, K)).clamp_(-MOST, MOST).to(torch.float8_e4m3fn)
        s["xs"] = torch.exp(0.3 * rnd(rows, _blocks(K))) / 90.0
        s["w"] = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
        for e in range(E):
            s["w"][e] = (90.0 * rnd(N, K)).clamp_(-MOST, MOST).to(torch.float8_e4m3fn)
        tall = 2 * _blocks(N // 2) if c["act"] else _blocks(N)             # up and gate have tiles of their own
        s["ws"] = torch.exp(0.3 * rnd(E, tall, _blocks(K))) * (K ** -0.5 / 90.0)
        s["out"] = torch.empty((M * k, N // 2 if c["act"] else N), dtype=dt, device="cuda")
    else:
        M, H, I = c["M"], c["H"], c["I"]
        s["x"] = rnd(M, H).to(dt)
        s["w13"] = (rnd(2 * I, H) * H ** -0.5).to(dt)
        s["w2"] = (rnd(H, I) * I ** -0.5).to(dt)
        s["dy"] = rnd(M, H).to(dt) if c["train"] else None
    if own:
        import serving_route_count_gb300 as moe
        s["moe"] = moe
        limit = c.get("limit") or math.inf
        if c["op"] == "fp8":            # what a program keeps for a layer: the plan and its workspace
            s["plan"] = moe.MoEFp8(c["E"], c["N"], c["K"], max_rows=c["M"] * c["k"], dtype=dt,
                                   act=moe.MOE_ACT_SWIGLU if c["act"] else moe.MOE_ACT_NONE, swiglu_limit=limit)
        elif c["op"] == "ff":
            s["plan"] = moe.MoEFeedForward(c["H"], c["I"], max_rows=c["M"], dtype=dt, swiglu_limit=limit)
    torch.cuda.synchronize()
    return s


# ------------------------------------------------------------------------------------ plain forms

def _quant(s, c):
    x = s["x"].float()
    tiles = c["form"] == "tiles"
    K, rows = x.shape[-1], x.shape[-2]
    pad = torch.nn.functional.pad(x, (0, -K % BLOCK, 0, -rows % BLOCK if tiles else 0))
    if tiles:
        pad = pad.reshape(*x.shape[:-2], _blocks(rows), BLOCK, _blocks(K), BLOCK)
        scale = (pad.abs().amax(dim=(-3, -1)) / MOST).clamp(min=LEAST)
        wide = scale[..., :, None, :, None]
    else:
        pad = pad.reshape(rows, _blocks(K), BLOCK)
        scale = (pad.abs().amax(dim=-1) / MOST).clamp(min=LEAST)
        wide = scale[..., None]
    q = (pad / wide).clamp(-MOST, MOST).to(torch.float8_e4m3fn)
    q = q.reshape(*x.shape[:-2], -1, _blocks(K) * BLOCK)[..., :rows, :K]
    return q.contiguous(), scale


def _values(q, scale):
    """What quantised rows stand for."""
    return q.float() * scale.repeat_interleave(BLOCK, dim=-1)[..., :q.shape[-1]]


def _weights(s, c):
    w = s["w"].float()
    halves = 2 if c["act"] else 1
    tall = s["ws"].shape[1] // halves
    per = s["ws"].reshape(c["E"], halves, tall, -1).repeat_interleave(BLOCK, dim=2)[:, :, :c["N"] // halves]
    per = per.reshape(c["E"], c["N"], -1).repeat_interleave(BLOCK, dim=2)[:, :, :c["K"]]
    return w.mul_(per)


def _swiglu(y, limit):
    up, gate = y.chunk(2, dim=-1)
    if limit:
        up, gate = up.clamp(-limit, limit), gate.clamp(max=limit)
    return gate / (1.0 + torch.exp(-gate)) * up


def _fp8(s, c):
    E, k, most = c["E"], c["k"], s["most"]
    x, w = _values(s["x"], s["xs"]), _weights(s, c)
    if E == 1:
        y = x @ w[0].T
        return (_swiglu(y, c["limit"]) if c["act"] else y).to(s["out"].dtype)
    off = s["offsets"].long()
    S = s["perm"].numel()
    q = torch.arange(S, device=off.device)
    e = torch.searchsorted(off, q, right=True) - 1                           # expert of each position
    if S <= E:                                                               # few rows: their own experts' weights
        row = s["perm"].long() // k if c["gather"] else q
        y = torch.bmm(w[e], x[row][:, :, None])[:, :, 0]
        return (_swiglu(y, c["limit"]) if c["act"] else y).to(s["out"].dtype)
    at = torch.arange(most, device=off.device)
    p = (off[:-1, None] + at).clamp(max=S - 1)                               # [E, most] positions, padded
    row = s["perm"].long()[p] // k if c["gather"] else p
    y = torch.bmm(x[row], w.transpose(1, 2))
    if c["act"]:
        y = _swiglu(y, c["limit"])
    return y[e, q - off[e]].to(s["out"].dtype)


def _ff(s, c):
    x, w13, w2 = s["x"].float(), s["w13"].float(), s["w2"].float()
    limit, dt = c["limit"], s["x"].dtype
    up, gate = (x @ w13.T).chunk(2, dim=-1)
    u, g = (up.clamp(-limit, limit), gate.clamp(max=limit)) if limit else (up, gate)
    sig = 1.0 / (1.0 + torch.exp(-g))
    h = g * sig * u
    y = h @ w2.T
    if not c["train"]:
        return y.to(dt)
    dy = s["dy"].float()
    dh = dy @ w2
    du = dh * (g * sig)
    dg = dh * u * (sig + g * sig * (1.0 - sig))
    if limit:
        du, dg = torch.where(up.abs() <= limit, du, 0.0), torch.where(gate <= limit, dg, 0.0)
    d = torch.cat((du, dg), dim=1)
    return y.to(dt), (d @ w13).to(dt), (d.T @ x).to(dt), (dy.T @ h).to(dt)


def run(s):
    c = s["c"]
    if not own:
        return {"quant": _quant, "fp8": _fp8, "ff": _ff}[c["op"]](s, c)
    moe = s["moe"]
    if c["op"] == "quant":
        return moe.moe_fp8_quant(s["x"], form=moe.MOE_FP8_TILES if c["form"] == "tiles" else moe.MOE_FP8_ROWS)
    if c["op"] == "fp8":
        return s["plan"](s["x"], s["xs"], s["w"], s["ws"], offsets=s["offsets"] if c["E"] > 1 else None,
                         perm=s["perm"] if c["gather"] else None, topk=c["k"], out=s["out"])
    if not c["train"]:
        return s["plan"](s["x"], s["w13"], s["w2"])
    y, saved = s["plan"].forward(s["x"], s["w13"], s["w2"])
    return (y, *s["plan"].backward(s["dy"], s["x"], s["w13"], s["w2"], saved))


# ------------------------------------------------------------------------------------ work and exact

def work(c):
    if c["op"] == "quant":
        n, size = c["E"] * c["N"] * c["K"], {"bf16": 2, "f16": 2, "f32": 4}[c["dtype"]]
        scales = c["E"] * (c["N"] if c["form"] == "rows" else _blocks(c["N"])) * _blocks(c["K"])
        return {"bytes": n * (size + 1) + 4 * scales, "flops": 2 * n}
    if c["op"] == "fp8":
        M, E, k, K, N = c["M"], c["E"], c["k"], c["K"], c["N"]
        touched = E * (1 - (1 - k / E) ** M)                      # expected, of evenly spread ids
        rows = M if c["gather"] else M * k
        wide = N // 2 if c["act"] else N
        scales = touched * _blocks(N) * _blocks(K) + rows * _blocks(K)
        return {"bytes": touched * N * K + rows * K + 4 * scales + 2 * M * k * wide, "flops": 2 * M * k * N * K}
    M, H, I = c["M"], c["H"], c["I"]
    if c["train"]:
        return {"bytes": 2 * (4 * M * H + 6 * H * I), "flops": 18 * M * H * I}
    return {"bytes": 2 * (2 * M * H + 3 * H * I), "flops": 6 * M * H * I}


def _e4m3(v):
    """Nearest e4m3 value of each 64-bit value, ties to even, saturating."""
    _, e = torch.frexp(v)                                         # |v| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-MOST, MOST)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "quant":
        x = s["x"] if c["form"] == "tiles" else s["x"][None]
        tall = BLOCK if c["form"] == "tiles" else 1
        codes = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        scales = torch.empty((x.shape[0], -(-x.shape[1] // tall), _blocks(c["K"])), dtype=torch.float64, device="cuda")
        for e in range(x.shape[0]):
            top = x[e].double().abs()
            for j in range(scales.shape[2]):
                part = top[:, j * BLOCK:(j + 1) * BLOCK].amax(1)
                part = torch.nn.functional.pad(part, (0, -len(part) % tall)).reshape(-1, tall).amax(1)
                # the scale is a 32-bit value, and codes are of the quotient by it
                scales[e, :, j] = torch.maximum((part / MOST), torch.full_like(part, LEAST)).float().double()
                each = scales[e, :, j].repeat_interleave(tall)[:x.shape[1], None]
                codes[e, :, j * BLOCK:(j + 1) * BLOCK] = _e4m3(x[e][:, j * BLOCK:(j + 1) * BLOCK].double() / each)
        return (codes, scales) if c["form"] == "tiles" else (codes[0], scales[0])
    if c["op"] == "fp8":
        out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        off = s["offsets"].tolist()
        halves = 2 if c["act"] else 1
        rows = c["N"] // halves
        at = torch.arange(c["K"], device="cuda") // BLOCK
        scale_row = torch.cat([torch.arange(rows, device="cuda") // BLOCK + h * (s["ws"].shape[1] // halves) for h in range(halves)])
        for e in range(c["E"]):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            pick = s["perm"][a:b].long() // c["k"] if c["gather"] else torch.arange(a, b, device="cuda")
            x = s["x"].view(torch.uint8)[pick].view(torch.float8_e4m3fn).double() * s["xs"].double()[pick][:, at]
            w = s["w"][e].double() * s["ws"][e].double()[scale_row][:, at]
            y = torch.einsum("mk,nk->mn", x, w)
            if c["act"]:
                u, g = y[:, :rows], y[:, rows:]
                if c["limit"]:
                    u, g = u.clamp(-c["limit"], c["limit"]), g.clamp(max=c["limit"])
                y = u * g * g.sigmoid()
            out[a:b] = y
        return out
    leaves = [s[n].double().requires_grad_(c["train"]) for n in ("x", "w13", "w2")]
    x, w13, w2 = leaves
    gate, up = torch.nn.functional.linear(x, w13[c["I"]:]), torch.nn.functional.linear(x, w13[:c["I"]])
    if c["limit"]:
        up, gate = up.clamp(-c["limit"], c["limit"]), gate.clamp(max=c["limit"])
    y = torch.nn.functional.linear(torch.nn.functional.silu(gate) * up, w2)
    if not c["train"]:
        return y
    return (y.detach(), *torch.autograd.grad(y, leaves, s["dy"].double()))
