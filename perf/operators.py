"""Timing cases of the 16-bit expert block: the router's top-k, the grouping of slots by expert,
the products grouped by expert, and the norms around the block.

Sizes are the layers of this repository (E=384, H=7168, I=576 or 1152, top-6; E=256, H=6144, I=512, top-8)
and generic ones around them.
"""
import math

import torch

own = False   # False: plain torch forms; True: the framework's operators

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # router: one token of a decode step (latency)
        {"name": "router_one_token", "op": "router", "M": 1, "E": 384, "k": 6, "score": "sigmoid", "groups": 1, "keep": 1,
         "renorm": True, "scale": 2.5, "dtype": "f32"},
        # group-limited selection over a medium batch whose logits come out of a 16-bit product
        {"name": "router_groups", "op": "router", "M": 777, "E": 256, "k": 8, "score": "sigmoid", "groups": 8, "keep": 4,
         "renorm": True, "scale": 2.5, "dtype": "bf16"},
        # softmax router of a large prefill
        {"name": "router_prefill", "op": "router", "M": 8192, "E": 256, "k": 8, "score": "softmax", "groups": 1, "keep": 1,
         "renorm": True, "scale": 1.0, "dtype": "f32"},
        # a verify step with padding rows (a quarter of the ids are -1)
        {"name": "group_decode", "op": "group", "M": 16, "E": 384, "k": 6, "skew": 0.0, "pad": 0.25},
        # a large prefill with skewed experts
        {"name": "group_prefill", "op": "group", "M": 8192, "E": 256, "k": 8, "skew": 0.8, "pad": 0.0},
        # fc1 + SwiGLU of a decode step: weight streaming
        {"name": "product_up_decode", "op": "product", "M": 8, "E": 256, "k": 8, "K": 6144, "N": 1024, "act": True,
         "gather": True, "skew": 0.0, "limit": 0.0, "dtype": "bf16"},
        # fc2 of a decode step: short K, wide N, rows already grouped
        {"name": "product_down_decode", "op": "product", "M": 16, "E": 384, "k": 6, "K": 576, "N": 7168, "act": False,
         "gather": False, "skew": 0.0, "limit": 0.0, "dtype": "bf16"},
        # fc1 + SwiGLU of a prefill: every expert touched by a ragged few dozen rows
        {"name": "product_up_prefill", "op": "product", "M": 2048, "E": 256, "k": 8, "K": 6144, "N": 1024, "act": True,
         "gather": True, "skew": 0.0, "limit": 7.0, "dtype": "bf16"},
        # few local experts with many rows, skewed: bound by the tensor cores
        {"name": "product_up_dense", "op": "product", "M": 4096, "E": 16, "k": 6, "K": 7168, "N": 2304, "act": True,
         "gather": True, "skew": 0.5, "limit": 7.0, "dtype": "f16"},
        # after the experts of one token: combine, post-norm, gate, residual, the next block's pre-norm
        {"name": "norm_one_token", "op": "norm", "M": 1, "H": 7168, "k": 6, "kind": "rms", "post": True, "gate": "channel",
         "scale": 0.5, "dtype": "bf16", "res": "bf16"},
        # the same for a prefill
        {"name": "norm_combine_prefill", "op": "norm", "M": 4096, "H": 7168, "k": 6, "kind": "rms", "post": True,
         "gate": "channel", "scale": 0.5, "dtype": "bf16", "res": "bf16"},
        # a dense block's output, gate per token, 32-bit residual stream
        {"name": "norm_dense_prefill", "op": "norm", "M": 8192, "H": 6144, "k": 0, "kind": "rms", "post": True, "gate": "token",
         "scale": 1.0, "dtype": "bf16", "res": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["router", "group", "product", "product", "norm"])
    if op == "router":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log(rng, max(2, 16 // groups), 512 // groups)
        keep = rng.randint(1, groups)
        return {"op": op, "M": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(12, E // groups * keep)),
                "score": rng.choice(["sigmoid", "softmax"]), "groups": groups, "keep": keep, "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op == "group":
        E = _log(rng, 4, 512)
        return {"op": op, "M": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(8, E)), "skew": rng.choice([0.0, 0.8]),
                "pad": rng.choice([0.0, 0.25])}
    if op == "product":
        E = _log(rng, 4, 384)
        act = rng.random() < 0.5
        K = 8 * _log(rng, 8, 896)
        most = min(7168, 1_600_000_000 // (E * K))         # as many weights as the largest listed layer
        N = _log(rng, 64, max(64, most))
        N = N // 2 * 2 if act else N
        M = _log(rng, 1, max(1, min(4096, int(4e11 / (2 * N * K * 8)))))
        return {"op": op, "M": M, "E": E, "k": rng.randint(1, min(8, E)), "K": K, "N": N, "act": act, "gather": rng.random() < 0.5,
                "skew": rng.choice([0.0, 0.5]), "limit": rng.choice([0.0, 7.0]), "dtype": rng.choice(["bf16", "f16"])}
    return {"op": op, "M": _log(rng, 1, 4096), "H": _log(rng, 64, 7168), "k": rng.choice([0, 2, 6]), "kind": rng.choice(["rms", "layer"]),
            "post": rng.random() < 0.7, "gate": rng.choice(["none", "channel", "token", "full"]), "scale": rng.choice([1.0, 0.22]),
            "dtype": rng.choice(["bf16", "f16"]), "res": rng.choice(["same", "f32"])}


def _ids(gen, M, E, k, skew):
    """Distinct ids of every token: the k largest of random keys, over a Zipf law where it is skewed."""
    g = -torch.log(-torch.log(torch.rand((M, E), generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)))
    if skew:
        g -= skew * torch.log(1.0 + torch.randperm(E, generator=gen, device="cuda"))
    return g.topk(k, dim=1).indices.to(torch.int32)


def _groups(ids, E):
    """offsets [E+1], perm [S] (past the last valid slot: -1) and slot_of [M, k] of distinct or padded ids."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    perm = torch.sort(key, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    slot_of = torch.empty_like(perm)
    slot_of[perm] = torch.arange(flat.numel(), device=ids.device)
    slot_of = torch.where(key < E, slot_of, -1)
    perm = torch.where(torch.arange(flat.numel(), device=ids.device) < offsets[E], perm, -1)
    return offsets.to(torch.int32), perm.to(torch.int32), slot_of.to(torch.int32).reshape(ids.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)
    rnd = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    s = {"c": c, "plan": None}
    M, k = c["M"], c["k"]
    if c["op"] == "router":
        s["logits"] = (1.5 * rnd(M, c["E"])).to(DT[c["dtype"]])
        s["bias"] = 0.1 * rnd(c["E"]) if c["score"] == "sigmoid" else None
    elif c["op"] == "group":
        ids = _ids(gen, M, c["E"], k, c["skew"])
        ids[M - int(M * c["pad"]):] = -1
        s["ids"] = ids
    elif c["op"] == "product":
        E, K, N, dt = c["E"], c["K"], c["N"], DT[c["dtype"]]
        ids = _ids(gen, M, E, k, c["skew"])
        s["offsets"], s["perm"], _ = _groups(ids, E)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())      # rows of the busiest expert
        s["x"] = rnd(M if c["gather"] else M * k, K).to(dt)
        s["w"] = torch.empty((E, N, K), dtype=dt, device="cuda")
        for e in range(E):
            s["w"][e] = rnd(N, K) * K ** -0.5
        s["out"] = torch.empty((M * k, N // 2 if c["act"] else N), dtype=dt, device="cuda")
    else:
        H, dt = c["H"], DT[c["dtype"]]
        rt = dt if c["res"] == "same" else DT[c["res"]]
        s["residual"] = (2.0 * rnd(M, H)).to(rt)
        s["y"] = rnd(M * k if k else M, H).to(dt)
        s["slot_of"] = s["weights"] = None
        if k:
            s["slot_of"] = torch.randperm(M * k, generator=gen, device="cuda").to(torch.int32).reshape(M, k)
            w = torch.rand((M, k), generator=gen, device="cuda") + 0.05
            s["weights"] = w / w.sum(1, keepdim=True)
        s["post"] = (1 + 0.1 * rnd(H)).to(dt) if c["post"] else None
        s["pre"] = (1 + 0.1 * rnd(H)).to(dt)
        shape = {"none": None, "channel": (1, H), "token": (M, 1), "full": (M, H)}[c["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(rnd(*shape)).to(dt)
        s["r_out"], s["out"] = torch.empty_like(s["residual"]), torch.empty((M, H), dtype=dt, device="cuda")
    if own:
        import serving_route_count_gb300 as moe
        s["moe"] = moe
        if c["op"] == "product":        # what a program keeps for a layer: the plan and its workspace
            s["plan"] = moe.MoEGrouped(c["E"], c["N"], c["K"], max_rows=M * k, dtype=DT[c["dtype"]],
                                       act=moe.MOE_ACT_SWIGLU if c["act"] else moe.MOE_ACT_NONE,
                                       swiglu_limit=c["limit"] or math.inf)
    torch.cuda.synchronize()
    return s


# ------------------------------------------------------------------------------------ plain forms

def _router(s, c):
    M, E, k, G = c["M"], c["E"], c["k"], c["groups"]
    l = s["logits"].float()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
        key = score + s["bias"]
    else:
        score = torch.exp(l - l.max(1, keepdim=True).values)
        score = score / score.sum(1, keepdim=True)
        key = l
    if G > 1:
        by = key.reshape(M, G, E // G)
        of_group = by.topk(min(2, E // G), dim=2).values.sum(2) if c["score"] == "sigmoid" else by.max(2).values
        best = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        stays = torch.zeros((M, G), dtype=torch.bool, device=l.device).scatter_(1, best, True)
        key = torch.where(stays[:, :, None], by, -math.inf).reshape(M, E)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), w * c["scale"]


def _swiglu(y, limit):
    up, gate = y.chunk(2, dim=-1)
    if limit:
        up, gate = up.clamp(-limit, limit), gate.clamp(max=limit)
    return gate / (1.0 + torch.exp(-gate)) * up


def _product(s, c):
    E, k, most = c["E"], c["k"], s["most"]
    off = s["offsets"].long()
    S = s["perm"].numel()
    q = torch.arange(S, device=off.device)
    e = torch.searchsorted(off, q, right=True) - 1                           # expert of each position
    if S <= E:                                                               # few rows: their own experts' weights
        row = s["perm"].long() // k if c["gather"] else q
        y = torch.bmm(s["w"][e].float(), s["x"].float()[row][:, :, None])[:, :, 0]
        return (_swiglu(y, c["limit"]) if c["act"] else y).to(s["x"].dtype)
    at = torch.arange(most, device=off.device)
    p = (off[:-1, None] + at).clamp(max=S - 1)                               # [E, most] positions, padded
    row = s["perm"].long()[p].clamp(min=0) // k if c["gather"] else p
    y = torch.bmm(s["x"].float()[row], s["w"].float().transpose(1, 2))
    if c["act"]:
        y = _swiglu(y, c["limit"])
    return y[e, q - off[e]].to(s["x"].dtype)


def _norm(y, w, kind, eps=1e-6):
    if kind == "layer":
        y = y - y.mean(1, keepdim=True)
    return y / torch.sqrt(y.square().mean(1, keepdim=True) + eps) * w.float()


def _block(s, c):
    y = s["y"].float()
    if c["k"]:
        y = (y[s["slot_of"].long()] * s["weights"][:, :, None]).sum(1)
    if c["post"]:
        y = _norm(y, s["post"], c["kind"])
    if s["gate"] is not None:
        y = y * s["gate"].float()
    r = s["residual"].float() + c["scale"] * y
    z = _norm(r, s["pre"], c["kind"])
    return r.to(s["residual"].dtype), z.to(s["y"].dtype)


def run(s):
    c = s["c"]
    if not own:
        if c["op"] == "group":
            return _groups(s["ids"], c["E"])
        return {"router": _router, "product": _product, "norm": _block}[c["op"]](s, c)
    moe = s["moe"]
    if c["op"] == "router":
        return moe.moe_router(s["logits"], c["k"], score=moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX,
                              bias=s["bias"], n_group=c["groups"], topk_group=c["keep"], renormalize=c["renorm"], scale=c["scale"])
    if c["op"] == "group":
        return moe.moe_group(s["ids"], c["E"])
    if c["op"] == "product":
        return s["plan"](s["x"], s["w"], s["offsets"], perm=s["perm"] if c["gather"] else None, topk=c["k"], out=s["out"])
    return moe.moe_block_norm(s["residual"], s["y"], slot_of=s["slot_of"], topk_weights=s["weights"], post_weight=s["post"],
                              gate=s["gate"], scale=c["scale"], pre_weight=s["pre"], eps=1e-6,
                              kind=moe.MOE_NORM_LAYER if c["kind"] == "layer" else moe.MOE_NORM_RMS,
                              residual_out=s["r_out"], out=s["out"])


# ------------------------------------------------------------------------------------ work and exact

def work(c):
    M, k = c["M"], c["k"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if c["op"] == "router":
        return {"bytes": M * c["E"] * size[c["dtype"]] + M * k * 8, "flops": 4 * M * c["E"]}
    if c["op"] == "group":
        return {"bytes": 4 * (3 * M * k + c["E"] + 1), "flops": 0}
    if c["op"] == "product":
        E, K, N = c["E"], c["K"], c["N"]
        touched = E * (1 - (1 - k / E) ** M)                      # expected, of evenly spread ids
        rows = M if c["gather"] else M * k
        wide = N // 2 if c["act"] else N
        return {"bytes": 2 * (touched * N * K + rows * K + M * k * wide) + 4 * (E + 1) + (4 * M * k if c["gather"] else 0),
                "flops": 2 * M * k * N * K}
    H = c["H"]
    res = 2 if c["res"] != "f32" else 4
    gate = {"none": 0, "channel": H, "token": M, "full": M * H}[c["gate"]]
    return {"bytes": M * H * (2 * max(1, k) + 2 * res + 2) + 8 * M * k + 2 * gate + 2 * H * (2 if c["post"] else 1),
            "flops": M * H * (2 * k + 12)}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "group":
        return None
    if c["op"] == "router":
        l = s["logits"].double()
        score = l.sigmoid() if c["score"] == "sigmoid" else l.softmax(1)
        # the choice is made among 32-bit scores
        key = score.float() + s["bias"] if c["score"] == "sigmoid" else s["logits"].float()
        M, E, G = c["M"], c["E"], c["groups"]
        if G > 1:
            parts = key.view(M, G, -1)
            two = parts.sort(2, descending=True).values[:, :, :2]
            rank = two.sum(2) if c["score"] == "sigmoid" else two[:, :, 0]
            order = rank.argsort(dim=1, descending=True, stable=True)
            gone = order[:, c["keep"]:]
            key = parts.clone().scatter_(1, gone[:, :, None].expand(-1, -1, E // G), -math.inf).view(M, E)
        ids = key.argsort(dim=1, descending=True, stable=True)[:, :c["k"]]
        w = torch.take_along_dim(score, ids, 1)
        return None, (w / w.sum(1, keepdim=True) if c["renorm"] else w) * c["scale"]
    if c["op"] == "product":
        off = s["offsets"].tolist()
        out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            x = s["x"][s["perm"][a:b].long() // c["k"]] if c["gather"] else s["x"][a:b]
            y = x.double() @ s["w"][e].double().T
            if c["act"]:
                half = c["N"] // 2
                u, g = y[:, :half], y[:, half:]
                if c["limit"]:
                    u, g = u.clamp(-c["limit"], c["limit"]), g.clamp(max=c["limit"])
                y = u * g * g.sigmoid()
            out[a:b] = y
        return out

    def normed(v, w):
        if c["kind"] == "layer":
            return torch.nn.functional.layer_norm(v, v.shape[1:], w.double(), None, 1e-6)
        return v * w.double() * (v.pow(2).sum(1, keepdim=True) / v.shape[1] + 1e-6).rsqrt()

    y = s["y"].double()
    if c["k"]:
        y = torch.einsum("mkh,mk->mh", y[s["slot_of"].long()], s["weights"].double()) if c["M"] <= 256 else sum(
            y[s["slot_of"][:, j].long()] * s["weights"][:, j:j + 1].double() for j in range(c["k"]))
    if c["post"]:
        y = normed(y, s["post"])
    r = s["residual"].double() + c["scale"] * (y if s["gate"] is None else y * s["gate"].double())
    return r, normed(r, s["pre"])
