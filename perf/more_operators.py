"""Workloads of a mixture-of-experts block's operators: routing, the experts' products over 4- and 6-bit
weights, and the norms before and after a block with its gate and residual scale, in plain torch (own = False)
and through the library (own = True)."""
import math

import torch

own = False

GROUP = 128     # weights of a row that share one scale
EPS = 1e-6


def listed():
    return [
        # one token of a decode step behind its router linear
        {"name": "route 1 x 128", "op": "route", "T": 1, "E": 128, "k": 8, "score": "softmax", "dtype": "f32", "bias": False, "groups": 1, "tops": 1, "best": 1, "renorm": True, "pad": 0},
        # the rows of a draft tree, experts in groups with a balance bias
        {"name": "route 8 x 256 groups", "op": "route", "T": 8, "E": 256, "k": 8, "score": "sigmoid", "dtype": "f32", "bias": True, "groups": 8, "tops": 4, "best": 2, "renorm": True, "pad": 0},
        # a prompt's tokens, some of the batch padding
        {"name": "route 8191 x 256 groups", "op": "route", "T": 8191, "E": 256, "k": 8, "score": "sigmoid", "dtype": "bf16", "bias": True, "groups": 8, "tops": 4, "best": 2, "renorm": True, "pad": 77},
        # a prompt's tokens over an odd number of experts
        {"name": "route 16000 x 60", "op": "route", "T": 16000, "E": 60, "k": 4, "score": "softmax", "dtype": "f32", "bias": False, "groups": 1, "tops": 1, "best": 1, "renorm": False, "pad": 0},
        # one token of a decode step: many small experts
        {"name": "experts 1 of 128", "op": "experts", "T": 1, "E": 128, "k": 8, "H": 2048, "I": 768, "bits": 4, "pad": 0},
        # the eight rows of a draft tree
        {"name": "experts 8 of 128", "op": "experts", "T": 8, "E": 128, "k": 8, "H": 2048, "I": 768, "bits": 4, "pad": 0},
        # three rows of verification, few experts as large as the 9B layer's gate, up and down
        {"name": "experts 3 of 8 large", "op": "experts", "T": 3, "E": 8, "k": 2, "H": 4096, "I": 12288, "bits": 4, "pad": 0},
        # int6 experts of a batch of sequences, two rows of it padding
        {"name": "experts 33 of 64 int6", "op": "experts", "T": 33, "E": 64, "k": 6, "H": 2048, "I": 1408, "bits": 6, "pad": 2},
        # a large serving batch: nearly every expert has many rows
        {"name": "experts 500 of 128", "op": "experts", "T": 500, "E": 128, "k": 8, "H": 2048, "I": 768, "bits": 4, "pad": 0},
        # one row behind the o linear of the 27B decoder: its fp32 output normalised, added, and normalised for the next linear
        {"name": "norm 1 x 5120", "op": "norm", "T": 1, "D": 5120, "u": "f32", "r": "bf16", "post": True, "gate": 0, "pre": True, "alpha": 1.0, "beta": 1.0, "offset": 0.0},
        # a prompt behind a gated block: one gate for each of its sequences
        {"name": "norm 8190 x 5120 gated", "op": "norm", "T": 8190, "D": 5120, "u": "bf16", "r": "bf16", "post": True, "gate": 5, "pre": True, "alpha": 1.0, "beta": 0.5, "offset": 0.0},
        # residuals in 32 bits, a learned scale for each channel, norms that hold their weight as 1 + w
        {"name": "norm 2049 x 4096 f32", "op": "norm", "T": 2049, "D": 4096, "u": "f32", "r": "f32", "post": True, "gate": 1, "pre": True, "alpha": 0.8, "beta": 1.0, "offset": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "norm"])
    if op == "route":
        e = rng.choice([8, 16, 24, 60, 64, 96, 128, 160, 256, 384, 512])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if e % g == 0 and e // g >= 4])
        tops = rng.randint(1, groups)
        k = rng.randint(1, min(12, tops * (e // groups)))
        t = _log(rng, 1, 16000 * 60 // e + 8000)
        return {"op": op, "T": t, "E": e, "k": k, "score": rng.choice(["softmax", "sigmoid"]), "dtype": rng.choice(["f32", "bf16"]), "bias": rng.choice([False, True]),
                "groups": groups, "tops": tops, "best": rng.choice([1, 2]), "renorm": rng.choice([True, False]), "pad": rng.randint(0, t // 9)}
    if op == "norm":
        d = 8 * _log(rng, 8, 1024)
        t = _log(rng, 1, 6000 * 5120 // max(d, 2560))
        gate = rng.choice([0, 1, 2, t])
        return {"op": op, "T": t + (t % gate if gate else 0), "D": d, "u": rng.choice(["f32", "bf16"]), "r": rng.choice(["f32", "bf16"]), "post": rng.choice([True, True, False]),
                "gate": gate, "pre": rng.choice([True, True, False]), "alpha": rng.choice([1.0, 0.7]), "beta": rng.choice([1.0, 0.5]), "offset": rng.choice([0.0, 1.0])}
    bits = rng.choice([4, 4, 6])
    e, k = rng.choice([(8, 2), (16, 1), (16, 4), (60, 4), (64, 6), (128, 8), (96, 8)])
    sizes = [(1024, 640), (2048, 384), (2048, 768), (2048, 1408), (2560, 896), (4096, 1280), (4096, 6016)]
    h, i = rng.choice([(h, i) for h, i in sizes if e * 3 * h * i * bits / 8 < 3.8e8])
    t = _log(rng, 1, min(500, 6.2e9 / (6 * k * h * i / 2)))
    return {"op": op, "T": t, "E": e, "k": k, "H": h, "I": i, "bits": bits, "pad": rng.randint(0, t // 9)}


def active(case):
    """Experts that at least one live row chose, for the popularity that the inputs are drawn with (expected, rounded)."""
    e, k, rows = case["E"], case["k"], case["T"] - case["pad"]
    return min(e, k * rows, round(e * (1 - (1 - k / e) ** rows)))


def work(case):
    t = case["T"]
    if case["op"] == "route":
        return {"bytes": t * (case["E"] * (2 if case["dtype"] == "bf16" else 4) + 8 * case["k"]), "flops": t * case["E"] * 8}
    if case["op"] == "norm":
        d, size = case["D"], {"bf16": 2, "f32": 4}
        b = t * d * (size[case["u"]] + 2 * size[case["r"]] + (2 if case["pre"] else 0)) + case["gate"] * d * 2
        return {"bytes": b, "flops": t * d * 10}
    h, i = case["H"], case["I"]
    weights = 3 * h * i * (case["bits"] / 8 + 2 / GROUP)
    live = (t - case["pad"]) * case["k"]
    return {"bytes": int(active(case) * weights) + t * h * 4, "flops": live * 6 * h * i}


# ------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _weights(g, experts, n, k, bits):
    """Codes as a checkpoint holds them (two in a byte, or four in three) and an fp16 scale for each row and 128 columns."""
    q = torch.randint(0, 256, (experts, n, k * bits // 8), dtype=torch.uint8, generator=g, device="cuda")
    c = 0.01 if bits == 4 else 0.0025
    s = torch.randn((experts, n, k // GROUP), generator=g, device="cuda").abs_().mul_(c).add_(c / 20).half()
    return q, s


def _inputs(case, seed):
    """Everything that comes from outside, from the seed alone."""
    g = _gen(seed)
    t = case["T"]
    if case["op"] == "route":
        e = case["E"]
        x = {"logits": (torch.randn((t, e), generator=g, device="cuda") * 1.5 + torch.randn((1, e), generator=g, device="cuda")).to(DTYPES[case["dtype"]])}
        if case["bias"]:
            x["bias"] = torch.randn(e, generator=g, device="cuda") * 0.05
        x["live"] = torch.tensor([t - case["pad"]], dtype=torch.int32, device="cuda")
        return x
    if case["op"] == "norm":
        d = case["D"]
        x = {"u": (torch.randn((t, d), generator=g, device="cuda") * 3).to(DTYPES[case["u"]]),
             "r": (torch.randn((t, d), generator=g, device="cuda") * 5).to(DTYPES[case["r"]])}
        x["r"][:, 5:: max(8, d // 4)] *= 30                                       # a residual stream's few large channels
        for name in ("post", "pre"):
            if case[name]:
                x[name] = (1 - case["offset"] + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
        if case["gate"]:
            x["gate"] = torch.randn((case["gate"], d), generator=g, device="cuda").to(torch.bfloat16)
        return x
    e, k, h, i = case["E"], case["k"], case["H"], case["I"]
    x = {}
    x["gq"], x["gs"] = _weights(g, e, 2 * i, h, case["bits"])
    x["dq"], x["ds"] = _weights(g, e, h, i, case["bits"])
    x["x"] = torch.randn((t, h), generator=g, device="cuda").to(torch.bfloat16)   # behind a norm
    p = torch.rand((t, e), generator=g, device="cuda")                            # experts that the rows chose, and with what weights
    x["ids"] = p.argsort(1, descending=True)[:, :k].int().contiguous()
    w = torch.rand((t, k), generator=g, device="cuda") + 0.1
    x["w"] = w / w.sum(1, keepdim=True)
    if case["pad"]:
        x["ids"][t - case["pad"]:] = -1                                           # rows of padding: no expert
        x["w"][t - case["pad"]:] = 0
    return x


# ------------------------------------------------------------------------------------- plain forms

def _route(case, s):
    """In 64 bits: neighbouring scores can lie nearer to each other than 32 bits tell."""
    l = s["logits"].double()
    t, e = l.shape
    if case["score"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-l))
    c = p + s["bias"].double() if case["bias"] else p
    if case["groups"] > 1:
        by = c.view(t, case["groups"], -1)
        score = by.sort(dim=2, descending=True)[0][:, :, : case["best"]].sum(2)
        best = score.sort(dim=1, descending=True, stable=True)[1][:, : case["tops"]]
        kept = torch.zeros_like(score, dtype=torch.bool).scatter_(1, best, True)
        c = c.masked_fill(~kept[:, :, None].expand_as(by).reshape(t, e), -math.inf)
    ids = c.sort(dim=1, descending=True, stable=True)[1][:, : case["k"]]
    w = p.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    live = torch.arange(t, device=l.device)[:, None] < s["live"]
    return torch.where(live, ids, -1).int(), torch.where(live, w * SCALE, 0).float()


SCALE = 2.5     # of routed weights


def _codes(q, bits):
    """[..., K * bits / 8] bytes -> [..., K] signed codes in fp32."""
    q = q.int()
    if bits == 4:
        v = torch.stack([q & 15, q >> 4], -1).flatten(-2)
        return torch.where(v > 7, v - 16, v).float()
    b = q.unflatten(-1, (-1, 3))
    w = b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16
    v = torch.stack([w & 63, w >> 6 & 63, w >> 12 & 63, w >> 18], -1).flatten(-2)
    return torch.where(v > 31, v - 64, v).float()


def _dense(q, s, bits):
    return (_codes(q, bits).unflatten(-1, (-1, GROUP)) * s.float()[..., None]).flatten(-2)


def _mlp(x, gu, down):
    """x [..., rows, H] through gate and up [..., 2 I, H] and down [..., H, I]."""
    g, u = (x @ gu.transpose(-1, -2)).chunk(2, -1)
    return (g / (1 + torch.exp(-g)) * u) @ down.transpose(-1, -2)


def _experts(case, s):
    t, k, e, bits = case["T"], case["k"], case["E"], case["bits"]
    x, w = s["x"].float(), torch.where(s["ids"] < 0, 0, s["w"])
    y = torch.zeros_like(x)
    if t * k <= 2 * e:                                   # few entries: each with its own expert's weights
        at = s["ids"].flatten().clamp(min=0).long()
        rows = torch.arange(t * k, device="cuda") // k
        part = []
        for i in range(0, t * k, 8):
            j = at[i: i + 8]
            part.append(_mlp(x[rows[i: i + 8], None], _dense(s["gq"][j], s["gs"][j], bits), _dense(s["dq"][j], s["ds"][j], bits))[:, 0])
        y = (torch.cat(part).view(t, k, -1) * w[..., None]).sum(1)
    else:                                                # many: every row through every expert, and what was chosen kept
        for i in range(e):
            wi = torch.where(s["ids"] == i, w, 0).sum(1, keepdim=True)
            y += wi * _mlp(x, _dense(s["gq"][i], s["gs"][i], bits), _dense(s["dq"][i], s["ds"][i], bits))
    return y.to(torch.bfloat16)


def _rms(x):
    return x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)


def _norm(case, s):
    n = s["u"].float()
    if case["post"]:
        n = _rms(n) * (s["post"].float() + case["offset"])
    if case["gate"]:
        n = n * s["gate"].float().repeat_interleave(case["T"] // case["gate"], 0)
    r = case["alpha"] * s["r"].float() + case["beta"] * n
    if not case["pre"]:
        return (r.to(s["r"].dtype),)
    return r.to(s["r"].dtype), (_rms(r) * (s["pre"].float() + case["offset"])).to(torch.bfloat16)


# ------------------------------------------------------------------------------------ prepare, run

def _packed(woq, q, s, n, k, bits):
    experts = q.shape[0]
    out = torch.empty(woq.woq_experts_bytes(bits, experts, n, k), dtype=torch.uint8, device="cuda").view(experts, -1)
    for i in range(experts):
        woq.woq_pack_device(bits, q[i], s[i].view(torch.int16), n, k, out[i])
    return out


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import weight_only_quantised_gb300 as woq
        s["woq"] = woq
        t = case["T"]
        if case["op"] == "route":
            s["ids"] = torch.empty((t, case["k"]), dtype=torch.int32, device="cuda")
            s["w"] = torch.empty((t, case["k"]), device="cuda")
        elif case["op"] == "norm":
            s["r_out"] = torch.empty_like(s["r"])
            s["out"] = torch.empty((t, case["D"]), dtype=torch.bfloat16, device="cuda") if case["pre"] else None
        else:
            h, i = case["H"], case["I"]
            s["gate_up"] = _packed(woq, s.pop("gq"), s.pop("gs"), 2 * i, h, case["bits"])
            s["down"] = _packed(woq, s.pop("dq"), s.pop("ds"), h, i, case["bits"])
            s["y"] = torch.empty((t, h), dtype=torch.bfloat16, device="cuda")
            s["ws"] = torch.zeros(woq.woq_experts_workspace(case["E"], t, case["k"], h, i), dtype=torch.uint8, device="cuda")
    return s


def run(state):
    s, case = state, state["case"]
    if not own:
        return {"route": _route, "experts": _experts, "norm": _norm}[case["op"]](case, s)
    woq = s["woq"]
    if case["op"] == "route":
        woq.woq_route(s["logits"], case["k"], s["ids"], s["w"], score=woq.ROUTE_SOFTMAX if case["score"] == "softmax" else woq.ROUTE_SIGMOID,
                      bias=s.get("bias"), groups=case["groups"], top_groups=case["tops"], group_best=case["best"], renormalise=case["renorm"], scale=SCALE, live=s["live"])
        return s["ids"], s["w"]
    if case["op"] == "norm":
        woq.woq_block_norm(s["u"], s["r"], s["r_out"], s["out"], post=s.get("post"), gate=s.get("gate"), pre=s.get("pre"), alpha=case["alpha"], beta=case["beta"],
                           offset=case["offset"], eps=EPS)
        return (s["r_out"], s["out"]) if case["pre"] else (s["r_out"],)
    woq.woq_experts_swiglu(case["bits"], case["E"], s["gate_up"], s["down"], s["x"], s["ids"], s["w"], case["I"], s["y"], s["ws"])
    return s["y"]


# ------------------------------------------------------------------------------------------- exact

def _exact_route(case, x):
    """Row by row from the definition, on the host; for many rows, the weights of the largest scores only."""
    import numpy as np
    l = x["logits"].double().cpu().numpy()
    b = x["bias"].double().cpu().numpy() if case["bias"] else np.zeros(case["E"])
    t, k, live = case["T"], case["k"], case["T"] - case["pad"]
    ids, w = np.full((t, k), -1, dtype=np.int32), np.zeros((t, k))
    size = case["E"] // case["groups"]
    z = np.exp(l - l.max(1, keepdims=True)) if case["score"] == "softmax" else None
    p = z / z.sum(1, keepdims=True) if z is not None else 1 / (1 + np.exp(-l))
    for r in range(live):
        c = p[r] + b
        groups = range(case["groups"])
        if case["groups"] > 1:
            score = [sum(sorted(c[g * size: (g + 1) * size])[-case["best"]:]) for g in groups]
            groups = sorted(groups, key=lambda g: (-score[g], g))[: case["tops"]]
        pool = np.concatenate([np.arange(g * size, (g + 1) * size) for g in sorted(groups)])
        chosen = pool[np.lexsort((pool, -c[pool]))[:k]]
        ids[r], w[r] = chosen, p[r, chosen]
        if case["renorm"]:
            w[r] /= w[r].sum()
    return torch.from_numpy(ids).cuda(), torch.from_numpy(w * SCALE).cuda()


def _exact_experts(case, x):
    """Expert by expert, over the rows that chose it."""
    t, k, h, i, bits = case["T"], case["k"], case["H"], case["I"], case["bits"]
    y = torch.zeros((t, h), dtype=torch.float64, device="cuda")

    def values(q, s, n, cols):
        j = torch.arange(cols, device="cuda")
        if bits == 4:
            v = (q.long()[:, j // 2] >> (4 * (j % 2))) & 15
        else:
            z = torch.cat([q.long(), torch.zeros((n, 1), dtype=torch.long, device="cuda")], 1)
            at = j * 6 // 8
            v = ((z[:, at] | z[:, at + 1] << 8) >> (j * 6 % 8)) & 63
        half = 1 << (bits - 1)
        return ((v + half) % (2 * half) - half).double() * s.double()[:, j // GROUP]

    for e in x["ids"].unique().tolist():
        if e < 0:
            continue
        rows, place = (x["ids"] == e).nonzero(as_tuple=True)
        gu = values(x["gq"][e], x["gs"][e], 2 * i, h)
        a = x["x"][rows].double() @ gu.T
        hidden = a[:, :i] * torch.sigmoid(a[:, :i]) * a[:, i:]
        y.index_add_(0, rows, x["w"][rows, place].double()[:, None] * (hidden @ values(x["dq"][e], x["ds"][e], h, i).T))
    return y


def _exact_norm(case, x):
    out, res = [], []
    every = case["T"] // case["gate"] if case["gate"] else 1
    for first in range(0, case["T"], 1024):
        u, r = x["u"][first: first + 1024].double(), x["r"][first: first + 1024].double()
        if case["post"]:
            u = u / torch.sqrt(u.pow(2).mean(1, keepdim=True) + EPS) * (x["post"].double() + case["offset"])
        if case["gate"]:
            u = u * x["gate"].double()[torch.arange(first, first + len(u), device="cuda") // every]
        z = r * case["alpha"] + u * case["beta"]
        res.append(z)
        if case["pre"]:
            out.append(z / torch.sqrt(z.pow(2).mean(1, keepdim=True) + EPS) * (x["pre"].double() + case["offset"]))
    return (torch.cat(res), torch.cat(out)) if case["pre"] else (torch.cat(res),)


def exact(case, seed):
    return {"route": _exact_route, "experts": _exact_experts, "norm": _exact_norm}[case["op"]](case, _inputs(case, seed))
