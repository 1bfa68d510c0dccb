"""Workloads of the 8-bit cache operators: rotary append, attention (full, and with a window and
sinks), and the page operations, in plain torch (own = False) and through the library (own = True)."""
import math

import torch

own = False

BLOCK = 64   # tokens that share one scale (per head)
TAIL = 72    # rows kept in bf16 behind the last full block: 63 and 8 drafts, rounded up
THETA = 1e6

# heads of the two decoders whose linears the library's benchmark runs, and a few generic ones
HEADS = {"27b": (40, 8, 128), "9b": (32, 8, 128), "d64": (14, 2, 64), "d256": (8, 2, 256), "mha": (6, 6, 128)}


def listed():
    return [
        # an image and a text prompt of the 27B decoder entering the cache: three position axes, bf16 qkv
        {"name": "prompt 8191 int8", "op": "prompt", "model": "27b", "fmt": "int8", "T": 8191, "axes": 3, "dtype": "bf16"},
        # a short text prompt, the qkv linear's fp32 output
        {"name": "prompt 333 e4m3", "op": "prompt", "model": "9b", "fmt": "e4m3", "T": 333, "axes": 1, "dtype": "f32"},
        # one token's step behind the qkv linear: append, read back, attend; short context, where latency counts
        {"name": "step M=1 ctx 777", "op": "step", "model": "27b", "fmt": "int8", "n": 1, "rows": 1, "ctx": 777, "axes": 1, "tree": "", "window": 0, "sinks": 0},
        # the eight rows of a draft tree at a long context
        {"name": "step tree ctx 16421", "op": "step", "model": "27b", "fmt": "e4m3", "n": 1, "rows": 8, "ctx": 16421, "axes": 3, "tree": "3,2,1,1", "window": 0, "sinks": 0},
        # a long conversation, one token
        {"name": "attend M=1 ctx 131071", "op": "attend", "model": "27b", "fmt": "int8", "n": 1, "rows": 1, "ctx": 131071, "tree": "", "window": 0, "sinks": 0},
        # multi-token verification of three rows
        {"name": "attend M=3 ctx 32785", "op": "attend", "model": "9b", "fmt": "e4m3", "n": 1, "rows": 3, "ctx": 32785, "tree": "", "window": 0, "sinks": 0},
        # a wide draft tree over a long conversation
        {"name": "attend tree ctx 65531", "op": "attend", "model": "27b", "fmt": "int8", "n": 1, "rows": 8, "ctx": 65531, "tree": "7", "window": 0, "sinks": 0},
        # eight requests of unequal lengths
        {"name": "attend 8 seqs 20000", "op": "attend", "model": "9b", "fmt": "int8", "n": 8, "rows": 1, "ctx": 20000, "tree": "", "window": 0, "sinks": 0},
        # a windowed layer: the last 4096 tokens and four sinks of a long conversation
        {"name": "window 4096 ctx 100003", "op": "attend", "model": "27b", "fmt": "int8", "n": 1, "rows": 1, "ctx": 100003, "tree": "", "window": 4096, "sinks": 4},
        # windowed layers of eight requests, four rows each
        {"name": "window 1000 8 seqs", "op": "attend", "model": "9b", "fmt": "e4m3", "n": 8, "rows": 4, "ctx": 9001, "tree": "", "window": 1000, "sinks": 65},
        # four continuations of one sequence: fork, accept different draft rows, look at the ends, free
        {"name": "fork and accept", "op": "fork", "model": "9b", "fmt": "int8", "layers": 16, "ctx": 4986, "forks": 4},
        # copies of a sequence, a hole in the pool, and the pool compacted
        {"name": "copy and compact", "op": "copy", "model": "9b", "fmt": "int8", "layers": 8, "ctx": 16411},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "step", "attend", "attend", "window", "fork", "copy"])
    model, fmt = rng.choice(["27b", "9b", "d64", "d256", "mha"]), rng.choice(["int8", "e4m3"])
    if op == "prompt":
        return {"op": op, "model": model, "fmt": fmt, "T": _log(rng, 3, 8000), "axes": rng.choice([1, 2, 3]), "dtype": rng.choice(["bf16", "f32"])}
    if op == "fork":
        return {"op": op, "model": model, "fmt": fmt, "layers": rng.randint(2, 16), "ctx": _log(rng, 20, 5000), "forks": rng.randint(1, 4)}
    if op == "copy":
        return {"op": op, "model": model, "fmt": fmt, "layers": rng.randint(1, 8), "ctx": _log(rng, 70, 16000)}
    n = rng.choice([1, 1, 2, 5, 8])
    rows = rng.choice([1, 1, 2, 3, 4, 8])
    c = {"op": "step" if op == "step" else "attend", "model": model, "fmt": fmt, "n": n, "rows": rows, "ctx": _log(rng, 1, 60000 // n),
         "tree": rng.choice(["3,2,1,1", "7", "2,2,2,1"]) if rows == 8 else "",
         "window": _log(rng, 1, 8000) if op == "window" else 0, "sinks": rng.choice([0, 1, 4, 65]) if op == "window" else 0}
    return dict(c, axes=rng.choice([1, 3])) if op == "step" else c


def lengths(case):
    """Tokens of each sequence: unequal, the longest is ctx."""
    n, ctx = case.get("n", 1), case["ctx"]
    return [max(0, ctx * (i + 1) // n - (i * 7) % 13 * (i + 1 < n)) for i in range(n)]


def tree_rows(case):
    """For each draft row the draft rows it sees, itself the last: a chain, or a root and levels of
    the given widths of which only the first choice goes on."""
    if not case["tree"]:
        return [list(range(m + 1)) for m in range(case["rows"])]
    path, rows = [0], [[0]]
    for w in case["tree"].split(","):
        first = len(rows)
        rows += [path + [first + j] for j in range(int(w))]
        path = path + [first]
    return rows


def keeps(case):
    """Draft rows that each fork accepts."""
    return [[0, 1, 2, 4, 5, 7], [0, 3], [], [0, 1, 2, 3, 4, 5, 6, 7]][: case["forks"]]


def seen(case, length):
    """Tokens of one sequence that any of its rows sees."""
    w = case["window"]
    return length if not w else min(length, w + case["sinks"])


def work(case):
    hq, h, d = HEADS[case["model"]]
    kv = 2 * h * d
    if case["op"] == "prompt":
        t = case["T"]
        item = 2 if case["dtype"] == "bf16" else 4
        # qkv in, q out, the codes written once and read back once, the read-back out
        return {"bytes": t * ((hq * d + kv) * item + hq * d * 2 + kv * (1 + 1 + 2)), "flops": t * (hq + h) * d * 3 + t * kv * 4}
    if case["op"] == "fork":
        tail = case["ctx"] % BLOCK
        b = f = 0
        for keep in keeps(case):
            rows = tail + len(keep)
            b += case["layers"] * kv * (2 * (tail + 8) * 2 + rows * 2 * 2)  # the tail read and written, the ends read and written
            f += case["layers"] * kv * rows * 2
        return {"bytes": b, "flops": f}
    if case["op"] == "copy":
        # two copies and the move of one (codes read and written each), the read-back
        return {"bytes": case["layers"] * kv * case["ctx"] * (3 * 2 + 1 + 2), "flops": case["layers"] * kv * case["ctx"]}
    tokens = sum(seen(case, x) for x in lengths(case))
    rows = case["n"] * case["rows"]
    b = tokens * (kv + 8 * h / BLOCK) + rows * hq * d * 4
    f = tokens * case["rows"] * hq * d * 4
    if case["op"] == "step":
        b += rows * ((hq * d + kv) * 4 + hq * d * 2 + 3 * kv * 2)
        f += rows * (hq + h) * d * 3
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _kv(g, shape, outliers):
    """Cached keys or values in bf16; keys have a few channels that are much larger, as after a rotation."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    if outliers:
        x[..., 3:: shape[-1] // 4] *= 6
    return x


def _axis_of(case, rot):
    """Axis of each frequency: time, height and width in turn, as for images between text."""
    return [i % case["axes"] for i in range(rot // 2)]


def _positions(case, g, rows, first):
    """Positions of each row on each axis: one image's grid inside running text."""
    p = torch.arange(rows, device="cuda", dtype=torch.int32) + first
    pos = [p]
    for a in range(1, case["axes"]):
        pos.append(p // (5 + a) + torch.randint(0, 3, (rows,), generator=g, device="cuda", dtype=torch.int32))
    return torch.stack(pos)


def _inputs(case, seed):
    """Everything that comes from outside, from the seed alone."""
    hq, h, d = HEADS[case["model"]]
    g = _gen(seed)
    x = {}
    if case["op"] == "prompt":
        t = case["T"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        x["qkv"] = torch.randn((t, (hq + 2 * h) * d), generator=g, device="cuda", dtype=dt)
        x["qkv"][:, hq * d + 3: (hq + h) * d: d // 4] *= 6
        x["pos"] = _positions(case, g, t, 0)
        return x
    if case["op"] in ("fork", "copy"):
        x["k"] = _kv(g, (case["layers"], case["ctx"], h, d), True)
        x["v"] = _kv(g, (case["layers"], case["ctx"], h, d), False)
        if case["op"] == "fork":
            x["pk"] = _kv(g, (case["layers"], 8, h, d), True)
            x["pv"] = _kv(g, (case["layers"], 8, h, d), False)
        return x
    n, rows = case["n"], case["rows"]
    x["k"] = _kv(g, (n, case["ctx"], h, d), True)
    x["v"] = _kv(g, (n, case["ctx"], h, d), False)
    if case["op"] == "step":
        x["qkv"] = torch.randn((n * rows, (hq + 2 * h) * d), generator=g, device="cuda")
        x["pos"] = _positions(case, g, n * rows, case["ctx"])
    else:
        x["q"] = torch.randn((n * rows, hq, d), generator=g, device="cuda", dtype=torch.bfloat16)
        x["pk"] = _kv(g, (n, rows, h, d), True)
        x["pv"] = _kv(g, (n, rows, h, d), False)
    return x


# ------------------------------------------------------------------------------------- plain forms

def _quantise(x, fmt):
    """x [..., blocks, 64, D] bf16 -> codes and one fp32 scale for each block: the largest magnitude
    over 127, or for e4m3 the least power of two that brings it to 448 or less."""
    x = x.float()
    top = x.abs().amax((-1, -2))
    if fmt == "int8":
        scale = top / torch.full((), 127.0, device=x.device)
    else:
        m, e = torch.frexp(top)                                            # 448 = 0.875 * 2^9
        scale = torch.where(top == 0, top, torch.ldexp(torch.ones_like(top), e - 9 + (m > 0.875)))
    y = x / torch.where(scale == 0, torch.ones_like(scale), scale)[..., None, None]
    return (y.round().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)), scale


def _dequantise(codes, scale):
    return codes.float() * scale[..., None, None]


def _table(rows, rot):
    """cos and sin of each position and frequency, from 64-bit angles."""
    f = THETA ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float()


def _rotate(x, pos, table, axis_of):
    """x [rows, heads, D] fp32; halves of D are the two parts of each pair."""
    cs = table[pos[axis_of].long(), torch.arange(axis_of.numel(), device=x.device)[:, None]].transpose(0, 1)[:, None]  # rows, 1, D/2, 2
    a, b = x.chunk(2, -1)
    c, s = cs[..., 0], cs[..., 1]
    return torch.cat([a * c - b * s, b * c + a * s], -1).to(torch.bfloat16)


def _split_rotate(s, qkv):
    hq, h, d = s["heads"]
    qkv = qkv.float().unflatten(1, (hq + 2 * h, d))
    r = _rotate(qkv[:, : hq + h], s["pos"], s["table"], s["axis_of"])
    return r[:, :hq], r[:, hq:], qkv[:, hq + h:].to(torch.bfloat16)


def _blocks(x, fmt):
    """The full blocks of x [..., tokens, H, D]: codes [..., H, blocks, 64, D] and scales; and the rest in bf16."""
    full = x.shape[-3] // BLOCK * BLOCK
    c, s = _quantise(x[..., :full, :, :].movedim(-2, -3).unflatten(-2, (-1, BLOCK)), fmt)
    return c, s, x[..., full:, :, :]


def _unblock(c, s, rest):
    """Back to bf16 tokens [..., tokens, H, D]."""
    y = _dequantise(c, s).flatten(-3, -2).movedim(-3, -2)
    return torch.cat([y.to(torch.bfloat16), rest], -3)


def _plain_sequences(case, x):
    """Sequences as a plain program holds them: codes and scales of full blocks, and 72 rows in bf16."""
    lens = torch.tensor(lengths(case), device="cuda")
    fulls = lens // BLOCK * BLOCK
    s = {"lens": lens, "fulls": fulls}
    i = torch.arange(TAIL, device="cuda")
    for name in ("k", "v"):
        b = x[name].shape[1] // BLOCK
        s[name + "c"], s[name + "s"] = _quantise(x[name][:, : b * BLOCK].movedim(-2, -3).unflatten(-2, (b, BLOCK)), case["fmt"])
        at = (fulls[:, None] + i).clamp(max=case["ctx"] - 1)
        tail = torch.where((fulls[:, None] + i < lens[:, None])[..., None, None], torch.take_along_dim(x[name], at[..., None, None], 1), 0)
        s[name + "t"] = tail
    return s


def _place(s, rows, k, v):
    """The draft rows [n, rows, H, D] behind each sequence's end."""
    at = (s["lens"] - s["fulls"])[:, None] + torch.arange(rows, device="cuda")
    for name, y in (("kt", k), ("vt", v)):
        s[name].scatter_(1, at[..., None, None].expand_as(y), y)


def _attend(case, s, q):
    """q [n * rows, Hq, D] against the cached tokens and the draft rows each row sees."""
    hq, h, d = s["heads"]
    n, rows = case["n"], case["rows"]
    k = torch.cat([_dequantise(s["kc"], s["ks"]).flatten(2, 3), s["kt"].float().movedim(1, 2)], 2)  # n, H, S, D
    v = torch.cat([_dequantise(s["vc"], s["vs"]).flatten(2, 3), s["vt"].float().movedim(1, 2)], 2)
    main = k.shape[2] - TAIL
    i = torch.arange(k.shape[2], device="cuda")
    fulls, lens = s["fulls"][:, None], s["lens"][:, None]
    token = torch.where(i < main, i, i - main + fulls)                                     # n, S
    cached = torch.where(i < main, i < fulls, token < lens)
    draft = torch.where(i < main, -1, token - lens)                                        # a draft row's number, or less than 0
    sees = s["sees"]                                                                       # rows, rows
    before = sees.long().cumsum(1) - 1                                                     # place of draft j among those seen
    drafted = (draft >= 0) & (draft < rows)
    j = draft.clamp(0, rows - 1)
    visible = cached[:, None] | (drafted[:, None] & sees[:, j].movedim(0, 1))              # n, rows, S
    place = torch.where(drafted[:, None], lens[:, None] + before[:, j].movedim(0, 1), token[:, None])
    if case["window"]:
        total = lens[:, None] + sees.sum(1)[None, :, None]
        visible &= (place < case["sinks"]) | (place >= total - case["window"])
    qh = q.float().reshape(n, rows, h, hq // h, d).movedim(2, 1).reshape(n, h, -1, d)
    m = visible[:, None, :, None].expand(n, h, rows, hq // h, -1).flatten(2, 3)
    w = (qh @ k.transpose(2, 3) * d ** -0.5).masked_fill(~m, -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True).clamp(min=-1e30))
    o = (w @ v) / w.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.reshape(n, h, rows, hq // h, d).movedim(1, 2).reshape(n * rows, hq, d).to(torch.bfloat16)


def _plain_prompt(case, s):
    q, k, v = _split_rotate(s, s["qkv"])
    return q, _unblock(*_blocks(k, case["fmt"])), _unblock(*_blocks(v, case["fmt"]))


def _plain_step(case, s):
    q, k, v = _split_rotate(s, s["qkv"])
    n, rows = case["n"], case["rows"]
    k, v = k.unflatten(0, (n, rows)), v.unflatten(0, (n, rows))
    _place(s, rows, k, v)
    return q, k, v, _attend(case, s, q)


def _plain_fork(case, s):
    tail, keep, count = case["ctx"] % BLOCK, s["keep"], s["count"]
    i = torch.arange(TAIL, device="cuda")
    at = torch.where(i < tail, i, tail + torch.take_along_dim(keep, (i - tail).clamp(0, 7)[None], 1))     # forks, 72
    out = []
    for name in ("kt", "vt"):
        y = s[name][:, None].expand(-1, at.shape[0], -1, -1, -1)
        y = torch.take_along_dim(y, at[None, :, :, None, None], 2)                                        # layers, forks, 72, H, D
        full = _dequantise(*_quantise(y[:, :, :BLOCK].movedim(-2, -3), case["fmt"])).movedim(-3, -2).to(torch.bfloat16)
        done = (tail + count >= BLOCK)[None, :, None, None, None]
        y = torch.cat([torch.where(done, full, y[:, :, :BLOCK]), y[:, :, BLOCK:]], 2)
        out.append([y[:, f, :e] for f, e in enumerate(s["ends"])])
    return out[0], out[1], case["ctx"] + count


def _plain_copy(case, s):
    pool, nb = s["pool"], case["ctx"] // BLOCK
    zero = torch.arange(nb, device="cuda")
    one, two = zero + nb, zero + 2 * nb
    tails = {}
    for name in ("kc", "vc", "ks", "vs"):
        pool[name][one] = pool[name][zero]
        pool[name][two] = pool[name][zero]
        pool[name][one] = pool[name][two]      # the hole that the first copy left is filled again
    for name in ("kt", "vt"):
        tails[name] = s[name].clone()
    k, v = (_unblock(pool[a + "c"][one].movedim(0, 2), pool[a + "s"][one].movedim(0, 2), tails[a + "t"]) for a in "kv")
    return k, v, one.int()


# ------------------------------------------------------------------------------- the library's calls

def _cache(case, x):
    """A cache that holds the case's sequences."""
    import weight_only_quantised_gb300 as woq
    hq, h, d = HEADS[case["model"]]
    layers = case.get("layers", 1)
    if case["op"] == "prompt":
        seqs, top, pages = 1, case["T"], case["T"] // BLOCK
    elif case["op"] == "fork":
        seqs, top, pages = 1 + case["forks"], case["ctx"] + 8, case["ctx"] // BLOCK + 1 + case["forks"]
    elif case["op"] == "copy":
        seqs, top, pages = 3, case["ctx"], 3 * (case["ctx"] // BLOCK)
    else:
        seqs, top, pages = case["n"], case["ctx"] + 8, sum(v // BLOCK for v in lengths(case)) + 1
    cfg = woq.KV8Config(format=woq.KV8_INT8 if case["fmt"] == "int8" else woq.KV8_E4M3, layers=layers, kv_heads=h, head_dim=d,
                        seqs=seqs, max_tokens=top, pages=max(1, pages))
    cache = torch.empty(woq.woq_kv8_bytes(cfg), dtype=torch.uint8, device="cuda")
    woq.woq_kv8_init(cfg, cache)
    s = {"woq": woq, "cfg": cfg, "cache": cache, "heads": (hq, h, d)}

    def fill(layer, seq, k, v):
        if k.shape[0]:
            woq.woq_kv8_append_prompt(cfg, cache, layer, seq, torch.cat([k, v], 1).flatten(1).contiguous(), 0, None)

    if case["op"] in ("fork", "copy"):
        if case["ctx"]:
            woq.woq_kv8_extend(cfg, cache, 0, case["ctx"])
        for i in range(layers):
            fill(i, 0, x["k"][i], x["v"][i])
    elif case["op"] != "prompt":
        for i, length in enumerate(lengths(case)):
            if length:
                woq.woq_kv8_extend(cfg, cache, i, length)
            fill(0, i, x["k"][i, :length], x["v"][i, :length])
    return s


def _rows_in(s, layer, seqs, rows, k, v):
    s["woq"].woq_kv8_append_rows(s["cfg"], s["cache"], layer, seqs, rows, torch.cat([k, v], -2).flatten(0, -3).flatten(1).contiguous(), 0, None)


def _own_rope(case, s, x):
    woq, (hq, h, d) = s["woq"], s["heads"]
    s["table"] = torch.empty((int(x["pos"].max()) + 1, d // 2, 2), device="cuda")
    woq.woq_rope_table(THETA, d, s["table"])
    s["rope"] = woq.Rope(s["table"], x["pos"], axis_of=_axis_of(case, d))


def _own_prompt(case, s):
    woq, cfg, cache = s["woq"], s["cfg"], s["cache"]
    woq.woq_kv8_free(cfg, cache, s["seqs"])
    woq.woq_kv8_extend(cfg, cache, 0, case["T"])
    woq.woq_kv8_append_prompt(cfg, cache, 0, 0, s["qkv"], s["heads"][0], s["q"], rope=s["rope"])
    woq.woq_kv8_read(cfg, cache, 0, 0, 0, s["k"], s["v"])
    return s["q"], s["k"], s["v"]


def _own_attend(case, s, q):
    s["woq"].woq_kv8_attention(s["cfg"], s["cache"], 0, s["seqs"], case["rows"], q, s["heads"][0], s["out"], s["ws"], s["heads"][2] ** -0.5,
                               window=case["window"], sinks=case["sinks"], vis=s["vis"])
    return s["out"]


def _own_step(case, s):
    woq, cfg, cache = s["woq"], s["cfg"], s["cache"]
    woq.woq_kv8_append_rows(cfg, cache, 0, s["seqs"], case["rows"], s["qkv"], s["heads"][0], s["q"], rope=s["rope"])
    for i, length in enumerate(lengths(case)):
        woq.woq_kv8_read(cfg, cache, 0, i, length, s["k"][i], s["v"][i])
    return s["q"], s["k"], s["v"], _own_attend(case, s, s["q"])


def _own_fork(case, s):
    woq, cfg, cache = s["woq"], s["cfg"], s["cache"]
    woq.woq_kv8_fork(cfg, cache, s["src"], s["dst"])
    woq.woq_kv8_accept(cfg, cache, s["dst"], s["keep"])
    first = case["ctx"] // BLOCK * BLOCK
    for f in range(case["forks"]):
        woq.woq_kv8_read(cfg, cache, -1, 1 + f, first, s["k"][f], s["v"][f])
    woq.woq_kv8_state(cfg, cache, lens=s["lens"])
    woq.woq_kv8_free(cfg, cache, s["dst"])
    return s["k"], s["v"], s["lens"][1:].long()


def _own_copy(case, s):
    woq, cfg, cache = s["woq"], s["cfg"], s["cache"]
    nb = case["ctx"] // BLOCK
    woq.woq_kv8_compact(cfg, cache, cfg.pages)         # all pages may be used again
    woq.woq_kv8_free(cfg, cache, s["copies"])
    woq.woq_kv8_copy(cfg, cache, cfg, cache, s["from"], s["copies"])
    woq.woq_kv8_free(cfg, cache, s["copies"][:1])
    woq.woq_kv8_compact(cfg, cache, max(1, 2 * nb))
    woq.woq_kv8_read(cfg, cache, -1, 2, 0, s["k"], s["v"])
    woq.woq_kv8_state(cfg, cache, table=s["table"])
    return s["k"], s["v"], s["table"][2, :nb]


# ------------------------------------------------------------------------------------ prepare, run

def prepare(case, seed):
    x = _inputs(case, seed)
    hq, h, d = HEADS[case["model"]]
    bf = {"dtype": torch.bfloat16, "device": "cuda"}
    rows = case.get("n", 1) * case.get("rows", 1)
    if own:
        s = _cache(case, x)
        woq, cfg, cache = s["woq"], s["cfg"], s["cache"]
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        if "pos" in x:
            _own_rope(case, s, x)
        if case["op"] == "prompt":
            s |= {"qkv": x["qkv"], "seqs": ints([0]), "q": torch.empty((case["T"], hq, d), **bf),
                  "k": torch.empty((case["T"], h, d), **bf), "v": torch.empty((case["T"], h, d), **bf)}
        elif case["op"] == "fork":
            s |= {"src": ints([0] * case["forks"]), "dst": ints(list(range(1, 1 + case["forks"]))), "lens": torch.empty(cfg.seqs, dtype=torch.int32, device="cuda"),
                  "keep": ints([sum(1 << j for j in v) for v in keeps(case)])}
            for i in range(case["layers"]):
                _rows_in(s, i, ints([0]), 8, x["pk"][i][None], x["pv"][i][None])
            for name in "kv":
                s[name] = [torch.empty((case["layers"], case["ctx"] % BLOCK + len(v), h, d), **bf) for v in keeps(case)]
        elif case["op"] == "copy":
            s |= {"from": ints([0, 0]), "copies": ints([1, 2]), "table": torch.empty((3, -(-case["ctx"] // BLOCK)), dtype=torch.int32, device="cuda"),
                  "k": torch.empty((case["layers"], case["ctx"], h, d), **bf), "v": torch.empty((case["layers"], case["ctx"], h, d), **bf)}
        else:
            n = case["n"]
            s |= {"seqs": ints(list(range(n))), "out": torch.empty((rows, hq, d), **bf),
                  "vis": ints([sum(1 << j for j in r) for r in tree_rows(case)] * n).view(n, case["rows"]),
                  "ws": torch.zeros(woq.woq_kv8_attention_workspace(cfg, n, case["rows"], hq), dtype=torch.uint8, device="cuda")}
            if case["op"] == "step":
                s |= {"qkv": x["qkv"], "q": torch.empty((rows, hq, d), **bf), "k": torch.empty((n, case["rows"], h, d), **bf), "v": torch.empty((n, case["rows"], h, d), **bf)}
            else:
                s["q"] = x["q"]
                _rows_in(s, 0, s["seqs"], case["rows"], x["pk"], x["pv"])
    else:
        s = {"heads": (hq, h, d)}
        if "pos" in x:
            s |= {"qkv": x["qkv"], "pos": x["pos"], "table": _table(int(x["pos"].max()) + 1, d), "axis_of": torch.tensor(_axis_of(case, d), device="cuda")}
        if case["op"] == "fork":
            tail = case["ctx"] % BLOCK
            for name in "kv":
                t = torch.zeros((case["layers"], TAIL, h, d), **bf)
                t[:, :tail] = x[name][:, case["ctx"] - tail:]
                t[:, tail: tail + 8] = x["p" + name]
                s[name + "t"] = t
            s["keep"] = torch.tensor([v + [0] * (8 - len(v)) for v in keeps(case)], device="cuda")
            s["count"] = torch.tensor([len(v) for v in keeps(case)], device="cuda")
            s["ends"] = [tail + len(v) for v in keeps(case)]
        elif case["op"] == "copy":
            nb = case["ctx"] // BLOCK
            s["pool"] = {}
            for name in "kv":
                c, sc, s[name + "t"] = _blocks(x[name], case["fmt"])                       # layers, H, blocks, 64, D
                for key, y in ((name + "c", c), (name + "s", sc)):
                    y = y.movedim(2, 0)
                    s["pool"][key] = torch.zeros((3 * nb, *y.shape[1:]), dtype=y.dtype, device="cuda")
                    s["pool"][key][:nb] = y
        elif case["op"] != "prompt":
            s |= _plain_sequences(case, x)
            m = case["rows"]
            s["sees"] = torch.tensor([[j in r for j in range(m)] for r in tree_rows(case)], device="cuda")
            if case["op"] == "attend":
                s["q"] = x["q"]
                _place(s, m, x["pk"], x["pv"])
    s["case"] = case
    return s


def run(state):
    case = state["case"]
    if case["op"] == "attend":
        return _own_attend(case, state, state["q"]) if own else _attend(case, state, state["q"])
    if own:
        return {"prompt": _own_prompt, "step": _own_step, "fork": _own_fork, "copy": _own_copy}[case["op"]](case, state)
    return {"prompt": _plain_prompt, "step": _plain_step, "fork": _plain_fork, "copy": _plain_copy}[case["op"]](case, state)


# ------------------------------------------------------------------------------------------- exact

def _values64(x, fmt):
    """What the cache stands for after it took in x [tokens, H, D] (bf16 values): 64-bit."""
    out = x.double().clone()
    full = x.shape[0] // BLOCK * BLOCK
    y = out[:full].reshape(-1, BLOCK, *x.shape[1:])
    top = y.abs().amax((1, 3), keepdim=True)
    s = (top / 127).float().double() if fmt == "int8" else torch.exp2(torch.ceil(torch.log2(top / 448)))   # held in 32 bits
    z = torch.where(s > 0, y / s, 0.0)
    if fmt == "int8":
        z = z.round()
    else:                                                                 # e4m3: 3 bits after the first, steps of 2^-9 below 2^-6
        step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
        z = (z / step).round() * step
    out[:full] = (z * s).reshape(full, *x.shape[1:])
    return out


def _rotate64(x, pos, axis_of):
    """Each pair turned as a complex number by its angle."""
    half = x.shape[-1] // 2
    turn = torch.stack([pos[a].double() * THETA ** (-i / half) for i, a in enumerate(axis_of)], 1)[:, None]
    z = torch.complex(x[..., :half].double(), x[..., half:].double()) * torch.polar(torch.ones_like(turn), turn)
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    x = _inputs(case, seed)
    hq, h, d = HEADS[case["model"]]
    fmt = case["fmt"]
    if case["op"] == "fork":
        first = case["ctx"] // BLOCK * BLOCK
        out = []
        for name in "kv":
            out.append([torch.stack([_values64(torch.cat([x[name][i, first:], x["p" + name][i][keep]]), fmt) for i in range(case["layers"])]) for keep in keeps(case)])
        return out[0], out[1], None
    if case["op"] == "copy":
        return [torch.stack([_values64(y, fmt) for y in x[name]]) for name in "kv"] + [None]
    if "qkv" in x:
        y = x["qkv"].reshape(-1, hq + 2 * h, d)
        ax = _axis_of(case, d)
        q, k, v = _rotate64(y[:, :hq], x["pos"], ax), _rotate64(y[:, hq:hq + h], x["pos"], ax), y[:, hq + h:]
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)                 # what the cache takes in
        if case["op"] == "prompt":
            return q, _values64(k, fmt), _values64(v, fmt)
        q = q.to(torch.bfloat16)
        x["pk"], x["pv"] = k.reshape(case["n"], -1, h, d), v.reshape(case["n"], -1, h, d)
    else:
        q = x["q"]
    rows, out = case["rows"], []
    for b, length in enumerate(lengths(case)):
        k, v = _values64(x["k"][b, :length], fmt), _values64(x["v"][b, :length], fmt)
        for m, sees in enumerate(tree_rows(case)):
            kk, vv = torch.cat([k, x["pk"][b][sees].double()]), torch.cat([v, x["pv"][b][sees].double()])
            at = torch.arange(len(kk), device="cuda")
            if case["window"]:
                at = at[(at < case["sinks"]) | (at >= len(kk) - case["window"])]
            qq = q[b * rows + m].double().reshape(h, hq // h, d)
            p = torch.softmax(torch.einsum("hgd,shd->hgs", qq, kk[at]) * d ** -0.5, -1)
            out.append(torch.einsum("hgs,shd->hgd", p, vv[at]).reshape(hq, d))
    o = torch.stack(out)
    return (q.double(), x["pk"].double(), x["pv"].double(), o) if case["op"] == "step" else o
