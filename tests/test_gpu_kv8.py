"""The 8-bit key/value cache on the GPU against the plain model (kv8_model.py): append and rotary
positions bit for bit, attention within a bound derived there, page operations exactly."""
import numpy as np
import pytest
import torch

from tests import kv8_model as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
woq = None


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    global woq
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import weight_only_quantised_gb300 as w
    woq = w
    torch.cuda.set_device(0)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def kv(g, tokens, heads, dim, scale=1.0):
    x = torch.randn((tokens, heads, dim), generator=g) * scale
    x[..., 3] *= 8
    return x.to(torch.bfloat16)


class Cache:
    """A cache on the GPU and its model side by side."""

    def __init__(self, fmt=0, layers=1, heads=2, dim=128, seqs=1, max_tokens=1000, pages=32):
        self.cfg = woq.KV8Config(format=fmt, layers=layers, kv_heads=heads, head_dim=dim, seqs=seqs,
                                 max_tokens=max_tokens, pages=pages)
        self.guard = torch.full((woq.woq_kv8_bytes(self.cfg) + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        self.buf = self.guard[:-4096]
        woq.woq_kv8_init(self.cfg, self.buf)
        self.model = [[M.Seq(heads, dim) for _ in range(seqs)] for _ in range(layers)]
        self.fmt, self.layers, self.heads, self.dim = fmt, layers, heads, dim

    def prompt(self, seq, g, tokens, scale=1.0):
        if tokens == 0:
            return
        woq.woq_kv8_extend(self.cfg, self.buf, seq, tokens)
        for i in range(self.layers):
            k, v = kv(g, tokens, self.heads, self.dim, scale), kv(g, tokens, self.heads, self.dim, scale)
            self.fill(i, seq, k, v)

    def fill(self, layer, seq, k, v):
        woq.woq_kv8_append_prompt(self.cfg, self.buf, layer, seq, torch.cat([k, v], 1).flatten(1).to(DEV), 0, None)
        self.model[layer][seq].extend(k, v)

    def draft(self, seqs, g, rows):
        for i in range(self.layers):
            k, v = kv(g, len(seqs) * rows, self.heads, self.dim), kv(g, len(seqs) * rows, self.heads, self.dim)
            self.place(i, seqs, rows, k, v)

    def place(self, layer, seqs, rows, k, v):
        woq.woq_kv8_append_rows(self.cfg, self.buf, layer, ints(seqs), rows, torch.cat([k, v], 1).flatten(1).to(DEV), 0, None)
        for e, s in enumerate(seqs):
            m = self.model[layer][s]
            m.pk = torch.cat([k[e * rows:(e + 1) * rows], m.pk[rows:]])
            m.pv = torch.cat([v[e * rows:(e + 1) * rows], m.pv[rows:]])

    def accept(self, seqs, keep):
        woq.woq_kv8_accept(self.cfg, self.buf, ints(seqs), ints(keep))
        for layer in self.model:
            for s, k in zip(seqs, keep):
                layer[s].accept(k)

    def read(self, layer, seq, first, count):
        k = torch.empty((count, self.heads, self.dim), dtype=torch.bfloat16, device=DEV)
        v = torch.empty_like(k)
        woq.woq_kv8_read(self.cfg, self.buf, layer, seq, first, k, v)
        return k.cpu(), v.cpu()

    def check(self, seq, draft=0):
        """Everything the sequence holds, in every layer, bit for bit."""
        for i in range(self.layers):
            m = self.model[i][seq]
            count = m.k.shape[0] + draft
            if count == 0:
                continue
            got = self.read(i, seq, 0, count)
            for a, b in zip(got, m.read(self.fmt, 0, count)):
                assert torch.equal(a, b), f"layer {i}: {(a != b).nonzero()[:4].tolist()}"
        self.sound()

    def state(self):
        cfg = self.cfg
        lens, refs = ints([0] * cfg.seqs), ints([0] * cfg.pages)
        table = torch.empty((cfg.seqs, -(-cfg.max_tokens // 64)), dtype=torch.int32, device=DEV)
        woq.woq_kv8_state(cfg, self.buf, lens, refs, table)
        return lens.cpu().tolist(), refs.cpu().tolist(), table.cpu()

    def sound(self, status=0):
        assert woq.woq_read_status(self.buf, clear=True) == status
        assert (self.guard[-4096:] == 0xA5).all(), "a write behind the cache"
        if self.cfg.pages < 4096:
            lens, refs, table = self.state()
            held = [0] * self.cfg.pages
            for s, n in enumerate(lens):
                for p in table[s, :n // 64].tolist():
                    held[p] += 1
            assert refs == held

    def attend(self, seqs, rows, group, g, window=0, sinks=0, vis=None, scale=None, layer=0, q=None, ws=None):
        """Runs the attention (twice: the results must be the same) and checks it against the model."""
        hq = self.heads * group
        if q is None:
            q = (torch.randn((len(seqs) * rows, hq, self.dim), generator=g) * 1.5).to(torch.bfloat16)
        scale = self.dim ** -0.5 if scale is None else scale
        masks = [[(2 << m) - 1 for m in range(rows)]] * len(seqs) if vis is None else vis
        outs = []
        if ws is None:
            ws = torch.zeros(woq.woq_kv8_attention_workspace(self.cfg, len(seqs), rows, hq), dtype=torch.uint8, device=DEV)
        for _ in range(2):
            out = torch.full((len(seqs) * rows + 2, hq, self.dim), 7.0, dtype=torch.bfloat16, device=DEV)
            woq.woq_kv8_attention(self.cfg, self.buf, layer, ints(seqs), rows, q.to(DEV), hq, out[1:-1], ws, scale,
                                  window=window, sinks=sinks, vis=None if vis is None else ints(vis))
            outs.append(out.cpu())
        self.sound()
        assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16)), "two runs differ"
        assert (outs[0][0] == 7).all() and (outs[0][-1] == 7).all(), "rows outside the call were written"
        assert woq.woq_read_status(ws) == 0
        worst = 0.0
        for e, s in enumerate(seqs):
            ref, bound = M.attention(self.model[layer][s], self.fmt, q[e * rows:(e + 1) * rows], masks[e], scale, window, sinks)
            got = outs[0][1 + e * rows:1 + (e + 1) * rows].double()
            assert torch.isfinite(got).all()
            assert ((got == 0) | (bound > 0)).all()
            worst = max(worst, float(((got - ref).abs() / bound.clamp(min=1e-300)).max()) if bound.any() else 0.0)
        assert worst <= 1.0, f"error is {worst:.3g} of the bound"
        return outs[0][1:-1]


FMTS = [0, 1]


# ----------------------------------------------------------------------------- append

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("tokens", [1, 63, 64, 65, 200])
def test_prompt_is_read_back(fmt, dim, tokens):
    c = Cache(fmt=fmt, dim=dim, heads=3, layers=2)
    c.prompt(0, gen(tokens), tokens)
    c.check(0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("parts", [(1, 1), (10, 54), (10, 200), (70, 3), (70, 58), (127, 1, 129), (5, 7, 0, 300)])
def test_prompts_in_parts_give_the_same_cache(fmt, parts):
    """Codes do not depend on how tokens arrive."""
    c = Cache(fmt=fmt, heads=2)
    g = gen(9)
    for t in parts:
        c.prompt(0, g, t)
        c.check(0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale", [1e-30, 2.0 ** -130, 1e30, 0.0])
def test_extreme_and_zero_values(fmt, scale):
    """Scales far from 1 (int8: the division's route), subnormal values, and blocks of zeros."""
    c = Cache(fmt=fmt, heads=1)
    c.prompt(0, gen(3), 130, scale)
    if fmt == 0 or scale in (1e-30, 1e30, 0.0):
        c.check(0)
    else:  # e4m3 scales stop at 2^-126
        c.sound()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,rot,axes,interleaved", [(128, 128, 1, False), (128, 128, 3, False), (64, 64, 2, True),
                                                     (256, 64, 3, False), (256, 256, 4, True), (64, 4, 1, False)])
def test_rotary_append(dtype, dim, rot, axes, interleaved):
    """Queries and keys of a prompt and of draft rows, from rows with a stride, bit for bit."""
    heads, hq, tokens, rows = 2, 6, 77, 5
    c = Cache(dim=dim, heads=heads, max_tokens=200)
    g = gen(rot + axes)
    table = torch.empty((4096, rot // 2, 2), device=DEV)
    woq.woq_rope_table(1e6, rot, table)
    tab = table.cpu()
    angle = np.arange(4096)[:, None] * 1e6 ** (-np.arange(0, rot, 2) / rot)
    want = torch.tensor(np.stack([np.cos(angle), np.sin(angle)], -1))
    assert ((tab.double() - want).abs() <= want.abs() * 2.0 ** -24 + 4096 * 2.0 ** -50).all()
    axis = [(i * 7 // 3) % axes for i in range(rot // 2)]
    width = (hq + 2 * heads) * dim
    for count, first in ((tokens, 0), (rows, tokens)):
        big = torch.randn((count, width + 24), generator=g).to(dtype)
        x = big[:, :width].float().unflatten(1, (-1, dim))
        pos = torch.randint(0, 4096, (axes, count), generator=g, dtype=torch.int32)
        pos[:, 0] = 4095
        rope = woq.Rope(table, pos.to(DEV), axis_of=axis, interleaved=interleaved)
        q_out = torch.zeros((count + 1, hq, dim), dtype=torch.bfloat16, device=DEV)
        view = big.to(DEV)[:, :width]
        if first == 0:
            woq.woq_kv8_extend(c.cfg, c.buf, 0, count)
            woq.woq_kv8_append_prompt(c.cfg, c.buf, 0, 0, view, hq, q_out[:-1], rope=rope)
        else:
            woq.woq_kv8_append_rows(c.cfg, c.buf, 0, None, rows, view, hq, q_out[:-1], rope=rope)
        r = M.rotate(x, tab, pos, axis, interleaved)
        assert torch.equal(q_out[:-1].cpu(), r[:, :hq]) and (q_out[-1] == 0).all()
        k, v = r[:, hq:hq + heads], x[:, hq + heads:].to(torch.bfloat16)
        if first == 0:
            c.model[0][0].extend(k, v)
        else:
            c.model[0][0].pk, c.model[0][0].pv = k, v
    c.check(0, draft=rows)


def test_positions_outside_the_table_are_reported():
    c = Cache(heads=1)
    table = torch.empty((10, 64, 2), device=DEV)
    woq.woq_rope_table(1e4, 128, table)
    x = torch.randn((3, 2 * 128), device=DEV)
    for bad in (10, -1, 2 ** 30):
        pos = ints([[0, bad, 1]])
        woq.woq_kv8_append_rows(c.cfg, c.buf, 0, ints([0]), 3, x, 0, None, rope=woq.Rope(table, pos))
        assert woq.woq_read_status(c.buf, clear=True) == woq.WOQ_DEVERR_POSITION
    k = c.read(0, 0, 0, 3)[0]
    assert torch.equal(k[1, 0], x[1, :128].cpu().to(torch.bfloat16))  # as by position 0


# ----------------------------------------------------------------------------- attention

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("length", [0, 1, 5, 63, 64, 65, 130, 700])
def test_one_token(fmt, dim, length):
    c = Cache(fmt=fmt, dim=dim)
    g = gen(length + dim)
    c.prompt(0, g, length)
    c.draft([0], g, 1)
    c.attend([0], 1, 5, g)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,group", [(1, 1), (2, 4), (3, 4), (3, 5), (4, 5), (5, 5), (7, 1), (8, 1), (8, 4), (8, 5), (8, 7), (8, 16),
                                        (1, 41), (1, 128), (5, 25), (3, 27)])
def test_rows_and_groups(fmt, rows, group):
    """Every number of query tiles, warps and groups."""
    c = Cache(fmt=fmt, heads=2)
    g = gen(rows * 31 + group)
    c.prompt(0, g, 250)
    c.draft([0], g, rows)
    c.attend([0], rows, group, g)


@pytest.mark.parametrize("dim,rows,group", [(64, 8, 16), (64, 2, 7), (64, 6, 4), (64, 7, 4), (64, 8, 5), (256, 8, 7), (256, 3, 4),
                                            (256, 5, 5), (256, 8, 16), (256, 2, 4), (256, 1, 100), (256, 3, 3), (64, 1, 100)])
def test_rows_and_groups_of_other_heads(dim, rows, group):
    c = Cache(fmt=rows % 2, dim=dim, heads=1)
    g = gen(rows * 31 + group)
    c.prompt(0, g, 333)
    c.draft([0], g, rows)
    c.attend([0], rows, group, g)


@pytest.mark.parametrize("widths", [(7,), (1, 1, 1, 1, 1, 1, 1), (3, 2, 1, 1), (2, 2, 2, 1)])
@pytest.mark.parametrize("length", [0, 60, 127])
def test_draft_trees(widths, length):
    """The planner's trees: each row sees its path."""
    c = Cache(heads=2)
    g = gen(length)
    c.prompt(0, g, length)
    c.draft([0], g, 8)
    c.attend([0], 8, 4, g, vis=[M.tree_masks(widths)])


@pytest.mark.parametrize("dim,group", [(128, 12), (64, 16), (256, 6)])
def test_draft_trees_and_windows_in_chunks(dim, group):
    """More queries than are worked on at once: each chunk has its own rows, masks and windows, and rows of two chunks meet in one row."""
    c = Cache(fmt=1, heads=2, dim=dim, seqs=3)
    g = gen(dim)
    for s, n in enumerate((500, 0, 127)):
        c.prompt(s, g, n)
    c.draft([0, 1, 2], g, 8)
    tree = M.tree_masks((3, 2, 1, 1))
    c.attend([2, 0, 1], 8, group, g, vis=[tree, [0] + tree[1:], tree])
    c.attend([2, 0, 1], 8, group, g, vis=[tree] * 3, window=70, sinks=3)
    c.attend([0, 1], 7, group, g, window=1)


def test_rows_that_see_nothing_and_old_drafts():
    c = Cache(heads=2)
    g = gen(0)
    c.draft([0], g, 8)
    out = c.attend([0], 2, 3, g, vis=[[0, 0b10000001]])
    assert (out[0] == 0).all() and (out[1] != 0).any()
    c.prompt(0, g, 70)
    c.draft([0], g, 8)
    c.attend([0], 2, 3, g, vis=[[0, 0b10000001]])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 64), (64, 0), (65, 4), (100, 65), (300, 1), (900, 7), (5000, 3), (130, 200), (64, 5000)])
def test_window_and_sinks(fmt, window, sinks):
    c = Cache(fmt=fmt, heads=2, seqs=4, pages=64)
    g = gen(window)
    lens = [799, 0, 64, 321]
    for s, n in enumerate(lens):
        c.prompt(s, g, n)
    c.draft([0, 1, 2, 3], g, 4)
    c.attend([0, 1, 2, 3], 4, 2, g, window=window, sinks=sinks)
    c.attend([0, 1, 2, 3], 4, 3, g, window=window, sinks=sinks)
    c.attend([3, 0], 4, 3, g, window=window, sinks=sinks, vis=[[1, 3, 5, 0], [8, 9, 15, 2]])


@pytest.mark.parametrize("fmt", FMTS)
def test_unequal_sequences_in_any_order(fmt):
    c = Cache(fmt=fmt, heads=3, seqs=7, max_tokens=2000, pages=96)
    g = gen(7)
    for s, n in enumerate([0, 1, 640, 1999, 63, 64, 1000]):
        c.prompt(s, g, n)
    c.draft(list(range(7)), g, 1)
    c.attend([6, 1, 3, 0, 5, 4, 2], 1, 4, g)
    c.attend([3, 3, 0, 3], 1, 4, g)  # a sequence may be named twice


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group,rows", [(5, 1), (4, 3), (5, 4), (5, 8), (7, 8)])
def test_long_context_over_many_ctas(fmt, group, rows):
    c = Cache(fmt=fmt, heads=8, max_tokens=9000, pages=150)
    g = gen(1)
    c.prompt(0, g, 9000 - 3)
    c.draft([0], g, rows)
    c.attend([0], rows, group, g)


@pytest.mark.parametrize("dim,rows,group", [(256, 1, 4), (256, 8, 4), (64, 8, 16)])
def test_long_context_of_other_heads(dim, rows, group):
    c = Cache(fmt=1, heads=2, dim=dim, max_tokens=9000, pages=150)
    g = gen(3)
    c.prompt(0, g, 9000 - 40)
    c.draft([0], g, rows)
    c.attend([0], rows, group, g)
    c.attend([0], rows, group, g, window=3000, sinks=100)


def test_one_workspace_for_every_shape():
    """What a launch needs zero is where every shape has it, and left zero."""
    c = Cache(heads=4, seqs=12, max_tokens=4000, pages=200)
    g = gen(11)
    lens = [3990, 0, 640, 1999, 63, 64, 1000, 5, 130, 200, 300, 1]
    for s, n in enumerate(lens):
        c.prompt(s, g, n)
    everyone = list(range(12))
    c.draft(everyone, g, 8)
    shapes = [([0], 1, 4), (everyone, 8, 16), ([0], 8, 5), (everyone, 1, 4), ([3, 0, 6], 3, 4), ([0], 8, 7), (everyone, 2, 4), ([2], 1, 2)]
    size = max(woq.woq_kv8_attention_workspace(c.cfg, len(s), rows, 4 * group) for s, rows, group in shapes)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    for s, rows, group in shapes:
        c.attend(s, rows, group, g, ws=ws)


@pytest.mark.parametrize("rows,group", [(1, 4), (3, 4), (8, 16)])
def test_more_items_than_ctas(rows, group):
    """Contiguous shares: items that begin in one CTA and end in another, one long among many short and empty ones."""
    c = Cache(fmt=1, heads=8, seqs=24, max_tokens=3000, pages=120)
    g = gen(12)
    lens = [(37 * s) % 200 for s in range(24)]
    lens[9], lens[10], lens[20] = 2999, 0, 0
    for s, n in enumerate(lens):
        c.prompt(s, g, n)
    c.draft(list(range(24)), g, rows)
    c.attend(list(range(24)), rows, group, g)
    c.attend([(7 * s) % 24 for s in range(40)], rows, group, g)
    c.attend([9] * 20, rows, group, g, window=700, sinks=70)


def test_two_streams_over_one_cache():
    """Reads of one cache may overlap; each stream has its own workspace."""
    c = Cache(heads=4, seqs=2, max_tokens=3000, pages=100)
    g = gen(13)
    c.prompt(0, g, 2990)
    c.prompt(1, g, 777)
    c.draft([0, 1], g, 8)
    runs = []
    for rows, group, seqs in ((1, 5, [0, 1]), (8, 5, [1, 0])):
        hq = 4 * group
        q = torch.randn((2 * rows, hq, 128), generator=g).to(torch.bfloat16).to(DEV)
        ws = torch.zeros(woq.woq_kv8_attention_workspace(c.cfg, 2, rows, hq), dtype=torch.uint8, device=DEV)
        want = torch.empty_like(q)
        args = (c.cfg, c.buf, 0, ints(seqs), rows, q, hq)
        woq.woq_kv8_attention(*args, want, ws, 0.1)
        outs = [torch.empty_like(q) for _ in range(20)]
        runs.append((torch.cuda.Stream(), args, ws, want, outs))
    torch.cuda.synchronize()
    for i in range(20):
        for stream, args, ws, _, outs in runs:
            with torch.cuda.stream(stream):
                woq.woq_kv8_attention(*args, outs[i], ws, 0.1)
    torch.cuda.synchronize()
    for _, _, _, want, outs in runs:
        assert all(torch.equal(want, out) for out in outs)
    c.sound()


@pytest.mark.parametrize("hq", [4, 20, 48])
def test_peaked_and_flat_scores(hq):
    """One token that outweighs all others far into the sequence, growing scores, and equal scores."""
    c = Cache(heads=1, max_tokens=700)
    g = gen(2)
    k, v = kv(g, 640, 1, 128, 0.3), kv(g, 640, 1, 128)
    q = torch.ones((1, hq, 128), dtype=torch.bfloat16)
    k[500] = 4.0
    k[:, 0, :] += (torch.arange(640) / 200)[:, None].to(torch.bfloat16)
    woq.woq_kv8_extend(c.cfg, c.buf, 0, 640)
    c.fill(0, 0, k, v)
    c.draft([0], g, 1)
    for scale in (1.0, 0.01, 0.0, -1.0):
        c.attend([0], 1, hq, g, q=q, scale=scale)


@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** 60])
def test_queries_far_from_one(size):
    c = Cache(heads=1)
    g = gen(4)
    c.prompt(0, g, 200)
    c.draft([0], g, 1)
    q = (torch.randn((1, 4, 128), generator=g) * size).to(torch.bfloat16)
    c.attend([0], 1, 4, g, q=q, scale=1.0 / size / 11)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hq", [2, 5, 9])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(fmt, hq):
    c = Cache(fmt=fmt, heads=1, max_tokens=400)
    g = gen(5)
    c.prompt(0, g, 190)
    k, v = kv(g, 3, 1, 128), kv(g, 3, 1, 128)
    k[1, 0, 5] = float("inf")
    v[2, 0, 7] = float("nan")
    x = torch.cat([k, v], 1).flatten(1).to(DEV)
    woq.woq_kv8_append_rows(c.cfg, c.buf, 0, ints([0]), 3, x, 0, None)
    m = c.model[0][0]
    m.pk, m.pv = k, v
    ws = torch.zeros(woq.woq_kv8_attention_workspace(c.cfg, 1, 4, hq), dtype=torch.uint8, device=DEV)
    q = torch.randn((4, hq, 128), generator=g).to(torch.bfloat16)
    out = torch.empty((4, hq, 128), dtype=torch.bfloat16, device=DEV)

    def run(vis, window=0, sinks=0):
        woq.woq_kv8_attention(c.cfg, c.buf, 0, ints([0]), 4, q.to(DEV), hq, out, ws, 0.1, vis=ints([vis]), window=window, sinks=sinks)
        return out.cpu()

    o = run([0b001, 0b011, 0b101, 0])
    clean = m.clone()
    clean.pk, clean.pv = torch.nan_to_num(k, 0, 0, 0), torch.nan_to_num(v, 0, 0, 0)
    ref, bound = M.attention(clean, fmt, q, [1, 1, 1, 0], 0.1)
    assert torch.isnan(o[1]).all() and torch.isnan(o[2]).all()
    for r in (0, 3):
        assert ((o[r].double() - ref[r]).abs() <= bound[r]).all()
    # once accepted and its block full, rows that see the block get NaN, rows behind a window do not
    woq.woq_kv8_accept(c.cfg, c.buf, ints([0]), ints([0b010]))
    c.model[0][0].k, c.model[0][0].v = torch.cat([m.k, k[1:2]]), torch.cat([m.v, v[1:2]])
    c.prompt(0, g, 60)
    o = run([0, 0, 0, 0])
    assert torch.isnan(o).all()
    k2 = c.model[0][0]
    tail = k2.clone()
    tail.k, tail.v = torch.nan_to_num(k2.k, 0, 0, 0), k2.v
    ref, bound = M.attention(tail, fmt, q, [0] * 4, 0.1, window=20, sinks=3)
    o = run([0, 0, 0, 0], window=20, sinks=3)
    assert ((o.double() - ref).abs() <= bound).all()
    # queries: NaN stays in its row
    q[2, 1, 0] = float("nan")
    o = run([0, 0, 0, 0], window=20, sinks=3)
    assert torch.isnan(o[2, 1]).all() and torch.isfinite(o[2, 0]).all() and torch.isfinite(o[[0, 1, 3]]).all()


# ----------------------------------------------------------------------------- pages

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_accept_moves_rows_and_fills_blocks(fmt, dim):
    c = Cache(fmt=fmt, dim=dim, layers=2, heads=2, seqs=3)
    g = gen(11)
    c.prompt(0, g, 59)
    c.prompt(2, g, 120)
    for keep in ([0b1, 0b10110001, 0], [0b11111111, 0b11, 0b10000000], [0b1010, 0, 0b11111111], [0b111, 0xFF, 0xFF],
                 [0xFF, 0xFF, 0xFF], [0x7E, 0x81, 0x10], [0xFF, 0x0F, 0xAA], [0xFF, 1, 0x55], [0xFF, 0xFF, 0xFF]):
        c.draft([0, 1, 2], g, 8)
        order = [2, 0, 1]
        c.accept(order, [keep[i] for i in order])
        for s in range(3):
            c.check(s)
    lens, _, _ = c.state()
    assert lens == [m.k.shape[0] for m in c.model[0]]


def test_decode_loop():
    """One token at a time over two block ends: append, attend, accept."""
    c = Cache(heads=2, max_tokens=200)
    g = gen(12)
    c.prompt(0, g, 60)
    for _ in range(70):
        c.draft([0], g, 1)
        c.accept([0], [1])
    c.draft([0], g, 1)
    c.attend([0], 1, 4, g)
    c.check(0, draft=1)


def test_fork_shares_pages_and_frees_them():
    c = Cache(layers=2, heads=2, seqs=5, pages=12, max_tokens=400)
    g = gen(13)
    c.prompt(0, g, 200)
    c.prompt(4, g, 10)
    c.draft([0], g, 8)
    woq.woq_kv8_fork(c.cfg, c.buf, ints([0, 0, 4]), ints([2, 1, 3]))
    for layer in c.model:
        layer[1], layer[2], layer[3] = layer[0].clone(), layer[0].clone(), layer[4].clone()
    lens, refs, _ = c.state()
    assert lens == [200, 200, 200, 10, 10] and refs[:3] == [3, 3, 3] and sum(refs) == 9
    c.accept([1, 2], [0b10101010, 0b1])
    for s in (0, 1, 2):
        c.check(s)
    for s in (1, 2):
        c.prompt(s, g, 100)
        c.check(s)
    c.check(0, draft=8)
    woq.woq_kv8_free(c.cfg, c.buf, ints([0, 3]))
    for layer in c.model:
        layer[0] = M.Seq(2, 128)
    c.check(1)
    c.check(2)
    woq.woq_kv8_free(c.cfg, c.buf, ints([2, 1, 4]))
    lens, refs, _ = c.state()
    assert lens == [0] * 5 and refs == [0] * 12


def test_copies_and_compaction():
    c = Cache(fmt=1, layers=3, heads=2, seqs=6, pages=20, max_tokens=400)
    g = gen(14)
    c.prompt(0, g, 200)
    c.prompt(1, g, 130)
    woq.woq_kv8_copy(c.cfg, c.buf, c.cfg, c.buf, ints([1, 0, 1]), ints([2, 3, 4]))
    for layer in c.model:
        layer[2], layer[3], layer[4] = layer[1].clone(), layer[0].clone(), layer[1].clone()
    lens, refs, table = c.state()
    assert table[2, :2].tolist() == [5, 6] and table[3, :3].tolist() == [7, 8, 9] and table[4, :2].tolist() == [10, 11]
    for s in range(5):
        c.check(s)
    woq.woq_kv8_fork(c.cfg, c.buf, ints([4]), ints([5]))
    for layer in c.model:
        layer[5] = layer[4].clone()
    woq.woq_kv8_free(c.cfg, c.buf, ints([0, 2]))
    for layer in c.model:
        layer[0], layer[2] = M.Seq(2, 128), M.Seq(2, 128)
    woq.woq_kv8_compact(c.cfg, c.buf, 6)          # seven pages are in use: they do not fit
    c.sound(woq.WOQ_DEVERR_PAGES)
    assert c.state()[1][:12] == [0, 0, 0, 1, 1, 0, 0, 1, 1, 1, 2, 2]
    woq.woq_kv8_compact(c.cfg, c.buf, 9)
    for s in range(6):
        c.check(s)
    lens, refs, table = c.state()
    assert refs == [1, 2, 2, 1, 1, 0, 0, 1, 1] + [0] * 11
    assert table[3, :3].tolist() == [7, 8, 0] and table[4, :2].tolist() == [1, 2] == table[5, :2].tolist()
    c.buf[woq.woq_kv8_page_offset(c.cfg, 9):] = 0xEE   # the pool's end is the caller's
    c.prompt(0, g, 128)
    woq.woq_kv8_extend(c.cfg, c.buf, 2, 64)            # no page is left below the limit
    c.sound(woq.WOQ_DEVERR_PAGES)
    for s in (0, 1, 3, 4, 5):
        c.check(s)
    assert (c.buf[woq.woq_kv8_page_offset(c.cfg, 9):] == 0xEE).all()
    woq.woq_kv8_compact(c.cfg, c.buf, 20)
    c.prompt(2, g, 64)
    c.check(2)


def test_copy_into_another_cache():
    a = Cache(layers=2, heads=2, seqs=2, pages=5, max_tokens=320)
    b = Cache(layers=2, heads=2, seqs=4, pages=9, max_tokens=1000)
    g = gen(15)
    a.prompt(0, g, 150)
    a.prompt(1, g, 64)
    b.prompt(1, g, 70)
    woq.woq_kv8_copy(a.cfg, a.buf, b.cfg, b.buf, ints([0, 1, 0]), ints([3, 0, 2]))
    for la, lb in zip(a.model, b.model):
        lb[3], lb[0], lb[2] = la[0].clone(), la[1].clone(), la[0].clone()
    for s in range(4):
        b.check(s)
    for s in range(2):
        a.check(s)
    b.prompt(3, g, 100)
    b.check(3)
    a.check(0)


def test_device_checks_change_nothing():
    """What only the device can see: flagged, and the cache stays as it was."""
    c = Cache(layers=1, heads=1, seqs=4, pages=4, max_tokens=200)
    g = gen(16)
    c.prompt(0, g, 130)
    c.prompt(1, g, 63)
    c.draft([0, 1], g, 8)
    before = c.guard.clone()
    before_status = before[:4].clone()

    def refused(status, fn, *args):
        fn(c.cfg, c.buf, *args)
        assert woq.woq_read_status(c.buf, clear=True) == status
        now = c.guard.clone()
        # the bookkeeping's scratch (moves, page list) may change; lengths, pages, tails and pool may not
        lens, refs, table = c.state()
        assert lens == [130, 63, 0, 0] and refs == [1, 1, 0, 0]
        tails = woq.woq_kv8_page_offset(c.cfg, 0) - 4 * 2 * 72 * 128 * 2
        assert torch.equal(now[tails:], before[tails:])

    S, P = woq.WOQ_DEVERR_STATE, woq.WOQ_DEVERR_PAGES
    refused(S, woq.woq_kv8_free, ints([0, 4]))
    refused(S, woq.woq_kv8_free, ints([-1]))
    refused(S, woq.woq_kv8_free, ints([1, 1]))
    refused(S, woq.woq_kv8_fork, ints([0]), ints([1]))            # not empty
    refused(S, woq.woq_kv8_fork, ints([0, 1]), ints([2, 2]))      # named twice
    refused(S, woq.woq_kv8_fork, ints([0, 2]), ints([2, 3]))      # a destination that is a source
    refused(S, woq.woq_kv8_fork, ints([0, 9]), ints([2, 3]))
    refused(S, woq.woq_kv8_accept, ints([0, 0]), ints([1, 1]))
    refused(S, woq.woq_kv8_accept, ints([0, 7]), ints([1, 1]))
    refused(S, woq.woq_kv8_accept, ints([0, 1]), ints([1, 256]))
    refused(S, woq.woq_kv8_extend, 1, 138)                        # longer than max_tokens
    refused(S, lambda cfg, buf: woq.woq_kv8_copy(cfg, buf, cfg, buf, ints([0]), ints([0])))
    refused(S, lambda cfg, buf: woq.woq_kv8_copy(cfg, buf, cfg, buf, ints([0, 2]), ints([2, 3])))
    refused(P, lambda cfg, buf: woq.woq_kv8_copy(cfg, buf, cfg, buf, ints([0, 0]), ints([2, 3])))
    refused(P, woq.woq_kv8_extend, 2, 64 * 3)
    refused(P, woq.woq_kv8_compact, 1)
    x = torch.zeros((5, 256), dtype=torch.bfloat16, device=DEV)
    refused(S, lambda cfg, buf: woq.woq_kv8_append_prompt(cfg, buf, 0, 0, x, 0, None))       # not what extend reserved
    k = torch.full((9, 1, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    refused(S, lambda cfg, buf: woq.woq_kv8_read(cfg, buf, 0, 0, 130, k, k.clone()))
    assert (k == 3).all()
    refused(S, lambda cfg, buf: woq.woq_kv8_append_rows(cfg, buf, 0, ints([4]), 5, x, 0, None))
    # an accept that all fits but for pages: three sequences full at once with two pages left
    c.prompt(2, g, 63)
    c.prompt(3, g, 63)
    c.draft([1, 2, 3], g, 8)
    woq.woq_kv8_accept(c.cfg, c.buf, ints([1, 2, 3]), ints([1, 1, 1]))
    c.sound(P)
    for s in range(4):
        c.check(s)
    c.accept([1, 3], [1, 3])
    for s in range(4):
        c.check(s)


def test_the_same_sequence_twice_and_padding_in_append_rows():
    c = Cache(heads=1, seqs=3)
    g = gen(17)
    c.prompt(1, g, 20)
    k, v = kv(g, 6, 1, 128), kv(g, 6, 1, 128)
    q_out = torch.full((6, 1, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    qkv = torch.cat([k, k, v], 1).flatten(1).to(DEV)
    woq.woq_kv8_append_rows(c.cfg, c.buf, 0, ints([1, 1, -1]), 2, qkv, 1, q_out)
    assert woq.woq_read_status(c.buf, clear=True) == woq.WOQ_DEVERR_STATE
    c.model[0][1].pk, c.model[0][1].pv = k[:2], v[:2]
    c.check(1, draft=2)
    assert torch.equal(q_out[:2].cpu(), k[:2]) and (q_out[2:] == 9).all()
    ws = torch.zeros(woq.woq_kv8_attention_workspace(c.cfg, 2, 2, 1), dtype=torch.uint8, device=DEV)
    out = torch.full((4, 1, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    woq.woq_kv8_attention(c.cfg, c.buf, 0, ints([5, 1]), 2, q_out[:4], 1, out, ws, 0.1)
    assert woq.woq_read_status(c.buf, clear=True) == woq.WOQ_DEVERR_STATE
    ref, bound = M.attention(c.model[0][1], 0, q_out[2:4].cpu(), [1, 3], 0.1)
    assert (out[:2] == 0).all() and ((out[2:].cpu().double() - ref).abs() <= bound).all()


def test_a_buffer_that_is_no_cache_is_left_alone():
    c = Cache(heads=1)
    other = woq.KV8Config(format=0, layers=1, kv_heads=1, head_dim=128, seqs=1, max_tokens=999, pages=32)
    junk = torch.full((woq.woq_kv8_bytes(c.cfg),), 0x5A, dtype=torch.uint8, device=DEV)
    x = torch.zeros((2, 256), dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(woq.woq_kv8_attention_workspace(c.cfg, 1, 2, 1), dtype=torch.uint8, device=DEV)
    out = torch.full((2, 1, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros((2, 1, 128), dtype=torch.bfloat16, device=DEV)
    for cfg, buf in ((c.cfg, junk), (other, c.buf)):
        woq.woq_kv8_extend(cfg, buf, 0, 2)
        woq.woq_kv8_append_prompt(cfg, buf, 0, 0, x, 0, None)
        woq.woq_kv8_append_rows(cfg, buf, 0, None, 2, x, 0, None)
        woq.woq_kv8_accept(cfg, buf, ints([0]), ints([1]))
        woq.woq_kv8_attention(cfg, buf, 0, None, 2, q, 1, out, ws, 1.0)
        woq.woq_kv8_free(cfg, buf, ints([0]))
        woq.woq_kv8_compact(cfg, buf, 1)
    torch.cuda.synchronize()
    assert (junk == 0x5A).all() and (out == 5).all()
    assert woq.woq_read_status(c.buf, clear=True) == woq.WOQ_DEVERR_HEADER
    assert c.state()[0] == [0]


# ----------------------------------------------------------------------------- as used together

def test_captured_step_on_another_stream():
    """Append, attention, accept captured in a graph on a side stream and replayed: the lengths live on
    the device, so each replay is the next step.  Two graphs share the workspace in turn."""
    heads, group, steps = 2, 4, 6
    hq = heads * group
    c = Cache(heads=heads, max_tokens=300, seqs=2)
    g = gen(20)
    c.prompt(0, g, 60)
    c.prompt(1, g, 125)
    seqs, keep = ints([1, 0]), ints([1, 0b101])
    qkv = torch.zeros((6, (hq + 2 * heads) * 128), device=DEV)
    pos = ints([[0] * 6])
    table = torch.empty((300, 64, 2), device=DEV)
    woq.woq_rope_table(1e4, 128, table)
    q = torch.empty((6, hq, 128), dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(woq.woq_kv8_attention_workspace(c.cfg, 2, 3, hq), dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(q), torch.empty_like(q)]
    stream = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for out in outs:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                woq.woq_kv8_append_rows(c.cfg, c.buf, 0, seqs, 3, qkv, hq, q, rope=woq.Rope(table, pos))
                woq.woq_kv8_attention(c.cfg, c.buf, 0, seqs, 3, q, hq, out, ws, 0.09)
                woq.woq_kv8_accept(c.cfg, c.buf, seqs, keep)
            graphs.append(graph)
        for step in range(steps):
            x = torch.randn(qkv.shape, generator=g)
            p = torch.randint(0, 300, (1, 6), generator=g, dtype=torch.int32)
            qkv.copy_(x)
            pos.copy_(p)
            graphs[step % 2].replay()
            stream.synchronize()
            r = M.rotate(x.unflatten(1, (-1, 128)), table.cpu(), p, [0] * 64)
            k, v = r[:, hq:hq + heads], x.unflatten(1, (-1, 128))[:, hq + heads:].to(torch.bfloat16)
            for e, s in enumerate([1, 0]):
                m = c.model[0][s]
                m.pk, m.pv = k[3 * e:3 * e + 3], v[3 * e:3 * e + 3]
                ref, bound = M.attention(m, 0, r[3 * e:3 * e + 3, :hq], [1, 3, 7], 0.09)
                got = outs[step % 2][3 * e:3 * e + 3].cpu().double()
                assert ((got - ref).abs() <= bound).all()
                m.accept([1, 0b101][e])
        for s in (0, 1):
            c.check(s)


def test_with_the_linears_and_the_planner():
    """A verify pass: qkv linear -> rotary append -> attention of the planner's tree -> o linear, then accept; the
    attention's bf16 output is the o linear's input."""
    import synthetic
    heads, group, hidden = 2, 4, 1024
    hq = heads * group
    n_qkv = (hq + 2 * heads) * 128
    planner = woq.TreePlanner()
    masks = M.tree_masks(planner.shape)
    c = Cache(heads=heads, max_tokens=400)
    g = gen(21)
    c.prompt(0, g, 123)
    packed = []
    for i, (n, k) in enumerate(((n_qkv, hidden), (hidden, hq * 128))):
        w, s = synthetic.weights(4, n, k, seed=30 + i)
        dst = torch.empty(woq.woq_packed_bytes(4, n, k), dtype=torch.uint8, device=DEV)
        woq.woq_pack_device(4, w.to(DEV), s.to(DEV).view(torch.int16), n, k, dst)
        packed.append(dst)
    lws = torch.zeros(max(woq.woq_workspace_bytes(4, 8, n_qkv, hidden), woq.woq_workspace_bytes(4, 8, hidden, hq * 128)),
                      dtype=torch.uint8, device=DEV)
    x = synthetic.activations(8, hidden, seed=5).to(DEV)
    qkv = torch.empty((8, n_qkv), device=DEV)
    table = torch.empty((200, 64, 2), device=DEV)
    woq.woq_rope_table(1e4, 128, table)
    depth = [bin(m).count("1") - 1 for m in masks]
    pos = torch.tensor([[123 + d for d in depth]], dtype=torch.int32)
    q, out = (torch.empty((8, hq * 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = torch.zeros(woq.woq_kv8_attention_workspace(c.cfg, 1, 8, hq), dtype=torch.uint8, device=DEV)
    y = torch.empty((8, hidden), device=DEV)
    woq.woq_w4a8_linear_bf16(packed[0], x, n_qkv, hidden, qkv, lws)
    woq.woq_kv8_append_rows(c.cfg, c.buf, 0, None, 8, qkv, hq, q, rope=woq.Rope(table, pos.to(DEV)))
    woq.woq_kv8_attention(c.cfg, c.buf, 0, None, 8, q, hq, out, ws, 0.002, vis=ints([masks]))
    woq.woq_w4a8_linear_bf16(packed[1], out, hidden, hq * 128, y, lws)
    torch.cuda.synchronize()
    rows = qkv.cpu().unflatten(1, (-1, 128))
    r = M.rotate(rows, table.cpu(), pos, [0] * 64)
    m = c.model[0][0]
    m.pk, m.pv = r[:, hq:hq + heads], rows[:, hq + heads:].to(torch.bfloat16)
    assert torch.equal(q.cpu().unflatten(1, (-1, 128)), r[:, :hq])
    ref, bound = M.attention(m, 0, r[:, :hq], masks, 0.002)
    assert ((out.cpu().double().unflatten(1, (-1, 128)) - ref).abs() <= bound).all()
    # the o linear of the same input by the two-call route is the same
    qi = torch.empty((8, hq * 128), dtype=torch.int8, device=DEV)
    a = torch.empty((8,), device=DEV)
    woq.woq_act_quant_int8(out, qi, a)
    y2 = torch.empty_like(y)
    woq.woq_w4a8_gemv(packed[1], qi, a, hidden, hq * 128, y2, lws)
    assert torch.equal(y, y2)
    c.accept([0], [masks[-1]])
    c.check(0)
