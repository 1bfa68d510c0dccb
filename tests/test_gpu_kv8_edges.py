"""The 8-bit key/value cache where it is easily wrong: values near the ends of bf16's range, plans of many entries
and plans that are made again, refused calls, another config's cache."""
import pytest
import torch

from tests import kv8_model as M
from tests import test_gpu_kv8 as base
from tests.test_gpu_kv8 import DEV, FMTS, Cache, gen, ints, kv

pytestmark = pytest.mark.gpu

woq = None


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    global woq
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import weight_only_quantised_gb300 as w
    woq = base.woq = w
    torch.cuda.set_device(0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim,hq,tokens,top", [(128, 4, 640, 117), (128, 20, 640, 117), (64, 48, 650, 117), (256, 3, 700, 117),
                                               (128, 5, 9000, 113), (128, 12, 9000, 113), (128, 5, 1000, -100), (128, 12, 1000, -100)])
def test_values_near_the_ends_of_the_range(fmt, dim, hq, tokens, top):
    """Magnitudes times tokens just below 2^127 (equal, rising and falling scores, so that weights pass the running
    maximum), and values near the other end.  The tail and the draft rows hold them too."""
    c = Cache(fmt=fmt, heads=1, dim=dim, max_tokens=tokens + 8, pages=160)
    g = gen(tokens + hq)

    def values(n):
        x = (1 + torch.rand((n, 1, dim), generator=g) * 0.5) * 2.0 ** (top - 1)
        return (x * torch.sign(torch.randn((1, 1, dim), generator=g))).to(torch.bfloat16)

    k = kv(g, tokens, 1, dim, 0.1)
    k[:, 0, :] += (torch.arange(tokens) / tokens * 4 / dim)[:, None].to(torch.bfloat16)
    woq.woq_kv8_extend(c.cfg, c.buf, 0, tokens)
    c.fill(0, 0, k, values(tokens))
    c.place(0, [0], 2, kv(g, 2, 1, dim, 0.1), values(2))
    q = torch.ones((2, hq, dim), dtype=torch.bfloat16)
    for scale in (0.0, 1.0, -1.0):
        c.attend([0], 2, hq, g, q=q, scale=scale)


def test_a_refused_extend_leaves_the_pending_prompt():
    """More tokens than fit, or than there are pages for: what the extend before it reserved can still be filled.  A
    prompt that was meant for the refused one is refused, even if it has as many tokens."""
    c = Cache(layers=2, heads=2, seqs=2, pages=5, max_tokens=400)
    g = gen(41)
    woq.woq_kv8_extend(c.cfg, c.buf, 0, 100)
    c.fill(0, 0, kv(g, 100, 2, 128), kv(g, 100, 2, 128))
    woq.woq_kv8_extend(c.cfg, c.buf, 0, 301)
    c.sound(woq.WOQ_DEVERR_STATE)
    woq.woq_kv8_extend(c.cfg, c.buf, 0, 290)
    c.sound(woq.WOQ_DEVERR_PAGES)
    c.fill(1, 0, kv(g, 100, 2, 128), kv(g, 100, 2, 128))
    c.check(0)
    c.prompt(1, g, 192)
    woq.woq_kv8_extend(c.cfg, c.buf, 0, 100)  # two pages, one is left
    c.sound(woq.WOQ_DEVERR_PAGES)
    x = torch.ones((100, 2 * 2 * 128), dtype=torch.bfloat16, device=DEV)
    for layer in range(2):
        woq.woq_kv8_append_prompt(c.cfg, c.buf, layer, 0, x, 0, None)
        c.sound(woq.WOQ_DEVERR_STATE)
    c.check(0)
    c.check(1)
    c.prompt(0, g, 50)
    c.check(0)


def test_state_of_another_configs_cache_and_of_no_cache():
    c = Cache(heads=1, seqs=2)
    other = woq.KV8Config(format=0, layers=1, kv_heads=1, head_dim=128, seqs=2, max_tokens=999, pages=32)
    junk = torch.full((woq.woq_kv8_bytes(c.cfg),), 0x5A, dtype=torch.uint8, device=DEV)
    c.prompt(0, gen(1), 70)
    lens, refs, table = ints([9] * 2), ints([9] * 32), torch.full((2, 16), 9, dtype=torch.int32, device=DEV)
    for cfg, buf in ((c.cfg, junk), (other, c.buf)):
        woq.woq_kv8_state(cfg, buf, lens, refs, table)
        torch.cuda.synchronize()
        assert (lens == 9).all() and (refs == 9).all() and (table == 9).all()
    assert (junk == 0x5A).all()
    assert woq.woq_read_status(c.buf, clear=True) == woq.WOQ_DEVERR_HEADER
    c.check(0)


def test_subnormal_values_in_e4m3():
    """Scales stop at 2^-126, and the codes below are the value's multiples of 2^-126 in e4m3."""
    c = Cache(fmt=1, heads=2)
    c.prompt(0, gen(3), 130, 2.0 ** -130)
    assert (c.model[0][0].k != 0).any()
    c.check(0)


@pytest.mark.parametrize("rows,group", [(1, 4), (3, 4), (8, 6)])
@pytest.mark.parametrize("n,heads", [(33, 2), (64, 2), (70, 2), (70, 1), (129, 1)])
def test_many_entries_that_are_cut(n, heads, rows, group):
    """No more items than CTAs, but more entries than a warp lays out at once; one of them is cut into pieces."""
    c = Cache(fmt=n % 2, heads=heads, seqs=n, max_tokens=4000, pages=70 + 3 * n, dim=64)
    g = gen(n)
    for s in range(n):
        c.prompt(s, g, 3990 if s == n - 2 else (53 * s) % 190)
    c.draft(list(range(n)), g, rows)
    c.attend(list(range(n)), rows, group, g)
    c.attend([(5 * s) % n for s in range(n)], rows, group, g, window=300, sinks=5)


@pytest.mark.parametrize("rows,group", [(1, 4), (3, 4), (8, 6)])
@pytest.mark.parametrize("captured", [False, True])
def test_attention_directly_behind_what_changes_lengths(rows, group, captured):
    """No kernel between a change of lengths and the attention."""
    heads, hq, n = 2, 2 * group, 4
    g = gen(31)
    c = Cache(heads=heads, seqs=n, max_tokens=2000, pages=100)
    lens = [1900, 130, 0, 700]
    for s, t in enumerate(lens):
        c.prompt(s, g, t)
    c.draft(list(range(n)), g, 8)
    q = torch.randn((n * rows, hq, 128), generator=g).to(torch.bfloat16)
    qd, seqs, vis = q.to(DEV), ints([3, 0, 2, 1]), torch.zeros((n, rows), dtype=torch.int32, device=DEV)
    ws = torch.zeros(woq.woq_kv8_attention_workspace(c.cfg, n, rows, hq), dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(qd), torch.empty_like(qd)]
    empty = lambda: M.Seq(heads, 128)  # noqa: E731
    m = c.model[0]

    def step(call, change):
        """attention, call, attention"""
        def run():
            for i in range(2):
                woq.woq_kv8_attention(c.cfg, c.buf, 0, seqs, rows, qd, hq, outs[i], ws, 0.1, vis=vis)
                if i == 0:
                    call()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run()
            run = graph.replay
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        for i in range(2):
            if i == 1:
                change()
            for e, s in enumerate([3, 0, 2, 1]):
                ref, bound = M.attention(m[s], 0, q[e * rows:(e + 1) * rows], [0] * rows, 0.1)
                assert ((outs[i][e * rows:(e + 1) * rows].cpu().double() - ref).abs() <= bound).all(), (i, e)
        c.sound()

    def becomes(**new):
        def change():
            for name, s in new.items():
                m[int(name[1:])] = s()
        return change

    def accept():
        m[0].accept(0xFF), m[1].accept(3), m[3].accept(0x81)

    lists = {k: ints(v) for k, v in dict(a=[0], b=[3], c=[1], d=[2], e=[0, 1, 3], f=[0xFF, 3, 0x81], g=[1, 3]).items()}
    step(lambda: woq.woq_kv8_accept(c.cfg, c.buf, lists["e"], lists["f"]), accept)
    step(lambda: woq.woq_kv8_free(c.cfg, c.buf, lists["a"]), becomes(s0=empty))
    step(lambda: woq.woq_kv8_fork(c.cfg, c.buf, lists["b"], lists["a"]), becomes(s0=lambda: m[3].clone()))
    step(lambda: woq.woq_kv8_copy(c.cfg, c.buf, c.cfg, c.buf, lists["c"], lists["d"]), becomes(s2=lambda: m[1].clone()))
    step(lambda: woq.woq_kv8_free(c.cfg, c.buf, lists["g"]), becomes(s1=empty, s3=empty))
    step(lambda: seqs.copy_(seqs), lambda: None)


@pytest.mark.parametrize("rows,group", [(1, 4), (3, 4)])
@pytest.mark.parametrize("captured", [False, True])
def test_attention_behind_the_end_of_a_long_sequence(rows, group, captured):
    """Freeing a long sequence takes some microseconds and ends with its length, so the attention behind it, in a
    graph, plans with the old length and has to plan anew (in 151 of 152 CTAs when this was written)."""
    g = gen(32)
    c = Cache(heads=1, seqs=3, dim=64, max_tokens=40000, pages=700)
    for s, t in enumerate((39990, 500, 190)):
        c.prompt(s, g, t)
    hq, n = group, 3
    q = torch.randn((n * rows, hq, 64), generator=g).to(torch.bfloat16)
    qd, seqs, gone = q.to(DEV), ints([1, 0, 2]), ints([0])
    vis = torch.zeros((n, rows), dtype=torch.int32, device=DEV)
    ws = torch.zeros(woq.woq_kv8_attention_workspace(c.cfg, n, rows, hq), dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(qd), torch.empty_like(qd)]

    def run():
        for i in range(2):
            woq.woq_kv8_attention(c.cfg, c.buf, 0, seqs, rows, qd, hq, outs[i], ws, 0.1, vis=vis)
            if i == 0:
                woq.woq_kv8_free(c.cfg, c.buf, gone)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        run = graph.replay
    torch.cuda.synchronize()
    run()
    torch.cuda.synchronize()
    for i in range(2):
        if i == 1:
            c.model[0][0] = M.Seq(1, 64)
        for e, s in enumerate((1, 0, 2)):
            ref, bound = M.attention(c.model[0][s], 0, q[e * rows:(e + 1) * rows], [0] * rows, 0.1)
            assert ((outs[i][e * rows:(e + 1) * rows].cpu().double() - ref).abs() <= bound).all(), (i, e)
    c.sound()


@pytest.mark.parametrize("rows,group", [(1, 4), (3, 4)])
def test_a_full_list_of_sequences(rows, group):
    """1024 entries: the most that a call takes."""
    n = 1024
    c = Cache(fmt=1, heads=2, dim=64, seqs=n, max_tokens=200, pages=2 * n)
    g = gen(51)
    for s in range(n):
        c.prompt(s, g, (37 * s) % 140)
    c.draft(list(range(n)), g, rows)
    c.attend([(5 * s) % n for s in range(n)], rows, group, g)
    keep = [(s * 7) % (1 << rows) for s in range(n)]
    c.accept(list(range(n)), keep)
    for s in (0, 1, 511, 1023):
        c.check(s)
    woq.woq_kv8_free(c.cfg, c.buf, ints(list(range(n))))
    c.model = [[M.Seq(2, 64) for _ in range(n)]]
    c.sound()


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(fmt):
    """The last layer of a cache of 11 GB holds what a cache of one layer holds, before and after its pages move."""
    heads, tokens, dim = 8, 40000, 128
    big = woq.KV8Config(format=fmt, layers=64, kv_heads=heads, head_dim=dim, seqs=3, max_tokens=tokens + 8, pages=1300)
    small = woq.KV8Config(format=fmt, layers=1, kv_heads=heads, head_dim=dim, seqs=1, max_tokens=tokens + 8, pages=630)
    assert woq.woq_kv8_page_offset(big, 626) > 1 << 32
    qkv = torch.randn((tokens, 2 * heads * dim), dtype=torch.bfloat16, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    new = torch.randn((8, 2 * heads * dim), dtype=torch.bfloat16, device=DEV, generator=torch.Generator(DEV).manual_seed(2))
    q = torch.randn((8, 5 * heads, dim), dtype=torch.bfloat16, device=DEV, generator=torch.Generator(DEV).manual_seed(3))

    def results(cfg, buf, layer, seq):
        out = []
        for rows in (1, 8):
            ws = torch.zeros(woq.woq_kv8_attention_workspace(cfg, 1, rows, 5 * heads), dtype=torch.uint8, device=DEV)
            out.append(torch.empty_like(q[:rows]))
            woq.woq_kv8_attention(cfg, buf, layer, ints([seq]), rows, q[:rows], 5 * heads, out[-1], ws, 0.09,
                                  vis=torch.zeros((1, rows), dtype=torch.int32, device=DEV))
        for _ in range(2):
            out.append(torch.empty((tokens + 8, heads, dim), dtype=torch.bfloat16, device=DEV))
        woq.woq_kv8_read(cfg, buf, layer, seq, 0, *out[2:])
        assert woq.woq_read_status(buf) == 0
        return out

    def filled(cfg, layer, seq, first):
        buf = torch.empty(woq.woq_kv8_bytes(cfg), dtype=torch.uint8, device=DEV)
        woq.woq_kv8_init(cfg, buf)
        for s in first + [seq]:
            woq.woq_kv8_extend(cfg, buf, s, tokens)
        woq.woq_kv8_append_prompt(cfg, buf, layer, seq, qkv, 0, None)
        woq.woq_kv8_append_rows(cfg, buf, layer, ints([seq]), 8, new, 0, None)
        woq.woq_kv8_accept(cfg, buf, ints([seq]), ints([0xFF]))
        return buf

    one = filled(small, 0, 0, [])
    want = results(small, one, 0, 0)
    buf = filled(big, 63, 2, [1])
    same = lambda seq: all(torch.equal(a, b) for a, b in zip(want, results(big, buf, 63, seq)))  # noqa: E731
    assert same(2)
    woq.woq_kv8_fork(big, buf, ints([2]), ints([0]))
    assert same(0)
    woq.woq_kv8_free(big, buf, ints([1]))
    woq.woq_kv8_compact(big, buf, 650)
    assert same(2) and same(0)
    woq.woq_kv8_compact(big, buf, 1300)
    woq.woq_kv8_copy(big, buf, big, buf, ints([0]), ints([1]))
    woq.woq_kv8_free(big, buf, ints([0, 2]))
    assert same(1)
