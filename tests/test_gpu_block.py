"""A block's norms, routing and experts on the GPU against their definitions in 64 bits (tests/block_model.py)."""
import itertools

import numpy as np
import pytest
import torch

from tests import block_model as M
from tests.helpers import encode_w4, encode_w6

pytestmark = pytest.mark.gpu
DEV = "cuda"
woq = None


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    global woq
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import weight_only_quantised_gb300 as w
    woq = w
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def guarded(shape, dtype):
    """A buffer with 256 bytes of a pattern on both sides; and what shows whether they still hold it."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    return raw[256: 256 + n].view(dtype).view(shape), lambda: bool((raw[:256] == 0x5A).all() and (raw[256 + n:] == 0x5A).all())


BF, F32 = torch.bfloat16, torch.float32

# ------------------------------------------------------------------------------------------- norms


def norm_case(T, D, ut, rt, post=True, gate_rows=0, pre=True, alpha=1.0, beta=1.0, offset=0.0, eps=1e-6, inplace=False, seed=0, u_scale=3.0):
    g = gen(seed + T + D)
    u = (torch.randn((T, D), generator=g) * u_scale).to(ut)
    r = (torch.randn((T, D), generator=g) * 5).to(rt)
    r[:, D // 3] *= 50
    w = lambda: (1 - offset + 0.2 * torch.randn(D, generator=g)).to(BF)  # noqa: E731
    post, pre = w() if post else None, w() if pre else None
    gate = torch.randn((gate_rows, D), generator=g).to(BF) if gate_rows else None
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    ro, ok_r = guarded((T, D), rt)
    out, ok_o = guarded((T, D), BF) if pre is not None else (None, lambda: True)
    rd = dev(r)
    if inplace:
        ro.copy_(rd)
        rd = ro
    woq.woq_block_norm(dev(u), rd, ro, out, post=dev(post), gate=dev(gate), pre=dev(pre), alpha=alpha, beta=beta, offset=offset, eps=eps)
    res, e_res, h, e_h = M.norm(u, r, post, gate, pre, alpha, beta, offset, eps)
    M.close(ro, res, e_res, M.B if rt is BF else M.U)
    if out is not None:
        M.close(out, h, e_h, M.B)
    assert ok_r() and ok_o()


@pytest.mark.parametrize("D", [8, 16, 136, 256, 1000, 4096, 5120, 8192, 8200, 12000, 16384])
@pytest.mark.parametrize("T", [1, 3, 37])
def test_norm_sizes(T, D):
    norm_case(T, D, F32, BF)
    norm_case(T, D, BF, F32, gate_rows=T, alpha=0.7, beta=0.5, offset=1.0)


@pytest.mark.parametrize("ut,rt", list(itertools.product([BF, F32], repeat=2)))
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_norm_types_and_parts(ut, rt, post, pre):
    for gate_rows in (0, 1, 3, 12):
        norm_case(12, 1032, ut, rt, post=post, pre=pre, gate_rows=gate_rows, alpha=0.9, beta=1.5)
    norm_case(5, 640, ut, rt, post=post, pre=pre, inplace=True, gate_rows=5)


def test_norm_many_rows():
    norm_case(70001, 64, BF, BF, gate_rows=1)
    norm_case(2048, 5120, BF, BF, gate_rows=4)


@pytest.mark.parametrize("scale", [1e-18, 1e-6, 1e6, 1e15])
def test_norm_magnitudes(scale):
    norm_case(3, 2048, F32, F32, u_scale=scale)
    norm_case(3, 2048, F32, F32, u_scale=scale, post=False, beta=1 / scale)


def test_norm_of_rows_of_zeros_and_of_nan():
    u, r = torch.randn((4, 256), device=DEV), torch.randn((4, 256), device=DEV)
    w = torch.ones(256, dtype=BF, device=DEV)
    u[1] = 0
    u[2, 7] = float("nan")
    a, b = torch.empty_like(r), torch.empty((4, 256), dtype=BF, device=DEV)
    woq.woq_block_norm(u, r, a, b, post=w, pre=w)
    assert torch.equal(a[1], r[1]) and a[2].isnan().all() and b[2].isnan().all()
    keep = [0, 1, 3]
    c, d = torch.empty_like(r[keep]), torch.empty_like(b[keep])
    woq.woq_block_norm(u[keep], r[keep], c, d, post=w, pre=w)
    assert torch.equal(a[keep], c) and torch.equal(b[keep], d)   # a row goes by itself


# ----------------------------------------------------------------------------------------- routing


def route_case(logits, k, bias=None, live=None, stride=0, **cfg):
    """logits: host tensor bf16 / fp32; the ids have to be those of 64 bits."""
    T, E = logits.shape
    full = torch.full((T, max(stride, E)), 99.0, dtype=logits.dtype)
    full[:, :E] = logits
    dl = full.to(DEV)[:, :E]
    ids, ok_i = guarded((T, k), torch.int32)
    w, ok_w = guarded((T, k), F32)
    woq.woq_route(dl, k, ids, w, bias=None if bias is None else bias.to(DEV), live=None if live is None else torch.tensor([live], dtype=torch.int32, device=DEV), **cfg)
    want_ids, want_w = M.route(logits.double().numpy(), dict(cfg, k=k), None if bias is None else bias.double().numpy(), live)
    got = ids.cpu().numpy()
    assert (got == want_ids).all(), (np.argwhere(got != want_ids)[:4], got[(got != want_ids).any(1)][:2], want_ids[(got != want_ids).any(1)][:2])
    gw = w.double().cpu().numpy()
    assert (np.isnan(gw) == np.isnan(want_w)).all()
    # softmax: the exponent's rounding (|x| 2^-24 for x up to 104) and a sum of 37 steps; 2^-17 relative, and the least fp32
    err = np.abs(gw - want_w)
    assert (np.isnan(gw) | (err <= 2.0 ** -17 * np.abs(want_w) + 1e-37)).all(), err.max()
    assert ok_i() and ok_w()
    return got, gw


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (7, 3), (31, 31), (32, 8), (33, 5), (60, 4), (128, 8), (160, 6), (256, 32), (384, 8), (512, 10), (1000, 9), (1024, 32)])
@pytest.mark.parametrize("score", [0, 1])
def test_route_sizes(E, k, score):
    g = gen(E + k)
    for T, dt in ((1, F32), (5, BF), (203, F32)):
        l = (torch.randn((T, E), generator=g) * 2).to(dt)
        route_case(l, k, score=score)
        route_case(l, k, score=score, renormalise=False, scale=2.5, stride=E + 8, bias=torch.randn(E, generator=g) * 0.1)


@pytest.mark.parametrize("E,groups,tops,best,k", [(64, 8, 4, 1, 6), (64, 8, 4, 2, 6), (256, 8, 4, 2, 8), (160, 8, 3, 1, 6), (60, 4, 1, 2, 15), (96, 32, 32, 2, 12), (96, 32, 5, 1, 12),
                                                  (1024, 2, 1, 2, 32), (24, 2, 2, 1, 3), (512, 16, 3, 2, 8)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_groups(E, groups, tops, best, k, score, with_bias):
    g = gen(E * groups + best)
    for dt in (F32, BF):
        l = (torch.randn((101, E), generator=g) * 1.5).to(dt)
        route_case(l, k, score=score, groups=groups, top_groups=tops, group_best=best, bias=torch.randn(E, generator=g) * 0.05 if with_bias else None)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("groups,tops,best", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_route_ties(score, groups, tops, best):
    """Few distinct logits (and biases): most places are decided by the lower number."""
    g = gen(7)
    l = torch.randint(-2, 3, (300, 64), generator=g).float() / 2
    cfg = dict(score=score, groups=groups, top_groups=tops, group_best=best)
    route_case(l, 9, **cfg)
    route_case(l.to(BF), 9, bias=torch.zeros(64), **cfg)
    route_case(l, 9, bias=torch.randint(0, 2, (64,), generator=g).float() / 4, **cfg)
    route_case(torch.zeros((3, 64)), 24, **cfg)
    l[:, ::3] = -0.0
    l[:, 1::3] = 0.0
    route_case(l, 9, **cfg)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_neighbours_nearer_than_fp32_tells(score, groups):
    """Scores that differ by some 1e-9: biases that make up for the difference of the scores, but for their own rounding."""
    g = gen(11)
    T, E = 64, 32
    l = (torch.randn((1, E), generator=g) * 0.7)
    x = l.double()
    s = torch.softmax(x, 1) if score == 0 else torch.sigmoid(x)
    bias = (0.75 - s[0]).float()                       # s + bias is 0.75 within 2^-26 or so, in every place
    rows = l.repeat(T, 1)
    rows[1:] = torch.nextafter(rows[1:], torch.full_like(rows[1:], 9.0)) if score else rows[1:]
    cfg = dict(score=score, groups=groups, top_groups=max(1, groups // 2), group_best=2 if groups > 1 else 1)
    route_case(rows, 10, bias=bias, **cfg)
    perm = torch.stack([torch.randperm(E, generator=g) for _ in range(T)])
    for i in range(0, T, 7):                           # the same pairs in other places
        route_case(l[:, perm[i]], 10, bias=bias[perm[i]], **cfg)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("groups", [1, 8])
@pytest.mark.parametrize("E,k", [(256, 8), (1024, 32), (100, 32)])
def test_route_many_neighbours(score, groups, E, k):
    """All scores within 2^-25 of each other: more than fit the short way of telling them apart."""
    if E % groups:
        groups = 4
    g = gen(E + k)
    l = torch.randn((5, E), generator=g) * 0.7
    x = l.double()
    for row in range(5):
        s = torch.softmax(x[row], 0) if score == 0 else torch.sigmoid(x[row])
        route_case(l[row: row + 1], k, bias=(0.75 - s).float(), score=score, groups=groups, top_groups=max(1, groups // 2), group_best=1)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_masked_infinite_and_nan(score, groups, with_bias):
    g = gen(13)
    inf, nan = float("inf"), float("nan")
    l = torch.randn((12, 32), generator=g)
    l[0] = -inf
    l[1] = -inf
    l[1, 5] = 1.0                                     # one left
    l[2, 8:] = -inf
    l[3, :16] = -inf
    l[4, 9] = nan
    l[5] = nan
    l[6, 20] = inf
    l[7, 3], l[7, 4], l[7, 9] = inf, nan, inf
    l[8] = -torch.finfo(F32).max                      # the type's lowest value is a logit like any other
    l[9, 4:] = -torch.finfo(F32).max
    l[10] = 80.0
    l[11, ::2], l[11, 1::2] = -95.0, -100.0
    bias = torch.randn(32, generator=g) * 0.1 if with_bias else None
    for best in ((1, 2) if groups > 1 else (1,)):
        for renorm in (False, True):
            route_case(l, 6, score=score, bias=bias, groups=groups, top_groups=max(1, groups // 2), group_best=best, renormalise=renorm)


def test_route_live_rows():
    l = torch.randn((9, 40), generator=gen(3))
    for live in (-1, 0, 1, 8, 9, 50):
        route_case(l, 4, live=live)


def test_route_many_rows():
    """Rows enough that some need 64 bits; a stride whose product passes 32 bits of bytes."""
    g = gen(5)
    l = (torch.randn((20000, 256), generator=g) * 1.5).to(BF)
    route_case(l, 8, score=1, bias=torch.randn(256, generator=g) * 0.02, groups=8, top_groups=4, group_best=2)
    wide = torch.zeros((5, 1 << 28), dtype=F32, device=DEV)          # row 4 starts at 4 GB
    x = torch.randn((5, 48), generator=g)
    wide[:, :48] = x.to(DEV)
    ids, w = torch.empty((5, 3), dtype=torch.int32, device=DEV), torch.empty((5, 3), device=DEV)
    woq.woq_route(wide[:, :48], 3, ids, w)
    assert (ids.cpu().numpy() == M.route(x.double().numpy(), dict(k=3))[0]).all()


# ----------------------------------------------------------------------------------------- experts


class Experts:
    def __init__(self, E, H, I, bits=4, seed=0, scale=0.02):
        rng = np.random.default_rng(seed + E + H + I)
        half = 1 << (bits - 1)
        self.E, self.H, self.I, self.bits = E, H, I, bits
        enc = encode_w4 if bits == 4 else encode_w6

        def make(n, k):
            q = rng.integers(-half, half, (E, n, k))
            s = (np.abs(rng.standard_normal((E, n, k // 128))) * scale * 8 / half + 1e-3).astype(np.float16)
            out = torch.empty(woq.woq_experts_bytes(bits, E, n, k), dtype=torch.uint8, device=DEV)
            for e in range(E):
                dst = out.view(E, -1)[e]
                woq.woq_pack_device(bits, torch.from_numpy(enc(q[e])).to(DEV), torch.from_numpy(s[e].view(np.int16)).to(DEV), n, k, dst)
            return out, torch.from_numpy(q * np.repeat(s.astype(np.float64), 128, axis=2))

        self.gate_up, self.gu = make(2 * I, H)
        self.down, self.d = make(H, I)

    def ws(self, T, k, extra=0):
        return torch.zeros(woq.woq_experts_workspace(self.E, T, k, self.H, self.I) + extra, dtype=torch.uint8, device=DEV)

    def call(self, x, ids, w, y, ws, **kw):
        woq.woq_experts_swiglu(self.bits, self.E, self.gate_up, self.down, x, ids, w, self.I, y, ws, **kw)

    def run(self, x, ids, w, ws=None):
        T, k = ids.shape
        ws = self.ws(T, k) if ws is None else ws
        y, ok = guarded((T, self.H), BF)
        self.call(x.to(DEV), ids.to(DEV), w.to(DEV), y, ws)
        assert ok()
        return y.cpu(), woq.woq_read_status(ws, clear=True)

    def check(self, x, ids, w, ws=None, status=0):
        y, s = self.run(x, ids, w, ws)
        assert s == status
        want, bound = M.experts(x, ids, w, self.gu, self.d)
        M.close(y, want, bound, M.B)
        return y


def chosen(g, T, E, k):
    ids = torch.rand((T, E), generator=g).argsort(1)[:, :k].int().contiguous()
    w = torch.rand((T, k), generator=g) + 0.1
    return ids, w / w.sum(1, keepdim=True)


@pytest.mark.parametrize("bits", [4, 6])
@pytest.mark.parametrize("E,k,H,I", [(1, 1, 128, 128), (4, 2, 256, 384), (3, 3, 384, 128), (16, 4, 1024, 640), (8, 2, 1152, 1280), (5, 1, 128, 1408)])
def test_experts_sizes(E, k, H, I, bits):
    m = Experts(E, H, I, bits)
    g = gen(E + H + bits)
    for T in (1, 2, 8, 9, 33):
        ids, w = chosen(g, T, E, k)
        m.check(torch.randn((T, H), generator=g).to(BF), ids, w)


@pytest.mark.parametrize("bits", [4, 6])
@pytest.mark.parametrize("T", [3, 20, 150, 700])
def test_experts_uneven_loads(T, bits):
    """Most rows choose the same expert; some places have none, some rows none at all; an expert twice in a row."""
    m = Experts(9, 256, 256, bits)
    g = gen(T)
    ids = torch.where(torch.rand((T, 3), generator=g) < 0.6, 4, torch.randint(-1, 9, (T, 3), generator=g)).int()
    ids[T // 2] = -1
    w = torch.randn((T, 3), generator=g)
    y = m.check(torch.randn((T, 256), generator=g).to(BF), ids, w)
    assert (y[T // 2] == 0).all()


def test_experts_of_no_row():
    m = Experts(4, 128, 128)
    ids = torch.full((6, 2), -1, dtype=torch.int32)
    y = m.check(torch.randn((6, 128), generator=gen(1)).to(BF), ids, torch.ones((6, 2)))
    assert (y == 0).all()


def test_experts_whose_number_is_out_of_range():
    m = Experts(4, 128, 128)
    g = gen(2)
    ids = torch.tensor([[0, 4], [1, -2], [2 ** 31 - 1, -2 ** 31], [3, 2]], dtype=torch.int32)
    m.check(torch.randn((4, 128), generator=g).to(BF), ids, torch.rand((4, 2), generator=g), status=woq.WOQ_DEVERR_STATE)


@pytest.mark.parametrize("T", [6, 40])
def test_experts_rows_go_by_themselves(T):
    """A row that is not finite makes its own results NaN, and nobody else's; the run does not change a bit."""
    m = Experts(4, 256, 128)
    g = gen(3)
    ids, w = chosen(g, T, 4, 2)
    x = torch.randn((T, 256), generator=g).to(BF)
    a, _ = m.run(x, ids, w)
    b, _ = m.run(x, ids, w)
    assert torch.equal(a, b)
    x[2, 17], x[5, 200] = float("nan"), float("inf")
    c, _ = m.run(x, ids, w)
    assert c[2].isnan().all() and not c[5].isfinite().any()
    keep = [i for i in range(T) if i not in (2, 5)]
    assert torch.equal(a[keep], c[keep])
    w[3, 1] = float("nan")
    d, _ = m.run(x, ids, w)
    assert d[3].isnan().all() and torch.equal(d[keep][[i for i in range(len(keep)) if keep[i] != 3]], a[[i for i in keep if i != 3]])


@pytest.mark.parametrize("bits", [4, 6])
@pytest.mark.parametrize("T", [4, 90])
def test_experts_outliers(T, bits):
    """A few channels far above the others, so that a group's elements lie many powers of two apart, and exact zeros."""
    m = Experts(6, 512, 256, bits)
    g = gen(T + bits)
    x = torch.randn((T, 512), generator=g) * torch.exp2(-torch.randint(0, 24, (T, 512), generator=g).float())
    x[:, 3::97] *= 1000
    x[1] = 0
    x[2, 128:256] = 0
    ids, w = chosen(g, T, 6, 3)
    y = m.check(x.to(BF), ids, w)
    assert (y[1] == 0).all()


def test_experts_many_places():
    """512 rows of 32 places each, of 40 experts: many items, and an expert for nearly every place."""
    m = Experts(40, 128, 128)
    g = gen(12)
    ids, w = chosen(g, 512, 40, 32)
    m.check(torch.randn((512, 128), generator=g).to(BF), ids, w)


def test_experts_of_a_wide_layer():
    """More tiles and groups than CTAs, one expert: every CTA has steps of several units."""
    m = Experts(2, 4096, 2560)
    g = gen(13)
    for T in (1, 5):
        m.check(torch.randn((T, 4096), generator=g).to(BF), torch.ones((T, 1), dtype=torch.int32), torch.ones((T, 1)))


@pytest.mark.parametrize("T", [1, 40])
def test_experts_a_wait_that_runs_out(T):
    """A CTA that copies no weights: its waits end, the status says so, y stays as it was; and the workspace works again once it
    is zero-filled."""
    m = Experts(8, 512, 384)
    g = gen(14)
    ids, w = chosen(g, T, 8, 2)
    x = torch.randn((T, 512), generator=g).to(BF)
    before, _ = m.run(x, ids, w)
    ws = m.ws(T, 2)
    y = torch.full((T, 512), 7.0, dtype=BF, device=DEV)
    for cta in (0, 3):
        woq.woq_tune_fault(1, cta, 20000)
        try:
            m.call(x.to(DEV), ids.to(DEV), w.to(DEV), y, ws)
            torch.cuda.synchronize()
        finally:
            woq.woq_tune_fault(0, 0, 0)
        assert (y == 7.0).all() and woq.woq_read_status(ws, clear=True) == woq.WOQ_DEVERR_TIMEOUT
        m.call(x.to(DEV), ids.to(DEV), w.to(DEV), y, ws)      # not yet zero-filled: nothing is written
        assert (y == 7.0).all()
        woq.woq_workspace_init(ws)
    m.call(x.to(DEV), ids.to(DEV), w.to(DEV), y, ws)
    assert torch.equal(y.cpu(), before) and woq.woq_read_status(ws) == 0


def test_two_graphs_share_a_workspace():
    """Graphs of two shapes that share a workspace, replayed in turn."""
    a, b = Experts(6, 256, 384), Experts(5, 384, 128, bits=6)
    g = gen(15)
    ws = torch.zeros(max(a.ws(30, 2).numel(), b.ws(3, 3).numel()), dtype=torch.uint8, device=DEV)
    jobs, want = [], []
    s = torch.cuda.Stream()
    for m, T, k in ((a, 30, 2), (b, 3, 3)):
        ids, w = chosen(g, T, m.E, k)
        x = torch.randn((T, m.H), generator=g).to(BF)
        want.append(m.run(x, ids, w)[0])
        args = [x.to(DEV), ids.to(DEV), w.to(DEV), torch.zeros((T, m.H), dtype=BF, device=DEV)]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                m.call(*args, ws)
        jobs.append((graph, args[3], args))
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, _, _ in jobs:
            graph.replay()
    torch.cuda.synchronize()
    for (_, y, _), ref in zip(jobs, want):
        assert torch.equal(y.cpu(), ref)


def test_experts_large_and_small_activations():
    m = Experts(2, 128, 128, scale=1.0)
    g = gen(4)
    for s in (1e-30, 1e-4, 30.0):
        ids, w = chosen(g, 5, 2, 1)
        m.check((torch.randn((5, 128), generator=g) * s).to(BF), ids, w)


@pytest.mark.parametrize("T", [3, 200])
def test_experts_headers(T):
    """A matrix of another shape: the rows that chose it keep their y, and the workspace says so; one that nobody chose
    says nothing."""
    m = Experts(4, 256, 128)
    g = gen(5)
    ids, w = chosen(g, T, 3, 2)
    ids[0] = torch.tensor([2, 1])
    ids[1] = torch.tensor([0, 1])
    x = torch.randn((T, 256), generator=g).to(BF)
    before, _ = m.run(x, ids, w)
    hit = (ids == 2).any(1)
    ws = m.ws(T, 2)
    for buf in (m.gate_up, m.down):
        for e, at in ((2, 0), (2, 8), (2, 16), (2, 20), (3, 16)):   # magic, bits, N, K of the third expert; the fourth's N
            word = buf.view(4, -1)[e][at: at + 4]
            held = word.clone()
            word += 1
            y = torch.full((T, 256), 7.0, dtype=BF, device=DEV)
            m.call(x.to(DEV), ids.to(DEV), w.to(DEV), y, ws)
            y = y.cpu()
            if e == 2:
                assert (y[hit] == 7.0).all() and torch.equal(y[~hit], before[~hit])
            else:
                assert torch.equal(y, before)
            assert woq.woq_read_status(ws, clear=True) == (woq.WOQ_DEVERR_HEADER if e == 2 else 0)
            word.copy_(held)
            m.call(x.to(DEV), ids.to(DEV), w.to(DEV), y := y.to(DEV), ws)
            assert torch.equal(y.cpu(), before) and woq.woq_read_status(ws) == 0


def test_experts_share_a_workspace_between_shapes():
    a, b = Experts(6, 256, 128), Experts(3, 128, 512, bits=6)
    ws = torch.zeros(max(a.ws(40, 2).numel(), b.ws(9, 3).numel()), dtype=torch.uint8, device=DEV)
    g = gen(6)
    for T in (40, 1, 7):
        ids, w = chosen(g, T, 6, 2)
        a.check(torch.randn((T, 256), generator=g).to(BF), ids, w, ws)
        ids, w = chosen(g, min(T, 9), 3, 3)
        b.check(torch.randn((min(T, 9), 128), generator=g).to(BF), ids, w, ws)


def test_experts_beyond_4_gb():
    """Matrices whose offsets pass 32 bits: one expert's bytes copied to the last places."""
    E, H, I = 900, 4096, 1280
    m = Experts(1, H, I)
    one, two = m.gate_up.numel(), m.down.numel()
    big, small = (torch.zeros(E * n, dtype=torch.uint8, device=DEV) for n in (one, two))
    assert big.numel() > 1 << 32
    big.view(E, -1)[:, :256] = m.gate_up[:256]    # every header in order
    small.view(E, -1)[:, :256] = m.down[:256]
    for e in (0, E - 1):
        big.view(E, -1)[e], small.view(E, -1)[e] = m.gate_up, m.down
    g = gen(7)
    x = torch.randn((2, H), generator=g).to(BF)
    want, bound = M.experts(x, torch.zeros((2, 1), dtype=torch.int32), torch.ones((2, 1)), m.gu, m.d)
    y = torch.empty((2, H), dtype=BF, device=DEV)
    ws = torch.zeros(woq.woq_experts_workspace(E, 2, 2, H, I), dtype=torch.uint8, device=DEV)
    ids = torch.tensor([[E - 1, 5], [7, E - 1]], dtype=torch.int32, device=DEV)      # the others' weights are 0
    woq.woq_experts_swiglu(4, E, big, small, x.to(DEV), ids, torch.ones((2, 2), device=DEV), I, y, ws)
    M.close(y, want, bound, M.B)


# ---------------------------------------------------------------------------------------- together


class Block:
    """norm -> router linear -> route -> experts -> norm, as a decoder's step runs them."""

    def __init__(self, T, seed=0):
        self.T, self.D, self.E, self.k = T, 512, 24, 4
        g = gen(seed)
        self.m = Experts(self.E, self.D, 256)
        rng = np.random.default_rng(seed)
        q = rng.integers(-8, 8, (self.E, self.D))
        s = np.full((self.E, self.D // 128), 0.01, dtype=np.float16)
        self.router = torch.empty(woq.woq_packed_bytes(4, self.E, self.D), dtype=torch.uint8, device=DEV)
        woq.woq_pack_device(4, torch.from_numpy(encode_w4(q)).to(DEV), torch.from_numpy(s.view(np.int16)).to(DEV), self.E, self.D, self.router)
        f = lambda *shape, dt=BF: torch.empty(shape, dtype=dt, device=DEV)  # noqa: E731
        w = lambda: (1 + 0.1 * torch.randn(self.D, generator=g)).to(BF).to(DEV)  # noqa: E731
        self.post, self.pre, self.post2, self.pre2 = w(), w(), w(), w()
        self.bias = (torch.randn(self.E, generator=g) * 0.05).to(DEV)
        self.u, self.r = f(T, self.D, dt=F32), f(T, self.D)
        self.r1, self.x, self.r2, self.out, self.y = (f(T, self.D) for _ in range(5))
        self.logits, self.w, self.ids = f(T, self.E, dt=F32), f(T, self.k, dt=F32), f(T, self.k, dt=torch.int32)
        self.lws = torch.zeros(woq.woq_workspace_bytes(4, T, self.E, self.D), dtype=torch.uint8, device=DEV)
        self.ws = self.m.ws(T, self.k)

    def fill(self, seed):
        g = gen(seed)
        self.u.copy_(torch.randn((self.T, self.D), generator=g))
        self.r.copy_(torch.randn((self.T, self.D), generator=g) * 2)

    def run(self):
        woq.woq_block_norm(self.u, self.r, self.r1, self.x, post=self.post, pre=self.pre)
        woq.woq_w4a8_linear_bf16(self.router, self.x, self.E, self.D, self.logits, self.lws)
        woq.woq_route(self.logits, self.k, self.ids, self.w, score=woq.ROUTE_SIGMOID, bias=self.bias, groups=4, top_groups=2, group_best=2, scale=2.5)
        self.m.call(self.x, self.ids, self.w, self.y, self.ws)
        woq.woq_block_norm(self.y, self.r1, self.r2, self.out, post=self.post2, pre=self.pre2)

    def check(self):
        """Each step against its definition on what the step before gave."""
        c = lambda t: t.cpu()  # noqa: E731
        res, e, h, eh = M.norm(c(self.u), c(self.r), c(self.post), None, c(self.pre), 1.0, 1.0, 0.0, 1e-6)
        M.close(self.r1, res, e, M.B)
        M.close(self.x, h, eh, M.B)
        ids, w = M.route(c(self.logits).double().numpy(), dict(score=1, k=self.k, groups=4, top_groups=2, group_best=2, scale=2.5), c(self.bias).double().numpy())
        assert (c(self.ids).numpy() == ids).all() and np.allclose(c(self.w).numpy(), w, rtol=2.0 ** -17)
        y, b = M.experts(c(self.x), c(self.ids), c(self.w), self.m.gu, self.m.d)
        M.close(self.y, y, b, M.B)
        res, e, h, eh = M.norm(c(self.y), c(self.r1), c(self.post2), None, c(self.pre2), 1.0, 1.0, 0.0, 1e-6)
        M.close(self.r2, res, e, M.B)
        M.close(self.out, h, eh, M.B)

    def results(self):
        return [t.clone() for t in (self.r1, self.x, self.logits, self.ids, self.w, self.y, self.r2, self.out)]


@pytest.mark.parametrize("T", [1, 3, 8])
def test_a_block_eager_and_captured(T):
    b = Block(T)
    b.fill(1)
    b.run()
    b.check()
    want = b.results()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            b.run()
            b.run()
    torch.cuda.synchronize()
    for t in (b.r1, b.x, b.y, b.r2, b.out, b.w):
        t.fill_(9)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, b.results()))
    for seed in (2, 3):                       # other inputs through the same graph
        b.fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        b.check()
    assert woq.woq_read_status(b.ws) == 0


def test_two_streams_at_once():
    """Two blocks with workspaces of their own, on two streams."""
    blocks = [Block(5, seed=1), Block(8, seed=2)]
    want = []
    for i, b in enumerate(blocks):
        b.fill(i)
        b.run()
        torch.cuda.synchronize()
        want.append(b.results())
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(20):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.run()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        assert all(torch.equal(p, q) for p, q in zip(w, b.results()))


def test_a_stream_given_by_name():
    m = Experts(4, 256, 128)
    g = gen(8)
    ids, w = chosen(g, 4, 4, 2)
    x = torch.randn((4, 256), generator=g).to(BF)
    want, _ = m.run(x, ids, w)
    s = torch.cuda.Stream()
    y, ws = torch.zeros((4, 256), dtype=BF, device=DEV), m.ws(4, 2)
    xd, di, dw = x.to(DEV), ids.to(DEV), w.to(DEV)
    torch.cuda.synchronize()
    m.call(xd, di, dw, y, ws, stream=s)
    s.synchronize()
    assert torch.equal(y.cpu(), want)


def test_empty_calls():
    z = lambda *s, dt=BF: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
    woq.woq_block_norm(z(0, 64), z(0, 64), z(0, 64), z(0, 64), pre=z(64))
    woq.woq_route(z(0, 16), 2, z(0, 2, dt=torch.int32), z(0, 2, dt=F32))
    m = Experts(2, 128, 128)
    m.call(z(0, 128), z(0, 2, dt=torch.int32), z(0, 2, dt=F32), z(0, 128), m.ws(1, 2))
    torch.cuda.synchronize()
