"""A block's routing and experts where their arithmetic is most easily wrong: codes that are all zero or small, near scores
that are not neighbours, results from run to run, workspaces after a wait that ran out."""
import numpy as np
import pytest
import torch

from tests import test_gpu_block as B
from tests.helpers import encode_w4, encode_w6

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
woq = None


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    global woq
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import weight_only_quantised_gb300 as w
    woq = B.woq = w
    torch.cuda.set_device(0)


# ------------------------------------------------------------------------------------------- codes


class Coded(B.Experts):
    """Experts of given codes, gate_up [E, 2 I, H] and down [E, H, I], under scales of 2^-6."""

    def __init__(self, bits, gate_up, down):
        self.E, self.H, self.I, self.bits = gate_up.shape[0], gate_up.shape[2], down.shape[2], bits
        enc = encode_w4 if bits == 4 else encode_w6

        def make(q):
            e, n, k = q.shape
            s = torch.from_numpy(np.full((n, k // 128), 2.0 ** -6, dtype=np.float16).view(np.int16)).to(DEV)
            out = torch.empty(woq.woq_experts_bytes(bits, e, n, k), dtype=torch.uint8, device=DEV)
            for i in range(e):
                woq.woq_pack_device(bits, torch.from_numpy(enc(q[i])).to(DEV), s, n, k, out.view(e, -1)[i])
            return out, torch.from_numpy(q * 2.0 ** -6)

        self.gate_up, self.gu = make(gate_up)
        self.down, self.d = make(down)


def codes(seed, bits, shape, most=None):
    half = 1 << (bits - 1)
    return np.random.default_rng(seed).integers(-half if most is None else -most, half if most is None else most + 1, shape)


@pytest.mark.parametrize("bits", [4, 6])
@pytest.mark.parametrize("H,I", [(256, 128), (384, 1408)])
@pytest.mark.parametrize("T", [3, 70])
def test_channels_whose_codes_are_zero(T, H, I, bits):
    """A down row of zeros gives 0 exactly: the products of a group are 128 multiples of 2^-15 (the offset's code times a half)
    that sum to less than 2^9, so 24 bits hold every sum on the way, and what takes the offset off is the same number
    rounded the same way."""
    down = codes(1, bits, (3, H, I))
    down[:, ::3] = 0
    m = Coded(bits, codes(2, bits, (3, 2 * I, H)), down)
    g = B.gen(T + I)
    ids, w = B.chosen(g, T, 3, 2)
    y = m.check(torch.randn((T, H), generator=g).to(BF), ids, w)
    assert (y[:, ::3] == 0).all()


@pytest.mark.parametrize("bits", [4, 6])
@pytest.mark.parametrize("T", [3, 70])
def test_up_rows_whose_codes_are_zero(T, bits):
    """As above for x, some of it far below the group's largest: U x is 0, so h and y are."""
    gate_up = codes(3, bits, (3, 512, 512))
    gate_up[:, 256:] = 0
    m = Coded(bits, gate_up, codes(4, bits, (3, 512, 256)))
    g = B.gen(T)
    ids, w = B.chosen(g, T, 3, 2)
    x = torch.randn((T, 512), generator=g) * torch.exp2(-torch.randint(0, 24, (T, 512), generator=g).float())
    x[:, 3::97] *= 1000
    y, status = m.run(x.to(BF), ids, w)
    assert status == 0 and (y == 0).all()


@pytest.mark.parametrize("bits", [4, 6])
@pytest.mark.parametrize("T", [8, 70])
def test_small_codes(T, bits):
    """Codes of -1, 0 and 1: an h's rounding counts with its weight, not with the offset (8 or 32 times that)."""
    m = Coded(bits, codes(5, bits, (3, 256, 256)), codes(6, bits, (3, 256, 128), 1))
    g = B.gen(T)
    ids, w = B.chosen(g, T, 3, 1)
    m.check(torch.randn((T, 256), generator=g).to(BF), ids, w)


# --------------------------------------------------------------------------------------- near scores


@pytest.mark.parametrize("E", [0, 64, 100, 256, 1024])
@pytest.mark.parametrize("l,k", [([20.0, 20, 21], 1), ([18.0] * 9 + [19], 8), ([25.0] + [18.0] * 40 + [19] + [18.0] * 20, 4)])
def test_route_equal_scores_hide_none(l, k, E):
    """Sigmoids that fp32 rounds to 1, most of them of the very same logit: the greater one behind them is chosen."""
    for at in (0, E // 3):
        row = torch.full((1, max(E, len(l))), 3.0)
        row[0, at: at + len(l)] = torch.tensor(l)[: row.shape[1] - at]
        B.route_case(row, k, bias=torch.zeros(row.shape[1]), score=1)


@pytest.mark.parametrize("groups", [1, 3])
def test_route_softmax_rounds_logits_together(groups):
    """l - m is the same in fp32 for the logits near 0."""
    l = torch.tensor([[20.0, 1e-7, 1e-7, 2e-7, 1e-7, -1.0]])
    B.route_case(l, 2, bias=torch.zeros(6), score=0, groups=groups, top_groups=max(1, groups - 1))


def test_route_a_larger_error_behind_the_next():
    route = lambda l, b: B.route_case(torch.tensor([l]), 1, bias=torch.tensor(b), score=1)  # noqa: E731
    route([-6.906785, -6.906797, 16.55], [0.0, 0.0, -0.998999])
    route([-17.9, -19.5, 1.1547612], [0.010547847, 0.010547847, -0.7498316])


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,k", [(6, 1), (6, 2), (24, 3), (60, 8), (200, 4), (256, 8), (700, 31), (900, 32)])
@pytest.mark.parametrize("t", [0.0, 0.01, -0.3])
def test_route_small_and_large_scores_about_one_value(E, k, score, t):
    """Scores of some 1e-9 under a bias of t, and large ones whose bias brings them to t within their error in fp32 (far more than
    the gaps of the small ones): which are chosen, and in what order, is not told by neighbours."""
    g = B.gen(E + k + int(100 * t))
    T, large = 150, max(2, E // 12)
    rows = torch.empty((T, E))
    rows[:] = torch.rand(E, generator=g) * 3 - 20 - (score == 0) * 2
    few = torch.randperm(E, generator=g)[:large]
    rows[:, few] = torch.rand(large, generator=g) * 2.5 - 0.5
    rows += (torch.rand((T, E), generator=g) < 0.3) * torch.randint(-2, 3, (T, E), generator=g) * 2.0 ** -23   # some ulps here and there
    x = rows[0].double()
    s = torch.softmax(x, 0) if score == 0 else torch.sigmoid(x)
    bias = torch.full((E,), t)
    bias[few] = (t - s[few] + (torch.rand(large, generator=g).double() - 0.5) * 2e-7).float()
    B.route_case(rows, k, bias=bias, score=score)
    if E % 4 == 0 and E // 2 >= k:
        B.route_case(rows, k, bias=bias, score=score, groups=4, top_groups=2, group_best=2)


# ------------------------------------------------------------------------------------- run to run


@pytest.mark.parametrize("bits", [4, 6])
@pytest.mark.parametrize("E,k,T", [(2, 2, 200), (2, 2, 2000), (5, 2, 33), (40, 8, 700)])
def test_experts_repeat_bit_for_bit(E, k, T, bits):
    """Several items of an expert, whose products are cut between CTAs at different steps: no sum goes by which warp or CTA
    comes first."""
    m = B.Experts(E, 2048, 640 if E < 40 else 256, bits)
    g = B.gen(T)
    ids, w = B.chosen(g, T, E, k)
    x, ids, w, ws = torch.randn((T, 2048), generator=g).to(BF).to(DEV), ids.to(DEV), w.to(DEV), m.ws(T, k)
    ys = torch.empty((60, T, 2048), dtype=BF, device=DEV)
    for y in ys:
        m.call(x, ids, w, y, ws)
    assert all(torch.equal(y, ys[0]) for y in ys) and woq.woq_read_status(ws) == 0


@pytest.mark.parametrize("T,k", [(1, 1), (1, 32), (3, 11), (9, 29), (255, 1), (256, 1), (8, 32), (257, 1), (600, 7), (1024, 32)])
def test_experts_places_of_any_number(T, k):
    """Runs of places of a warp, and items, that end anywhere; places without an expert among them, or all of one expert."""
    m = B.Experts(7, 128, 128)
    g = B.gen(T * k)
    w = torch.randn((T, k), generator=g)
    x = torch.randn((T, 128), generator=g).to(BF)
    keep = torch.randperm(T, generator=g)[:40]
    for ids in (torch.randint(-1, 7, (T, k), generator=g).int(), torch.full((T, k), 6, dtype=torch.int32), torch.where(torch.rand((T, k), generator=g) < 0.9, -1, 5).int()):
        y, status = m.run(x, ids, w)
        want, bound = B.M.experts(x[keep], ids[keep], w[keep], m.gu, m.d)
        B.M.close(y[keep], want, bound, B.M.B)
        assert status == 0 and (y[(ids < 0).all(1)] == 0).all()


# ------------------------------------------------------------------------------ a wait that ran out


@pytest.mark.parametrize("bits", [4, 6])
@pytest.mark.parametrize("T", [1, 6])
def test_experts_calls_directly_behind_one_that_gave_up(T, bits):
    """CTAs with a few steps have issued all their copies before a wait runs out: they end with none under way, and the calls
    behind them on another workspace, which take their place on the SMs, are right."""
    m = B.Experts(8, 512, 384, bits)
    g = B.gen(14)
    ids, w = B.chosen(g, T, 8, 2)
    x = torch.randn((T, 512), generator=g).to(BF)
    want, _ = m.run(x, ids, w)
    x, ids, w, ws, other = x.to(DEV), ids.to(DEV), w.to(DEV), m.ws(T, 2), m.ws(T, 2)
    y = torch.full((T, 512), 7.0, dtype=BF, device=DEV)
    for cta in range(4):
        woq.woq_tune_fault(1, cta, 5000)
        try:
            m.call(x, ids, w, y, ws)
        finally:
            woq.woq_tune_fault(0, 0, 0)
        behind = [torch.zeros((T, 512), dtype=BF, device=DEV) for _ in range(3)]
        for z in behind:
            m.call(x, ids, w, z, other)
        assert all(torch.equal(z.cpu(), want) for z in behind) and woq.woq_read_status(other) == 0
        assert woq.woq_read_status(ws, clear=True) & woq.WOQ_DEVERR_TIMEOUT
        woq.woq_workspace_init(ws)
    assert (y == 7.0).all()


@pytest.mark.parametrize("T", [1, 40])
def test_experts_every_call_that_writes_nothing_says_so(T):
    """Behind a wait that ran out, and a status that was read and cleared: y is not written, and the status says it each time."""
    m = B.Experts(8, 512, 384)
    g = B.gen(16)
    ids, w = B.chosen(g, T, 8, 2)
    args = torch.randn((T, 512), generator=g).to(BF).to(DEV), ids.to(DEV), w.to(DEV)
    ws, y = m.ws(T, 2), torch.full((T, 512), 7.0, dtype=BF, device=DEV)
    woq.woq_tune_fault(1, 0, 5000)
    try:
        m.call(*args, y, ws)
    finally:
        woq.woq_tune_fault(0, 0, 0)
    for _ in range(3):
        assert (y == 7.0).all() and woq.woq_read_status(ws, clear=True) == woq.WOQ_DEVERR_TIMEOUT
        m.call(*args, y, ws)
    woq.woq_workspace_init(ws)
    m.call(*args, y, ws)
    assert torch.equal(y.cpu(), m.run(*(t.cpu() for t in args))[0]) and woq.woq_read_status(ws) == 0


# ------------------------------------------------------------------------------------ largest calls


def sampled(m, T, k, g, rows, **kw):
    """A call of T rows, some of them against their definition."""
    ids, w = B.chosen(g, T, m.E, k)
    x = torch.randn((T, m.H), generator=g).to(BF)
    y, status = m.run(x, ids, w)
    keep = torch.randperm(T, generator=g)[:rows]
    want, bound = B.M.experts(x[keep], ids[keep], w[keep], m.gu, m.d)
    B.M.close(y[keep], want, bound, B.M.B)
    assert status == 0


@pytest.mark.parametrize("bits", [4, 6])
@pytest.mark.parametrize("E,T,k", [(1024, 4096, 8), (1024, 2048, 16), (1, 32768, 1), (300, 1, 32)])
def test_experts_most_places(E, T, k, bits):
    sampled(B.Experts(E, 128, 128, bits), T, k, B.gen(E + T), 40)


@pytest.mark.parametrize("bits", [4, 6])
@pytest.mark.parametrize("H,I", [(32768, 128), (128, 32768)])
def test_experts_widest(H, I, bits):
    m = B.Experts(2, H, I, bits, scale=0.002)
    for T in (1, 19):
        sampled(m, T, 2, B.gen(T), 4)


def test_norm_and_route_of_more_rows_than_a_grid_dimension_takes_in_y():
    """70,000 rows and more: rows lie along x."""
    T = 140000
    g = B.gen(9)
    l = torch.randn((T, 8), generator=g)
    B.route_case(l, 2)
    B.norm_case(T, 8, F32, BF)


@pytest.mark.parametrize("bits", [4, 6])
@pytest.mark.parametrize("scale", [1e-38, 1e-20, 1e12])
def test_experts_of_very_small_and_large_rows(scale, bits):
    """As far as gate times up is within fp32's range (and x among bf16's smallest)."""
    m = B.Experts(2, 256, 128, bits, scale=0.1)
    g = B.gen(4)
    ids, w = B.chosen(g, 9, 2, 1)
    m.check((torch.randn((9, 256), generator=g) * scale).to(BF), ids, w)
