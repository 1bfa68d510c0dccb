"""The block's C ABI and binding on the host: sizes, and every refusal that is decided before a launch (no GPU is touched:
the addresses are never dereferenced)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

P = ctypes.c_void_p
A = 0x10000
BIG = 1 << 40


@pytest.fixture(scope="module")
def woq():
    import weight_only_quantised_gb300 as w
    return w


def norm(woq, **kw):
    a = dict(u=A, ut=0, r=A, ro=A, rt=0, out=A, T=2, D=128, post=A, gate=A, rows=1, pre=A, alpha=1.0, beta=1.0, offset=0.0, eps=1e-6)
    a.update(kw)
    return woq.lib.woq_block_norm(P(a["u"]), a["ut"], P(a["r"]), P(a["ro"]), a["rt"], P(a["out"]), a["T"], a["D"], P(a["post"]), P(a["gate"]),
                                  a["rows"], P(a["pre"]), a["alpha"], a["beta"], a["offset"], a["eps"], None)


@pytest.mark.parametrize("kw", [dict(ut=2), dict(ut=-1), dict(rt=2), dict(T=-1), dict(D=0), dict(D=12), dict(D=16392), dict(rows=0), dict(rows=3),
                                dict(rows=-1), dict(eps=-1e-9), dict(eps=float("nan")), dict(alpha=float("inf")), dict(beta=float("nan")),
                                dict(offset=float("inf"))])
def test_norm_arguments_out_of_range(woq, kw):
    assert norm(woq, **kw) == woq.WOQ_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(u=None), dict(r=None), dict(ro=None), dict(pre=None)])
def test_norm_null(woq, kw):
    assert norm(woq, **kw) == woq.WOQ_ERR_NULL


@pytest.mark.parametrize("name", ["u", "r", "ro", "out", "post", "gate", "pre"])
def test_norm_alignment(woq, name):
    assert norm(woq, **{name: A + 8}) == woq.WOQ_ERR_ALIGN


def test_norm_of_no_rows(woq):
    assert norm(woq, T=0, u=None, r=None, ro=None, out=None) == woq.WOQ_OK


def route(woq, cfg=None, **kw):
    c = dict(score=0, experts=64, k=4, groups=1, top_groups=1, group_best=1, renormalise=1, scale=1.0)
    c.update(cfg or {})
    a = dict(logits=A, dtype=0, stride=64, T=2, bias=None, live=None, ids=A, weights=A)
    a.update(kw)
    r = woq._Router(*[c[n] for n, _ in woq._Router._fields_])
    return woq.lib.woq_route(ctypes.byref(r), P(a["logits"]), a["dtype"], a["stride"], a["T"], P(a["bias"]), P(a["live"]), P(a["ids"]), P(a["weights"]), None)


@pytest.mark.parametrize("cfg", [dict(score=2), dict(score=-1), dict(experts=0), dict(experts=1025), dict(k=0), dict(k=33), dict(experts=3), dict(groups=0),
                                 dict(groups=5), dict(groups=64), dict(groups=8, top_groups=9), dict(top_groups=0), dict(top_groups=2), dict(group_best=3),
                                 dict(group_best=0), dict(experts=32, groups=32, group_best=2, top_groups=32), dict(groups=32, top_groups=1),
                                 dict(renormalise=2), dict(scale=float("nan")), dict(scale=float("inf"))])
def test_routers_out_of_range(woq, cfg):
    assert route(woq, cfg) == woq.WOQ_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(T=-1), dict(stride=63)])
def test_route_arguments_out_of_range(woq, kw):
    assert route(woq, **kw) == woq.WOQ_ERR_SHAPE


def test_route_pointers(woq):
    for name in ("logits", "ids", "weights"):
        assert route(woq, **{name: None}) == woq.WOQ_ERR_NULL
    assert route(woq, logits=A + 8) == woq.WOQ_ERR_ALIGN
    for name in ("ids", "weights", "bias", "live"):
        assert route(woq, **{name: A + 2}) == woq.WOQ_ERR_ALIGN
    assert woq.lib.woq_route(None, P(A), 0, 64, 2, None, None, P(A), P(A), None) == woq.WOQ_ERR_NULL
    assert route(woq, T=0, logits=None, ids=None, weights=None) == woq.WOQ_OK


def experts(woq, **kw):
    a = dict(bits=4, E=8, gu=A, gub=BIG, down=A, db=BIG, x=A, ids=A, w=A, T=2, k=2, H=256, I=128, y=A, ws=A, wsb=BIG)
    a.update(kw)
    return woq.lib.woq_experts_swiglu(a["bits"], a["E"], P(a["gu"]), a["gub"], P(a["down"]), a["db"], P(a["x"]), P(a["ids"]), P(a["w"]), a["T"], a["k"],
                                      a["H"], a["I"], P(a["y"]), P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("kw", [dict(bits=5), dict(bits=8), dict(E=0), dict(E=1025), dict(T=-1), dict(k=0), dict(k=33), dict(H=64), dict(H=200), dict(H=0),
                                dict(H=32896), dict(I=0), dict(I=130), dict(I=32896), dict(T=16385)])
def test_expert_arguments_out_of_range(woq, kw):
    assert experts(woq, **kw) == woq.WOQ_ERR_SHAPE


def test_expert_pointers_and_sizes(woq):
    for name in ("gu", "down", "x", "ids", "w", "y", "ws"):
        assert experts(woq, **{name: None}) == woq.WOQ_ERR_NULL
    for name in ("gu", "down", "x", "y", "ws"):
        assert experts(woq, **{name: A + 8}) == woq.WOQ_ERR_ALIGN
    for name in ("ids", "w"):
        assert experts(woq, **{name: A + 2}) == woq.WOQ_ERR_ALIGN
    gu, d = woq.woq_experts_bytes(4, 8, 256, 256), woq.woq_experts_bytes(4, 8, 256, 128)
    assert gu == 8 * woq.woq_packed_bytes(4, 256, 256) and d == 8 * woq.woq_packed_bytes(4, 256, 128)
    assert experts(woq, gub=gu - 1) == woq.WOQ_ERR_LAYOUT
    assert experts(woq, db=d - 1) == woq.WOQ_ERR_LAYOUT
    assert experts(woq, wsb=woq.woq_experts_workspace(8, 2, 2, 256, 128) - 1) == woq.WOQ_ERR_WORKSPACE
    assert experts(woq, T=0, gu=None, down=None, x=None, ids=None, w=None, y=None, ws=None) == woq.WOQ_OK


def test_expert_sizes(woq):
    assert woq.woq_experts_bytes(4, 0, 256, 256) == 0 and woq.woq_experts_bytes(4, 8, 256, 100) == 0 and woq.woq_experts_bytes(5, 8, 256, 256) == 0
    assert woq.woq_experts_bytes(6, 1024, 32768, 32768) == 1024 * woq.woq_packed_bytes(6, 32768, 32768) > 1 << 32
    # h and the parts of each place
    assert woq.woq_experts_workspace(128, 500, 8, 2048, 768) >= 4000 * (768 * 2 + 2048 * 4)
    assert woq.woq_experts_workspace(8, 16385, 2, 128, 128) == 0 and woq.woq_experts_workspace(8, 1, 1, 130, 128) == 0


def cpu(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_the_binding_looks_at_shapes_and_types(woq):
    bf, i32 = torch.bfloat16, torch.int32
    with pytest.raises(ValueError, match="CUDA"):
        woq.woq_block_norm(cpu(2, 64), cpu(2, 64), cpu(2, 64), None)
    with pytest.raises(ValueError, match="u: expected bfloat16 or float32"):
        woq.woq_block_norm(cpu(2, 64, dtype=torch.float16), cpu(2, 64), cpu(2, 64), None)
    with pytest.raises(ValueError, match="r_out"):
        woq.woq_block_norm(cpu(2, 64), cpu(2, 64), cpu(2, 64, dtype=bf), None)
    with pytest.raises(ValueError, match="gate"):
        woq.woq_block_norm(cpu(5, 64), cpu(5, 64), cpu(5, 64), None, gate=cpu(2, 64, dtype=bf))
    with pytest.raises(ValueError, match="gate"):
        woq.woq_block_norm(cpu(4, 64), cpu(4, 64), cpu(4, 64), None, gate=cpu(2, 32, dtype=bf))
    with pytest.raises(ValueError, match="logits"):
        woq.woq_route(cpu(4, 64, dtype=torch.float64), 2, cpu(4, 2, dtype=i32), cpu(4, 2))
    with pytest.raises(ValueError, match="logits"):
        woq.woq_route(cpu(64, 4).t(), 2, cpu(4, 2, dtype=i32), cpu(4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        woq.woq_route(cpu(4, 64), 2, cpu(4, 2, dtype=i32), cpu(4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        woq.woq_experts_swiglu(4, 2, cpu(9, dtype=torch.uint8), cpu(9, dtype=torch.uint8), cpu(1, 128, dtype=bf), cpu(1, 1, dtype=i32), cpu(1, 1), 128,
                               cpu(1, 128, dtype=bf), cpu(9, dtype=torch.uint8))
