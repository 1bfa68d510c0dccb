"""Sizes and strides that a C int does not hold: the binding refuses them, as their low 32 bits would be taken for a call of
another shape (tensors without memory: what is refused comes before anything is looked at on a device)."""
import pytest

torch = pytest.importorskip("torch")
BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8
BIG = 1 << 32


@pytest.fixture(scope="module")
def woq():
    import weight_only_quantised_gb300 as w
    return w


def t(*shape, dtype=torch.float32, stride=None):
    return torch.empty_strided(shape, (stride, 1), dtype=dtype, device="meta") if stride else torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("rows,width", [(BIG + 2, 8), (1, BIG + 8), (1 << 31, 8)])
def test_norm(woq, rows, width):
    with pytest.raises(ValueError, match="u: sizes up to"):
        woq.woq_block_norm(t(rows, width), t(rows, width), t(rows, width), None)


@pytest.mark.parametrize("stride", [BIG + 64, 1 << 31])
def test_route(woq, stride):
    with pytest.raises(ValueError, match="logits: row strides up to"):
        woq.woq_route(t(2, 64, stride=stride), 2, t(2, 2, dtype=I32), t(2, 2))
    with pytest.raises(ValueError, match="logits: sizes up to"):
        woq.woq_route(t(stride, 64), 2, t(stride, 2, dtype=I32), t(stride, 2))


@pytest.mark.parametrize("rows,k,inner", [(BIG + 1, 1, 128), (2, BIG + 1, 128), (2, 1, BIG + 128), (2, 1, 128 - BIG)])
def test_experts(woq, rows, k, inner):
    with pytest.raises(ValueError, match="sizes up to"):
        woq.woq_experts_swiglu(4, 2, t(9, dtype=U8), t(9, dtype=U8), t(rows, 128, dtype=BF), t(rows, k, dtype=I32), t(rows, k), inner,
                               t(rows, 128, dtype=BF), t(9, dtype=U8))


def test_linears_and_the_cache(woq):
    with pytest.raises(ValueError, match="x_bf16: sizes up to"):
        woq.woq_act_quant_int8(t(1, BIG + 128, dtype=BF), t(1, BIG + 128, dtype=torch.int8), t(1))
    cfg = woq.KV8Config(head_dim=128, kv_heads=1, layers=1, pages=4, seqs=2, max_tokens=256)
    with pytest.raises(ValueError, match="qkv: row strides up to"):
        woq.woq_kv8_append_rows(cfg, t(9, dtype=U8), 0, None, 1, t(2, 512, dtype=BF, stride=BIG + 512), 2, t(2, 256, dtype=BF))
