"""Refusals of the cache's Python binding that look at shapes only (no GPU is touched)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def woq():
    import weight_only_quantised_gb300 as w
    return w


def ints(n):
    return torch.zeros(n, dtype=torch.int32)


@pytest.mark.parametrize("shape", [(10, 64, 2), (10, 32), (10, 32, 3), (640,)])
def test_a_rotary_table_of_another_shape(woq, shape):
    """A table for rot_dim 64 has 32 pairs a row: Rope takes rot_dim from the shape."""
    with pytest.raises(ValueError, match="64 / 2"):
        woq.woq_rope_table(1e4, 64, torch.zeros(shape))


def test_a_rotary_table_of_another_type(woq):
    with pytest.raises(ValueError, match="float32"):
        woq.woq_rope_table(1e4, 64, torch.zeros((10, 32, 2), dtype=torch.int32))


@pytest.mark.parametrize("a,b", [(3, 2), (2, 3), (1, 0)])
def test_lists_of_unequal_lengths(woq, a, b):
    cfg = woq.KV8Config(format=0, layers=1, kv_heads=1, head_dim=64, seqs=4, max_tokens=100, pages=4)
    cache = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="entries for"):
        woq.woq_kv8_fork(cfg, cache, ints(a), ints(b))
    with pytest.raises(ValueError, match="entries for"):
        woq.woq_kv8_copy(cfg, cache, cfg, cache, ints(a), ints(b))
