"""The 8-bit cache's C ABI on the host: sizes, and every refusal that is decided before a launch (no GPU is
touched: the addresses are never dereferenced)."""
import ctypes

import pytest

P = ctypes.c_void_p
FAKE = 0x10000
BIG = 1 << 40


@pytest.fixture(scope="module")
def woq():
    import weight_only_quantised_gb300 as w
    return w


def config(woq, **kw):
    return woq.KV8Config(**dict(dict(format=0, layers=2, kv_heads=4, head_dim=128, seqs=3, max_tokens=1000, pages=20), **kw))


def test_sizes(woq):
    c = config(woq)
    page = 2 * 4 * (128 * 128 + 16)
    assert woq.woq_kv8_page_offset(c, 20) == woq.woq_kv8_bytes(c)
    assert woq.woq_kv8_page_offset(c, 3) - woq.woq_kv8_page_offset(c, 0) == 3 * page
    # the bookkeeping and the bf16 tails (72 rows of keys and values) come before the pages
    tails = 2 * 3 * 4 * 2 * 72 * 128 * 2
    assert tails < woq.woq_kv8_page_offset(c, 0) < tails + 32768
    # sizes of a long cache pass 32 bits
    long = config(woq, layers=64, kv_heads=8, max_tokens=1 << 20, pages=1 << 14)
    assert woq.woq_kv8_bytes(long) > 64 * 8 * (128 * 128 + 16) * (1 << 14) > 1 << 32
    assert woq.woq_kv8_page_offset(c, 21) == 0 and woq.woq_kv8_page_offset(c, -1) == 0


@pytest.mark.parametrize("bad", [dict(format=2), dict(format=-1), dict(layers=0), dict(layers=1025), dict(kv_heads=0),
                                 dict(kv_heads=257), dict(head_dim=96), dict(head_dim=0), dict(seqs=0), dict(seqs=1025),
                                 dict(max_tokens=0), dict(max_tokens=(1 << 24) + 1), dict(pages=0), dict(pages=(1 << 24) + 1)])
def test_configs_out_of_range(woq, bad):
    c = config(woq, **bad)
    assert woq.woq_kv8_bytes(c) == 0 and woq.woq_kv8_page_offset(c, 0) == 0
    assert woq.lib.woq_kv8_init(ctypes.byref(c), P(FAKE), BIG, None) == woq.WOQ_ERR_SHAPE
    assert woq.woq_kv8_attention_workspace(c, 1, 1, 4) == 0


def every_call(woq, c, cache=FAKE, size=BIG):
    """Each entry that takes a cache, with arguments that are otherwise in order."""
    L, r, a = woq.lib, ctypes.byref(c), P(FAKE)
    buf = P(cache) if cache else None
    return {
        "init": lambda: L.woq_kv8_init(r, buf, size, None),
        "append_rows": lambda: L.woq_kv8_append_rows(r, buf, size, 0, None, 1, 1, a, 0, 4096, 8, None, a, None),
        "append_prompt": lambda: L.woq_kv8_append_prompt(r, buf, size, 0, 0, 5, a, 0, 4096, 8, None, a, None),
        "accept": lambda: L.woq_kv8_accept(r, buf, size, None, 1, a, None),
        "extend": lambda: L.woq_kv8_extend(r, buf, size, 0, 5, None),
        "attention": lambda: L.woq_kv8_attention(r, buf, size, 0, None, 1, 1, a, 8, None, 1.0, 0, 0, a, a, BIG, None),
        "fork": lambda: L.woq_kv8_fork(r, buf, size, a, a, 1, None),
        "free": lambda: L.woq_kv8_free(r, buf, size, a, 1, None),
        "copy_from": lambda: L.woq_kv8_copy(r, buf, size, r, P(1 << 50), BIG, a, a, 1, None),
        "copy_to": lambda: L.woq_kv8_copy(r, P(1 << 50), BIG, r, buf, size, a, a, 1, None),
        "compact": lambda: L.woq_kv8_compact(r, buf, size, 5, None),
        "read": lambda: L.woq_kv8_read(r, buf, size, 0, 0, 0, 5, a, a, None),
        "state": lambda: L.woq_kv8_state(r, buf, size, None, None, None, None),
    }


def test_every_call_checks_its_cache(woq):
    c = config(woq)
    for name, call in every_call(woq, c, cache=0).items():
        assert call() == woq.WOQ_ERR_NULL, name
    for name, call in every_call(woq, c, cache=FAKE + 8).items():
        assert call() == woq.WOQ_ERR_ALIGN, name
    for name, call in every_call(woq, c, size=woq.woq_kv8_bytes(c) - 1).items():
        assert call() == woq.WOQ_ERR_LAYOUT, name
    for name, call in every_call(woq, config(woq, head_dim=80)).items():
        assert call() == woq.WOQ_ERR_SHAPE, name
    assert woq.lib.woq_kv8_init(None, P(FAKE), BIG, None) == woq.WOQ_ERR_NULL


def test_append_arguments(woq):
    c = config(woq)
    L, r = woq.lib, ctypes.byref(c)
    S, N, A = woq.WOQ_ERR_SHAPE, woq.WOQ_ERR_NULL, woq.WOQ_ERR_ALIGN

    def rows(layer=0, seqs=None, n=1, rows=1, qkv=P(FAKE), dtype=0, stride=2048, hq=8, rope=None, out=P(FAKE)):
        return L.woq_kv8_append_rows(r, P(FAKE), BIG, layer, seqs, n, rows, qkv, dtype, stride, hq, rope, out, None)

    for bad in (dict(layer=2), dict(layer=-1), dict(n=-1), dict(n=1025), dict(rows=0), dict(rows=9), dict(dtype=2),
                dict(stride=2040), dict(stride=2052), dict(hq=-1), dict(hq=9)):
        assert rows(**bad) == S, bad
    assert rows(n=0, qkv=None) == woq.WOQ_OK
    assert rows(qkv=None) == N and rows(out=None) == N
    assert rows(qkv=P(FAKE + 4)) == A and rows(out=P(FAKE + 8)) == A and rows(seqs=P(FAKE + 2)) == A

    def prompt(layer=0, seq=0, tokens=3, **kw):
        return L.woq_kv8_append_prompt(r, P(FAKE), BIG, layer, seq, tokens, P(FAKE), 0, 2048, 8, None, P(FAKE), None)

    for bad in (dict(layer=2), dict(seq=3), dict(seq=-1), dict(tokens=-1), dict(tokens=1001)):
        assert prompt(**bad) == S, bad
    assert prompt(tokens=0) == woq.WOQ_OK

    def rope(table=FAKE, positions=10, rot=128, inter=0, axes=1, pos=FAKE, axis=None):
        arr = None if axis is None else (ctypes.c_uint8 * 64)(*axis)
        s = woq._Rope(table, positions, rot, inter, axes, pos, None if arr is None else ctypes.cast(arr, P))
        return rows(rope=ctypes.byref(s))

    for bad in (dict(rot=2), dict(rot=130), dict(rot=256), dict(rot=6), dict(positions=0), dict(axes=0), dict(axes=5),
                dict(inter=2), dict(axes=2, axis=[0] * 63 + [2])):
        assert rope(**bad) == S, bad
    assert rope(pos=None) == N and rope(table=FAKE + 4) == A and rope(pos=FAKE + 1) == A
    t = L.woq_rope_table
    assert t(1e4, 6, 5, P(FAKE), None) == S and t(1e4, 260, 5, P(FAKE), None) == S and t(0.0, 64, 5, P(FAKE), None) == S
    assert t(float("nan"), 64, 5, P(FAKE), None) == S and t(float("inf"), 64, 5, P(FAKE), None) == S
    assert t(1e4, 64, -1, P(FAKE), None) == S and t(1e4, 64, 0, None, None) == woq.WOQ_OK
    assert t(1e4, 64, 5, None, None) == N and t(1e4, 64, 5, P(FAKE + 4), None) == A


def test_attention_arguments(woq):
    c = config(woq)
    L = woq.lib
    S, N, A = woq.WOQ_ERR_SHAPE, woq.WOQ_ERR_NULL, woq.WOQ_ERR_ALIGN

    def call(cfg=c, layer=0, seqs=None, n=1, rows=1, q=P(FAKE), hq=8, vis=None, scale=1.0, window=0, sinks=0,
             out=P(FAKE), ws=P(FAKE), wsb=BIG):
        return L.woq_kv8_attention(ctypes.byref(cfg), P(FAKE), BIG, layer, seqs, n, rows, q, hq, vis, scale, window, sinks,
                                   out, ws, wsb, None)

    for bad in (dict(layer=2), dict(n=-1), dict(n=1025), dict(rows=0), dict(rows=9), dict(hq=0), dict(hq=6),
                dict(rows=8, hq=4 * 17), dict(scale=float("inf")), dict(scale=float("nan")), dict(window=-1), dict(sinks=-1),
                dict(window=(1 << 30) + 1), dict(sinks=(1 << 30) + 1)):
        assert call(**bad) == S, bad
    assert call(cfg=config(woq, head_dim=256), rows=8, hq=4 * 17) == S
    assert call(n=0, q=None) == woq.WOQ_OK
    assert call(q=None) == N and call(out=None) == N and call(ws=None) == N
    assert call(q=P(FAKE + 2)) == A and call(out=P(FAKE + 8)) == A and call(ws=P(FAKE + 8)) == A and call(vis=P(FAKE + 1)) == A


def test_page_arguments(woq):
    c = config(woq)
    L, r, a = woq.lib, ctypes.byref(c), P(FAKE)
    S, N, A = woq.WOQ_ERR_SHAPE, woq.WOQ_ERR_NULL, woq.WOQ_ERR_ALIGN
    cache = (r, a, BIG)
    for n in (-1, 1025):
        assert L.woq_kv8_fork(*cache, a, a, n, None) == S and L.woq_kv8_free(*cache, a, n, None) == S
        assert L.woq_kv8_accept(*cache, a, n, a, None) == S
    assert L.woq_kv8_fork(*cache, None, a, 1, None) == N and L.woq_kv8_fork(*cache, a, None, 1, None) == N
    assert L.woq_kv8_free(*cache, None, 1, None) == N and L.woq_kv8_accept(*cache, None, 1, None, None) == N
    assert L.woq_kv8_fork(*cache, P(FAKE + 1), a, 1, None) == A and L.woq_kv8_accept(*cache, None, 1, P(FAKE + 2), None) == A
    assert L.woq_kv8_fork(*cache, None, None, 0, None) == woq.WOQ_OK and L.woq_kv8_free(*cache, None, 0, None) == woq.WOQ_OK
    for limit in (0, 21, -5):
        assert L.woq_kv8_compact(*cache, limit, None) == S
    for seq, tokens in ((3, 1), (-1, 1), (0, -1), (0, 1001)):
        assert L.woq_kv8_extend(*cache, seq, tokens, None) == S
    for layer, seq, first, count in ((2, 0, 0, 1), (-2, 0, 0, 1), (0, 3, 0, 1), (0, -1, 0, 1), (0, 0, -1, 1), (0, 0, 0, -1),
                                     (0, 0, 1000, 9), (0, 0, 2 ** 31 - 1, 2 ** 31 - 1)):
        assert L.woq_kv8_read(*cache, layer, seq, first, count, a, a, None) == S
    assert L.woq_kv8_read(*cache, 0, 0, 0, 0, None, None, None) == woq.WOQ_OK
    assert L.woq_kv8_read(*cache, 0, 0, 0, 1, None, a, None) == N and L.woq_kv8_read(*cache, 0, 0, 0, 1, a, P(FAKE + 8), None) == A
    assert L.woq_kv8_state(*cache, P(FAKE + 1), None, None, None) == A


def test_copies_between_caches(woq):
    c = config(woq)
    L, a = woq.lib, P(FAKE)
    size = woq.woq_kv8_bytes(c)

    def copy(other, at):
        return L.woq_kv8_copy(ctypes.byref(c), a, BIG, ctypes.byref(other), P(at), BIG, a, a, 1, None)

    for other in (dict(format=1), dict(layers=1), dict(kv_heads=8), dict(head_dim=64)):
        assert copy(config(woq, **other), 1 << 50) == woq.WOQ_ERR_SHAPE, other
    assert copy(config(woq, pages=21), FAKE) == woq.WOQ_ERR_LAYOUT           # one buffer, two configs
    for at in (FAKE + 16, FAKE + size // 16 * 16 - 16):
        assert copy(c, at) == woq.WOQ_ERR_LAYOUT                             # overlapping buffers


def test_binding_refusals(woq):
    torch = pytest.importorskip("torch")
    c = config(woq)
    cache = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        woq.woq_kv8_init(c, cache)
    with pytest.raises(ValueError, match="2-D"):
        woq.woq_kv8_append_rows(c, cache, 0, None, 1, torch.zeros(8), 8, None)
    with pytest.raises(ValueError, match="the call needs"):
        woq.woq_kv8_append_rows(c, cache, 0, None, 3, torch.zeros((4, 2048)), 8, None)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        woq.woq_kv8_append_prompt(c, cache, 0, 0, torch.zeros((4, 2048), dtype=torch.float16), 8, None)
    with pytest.raises(ValueError, match="neighbouring"):
        woq.woq_kv8_append_prompt(c, cache, 0, 0, torch.zeros((4, 2047)), 8, None)
    with pytest.raises(ValueError, match="entries for"):
        woq.woq_kv8_accept(c, cache, torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="the call needs"):
        woq.woq_kv8_attention(c, cache, 0, None, 2, torch.zeros((3, 8, 128), dtype=torch.bfloat16), 8, None, None, 1.0)
    with pytest.raises(ValueError, match="same multiple"):
        woq.woq_kv8_read(c, cache, 0, 0, 0, torch.zeros((5, 4, 128)), torch.zeros((4, 4, 128)))
