"""The attention's launch shape, and its ring of stages, on the CPU.

A copy's end and a stage's release are barriers that a waiter asks for by the parity of a phase; asked two
phases ahead, a barrier answers at once.  The model below runs a CTA's ring with copies that end in any order
and warps of any speed, answers every wait as the hardware does, and reports a wait that was answered too early."""
import random

import pytest

SMEM, SMS = 232448, 152


@pytest.fixture(scope="module")
def woq():
    import weight_only_quantised_gb300 as w
    return w


def plan(woq, dim, rows, group, n=1, heads=2, smem=SMEM):
    c = woq.KV8Config(format=0, layers=1, kv_heads=heads, head_dim=dim, seqs=max(n, 1), max_tokens=1000, pages=20)
    return woq.woq_kv8_plan_attention(c, n, rows, heads * group, SMS, smem)


SHAPES = [(dim, rows, group) for dim in (64, 128, 256) for rows in range(1, 9) for group in (1, 2, 3, 4, 5, 6, 7, 8, 16)
          if rows * group <= 128]


@pytest.mark.parametrize("n", [1, 8, 1024])
def test_every_shape_has_a_plan_that_fits(woq, n):
    for dim, rows, group in SHAPES:
        p = plan(woq, dim, rows, group, n)
        per = p["warps"] // p["query_groups"]
        assert p["query_groups"] == (4 if rows * group > 8 or dim == 256 else 1)  # teams of four warps
        assert p["warps"] == per * p["query_groups"] and 1 <= p["warps"] <= 12
        assert p["stages"] % per == 0 and 2 * per <= p["stages"] <= 32, (dim, rows, group, p)
        assert p["stages"] * (128 * dim + 16) < p["smem_bytes"] <= SMEM
        assert p["ctas"] == SMS


def test_refusals(woq):
    for args in ((128, 8, 17), (256, 8, 17), (128, 0, 4), (128, 9, 1)):
        with pytest.raises(woq.WoqError, match="M, N, K"):
            plan(woq, *args)
    with pytest.raises(woq.WoqError):
        plan(woq, 128, 1, 4, smem=30000)  # not two stages
    assert woq.lib.woq_kv8_plan_attention(None, 1, 1, 1, 1, 1, None) == woq.WOQ_ERR_NULL


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passes(self, parity):  # the last phase that ended has this parity
        return (self.phase - 1) & 1 == parity


def ring_is_sound(stages, per, groups, blocks, rng):
    full = [Barrier(1) for _ in range(stages)]
    empty = [Barrier(groups) for _ in range(stages)]
    issued, flying = 0, []
    nxt = {(g, s): s for g in range(groups) for s in range(per)}
    idle = 0
    while any(b < blocks for b in nxt.values()):
        idle += 1
        if idle > 10000:
            return False  # stuck
        what = rng.random()
        if what < 0.3 and issued < blocks:
            st = issued % stages
            if issued < stages or empty[st].passes((issued // stages - 1) & 1):
                flying.append(issued)
                issued += 1
                idle = 0
        elif what < 0.6 and flying:
            b = flying.pop(rng.randrange(len(flying)) if rng.random() < 0.5 else -1)
            full[b % stages].arrive()
            idle = 0
        else:
            key = rng.choice([k for k, b in nxt.items() if b < blocks])
            b = nxt[key]
            if full[b % stages].passes((b // stages) & 1):
                if full[b % stages].phase != b // stages + 1:
                    return False  # answered too early: the copy of an earlier block is still under way
                empty[b % stages].arrive()
                nxt[key] = b + per
                idle = 0
    return True


def test_the_ring_never_answers_early(woq):
    shapes = {(p["stages"], p["warps"] // p["query_groups"], p["query_groups"])
              for p in (plan(woq, *s) for s in SHAPES)}
    rng = random.Random(5)
    for s in sorted(shapes):
        for _ in range(10):
            assert ring_is_sound(*s, blocks=6 * s[0], rng=rng), s
    # the model sees the mistake: stages that are no multiple of the warps
    assert not all(ring_is_sound(12, 8, 1, 100, rng) for _ in range(10))
