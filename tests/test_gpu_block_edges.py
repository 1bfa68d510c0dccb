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
