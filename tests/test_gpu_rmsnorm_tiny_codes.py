"""Codes of blocks whose scale lies near the smallest normal numbers, bit for bit the
definition's E4M3(fl32(y / s)): rests of the quotients underflow there.

Rows of +-1 with eps = 3 have rstd = 1 / 2, so y = g / 2 is exact.  The gain puts one
value that sets the scale and 63 next to ties of the code into every block."""

import numpy as np
import pytest
import torch

import quantized_rank_fine_b200 as q
from oracle import norm
from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

LEVELS = [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:127]     # up to 448
TIES = np.array([(a + b) / 2 for a, b in zip(LEVELS, LEVELS[1:])])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def blocks(exponent, width, n, seed):
    """n values of y in fp32: per block of `width` one maximum for a scale of 2^exponent to
    2^(exponent + 1), the others within three steps of a tie times the scale."""
    rng = np.random.default_rng(seed)
    top = (448 * 2.0 ** exponent * (1 + rng.random(n // width))).astype(np.float32)
    s = (top.astype(np.float64) / 448).astype(np.float32)
    y = (rng.choice(TIES, (n // width, width)) * s.astype(np.float64)[:, None]).astype(np.float32)
    for _ in range(3):
        to = rng.integers(-1, 2, y.shape)
        y = np.where(to > 0, np.nextafter(y, np.float32(1)), np.where(to < 0, np.nextafter(y, np.float32(0)), y))
    y = np.minimum(y, top[:, None])
    y[:, 0] = top
    return y.reshape(-1)


@pytest.mark.parametrize("exponent", [-126, -122, -118, -114, -100, -70, -62, -60, -58, -40])
@pytest.mark.parametrize("block", [0, 64])
def test_codes(exponent, block):
    for n, M in ((65536, 2), (4096, 3), (4096, 700)):      # eight, one and two vectors a thread
        y = blocks(exponent, block or n, n, 200 + exponent)
        x = np.where(np.arange(n) % 3 == 0, -1.0, 1.0)
        xt = torch.from_numpy(np.tile(x, (M, 1))).to(BF).cuda()
        g = torch.from_numpy(2.0 * y.astype(np.float64)).float().cuda()
        o = q.qlora_rmsnorm_fwd(xt, g, 3.0, want_y=False, quant_block=block)
        v, s = norm.quantize_e4m3((x * y.astype(np.float64))[None], block)
        got = o.act.codes.view(torch.float8_e4m3fn).double().cpu().numpy()
        assert np.array_equal(o.act.scales.double().cpu().numpy(), np.repeat(s, M, axis=0))
        assert np.array_equal(got, np.repeat(v, M, axis=0)), f"{int((got[0] != v[0]).sum())} codes of {n}"
