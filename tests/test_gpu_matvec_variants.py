"""The matrix-vector product's variants on weights of more than 2^21 numbers: both tile
widths, with a last tile cut short and a last stage of half its rows, one or two token
tiles, every class of adapter rank, and the three kinds of x.  Tolerances are those of
test_gpu_matvec_precision."""

import pytest
import torch

import quantized_rank_fine_b200 as q
from tests.helpers import assert_guards, guarded, require_gpu
from tests.test_gpu_matvec_precision import check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# A cluster shares the stages of a column tile; the plan weighs how many clusters fit.
# On a B200: 256 columns with one stage and with two a CTA (last tiles of 64, 128 and
# 192 columns), 256 with eight or more, 128 with three to eight, and 128 or 256 by
# the rank, so that rings of every depth are refilled.
SIZES = [(576, 7232), (1088, 7296), (1088, 7360), (4160, 7360), (4160, 2112), (8256, 3776)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(scope="module")
def weights():
    """(weight, its values in float64, adapters of 256 columns) of a size, the last one kept."""
    kept = {}

    def get(K, N):
        if (K, N) not in kept:
            kept.clear()
            gen = torch.Generator(device="cuda").manual_seed(K + N)
            codes = torch.randint(0, 256, (K * N // 2,), generator=gen, device="cuda", dtype=torch.uint8)
            s = torch.exp(torch.randn((K, N // 16), generator=gen, device="cuda")) * 0.01
            v = torch.stack((codes & 15, codes >> 4), 1).view(K, N).double() - 8
            w64 = v * s.double().repeat_interleave(16, dim=1)
            A = (torch.randn((K, 256), generator=gen, device="cuda") / K ** 0.5).to(BF)
            B = (torch.randn((256, N), generator=gen, device="cuda") * 0.05).to(BF)
            kept[K, N] = q.int_weight(codes, s.view(-1), K, N), w64, A, B
        return kept[K, N]

    yield get
    kept.clear()
    torch.cuda.empty_cache()


def _x(M, K, x8, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, K), generator=gen, device="cuda")
    if x8 is None:
        X = x.to(BF)
        return X, X.double()
    b = (x * torch.exp(torch.randn(K, generator=gen, device="cuda"))).view(M, -1, x8 or K)
    s = b.abs().amax(2) / 448
    c = (b / s[:, :, None]).to(torch.float8_e4m3fn)
    return q.Act8(c.view(M, K).view(torch.uint8), s, x8), (c.double() * s.double()[:, :, None]).view(M, K)


@pytest.mark.parametrize("K,N", SIZES)
@pytest.mark.parametrize("M", [1, 8, 9, 16])
@pytest.mark.parametrize("x8", [None, 0, 64])
def test_every_rank_class(weights, K, N, M, x8):
    w, w64, A, B = weights(K, N)
    X, x64 = _x(M, K, x8, M)
    ws = q.Workspace()
    for r in (0, 8, 64, 72, 136, 256):
        a, b = (A[:, :r].contiguous(), B[:r].contiguous()) if r else (None, None)
        bufy, Y = guarded((M, N), BF)
        bufv, V = guarded((M, max(r, 8)), BF)
        _, v = q.qlora_matvec(w, X, ws, a, b, adapter_scale=2.0, save_V=True, Y=Y, V=V if r else None)
        assert_guards([bufy, bufv], f"matvec, rank {r}")
        assert ws.status() == 0
        check(Y, v, x64, a, b, w64, 2.0)
        assert torch.equal(q.qlora_matvec(w, X, ws, a, b, adapter_scale=2.0)[0], Y)
