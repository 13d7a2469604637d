"""The operators together, as a decoder uses them around the adapted layer: a
training step (norm, layer with dropout, residual join with dropout, norm, and all
of their gradients) against float64 autograd, and a decode chain (norm to 8 bits,
matrix-vector product) against float64."""

import numpy as np
import pytest
import torch

import quantized_rank_fine_b200 as q
from oracle import intq, norm
from tests.helpers import layer_on_gpu, oracle_weight, require_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _rms(h, g):
    return h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * g


def test_training_block():
    """h0 -> norm -> adapted layer (adapter dropout) -> dropout + residual -> norm.
    Every stored tensor is bf16, so each gradient is within a few half steps
    (2^-8 each, seven roundings on the longest path) of float64 autograd."""
    M, n, r, p = 192, 512, 16, 0.1
    t, w = layer_on_gpu(n, n, M, r, tag="block")
    gen = torch.Generator(device="cuda").manual_seed(0)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")
    h0, g1, g2 = rn(M, n).to(BF), (1 + 0.2 * rn(n)).to(BF), 1 + 0.2 * rn(n)
    dy, dh = rn(M, n).to(BF), rn(M, n).to(BF)
    da, dr = q.Dropout(p, 1, 3), q.Dropout(p, 2, 3)
    ws = q.Workspace()

    n1 = q.qlora_rmsnorm_fwd(h0, g1, EPS, save_rstd=True)
    Y, V = q.qlora_linear_fwd(w, n1.Y, t["A"], t["B"], ws, adapter_scale=2.0, dropout=da)
    n2 = q.qlora_rmsnorm_fwd(Y, g2, EPS, residual=h0, dropout=dr, save_rstd=True)
    dY, dres, dg2 = q.qlora_rmsnorm_bwd(dy, n2.H, g2, n2.rstd, ws, dH=dh, dropout=dr)
    dX, dA, dB = q.qlora_linear_bwd(w, n1.Y, V, dY, t["A"], t["B"], ws, adapter_scale=2.0, dropout=da)
    _, dh0, dg1 = q.qlora_rmsnorm_bwd(dX, h0, g1, n1.rstd, ws, dH=dres)
    assert ws.status() == 0

    Wq = torch.from_numpy(np.asarray(oracle_weight(w))).double().cuda()
    ka = torch.from_numpy(norm.keep_mask(p, 1, 3, M, r)).cuda().double() * norm.keep_scale(p)
    kr = torch.from_numpy(norm.keep_mask(p, 2, 3, M, n)).cuda().double() * norm.keep_scale(p)
    leaf = {k: v.double().requires_grad_() for k, v in dict(h0=h0, g1=g1, g2=g2, A=t["A"], B=t["B"]).items()}
    x1 = _rms(leaf["h0"], leaf["g1"])
    y = x1 @ Wq + (2.0 * ka * (x1 @ leaf["A"])) @ leaf["B"]
    h1 = leaf["h0"] + kr * y
    out = _rms(h1, leaf["g2"])
    ((out * dy.double()).sum() + (h1 * dh.double()).sum()).backward()
    for name, got, want in (("Y2", n2.Y, out), ("H", n2.H, h1), ("dh0", dh0, leaf["h0"].grad), ("dg1", dg1, leaf["g1"].grad),
                            ("dg2", dg2, leaf["g2"].grad), ("dA", dA, leaf["A"].grad), ("dB", dB, leaf["B"].grad)):
        rel = ((got.double() - want).norm() / want.norm()).item()
        assert rel <= 7 * 2.0 ** -8, f"{name}: {rel:.2e}"


@pytest.mark.parametrize("M", [1, 4, 16])
@pytest.mark.parametrize("block", [0, 64])
def test_decode_chain(M, block):
    """Norm to 8 bits -> up projection -> norm with the residual -> next projection,
    each stage against float64 on the stage's own inputs (an 8-bit stage's error is
    the codes' and belongs to the codes, which are read back)."""
    n, r = 512, 8
    gen = torch.Generator(device="cuda").manual_seed(M)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")
    h, g = rn(M, n).to(BF), (1 + 0.2 * rn(n)).to(BF)
    A, B = (rn(n, r) / n ** 0.5).to(BF), (rn(r, n) * 0.05).to(BF)
    codes, scales = q.qlora_quantize_int(rn(n, n) * 0.04, 4)
    w = q.int_weight(codes, scales, n, n)
    w64 = torch.from_numpy(intq.dequantize_int(codes.cpu().numpy(), scales.cpu().numpy(), n, n)).cuda().double()
    ws = q.Workspace()
    branch = torch.zeros_like(h)
    for _ in range(3):
        o = q.qlora_rmsnorm_fwd(branch, g, EPS, residual=h, want_y=False, quant_block=block)
        y, _ = q.qlora_matvec(w, o.act, ws, A, B)
        h64 = h.double() + branch.double()
        assert torch.equal(o.H, h64.float().to(BF))
        x64 = (o.act.codes.view(torch.float8_e4m3fn).double().view(M, -1, block or n) * o.act.scales.double()[:, :, None]).view(M, n)
        y64 = _rms(o.H.double(), g.double())
        assert (x64 - y64).norm() <= 2.0 ** -4 * y64.norm()
        want = x64 @ w64 + (x64 @ A.double()) @ B.double()
        assert (y.double() - want).norm() <= 2.0 ** -7.5 * want.norm()
        h, branch = o.H, y
    assert ws.status() == 0
