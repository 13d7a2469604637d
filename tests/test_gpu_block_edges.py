"""Calls around the layer that the documentation allows and everyday use brings:
in-place residual streams, calls of one workspace that outgrow it under a captured
graph, mixed chains of the library's dependent launches, kernel timers."""

import numpy as np
import pytest
import torch

import quantized_rank_fine_b200 as q
from oracle import norm
from tests.helpers import layer_on_gpu, require_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _rn(*s, seed=0):
    return torch.randn(s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("M,n", [(5, 64), (700, 1032), (40, 4096), (6, 11008), (3, 32768)])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_residual_stream_in_place(M, n, p):
    x, res, g, dy, dH = _rn(M, n, seed=1).to(BF), _rn(M, n, seed=2).to(BF), _rn(n, seed=3), _rn(M, n, seed=4).to(BF), _rn(M, n, seed=5).to(BF)
    d = q.Dropout(p, 1, 1) if p else None
    ws = q.Workspace()
    a = q.qlora_rmsnorm_fwd(x, g, 1e-5, res, d, save_rstd=True)
    h = res.clone()
    b = q.qlora_rmsnorm_fwd(x, g, 1e-5, h, d, save_rstd=True, H=h)
    assert b.H is h and torch.equal(a.H, h) and torch.equal(a.Y, b.Y)
    want = q.qlora_rmsnorm_bwd(dy, h, g, a.rstd, ws, dH, d)
    buf = dH.clone()
    got = q.qlora_rmsnorm_bwd(dy, h, g, a.rstd, ws, buf, d, dR=buf)
    assert all(torch.equal(u, v) for u, v in zip(got, want)) and got[1] is buf
    buf = dy.clone()
    got = q.qlora_rmsnorm_bwd(buf, h, g, a.rstd, ws, dH, d, dR=buf)
    assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_probability_that_is_zero_in_fp32():
    x, g = _rn(4, 64).to(BF), torch.ones(64, device="cuda")
    d = q.Dropout(1e-60, 1, 1)
    o = q.qlora_rmsnorm_fwd(x, g, 1e-5, dropout=d, save_rstd=True)
    assert o.H is None
    dX, dR, _ = q.qlora_rmsnorm_bwd(x, x, g, o.rstd, q.Workspace(), dropout=d)
    assert dX is dR


def test_probability_close_to_one():
    """The largest fp32 below 1: almost everything is dropped, kept values times 2^24."""
    p = 1.0 - 2.0 ** -24
    x = torch.ones((64, 4096), dtype=BF, device="cuda")
    m = q.qlora_dropout_mask(64, 4096, q.Dropout(p, 5, 5))
    o = q.qlora_rmsnorm_fwd(x, torch.ones(4096, device="cuda"), 1.0, torch.zeros_like(x), q.Dropout(p, 5, 5))
    assert torch.equal(o.H != 0, m.bool()) and int(m.sum()) <= 3
    assert torch.equal(o.H[m.bool()].float(), torch.full((int(m.sum()),), 2.0 ** 24, device="cuda"))


def test_workspace_outgrown_under_a_captured_graph():
    """A graph captured on a small workspace still runs right after a larger call made
    the workspace grow and other tensors took what memory was free."""
    n = 512
    h, g, dy = _rn(40, n, seed=1).to(BF), _rn(n, seed=2), _rn(40, n, seed=3).to(BF)
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-5)
    ws = q.Workspace()
    dG = torch.empty(n, device="cuda")
    q.qlora_rmsnorm_bwd(dy, h, g, rstd, ws, dG=dG)
    want = dG.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qlora_rmsnorm_bwd(dy, h, g, rstd, ws, dG=dG)
    small = ws.buf.numel()
    H = _rn(4000, 4096, seed=4).to(BF)
    q.qlora_rmsnorm_bwd(H, H, _rn(4096), torch.ones(4000, device="cuda"), ws)
    assert ws.buf.numel() > small
    canary = [torch.full((small,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    dG.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dG, want)
    assert all(int((c != 7).sum()) == 0 for c in canary)


def test_mixed_chain_of_dependent_launches():
    """Norm, NF4 layer (small M and GEMM), integer matvec and quantiser back to back
    without synchronisation, each reading what the one before wrote, many times over:
    the bits of the same chain run with a synchronisation after every call."""
    K, r, M = 512, 8, 8
    t, w = layer_on_gpu(K, K, 64, r, tag="chain")
    g = torch.ones(K, device="cuda")
    W0 = _rn(K, K, seed=7) * 0.05
    codes, scales = q.qlora_quantize_int(W0, 4)
    ws = q.Workspace()
    x0 = _rn(M, K, seed=8).to(BF)

    def chain(sync):
        def s(v):
            if sync:
                torch.cuda.synchronize()
            return v
        h = x0
        for i in range(3):
            o = s(q.qlora_rmsnorm_fwd(h, g, 1e-5, residual=x0, dropout=q.Dropout(0.1, i, 0), quant_block=64))
            y, _ = s(q.qlora_linear_fwd(w, o.Y, t["A"], t["B"], ws))
            o = s(q.qlora_rmsnorm_fwd(y, g, 1e-5, residual=o.H, want_y=False, quant_block=0))
            s(q.qlora_quantize_int(W0, 4, out=(codes, scales)))
            h, _ = s(q.qlora_matvec(q.int_weight(codes, scales, K, K), o.act, ws, t["A"], t["B"]))
            big = h.repeat(8, 1)
            o = s(q.qlora_rmsnorm_fwd(big, g, 1e-5, save_rstd=True))
            y, v = s(q.qlora_linear_fwd(w, o.Y, t["A"], t["B"], ws))
            dx, _, _ = s(q.qlora_linear_bwd(w, o.Y, v, y, t["A"], t["B"], ws))
            _, dr, _ = s(q.qlora_rmsnorm_bwd(dx, big, g, o.rstd, ws))
            h = dr[:M].contiguous()
        return h

    want = chain(True)
    for _ in range(30):
        assert torch.equal(chain(False), want)
    assert ws.status() == 0


def test_two_streams_share_nothing():
    """The same calls on two streams at once, each with a workspace of its own."""
    K = 1024
    codes, scales = q.qlora_quantize_int(_rn(K, K) * 0.05, 4)
    w = q.int_weight(codes, scales, K, K)
    xs = [_rn(4, K, seed=i).to(BF) for i in range(2)]
    g = torch.ones(K, device="cuda")
    want = []
    for x in xs:
        o = q.qlora_rmsnorm_fwd(x, g, 1e-5, quant_block=64)
        want.append(q.qlora_matvec(w, o.act, q.Workspace())[0])
    torch.cuda.synchronize()
    streams, wss = [torch.cuda.Stream() for _ in xs], [q.Workspace() for _ in xs]
    outs = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                o = q.qlora_rmsnorm_fwd(xs[i], g, 1e-5, quant_block=64)
                outs[i].append(q.qlora_matvec(w, o.act, wss[i])[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in outs[i])


def test_kernel_timers_and_launch_count():
    x, g = _rn(64, 512).to(BF), torch.ones(512, device="cuda")
    codes, scales = q.qlora_quantize_int(_rn(512, 256), 4)
    w = q.int_weight(codes, scales, 512, 256)
    ws = q.Workspace()
    o = q.qlora_rmsnorm_fwd(x, g, 1e-5, save_rstd=True)
    for kind, call, launches in ((q.KERNEL_RMSNORM, lambda: q.qlora_rmsnorm_fwd(x, g, 1e-5), 1),
                                 (q.KERNEL_RMSNORM_BWD, lambda: q.qlora_rmsnorm_bwd(x, x, g, o.rstd, ws), 2),
                                 (q.KERNEL_MATVEC, lambda: q.qlora_matvec(w, x[:3].contiguous(), ws), 1)):
        tm = q.KernelTimer(kind, 2)
        n0 = q.qlora_launch_count()
        call()
        call()
        assert q.qlora_launch_count() - n0 == 2 * launches
        torch.cuda.synchronize()
        assert all(0 < t < 50 for t in tm.times_ms())
        tm.disarm()


def test_norms_past_32_bit_offsets():
    """More than 2^31 elements: the last rows are where 64-bit offsets put them, and
    their masks count elements in 64 bits."""
    n, M = 65536, 32776
    x = torch.zeros((M, n), dtype=BF, device="cuda")
    last = _rn(2, n, seed=3).to(BF)
    x[-2:] = last
    g = _rn(n, seed=4)
    d = q.Dropout(0.25, 7, 9)
    s = norm.keep_scale(0.25)
    keep = torch.from_numpy(norm.words(7, 9, (M - 2) * n, 2 * n).reshape(2, n) >= np.uint32(2 ** 30)).cuda()
    o = q.qlora_rmsnorm_fwd(x, g, 1e-5, dropout=d, save_rstd=True)
    h = torch.where(keep, last.double() * s, 0.0).to(BF)
    assert torch.equal(o.H[-2:], h) and torch.count_nonzero(o.H[:-2]) == 0
    a = q.qlora_rmsnorm_fwd(h, g, 1e-5, save_rstd=True)
    assert torch.equal(o.Y[-2:], a.Y) and torch.equal(o.rstd[-2:], a.rstd) and torch.count_nonzero(o.Y[:-2]) == 0
    dX, dR, _ = q.qlora_rmsnorm_bwd(x, o.H, g, o.rstd, q.Workspace(), dropout=d, need_dG=False, dR=o.Y)
    want = q.qlora_rmsnorm_bwd(last, h, g, a.rstd, q.Workspace(), need_dG=False)[1]
    assert torch.equal(dR[-2:], want) and torch.count_nonzero(dX[:-2]) == 0 and torch.count_nonzero(dX[-2:][~keep]) == 0
    # dX is the rounding of the unrounded gradient times s: two roundings of half a step
    ref = torch.where(keep, want.double() * s, 0.0)
    assert ((dX[-2:].double() - ref).abs() <= 2.0 ** -7 * 1.01 * ref.abs()).all()
    del x, o, dX, dR
    torch.cuda.empty_cache()
