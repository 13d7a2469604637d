"""GPU parity of the residual addition with RMS norm and of its gradient against
the float64 oracle on the same bytes.

Tolerances, from the arithmetic:
* a bf16 result is off by half a step, 2^-8 of it; an fp32 sum of n positive terms
  in a tree over threads has at most 8 x 8 + 10 roundings on a path, so rstd
  (half of the relative error of the sum, and three roundings) is within 2^-18 and
  y within 2^-17;
* E4M3: half a step is 2^-4 of a normal value and 2^-10 scales below;
* dh is a difference, so its fp32 part is bounded by the terms' magnitudes times
  2^-17 (the same path length), and dG by the path over rows and parts."""

import numpy as np
import pytest
import torch

import quantized_rank_fine_b200 as q
from oracle import norm
from tests.helpers import assert_guards, guarded, require_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _np(t):
    return t.double().cpu().numpy()


def _inputs(M, n, seed=0, g32=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    chan = torch.exp(r(n))
    d = {"x": r(M, n).to(BF), "res": (r(M, n) * chan).to(BF), "g": 1 + 0.3 * r(n), "dy": r(M, n).to(BF),
         "dH": r(M, n).to(BF)}
    if not g32:
        d["g"] = d["g"].to(BF)
    return d


def _check_q(act, y, block):
    v = _np(act.codes.view(torch.float8_e4m3fn).float())
    s = _np(act.scales)
    want = np.abs(y.reshape(y.shape[0], -1, block or y.shape[1])).max(axis=2) / 448.0
    assert np.all(np.abs(s - want) <= 2.0 ** -17 * want)
    sc = np.repeat(s, y.shape[1] // s.shape[1], axis=1)
    assert np.all(np.abs(v * sc - y) <= (2.0 ** -4 + 2.0 ** -15) * np.abs(y) + sc * (2.0 ** -10 + 2.0 ** -15))


SHAPES = [(1, 8), (3, 64), (5, 72), (2, 1032), (4, 4096), (130, 4096), (3, 8192), (2, 8200), (3, 11008), (2, 16392),
          (2, 32768), (1, 32776), (2, 65536), (700, 256)]


@pytest.mark.parametrize("M,n", SHAPES)
@pytest.mark.parametrize("res,p,g32", [(True, 0.0, False), (False, 0.0, True), (True, 0.3, True), (False, 0.1, False)])
def test_forward(M, n, res, p, g32):
    d = _inputs(M, n, M + n, g32)
    drop = q.Dropout(p, 0x123456789ABCDEF1, 77) if p else None
    bufs, H = guarded((M, n), BF)
    bufy, Y = guarded((M, n), BF)
    o = q.qlora_rmsnorm_fwd(d["x"], d["g"], EPS, d["res"] if res else None, drop, save_rstd=True, H=H, Y=Y,
                            quant_block=0)
    assert_guards([bufs, bufy], "rmsnorm_fwd")
    keep = norm.keep_mask(p, drop.seed, drop.offset, M, n) if p else None
    h, y, rstd = norm.rmsnorm(_np(d["x"]), _np(d["res"]) if res else None, _np(d["g"]), EPS, keep, p)
    assert np.array_equal(_np(o.H), h)
    assert np.all(np.abs(_np(o.rstd) - rstd) <= 2.0 ** -18 * rstd)
    assert np.all(np.abs(_np(o.Y) - y) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(y))
    _check_q(o.act, y, 0)
    if n % 64 == 0:
        o2 = q.qlora_rmsnorm_fwd(d["x"], d["g"], EPS, d["res"] if res else None, drop, want_y=False, quant_block=64)
        assert o2.Y is None and (o2.H is None) == (not res and not p)
        _check_q(o2.act, y, 64)
    # without the 8-bit output, and again: the same bits
    o3 = q.qlora_rmsnorm_fwd(d["x"], d["g"], EPS, d["res"] if res else None, drop, save_rstd=True)
    assert torch.equal(o3.Y, o.Y) and torch.equal(o3.rstd, o.rstd)


def test_codes_are_the_oracles_where_y_is_exact():
    """Rows whose mean square and gain are powers of two: y is exact, so the codes
    and scales are the definition's bit for bit (ties and subnormal codes among them)."""
    M, n = 6, 128
    rng = np.random.default_rng(0)
    x = np.ones((M, n))
    x[:, ::2] = -1.0
    g = np.ldexp(rng.integers(1, 256, n).astype(np.float64), rng.integers(-14, 2, n))
    g[:64] = np.arange(64) / 64.0 * 448.0      # multiples of 7: ties of the 3-bit mantissa
    xt = torch.from_numpy(x).to(BF).cuda()
    gt = torch.from_numpy(g).float().cuda()
    # eps = 3: mean square 1 + 3 = 4, rstd = 1/2
    for block in (0, 64):
        o = q.qlora_rmsnorm_fwd(xt, gt, 3.0, want_y=False, quant_block=block)
        v, s = norm.quantize_e4m3(x * 0.5 * g, block)
        assert np.array_equal(_np(o.act.scales), s)
        assert np.array_equal(_np(o.act.codes.view(torch.float8_e4m3fn).float()), v)


def test_codes_of_random_quotients():
    """y made exact again (rstd = 1/2 on rows of +-1, gains of 24 bits): a million
    quotients y / s over many scales, every code as from the IEEE quotient."""
    M, n = 64, 16384
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = (torch.randint(0, 2, (M, n), generator=gen, device="cuda") * 2 - 1).to(BF)
    for lo in (-20, -60):
        g = torch.randn(n, generator=gen, device="cuda") * torch.exp2(torch.randint(lo, 8, (n,), generator=gen, device="cuda").float())
        o = q.qlora_rmsnorm_fwd(x, g, 3.0, want_y=False, quant_block=64)
        v, s = norm.quantize_e4m3(_np(x[:1]) * 0.5 * _np(g), 64)
        got = _np(o.act.codes.view(torch.float8_e4m3fn).float())
        assert np.array_equal(_np(o.act.scales), np.repeat(s, M, axis=0))
        sign = _np(x) * _np(x[:1])
        assert np.array_equal(got, sign * v)


def test_zero_rows_and_nonfinite_values():
    n = 256
    d = _inputs(4, n)
    x = d["x"].clone()
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 70] = float("inf")
    o = q.qlora_rmsnorm_fwd(x, d["g"], EPS, save_rstd=True, quant_block=64)
    assert torch.count_nonzero(o.Y[0]) == 0 and torch.count_nonzero(o.act.codes[0]) == 0
    assert torch.count_nonzero(o.act.scales[0]) == 0
    deq = o.act.codes.view(torch.float8_e4m3fn).float().view(4, -1, 64) * o.act.scales[:, :, None]
    assert torch.isnan(o.Y[1]).all() and torch.isnan(deq[1]).all()
    assert torch.isnan(o.Y[2, 70]) and torch.isnan(deq[2, 1]).all()
    # the other rows do not see them
    clean = q.qlora_rmsnorm_fwd(d["x"], d["g"], EPS, quant_block=64)
    assert torch.equal(clean.Y[3], o.Y[3]) and torch.equal(clean.act.codes[3], o.act.codes[3])


def test_tiny_blocks_quantise():
    """Blocks of very small values: a scale that would be subnormal is zero, and so is
    the block; a small normal one quantises as any other.  No NaN."""
    n = 128
    g = torch.full((n,), 1e-30, device="cuda")
    g[64:] = 2.0 ** -140
    x = _inputs(2, n)["x"]
    o = q.qlora_rmsnorm_fwd(x, g, EPS, want_y=False, quant_block=64)
    v = _np(o.act.codes.view(torch.float8_e4m3fn).float())
    _, y, _ = norm.rmsnorm(_np(x), None, _np(g), EPS)
    s = _np(o.act.scales)
    assert np.count_nonzero(v[:, 64:]) == 0 and np.count_nonzero(s[:, 1]) == 0 and np.all(s[:, 0] > 0)
    assert np.all(np.abs(v[:, :64] * s[:, :1] - y[:, :64]) <= (2.0 ** -4 + 2.0 ** -15) * np.abs(y[:, :64]) + s[:, :1] * 2.0 ** -9)


def test_dropped_values_do_not_count():
    """NaN and infinity at dropped places of the branch leave every output finite."""
    M, n, p = 8, 512, 0.5
    d = _inputs(M, n, 12)
    drop = q.Dropout(p, 3, 4)
    keep = torch.from_numpy(norm.keep_mask(p, 3, 4, M, n)).cuda()
    bad = torch.where(keep, d["x"], torch.tensor(float("nan"), dtype=BF, device="cuda"))
    bad[:, ::3] = torch.where(keep[:, ::3], bad[:, ::3], torch.tensor(float("inf"), dtype=BF, device="cuda"))
    a = q.qlora_rmsnorm_fwd(bad, d["g"], EPS, d["res"], drop, quant_block=64)
    b = q.qlora_rmsnorm_fwd(d["x"], d["g"], EPS, d["res"], drop, quant_block=64)
    assert torch.equal(a.H, b.H) and torch.equal(a.Y, b.Y) and torch.equal(a.act.codes, b.act.codes)


@pytest.mark.parametrize("M,n", SHAPES)
@pytest.mark.parametrize("dH,p,g32", [(True, 0.0, False), (False, 0.0, True), (True, 0.3, False)])
def test_backward(M, n, dH, p, g32):
    d = _inputs(M, n, 7 * M + n, g32)
    drop = q.Dropout(p, 99, 1 << 40) if p else None
    h = d["res"]
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    ws = q.Workspace()
    bufr, dR = guarded((M, n), BF)
    bufx, dX = guarded((M, n), BF)
    bufg, dG = guarded((n,), torch.float32)
    gx, gr, gg = q.qlora_rmsnorm_bwd(d["dy"], h, d["g"], rstd, ws, d["dH"] if dH else None, drop, dR=dR, dX=dX, dG=dG)
    assert_guards([bufr, bufx, bufg], "rmsnorm_bwd")
    keep = norm.keep_mask(p, drop.seed, drop.offset, M, n) if p else None
    dy, hn, g, rs = _np(d["dy"]), _np(h), _np(d["g"]), _np(rstd)[:, None]
    e = _np(d["dH"]) if dH else np.zeros((M, n))
    dx, dh, dg = norm.rmsnorm_backward(dy, hn, g, rs[:, 0], e, keep, p)
    terms = rs * np.abs(dy * g) + rs ** 3 * np.abs(hn) * np.abs(dy * g * hn).mean(1, keepdims=True) + np.abs(e)
    assert np.all(np.abs(_np(gr) - dh) <= 2.0 ** -8 * np.abs(dh) + 2.0 ** -17 * terms)
    sc = norm.keep_scale(p) if p else 1.0
    assert np.all(np.abs(_np(gx) - dx) <= 2.0 ** -8 * np.abs(dx) + 2.0 ** -17 * sc * terms)
    path = M / 148 + 600
    assert np.all(np.abs(_np(gg) - dg) <= path * 2.0 ** -24 * np.abs(dy * hn * rs).sum(0))
    if p:
        assert torch.count_nonzero(gx[torch.from_numpy(~keep).cuda()]) == 0
    # frozen gain; accumulation; the same bits again
    fx, fr, none = q.qlora_rmsnorm_bwd(d["dy"], h, d["g"], rstd, ws, d["dH"] if dH else None, drop, need_dG=False)
    assert none is None and torch.equal(fr, gr) and torch.equal(fx, gx)
    acc = torch.ones_like(gg)
    q.qlora_rmsnorm_bwd(d["dy"], h, d["g"], rstd, ws, d["dH"] if dH else None, drop, accumulate=True, dG=acc)
    assert torch.equal(acc, gg + 1)


def test_backward_against_differences():
    """The kernels' own forward differenced: sum(dY y) in float64 along one random
    direction of h and of g, from bf16 outputs of fp32 arithmetic averaged over many
    elements (steps of 2^-4 keep the outputs' rounding below the change)."""
    M, n = 64, 512
    d = _inputs(M, n, 3, True)
    h = d["res"]
    rstd = q.qlora_rmsnorm_fwd(h, d["g"], EPS, save_rstd=True).rstd
    gx, _, gg = q.qlora_rmsnorm_bwd(d["dy"], h, d["g"], rstd, q.Workspace())
    dy = d["dy"].double()
    g64, h64 = d["g"].double(), h.double()

    def loss(hh, gg_):
        return (dy * hh * torch.rsqrt(hh.square().mean(1, keepdim=True) + EPS) * gg_).sum().item()

    u = torch.randn(M, n, device="cuda", dtype=torch.float64, generator=torch.Generator("cuda").manual_seed(1))
    t = 1e-5
    num = (loss(h64 + t * u, g64) - loss(h64 - t * u, g64)) / (2 * t)
    ana = (gx.double() * u).sum().item()
    # each dx is off by half a bf16 step: 2^-8 of it, independent signs
    slack = 6 * 2.0 ** -8 * (gx.double() * u).square().sum().sqrt().item()
    assert abs(num - ana) <= slack
    ug = u[0]
    num = (loss(h64, g64 + t * ug) - loss(h64, g64 - t * ug)) / (2 * t)
    assert abs(num - (gg.double() * ug).sum().item()) <= 1e-5 * (gg.double() * ug).abs().sum().item()


def test_side_stream_and_graph_counter():
    """A forward and a backward captured in a graph on a side stream: every replay
    reads the device counter, so it draws the mask of its own step, and both
    directions of one replay draw the same one."""
    M, n, p = 96, 1024, 0.25
    d = _inputs(M, n, 5)
    cnt = torch.zeros(1, dtype=torch.int64, device="cuda")
    drop = q.Dropout(p, 11, 1000, cnt)
    ws = q.Workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        o = q.qlora_rmsnorm_fwd(d["x"], d["g"], EPS, d["res"], drop, save_rstd=True)
        return o, q.qlora_rmsnorm_bwd(d["dy"], o.H, d["g"], o.rstd, ws, d["dH"], drop)

    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o, grads = step()
    for i in range(3):
        cnt.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        eager = q.Dropout(p, 11, 1000 + i)
        oe = q.qlora_rmsnorm_fwd(d["x"], d["g"], EPS, d["res"], eager, save_rstd=True)
        ge = q.qlora_rmsnorm_bwd(d["dy"], oe.H, d["g"], oe.rstd, q.Workspace(), d["dH"], eager)
        assert torch.equal(o.H, oe.H) and torch.equal(o.Y, oe.Y)
        assert all(torch.equal(a, b) for a, b in zip(grads, ge))
        keep = torch.from_numpy(norm.keep_mask(p, 11, 1000 + i, M, n)).cuda()
        assert torch.count_nonzero(grads[0][~keep]) == 0


def test_explicit_stream_argument():
    M, n = 64, 4096
    d = _inputs(M, n, 8)
    want = q.qlora_rmsnorm_fwd(d["x"], d["g"], EPS, d["res"], save_rstd=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = q.qlora_rmsnorm_fwd(d["x"], d["g"], EPS, d["res"], save_rstd=True, stream=s)
    ws = q.Workspace()
    gb = q.qlora_rmsnorm_bwd(d["dy"], got.H, d["g"], got.rstd, ws, stream=s)
    s.synchronize()
    wb = q.qlora_rmsnorm_bwd(d["dy"], want.H, d["g"], want.rstd, q.Workspace())
    assert torch.equal(got.Y, want.Y) and torch.equal(gb[1], wb[1]) and torch.equal(gb[2], wb[2])


def test_rows_past_32_bit_offsets():
    """2^32 elements and more: the last rows against the same rows alone."""
    n = 65536
    M = (1 << 16) + 3
    x = torch.zeros((M, n), dtype=BF, device="cuda")
    tail = _inputs(4, n, 21)
    x[-4:] = tail["x"]
    o = q.qlora_rmsnorm_fwd(x, tail["g"], EPS, save_rstd=True)
    t = q.qlora_rmsnorm_fwd(tail["x"], tail["g"], EPS, save_rstd=True)
    assert torch.equal(o.Y[-4:], t.Y) and torch.equal(o.rstd[-4:], t.rstd)
    assert torch.count_nonzero(o.Y[:8]) == 0
    dy = torch.zeros_like(x)
    dy[-4:] = tail["dy"]
    _, dr, dg = q.qlora_rmsnorm_bwd(dy, x, tail["g"], o.rstd, q.Workspace())
    _, er, eg = q.qlora_rmsnorm_bwd(tail["dy"], tail["x"], tail["g"], t.rstd, q.Workspace())
    assert torch.equal(dr[-4:], er)
    assert torch.allclose(dg, eg, rtol=1e-5, atol=1e-5)
    del x, dy, o, dr
    torch.cuda.empty_cache()


def test_refusals_on_the_device():
    d = _inputs(4, 128)
    lib, s = q.lib(), torch.cuda.current_stream().cuda_stream
    x, g, y = d["x"], d["g"], torch.empty_like(d["x"])
    args = lambda X, Y: (X, None, g.data_ptr(), 1, 1e-5, 2, 128, None, None, Y, None, None, 0, None, s)
    assert lib.qlora_rmsnorm_fwd(*args(x.data_ptr(), y.data_ptr())) == 0
    assert lib.qlora_rmsnorm_fwd(*args(x.data_ptr() + 2, y.data_ptr())) == 3        # not 16-byte aligned
    host = torch.empty((4, 128), dtype=BF)
    assert lib.qlora_rmsnorm_fwd(*args(host.data_ptr(), y.data_ptr())) == 1         # host memory
    cnt = torch.zeros(2, dtype=torch.int64, device="cuda")
    import ctypes
    bad = ctypes.byref(q._Dropout(0.5, 1, 1, cnt.data_ptr() + 4))
    assert lib.qlora_dropout_mask(bad, 4, 8, y.data_ptr(), s) == 3                  # counter not 8-byte aligned
    ok = ctypes.byref(q._Dropout(0.5, 1, 1, cnt.data_ptr() + 8))
    assert lib.qlora_dropout_mask(ok, 4, 8, y.data_ptr(), s) == 0
