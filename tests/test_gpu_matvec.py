"""GPU parity of the matrix-vector product with an integer weight (one scale per
16 weights) against float64 on the same bytes, for bf16 and 8-bit activations.

Tolerances: the output is rounded to bf16 (half a step, 2^-8 of it); each product
x scale q is formed from an operand rounded to bf16 at most (2^-8 of the product,
independent signs), so the norm of the error stays below 2^-8 of the result's norm
(two uniform errors of variance 2^-16 / 3 each) and a single element's below
2^-8 of itself plus 2^-8 of the root of the sum of its squared products times six
(six standard deviations, of which each product's error has at most 1 / sqrt 3).
V is off by half a step, or a whole one where two fp32 sums round apart."""

import numpy as np
import pytest
import torch

import quantized_rank_fine_b200 as q
from oracle import intq
from tests.helpers import assert_guards, guarded, require_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _case(M, K, N, r, x8, seed=0, bits=4):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")
    codes, scales = q.qlora_quantize_int(rn(K, N) * 0.02, bits)
    w = q.int_weight(codes, scales, K, N)
    if x8 is None:
        X = rn(M, K).to(BF)
        x64 = X.double()
    else:
        y = rn(M, K) * torch.exp(rn(K))
        b = y.view(M, -1, x8 or K)
        s = b.abs().amax(2) / 448
        X = q.Act8((b / s[:, :, None]).to(torch.float8_e4m3fn).view(M, K).view(torch.uint8), s.contiguous(), x8)
        x64 = (X.codes.view(torch.float8_e4m3fn).double().view(M, -1, x8 or K) * s.double()[:, :, None]).view(M, K)
    A = (rn(K, r) / K ** 0.5).to(BF) if r else None
    B = (rn(r, N) * 0.05).to(BF) if r else None
    w64 = torch.from_numpy(intq.dequantize_int(codes.cpu().numpy(), scales.cpu().numpy(), K, N)).cuda().double()
    return w, X, x64, A, B, w64


def _check(Y, V, x64, A, B, w64, scale=1.0):
    y = x64 @ w64
    sq = (x64 ** 2) @ (w64 ** 2)
    if A is not None:
        v = scale * (x64 @ A.double())
        if V is not None:
            mag = abs(scale) * (x64.abs() @ A.double().abs())
            assert ((V.double() - v).abs() <= 2.0 ** -8 * v.abs() + 2.0 ** -15 * mag).all()
        y = y + v @ B.double()
        sq = sq + (v ** 2) @ (B.double() ** 2)
    e = Y.double() - y
    assert torch.isfinite(Y).all()
    assert e.norm() <= 2.0 ** -8 * y.norm(), f"relative error {(e.norm() / y.norm()).item():.2e}"
    assert (e.abs() <= 2.0 ** -8 * y.abs() + 6 * 2.0 ** -8 / 3 ** 0.5 * sq.sqrt()).all()


SHAPES = [(64, 64), (64, 192), (320, 192), (192, 320), (1024, 64), (576, 704), (4096, 256), (256, 4160), (2048, 1536)]


@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("M", [1, 2, 5, 8, 9, 16])
@pytest.mark.parametrize("x8", [None, 0, 64])
def test_matvec(M, K, N, x8):
    for r in (0, 16):
        w, X, x64, A, B, w64 = _case(M, K, N, r, x8, K + N + M)
        ws = q.Workspace()
        buf, Y = guarded((M, N), BF)
        bufv, V = guarded((M, max(r, 8)), BF)
        Yo, Vo = q.qlora_matvec(w, X, ws, A, B, save_V=True, Y=Y, V=V if r else None)
        assert_guards([buf, bufv], "matvec")
        assert ws.status() == 0
        _check(Y, Vo, x64, A, B, w64)
        # V kept in the workspace; the same bits again
        Y2, none = q.qlora_matvec(w, X, ws, A, B)
        assert none is None and torch.equal(Y2, Y)


@pytest.mark.parametrize("r", [8, 24, 64, 72, 136, 256])
@pytest.mark.parametrize("M", [3, 16])
def test_ranks_and_scale(M, r):
    for x8 in (None, 64):
        w, X, x64, A, B, w64 = _case(M, 640, 448, r, x8, r)
        Y, V = q.qlora_matvec(w, X, q.Workspace(), A, B, adapter_scale=-0.5, save_V=True)
        _check(Y, V, x64, A, B, w64, -0.5)


@pytest.mark.parametrize("bits", [2, 3])
def test_narrow_integers(bits):
    w, X, x64, A, B, w64 = _case(4, 512, 320, 8, None, 3, bits)
    Y, V = q.qlora_matvec(w, X, q.Workspace(), A, B, save_V=True)
    _check(Y, V, x64, A, B, w64)


@pytest.mark.parametrize("M,K,N,r,x8", [(1, 4096, 4096, 16, None), (4, 11008, 4096, 16, 64), (16, 4096, 11008, 64, 0)])
def test_projection_sizes(M, K, N, r, x8):
    w, X, x64, A, B, w64 = _case(M, K, N, r, x8, 5)
    Y, V = q.qlora_matvec(w, X, q.Workspace(), A, B, save_V=True)
    _check(Y, V, x64, A, B, w64)


def test_every_code_and_exact_values():
    """All sixteen codes (0 is -8, which the quantiser never writes), power-of-two
    scales and small integers: the result is exact, so it is compared for equality."""
    K, N, M = 128, 128, 8
    rng = np.random.default_rng(0)
    code = rng.integers(0, 16, (K, N)).astype(np.uint8)
    flat = code.reshape(-1, 2)
    codes = torch.from_numpy((flat[:, 0] | (flat[:, 1] << 4)).astype(np.uint8)).cuda()
    sc = 2.0 ** rng.integers(-3, 2, (K, N // 16))
    x = rng.integers(-3, 4, (M, K)).astype(np.float64)
    x[:, rng.permutation(K)[:K - 6]] = 0          # few terms: sums stay within bf16's 8 bits more often
    y = x @ ((code.astype(np.float64) - 8) * np.repeat(sc, 16, axis=1))
    w = q.int_weight(codes, torch.from_numpy(sc).float().cuda().reshape(-1), K, N)
    Y, _ = q.qlora_matvec(w, torch.from_numpy(x).to(BF).cuda(), q.Workspace())
    assert torch.equal(Y, torch.from_numpy(y).float().to(BF).cuda())


def test_zero_scales_and_zero_rows():
    w, X, x64, _, _, w64 = _case(4, 256, 192, 0, None, 9)
    w.dq_scales.view(256, 12)[:, 5] = 0
    X[2] = 0
    Y, _ = q.qlora_matvec(w, X, q.Workspace())
    assert torch.count_nonzero(Y[:, 80:96]) == 0 and torch.count_nonzero(Y[2]) == 0


def test_nan_stays_in_its_row():
    w, X, x64, A, B, w64 = _case(9, 256, 192, 8, None, 9)
    Y0, V0 = q.qlora_matvec(w, X, q.Workspace(), A, B, save_V=True)
    X2 = X.clone()
    X2[3, 77] = float("nan")
    X2[8, 1] = float("inf")
    Y, V = q.qlora_matvec(w, X2, q.Workspace(), A, B, save_V=True)
    assert torch.isnan(Y[3]).all() and not torch.isfinite(Y[8]).all()
    rows = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(Y[rows], Y0[rows]) and torch.equal(V[rows], V0[rows])


@pytest.mark.parametrize("K,N", [(256, 192), (2048, 1536)])
@pytest.mark.parametrize("x8", [None, 0, 64])
def test_infinities_stay_visible(K, N, x8):
    """An infinity in A, in B or in a scale of the weight: what it reaches is not
    finite, and every other output keeps its bits."""
    w, X, x64, A, B, w64 = _case(5, K, N, 16, x8, 21)
    Y0, V0 = q.qlora_matvec(w, X, q.Workspace(), A, B, save_V=True)
    A2 = A.clone()
    A2[70, 3] = float("inf")
    Y, V = q.qlora_matvec(w, X, q.Workspace(), A2, B, save_V=True)
    assert not torch.isfinite(Y).any() and not torch.isfinite(V[:, 3]).any()
    keep = [i for i in range(16) if i != 3]
    assert torch.equal(V[:, keep], V0[:, keep])
    B2 = B.clone()
    B2[9, 100] = float("-inf")
    Y, V = q.qlora_matvec(w, X, q.Workspace(), A, B2, save_V=True)
    cols = torch.arange(N, device="cuda") != 100
    assert not torch.isfinite(Y[:, 100]).any() and torch.equal(Y[:, cols], Y0[:, cols]) and torch.equal(V, V0)
    w.dq_scales.view(K, N // 16)[31, 2] = float("inf")
    Y, V = q.qlora_matvec(w, X, q.Workspace(), A, B, save_V=True)
    cols = torch.arange(N, device="cuda") // 16 != 2
    assert not torch.isfinite(Y[:, 32:48]).any() and torch.equal(Y[:, cols], Y0[:, cols]) and torch.equal(V, V0)


def test_matches_the_layer_forward():
    """The layer's forward on the same integer weight multiplies with bf16(w')."""
    w, X, x64, A, B, w64 = _case(8, 1024, 768, 16, None, 2)
    ws = q.Workspace()
    Y, V = q.qlora_matvec(w, X, ws, A, B, adapter_scale=2.0, save_V=True)
    Yl, Vl = q.qlora_linear_fwd(w, X, A, B, ws, adapter_scale=2.0)
    assert (Y.double() - Yl.double()).norm() <= 2.0 ** -7 * Yl.double().norm()
    assert (V.double() - Vl.double()).norm() <= 2.0 ** -8 * Vl.double().norm()


def test_graph_replay_and_chain():
    """Calls back to back, each reading what the one before wrote, in a captured
    graph, against the same calls one by one with a synchronisation between."""
    K = 512
    gen = torch.Generator(device="cuda").manual_seed(0)
    ws = q.Workspace()
    weights = []
    for i in range(6):
        codes, scales = q.qlora_quantize_int(torch.randn((K, K), generator=gen, device="cuda") * 0.05, 4)
        weights.append(q.int_weight(codes, scales, K, K))
    A = (torch.randn((K, 8), generator=gen, device="cuda") * 0.05).to(BF)
    B = (torch.randn((8, K), generator=gen, device="cuda") * 0.05).to(BF)
    x = torch.randn((5, K), generator=gen, device="cuda").to(BF)

    def chain(sync):
        h = x
        for i, w in enumerate(weights):
            h, _ = q.qlora_matvec(w, h, ws, *((A, B) if i % 2 else (None, None)))
            if sync:
                torch.cuda.synchronize()
        return h

    want = chain(True)
    for _ in range(20):
        assert torch.equal(chain(False), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain(False)
    for _ in range(20):
        got.zero_()
        g.replay()
        assert torch.equal(got, want)


def test_first_call_of_a_variant_inside_a_capture():
    """A variant that no call has prepared yet (120 adapter columns, row scales) is
    captured at once; the replay has the bits of a call made after it."""
    for K, N in ((512, 256), (2048, 1536)):
        w, X, x64, A, B, w64 = _case(13, K, N, 120, 0, 31)
        ws = q.Workspace()
        ws.get(1 << 16)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            Y, V = q.qlora_matvec(w, X, ws, A, B, save_V=True)
        g.replay()
        torch.cuda.synchronize()
        _check(Y, V, x64, A, B, w64)
        want = q.qlora_matvec(w, X, ws, A, B, save_V=True)
        assert torch.equal(Y, want[0]) and torch.equal(V, want[1])


def test_two_host_threads():
    """Calls from two threads at once, each on a stream and a workspace of its own."""
    import threading
    w, X, x64, A, B, w64 = _case(6, 1024, 768, 16, 64, 33)
    want, _ = q.qlora_matvec(w, X, q.Workspace(), A, B)
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        st, ws = torch.cuda.Stream(), q.Workspace()
        with torch.cuda.stream(st):
            ys = [q.qlora_matvec(w, X, ws, A, B)[0] for _ in range(50)]
        st.synchronize()
        got[i] = ys

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(y, want) for ys in got for y in ys)


def test_fresh_weights_each_call():
    """A weight quantised by the call just before is read whole."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    ws = q.Workspace()
    K, N = 1024, 512
    codes = torch.empty(K * N // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(K * N // 16, dtype=torch.float32, device="cuda")
    w = q.int_weight(codes, scales, K, N)
    X = torch.randn((2, K), generator=gen, device="cuda").to(BF)
    W0 = [torch.randn((K, N), generator=gen, device="cuda") for _ in range(8)]
    outs = []
    for W in W0:
        q.qlora_quantize_int(W, 4, out=(codes, scales))
        outs.append(q.qlora_matvec(w, X, ws)[0])
    torch.cuda.synchronize()
    for W, Y in zip(W0, outs):
        q.qlora_quantize_int(W, 4, out=(codes, scales))
        torch.cuda.synchronize()
        assert torch.equal(q.qlora_matvec(w, X, ws)[0], Y)


def test_side_stream():
    w, X, x64, A, B, w64 = _case(3, 2048, 512, 16, 64, 4)
    want, _ = q.qlora_matvec(w, X, q.Workspace(), A, B)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, _ = q.qlora_matvec(w, X, q.Workspace(), A, B, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_more_columns_than_32_bit_weights():
    """A weight of more than 2^31 elements: its last rows and columns are read where they are."""
    K, N = 256, 1 << 23
    codes = torch.full((K * N // 2,), 0x88, dtype=torch.uint8, device="cuda")      # all zeros
    scales = torch.full((K * N // 16,), 0.5, device="cuda")
    codes.view(K, N // 2)[-1, -1] = 0xF8                                           # the very last weight: +7
    codes.view(K, N // 2)[-1, 0] = 0x89                                            # first of the last row: +1
    w = q.int_weight(codes, scales, K, N)
    X = torch.ones((2, K), dtype=BF, device="cuda")
    X[1] = 2
    Y, _ = q.qlora_matvec(w, X, q.Workspace())
    assert Y[0, -1] == 3.5 and Y[1, -1] == 7.0 and Y[0, 0] == 0.5 and Y[1, 0] == 1.0
    assert torch.count_nonzero(Y) == 4
    del codes, scales, Y
    torch.cuda.empty_cache()
