"""The counter-based dropout: its mask against the oracle's words, and the layer's
calls under it bit for bit against the same calls given that mask as bytes."""

import numpy as np
import pytest
import torch

import quantized_rank_fine_b200 as q
from oracle import linear, norm
from tests.helpers import assert_close, assert_guards, guarded, layer_on_gpu, oracle_weight, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("M,n", [(1, 1), (1, 15), (3, 17), (16, 8), (300, 40), (1000, 64), (7, 4099)])
@pytest.mark.parametrize("p,seed,offset", [(0.0, 1, 0), (0.05, (1 << 64) - 1, 3), (0.5, 7, (1 << 64) - 1),
                                           (0.999, 1 << 40, 1 << 33)])
def test_mask_bytes(M, n, p, seed, offset):
    buf, out = guarded((M, n), torch.uint8)
    q.qlora_dropout_mask(M, n, q.Dropout(p, seed, offset), out=out)
    assert_guards([buf], "dropout_mask")
    assert np.array_equal(out.cpu().numpy(), norm.keep_mask(p, seed, offset, M, n).astype(np.uint8))


def test_mask_counter_adds_modulo_two_to_the_64():
    cnt = torch.tensor([5], dtype=torch.int64, device="cuda")
    a = q.qlora_dropout_mask(64, 64, q.Dropout(0.5, 3, (1 << 64) - 2, cnt))
    assert torch.equal(a, q.qlora_dropout_mask(64, 64, q.Dropout(0.5, 3, 3)))


def test_mask_past_32_bit_counters():
    """Elements past 2^34, whose Philox block number needs its high word."""
    M, n = (1 << 14) + 1, 1 << 20
    m = q.qlora_dropout_mask(M, n, q.Dropout(0.3, 42, 17))
    first = M * n - 4096
    t = np.uint32(np.rint(np.float64(np.float32(0.3)) * 2 ** 32))
    assert np.array_equal(m.view(-1)[first:].cpu().numpy(), (norm.words(42, 17, first, 4096) >= t).astype(np.uint8))
    del m
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,n_in,n_out,r", [(1, 128, 64, 8), (16, 512, 320, 16), (8, 256, 256, 72), (17, 320, 192, 24),
                                            (300, 512, 768, 64), (130, 256, 512, 256), (2048, 1024, 1024, 16)])
@pytest.mark.parametrize("p", [0.05, 0.5])
def test_layer_equals_stored_mask(M, n_in, n_out, r, p):
    t, w = layer_on_gpu(n_in, n_out, M, r, tag="ctr")
    d = q.Dropout(p, 0xDEADBEEFCAFE, 5)
    keep = q.qlora_dropout_mask(M, r, d)
    ws = q.Workspace()
    kw, kk = dict(adapter_scale=2.0, dropout=d), dict(adapter_scale=2.0, dropout_keep=keep, dropout_p=p)
    Y, V = q.qlora_linear_fwd(w, t["X"], t["A"], t["B"], ws, **kw)
    Yk, Vk = q.qlora_linear_fwd(w, t["X"], t["A"], t["B"], ws, **kk)
    assert torch.equal(Y, Yk) and torch.equal(V, Vk)
    assert torch.count_nonzero(V[keep == 0]) == 0
    for v in (V, None):
        got = q.qlora_linear_bwd(w, t["X"], v, t["dY"], t["A"], t["B"], ws, **kw)
        want = q.qlora_linear_bwd(w, t["X"], v, t["dY"], t["A"], t["B"], ws, **kk)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    sa, sb = q.adam_state(t["A"], t["B"]), q.adam_state(t["A"], t["B"])
    A1, B1, A2, B2 = t["A"].clone(), t["B"].clone(), t["A"].clone(), t["B"].clone()
    x1 = q.qlora_linear_bwd_adam(w, t["X"], V, t["dY"], A1, B1, sa, 1, ws, **kw)
    x2 = q.qlora_linear_bwd_adam(w, t["X"], V, t["dY"], A2, B2, sb, 1, ws, **kk)
    assert torch.equal(x1, x2) and torch.equal(A1, A2) and torch.equal(B1, B2)
    assert all(torch.equal(sa[k], sb[k]) for k in sa)
    assert ws.status() == 0


def test_layer_against_oracle():
    M, n_in, n_out, r, p = 200, 320, 448, 16, 0.1
    t, w = layer_on_gpu(n_in, n_out, M, r, tag="ctro")
    d = q.Dropout(p, 9, 9)
    ws = q.Workspace()
    Y, V = q.qlora_linear_fwd(w, t["X"], t["A"], t["B"], ws, adapter_scale=2.0, dropout=d)
    dX, dA, dB = q.qlora_linear_bwd(w, t["X"], V, t["dY"], t["A"], t["B"], ws, adapter_scale=2.0, dropout=d)
    k = norm.keep_mask(p, 9, 9, M, r)
    Wq = oracle_weight(w)
    Yr, Vr = linear.forward(t["X"], t["A"], t["B"], Wq, 2.0, k, p)
    g = linear.backward(t["X"], t["A"], t["B"], Wq, t["dY"], 2.0, k, p)
    for name, got, ref in (("Y", Y, Yr), ("V", V, Vr), ("dX", dX, g["dX"]), ("dA", dA, g["dA"]), ("dB", dB, g["dB"])):
        assert_close(got, ref, name)


def test_layer_p_zero_is_the_plain_layer():
    t, w = layer_on_gpu(256, 256, 64, 8, tag="ctr0")
    ws = q.Workspace()
    Y, V = q.qlora_linear_fwd(w, t["X"], t["A"], t["B"], ws, dropout=q.Dropout(0.0, 1))
    Y0, V0 = q.qlora_linear_fwd(w, t["X"], t["A"], t["B"], ws)
    assert torch.equal(Y, Y0) and torch.equal(V, V0)


def test_layer_counter_in_a_replayed_graph():
    """One captured training step, replayed: each replay uses the mask of the step
    number on the device, in the forward and the backward."""
    M, n_in, n_out, r, p = 64, 256, 256, 16, 0.5
    t, w = layer_on_gpu(n_in, n_out, M, r, tag="ctrg")
    cnt = torch.zeros(1, dtype=torch.int64, device="cuda")
    d = q.Dropout(p, 1, 0, cnt)
    ws = q.Workspace()

    def step(drop):
        Y, V = q.qlora_linear_fwd(w, t["X"], t["A"], t["B"], ws, dropout=drop)
        return (Y, V) + q.qlora_linear_bwd(w, t["X"], V, t["dY"], t["A"], t["B"], ws, dropout=drop)

    step(d)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(d)
    masks = set()
    for i in range(3):
        cnt.fill_(i)
        g.replay()
        torch.cuda.synchronize()
        want = step(q.Dropout(p, 1, i))
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        masks.add(q.qlora_dropout_mask(M, r, q.Dropout(p, 1, i)).cpu().numpy().tobytes())
    assert len(masks) == 3
