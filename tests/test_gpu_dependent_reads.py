"""Chains without a synchronisation in which a matrix-vector product reads what the
kernel in front has just written over the same memory: scales of 8-bit activations,
and adapters after an optimizer step.  The bits are those of the same chain with a
synchronisation after every call."""

import ctypes

import pytest
import torch

import quantized_rank_fine_b200 as q
from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _rn(*s, seed=0):
    return torch.randn(s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _weight(K, N, seed):
    return q.int_weight(*q.qlora_quantize_int(_rn(K, N, seed=seed) * 0.05, 4), K, N)


def _ok(status):
    assert status == 0


@pytest.mark.parametrize("M,K,N", [(1, 1024, 1024), (4, 2048, 2048), (16, 4096, 1024), (8, 1088, 320)])
@pytest.mark.parametrize("block", [0, 64])
def test_scales_rewritten_in_place(M, K, N, block):
    """One buffer of codes and one of scales for every step; the gain's size changes from
    step to step, so a scale of the step before is wrong by a factor."""
    w, ws = _weight(K, N, 1), q.Workspace()
    ws.get(1280)
    A, B = (_rn(K, 16, seed=2) / K ** 0.5).to(BF), (_rn(16, N, seed=3) * 0.05).to(BF)
    steps = 24
    xs = [_rn(M, K, seed=10 + i).to(BF) for i in range(steps)]
    gains = [_rn(K, seed=50 + i) * 2.0 ** (i % 7 - 3) for i in range(steps)]
    codes = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    scales = torch.empty((M, K // block if block else 1), device="cuda")
    lib, cw = q.lib(), w.c_struct()

    def chain(sync):
        s = torch.cuda.current_stream().cuda_stream
        ys = [torch.zeros((M, N), dtype=BF, device="cuda") for _ in range(steps)]
        torch.cuda.synchronize()
        for x, g, y in zip(xs, gains, ys):
            _ok(lib.qlora_rmsnorm_fwd(x.data_ptr(), None, g.data_ptr(), q.QLORA_F32, 1e-5, M, K, None, None, None,
                                      codes.data_ptr(), scales.data_ptr(), block, None, s))
            if sync:
                torch.cuda.synchronize()
            _ok(lib.qlora_matvec(ctypes.byref(cw), codes.data_ptr(), scales.data_ptr(), block, M, A.data_ptr(),
                                 B.data_ptr(), 16, 1.0, y.data_ptr(), None, ws.buf.data_ptr(), ws.buf.numel(), s))
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return ys

    want = chain(True)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))
    assert ws.status() == 0


@pytest.mark.parametrize("M", [1, 12])
def test_adapters_rewritten_by_an_optimizer_step(M):
    """The fused optimizer step writes A and B in place; the product right after reads them."""
    K, N, r, steps = 1024, 768, 16, 12
    w = _weight(K, N, 4)
    X, dY, x = _rn(64, K, seed=5).to(BF), _rn(64, N, seed=6).to(BF), _rn(M, K, seed=7).to(BF)
    A0, B0 = (_rn(K, r, seed=8) / K ** 0.5).to(BF), (_rn(r, N, seed=9) * 0.05).to(BF)

    def chain(sync):
        def s(v):
            if sync:
                torch.cuda.synchronize()
            return v
        A, B, ws, out = A0.clone(), B0.clone(), q.Workspace(), []
        state = q.adam_state(A, B)
        for i in range(steps):
            s(q.qlora_linear_bwd_adam(w, X, None, dY, A, B, state, i + 1, ws, lr=0.1, need_dX=False))
            out.append(s(q.qlora_matvec(w, x, ws, A, B))[0])
        torch.cuda.synchronize()
        assert ws.status() == 0
        return out

    want = chain(True)
    assert not torch.equal(want[0], want[-1])
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))
