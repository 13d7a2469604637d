"""What the matrix-vector product on the integer base keeps of its numbers, at every
size of the weight.

Tolerance.  With P the root of the sum of the squared products x s q (and V B), and
eps / 2 of a type its half step:
* Y is rounded to bf16 once: 2^-8 of |y|;
* each product's factor x s goes in as two bf16 terms: 2^-8 of what the first leaves,
  which is 2^-8 of it, so 2^-16 at most, of independent signs; six standard deviations
  of a uniform error are 6 / sqrt 3 of that times P, below 2^-14 P.  V B is held to
  the same (V as two bf16 terms, x as two where it has block scales);
* fp32 sums: K / 16 products of a tile and at most 32 parts follow one another, two
  terms each, every sum within 2^-23 of a partial sum, which is of the size of P or
  smaller: (K / 16 + 32) 2^-22 P.
One term alone would leave errors of 2^-8 / sqrt 3 of each product, 2^-9.3 P in the
root mean square, six times the bound at K = 4096."""

import numpy as np
import pytest
import torch

import quantized_rank_fine_b200 as q
from tests.helpers import require_gpu
from tests.test_gpu_matvec import _case

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def check(Y, V, x64, A, B, w64, scale=1.0):
    """Y (and V, unless None) against 64 bits, by the tolerance above."""
    K = x64.shape[1]
    fine = 2.0 ** -14 + (K / 16 + 32) * 2.0 ** -22
    y, p2 = x64 @ w64, (x64 ** 2) @ (w64 ** 2)
    if A is not None:
        v = scale * (x64 @ A.double())
        pv2 = scale ** 2 * ((x64 ** 2) @ (A.double() ** 2))
        if V is not None:
            assert torch.isfinite(V).all()
            assert ((V.double() - v).abs() <= 2.0 ** -8 * v.abs() + fine * pv2.sqrt()).all()
        y, p2 = y + v @ B.double(), p2 + (v ** 2 + pv2) @ (B.double() ** 2)
    assert torch.isfinite(Y).all()
    over = (Y.double() - y).abs() / (2.0 ** -8 * y.abs() + fine * p2.sqrt()).clamp(min=1e-300)
    assert over.max() <= 1.0, f"{over.max().item():.2f} times the bound"


@pytest.mark.parametrize("K,N", [(64, 64), (576, 704), (2048, 1024), (2048, 1536), (4096, 1088), (1024, 4160)])
@pytest.mark.parametrize("M", [1, 8, 16])
@pytest.mark.parametrize("x8", [None, 0, 64])
def test_random_values(M, K, N, x8):
    for r in (0, 16):
        w, X, x64, A, B, w64 = _case(M, K, N, r, x8, K + N + M)
        ws = q.Workspace()
        Y, V = q.qlora_matvec(w, X, ws, A, B, save_V=True)
        assert ws.status() == 0
        check(Y, V, x64, A, B, w64)


@pytest.mark.parametrize("K,N", [(128, 256), (256, 8256), (1024, 4096)])
@pytest.mark.parametrize("M", [3, 13])
@pytest.mark.parametrize("x8", [None, 0, 64])
def test_products_that_cancel(M, K, N, x8):
    """Token m sees two rows, a and -a, of the same codes and of scales that are 2^-10
    apart: what is left is 2^-10 of each product, which two terms hold to 2^-15."""
    rng = np.random.default_rng(K + N + M)
    code = rng.integers(0, 16, (K // 2, N)).astype(np.uint8).repeat(2, axis=0)
    s = np.exp(rng.normal(size=(K // 2, N // 16))).astype(np.float32).repeat(2, axis=0)
    s[1::2] *= np.float32(1 + 2.0 ** -10)
    a = rng.integers(8, 16, M) / 8.0          # four bits: a code, and exact in bf16
    x = np.zeros((M, K))
    at = 2 * rng.integers(0, K // 2, M)
    x[np.arange(M), at], x[np.arange(M), at + 1] = a, -a
    xs = np.exp(rng.normal(size=(M, K // x8 if x8 else 1))).astype(np.float32)
    flat = code.reshape(-1, 2)
    w = q.int_weight(torch.from_numpy((flat[:, 0] | (flat[:, 1] << 4)).astype(np.uint8)).cuda(),
                     torch.from_numpy(s.reshape(-1)).cuda(), K, N)
    xt = torch.from_numpy(x).float().cuda()
    if x8 is None:
        X, x64 = xt.to(BF), x
    else:
        X = q.Act8(xt.to(torch.float8_e4m3fn).view(torch.uint8), torch.from_numpy(xs).cuda(), x8)
        x64 = x * xs.astype(np.float64).repeat(K // xs.shape[1], axis=1)
    w64 = (code.astype(np.float64) - 8) * s.astype(np.float64).repeat(16, axis=1)
    y, size = x64 @ w64, np.abs(x64) @ np.abs(w64)
    Y = q.qlora_matvec(w, X, q.Workspace())[0].double().cpu().numpy()
    # two products, each within 2^-16 and an fp32 rounding or two of itself
    assert np.all(np.abs(Y - y) <= 2.0 ** -8 * np.abs(y) + (2.0 ** -16 + 2.0 ** -21) * size)
