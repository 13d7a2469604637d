"""Host-side refusals of the norm, dropout and matrix-vector calls: every case
fails its argument check before any device access (CPU only)."""

import ctypes
import os

import pytest

import quantized_rank_fine_b200 as q

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced
INVALID, SHAPE, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(q.LIB_PATH):
        from quantized_rank_fine_b200 import build
        build.build()
    return q.lib()


def _drop(p, counter=None):
    return ctypes.byref(q._Dropout(p, 1, 2, counter))


def _fwd(L, X=FAKE, R=FAKE, G=FAKE, gd=0, eps=1e-5, M=4, n=128, drop=None, H=FAKE, Y=FAKE, Q=None, qs=None, block=0,
         rstd=None):
    return L.qlora_rmsnorm_fwd(X, R, G, gd, eps, M, n, drop, H, Y, Q, qs, block, rstd, None)


@pytest.mark.parametrize("kw,want", [
    (dict(X=None), INVALID), (dict(G=None), INVALID), (dict(gd=2), INVALID), (dict(gd=-1), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1e-5), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(Y=None), INVALID), (dict(Q=FAKE), INVALID),
    (dict(Q=FAKE, qs=FAKE, block=32), INVALID), (dict(Q=FAKE, qs=FAKE, block=-1), INVALID),
    (dict(M=0), SHAPE), (dict(M=-3), SHAPE), (dict(M=1 << 31), SHAPE), (dict(n=0), SHAPE), (dict(n=12), SHAPE),
    (dict(n=65544), SHAPE), (dict(n=72, Q=FAKE, qs=FAKE, block=64), SHAPE),
])
def test_rmsnorm_fwd_rejects(L, kw, want):
    assert _fwd(L, **kw) == want


@pytest.mark.parametrize("p", [1.0, 1.5, -0.25, float("nan"), float("inf")])
def test_dropout_probability_rejected(L, p):
    assert _fwd(L, drop=_drop(p)) == INVALID
    assert L.qlora_dropout_mask(_drop(p), 4, 8, FAKE, None) == INVALID
    assert _bwd(L, drop=_drop(p), dX=FAKE) == INVALID
    w = q._Weight(0x10000, 0x10000, 0x10000, 256, 256)
    o = q._LinearOpts(1.0, q.QLORA_DROPOUT_COUNTER, None, 0.0, q._Dropout(p, 1, 2, None))
    assert L.qlora_linear_fwd_ex(ctypes.byref(w), FAKE, 64, FAKE, FAKE, 8, FAKE, None, ctypes.byref(o), FAKE, 1 << 30,
                                 None) == INVALID


def _bwd(L, dY=FAKE, H=FAKE, G=FAKE, gd=1, rstd=FAKE, dH=None, M=4, n=128, drop=None, dR=FAKE, dX=None, dG=FAKE,
         flags=0, ws=FAKE, nb=1 << 30):
    return L.qlora_rmsnorm_bwd(dY, H, G, gd, rstd, dH, M, n, drop, dR, dX, dG, flags, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dY=None), INVALID), (dict(H=None), INVALID), (dict(G=None), INVALID), (dict(gd=7), INVALID),
    (dict(rstd=None), INVALID), (dict(dR=None), INVALID), (dict(flags=2), INVALID), (dict(dX=FAKE), INVALID),
    (dict(M=0), SHAPE), (dict(n=20), SHAPE), (dict(ws=None), WORKSPACE), (dict(nb=1280), WORKSPACE),
])
def test_rmsnorm_bwd_rejects(L, kw, want):
    assert _bwd(L, **kw) == want


def test_dropout_without_probability_is_none(L):
    """p = 0 is no dropout, so a dX of its own is refused as without one."""
    assert _bwd(L, drop=_drop(0.0), dX=FAKE) == INVALID


def test_rmsnorm_ws_bytes(L):
    assert L.qlora_rmsnorm_ws_bytes(0, 128) == 0 and L.qlora_rmsnorm_ws_bytes(4, 100) == 0
    nb = L.qlora_rmsnorm_ws_bytes(4, 128)
    assert nb > 1280
    assert _bwd(L, nb=nb - 1) == WORKSPACE


def _mv(L, w=None, X=FAKE, xs=None, block=0, M=4, A=FAKE, B=FAKE, r=8, s=1.0, Y=FAKE, V=None,
        ws=FAKE, nb=1 << 30):
    w = w or q._Weight(0x10000, 0, 0x10000, 256, 128, q.QLORA_FMT_INT16)
    return L.qlora_matvec(ctypes.byref(w), X, xs, block, M, A, B, r, s, Y, V, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(X=None), INVALID), (dict(Y=None), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID),
    (dict(r=0), INVALID), (dict(r=0, A=None, B=None, V=FAKE), INVALID), (dict(s=float("nan")), INVALID),
    (dict(xs=FAKE, block=32), INVALID), (dict(w=q._Weight(0x10000, 0x10000, 0x10000, 256, 128, 0)), INVALID),
    (dict(M=0), SHAPE), (dict(M=17), SHAPE), (dict(r=4), SHAPE), (dict(r=12), SHAPE), (dict(r=264), SHAPE),
    (dict(w=q._Weight(0x10000, 0, 0x10000, 256, 96, 2)), SHAPE), (dict(w=q._Weight(0x10000, 0, 0x10000, 32, 64, 2)), SHAPE),
    (dict(ws=None), WORKSPACE), (dict(nb=1279), WORKSPACE),
])
def test_matvec_rejects(L, kw, want):
    assert _mv(L, **kw) == want


def test_counter_option_excludes_a_stored_mask(L):
    w = q._Weight(0x10000, 0x10000, 0x10000, 256, 256)
    o = q._LinearOpts(1.0, q.QLORA_DROPOUT_COUNTER, FAKE, 0.1, q._Dropout(0.1, 1, 2, None))
    args = (FAKE, 64, FAKE, FAKE, 8, FAKE, None, ctypes.byref(o), FAKE, 1 << 30, None)
    assert L.qlora_linear_fwd_ex(ctypes.byref(w), *args) == INVALID
    # without the flag the member is not read
    o = q._LinearOpts(1.0, 0, None, 0.0, q._Dropout(7.0, 1, 2, None))
    assert L.qlora_linear_fwd_ex(ctypes.byref(w), FAKE, 64, FAKE, FAKE, 12, FAKE, None, ctypes.byref(o), FAKE, 1 << 30,
                                 None) == SHAPE


def test_dropout_mask_shape(L):
    assert L.qlora_dropout_mask(_drop(0.5), 0, 8, FAKE, None) == SHAPE
    assert L.qlora_dropout_mask(_drop(0.5), 1 << 21, 1 << 20, FAKE, None) == SHAPE
    assert L.qlora_dropout_mask(None, 1, 8, FAKE, None) == INVALID


def test_binding_checks_shapes_and_types():
    """The binding refuses tensors of another shape or type before it allocates."""
    import torch
    bf, f32 = torch.bfloat16, torch.float32
    x, g = torch.zeros(4, 64, dtype=bf), torch.ones(64, dtype=bf)
    ws = q.Workspace("cpu")
    for bad in (dict(residual=torch.zeros(3, 64, dtype=bf)), dict(residual=torch.zeros(4, 64)),
                dict(H=torch.zeros(4, 72, dtype=bf)), dict(Y=torch.zeros(4, 64, dtype=f32))):
        with pytest.raises(ValueError):
            q.qlora_rmsnorm_fwd(x, g, **bad)
    with pytest.raises(ValueError):
        q.qlora_rmsnorm_fwd(x.float(), g)
    with pytest.raises(ValueError):
        q.qlora_rmsnorm_fwd(x, g[:32])
    with pytest.raises(ValueError):
        q.qlora_rmsnorm_fwd(x, g.half())
    for bad in (dict(dH=torch.zeros(4, 8, dtype=bf)), dict(dG=torch.zeros(64, dtype=bf)), dict(dG=torch.zeros(32))):
        with pytest.raises(ValueError):
            q.qlora_rmsnorm_bwd(x, x, g, torch.ones(4), ws, **bad)
    with pytest.raises(ValueError):
        q.qlora_rmsnorm_bwd(x, x, g, torch.ones(4), ws, accumulate=True)
    w = q.int_weight(torch.zeros(64 * 64, dtype=torch.uint8), torch.zeros(64 * 8), 64, 128)
    for X in (torch.zeros(4, 128, dtype=bf), torch.zeros(4, 64), q.Act8(torch.zeros(4, 64, dtype=bf), torch.ones(4, 1)),
              q.Act8(torch.zeros(4, 64, dtype=torch.uint8), torch.ones(4, 2)),
              q.Act8(torch.zeros(4, 64, dtype=torch.uint8), torch.ones(4, 1), 32)):
        with pytest.raises(ValueError):
            q.qlora_matvec(w, X, ws)
    with pytest.raises(ValueError):
        q.qlora_matvec(w, x, ws, torch.zeros(64, 8, dtype=bf), torch.zeros(8, 64, dtype=bf))
    for d in (q.Dropout(0.1, -1), q.Dropout(0.1, 1 << 64), q.Dropout(0.1, 0, -1),
              q.Dropout(0.1, 0, 0, torch.zeros(1, dtype=torch.int32)), q.Dropout(0.1, 0, 0, torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            d.c_struct()
