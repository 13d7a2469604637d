"""Pins of the norm / dropout oracle against something other than itself: the
generator's published known-answer vectors, bf16 rounding against torch, the norm
against a library routine, gradients against differences."""

import numpy as np
import pytest
import torch

from oracle import norm


@pytest.mark.parametrize("ctr,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(ctr, key, want):
    """The known-answer vectors published with the generator."""
    assert tuple(norm.philox4x32_10(ctr, key)) == want


def test_words_are_the_blocks():
    seed, off = 0x299F31D0A4093822, 0x0370734413198A2E
    w = norm.words(seed, off, 5, 30)
    for i in range(30):
        e = 5 + i
        blk = norm.philox4x32_10((e // 4, 0, off & 0xFFFFFFFF, off >> 32), (seed & 0xFFFFFFFF, seed >> 32))
        assert int(w[i]) == blk[e % 4]
    first = (1 << 34) + 6     # a counter past 32 bits
    blk = norm.philox4x32_10(((first // 4) & 0xFFFFFFFF, first // 4 >> 32, 9, 0), (7, 0))
    assert norm.words(7, 9, first, 2).tolist() == blk[2:4]


def test_keep_mask_share():
    """The kept share is 1 - p within five standard deviations."""
    for p in (0.05, 0.5, 0.9):
        k = norm.keep_mask(p, 3, 1, 512, 512)
        assert abs(k.mean() - (1 - p)) < 5 * np.sqrt(p * (1 - p) / k.size)
    assert norm.keep_mask(0.0, 3, 1, 8, 8).all()


def test_round_bf16_is_one_rounding():
    rng = np.random.default_rng(0)
    x = rng.normal(size=4096).astype(np.float32)
    assert np.array_equal(norm.round_bf16(x), torch.from_numpy(x).bfloat16().double().numpy())
    # just above a tie: through binary32 this would become the tie and go to even
    assert norm.round_bf16(np.array([1.0 + 2.0 ** -8 + 2.0 ** -40]))[0] == 1.0 + 2.0 ** -7
    assert norm.round_bf16(np.array([1.0 + 2.0 ** -8]))[0] == 1.0


def test_rmsnorm_matches_library():
    rng = np.random.default_rng(1)
    x = norm.round_bf16(rng.normal(size=(5, 72)))
    g = rng.normal(size=72)
    _, y, _ = norm.rmsnorm(x, None, g, 1e-5)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (72,), torch.from_numpy(g), eps=float(np.float32(1e-5)))
    assert np.allclose(y, want.numpy(), rtol=1e-12, atol=0)


def test_backward_matches_differences():
    """Central differences of sum(dy y) + sum(dH h) in float64 (without the
    rounding of h), with respect to h and g; step 1e-5, so about 1e-9 off."""
    rng = np.random.default_rng(2)
    M, n, eps, d = 3, 16, float(np.float32(1e-5)), 1e-5
    h, g, dy, dH = rng.normal(size=(M, n)), rng.normal(size=n), rng.normal(size=(M, n)), rng.normal(size=(M, n))

    def loss(h, g):
        return (dy * h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * g).sum() + (dH * h).sum()

    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    keep = rng.random((M, n)) < 0.5
    dx, dh, dg = norm.rmsnorm_backward(dy, h, g, rstd, dH, keep, 0.5)
    for i in range(M):
        for j in range(n):
            e = np.zeros((M, n))
            e[i, j] = d
            assert abs((loss(h + e, g) - loss(h - e, g)) / (2 * d) - dh[i, j]) < 1e-7
    for j in range(n):
        e = np.zeros(n)
        e[j] = d
        assert abs((loss(h, g + e) - loss(h, g - e)) / (2 * d) - dg[j]) < 1e-7
    assert np.array_equal(dx, dh * keep * 2.0)


@pytest.mark.parametrize("block", [0, 64])
def test_quantize_e4m3_is_nearest(block):
    rng = np.random.default_rng(3)
    y = rng.normal(size=(4, 128))
    y[1] = 0.0
    v, s = norm.quantize_e4m3(y, block)
    sc = np.repeat(s, 128 // s.shape[1], axis=1)
    # half a step: 2^-4 of a normal value, 2^-10 below the normals; fl32 roundings on top
    assert np.all(np.abs(v * sc - y) <= (2.0 ** -4 + 2.0 ** -20) * np.abs(y) + sc * 2.0 ** -10)
    assert np.all(v[1] == 0) and np.abs(v).max() == 448.0
