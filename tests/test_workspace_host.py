"""The binding's Workspace: how it grows, what it keeps and gives back (CPU only, with a
stand-in for the library, which would need a device to zero a buffer)."""

import pytest
import torch

import quantized_rank_fine_b200 as q


class FakeLibrary:
    def __init__(self):
        self.inited = []

    def qlora_ws_init(self, ptr, nbytes, stream):
        self.inited.append((ptr, nbytes, stream))
        return 0


@pytest.fixture
def fake(monkeypatch):
    lib = FakeLibrary()
    monkeypatch.setattr(q, "lib", lambda: lib)
    return lib


def held(ws):
    return ws.buf.numel() + sum(b.numel() for b in ws.outgrown)


def test_first_buffer_has_the_size_asked_for(fake):
    ws = q.Workspace("cpu")
    assert ws.get(5000, 7).numel() == 5000 and fake.inited == [(ws.buf.data_ptr(), 5000, 7)]
    assert ws.get(100, 7) is ws.buf and ws.get(5000, 7) is ws.buf and len(fake.inited) == 1
    assert q.Workspace("cpu").get(1, 7).numel() == 256


def test_outgrown_buffers_are_kept(fake):
    """A captured graph may still write to them."""
    ws = q.Workspace("cpu")
    first = ws.get(1280, 7)
    second = ws.get(100000, 7)
    assert second is not first and any(b is first for b in ws.outgrown)


@pytest.mark.parametrize("step", [1, 256, 4096, 1 << 16])
def test_memory_held_by_a_size_that_creeps_up(fake, step):
    """However the size asked for grows, everything held is below a constant times it."""
    ws = q.Workspace("cpu")
    n = 1280
    for _ in range(400):
        ws.get(n, 7)
        assert ws.buf.numel() >= n
        assert held(ws) <= 4.5 * n + 2048
        n += step


def test_release(fake):
    ws = q.Workspace("cpu")
    ws.get(1280, 7)
    ws.get(5000, 7)
    newest = ws.get(50000, 7)
    assert len(ws.outgrown) == 2
    ws.release_outgrown()
    assert ws.outgrown == [] and ws.get(50000, 7) is newest
    q.Workspace("cpu").release_outgrown()
