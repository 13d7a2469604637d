"""The binding's Workspace on the device: the status of buffers that it outgrew, and the
stream that a new one belongs to."""

import pytest
import torch

import quantized_rank_fine_b200 as q
from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu

QLORA_ERR_TIMEOUT = 7


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("kind", [0, 1])
def test_timeout_in_an_outgrown_buffer_is_reported(kind):
    """A wait gives up on a buffer that the workspace has outgrown by the time that the
    status is read; reading clears it there too."""
    ws = q.Workspace()
    q.qlora_selftest_wait_timeout(ws, kind, limit_us=50)
    ws.get(4 * ws.buf.numel())
    ws.get(16 * ws.buf.numel())
    assert len(ws.outgrown) == 2
    assert ws.status() == QLORA_ERR_TIMEOUT
    assert ws.status() == 0


def test_timeouts_in_several_buffers_are_read_at_once():
    ws = q.Workspace()
    for _ in range(3):
        q.qlora_selftest_wait_timeout(ws, 0, limit_us=50)
        ws.get(2 * ws.buf.numel())
    assert ws.status() == QLORA_ERR_TIMEOUT
    assert ws.status() == 0


def test_new_buffer_belongs_to_the_stream_of_the_call():
    """A buffer first asked for by a call on another stream is not memory that the current
    stream, still busy, has only just let go of: it stays zero."""
    n = 1 << 20
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        old = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda._sleep(20_000_000)          # about 10 ms
        for t in old:
            t.fill_(0xFF)
        t = None
        old.clear()
        ws = q.Workspace()
        ws.get(n, side)
        torch.cuda.synchronize()
        assert torch.count_nonzero(ws.buf) == 0
