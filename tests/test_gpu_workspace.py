"""The binding's Workspace on the device: the status of buffers that it outgrew."""

import pytest

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
