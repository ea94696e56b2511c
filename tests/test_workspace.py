"""The binding's workspaces and streams, as far as that goes without a GPU."""
from types import SimpleNamespace

import pytest
import torch

import dynamic_block_sparse_shape_b200 as P


@pytest.fixture
def dirty(monkeypatch):
    """Fresh memory that is not zero."""
    made = torch.empty

    def empty(*a, **k):
        t = made(*a, **k)
        return t.fill_(171) if t.dtype == torch.uint8 else t

    monkeypatch.setattr(torch, "empty", empty)


@pytest.mark.parametrize("nbytes", [1, 256, 257, 100000])
def test_only_the_status_word_is_cleared(dirty, nbytes):
    """The calls write the rest before they read it; clearing all of it would cost as much as some of them."""
    ws = P.Workspace("cpu", nbytes)
    for need in (nbytes, nbytes + 5000):
        ws.ensure(need)
        assert ws.ptr.value % 256 == 0 and ws.nbytes >= max(need, 256)
        at = ws.ptr.value - ws.buf.data_ptr()
        head, rest = ws.buf[at:at + 256], torch.cat((ws.buf[:at], ws.buf[at + 256:]))
        assert (head == 0).all() and (rest == 171).all()


def test_a_buffer_is_kept_until_it_is_too_small():
    ws = P.Workspace("cpu", 5000)
    first = ws.buf
    ws.buf[-1] = 9
    for need in (1, 4999, 5000):
        assert ws.ensure(need).buf is first and ws.nbytes >= need
    assert ws.ensure(5001).buf is not first and ws.kept == []
    ws.captured = True  # as a stream capture leaves it
    held = ws.buf
    ws.ensure(1 << 20)
    assert ws.kept[0] is held and not ws.captured


def test_a_workspace_of_another_device_is_refused():
    call = object.__new__(P._On)
    call.device = 0
    with pytest.raises(P.PrismError) as e:
        call.workspace(P.Workspace("cpu"), 1024, "a call")
    assert e.value.status == 4


def test_a_stream_of_another_device_is_refused():
    """Also when both are the default stream, whose handle is the same on every device."""
    tensor, stream = SimpleNamespace(get_device=lambda: 0), SimpleNamespace(device_index=1, cuda_stream=0)
    with pytest.raises(P.PrismError, match="another device"):
        P._On([tensor], stream, "a call")


def test_refusals_of_kept_status():
    """Host checks of the status calls, before any CUDA call."""
    from dynamic_block_sparse_shape_b200 import build
    build.build()
    assert P.lib().prism_clear_device_status(None, None) == 4
    assert P.lib().prism_clear_device_status(8, None) == 4
    assert P.lib().prism_keep_device_status(None, None) == 4
    assert P.lib().prism_check_kept_status(None, None) == 4
    assert P.lib().prism_check_kept_status(8, None) == 4
