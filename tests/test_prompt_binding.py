"""The binding of the prompt chunk's entry points: what it passes on to the library.  No GPU: host tensors that say they are on
device 0, and a library that only takes down its arguments."""
import contextlib
import threading

import pytest
import torch

import gated_delta_rule_16_gb300 as gdn
from gated_delta_rule_16_gb300 import _binding, paged, prompt
from test_paged_binding import Library, Stream, decode, empty, fake  # noqa: F401


class PromptLibrary(Library):
    """Workspaces of 1000 bytes per row; a call's status is what `status` says at its address."""

    def __init__(self):
        super().__init__()
        self.status = {}

    def gdn_paged_prefill_workspace_bytes(self, cache, B, n, heads):
        return 1000 * n

    def gdn_paged_prefill(self, *args):
        self.calls.append(args)
        return 0

    def gdn_paged_prefill_status(self, address, stream):
        return self.status.get((address, stream), 0)


@pytest.fixture
def lib(fake, monkeypatch):  # noqa: F811
    monkeypatch.setattr(paged, "_local", paged._Local())
    monkeypatch.setattr(prompt, "_ws_bytes", {})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    return fake(PromptLibrary())


def prefill(n=3, **kw):
    cache = empty((3, 16, 2, 64), torch.bfloat16)
    return gdn.gdn_paged_prefill(empty((n, 4, 64), torch.bfloat16), cache, cache, empty((1, 3), torch.int32), empty((1,), torch.int32),
                                 empty((2,), torch.int32), **kw)


def test_status_of_a_call_without_a_workspace(lib):
    with pytest.raises(ValueError, match="no call"):
        gdn.gdn_paged_prefill_status()
    prefill()
    first = lib.calls[-1][-3]
    assert gdn.gdn_paged_prefill_status() == 0
    lib.status[first, 7] = 10
    assert gdn.gdn_paged_prefill_status() == 10
    decode()  # whose workspace is another: the status is still of the call that it belongs to
    assert lib.calls[-1][-3] != first and gdn.gdn_paged_prefill_status() == 10
    prefill(n=50)  # a larger one: the status is the last call's
    assert lib.calls[-1][-3] != first and lib.calls[-1][-2] >= 50000
    assert gdn.gdn_paged_prefill_status() == 0
    with pytest.raises(ValueError, match="no call"):
        gdn.gdn_paged_prefill_status(stream=Stream(9))  # no call of this stream's
    with pytest.raises(ValueError, match="no call"):
        gdn.gdn_paged_prefill_status(gdn.Workspace())


def test_status_of_a_call_without_a_workspace_is_the_threads_own(lib):
    prefill()
    lib.status[lib.calls[-1][-3], 7] = 10
    got = []

    def other():
        with pytest.raises(ValueError, match="no call"):
            gdn.gdn_paged_prefill_status()
        prefill()
        got.append(gdn.gdn_paged_prefill_status())
    t = threading.Thread(target=other)
    t.start()
    t.join()
    assert got == [0] and gdn.gdn_paged_prefill_status() == 10
    assert _binding._lib is lib
