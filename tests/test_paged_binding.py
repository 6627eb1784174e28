"""The binding of the decode-step entry points: what it passes on to the library.  No GPU: host tensors that say they are on
device 0, and a library that only takes down its arguments."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import gated_delta_rule_16_gb300 as gdn
from gated_delta_rule_16_gb300 import _binding, paged


class OnDevice(torch.Tensor):
    def get_device(self):
        return 0


def empty(shape, dtype=torch.float32, device=None):
    return torch.empty(shape, dtype=dtype).as_subclass(OnDevice)


class Library:
    """Workspaces of 1000 bytes per query head; calls wait at `meet`, then are noted."""

    def __init__(self, meet=None):
        self.meet, self.calls = meet, []

    def gdn_paged_decode_workspace_bytes(self, cache, heads):
        return 1000 * heads

    def gdn_paged_decode(self, *args):
        if self.meet:
            self.meet.wait(10)
        self.calls.append(args)
        return 0


@pytest.fixture
def fake(monkeypatch):
    def use(lib, stream=7):
        monkeypatch.setattr(_binding, "_lib", lib)
        monkeypatch.setattr(paged, "_current_device", lambda: 0)
        monkeypatch.setattr(paged, "_current_stream", lambda dev: stream)
        monkeypatch.setattr(paged, "_empty", empty)
        monkeypatch.setattr(paged, "_ws_bytes", {})
        return lib
    return use


def decode(heads=4, **kw):
    cache = empty((3, 16, 2, 64), torch.bfloat16)
    return gdn.gdn_paged_decode(empty((2, heads, 64), torch.bfloat16), cache, cache, empty((2, 3), torch.int32), empty((2,), torch.int32), **kw)


def test_threads_on_one_stream_have_workspaces_of_their_own(fake):
    # a call is two launches, between which another thread's may come: both calls are in the library at once here
    lib = fake(Library(threading.Barrier(2)))
    errors = []

    def run(heads):
        try:
            for _ in range(3):
                decode(heads)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(h,)) for h in (4, 8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    by_heads = {h: {a[-3] for a in lib.calls if a[2] == h} for h in (4, 8)}
    assert len(lib.calls) == 6 and all(a[-2] >= 1000 * a[2] for a in lib.calls)
    assert len(by_heads[4]) == len(by_heads[8]) == 1      # a thread keeps its own from call to call
    assert by_heads[4] != by_heads[8]


class Stream:
    def __init__(self, handle, device_index=0):
        self.cuda_stream, self.device_index = handle, device_index


@pytest.mark.parametrize("op", ["tables", "decode", "sample"])
def test_outputs_and_workspace_are_made_on_the_calls_stream(fake, monkeypatch, op):
    # memory that is free in the current stream's order may still be in use when the call runs on another one
    now, made, recorded = [7], [], []

    class Within:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            self.before, now[0] = now[0], self.stream.cuda_stream

        def __exit__(self, *_):
            now[0] = self.before

    class Noted(Library):
        def gdn_page_tables(self, *args):
            self.calls.append(args)
            return 0

        gdn_sample = gdn_page_tables

    def tracked(shape, dtype=torch.float32, device=None):
        t = empty(shape, dtype)
        made.append((now[0], t.data_ptr()))
        return t

    lib = fake(Noted())
    monkeypatch.setattr(paged, "_current_stream", lambda dev: now[0])
    monkeypatch.setattr(paged, "_empty", tracked)
    monkeypatch.setattr(torch.cuda, "stream", Within)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: Stream(now[0]))
    monkeypatch.setattr(OnDevice, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s.cuda_stream)), raising=False)
    i32 = lambda *shape: empty(shape, torch.int32)
    # one output given, which torch has made for the current stream
    if op == "tables":
        given = i32(4)
        call = lambda s: gdn.gdn_page_tables(i32(2), i32(5), i32(2, 3), page=16, n_slots=4, counts=given, stream=s)
    elif op == "decode":
        given = empty((2, 4))
        call = lambda s: decode(lse=given, stream=s)
    else:
        given = empty((2,))
        call = lambda s: gdn.gdn_sample(empty((2, 9)), empty((2, 9)), logprobs=given, stream=s)
    got = call(Stream(9))
    assert lib.calls[-1][-1] == 9 and now[0] == 7
    assert made and all(stream == 9 for stream, _ in made)
    assert (given.data_ptr(), 9) in recorded
    assert all((t.data_ptr(), 7) in recorded for t in got if t is not given)
    with pytest.raises(ValueError):
        call(Stream(9, device_index=1))
    # the current stream, given or not: nothing to record
    made.clear(), recorded.clear()
    call(None), call(Stream(7))
    assert all(stream == 7 for stream, _ in made) and not recorded and [a[-1] for a in lib.calls[-2:]] == [7, 7]


def test_import_with_a_torch_without_cuda():
    # what such a torch lacks; the calls refuse host tensors before they would need it
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import gated_delta_rule_16_gb300 as gdn\n"
            "try: gdn.gdn_sample(torch.zeros(2, 8), torch.zeros(2, 8))\n"
            "except ValueError as e: print('refused:', e)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0 and "refused: logits must be a CUDA tensor" in r.stdout, r.stderr


def test_status_is_asked_on_the_counts_device(fake, monkeypatch):
    # stream 0 is the current device's: another device's would not wait for the call that writes the counts
    now = [1]

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, now[0] = now[0], self.dev

        def __exit__(self, *_):
            now[0] = self.before

    class Asked(Library):
        def gdn_page_tables_status(self, counts, stream):
            self.calls.append((now[0], stream))
            return 9

    lib = fake(Asked(), stream=0)
    monkeypatch.setattr(paged, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    counts = empty((4,), torch.int32)
    assert gdn.gdn_page_tables_status(counts) == 9
    now[0] = 0
    assert gdn.gdn_page_tables_status(counts) == 9
    assert lib.calls == [(0, 0), (0, 0)] and now[0] == 0
