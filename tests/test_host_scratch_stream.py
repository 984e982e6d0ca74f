"""A workspace that the bindings allocate belongs to the stream of the call: on the
host, with the library, the allocator and torch's stream context replaced by fakes
that record what they are asked for."""

import contextlib
import types

import pytest
import torch

from paged_kv_attention_17_gb300 import _binding as B


class Recorder:
    """Which stream was current when each workspace was allocated, and the streams
    and workspaces that the library was called with."""

    def __init__(self, monkeypatch):
        self.current, self.allocated, self.calls = 0x1000, [], []
        empty = torch.empty

        def fake_empty(*size, dtype=None, device=None):
            t = empty(*size, dtype=dtype)
            if dtype == torch.uint8:
                self.allocated.append((t.data_ptr(), self.current))
            return t

        @contextlib.contextmanager
        def fake_context(stream):
            before, self.current = self.current, stream.cuda_stream
            yield
            self.current = before

        def stream_of(handle):
            return types.SimpleNamespace(cuda_stream=handle)

        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(torch, "empty", fake_empty)
        monkeypatch.setattr(torch.cuda, "stream", fake_context)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream_of(self.current))
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: stream_of(0))
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: stream_of(handle))
        monkeypatch.setattr(B, "lib", lambda: self)
        monkeypatch.setattr(B, "_device_and_stream", lambda cache, stream: (
            0, self.current if stream is None else getattr(stream, "cuda_stream", stream)))
        monkeypatch.setattr(B, "_calls", types.SimpleNamespace(attention=self.e2m1))
        for name in ("pkv_attention_varlen_e2m1", "pkv_write_attention_varlen_e2m1"):
            monkeypatch.setitem(B._address, name, 1)

    def e2m1(self, *a):
        self.calls.append((a[-6].data_ptr(), a[-1]))
        return 0

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 4096
        if name.endswith("splits") or name.endswith("splits_e2m1"):
            return lambda *a: 3

        def call(*a):
            # the stream is last; the workspace pointer is followed by its 4096 bytes
            at = max(i for i, x in enumerate(a) if isinstance(x, int) and x == 4096) - 1
            self.calls.append((a[at].value, a[-1].value or 0))
            return 0
        return call


def run(name, stream):
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    new = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    slots = torch.zeros(2, dtype=torch.int64)
    codes = torch.zeros(4, 16, 2, 128, dtype=torch.uint8)
    pages = torch.zeros(4, 2, 9 * 128, dtype=torch.uint8)
    plain = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    qsl, lens = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 2, dtype=torch.int32)
    cache = codes if "e4m3" in name else pages if "e2m1" in name else plain
    f = getattr(B, name.split("/")[0])
    if "cascade" in name:
        scales = (0.5, 0.5) if "e4m3" in name else None
        f(q, cache, cache, q, qsl, lens, table, table[0], 1, 32, 0.1, kv_scales=scales, stream=stream)
        return
    args = [q, cache, cache, q, qsl, lens, table, 1, 32, 0.1]
    if "write" in name:
        args = [new, new, slots] + args
    if "e4m3" in name or "e2m1" in name:
        args += [0.5, 0.5]
    f(*args, stream=stream, **({"window": 20} if "window" in name else {}))


NAMES = ["pkv_attention_varlen", "pkv_attention_varlen/window", "pkv_write_attention_varlen",
         "pkv_attention_varlen_e4m3", "pkv_attention_varlen_e4m3/window",
         "pkv_write_attention_varlen_e4m3", "pkv_cascade_attention", "pkv_cascade_attention/e4m3",
         "pkv_attention_varlen_e2m1", "pkv_write_attention_varlen_e2m1"]


@pytest.mark.parametrize("stream", [None, 0x1000, 0x2000, 0, 2, types.SimpleNamespace(cuda_stream=0x3000)])
@pytest.mark.parametrize("name", NAMES)
def test_the_workspace_belongs_to_the_stream_of_the_call(monkeypatch, name, stream):
    r = Recorder(monkeypatch)
    run(name, stream)
    want = 0x1000 if stream is None else getattr(stream, "cuda_stream", stream)
    assert len(r.calls) == 1 and len(r.allocated) == 1
    (pointer, launched), (allocated, owner) = r.calls[0], r.allocated[0]
    assert launched == want
    assert pointer == allocated
    assert owner == want
    assert r.current == 0x1000
