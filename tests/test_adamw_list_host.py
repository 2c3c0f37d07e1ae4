"""Host checks of the AdamW list's own device table: which stream's memory it
is, on which stream it is written, what is waited for, and which streams' work
keeps the memory.  torch's streams are stood in for, so that the order of the
calls can be looked at without a GPU."""
import contextlib
import types

import pytest
import torch

import token_dispatch_grouped_top_amd as mok


class Stream:
    def __init__(self, handle, gpu=0):
        self.cuda_stream, self.device, self.capturing = handle, torch.device("cuda", gpu), False


class Buffer:
    """A dense tensor on the stand-in's GPU 0, taken from the current stream's memory."""

    def __init__(self, gpu, n, dtype=torch.float32):
        self.gpu, self.n, self.dtype, self.home = gpu, n, dtype, gpu.current
        self.device, self.shape, self.used_on = torch.device("cuda", 0), (n,), []

    def numel(self):
        return self.n

    def stride(self):
        return (1,)

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 20

    def element_size(self):
        return self.dtype.itemsize

    def record_stream(self, stream):
        self.gpu.log.append(("record", self, stream.cuda_stream))
        self.used_on.append(stream.cuda_stream)


class Gpu:
    def __init__(self):
        self.default = self.current = Stream(0)
        self.log, self.device = [], 0

    def tensors(self, count=2):
        return [{name: Buffer(self, 64) for name in ("p", "grad", "m", "v")} for _ in range(count)]

    def did(self, what):
        return [x[1:] for x in self.log if x[0] == what]


@pytest.fixture
def gpu(monkeypatch):
    g = Gpu()

    @contextlib.contextmanager
    def on(stream):
        before, g.current = g.current, stream
        try:
            yield
        finally:
            g.current = before

    def wait(name):
        return lambda self=None, *a: g.log.append((name, self or g.current))

    def external(handle, device=None):
        assert handle != 0                     # torch makes a new stream of a handle of 0
        return Stream(handle)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: g.current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: g.default)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: g.current.capturing)
    monkeypatch.setattr(torch.cuda, "synchronize", wait("synchronize all"))
    monkeypatch.setattr(Stream, "synchronize", wait("synchronize"), raising=False)
    monkeypatch.setattr(torch, "empty", lambda n, dtype=None, device=None: Buffer(g, n, dtype))
    monkeypatch.setattr(mok, "_device", lambda: g.device)
    monkeypatch.setattr(mok, "_stream_of",
                        lambda s, device: g.current.cuda_stream if s is None else s if isinstance(s, int) else s.cuda_stream)
    monkeypatch.setattr(mok, "_stream", lambda s: mok._stream_of(s, 0))
    monkeypatch.setattr(mok, "mok_adamw_build_table",
                        lambda c, table, plan, stream=None: g.log.append(("write", table, mok._stream_of(stream, 0))))
    monkeypatch.setattr(mok, "_lib", types.SimpleNamespace(
        mok_adamw_table_size=mok._lib.mok_adamw_table_size,
        mok_adamw_step=lambda table, plan, hyper, scalars, stream: g.log.append(("step", stream)) or mok.MOK_OK))
    return g


def _step(lst, stream=None):
    mok.mok_adamw_step(lst, 1e-3, 0.9, 0.95, 1e-8, 1, stream=stream)


def _given(g, how):
    """(the argument, the stream it means)"""
    side = Stream(7)
    return {"none": (None, g.current), "object": (side, side), "handle": (9, Stream(9)), "zero": (0, g.default)}[how]


@pytest.mark.parametrize("how", ["none", "object", "handle", "zero"])
@pytest.mark.parametrize("current", [0, 5])
def test_table_is_memory_of_the_stream_that_writes_it(gpu, how, current):
    """Else work still pending on the current stream, in whose memory the block was before, could write over it."""
    gpu.current = gpu.default if current == 0 else Stream(current)
    argument, stream = _given(gpu, how)
    before = gpu.current
    lst = mok.AdamwTensors(gpu.tensors(), stream=argument)
    (table, written_on), = gpu.did("write")
    assert table is lst.table
    assert table.home.cuda_stream == written_on == stream.cuda_stream
    # that stream alone is waited for, behind the writing
    (waited,), = gpu.did("synchronize")
    assert waited.cuda_stream == stream.cuda_stream and not gpu.did("synchronize all")
    assert [x[0] for x in gpu.log if x[0] != "record"] == ["write", "synchronize"]
    assert gpu.current is before


def test_memory_is_kept_for_steps_on_other_streams(gpu):
    """A list that is dropped while a step runs on a side stream: its table's memory and its tensors' are not given out
    again before that step is done."""
    ts = gpu.tensors(3)
    lst = mok.AdamwTensors(ts)
    _step(lst)
    assert not gpu.did("record") or all(s == 0 for _, s in gpu.did("record"))   # nothing to do on their own stream
    for argument, handle in ((Stream(7), 7), (9, 9), (Stream(7), 7), (9, 9)):
        gpu.log.clear()
        first = handle not in lst.table.used_on
        _step(lst, argument)
        assert [x for x in gpu.log if x[0] == "step"] == [("step", handle)]
        assert lst.table.used_on.count(handle) == 1                         # once for each stream is enough
        assert bool(gpu.did("record")) == first
        for t in ts:
            assert all(x.used_on.count(handle) == 1 for x in t.values())
    gpu.current = Stream(11)                                                # the current stream, another than at the building
    _step(lst)
    assert 11 in lst.table.used_on and all(11 in x.used_on for t in ts for x in t.values())
    gpu.current = gpu.default
    _step(lst, 0)
    assert gpu.did("step")[-1] == (0,)


def test_table_of_a_side_stream_is_kept_for_steps_on_the_current_one(gpu):
    lst = mok.AdamwTensors(gpu.tensors(), stream=Stream(7))
    _step(lst)
    assert lst.table.home.cuda_stream == 7 and 0 in lst.table.used_on
    _step(lst, Stream(7))
    assert all(7 in x.used_on for t in lst.tensors for x in t.values())     # theirs is the current stream's memory


def test_a_stream_that_is_captured_is_not_waited_for(gpu):
    """Neither is the GPU: what counts is the stream that is written on, not the current one."""
    side = Stream(7)
    side.capturing = True
    mok.AdamwTensors(gpu.tensors(), stream=side)
    assert gpu.did("write") and not gpu.did("synchronize") and not gpu.did("synchronize all")
    gpu.log.clear()
    gpu.current = side
    mok.AdamwTensors(gpu.tensors())
    assert gpu.did("write") and not gpu.did("synchronize") and not gpu.did("synchronize all")


def test_writing_beside_a_capture_is_refused(gpu):
    """Waiting for another stream would end the current stream's capture; not waiting would leave the captured steps
    without a table."""
    gpu.current = Stream(5)
    gpu.current.capturing = True
    with pytest.raises(ValueError, match="stream.*captur"):
        mok.AdamwTensors(gpu.tensors(), stream=Stream(7))
    assert not gpu.log and gpu.current.cuda_stream == 5


def test_step_of_a_list_on_another_gpu_is_refused(gpu):
    lst = mok.AdamwTensors(gpu.tensors())
    gpu.device = 1
    with pytest.raises(ValueError, match="list.*current GPU"):
        _step(lst)
    assert not gpu.did("step")
    gpu.device = 0
    _step(lst)
    assert gpu.did("step") == [(0,)]


def test_building_on_a_stream_of_another_gpu_is_refused(gpu):
    with pytest.raises(ValueError, match="stream.*current GPU"):
        mok.AdamwTensors(gpu.tensors(), stream=Stream(7, gpu=1))
    assert not gpu.log


def test_an_empty_list_has_nothing_to_keep(gpu):
    lst = mok.AdamwTensors([])
    _step(lst, Stream(7))
    assert gpu.did("step") == [(7,)] and not gpu.did("record")


def test_an_empty_list_needs_no_gpu():
    mok.mok_adamw_step(mok.AdamwTensors([]), 1e-3, 0.9, 0.95, 1e-8, 1, stream=0)
