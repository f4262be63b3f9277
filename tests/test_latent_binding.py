"""Latent attention: what the Python layer refuses before the library is called, on tensors that only
claim a device (CPU only: nothing is launched)."""
import contextlib

import pytest
import torch

import sparse_paged_attention_gb300 as spa


class OnDevice(torch.Tensor):
    """A host tensor that says it is on GPU `index`."""
    index = 0

    def get_device(self):
        return self.index

    def record_stream(self, stream):
        pass


class OnOtherDevice(OnDevice):
    index = 1


def claim(t, cls=OnDevice):
    return t.as_subclass(cls)


def zeros(*shape, dtype=torch.bfloat16):
    return claim(torch.zeros(shape, dtype=dtype))


def pools(block_table):
    return (spa.LatentPool(zeros(4, 8, 80), block_table, 16),
            spa.LatentPool(zeros(4, 8, 96, dtype=torch.uint8), block_table, 16,
                           zeros(32, dtype=torch.float32)))


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    """The library is not there to be called."""
    monkeypatch.setattr(spa, "load_library", lambda: None)


@pytest.mark.parametrize("where", ["host", "another GPU"])
def test_block_table_elsewhere_is_refused(where):
    bt = torch.zeros((1, 4), dtype=torch.int32)
    if where != "host":
        bt = claim(bt, OnOtherDevice)
    pos = zeros(3, dtype=torch.int32)
    bf16, e4m3 = pools(bt)
    for pool, write, read, decode in (
            (bf16, spa.sparse_attn_latent_write, spa.sparse_attn_latent_read, spa.sparse_attn_latent_decode),
            (e4m3, spa.sparse_attn_latent_write_fp8, spa.sparse_attn_latent_read_fp8,
             spa.sparse_attn_latent_decode_fp8)):
        with pytest.raises(ValueError, match="block_table"):
            write(zeros(3, 64), zeros(3, 16), pos, pool)
        with pytest.raises(ValueError, match="block_table"):
            read(pos, pool)
        with pytest.raises(ValueError, match="block_table"):
            decode(zeros(3, 2, 64), zeros(3, 2, 16), pool, pos, scale=1.0)
        with pytest.raises(ValueError, match="block_table"):
            spa.bind_latent_decode(zeros(3, 2, 64), zeros(3, 2, 16), pool, pos, scale=1.0,
                                   fp8=pool is e4m3)
        with pytest.raises(ValueError, match="block_table"):
            spa.sparse_attn_latent_decode_workspace_size(zeros(3, 2, 64), pool, pos, fp8=pool is e4m3)


class FakeLibrary:
    """Entry points that note the stream they are called on (their last argument)."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*args):
            self.streams.append(args[-1])
            return 0
        call.__name__ = name
        return (lambda *_: 4096) if name.endswith("workspace_size") else call


@pytest.fixture
def device(monkeypatch):
    """One GPU whose current stream is 7; notes the stream that every torch.empty is made on."""
    lib, now, made = FakeLibrary(), [7], []
    empty = torch.empty

    class Stream:
        def __init__(self, handle, device=None):
            self.cuda_stream = handle

    @contextlib.contextmanager
    def on(stream):
        now.append(stream.cuda_stream)
        yield
        now.pop()

    def note_empty(*args, device=None, **kw):
        made.append(now[-1])
        return claim(empty(*args, **kw))
    monkeypatch.setattr(spa, "load_library", lambda: lib)
    monkeypatch.setattr(torch, "empty", note_empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(now[-1]))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: now[-1], raising=False)
    return lib, made, Stream


@pytest.mark.parametrize("given", [None, 7, 9, "object", 0])
def test_memory_comes_from_the_stream_of_the_call(device, given):
    """out and workspace of a call on another stream than the current one are that stream's memory."""
    lib, made, Stream = device
    stream = Stream(9) if given == "object" else given
    want = 7 if given is None else 9 if given == "object" else given
    bt, pos = zeros(1, 4, dtype=torch.int32), zeros(3, dtype=torch.int32)
    cu = zeros(2, dtype=torch.int32)
    for pool, suffix in zip(pools(bt), ("", "_fp8")):
        getattr(spa, "sparse_attn_latent_read" + suffix)(pos, pool, stream=stream)
        assert made == [want]
        getattr(spa, "sparse_attn_latent_decode" + suffix)(zeros(3, 2, 64), zeros(3, 2, 16), pool, pos,
                                                           scale=1.0, stream=stream)
        assert made == [want] * 3                    # out and workspace
        spa.bind_latent_decode(zeros(3, 2, 64), zeros(3, 2, 16), pool, pos, scale=1.0, fp8=bool(suffix),
                               stream=stream)()
        assert made == [want] * 5
        made.clear()
    spa.sparse_attn_latent_prefill(zeros(3, 2, 24), zeros(3, 2, 16), zeros(3, 8), zeros(3, 2, 16), cu, cu,
                                   scale=1.0, stream=stream)
    assert made == [want] and lib.streams == [want] * 7


def test_workspaces_with_gaps_or_repeats_are_refused(device):
    """The bytes of a workspace are counted from its address on, which only holds for contiguous ones."""
    bt, pos = zeros(1, 4, dtype=torch.int32), zeros(3, dtype=torch.int32)
    paged = spa.PagedPool(zeros(4, 8, 2, 64), bt)
    topk = zeros(3, 8, dtype=torch.int32)
    for ws in (zeros(1, dtype=torch.uint8).expand(4096), zeros(8192, dtype=torch.uint8)[::2]):
        for pool, suffix in zip(pools(bt), ("", "_fp8")):
            args = (zeros(3, 2, 64), zeros(3, 2, 16), pool, pos)
            with pytest.raises(ValueError, match="workspace"):
                getattr(spa, "sparse_attn_latent_decode" + suffix)(*args, scale=1.0, workspace=ws)
            with pytest.raises(ValueError, match="workspace"):
                spa.bind_latent_decode(*args, scale=1.0, workspace=ws, fp8=bool(suffix))
        for decode in (spa.sparse_attn_paged_decode, spa.bind_decode):
            with pytest.raises(ValueError, match="workspace"):
                decode(zeros(3, 2, 64), paged, None, topk, pos, window=16, ratio=4, scale=1.0, workspace=ws)


def test_bound_call_on_another_device_is_refused(device, monkeypatch):
    """A bound call goes to the current device's stream, so its tensors have to be there."""
    lib, _, _ = device
    bt, pos = zeros(1, 4, dtype=torch.int32), zeros(3, dtype=torch.int32)
    for fp8, pool in enumerate(pools(bt)):
        call = spa.bind_latent_decode(zeros(3, 2, 64), zeros(3, 2, 16), pool, pos, scale=1.0, fp8=bool(fp8))
        call()
        assert len(lib.streams) == fp8 + 1
        with monkeypatch.context() as m:
            m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
            with pytest.raises(ValueError, match="current device"):
                call()
        assert len(lib.streams) == fp8 + 1
