"""Scratch that a call allocates for itself belongs to the stream it launches
on. (An allocator hands a freed block on in the order of the stream it was
allocated on: a block of another stream may be written by what runs there
while the call's kernels use it.) Streams, allocations and launches are
recorded by fakes; no GPU."""
import contextlib

import pytest
import torch

from hybrid_local_global_b200 import native
from hybrid_local_global_b200.stack import AttentionStack
from hybrid_local_global_b200.workloads import WORKLOADS


class Tensor:
    """What the binding looks at of a CUDA tensor."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, "cuda:0", True

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def numel(self):
        return self.shape.numel()

    nbytes = property(numel)


class Stream:
    cuda_stream = 7
    device = torch.device("cuda", 0)


SIDE = Stream()


@pytest.fixture
def log(monkeypatch):
    """[(what, stream)]: allocations by the stream that is current, launches by theirs."""
    events, current = [], ["current"]

    @contextlib.contextmanager
    def switch(stream):
        current.append(stream)
        try:
            yield
        finally:
            current.pop()

    def empty(*shape, dtype=None, device=None):
        events.append(("alloc", current[-1]))
        return Tensor(*shape, dtype=dtype)

    def launch(*args):
        raw = getattr(args[-1], "value", args[-1])
        events.append(("launch", SIDE if raw == SIDE.cuda_stream else "current"))
        return 0

    monkeypatch.setattr(torch.cuda, "stream", switch)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: type("S", (), {"cuda_stream": 3}))
    monkeypatch.setattr(native, "_raw_stream", lambda index: 3)
    monkeypatch.setattr(native, "_current_device", lambda: 0)
    for f in ("_prefill", "_decode", "_multi", "_prefill_paged", "_decode_paged", "_multi_paged", "_prefill_sinks",
              "_decode_sinks", "_pages_reserve", "_pages_compact"):
        monkeypatch.setattr(native, f, launch)
    return events


def i32(*shape):
    return Tensor(*shape, dtype=torch.int32)


def page_book():
    book = object.__new__(native.PageBook)
    book.n_seqs, book.pages_per_seq, book.n_pages, book.page_size, book._index, book._ref = 2, 3, 7, 128, 0, None
    return book


ROPE = dict(rope_frac=0.25, rope_theta=1e6, scale=0.04)
ROWS, STEP = (2, 16, 8, 512), (2, 8, 512)
NEW, ONE = (2, 16, 1, 512), (2, 1, 512)
POOL, CACHE = (20, 1, 128, 512), (2, 1, 1024, 512)


def calls(stream):
    t = Tensor
    before, lens = dict(seq_lens_before=i32(2)), dict(seq_lens=i32(2), max_seq_len=1000)
    rows = [t(*ROWS), t(*NEW), t(*NEW)]
    step = [t(*STEP), t(*ONE), t(*ONE)]
    pools, caches = [t(*POOL), t(*POOL)], [t(*CACHE), t(*CACHE)]
    table = i32(2, 8)
    kw = dict(ROPE, stream=stream)
    yield "prefill", lambda: native.gemma_attn_prefill(*rows, *caches, window=0, out=t(*ROWS), **before, **kw)
    yield "decode", lambda: native.gemma_attn_decode(*step, *caches, window=0, out=t(*STEP), **lens, **kw)
    yield "multi", lambda: native.gemma_attn_decode_multi(*rows, *caches, window=0, out=t(*ROWS), **lens, **kw)
    yield "prefill_paged", lambda: native.gemma_attn_prefill_paged(*rows, *pools, table, out=t(*ROWS), **before, **kw)
    yield "decode_paged", lambda: native.gemma_attn_decode_paged(*step, *pools, table, out=t(*STEP), **lens, **kw)
    yield "multi_paged", lambda: native.gemma_attn_decode_multi_paged(*rows, *pools, table, out=t(*ROWS), **lens, **kw)
    yield "prefill_sinks", lambda: native.gemma_attn_prefill_sinks(*rows, *pools, table, window=64, sinks=4,
                                                                   out=t(*ROWS), **before, **kw)
    yield "decode_sinks", lambda: native.gemma_attn_decode_sinks(*step, *pools, table, window=64, sinks=4,
                                                                 out=t(*STEP), **lens, **kw)
    yield "reserve", lambda: native.gemma_kv_pages_reserve(page_book(), [], seq_lens=i32(2), new_tokens=i32(2),
                                                           lacking=i32(1), stream=stream)
    yield "compact", lambda: native.gemma_kv_pages_compact(page_book(), [], n_live=i32(1), stream=stream)


NAMES = [name for name, _ in calls(None)]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("stream", [None, SIDE], ids=["current", "side"])
def test_workspace_is_allocated_on_the_stream_of_the_launch(log, name, stream):
    dict(calls(stream))[name]()
    on = stream or "current"
    # a single token under a window plus sinks needs no workspace
    assert log == ([] if name == "decode_sinks" else [("alloc", on)]) + [("launch", on)]


def test_window_workspace_of_a_stack(log, monkeypatch):
    recorded = []
    monkeypatch.setattr(Tensor, "record_stream", lambda self, s: recorded.append(s), raising=False)
    st = AttentionStack(WORKLOADS["31b_verify_b64_k4"], "cpu", alloc_caches=False)
    a = st._window_workspace(3, 1000, SIDE)
    assert log == [("alloc", SIDE)] and recorded == [SIDE]
    assert st._window_workspace(3, 900) is a and len(log) == 1
    assert [getattr(s, "cuda_stream") for s in recorded] == [7, 3]  # used there too, before it may be replaced
    assert st._window_workspace(3, 2000, SIDE) is not a and log[1:] == [("alloc", SIDE)]
