"""The binding's serving methods without a GPU: where their outputs are allocated and what they refuse."""
import contextlib

import pytest
import torch

import decode_attention_host_b200 as dkv


def handle(kv_dtype=dkv.DKV_KV_BF16):
    """A DecodeAttention of 4 query heads over 2 kv heads, D = 64, without its library handle."""
    a = object.__new__(dkv.DecodeAttention)
    a.cfg = dkv.DkvConfig(4, 2, 64, 16, kv_dtype, 0.0, 0.0, 8, 8, 0, 0)
    a.handle = None
    return a


class FakeStream:
    cuda_stream = 77
    device = torch.device("cuda", 0)


class OnGpu:
    """What extend reads of a tensor on GPU 0."""

    def __init__(self, n, dtype=torch.int32):
        self.n, self.dtype, self.device, self.is_cuda = n, dtype, torch.device("cuda", 0), True
        self.shape = torch.Size([n])

    def numel(self):
        return self.n

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0


class KV:
    batch, stride, num_kv_heads, head_dim, host_split, num_dev_blocks = 2, 4, 2, 64, 0, 8
    table_dev, seq_lens_dev = OnGpu(8), OnGpu(2)


def test_extend_allocates_its_outputs_on_the_stream_that_writes_them(monkeypatch):
    """torch hands memory out in the order of the stream that is current at the allocation: what a kernel on `stream`
    writes has to come from that stream's memory, or work still queued elsewhere may own it."""
    current, seen, calls = [], [], []

    @contextlib.contextmanager
    def use(s):
        current.append(s)
        yield
        current.pop()

    def empty(*size, **kw):
        seen.append(current[-1] if current else None)
        return OnGpu(size[0], kw["dtype"])

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: FakeStream)
    monkeypatch.setattr(dkv, "dkv_extend_tables", lambda *a: calls.append(a))
    s = FakeStream()
    q_start, slots = handle().extend(KV, OnGpu(2), OnGpu(8), OnGpu(1), 40, stream=s)
    assert seen == [s, s] and calls[0][-1] == 77
    assert (q_start.numel(), slots.numel(), slots.dtype) == (3, 40, torch.int64)
