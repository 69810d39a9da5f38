"""The binding's serving methods without a GPU: where their outputs are allocated and what they refuse."""
import contextlib
from types import SimpleNamespace

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
    k_host = v_host = SimpleNamespace(ptr=0)
    k_dev = v_dev = OnGpu(8)


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


def tensors(dtype=torch.bfloat16):
    """Arguments that fit the handle and the cache, but for where they lie: CPU memory."""
    rows, batch = 5, KV.batch
    return dict(q16=torch.zeros((rows, 4, 64), dtype=dtype), out16=torch.zeros((rows, 4, 64), dtype=dtype),
                q32=torch.zeros((batch, 4, 64)), out32=torch.zeros((batch, 4, 64)),
                k=torch.zeros((rows, 2, 64), dtype=dtype), v=torch.zeros((rows, 2, 64), dtype=dtype),
                slots=torch.zeros(rows, dtype=torch.int64), q_start=torch.zeros(batch + 1, dtype=torch.int32),
                new=torch.zeros(batch, dtype=torch.int32), ids=torch.zeros(8, dtype=torch.int32),
                count=torch.zeros(1, dtype=torch.int32))


def call(name, t, kv=KV, a=None):
    a = a or handle()
    s = FakeStream()
    if name == "window":
        a.window(t["q32"], kv, t["out32"], 4, stream=s)
    elif name == "chunk":
        a.chunk(t["q16"], t["q_start"], kv, t["out16"], stream=s, k_stage=t.get("k_stage"), v_stage=t.get("v_stage"))
    elif name == "store":
        a.store(t["k"], t["v"], t["slots"], kv, stream=s)
    else:
        a.extend(kv, t["new"], t["ids"], t["count"], 8, stream=s)


@pytest.fixture
def no_calls(monkeypatch):
    """Any call that reaches the library is a failure."""
    for f in ("dkv_extend_tables", "dkv_store_kv", "dkv_attn_chunk", "dkv_attn_decode_window"):
        monkeypatch.setattr(dkv, f, lambda *a: pytest.fail("the call reached the library"))


@pytest.mark.parametrize("name,key,bad", [
    ("window", "q32", torch.zeros((2, 4, 64), dtype=torch.bfloat16)),       # read as fp32, past its end
    ("window", "q32", torch.zeros((2, 4, 64), dtype=torch.float16)),
    ("window", "out32", torch.zeros((2, 4, 64), dtype=torch.bfloat16)),     # written past its end
    ("window", "q32", torch.zeros((1, 4, 64))),
    ("window", "q32", torch.zeros((2, 2, 64))),
    ("window", "q32", torch.zeros((2, 4, 128))[..., ::2]),
    ("window", "out32", torch.zeros((2, 64, 4)).transpose(1, 2)),
    ("chunk", "q16", torch.zeros((5, 4, 64), dtype=torch.float16)),
    ("chunk", "q16", torch.zeros((5, 4, 64), dtype=torch.int16)),
    ("chunk", "out16", torch.zeros((5, 4, 64), dtype=torch.float16)),
    ("store", "k", torch.zeros((5, 2, 64), dtype=torch.float16)),
    ("store", "v", torch.zeros((5, 2, 64), dtype=torch.float16)),
    ("store", "v", torch.zeros((5, 2, 64), dtype=torch.int16)),
])
def test_a_tensor_that_the_kernels_would_misread_is_refused(no_calls, name, key, bad):
    t = tensors()
    if name == "chunk" and key == "q16":    # out of the same type: the pair is consistent, and not the handle's
        t["out16"] = torch.zeros_like(bad)
    t[key] = bad
    with pytest.raises(ValueError, match="float32|bfloat16"):
        call(name, t)


@pytest.mark.parametrize("name", ["window", "chunk", "store", "extend"])
def test_a_cpu_tensor_is_refused(no_calls, name):
    with pytest.raises(ValueError, match="must be on GPU 0"):
        call(name, tensors())


@pytest.mark.parametrize("name", ["window", "chunk", "store", "extend"])
def test_a_cache_of_another_shape_is_refused(no_calls, name):
    for field, value in (("num_kv_heads", 1), ("head_dim", 128), ("block_size", 32)):
        kv = type("Other", (KV,), {field: value})
        t = tensors()
        t["k"] = t["v"] = torch.zeros((5, kv.num_kv_heads, kv.head_dim), dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="cache"):
            call(name, t, kv)


def test_staging_buffers_too_small_are_refused(no_calls):
    kv = type("Host", (KV,), {"host_split": 3})
    t = tensors()
    block = 2 * 16 * 64
    for k, v in ((torch.zeros(3 * block - 1, dtype=torch.int16), torch.zeros(3 * block, dtype=torch.int16)),
                 (torch.zeros(3 * block, dtype=torch.int16), torch.zeros((6 * block,), dtype=torch.int16)[::2]),
                 (torch.zeros(3 * block, dtype=torch.int16), None)):
        with pytest.raises(ValueError, match="k_stage and v_stage"):
            call("chunk", {**t, "k_stage": k, "v_stage": v}, kv)
