"""The binding's serving methods on the GPU: streams other than the current one."""
from types import SimpleNamespace

import torch
import pytest

import decode_attention_host_b200 as dkv

pytestmark = pytest.mark.gpu


def test_extend_on_another_stream_takes_no_memory_that_the_current_one_still_writes():
    batch, s, cols, slots = 3, 16, 8, 4096
    kv = SimpleNamespace(batch=batch, stride=cols, num_kv_heads=1, head_dim=64, host_split=0, num_dev_blocks=64,
                         table_dev=torch.full((batch, cols), -1, dtype=torch.int32, device="cuda"),
                         seq_lens_dev=torch.zeros(batch, dtype=torch.int32, device="cuda"))
    attn = dkv.DecodeAttention(1, 1, 64, s, dkv.DKV_KV_BF16, 0.0, batch, cols)
    new = torch.tensor([20, 0, 33], dtype=torch.int32, device="cuda")
    free_ids = torch.arange(64, dtype=torch.int32, device="cuda")
    count = torch.tensor([64], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    big = torch.randn((4096, 4096), device="cuda")
    # the current stream's queue ends with a write to memory that its allocator already counts as free
    old = torch.empty(slots, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        big = big @ big * 1e-3
    old.fill_(-7)
    del old
    q_start, slot_map = attn.extend(kv, new, free_ids, count, slots, stream=side)
    torch.cuda.synchronize()
    assert attn.status() == 0 and q_start.tolist() == [0, 20, 20, 53]
    ids = [63] * 16 + [62] * 4 + [61] * 16 + [60] * 16 + [59]
    rows = list(range(20)) + list(range(33))
    want = [i * s + r % s for i, r in zip(ids, rows)] + [-1] * (slots - 53)
    assert slot_map.tolist() == want and count.item() == 59
    attn.close()
