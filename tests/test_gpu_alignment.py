"""The serving entry points refuse addresses that their kernels could not load from (needs a B200)."""
import pytest
import torch

import decode_attention_host_b200 as dkv
from tests.test_gpu_chunk import Chunk
from tests.test_gpu_tables import Store
from tests.test_gpu_window import Window

pytestmark = pytest.mark.gpu


def refused(call, **bad):
    for name, ptr in bad.items():
        with pytest.raises(dkv.DkvError) as e:
            call(**{name: ptr.data_ptr() + 2})
        assert e.value.code == dkv.DKV_ERR_INVALID_ARG and "aligned" in str(e.value), name


def test_addresses_between_two_numbers_are_refused():
    st = torch.cuda.current_stream().cuda_stream
    c = Chunk([20], [8])
    k = c.cache
    args = dict(q=c.q, q_stride=c.hq * c.d, q_start=c.q_start, total_rows=8, k_host=None, v_host=None, k_dev=k.k_dev,
                v_dev=k.v_dev, block_table=k.table_dev, seq_lens=k.seq_lens_dev, host_split=0, out=c.out, window=0,
                sinks=0, include_self=1, stream=st, batch=1, block_table_stride=k.stride,
                num_dev_blocks=k.num_dev_blocks, k_stage=None, v_stage=None)
    refused(lambda **kw: dkv.dkv_attn_chunk(c.attn.handle, *{**args, **kw}.values()), q_start=c.q_start,
            block_table=k.table_dev, seq_lens=k.seq_lens_dev)
    w = Window([20], 8, 2)
    k = w.cache
    args2 = dict(window=8, sinks=2, include_self=0, q=w.q, k_host=None, v_host=None, k_dev=k.k_dev, v_dev=k.v_dev,
                 block_table=k.table_dev, seq_lens=k.seq_lens_dev, host_split=0, out=w.out, stream=st, batch=1,
                 block_table_stride=k.stride, num_dev_blocks=k.num_dev_blocks)
    refused(lambda **kw: dkv.dkv_attn_decode_window(w.attn.handle, *{**args2, **kw}.values()), out=w.out,
            block_table=k.table_dev, seq_lens=k.seq_lens_dev)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, new, table, ids, count, left, q_start = i32(1), i32(1), i32(4), i32(4), i32(1), i32(1), i32(2)
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    args3 = dict(seq_lens=lens, new_lens=new, batch=1, block_table=table, block_table_stride=4, free_ids=ids,
                 free_capacity=4, free_count=count, free_left=left, q_start=q_start, slot_map=slots, max_slots=4,
                 stream=st)
    refused(lambda **kw: dkv.dkv_extend_tables(w.attn.handle, *{**args3, **kw}.values()), seq_lens=lens, new_lens=new,
            block_table=table, free_ids=ids, free_count=count, free_left=left, q_start=q_start, slot_map=slots)
    torch.cuda.synchronize()
    for x in (c, w):
        assert x.attn.status() == 0 and (x.out == 7.0).all()
        x.run()
        x.verify()
        x.free()
    s = Store(4)
    s.call()
    s.verify()
    s.free()
