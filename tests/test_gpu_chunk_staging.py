"""Chunk attention with staged host pools (needs a B200): a refused call has copied nothing and taken no hook."""
import pytest
import torch

import decode_attention_host_b200 as dkv
from tests.test_gpu_chunk import Chunk

pytestmark = pytest.mark.gpu


def test_a_refused_call_leaves_the_staging_buffers_and_the_stall_hook():
    c = Chunk([300], [20], hkv=8, host=1.0, seed=31)
    k = c.cache
    n = k.host_split * k.hkv * k.s * k.d
    stage = [torch.full((n,), -9, dtype=torch.int16, device="cuda") for _ in "kv"]
    too_many = 2 ** 31 // (k.hkv * k.s)      # blocks of a device pool with 2^31 token rows; refused, so never read
    dkv.dkv_debug_stall_copy(True)
    with pytest.raises(dkv.DkvError) as e:
        dkv.dkv_attn_chunk(c.attn.handle, c.q, c.hq * c.d, c.q_start, 20, k.k_host.ptr, k.v_host.ptr, k.k_dev, k.v_dev,
                           k.table_dev, k.seq_lens_dev, k.host_split, c.out, 0, 0, 1,
                           torch.cuda.current_stream().cuda_stream, 1, k.stride, too_many, *stage)
    assert e.value.code == dkv.DKV_ERR_INVALID_ARG and "token rows" in str(e.value)
    torch.cuda.synchronize()
    assert all((x == -9).all() for x in stage) and (c.out == 7.0).all()
    c.run()                                  # the hook is still armed: it belongs to the next call that launches
    assert c.attn.status() == dkv.DKV_STATUS_COPY_TIMEOUT
    c.run(k_stage=stage[0], v_stage=stage[1])
    c.verify()
    c.free()
