"""Decode attention over a sliding window and sinks (needs a B200), against the 64-bit definition."""
import pytest
import torch

import decode_attention_host_b200 as dkv
from tests import serving_cases as sc

pytestmark = pytest.mark.gpu

LIB = {"bf16": dkv.DKV_KV_BF16, "f16": dkv.DKV_KV_F16}


class Window:
    def __init__(self, ctx, window, sinks, hkv=2, g=4, d=128, s=16, dtype="bf16", base=5e5, host=0.0, std=1.0, self_=0,
                 seed=0, max_batch=None, dev_blocks=None):
        self.ctx, self.win, self.sinks, self.self_, self.base = list(ctx), window, sinks, self_, base

        def keep(b, j):
            lo = max(0, ctx[b] + self_ - window)
            return (j + 1) * s > lo or j * s < min(sinks, lo)
        self.cache = sc.Cache([c + self_ for c in ctx], hkv, d, s, dtype, seed, host=host, std=std, keep=keep,
                              dev_blocks=dev_blocks)
        self.cache.set_lens(ctx)
        self.attn = dkv.DecodeAttention(hkv * g, hkv, d, s, LIB[dtype], base, max_batch or len(ctx), self.cache.stride)
        gen = torch.Generator().manual_seed(seed + 1)
        self.q = torch.randn((len(ctx), hkv * g, d), generator=gen).cuda()
        self.out = torch.full_like(self.q, 7.0)

    def run(self, stream=None):
        self.attn.window(self.q, self.cache, self.out, self.win, self.sinks, bool(self.self_), stream=stream)
        torch.cuda.synchronize()
        return self.out

    def verify(self):
        assert self.attn.status() == 0
        worst = 0.0
        for b, c in enumerate(self.ctx):
            want = sc.attend64(self.q[b:b + 1], self.cache.k[b], self.cache.v[b], c, self.base, self.self_, self.win,
                               self.sinks)
            worst = max(worst, sc.check(self.out[b:b + 1], want[0], sc.bound32(want[1], want[2])))
        return worst

    def free(self):
        self.attn.close()
        self.cache.free()


def once(*a, **kw):
    w = Window(*a, **kw)
    w.run()
    worst = w.verify()
    w.free()
    return worst


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("base", [0.0, 1e4])
@pytest.mark.parametrize("g", [1, 2, 4])
@pytest.mark.parametrize("d", [64, 128])
def test_shapes_and_types(d, g, base, dtype):
    once([0, 5, 300, 777], 100, 5, g=g, d=d, dtype=dtype, base=base, seed=d + g)


@pytest.mark.parametrize("self_", [0, 1])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (15, 16), (16, 0), (17, 17), (100, 4), (128, 128),
                                          (500, 33), (64, 4000), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows_and_sinks(window, sinks, self_):
    once([0, 1, 16, 17, 100, 101, 140, 1000, 999, 33], window, sinks, self_=self_, seed=window % 97)


@pytest.mark.parametrize("s", [16, 48, 64, 256, 1024])
def test_block_sizes(s):
    once([s - 1, s, 3 * s + 5, 5 * s], 300, 20, s=s, seed=s, dtype="f16", base=1e4)


@pytest.mark.parametrize("host", [0.3, 1.0])
def test_host_blocks(host):
    once([300, 90, 2000], 256, 40, host=host, seed=3)


def test_long_contexts():
    once([60000, 30001], 8192, 64, s=32, seed=4)


def test_many_sequences():
    once([(i * 61) % 900 for i in range(100)], 200, 4, seed=5, hkv=1)


def test_pool_beyond_32_bit_offsets():
    once([500], 200, 20, hkv=8, g=1, dev_blocks=140000, seed=9)


def test_large_window_is_the_plain_decode_step():
    w = Window([700, 33, 0], 10 ** 6, 0)
    w.run()
    w.verify()
    w.attn(w.q, w.cache, w.out)
    torch.cuda.synchronize()
    w.verify()
    w.free()


def test_stream_repeat_and_graph():
    w = Window([5000, 100], 700, 9, seed=12)
    first = w.run().clone()
    s = torch.cuda.Stream()
    w.run(stream=s)
    assert torch.equal(first, w.out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.attn.window(w.q, w.cache, w.out, w.win, w.sinks)
    # a shorter sequence in the same buffers; its window still lies in blocks that the cache holds
    w.ctx = [4995, 60]
    w.cache.set_lens(w.ctx)
    w.win = 690
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        w.attn.window(w.q, w.cache, w.out, w.win, w.sinks)
    g2.replay()
    torch.cuda.synchronize()
    w.verify()
    w.ctx, w.win = [5000, 100], 700
    w.cache.set_lens(w.ctx)
    g.replay()
    torch.cuda.synchronize()
    w.verify()
    w.free()


def test_bad_ids_and_lengths_poison_their_rows():
    w = Window([500, 500], 100, 20, seed=14)
    good = w.run().clone()
    keep = w.cache.table_dev.clone()
    w.cache.table_dev[1, 0] = w.cache.host_split + w.cache.num_dev_blocks   # a sink block
    w.run()
    assert w.attn.status() == dkv.DKV_STATUS_BAD_BLOCK_ID
    assert w.out[1].isnan().all() and torch.equal(w.out[0], good[0])
    w.cache.table_dev.copy_(keep)
    w.cache.table_dev[1, 3] = 2 ** 31 - 1                                      # an evicted block
    w.run()
    assert w.attn.status() == 0 and torch.equal(w.out, good)
    for bad in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        w.cache.set_lens([bad, 500])
        w.run()
        assert w.attn.status() == dkv.DKV_STATUS_BAD_SEQ_LEN
        assert w.out[0].isnan().all() and torch.equal(w.out[1], good[1])
    w.free()


def test_unseen_values_do_not_matter():
    w = Window([333], 100, 4, seed=16)
    lo = 333 - 100
    for pool, fill in ((w.cache.k_dev, float("nan")), (w.cache.v_dev, float("inf"))):
        pool[int(w.cache.table[0, lo // 16]), :, :lo % 16] = fill
        pool[int(w.cache.table[0, 0]), :, 4:] = fill
    w.run()
    w.verify()
    w.free()


def test_refusals():
    w = Window([20], 8, 2, seed=18)
    k = w.cache
    st = torch.cuda.current_stream().cuda_stream

    def call(**kw):
        d = dict(window=8, sinks=2, include_self=0, q=w.q, k_host=None, v_host=None, k_dev=k.k_dev, v_dev=k.v_dev,
                 block_table=k.table_dev, seq_lens=k.seq_lens_dev, host_split=0, out=w.out, stream=st, batch=1,
                 block_table_stride=k.stride, num_dev_blocks=k.num_dev_blocks)
        d.update(kw)
        dkv.dkv_attn_decode_window(w.attn.handle, *d.values())

    for kw in (dict(q=None), dict(out=None), dict(block_table=None), dict(seq_lens=None), dict(k_dev=None),
               dict(v_dev=None), dict(batch=-1), dict(batch=2), dict(block_table_stride=0), dict(window=0),
               dict(window=-3), dict(sinks=-1), dict(include_self=2), dict(include_self=-1), dict(host_split=-1),
               dict(num_dev_blocks=-1), dict(host_split=1), dict(q=w.q.data_ptr() + 4),
               dict(v_dev=k.v_dev.data_ptr() + 2), dict(host_split=1, k_host=k.k_dev, v_host=k.v_dev)):
        with pytest.raises(dkv.DkvError) as e:
            call(**kw)
        assert e.value.code == dkv.DKV_ERR_INVALID_ARG and str(e.value), kw
    call(batch=0)
    call()
    torch.cuda.synchronize()
    w.verify()
    w.free()
