"""Engine steps through all entry points of a growing cache (needs a B200): tables and slots, K/V store, chunk
attention, windowed and plain decode, eagerly and as one captured graph, against the 64-bit definition."""
import pytest
import torch

import decode_attention_host_b200 as dkv
from tests import serving_cases as sc

pytestmark = pytest.mark.gpu


class Engine:
    """Three requests on an empty cache with room to grow; keeps the logical K/V rows beside it."""

    def __init__(self, window, sinks, host_blocks=0, dtype="bf16", hkv=2, g=4, d=128, s=16, base=5e5, batch=3,
                 cols=64):
        self.window, self.sinks, self.base, self.dtype = window, sinks, base, dtype
        self.hkv, self.hq, self.d, self.s = hkv, hkv * g, d, s
        blocks = batch * cols
        self.kv = kv = type("KV", (), {})()
        kv.batch, kv.stride, kv.num_kv_heads, kv.head_dim = batch, cols, hkv, d
        kv.host_split, kv.num_dev_blocks = host_blocks, blocks - host_blocks
        kv.k_host, kv.v_host = (dkv.HostPool(host_blocks * hkv * s * d) for _ in "kv")
        shape = (blocks - host_blocks, hkv, s, d)
        kv.k_dev, kv.v_dev = (torch.full(shape, float("nan"), dtype=sc.DTYPES[dtype], device="cuda") for _ in "kv")
        kv.table_dev = torch.full((batch, cols), -1, dtype=torch.int32, device="cuda")
        kv.seq_lens_dev = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.gen = torch.Generator().manual_seed(5)
        self.free_ids = torch.randperm(blocks, generator=self.gen).to(torch.int32).cuda()
        self.count = torch.tensor([blocks], dtype=torch.int32, device="cuda")
        self.attn = dkv.DecodeAttention(self.hq, hkv, d, s, dkv.DKV_KV_BF16 if dtype == "bf16" else dkv.DKV_KV_F16,
                                        base, batch, cols)
        self.k = [torch.zeros((0, hkv, d), dtype=sc.DTYPES[dtype]) for _ in range(batch)]
        self.v = list(self.k)
        # the buffers that a captured step keeps: 256 rows of a fused q, k, v projection
        self.rows = 256
        width = (self.hq + 2 * hkv) * d
        self.qkv = torch.zeros((self.rows, width), dtype=sc.DTYPES[dtype], device="cuda")
        self.new = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.out = torch.empty((self.rows, self.hq, d), dtype=sc.DTYPES[dtype], device="cuda")
        self.q_dec = torch.zeros((batch, self.hq, d), device="cuda")
        self.dec = torch.empty_like(self.q_dec)
        self.plain = torch.empty_like(self.q_dec)

    def draw(self, new):
        self.ctx, self.lens = [len(x) for x in self.k], list(new)
        qkv = torch.randn((sum(new), self.qkv.shape[1]), generator=self.gen).to(self.qkv.dtype)
        self.qkv.fill_(float("nan"))
        self.qkv[:sum(new)] = qkv.cuda()
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.q_dec.copy_(torch.randn(self.q_dec.shape, generator=self.gen))
        at, a, b = 0, self.hq * self.d, (self.hq + self.hkv) * self.d
        for i, n in enumerate(new):
            r = qkv[at:at + n]
            self.k[i] = torch.cat((self.k[i], r[:, a:b].unflatten(1, (self.hkv, self.d))))
            self.v[i] = torch.cat((self.v[i], r[:, b:].unflatten(1, (self.hkv, self.d))))
            at += n

    def step(self):
        kv, a, b = self.kv, self.hq * self.d, (self.hq + self.hkv) * self.d
        q_start, slots = self.attn.extend(kv, self.new, self.free_ids, self.count, self.rows)
        heads = lambda x: x.unflatten(1, (-1, self.d))  # noqa: E731
        self.attn.store(heads(self.qkv[:, a:b]), heads(self.qkv[:, b:]), slots, kv)
        self.attn.chunk(heads(self.qkv[:, :a]), q_start, kv, self.out, self.window, self.sinks)
        kv.seq_lens_dev += self.new
        self.attn.window(self.q_dec, kv, self.dec, self.window or 10 ** 6, self.sinks)
        self.attn(self.q_dec, kv, self.plain)

    def verify(self):
        torch.cuda.synchronize()
        assert self.attn.status() == 0
        assert self.kv.seq_lens_dev.tolist() == [len(x) for x in self.k]
        used = sum(-(-len(x) // self.s) for x in self.k)
        assert self.count.item() == self.free_ids.numel() - used
        at = 0
        for i, n in enumerate(self.lens):
            if n:
                q = self.qkv[at:at + n, :self.hq * self.d].unflatten(1, (self.hq, self.d))
                want = sc.attend64(q, self.k[i], self.v[i], self.ctx[i], self.base, 1, self.window, self.sinks)
                sc.check(self.out[at:at + n], want[0], sc.bound16(*want, self.dtype))
            at += n
            for out, win in ((self.dec, self.window), (self.plain, 0)):
                want = sc.attend64(self.q_dec[i:i + 1], self.k[i], self.v[i], len(self.k[i]), self.base, 0, win,
                                   self.sinks)
                sc.check(out[i:i + 1], want[0], sc.bound32(want[1], want[2]))


STEPS = ([130, 0, 17], [1, 1, 1], [1, 200, 1], [15, 1, 0], [64, 64, 64])


@pytest.mark.parametrize("window,sinks,host", [(0, 0, 0), (100, 5, 0), (100, 5, 60)])
def test_steps(window, sinks, host):
    e = Engine(window, sinks, host)
    for new in STEPS:
        e.draw(new)
        e.step()
        e.verify()


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_steps_as_one_captured_graph(window, sinks):
    e = Engine(window, sinks, dtype="f16", base=1e4)
    e.draw([0, 0, 0])
    e.step()        # warm-up on an empty step
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e.step()
    for new in STEPS:
        e.draw(new)
        g.replay()
        e.verify()


def test_first_calls_of_a_handle_inside_a_capture():
    e = Engine(100, 5, host_blocks=20)
    e.draw(STEPS[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e.step()
    g.replay()
    e.verify()
    for new in STEPS[1:]:
        e.draw(new)
        g.replay()
        e.verify()


def test_two_graphs_of_one_handle_replayed_in_turn():
    e = Engine(100, 5)
    graphs = []
    for new in STEPS[:2]:
        e.draw(new)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            e.step()
        g.replay()
        e.verify()
        graphs.append(g)
    for i, new in enumerate(STEPS[2:]):
        e.draw(new)
        graphs[i % 2].replay()
        e.verify()


def test_two_handles_on_two_streams():
    es = [Engine(100, 5), Engine(0, 0, dtype="f16")]
    streams = [torch.cuda.Stream() for _ in es]
    for new in STEPS:
        for e in es:
            e.draw(new)
        torch.cuda.synchronize()
        for e, s in zip(es, streams):
            with torch.cuda.stream(s):
                e.step()
        torch.cuda.synchronize()
        for e in es:
            e.verify()
