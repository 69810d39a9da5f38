"""Attention of a chunk of new tokens over the paged cache (needs a B200), against the 64-bit definition."""
import pytest
import torch

import decode_attention_host_b200 as dkv
from tests import serving_cases as sc

pytestmark = pytest.mark.gpu

LIB = {"bf16": dkv.DKV_KV_BF16, "f16": dkv.DKV_KV_F16}


class Chunk:
    def __init__(self, ctx, new, hkv=2, g=4, d=128, s=16, dtype="bf16", base=5e5, host=0.0, std=1.0, window=0, sinks=0,
                 self_=1, seed=0, pad=0, gap=0, max_batch=None, dev_blocks=None, spare_lens=0):
        self.ctx, self.new, self.window, self.sinks, self.self_ = list(ctx), list(new), window, sinks, self_
        self.dtype, self.base, self.pad = dtype, base, pad
        end = [c + max(0, n - 1 + self_) for c, n in zip(ctx, new)]

        def keep(b, j):      # blocks that no query sees are absent from the table
            if not window:
                return new[b] > 0
            lo = max(0, ctx[b] + self_ - window)
            return new[b] > 0 and ((j + 1) * s > lo or j * s < min(sinks, lo))
        self.cache = sc.Cache(end, hkv, d, s, dtype, seed, host=host, std=std, keep=keep, dev_blocks=dev_blocks)
        self.cache.set_lens(ctx)
        self.hq, self.d = hkv * g, d
        self.attn = dkv.DecodeAttention(self.hq, hkv, d, s, LIB[dtype], base, max_batch or len(ctx), self.cache.stride)
        gen = torch.Generator().manual_seed(seed + 1)
        total = sum(new)
        buf = torch.full((total + pad, self.hq * d + gap), float("nan"), dtype=sc.DTYPES[dtype])
        buf[:total, :self.hq * d] = torch.randn((total, self.hq * d), generator=gen).to(buf.dtype)
        self.q = buf.cuda()[:, :self.hq * d].unflatten(1, (self.hq, d))
        self.q_start = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32).cuda()
        self.out = torch.full((total + pad, self.hq, d), 7.0, dtype=buf.dtype, device="cuda")

    def run(self, **kw):
        self.attn.chunk(self.q, self.q_start, self.cache, self.out, self.window, self.sinks, bool(self.self_), **kw)
        torch.cuda.synchronize()
        return self.out

    def verify(self, out=None, rotated=True):
        out = self.out if out is None else out
        assert self.attn.status() == 0
        at, worst = 0, 0.0
        for b, n in enumerate(self.new):
            if n == 0:
                continue
            want = sc.attend64(self.q[at:at + n], self.cache.k[b], self.cache.v[b], self.ctx[b], self.base, self.self_,
                               self.window, self.sinks)
            worst = max(worst, sc.check(out[at:at + n], want[0], sc.bound16(*want, self.dtype, bool(self.base))))
            at += n
        if self.pad:
            assert (out[at:] == 7.0).all(), "rows behind the last sequence changed"
        return worst

    def free(self):
        self.attn.close()
        self.cache.free()


def once(*a, **kw):
    c = Chunk(*a, **kw)
    c.run()
    worst = c.verify()
    c.free()
    return worst


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("base", [0.0, 1e4])
@pytest.mark.parametrize("g", [1, 2, 4])
@pytest.mark.parametrize("d", [64, 128])
def test_shapes_and_types(d, g, base, dtype):
    once([70, 0, 301], [130, 65, 1], hkv=2, g=g, d=d, dtype=dtype, base=base, seed=d + g)


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 1000])
@pytest.mark.parametrize("new", [1, 2, 31, 32, 33, 64, 65, 129])
def test_edges_of_lengths(ctx, new):
    once([ctx], [new], hkv=1, g=4, seed=ctx + new)


@pytest.mark.parametrize("new", [1, 127, 128, 129, 255, 256, 257, 700])
def test_edges_of_lengths_mha(new):
    once([33], [new], hkv=3, g=1, dtype="f16", base=1e4, seed=new)


def test_ragged_batch_with_empty_sequences():
    once([0, 500, 3, 0, 77, 1200, 16], [5, 0, 300, 0, 1, 64, 16], seed=3, pad=5)


def test_every_sequence_empty():
    c = Chunk([4, 9], [0, 0], pad=3)
    c.run()
    assert (c.out == 7.0).all() and c.attn.status() == 0
    c.free()


def test_no_token_visible_gives_zero_rows():
    # without the tokens themselves the first query of an empty context sees nothing
    c = Chunk([0, 40], [70, 70], self_=0)
    c.run()
    assert (c.out[0] == 0).all()
    c.verify()
    c.free()


def test_one_query_without_self_is_the_decode_step():
    c = Chunk([700, 33], [1, 1], self_=0, hkv=2, g=4)
    c.run()
    q = c.q.float().contiguous()
    out = torch.empty_like(q)
    c.attn(q, c.cache, out)
    torch.cuda.synchronize()
    bound = 2 * sc.HALF_STEP["bf16"] * (out.abs() + 1)
    assert ((c.out.float() - out).abs() <= bound).all()
    c.free()


@pytest.mark.parametrize("s", [16, 32, 48, 64, 80, 128, 256, 1024])
def test_block_sizes(s):
    once([s - 1, 3 * s + 5, 0], [2, s + 1, 40], s=s, seed=s)


@pytest.mark.parametrize("self_", [0, 1])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (16, 0), (100, 4), (128, 128), (129, 130), (500, 17),
                                          (4000, 64), (64, 4000), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows_and_sinks(window, sinks, self_):
    once([0, 1000, 333, 64], [100, 70, 300, 1], window=window, sinks=sinks, self_=self_, seed=window % 97 + sinks % 89)


@pytest.mark.parametrize("s", [16, 48, 256])
def test_window_with_block_sizes(s):
    once([900, 2100], [150, 3], s=s, window=300, sinks=20, dtype="f16", base=1e4, seed=s)


@pytest.mark.parametrize("staged", [False, True])
@pytest.mark.parametrize("host", [0.3, 1.0])
def test_host_blocks(host, staged):
    c = Chunk([300, 90], [150, 40], host=host, seed=11, window=200 if staged else 0, sinks=5 if staged else 0)
    kw = {}
    if staged:
        n = c.cache.host_split * c.cache.hkv * c.cache.s * c.cache.d
        kw = {"k_stage": torch.empty(n, dtype=torch.int16, device="cuda"),
              "v_stage": torch.empty(n, dtype=torch.int16, device="cuda")}
    c.run(**kw)
    c.verify()
    c.free()


def test_strided_queries_and_padded_rows():
    once([50, 600], [90, 33], gap=264, pad=9, seed=5)


def test_long_context_few_rows():
    once([20000, 11111], [3, 9], hkv=2, g=4, s=64, seed=6)


def test_long_chunk():
    once([1500], [1100], hkv=1, g=2, d=64, dtype="f16", base=1e4, seed=7)


def test_many_sequences():
    once([(37 * i) % 400 for i in range(90)], [(i * 13) % 41 for i in range(90)], hkv=2, g=4, seed=8)


# Grids that fill the GPU are not split, so that a CTA walks over many tiles.

@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 40), (130, 200)])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
@pytest.mark.parametrize("rows", [1, 40, 128, 140, 256, 300])
def test_many_tiles_in_one_walk(rows, dtype, d, window, sinks):
    # an odd and an even number of tiles, one, two and none behind the sinks
    ctx = [1500 - rows, 1300, 130, 5, 700, 260]
    once(ctx, [rows] * 6, hkv=32, g=1, d=d, dtype=dtype, window=window, sinks=sinks, seed=rows)


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 40)])
@pytest.mark.parametrize("dtype,d,s", [("bf16", 128, 16), ("f16", 128, 64), ("bf16", 64, 32), ("f16", 64, 128)])
@pytest.mark.parametrize("new", [256, 257, 300, 384, 385, 512])
def test_long_chunks(new, dtype, d, s, window, sinks):
    # 4 to 8 row tiles of 256 rows, an even and an odd number, full and ragged ends; walks whole and split
    once([700, 0, 33], [new] * 3, hkv=16, g=4, d=d, s=s, dtype=dtype, window=window, sinks=sinks, seed=new)
    once([1000], [new], hkv=1, g=4, d=d, s=s, dtype=dtype, window=window, sinks=sinks, self_=0, seed=new + 1)


def test_long_chunks_with_short_and_empty_ones():
    once([0, 64, 1000, 3], [900, 0, 1, 700], hkv=8, g=4, host=0.2, seed=30, pad=3)


@pytest.mark.parametrize("g", [2, 4])
def test_many_tiles_of_shared_heads(g):
    once([900 + 61 * i for i in range(12)], [17 + 9 * i for i in range(12)], hkv=16, g=g, s=32, seed=g)


def test_short_chunks_on_average_with_a_long_one():
    once([100, 0, 700, 30, 1000], [1, 2, 1, 1, 150], hkv=2, g=4, seed=20)
    once([100, 0, 700, 30, 1000] * 8, ([1, 2, 1, 1, 150] + [1] * 5 * 7), hkv=8, g=2, seed=21)


def test_reference_raised_in_many_tiles():
    # scores that grow with the position: the running maximum moves in every tile, and must be followed
    c = Chunk([1500, 1400], [128, 30], hkv=32, g=1, base=0.0, dtype="f16", seed=22)
    for b in range(2):
        e = len(c.cache.k[b])
        ramp = torch.linspace(-40, 60, e)[:, None]
        c.cache.k[b][:, :, 0] = ramp.half()
        for j in range(-(-e // 16)):
            bid = int(c.cache.table[b, j])
            if bid >= 0:
                c.cache.k_dev[bid, :, :min(16, e - 16 * j), 0] = c.cache.k[b][16 * j:16 * j + 16, :, 0].T.cuda()
    c.q[..., 0] = 8.0
    c.run()
    c.verify()
    c.free()


def test_operands_beyond_fp16_poison_the_rows_that_see_them():
    c = Chunk([300, 300], [20, 20], seed=23)
    c.run()
    good = c.out.clone()
    bid = int(c.cache.table[1, 5])
    c.cache.k_dev[bid, :, 3, 7] = 1e5
    c.run()
    assert c.attn.status() == dkv.DKV_STATUS_RANGE
    assert torch.equal(c.out[:20], good[:20]) and c.out[20:].isnan().all()
    c.cache.k_dev[bid, :, 3, 7] = 6e4            # the largest that is sure to fit after rotation is 65504 / sqrt(2)
    c.cache.k_dev[bid, :, 3, 7 + 64] = 0.0
    c.run()
    assert c.attn.status() == 0 and torch.isfinite(c.out.float()).all()
    # behind the last visible token anything may be stored
    last = int(c.cache.table[1, (300 + 19) // 16])
    c.cache.k_dev[bid, :, 3, 7] = 0.0
    c.cache.k_dev[last, :, (300 + 19) % 16 + 1:] = 1e38
    c.run()
    assert c.attn.status() == 0 and torch.isfinite(c.out.float()).all()
    c.q[25, 3, 9] = 1e6
    c.run()
    assert c.attn.status() == dkv.DKV_STATUS_RANGE and c.out[25, 3].isnan().all()
    c.free()


def test_pool_beyond_32_bit_offsets():
    # 140000 blocks of 16384 elements: K and V offsets pass 2^31 elements and 2^32 bytes
    once([200], [70], hkv=8, g=1, dev_blocks=140000, seed=9)


def test_large_keys_and_peaked_weights():
    once([600, 90], [64, 64], std=8.0, dtype="f16", base=1e4, seed=10)
    once([600, 90], [64, 64], std=8.0, dtype="bf16", base=1e4, seed=10)


def test_explicit_stream_and_repeat_are_deterministic():
    c = Chunk([5000, 100], [40, 200], seed=12)
    first = c.run().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.out.fill_(7.0)
    torch.cuda.synchronize()
    c.run(stream=s)
    assert torch.equal(first, c.out)
    c.verify()
    c.free()


def test_captured_graph_follows_lengths_and_tables():
    c = Chunk([900, 30], [60, 20], seed=13)
    c.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attn.chunk(c.q, c.q_start, c.cache, c.out)
    c.out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    c.verify()
    # other lengths in the same buffers: shorter contexts, rows shifted between the sequences
    c.ctx, c.new = [800, 3], [50, 27]
    c.cache.set_lens(c.ctx)
    c.q_start.copy_(torch.tensor([0, 50, 77], dtype=torch.int32))
    c.out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    c.verify()
    assert (c.out[77:] == 7.0).all()
    c.free()


def test_bad_block_id_poisons_its_rows_only():
    c = Chunk([200, 200], [40, 40], seed=14)
    c.run()
    good = c.out.clone()
    bad = c.cache.host_split + c.cache.num_dev_blocks
    for value in (bad, -1, -2 ** 31, 2 ** 31 - 1):
        c.cache.table_dev[1, 3] = value
        c.out.fill_(7.0)
        c.run()
        assert c.attn.status() == dkv.DKV_STATUS_BAD_BLOCK_ID
        assert torch.equal(c.out[:40], good[:40]) and c.out[40:].isnan().all()
    assert c.attn.status() == 0
    c.free()


@pytest.mark.parametrize("lens", [-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
def test_bad_length_poisons_its_rows_only(lens):
    c = Chunk([200, 200], [40, 40], seed=15)
    c.run()
    good = c.out.clone()
    c.cache.set_lens([lens, 200])
    c.out.fill_(7.0)
    c.run()
    assert c.attn.status() == dkv.DKV_STATUS_BAD_SEQ_LEN
    assert c.out[:40].isnan().all() and torch.equal(c.out[40:], good[40:])
    c.free()


def test_infinite_and_nan_values_of_unseen_tokens_do_not_matter():
    # tokens that no query of the chunk sees: behind its last token in the same block, and between sinks and window
    c = Chunk([333], [20], window=100, sinks=4, seed=16)
    lo = 333 + 1 - 100
    for pool, fill in ((c.cache.k_dev, float("nan")), (c.cache.v_dev, float("inf"))):
        bid = int(c.cache.table[0, lo // 16]) - c.cache.host_split
        pool[bid, :, :lo % 16] = fill
        bid = int(c.cache.table[0, 0]) - c.cache.host_split
        pool[bid, :, 4:] = fill
    c.run()
    c.verify()
    c.free()


def test_nan_key_reaches_the_rows_that_see_it():
    c = Chunk([0], [40], hkv=1, g=4, seed=17)
    bid = int(c.cache.table[0, 1]) - c.cache.host_split
    c.cache.k_dev[bid, 0, 4, 5] = float("nan")       # token 20
    c.run()
    assert torch.isfinite(c.out[:20].float()).all() and c.out[20:].isnan().all()
    c.free()


@pytest.mark.parametrize("new", [[130, 20], [9, 3], [400, 300]])
def test_a_copy_that_never_completes_times_out_and_is_reported(new):
    """Every wait is bounded: a key tile that never lands (the hook arms its barrier and issues no copy) ends the
    waits of its CTA after about 2 s each, with NaN rows there; the other rows and the next call are clean."""
    c = Chunk([1500, 600], new, hkv=40, g=4, seed=24)      # more units than SMs: the walk is not split
    c.run()
    good = c.out.clone()
    dkv.dkv_debug_stall_copy(True)
    c.run()
    assert c.attn.status() == dkv.DKV_STATUS_COPY_TIMEOUT
    bad = c.out.isnan().any(-1)
    assert bad.any() and not bad.all()
    assert torch.equal(c.out[~bad], good[~bad])
    c.run()
    assert c.attn.status() == 0 and torch.equal(c.out, good)
    c.free()


def test_refusals():
    c = Chunk([20], [8], seed=18)
    a, k = c.attn, c.cache
    st = torch.cuda.current_stream().cuda_stream

    def call(**kw):
        d = dict(q=c.q, q_stride=c.hq * c.d, q_start=c.q_start, total_rows=8, k_host=None, v_host=None, k_dev=k.k_dev,
                 v_dev=k.v_dev, block_table=k.table_dev, seq_lens=k.seq_lens_dev, host_split=0, out=c.out, window=0,
                 sinks=0, include_self=1, stream=st, batch=1, block_table_stride=k.stride,
                 num_dev_blocks=k.num_dev_blocks, k_stage=None, v_stage=None)
        d.update(kw)
        dkv.dkv_attn_chunk(a.handle, *d.values())

    p = c.q.data_ptr()
    host = dkv.HostPool(1 << 16)
    for kw in (dict(q=None), dict(out=None), dict(q_start=None), dict(block_table=None), dict(seq_lens=None),
               dict(k_dev=None), dict(v_dev=None), dict(batch=-1), dict(batch=2), dict(total_rows=-1),
               dict(block_table_stride=0), dict(q_stride=c.hq * c.d - 8), dict(q_stride=c.hq * c.d + 4),
               dict(q=p + 8), dict(out=c.out.data_ptr() + 2), dict(window=-1), dict(sinks=-1), dict(include_self=2),
               dict(host_split=-1), dict(num_dev_blocks=-1), dict(host_split=1), dict(k_dev=k.k_dev.data_ptr() + 8),
               dict(k_dev=host.ptr), dict(host_split=1, k_host=k.k_dev, v_host=k.v_dev),
               dict(k_stage=k.k_dev), dict(host_split=1, k_host=host.ptr, v_host=host.ptr, k_stage=host.ptr,
                                           v_stage=host.ptr)):
        with pytest.raises(dkv.DkvError) as e:
            call(**kw)
        assert e.value.code == dkv.DKV_ERR_INVALID_ARG and str(e.value), kw
    call(batch=0)
    call(total_rows=0)
    call()
    torch.cuda.synchronize()
    c.verify()
    with pytest.raises(ValueError):
        a.chunk(c.q[:, :1], c.q_start, k, c.out)
    host.free()
    c.free()
