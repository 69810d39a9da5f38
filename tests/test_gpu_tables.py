"""Block tables, slot maps and the K/V store (needs a B200): whole numbers and copied bits, so all equal."""
import numpy as np
import pytest
import torch

import decode_attention_host_b200 as dkv

pytestmark = pytest.mark.gpu


class Tables:
    def __init__(self, ctx, new, s=16, seed=0, spare=7, pad=3, max_batch=None, stride=None):
        rng = np.random.default_rng(seed)
        self.ctx, self.new, self.s = np.array(ctx, np.int64), np.array(new, np.int64), s
        held, total = -(-self.ctx // s), -(-(self.ctx + self.new) // s)
        self.stride = stride or int(max(1, total.max(initial=1)))
        ids = rng.permutation(int(total.sum()) + spare).astype(np.int32)
        self.table = np.full((len(ctx), self.stride), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.free_ids = ids[at:].copy()
        self.max_slots = int(self.new.sum()) + pad
        self.dev = {k: torch.from_numpy(np.asarray(v, np.int32)).cuda() for k, v in (
            ("ctx", self.ctx), ("new", self.new), ("table", self.table), ("ids", self.free_ids),
            ("count", [len(self.free_ids)]))}
        self.left = torch.full((1,), -7, dtype=torch.int32, device="cuda")
        self.q_start = torch.full((len(ctx) + 1,), -7, dtype=torch.int32, device="cuda")
        self.slots = torch.full((max(1, self.max_slots),), -7, dtype=torch.int64, device="cuda")
        self.attn = dkv.DecodeAttention(1, 1, 64, s, dkv.DKV_KV_F16, 0.0, max_batch or len(ctx), self.stride)

    def call(self, **kw):
        d = dict(seq_lens=self.dev["ctx"], new_lens=self.dev["new"], batch=len(self.ctx), block_table=self.dev["table"],
                 block_table_stride=self.stride, free_ids=self.dev["ids"], free_capacity=len(self.free_ids),
                 free_count=self.dev["count"], free_left=self.left, q_start=self.q_start, slot_map=self.slots,
                 max_slots=self.max_slots, stream=torch.cuda.current_stream().cuda_stream)
        d.update(kw)
        dkv.dkv_extend_tables(self.attn.handle, *d.values())
        torch.cuda.synchronize()

    def want(self):
        table, top, slots = self.table.copy(), len(self.free_ids), []
        for b, (c, n) in enumerate(zip(self.ctx.tolist(), self.new.tolist())):
            for j in range(-(-c // self.s), -(-(c + n) // self.s)):
                top -= 1
                table[b, j] = self.free_ids[top]
            slots += [int(table[b, p // self.s]) * self.s + p % self.s for p in range(c, c + n)]
        slots += [-1] * (self.max_slots - len(slots))
        return table, [0] + np.cumsum(self.new).tolist(), slots, top

    def verify(self, left=None):
        table, q_start, slots, top = self.want()
        assert self.attn.status() == 0
        assert np.array_equal(self.dev["table"].cpu().numpy(), table)
        assert self.q_start.tolist() == q_start
        assert self.slots[:self.max_slots].tolist() == slots
        assert (self.left if left is None else left).item() == top

    def verify_refused(self, status):
        assert self.attn.status() == status
        assert np.array_equal(self.dev["table"].cpu().numpy(), self.table)
        assert not self.q_start.any() and (self.slots[:self.max_slots] == -1).all()


@pytest.mark.parametrize("s", [16, 48, 1024])
@pytest.mark.parametrize("ctx,new", [
    ([0], [0]), ([0], [1]), ([15], [1]), ([16], [1]), ([17], [15]), ([16], [16]), ([1], [1000]),
    ([0, 5, 16, 31, 700], [33, 0, 1, 1, 0]), ([0, 0, 0], [0, 0, 0])])
def test_small(ctx, new, s):
    t = Tables(ctx, new, s)
    t.call()
    t.verify()


@pytest.mark.parametrize("batch", [1, 31, 32, 33, 511, 512, 513, 1500])
def test_batches(batch):
    rng = np.random.default_rng(batch)
    t = Tables(rng.integers(0, 300, batch), rng.integers(0, 90, batch), seed=batch)
    t.call()
    t.verify()


def test_a_million_slots():
    rng = np.random.default_rng(5)
    t = Tables(rng.integers(0, 5000, 300), rng.integers(0, 7000, 300), s=32, seed=5)
    t.call()
    t.verify()


def test_largest_batch():
    t = Tables([3] * 8192, [14] * 8192, seed=6)
    t.call()
    t.verify()
    with pytest.raises(dkv.DkvError) as e:
        big = Tables([0], [1], max_batch=8193)
        big.call(batch=8193)
    assert e.value.code == dkv.DKV_ERR_UNSUPPORTED


def test_count_in_place_and_repeated_growth():
    t = Tables([0, 30, 7], [20, 3, 0], stride=40, spare=60)
    t.call(free_left=t.dev["count"])
    t.verify(left=t.dev["count"])
    # the next step goes on from there
    table, _, _, top = t.want()
    t.table, t.free_ids = table, t.free_ids[:top]
    t.ctx = t.ctx + t.new
    t.new = np.array([1, 1, 200])
    t.max_slots = 210
    t.slots = torch.full((210,), -7, dtype=torch.int64, device="cuda")
    for k, v in (("ctx", t.ctx), ("new", t.new)):
        t.dev[k].copy_(torch.from_numpy(v.astype(np.int32)))
    t.call(free_left=t.dev["count"], free_capacity=len(t.dev["ids"]))
    t.verify(left=t.dev["count"])


def test_captured_graph_follows_the_lengths():
    t = Tables([100, 7, 0], [5, 1, 0], stride=30, spare=40, pad=60)
    t.call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dkv.dkv_extend_tables(t.attn.handle, t.dev["ctx"], t.dev["new"], 3, t.dev["table"], 30, t.dev["ids"],
                              len(t.free_ids), t.dev["count"], t.left, t.q_start, t.slots, t.max_slots,
                              torch.cuda.current_stream().cuda_stream)
    t.ctx, t.new = np.array([100, 7, 0]), np.array([0, 40, 17])
    t.dev["table"].copy_(torch.from_numpy(t.table))
    t.dev["new"].copy_(torch.from_numpy(t.new.astype(np.int32)))
    for _ in range(3):      # replays on the same input give the same answer
        g.replay()
    torch.cuda.synchronize()
    t.verify()


@pytest.mark.parametrize("what,status", [
    ("blocks", dkv.DKV_STATUS_NO_FREE_BLOCKS), ("count", dkv.DKV_STATUS_NO_FREE_BLOCKS),
    ("negative count", dkv.DKV_STATUS_NO_FREE_BLOCKS), ("slots", dkv.DKV_STATUS_NO_SLOTS),
    ("ctx", dkv.DKV_STATUS_BAD_SEQ_LEN), ("new", dkv.DKV_STATUS_BAD_SEQ_LEN), ("long", dkv.DKV_STATUS_BAD_SEQ_LEN),
    ("huge", dkv.DKV_STATUS_BAD_SEQ_LEN)])
def test_what_cannot_be_served_changes_nothing(what, status):
    t = Tables([100, 7, 0], [30, 1, 18])
    count = len(t.free_ids)
    if what == "blocks":
        t.dev["count"].fill_(3)
        count = 3
    elif what == "count":
        t.dev["count"].fill_(len(t.free_ids) + 1)
        count += 1
    elif what == "negative count":
        t.dev["count"].fill_(-1)
        count = -1
    elif what == "slots":
        t.max_slots = 48
    elif what == "ctx":
        t.dev["ctx"][1] = -1
    elif what == "new":
        t.dev["new"][2] = -2 ** 31
    elif what == "long":
        t.dev["new"][0] = t.stride * 16 - 100 + 1
    elif what == "huge":
        t.dev["new"][0] = 2 ** 31 - 1
    t.call()
    t.verify_refused(status)
    assert t.left.item() == count


def test_negative_ids_are_not_mapped():
    t = Tables([20], [40])
    t.dev["table"][0, 1] = -1
    t.dev["ids"][-1] = -5
    t.call()
    assert t.attn.status() == dkv.DKV_STATUS_BAD_BLOCK_ID
    assert (t.slots[:28] == -1).all() and (t.slots[28:40] >= 0).all()


def test_table_refusals():
    t = Tables([20], [40])
    for kw in (dict(seq_lens=None), dict(new_lens=None), dict(batch=0), dict(batch=-1), dict(batch=2),
               dict(block_table=None), dict(block_table_stride=0), dict(free_ids=None), dict(free_capacity=-1),
               dict(free_count=None), dict(free_left=None), dict(q_start=None), dict(slot_map=None),
               dict(max_slots=-1), dict(max_slots=(1 << 30) + 1), dict(slot_map=t.slots.data_ptr() + 4)):
        with pytest.raises(dkv.DkvError) as e:
            t.call(**kw)
        assert e.value.code == dkv.DKV_ERR_INVALID_ARG, kw
    t.call()
    t.verify()


# --------------------------------------------------------------------------- store

class Store:
    def __init__(self, rows, hkv=2, d=128, s=16, dtype=torch.bfloat16, host=0, gap=0, seed=0, dev_blocks=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.hkv, self.d, self.s, self.host = rows, hkv, d, s, host
        self.dev = dev_blocks or -(-max(rows, 1) // s) + 2
        w = hkv * d
        self.buf = torch.randn((max(rows, 1), 2 * w + gap), generator=g, device="cuda").to(dtype)
        self.k_new, self.v_new = (self.buf[:, o:o + w].unflatten(1, (hkv, d)) for o in (0, w))
        make = torch.empty if dev_blocks else torch.zeros
        self.k_dev, self.v_dev = (make((self.dev, hkv, s, d), dtype=dtype, device="cuda") for _ in "kv")
        self.pools = [dkv.HostPool(host * hkv * s * d) for _ in "kv"]
        for p in self.pools:
            p.array[:] = 0
        self.attn = dkv.DecodeAttention(hkv, hkv, d, s, dkv.DKV_KV_BF16 if dtype == torch.bfloat16 else dkv.DKV_KV_F16,
                                        0.0, 1, 4)
        total = (self.dev + host) * s
        self.slots = torch.randperm(total if not dev_blocks else 4000, generator=g, device="cuda")[:rows]
        if dev_blocks:
            self.slots = total - 1 - self.slots

    def call(self, **kw):
        k = dict(k_new=self.k_new, v_new=self.v_new, row_stride=self.buf.stride(0), slot_map=self.slots,
                 num_rows=self.rows, host_split=self.host, k_host=self.pools[0].ptr if self.host else None,
                 v_host=self.pools[1].ptr if self.host else None, k_dev=self.k_dev, v_dev=self.v_dev,
                 stream=torch.cuda.current_stream().cuda_stream, num_dev_blocks=self.dev)
        k.update(kw)
        dkv.dkv_store_kv(self.attn.handle, *k.values())
        torch.cuda.synchronize()

    def pool(self, i):
        dev = (self.k_dev, self.v_dev)[i].view(torch.int16)
        n = self.host * self.hkv * self.s * self.d
        h = torch.from_numpy(self.pools[i].array[:n].astype(np.int16)).view(self.host, self.hkv, self.s, self.d).cuda()
        return torch.cat((h, dev))

    def verify(self, live=None):
        for i, new in enumerate((self.k_new, self.v_new)):
            want = torch.zeros_like(self.pool(i))
            use = self.slots >= 0 if live is None else live
            slot = self.slots[use]
            want[slot // self.s, :, slot % self.s] = new.view(torch.int16)[:self.rows][use]
            assert torch.equal(self.pool(i), want)

    def free(self):
        self.attn.close()
        for p in self.pools:
            p.free()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hkv,d,s", [(1, 64, 16), (8, 128, 16), (3, 64, 48), (32, 128, 64), (5, 128, 1024)])
@pytest.mark.parametrize("rows", [1, 3, 130])
def test_store(rows, hkv, d, s, dtype):
    st = Store(rows, hkv, d, s, dtype, seed=rows)
    st.call()
    assert st.attn.status() == 0
    st.verify()
    st.free()


def test_store_skips_strides_and_host_blocks():
    st = Store(200, hkv=4, host=9, gap=264, seed=2)
    st.slots[::7] = -1
    st.slots[5] = -2 ** 62
    st.call()
    assert st.attn.status() == 0
    st.verify()
    st.free()


def test_store_beyond_both_pools_is_skipped():
    st = Store(50, host=3, seed=3)
    bad = torch.zeros(50, dtype=torch.bool, device="cuda")
    bad[[0, 13, 49]] = True
    st.slots[0], st.slots[13], st.slots[49] = (st.dev + 3) * 16, 2 ** 62, (st.dev + 3) * 16 + 5
    st.call()
    assert st.attn.status() == dkv.DKV_STATUS_BAD_BLOCK_ID
    st.verify(live=~bad)
    st.free()


def test_store_beyond_32_bit_offsets():
    st = Store(60, hkv=8, dev_blocks=140000, seed=4)
    st.call()
    assert st.attn.status() == 0
    for pool, new in ((st.k_dev, st.k_new), (st.v_dev, st.v_new)):
        assert torch.equal(pool[st.slots // 16, :, st.slots % 16].view(torch.int16), new.contiguous().view(torch.int16))
    st.free()


def test_store_refusals():
    st = Store(4)
    for kw in (dict(k_new=None), dict(v_new=None), dict(slot_map=None), dict(num_rows=-1), dict(row_stride=248),
               dict(row_stride=516), dict(k_new=st.buf.data_ptr() + 8), dict(slot_map=st.slots.data_ptr() + 4),
               dict(k_dev=None), dict(host_split=1), dict(host_split=-1), dict(num_dev_blocks=-1),
               dict(v_dev=st.v_dev.data_ptr() + 2)):
        with pytest.raises(dkv.DkvError) as e:
            st.call(**kw)
        assert e.value.code == dkv.DKV_ERR_INVALID_ARG, kw
    st.call(num_rows=0)
    assert not st.k_dev.any()
    st.call()
    st.verify()
    st.free()


def test_binding_refusals():
    class KV:
        num_kv_heads, head_dim, host_split, num_dev_blocks, batch, stride = 2, 128, 0, 4, 1, 4
    st = Store(4)
    bad = [(st.k_new[:, :, ::2], st.v_new, st.slots), (st.k_new.float(), st.v_new, st.slots),
           (st.k_new, st.v_new.contiguous(), st.slots), (st.k_new, st.v_new, st.slots.int()),
           (st.k_new, st.v_new, st.slots[:3])]
    for k, v, slots in bad:
        with pytest.raises(ValueError):
            st.attn.store(k, v, slots, KV)
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    for new, ids, count in ((one.long(), one, one), (one, one.long(), one), (one, one, one.float()),
                            (torch.ones(2, dtype=torch.int32, device="cuda"), one, one)):
        with pytest.raises(ValueError):
            st.attn.extend(KV, new, ids, count, 4)
    st.free()
