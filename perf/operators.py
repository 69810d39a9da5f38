"""Cases, plain forms and exact values of the serving operators around the paged cache.

Four operators are measured, in the order in which one engine step calls them:

- ``tables``: block tables grown and slot maps written on the GPU from request lengths;
- ``store``: new K/V rows scattered to their slots of the paged pools;
- ``chunk``: attention of chunks of new tokens over the paged cache, causal, optionally with a
  sliding window and sinks;
- ``window``: decode attention over a sliding window and a few first tokens that stay visible.

Keys are stored un-rotated and rotated when they are read (NeoX RoPE, token t at position t).
With ``own`` false, ``run`` computes the plain form out of elementary torch operations; with
``own`` true it calls the library.
"""
import math

import torch

own = False

_DEV = "cuda"
_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------------- cases

def _attn(name, op, batch, hq, hkv, d, bs, dtype, std, base, ctx, new, window=0, sinks=0, self_visible=1,
          host_sinks=False):
    return {"name": name, "op": op, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "bs": bs, "dtype": dtype,
            "std": std, "base": base, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0], "new_hi": new[1],
            "window": window, "sinks": sinks, "self_visible": self_visible, "host_sinks": host_sinks}


def listed():
    return [
        # every decode step of a batch: one new token each, a new block now and then (latency)
        {"name": "tables_decode_b64", "op": "tables", "batch": 64, "bs": 16, "ctx_lo": 1, "ctx_hi": 16384,
         "new_lo": 1, "new_hi": 1},
        # admission of a large batch of ragged prompts at once: about a million slots
        {"name": "tables_admit_b512", "op": "tables", "batch": 512, "bs": 16, "ctx_lo": 0, "ctx_hi": 1024,
         "new_lo": 1, "new_hi": 4096},
        # the K/V rows of one decode step of 16 sequences (latency)
        {"name": "store_step_16", "op": "store", "rows": 16, "hkv": 8, "d": 128, "bs": 16, "dtype": "bf16",
         "gap": 0, "pad": 0},
        # the K/V rows of a step of full prefill chunks, sliced out of a fused projection's rows; MHA
        {"name": "store_prefill_8192", "op": "store", "rows": 8192, "hkv": 32, "d": 128, "bs": 16, "dtype": "f16",
         "gap": 4096, "pad": 37},
        # a short prompt on the small model: one launch's latency
        _attn("chunk_tiny_gqa", "chunk", 1, 4, 1, 64, 16, "f16", 1.0, 1e4, (512, 512), (64, 64)),
        # a mixed batch: ragged chunks on ragged contexts, some of one token
        _attn("chunk_ragged_b8", "chunk", 8, 32, 8, 128, 16, "bf16", 1.0, 5e5, (0, 8192), (1, 512)),
        # one full chunk of a long prompt: the largest compute
        _attn("chunk_long_prompt", "chunk", 1, 32, 8, 128, 16, "bf16", 1.0, 5e5, (30720, 30720), (2048, 2048)),
        # verification of short drafts on long contexts: few rows, all of the cache is read
        _attn("chunk_verify_64k", "chunk", 4, 32, 8, 128, 32, "bf16", 1.0, 5e5, (65500, 65500), (8, 8)),
        # prefill of a sliding-window MHA model: evicted blocks are gone from the table
        _attn("chunk_window_mha", "chunk", 2, 32, 32, 128, 16, "f16", 0.5, 1e4, (9000, 14336), (1024, 1900),
              window=4096, sinks=64),
        # one short windowed decode step (latency)
        _attn("window_tiny_gqa", "window", 1, 4, 1, 64, 16, "f16", 1.0, 1e4, (512, 512), (0, 0), window=256, sinks=4,
              self_visible=0),
        # a wide decode batch on a windowed GQA model: the largest read
        _attn("window_b64_4k", "window", 64, 32, 8, 128, 16, "bf16", 1.0, 5e5, (6000, 32768), (0, 0), window=4096,
              sinks=16, self_visible=1),
        # ragged lengths around the window on an MHA model, the sinks offloaded to mapped host memory
        _attn("window_mha_host", "window", 16, 32, 32, 128, 16, "f16", 0.5, 1e4, (0, 4000), (0, 0), window=1024,
              sinks=4, self_visible=0, host_sinks=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "store", "chunk", "chunk", "window", "window"])
    if op == "tables":
        hi = _log(rng, 1, 4096)
        return {"op": op, "batch": _log(rng, 1, 512), "bs": rng.choice([16, 32, 48, 64, 256]), "ctx_lo": 0,
                "ctx_hi": _log(rng, 1, 16384), "new_lo": rng.randint(0, hi), "new_hi": hi}
    if op == "store":
        rows = _log(rng, 1, 8192)
        return {"op": op, "rows": rows, "hkv": rng.choice([1, 2, 4, 8, 16, 32]), "d": rng.choice([64, 128]),
                "bs": rng.choice([16, 32, 48, 64]), "dtype": rng.choice(["bf16", "f16"]),
                "gap": rng.choice([0, 8, 512, 4096]), "pad": rng.randint(0, rows - 1) // 2}
    while True:
        hkv = rng.choice([1, 2, 4, 8, 16, 32])
        g = rng.choice([1, 2, 4])
        d, bs = rng.choice([64, 128]), rng.choice([16, 32, 48, 64, 128])
        dtype = rng.choice(["bf16", "f16"])
        std, base = rng.choice([(1.0, 5e5), (0.5, 1e4), (0.5, 0.0)])
        if hkv * g > 32:
            continue
        if op == "chunk":
            batch = _log(rng, 1, 12)
            ctx = _log(rng, 1, 65536)
            new = _log(rng, 1, 2048)
            window = rng.choice([0, 0, _log(rng, 16, 8192)])
            sinks = rng.randint(0, 100) if window else 0
            c = _attn("", op, batch, hkv * g, hkv, d, bs, dtype, std, base, (ctx // rng.randint(1, 4), ctx),
                      (rng.randint(1, new), new), window, sinks, rng.randint(0, 1))
            if batch * hkv * g * new * (ctx + new) > 2.2e9 or batch * hkv * d * (ctx + new) > 3.5e8:
                continue
        else:
            batch = _log(rng, 1, 64)
            ctx = _log(rng, 1, 65536)
            window = _log(rng, 16, 8192)
            c = _attn("", op, batch, hkv * g, hkv, d, bs, dtype, std, base, (ctx // rng.randint(1, 4), ctx), (0, 0),
                      window, rng.randint(0, 100), rng.randint(0, 1))
            if batch * hkv * d * min(window, ctx) > 2.7e8:
                continue
        if work(c)["flops"] > 1.1e12:
            continue
        del c["name"]
        return c


# --------------------------------------------------------------------------- inputs

def _spread(lo, hi, n):
    """n whole numbers spread over [lo, hi]; both ends are among them where n allows."""
    got = [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + 0.5) % 1.0)) for i in range(n)]
    got[0] = hi
    if n > 1:
        got[1] = lo
    return got


def _lens(c):
    return _spread(c["ctx_lo"], c["ctx_hi"], c["batch"]), _spread(c["new_lo"], c["new_hi"], c["batch"])[::-1]


def _end(c, ctx, new):
    """Cached tokens that a call on this case may read: the context, the chunk, and a decode step's own token."""
    return ctx + (new if c["op"] == "chunk" else c["self_visible"])


def _visible(c, ctx, new):
    """Tokens of one sequence that some query of the call sees."""
    n = new if c["op"] == "chunk" else 1
    hi = ctx + n - 1 + c["self_visible"]
    if not c["window"]:
        return max(0, hi)
    lo = max(0, ctx + c["self_visible"] - c["window"])
    return max(0, hi - lo) + min(c["sinks"], lo)


def _pairs(c, ctx, new):
    """(query, token) pairs of one sequence that the mask leaves."""
    n = new if c["op"] == "chunk" else 1
    total = 0
    for i in range(n):
        hi = ctx + i + c["self_visible"]
        lo = max(0, hi - c["window"]) if c["window"] else 0
        total += hi - lo + min(c["sinks"], lo)
    return total


def work(case):
    c = case
    if c["op"] == "tables":
        ctx, new = _lens(c)
        blocks = sum((a + b + c["bs"] - 1) // c["bs"] - (a + c["bs"] - 1) // c["bs"] for a, b in zip(ctx, new))
        return {"bytes": 12 * c["batch"] + 8 * blocks + 8 * sum(new), "flops": 0}
    if c["op"] == "store":
        return {"bytes": 8 * c["rows"] + (c["rows"] - c["pad"]) * c["hkv"] * c["d"] * 2 * 2 * 2, "flops": 0}
    ctx, new = _lens(c)
    seen = sum(_visible(c, a, b) for a, b in zip(ctx, new))
    rows = sum(new) if c["op"] == "chunk" else c["batch"]
    size = 2 if c["op"] == "chunk" else 4
    pairs = sum(_pairs(c, a, b) for a, b in zip(ctx, new))
    return {"bytes": seen * c["hkv"] * c["d"] * 4 + 2 * rows * c["hq"] * c["d"] * size,
            "flops": 4 * pairs * c["hq"] * c["d"]}


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=_DEV)


_handles = {}


def _handle(hq, hkv, d, bs, dtype, base, batch, blocks):
    """The library handle that a program keeps for its model: one for each shape."""
    import decode_attention_host_b200 as dkv
    key = (hq, hkv, d, bs, dtype, base, batch, blocks)
    if key not in _handles:
        _handles[key] = dkv.DecodeAttention(hq, hkv, d, bs, dkv.DKV_KV_BF16 if dtype == "bf16" else dkv.DKV_KV_F16,
                                            base, batch, blocks)
    return _handles[key].handle


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=_DEV).manual_seed(int(seed) * 7 + 3)

    def normal(shape, std, dtype):
        return (torch.randn(shape, generator=gen, device=_DEV) * std).to(dtype)

    def perm(n):
        return torch.randperm(n, generator=gen, device=_DEV).to(torch.int32)

    s = {"case": dict(c)}
    if c["op"] == "tables":
        ctx, new = _lens(c)
        held = [-(-a // c["bs"]) for a in ctx]
        total = [-(-(a + b) // c["bs"]) for a, b in zip(ctx, new)]
        cap, taken = max(1, max(total)), sum(total) - sum(held)
        ids = perm(sum(total) + 64)
        col = torch.arange(cap, device=_DEV)
        start = torch.tensor([0] + held, device=_DEV).cumsum(0)[:-1]
        at = (start[:, None] + col[None, :]).clamp(max=len(ids) - 1)
        s["table"] = torch.where(col[None, :] < _ints(held)[:, None], ids[at], -1).to(torch.int32).contiguous()
        s["free_ids"] = ids[sum(held):].clone()
        s["free_count"] = _ints([taken + 64])
        s["ctx"], s["new"] = _ints(ctx), _ints(new)
        s["slots"] = sum(new) + 5       # a few entries behind the last sequence
        if own:
            s["handle"] = _handle(1, 1, 64, c["bs"], "bf16", 0.0, c["batch"], cap)
        return s
    if c["op"] == "store":
        n, width = c["rows"], c["hkv"] * c["d"]
        nblk = -(-n // c["bs"]) + 8
        dt = _DTYPES[c["dtype"]]
        s["new_kv"] = normal((n, 2 * width + c["gap"]), 1.0, dt)   # K, V and what else the projection gives
        shape = (nblk, c["hkv"], c["bs"], c["d"])
        s["k_pool"], s["v_pool"] = torch.zeros(shape, dtype=dt, device=_DEV), torch.zeros(shape, dtype=dt, device=_DEV)
        slots = perm(nblk * c["bs"])[:n].to(torch.int64)
        if c["pad"]:
            slots[-c["pad"]:] = -1
        s["slots"] = slots
        if own:
            s["handle"] = _handle(c["hkv"], c["hkv"], c["d"], c["bs"], c["dtype"], 0.0, 1, nblk)
        return s
    ctx, new = _lens(c)
    bs, dt = c["bs"], _DTYPES[c["dtype"]]
    end = [_end(c, a, b) for a, b in zip(ctx, new)]
    cap = max(1, max(-(-e // bs) for e in end))
    col = torch.arange(cap, device=_DEV)[None, :]
    live = col * bs < _ints(end)[:, None]
    sink = torch.zeros_like(live)
    if c["window"]:     # blocks that no query of this call sees are gone from the table
        lo = (_ints(ctx) + c["self_visible"] - c["window"]).clamp(min=0)[:, None]
        sink = live & (col * bs < c["sinks"]) & ((col + 1) * bs <= lo)
        live = live & (((col + 1) * bs > lo) | (col * bs < c["sinks"]))
    host = sink if c["host_sinks"] else torch.zeros_like(live)
    dev = live & ~host
    s["host_split"], s["dev_blocks"] = int(host.sum()), max(1, int(dev.sum()))
    rank = dev.flatten().long().cumsum(0).view_as(dev) - 1
    hrank = host.flatten().long().cumsum(0).view_as(host) - 1
    ids = perm(s["dev_blocks"]).long()[rank.clamp(min=0)] + s["host_split"]
    s["table"] = torch.where(dev, ids, torch.where(host, hrank, -1)).to(torch.int32).contiguous()
    shape = (s["dev_blocks"], c["hkv"], bs, c["d"])
    s["k_pool"], s["v_pool"] = normal(shape, c["std"], dt), normal(shape, c["std"], dt)
    s["k_host"] = s["v_host"] = None
    if s["host_split"]:
        shape = (s["host_split"], c["hkv"], bs, c["d"])
        s["k_host"], s["v_host"] = (normal(shape, c["std"], dt).cpu().pin_memory() for _ in "kv")
    s["ctx"] = _ints(ctx)
    if c["op"] == "chunk":
        s["q"] = normal((sum(new), c["hq"], c["d"]), 1.0, dt)
        s["q_start"] = torch.tensor([0] + new, device=_DEV).cumsum(0).to(torch.int32)
        s["max_new"] = max(new)
    else:
        s["q"] = normal((c["batch"], c["hq"], c["d"]), 1.0, torch.float32)
    if own:
        s["handle"] = _handle(c["hq"], c["hkv"], c["d"], bs, c["dtype"], c["base"], c["batch"], cap)
    return s


# --------------------------------------------------------------------------- the library's calls

def _own(s):
    import decode_attention_host_b200 as dkv
    c, stream = s["case"], torch.cuda.current_stream().cuda_stream
    if c["op"] == "tables":
        batch, cap = s["table"].shape
        left = torch.empty(1, dtype=torch.int32, device=_DEV)
        q_start = torch.empty(batch + 1, dtype=torch.int32, device=_DEV)
        slot_map = torch.empty(s["slots"], dtype=torch.int64, device=_DEV)
        dkv.dkv_extend_tables(s["handle"], s["ctx"], s["new"], batch, s["table"], cap, s["free_ids"],
                              s["free_ids"].numel(), s["free_count"], left, q_start, slot_map, s["slots"], stream)
        return {"table": s["table"], "q_start": q_start, "slot_map": slot_map, "free_left": left}
    if c["op"] == "store":
        width = c["hkv"] * c["d"]
        dkv.dkv_store_kv(s["handle"], s["new_kv"], s["new_kv"][:, width:], s["new_kv"].stride(0), s["slots"],
                         c["rows"], 0, None, None, s["k_pool"], s["v_pool"], stream, s["k_pool"].shape[0])
        return {"k": s["k_pool"], "v": s["v_pool"]}
    out = torch.empty_like(s["q"])
    batch, cap = s["table"].shape
    if c["op"] == "chunk":
        dkv.dkv_attn_chunk(s["handle"], s["q"], c["hq"] * c["d"], s["q_start"], s["q"].shape[0], s["k_host"],
                           s["v_host"], s["k_pool"], s["v_pool"], s["table"], s["ctx"], s["host_split"], out,
                           c["window"], c["sinks"], c["self_visible"], stream, batch, cap, s["dev_blocks"], None, None)
    else:
        dkv.dkv_attn_decode_window(s["handle"], c["window"], c["sinks"], c["self_visible"], s["q"], s["k_host"],
                                   s["v_host"], s["k_pool"], s["v_pool"], s["table"], s["ctx"], s["host_split"], out,
                                   stream, batch, cap, s["dev_blocks"])
    return out


# --------------------------------------------------------------------------- the plain forms

def _rotate(x, pos, base):
    """NeoX RoPE of x [..., T, D] at positions pos (broadcast to [..., T]): angles in 64 bits, products in 32."""
    if not base:
        return x
    half = x.shape[-1] // 2
    i = torch.arange(half, device=x.device, dtype=torch.float64)
    th = pos.double()[..., None] * torch.pow(torch.tensor(base, device=x.device, dtype=torch.float64), -i / half)
    cos, sin = torch.cos(th).float(), torch.sin(th).float()
    a, b = x[..., :half], x[..., half:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _cache(s, pos):
    """K and V rows of the tokens pos [B, T] in 32 bits, [B, Hkv, T, D]; rows of absent blocks are any row."""
    c = s["case"]
    blk = torch.gather(s["table"].long(), 1, pos // c["bs"]).clamp(min=0)
    k, v = s["k_pool"], s["v_pool"]
    if s["host_split"]:
        k, v = (torch.cat((h.to(_DEV, non_blocking=True), p)) for h, p in ((s["k_host"], k), (s["v_host"], v)))
    else:
        blk = blk - s["host_split"]
    row = pos % c["bs"]
    return k[blk, :, row].float().transpose(1, 2), v[blk, :, row].float().transpose(1, 2)


def _attend(q, k, v, seen, scale):
    """q [B, Hkv, G, N, D], k and v [B, Hkv, T, D], seen [B, 1, 1, N, T]: softmax attention, empty rows zero."""
    b, h, g, n, d = q.shape
    x = torch.matmul(q.reshape(b, h, g * n, d), k.transpose(2, 3)).view(b, h, g, n, -1) * scale
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    x = x.masked_fill(~seen, 0.0)
    total = x.sum(-1, keepdim=True)
    v = torch.where(seen.any(3).transpose(2, 3), v, torch.zeros_like(v))   # rows that no query sees take no part
    o = torch.matmul(x.view(b, h, g * n, -1), v).view(b, h, g, n, d)
    return torch.where(total > 0, o / torch.where(total > 0, total, torch.ones_like(total)), torch.zeros_like(o))


def run(state):
    s = state
    if own:
        return _own(s)
    c = s["case"]
    if c["op"] == "tables":
        bs, cap = c["bs"], s["table"].shape[1]
        ctx, new = s["ctx"].long(), s["new"].long()
        q_start = torch.cat((torch.zeros_like(new[:1]), new.cumsum(0)))
        held, total = (ctx + bs - 1) // bs, (ctx + new + bs - 1) // bs
        first = (total - held).cumsum(0) - (total - held)       # rank of each sequence's first new block
        col = torch.arange(cap, device=_DEV)[None, :]
        rank = first[:, None] + col - held[:, None]
        fresh = (col >= held[:, None]) & (col < total[:, None])
        ids = s["free_ids"][(s["free_count"].long() - 1 - rank).clamp(0, s["free_ids"].numel() - 1)]
        table = torch.where(fresh, ids, s["table"])
        s["table"].copy_(table)
        at = torch.arange(s["slots"], device=_DEV)
        seq = (torch.searchsorted(q_start, at, right=True) - 1).clamp(max=c["batch"] - 1)
        pos = ctx[seq] + at - q_start[seq]
        slot = table[seq, (pos // bs).clamp(max=cap - 1)].long() * bs + pos % bs
        slot = torch.where(at < q_start[-1], slot, torch.full_like(slot, -1))
        left = (s["free_count"].long() - (total - held).sum()).to(torch.int32)
        return {"table": s["table"], "q_start": q_start.to(torch.int32), "slot_map": slot, "free_left": left}
    if c["op"] == "store":
        width, slots = c["hkv"] * c["d"], s["slots"]
        live = slots >= 0
        at = torch.arange(c["rows"], device=_DEV)
        src = torch.where(live, at, live.long().argmax())       # padding rows repeat the first live one
        rows, slot = s["new_kv"][src], slots[src]
        blk, row = slot // c["bs"], slot % c["bs"]
        s["k_pool"][blk, :, row] = rows[:, :width].view(-1, c["hkv"], c["d"])
        s["v_pool"][blk, :, row] = rows[:, width:2 * width].view(-1, c["hkv"], c["d"])
        return {"k": s["k_pool"], "v": s["v_pool"]}
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    batch, cap = s["table"].shape
    scale, ctx = 1.0 / math.sqrt(d), s["ctx"].long()
    if c["op"] == "chunk":
        n, total = s["max_new"], s["q"].shape[0]
        start = s["q_start"].long()
        i = torch.arange(n, device=_DEV)
        q = s["q"][(start[:-1, None] + i).clamp(max=total - 1)].float()          # [B, N, Hq, D], padded
        at = ctx[:, None] + i                                                     # positions of the queries
        q = _rotate(q.transpose(1, 2), at[:, None, :], c["base"]).view(batch, hkv, hq // hkv, n, d)
        t = torch.arange(cap * c["bs"], device=_DEV)[None, :].expand(batch, -1)
        hi = (at + c["self_visible"])[:, :, None]
        seen = (t[:, None, :] < hi) & (i[None, :, None] < (start[1:] - start[:-1])[:, None, None])
        if c["window"]:
            seen = seen & ((t[:, None, :] >= hi - c["window"]) | (t[:, None, :] < c["sinks"]))
        k, v = _cache(s, t)
        o = _attend(q, _rotate(k, t[:, None, :], c["base"]), v, seen[:, None, None], scale)
        row = torch.arange(total, device=_DEV)
        seq = torch.searchsorted(start, row, right=True) - 1
        return o.reshape(batch, hq, n, d).transpose(1, 2)[seq, row - start[seq]].to(s["q"].dtype)
    hi = ctx + c["self_visible"]
    sink, win = torch.arange(c["sinks"], device=_DEV), torch.arange(c["window"], device=_DEV)
    lo = (hi - c["window"]).clamp(min=0)
    t = torch.cat((sink[None, :].expand(batch, -1), lo[:, None] + win[None, :]), 1)
    seen = torch.cat((sink[None, :] < lo[:, None], (lo[:, None] + win[None, :]) < hi[:, None]), 1)
    t = t.clamp(max=cap * c["bs"] - 1)
    k, v = _cache(s, t)
    q = _rotate(s["q"], ctx[:, None].expand(batch, hq), c["base"]).view(batch, hkv, hq // hkv, 1, d)
    o = _attend(q, _rotate(k, t[:, None, :], c["base"]), v, seen[:, None, None, None, :], scale)
    return o.reshape(batch, hq, d)


# --------------------------------------------------------------------------- exact values

def exact(case, seed):
    """The definition, sequence by sequence and head by head, in 64 bits; rotation as a complex product."""
    c = case
    if c["op"] == "tables":
        return None
    s = prepare(c, seed)
    if c["op"] == "store":
        out, width = {}, c["hkv"] * c["d"]
        slots = s["slots"].tolist()
        keep = [i for i, x in enumerate(slots) if x >= 0]
        dst = torch.tensor([slots[i] for i in keep], device=_DEV)
        for name, off in (("k", 0), ("v", width)):
            pool = s[name + "_pool"].double().transpose(1, 2).reshape(-1, width)       # one line for each slot
            pool[dst] = s["new_kv"][keep, off:off + width].double()
            out[name] = pool.view(-1, c["bs"], c["hkv"], c["d"]).transpose(1, 2).contiguous()
        return out
    bs, hkv, d, base = c["bs"], c["hkv"], c["d"], c["base"]
    group, half = c["hq"] // hkv, d // 2
    freq = [base ** (-2.0 * i / d) if base else 0.0 for i in range(half)]
    freq = torch.tensor(freq, dtype=torch.float64, device=_DEV)

    def turned(x, pos):
        ang = pos.double()[:, None] * freq[None, :]
        z = torch.complex(x[:, :half], x[:, half:]) * torch.polar(torch.ones_like(ang), ang)
        return torch.cat((z.real, z.imag), 1)

    ctx, new = _lens(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=_DEV)
    first = 0
    for b in range(c["batch"]):
        n = new[b] if c["op"] == "chunk" else 1
        at = ctx[b] + torch.arange(n, device=_DEV)
        end = ctx[b] + n - 1 + c["self_visible"]
        t = torch.arange(max(0, end), device=_DEV)
        if c["window"]:
            lo = max(0, ctx[b] + c["self_visible"] - c["window"])
            t = t[(t >= lo) | (t < c["sinks"])]
        if len(t) == 0:
            first += n
            continue
        blocks = s["table"][b].long()[t // bs]
        on_host = (blocks < s["host_split"])[:, None]
        last = at[:, None] + c["self_visible"]
        seen = t[None, :] < last
        if c["window"]:
            seen = seen & ((t[None, :] >= last - c["window"]) | (t[None, :] < c["sinks"]))
        for h in range(hkv):
            k = s["k_pool"][(blocks - s["host_split"]).clamp(min=0), h, t % bs].double()
            v = s["v_pool"][(blocks - s["host_split"]).clamp(min=0), h, t % bs].double()
            if s["host_split"]:
                hb = blocks.clamp(max=s["host_split"] - 1)
                k = torch.where(on_host, s["k_host"].to(_DEV)[hb, h, t % bs].double(), k)
                v = torch.where(on_host, s["v_host"].to(_DEV)[hb, h, t % bs].double(), v)
            k = turned(k, t).T
            for j in range(h * group, (h + 1) * group):
                x = turned(s["q"][first:first + n, j].double(), at) @ k
                x = torch.where(seen, x / d ** 0.5, -math.inf)
                p = torch.softmax(x, 1)
                p = torch.where(seen.any(1, keepdim=True), p, torch.zeros_like(p))
                out[first:first + n, j] = p @ v
        first += n
    return out
