"""Shared set-up of the serving tests: a paged cache with poisoned gaps, and the 64-bit references.

Every pool row that no call may read holds NaN, and every table entry that no call may read holds an
invalid id, so a read outside the visible tokens shows in the output or in the status word.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import decode_attention_host_b200 as dkv

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # largest relative error of one rounding
NAN16 = 0x7FFF                                           # a NaN in both 16-bit types


class Cache:
    """Logical K/V rows of ragged sequences in shuffled blocks of a host and a device pool.

    ``end[b]`` tokens of sequence b are stored; blocks j with keep(b, j) false are left out of the table
    (-1) and of the pools.  Has the attributes of dkv.PagedKV that DecodeAttention reads.
    """

    def __init__(self, end, hkv, d, s, dtype, seed, host=0.0, std=1.0, keep=None, spare=3, extra_cols=2,
                 dev_blocks=None):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.end, self.hkv, self.d, self.s, self.dtype = list(end), hkv, d, s, dtype
        self.batch, self.num_kv_heads, self.head_dim, self.block_size = len(end), hkv, d, s
        dt = DTYPES[dtype]
        self.k = [(torch.randn((e, hkv, d), generator=g) * std).to(dt) for e in end]
        self.v = [(torch.randn((e, hkv, d), generator=g) * std).to(dt) for e in end]
        need = [-(-e // s) for e in end]
        self.stride = max(1, max(need)) + extra_cols
        where = {}
        for b, n in enumerate(need):
            for j in range(n):
                if keep is None or keep(b, j):
                    where[b, j] = rng.random() < host
        n_host = sum(where.values())
        n_dev = len(where) - n_host
        self.host_split = n_host + (spare if host > 0 else 0)
        self.num_dev_blocks = max(n_dev + spare, dev_blocks or 0)
        host_ids = rng.permutation(self.host_split)[:n_host].tolist()
        if dev_blocks:      # the last blocks of a pool too large to fill
            dev_ids = (self.num_dev_blocks - 1 - rng.permutation(n_dev + spare)[:n_dev] + self.host_split).tolist()
        else:
            dev_ids = (rng.permutation(self.num_dev_blocks)[:n_dev] + self.host_split).tolist()
        table = np.full((self.batch, self.stride), -1, np.int32)
        shape = (hkv, s, d)
        blk = hkv * s * d
        self.k_host, self.v_host = dkv.HostPool(self.host_split * blk), dkv.HostPool(self.host_split * blk)
        pools = {}
        for name in ("k", "v"):
            (self.k_host if name == "k" else self.v_host).array[:] = NAN16
            make = torch.empty if dev_blocks else torch.full
            args = ((self.num_dev_blocks, *shape),) if dev_blocks else ((self.num_dev_blocks, *shape), NAN16)
            pools[name] = make(*args, dtype=torch.int16, device="cuda").view(dt)
        host_view = {"k": self._host_view(self.k_host), "v": self._host_view(self.v_host)}
        for (b, j), on_host in where.items():
            n = min(s, end[b] - j * s)
            bid = host_ids.pop() if on_host else dev_ids.pop()
            table[b, j] = bid
            for name, rows in (("k", self.k[b]), ("v", self.v[b])):
                part = rows[j * s:j * s + n].transpose(0, 1)
                if on_host:
                    host_view[name][bid, :, :n] = part
                else:
                    pools[name][bid - self.host_split, :, :n] = part.cuda()
                    if dev_blocks:
                        pools[name][bid - self.host_split, :, n:] = float("nan")
        self.k_dev, self.v_dev = pools["k"], pools["v"]
        self.table = table
        self.table_dev = torch.from_numpy(table).cuda()
        self.seq_lens_dev = torch.tensor(end, dtype=torch.int32, device="cuda")

    def _host_view(self, pool):
        n = self.host_split * self.hkv * self.s * self.d
        return torch.from_numpy(pool.array[:n].view(np.int16)).view(DTYPES[self.dtype]).view(
            self.host_split, self.hkv, self.s, self.d)

    def set_lens(self, lens):
        self.seq_lens_dev.copy_(torch.tensor(list(lens), dtype=torch.int32))

    def free(self):
        torch.cuda.synchronize()
        self.k_host.free()
        self.v_host.free()


def rotate64(x, pos, base):
    """NeoX RoPE in 64 bits: x [..., T, D] at positions pos [T]."""
    if not base:
        return x
    d = x.shape[-1]
    w = torch.tensor([base ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None] * w
    c, s = torch.cos(ang), torch.sin(ang)
    a, b = x[..., :d // 2], x[..., d // 2:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def visible(ctx, n, self_, window, sinks):
    """bool [n, ctx + n]: token t is seen by query i."""
    hi = torch.arange(n)[:, None] + ctx + self_
    t = torch.arange(ctx + n)[None, :]
    m = t < hi
    if window:
        m = m & ((t >= hi - window) | (t < sinks))
    return m


def attend64(q, k, v, ctx, base, self_, window, sinks, scale=None):
    """q [n, Hq, D] at positions ctx .., k and v [>= ctx + n - 1 + self, Hkv, D]: (out, mass, spread).

    mass[n, Hq, D] = sum_t p_t |v_t| and spread[n, Hq] = max over visible t of scale * sum over pairs
    |q pair| |k pair|: what rounding errors of the weights and of the rotated operands multiply.
    """
    n, hq, d = q.shape
    hkv = k.shape[1]
    scale = scale or 1.0 / math.sqrt(d)
    m = visible(ctx, n, self_, window, sinks)[:, :k.shape[0]].cuda()
    t = torch.arange(m.shape[1], device="cuda")
    kk, vv = (x[:m.shape[1]].cuda().double().permute(1, 0, 2) for x in (k, v))
    kk, vv = (torch.where(m.any(0)[None, :, None], x, torch.zeros_like(x)) for x in (kk, vv))
    kk = rotate64(kk, t, base).repeat_interleave(hq // hkv, 0)
    vv = vv.repeat_interleave(hq // hkv, 0)
    qq = rotate64(q.cuda().double().permute(1, 0, 2), ctx + torch.arange(n, device="cuda"), base)
    s = (qq @ kk.transpose(1, 2) * scale).masked_fill(~m, -math.inf)
    p = torch.softmax(s, -1)
    p = torch.where(m.any(1)[None, :, None], p, torch.zeros_like(p))
    norm = lambda x: torch.sqrt(x[..., :d // 2] ** 2 + x[..., d // 2:] ** 2)  # noqa: E731
    spread = (norm(qq) @ norm(kk).transpose(1, 2) * scale).masked_fill(~m, 0.0)
    spread = spread.amax(-1) if m.shape[1] else torch.zeros(hq, n, device="cuda")
    return (p @ vv).permute(1, 0, 2), (p @ vv.abs()).permute(1, 0, 2), spread.permute(1, 0)


def bound16(out, mass, spread, dtype, rotated=True):
    """Largest error of a 16-bit output computed from 16-bit weights and 16-bit rotated operands.

    A weight exp(s) is off by its own rounding u and by the error of s: both operands of each score are
    rotated in fp32 and rounded once to fp16 (2^-11 each, per component, so 2^-11 of the pair's norm; the
    fp32 angle adds 2^-19), or taken as stored.  The weights' sum is off by no more, so the output is off
    by at most 2 (u + ds) sum p |v|, and by its own rounding u |out|.  2^-18 covers the fp32 sums.
    """
    u = HALF_STEP[dtype]
    ds = (2.0 * (2.0 ** -11 + 2.0 ** -19) if rotated else 0.0) * spread + 2.0 ** -18 * (1 + spread)
    ds = torch.expm1(ds)
    return u * out.abs() + 2.05 * (u + ds)[..., None] * mass + 1e-7


def bound32(mass, spread):
    """Largest error of the fp32 decode output: rotated keys are off by at most 5e-5 of the pair's norm (the
    recurrence's documented bound), queries by 1e-6; weights are split into two 16-bit parts (2^-16)."""
    ds = torch.expm1(5.2e-5 * spread + 2.0 ** -18 * (1 + spread))
    return 2.05 * (2.0 ** -16 + ds)[..., None] * mass + 1e-7


def check(got, want, bound):
    got = got.double()
    assert torch.isfinite(got).all(), "non-finite output"
    worst = ((got - want).abs() - bound).amax().item() if got.numel() else -1.0
    ratio = ((got - want).abs() / bound).amax().item() if got.numel() else 0.0
    assert worst <= 0, f"error {ratio:.2f} times its bound"
    return ratio
