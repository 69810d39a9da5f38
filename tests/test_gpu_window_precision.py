"""Precision of the windowed decode (needs a B200): its fp32 output against the 64-bit definition, under bounds that
follow from how the kernel holds weights and rotations."""
from types import SimpleNamespace

import pytest
import torch

import decode_attention_host_b200 as dkv
from tests import serving_cases as sc

pytestmark = pytest.mark.gpu

# A weight is 2^(s - ref + bias) in 32 bits, split into three bf16 parts (2^-9 each: 2^-27) or two fp16 parts (2^-11
# each: 2^-22; the second one counts in steps of 2^-11, so that what falls under fp16's smallest number is off by
# 2^-43 of the reference).  ex2.approx is off by 2^-22.
FLOOR = {"f16": 2.0 ** -43, "bf16": 0.0}
SPLIT = {"f16": 2.0 ** -22, "bf16": 2.0 ** -27}


def weight_bound(dtype, spread, adds):
    """Relative error of sum p |v| for scores that are one product each (a single non-zero component of q and k, no
    rotation): 4 roundings of the score, the exponential, the parts, and `adds` fp32 additions in a chain (2^-23 each:
    the tensor core may cut instead of rounding), in the output and in the sum that divides it."""
    return 2.0 * torch.expm1(4 * 2.0 ** -24 * spread)[..., None] + 2 * 2.0 ** -22 + SPLIT[dtype] + \
        2 * adds * 2.0 ** -23


def shared(ctx, batch, hkv, d, s, dtype, k, v):
    """`batch` sequences of `ctx` tokens that all name the same blocks: k, v [ctx, hkv, d] in a device pool."""
    n = -(-ctx // s)
    pools = []
    for x in (k, v):
        p = torch.full((n * s, hkv, d), float("nan"), dtype=sc.DTYPES[dtype])
        p[:ctx] = x
        pools.append(p.view(n, s, hkv, d).transpose(1, 2).contiguous().cuda())
    none = SimpleNamespace(ptr=0)
    return SimpleNamespace(batch=batch, stride=n, num_kv_heads=hkv, head_dim=d, block_size=s, host_split=0,
                           num_dev_blocks=n, k_host=none, v_host=none, k_dev=pools[0], v_dev=pools[1],
                           table_dev=torch.arange(n, dtype=torch.int32, device="cuda").repeat(batch, 1),
                           seq_lens_dev=torch.full((batch,), ctx, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("gap", [12.0, 17.5, 20.0])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_small_weights_beside_a_sink(dtype, gap):
    """One dominating token whose value is zero, the other weights up to 2^-28.9 of its own and of one sign."""
    ctx, batch, hkv, d = 8192, 148, 8, 64
    k, v = torch.zeros((ctx, hkv, d)), torch.full((ctx, hkv, d), 60.0)
    k[0, :, 0], v[0] = gap, 0.0
    kv = shared(ctx, batch, hkv, d, 64, dtype, k.to(sc.DTYPES[dtype]), v.to(sc.DTYPES[dtype]))
    attn = dkv.DecodeAttention(hkv, hkv, d, 64, dkv.DKV_KV_BF16 if dtype == "bf16" else dkv.DKV_KV_F16, 0.0, batch,
                               kv.stride)
    q = torch.zeros((batch, hkv, d), device="cuda")
    q[..., 0] = d ** 0.5
    out = torch.full_like(q, 7.0)
    attn.window(q, kv, out, ctx)
    torch.cuda.synchronize()
    assert attn.status() == 0
    want, mass, spread = sc.attend64(q[:1], k, v, ctx, 0.0, 0, ctx, 0)
    bound = weight_bound(dtype, spread, ctx // 16) * mass + ctx * FLOOR[dtype] * 60.0 + 2.0 ** -24 * want.abs()
    for b in range(batch):
        sc.check(out[b:b + 1], want, bound)
    attn.close()
