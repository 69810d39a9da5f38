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


def attn_of(kv, dtype, g, base, scale=0.0):
    return dkv.DecodeAttention(kv.num_kv_heads * g, kv.num_kv_heads, kv.head_dim, kv.block_size,
                               dkv.DKV_KV_BF16 if dtype == "bf16" else dkv.DKV_KV_F16, base, kv.batch, kv.stride,
                               scale=scale)


def two_token_case():
    """Scores of two tokens, 0 and up to +-1 apart: q (component 0) of 300 sequences x 16 heads."""
    g = torch.Generator().manual_seed(7)
    return torch.rand((300, 16), generator=g) * 2 - 1


@pytest.mark.parametrize("g", [1, 2, 4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_weights_of_two_tokens(dtype, d, g):
    """The second token's value is 1, the first one's 0: the output is a weight, and shows its every bit."""
    s = two_token_case()
    batch, hq = s.shape
    hkv = hq // g
    k, v = torch.zeros((2, hkv, d)), torch.zeros((2, hkv, d))
    k[1, :, 0] = v[1] = 1.0
    kv = shared(2, batch, hkv, d, 16, dtype, k.to(sc.DTYPES[dtype]), v.to(sc.DTYPES[dtype]))
    attn = attn_of(kv, dtype, g, 0.0, scale=1.0)
    q = torch.zeros((batch, hq, d), device="cuda")
    q[..., 0] = s.cuda()
    out = torch.full_like(q, 7.0)
    attn.window(q, kv, out, 2)
    torch.cuda.synchronize()
    assert attn.status() == 0
    want = torch.sigmoid(s.double())[..., None].expand(batch, hq, d).cuda()
    sc.check(out, want, weight_bound(dtype, s.abs().double(), 2).cuda() * want + 2.0 ** -24 * want)
    attn.close()


# Rotation state of a key: a seed from __sincosf (2^-20.8 of the pair), then one fp32 rotation by 4 positions for each
# step, 63 at most.  Root mean square over tokens and pairs, of the pair's norm: the step factors' own rounding,
# 2^-24 / sqrt(12) in each of two, is the same in every step and adds up to 63 / sqrt(3) times 2.4e-8 = 8.8e-7; two
# roundings of each step add up like a walk, sqrt(63 / 2) * 2 * 1.7e-8 = 1.9e-7; the seeds of key and query are off by
# 5.5e-7 each at most.  Together 1.2e-6.
ROTATION_RMS = 1.2e-6
SCORE = 4.0             # |q| |k| scale of each pair


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,base", [(64, 1e4), (128, 1e4), (128, 5e5)])
def test_rotation_of_each_pair(d, base, dtype):
    """One kv head for each pair, with nothing else in q and k; v of token t is the unit vector t mod D: the output
    holds the weights one by one.  256 tokens of a sequence are one chain of rotations."""
    pairs, ctx = d // 2, 256
    batch = 4736 // pairs     # enough sequences that a unit is a whole sequence
    k, v = torch.zeros((ctx, pairs, d)), torch.zeros((ctx, pairs, d))
    h = torch.arange(pairs)
    k[:, h, h] = 1.0
    t = torch.arange(ctx)
    v[t, :, t % d] = 1.0
    kv = shared(ctx, batch, pairs, d, 16, dtype, k.to(sc.DTYPES[dtype]), v.to(sc.DTYPES[dtype]))
    attn = attn_of(kv, dtype, 1, base, scale=1.0)
    q = torch.zeros((batch, pairs, d), device="cuda")
    q[:, h, h] = SCORE
    out = torch.full_like(q, 7.0)
    attn.window(q, kv, out, ctx)
    torch.cuda.synchronize()
    assert attn.status() == 0 and torch.equal(out, out[:1].expand_as(out))
    want = sc.attend64(q[:1], k, v, ctx, base, 0, ctx, 0, scale=1.0)[0]
    off = (out[:1].double() / want - 1.0)
    rms = off.pow(2).mean().sqrt().item()
    # the weights' sum moves all of a row's weights alike, by no more; 5e-7 for the weights themselves
    assert rms <= 2 ** 0.5 * ROTATION_RMS * SCORE + 5e-7, rms
    attn.close()


def test_a_repeat_on_another_stream_writes_every_output():
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((900, 2, 128), generator=g).bfloat16() for _ in "kv")
    kv = shared(900, 5, 2, 128, 16, "bf16", k, v)
    attn = attn_of(kv, "bf16", 4, 1e4)
    q = torch.randn((5, 8, 128), generator=g).cuda()
    out = torch.full_like(q, 7.0)
    attn.window(q, kv, out, 300, 4)
    torch.cuda.synchronize()
    first = out.clone()
    out.fill_(7.0)
    torch.cuda.synchronize()
    attn.window(q, kv, out, 300, 4, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(first, out) and not (out == 7.0).any()
    # a window over everything is the plain decode step: either call writes every output
    for call in (lambda: attn.window(q, kv, out, 900), lambda: attn(q, kv, out)):
        out.fill_(7.0)
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        for b in range(5):
            want = sc.attend64(q[b:b + 1], k, v, 900, 1e4, 0, 0, 0)
            sc.check(out[b:b + 1], want[0], sc.bound32(want[1], want[2]))
    attn.close()
