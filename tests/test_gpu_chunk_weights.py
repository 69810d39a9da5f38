"""Chunk attention with weights far below a row's largest (needs a B200): one dominating token, an attention sink, and
tens of thousands of small weights of one sign, whose sum is the whole of the output."""
import pytest
import torch

from tests import serving_cases as sc
from tests.test_gpu_chunk import Chunk

pytestmark = pytest.mark.gpu

# A weight is held in fp16 as 2^(s - ref + 11), the reference at most 2^4 below the row's maximum: a normal number
# down to 2^-25 of the reference, and below that off by at most half a subnormal step, 2^-25, so 2^-36 of it.
FLOOR = 2.0 ** -36


@pytest.mark.parametrize("gap", [12.0, 17.5, 20.0])
@pytest.mark.parametrize("new", [3, 300])          # 128 rows to a CTA, and 256
@pytest.mark.parametrize("d,dtype", [(64, "f16"), (128, "f16"), (64, "bf16")])
def test_small_weights_beside_a_sink(d, dtype, new, gap):
    ctx = 65536
    c = Chunk([ctx], [new], hkv=1, g=1, d=d, s=64, dtype=dtype, base=0.0, seed=41)
    k, bid = c.cache, int(c.cache.table[0, 0]) - c.cache.host_split
    k.k_dev.zero_()
    k.v_dev.fill_(60.0)
    k.k[0].zero_()
    k.v[0].fill_(60.0)
    for kk, vv in ((k.k_dev[bid, 0, 0], k.v_dev[bid, 0, 0]), (k.k[0][0, 0], k.v[0][0, 0])):
        kk[0] = gap
        vv.zero_()
    c.q.zero_()
    c.q[..., 0] = d ** 0.5
    c.run()
    assert c.attn.status() == 0
    out, mass, spread = sc.attend64(c.q, k.k[0], k.v[0], ctx, 0.0, 1, 0, 0)
    floor = (ctx + new) * FLOOR * 60.0 if dtype == "f16" else 0.0
    sc.check(c.out, out, sc.bound16(out, mass, spread, dtype, rotated=False) + floor)
    c.free()
