"""Chunk attention: the error that its roundings leave, and no more (needs a B200).

One rounding to fp16 of a number with a log-uniform mantissa is off by 2^-11 / sqrt(3) * sqrt((3/8) / ln 2) = 2.07e-4
of it, root mean square; to bf16 by 8 times that.  With q, k and v drawn from N(0, 1) the scores have variance 1, and
  - the output's own rounding and that of the weights leave one rounding of the cache's type each,
  - rotated queries and keys, held in fp16, move each score by scale * sqrt(sum q^2 k^2) * 2.07e-4 each, 2.07e-4 in the
    mean, and the output by as much of its norm; without rotation they are exact.
The squares add up.  The bound lies 10% above: the sums run over more than 10^4 outputs.
"""
import pytest
import torch

from tests import serving_cases as sc
from tests.test_gpu_chunk import Chunk

pytestmark = pytest.mark.gpu

ONE = 2.0 ** -11 / 3 ** 0.5 * (0.375 / 0.6931) ** 0.5


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("base", [0.0, 1e4])
@pytest.mark.parametrize("ctx,new,hkv,g,d,s", [
    (512, 64, 1, 4, 64, 16), (3000, 300, 2, 1, 64, 64), (3000, 300, 2, 1, 128, 128), (4000, 20, 2, 4, 128, 48)])
def test_error_of_a_chunk_is_that_of_its_roundings(ctx, new, hkv, g, d, s, base, dtype):
    c = Chunk([ctx], [new], hkv=hkv, g=g, d=d, s=s, dtype=dtype, base=base, seed=51 + d + new)
    c.run()
    c.verify()
    want = sc.attend64(c.q, c.cache.k[0], c.cache.v[0], ctx, base, 1, 0, 0)[0]
    rel = ((c.out.double() - want).norm() / want.norm()).item()
    own = ONE * (8 if dtype == "bf16" else 1)
    assert rel <= 1.1 * (2 * own ** 2 + (2 * ONE ** 2 if base else 0.0)) ** 0.5, rel
    c.free()
