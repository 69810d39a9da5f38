"""Which rows of a chunk become NaN (needs a B200): those that see a token of an invalid block or with a key out of
range, and the query out of range itself; the rows computed together with them keep their values."""
import pytest
import torch

import decode_attention_host_b200 as dkv
from tests.test_gpu_chunk import Chunk

pytestmark = pytest.mark.gpu

CTX, NEW = 100, 60      # 240 rows of a kv head: one CTA of 256 rows, or two of 128 beside an empty sequence


def make(window, beside, dtype="bf16"):
    # a second sequence without rows halves the average rows of a sequence, and with it the rows of a CTA
    c = Chunk([CTX] + [5] * beside, [NEW] + [0] * beside, window=window, sinks=2 if window else 0, dtype=dtype, seed=61)
    c.run()
    assert c.attn.status() == 0
    return c, c.out.clone()


def seeing(tokens, window):
    """bool [NEW]: the rows that see one of the tokens."""
    hi = torch.arange(NEW) + CTX + 1
    m = torch.zeros(NEW, dtype=torch.bool)
    for t in tokens:
        m |= (t < hi) & ((t >= hi - window) | (t < 2) if window else torch.ones(NEW, dtype=torch.bool))
    return m.cuda()


def verify(c, good, nan_rows, status):
    c.out.fill_(7.0)
    c.run()
    assert c.attn.status() == status
    assert c.out[nan_rows].isnan().all() and torch.equal(c.out[~nan_rows], good[~nan_rows])


@pytest.mark.parametrize("beside", [0, 1])
@pytest.mark.parametrize("window,token", [(0, 0), (0, 99), (0, 100), (0, 141), (0, 159), (20, 1), (20, 85), (20, 100),
                                          (20, 141), (20, 159)])
def test_a_key_out_of_range(window, token, beside):
    c, good = make(window, beside)
    bid = int(c.cache.table[0, token // 16]) - c.cache.host_split
    c.cache.k_dev[bid, :, token % 16, 3] = 1e6
    verify(c, good, seeing([token], window), dkv.DKV_STATUS_RANGE)
    c.free()


@pytest.mark.parametrize("beside", [0, 1])
@pytest.mark.parametrize("window,block", [(0, 0), (0, 6), (0, 7), (0, 9), (20, 0), (20, 6), (20, 7), (20, 9)])
def test_an_invalid_block(window, block, beside):
    c, good = make(window, beside)
    c.cache.table_dev[0, block] = -5
    verify(c, good, seeing(range(16 * block, 16 * block + 16), window), dkv.DKV_STATUS_BAD_BLOCK_ID)
    c.free()


@pytest.mark.parametrize("beside", [0, 1])
def test_a_query_out_of_range(beside):
    c, good = make(0, beside)
    c.q[25, 3, 9] = 1e6
    c.q[41, 0, 70] = -1e6
    c.out.fill_(7.0)
    c.run()
    assert c.attn.status() == dkv.DKV_STATUS_RANGE
    nan = torch.zeros(c.out.shape[:2], dtype=torch.bool, device="cuda")
    nan[25, 3] = nan[41, 0] = True
    assert c.out[nan].isnan().all() and torch.equal(c.out[~nan], good[~nan])
    c.free()


def test_a_key_that_rounds_to_the_largest_number_is_in_range():
    c, _ = make(0, 0)
    bid = int(c.cache.table[0, 0]) - c.cache.host_split     # token 0 is not turned
    c.cache.k_dev[bid, :, 0, 3] = 65280.0                   # the largest bf16 below 65504
    c.out.fill_(7.0)
    c.run()
    assert c.attn.status() == 0 and torch.isfinite(c.out.float()).all()
    c.free()
