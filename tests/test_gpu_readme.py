"""The serving step that the README shows, run as it stands there (needs a B200), on the framework's own cache."""
import re
from pathlib import Path

import numpy as np
import pytest
import torch

import decode_attention_host_b200 as dkv
from tests import serving_cases as sc

pytestmark = pytest.mark.gpu

ROOT = Path(__file__).resolve().parent.parent


def test_the_serving_step_of_the_readme():
    blocks = re.findall(r"```python\n(.*?)```", (ROOT / "README.md").read_text(), re.S)
    step = next(b for b in blocks if "attn.extend" in b)
    Hq, Hkv, D, lens, new = 8, 2, 128, np.array([300, 0, 77], np.int32), [20, 130, 1]
    g = torch.Generator().manual_seed(1)
    draw = lambda *s: torch.randn(s, generator=g).bfloat16()  # noqa: E731
    old = [[draw(n, Hkv, D) for n in lens] for _ in "kv"]
    bits = np.zeros((2, len(lens), Hkv, lens.max(), D), np.uint16)
    for i in range(2):
        for b, n in enumerate(lens):
            bits[i, b, :, :n] = old[i][b].transpose(0, 1).contiguous().view(torch.int16).numpy().view(np.uint16)
    rows = sum(new)
    q, k_new, v_new = draw(rows, Hq, D), draw(rows, Hkv, D), draw(rows, Hkv, D)
    q_dec = torch.randn((len(lens), Hq, D), generator=g)
    env = dict(dkv=dkv, k=bits[0], v=bits[1], lens=lens, Hq=Hq, Hkv=Hkv, D=D, max_slots=256,
               new_lens=torch.tensor(new, dtype=torch.int32, device="cuda"), q=q.cuda(), k_new=k_new.cuda(),
               v_new=v_new.cuda(), q_dec=q_dec.cuda(), out=torch.full((rows, Hq, D), 7.0).bfloat16().cuda(),
               out_dec=torch.full((len(lens), Hq, D), 7.0, device="cuda"))
    exec(step, env)
    torch.cuda.synchronize()
    kv, attn = env["kv"], env["attn"]
    assert attn.status() == 0
    at, taken = 0, 0
    for b, n in enumerate(new):
        ctx = int(lens[b])
        kk, vv = (torch.cat((o[b], x[at:at + n])) for o, x in zip(old, (k_new, v_new)))
        want = sc.attend64(q[at:at + n], kk, vv, ctx, 5e5, 1, 100, 16)
        sc.check(env["out"][at:at + n], want[0], sc.bound16(*want, "bf16"))
        want = sc.attend64(q_dec[b:b + 1], kk, vv, ctx + n, 5e5, 0, 100, 16)
        sc.check(env["out_dec"][b:b + 1], want[0], sc.bound32(want[1], want[2]))
        at += n
        taken += -(-(ctx + n) // 16) - -(-ctx // 16)
    assert kv.free_count.item() == 128 - taken and kv.seq_lens_dev.tolist() == (lens + new).tolist()
    attn.close()
    kv.free()


def test_a_cache_without_spare_blocks_grows_by_none():
    lens = np.array([16], np.int32)
    bits = np.zeros((1, 1, 16, 64), np.uint16)
    kv = dkv.PagedKV(bits, bits, lens, 16, dkv.DKV_PLACE_PREFIX_HOST, 0.0, stride=4)
    attn = dkv.DecodeAttention(1, 1, 64, 16, dkv.DKV_KV_F16, 0.0, 1, 4)
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    attn.extend(kv, one, kv.free_ids, kv.free_count, 4)
    assert attn.status() == dkv.DKV_STATUS_NO_FREE_BLOCKS and kv.table_dev.tolist() == [[0, -1, -1, -1]]
    with pytest.raises(ValueError):
        dkv.PagedKV(bits, bits, lens, 16, dkv.DKV_PLACE_PREFIX_HOST, 0.0, spare_blocks=-1)
    attn.close()
    kv.free()
