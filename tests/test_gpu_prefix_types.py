"""Shared prefixes: the types and head sizes of the CUDA cores over every cache,
and e4m3 values that are not finite."""
import pytest
import torch

import test_gpu_prefix_attention as tp
from test_gpu_prefix_attention import _built   # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,qt,hd", [("e4m3", "bf16", 32), ("e4m3", "bf16", 512), ("f32", "bf16", 32), ("f32", "bf16", 64), ("f32", "bf16", 128),
                                      ("f32", "bf16", 256), ("f32", "bf16", 512), ("f32", "f32", 512), ("e4m3", "f32", 32), ("e4m3", "f32", 512),
                                      ("bf16", "f32", 32), ("bf16", "f32", 512), ("e4m3", "f32", 128)])
def test_types_and_heads(kv, qt, hd):
    """Two groups and a sequence of none, prefixes that end inside pages, one sequence without a new row."""
    start, pre = [0, 3, 5], [150, 33]
    own, n, page, hkv, G = [10, 0, 65, 7, 0, 90], [3, 1, 0, 2, 3, 3], 32, 2, 3
    lens = [a + tp.of_group(b, start, pre)[0] for b, a in enumerate(own)]
    pool = tp.shared_pool(lens, n, start, pre, page, hkv, hd, kv, 1, "slot")
    q = tp.queries(6, 3, hkv * G, hd, torch.bfloat16 if qt == "bf16" else torch.float32, seed=3)
    gain = 1 + 0.1 * torch.randn(hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    out, st = tp.run(pool, q, lens, start, pre, n, gain, rope_theta=1e4)
    assert st == tp.mtp().MTP_OK
    tp.check(pool, out, q, gain, lens, n, start, pre, 1e4)


@pytest.mark.parametrize("hd", [32, 64, 128, 256, 512])
@pytest.mark.parametrize("qt", ["bf16", "f32"])
def test_e4m3_values_that_are_not_finite(qt, hd):
    """A NaN of the prefix reaches its group's rows in its dimension, one of a
    sequence's own positions the rows that attend it."""
    m = tp.mtp()
    lens, start, pre = [150, 130, 140, 300], [0, 2, 3], [100, 0]
    pool = tp.shared_pool(lens, [2] * 4, start, pre, 16, 1, hd, "e4m3", 18)
    q = tp.queries(4, 2, 4, hd, torch.bfloat16 if qt == "bf16" else torch.float32, seed=19)
    want, _ = tp.run(pool, q, lens, start, pre, rope_theta=1e4)
    codes = pool.v.view(torch.uint8)
    codes[int(pool.table[0, 3]), 0, 5, 9] = 0x7F               # position 53: in the prefix of 0 and 1
    codes[int(pool.table[1, 8]), 0, 3, 20] = 0xFF              # position 131: row 1 of sequence 1
    codes[int(pool.table[3, 18]), 0, 13, 2] = 0x7F             # position 301: row 1 of sequence 3
    out, st = tp.run(pool, q, lens, start, pre, rope_theta=1e4)
    assert st == m.MTP_OK
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:2, :, :, 9] = True
    hit[1, 1, :, 20] = True
    hit[3, 1, :, 2] = True
    assert out[hit].isnan().all()
    assert ((out.float() - want.float()).abs()[~hit] <= 2.0 ** -5 * (1 + want.float().abs()[~hit])).all()


def test_a_key_that_is_not_finite_stays_with_the_rows_that_attend_it():
    for kv, hd in (("bf16", 64), ("bf16", 128), ("bf16", 256), ("e4m3", 128), ("e4m3", 256), ("f32", 64)):
        lens, start, pre = [150, 130, 140, 300], [0, 2, 3], [100, 0]
        pool = tp.shared_pool(lens, [2] * 4, start, pre, 16, 1, hd, kv, 21)
        q = tp.queries(4, 2, 4, hd, torch.bfloat16 if kv != "f32" else torch.float32, seed=22)
        want, _ = tp.run(pool, q, lens, start, pre, rope_theta=1e4)
        cell = int(pool.table[1, 8]), 0, 3, 20                  # position 131 of sequence 1: its row 1
        if kv == "e4m3":
            pool.k.view(torch.uint8)[cell] = 0x7F
        else:
            pool.k[cell] = float("nan")
        out, st = tp.run(pool, q, lens, start, pre, rope_theta=1e4)
        assert st == tp.mtp().MTP_OK
        keep = torch.ones_like(out, dtype=torch.bool)
        keep[1, 1] = False
        assert ((out.float() - want.float()).abs()[keep] <= 2.0 ** -5 * (1 + want.float().abs()[keep])).all()
