"""mtp_kv_append into an e4m3 cache around the sizes at which its launch
changes: calls of few rows a page run in one block shape, larger ones in
blocks as narrow as half of their rows' 16-element units, the largest in
blocks of a fixed width."""
import pytest
import torch

import paged_common as pc
from test_gpu_kv_append import check, rows, snapshot

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mtp_speculative_decoding_gb300 import build
    build.build()


def append_and_check(hd, hkv, page, M, lens, n_new, norm, inp, theta=1e6):
    import mtp_speculative_decoding_gb300 as m
    B = len(lens)
    n = n_new or [M] * B
    pool = pc.Pool(B, (max(lens) + M + page - 1) // page + 1, page, hkv, hd, "e4m3", seed=1)
    pool.fill(lens, seed=2)
    k, v = rows(B, M, hkv, hd, inp, seed=3)
    gain = 1 + 0.1 * torch.randn(hd, device="cuda") if norm else None
    before = snapshot(pool)
    scales = {"k": pool.ks.clone(), "v": pool.vs.clone()}
    h = pool.handle(rope_theta=theta)
    ws = m.alloc_workspace(m.kv_workspace_size(h, B, M, hkv))
    m.kv_append(h, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), ws,
                n_new=None if n_new is None else torch.tensor(n, dtype=torch.int32, device="cuda"), k_norm=gain)
    assert m.last_error(ws) == m.MTP_OK
    check(pool, before, k, v, gain, lens, n, theta, scales)


@pytest.mark.parametrize("inp", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("M", [8, 9, 11, 13, 14, 15, 16, 17, 31])
def test_few_rows_of_the_largest_heads(M, page, norm, inp):
    """head_dim 512 has 256 rotation pairs and, from 9 to 14 rows, fewer
    threads than that.  Pages that start with the call, that it continues, and
    that it crosses."""
    append_and_check(512, 2, page, M, [0, 5, page - 3], [M, M, M - 1], norm, inp)


# rows at which a page's units pass 256 and 1024 (units of 16 elements)
@pytest.mark.parametrize("hd,M", [(hd, most * 16 // hd + d) for hd in (32, 64, 128, 256, 512) for most in (256, 1024) for d in (0, 1)
                                  if most * 16 // hd + d <= 257])
def test_either_side_of_a_change_of_launch(hd, M):
    append_and_check(hd, 1, 256, M, [0, 250], None, True, torch.bfloat16)
