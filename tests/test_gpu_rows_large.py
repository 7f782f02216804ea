"""The largest calls: as many packed rows as a call takes, and rows, outputs,
caches and parts that lie more than 2^31 elements behind their beginnings."""
import pytest
import torch

import paged_common as pc
import rows_common as rc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mtp_speculative_decoding_gb300 import build
    build.build()


def mtp():
    import mtp_speculative_decoding_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def normal(shape, seed):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(seed))


class Cache(pc.Pool):
    """Sequence b's page j is page b * max_pages + j of a pool in which every slot is written."""

    def __init__(self, B, max_pages, page, hkv, hd, seed):
        self.dtype, self.page, self.hkv, self.hd, self.B, self.max_pages = "bf16", page, hkv, hd, B, max_pages
        self.k, self.v = normal((B * max_pages, hkv, page, hd), seed), normal((B * max_pages, hkv, page, hd), seed + 1)
        self.ks = self.vs = None
        self.table = torch.arange(B * max_pages, dtype=torch.int32, device="cuda").view(B, max_pages)


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def test_prompts_of_as_many_rows_as_a_call_takes():
    """1024 prompts of 1024 rows, 16 heads of 256 over as many: 2^32 elements of
    queries, outputs, keys and values each."""
    m = mtp()
    B, n, page, hq, hd = m.MTP_MAX_PAGED_BATCH, 1024, 256, 16, 256
    T = B * n
    assert T == m.MTP_MAX_PROMPT_ROWS
    pool = Cache(B, n // page, page, hq, hd, 1)
    q = normal((T, hq, hd), 3)
    out = torch.full_like(q, 7.0)
    h = pool.handle(rope_theta=1e6)
    ws = m.alloc_workspace(m.prompt_workspace_size(h, B, T, hq))
    m.prompt_attention(h, q, i32([n * b for b in range(B + 1)]), i32([0] * B), out, ws)
    assert m.last_error(ws) == m.MTP_OK
    for b in (0, 1, 511, 512, 1023):
        for rows in (slice(0, 40), slice(n - 40, n)):
            p0 = rows.start
            r = slice(b * n + p0, b * n + rows.stop)
            rc.check(out[r], *rc.attend(pool, b, q[r], None, p0, 1e6), rows.stop, "bf16")


def test_cuda_cores_behind_2_31_elements():
    """Head dimension 512: short prompts among the last rows of a large buffer."""
    m = mtp()
    B, T, page, hq, hd = 9, 9 * 2 ** 16, 256, 8, 512
    pool = Cache(B, 1, page, 1, hd, 4)
    q = normal((T, hq, hd), 5)
    out = torch.full_like(q, 7.0)
    h = pool.handle(rope_theta=1e4)
    ws = m.alloc_workspace(m.prompt_workspace_size(h, B, T, hq))
    at = [T - 300] + [T - 250 + 20 * b for b in range(B)]
    assert at[0] * hq * hd > 2 ** 31
    m.prompt_attention(h, q, i32(at), i32([0] * B), out, ws)
    assert m.last_error(ws) == m.MTP_OK
    for b in range(B):
        r = slice(at[b], at[b + 1])
        rc.check(out[r], *rc.attend(pool, b, q[r], None, 0, 1e4), page, "bf16")
    assert (out[: at[0]] == 7.0).all() and (out[at[-1]:] == 7.0).all()


def test_shared_prefixes_behind_2_31_elements():
    """1024 sequences of 64 rows, 144 heads of 256: queries, outputs and parts pass 2^31."""
    m = mtp()
    B, M, page, hkv, G, hd, P = m.MTP_MAX_PAGED_BATCH, m.MTP_MAX_ATTN_ROWS, 64, 9, 16, 256, 200
    pool = Cache(B, 5, page, hkv, hd, 6)
    q = normal((B, M, hkv * G, hd), 8)
    assert q.numel() > 2 ** 31
    out = torch.full_like(q, 7.0)
    h = pool.handle(rope_theta=1e6)
    ws = m.alloc_workspace(m.prefix_workspace_size(h, B, M, hkv * G))
    lens = [P + b % 50 for b in range(B)]
    m.prefix_attention(h, q, i32(lens), i32([0, 500, B]), i32([P, P]), out, ws)
    assert m.last_error(ws) == m.MTP_OK
    for b in (0, 499, 500, 901, B - 1):
        ref = rc.attend(pool, b, q[b], None, lens[b], 1e6, prefix=P, first=0 if b < 500 else 500)
        rc.check(out[b], *ref, lens[b] + M, "bf16")


def test_rotation_behind_2_31_elements():
    m = mtp()
    T, hq, hd = m.MTP_MAX_PROMPT_ROWS, 9, 256
    q, k = normal((T, hq, hd), 9), normal((T, 1, hd), 10)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, T), generator=torch.Generator().manual_seed(11)).to(torch.int32).cuda()
    rows = torch.cat([torch.arange(0, 50), torch.arange(T - 50, T), torch.arange(T // 2, T // 2 + 50)]).cuda()
    want = [rc.rotate(x[rows], None, pos[:, rows], (44, 42, 42), 1e6, True) for x in (q, k)]
    assert q.numel() > 2 ** 31
    m.rotate_axes(q, k, pos, (44, 42, 42), 1e6, q, k, interleaved=True)       # in place
    for x, (ref, tol) in zip((q, k), want):
        got = x[rows].double()
        # beside the fp32 bound: a frequency keeps 48 bits and its product with a position the
        # last bits of two fp32 sums, 2^-18 turns at 2^31 positions, 2^-15 of a pair's magnitude;
        # the sine and cosine instructions 2^-20; the result rounds to bf16
        off = 2 * tol + 2.0 ** -15 * (tol * 2.0 ** 19)
        assert ((got - ref).abs() <= off + 2.0 ** -8 * (ref.abs() + off)).all()
