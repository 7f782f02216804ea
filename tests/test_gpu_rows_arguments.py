"""Calls of the attention of prompts and of shared prefixes that the header
allows and few programs make: outputs and queries at any 16-byte address,
windows without an end, bounds that do not ascend, dirty workspaces."""
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


def rand(shape, dtype, seed):
    return torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(dtype)


def at_address(x, byte):
    """A copy of x whose address is `byte` behind a 256-byte boundary."""
    n = byte // x.element_size()
    y = torch.empty(x.numel() + 256, dtype=x.dtype, device="cuda")
    assert y.data_ptr() % 256 == 0 and byte % x.element_size() == 0
    y = y[n:n + x.numel()].view(x.shape)
    y.copy_(x)
    assert y.data_ptr() % 256 == byte
    return y


def prompt(pool, q, row_start, lens, out=None, ws=None, **kw):
    m = mtp()
    h = pool.handle(**kw)
    T, hq, _ = q.shape
    ws = m.alloc_workspace(m.prompt_workspace_size(h, len(lens), T, hq)) if ws is None else ws
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    m.prompt_attention(h, q, i32(row_start), i32(lens), out, ws)
    return out, m.last_error(ws)


@pytest.mark.parametrize("byte", [16, 32, 48, 240])
@pytest.mark.parametrize("kv,qt,hd", [("bf16", "bf16", 64), ("bf16", "bf16", 128), ("bf16", "bf16", 256), ("e4m3", "bf16", 64), ("e4m3", "bf16", 128),
                                      ("e4m3", "bf16", 256), ("f32", "f32", 64), ("bf16", "bf16", 512)])
def test_outputs_and_queries_at_any_16_byte_address(kv, qt, hd, byte):
    m = mtp()
    dt = torch.bfloat16 if qt == "bf16" else torch.float32
    n, lens, hq = [150, 3], [40, 300], 2
    pool = pc.Pool(2, 24, 16, 1, hd, kv, seed=1)
    pool.fill([a + c for a, c in zip(lens, n)], seed=2)
    q = rand((sum(n), hq, hd), dt, 3)
    want, st = prompt(pool, q, [0, 150, 153], lens, rope_theta=1e4)
    assert st == m.MTP_OK
    out, st = prompt(pool, at_address(q, byte), [0, 150, 153], lens, out=at_address(torch.full_like(q, 7.0), byte), rope_theta=1e4)
    assert st == m.MTP_OK and torch.equal(out, want)
    # shared prefixes
    h = pool.handle(rope_theta=1e4)
    B, M = 2, 3
    qq = q[:B * M].reshape(B, M, hq, hd).contiguous()
    ws = m.alloc_workspace(m.prefix_workspace_size(h, B, M, hq))
    outs = []
    for b in (0, byte):
        o = at_address(torch.full_like(qq, 7.0), b)
        m.prefix_attention(h, at_address(qq, b), i32([40, 300]), i32([0, 2]), i32([37]), o, ws)
        assert m.last_error(ws) == m.MTP_OK
        outs.append(o)
    assert torch.equal(*outs)


@pytest.mark.parametrize("kv,qt,hd", [("bf16", "bf16", 64), ("bf16", "bf16", 128), ("bf16", "bf16", 256), ("e4m3", "bf16", 128),
                                      ("e4m3", "bf16", 256), ("f32", "f32", 64)])
@pytest.mark.parametrize("G", [1, 4, 16])
def test_windows_as_long_as_an_int_goes(kv, qt, hd, G):
    """A window that reaches over everything is no window, up to 2^31 - 1, with any sink."""
    m = mtp()
    n, lens = [400, 70, 1], [0, 333, 600]
    pool = pc.Pool(3, 13, 64, 1, hd, kv, seed=4)
    pool.fill([a + c for a, c in zip(lens, n)], seed=5)
    q = rand((471, G, hd), torch.bfloat16 if qt == "bf16" else torch.float32, 6)
    at = [0, 400, 470, 471]
    want, st = prompt(pool, q, at, lens, rope_theta=1e4)
    assert st == m.MTP_OK
    for b, a in enumerate(lens):
        r = slice(at[b], at[b + 1])
        rc.check(want[r], *rc.attend(pool, b, q[r], None, a, 1e4), a + n[b], kv)
    top = 2 ** 31 - 1
    for window, sink in ((top, 0), (top, top), (top - 15, 4), (top - 255, 0), (top - 256, 1000), (2 ** 30, top), (671, 0), (601, 9)):
        out, st = prompt(pool, q, at, lens, rope_theta=1e4, window=window, sink=sink)
        assert st == m.MTP_OK and torch.equal(out, want), (window, sink)


def left_in(at, T):
    """Sequences whose rows are theirs alone and within [0, T]."""
    return [b for b in range(len(at) - 1) if 0 <= at[b] <= at[b + 1] <= T and max(at[: b + 1]) <= at[b] and min(at[b + 1:]) >= at[b + 1]]


@pytest.mark.parametrize("kv,qt,hd", [("bf16", "bf16", 64), ("bf16", "bf16", 128), ("bf16", "bf16", 256), ("e4m3", "bf16", 128),
                                      ("e4m3", "bf16", 256), ("f32", "f32", 64), ("bf16", "bf16", 512)])
def test_bounds_that_do_not_ascend(kv, qt, hd):
    """What two sequences would claim is left out with both of them, for every KV
    head, and the others are right."""
    m = mtp()
    B, T, hkv, G = 5, 150, 2, 2
    pool = pc.Pool(B, 16, 16, hkv, hd, kv, seed=7)
    pool.fill([210] * B, seed=8)
    lens = [60] * B
    q = rand((T, hkv * G, hd), torch.bfloat16 if qt == "bf16" else torch.float32, 9)
    h = pool.handle(rope_theta=1e4)
    ws = m.alloc_workspace(m.prompt_workspace_size(h, B, T, hkv * G))
    ref = {}
    g = torch.Generator().manual_seed(10)
    bounds = [[0, 40, 30, 70, 110, 150], [10, 5, 5, 60, 60, 100], [150, 110, 70, 30, 20, 0], [0, 150, 20, 30, 60, 150], [0, 30, 60, 90, 120, 119],
              [-5, 20, 10, 60, 90, 151], [0, 2 ** 31 - 1, -2 ** 31, 20, 20, 150]]
    bounds += [(torch.randint(0, 6, (B + 1,), generator=g).sort().values + torch.randint(0, 2, (B + 1,), generator=g)).mul(25).tolist()
               for _ in range(8)]
    for at in bounds:
        ws.fill_(0xFF)
        out, st = prompt(pool, q, at, lens, ws=ws, rope_theta=1e4)
        good = left_in(at, T)
        assert st == (m.MTP_OK if len(good) == B else m.MTP_ERR_ARG), at
        used = torch.zeros(T, dtype=torch.bool)
        for b in good:
            r0, r1 = at[b], at[b + 1]
            used[r0:r1] = True
            if r1 > r0:
                if (b, r0, r1) not in ref:
                    ref[b, r0, r1] = rc.attend(pool, b, q[r0:r1], None, 60, 1e4)
                rc.check(out[r0:r1], *ref[b, r0, r1], 60 + r1 - r0, kv)
        assert (out[~used] == 7.0).all(), at


@pytest.mark.parametrize("kv,qt,hd", [("bf16", "bf16", 64), ("bf16", "bf16", 256), ("e4m3", "bf16", 128), ("f32", "f32", 64), ("bf16", "bf16", 512),
                                      ("e4m3", "bf16", 32)])
def test_groups_that_do_not_ascend(kv, qt, hd):
    """All sequences are left out, with every type."""
    m = mtp()
    B, M, hq = 6, 2, 4
    pool = pc.Pool(B, 8, 16, 2, hd, kv, seed=11)
    pool.fill([100] * B, seed=12)
    q = rand((B, M, hq, hd), torch.bfloat16 if qt == "bf16" else torch.float32, 13)
    h = pool.handle(rope_theta=1e4)
    ws = m.alloc_workspace(m.prefix_workspace_size(h, B, M, hq))
    for start, pre in (([0, 3, 2, 6], [20, 20, 20]), ([6, 0], [20]), ([0, 6, 0, 6], [20, 40, 30]), ([0, 2, 4, 3], [20, 20, 20]), ([3, 2], [0])):
        ws.fill_(0xFF)
        out = torch.full_like(q, 7.0)
        m.prefix_attention(h, q, i32([80] * B), i32(start), i32(pre), out, ws)
        assert m.last_error(ws) == m.MTP_ERR_ARG and (out == 7.0).all(), start
    for start, pre, n in (([2, 2, 5], [30, 20], 6), ([-1, 2, 6], [20, 20], 4)):     # bounds that ascend: [-1, 2) alone is out
        out = torch.full_like(q, 7.0)
        m.prefix_attention(h, q, i32([80] * B), i32(start), i32(pre), out, ws)
        assert m.last_error(ws) == (m.MTP_OK if n == 6 else m.MTP_ERR_ARG)
        assert (out[: B - n] == 7.0).all() and not (out[B - n:] == 7.0).any(), start


@pytest.mark.parametrize("kv,qt,hd", [("bf16", "bf16", 64), ("bf16", "bf16", 256), ("e4m3", "bf16", 128), ("f32", "f32", 64), ("bf16", "bf16", 512)])
def test_groups_without_a_sequence(kv, qt, hd):
    """Whatever their prefix is, they concern no one: the same status with every type."""
    m = mtp()
    B, M, hq = 3, 2, 4
    pool = pc.Pool(B, 4, 16, 2, hd, kv, seed=14)
    pool.fill([42] * B, seed=15)
    q = rand((B, M, hq, hd), torch.bfloat16 if qt == "bf16" else torch.float32, 16)
    h = pool.handle(rope_theta=1e4)
    ws = m.alloc_workspace(m.prefix_workspace_size(h, B, M, hq))
    for start, pre, shared in (([0, 0], [1000], 0), ([0, 0, 3], [-4, 20], 1), ([0, 3, 3], [20, 2 ** 31 - 1], 1), ([3, 3, 3], [65, -1], 0),
                               ([-5, -2], [20], 0), ([4, 9], [20], 0)):
        out = torch.full_like(q, 7.0)
        m.prefix_attention(h, q, i32([40] * B), i32(start), i32(pre), out, ws)
        assert m.last_error(ws) == m.MTP_OK, start
        for b in range(B):
            rc.check(out[b], *rc.attend(pool, b, q[b], None, 40, 1e4, prefix=20 if shared else 0, first=0), 42, kv)
