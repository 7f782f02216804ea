"""mtp_prefix_attention against a plain 64-bit form: types, head sizes, groups
of sequences, prefixes that end inside pages and tiles, and rows it must leave
alone."""
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


def queries(B, M, hq, hd, dtype, seed, extra=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(B, M, hq + extra, hd, device="cuda", generator=g).to(dtype)[:, :, :hq]


def shared_pool(lens, n, start, pre, page, hkv, hd, kv, seed, layout="head"):
    """A pool whose groups' whole prefix pages appear in the first sequence's
    table row only: the others' entries are pages of no one (-1)."""
    pool = pc.Pool(len(lens), max(a + c for a, c in zip(lens, n)) // page + 2, page, hkv, hd, kv, seed=seed, layout=layout)
    pool.fill([a + c for a, c in zip(lens, n)], seed=seed + 1)
    for i, p in enumerate(pre):
        for b in range(start[i] + 1, start[i + 1]):
            pool.table[b, : p // page] = -1
    return pool


def run(pool, q, lens, start, pre, n_new=None, gain=None, ws=None, scale=None, **kw):
    m = mtp()
    h = pool.handle(**kw)
    B, M, hq, _ = q.shape
    ws = m.alloc_workspace(m.prefix_workspace_size(h, B, M, hq)) if ws is None else ws
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    m.prefix_attention(h, q, i32(lens), i32(start), i32(pre), out, ws, n_new=None if n_new is None else i32(n_new), q_norm=gain,
                       attn_scale=scale)
    return out, m.last_error(ws)


def of_group(b, start, pre):
    for i in range(len(pre)):
        if start[i] <= b < start[i + 1]:
            return pre[i], start[i]
    return 0, b


def check(pool, out, q, gain, lens, n, start, pre, theta, scale=None, random=True, absent=None, skip=()):
    for b, c in enumerate(n):
        P, first = of_group(b, start, pre)
        if c and b not in skip:
            ref = rc.attend(pool, b, q[b, :c], gain, lens[b], theta, scale=scale, prefix=P, first=first, absent=(absent or {}).get(b, ()))
            rc.check(out[b, :c], *ref, lens[b] + c, pool.dtype, random)
        assert (out[b, c:] == 7.0).all(), "a row behind the sequence's last has changed"


CASES = [
    # kv, q, hd, hkv, G, page, M, own lengths behind the prefix, n_new, group_start, prefix_len, norm, theta, layout
    ("bf16", "bf16", 256, 2, 4, 16, 1, [60, 0, 7, 60], None, [0, 4], [1000], True, 1e6, "head"),
    ("bf16", "bf16", 256, 4, 4, 64, 3, [10, 0, 300, 129, 64, 1], [3, 0, 3, 1, 2, 3], [0, 4, 6], [640, 250], True, 1e6, "slot"),
    ("bf16", "bf16", 256, 1, 7, 32, 5, [3] * 20, None, [0, 20], [700], False, 1e4, "head"),          # 700 rows of one KV head
    ("bf16", "bf16", 128, 2, 2, 32, 1, [130, 5, 0, 77, 90], None, [0, 5], [513], False, 1e4, "slot"),
    ("bf16", "bf16", 128, 1, 8, 128, 17, [40, 300], [17, 2], [0, 2], [400], True, 1e6, "head"),
    ("bf16", "bf16", 128, 2, 4, 16, 2, [1] * 9, None, [0, 1, 1, 4, 9], [33, 50, 0, 128], True, 1e4, "head"),   # one, none, no prefix
    ("bf16", "bf16", 64, 2, 4, 16, 3, [9, 100, 0], None, [0, 3], [127], True, 1e4, "slot"),
    ("bf16", "bf16", 64, 1, 16, 32, 64, [5, 200], [64, 33], [0, 2], [129], False, 1e4, "head"),
    ("bf16", "bf16", 128, 1, 4, 32, 2, [50, 60, 70, 80, 90], None, [1, 3], [300], False, 1e4, "head"),   # sequences of no group
    ("bf16", "bf16", 256, 1, 4, 32, 2, [50, 60, 700], None, [0], [], False, 1e4, "head"),                  # no group at all
    ("e4m3", "bf16", 256, 2, 4, 64, 4, [60, 0, 7, 160, 700], [4, 4, 0, 3, 4], [0, 2, 5], [1000, 300], True, 1e6, "head"),
    ("e4m3", "bf16", 256, 1, 8, 16, 1, [20] * 40, None, [0, 40], [500], False, 1e4, "slot"),
    ("e4m3", "bf16", 128, 2, 7, 32, 3, [100, 5, 31], None, [0, 3], [260], True, 1e4, "slot"),
    ("e4m3", "bf16", 64, 1, 4, 128, 2, [100, 0, 31], None, [0, 3], [1], True, 1e4, "head"),
    ("f32", "f32", 128, 2, 4, 16, 3, [10, 0, 33], [3, 3, 1], [0, 3], [50], True, 1e4, "slot"),
    ("bf16", "f32", 256, 1, 3, 32, 2, [15, 3], None, [0, 2], [90], True, 1e6, "slot"),
    ("e4m3", "f32", 64, 1, 2, 32, 2, [15, 3], None, [0, 2], [90], True, 1e6, "slot"),
    ("bf16", "bf16", 512, 1, 2, 64, 2, [15, 3], None, [0, 2], [90], True, 1e6, "head"),
    ("bf16", "bf16", 32, 2, 2, 16, 2, [15, 3], None, [0, 2], [90], True, 1e6, "head"),
]


@pytest.mark.parametrize("kv,qt,hd,hkv,G,page,M,own,n_new,start,pre,norm,theta,layout", CASES)
def test_rows_attend_a_shared_prefix(kv, qt, hd, hkv, G, page, M, own, n_new, start, pre, norm, theta, layout):
    B = len(own)
    n = n_new or [M] * B
    lens = [a + of_group(b, start, pre)[0] for b, a in enumerate(own)]
    pool = shared_pool(lens, n, start, pre, page, hkv, hd, kv, 1, layout)
    q = queries(B, M, hkv * G, hd, torch.bfloat16 if qt == "bf16" else torch.float32, seed=3)
    gain = 1 + 0.1 * torch.randn(hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)) if norm else None
    out, st = run(pool, q, lens, start, pre, n_new, gain, rope_theta=theta)
    assert st == mtp().MTP_OK
    check(pool, out, q, gain, lens, n, start, pre, theta)


@pytest.mark.parametrize("kv,hd,hkv,G,M", [("bf16", 256, 2, 4, 3), ("e4m3", 256, 1, 4, 2), ("bf16", 128, 2, 2, 1), ("bf16", 64, 1, 8, 4)])
def test_a_large_ragged_batch(kv, hd, hkv, G, M):
    """Prefixes and own parts cut between CTAs; twice the same bits, whatever the
    workspace held."""
    m = mtp()
    g = torch.Generator().manual_seed(5)
    B, page = 90, 32
    start, pre = [0, 1, 50, 50, 70, 90], [77, 2000, 5, 0, 999]
    own = torch.randint(0, 400, (B,), generator=g).tolist()
    n = torch.randint(0, M + 1, (B,), generator=g).tolist()
    lens = [a + of_group(b, start, pre)[0] for b, a in enumerate(own)]
    pool = shared_pool(lens, n, start, pre, page, hkv, hd, kv, 6)
    q = queries(B, M, hkv * G, hd, torch.bfloat16, seed=7)
    ws = m.alloc_workspace(m.prefix_workspace_size(pool.handle(), B + 30, M, hkv * G))
    ws.fill_(0xFF)
    out, st = run(pool, q, lens, start, pre, n, ws=ws, rope_theta=1e6)
    assert st == m.MTP_OK
    check(pool, out, q, None, lens, n, start, pre, 1e6)
    ws.fill_(0x5A)
    again, _ = run(pool, q, lens, start, pre, n, ws=ws, rope_theta=1e6)
    assert torch.equal(out, again)


def test_the_largest_batch_and_as_many_groups():
    m = mtp()
    for kv, hd, G, k in (("bf16", 256, 4, 1024), ("e4m3", 128, 2, 3), ("bf16", 64, 1, 511)):
        B, M, page = m.MTP_MAX_PAGED_BATCH, 2, 16
        g = torch.Generator().manual_seed(8)
        start = [0] + sorted((torch.randperm(B - 1, generator=g)[: k - 1] + 1).tolist()) + [B]
        pre = torch.randint(0, 40, (k,), generator=g).tolist()
        own = torch.randint(0, 20, (B,), generator=g).tolist()
        lens = [a + of_group(b, start, pre)[0] for b, a in enumerate(own)]
        pool = shared_pool(lens, [M] * B, start, pre, page, 1, hd, kv, 9)
        q = queries(B, M, G, hd, torch.bfloat16, seed=10)
        out, st = run(pool, q, lens, start, pre, rope_theta=1e4)
        assert st == m.MTP_OK
        check(pool, out, q, None, lens, [M] * B, start, pre, 1e4, skip=set(range(B)) - set(range(0, B, 41)) - {B - 1})


@pytest.mark.parametrize("kv,hd", [("bf16", 128), ("bf16", 256), ("e4m3", 256), ("e4m3", 128)])
def test_far_scores(kv, hd):
    """The largest score in the prefix for some rows, in their own part for others."""
    pool = shared_pool([800] * 6, [2] * 6, [0, 6], [700], 32, 1, hd, kv, 11)
    q = queries(6, 2, 4, hd, torch.bfloat16, seed=13) * 8
    out, st = run(pool, q, [800] * 6, [0, 6], [700], rope_theta=1e4, scale=0.25)
    assert st == mtp().MTP_OK
    check(pool, out, q, None, [800] * 6, [2] * 6, [0, 6], [700], 1e4, scale=0.25, random=False)


@pytest.mark.parametrize("kv,hd", [("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_absent_pages_are_masked_and_reported(kv, hd):
    m = mtp()
    lens, start, pre = [150, 130, 140], [0, 3], [100]
    pool = shared_pool(lens, [2] * 3, start, pre, 16, 1, hd, kv, 14)
    pool.table[0, 2], pool.table[1, 7] = -5, 10 ** 7          # a page of the prefix; one of sequence 1's own
    q = queries(3, 2, 4, hd, torch.bfloat16 if kv != "f32" else torch.float32, seed=15)
    out, st = run(pool, q, lens, start, pre, rope_theta=1e4)
    assert st == m.MTP_ERR_ARG
    gone = {b: list(range(32, 48)) for b in range(3)}
    gone[1] = gone[1] + list(range(112, 128))
    pool.table[0, 2] = pool.table[1, 7] = 0
    check(pool, out, q, None, lens, [2] * 3, start, pre, 1e4, absent=gone)


def test_what_is_out_of_range_is_left_out():
    m = mtp()
    lens, pre = [150, 130, 140, 20], [100]
    for start, bad in (([0, 4], [3]),              # kv_len 20 below the prefix
                       ([0, 3], []), ([2, 3], [])):
        pool = shared_pool(lens, [2] * 4, [0, 0], pre, 16, 1, 128, "bf16", 16)
        q = queries(4, 2, 2, 128, torch.bfloat16, seed=17)
        out, st = run(pool, q, lens, start, pre, rope_theta=1e4)
        assert st == (m.MTP_ERR_ARG if bad else m.MTP_OK)
        check(pool, out, q, None, lens, [0 if b in bad else 2 for b in range(4)], start, pre, 1e4)
    for n_new, more in (([2, -1, 2, 2], 0), ([2, 3, 2, 2], 0), (None, 1000)):
        ll = list(lens)
        ll[1] += more
        out, st = run(pool, q, ll, [0, 3], pre, n_new, rope_theta=1e4)
        assert st == m.MTP_ERR_ARG
        check(pool, out, q, None, lens, [2, 0, 2, 2], [0, 3], pre, 1e4)
    for start, plen in (([0, 9], pre), ([-1, 4], pre), ([3, 0], pre), ([0, 4], [-7])):      # in no order, outside, negative
        out, st = run(pool, q, lens, start, plen, rope_theta=1e4)
        assert st == m.MTP_ERR_ARG


def test_values_that_are_not_finite():
    m = mtp()
    for kv, hd in (("bf16", 128), ("bf16", 256), ("f32", 128)):
        lens, start, pre = [150, 130, 140], [0, 2, 3], [100, 0]
        pool = shared_pool(lens, [2] * 3, start, pre, 16, 1, hd, kv, 18)
        q = queries(3, 2, 4, hd, torch.bfloat16 if kv != "f32" else torch.float32, seed=19)
        want, _ = run(pool, q, lens, start, pre, rope_theta=1e4)
        pool.v[int(pool.table[0, 3]), 0, 5, 9] = float("inf")       # position 53: in the prefix of 0 and 1
        pool.v[int(pool.table[1, 8]), 0, 3, 20] = float("nan")      # position 131: row 1 of sequence 1
        out, st = run(pool, q, lens, start, pre, rope_theta=1e4)
        assert st == m.MTP_OK
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[:2, :, :, 9] = True
        assert (out[hit] == float("inf")).all()
        hit[1, 1, :, 20] = True
        assert out[1, 1, :, 20].isnan().all()
        assert ((out.float() - want.float()).abs()[~hit] <= 2.0 ** -5 * (1 + want.float().abs()[~hit])).all()


def test_same_rows_as_the_verify_steps_attention():
    """With the prefix's pages in every table row, mtp_paged_attention gives the
    same answers within both roundings."""
    m = mtp()
    for kv, hd in (("bf16", 256), ("e4m3", 128)):
        B, M, hq, page, P = 7, 3, 8, 32, 320
        lens = [P + x for x in (0, 5, 32, 100, 64, 1, 200)]
        pool = shared_pool(lens, [M] * B, [0, B], [P], page, 2, hd, kv, 20)
        q = queries(B, M, hq, hd, torch.bfloat16, seed=21)
        out, st = run(pool, q, lens, [0, B], [P], rope_theta=1e6)
        assert st == m.MTP_OK
        pool.table[1:, : P // page] = pool.table[0, : P // page]
        h = pool.handle(rope_theta=1e6)
        ws = m.alloc_workspace(m.kv_workspace_size(h, B, M, hq))
        other = torch.empty_like(out)
        m.paged_attention(h, q, i32(lens), other, ws)
        d = out.double() - other.double()
        assert d.square().mean().sqrt() <= 2.0 ** -7 * other.double().square().mean().sqrt()


def test_captured_and_on_another_stream():
    m = mtp()
    B, M, hq, hd, P = 5, 2, 8, 256, 300
    lens = [P + x for x in (0, 5, 32, 100, 64)]
    pool = shared_pool(lens, [M] * B, [0, B], [P], 32, 2, hd, "bf16", 22)
    q = queries(B, M, hq, hd, torch.bfloat16, seed=23)
    want, _ = run(pool, q, lens, [0, B], [P], rope_theta=1e4)
    h = pool.handle(rope_theta=1e4)
    ws = m.alloc_workspace(m.prefix_workspace_size(h, B, M, hq))
    out = torch.zeros_like(want)
    ln, st, pl = i32(lens), i32([0, B]), i32([P])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    m.prefix_attention(h, q, ln, st, pl, out, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.prefix_attention(h, q, ln, st, pl, out, ws)
    ln.sub_(i32([0, 3, 1, 50, 64]))
    g.replay()
    torch.cuda.synchronize()
    other, _ = run(pool, q, ln.tolist(), [0, B], [P], rope_theta=1e4)
    assert torch.equal(out, other)
