"""mtp_paged_attention against a plain 64-bit form: types, head sizes, groups,
pages, lengths, windows, absent pages, values that are not finite, and rows
it must leave alone."""
import pytest
import torch

import paged_common as pc

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
    """Rows as a slice of a fused projection's output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, M, (hq + extra) * hd, device="cuda", generator=g).to(dtype)
    return x[..., : hq * hd].unflatten(-1, (hq, hd))


def run(pool, q, lens, n_new=None, gain=None, ws=None, scale=None, **kw):
    m = mtp()
    h = pool.handle(**kw)
    B, M, hq, _ = q.shape
    ws = m.alloc_workspace(m.kv_workspace_size(h, B, M, hq)) if ws is None else ws
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    m.paged_attention(h, q, i32(lens), out, ws, n_new=None if n_new is None else i32(n_new), q_norm=gain, attn_scale=scale)
    return out, m.last_error(ws)


def check(pool, out, q, gain, lens, n_new, theta, window=0, sink=0, scale=None, absent=None):
    low = q.dtype == torch.bfloat16
    ref, mass, dots = pc.attention(pool, q, gain, lens, n_new, theta, window, sink, scale, absent)
    tol = pc.attention_tol(ref, mass, dots, q.shape[-1], max(a + n for a, n in zip(lens, n_new)), low)
    for b, n in enumerate(n_new):
        err = (out[b, :n].double() - ref[b, :n]).abs()
        assert (err <= tol[b, :n]).all(), (b, float((err / tol[b, :n].clamp(min=1e-30)).max()))
        assert (out[b, n:] == 7.0).all(), "a row behind the sequence's last has changed"


CASES = [
    # kv, q, hd, hkv, G, page, M, lens, n_new, norm, theta, window, sink, layout
    ("bf16", "bf16", 256, 2, 4, 16, 1, [999], None, True, 1e6, 0, 0, "head"),
    ("bf16", "bf16", 256, 4, 4, 64, 4, [0, 1, 127, 128, 700], None, True, 1e6, 0, 0, "slot"),
    ("bf16", "bf16", 128, 1, 1, 32, 1, [0], None, False, 0.0, 0, 0, "head"),
    ("bf16", "bf16", 128, 2, 7, 128, 5, [63, 300], [5, 2], True, 1e4, 0, 0, "slot"),
    ("bf16", "bf16", 64, 2, 8, 16, 3, [250, 17, 0], [3, 0, 1], True, 1e4, 0, 0, "head"),
    ("bf16", "bf16", 512, 1, 4, 64, 3, [200, 5], None, True, 1e6, 0, 0, "slot"),
    ("bf16", "bf16", 128, 1, 16, 256, 17, [400], None, False, 1e4, 0, 0, "head"),      # 272 rows of one KV head
    ("bf16", "bf16", 256, 1, 8, 32, 64, [130, 0], [64, 33], True, 1e6, 0, 0, "slot"),
    ("bf16", "bf16", 32, 2, 2, 16, 3, [40, 3], None, True, 1e4, 0, 0, "head"),
    ("bf16", "bf16", 128, 2, 4, 32, 4, [600, 90, 5], None, False, 1e4, 100, 4, "slot"),
    ("bf16", "bf16", 256, 1, 4, 64, 3, [1500, 1023, 1025], None, False, 1e4, 1024, 130, "head"),
    ("bf16", "bf16", 64, 1, 4, 16, 9, [500], None, True, 1e4, 1, 0, "head"),            # a window of one
    ("e4m3", "bf16", 256, 4, 4, 64, 3, [700, 64, 0, 1], [3, 3, 3, 2], True, 1e6, 0, 0, "head"),
    ("e4m3", "bf16", 128, 2, 8, 16, 1, [333, 15], None, True, 1e4, 0, 0, "slot"),
    ("e4m3", "bf16", 64, 2, 4, 32, 5, [200, 31], None, False, 1e4, 0, 0, "head"),
    ("e4m3", "bf16", 512, 1, 2, 128, 2, [300], None, True, 1e6, 0, 0, "slot"),
    ("e4m3", "bf16", 256, 1, 16, 32, 17, [260, 100], [17, 4], True, 1e6, 0, 0, "head"),
    ("e4m3", "bf16", 128, 2, 4, 256, 4, [900, 300], None, False, 1e4, 200, 20, "slot"),
    ("e4m3", "bf16", 32, 1, 2, 16, 2, [30], None, True, 0.0, 0, 0, "head"),
    ("f32", "f32", 128, 2, 4, 16, 3, [100, 0, 33], [3, 3, 1], True, 1e4, 0, 0, "slot"),
    ("f32", "f32", 256, 1, 2, 64, 20, [70], None, True, 1e6, 0, 0, "head"),
    ("f32", "bf16", 64, 1, 4, 32, 2, [65], None, False, 1e4, 0, 0, "head"),
    ("bf16", "f32", 512, 1, 3, 32, 2, [150], None, True, 1e6, 50, 7, "slot"),
    ("e4m3", "f32", 256, 2, 4, 64, 4, [180, 63], None, True, 1e6, 0, 0, "head"),
    # more rows than a 16-row tile at the largest head dimension, and of all tile heights
    ("bf16", "bf16", 512, 1, 8, 32, 4, [300, 3], [4, 1], True, 1e6, 0, 0, "head"),
    ("e4m3", "bf16", 512, 2, 16, 64, 3, [260], None, False, 1e6, 0, 0, "slot"),
    ("e4m3", "bf16", 64, 1, 16, 16, 64, [200, 0], [64, 7], True, 1e4, 0, 0, "head"),
    ("e4m3", "bf16", 128, 1, 8, 64, 33, [150], None, True, 1e4, 70, 9, "slot"),
    ("bf16", "bf16", 64, 2, 4, 32, 8, [513, 40], None, True, 1e4, 0, 0, "slot"),
    # sequences that bring nothing between ones that do, each cut into parts
    ("bf16", "bf16", 128, 1, 4, 64, 2, [1500, 900, 0, 2000], [2, 0, 0, 1], False, 1e4, 0, 0, "head"),
    ("f32", "f32", 64, 1, 2, 16, 2, [400, 300, 200], [0, 2, 0], False, 1e4, 0, 0, "head"),
]


@pytest.mark.parametrize("kv,qt,hd,hkv,G,page,M,lens,n_new,norm,theta,window,sink,layout", CASES)
def test_rows_attend_the_cache(kv, qt, hd, hkv, G, page, M, lens, n_new, norm, theta, window, sink, layout):
    B = len(lens)
    n = n_new or [M] * B
    pool = pc.Pool(B, (max(lens) + M + page - 1) // page + 1, page, hkv, hd, kv, seed=1, layout=layout)
    pool.fill([a + c for a, c in zip(lens, n)], seed=2)
    q = queries(B, M, hkv * G, hd, torch.bfloat16 if qt == "bf16" else torch.float32, seed=3)
    gain = 1 + 0.1 * torch.randn(hd, device="cuda") if norm else None
    out, st = run(pool, q, lens, n_new, gain, rope_theta=theta, window=window, sink=sink)
    assert st == mtp().MTP_OK
    check(pool, out, q, gain, lens, n, theta, window, sink)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_many_sequences_of_ragged_lengths(kv):
    """More items than CTAs and items cut between CTAs, in one call; and the
    same call twice gives the same bits."""
    g = torch.Generator().manual_seed(4)
    B, M, hkv, G, hd, page = 90, 3, 2, 4, 128, 32
    lens = torch.randint(0, 900, (B,), generator=g).tolist()
    lens[7], lens[8] = 4000, 0
    n = torch.randint(0, M + 1, (B,), generator=g).tolist()
    pool = pc.Pool(B, (max(lens) + M) // page + 2, page, hkv, hd, kv, seed=5)
    pool.fill([a + c for a, c in zip(lens, n)], seed=6)
    q = queries(B, M, hkv * G, hd, torch.bfloat16, seed=7)
    out, st = run(pool, q, lens, n, rope_theta=1e6)
    assert st == mtp().MTP_OK
    check(pool, out, q, None, lens, n, 1e6)
    again, _ = run(pool, q, lens, n, rope_theta=1e6)
    assert torch.equal(out, again)


@pytest.mark.parametrize("kv,hd,hkv,G,M", [("bf16", 64, 2, 2, 2), ("e4m3", 128, 4, 2, 1), ("bf16", 64, 1, 16, 9)])
def test_many_short_sequences_beside_long_ones(kv, hd, hkv, G, M):
    """Shares that count what beginning an item costs: CTAs with many items of
    one tile, with a part of a long one, and with none."""
    g = torch.Generator().manual_seed(41)
    B, page = 500, 16
    lens = torch.randint(0, 120, (B,), generator=g).tolist()
    for b, x in ((0, 3000), (3, 5001), (250, 6000), (251, 0), (499, 4345)):
        lens[b] = x
    n = torch.randint(0, M + 1, (B,), generator=g).tolist()
    n[0] = n[250] = n[499] = M
    pool = pc.Pool(B, (max(lens) + M) // page + 2, page, hkv, hd, kv, seed=42)
    pool.fill([a + c for a, c in zip(lens, n)], seed=43)
    q = queries(B, M, hkv * G, hd, torch.bfloat16, seed=44)
    out, st = run(pool, q, lens, n, rope_theta=1e6)
    assert st == mtp().MTP_OK
    check(pool, out, q, None, lens, n, 1e6)


@pytest.mark.parametrize("kv,hd,G,M", [("bf16", 512, 8, 3), ("e4m3", 256, 4, 3), ("bf16", 64, 2, 1)])
def test_the_largest_batch(kv, hd, G, M):
    """MTP_MAX_PAGED_BATCH sequences, one call of append and one of attention."""
    m = mtp()
    B, page = m.MTP_MAX_PAGED_BATCH, 16
    g = torch.Generator().manual_seed(31)
    lens = torch.randint(0, 40, (B,), generator=g).tolist()
    n = torch.randint(0, M + 1, (B,), generator=g).tolist()
    pool = pc.Pool(B, 4, page, 1, hd, kv, seed=32)
    pool.fill(lens, seed=33)
    q = queries(B, M, G, hd, torch.bfloat16, seed=34, extra=2)
    qkv = torch.randn(B, M, 2 * hd, device="cuda").to(torch.bfloat16)
    h = pool.handle(rope_theta=1e4)
    ws = m.alloc_workspace(m.kv_workspace_size(h, B, M, G))
    m.kv_append(h, qkv[..., :hd].unflatten(-1, (1, hd)), qkv[..., hd:].unflatten(-1, (1, hd)), i32(lens), ws, n_new=i32(n))
    assert m.last_error(ws) == m.MTP_OK
    out, st = run(pool, q, lens, n, ws=ws, rope_theta=1e4)
    assert st == m.MTP_OK
    pick = list(range(0, B, 37)) + [B - 1]
    sub = pc.Pool.__new__(pc.Pool)
    sub.__dict__.update(pool.__dict__)
    sub.table = pool.table[pick]
    check(sub, out[pick], q[pick], None, [lens[b] for b in pick], [n[b] for b in pick], 1e4)
    # a workspace sized for the largest batch serves a small one
    out2, st = run(sub, q[pick], [lens[b] for b in pick], [n[b] for b in pick], ws=ws, rope_theta=1e4)
    assert st == m.MTP_OK
    check(sub, out2, q[pick], None, [lens[b] for b in pick], [n[b] for b in pick], 1e4)


def test_one_long_sequence():
    for kv, hd in (("bf16", 128), ("e4m3", 256)):
        lens, M = [20011], 2
        pool = pc.Pool(1, lens[0] // 128 + 2, 128, 1, hd, kv, seed=8)
        pool.fill([lens[0] + M], seed=9)
        q = queries(1, M, 4, hd, torch.bfloat16, seed=10)
        out, st = run(pool, q, lens, rope_theta=1e6)
        assert st == mtp().MTP_OK
        check(pool, out, q, None, lens, [M], 1e6)


def test_far_scores_and_spread_scales():
    """Scores a hundred apart with their maximum anywhere, and value scales
    2^30 apart between pages: the running maximum and the sums hold."""
    for kv in ("bf16", "e4m3"):
        lens, M, hd = [1200], 2, 128
        pool = pc.Pool(1, 42, 32, 1, hd, kv, seed=11)
        pool.fill([1202], seed=12)
        if kv == "e4m3":
            pool.vs[pool.table[0].long()[::3]] *= 2.0 ** -30
            pool.ks[pool.table[0].long()[5:9]] *= 4
        q = queries(1, M, 4, hd, torch.bfloat16, seed=13) * 8
        out, st = run(pool, q, lens, rope_theta=1e4, scale=0.25)
        assert st == mtp().MTP_OK
        check(pool, out, q, None, lens, [M], 1e4, scale=0.25)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_many_small_weights_beside_a_spike(kv):
    """One position's score is 11 above 6000 equal ones: together they outweigh
    it, so none of their small weights may be lost."""
    lens, hd = [6000], 128
    pool = pc.Pool(1, 190, 32, 1, hd, kv, seed=14)
    pool.fill([6001], seed=15)
    q = torch.zeros(1, 1, 1, hd, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    for w, val in (("k", 0.0), ("v", 1.0)):
        t = getattr(pool, w)
        pages = pool.table[0].long()
        if kv == "e4m3":
            getattr(pool, w + "s")[pages] = 2.0 ** -6
            t.view(torch.uint8)[pages] = torch.tensor(val * 64).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        else:
            t[pages] = val
    spike = 3000
    pg, sl = int(pool.table[0, spike // 32]), spike % 32
    one = torch.tensor(5.5 * (64 if kv == "e4m3" else 1)).to(pool.k.dtype)
    if kv == "e4m3":
        pool.k.view(torch.uint8)[pg, 0, sl, 0] = one.view(torch.uint8).cuda()
        pool.v.view(torch.uint8)[pg, 0, sl] = 0
    else:
        pool.k[pg, 0, sl, 0] = one.cuda()
        pool.v[pg, 0, sl] = 0
    out, st = run(pool, q, lens, scale=2.0)
    assert st == mtp().MTP_OK
    check(pool, out, q, None, lens, [1], 0.0, scale=2.0)


@pytest.mark.parametrize("kv,qt", [("bf16", "bf16"), ("e4m3", "bf16"), ("bf16", "f32")])
def test_absent_pages_are_masked_and_reported(kv, qt):
    m = mtp()
    lens, M, page, hd = [200, 40, 20], 2, 16, 128
    pool = pc.Pool(3, 14, page, 2, hd, kv, seed=16)
    pool.fill([202, 42, 22], seed=17)
    good = pool.table.clone()
    pool.table[0, 3] = -1
    pool.table[0, 12] = 1 << 30
    pool.table[2, :2] = -5                                   # all that sequence 2 has
    absent = {(0, t) for t in range(48, 64)} | {(0, t) for t in range(192, 208)} | {(2, t) for t in range(0, 32)}
    q = queries(3, M, 8, hd, torch.bfloat16 if qt == "bf16" else torch.float32, seed=18)
    out, st = run(pool, q, lens, rope_theta=1e4)
    assert st == m.MTP_ERR_ARG
    bad = pool.table
    pool.table = good
    check(pool, out, q, None, lens, [M] * 3, 1e4, absent=absent)
    assert not out[2].any()                                  # attends nothing: zeros
    # outside the window an absent page is no error
    pool.table = bad
    pool.table[0, 12], pool.table[2] = good[0, 12], good[2]
    out, st = run(pool, q, lens, rope_theta=1e4, window=32)
    assert st == m.MTP_OK
    pool.table = good
    check(pool, out, q, None, lens, [M] * 3, 1e4, window=32)


def test_bad_lengths_are_left_out_and_reported():
    m = mtp()
    pool = pc.Pool(4, 4, 16, 1, 128, "bf16", seed=19)
    pool.fill([22, 0, 0, 12], seed=20)
    q = queries(4, 2, 4, 128, torch.bfloat16, seed=21)
    lens, n = [20, -3, 63, 10], [2, 2, 2, 3]
    out, st = run(pool, q, lens, n)
    assert st == m.MTP_ERR_ARG
    check(pool, out, q, None, [20, 0, 0, 0], [2, 0, 0, 0], 0.0)
    out, st = run(pool, q, [20, 0, 0, 10], [2, 0, 0, 2])
    assert st == m.MTP_OK
    check(pool, out, q, None, [20, 0, 0, 10], [2, 0, 0, 2], 0.0)


@pytest.mark.parametrize("kv,qt,hd", [("bf16", "bf16", 128), ("bf16", "bf16", 256), ("bf16", "f32", 128), ("bf16", "bf16", 64)])
def test_values_that_are_not_finite_stay_with_the_rows_that_attend_them(kv, qt, hd):
    """A new row's value holds an infinity and a NaN: the rows before it do not
    attend it and stay finite, the others get them where the definition does."""
    lens, M, page = [123], 6, 16
    pool = pc.Pool(1, 10, page, 1, hd, kv, seed=22)
    pool.fill([129], seed=23)
    for t, d, x in ((126, 3, float("inf")), (127, 40, float("nan")), (127, 3, float("inf")), (128, 5, -float("inf"))):
        pool.v[int(pool.table[0, t // page]), 0, t % page, d] = x
    pool.k[int(pool.table[0, 128 // page]), 0, 128 % page, 0] = float("nan")       # only the last row attends it
    q = queries(1, M, 4, hd, torch.bfloat16 if qt == "bf16" else torch.float32, seed=24)
    out, st = run(pool, q, lens, rope_theta=1e4)
    assert st == mtp().MTP_OK
    ref, mass, dots = pc.attention(pool, q, None, lens, [M], 1e4)
    tol = pc.attention_tol(ref, mass, dots, hd, 129, qt == "bf16")
    assert torch.isnan(out[0, 5]).all()
    o, r = out[0, :5].double(), ref[0, :5]
    assert torch.equal(torch.isfinite(o), torch.isfinite(r))
    assert torch.equal(torch.isnan(o), torch.isnan(r)) and torch.equal(o[torch.isinf(r)], r[torch.isinf(r)])
    f = torch.isfinite(r)
    assert ((o - r).abs()[f] <= tol[0, :5][f]).all()
    # behind a window's start too
    w = 50
    pool.v[int(pool.table[0, 75 // page]), 0, 75 % page, 9] = float("inf")
    pool.v[int(pool.table[0, 72 // page]), 0, 72 % page, 9] = float("nan")        # before every row's window
    out, _ = run(pool, q, lens, rope_theta=1e4, window=w)
    ref, _, _ = pc.attention(pool, q, None, lens, [M], 1e4, window=w)
    assert torch.equal(torch.isfinite(out[0, :5].double()), torch.isfinite(ref[0, :5]))


def test_captured_replayed_and_on_two_streams():
    m = mtp()
    lens, M = [500, 90], 3
    pool = pc.Pool(2, 9, 64, 2, 128, "bf16", seed=25)
    pool.fill([503, 93], seed=26)
    q = queries(2, M, 8, 128, torch.bfloat16, seed=27)
    first, _ = run(pool, q, lens, rope_theta=1e4)
    h = pool.handle(rope_theta=1e4)
    size = m.kv_workspace_size(h, 2, M, 8)
    ws = [m.alloc_workspace(size) for _ in range(2)]
    outs = [torch.zeros_like(q.contiguous()) for _ in range(2)]
    ln = i32(lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for s, w, o in zip(streams, ws, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            m.paged_attention(h, q, ln, o, w)
        graphs.append(g)
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, ws):
        assert torch.equal(o, first) and m.last_error(w) == m.MTP_OK
    # new lengths in the captured graph's own buffers: the schedule is made on the device
    ln.copy_(i32([77, 90]))
    graphs[0].replay()
    torch.cuda.synchronize()
    again, _ = run(pool, q, [77, 90], rope_theta=1e4)
    assert torch.equal(outs[0], again)


def test_a_small_workspace_is_refused():
    m = mtp()
    pool = pc.Pool(1, 3, 16, 1, 128, "bf16", seed=28)
    pool.fill([20], seed=29)
    q = queries(1, 1, 4, 128, torch.bfloat16, seed=30)
    h = pool.handle()
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    with pytest.raises(m.MTPError) as e:
        m.paged_attention(h, q, i32([19]), out, m.alloc_workspace(512))
    assert e.value.code == m.MTP_ERR_WORKSPACE and (out == 7.0).all()
    with pytest.raises(ValueError):
        m.paged_attention(h, q.expand(2, -1, -1, -1), i32([19, 19]), out.expand(2, -1, -1, -1).contiguous(), m.alloc_workspace(1 << 22))
