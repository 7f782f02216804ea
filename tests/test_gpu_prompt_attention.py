"""mtp_prompt_attention against a plain 64-bit form: types, head sizes, groups,
pages, packed lengths, cached positions, windows, absent pages, values that are
not finite, and rows it must leave alone."""
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


def queries(T, hq, hd, dtype, seed, extra=3):
    """Rows as a slice of a fused projection's output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, hq + extra, hd, device="cuda", generator=g).to(dtype)[:, :hq]


def starts(n, front=0):
    s = [front]
    for x in n:
        s.append(s[-1] + x)
    return s


def run(pool, q, row_start, lens, gain=None, ws=None, scale=None, out=None, **kw):
    m = mtp()
    h = pool.handle(**kw)
    T, hq, _ = q.shape
    ws = m.alloc_workspace(m.prompt_workspace_size(h, len(lens), T, hq)) if ws is None else ws
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    m.prompt_attention(h, q, i32(row_start), i32(lens), out, ws, q_norm=gain, attn_scale=scale)
    return out, m.last_error(ws)


def check(pool, out, q, gain, row_start, lens, theta, window=0, sink=0, scale=None, absent=None, random=True):
    used = torch.zeros(q.shape[0], dtype=torch.bool)
    for b, a in enumerate(lens):
        r0, r1 = row_start[b], row_start[b + 1]
        used[r0:r1] = True
        if r1 > r0:
            ref = rc.attend(pool, b, q[r0:r1], gain, a, theta, window, sink, scale, (absent or {}).get(b, ()))
            rc.check(out[r0:r1], *ref, a + r1 - r0, pool.dtype, random)
    assert (out[~used] == 7.0).all(), "a row of no sequence has changed"


CASES = [
    # kv, q, hd, hkv, G, page, cached, n, norm, theta, window, sink, layout
    ("bf16", "bf16", 256, 2, 4, 16, [0], [77], True, 1e6, 0, 0, "head"),
    ("bf16", "bf16", 256, 1, 4, 64, [0], [1], True, 1e6, 0, 0, "slot"),
    ("bf16", "bf16", 256, 4, 4, 64, [0, 5, 1000, 63, 127], [300, 1, 64, 0, 129], True, 1e6, 0, 0, "slot"),
    ("bf16", "bf16", 256, 1, 7, 32, [0, 130], [1500, 33], False, 1e4, 0, 0, "head"),
    ("bf16", "bf16", 256, 2, 1, 128, [3, 0], [700, 256], True, 1e6, 0, 0, "slot"),
    ("bf16", "bf16", 256, 1, 16, 256, [100], [90], True, 1e6, 0, 0, "head"),
    ("bf16", "bf16", 128, 2, 2, 32, [0, 0, 0, 0, 0], [513, 1, 127, 128, 640], False, 1e4, 0, 0, "head"),
    ("bf16", "bf16", 128, 1, 7, 16, [64, 2000], [200, 3], True, 1e4, 0, 0, "slot"),
    ("bf16", "bf16", 128, 2, 8, 128, [0, 1], [1100, 31], True, 1e6, 0, 0, "head"),
    ("bf16", "bf16", 128, 1, 1, 64, [0], [2049], False, 0.0, 0, 0, "head"),
    ("bf16", "bf16", 64, 2, 4, 16, [0, 17, 900], [300, 0, 100], True, 1e4, 0, 0, "slot"),
    ("bf16", "bf16", 64, 8, 1, 64, [0], [1025], False, 1e4, 0, 0, "head"),
    # windows: shorter and longer than a tile, sinks that reach over the window's start
    ("bf16", "bf16", 256, 1, 4, 64, [0, 1500], [1400, 70], False, 1e4, 1024, 130, "head"),
    ("bf16", "bf16", 256, 2, 4, 32, [0, 40], [500, 200], True, 1e4, 100, 4, "slot"),
    ("bf16", "bf16", 128, 2, 2, 32, [0, 2500], [900, 260], False, 1e4, 128, 0, "slot"),
    ("bf16", "bf16", 128, 1, 4, 16, [0, 333], [400, 50], True, 1e4, 1, 0, "head"),
    ("bf16", "bf16", 64, 1, 4, 16, [7], [600], True, 1e4, 300, 270, "head"),
    ("e4m3", "bf16", 256, 2, 4, 64, [0, 700, 5], [300, 64, 1], True, 1e6, 0, 0, "head"),
    ("e4m3", "bf16", 256, 1, 8, 16, [1000], [257], False, 1e4, 0, 0, "slot"),
    ("e4m3", "bf16", 256, 1, 4, 32, [0, 200], [700, 90], True, 1e4, 200, 20, "slot"),
    ("e4m3", "bf16", 128, 2, 7, 32, [0, 31], [400, 130], True, 1e4, 0, 0, "slot"),
    ("e4m3", "bf16", 128, 1, 2, 256, [300], [900], False, 1e6, 0, 0, "head"),
    ("e4m3", "bf16", 64, 2, 4, 16, [0, 250], [513, 2], True, 1e4, 0, 0, "head"),
    ("e4m3", "bf16", 64, 1, 16, 128, [60], [129], False, 1e4, 90, 5, "slot"),
    # the types and heads of the CUDA cores
    ("f32", "f32", 128, 2, 4, 16, [0, 33], [130, 20], True, 1e4, 0, 0, "slot"),
    ("f32", "bf16", 64, 1, 4, 32, [65], [40], False, 1e4, 0, 0, "head"),
    ("bf16", "f32", 256, 1, 3, 32, [150], [50], True, 1e6, 50, 7, "slot"),
    ("e4m3", "f32", 256, 2, 2, 64, [0], [180], True, 1e6, 0, 0, "head"),
    ("bf16", "bf16", 512, 1, 2, 64, [10], [140], True, 1e6, 0, 0, "head"),
    ("e4m3", "bf16", 512, 1, 2, 64, [10], [40], True, 1e6, 0, 0, "head"),
    ("bf16", "bf16", 32, 2, 2, 16, [0, 3], [100, 9], True, 1e4, 0, 0, "head"),
    ("e4m3", "bf16", 32, 1, 2, 16, [30], [70], False, 0.0, 30, 3, "slot"),
]


@pytest.mark.parametrize("kv,qt,hd,hkv,G,page,lens,n,norm,theta,window,sink,layout", CASES)
def test_prompts_attend_the_cache(kv, qt, hd, hkv, G, page, lens, n, norm, theta, window, sink, layout):
    front, back = 2, 3                                 # rows of no sequence
    ends = [a + c for a, c in zip(lens, n)]
    pool = pc.Pool(len(lens), (max(ends) + page - 1) // page + 1, page, hkv, hd, kv, seed=1, layout=layout)
    pool.fill(ends, seed=2)
    at = starts(n, front)
    q = queries(at[-1] + back, hkv * G, hd, torch.bfloat16 if qt == "bf16" else torch.float32, seed=3)
    gain = 1 + 0.1 * torch.randn(hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)) if norm else None
    out, st = run(pool, q, at, lens, gain, rope_theta=theta, window=window, sink=sink)
    assert st == mtp().MTP_OK
    check(pool, out, q, gain, at, lens, theta, window, sink)


@pytest.mark.parametrize("kv,hd,hkv,G", [("bf16", 256, 1, 4), ("bf16", 128, 2, 2), ("e4m3", 256, 1, 4), ("e4m3", 128, 1, 8), ("bf16", 64, 2, 2)])
def test_many_prompts_of_ragged_lengths(kv, hd, hkv, G):
    """More row tiles than the GPU holds at a time, tiles cut between CTAs, and
    empty prompts between them; the same call twice gives the same bits, and a
    workspace of a larger call serves it."""
    m = mtp()
    g = torch.Generator().manual_seed(4)
    B, page = 60, 32
    n = torch.randint(0, 260, (B,), generator=g).tolist()
    lens = torch.randint(0, 300, (B,), generator=g).tolist()
    n[7], lens[7], n[8], n[9], lens[30] = 1700, 0, 0, 1, 5000
    ends = [a + c for a, c in zip(lens, n)]
    pool = pc.Pool(B, max(ends) // page + 2, page, hkv, hd, kv, seed=5)
    pool.fill(ends, seed=6)
    at = starts(n)
    q = queries(at[-1], hkv * G, hd, torch.bfloat16, seed=7)
    h = pool.handle(rope_theta=1e6)
    ws = m.alloc_workspace(m.prompt_workspace_size(h, B + 100, at[-1] + 5000, hkv * G))
    ws.fill_(0xFF)
    out, st = run(pool, q, at, lens, ws=ws, rope_theta=1e6)
    assert st == m.MTP_OK
    check(pool, out, q, None, at, lens, 1e6)
    ws.fill_(0x5A)
    again, _ = run(pool, q, at, lens, ws=ws, rope_theta=1e6)
    assert torch.equal(out, again)


def test_the_largest_batch():
    for kv, hd, G in (("bf16", 256, 4), ("e4m3", 64, 2), ("bf16", 128, 1)):
        m = mtp()
        B, page = m.MTP_MAX_PAGED_BATCH, 16
        g = torch.Generator().manual_seed(31)
        lens, n = (torch.randint(0, 30, (B,), generator=g).tolist() for _ in range(2))
        pool = pc.Pool(B, 4, page, 1, hd, kv, seed=32)
        pool.fill([a + c for a, c in zip(lens, n)], seed=33)
        at = starts(n)
        q = queries(at[-1], G, hd, torch.bfloat16, seed=34)
        out, st = run(pool, q, at, lens, rope_theta=1e4)
        assert st == m.MTP_OK
        for b in list(range(0, B, 37)) + [B - 1]:
            if n[b]:
                r = rc.attend(pool, b, q[at[b]:at[b + 1]], None, lens[b], 1e4)
                rc.check(out[at[b]:at[b + 1]], *r, 60, kv)


def test_one_long_context():
    for kv, hd in (("bf16", 128), ("e4m3", 256), ("bf16", 256)):
        lens, n = [20011], 5
        pool = pc.Pool(1, lens[0] // 128 + 2, 128, 1, hd, kv, seed=8)
        pool.fill([lens[0] + n], seed=9)
        q = queries(n, 4, hd, torch.bfloat16, seed=10)
        out, st = run(pool, q, [0, n], lens, rope_theta=1e6)
        assert st == mtp().MTP_OK
        check(pool, out, q, None, [0, n], lens, 1e6)


@pytest.mark.parametrize("kv,hd", [("bf16", 128), ("bf16", 256), ("e4m3", 128), ("e4m3", 256), ("f32", 64)])
def test_far_scores_and_spread_scales(kv, hd):
    """Scores a hundred apart with their maximum anywhere, and page scales far
    apart: the running maximum and the sums hold."""
    n = 700
    pool = pc.Pool(1, 40, 32, 1, hd, kv, seed=11)
    pool.fill([n + 100], seed=12)
    if kv == "e4m3":
        pool.vs[pool.table[0].long()[::3]] *= 2.0 ** -12
        pool.ks[pool.table[0].long()[5:9]] *= 4
    q = queries(n, 4, hd, torch.bfloat16, seed=13) * 8
    out, st = run(pool, q, [0, n], [100], rope_theta=1e4, scale=0.25)
    assert st == mtp().MTP_OK
    check(pool, out, q, None, [0, n], [100], 1e4, scale=0.25, random=False)


@pytest.mark.parametrize("kv,hd", [("bf16", 128), ("bf16", 256), ("e4m3", 256), ("f32", 128)])
def test_absent_pages_are_masked_and_reported(kv, hd):
    m = mtp()
    pool = pc.Pool(2, 30, 16, 2, hd, kv, seed=14)
    pool.fill([400, 200], seed=15)
    pool.table[0, 3], pool.table[0, 20], pool.table[1, :13] = -1, 10 ** 6, -1      # sequence 1 has nothing at all
    q = queries(500, 4, hd, torch.bfloat16 if kv != "f32" else torch.float32, seed=16)
    out, st = run(pool, q, [0, 350, 500], [50, 50], rope_theta=1e4)
    assert st == m.MTP_ERR_ARG
    gone = {0: list(range(48, 64)) + list(range(320, 336)), 1: list(range(200))}
    for t in (3, 20):
        pool.table[0, t] = 0
    pool.table[1, :13] = 0
    check(pool, out, q, None, [0, 350, 500], [50, 50], 1e4, absent=gone)
    assert (out[350:] == 0).all()


def test_pages_outside_the_windows_may_be_absent():
    m = mtp()
    pool = pc.Pool(1, 60, 16, 1, 128, "bf16", seed=17)
    pool.fill([900], seed=18)
    q = queries(200, 4, 128, torch.bfloat16, seed=19)
    saved = pool.table.clone()
    pool.table[0, 1:37] = -1                                # rows from 700 on, a window of 100: [601, ..) and [0, 4)
    out, st = run(pool, q, [0, 200], [700], rope_theta=1e4, window=100, sink=4)
    assert st == m.MTP_OK
    pool.table.copy_(saved)
    check(pool, out, q, None, [0, 200], [700], 1e4, 100, 4)


def test_sequences_out_of_range_are_left_out():
    m = mtp()
    pool = pc.Pool(5, 8, 16, 1, 128, "bf16", seed=20)
    pool.fill([100] * 5, seed=21)
    q = queries(200, 2, 128, torch.bfloat16, seed=22)
    for at, lens, good in (([0, 40, 80, 120, 160, 200], [60, -1, 60, 100, 60], [0, 2, 4]),     # 100 + 40 > 128
                           ([-5, 40, 80, 120, 160, 200], [60] * 5, [1, 2, 3, 4]),
                           ([0, 40, 80, 120, 160, 201], [60] * 5, [0, 1, 2, 3]),
                           ([0, 40, 30, 70, 110, 150], [60] * 5, [0, 2, 3, 4])):
        out, st = run(pool, q, at, lens, rope_theta=1e4)
        assert st == m.MTP_ERR_ARG
        if at[2] == 30:      # rows 30..39 belong to two sequences: either's answer
            out[30:40] = 7.0
            for b in (3, 4):
                rc.check(out[at[b]:at[b + 1]], *rc.attend(pool, b, q[at[b]:at[b + 1]], None, 60, 1e4), 100, "bf16")
            continue
        for b in range(5):
            r0, r1 = max(0, at[b]), min(200, at[b + 1])
            if b in good:
                rc.check(out[r0:r1], *rc.attend(pool, b, q[r0:r1], None, 60, 1e4), 100, "bf16")
            else:
                assert (out[r0:r1] == 7.0).all()


@pytest.mark.parametrize("kv,hd", [("bf16", 128), ("bf16", 256), ("e4m3", 256), ("e4m3", 64), ("f32", 64)])
def test_values_that_are_not_finite_reach_the_rows_that_attend_them(kv, hd):
    m = mtp()
    n, G = 300, 2
    pool = pc.Pool(1, 24, 16, 1, hd, kv, seed=23)
    pool.fill([n], seed=24)
    q = queries(n, G, hd, torch.bfloat16 if kv != "f32" else torch.float32, seed=25)
    want, _ = run(pool, q, [0, n], [0], rope_theta=1e4)
    nan, inf = (200, 3), (260, 7)                       # (position, dimension)
    cell = lambda t: (int(pool.table[0, t // 16]), 0, t % 16)   # noqa: E731
    if kv == "e4m3":
        pool.v.view(torch.uint8)[cell(nan[0]) + (nan[1],)] = 0x7F
    else:
        pool.v[cell(nan[0]) + (nan[1],)] = float("nan")
        pool.v[cell(inf[0]) + (inf[1],)] = float("-inf")
    out, st = run(pool, q, [0, n], [0], rope_theta=1e4)
    assert st == m.MTP_OK
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[nan[0]:, :, nan[1]] = True
    assert out[hit].isnan().all()
    if kv != "e4m3":
        assert (out[inf[0]:, :, inf[1]] == float("-inf")).all()
        hit[inf[0]:, :, inf[1]] = True
    # the other dimensions and the rows before them: as before, up to how they are summed
    d = (out.float() - want.float()).abs()[~hit]
    assert (d <= 2.0 ** -5 * (1 + want.float().abs()[~hit])).all()


def test_masks_of_nan_slots_hold_in_every_tile():
    """Slots behind a sequence's end, pages of other sequences and the rest of a
    tile are NaN (the pool is made so): none of it shows.  Lengths around the
    edges of tiles and pages."""
    for hd in (64, 128, 256):
        for kv in ("bf16", "e4m3"):
            n = [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257]
            pool = pc.Pool(len(n), 18, 16, 1, hd, kv, seed=26)
            pool.fill(n, seed=27)
            q = queries(sum(n), 1, hd, torch.bfloat16, seed=28)
            out, st = run(pool, q, starts(n), [0] * len(n), rope_theta=1e4)
            assert st == mtp().MTP_OK
            check(pool, out, q, None, starts(n), [0] * len(n), 1e4)


def test_same_rows_as_the_verify_steps_attention():
    """Up to 64 rows a sequence mtp_paged_attention takes too: the same answers
    within both roundings."""
    m = mtp()
    for kv, hd, G in (("bf16", 256, 4), ("e4m3", 128, 4)):
        B, M, page, lens = 3, 40, 32, [0, 100, 1000]
        pool = pc.Pool(B, 40, page, 2, hd, kv, seed=29)
        pool.fill([a + M for a in lens], seed=30)
        q = queries(B * M, 2 * G, hd, torch.bfloat16, seed=31, extra=0)
        out, _ = run(pool, q, [0, M, 2 * M, 3 * M], lens, rope_theta=1e6)
        h = pool.handle(rope_theta=1e6)
        ws = m.alloc_workspace(m.kv_workspace_size(h, B, M, 2 * G))
        other = torch.empty(B, M, 2 * G, hd, dtype=torch.bfloat16, device="cuda")
        m.paged_attention(h, q.view(B, M, 2 * G, hd), i32(lens), other, ws)
        d = out.double() - other.view_as(out).double()
        assert d.square().mean().sqrt() <= 2.0 ** -7 * other.double().square().mean().sqrt()


def test_captured_and_on_another_stream():
    m = mtp()
    for hd, kv in ((256, "bf16"), (128, "e4m3")):
        n, lens = [200, 3, 90], [0, 500, 40]
        pool = pc.Pool(3, 20, 32, 2, hd, kv, seed=35)
        pool.fill([a + c for a, c in zip(lens, n)], seed=36)
        at, hq = starts(n), 8
        q = queries(at[-1], hq, hd, torch.bfloat16, seed=37)
        want, _ = run(pool, q, at, lens, rope_theta=1e4)
        h = pool.handle(rope_theta=1e4)
        ws = m.alloc_workspace(m.prompt_workspace_size(h, 3, at[-1], hq))
        out = torch.zeros_like(want)
        a, ln = i32(at), i32(lens)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        m.prompt_attention(h, q, a, ln, out, ws, stream=s)
        s.synchronize()
        assert torch.equal(out, want)
        # two graphs that share the workspace, replayed in turn with other lengths
        graphs, outs = [], [torch.zeros_like(want) for _ in range(2)]
        for o in outs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                m.prompt_attention(h, q, a, ln, o, ws)
            graphs.append(g)
        graphs[0].replay()
        a.copy_(i32([0, 150, 150, 290]))
        ln.copy_(i32([0, 500, 0]))
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want)
        other, _ = run(pool, q, [0, 150, 150, 290], [0, 500, 0], out=torch.zeros_like(want), rope_theta=1e4)
        # (sequence 2's last ten positions were never written: NaN on both sides)
        assert torch.equal(outs[1].nan_to_num(9.0), other.nan_to_num(9.0))


def test_no_row_at_all():
    m = mtp()
    pool = pc.Pool(2, 4, 16, 1, 128, "bf16", seed=38)
    q = queries(6, 2, 128, torch.bfloat16, seed=39)
    out, st = run(pool, q, [3, 3, 3], [0, 0], rope_theta=1e4)
    assert st == m.MTP_OK and (out == 7.0).all()
