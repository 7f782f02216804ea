"""Attention of prompts and of shared prefixes with scores far apart: the largest
in the first, a middle or the last tile, or rising from tile to tile by steps
around those that move a row's reference.  The scores are exact in every type
(scores_common.py), so the bound is a probability's and the result's rounding
and little more; a result that is zero, negated or scaled wrongly is outside."""
import pytest
import torch

import paged_common as pc
import scores_common as sc

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


def put_scores(pool, b, z):
    """Keys whose scores are z on sequence b's positions [0, len(z)); e4m3: page scales 1/2, 1, 2."""
    t = torch.arange(z.numel(), device="cuda")
    pg, slot = pool.table[b].long()[t // pool.page], t % pool.page
    k = sc.keys(z.cuda(), pool.hd)
    if pool.dtype == "e4m3":
        pages = pool.table[b].long()[: -(-z.numel() // pool.page)]
        pool.ks[pages] = torch.exp2((torch.arange(pages.numel(), device="cuda") % 3 - 1).float())[:, None]
        codes = (k / pool.ks[pg].double()).to(torch.float8_e4m3fn).view(torch.uint8)
        pool.k.view(torch.uint8)[pg, 0, slot] = codes
    else:
        pool.k[pg, 0, slot] = k.to(pool.k.dtype)


def step_of(kv):
    return {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -11, "f32": 0.0}[kv]


def check(out, z, v, kv, T):
    """out [rows, heads, hd] against scores z [rows, T] (-inf: not attended) times the heads' factors."""
    power = []
    for h, f in enumerate(sc.FACTORS):
        ref, mass = sc.plain(z * f, v)
        tol = sc.bound(ref, mass, float(z[z > -1e9].abs().max()) * f, T, step_of(kv))
        err = (out[:, h].double() - ref).abs()
        assert (err <= tol).all(), (h, float((err / tol).max()))
        power += [((ref.abs() > tol).double().mean(), (2 * ref.abs() > tol).double().mean())]
    assert min(float(x) for pair in power for x in pair) > 0.8      # zeros and the negated result are outside


FORMS = [("bf16", 64), ("bf16", 128), ("bf16", 256), ("e4m3", 64), ("e4m3", 128), ("e4m3", 256), ("f32", 64), ("bf16", 512)]


@pytest.mark.parametrize("kind", sc.KINDS)
@pytest.mark.parametrize("kv,hd", FORMS)
def test_prompts(kv, hd, kind):
    m = mtp()
    g = torch.Generator().manual_seed(1)
    before, n = 300, 420                       # six tiles; rows see from three of them on
    T = before + n
    pool = pc.Pool(1, T // 32 + 2, 32, 1, hd, kv, seed=2)
    pool.fill([T], seed=3)
    z = sc.scores(kind, T, g)
    put_scores(pool, 0, z)
    q = sc.rows((n,), hd, g, "cuda")
    h = pool.handle()                          # (rope_theta 0)
    ws = m.alloc_workspace(m.prompt_workspace_size(h, 1, n, 4))
    out = torch.full_like(q, 7.0)
    m.prompt_attention(h, q, i32([0, n]), i32([before]), out, ws, attn_scale=1.0)
    assert m.last_error(ws) == m.MTP_OK
    p = torch.arange(before, T, device="cuda")
    see = torch.arange(T, device="cuda") <= p[:, None]
    v = pool.rows("v", 0, torch.arange(T))[0]
    check(out, z.cuda().expand(n, T).masked_fill(~see, -torch.inf), v, kv, T)


@pytest.mark.parametrize("kind", ("rising 5.625", "rising 2.875", "first", "last", "far"))
@pytest.mark.parametrize("kv,hd", FORMS[:6])
def test_a_long_item_cut_between_workers(kv, hd, kind):
    """Few rows behind many tiles: every part has a reference of its own."""
    m = mtp()
    g = torch.Generator().manual_seed(4)
    T, n = 9000, 5
    pool = pc.Pool(1, T // 64 + 2, 64, 1, hd, kv, seed=5)
    pool.fill([T], seed=6)
    z = sc.scores(kind, T, g)
    put_scores(pool, 0, z)
    q = sc.rows((n,), hd, g, "cuda")
    h = pool.handle()
    ws = m.alloc_workspace(m.prompt_workspace_size(h, 1, n, 4))
    out = torch.full_like(q, 7.0)
    m.prompt_attention(h, q, i32([0, n]), i32([T - n]), out, ws, attn_scale=1.0)
    assert m.last_error(ws) == m.MTP_OK
    see = torch.arange(T, device="cuda") <= torch.arange(T - n, T, device="cuda")[:, None]
    check(out, z.cuda().expand(n, T).masked_fill(~see, -torch.inf), pool.rows("v", 0, torch.arange(T))[0], kv, T)


@pytest.mark.parametrize("kind", sc.KINDS)
@pytest.mark.parametrize("kv,hd", FORMS)
def test_windows(kv, hd, kind):
    """The largest scores leave the window, or stay with the sink."""
    m = mtp()
    g = torch.Generator().manual_seed(7)
    T, window, sink = 700, 200, 20
    pool = pc.Pool(1, T // 16 + 2, 16, 1, hd, kv, seed=8)
    pool.fill([T], seed=9)
    z = sc.scores(kind, T, g)
    z[19] = 9.0
    put_scores(pool, 0, z)
    q = sc.rows((T,), hd, g, "cuda")
    h = pool.handle(window=window, sink=sink)
    ws = m.alloc_workspace(m.prompt_workspace_size(h, 1, T, 4))
    out = torch.full_like(q, 7.0)
    m.prompt_attention(h, q, i32([0, T]), i32([0]), out, ws, attn_scale=1.0)
    assert m.last_error(ws) == m.MTP_OK
    t = torch.arange(T, device="cuda")
    see = (t <= t[:, None]) & ((t > t[:, None] - window) | (t < sink))
    check(out, z.cuda().expand(T, T).masked_fill(~see, -torch.inf), pool.rows("v", 0, torch.arange(T))[0], kv, T)


@pytest.mark.parametrize("kind", sc.KINDS)
@pytest.mark.parametrize("kv,hd", FORMS)
def test_shared_prefixes(kv, hd, kind):
    """The largest score in the prefix for some sequences, in their own positions for others."""
    m = mtp()
    g = torch.Generator().manual_seed(10)
    B, M, P, page = 8, 2, 690, 32
    lens = [P + x for x in (0, 5, 130, 200, 64, 1, 300, 40)]
    pool = pc.Pool(B, (max(lens) + M) // page + 2, page, 1, hd, kv, seed=11)
    pool.fill([a + M for a in lens], seed=12)
    zs = []
    for b, a in enumerate(lens):
        z = sc.scores(kind, a + M, g)
        z[P:] += (0.0, 8.0, 5.5, -8.0)[b % 4]
        if b:
            z[:P] = zs[0][:P]
        zs.append(z)
        put_scores(pool, b, z)
    for b in range(1, B):
        pool.table[b, : P // page] = -1        # whole pages of the prefix: the first sequence's
    q = sc.rows((B, M), hd, g, "cuda")
    h = pool.handle()
    ws = m.alloc_workspace(m.prefix_workspace_size(h, B, M, 4))
    out = torch.full_like(q, 7.0)
    m.prefix_attention(h, q, i32(lens), i32([0, B]), i32([P]), out, ws, attn_scale=1.0)
    assert m.last_error(ws) == m.MTP_OK
    for b, a in enumerate(lens):
        T = a + M
        v = torch.cat([pool.rows("v", 0, torch.arange(P))[0], pool.rows("v", b, torch.arange(P, T))[0]])
        see = torch.arange(T, device="cuda") <= torch.arange(a, T, device="cuda")[:, None]
        check(out[b], zs[b].cuda().expand(M, T).masked_fill(~see, -torch.inf), v, kv, T)
