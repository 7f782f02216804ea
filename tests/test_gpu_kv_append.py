"""mtp_kv_append against a plain 64-bit form: types, head sizes, page sizes,
lengths, layouts, the 8-bit scales' rule, and what it must leave alone."""
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


def rows(B, M, hkv, hd, dtype, seed, hq=2):
    """k and v rows as slices of a fused projection's output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(B, M, (hq + 2 * hkv) * hd, device="cuda", generator=g).to(dtype)
    k = qkv[..., hq * hd:(hq + hkv) * hd].unflatten(-1, (hkv, hd))
    v = qkv[..., (hq + hkv) * hd:].unflatten(-1, (hkv, hd))
    return k, v


def snapshot(pool):
    bits = {"f32": torch.int32, "bf16": torch.int16, "e4m3": torch.uint8}[pool.dtype]
    return {w: getattr(pool, w).view(bits).clone() for w in "kv"}


def check(pool, before, k, v, gain, lens, n_new, theta, scales_before=None):
    """Every written slot against the definition, every other byte unchanged."""
    after = snapshot(pool)
    for w, src in (("k", k), ("v", v)):
        touched = torch.zeros(before[w].shape[:3], dtype=torch.bool, device="cuda")
        for b, n in enumerate(n_new):
            if n == 0:
                continue
            pos = torch.arange(lens[b], lens[b] + n, device="cuda")
            x = pc.turn(src[b, :n], gain, pos, theta) if w == "k" else src[b, :n].double()
            x = x.transpose(0, 1)                                      # [heads, n, hd]
            tol = pc.turn_tol(x) if w == "k" else torch.zeros_like(x)
            got = pool.rows(w, b, pos)
            pg = pool.table[b].long()[pos // pool.page]
            touched[pg, :, pos % pool.page] = True
            if pool.dtype == "f32":
                assert ((got - x).abs() <= tol).all()
            elif pool.dtype == "bf16":
                assert ((got - x).abs() <= tol + 2.0 ** -8 * (x.abs() + tol)).all()
            else:
                scale = getattr(pool, w + "s")
                for page0 in range(lens[b] // pool.page, (lens[b] + n - 1) // pool.page + 1):
                    lo, hi = max(lens[b], page0 * pool.page), min(lens[b] + n, (page0 + 1) * pool.page)
                    p = int(pool.table[b, page0])
                    y = x[:, lo - lens[b]:hi - lens[b]]
                    t = tol[:, lo - lens[b]:hi - lens[b]]
                    off = lo % pool.page
                    for h in range(pool.hkv):
                        s = float(scale[p, h])
                        amax = float(y[h].abs().max())
                        want = {pc.pow2_scale(amax * (1 + 2.0 ** -19)), pc.pow2_scale(amax * (1 - 2.0 ** -19))}
                        if off:
                            want = {max(a, float(scales_before[w][p, h])) for a in want}
                        assert s in want, (w, b, page0, h, s, want)
                        d = (got[h, lo - lens[b]:hi - lens[b]] - y[h]).abs()
                        assert (d <= t[h] + torch.maximum(2.0 ** -4 * (y[h].abs() + t[h]), torch.tensor(2.0 ** -10 * s).double())).all()
                        if off:   # older codes: the same values, re-rounded where the scale grew
                            old = before[w][p, h, :off].view(torch.float8_e4m3fn).double() * float(scales_before[w][p, h])
                            new = after[w][p, h, :off].view(torch.float8_e4m3fn).double() * s
                            if s == float(scales_before[w][p, h]):
                                assert torch.equal(before[w][p, h, :off], after[w][p, h, :off])
                            else:
                                assert ((old - new).abs() <= torch.maximum(2.0 ** -4 * old.abs(), torch.tensor(2.0 ** -10 * s).double())).all()
                    touched[p, :, :off] = True
        keep = ~touched[..., None].expand_as(before[w])
        assert torch.equal(before[w][keep], after[w][keep]), "a slot that no row went to has changed"


CASES = [
    # kv, in, hd, hkv, page, B, M, lens, n_new, norm, theta, layout
    ("bf16", "bf16", 256, 4, 64, 2, 4, [0, 61], None, True, 1e6, "head"),
    ("bf16", "f32", 128, 8, 32, 1, 1, [31], None, False, 1e4, "slot"),
    ("bf16", "bf16", 64, 3, 16, 3, 5, [16, 0, 7], [5, 0, 2], True, 1e4, "slot"),
    ("bf16", "f32", 512, 1, 128, 2, 130, [127, 1], [130, 77], True, 1e6, "head"),
    ("bf16", "bf16", 32, 2, 16, 2, 17, [3, 15], [17, 16], True, 1e4, "head"),
    ("bf16", "bf16", 256, 4, 64, 1, 3000, [5], None, True, 1e6, "slot"),
    ("f32", "f32", 128, 2, 16, 2, 3, [14, 0], [3, 1], True, 1e4, "head"),
    ("f32", "bf16", 256, 1, 256, 1, 40, [250], None, False, 0.0, "slot"),
    ("e4m3", "bf16", 256, 4, 64, 3, 4, [0, 62, 64], [4, 4, 0], True, 1e6, "head"),
    ("e4m3", "f32", 128, 2, 16, 2, 1, [0, 15], None, False, 1e4, "slot"),
    ("e4m3", "bf16", 64, 8, 32, 2, 100, [31, 0], [100, 33], True, 1e4, "slot"),
    ("e4m3", "f32", 512, 2, 256, 1, 300, [100], None, True, 1e6, "head"),      # more rows of a page than a CTA keeps
    ("e4m3", "bf16", 512, 1, 128, 2, 128, [0, 128], None, True, 1e6, "slot"),
    ("e4m3", "bf16", 32, 2, 16, 2, 6, [13, 2], None, True, 0.0, "head"),
    ("e4m3", "bf16", 256, 1, 16, 64, 3, list(range(64)), None, False, 1e7, "head"),
]


@pytest.mark.parametrize("kv,inp,hd,hkv,page,B,M,lens,n_new,norm,theta,layout", CASES)
def test_rows_reach_their_slots(kv, inp, hd, hkv, page, B, M, lens, n_new, norm, theta, layout):
    m = mtp()
    n = n_new or [M] * B
    pool = pc.Pool(B, (max(lens) + M + page - 1) // page + 1, page, hkv, hd, kv, seed=1, layout=layout)
    pool.fill(lens, seed=2)
    k, v = rows(B, M, hkv, hd, torch.bfloat16 if inp == "bf16" else torch.float32, seed=3)
    gain = 1 + 0.1 * torch.randn(hd, device="cuda") if norm else None
    before = snapshot(pool)
    sb = {"k": pool.ks.clone(), "v": pool.vs.clone()} if kv == "e4m3" else None
    h = pool.handle(rope_theta=theta)
    ws = m.alloc_workspace(m.kv_workspace_size(h, B, M, hkv))
    m.kv_append(h, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), ws,
                n_new=None if n_new is None else torch.tensor(n, dtype=torch.int32, device="cuda"), k_norm=gain)
    assert m.last_error(ws) == m.MTP_OK
    check(pool, before, k, v, gain, lens, n, theta, sb)


def test_far_positions_keep_their_angle():
    """Positions of a million: the angle in fp32 would be off by whole turns'
    thousandths; the tolerance is the same as at position 0."""
    m = mtp()
    page, B, M, hkv, hd = 256, 2, 3, 1, 128
    lens = [1000003, (1 << 24) + 12345]
    pool = pc.Pool(B, 8, page, hkv, hd, "f32", seed=4)
    full = torch.full((B, lens[1] // page + 2), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        full[b, lens[b] // page: lens[b] // page + 2] = pool.table[b, :2]
    pool.table = full
    k, v = rows(B, M, hkv, hd, torch.float32, seed=5)
    before = snapshot(pool)
    h = pool.handle(rope_theta=1e4)
    ws = m.alloc_workspace(m.kv_workspace_size(h, B, M, hkv))
    m.kv_append(h, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), ws)
    assert m.last_error(ws) == m.MTP_OK
    check(pool, before, k, v, None, lens, [M] * B, 1e4)


def test_scale_grows_in_place_and_starts_anew_on_a_new_page():
    m = mtp()
    page, hkv, hd = 16, 2, 64
    pool = pc.Pool(1, 4, page, hkv, hd, "e4m3", seed=6)
    h = pool.handle()
    ws = m.alloc_workspace(m.kv_workspace_size(h, 1, 16, hkv))
    g = torch.Generator(device="cuda").manual_seed(7)
    at = 0
    for n, mag in ((3, 1e-3), (4, 1.0), (2, 1e-2), (7, 300.0), (5, 1e-4), (0, 1.0), (11, 50.0)):
        x = torch.randn(1, max(n, 1), hkv, hd, device="cuda", generator=g) * mag
        y = torch.randn(1, max(n, 1), hkv, hd, device="cuda", generator=g) * mag * 3
        before, sb = snapshot(pool), {"k": pool.ks.clone(), "v": pool.vs.clone()}
        m.kv_append(h, x, y, torch.tensor([at], dtype=torch.int32, device="cuda"), ws,
                    n_new=torch.tensor([n], dtype=torch.int32, device="cuda"))
        assert m.last_error(ws) == m.MTP_OK
        check(pool, before, x, y, None, [at], [n], 0.0, sb)
        at += n
    # rejected drafts: the same positions are written again, the scale only grows
    top = pool.ks.clone()
    x = torch.randn(1, 4, hkv, hd, device="cuda", generator=g)
    before, sb = snapshot(pool), {"k": pool.ks.clone(), "v": pool.vs.clone()}
    m.kv_append(h, x, x, torch.tensor([at - 4], dtype=torch.int32, device="cuda"), ws)
    check(pool, before, x, x, None, [at - 4], [4], 0.0, sb)
    pg = int(pool.table[0, (at - 1) // page])
    assert (pool.ks[pg] >= top[pg]).all()


def test_borders_of_the_scale_and_values_that_are_not_finite():
    m = mtp()
    pool = pc.Pool(1, 2, 16, 1, 32, "e4m3", seed=8)
    h = pool.handle()
    ws = m.alloc_workspace(m.kv_workspace_size(h, 1, 16, 1))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    for amax in (448.0, 448.0 * (1 + 2.0 ** -20), 447.9, 0.0, 2.0 ** -60, 448 * 2.0 ** 39, 3e38, 1.75, 1.7500001, 1e-42):
        x = torch.zeros(1, 1, 1, 32, device="cuda")
        x[0, 0, 0, 5] = -amax
        m.kv_append(h, x, x, zero, ws)
        s = float(pool.ks[int(pool.table[0, 0]), 0])
        assert s == pc.pow2_scale(float(x.abs().max())), amax
        got = float(pool.rows("v", 0, [0])[0, 0, 5])
        assert abs(got + float(x.abs().max())) <= max(2.0 ** -4 * float(x.abs().max()), 2.0 ** -10 * s) or amax > 448 * 2.0 ** 40
        if amax > 448 * 2.0 ** 40:
            assert got == -448 * 2.0 ** 40          # saturates
    x = torch.randn(1, 3, 1, 32, device="cuda")
    x[0, 0, 0, 3], x[0, 1, 0, 4], x[0, 2, 0, 5] = float("nan"), float("inf"), -float("inf")
    m.kv_append(h, x, x, zero, ws)
    got = pool.rows("v", 0, [0, 1, 2])[0]
    bad = ~torch.isfinite(x[0, :, 0])
    assert torch.equal(torch.isnan(got), bad)
    fine = x[0, :, 0].masked_fill(bad, 0).double()
    assert float(pool.vs[int(pool.table[0, 0]), 0]) == pc.pow2_scale(float(fine.abs().max()))


def test_bad_lengths_and_absent_pages_leave_the_rest_alone():
    m = mtp()
    page, B, M, hkv, hd = 16, 5, 20, 2, 64
    for kv in ("bf16", "e4m3"):
        pool = pc.Pool(B, 4, page, hkv, hd, kv, seed=9)
        lens, n = [0, -1, 60, 5, 10], [20, 3, 5, 21, 20]     # 1: negative, 2: past the table, 3: more rows than M
        pool.table[4, 1] = -1                                 # positions 16..29 of sequence 4 have no page
        pool.fill([0, 0, 0, 0, 10], seed=1)
        k, v = rows(B, M, hkv, hd, torch.bfloat16, seed=10)
        before = snapshot(pool)
        sb = {"k": pool.ks.clone(), "v": pool.vs.clone()} if kv == "e4m3" else None
        h = pool.handle(rope_theta=1e4)
        ws = m.alloc_workspace(m.kv_workspace_size(h, B, M, hkv))
        m.kv_append(h, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), ws,
                    n_new=torch.tensor(n, dtype=torch.int32, device="cuda"))
        assert m.last_error(ws) == m.MTP_ERR_ARG
        check(pool, before, k, v, None, [0, 0, 0, 0, 10], [20, 0, 0, 0, 6], 1e4, sb)
        m.kv_append(h, k[:1], v[:1], torch.zeros(1, dtype=torch.int32, device="cuda"), ws)
        assert m.last_error(ws) == m.MTP_OK                  # the next good call's status


def test_pool_beyond_32_bit_offsets():
    m = mtp()
    n, hkv, page, hd = 36000, 4, 64, 256                      # 2.4e9 elements each
    k = torch.zeros(n, hkv, page, hd, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[n - 1, 3]], dtype=torch.int32, device="cuda")
    h = m.make_kv_cache(k, v, table)
    ws = m.alloc_workspace(m.kv_workspace_size(h, 1, 70, 16))
    x, y = rows(1, 70, hkv, hd, torch.bfloat16, seed=11)
    m.kv_append(h, x, y, torch.zeros(1, dtype=torch.int32, device="cuda"), ws)
    assert m.last_error(ws) == m.MTP_OK
    assert torch.equal(k[n - 1], x[0, :64].transpose(0, 1)) and torch.equal(v[n - 1], y[0, :64].transpose(0, 1))
    assert torch.equal(k[3, :, :6], x[0, 64:].transpose(0, 1)) and not k[3, :, 6:].any() and not k[4].any()
    q = torch.randn(1, 1, 16, hd, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    m.paged_attention(h, q, torch.tensor([69], dtype=torch.int32, device="cuda"), out, ws)
    p = torch.softmax(q[0, 0].double().view(hkv, 4, hd) @ x[0].double().permute(1, 2, 0) / 16, -1)
    vv = y[0].double().transpose(0, 1)
    ref, mass = (p @ vv).view(16, hd), (p @ vv.abs()).view(16, hd)
    tol = pc.attention_tol(ref, mass, torch.full((16,), 60.0, dtype=torch.float64, device="cuda"), hd, 70, True)
    assert ((out[0, 0].double() - ref).abs() <= tol).all()


def test_captured_and_replayed_on_another_stream():
    m = mtp()
    page, B, M, hkv, hd = 32, 4, 3, 2, 128
    s = torch.cuda.Stream()
    pools = [pc.Pool(B, 4, page, hkv, hd, "e4m3", seed=12) for _ in range(2)]
    k, v = rows(B, M, hkv, hd, torch.bfloat16, seed=13)
    lens = torch.tensor([0, 30, 31, 32], dtype=torch.int32, device="cuda")
    for p in pools:
        p.fill([0, 30, 31, 32], seed=14)
    h = pools[0].handle(rope_theta=1e4)
    ws = m.alloc_workspace(m.kv_workspace_size(h, B, M, hkv))
    m.kv_append(h, k, v, lens, ws)
    h2 = pools[1].handle(rope_theta=1e4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            m.kv_append(h2, k, v, lens, ws)
        g.replay()
        g.replay()
    s.synchronize()
    for w in ("k", "v"):
        assert torch.equal(getattr(pools[0], w).view(torch.uint8), getattr(pools[1], w).view(torch.uint8))
    assert torch.equal(pools[0].ks.nan_to_num(-1), pools[1].ks.nan_to_num(-1))
