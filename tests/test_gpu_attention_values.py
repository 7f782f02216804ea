"""mtp_paged_attention where single values decide: the bits that the
tensor-core path keeps of a probability, infinite and NaN values, scores of any
size, and page scales that are none."""
import math

import pytest
import torch

import paged_common as pc
from test_gpu_paged_attention import check, queries, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mtp_speculative_decoding_gb300 import build
    build.build()


def mtp():
    import mtp_speculative_decoding_gb300 as m
    return m


def put(pool, w, t, x):
    """Row t of sequence 0, KV head 0, becomes x (e4m3: codes under a scale of 1)."""
    pg, sl = int(pool.table[0, t // pool.page]), t % pool.page
    x = torch.as_tensor(x, dtype=torch.float32, device="cuda")
    if pool.dtype == "e4m3":
        getattr(pool, w).view(torch.uint8)[pg, 0, sl] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        getattr(pool, w)[pg, 0, sl] = x.to(pool.k.dtype)


# ---------------------------------------------------------------------------
# the bits of a probability
# ---------------------------------------------------------------------------

def parts_left(e, dtype, parts):
    """What `parts` successive roundings to dtype leave of e."""
    for _ in range(parts):
        e = e - e.to(torch.float32).to(dtype).double()
    return e


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_the_bits_of_a_probability(kv):
    """Two groups of positions with values +1 and -1 whose probabilities nearly
    cancel, chosen so that one operand part fewer than the path keeps would
    round every one of a group up and of the other down.

    The probabilities keep 16 bits (bf16: two parts, off by at most 2^-16 of
    each) or 9 (e4m3: three e5m2 parts, 2^-9, of a binary16 that is off by
    2^-11).  Everything else: the query is 1 in the dimensions that the keys
    use, so a score z (at most 1.1 in size) is a sum of 4 products, each off
    by what the query's parts leave (2^-16 or 2^-12) of sum |q k| <= 1.2 and
    by the accumulation's 2 (2 hd + 80) u; a probability is off by twice
    that (numerator and sum).  The two sums run over 129 terms: 2 (2 T + 200)
    u of the mass.  The output rounds to bf16, 2^-8 of itself, and it is
    small: at most 2^-8 of the mass, or 2^-5 against e4m3."""
    hd, n, T = 128, 64, 129
    low = {"bf16": torch.bfloat16, "e4m3": torch.float8_e5m2}[kv]
    keeps = {"bf16": 2, "e4m3": 3}[kv]
    # keys: one or two representable numbers whose sum is the score, in natural units
    if kv == "bf16":
        a = -torch.arange(32, 160, dtype=torch.float64) / 256                       # bf16 numbers
    else:
        a = -torch.arange(8, 16, dtype=torch.float64) / 16                          # e4m3 numbers
    b = -torch.arange(8, 16, dtype=torch.float64) / 512
    c = (a[:, None] + b[None]).reshape(-1)
    e = torch.exp(c)                                                                # relative to the largest, exp(0)
    assert float(c.min()) > -1.1
    scale = 2.0 ** (11 if kv == "e4m3" else 0)                                      # where the path places the largest
    fewer = parts_left(e * scale, low, keeps - 1) / scale / e
    best = None
    for i in fewer.argsort()[:24].tolist():                                         # left over: negative, so too large
        for j in fewer.argsort(descending=True)[:24].tolist():
            gap = abs(float((e[i] - e[j]) / (e[i] + e[j])))
            lost = float(fewer[j] - fewer[i]) / 2
            if gap < (2.0 ** -8 if kv == "bf16" else 2.0 ** -5) and (best is None or lost > best[0]):
                best = (lost, i, j)
    lost, i, j = best
    pool = pc.Pool(1, 9, 16, 1, hd, kv, seed=1)
    pool.fill([T], seed=2)
    if kv == "e4m3":
        pool.ks[:] = 1.0
        pool.vs[:] = 1.0
    for t in range(T):
        which = 0 if t == 0 else i if t % 2 else j
        k, v = torch.zeros(hd), torch.zeros(hd)
        if t > 0:
            k[0], k[1] = float(a[which // 8]), float(b[which % 8])
            v[:] = 1.0 if t % 2 else -1.0
        put(pool, "k", t, k)
        put(pool, "v", t, v)
    q = torch.zeros(1, 1, 1, hd, dtype=torch.bfloat16, device="cuda")
    q[..., :2] = 1.0
    out, st = run(pool, q, [T - 1], scale=1.0)
    assert st == mtp().MTP_OK
    w = torch.exp(pool.rows("k", 0, list(range(T)))[0, :, :2].sum(-1))
    v = pool.rows("v", 0, list(range(T)))[0]
    ref, mass = (w @ v) / w.sum(), (w @ v.abs()) / w.sum()
    z_err = 1.2 * ((2.0 ** -16 if kv == "bf16" else 2.0 ** -12) + 2 * (2 * hd + 80) * pc.U)
    tol = ((2.0 ** -16 if kv == "bf16" else 2.0 ** -9 + 2.0 ** -11) + 2 * z_err + 2 * (2 * T + 200) * pc.U) * mass
    assert lost * 128 / 129 > 1.5 * float((tol / mass).max()), "the case would not show a part fewer"
    assert ((out[0, 0, 0].double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)).all()


# ---------------------------------------------------------------------------
# values that are not finite
# ---------------------------------------------------------------------------

def same_where_not_finite(out, ref):
    out = out.double()
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    assert torch.equal(torch.isinf(out), torch.isinf(ref))
    assert torch.equal(out[torch.isinf(out)], ref[torch.isinf(ref)])


INF = float("inf")
NAN = float("nan")
PLANTED = [  # position, dimension, value: far back, in the middle of a tile, in the last one, pairs that cancel, NaN
    (5, 3, INF), (300, 4, -INF), (130, 7, INF), (520, 7, INF), (131, 9, INF), (640, 9, -INF), (200, 11, NAN), (690, 12, -INF),
    (700, 14, INF), (701, 15, INF), (702, 15, -INF), (703, 16, NAN), (0, 40, -INF)]


@pytest.mark.parametrize("spread", [1.0, 8.0])
@pytest.mark.parametrize("kv,qt,hd,G,M,window", [
    ("bf16", "bf16", 64, 2, 4, 0), ("bf16", "bf16", 128, 4, 4, 0), ("bf16", "bf16", 256, 4, 4, 0), ("bf16", "bf16", 512, 4, 4, 0),
    ("bf16", "bf16", 128, 8, 4, 0), ("bf16", "bf16", 256, 16, 4, 0), ("bf16", "bf16", 64, 16, 4, 0), ("bf16", "bf16", 512, 8, 4, 0),
    ("bf16", "bf16", 128, 4, 4, 190), ("bf16", "f32", 128, 2, 4, 0), ("f32", "f32", 64, 2, 4, 190), ("bf16", "bf16", 32, 2, 4, 0)])
def test_infinite_values_that_rows_attend(kv, qt, hd, G, M, window, spread):
    """An infinity among the attended values gives that infinity in its
    dimension, whatever its weight is, two of them of different signs or a NaN
    give NaN, and every other output stays what it is.  spread 8: the scores
    lie hundreds apart, so most weights are below what fp32 holds."""
    lens = [700]
    pool = pc.Pool(1, 45, 16, 1, hd, kv, seed=3)
    pool.fill([704], seed=4)
    for t, d, x in PLANTED:
        pool.v[int(pool.table[0, t // 16]), 0, t % 16, d % hd] = x
    q = queries(1, M, G, hd, torch.bfloat16 if qt == "bf16" else torch.float32, seed=5) * spread
    scale = None if spread == 1.0 else 4.0 / math.sqrt(hd)
    out, st = run(pool, q, lens, rope_theta=1e4, window=window, scale=scale)
    assert st == mtp().MTP_OK
    # weights of 64 bits: none is 0
    ref, mass, dots = pc.attention(pool, q, None, lens, [M], 1e4, window, 0, scale)
    same_where_not_finite(out, ref)
    tol = pc.attention_tol(ref, mass, dots, hd, 704, qt == "bf16")
    fine = torch.isfinite(ref)
    assert ((out.double() - ref).abs()[fine] <= tol[fine]).all()


@pytest.mark.parametrize("hd,G,M", [(128, 4, 3), (256, 8, 4), (64, 16, 4)])
def test_infinite_values_of_whole_items(hd, G, M):
    """Many sequences, so that most are not cut into parts."""
    B, page = 200, 16
    lens = [(37 * b) % 300 for b in range(B)]
    pool = pc.Pool(B, (max(lens) + M) // page + 1, page, 1, hd, "bf16", seed=6)
    pool.fill([n + M for n in lens], seed=7)
    for b in range(0, B, 3):
        t = (11 * b) % (lens[b] + 1)
        pool.v[int(pool.table[b, t // page]), 0, t % page, b % hd] = INF if b % 2 else -INF
    q = queries(B, M, G, hd, torch.bfloat16, seed=8)
    out, st = run(pool, q, lens, rope_theta=1e4)
    assert st == mtp().MTP_OK
    pick = list(range(0, B, 7))
    sub = pc.Pool.__new__(pc.Pool)
    sub.__dict__.update(pool.__dict__)
    sub.table = pool.table[pick]
    ref, mass, dots = pc.attention(sub, q[pick], None, [lens[b] for b in pick], [M] * len(pick), 1e4)
    same_where_not_finite(out[pick], ref)
    tol = pc.attention_tol(ref, mass, dots, hd, 310, True)
    fine = torch.isfinite(ref)
    assert ((out[pick].double() - ref).abs()[fine] <= tol[fine]).all()


@pytest.mark.parametrize("qt", ["bf16", "f32"])
@pytest.mark.parametrize("hd,G,M", [(128, 4, 6), (64, 8, 6), (256, 2, 6)])
def test_nan_codes_of_an_8_bit_cache_stay_with_the_rows_that_attend_them(hd, G, M, qt):
    lens, page = [123], 16
    for window in (0, 50):
        pool = pc.Pool(1, 10, page, 1, hd, "e4m3", seed=9)
        pool.fill([129], seed=10)
        codes = pool.v.view(torch.uint8)
        for t, d in ((126, 3), (127, 40), (128, 5), (75, 9), (72, 10), (20, 11)):
            codes[int(pool.table[0, t // page]), 0, t % page, d] = 0x7F
        pool.k.view(torch.uint8)[int(pool.table[0, 8]), 0, 0, 0] = 0xFF        # position 128: only the last row attends it
        q = queries(1, M, G, hd, torch.bfloat16 if qt == "bf16" else torch.float32, seed=11)
        out, st = run(pool, q, lens, rope_theta=1e4, window=window)
        assert st == mtp().MTP_OK
        ref, mass, dots = pc.attention(pool, q, None, lens, [M], 1e4, window)
        assert torch.isnan(out[0, 5]).all()
        same_where_not_finite(out[0, :5], ref[0, :5])
        tol = pc.attention_tol(ref, mass, dots, hd, 129, qt == "bf16")
        fine = torch.isfinite(ref)
        assert ((out.double() - ref).abs()[fine] <= tol[fine]).all()


# ---------------------------------------------------------------------------
# scores of any size
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv,qt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("e4m3", "bf16"), ("e4m3", "f32")])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_scores_of_any_size(kv, qt, sign):
    """Every score is the same number of 2^100's size, so the weights are equal
    and the output is the mean of the values."""
    hd, lens, M = 128, [400], 2
    pool = pc.Pool(1, 27, 16, 1, hd, kv, seed=12)
    pool.fill([402], seed=13)
    pages = pool.table[0].long()
    if kv == "e4m3":
        pool.k.view(torch.uint8)[pages] = torch.tensor(sign).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        pool.ks[pages] = 2.0 ** 38
        pool.vs[pages] = 2.0 ** -6
        q = torch.full((1, M, 4, hd), 2.0 ** 60, dtype=torch.bfloat16, device="cuda")
    else:
        pool.k[pages] = sign * 2.0 ** 49
        q = torch.full((1, M, 4, hd), 2.0 ** 49, dtype=torch.bfloat16, device="cuda")
    q = q if qt == "bf16" else q.float()
    out, st = run(pool, q, lens, scale=1.0)
    assert st == mtp().MTP_OK
    for j in range(M):
        v = pool.rows("v", 0, list(range(lens[0] + j + 1)))[0]
        ref, mass = v.mean(0), v.abs().mean(0)
        tol = (2 * 402 + 200) * pc.U * mass
        if qt == "bf16":
            tol = tol + 2.0 ** -8 * (ref.abs() + mass * 2.0 ** -9)
            if kv == "e4m3":
                tol = tol + 2.0 ** -9 * mass
        else:
            tol = tol + pc.U * ref.abs()
        assert ((out[0, j].double() - ref).abs() <= tol).all(), j


@pytest.mark.parametrize("kv,qt,hd", [("f32", "f32", 64), ("bf16", "f32", 128), ("bf16", "bf16", 32)])
def test_scores_of_minus_infinity_on_the_cuda_cores(kv, qt, hd):
    """A key whose score is -inf has no weight, and a row with no other scores
    gives zeros."""
    pool = pc.Pool(2, 3, 16, 1, hd, kv, seed=20)
    pool.fill([33, 20], seed=21)
    q = queries(2, 1, 2, hd, torch.bfloat16 if qt == "bf16" else torch.float32, seed=22)
    q[..., 0] = 1.0
    gone = [(0, t) for t in (0, 7, 31, 32)] + [(1, t) for t in range(20)]
    for b, t in gone:
        pool.k[int(pool.table[b, t // 16]), 0, t % 16, 0] = -INF
    out, st = run(pool, q, [32, 19])
    assert st == mtp().MTP_OK
    check(pool, out, q, None, [32, 19], [1, 1], 0.0, absent=set(gone))
    assert not out[1].any()


# ---------------------------------------------------------------------------
# page scales
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("qt", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("bad", [0.0, -0.25, 0.3, 2.0 ** -41, 2.0 ** 41, INF, NAN])
def test_a_scale_that_is_no_power_of_two_is_reported(bad, which, qt):
    """Such a page counts as absent: its positions are masked, and the status
    says so; the other pages' are not touched.  Where no row attends the page
    its scales are not looked at."""
    m = mtp()
    lens, M, page, hd = [200], 2, 16, 128
    pool = pc.Pool(1, 14, page, 2, hd, "e4m3", seed=14)
    pool.fill([202], seed=15)
    q = queries(1, M, 8, hd, torch.bfloat16 if qt == "bf16" else torch.float32, seed=16)
    good = getattr(pool, which).clone()
    getattr(pool, which)[int(pool.table[0, 3])] = bad
    out, st = run(pool, q, lens, rope_theta=1e4)
    assert st == m.MTP_ERR_ARG
    out2, st2 = run(pool, q, lens, rope_theta=1e4, window=32)
    assert st2 == m.MTP_OK
    getattr(pool, which).copy_(good)
    check(pool, out, q, None, lens, [M], 1e4, absent={(0, t) for t in range(48, 64)})
    check(pool, out2, q, None, lens, [M], 1e4, window=32)


def test_the_borders_of_a_scale():
    for s in (2.0 ** -40, 2.0 ** 40):
        pool = pc.Pool(1, 3, 16, 1, 128, "e4m3", seed=17)
        pool.fill([20], seed=18)
        pool.vs[pool.table[0].long()] = s
        pool.ks[pool.table[0].long()] = 2.0 ** -40
        for dt in (torch.bfloat16, torch.float32):
            q = queries(1, 1, 4, 128, dt, seed=19)
            out, st = run(pool, q, [19], scale=2.0 ** 30)
            assert st == mtp().MTP_OK
            check(pool, out, q, None, [19], [1], 0.0, scale=2.0 ** 30)
