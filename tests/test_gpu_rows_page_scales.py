"""Value scales of an e4m3 cache's pages far apart: what is rounded is a
probability times its page's value scale, to fp16 around the row's largest."""
import pytest
import torch

import paged_common as pc
import scores_common as sc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mtp_speculative_decoding_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# value scale of page class 0, 1, 2 (log2) and their scores: weights that differ by
# the scales alone (20 and 40 bits below the largest), by 24, 26, 33 bits, and scales
# that the probabilities make up for
SPREADS = [((10, -10, -30), (0.0, 0.0, 0.0)), ((20, -4, -6), (0.0, 0.0, 0.0)), ((33, 0, -4), (0.0, 0.0, 0.0)),
           ((10, -10, -30), (-13.875, 0.0, 0.0)), ((40, 0, -40), (-28.0, 0.0, 28.0)), ((0, 0, 0), (0.0, -17.375, -24.25)), ((-40, 40, 0), (0.0, 0.0, 0.0))]


@pytest.mark.parametrize("scales,tops", SPREADS)
@pytest.mark.parametrize("hd", [64, 128, 256, 512])
@pytest.mark.parametrize("qt", ["bf16", "f32"])
def test_page_scales_far_apart(qt, hd, scales, tops):
    """A weight w = p * scale is off by 2^-11 of itself, or by 2^-36 of the row's
    largest where that is more (half a step of fp16's smallest numbers, the
    largest weight being 2^11 to 2^15).  fp32 queries and head dimension 512 lose
    nothing of it."""
    import mtp_speculative_decoding_gb300 as m
    n, before, page = 200, 250, 16
    T = before + n
    g = torch.Generator().manual_seed(1)
    pool = pc.Pool(1, T // page + 2, page, 1, hd, "e4m3", seed=2)
    pool.fill([T], seed=3)
    t = torch.arange(T)
    cls = (t // page) % 3
    z = torch.tensor(tops, dtype=torch.float64)[cls] + torch.randint(-8, 1, (T,), generator=g) / 8
    pages = pool.table[0].long()[: -(-T // page)]
    pool.ks[pages] = 1.0
    pool.vs[pages] = torch.exp2(torch.tensor(scales, dtype=torch.float32))[torch.arange(pages.numel()) % 3].cuda()[:, None]
    pg, slot = pages[t.cuda() // page], t.cuda() % page
    pool.k.view(torch.uint8)[pg, 0, slot] = sc.keys(z, hd).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    # dimensions to themselves: the first half to class 0, a quarter each to 1 and 2
    code = pool.v.view(torch.uint8)[pg, 0, slot].clone()
    dim = torch.arange(hd, device="cuda")
    own = torch.where(dim < hd // 2, 0, torch.where(dim < 3 * hd // 4, 1, 2))
    code[cls.cuda()[:, None] != own] = 0
    pool.v.view(torch.uint8)[pg, 0, slot] = code
    q = sc.rows((n,), hd, g, "cuda").to(torch.bfloat16 if qt == "bf16" else torch.float32)
    h = pool.handle()
    ws = m.alloc_workspace(m.prompt_workspace_size(h, 1, n, 4))
    out = torch.full_like(q, 7.0)
    m.prompt_attention(h, q, i32([0, n]), i32([before]), out, ws, attn_scale=1.0)
    assert m.last_error(ws) == m.MTP_OK
    see = t.cuda() <= torch.arange(before, T, device="cuda")[:, None]
    v = pool.rows("v", 0, t)[0]
    codes = code.view(torch.float8_e4m3fn).double().abs()
    vs = pool.vs[pg, 0].double()
    low = qt == "bf16" and hd < 512
    for k, f in enumerate(sc.FACTORS):
        p = torch.softmax((z.cuda() * f).expand(n, T).masked_fill(~see, -torch.inf), -1)
        w = p * vs
        ref = p @ v
        off = torch.maximum(2.0 ** -11 * w, 2.0 ** -36 * w.amax(-1, keepdim=True)) * see if low else torch.zeros_like(w)
        rel = 2 * 8 * sc.U * (float(z.abs().max()) * f + 64) + (2 * T + 200) * sc.U
        tol = off @ codes + rel * (p @ v.abs())
        # fp32: a weight never falls below 2^-149 of the row's largest (an infinite value keeps its
        # sign), neither where a position is added nor where the sum so far is scaled down.  Scores
        # rise by more than 149 bits once at most (they span 2 * 56 nats, 162 bits), and a lane
        # group's sum meets the others five times: with the position itself 7 * 2^-149 of |v| at most
        if not low:
            tol = tol + 2.0 ** -146 * (see.double() @ v.abs())
        tol = tol + (2.0 ** -8 if qt == "bf16" else sc.U) * (ref.abs() + tol)
        err = (out[:, k].double() - ref).abs()
        assert (err <= tol).all(), (k, float((err / tol.clamp(min=1e-300)).max()))
        # what lies within 2^-25 of the row's largest weight keeps its bits: seen in the dimensions of its own
        for c in range(3):
            mine = (cls.cuda() == c)[None] & see
            held = (torch.where(mine, w, torch.inf).amin(-1) >= 2.0 ** -25 * w.amax(-1)) if low else torch.ones(n, dtype=torch.bool, device="cuda")
            d = own == c
            strict = (2.0 ** -11 + rel if low else rel) * (p @ v.abs()) + (0.0 if low else 2.0 ** -146) * (see.double() @ v.abs())
            strict = strict + (2.0 ** -8 if qt == "bf16" else sc.U) * (ref.abs() + strict)
            assert (err <= strict)[held][:, d].all(), (k, c)
