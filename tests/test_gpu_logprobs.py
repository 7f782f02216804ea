"""mtp_token_logprobs against a plain 64-bit form: types, sizes, alignments,
masked and degenerate rows, ties, and skipped rows."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mtp_speculative_decoding_gb300 import build
    build.build()


def run(z, tokens, K, outputs="lept"):
    import mtp_speculative_decoding_gb300 as m
    lead = z.shape[:-1]
    lp = torch.full(lead, 7.0, device="cuda")
    ent = torch.full(lead, 7.0, device="cuda")
    ids = torch.full((*lead, K), -7, dtype=torch.int32, device="cuda") if K else None
    top = torch.full((*lead, K), 7.0, device="cuda") if K else None
    m.token_logprobs(z, tokens, lp if "l" in outputs else None, ent if "e" in outputs else None,
                     ids if "t" in outputs else None, top if "p" in outputs else None)
    torch.cuda.synchronize()
    return lp, ent, ids, top


def check(z, tokens, K, got):
    """The sum of V exponentials: each is off by 2^-22 (the instruction) and
    the rounding of its exponent, |d| 2^-23 (weighted by p: at most the
    entropy-like mean of |d|); a thread adds at most V / 512 + 32 of them and
    30 sums join threads, warps and pieces, 2^-24 each.  The logarithm is off
    by that relative error; z - max and the last difference round once."""
    lp, ent, ids, top = (None if t is None else t.reshape(-1, *(t.shape[z.dim() - 1:])) for t in got)
    z = z.reshape(-1, z.shape[-1])
    tokens = tokens.reshape(-1).tolist() if tokens is not None else [None] * z.shape[0]
    V = z.shape[1]
    for r, t in enumerate(tokens):
        if t is not None and not 0 <= t < V:
            assert lp[r] == 7.0 and ent[r] == 7.0
            assert K == 0 or ((ids[r] == -7).all() and (top[r] == 7.0).all())
            continue
        x = z[r].double()
        x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
        m = x.max()
        p = torch.softmax(x, 0)
        d = torch.where(p > 0, x - m, torch.zeros_like(x))
        ls = torch.exp(x - m).sum().log()
        ad = float((p * d.abs()).sum())
        eps = (V / 512 + 64) * 2.0 ** -24 + 2.0 ** -22 + ad * 2.0 ** -22
        if t is not None:
            want = float(x[t] - m - ls)
            if math.isinf(want):
                assert float(lp[r]) == want
            else:
                assert abs(float(lp[r]) - want) <= eps + 2.0 ** -22 * abs(want)
        H = float(ls - (p * d).sum())
        assert abs(float(ent[r]) - H) <= eps * (2 + ad) + 2.0 ** -22 * (ad + float(ls))
        if K:
            real = min(K, int((x > -math.inf).sum()))
            order = torch.sort(x, descending=True, stable=True)[1][:real]
            assert ids[r, :real].tolist() == order.tolist()
            assert (ids[r, real:] == -1).all() and (top[r, real:] == -math.inf).all()
            want = x[order] - m - ls
            assert ((top[r, :real].double() - want).abs() <= eps + 2.0 ** -22 * want.abs()).all()


def logits(rows, V, dtype, seed, std=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, V, device="cuda", generator=g) * std).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,K", [(1, 1, 1), (3, 2, 5), (2, 31, 32), (5, 1000, 8), (4, 4097, 17), (2, 16385, 20), (4, 262144, 5),
                                      (33, 50257, 32), (700, 9001, 16), (1, 248320, 0), (12, 131071, 1)])
def test_rows_of_all_sizes(dtype, rows, V, K):
    z = logits(rows, V, dtype, seed=rows + V)
    tok = torch.randint(0, V, (rows,), device="cuda", dtype=torch.int32)
    tok[rows // 2] = z[rows // 2].argmax()
    check(z, tok, K, run(z, tok, K))


def test_a_verify_windows_rows():
    """[B, 1+N, V] logits with a verify's -1 padded tokens, and ids outside the vocabulary."""
    z = logits(12, 5003, torch.bfloat16, seed=1).view(4, 3, 5003)
    tok = torch.tensor([[5, 17, 2], [4, -1, -1], [5002, 0, -1], [5003, 9, 1 << 30]], dtype=torch.int32, device="cuda")
    check(z, tok, 6, run(z, tok, 6))


def test_rows_at_a_stride_and_odd_starts():
    buf = logits(9, 4000, torch.bfloat16, seed=2)
    for lo, V in ((1, 3001), (7, 3993), (8, 17), (3, 1)):
        z = buf[:, lo:lo + V]
        tok = torch.randint(0, V, (9,), device="cuda", dtype=torch.int32)
        check(z, tok, 4, run(z, tok, 4))
    f = logits(5, 999, torch.float32, seed=3)[:, 2:]
    tok = torch.zeros(5, dtype=torch.int32, device="cuda")
    check(f, tok, 3, run(f, tok, 3))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [70, 5000, 262144])
def test_masked_and_tied_rows(dtype, V):
    low = torch.finfo(dtype).min
    z = logits(12, V, dtype, seed=4)
    z[0] = 0.0                                    # all tied: the lowest ids
    z[1] = low                                    # all at the type's lowest: uniform
    z[2] = -math.inf
    z[2, V - 3:] = torch.tensor([1.0, 1.0, -2.0], dtype=dtype)     # three tokens allowed
    z[3] = low
    z[3, V // 2] = 3.0                            # one allowed, the others at the lowest
    z[4, ::2] = float("nan")
    z[5] = torch.arange(V, device="cuda").float().mul(200.0 / V).to(dtype)        # ascending
    z[6] = -torch.arange(V, device="cuda").float().mul(200.0 / V).to(dtype)       # descending
    z[7] = torch.where(torch.arange(V, device="cuda") % 2 == 0, low, -math.inf).to(dtype)
    z[8, :] = torch.where(torch.rand(V, device="cuda") < 0.5, 1.0, 2.0).to(dtype)  # two values, long ties
    z[9] = float("nan")
    z[9, 5] = -4.0
    z[10, 7] = 60000.0                            # one logit far above all others
    z[11] = torch.where(torch.arange(V, device="cuda") < V - 40, low, 1e30).to(dtype)
    tok = torch.tensor([3, 5, V - 2, V // 2, 0, V - 1, 0, 2, 1, 5, 7, V - 1], dtype=torch.int32, device="cuda")
    for K in (0, 1, 20, 32):
        check(z, tok, K, run(z, tok, K))


def test_rows_without_a_distribution_are_nan():
    z = logits(4, 3000, torch.float32, seed=5)
    z[0] = -math.inf
    z[1] = float("nan")
    z[2, 100] = math.inf
    lp, ent, ids, top = run(z, torch.tensor([1, 2, 100, 3], dtype=torch.int32, device="cuda"), 3)
    assert torch.isnan(lp[:3]).all() and torch.isnan(ent[:3]).all() and torch.isfinite(lp[3])
    assert (ids[:2] == -1).all() and (top[:2] == -math.inf).all()
    assert ids[2, 0] == 100 and torch.isnan(top[2]).all()


def test_optional_outputs_and_no_tokens():
    z = logits(6, 20000, torch.bfloat16, seed=6)
    full = run(z, None, 7)
    assert (full[0] == 7.0).all()                 # no tokens: no log probability
    for outs in ("e", "t", "p", "l"):
        got = run(z, torch.zeros(6, dtype=torch.int32, device="cuda"), 7, outs)
        for name, x, y in zip("letp", got, full):
            if name != "l":
                assert torch.equal(x, y) if name in outs else ((x == 7.0).all() or (x == -7).all())


def test_same_bits_again_captured_and_on_another_stream():
    import mtp_speculative_decoding_gb300 as m
    z = logits(40, 100003, torch.bfloat16, seed=7)
    tok = torch.randint(0, 100003, (40,), device="cuda", dtype=torch.int32)
    a = run(z, tok, 20)
    outs = [torch.zeros_like(t) for t in a]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        m.token_logprobs(z, tok, *outs)
    with torch.cuda.stream(s):
        g.replay()
        g.replay()
    s.synchronize()
    for x, y in zip(a, outs):
        assert torch.equal(x, y)


def test_more_than_32_bits_of_logits():
    z = torch.zeros(17000, 131072, dtype=torch.bfloat16, device="cuda")      # 2.2e9 elements
    z[16999, 131071] = 5.0
    tok = torch.full((17000,), -1, dtype=torch.int32, device="cuda")
    tok[16999] = 131071
    tok[16000] = 9
    lp, ent, ids, _ = run(z, tok, 2)
    assert abs(float(lp[16999]) - (5 - math.log(131071 + math.exp(5)))) < 1e-4
    assert abs(float(lp[16000]) + math.log(131072)) < 1e-4 and ids[16999].tolist() == [131071, 0] and ids[16000].tolist() == [0, 1]
    assert lp[0] == 7.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,K", [(2154, 32), (600, 32), (4099, 20), (1100, 1), (517, 8)])
def test_rows_that_few_warps_hold(dtype, V, K):
    z = logits(37, V, dtype, 61)
    tok = torch.arange(37, dtype=torch.int32, device="cuda") * 13
    check(z, tok, K, run(z, tok, K))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("at,n", [(0, 1000), (70001, 1000), (131000, 200), (5, 31), (199000, 1000)])
def test_an_allowed_set_that_lies_together(dtype, at, n):
    """Everything masked but one run of logits: a few warps hold all candidates."""
    z = logits(5, 200000, dtype, 62)
    keep = torch.zeros(200000, dtype=torch.bool, device="cuda")
    keep[at:at + n] = True
    z = z.masked_fill(~keep, -math.inf)
    tok = torch.full((5,), at, dtype=torch.int32, device="cuda")
    check(z, tok, 32, run(z, tok, 32))
