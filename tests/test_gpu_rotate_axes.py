"""mtp_rotate_axes against a plain 64-bit form: types, head sizes, sections,
strides, far and negative positions, in place."""
import pytest
import torch

import rows_common as rc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mtp_speculative_decoding_gb300 import build
    build.build()


def mtp():
    import mtp_speculative_decoding_gb300 as m
    return m


def rows(T, hq, hk, hd, dtype, seed):
    """Query and key rows as slices of a fused projection's output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, hq + 2 * hk + 1, hd, device="cuda", generator=g).to(dtype)
    return x[:, :hq], x[:, hq:hq + hk]


def check(out, x, gain, pos, sections, theta, inter):
    ref, tol = rc.rotate(x, gain, pos, sections, theta, inter)
    step = 2.0 ** -8 if out.dtype == torch.bfloat16 else rc.U
    err = (out.double() - ref).abs()
    # 16-bit rows take the sine and cosine instructions: 2^-20 of the pair's magnitude more
    bound = tol * (1.5 if out.dtype == torch.bfloat16 else 1.0) + step * (ref.abs() + 2 * tol)
    assert (err <= bound).all(), float((err / bound.clamp(min=1e-30)).max())


CASES = [
    # T, hq, hk, hd, sections, interleaved, dtype, norm, theta
    (1, 1, 1, 128, (24, 20, 20), False, "bf16", True, 1e6),
    (4, 16, 4, 256, (44, 42, 42), True, "bf16", True, 1e6),
    (77, 7, 1, 128, (16, 24, 24), False, "bf16", False, 1e4),
    (1023, 8, 2, 64, (8, 12, 12), True, "bf16", True, 1e7),
    (33, 3, 3, 32, (8, 4, 4), True, "f32", True, 1e4),
    (500, 4, 2, 256, (11, 11, 10), True, "f32", True, 1e7),       # a quarter of the head
    (129, 5, 2, 512, (100, 78, 78), False, "f32", False, 1e4),
    (65, 2, 2, 512, (24,), False, "bf16", True, 1e4),             # one axis, partial
    (50, 6, 3, 128, (2, 3, 1, 2), True, "bf16", False, 1e4),      # four axes, 8 pairs
    (50, 6, 3, 128, (0, 0, 64), False, "f32", False, 1e4),        # empty sections
    (50, 6, 3, 128, (1, 62, 1), True, "f32", False, 1e4),         # a section beyond its turns
    (3001, 16, 8, 128, (16, 24, 24), False, "bf16", True, 1e6),
]


@pytest.mark.parametrize("T,hq,hk,hd,sections,inter,dtype,norm,theta", CASES)
@pytest.mark.parametrize("inplace", [False, True])
def test_rows_turn(T, hq, hk, hd, sections, inter, dtype, norm, theta, inplace):
    m = mtp()
    q, k = rows(T, hq, hk, hd, torch.bfloat16 if dtype == "bf16" else torch.float32, 1)
    x = (q.clone(), k.clone())
    g = torch.Generator(device="cuda").manual_seed(2)
    gains = [1 + 0.1 * torch.randn(hd, device="cuda", generator=g) if norm else None for _ in range(2)]
    pos = torch.randint(-3000, 130000, (len(sections), T), device="cuda", generator=g, dtype=torch.int32)
    oq, ok = (q, k) if inplace else (torch.full_like(x[0], 7.0), torch.full_like(x[1], 7.0))
    m.rotate_axes(q, k, pos, sections, theta, oq, ok, interleaved=inter, q_norm=gains[0], k_norm=gains[1])
    check(oq, x[0], gains[0], pos, sections, theta, inter)
    check(ok, x[1], gains[1], pos, sections, theta, inter)
    if not inplace:
        assert torch.equal(q, x[0]) and torch.equal(k, x[1])


def test_what_lies_between_the_rows_keeps_its_bytes():
    m = mtp()
    x = torch.randn(40, 9, 128, device="cuda").to(torch.bfloat16)
    before = x.clone()
    pos = torch.arange(40, device="cuda", dtype=torch.int32).expand(3, 40).contiguous()
    m.rotate_axes(x[3:20, 1:5], x[3:20, 6:8], pos[:, 3:20].contiguous(), (24, 20, 20), 1e4, x[3:20, 1:5], x[3:20, 6:8])
    same = torch.ones(40, 9, dtype=torch.bool)
    same[3:20, 1:5] = same[3:20, 6:8] = False
    assert torch.equal(x[same], before[same])
    check(x[3:20, 1:5], before[3:20, 1:5], None, pos[:, 3:20], (24, 20, 20), 1e4, False)


def test_queries_alone_and_heads_of_stride_zero():
    m = mtp()
    q = torch.randn(21, 1, 64, device="cuda").expand(21, 5, 64)       # one row for every head
    pos = torch.randint(0, 900, (2, 21), device="cuda", dtype=torch.int32)
    out = torch.empty(5, 21, 64, device="cuda").transpose(0, 1)        # heads outermost
    m.rotate_axes(q, None, pos, (16, 16), 1e4, out)
    check(out, q, None, pos, (16, 16), 1e4, False)


def test_equal_positions_are_one_position():
    """Text: all axes at one position turn as a single axis does, bit for bit."""
    m = mtp()
    q, k = rows(60, 4, 2, 128, torch.bfloat16, 5)
    pos = torch.randint(0, 70000, (1, 60), device="cuda", dtype=torch.int32)
    one, many = (tuple(torch.empty_like(x) for x in (q, k)) for _ in range(2))
    m.rotate_axes(q, k, pos, (64,), 1e6, *one)
    m.rotate_axes(q, k, pos.expand(3, 60).contiguous(), (24, 20, 20), 1e6, *many, interleaved=True)
    assert all(torch.equal(a, b) for a, b in zip(one, many))


def test_the_farthest_positions():
    m = mtp()
    q = torch.randn(4, 2, 64, device="cuda")
    pos = torch.tensor([[2**31 - 1, -2**31, 2**30 + 12345, 0]] * 2, device="cuda", dtype=torch.int32)
    out = torch.empty_like(q)
    m.rotate_axes(q, None, pos, (16, 16), 1e4, out)
    # an angle keeps 2^-45 of its size: 2^31 radians are off by 2^-14
    ref, tol = rc.rotate(q, None, pos, (16, 16), 1e4, False)
    assert ((out.double() - ref).abs() <= tol + 2.0 ** -13 * q.abs().amax()).all()


def test_values_that_are_not_finite_stay_in_their_row():
    m = mtp()
    q = torch.randn(6, 4, 128, device="cuda").to(torch.bfloat16)
    q[2, 1, 5], q[4, 3, 100] = float("nan"), float("inf")
    pos = torch.arange(6, device="cuda", dtype=torch.int32).expand(3, 6).contiguous()
    out = torch.empty_like(q)
    m.rotate_axes(q, None, pos, (24, 20, 20), 1e4, out, q_norm=torch.ones(128, device="cuda"))
    bad = (~out.isfinite()).any(-1)
    want = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    want[2, 1] = want[4, 3] = True
    assert torch.equal(bad, want)


def test_captured_and_on_another_stream():
    m = mtp()
    q, k = rows(300, 8, 2, 128, torch.bfloat16, 7)
    pos = torch.randint(0, 9000, (3, 300), device="cuda", dtype=torch.int32)
    want = (torch.empty_like(q), torch.empty_like(k))
    m.rotate_axes(q, k, pos, (24, 20, 20), 1e6, *want)
    got = (torch.zeros_like(q), torch.zeros_like(k))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    m.rotate_axes(q, k, pos, (24, 20, 20), 1e6, *got, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.rotate_axes(q, k, pos, (24, 20, 20), 1e6, *got)
    pos.add_(17)
    m.rotate_axes(q, k, pos, (24, 20, 20), 1e6, *want)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
