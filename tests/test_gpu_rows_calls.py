"""Calls of the attention of prompts and of shared prefixes beside one another:
from two host threads on two streams, as two captured graphs with one workspace,
and many rows that are computed again."""
import ctypes as C

import pytest
import torch

import paged_common as pc
import rows_common as rc
from test_gpu_paged_threads import together

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mtp_speculative_decoding_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Prefix:
    """B sequences of M rows behind one prefix of P positions."""

    def __init__(self, B, M, P, hd, kv, seed, spare=0):
        import mtp_speculative_decoding_gb300 as m
        self.m, self.M, self.P, self.lens = m, M, P, [P + b % 3 for b in range(B)]
        self.pool = pc.Pool(B, (P + 3 + M) // 16 + 2, 16, 1, hd, kv, seed=seed)
        self.pool.table[:, : P // 16] = self.pool.table[:1, : P // 16].clone()
        self.pool.fill([n + M for n in self.lens], seed=seed + 1)
        self.h = self.pool.handle(rope_theta=1e4)
        self.q = torch.randn(B, M, 2, hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(torch.bfloat16)
        self.out = torch.full_like(self.q, 7.0)
        self.at = i32(self.lens), i32([0, B]), i32([P])
        self.size = m.prefix_workspace_size(self.h, B, M, 2)
        self.ws = m.alloc_workspace(self.size + spare)

    def raw(self, stream):
        q = self.q
        args = (C.byref(self.h), q.shape[0], self.M, 2, self.at[0].data_ptr(), None, 1, self.at[1].data_ptr(), self.at[2].data_ptr(),
                q.data_ptr(), self.m.MTP_DTYPE_BF16, q.stride(0), q.stride(1), q.stride(2), None, 1e-6, 0.0, self.out.data_ptr(),
                self.ws.data_ptr(), self.ws.numel(), stream.cuda_stream)
        return lambda: self.m.lib().mtp_prefix_attention(*args)

    def call(self):
        self.m.prefix_attention(self.h, self.q, *self.at, self.out, self.ws)

    def check(self):
        assert self.m.last_error(self.ws) == 0
        for b in range(0, len(self.lens), max(1, len(self.lens) // 5)):
            ref = rc.attend(self.pool, b, self.q[b], None, self.lens[b], 1e4, prefix=self.P, first=0)
            rc.check(self.out[b], *ref, self.lens[b] + self.M, self.pool.dtype)


class Prompt:
    """Prompts of n rows each behind the cached positions lens."""

    def __init__(self, n, lens, hd, kv, seed):
        import mtp_speculative_decoding_gb300 as m
        self.m, self.n, self.lens = m, n, lens
        ends = [a + c for a, c in zip(lens, n)]
        self.pool = pc.Pool(len(n), max(ends) // 32 + 1, 32, 1, hd, kv, seed=seed)
        self.pool.fill(ends, seed=seed + 1)
        self.h = self.pool.handle(rope_theta=1e4)
        self.at = [0]
        for c in n:
            self.at.append(self.at[-1] + c)
        self.q = torch.randn(self.at[-1], 2, hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(torch.bfloat16)
        self.out = torch.full_like(self.q, 7.0)
        self.dev = i32(self.at), i32(lens)
        self.size = m.prompt_workspace_size(self.h, len(n), self.at[-1], 2)
        self.ws = m.alloc_workspace(self.size)

    def raw(self, stream):
        q = self.q
        args = (C.byref(self.h), len(self.n), q.shape[0], 2, self.dev[1].data_ptr(), self.dev[0].data_ptr(), q.data_ptr(),
                self.m.MTP_DTYPE_BF16, q.stride(0), q.stride(1), None, 1e-6, 0.0, self.out.data_ptr(), self.ws.data_ptr(),
                self.ws.numel(), stream.cuda_stream)
        return lambda: self.m.lib().mtp_prompt_attention(*args)

    def call(self):
        self.m.prompt_attention(self.h, self.q, *self.dev, self.out, self.ws)

    def check(self):
        assert self.m.last_error(self.ws) == 0
        for b, c in enumerate(self.n):
            r = slice(self.at[b], self.at[b + 1])
            if c:
                rc.check(self.out[r], *rc.attend(self.pool, b, self.q[r], None, self.lens[b], 1e4), self.lens[b] + c, self.pool.dtype)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_two_host_threads(kv):
    """A large and a small batch: their kernels ask for different amounts of shared memory."""
    large, small, prompt = Prefix(1000, 1, 64, 64, kv, 1), Prefix(3, 2, 200, 256, kv, 2), Prompt([300, 1, 77], [0, 500, 3], 128, kv, 3)
    calls = [x.raw(torch.cuda.Stream()) for x in (large, small, prompt)]
    torch.cuda.synchronize()
    assert together(calls, 300) == [0, 0, 0]
    for x in (large, small, prompt):
        x.check()


def test_two_captured_graphs_with_one_workspace():
    a, b = Prefix(6, 3, 300, 256, "bf16", 4), Prompt([400, 9], [0, 130], 256, "bf16", 5)
    a.ws = b.ws = a.ws if a.size >= b.size else b.ws
    graphs = []
    for x in (a, b):
        x.call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.call()
        graphs.append(g)
    want = [x.out.clone() for x in (a, b)]
    for turn in range(4):
        for x in (a, b):
            x.out.fill_(7.0)
        for g in (graphs if turn % 2 else graphs[::-1]):
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x.out, w) for x, w in zip((a, b), want))
    a.check()
    b.check()


def test_a_workspace_for_more_holds_fewer():
    big = Prefix(40, 4, 100, 128, "bf16", 6)
    x = Prefix(7, 1, 130, 128, "bf16", 7)
    x.ws = big.ws
    for y in (big, x, big):
        y.call()
        y.check()


@pytest.mark.parametrize("kv,hd", [("bf16", 256), ("e4m3", 128)])
def test_every_row_computed_again(kv, hd):
    """A value that is infinite at position 0: every row is computed anew, and the others' dimensions keep their values."""
    x = Prompt([700, 50], [0, 0], hd, kv, 8)
    if kv == "e4m3":
        x.pool.v.view(torch.uint8)[int(x.pool.table[0, 0]), 0, 0, 5] = 0x7F       # NaN
    else:
        x.pool.v[int(x.pool.table[0, 0]), 0, 0, 5] = float("inf")
    x.call()
    assert x.m.last_error(x.ws) == 0
    odd = x.out[:700, :, 5]
    assert (odd.isnan() if kv == "e4m3" else odd == float("inf")).all()
    ref, mass, dots = rc.attend(x.pool, 0, x.q[:700], None, 0, 1e4)
    keep = [i for i in range(hd) if i != 5]
    rc.check(x.out[:700][..., keep], ref[..., keep], mass[..., keep], dots, 700, "f32")
    ref = rc.attend(x.pool, 1, x.q[700:], None, 0, 1e4)
    rc.check(x.out[700:], *ref, 50, kv)


@pytest.mark.parametrize("kv", ["bf16", "f32"])
def test_groups_that_overlap_are_reported(kv):
    """Bounds that go up and down again: many groups of all sequences, more items than a plan holds."""
    x = Prefix(12, 16, 90, 128, kv, 9)
    start = i32([0, 12] * 6 + [0])
    x.m.prefix_attention(x.h, x.q, x.at[0], start, i32([90] * 12), x.out, x.ws)
    assert x.m.last_error(x.ws) == x.m.MTP_ERR_ARG
    if kv == "bf16":
        assert (x.out == 7.0).all()
    x.call()
    x.check()
