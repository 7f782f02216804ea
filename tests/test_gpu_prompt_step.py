"""A prompt's calls together, as a server makes them: rows rotated by several
positions, appended to the paged cache as they are, attended as packed prompts;
then verify windows of sequences that share the first prompt's pages."""
import pytest
import torch

import paged_common as pc
import rows_common as rc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mtp_speculative_decoding_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Layer:
    """One attention layer of the target over a paged cache."""

    def __init__(self, kv, hd, hkv, G, page, B, pages, seed):
        import mtp_speculative_decoding_gb300 as mtp
        self.m, self.hd, self.hkv, self.hq, self.B = mtp, hd, hkv, hkv * G, B
        self.pool = pc.Pool(B, pages, page, hkv, hd, kv, seed=seed)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.gains = [1 + 0.1 * torch.randn(hd, device="cuda", generator=self.g) for _ in "qk"]
        self.sections = (hd // 4, hd // 8, hd // 8)

    def rows(self, T):
        """A fused projection's output: its queries, keys and values [T, heads, head_dim]."""
        x = torch.randn(T, self.hq + 2 * self.hkv, self.hd, device="cuda", generator=self.g).to(torch.bfloat16)
        return x, x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]

    def turn(self, q, k, pos):
        """In place; against the formula."""
        want = [rc.rotate(x, gain, pos, self.sections, 1e6, True) for x, gain in zip((q, k), self.gains)]
        self.m.rotate_axes(q, k, pos, self.sections, 1e6, q, k, interleaved=True, q_norm=self.gains[0], k_norm=self.gains[1])
        for x, (ref, bound) in zip((q, k), want):
            assert ((x.double() - ref).abs() <= bound + 2.0 ** -8 * (ref.abs() + bound)).all()

    def held(self, b, pos, k, v):
        """What the cache holds at the positions pos of sequence b: these rows, rounded once."""
        for w, x in (("k", k), ("v", v)):
            x = x.double().transpose(0, 1)
            d = (self.pool.rows(w, b, pos) - x).abs()
            # (e4m3: a page's scale is at most twice its largest value / 448, and no value here reaches 8;
            # below a normal code a value is off by 2^-10 scales)
            step, floor = (0.0, 0.0) if self.pool.dtype == "bf16" else (2.0 ** -4, 2.0 ** -10 * 2 * 8 / 448)
            assert x.abs().max() < 8 and (d <= step * x.abs() + floor).all()


@pytest.mark.parametrize("kv,hd,G,P", [("bf16", 256, 4, 192), ("bf16", 128, 2, 208), ("e4m3", 256, 4, 192), ("e4m3", 64, 7, 64)])
def test_a_shared_prompt_and_what_follows(kv, hd, G, P):
    B, page, M = 4, 16, 3
    a = Layer(kv, hd, 2, G, page, B, P // page + 8, seed=31)
    m, pool = a.m, a.pool
    one = m.make_kv_cache(pool.k, pool.v, pool.table[:1], pool.ks, pool.vs)
    ws = m.alloc_workspace(max(m.kv_workspace_size(one, B, P, a.hq), m.prompt_workspace_size(one, B, 2 * P, a.hq),
                               m.prefix_workspace_size(one, B, M, a.hq)))
    # the shared prompt: text, then a picture of 8 columns
    t = torch.arange(P, device="cuda")
    pos = torch.stack([t.clamp(max=40), torch.where(t > 40, 40 + (t - 40) // 8, t), torch.where(t > 40, 40 + (t - 40) % 8, t)]).to(torch.int32)
    x, q, k, v = a.rows(P)
    a.turn(q, k, pos)
    m.kv_append(one, k[None], v[None], i32([0]), ws)
    out = torch.full((P, a.hq, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    m.prompt_attention(one, q, i32([0, P]), i32([0]), out, ws)
    assert m.last_error(ws) == 0
    a.held(0, range(P), k, v)
    rc.check(out, *rc.attend(pool, 0, q, None, 0, 0.0), P, kv)
    # sequences behind it, their prompts packed
    pool.table[1:, : P // page] = pool.table[:1, : P // page]
    cache = pool.handle()
    n = [0, 40, 1, 57]
    at = [0, 0, 40, 41, 98]
    x, q, k, v = a.rows(at[-1])
    text = torch.cat([torch.arange(c) for c in n]).cuda() + 70
    a.turn(q, k, text.to(torch.int32).expand(3, -1).contiguous())
    pads = [torch.zeros(B, max(n), 2, hd, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    for b in range(B):
        for p, y in zip(pads, (k, v)):
            p[b, :n[b]] = y[at[b]:at[b + 1]]
    m.kv_append(cache, *pads, i32([P] * B), ws, n_new=i32(n))
    out = torch.full((at[-1], a.hq, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    m.prompt_attention(cache, q, i32(at), i32([P] * B), out, ws)
    assert m.last_error(ws) == 0
    for b in range(B):
        if n[b]:
            r = slice(at[b], at[b + 1])
            a.held(b, range(P, P + n[b]), k[r], v[r])
            rc.check(out[r], *rc.attend(pool, b, q[r], None, P, 0.0), P + n[b], kv)
    # two verify windows; the calls of one captured, replayed on the next one's inputs
    lens = [P + c for c in n]
    ln, group, pre = i32(lens), i32([0, B]), i32([P])
    fused = a.rows(B * M)[0]
    q, k, v = (fused[:, i:j].unflatten(0, (B, M)) for i, j in ((0, a.hq), (a.hq, a.hq + 2), (a.hq + 2, a.hq + 4)))
    pos = torch.zeros(3, B * M, dtype=torch.int32, device="cuda")
    out = torch.empty(B, M, a.hq, hd, dtype=torch.bfloat16, device="cuda")
    other = torch.empty_like(out)

    def step():
        m.rotate_axes(fused[:, :a.hq], fused[:, a.hq:a.hq + 2], pos, a.sections, 1e6, fused[:, :a.hq], fused[:, a.hq:a.hq + 2],
                      interleaved=True, q_norm=a.gains[0], k_norm=a.gains[1])
        m.kv_append(cache, k, v, ln, ws)
        m.prefix_attention(cache, q, ln, group, pre, out, ws)
        m.paged_attention(cache, q, ln, other, ws)

    graph = None
    for turn in range(3):
        fused.copy_(a.rows(B * M)[0])
        pos.copy_((ln[:, None] + torch.arange(M, device="cuda")).flatten().expand(3, -1))
        want = rc.rotate(fused[:, :a.hq], a.gains[0], pos, a.sections, 1e6, True)
        if turn == 0:
            step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        assert m.last_error(ws) == 0
        assert ((fused[:, :a.hq].double() - want[0]).abs() <= want[1] + 2.0 ** -8 * (want[0].abs() + want[1])).all()
        for b in range(B):
            end = int(ln[b]) + M
            a.held(b, range(end - M, end), k[b], v[b])
            ref = rc.attend(pool, b, q[b], None, int(ln[b]), 0.0)
            rc.check(out[b], *ref, end, kv)
            assert ((other[b].double() - ref[0]).abs() <= pc.attention_tol(*ref, hd, end, True)).all()
        ln += i32([1, 3, 2, 0])
