"""A speculative step's calls together, as a server makes them: the target's
rows into the paged cache, the drafter's cross-attention and the target's
attention over that same cache, the verify, and the emitted tokens' log
probabilities."""
import math

import pytest
import torch

import paged_common as pc
import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mtp_speculative_decoding_gb300 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_the_drafter_reads_what_the_append_wrote():
    """Consecutive pages of a sequence are an mtp_kv_view: a cache filled by
    mtp_kv_append drafts bit for bit what the same keys and values drafted
    from a view laid out by hand."""
    import mtp_speculative_decoding_gb300 as mtp
    from mtp_speculative_decoding_gb300.device import to_device, upload_draft
    m = synth.ModelSpec(d_t=256, d_a=128, n_blocks=2, n_q_heads=4, head_dim=64, n_kv_heads=2, d_ff=256, vocab=1000, dtype="bf16",
                        block_view=(0, 0))
    B, cap, page = 3, 96, 32
    w = synth.make_draft_workload("paged", m, [synth.ViewSpec(cap=cap, window=0, rope_theta=1e4)], B, 3, [96, 40, 65], 5)
    dev = upload_draft(w)
    want = torch.empty((B, 3), dtype=torch.int32, device="cuda")
    zw = torch.empty((B, 3, m.vocab), device="cuda")
    dev.run(want, out_logits=zw)
    # the same positions through the paged cache (keys as stored: no rotation), in uneven calls
    src = [to_device(w.views[0][n]) for n in ("k", "v")]                     # [B, Hkv, cap, hd]
    table = i32([[b * (cap // page) + i for i in range(cap // page)] for b in range(B)])
    # a [page][slot][head] pool: stride_p == page * stride_t, so consecutive pages are a plain view
    kv = [torch.full((B * cap // page, page, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    c = mtp.make_kv_cache(kv[0].permute(0, 2, 1, 3), kv[1].permute(0, 2, 1, 3), table)
    ws = mtp.alloc_workspace(mtp.kv_workspace_size(c, B, 50, 4))
    done = [0] * B
    for n in ([50, 40, 1], [46, 0, 50], [0, 0, 14]):
        x = [torch.zeros(B, 50, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        for b in range(B):
            for t, s in zip(x, src):
                t[b, :n[b]] = s[b, :, done[b]:done[b] + n[b]].transpose(0, 1)
        mtp.kv_append(c, x[0], x[1], i32(done), ws, n_new=i32(n))
        assert mtp.last_error(ws) == mtp.MTP_OK
        done = [a + e for a, e in zip(done, n)]
    assert done == [96, 40, 65]
    view = [t.view(B, cap, 2, 64).permute(0, 2, 1, 3) for t in kv]
    got = torch.empty_like(want)
    zg = torch.empty_like(zw)
    mtp.draft_block(dev.cfg, dev.weights, [mtp.make_view(view[0], view[1], cap, 0, 1e4)], dev.kv_len, dev.last_tok, dev.h_prev, got,
                    dev.ws, out_logits=zg)
    torch.cuda.synchronize()
    assert mtp.last_error(dev.ws) == 0
    assert torch.equal(want, got) and torch.equal(zw, zg)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_two_windows_of_a_target_layer(kv):
    """Two verify windows in a row: append, attend, logits, verify, log
    probabilities; the second window overwrites the rejected rows.  Each
    step's outputs against the plain forms on what the step before left."""
    import mtp_speculative_decoding_gb300 as mtp
    B, N, hq, hkv, hd, V, page, theta = 4, 3, 8, 2, 128, 3001, 16, 1e4
    M = N + 1
    g = torch.Generator(device="cuda").manual_seed(1)
    pool = pc.Pool(B, 8, page, hkv, hd, kv, seed=2)
    lens = [0, 13, 40, 64]
    pool.fill(lens, seed=3)
    gain_q, gain_k = (1 + 0.1 * torch.randn(hd, device="cuda", generator=g) for _ in range(2))
    head = torch.randn(V, hq * hd, device="cuda", generator=g).to(torch.bfloat16) * 0.3
    c = pool.handle(rope_theta=theta)
    ws = mtp.alloc_workspace(max(mtp.kv_workspace_size(c, B, M, hq), mtp.workspace_size(None, B, N, V)))
    for step in range(2):
        qkv = torch.randn(B, M, (hq + 2 * hkv) * hd, device="cuda", generator=g).to(torch.bfloat16)
        q = qkv[..., :hq * hd].unflatten(-1, (hq, hd))
        k = qkv[..., hq * hd:(hq + hkv) * hd].unflatten(-1, (hkv, hd))
        v = qkv[..., (hq + hkv) * hd:].unflatten(-1, (hkv, hd))
        ln = i32(lens)
        mtp.kv_append(c, k, v, ln, ws, k_norm=gain_k)
        out = torch.empty(B, M, hq, hd, dtype=torch.bfloat16, device="cuda")
        mtp.paged_attention(c, q, ln, out, ws, q_norm=gain_q)
        assert mtp.last_error(ws) == mtp.MTP_OK
        ref, mass, dots = pc.attention(pool, q, gain_q, lens, [M] * B, theta)
        assert ((out.double() - ref).abs() <= pc.attention_tol(ref, mass, dots, hd, 80, True)).all()
        # what the cache holds: this window's keys, turned
        for b in range(B):
            pos = torch.arange(lens[b], lens[b] + M, device="cuda")
            x = pc.turn(k[b], gain_k, pos, theta).transpose(0, 1)
            step_ = 2.0 ** -4 if kv == "e4m3" else 2.0 ** -8
            d = (pool.rows("k", b, pos) - x).abs()
            floor = 2.0 ** -10 * 2.0 ** -4 if kv == "e4m3" else 0.0      # scales here are below 2^-4
            assert (d <= step_ * x.abs() * (1 + 2.0 ** -10) + floor + pc.turn_tol(x)).all()
        z = (out.view(B * M, hq * hd) @ head.T).view(B, M, V)
        drafts = z[:, :N].float().argmax(-1).to(torch.int32)
        for b in range(B):                         # reject from position b % (N + 1) on
            if b % (N + 1) < N:
                drafts[b, b % (N + 1):] = (drafts[b, b % (N + 1):] + 1) % V
        toks = torch.empty(B, M, dtype=torch.int32, device="cuda")
        acc = torch.empty(B, dtype=torch.int32, device="cuda")
        mtp.verify_greedy(z, drafts, toks, acc, ws)
        lp, ent = (torch.full((B, M), 7.0, device="cuda") for _ in range(2))
        ids = torch.full((B, M, 4), -7, dtype=torch.int32, device="cuda")
        top = torch.full((B, M, 4), 7.0, device="cuda")
        mtp.token_logprobs(z, toks, lp, ent, ids, top)
        torch.cuda.synchronize()
        assert acc.tolist() == [b % (N + 1) for b in range(B)]
        logp = torch.log_softmax(z.double(), -1)
        for b in range(B):
            for i in range(M):
                t = int(toks[b, i])
                assert (t >= 0) == (i <= int(acc[b]))
                if t < 0:
                    assert lp[b, i] == 7.0 and (ids[b, i] == -7).all()
                    continue
                assert int(ids[b, i, 0]) == t      # greedy: the emitted token is the best
                assert abs(float(lp[b, i]) - float(logp[b, i, t])) <= 1e-5 * (1 + abs(float(logp[b, i, t])))
                assert math.isclose(float(lp[b, i]), float(top[b, i, 0]), rel_tol=0, abs_tol=1e-6)
        lens = [a + int(n) + 1 for a, n in zip(lens, acc.tolist())]
