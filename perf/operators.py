"""The cases by which the target's side of a speculative step is measured.

Three operators stand around the draft and verify calls of this library:

  append     the target's new key and value rows go into its paged KV cache,
             keys normed and rotated on the way, in bf16 or in 8 bits (e4m3)
             with one power-of-two scale per page and KV head;
  attention  the 1 + N rows of a verify step (or the single row of plain
             decoding) attend the paged cache;
  logprobs   log probability, entropy and top alternatives of the emitted
             tokens, from the target's logits.

`run` computes them in plain torch operations, or, with `own`, through the
library's entry points.  `exact` says from the definitions, in 64 bits, what
comes out.
"""
import math

import torch

own = False

# the 16 query heads x 256 against 4 KV heads of the assistant's and the NextN
# drafter's targets, and the edge model's 8 against 2
_BIG = {"hq": 16, "hkv": 4, "hd": 256}
_EDGE = {"hq": 8, "hkv": 2, "hd": 256}


def listed():
    return [
        # one user's verify step: four rows, the call's latency is what counts
        {"name": "append b1 m4 bf16", "op": "append", "kv": "bf16", "inp": "bf16", "norm": True, "B": 1, "M": 4, "ctx": 8192,
         "page": 64, "ragged": False, "theta": 1e6, **_BIG},
        # a full batch's verify step into the 8-bit cache, some windows cut short
        {"name": "append b64 m3 e4m3", "op": "append", "kv": "e4m3", "inp": "bf16", "norm": True, "B": 64, "M": 3, "ctx": 4096,
         "page": 64, "ragged": True, "theta": 1e6, **_BIG},
        # prompts of a batch going into the 8-bit cache
        {"name": "append prompts e4m3", "op": "append", "kv": "e4m3", "inp": "bf16", "norm": True, "B": 8, "M": 4096, "ctx": 70,
         "page": 64, "ragged": True, "theta": 1e6, **_BIG},
        # one long prompt, fp32 activations, a bf16 cache, an odd length
        {"name": "append prompt 8191 f32 in", "op": "append", "kv": "bf16", "inp": "f32", "norm": False, "B": 1, "M": 8191, "ctx": 0,
         "page": 32, "ragged": False, "theta": 1e4, "hq": 16, "hkv": 8, "hd": 128},
        # plain decoding of one sequence with a short context: the smallest call
        {"name": "attn b1 m1 bf16 ctx999", "op": "attention", "kv": "bf16", "norm": True, "B": 1, "M": 1, "ctx": 999, "page": 16,
         "ragged": False, "window": 0, "sink": 0, "theta": 1e6, **_EDGE},
        # one user's verify step at 8192 cached positions
        {"name": "attn b1 m4 bf16 ctx8192", "op": "attention", "kv": "bf16", "norm": True, "B": 1, "M": 4, "ctx": 8192, "page": 64,
         "ragged": False, "window": 0, "sink": 0, "theta": 1e6, **_BIG},
        # sixteen sequences of 2k to 32k positions, 8-bit cache: the largest
        {"name": "attn b16 m5 e4m3 2k-32k", "op": "attention", "kv": "e4m3", "norm": True, "B": 16, "M": 5, "ctx": 32768, "page": 64,
         "ragged": True, "window": 0, "sink": 0, "theta": 1e6, **_BIG},
        # the full batch's verify step, 8-bit cache
        {"name": "attn b64 m3 e4m3 ctx4096", "op": "attention", "kv": "e4m3", "norm": True, "B": 64, "M": 3, "ctx": 4096, "page": 64,
         "ragged": False, "window": 0, "sink": 0, "theta": 1e6, **_BIG},
        # the same step in a sliding layer: 1024 positions and the attention sink
        {"name": "attn b64 m3 bf16 window", "op": "attention", "kv": "bf16", "norm": False, "B": 64, "M": 3, "ctx": 4096, "page": 32,
         "ragged": True, "window": 1024, "sink": 4, "theta": 1e4, **_BIG},
        # one user's four verify rows, five alternatives each
        {"name": "logprobs 4 rows top5", "op": "logprobs", "dtype": "bf16", "rows": 4, "V": 262144, "top": 5, "skip": 0.0},
        # a full batch: rows behind the accepted prefix are marked and skipped
        {"name": "logprobs 192 rows top20", "op": "logprobs", "dtype": "bf16", "rows": 192, "V": 262144, "top": 20, "skip": 0.25},
        # fp32 logits, log probability and entropy alone
        {"name": "logprobs 128 rows f32", "op": "logprobs", "dtype": "f32", "rows": 128, "V": 248320, "top": 0, "skip": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "logprobs"])
    if op == "logprobs":
        rows, V = _log_int(rng, 1, 256), _log_int(rng, 1000, 262144)
        while rows * V > 192 * 262144:
            rows = max(1, rows // 2)
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "rows": rows, "V": V, "top": rng.choice([0, 1, 5, 8, 20, 32]),
                "skip": rng.choice([0.0, 0.3])}
    hd, hkv, group = rng.choice([64, 128, 256, 256]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 4, 7, 8])
    c = {"op": op, "kv": rng.choice(["bf16", "e4m3"]), "norm": rng.random() < 0.5, "page": rng.choice([16, 32, 64, 128]),
         "ragged": rng.random() < 0.5, "theta": rng.choice([1e4, 1e6, 1e7]), "hq": hkv * group, "hkv": hkv, "hd": hd}
    if op == "append":
        c.update(inp=rng.choice(["bf16", "bf16", "f32"]), B=_log_int(rng, 1, 64), M=_log_int(rng, 1, 4096), ctx=rng.randint(0, 20000))
        while c["B"] * c["M"] * hkv * hd > 8 * 4096 * 1024:
            c["M"] = max(1, c["M"] // 2)
        return c
    c.update(B=_log_int(rng, 1, 64), M=rng.randint(1, 17), ctx=_log_int(rng, 1, 32768), window=0, sink=0)
    if rng.random() < 0.25:
        c.update(window=rng.choice([128, 512, 1000, 1024]), sink=rng.choice([0, 4, 130]))
    while c["B"] * (c["ctx"] + 17) * hkv * hd > 16 * 32768 * 1024 // 2 or c["B"] * (c["ctx"] + 17) * hkv * group * c["M"] * hd * 4 > 12e9:
        c["B" if c["B"] > 1 else "ctx"] //= 2
    return c


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

_KV = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "f32": torch.float32}


def _lengths(case, seed):
    """Cached positions and new rows of every sequence (host lists, from the seed)."""
    g = torch.Generator().manual_seed(seed * 7 + 1)
    B, M, ctx = case["B"], case["M"], case["ctx"]
    if case["ragged"]:
        kv = torch.randint(ctx // 16, ctx + 1, (B,), generator=g)
        n = torch.randint(0 if M > 1 else 1, M + 1, (B,), generator=g)
        n[0] = M
    else:
        kv, n = torch.full((B,), ctx), torch.full((B,), M)
    if not case["ragged"] and case["op"] == "append" and ctx:
        kv = torch.randint(ctx // 2, ctx + 1, (B,), generator=g)
    return kv.tolist(), n.tolist(), g


def _gain(hd, gen):
    return 1.0 + 0.02 * torch.randn(hd, device="cuda", generator=gen)


def _cache(case, kv_len, n_new, gen, host_gen):
    """The cache as a server has it: pages in no order, slots that hold no
    position are NaN, table entries past a sequence's end are -1.  For the
    append the pages before the ones it touches are a prefix that all
    sequences share."""
    B, ps, hkv, hd, kvt = case["B"], case["page"], case["hkv"], case["hd"], case["kv"]
    ends = [a + n for a, n in zip(kv_len, n_new)]
    per = [max(1, -(-e // ps)) for e in ends]
    maxp = -(-(case["ctx"] + case["M"]) // ps) + 1
    firsts = [0] * B if case["op"] == "attention" else [a // ps for a in kv_len]
    shared = 0 if case["op"] == "attention" else 8
    n_pages = shared + B * (maxp if case["op"] == "attention" else (case["M"] + ps - 2) // ps + 1) + 3
    order = torch.randperm(n_pages, generator=host_gen).tolist()
    table = torch.full((B, maxp), -1, dtype=torch.int32)
    nxt = shared
    for b in range(B):
        for i in range(per[b]):
            if i < firsts[b]:
                table[b, i] = order[i % shared]
            else:
                table[b, i] = order[nxt]
                nxt += 1
    dt = _KV[kvt]
    out = {"table": table.cuda(), "kv_len": torch.tensor(kv_len, dtype=torch.int32, device="cuda"),
           "n_new": torch.tensor(n_new, dtype=torch.int32, device="cuda")}
    for w in "kv":
        x = torch.empty((n_pages, ps, hkv, hd), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        if kvt == "e4m3":
            # codes as an append would have left them: the largest in the top three binades
            scale = torch.exp2(torch.randint(-7, -4, (n_pages, hkv), device="cuda", generator=gen).float())
            out[w + "_scale"] = scale
            x = (x.float() / scale[:, None, :, None]).clamp(-448, 448).to(dt)
        else:
            x = x.to(dt)
        # slots without a position: NaN
        used = torch.zeros((n_pages, ps), dtype=torch.bool, device="cuda")
        pos = torch.arange(maxp * ps, device="cuda")
        last = out["kv_len"] if case["op"] == "append" else out["kv_len"] + out["n_new"]
        pages = out["table"].long()[:, pos // ps]
        held = (pos[None] < last[:, None]) & (pages >= 0)
        used.view(-1)[(pages * ps + pos[None] % ps)[held]] = True
        if kvt == "e4m3":
            x.view(torch.uint8)[~used] = 0x7F
        else:
            x[~used] = float("nan")
        out[w] = x.permute(0, 2, 1, 3)   # [pages, KV heads, slots, hd], as the library takes it
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 3 + 2)
    s = {"case": case}
    if case["op"] == "logprobs":
        rows, V = case["rows"], case["V"]
        z = torch.empty((rows, V), dtype=torch.float32, device="cuda").normal_(generator=gen).mul_(2.5)
        # a head of likely tokens over a wide tail, as a model's logits have
        hot = torch.randint(0, V, (rows, 12), device="cuda", generator=gen)
        z.scatter_add_(1, hot, 9.0 + 3.0 * torch.randn((rows, 12), device="cuda", generator=gen))
        s["logits"] = z.to(torch.bfloat16) if case["dtype"] == "bf16" else z
        tok = hot[:, 0].to(torch.int32)
        any_tok = torch.randint(0, V, (rows,), device="cuda", generator=gen, dtype=torch.int32)
        tok = torch.where(torch.rand(rows, device="cuda", generator=gen) < 0.2, any_tok, tok)
        s["tokens"] = torch.where(torch.rand(rows, device="cuda", generator=gen) < case["skip"], torch.full_like(tok, -1), tok)
        s["tokens"][0] = any_tok[0]
        s["logprob"] = torch.zeros(rows, device="cuda")
        s["entropy"] = torch.zeros(rows, device="cuda")
        if case["top"]:
            s["top_ids"] = torch.zeros((rows, case["top"]), dtype=torch.int32, device="cuda")
            s["top_logprobs"] = torch.zeros((rows, case["top"]), device="cuda")
        return s
    kv_len, n_new, host_gen = _lengths(case, seed)
    s.update(_cache(case, kv_len, n_new, gen, host_gen))
    B, M, hq, hkv, hd = case["B"], case["M"], case["hq"], case["hkv"], case["hd"]
    # the rows as the fused query / key / value projection leaves them
    dt = torch.float32 if case.get("inp") == "f32" else torch.bfloat16
    qkv = torch.empty((B, M, (hq + 2 * hkv) * hd), dtype=dt, device="cuda").normal_(generator=gen)
    s["q"] = qkv[..., :hq * hd].unflatten(-1, (hq, hd))
    s["k_new"] = qkv[..., hq * hd:(hq + hkv) * hd].unflatten(-1, (hkv, hd))
    s["v_new"] = qkv[..., (hq + hkv) * hd:].unflatten(-1, (hkv, hd))
    s["gain"] = _gain(hd, gen) if case["norm"] else None
    if case["op"] == "attention":
        s["out"] = torch.zeros((B, M, hq, hd), dtype=dt, device="cuda")
    return s


# ----------------------------------------------------------------------------
# the operators
# ----------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state)
    return {"append": _plain_append, "attention": _plain_attention, "logprobs": _plain_logprobs}[op](state)


def _own(s):
    import mtp_speculative_decoding_gb300 as mtp
    c = s["case"]
    if c["op"] == "logprobs":
        mtp.token_logprobs(s["logits"], s["tokens"], s["logprob"], s["entropy"], s.get("top_ids"), s.get("top_logprobs"))
        return {k: s[k] for k in ("logprob", "entropy", "top_ids", "top_logprobs") if k in s}
    if "handle" not in s:   # what a server makes once for a layer's cache
        s["handle"] = mtp.make_kv_cache(s["k"], s["v"], s["table"], s.get("k_scale"), s.get("v_scale"), rope_theta=c["theta"],
                                        window=c.get("window", 0), sink=c.get("sink", 0))
        s["ws"] = mtp.alloc_workspace(mtp.kv_workspace_size(s["handle"], c["B"], c["M"], c["hq"]))
    if c["op"] == "append":
        mtp.kv_append(s["handle"], s["k_new"], s["v_new"], s["kv_len"], s["ws"], n_new=s["n_new"], k_norm=s["gain"], rms_eps=1e-6)
        return {k: s[k] for k in ("k", "v", "k_scale", "v_scale") if k in s}
    mtp.paged_attention(s["handle"], s["q"], s["kv_len"], s["out"], s["ws"], n_new=s["n_new"], q_norm=s["gain"], rms_eps=1e-6)
    return s["out"]


def _plain_rotate(x, gain, pos, theta):
    """rmsnorm (when there is a gain), then the rotation of the pairs (i, i + hd/2) by pos * theta^(-2i/hd); x [B, M, H, hd]."""
    x = x.float()
    hd = x.shape[-1]
    if gain is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gain
    freq = theta ** (-torch.arange(0, hd, 2, device=x.device, dtype=torch.float64) / hd)
    ang = pos.double()[..., None] * freq   # angles of far positions lose their fraction in 32 bits
    cos, sin = torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]
    a, b = x[..., :hd // 2], x[..., hd // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    c = s["case"]
    M, ps = c["M"], c["page"]
    j = torch.arange(M, device="cuda")
    pos = s["kv_len"].long()[:, None] + j
    live = j[None] < s["n_new"][:, None]
    rows = {"k": _plain_rotate(s["k_new"], s["gain"], pos, c["theta"]), "v": s["v_new"].float()}
    table = s["table"].long()
    out = {}
    for w in "kv":
        cache = s[w].permute(0, 2, 1, 3)    # [pages, slots, heads, hd]
        page = table.gather(1, pos.clamp(max=table.shape[1] * ps - 1) // ps)
        if c["kv"] != "e4m3":
            cache[page[live], pos[live] % ps] = rows[w][live].to(cache.dtype)
            out[w] = s[w]
            continue
        scale, codes = s[w + "_scale"], cache.view(torch.uint8)
        # the pages that each sequence's rows fall into
        n_touch = (M - 1 + ps - 1) // ps + 1
        t = s["kv_len"].long()[:, None] // ps + torch.arange(n_touch, device="cuda")
        hit = (t * ps < (s["kv_len"] + s["n_new"]).long()[:, None]) & (s["n_new"] > 0)[:, None]
        pid = table.gather(1, t.clamp(max=table.shape[1] - 1))[hit]
        b_of, first = hit.nonzero()[:, 0], (t * ps)[hit]
        slot = first[:, None] + torch.arange(ps, device="cuda")            # position of every slot of those pages
        jj = slot - s["kv_len"].long()[b_of][:, None]
        new = (jj >= 0) & (jj < s["n_new"].long()[b_of][:, None])
        old = jj < 0
        x = rows[w][b_of[:, None], jj.clamp(0, M - 1)]                       # [touched, slots, heads, hd]
        amax = x.abs().masked_fill(~new[..., None, None], 0.0).amax((1, 3))   # [touched, heads]
        _, e = torch.frexp(amax / 448)
        want = torch.exp2(torch.where(torch.frexp(amax / 448)[0] == 0.5, e - 1, e).clamp(-40, 40).float())
        want = torch.where(amax > 0, want, torch.full_like(want, 2.0 ** -40))
        had = scale[pid]
        now = torch.where(old.any(1)[:, None], torch.maximum(want, had), want)
        kept = codes[pid].view(torch.float8_e4m3fn).float() * (had / now)[:, None, :, None]
        fresh = (x / now[:, None, :, None]).clamp(-448, 448)
        value = torch.where(new[..., None, None], fresh, kept).to(torch.float8_e4m3fn).view(torch.uint8)
        write = new | old
        codes[pid[:, None].expand_as(slot)[write], (slot % ps)[write]] = value[write]
        scale[pid] = now
        out[w], out[w + "_scale"] = s[w], scale
    return out


def _plain_attention(s):
    c = s["case"]
    M, ps, hq, hkv, hd = c["M"], c["page"], c["hq"], c["hkv"], c["hd"]
    B, G = c["B"], hq // hkv
    j = torch.arange(M, device="cuda")
    pos = s["kv_len"].long()[:, None] + j
    q = _plain_rotate(s["q"], s["gain"], pos, c["theta"]).view(B, M, hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, hkv, M * G, hd)
    end = (s["kv_len"] + s["n_new"]).long()
    t = torch.arange((c["ctx"] + M + ps - 1) // ps * ps, device="cuda")
    page = s["table"].long()[:, : t.numel() // ps]
    held = t[None] < end[:, None]
    x = {}
    for w in "kv":
        pages = s[w][page.clamp(min=0)].float()                              # [B, pages, heads, slots, hd]
        if c["kv"] == "e4m3":
            pages = pages * s[w + "_scale"][page.clamp(min=0)][..., None, None]
        pages = pages.permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, hd)
        x[w] = pages.masked_fill(~held[:, None, :, None], 0.0)
    z = torch.matmul(q, x["k"].transpose(2, 3)) * (1.0 / math.sqrt(hd))
    p = pos[:, :, None]
    see = (t <= p) & held[:, None]
    if c["window"]:
        lo = (p + 1 - c["window"]).clamp(min=0)
        see &= (t >= lo) | (t < c["sink"])
    z = z.masked_fill(~see[:, None, :, None].expand(B, 1, M, G, t.numel()).reshape(B, 1, M * G, -1), -math.inf)
    z = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-1e30))
    o = torch.matmul(z, x["v"]) / z.sum(-1, keepdim=True)
    o = o.view(B, hkv, M, G, hd).permute(0, 2, 1, 3, 4).reshape(B, M, hq, hd).to(s["out"].dtype)
    s["out"].copy_(torch.where((j[None] < s["n_new"][:, None])[..., None, None], o, s["out"]))
    return s["out"]


def _plain_logprobs(s):
    c = s["case"]
    z = s["logits"].float()
    live = s["tokens"] >= 0
    m = z.amax(-1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    total = e.sum(-1)
    lse = torch.log(total)
    keep = {"logprob": d.gather(1, s["tokens"].long().clamp(min=0)[:, None])[:, 0] - lse,
            "entropy": lse - (e * d).sum(-1) / total}
    if c["top"]:
        bits = (z + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) * (1 << 32) + ((1 << 32) - 1 - torch.arange(c["V"], device="cuda"))
        ids = ((1 << 32) - 1) - (torch.topk(key, c["top"], dim=-1)[0] & 0xFFFFFFFF)   # ties go to the lowest index
        keep["top_ids"] = ids.to(torch.int32)
        keep["top_logprobs"] = d.gather(1, ids) - lse[:, None]
    for k, v in keep.items():
        s[k].copy_(torch.where(live if v.dim() == 1 else live[:, None], v, s[k]))
    return {k: s[k] for k in keep}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "logprobs":
        esz = 2 if c["dtype"] == "bf16" else 4
        rows = c["rows"] * (1.0 - c["skip"])
        return {"bytes": rows * (c["V"] * esz + 12 + 8 * c["top"]), "flops": rows * c["V"] * 6.0}
    kv, n, _ = _lengths(c, 0)
    esz = {"bf16": 2, "f32": 4, "e4m3": 1}[c["kv"]]
    if c["op"] == "append":
        elems = sum(n) * c["hkv"] * c["hd"] * 2
        return {"bytes": elems * ((4 if c["inp"] == "f32" else 2) + esz), "flops": elems * 6.0}
    span = 0.0
    pairs = 0.0
    for a, m in zip(kv, n):
        if m == 0:
            continue
        seen = a + m
        if c["window"]:
            seen = min(seen, c["window"] + m - 1 + c["sink"])
        span += seen
        pairs += m * min(a + (m + 1) / 2, c["window"] + c["sink"] if c["window"] else 1e18)
    io = sum(n) * c["hq"] * c["hd"] * 4.0
    return {"bytes": span * c["hkv"] * c["hd"] * 2 * esz + io, "flops": pairs * c["hq"] * c["hd"] * 4.0}


# ----------------------------------------------------------------------------
# the definitions, in 64 bits
# ----------------------------------------------------------------------------

def _e4m3_nearest(x):
    """The nearest value of e4m3 (ties to even code, at most 448) to each x."""
    _, e = torch.frexp(x)
    step = torch.exp2((torch.maximum(e - 1, torch.full_like(e, -6)) - 3).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def _normed_turned(x, gain, positions, theta):
    """One sequence's rows x [m, heads, hd] at the positions [m], as complex pairs."""
    x = x.double()
    h = x.shape[-1] // 2
    if gain is not None:
        x = x / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / (2 * h) + 1e-6) * gain.double()
    i = torch.arange(h, device=x.device, dtype=torch.float64)
    turn = positions.double()[:, None] * torch.exp(-math.log(theta) * i / h)
    z = torch.complex(x[..., :h], x[..., h:]) * torch.polar(torch.ones_like(turn), turn)[:, None]
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "logprobs": _exact_logprobs}[case["op"]](case, s)


def _exact_append(c, s):
    ps, kv = c["page"], s["kv_len"].tolist()
    got = {}
    for w in "kv":
        cache = s[w].double()                  # [pages, heads, slots, hd]
        scale = s[w + "_scale"].double() if c["kv"] == "e4m3" else None
        for b, n in enumerate(s["n_new"].tolist()):
            if n == 0:
                continue
            p = torch.arange(kv[b], kv[b] + n, device="cuda")
            x = _normed_turned(s["k_new"][b, :n], s["gain"], p, c["theta"]) if w == "k" else s["v_new"][b, :n].double()
            if scale is None:
                cache[s["table"][b].long()[p // ps], :, p % ps] = x
                continue
            at = 0
            while at < n:                          # page by page
                page, off = int(s["table"][b, (kv[b] + at) // ps]), (kv[b] + at) % ps
                m = min(ps - off, n - at)
                y = x[at:at + m].transpose(0, 1)   # [heads, rows, hd]
                big = y.abs().amax((1, 2))
                k = torch.ceil(torch.log2(big.clamp(min=2.0 ** -60) / 448))
                k = torch.where(big > 448 * torch.exp2(k), k + 1, torch.where(big <= 448 * torch.exp2(k - 1), k - 1, k)).clamp(-40, 40)
                now = torch.exp2(k)
                if off:
                    now = torch.maximum(now, scale[page])
                    cache[page, :, :off] = _e4m3_nearest(cache[page, :, :off] * (scale[page] / now)[:, None, None])
                cache[page, :, off:off + m] = _e4m3_nearest(y / now[:, None, None])
                scale[page] = now
                at += m
        got[w] = cache
        if scale is not None:
            got[w + "_scale"] = scale
    return got


def _exact_attention(c, s):
    out = s["out"].double()
    ps, G = c["page"], c["hq"] // c["hkv"]
    for b, (a, n) in enumerate(zip(s["kv_len"].tolist(), s["n_new"].tolist())):
        if n == 0:
            continue
        t = torch.arange(a + n, device="cuda")
        page = s["table"][b].long()[t // ps]
        q = _normed_turned(s["q"][b, :n], s["gain"], t[a:], c["theta"])
        for h in range(c["hkv"]):
            k, v = s["k"][page, h, t % ps].double(), s["v"][page, h, t % ps].double()
            if c["kv"] == "e4m3":
                k, v = k * s["k_scale"][page, h].double()[:, None], v * s["v_scale"][page, h].double()[:, None]
            for j in range(n):
                first = max(0, a + j + 1 - c["window"]) if c["window"] else 0
                see = torch.cat([t[: min(c["sink"], first)], t[first: a + j + 1]])
                prob = torch.softmax(q[j, h * G:(h + 1) * G] @ k[see].T / math.sqrt(c["hd"]), -1)
                out[b, j, h * G:(h + 1) * G] = prob @ v[see]
    return out


def _exact_logprobs(c, s):
    got = {"logprob": s["logprob"].double(), "entropy": s["entropy"].double()}
    if c["top"]:
        got["top_ids"], got["top_logprobs"] = s["top_ids"].clone(), s["top_logprobs"].double()
    for r, tok in enumerate(s["tokens"].tolist()):
        if tok < 0:
            continue
        z = s["logits"][r].double()
        logp = torch.log_softmax(z, 0)
        got["logprob"][r] = logp[tok]
        got["entropy"][r] = -(logp.exp() * logp).sum()
        if c["top"]:
            order = torch.sort(z, descending=True, stable=True)[1][: c["top"]]
            got["top_ids"][r], got["top_logprobs"][r] = order.to(torch.int32), logp[order]
    return got
