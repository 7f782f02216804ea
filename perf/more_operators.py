"""The cases by which the target's work on prompts and on shared prefixes is measured.

  rotate   query and key rows of a target that sees images and video: norm, then
           a rotation whose pairs go by several positions (time, height, width),
           before the rows go into a cache that does not rotate;
  prompt   the rows of whole prompts, packed one after another, attend the paged
           cache that holds their keys and values already (causal, or a window
           with an attention sink), with or without positions cached before;
  prefix   the rows of a decoding batch whose sequences share long prefixes: each
           group's prefix is read and computed once for all of its rows.

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
        # one user's verify step: four rows behind an image, the call's latency is what counts
        {"name": "rotate 4 rows", "op": "rotate", "dtype": "bf16", "rows": 4, "sections": "44,42,42", "interleaved": True, "norm": True,
         "theta": 1e6, **_BIG},
        # a prompt with images, every pair turned, sections one after another
        {"name": "rotate 8192 rows bf16", "op": "rotate", "dtype": "bf16", "rows": 8192, "sections": "16,24,24", "interleaved": False,
         "norm": False, "theta": 1e6, "hq": 16, "hkv": 8, "hd": 128},
        # fp32 activations, a quarter of the head turned, an odd number of rows
        {"name": "rotate 4093 rows f32 partial", "op": "rotate", "dtype": "f32", "rows": 4093, "sections": "11,11,10", "interleaved": True,
         "norm": True, "theta": 1e7, **_BIG},
        # one short question to the edge model: the smallest call
        {"name": "prompt 77 edge", "op": "prompt", "kv": "bf16", "norm": True, "B": 1, "rows": 77, "ctx": 0, "page": 16, "ragged": False,
         "window": 0, "sink": 0, "theta": 1e6, **_EDGE},
        # one long prompt: the largest
        {"name": "prompt 8192 bf16", "op": "prompt", "kv": "bf16", "norm": True, "B": 1, "rows": 8192, "ctx": 0, "page": 64, "ragged": False,
         "window": 0, "sink": 0, "theta": 1e6, **_BIG},
        # prompts of different lengths packed into one call, heads of 128
        {"name": "prompts packed hd128", "op": "prompt", "kv": "bf16", "norm": False, "B": 13, "rows": 2048, "ctx": 0, "page": 32, "ragged": True,
         "window": 0, "sink": 0, "theta": 1e4, "hq": 16, "hkv": 8, "hd": 128},
        # the next piece of a long prompt, the earlier ones in the 8-bit cache
        {"name": "prompt piece e4m3", "op": "prompt", "kv": "e4m3", "norm": True, "B": 2, "rows": 1024, "ctx": 15000, "page": 64, "ragged": False,
         "window": 0, "sink": 0, "theta": 1e6, **_BIG},
        # a sliding layer over packed prompts
        {"name": "prompts window bf16", "op": "prompt", "kv": "bf16", "norm": True, "B": 5, "rows": 4096, "ctx": 0, "page": 32, "ragged": True,
         "window": 1024, "sink": 4, "theta": 1e4, **_BIG},
        # four users of the edge model behind one instruction, plain decoding
        {"name": "prefix b4 m1 edge", "op": "prefix", "kv": "bf16", "norm": True, "B": 4, "M": 1, "groups": 1, "prefix": 1000, "ctx": 60,
         "page": 16, "ragged": False, "theta": 1e6, **_EDGE},
        # a full batch's verify step behind one long document
        {"name": "prefix b64 m3 8192", "op": "prefix", "kv": "bf16", "norm": True, "B": 64, "M": 3, "groups": 1, "prefix": 8192, "ctx": 512,
         "page": 64, "ragged": True, "theta": 1e6, **_BIG},
        # the 8-bit cache, four groups with prefixes of their own
        {"name": "prefix b64 m4 4 groups e4m3", "op": "prefix", "kv": "e4m3", "norm": True, "B": 64, "M": 4, "groups": 4, "prefix": 4096,
         "ctx": 700, "page": 64, "ragged": True, "theta": 1e6, **_BIG},
        # many short answers, heads of 128, a prefix that ends inside a page
        {"name": "prefix b128 m1 hd128", "op": "prefix", "kv": "bf16", "norm": False, "B": 128, "M": 1, "groups": 1, "prefix": 5001, "ctx": 130,
         "page": 32, "ragged": True, "theta": 1e4, "hq": 16, "hkv": 8, "hd": 128},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rotate", "prompt", "prompt", "prefix", "prefix"])
    hd, hkv, group = rng.choice([64, 128, 256, 256]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 4, 7, 8])
    c = {"op": op, "norm": rng.random() < 0.5, "theta": rng.choice([1e4, 1e6, 1e7]), "hq": hkv * group, "hkv": hkv, "hd": hd}
    if op == "rotate":
        pairs = hd // 2 if rng.random() < 0.6 else hd // 8
        h = rng.randint(1, pairs // 3)
        w = rng.choice([h, rng.randint(1, pairs // 3)])
        c.update(dtype=rng.choice(["bf16", "bf16", "f32"]), rows=_log_int(rng, 1, 16384), interleaved=rng.random() < 0.5,
                 sections="%d,%d,%d" % (pairs - h - w, h, w))
        while c["rows"] * (c["hq"] + hkv) * hd > 16384 * 24 * 128:
            c["rows"] = max(1, c["rows"] // 2)
        return c
    c.update(kv=rng.choice(["bf16", "bf16", "e4m3"]), page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.5)
    if op == "prompt":
        c.update(B=_log_int(rng, 1, 24), rows=_log_int(rng, 1, 8192), ctx=rng.choice([0, 0, _log_int(rng, 1, 16000)]), window=0, sink=0)
        if rng.random() < 0.25:
            c.update(window=rng.choice([128, 512, 1000, 1024]), sink=rng.choice([0, 4, 130]))
        while (c["B"] * c["rows"] * (c["rows"] + c["ctx"]) * c["hq"] * hd > 8192 * 8192 * 16 * 256
               or c["B"] * c["rows"] * (c["rows"] + c["ctx"]) * c["hq"] > 2.2e9):
            c["B" if c["B"] > 1 else "rows"] //= 2
        return c
    c.update(B=_log_int(rng, 2, 128), M=rng.choice([1, 1, 3, 5, rng.randint(1, 17)]), prefix=_log_int(rng, 16, 16000), ctx=_log_int(rng, 1, 1500))
    c["groups"] = min(rng.choice([1, 1, 2, 5]), c["B"])
    while c["B"] * (c["prefix"] + c["ctx"] + 17) * (c["hkv"] * hd + c["hq"] * c["M"]) > 1.6e9:
        c["prefix" if c["prefix"] > 500 else "B"] //= 2
        c["groups"] = max(1, min(c["groups"], c["B"]))
    return c


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "f32": torch.float32}


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _packed(case):
    """Rows of a prompt call's buffers: ragged prompts fill it, or leave rows behind the last one."""
    return case["rows"] + (case["B"] - 1) * case["rows"] // (2 if case["ragged"] else 1)


def _lengths(case, seed):
    """Cached positions, new rows and, for shared prefixes, the group's bounds and
    prefix lengths (host lists, from the seed)."""
    g = torch.Generator().manual_seed(seed * 7 + 1)
    B, ctx = case["B"], case["ctx"]
    M = case["M"] if case["op"] == "prefix" else case["rows"]
    if case["ragged"]:
        kv = torch.randint(ctx // 16, ctx + 1, (B,), generator=g).tolist()
        n = torch.randint(1 if M == 1 else 0, M + 1, (B,), generator=g).tolist()
        n[0] = M
    else:
        kv, n = [ctx] * B, [M] * B
    if case["op"] == "prompt":   # what does not fit the call's buffer of rows is cut
        rest, room = sum(n[1:]), _packed(case) - n[0]
        n[1:] = [x * room // rest if rest > room else x for x in n[1:]]
        return kv, n, None, None, g
    k, P = case["groups"], case["prefix"]
    cut = sorted((torch.randperm(B - 1, generator=g)[: k - 1] + 1).tolist()) if case["ragged"] else [B * i // k for i in range(1, k)]
    start = [0, *cut, B]
    pre = [P] + torch.randint(P // 2, P + 1, (k - 1,), generator=g).tolist()
    of = [i for i in range(k) for _ in range(start[i], start[i + 1])]
    return [a + pre[of[b]] for b, a in enumerate(kv)], n, start, pre, g


def _cache(case, kv_len, n_new, start, pre, gen, host_gen):
    """The cache as a server has it: pages in no order, slots that hold no
    position are NaN, table entries past a sequence's end are -1.  Sequences of a
    group have the pages of their prefix in common; the rest of a page in which
    a prefix ends is each sequence's own."""
    B, ps, hkv, hd, kvt = case["B"], case["page"], case["hkv"], case["hd"], case["kv"]
    ends = [a + n for a, n in zip(kv_len, n_new)]
    per = [max(1, -(-e // ps)) for e in ends]
    maxp = max(per) + 1
    group = [i for i in range(len(pre)) for _ in range(start[i], start[i + 1])] if pre else list(range(B))
    first = [start[i] for i in group] if pre else list(range(B))
    common = [pre[i] // ps for i in group] if pre else [0] * B
    n_pages = sum(per) - sum(c for b, c in enumerate(common) if first[b] != b) + 3
    order = torch.randperm(n_pages, generator=host_gen)
    table = torch.full((B, maxp), -1, dtype=torch.int32)
    held = torch.zeros((n_pages, ps), dtype=torch.bool)
    nxt = 0
    for b in range(B):
        keep = common[b] if first[b] != b else 0
        table[b, :keep] = table[first[b], :keep]
        table[b, keep:per[b]] = order[nxt:nxt + per[b] - keep]
        nxt += per[b] - keep
        slots = torch.arange(per[b] * ps)
        live = slots < ends[b]
        if pre and first[b] != b:
            live &= slots >= pre[group[b]]
        held[table[b, slots[live] // ps].long(), slots[live] % ps] = True
    held = held.cuda()
    out = {"table": table.cuda(), "kv_len": _i32(kv_len), "n_new": _i32(n_new)}
    for w in "kv":
        x = torch.empty((n_pages, ps, hkv, hd), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        if kvt == "e4m3":
            # codes as an append would have left them: the largest in the top three binades
            scale = torch.exp2(torch.randint(-7, -4, (n_pages, hkv), device="cuda", generator=gen).float())
            out[w + "_scale"] = scale
            x = (x.float() / scale[:, None, :, None]).clamp(-448, 448).to(_DT[kvt])
            x.view(torch.uint8)[~held] = 0x7F
        else:
            x[~held] = float("nan")
        out[w] = x.permute(0, 2, 1, 3)   # [pages, KV heads, slots, hd], as the library takes it
    return out


def _image_positions(rows, gen):
    """Time, height and width of a prompt's tokens: stretches of text, where all
    three advance together, around images of up to 32 x 32 patches."""
    at, t, parts = int(torch.randint(0, 100000, (1,), generator=gen)), 0, []
    while t < rows:
        n = int(torch.randint(1, 200, (1,), generator=gen))
        parts.append((at + torch.arange(n)).expand(3, n))
        h, w = torch.randint(2, 33, (2,), generator=gen).tolist()
        at += n
        y, x = torch.arange(h * w) // w, torch.arange(h * w) % w
        parts.append(torch.stack([torch.full((h * w,), at), at + y, at + x]))
        at += max(h, w)
        t += n + h * w
    return torch.cat(parts, 1)[:, :rows].to(torch.int32).contiguous().cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 3 + 2)
    s = {"case": case}
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    gain = [1.0 + 0.02 * torch.randn(hd, device="cuda", generator=gen) if case["norm"] else None for _ in range(2)]
    dt = _DT[case.get("dtype", "bf16")]
    if case["op"] == "rotate":
        s["pos"] = _image_positions(case["rows"], torch.Generator().manual_seed(seed * 7 + 1))
        lead = (case["rows"],)
        s["sections"] = tuple(int(x) for x in case["sections"].split(","))
    else:
        kv_len, n_new, start, pre, host_gen = _lengths(case, seed)
        s.update(_cache(case, kv_len, n_new, start, pre, gen, host_gen))
        if case["op"] == "prompt":
            ends = torch.tensor([0, *n_new]).cumsum(0)
            s["row_start"], s["longest"], s["reach"] = ends.to(torch.int32).cuda(), max(n_new), max(a + n for a, n in zip(kv_len, n_new))
            lead = (_packed(case),)
        else:
            s["group_start"], s["prefix_len"], s["reach"] = _i32(start), _i32(pre), max(a + n for a, n in zip(kv_len, n_new))
            lead = (case["B"], case["M"])
    # the rows as the fused query / key / value projection leaves them
    qkv = torch.empty((*lead, (hq + 2 * hkv) * hd), dtype=dt, device="cuda").normal_(generator=gen)
    s["q"] = qkv[..., :hq * hd].unflatten(-1, (hq, hd))
    s["gain"] = gain[0]
    s["out"] = torch.zeros((*lead, hq, hd), dtype=dt, device="cuda")
    if case["op"] == "rotate":
        s["k"], s["k_gain"] = qkv[..., hq * hd:(hq + hkv) * hd].unflatten(-1, (hkv, hd)), gain[1]
        s["out_k"] = torch.zeros((*lead, hkv, hd), dtype=dt, device="cuda")
    return s


# ----------------------------------------------------------------------------
# the operators
# ----------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state)
    return {"rotate": _plain_rotate, "prompt": _plain_prompt, "prefix": _plain_prefix}[op](state)


def _own(s):
    import mtp_speculative_decoding_gb300 as mtp
    c = s["case"]
    if c["op"] == "rotate":
        mtp.rotate_axes(s["q"], s["k"], s["pos"], s["sections"], c["theta"], s["out"], s["out_k"], interleaved=c["interleaved"],
                        q_norm=s["gain"], k_norm=s["k_gain"], rms_eps=1e-6)
        return {"q": s["out"], "k": s["out_k"]}
    if "handle" not in s:   # what a server makes once for a layer's cache
        s["handle"] = mtp.make_kv_cache(s["k"], s["v"], s["table"], s.get("k_scale"), s.get("v_scale"), rope_theta=c["theta"],
                                        window=c.get("window", 0), sink=c.get("sink", 0))
        size = (mtp.prompt_workspace_size(s["handle"], c["B"], s["q"].shape[0], c["hq"]) if c["op"] == "prompt" else
                mtp.prefix_workspace_size(s["handle"], c["B"], c["M"], c["hq"]))
        s["ws"] = mtp.alloc_workspace(size)
    if c["op"] == "prompt":
        mtp.prompt_attention(s["handle"], s["q"], s["row_start"], s["kv_len"], s["out"], s["ws"], q_norm=s["gain"], rms_eps=1e-6)
    else:
        mtp.prefix_attention(s["handle"], s["q"], s["kv_len"], s["group_start"], s["prefix_len"], s["out"], s["ws"], n_new=s["n_new"],
                             q_norm=s["gain"], rms_eps=1e-6)
    return s["out"]


def _normed(x, gain):
    x = x.float()
    return x if gain is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gain


def _turned(x, ang):
    """The rotation of the pairs (i, i + r) of the first 2 r dimensions, r = ang.shape[-1]; x [..., H, hd], ang [..., r] in 64 bits."""
    r = ang.shape[-1]
    cos, sin = torch.cos(ang).float()[..., None, :], torch.sin(ang).float()[..., None, :]
    a, b = x[..., :r], x[..., r:2 * r]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * r:]], -1)


def _plain_rotate(s):
    c, sec = s["case"], torch.tensor(s["sections"], device="cuda")
    pairs, n = sum(s["sections"]), len(s["sections"])
    i = torch.arange(pairs, device="cuda")
    if c["interleaved"]:
        axis = torch.where(i < n * sec[i % n], i % n, 0)
    else:
        axis = torch.searchsorted(sec.cumsum(0), i, right=True)
    ang = s["pos"].double()[axis].T * c["theta"] ** (-i.double() / pairs)   # angles of far positions lose their fraction in 32 bits
    s["out"].copy_(_turned(_normed(s["q"], s["gain"]), ang))
    s["out_k"].copy_(_turned(_normed(s["k"], s["k_gain"]), ang))
    return {"q": s["out"], "k": s["out_k"]}


def _attend(s, q, pos, table, live):
    """Rows q [B, M, hq, hd] at the positions pos [B, M] against the pages of table; rows that are not live may come out as anything."""
    c = s["case"]
    B, M, hq, hd = q.shape
    hkv, ps = c["hkv"], c["page"]
    G = hq // hkv
    freq = c["theta"] ** (-torch.arange(0, hd, 2, device="cuda", dtype=torch.float64) / hd)
    q = _turned(_normed(q, s["gain"]), pos.double()[..., None] * freq).view(B, M, hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, hkv, M * G, hd)
    end = (s["kv_len"] + s["n_new"]).long()
    t = torch.arange((s["reach"] + ps - 1) // ps * ps, device="cuda")
    page = table.long()[:, : t.numel() // ps].clamp(min=0)
    held = t < end[:, None]
    x = {}
    for w in "kv":
        pages = s[w][page].float()                              # [B, pages, heads, slots, hd]
        if c["kv"] == "e4m3":
            pages = pages * s[w + "_scale"][page][..., None, None]
        x[w] = pages.permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, hd).masked_fill(~held[:, None, :, None], 0.0)
    z = torch.matmul(q, x["k"].transpose(2, 3)) * (1.0 / math.sqrt(hd))
    p = pos[:, :, None]
    see = (t <= p) & held[:, None]
    if c.get("window"):
        see &= (t > p - c["window"]) | (t < c["sink"])
    z.view(B, hkv, M, G, -1).masked_fill_(~see[:, None, :, None], -math.inf)
    z = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-1e30))
    o = torch.matmul(z, x["v"]) / z.sum(-1, keepdim=True)
    return o.view(B, hkv, M, G, hd).permute(0, 2, 1, 3, 4).reshape(B, M, hq, hd)


def _plain_prompt(s):
    j = torch.arange(s["longest"], device="cuda")
    live = j < s["n_new"][:, None]
    row = torch.where(live, s["row_start"].long()[:-1, None] + j, 0)
    o = _attend(s, s["q"][row], s["kv_len"].long()[:, None] + j, s["table"], live)
    s["out"][row[live]] = o[live].to(s["out"].dtype)
    return s["out"]


def _plain_prefix(s):
    j = torch.arange(s["case"]["M"], device="cuda")
    live = j < s["n_new"][:, None]
    b = torch.arange(s["case"]["B"], device="cuda")
    group = torch.searchsorted(s["group_start"].long()[1:], b, right=True)
    first, P = s["group_start"].long()[group], s["prefix_len"].long()[group]
    ps, maxp = s["case"]["page"], s["table"].shape[1]
    # every sequence's own view of the prefix; where it ends inside a page, that page is
    # put together behind the pool's last one
    table = torch.where(torch.arange(maxp, device="cuda") < (P // ps)[:, None], s["table"][first], s["table"])
    at = (P // ps).clamp(max=maxp - 1)
    mine, theirs = s["table"][b, at].long().clamp(min=0), s["table"][first, at].long().clamp(min=0)
    low = (torch.arange(ps, device="cuda") < (P % ps)[:, None])[:, None, :, None]
    pool = dict(s)
    n = s["k"].shape[0]
    for w in "kv":
        x, y = s[w][mine], s[w][theirs]
        if s["case"]["kv"] == "e4m3":   # (as values: their pages' scales differ)
            x, y = x.float() * s[w + "_scale"][mine][..., None, None], y.float() * s[w + "_scale"][theirs][..., None, None]
            pool[w] = torch.cat([s[w].float() * s[w + "_scale"][..., None, None], torch.where(low, y, x)])
            pool[w + "_scale"] = torch.ones((n + b.numel(), s["case"]["hkv"]), device="cuda")
        else:
            pool[w] = torch.cat([s[w], torch.where(low, y, x)])
    table[b, at] = torch.where(P % ps > 0, (n + b).to(torch.int32), table[b, at])
    o = _attend(pool, s["q"], s["kv_len"].long()[:, None] + j, table, live)
    s["out"][live] = o[live].to(s["out"].dtype)
    return s["out"]


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "rotate":
        elems = c["rows"] * (c["hq"] + c["hkv"]) * float(c["hd"])
        return {"bytes": elems * 2 * (4 if c["dtype"] == "f32" else 2) + 12.0 * c["rows"], "flops": elems * 6.0}
    kv, n, start, pre, _ = _lengths(c, 0)
    esz = 1 if c["kv"] == "e4m3" else 2
    W, span, pairs = c.get("window", 0), 0.0, 0.0
    for b, (a, m) in enumerate(zip(kv, n)):
        if m == 0:
            continue
        if W:
            span += min(a + m, W + m - 1 + c["sink"])
            pairs += sum(min(a + j + 1, W + c["sink"]) for j in range(m))
        else:
            span += a + m
            pairs += m * (a + (m + 1) / 2)
    if pre:
        for i, p in enumerate(pre):
            having = sum(m > 0 for m in n[start[i]:start[i + 1]])
            span -= p * max(0, having - 1)
    return {"bytes": span * c["hkv"] * c["hd"] * 2 * esz + sum(n) * c["hq"] * c["hd"] * 4.0, "flops": pairs * c["hq"] * c["hd"] * 4.0}


# ----------------------------------------------------------------------------
# the definitions, in 64 bits
# ----------------------------------------------------------------------------

def _spun(x, gain, turn):
    """rmsnorm (when there is a gain), then the pairs as complex numbers times e^(i turn); x [m, heads, hd], turn [m, r]."""
    x = x.double()
    if gain is not None:
        x = x / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / x.shape[-1] + 1e-6) * gain.double()
    r = turn.shape[-1]
    z = torch.complex(x[..., :r], x[..., r:2 * r]) * torch.polar(torch.ones_like(turn), turn)[:, None]
    return torch.cat([z.real, z.imag, x[..., 2 * r:]], -1)


def exact(case, seed):
    c = case
    if c["op"] != "rotate":
        kv, n, _, _, _ = _lengths(c, seed)
        if sum(m * (a + m) for a, m in zip(kv, n)) * c["hq"] * c["hd"] * 4.0 > 6e12:
            return None
    s = prepare(case, seed)
    if c["op"] == "rotate":
        return _exact_rotate(c, s)
    return _exact_attention(c, s)


def _exact_rotate(c, s):
    sec, n = s["sections"], len(s["sections"])
    pairs = sum(sec)
    if c["interleaved"]:
        axis = [i % n if i < n * sec[i % n] else 0 for i in range(pairs)]
    else:
        axis = [a for a in range(n) for _ in range(sec[a])]
    turn = torch.stack([s["pos"][a].double() * math.exp(-math.log(c["theta"]) * i / pairs) for i, a in enumerate(axis)], 1)
    return {"q": _spun(s["q"], s["gain"], turn), "k": _spun(s["k"], s["k_gain"], turn)}


def _exact_attention(c, s):
    out = s["out"].double()
    ps, hkv, hd, G, W = c["page"], c["hkv"], c["hd"], c["hq"] // c["hkv"], c.get("window", 0)
    rows = s["row_start"].tolist() if c["op"] == "prompt" else None
    start = s["group_start"].tolist() if c["op"] == "prefix" else None
    wave = torch.exp(-math.log(c["theta"]) * torch.arange(hd // 2, device="cuda", dtype=torch.float64) * 2 / hd)
    for b, (a, n) in enumerate(zip(s["kv_len"].tolist(), s["n_new"].tolist())):
        if n == 0:
            continue
        t = torch.arange(a + n, device="cuda")
        page = s["table"][b].long()[t // ps]
        if start:
            i = max(x for x in range(len(start) - 1) if start[x] <= b)
            page = torch.where(t < int(s["prefix_len"][i]), s["table"][start[i]].long()[t // ps], page)
        src, dst = (s["q"][rows[b]:rows[b] + n], out[rows[b]:rows[b] + n]) if rows else (s["q"][b, :n], out[b, :n])
        q = _spun(src, s["gain"], t[a:].double()[:, None] * wave)
        for h in range(hkv):
            k, v = s["k"][page, h, t % ps].double(), s["v"][page, h, t % ps].double()
            if c["kv"] == "e4m3":
                k, v = k * s["k_scale"][page, h].double()[:, None], v * s["v_scale"][page, h].double()[:, None]
            for j in range(0, n, 256):
                m = min(256, n - j)
                far = a + j + m                     # positions that any of these rows sees
                p = t[a + j:far]
                hide = t[:far] > p[:, None]
                if W:
                    hide |= (t[:far] <= p[:, None] - W) & (t[:far] >= c["sink"])
                z = torch.einsum("mgd,td->mgt", q[j:j + m, h * G:(h + 1) * G], k[:far]) / math.sqrt(hd)
                prob = torch.softmax(z.masked_fill(hide[:, None], -math.inf), -1)
                dst[j:j + m, h * G:(h + 1) * G] = torch.einsum("mgt,td->mgd", prob, v[:far])
    return out
