"""Plain 64-bit forms of the attention of prompts and of shared prefixes and of
the rotation by several positions, for the GPU tests.  They share no code with
the library.

Tolerances follow from the roundings.  u = 2^-24 is the fp32 half step; a value
rounded to bf16 is off by at most 2^-8 of itself, to fp16 by 2^-11.
"""
import math

import torch

import paged_common as pc

U = pc.U


def attend(pool, b, q, gain, start, theta, window=0, sink=0, scale=None, absent=(), prefix=0, first=None):
    """Rows q [n, hq, hd] of sequence b at positions start + j, in 64 bits: the
    result, sum p |v| and, per row, the largest sum |q k| (for the error bounds).
    absent: positions that are masked; positions below prefix lie on the pages of
    sequence `first`."""
    n, hq, hd = q.shape
    G, end = hq // pool.hkv, start + n
    scale = 1 / math.sqrt(hd) if scale is None else scale
    p = torch.arange(start, end, device="cuda")
    qq = pc.turn(q, gain, p, theta).view(n, pool.hkv, G, hd)
    t = torch.arange(end, device="cuda")

    def rows(w):
        own = pool.rows(w, b, t[prefix:])
        return torch.cat([pool.rows(w, first, t[:prefix]), own], 1) if prefix else own
    k, v = rows("k"), rows("v")
    see = t <= p[:, None]
    if window:
        see &= (t > p[:, None] - window) | (t < sink)
    if len(absent):
        see[:, list(absent)] = False
    held = see.any(0)
    k, v = (x.masked_fill(~held[None, :, None], 0.0) for x in (k, v))
    z = torch.einsum("nhgd,htd->nhgt", qq, k) * scale
    z = z.masked_fill(~see[:, None, None], -math.inf)
    pr = torch.softmax(z, -1).nan_to_num(0.0)        # a row that attends nothing gives zeros
    out = torch.einsum("nhgt,htd->nhgd", pr, v).reshape(n, hq, hd)
    mass = torch.einsum("nhgt,htd->nhgd", pr, v.abs()).reshape(n, hq, hd)
    dots = torch.einsum("nhgd,htd->nhgt", qq.abs(), k.abs()).masked_fill(~see[:, None, None], 0.0).amax(-1).reshape(n, hq) * scale
    return out, mass, dots


def tol(ref, mass, dots, hd, T, q_step, out_step):
    """A score is off by q_step sum |q k| (the rounding of a rotated query, 0 in
    fp32) and (2 hd + 80) u of it (sums of hd products truncated in the matrix
    unit, the norm's and rotation's 32 u); its exponential by that and 4 u, the
    sum that divides by as much again; a probability by q_step of itself; the
    weighted sum adds 2 T + 200 roundings, and the result its own rounding."""
    ds = dots[..., None] * (q_step + (2 * hd + 80) * U)
    rel = 2 * ds + (2 * T + 200) * U + q_step
    return rel * mass + out_step * (ref.abs() + rel * mass)


def check(out, ref, mass, dots, T, kv, random=True):
    """kv: the cache's type.  Against random keys and values the three roundings
    (query, probability, result) are independent and each is off by 2^-8 / 3 rms
    of its value at most: together below 2^-8 of the result's rms."""
    low = out.dtype == torch.bfloat16
    tensor = low and kv != "f32" and out.shape[-1] in (64, 128, 256)
    q_step = (2.0 ** -8 if kv == "bf16" else 2.0 ** -11) if tensor else 0.0
    err = (out.double() - ref).abs()
    bound = tol(ref, mass, dots, out.shape[-1], T, q_step, 2.0 ** -8 if low else U)
    assert (err <= bound).all(), float((err / bound.clamp(min=1e-30)).max())
    if random and low and ref.numel() > 4096:
        assert err.square().mean().sqrt() <= 2.0 ** -8 * ref.square().mean().sqrt()


def axis_of(i, sections, interleaved):
    n = len(sections)
    if interleaved:
        return i % n if i < n * sections[i % n] else 0
    a = 0
    while i >= sum(sections[: a + 1]):
        a += 1
    return a


def rotate(x, gain, positions, sections, theta, interleaved, eps=1e-6):
    """x [T, H, hd] normed and turned in 64 bits, and the bound of its fp32 error
    (pc.turn_tol: of a pair's magnitude; of the value itself where nothing turns)."""
    x = x.double()
    pairs = sum(sections)
    if gain is not None:
        x = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * gain.double()
    ang = torch.stack([positions[axis_of(i, sections, interleaved)].double() * theta ** (-i / pairs) for i in range(pairs)], -1)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b, rest = x[..., :pairs], x[..., pairs:2 * pairs], x[..., 2 * pairs:]
    m = (a.square() + b.square()).sqrt()
    return torch.cat([a * c - b * s, a * s + b * c, rest], -1), 2.0 ** -19 * torch.cat([m, m, rest.abs()], -1)
