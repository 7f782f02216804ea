"""Plain 64-bit forms of the paged cache's operators and of the token log
probabilities, for the GPU tests.  They share no code with the library.

Tolerances follow from the roundings.  u = 2^-24 is the fp32 half step; a
value rounded to bf16 is off by at most 2^-8 of itself, to e4m3 by at most
2^-4 of itself or 2^-10 scales (below the smallest normal code).
"""
import math

import torch

U = 2.0 ** -24


def turn(x, gain, pos, theta, eps=1e-6):
    """rope(rmsnorm(x)) in 64 bits: x [..., m, heads, hd] at positions pos [m]."""
    x = x.double()
    hd = x.shape[-1]
    if gain is not None:
        x = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * gain.double()
    if theta > 0:
        f = theta ** (-torch.arange(hd // 2, device=x.device, dtype=torch.float64) * 2 / hd)
        ang = pos.double()[:, None] * f
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        a, b = x[..., : hd // 2], x[..., hd // 2:]
        x = torch.cat([a * c - b * s, a * s + b * c], -1)
    return x


def turn_tol(x):
    """Bound of the fp32 error of turn(): the norm's sum of hd squares is 16
    products a thread and 5 sums between threads (21 u, half of it on the
    root), root, quotient, two products (4 u), cos and sin at 2 units in the
    last place and 2 u from the angle (6 u), two roundings of the rotation:
    below 32 u = 2^-19 of the pair's magnitude."""
    h = x.shape[-1] // 2
    m = (x[..., :h].square() + x[..., h:].square()).sqrt()
    return 2.0 ** -19 * torch.cat([m, m], -1)


def pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s, within [2^-40, 2^40]."""
    if not amax > 0:
        return 2.0 ** -40
    k = math.ceil(math.log2(amax / 448))
    while amax > 448 * 2.0 ** k:
        k += 1
    while amax <= 448 * 2.0 ** (k - 1):
        k -= 1
    return 2.0 ** max(-40, min(40, k))


def attended(p, window, sink):
    """The positions a row at position p attends, ascending."""
    lo = max(0, p + 1 - window) if window else 0
    return list(range(min(sink, lo))) + list(range(lo, p + 1))


class Pool:
    """A paged cache on the GPU: pages handed out in random order, everything
    not written NaN."""

    def __init__(self, B, max_pages, page, hkv, hd, dtype, seed, layout="head", spare=2):
        g = torch.Generator().manual_seed(seed)
        n = B * max_pages + spare
        tdt = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[dtype]
        self.dtype, self.page, self.hkv, self.hd, self.B, self.max_pages = dtype, page, hkv, hd, B, max_pages

        def buf():
            shape = (n, hkv, page, hd) if layout == "head" else (n, page, hkv, hd)
            if dtype == "e4m3":
                t = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(tdt)
            else:
                t = torch.full(shape, float("nan"), dtype=tdt, device="cuda")
            return t if layout == "head" else t.permute(0, 2, 1, 3)

        self.k, self.v = buf(), buf()
        self.ks = torch.full((n, hkv), float("nan"), device="cuda") if dtype == "e4m3" else None
        self.vs = torch.full((n, hkv), float("nan"), device="cuda") if dtype == "e4m3" else None
        self.table = torch.randperm(n, generator=g)[: B * max_pages].view(B, max_pages).to(torch.int32).cuda()

    def handle(self, **kw):
        import mtp_speculative_decoding_gb300 as mtp
        return mtp.make_kv_cache(self.k, self.v, self.table, self.ks, self.vs, **kw)

    def rows(self, w, b, positions):
        """Cached rows of sequence b in 64 bits: [heads, positions, hd]."""
        t = torch.as_tensor(positions, device="cuda", dtype=torch.long)
        pg = self.table[b].long()[t // self.page]
        x = getattr(self, w)[pg, :, t % self.page].double()
        if self.dtype == "e4m3":
            x = x * getattr(self, w + "s")[pg].double()[..., None]
        return x.transpose(0, 1)

    def fill(self, lens, seed, std=1.0):
        """Positions [0, lens[b]) hold N(0, std^2) (e4m3: codes and scales of their own)."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        for w in "kv":
            for b, n in enumerate(lens):
                for p in range(0, n, self.page):
                    m = min(self.page, n - p)
                    pg = int(self.table[b, p // self.page])
                    x = torch.randn(self.hkv, m, self.hd, device="cuda", generator=g) * std
                    t = getattr(self, w)
                    if self.dtype == "e4m3":
                        s = torch.exp2(torch.randint(-8, -5, (self.hkv,), device="cuda", generator=g).float())
                        getattr(self, w + "s")[pg] = s
                        x = (x / s[:, None, None]).clamp(-448, 448)
                        t.view(torch.uint8)[pg, :, :m] = x.to(torch.float8_e4m3fn).view(torch.uint8)
                    else:
                        t[pg, :, :m] = x.to(t.dtype)


def attention(pool, q, gain, lens, n_new, theta, window=0, sink=0, scale=None, absent=None):
    """Rows' attention in 64 bits and, per row, Sum p |v| and the largest
    Sum |q k| (for the error bounds).  absent: set of (b, position) masked."""
    B, M, hq, hd = q.shape
    G = hq // pool.hkv
    scale = 1 / math.sqrt(hd) if scale is None else scale
    out = torch.zeros(B, M, hq, hd, dtype=torch.float64, device="cuda")
    mass = torch.zeros_like(out)
    dots = torch.zeros(B, M, hq, dtype=torch.float64, device="cuda")
    for b in range(B):
        for j in range(n_new[b]):
            p = lens[b] + j
            see = [t for t in attended(p, window, sink) if not absent or (b, t) not in absent]
            if not see:
                continue
            qq = turn(q[b, j:j + 1], gain, torch.tensor([p], device="cuda"), theta)[0].view(pool.hkv, G, hd)
            k, v = pool.rows("k", b, see), pool.rows("v", b, see)
            z = torch.einsum("hgd,htd->hgt", qq, k) * scale
            pr = torch.softmax(z, -1)
            out[b, j] = torch.einsum("hgt,htd->hgd", pr, v).reshape(hq, hd)
            mass[b, j] = torch.einsum("hgt,htd->hgd", pr, v.abs()).reshape(hq, hd)
            dots[b, j] = torch.einsum("hgd,htd->hgt", qq.abs(), k.abs()).amax(-1).reshape(hq) * scale
    return out, mass, dots


def attention_tol(ref, mass, dots, hd, T, low):
    """low False, everything fp32: a score is off by at most (hd + 40) u of
    Sum |q k| (products and sums of hd terms, and turn()'s 32 u on q), its
    exponential by that and 4 u, and the same for the sum that divides; the
    weighted sum adds T + 64 roundings.  low True, the tensor cores: q keeps
    16 bits or more (2^-16) and the products accumulate in fp32 with a
    truncation each (2 u a term), the probabilities keep a half step of bf16
    (2^-8 of each, so 2^-8 of Sum p |v|), and the result rounds to bf16."""
    ds = dots[..., None] * ((2 * hd + 80) * U + 2.0 ** -16 if low else (hd + 40) * U)
    rel = 2 * ds + (2 * T + 200) * U
    if low:
        return (2.0 ** -8 + rel) * mass + 2.0 ** -8 * (ref.abs() + (2.0 ** -8 + rel) * mass)
    return rel * mass + U * ref.abs()
