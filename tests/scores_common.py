"""Scores that the caches hold exactly, for the tests of the running maxima.

A score is a multiple of 1/8 below 128, written in binary over ten dimensions of
the key (one power of two or nothing each, with the score's sign); the query has
one power of two in all of them.  Products and sums are then exact in bf16, fp16
and e4m3 whatever the order, and what is left is small (see `bound`): a sum that
is scaled wrongly, or not at all, lies far outside.
"""
import math

import torch

U = 2.0 ** -24
DIGITS = 10
FACTORS = (1.0, 0.5, 2.0, 1.0)    # query heads
TILE = 128


def keys(z, hd):
    """Scores z [T] (multiples of 1/8) as key rows [T, hd]."""
    z = z.double()
    k = torch.zeros((z.numel(), hd), dtype=torch.float64, device=z.device)
    units = (z.abs() * 8).round()
    assert torch.equal(units / 8, z.abs()) and float(units.max()) < 2 ** DIGITS
    for i in range(DIGITS):
        k[:, i] = torch.floor(units / 2 ** i) % 2 * 2.0 ** (i - 3) * z.sign()
    return k


def rows(shape, hd, gen, device="cpu"):
    """Query rows [*shape, heads, hd] in bf16: a head's factor in the digits'
    dimensions, anything behind them (the keys are zero there)."""
    q = torch.randn((*shape, len(FACTORS), hd), generator=gen).to(device)
    for h, f in enumerate(FACTORS):
        q[..., h, :DIGITS] = f
    return q.to(torch.bfloat16)


KINDS = ("rising 5.5", "rising 5.625", "rising 2.75", "rising 2.875", "rising 11", "falling 5.625", "first", "middle", "last", "far", "even")


def scores(kind, T, gen, low=-12.0, high=-6.0):
    """Scores of T positions, multiples of 1/8: what rises does so from tile to tile by a
    step just below or above those that move a reference (8 bits are 5.545, 4 bits 2.773), at
    positions behind a tile's first 16."""
    z = torch.randint(int(low * 8), int(high * 8) + 1, (T,), generator=gen).double() / 8
    tiles = -(-T // TILE)
    at = [min(T - 1, TILE * i + 16 + int(torch.randint(0, TILE - 16, (1,), generator=gen))) for i in range(tiles)]
    name, _, step = kind.partition(" ")
    if name == "rising":
        for i, t in enumerate(at):
            z[t] = float(step) * (i % 6)
    elif name == "falling":
        for i, t in enumerate(at):
            z[t] = float(step) * (5 - i % 6)
    elif name in ("first", "middle", "last"):
        z[at[{"first": 0, "middle": tiles // 2, "last": tiles - 1}[name]]] = 40.0
        z[at[tiles // 2] - 3] = 39.0
    elif name == "far":
        z = torch.randint(-60 * 8, 60 * 8, (T,), generator=gen).double() / 8
    return z


def bound(ref, mass, largest, T, step):
    """ref, mass = sum p |v|: a score of `largest` at most is off by the roundings
    of the scale, of the product and of the reference (8 u of it and of 64 bits),
    its exponential by that and 4 u, and the sum that divides by as much; a
    probability is rounded by `step` of itself; the weighted sum adds 2 T + 200
    roundings; the result rounds to bf16."""
    rel = 2 * 8 * U * (largest + 64) + (2 * T + 200) * U + step
    return rel * mass + 2.0 ** -8 * (ref.abs() + rel * mass)


def plain(z, v):
    """Softmax of z [.., T] over v [T, hd] in 64 bits, and sum p |v|."""
    p = torch.softmax(z, -1)
    return p @ v, p @ v.abs()


def by_tiles(z, v, slack, mistake):
    """The same tile by tile with a reference that moves when a score lies more than
    `slack` above it, and one mistake at its last move: the accumulator is not
    scaled, or the sum is not, or only the accumulator's second half is.  With it,
    whether there was such a move."""
    tiles = range(0, len(z), TILE)
    moves, m = [], -math.inf
    for i in tiles:
        top = float(z[i:i + TILE].max())
        if top > m + slack:
            moves.append(i)
            m = top
    last = moves[-1] if len(moves) > 1 else -1
    l, o, m = 0.0, torch.zeros(v.shape[1], dtype=torch.float64), -math.inf
    for i in tiles:
        if i in moves:
            top = float(z[i:i + TILE].max())
            f = math.exp(m - top)
            l *= 1.0 if i == last and mistake == "sum" else f
            o[len(o) // 2:] *= 1.0 if i == last and mistake == "accumulator" else f
            o[:len(o) // 2] *= 1.0 if i == last and mistake in ("accumulator", "half") else f
            m = top
        p = torch.exp(z[i:i + TILE] - m)
        l += float(p.sum())
        o += p @ v[i:i + TILE]
    return o / l, last > 0
