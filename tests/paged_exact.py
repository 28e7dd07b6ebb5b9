"""The paged decode in 64 bits on the device, with an error bound for every output element, and
inputs whose attention weights need all 24 bits of fp32."""
import math

import numpy as np

from paged_helpers import torch_mod


def attend_rows(q, k, v, ak, av, scale, steps):
    """q [g][d] over k, v [n][d] in fp64; ak, av: magnitudes |K~|, |V~| as mixed. Returns out, lse and bounds.

    Scores: at most 20 accumulation, mixing and scaling steps, each off by at most 2^-22 of the sum of
    magnitudes S_t of that row. Weight t is off by its own score's error and, through the normaliser,
    by the weighted mean of all of them; exp2 in weight and normaliser by 2^-22 each, twice (within a
    warp's share and between shares); a tile's products sum in up to 4 tensor-core steps of 2^-22 of
    their magnitudes; `steps` fp32 half steps for rescaling and joining, output and normaliser alike.
    """
    torch = torch_mod()
    z = (q @ k.T) * scale
    lse = torch.logsumexp(z, dim=1)
    p = torch.exp(z - lse[:, None])
    dz = 20 * 2.0 ** -22 * (q.abs() @ ak.T) * scale
    rel = dz + (p * dz).sum(1, keepdim=True) + 4 * 2.0 ** -22 + 2 * steps * 2.0 ** -24
    bound = (p * rel) @ av + 4 * 2.0 ** -22 * (p @ av)
    # log2 and the scale to natural units: 2^-19 and 4 half steps of the value
    lse_bound = (p * dz).sum(1) + 2 * 2.0 ** -22 + steps * 2.0 ** -24 + 2.0 ** -19 + lse.abs() * 2.0 ** -22
    return p @ v, lse, bound, lse_bound


def exact_decode(pool, q, layer_map, w=None, selected=None, steps=0, scale=None):
    """out, lse and their bounds [L][B][Hq]([d]) of a decode of `pool`; selected [L][B][Hkv][top] or None."""
    torch = torch_mod()
    L, B, Hq, d = q.shape
    g, page = Hq // pool.Hkv, pool.page
    scale = float(np.float32(1.0 / math.sqrt(d))) if scale is None else scale
    out, bound = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    lbound = torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    for l, (kind, s0, s1) in enumerate(layer_map):
        mix = kind == pool.K.KVS_SRC_MIX
        for b in range(B):
            n = int(pool.lens[b])
            if n == 0:
                continue
            held = -(-n // page)
            for j in range(pool.Hkv):
                blocks = np.arange(held) if selected is None else selected[l][b][j]
                at = (blocks[blocks >= 0][:, None] * page + np.arange(page)).reshape(-1)
                at = torch.from_numpy(at[at < n]).cuda()
                pages = torch.from_numpy(pool.table[b, :held]).cuda().long()[at // page]

                def rows(x):
                    a = x[s0, pages, j, at % page].double()
                    if not mix:
                        return a, a.abs()
                    wj, w1 = float(np.float32(w[l][j])), float(np.float32(1) - np.float32(w[l][j]))
                    c = x[s1, pages, j, at % page].double()
                    return wj * a + w1 * c, abs(wj) * a.abs() + abs(w1) * c.abs()
                (kk, ak), (vv, av) = rows(pool.k), rows(pool.v)
                h = slice(j * g, (j + 1) * g)
                out[l, b, h], lse[l, b, h], bound[l, b, h], lbound[l, b, h] = \
                    attend_rows(q[l, b, h].double(), kk, vv, ak, av, scale, steps)
    return out, lse, bound, lbound


def check_exact(out, lse, want, what):
    torch = torch_mod()
    o, s, ob, sb = want
    assert torch.isfinite(out).all(), what
    over = (out.double() - o).abs() / ob.clamp_min(1e-300)
    assert ((out.double() - o).abs() <= ob).all(), f"{what}: {over.max().item():.2f} of an element's bound"
    empty = torch.isinf(s)
    assert torch.equal(torch.isneginf(lse), empty), what
    assert ((lse.double() - s).abs()[~empty] <= sb[~empty]).all(), what


# ---- inputs with exact scores and weights of 24 bits: scale ln 2, so that a weight is 2^score;
# scores in (-2, 0] on a grid of 1/32, exact in any order; token t's value is 1 in channel t alone
# (and 0 elsewhere), so output channel t is weight t itself
WEIGHT_SCALE = float(np.float32(math.log(2.0)))
WEIGHT_LENS = [2, 5, 16, 17, 33, 1, 24]


def weight_keys(n):
    """The two key channels in use, [n][2], negated steps: the first token of every 16 scores 0."""
    t = np.arange(n)
    k = -np.stack([t % 2, (5 * t) % 8], axis=1).astype(np.float64)
    k[t % 16 == 0] = 0
    return k


def weight_queries(g):
    return np.stack([np.ones(g), (1 + np.arange(g) % 4) / 32.0], axis=1)


def weights_exact(n, g):
    """[g][n] weights in 64 bits."""
    p = np.exp2((weight_queries(g) @ weight_keys(n).T) * (WEIGHT_SCALE / math.log(2.0)))
    return p / p.sum(1, keepdims=True)


# relative error of an output that is one weight: exp2 at most 2^-22 off, twice in the weight and twice
# in the normaliser (rescaling between shares); the normaliser's sum (12 half steps at most: a lane's
# rows, three exchanges, a warp's few tiles, the joins), its reciprocal, the product, the mixed
# weight's own rounding and one more of the sum of two sources, 16 in all: (16 + 16) half steps
WEIGHT_TOL = 32 * 2.0 ** -24
