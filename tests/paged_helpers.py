"""Inputs and oracle runs shared by the paged GPU tests."""
import numpy as np

import oracle.paged_ref as paged


def torch_mod():
    import torch
    return torch


class Pool:
    """A paged cache on the device with the same values in fp64 on the host; every row that no
    sequence holds is NaN."""

    def __init__(self, K, dtype, slots, Hkv, page, d, lens, seed, max_blocks=None, spare=3, bounds=False):
        torch = torch_mod()
        self.K, self.page, self.Hkv, self.d, self.slots = K, page, Hkv, d, slots
        self.lens = np.asarray(lens, dtype=np.int32)
        self.tdt = torch.float32 if dtype == "f32" else torch.bfloat16
        B = len(lens)
        P = max_blocks or max(1, -(-int(self.lens.max()) // page))
        held = [-(-int(n) // page) for n in self.lens]
        N = sum(held) + spare
        rng = np.random.default_rng(seed)
        ids = rng.permutation(N)
        self.table = np.full((B, P), -7, dtype=np.int32)       # never read past a sequence's blocks
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = ids[at:at + h]
            at += h
        live = np.zeros((N, page), bool)
        for b, n in enumerate(self.lens):
            for t in range(int(n)):
                live[self.table[b, t // page], t % page] = True
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def draw():
            x = torch.randn(slots, N, Hkv, page, d, generator=gen, device="cuda").to(self.tdt)
            return x.masked_fill(~torch.from_numpy(live).cuda()[None, :, None, :, None], float("nan"))
        self.k, self.v = draw(), draw()
        self.num_pages = N
        self.block_table = torch.from_numpy(self.table).cuda()
        self.lengths = torch.from_numpy(self.lens).cuda()
        self.codes = self.scales = None
        if bounds:
            c = np.full((slots, N, Hkv, 2, d), 99, np.int8)
            s = np.full((slots, N, Hkv), np.nan, np.float32)
            k = self.k.double().cpu().numpy()
            for b, n in enumerate(self.lens):
                for blk in range(held[b]):
                    rows = min(page, int(n) - blk * page)
                    ph = self.table[b, blk]
                    for sl in range(slots):
                        for j in range(Hkv):
                            c[sl, ph, j], s[sl, ph, j] = paged.bounds(k[sl, ph, j, :rows])
            self.hcodes, self.hscales = c, s
            self.codes, self.scales = torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()

    def pages(self, **kw):
        f = dict(k=self.k, v=self.v, block_table=self.block_table, lengths=self.lengths, bound_codes=self.codes,
                 bound_scale=self.scales)
        f.update(kw)
        return self.K.Pages(**f)

    def host(self):
        return self.k.double().cpu().numpy(), self.v.double().cpu().numpy()


def oracle_decode(pool, q, layer_map, w=None, selected=None, lens=None, table=None):
    """q [L][B][Hq][d] fp64; selected [L][B][Hkv][top] or None. Returns out, lse, and an error bound of each."""
    K = pool.K
    k, v = pool.host()
    L, B, Hq, d = q.shape
    g = Hq // pool.Hkv
    lens = pool.lens if lens is None else lens
    table = pool.table if table is None else table
    out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    tol_o, tol_l = 0.0, 0.0
    for l, (kind, s0, s1) in enumerate(layer_map):
        for b in range(B):
            n = int(lens[b])
            for j in range(pool.Hkv):
                blocks = range(-(-n // pool.page)) if selected is None else selected[l][b][j]
                rows = lambda x, s: paged.rows_of(x[s, :, j], table[b], blocks, n, pool.page, pool.num_pages)  # noqa: E731
                kk, vv = rows(k, s0), rows(v, s0)
                if kind == K.KVS_SRC_MIX:
                    wj = float(np.float32(w[l][j]))
                    w1 = float(np.float32(1) - np.float32(w[l][j]))
                    ak = np.abs(wj * kk) + np.abs(w1 * rows(k, s1))
                    av = np.abs(wj * vv) + np.abs(w1 * rows(v, s1))
                    kk, vv = wj * kk + w1 * rows(k, s1), wj * vv + w1 * rows(v, s1)
                else:
                    ak, av = np.abs(kk), np.abs(vv)
                h = slice(j * g, (j + 1) * g)
                scale = float(np.float32(1.0 / np.sqrt(np.float32(d))))
                out[l, b, h], lse[l, b, h] = paged.attend(q[l, b, h], kk, vv, scale)
                if len(kk):
                    # scores: at most 16 accumulation steps, each off by at most 2^-22 of the sum of
                    # magnitudes S (tensor-core steps truncate), and the scale's own half step
                    S = (np.abs(q[l, b, h]) @ ak.T).max() * scale
                    ds = 20 * 2.0 ** -22 * S
                    # weights: the scores' error twice (weight and normaliser), exp2 to 2^-21, the parts
                    # of p to 2^-23; sums over the tiles and joins in fp32: 64 half steps cover them
                    rel = 2 * ds + 2.0 ** -21 + 2.0 ** -23 + 64 * 2.0 ** -24
                    tol_o = max(tol_o, rel * av.max())
                    tol_l = max(tol_l, ds + 2.0 ** -19 + np.abs(lse[l, b, h]).max() * 2.0 ** -22)
    return out, lse, tol_o, tol_l


def check(got_out, got_lse, want, what):
    out, lse, to, tl = want
    o, s = got_out.double().cpu().numpy(), got_lse.double().cpu().numpy()
    assert np.all(np.isfinite(o)), f"{what}: non-finite output"
    assert np.abs(o - out).max() <= to, f"{what}: {np.abs(o - out).max():.3e} > {to:.3e}"
    assert np.array_equal(np.isneginf(s), np.isneginf(lse)), what
    live = ~np.isneginf(lse)
    assert not live.any() or np.abs(s[live] - lse[live]).max() <= tl, f"{what}: lse {np.abs(s[live] - lse[live]).max():.3e} > {tl:.3e}"
