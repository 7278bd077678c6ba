"""Problems for the tree attention, and its definition in 64 bits (torch, CPU).

The tolerance is that of the chunk attention (tests/_chunk_ref.py): the same
sums over the positions that a row sees.
"""

from dataclasses import dataclass

import numpy as np
import torch

from tests._chunk_ref import HALF, POISON, Case, decode_table


def random_tree(n, gen):
    """Parents of n nodes, each behind its parent."""
    pick = torch.rand(max(n, 1), generator=gen).tolist()
    return [-1] + [int(pick[i] * i) for i in range(1, n)]


def ancestors(parents):
    """What each node sees (its ancestors and itself), as truth values, and its depth."""
    n = len(parents)
    sees, depth = np.zeros((n, n), dtype=bool), np.zeros(n, dtype=np.int32)
    for i, p in enumerate(parents):
        if p >= 0:
            sees[i], depth[i] = sees[p], depth[p] + 1
        sees[i, i] = True
    return sees, depth


def words_of(sees, words):
    """Truth values [n][n] as 32-bit words."""
    bits = np.zeros((sees.shape[0], 32 * words), dtype=np.uint64)
    bits[:, :sees.shape[1]] = sees
    w = (bits.reshape(-1, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)


@dataclass
class TreeCase(Case):
    masks: list = None   # per request: truth values [n][n]; None: random trees
    depths: list = None  # per request: [n]
    spare: int = 1       # words of a mask row beyond those needed, all ones

    def __post_init__(self):
        g = torch.Generator().manual_seed(self.seed + 77)
        if self.masks is None:
            both = [ancestors(random_tree(n, g)) if n else (np.zeros((0, 0), bool), np.zeros(0, np.int32))
                    for n, _ in self.requests]
            self.masks = [x for x, _ in both]
            self.depths = [d for _, d in both]
        if self.depths is None:
            self.depths = [np.zeros(n, dtype=np.int32) for n, _ in self.requests]
        super().__post_init__()
        need = -(-self.max_q // 32)
        self.words = need + self.spare
        self.mask = np.full((self.total, self.words), -1, dtype=np.int32)
        self.depth = np.zeros(self.total, dtype=np.int32)
        for b, (n, kv) in enumerate(self.requests):
            rows = slice(int(self.cu[b]), int(self.cu[b]) + n)
            full = np.ones((n, 32 * self.words), dtype=bool)  # bits past the last node are ignored
            full[:, :n] = self.masks[b]
            self.mask[rows] = words_of(full, self.words)
            self.depth[rows] = self.depths[b]
            if n:
                unseen = torch.from_numpy(np.flatnonzero(~self.sees(b).any(0)))
                blk = self.table[b].long()[unseen // self.page]
                self.k[blk, unseen % self.page] = POISON[self.fmt]
                self.v[blk, unseen % self.page] = POISON[self.fmt]

    def sees(self, b):
        """Truth values [n][kv] of a request."""
        n, kv = self.requests[b]
        t, base = np.arange(max(kv, 0)), kv - n
        out = np.broadcast_to(t < base, (n, t.size)).copy()
        if self.window:
            at = base + np.clip(self.depths[b], 0, max(n - 1, 0))[:, None]
            out &= (at - t < self.window) | (t < self.sinks)
        nodes = t >= base
        out[:, nodes] = self.masks[b][:, t[nodes] - base]
        return out

    def reference(self, bad_blocks=()):
        """(out, tolerance without the P term, cond): float64 [total][Hq][D]; rows behind the last request NaN."""
        tab = decode_table(self.fmt)
        shape = (self.total, self.Hq, self.D)
        out, tol, cond = (torch.full(shape, float("nan"), dtype=torch.float64) for _ in range(3))
        vs = float(np.float32(self.v_scale))
        z_scale = float(np.float32(self.softmax_scale)) * float(np.float32(self.k_scale))
        for b, (n, kv) in enumerate(self.requests):
            if n == 0:
                continue
            rows = slice(int(self.cu[b]), int(self.cu[b]) + n)
            t = torch.arange(max(kv, 0))
            blk = self.table[b].long()[t // self.page]
            there = torch.tensor([int(x) not in bad_blocks for x in blk], dtype=torch.bool)
            sees = torch.from_numpy(self.sees(b)) & there[None]
            some = sees.any(0)  # positions that no row sees do not enter the arithmetic
            t, blk, sees = t[some], blk[some], sees[:, some]
            N = int(sees.sum(1).max()) if n else 0
            for h in range(self.Hq):
                K, V = (tab[c[blk, t % self.page, h // self.group].long()] for c in (self.k, self.v))
                q = self.q[rows, h].double()
                z = torch.where(sees, (q @ K.T) * z_scale, -float("inf"))
                w = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-1e300)) if t.numel() else z
                s = w.sum(-1, keepdim=True)
                w = torch.where(s == 0, 0.0, w / s)  # a NaN logit makes the row NaN
                wv = torch.where(sees, w, 0.0)
                if bool(torch.isfinite(V).all()):
                    o = wv @ V
                else:  # a non-finite V reaches exactly the rows that see it
                    o = torch.stack([(wv[i, sees[i], None] * V[sees[i]]).sum(0) for i in range(n)])
                o = o * vs
                out[rows, h] = o
                Vf = torch.nan_to_num(V, nan=0.0, posinf=0.0, neginf=0.0)
                of = torch.nan_to_num(o, nan=0.0, posinf=0.0, neginf=0.0)
                c = (torch.nan_to_num(wv) @ Vf.abs()) * vs
                # (a logit that is not finite has no error: its weight is exactly 0, or the row is NaN)
                a = (q.abs() @ torch.nan_to_num(K, nan=0.0, posinf=0.0, neginf=0.0).abs().T) * abs(z_scale)
                cq = torch.einsum("ij,ijd->id", torch.nan_to_num(wv) * a, (vs * Vf[None] - of[:, None]).abs()) \
                    if t.numel() * n * self.D < 6e7 else (torch.nan_to_num(wv) * a).sum(-1, keepdim=True) * 2 * vs * \
                    float(Vf.abs().max())
                vmax = float(Vf.abs().max()) * vs if t.numel() else 0.0
                tol[rows, h] = HALF[self.dtype] * of.abs() + (N / 16 + 32) * 2.0 ** -23 * c + \
                    (self.D / 16 + 16) * 2.0 ** -23 * cq + N * 2.0 ** -31 * vmax + 2.0 ** -25
                cond[rows, h] = c
        return out, tol, cond
