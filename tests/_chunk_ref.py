"""Problems for the chunk attention, and its definition in 64 bits (torch, CPU).

Tolerance, per output element (derived, not fitted):

    half * |ref|                                one rounding to the output type (half an ulp: fp16 2^-11, bf16 2^-8)
  + p_err * cond                                probabilities rounded to fp16: 2^-11 each
  + (N/16 + 32) 2^-23 * cond                    FP32 PV sums: one truncation (2^-23) per K16 step of N tokens, and 32
                                                for the weights (ex2.approx 2^-22, its argument), joins, normalisation
  + (D/16 + 16) 2^-23 * cond_qk                 FP32 logits: one truncation per K16 step of D, and 16 for the scaling
  + N 2^-31 max|V| + 2^-25                      probabilities and outputs in the fp16 subnormal range

with cond = v_scale sum_j w_j |V_j| and cond_qk = sum_j w_j a_j |v_scale V_j - out|, a_j the scaled sum of |q_d k_jd|
(the first-order change of the output under logit errors relative to a_j).
"""

from dataclasses import dataclass, field

import numpy as np
import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
POISON = {"e4m3": 0x7F, "e5m2": 0x7E}  # NaN codes


def decode_table(fmt):
    kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    return torch.arange(256, dtype=torch.int32).to(torch.uint8).view(kind).double()


@dataclass
class Case:
    requests: list  # (new tokens, positions with them)
    Hq: int = 4
    Hkv: int = 2
    D: int = 128
    page: int = 16
    window: int = 0
    sinks: int = 0
    dtype: torch.dtype = torch.float16
    fmt: str = "e4m3"
    softmax_scale: float = None
    k_scale: float = 0.02
    v_scale: float = 0.5
    seed: int = 0
    q_scale: float = 1.0
    extra_rows: int = 0       # rows of q behind the last request
    k: torch.Tensor = field(default=None, repr=False)

    def __post_init__(self):
        g = torch.Generator().manual_seed(self.seed + 1000)
        B, G = len(self.requests), self.Hq // self.Hkv
        self.softmax_scale = self.D ** -0.5 if self.softmax_scale is None else self.softmax_scale
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in self.requests])]).astype(np.int32)
        self.total = int(self.cu[-1]) + self.extra_rows
        self.max_q = max([n for n, _ in self.requests] + [1])
        self.max_kv = max([kv for _, kv in self.requests] + [1])
        self.cols = -(-self.max_kv // self.page)
        self.blocks = 1 + B * self.cols
        self.q = (torch.randn(self.total, self.Hq, self.D, generator=g) * self.q_scale).to(self.dtype)
        kind = torch.float8_e4m3fn if self.fmt == "e4m3" else torch.float8_e5m2
        shape = (self.blocks, self.page, self.Hkv, self.D)
        # K of unit variance after its scale, V of two
        self.k = (torch.randn(shape, generator=g) / self.k_scale).clamp(-FMAX[self.fmt], FMAX[self.fmt]).to(kind).view(torch.uint8)
        self.v = (torch.randn(shape, generator=g) / 0.25).to(kind).view(torch.uint8)
        self.table = (1 + torch.randperm(B * self.cols, generator=g)).to(torch.int32).view(B, self.cols) if B else \
            torch.zeros(0, self.cols, dtype=torch.int32)
        self.kv_len = np.array([kv for _, kv in self.requests], dtype=np.int32)
        self.group = G
        # poison every slot that no new token may see
        keep = torch.zeros(self.blocks, self.page, dtype=torch.bool)
        for b, (n, kv) in enumerate(self.requests):
            if n == 0:
                continue
            for t in self.seen(n, kv):
                keep[self.table[b, t // self.page].long(), t % self.page] = True
        self.k[~keep] = POISON[self.fmt]
        self.v[~keep] = POISON[self.fmt]

    def seen(self, n, kv):
        t = np.arange(max(kv, 0))
        if self.window:
            t = t[(t >= kv - n - self.window + 1) | (t < self.sinks)]
        return t

    def reference(self, bad_blocks=()):
        """(out, tolerance without the P term, cond): float64 [total][Hq][D]; rows behind the last request NaN."""
        tab = decode_table(self.fmt)
        shape = (self.total, self.Hq, self.D)
        out, tol, cond = (torch.full(shape, float("nan"), dtype=torch.float64) for _ in range(3))
        vs, z_scale = float(np.float32(self.v_scale)), float(np.float32(self.softmax_scale)) * float(np.float32(self.k_scale))
        for b, (n, kv) in enumerate(self.requests):
            if n == 0:
                continue
            rows = slice(int(self.cu[b]), int(self.cu[b]) + n)
            t = torch.from_numpy(self.seen(n, kv)).long()
            blk = self.table[b].long()[t // self.page]
            there = torch.tensor([int(x) not in bad_blocks for x in blk], dtype=torch.bool)
            at = kv - n + torch.arange(n)
            sees = (t[None] <= at[:, None]) & there[None]
            if self.window:
                sees &= (at[:, None] - t[None] < self.window) | (t[None] < self.sinks)
            blk = torch.where(there, blk, 0)
            for h in range(self.Hq):
                g = h // self.group
                K, V = (tab[c[blk, t % self.page, g].long()] for c in (self.k, self.v))
                K = torch.where(there[:, None], K, 0.0)
                q = self.q[rows, h].double()
                z = torch.full((n, t.numel()), -float("inf"), dtype=torch.float64)
                zz = (q @ K.T) * z_scale
                z = torch.where(sees, zz, z)
                w = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-1e300)) if t.numel() else z
                s = w.sum(-1, keepdim=True)
                w = torch.where(s == 0, 0.0, w / s)  # a NaN logit makes the row NaN
                wv = torch.where(sees, w, 0.0)
                any_bad = not bool(torch.isfinite(V).all())
                if any_bad:  # a non-finite V reaches exactly the rows that see it
                    o = torch.zeros(n, self.D, dtype=torch.float64)
                    for i in range(n):
                        o[i] = (wv[i, sees[i], None] * V[sees[i]]).sum(0)
                else:
                    o = wv @ V
                o = o * vs
                out[rows, h] = o
                Vf = torch.nan_to_num(V, nan=0.0, posinf=0.0, neginf=0.0)
                c = (wv @ Vf.abs()) * vs
                a = (q.abs() @ torch.nan_to_num(K).abs().T) * abs(z_scale)
                of = torch.nan_to_num(o, nan=0.0, posinf=0.0, neginf=0.0)
                cq = torch.einsum("ij,ijd->id", torch.nan_to_num(wv) * a, (vs * Vf[None] - of[:, None]).abs()) \
                    if t.numel() * n * self.D < 6e7 else (torch.nan_to_num(wv) * a).sum(-1, keepdim=True) * 2 * vs * (
                        float(Vf.abs().max()) if t.numel() else 0.0)
                N = t.numel()
                vmax = float(Vf.abs().max()) * vs if N else 0.0
                tol[rows, h] = HALF[self.dtype] * of.abs() + (N / 16 + 32) * 2.0 ** -23 * c + \
                    (self.D / 16 + 16) * 2.0 ** -23 * cq + N * 2.0 ** -31 * vmax + 2.0 ** -25
                cond[rows, h] = c
        return out, tol, cond
