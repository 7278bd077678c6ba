"""GPU parity of the gathered attention weights (fp8kv_attn_cache_score) with their definition in 64 bits.

Tolerance, per position t of a KV head (derived, not fitted), over the rows r that see it:

    sum_r p_rt [ (D/16 + 16) 2^-23 (a_rt + sum_s p_rs a_rs)   FP32 logits: one truncation per K16 step of D, 16 for the
                                                             scaling; a weight moves by its own logit's error and, through
                                                             the sum, by the mean one
               + (N/64 + 32) 2^-23 ]                         the row's sum of N weights (in chains of N/64 at most), ex2 (2^-22),
                                                             its argument, the quotient
  + (R/64 + 80) 2^-24 sum_r p_rt                             adding R rows: chains of 32, then tiles, then groups
  + 2^-23 |decay score_in| + 2^-120                          one fma; weights in the subnormal range

with a_rt the scaled sum of |q_d k_td|.
"""

import copy
import math

import numpy as np
import pytest
import torch

from tests._chunk_ref import Case, decode_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_e4m3_paged_gb300 import build_lib

    build_lib.build()


def reference(c, before=None, decay=1.0, bad_blocks=()):
    """(score, tolerance): float64 [B][Hkv][max_kv]; NaN where nothing is written."""
    tab = decode_table(c.fmt)
    out, tol = (torch.full((len(c.requests), c.Hkv, c.max_kv), float("nan"), dtype=torch.float64) for _ in range(2))
    z_scale = float(np.float32(c.softmax_scale)) * float(np.float32(c.k_scale))
    for b, (n, kv) in enumerate(c.requests):
        if n == 0 or kv <= 0:
            continue
        rows = slice(int(c.cu[b]), int(c.cu[b]) + n)
        t = torch.arange(kv)
        blk = c.table[b].long()[t // c.page]
        there = torch.tensor([int(x) not in bad_blocks for x in blk], dtype=torch.bool)
        at = kv - n + torch.arange(n)
        sees = (t[None] <= at[:, None]) & there[None]
        blk = torch.where(there, blk, 0)
        for g in range(c.Hkv):
            K = tab[c.k[blk, t % c.page, g].long()]
            Kf = torch.nan_to_num(K, nan=0.0, posinf=0.0, neginf=0.0).abs()
            total, err = torch.zeros(kv, dtype=torch.float64), torch.zeros(kv, dtype=torch.float64)
            for h in range(g * c.group, (g + 1) * c.group):
                q = c.q[rows, h].double()
                z = torch.where(sees, (q @ K.T) * z_scale, -float("inf"))
                top = z.amax(-1, keepdim=True)
                w = torch.where(top == -float("inf"), 0.0, torch.exp(z - top))
                s = w.sum(-1, keepdim=True)
                w = torch.where(s == 0, 0.0, w / s)
                w = torch.where(sees, w, 0.0)
                wf = torch.nan_to_num(w)
                a = (q.abs() @ Kf.T) * abs(z_scale)
                mean = (wf * torch.nan_to_num(a)).sum(-1, keepdim=True)
                err += (wf * ((c.D / 16 + 16) * 2.0 ** -23 * (a + mean) + (kv / 64 + 32) * 2.0 ** -23)).sum(0)
                total += w.sum(0)
            old = torch.zeros(kv, dtype=torch.float64)
            if before is not None:
                old = torch.where(t < kv - n, before[b, g, :kv].double() * float(np.float32(decay)), 0.0)
            out[b, g, :kv] = total + old
            tol[b, g, :kv] = err + (n * c.group / 64 + 80) * 2.0 ** -24 * torch.nan_to_num(total) + \
                2.0 ** -23 * old.abs() + 2.0 ** -120
    return out, tol


class Run:
    def __init__(self, c, kernel=0, num_splits=0, before=None, decay=1.0, spread=False, in_place=False, **over):
        from fp8_e4m3_paged_gb300 import binding as B

        self.B, self.c = B, c
        dev = "cuda"
        self.cu, self.kv_len = torch.from_numpy(c.cu).to(dev), torch.from_numpy(c.kv_len).to(dev)
        self.table = c.table.to(dev)
        q, k = c.q.to(dev), c.k.to(dev)
        self.score = torch.full((len(c.requests), c.Hkv, c.max_kv), -7.0, device=dev)
        self.before = None if before is None else before.to(dev)
        if spread:
            qw = torch.zeros(c.total, c.Hq + 1, c.D + 8, dtype=q.dtype, device=dev)
            qw[:, :c.Hq, :c.D] = q
            q = qw[:, :c.Hq, :c.D]
            both = torch.full((c.blocks, c.page, 2, c.Hkv, c.D), 0x7F, dtype=torch.uint8, device=dev)
            both[:, :, 0] = k
            k = both[:, :, 0]
            self.score = torch.full((len(c.requests), c.Hkv + 1, c.max_kv + 7), -7.0, device=dev)[:, :c.Hkv, 3:3 + c.max_kv]
        if in_place:
            self.score.copy_(self.before)
            self.before = self.score
        self.q, self.k = q, k
        desc = dict(batch=len(c.requests), total_q=c.total, max_q=c.max_q, num_q_heads=c.Hq, num_kv_heads=c.Hkv,
                    head_dim=c.D, page_size=c.page, max_kv_len=c.max_kv, max_blocks=c.cols, num_kv_blocks=c.blocks,
                    dtype=B.DTYPE_F16 if c.dtype == torch.float16 else B.DTYPE_BF16,
                    kv_format=B.KV_E4M3 if c.fmt == "e4m3" else B.KV_E5M2, kernel=kernel, num_splits=num_splits)
        desc.update(over)
        self.plan = B.fp8kv_attn_cache_score_plan(B.make_chunk_desc(**desc))
        self.ws = torch.full((self.plan.workspace_bytes,), 0xFF, dtype=torch.uint8, device=dev)
        self.ws[:4] = 0
        self.args = B.make_cache_score_args(q=q, k_cache=k, block_table=self.table, cu_q=self.cu, kv_len=self.kv_len,
                                            softmax_scale=c.softmax_scale, k_scale=c.k_scale, score=self.score,
                                            score_in=self.before, decay=decay, workspace=self.ws)

    def __call__(self, stream=None):
        s = torch.cuda.current_stream() if stream is None else stream
        self.B.CacheScoreCall(self.plan, self.args).run(s.cuda_stream)
        s.synchronize()
        return self.score.cpu()

    def status(self):
        return int(self.ws[:4].view(torch.int32).item())


def check(got, c, ref, untouched=-7.0):
    out, tol = ref
    for b, (n, kv) in enumerate(c.requests):
        end = kv if n and kv > 0 else 0
        left = untouched if isinstance(untouched, float) else untouched[b, :, end:]
        assert (got[b, :, end:] == left).all(), "positions behind the last one were written"
        g, r, bound = got[b, :, :end].double(), out[b, :, :end], tol[b, :, :end]
        assert torch.equal(torch.isnan(g), torch.isnan(r)), "NaN in other places"
        d = torch.where(torch.isnan(r), 0.0, (g - torch.nan_to_num(r)).abs())
        worst = float((d / bound).nan_to_num().max()) if end else 0.0
        assert worst <= 1.0, f"request {b}: {worst:.3f} of the bound"


def kernels(c):
    tile = [(2, 0), (2, 1), (2, 3), (0, 0)]
    return tile + [(1, 0), (1, 1), (1, 3), (1, 11)] if c.max_q * c.group <= 256 else tile


CASES = {
    "decode": Case([(1, 1), (1, 2), (1, 611), (1, 64), (1, 65), (1, 1023)], Hq=6, Hkv=1, D=256),
    "decode_gqa4": Case([(1, 700), (1, 17), (1, 128), (1, 5000)], Hq=8, Hkv=2, D=128, page=3),
    "decode_gqa8": Case([(1, 700), (1, 17), (1, 129)], Hq=16, Hkv=2, D=128, page=16, dtype=torch.bfloat16),
    "decode_group1": Case([(1, 300), (1, 33)], Hq=3, Hkv=3, D=64, page=5, fmt="e5m2", k_scale=0.001),
    "decode_group12": Case([(1, 333), (1, 1)], Hq=24, Hkv=2, D=128, page=4, dtype=torch.bfloat16),
    "drafts": Case([(3, 130), (4, 4), (2, 777)], Hq=8, Hkv=2, D=64, fmt="e5m2", k_scale=0.001),
    "last_rows": Case([(32, 700), (7, 130), (32, 32), (1, 400)], Hq=8, Hkv=2, D=128),
    "last_rows_bf16": Case([(20, 333), (31, 900)], Hq=16, Hkv=2, D=128, dtype=torch.bfloat16, page=64),
    "wide": Case([(100, 431), (3, 3), (22, 700)], Hq=6, Hkv=1, D=256, page=1728),
    "wide_e5m2": Case([(65, 200), (22, 150)], Hq=4, Hkv=2, D=256, fmt="e5m2", k_scale=0.001, dtype=torch.bfloat16),
    "narrow": Case([(200, 200), (31, 700)], Hq=4, Hkv=4, D=64, page=7),
    "prompt": Case([(700, 700), (300, 2500)], Hq=8, Hkv=2, D=128),
    "prompt_odd_group": Case([(333, 350), (90, 91)], Hq=5, Hkv=1, D=128, page=1),
    "dead_rows": Case([(9, 4), (3, 0), (20, 19), (1, 0)], Hq=4, Hkv=2, D=128),
    "dead_rows_many": Case([(200, 50), (70, 0)], Hq=4, Hkv=2, D=128),
    "empty_requests": Case([(0, 0), (0, 100), (2, 2), (0, 0)], Hq=4, Hkv=2, D=128, extra_rows=5),
    "many_requests": Case([(1 + i % 4, 1 + (i * 37) % 210 + i % 4) for i in range(75)], Hq=2, Hkv=1, D=64),
    "negative_scale": Case([(20, 200), (1, 90)], Hq=4, Hkv=2, D=128, softmax_scale=-0.11),
    "large_logits": Case([(20, 200), (1, 90)], Hq=4, Hkv=2, D=128, q_scale=30.0),
    "page_past_tile": Case([(5, 260)], Hq=4, Hkv=2, D=128, page=256),
}


@pytest.mark.parametrize("name", CASES)
def test_every_kernel(name):
    c = CASES[name]
    ref = reference(c)
    for kernel, S in kernels(c):
        r = Run(c, kernel, S)
        check(r(), c, ref)
        assert r.status() == 0, (kernel, S)


@pytest.mark.parametrize("name", ["decode_gqa4", "last_rows", "prompt", "dead_rows", "empty_requests"])
@pytest.mark.parametrize("in_place", [False, True])
def test_added_to_what_was_gathered(name, in_place):
    c = CASES[name]
    before = torch.rand((len(c.requests), c.Hkv, c.max_kv), generator=torch.Generator().manual_seed(1)) * 9
    for b, (n, kv) in enumerate(c.requests):
        before[b, :, max(kv - n, 0):] = float("nan")  # positions of new tokens start anew, whatever lies there
    ref = reference(c, before, 0.875)
    for kernel, S in kernels(c):
        got = Run(c, kernel, S, before, 0.875, in_place=in_place)()
        left = before if in_place else -7.0
        for b, (n, kv) in enumerate(c.requests):  # (NaN compares with nothing)
            if in_place:
                end = kv if n and kv > 0 else 0
                assert torch.equal(got[b, :, end:].nan_to_num(5.0), before[b, :, end:].nan_to_num(5.0))
                got[b, :, end:] = -7.0
        check(got, c, ref)


@pytest.mark.parametrize("name", ["decode_gqa4", "last_rows", "wide", "narrow"])
def test_strides(name):
    c = CASES[name]
    ref = reference(c)
    for kernel, S in kernels(c):
        check(Run(c, kernel, S, spread=True)(), c, ref)


def test_more_requests_than_shares():
    """Batches whose CTAs do not find their shares from the lengths: partitions of one length."""
    c = Case([(9 + i % 9, 20 + (i * 37) % 150 + 9) for i in range(150)] + [(20, 3000)], Hq=4, Hkv=2, D=64)
    r = Run(c, 2)
    assert r.plan.per_head == 0
    check(r(), c, reference(c))


def test_rows_before_the_first_position():
    """Row blocks whose tokens all stand in front of position 0."""
    c = Case([(2000, 50), (700, 300)], Hq=4, Hkv=2, D=128)
    check(Run(c, 2)(), c, reference(c))


def test_one_long_partition():
    """2^25 positions, all rows' sums in one partition: the column pass waits for the row pass however long that takes, and
    the sums hold.  All positions are in one block of 1024, so position t weighs what t mod 1024 does."""
    from fp8_e4m3_paged_gb300 import binding as B

    L, n, Hq, D, page = 1 << 25, 33, 4, 64, 1024
    gen = torch.Generator().manual_seed(5)
    q = torch.randn(n, Hq, D, generator=gen).half()
    k = torch.randn(1, page, 1, D, generator=gen).to(torch.float8_e4m3fn)
    logits = torch.einsum("nhd,td->nht", q.double(), k[0, :, 0].double()) * 0.125
    # every new token sees all positions in front of them; at most 32 of 2^25 others are not in a token's sum, which
    # moves no weight by more than 33 * 2^-25 times the largest one over the mean
    w = torch.exp(logits - logits.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True) / (L // page)
    want = w.sum((0, 1))
    assert 33 * float((w.amax(-1) / w.mean(-1)).max()) * 2.0 ** -25 < 2.0 ** -12
    plan = B.fp8kv_attn_cache_score_plan(B.make_chunk_desc(
        batch=1, total_q=n, max_q=n, num_q_heads=Hq, num_kv_heads=1, head_dim=D, page_size=page, max_kv_len=L,
        max_blocks=L // page, num_kv_blocks=1, kernel=B.CHUNK_TILE, num_splits=1, num_sms=152))
    assert plan.num_splits == 1 and plan.stat_part >= L
    score = torch.zeros(1, 1, L, device="cuda")
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    args = B.make_cache_score_args(
        q=q.cuda(), k_cache=k.cuda().view(torch.uint8), block_table=torch.zeros(1, L // page, dtype=torch.int32, device="cuda"),
        cu_q=torch.tensor([0, n], dtype=torch.int32, device="cuda"), kv_len=torch.tensor([L], dtype=torch.int32, device="cuda"),
        score=score, workspace=ws, softmax_scale=0.125, k_scale=1.0)
    B.CacheScoreCall(plan, args).run(torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) == 0
    got = score[0, 0, : L - page].view(-1, page).cpu().double()
    # Logits of 64 FP32 products and sums, |z| < 8, base 2 at 2^4 (each term at most 2^-20 in all: 2^-14 with the factor), the
    # exponential 2^-22, sums by the kernel's compensated addition of 32 terms each (2^-19), the positions left out above
    # (2^-12): 2^-11 covers them.
    assert ((got - want).abs() <= 2.0 ** -11 * want).all()


@pytest.mark.parametrize("kernel", [1, 2])
def test_pages_past_32_bits(kernel):
    """Pages 600 MB apart: byte offsets up to 6 GB."""
    from fp8_e4m3_paged_gb300 import binding as B

    c = Case([(5, 60), (1, 40)], Hq=8, Hkv=2, D=128, page=16)
    far = (600 << 20) // 128 * 128
    r = Run(c, kernel)
    pool = torch.empty(c.blocks * far, dtype=torch.uint8, device="cuda")
    assert pool.numel() > 1 << 32
    k = pool.as_strided((c.blocks, 16, 2, 128), (far, 256, 128, 1))
    k.copy_(r.k)
    r.args = B.make_cache_score_args(q=r.q, k_cache=k, block_table=r.table, cu_q=r.cu, kv_len=r.kv_len, score=r.score,
                                     workspace=r.ws, softmax_scale=c.softmax_scale, k_scale=c.k_scale)
    check(r(), c, reference(c))


def test_device_scale():
    from fp8_e4m3_paged_gb300 import binding as B

    for name in ("decode_gqa4", "last_rows"):
        c = CASES[name]
        ref = reference(c)
        scale = torch.tensor([c.k_scale], dtype=torch.float32, device="cuda")
        for kernel in (1, 2):
            r = Run(c, kernel)
            kw = dict(q=r.q, k_cache=r.k, block_table=r.table, cu_q=r.cu, kv_len=r.kv_len, score=r.score, workspace=r.ws,
                      softmax_scale=c.softmax_scale, k_scale=float("nan"), k_scale_dev=scale)
            r.args = B.make_cache_score_args(**kw)
            check(r(), c, ref)
            # a NaN scale: every position that a token sees
            scale.fill_(float("nan"))
            got = r()
            for b, (n, kv) in enumerate(c.requests):
                assert torch.isnan(got[b, :, :kv]).all() and (got[b, :, kv:] == -7.0).all()
            scale.fill_(c.k_scale)


def test_two_calls_at_once():
    """Calls in flight on streams of their own, each with its workspace."""
    c, d = CASES["prompt"], CASES["decode_gqa4"]
    a, b = Run(c, 2), Run(d, 1)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.B.CacheScoreCall(a.plan, a.args).run(s.cuda_stream)
        b.B.CacheScoreCall(b.plan, b.args).run(t.cuda_stream)
    torch.cuda.synchronize()
    check(a.score.cpu(), c, reference(c))
    check(b.score.cpu(), d, reference(d))


def test_calls_in_a_row():
    """The second kernel of a call starts early; the next call on the same buffers starts behind it."""
    for name in ("decode_gqa4", "last_rows", "prompt"):
        c = CASES[name]
        zero = torch.zeros((len(c.requests), c.Hkv, c.max_kv))
        once = Run(c, 0, before=zero)()
        r = Run(c, 0, before=zero.clone(), in_place=True)
        s = torch.cuda.current_stream()
        torch.cuda.synchronize()
        for _ in range(6):
            r.B.CacheScoreCall(r.plan, r.args).run(s.cuda_stream)
        torch.cuda.synchronize()
        got = r.score.cpu()
        for b, (n, kv) in enumerate(c.requests):
            # in front of the new tokens six times the weights (five roundings), at them one time
            want = once[b, :, :kv].double() * torch.where(torch.arange(kv) < kv - n, 6.0, 1.0)
            assert ((got[b, :, :kv].double() - want).abs() <= 6 * 2.0 ** -24 * want).all()


def test_the_same_bits_every_time():
    for name in ("decode_gqa4", "prompt", "wide"):
        r = Run(CASES[name])
        first = r().clone()
        for _ in range(3):
            assert torch.equal(r(), first)


@pytest.mark.parametrize("softmax_scale", [1e4, 1e8])
def test_huge_logits(softmax_scale):
    """Logits of 10^8 and 10^12 (queries and keys are finite: 3000 times five sigma is an fp16 number), so past 2^22,
    where a maximum and its exponents are rounded: nothing turns NaN or infinite."""
    for requests in ([(1, 300), (1, 77)], [(40, 300), (9, 77)]):
        c = Case(requests, Hq=4, Hkv=2, D=128, q_scale=3e3, softmax_scale=softmax_scale)
        for kernel, S in kernels(c):
            got = Run(c, kernel, S)()
            for b, (n, kv) in enumerate(requests):
                x = got[b, :, :kv].double()
                assert torch.isfinite(x).all() and (x >= 0).all()
                # every row's weights sum to 1: each is off by its logit's rounding at most, and those cancel
                # only within what they are, so the sum is held to the rows' number alone
                assert ((x.sum(-1) - n * c.group).abs() < 1e-3 * n * c.group).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_nonfinite_codes(fmt):
    """A NaN logit, or +inf, makes the positions that its row sees NaN, and no others; -inf weighs nothing."""
    for requests in ([(1, 150), (2, 200)], [(12, 150), (70, 200)]):
        base = Case(requests, Hq=4, Hkv=2, D=128, fmt=fmt, k_scale=0.02 if fmt == "e4m3" else 0.001)
        for code in ([0x7F] if fmt == "e4m3" else [0x7E, 0x7C, 0xFC]):
            c = copy.deepcopy(base)
            c.q = c.q.abs() + c.q.new_tensor(2.0 ** -6)  # +inf times q is +inf
            for b, back in ((0, 1), (1, 2)):
                t = requests[b][1] - back  # only the last tokens see it
                c.k[c.table[b, t // c.page].long(), t % c.page, 1, 5] = code
            ref = reference(c)
            for kernel, S in kernels(c):
                r = Run(c, kernel, S)
                got = r()
                out, _ = ref
                for b, (n, kv) in enumerate(requests):
                    g, o = got[b, :, :kv].double(), out[b, :, :kv]
                    t = kv - (1, 2)[b]
                    if code != 0xFC:
                        # (positions whose own logit is -inf do not arise here)
                        assert torch.equal(torch.isnan(g), torch.isnan(o))
                    else:
                        assert torch.isfinite(g).all() and g[1, t] == 0
                if code == 0xFC:
                    check(got, c, ref)


def test_bad_blocks_and_lengths():
    for requests in ([(1, 400), (2, 200)], [(26, 400), (9, 200)]):
        c = Case(requests, Hq=4, Hkv=2, D=128)
        bad = copy.deepcopy(c)
        hidden = [int(c.table[0, 350 // c.page]), int(c.table[1, 195 // c.page])]
        ref = reference(c, bad_blocks=hidden)
        for b, t in ((0, 350), (1, 195)):
            bad.table[b, t // c.page] = 1 << 20 if b else -1
        for kernel, S in kernels(c):
            r = Run(bad, kernel, S)
            check(r(), bad, ref)
            assert r.status() == r.B.STATUS_BAD_BLOCK
            r = Run(c, kernel, S, max_kv_len=300, max_blocks=c.cols)  # kv_len 400 is clamped
            got = r()
            assert r.status() == r.B.STATUS_BAD_LEN
            short = copy.deepcopy(c)
            short.requests = [(requests[0][0], 300), requests[1]]
            check(got, short, reference(short))


def test_replay_on_other_lengths_and_streams():
    for name in ("decode_gqa4", "last_rows"):
        c = CASES[name]
        s = torch.cuda.Stream()
        for kernel in (1, 2) if name == "decode_gqa4" else (2,):
            r = Run(c, kernel)
            s.wait_stream(torch.cuda.current_stream())
            check(r(s), c, reference(c))
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                r.B.CacheScoreCall(r.plan, r.args).run(torch.cuda.current_stream().cuda_stream)
            d = copy.deepcopy(c)
            d.requests = [(n, max(n, kv // 2)) for n, kv in c.requests]
            r.kv_len.copy_(torch.tensor([kv for _, kv in d.requests], dtype=torch.int32))
            r.score.fill_(-7.0)
            g.replay()
            torch.cuda.synchronize()
            check(r.score.cpu(), d, reference(d))


@pytest.mark.parametrize("requests,group,kernel", [([(1, 140001)], 4, 0), ([(1, 140001)], 4, 2), ([(20, 90000)], 8, 0)])
def test_long_context(requests, group, kernel):
    c = Case(requests, Hq=group, Hkv=1, D=64, page=64)
    check(Run(c, kernel)(), c, reference(c))


@pytest.mark.parametrize("d,dtype", [(128, torch.float16), (256, torch.bfloat16), (64, torch.float16)])
def test_long_prompt(d, dtype):
    """Many row blocks, and positions over several CTAs and groups."""
    c = Case([(2600, 4700)], Hq=4, Hkv=2, D=d, dtype=dtype)
    ref = reference(c)
    for over in (dict(), dict(num_sms=1), dict(num_splits=2)):
        r = Run(c, 2, **over)
        check(r(), c, ref)
    assert Run(c, 2).plan.row_groups > 1 and Run(c, 2, num_sms=1).plan.row_groups == 1


def test_score_select_move_attend():
    """A context is cut down: weights of the last rows, choice, move, and attention over what stays.

    The attention over the kept positions, in the cache's own pages, equals that of the definition over the same
    positions, for a list per KV head."""
    from fp8_e4m3_paged_gb300 import binding as B

    c = Case([(8, 900), (8, 333), (8, 100)], Hq=8, Hkv=2, D=128, page=16)
    r = Run(c)
    s = torch.cuda.current_stream().cuda_stream
    score = r()
    budget, sinks, recent = 200, 4, 8
    keep = torch.zeros((3, 2, budget), dtype=torch.int32, device="cuda")
    n_keep = torch.zeros(3, dtype=torch.int32, device="cuda")
    v = c.v.cuda()
    after = torch.zeros_like(r.score)
    B.fp8kv_attn_cache_select(B.make_cache_select_args(score=r.score, kv_len=r.kv_len, budget=budget, sinks=sinks,
                                                       recent=recent, keep=keep, n_keep=n_keep), s)
    B.fp8kv_attn_cache_move(B.make_cache_move_args(k_cache=r.k, v_cache=v, block_table=r.table, src=keep, count=n_keep,
                                                   score=r.score, score_out=after), s)
    q = torch.randn((3, 8, 128), generator=torch.Generator().manual_seed(3)).half().cuda()
    out = torch.zeros_like(q)
    plan = B.fp8kv_attn_chunk_plan(B.make_chunk_desc(
        batch=3, total_q=3, max_q=1, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, max_kv_len=budget,
        max_blocks=c.cols, num_kv_blocks=c.blocks))
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    args = B.make_chunk_args(q=q, k_cache=r.k, v_cache=v, out=out, workspace=ws, softmax_scale=c.softmax_scale,
                             k_scale=c.k_scale, v_scale=c.v_scale, block_table=r.table, cu_q=cu, kv_len=n_keep)
    B.fp8kv_attn_chunk(plan, args, s)
    torch.cuda.synchronize()
    assert n_keep.tolist() == [200, 200, 100]
    tab = decode_table(c.fmt)
    kept = keep.cpu()
    for b, (n, kv) in enumerate(c.requests):
        for g in range(2):
            line = kept[b, g, :n_keep[b]].long()
            assert torch.equal(after[b, g, :len(line)].cpu(), score[b, g, line])
            if kv > budget:  # nothing that went weighs more than what stayed of those between
                gone = torch.ones(kv, dtype=torch.bool)
                gone[line] = False
                between = line[(line >= sinks) & (line < kv - recent)]
                assert score[b, g, :kv][gone].max() <= score[b, g, between].min()
            blk = c.table[b].long()[line // 16]
            K, V = (tab[x[blk, line % 16, g].long()] for x in (c.k, c.v))
            w = torch.softmax(q[b, 4 * g:4 * g + 4].cpu().double() @ K.T * c.softmax_scale * c.k_scale, -1)
            want = w @ V * c.v_scale
            bound = 2.0 ** -11 * want.abs() + (2.0 ** -11 + 2.0 ** -14) * (w @ V.abs()) * c.v_scale + 2.0 ** -24
            assert ((out[b, 4 * g:4 * g + 4].cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("n", [1, 20, 50, 100])
@pytest.mark.parametrize("where", ["last", "pages"])
def test_nan_with_nothing_finite_beside_it(n, where):
    """A NaN logit reaches its row where every other logit that the row sees of the same columns is masked, or NaN too: in
    the newest position alone behind whole tiles, and all over the first columns of tiles (n: one and two row tiles, and
    several row blocks)."""
    for kv in (129, 257, 385):
        c = Case([(n, kv), (1, 40)], Hq=8, Hkv=2, D=128)
        bad = [kv - 1] if where == "last" else [t for t in [*range(32), *range(128, 160)] if t < kv]
        for t in bad:
            c.k[c.table[0, t // c.page].long(), t % c.page, 1, 5] = 0x7F
        ref = reference(c)
        assert torch.isnan(ref[0][0, 1, :kv]).all() and torch.isfinite(ref[0][0, 0, :kv]).all()
        for kernel, S in kernels(c):
            check(Run(c, kernel, S)(), c, ref)


@pytest.mark.parametrize("n", [1, 3, 12, 60])
@pytest.mark.parametrize("code", [0x7E, 0x7C])
def test_minus_infinity_in_a_row_that_is_nan(n, code):
    """Positions whose own logit is -inf are NaN too where a row that sees them is; those in a block out of range, which no
    row sees, are not.  (n: up to 16 query vectors, more, and row tiles.)"""
    c = Case([(n, 200), (1, 77)], Hq=8, Hkv=2, D=128, fmt="e5m2", k_scale=0.001)
    c.q = c.q.abs() + c.q.new_tensor(2.0 ** -6)  # (an infinity times q keeps its sign)
    t = 200 - n  # the first new token: all rows see it
    c.k[c.table[0, t // c.page].long(), t % c.page, 1, 5] = code
    for low in (7, 100, 150):
        c.k[c.table[0, low // c.page].long(), low % c.page, 1, 9] = 0xFC
    hidden = int(c.table[0, 40 // c.page])
    ref = reference(c, bad_blocks=[hidden])
    out = ref[0][0, 1, :200]
    assert torch.isnan(out[[7, 100, 150]]).all() and (out[32:48] == 0).all()
    bad = copy.deepcopy(c)
    bad.table[0, 40 // c.page] = -1
    for kernel, S in kernels(c):
        check(Run(bad, kernel, S)(), bad, ref)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("power", [3, 5, 6, 7, 9, 11, 13, 15, 17, 19, 20, 21, 22, 24, "mixed", "apart"])
def test_equal_keys_share_a_row(power, dtype):
    """Where all of a row's logits are equal its weights are 1 / (positions seen), however large the logits are.

    Per row, relative: the logits of a row are the same number x, so in exact arithmetic of the exponent the factor 2^(x - m)
    cancels.  Up to |x| = 2^7 that is off by the rounding of numbers of that size at the most, 2 x 2^-18 ln 2 in all; past it
    both passes round the same product.  The row's sum of N weights (N/64 + 32) 2^-23 (as above), the sum over R rows (R/64 + 80) 2^-24."""
    for requests in ([(1, 3), (2, 300)], [(30, 300), (1, 129), (40, 45)], [(100, 700), (70, 200)]):
        c = Case(requests, Hq=8, Hkv=2, D=128, dtype=dtype, softmax_scale=45.0, k_scale=1.0)
        c.k[:] = 0x38  # 1.0
        # (mixed: within eight tokens, a warp's 32 rows; apart: from eight to eight)
        p = torch.full((c.total,), float(power)) if not isinstance(power, str) else \
            torch.tensor([22.0, 21.0, 3.0, 6.0, 13.0, 20.0])[torch.arange(c.total) // (1 if power == "mixed" else 8) % 6]
        # 128 q 45 log2 e = 2^13.02 q
        c.q[:] = (torch.where(torch.arange(c.Hq)[None] % 2 == 1, -1.0, 1.0) * 2.0 ** (p[:, None] - 13))[..., None].to(dtype)
        want = torch.full((len(requests), 2, c.max_kv), float("nan"), dtype=torch.float64)
        tol = want.clone()
        for b, (n, kv) in enumerate(requests):
            for t in range(kv):
                seen = torch.arange(max(t, kv - n), kv) + 1  # positions that each row that sees t sees
                want[b, :, t] = c.group * (1.0 / seen.double()).sum()
            tol[b, :, :kv] = want[b, :, :kv] * (2.0 ** -17 * math.log(2) + (kv / 64 + 32) * 2.0 ** -23 +
                                                (n * c.group / 64 + 80) * 2.0 ** -24)
        for kernel, S in kernels(c):
            check(Run(c, kernel, S)(), c, (want, tol))
