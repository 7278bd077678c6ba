"""GPU parity of the tree attention (fp8kv_attn_tree) with its definition in 64 bits.

Trees of every size from one node on, masks that are no trees, rows that see nothing, windows by depth, partitions, both
kernels, page sizes that end inside a tile, non-finite codes, bad blocks and depths, graph replay, and a verify step
from the write of its drafts on.  Every slot that no node may see holds a NaN code.
"""

import copy

import numpy as np
import pytest
import torch

from tests._chunk_ref import POISON
from tests._tree_ref import TreeCase, ancestors, words_of

pytestmark = pytest.mark.gpu

P_ERR = 2.0 ** -11  # probabilities as fp16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_e4m3_paged_gb300 import build_lib

    build_lib.build()


class Run:
    """Device buffers and plan of a case."""

    def __init__(self, c, kernel=0, num_splits=0, spread=False, **over):
        from fp8_e4m3_paged_gb300 import binding as B

        self.B, self.c = B, c
        dev = "cuda"
        self.cu, self.kv_len = torch.from_numpy(c.cu).to(dev), torch.from_numpy(c.kv_len).to(dev)
        self.mask, self.depth = torch.from_numpy(c.mask).to(dev), torch.from_numpy(c.depth).to(dev)
        self.table = c.table.to(dev)
        q, k, v = c.q.to(dev), c.k.to(dev), c.v.to(dev)
        self.out = torch.full((c.total, c.Hq, c.D), 7.0, dtype=q.dtype, device=dev)
        if spread:  # rows, heads, pages and mask rows further apart than they need to be
            qw = torch.zeros(c.total, c.Hq + 1, c.D + 8, dtype=q.dtype, device=dev)
            qw[:, :c.Hq, :c.D] = q
            q = qw[:, :c.Hq, :c.D]
            both = torch.full((c.blocks, c.page, 2, c.Hkv, c.D), 0x7F, dtype=torch.uint8, device=dev)
            both[:, :, 0], both[:, :, 1] = k, v
            k, v = both[:, :, 0], both[:, :, 1]
            wide = torch.full((c.total, c.words + 3), -1, dtype=torch.int32, device=dev)
            wide[:, :c.words] = self.mask
            self.mask = wide[:, :c.words]
        self.q, self.k, self.v = q, k, v
        desc = dict(batch=len(c.requests), total_q=c.total, max_q=c.max_q, num_q_heads=c.Hq, num_kv_heads=c.Hkv,
                    head_dim=c.D, page_size=c.page, max_kv_len=c.max_kv, max_blocks=c.cols, num_kv_blocks=c.blocks,
                    window=c.window, sinks=c.sinks,
                    dtype=B.DTYPE_F16 if c.dtype == torch.float16 else B.DTYPE_BF16,
                    kv_format=B.KV_E4M3 if c.fmt == "e4m3" else B.KV_E5M2, kernel=kernel, num_splits=num_splits)
        desc.update(over)
        self.plan = B.fp8kv_attn_tree_plan(B.make_chunk_desc(**desc))
        self.ws = torch.full((self.plan.workspace_bytes,), 0xFF, dtype=torch.uint8, device=dev)
        self.ws[:4] = 0
        self.args = B.make_tree_args(q=q, k_cache=k, v_cache=v, out=self.out, workspace=self.ws, mask=self.mask,
                                     depth=self.depth, softmax_scale=c.softmax_scale, block_table=self.table,
                                     cu_q=self.cu, kv_len=self.kv_len, k_scale=c.k_scale, v_scale=c.v_scale)

    def __call__(self, stream=None):
        s = torch.cuda.current_stream() if stream is None else stream
        self.B.TreeCall(self.plan, self.args).run(s.cuda_stream)
        s.synchronize()
        return self.out.cpu().double()

    def status(self):
        return int(self.ws[:4].view(torch.int32).item())


def check(got, c, ref=None):
    out, tol, cond = c.reference() if ref is None else ref
    used = int(c.cu[-1])
    assert (got[used:] == 7.0).all(), "rows behind the last request were written"
    g, r = got[:used], out[:used]
    bound = tol[:used] + P_ERR * cond[:used]
    assert torch.equal(torch.isnan(g), torch.isnan(r)), "NaN in other places"
    inf = torch.isinf(r)
    assert torch.equal(torch.isinf(g), inf) and torch.equal(g[inf], r[inf]), "infinities in other places"
    fine = torch.isfinite(r)
    d = torch.where(fine, (g - torch.nan_to_num(r, posinf=0, neginf=0)).abs(), 0.0)
    worst = (torch.where(fine, d / bound, 0.0)).max() if used else torch.tensor(0.0)
    assert worst <= 1.0, f"{float(worst):.3f} of the bound"


def kernels():
    return [(1, 0), (1, 1), (1, 3), (1, 11), (2, 0), (2, 1), (2, 3), (0, 0)]


def _odd_masks(sizes, seed):
    """Masks of any pattern, some rows of them empty."""
    r = np.random.default_rng(seed)
    out = [r.random((n, n)) < 0.4 for n in sizes]
    for x in out:
        x[::3] = False
    return out


CASES = {
    "one_node": TreeCase([(1, 1), (1, 2), (1, 700), (1, 129)], Hq=6, Hkv=1, D=256),
    "small": TreeCase([(9, 130), (26, 637), (2, 2)], Hq=8, Hkv=2, D=128),
    "small_bf16": TreeCase([(16, 300), (5, 77), (31, 31)], Hq=8, Hkv=2, D=128, dtype=torch.bfloat16, page=5),
    "narrow_e5m2": TreeCase([(33, 200), (7, 500)], Hq=4, Hkv=4, D=64, fmt="e5m2", k_scale=0.001, page=7),
    "wide": TreeCase([(26, 637), (3, 40)], Hq=6, Hkv=1, D=256, page=1728),
    "word_edges": TreeCase([(31, 95), (32, 160), (33, 97), (64, 64), (65, 193)], Hq=4, Hkv=2, D=128, page=16),
    "odd_group": TreeCase([(77, 300), (40, 290)], Hq=5, Hkv=1, D=128, page=1),
    "many_nodes": TreeCase([(300, 811), (129, 129)], Hq=2, Hkv=1, D=128, seed=3),
    "group12": TreeCase([(22, 333), (1, 1)], Hq=24, Hkv=2, D=128, page=4, dtype=torch.bfloat16),
    "any_mask": TreeCase([(40, 120), (17, 17), (70, 300)], Hq=4, Hkv=2, D=128, masks=_odd_masks((40, 17, 70), 1)),
    "no_context": TreeCase([(40, 40), (3, 3)], Hq=4, Hkv=2, D=128, masks=_odd_masks((40, 3), 2), extra_rows=9),
    "behind_position_0": TreeCase([(9, 4), (3, 0), (140, 130)], Hq=4, Hkv=2, D=128,
                                  masks=[np.ones((n, n), bool) for n in (9, 3, 140)]),
    "window": TreeCase([(26, 900), (9, 140), (5, 5), (33, 134)], Hq=8, Hkv=2, D=128, window=129, sinks=4),
    "window_short": TreeCase([(40, 300), (20, 300)], Hq=4, Hkv=2, D=128, window=3, sinks=0),
    "window_sinks_past_base": TreeCase([(30, 60), (12, 200)], Hq=4, Hkv=2, D=64, window=20, sinks=100,
                                       dtype=torch.bfloat16),
    "empty_requests": TreeCase([(0, 0), (0, 100), (12, 120), (0, 0)], Hq=4, Hkv=2, D=128, extra_rows=5),
    "many_requests": TreeCase([(1 + i % 9, 9 + (i * 37) % 210 + i % 4) for i in range(75)], Hq=2, Hkv=1, D=64),
    "negative_scale": TreeCase([(20, 200), (4, 90)], Hq=4, Hkv=2, D=128, softmax_scale=-0.11),
}


@pytest.mark.parametrize("name", CASES)
def test_every_kernel(name):
    c = CASES[name]
    ref = c.reference()
    for kernel, S in kernels():
        r = Run(c, kernel, S)
        check(r(), c, ref)
        assert r.status() == 0, (kernel, S)


@pytest.mark.parametrize("kernel,S", [(1, 2), (2, 1), (2, 2)])
def test_strides(kernel, S):
    for name in ("small", "window", "wide"):
        c = CASES[name]
        check(Run(c, kernel, S, spread=True)(), c)


def test_a_causal_mask_is_the_chunk_attention():
    """A chain of drafts gives bit for bit what fp8kv_attn_chunk gives with the same kernel and partitions."""
    from fp8_e4m3_paged_gb300 import binding as B

    sizes = [(40, 300), (7, 30)]
    c = TreeCase(sizes, Hq=8, Hkv=2, D=128, masks=[np.tril(np.ones((n, n), bool)) for n, _ in sizes])
    for kernel in (1, 2):
        r = Run(c, kernel, 1)
        got = r().clone()
        plan = B.fp8kv_attn_chunk_plan(B.make_chunk_desc(
            batch=2, total_q=c.total, max_q=c.max_q, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=c.page,
            max_kv_len=c.max_kv, max_blocks=c.cols, num_kv_blocks=c.blocks, kernel=kernel, num_splits=1))
        B.fp8kv_attn_chunk(plan, r.args.chunk, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(got, r.out.cpu().double())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_nonfinite_codes(fmt):
    """NaN and infinite codes of K and V, in the context and in nodes, reach the rows that see them and no others."""
    base = TreeCase([(12, 150), (70, 200)], Hq=4, Hkv=2, D=128, fmt=fmt, k_scale=0.02 if fmt == "e4m3" else 0.001)
    codes = [0x7F] if fmt == "e4m3" else [0x7E, 0x7C, 0xFC]
    for cache in ("k", "v"):
        for code in codes:
            c = copy.deepcopy(base)
            x = getattr(c, cache)
            for b, t in ((0, 140), (1, 133), (1, 180)):  # node 2, node 3, node 50
                x[c.table[b, t // c.page].long(), t % c.page, 1, 5] = code
            if cache == "v":
                x[c.table[0, 0].long(), 3, 0, 9] = code  # in the context: every row of the request
            ref = c.reference()
            for kernel, S in ((1, 1), (1, 3), (2, 1), (2, 2)):
                check(Run(c, kernel, S)(), c, ref)


def test_bad_blocks_and_depths():
    c = TreeCase([(26, 400), (9, 200)], Hq=4, Hkv=2, D=128, window=100, sinks=2)
    bad = copy.deepcopy(c)
    hidden = [int(c.table[0, 350 // c.page]), int(c.table[1, 195 // c.page])]
    ref = c.reference(bad_blocks=hidden)
    for b, t in ((0, 350), (1, 195)):
        bad.table[b, t // c.page] = 1 << 20 if b else -1
    for kernel, S in ((1, 1), (1, 2), (2, 1), (2, 2)):
        r = Run(bad, kernel, S)
        check(r(), bad, ref)
        assert r.status() == r.B.STATUS_BAD_BLOCK
    deep = copy.deepcopy(c)
    deep.depths = [d.copy() for d in c.depths]
    deep.depths[0][3], deep.depths[1][8] = -5, 1 << 30  # clamped to 0 and 8
    deep.depth[3], deep.depth[26 + 8] = -5, 1 << 30
    ref = deep.reference()
    for kernel in (1, 2):
        r = Run(deep, kernel, 1)
        check(r(), deep, ref)
        assert r.status() == r.B.STATUS_BAD_LEN


def test_other_stream_and_replay_with_other_trees():
    c = TreeCase([(26, 637), (9, 200), (40, 90)], Hq=8, Hkv=2, D=128)
    d = TreeCase([(26, 500), (9, 150), (40, 70)], Hq=8, Hkv=2, D=128, seed=0, masks=_odd_masks((26, 9, 40), 9))
    for kernel, S in ((1, 0), (2, 2), (2, 0)):
        s = torch.cuda.Stream()
        r = Run(c, kernel, S)
        s.wait_stream(torch.cuda.current_stream())
        check(r(s), c)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r.B.TreeCall(r.plan, r.args).run(torch.cuda.current_stream().cuda_stream)
        # other lengths, masks and bytes in the same buffers
        r.kv_len.copy_(torch.from_numpy(d.kv_len))
        r.mask.copy_(torch.from_numpy(d.mask))
        r.k.copy_(c.k), r.v.copy_(c.v)
        e = copy.deepcopy(d)
        e.k, e.v, e.table, e.q = c.k, c.v, c.table, c.q
        e.max_kv, e.cols, e.blocks = c.max_kv, c.cols, c.blocks
        g.replay()
        torch.cuda.synchronize()
        check(r.out.cpu().double(), e)


def test_many_requests_and_row_blocks():
    """Batches whose CTAs do not find their shares from the lengths: partitions of one length."""
    for c in (TreeCase([(1 + i % 5, 9 + (i * 37) % 90) for i in range(140)] + [(5, 3000)], Hq=2, Hkv=1, D=64),
              TreeCase([(300, 2900), (5, 40), (0, 7)], Hq=2, Hkv=1, D=128)):
        ref = c.reference()
        r = Run(c, 2)
        assert r.plan.per_head == 0 and r.plan.num_splits > 1
        check(r(), c, ref)


def test_shares_with_nothing_to_see():
    """Requests without positions, without tokens, with a mask that is empty, beside a long one."""
    n = [3, 0, 40, 5, 1, 0]
    c = TreeCase([(3, 0), (0, 50), (40, 1500), (5, 5), (1, 1), (0, 0)], Hq=8, Hkv=2, D=128,
                 masks=[np.zeros((k, k), bool) for k in n], extra_rows=3)
    r = Run(c, 2)
    assert r.plan.per_head > 0
    got = r()
    check(got, c)
    assert (got[:3] == 0).all() and (got[43:49] == 0).all()


@pytest.mark.parametrize("kernel", [1, 2])
def test_pages_past_32_bits(kernel):
    """Pages 600 MB apart: byte offsets up to 6 GB."""
    from fp8_e4m3_paged_gb300 import binding as B

    c = TreeCase([(9, 60), (20, 40)], Hq=8, Hkv=2, D=128, page=16)
    far = (600 << 20) // 128 * 128
    r = Run(c, kernel)
    pool = torch.empty(c.blocks * far, dtype=torch.uint8, device="cuda")
    assert pool.numel() > 1 << 32
    k = pool.as_strided((c.blocks, 16, 2, 128), (far, 256, 128, 1))
    v = pool.as_strided((c.blocks, 16, 2, 128), (far, 256, 128, 1), 4096)
    k.copy_(c.k.cuda())
    v.copy_(c.v.cuda())
    r.args = B.make_tree_args(q=r.q, k_cache=k, v_cache=v, out=r.out, workspace=r.ws, mask=r.mask, depth=r.depth,
                              softmax_scale=c.softmax_scale, block_table=r.table, cu_q=r.cu, kv_len=r.kv_len,
                              k_scale=c.k_scale, v_scale=c.v_scale)
    check(r(), c)


def test_two_graphs_share_no_workspace():
    """Two calls in flight on streams of their own, each with its workspace."""
    c, d = CASES["many_nodes"], CASES["small"]
    a, b = Run(c, 2, 3), Run(d, 1, 3)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.B.TreeCall(a.plan, a.args).run(s.cuda_stream)
        b.B.TreeCall(b.plan, b.args).run(t.cuda_stream)
    torch.cuda.synchronize()
    check(a.out.cpu().double(), c)
    check(b.out.cpu().double(), d)


def test_long_context():
    """A context past one FP32 sum's positions, and a tree behind it."""
    c = TreeCase([(10, 70001)], Hq=2, Hkv=1, D=64, page=64)
    ref = c.reference()
    for kernel, S in ((0, 0), (1, 0), (1, 1), (2, 0)):
        check(Run(c, kernel, S)(), c, ref)


def test_largest_tree():
    n = 1024
    sees, depth = ancestors([-1] + [i // 2 for i in range(n - 1)])
    c = TreeCase([(n, 1400)], Hq=1, Hkv=1, D=64, masks=[sees], depths=[depth], window=50, sinks=1)
    assert words_of(sees, 32).shape == (n, 32)
    ref = c.reference()
    for kernel in (0, 1, 2):
        check(Run(c, kernel)(), c, ref)


def test_a_nodes_path_is_what_it_would_be_alone():
    """Each leaf's output equals a causal verify of its path, its rows written to a cache of their own."""
    from fp8_e4m3_paged_gb300 import binding as B

    c = TreeCase([(15, 100)], Hq=4, Hkv=2, D=128, spare=0)
    got = Run(c)()
    base = 85
    for leaf in (3, 14):
        path = np.flatnonzero(c.masks[0][leaf])
        kv = base + len(path)
        table = torch.arange(1, 1 + -(-kv // 16), dtype=torch.int32)[None].cuda()
        k, v = (torch.full((1 + table.shape[1], 16, 2, 128), POISON["e4m3"], dtype=torch.uint8) for _ in "kv")
        for t in range(kv):
            s = t if t < base else base + int(path[t - base])
            for x, y in ((k, c.k), (v, c.v)):
                x[1 + t // 16, t % 16] = y[c.table[0, s // c.page].long(), s % c.page]
        q = c.q[torch.from_numpy(path)].cuda()
        out = torch.zeros_like(q)
        plan = B.fp8kv_attn_chunk_plan(B.make_chunk_desc(
            batch=1, total_q=len(path), max_q=len(path), num_q_heads=4, num_kv_heads=2, head_dim=128, page_size=16,
            max_kv_len=kv, max_blocks=table.shape[1], num_kv_blocks=k.shape[0]))
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        args = B.make_chunk_args(q=q, k_cache=k.cuda(), v_cache=v.cuda(), out=out, workspace=ws,
                                 softmax_scale=c.softmax_scale, k_scale=c.k_scale, v_scale=c.v_scale,
                                 block_table=table, cu_q=torch.tensor([0, len(path)], dtype=torch.int32).cuda(),
                                 kv_len=torch.tensor([kv], dtype=torch.int32).cuda())
        B.fp8kv_attn_chunk(plan, args, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        _, tol, cond = c.reference()
        rows = torch.from_numpy(path)
        assert ((out.cpu().double() - got[rows]).abs() <= 2 * (tol[rows] + P_ERR * cond[rows])).all()
