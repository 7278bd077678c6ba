"""GPU parity of the chunk attention (fp8kv_attn_chunk) with its definition in 64 bits.

Ragged batches, single tokens, windows with sinks, both cache formats, both
query types, head dims 64/128/256, page sizes that end inside a tile,
partitions, strides, dead rows, rows behind the last request, non-finite
codes, bad blocks and lengths, graph replay, streams.  Every cache slot that no
new token may see holds a NaN code.
"""

import copy

import numpy as np
import pytest
import torch

from tests._chunk_ref import POISON, Case, decode_table

pytestmark = pytest.mark.gpu

P_ERR = 2.0 ** -11  # probabilities as fp16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_e4m3_paged_gb300 import build_lib

    build_lib.build()
    import oracle

    oracle.build()


class Run:
    """Device buffers and plan of a case."""

    def __init__(self, c, kernel=0, num_splits=0, spread=False, device_scales=False, **over):
        from fp8_e4m3_paged_gb300 import binding as B

        self.B, self.c = B, c
        dev = "cuda"
        self.cu = torch.from_numpy(c.cu).to(dev)
        self.kv_len = torch.from_numpy(c.kv_len).to(dev)
        self.table = c.table.to(dev)
        q, k, v = c.q.to(dev), c.k.to(dev), c.v.to(dev)
        if spread:  # rows, heads and pages further apart than they need to be
            qw = torch.zeros(c.total, c.Hq + 1, c.D + 8, dtype=q.dtype, device=dev)
            qw[:, :c.Hq, :c.D] = q
            q = qw[:, :c.Hq, :c.D]
            ow = torch.full((c.total, c.Hq + 2, c.D + 16), 7.0, dtype=q.dtype, device=dev)
            self.out_all, self.out = ow, ow[:, :c.Hq, :c.D]
            both = torch.full((c.blocks, c.page, 2, c.Hkv, c.D), 0x7F, dtype=torch.uint8, device=dev)
            both[:, :, 0], both[:, :, 1] = k, v
            k, v = both[:, :, 0], both[:, :, 1]
        else:
            self.out = torch.full((c.total, c.Hq, c.D), 7.0, dtype=q.dtype, device=dev)
        self.q, self.k, self.v = q, k, v
        desc = dict(batch=len(c.requests), total_q=c.total, max_q=c.max_q, num_q_heads=c.Hq, num_kv_heads=c.Hkv,
                    head_dim=c.D, page_size=c.page, max_kv_len=c.max_kv, max_blocks=c.cols, num_kv_blocks=c.blocks,
                    window=c.window, sinks=c.sinks,
                    dtype=B.DTYPE_F16 if c.dtype == torch.float16 else B.DTYPE_BF16,
                    kv_format=B.KV_E4M3 if c.fmt == "e4m3" else B.KV_E5M2, kernel=kernel, num_splits=num_splits)
        desc.update(over)
        self.plan = B.fp8kv_attn_chunk_plan(B.make_chunk_desc(**desc))
        self.ws = torch.full((self.plan.workspace_bytes,), 0xFF, dtype=torch.uint8, device=dev)
        self.ws[:4] = 0
        self.scales = [torch.tensor([x], dtype=torch.float32, device=dev) for x in (c.k_scale, c.v_scale)]
        sc = dict(k_scale_dev=self.scales[0], v_scale_dev=self.scales[1]) if device_scales else \
            dict(k_scale=c.k_scale, v_scale=c.v_scale)
        self.args = B.make_chunk_args(q=q, k_cache=k, v_cache=v, out=self.out, workspace=self.ws,
                                      softmax_scale=c.softmax_scale, block_table=self.table, cu_q=self.cu,
                                      kv_len=self.kv_len, **sc)

    def __call__(self, stream=None):
        s = torch.cuda.current_stream() if stream is None else stream
        self.B.fp8kv_attn_chunk(self.plan, self.args, s.cuda_stream)
        s.synchronize()
        return self.out.cpu().double()

    def status(self):
        return int(self.ws[:4].view(torch.int32).item())


def check(got, c, ref=None, rows=None):
    out, tol, cond = c.reference() if ref is None else ref
    used = int(c.cu[-1]) if rows is None else rows
    assert (got[int(c.cu[-1]):] == 7.0).all(), "rows behind the last request were written"
    g, r = got[:used], out[:used]
    bound = tol[:used] + P_ERR * cond[:used]
    assert torch.equal(torch.isnan(g), torch.isnan(r)), "NaN in other places"
    inf = torch.isinf(r)
    assert torch.equal(torch.isinf(g), inf) and torch.equal(g[inf], r[inf]), "infinities in other places"
    fine = torch.isfinite(r)
    d = torch.where(fine, (g - torch.nan_to_num(r, posinf=0, neginf=0)).abs(), 0.0)
    worst = (torch.where(fine, d / bound, 0.0)).max() if used else torch.tensor(0.0)
    assert worst <= 1.0, f"{float(worst):.3f} of the bound"
    return float(worst)


def kernels(c):
    """Every kernel that takes the case: (kernel, partitions)."""
    return [(1, 0), (1, 1), (1, 3), (1, 11), (2, 0), (2, 1), (2, 3), (0, 0)]


CASES = {
    "decode": Case([(1, 1), (1, 2), (1, 611), (1, 64), (1, 65), (1, 1023)], Hq=6, Hkv=1, D=256),
    "decode_gqa8": Case([(1, 700), (1, 17), (1, 128)], Hq=16, Hkv=2, D=128, page=3),
    "decode_group1": Case([(1, 300), (1, 33)], Hq=3, Hkv=3, D=64, page=5, fmt="e5m2", k_scale=0.001),
    "decode_group12": Case([(1, 333), (1, 1)], Hq=24, Hkv=2, D=128, page=4, dtype=torch.bfloat16),
    "drafts": Case([(3, 130), (8, 8), (5, 777)], Hq=4, Hkv=2, D=64, fmt="e5m2", k_scale=0.001, window=50, sinks=1),
    "ragged": Case([(1, 130), (0, 40), (33, 33), (7, 500), (150, 401)], Hq=8, Hkv=2, D=128),
    "ragged_bf16": Case([(70, 70), (1, 257), (129, 300)], Hq=8, Hkv=2, D=128, dtype=torch.bfloat16, page=64),
    "wide": Case([(100, 431), (3, 3)], Hq=6, Hkv=1, D=256, page=1728),
    "wide_e5m2": Case([(65, 200), (22, 150)], Hq=4, Hkv=2, D=256, fmt="e5m2", k_scale=0.001, dtype=torch.bfloat16),
    "narrow": Case([(200, 200), (31, 700)], Hq=4, Hkv=4, D=64, page=7),
    "odd_group": Case([(77, 300), (200, 290)], Hq=5, Hkv=1, D=128, page=1),
    "window_decode": Case([(1, 900), (1, 130), (1, 5), (1, 134), (1, 1)], Hq=8, Hkv=2, D=128, window=129, sinks=4),
    "window_long_sinks": Case([(1, 900), (2, 300)], Hq=4, Hkv=2, D=128, window=20, sinks=100),
    "window_prompt": Case([(500, 500), (90, 700)], Hq=4, Hkv=2, D=128, window=100, sinks=3, dtype=torch.bfloat16),
    "window_one": Case([(40, 300), (1, 300)], Hq=2, Hkv=1, D=128, window=1),
    "window_wide": Case([(300, 800)], Hq=2, Hkv=1, D=256, window=257, sinks=1, page=16),
    "window_past_all": Case([(30, 300)], Hq=2, Hkv=1, D=64, window=5000, sinks=9),
    "dead_rows": Case([(9, 4), (3, 0), (20, 19), (1, 0)], Hq=4, Hkv=2, D=128),
    "dead_rows_many": Case([(200, 50), (70, 0)], Hq=4, Hkv=2, D=128, window=16, sinks=2),
    "empty_requests": Case([(0, 0), (0, 100), (2, 2), (0, 0)], Hq=4, Hkv=2, D=128, extra_rows=5),
    "behind_the_last": Case([(40, 90), (3, 60)], Hq=8, Hkv=2, D=64, extra_rows=70),
    "many_requests": Case([(1 + i % 4, 1 + (i * 37) % 210 + i % 4) for i in range(75)], Hq=2, Hkv=1, D=64),
    "negative_scale": Case([(20, 200), (1, 90)], Hq=4, Hkv=2, D=128, softmax_scale=-0.11),
    "large_logits": Case([(20, 200), (1, 90)], Hq=4, Hkv=2, D=128, q_scale=30.0),
    "long": Case([(3, 5000), (1, 4097)], Hq=4, Hkv=2, D=128),
    "one_chunk": Case([(150, 3000)], Hq=8, Hkv=2, D=128),          # partitions by waves
    "one_chunk_wide": Case([(130, 2100)], Hq=3, Hkv=1, D=256, dtype=torch.bfloat16),
    "many_vectors_few_positions": Case([(40, 90)], Hq=12, Hkv=1, D=64),
    # enough CTAs and positions that the stream kernel takes the requests by length
    "ragged_decodes": Case([(1 if i % 5 else 0, 1 + (i * 397) % 1500) for i in range(128)], Hq=6, Hkv=3, D=64),
    "ragged_window_decodes": Case([(1 + i % 2, 2 + (i * 731) % 1800) for i in range(90)], Hq=8, Hkv=4, D=64,
                                  window=1100, sinks=4, dtype=torch.bfloat16),
    "more_requests_than_are_sorted": Case([(1, 1 + (i * 211) % 1200) for i in range(131)], Hq=4, Hkv=4, D=64),
}


@pytest.mark.parametrize("name", CASES)
def test_parity(name):
    c = CASES[name]
    ref = c.reference()
    for kernel, splits in kernels(c):
        r = Run(c, kernel, splits)
        got = r()
        try:
            check(got, c, ref)
        except AssertionError as e:
            raise AssertionError(f"kernel {r.plan.kernel}, {r.plan.num_splits} partitions: {e}") from None
        assert r.status() == 0
        again = r()
        assert torch.equal(got, again), "two calls differ"


@pytest.mark.parametrize("name", ["decode", "ragged", "drafts", "window_prompt", "wide"])
def test_strides_and_device_scales(name):
    c = CASES[name]
    for kernel, splits in kernels(c):
        r = Run(c, kernel, splits, spread=True, device_scales=True)
        check(r(), c)
        assert (r.out_all[:, c.Hq:] == 7.0).all() and (r.out_all[:, :, c.D:] == 7.0).all()


def test_bf16_rows_of_very_different_size():
    c = Case([(40, 200), (2, 33)], Hq=4, Hkv=2, D=128, dtype=torch.bfloat16, softmax_scale=1.0)
    size = torch.tensor([1e-30, 1e-6, 1.0, 300.0])[torch.arange(c.total) % 4]
    c.q = (c.q.float() * size[:, None, None] * 0.02).to(torch.bfloat16)
    c.q[5] = 0
    for kernel, splits in kernels(c):
        check(Run(c, kernel, splits)(), c)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_nonfinite_codes_reach_the_rows_that_see_them(fmt, D):
    """A non-finite V code makes that column of exactly the rows that see the
    token non-finite; a NaN K code the whole output of those rows."""
    for requests, window in (([(4, 90), (3, 40)], 0), ([(4, 90), (3, 40)], 20), ([(120, 150)], 30)):
        c = Case(requests, Hq=4, Hkv=2, D=D, fmt=fmt, k_scale=0.02 if fmt == "e4m3" else 0.001, window=window, seed=3)
        nan = 0x7F
        kv0 = c.requests[0][1]

        def put(cache, t, g, d, code):
            cache[c.table[0, t // c.page].long(), t % c.page, g, d] = code

        put(c.v, kv0 - 3, 0, 5, nan)          # seen by the last rows only
        put(c.v, kv0 - 2, 1, D - 1, nan)
        put(c.k, kv0 - 1, 1, 7, nan)          # the last row of KV head 1
        if fmt == "e5m2":
            put(c.v, kv0 - 4, 0, 9, 0x7C)     # +inf
            put(c.v, kv0 - 2, 0, 9, 0x7C)
            put(c.v, kv0 - 4, 0, 10, 0xFC)    # -inf
            put(c.v, kv0 - 4, 0, 11, 0x7C)    # both signs
            put(c.v, kv0 - 1, 0, 11, 0xFC)
        ref = c.reference()
        assert torch.isnan(ref[0]).any() and not torch.isnan(ref[0]).all()
        for kernel, splits in kernels(c):
            check(Run(c, kernel, splits)(), c, ref)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_nonfinite_queries_reach_their_own_rows_only(dtype):
    c = Case([(20, 200), (40, 300), (1, 90)], Hq=4, Hkv=2, D=128, dtype=dtype)
    clean = c.reference()
    c.q[3, 0, 5] = float("nan")
    c.q[30, 2, 7] = float("inf")
    c.q[60, 3, 0] = float("-inf")
    c.q[17, 1] = float("nan")
    bad = torch.zeros(c.total, c.Hq, dtype=torch.bool)
    for row, h in ((3, 0), (30, 2), (60, 3), (17, 1)):
        bad[row, h] = True
    for kernel, splits in kernels(c):
        got = Run(c, kernel, splits)()
        assert torch.isnan(got[bad]).all()
        got[bad] = clean[0][bad]
        check(got, c, clean)


def test_requests_that_share_blocks():
    """A shared prefix: one block in several tables, and twice in one."""
    c = Case([(5, 160), (30, 170), (1, 64)], Hq=8, Hkv=2, D=128, page=16)
    c.table[1, :8] = c.table[0, :8]
    c.table[2, :4] = c.table[0, 0]
    ref = c.reference()
    for kernel, splits in kernels(c):
        check(Run(c, kernel, splits)(), c, ref)


def test_bad_blocks_count_as_not_visible():
    c = Case([(40, 200), (3, 70)], Hq=4, Hkv=2, D=128, page=16, seed=5)
    victims = [int(c.table[0, 2]), int(c.table[1, 0])]
    ref = c.reference(bad_blocks=victims)
    c.table[0, 2] = c.blocks
    c.table[1, 0] = -1
    for kernel, splits in kernels(c):
        r = Run(c, kernel, splits)
        check(r(), c, ref)
        assert r.status() == r.B.STATUS_BAD_BLOCK


def test_lengths_are_clamped():
    c = Case([(4, 90), (3, 60)], Hq=4, Hkv=2, D=128)
    for kernel, splits in [(1, 0), (2, 0), (2, 2), (1, 2)]:
        r = Run(c, kernel, splits)
        r.kv_len[0] = 10 ** 9           # as max_kv_len
        check(r(), c)
        assert r.status() == r.B.STATUS_BAD_LEN
        r = Run(c, kernel, splits)
        r.kv_len[1] = -5                # as 0: nothing to see
        got = r()
        assert (got[4:7] == 0).all() and r.status() == r.B.STATUS_BAD_LEN
        r = Run(c, kernel, splits)
        r.cu[2] = 100                   # past total_q
        check(r(), c)
        assert r.status() == r.B.STATUS_BAD_LEN
        r = Run(c, kernel, splits)
        r.cu[1] = -3                    # request 0 is empty, request 1 begins at row 0
        r()
        assert r.status() == r.B.STATUS_BAD_LEN
        r = Run(c, kernel, splits, max_q=3)  # request 0 has one more than the plan
        r()
        assert r.status() == r.B.STATUS_BAD_LEN


def test_graph_replay_with_other_lengths():
    big = Case([(6, 300), (2, 200), (4, 90)], Hq=8, Hkv=2, D=128, window=70, sinks=2)
    others = [Case([(2, 300), (6, 90), (1, 1)], Hq=8, Hkv=2, D=128, window=70, sinks=2, extra_rows=3),
              Case([(0, 0), (6, 200), (3, 50)], Hq=8, Hkv=2, D=128, window=70, sinks=2, extra_rows=3)]
    for kernel, splits in [(0, 0), (2, 2), (2, 1)]:
        r = Run(big, kernel, splits)
        side = torch.cuda.Stream()
        r(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            r.B.fp8kv_attn_chunk(r.plan, r.args, side.cuda_stream)
        for c in [big] + others:
            r.q.copy_(c.q)
            n = min(r.k.shape[0], c.k.shape[0])
            r.k[:n].copy_(c.k[:n])
            r.v[:n].copy_(c.v[:n])
            r.table[:, :c.cols].copy_(c.table)
            r.cu.copy_(torch.from_numpy(c.cu))
            r.kv_len.copy_(torch.from_numpy(c.kv_len))
            r.out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            check(r.out.cpu().double(), c)
            assert r.status() == 0


def test_two_calls_at_once_with_a_workspace_each():
    c, d = CASES["ragged"], CASES["window_prompt"]
    rc, rd = c.reference(), d.reference()
    a, b = Run(c, 2, 2), Run(d, 2, 2)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.B.fp8kv_attn_chunk(a.plan, a.args, s.cuda_stream)
        b.B.fp8kv_attn_chunk(b.plan, b.args, t.cuda_stream)
    torch.cuda.synchronize()
    check(a.out.cpu().double(), c, rc)
    check(b.out.cpu().double(), d, rd)


def test_cache_offsets_past_32_bits():
    """Blocks 700 MB apart: byte offsets pass 2^31 and 2^32."""
    c = Case([(3, 100), (20, 64)], Hq=4, Hkv=2, D=128, page=16)
    stride = 700 << 20
    for kernel, splits in [(0, 0), (2, 1)]:
        r = Run(c, kernel, splits)
        blocks = c.blocks
        pool = torch.empty(stride * (blocks - 1) + c.page * c.Hkv * c.D, dtype=torch.uint8, device="cuda")
        view = pool.as_strided((blocks, c.page, c.Hkv, c.D), (stride, c.Hkv * c.D, c.D, 1))
        view.copy_(r.k)
        r.args.k_cache, r.args.k_stride_block = view.data_ptr(), stride
        check(r(), c)
        view.copy_(r.v)
        r.args.k_cache, r.args.k_stride_block = r.k.data_ptr(), r.k.stride(0)
        r.args.v_cache, r.args.v_stride_block = view.data_ptr(), stride
        check(r(), c)
        del pool, view


def test_matches_the_decode_path():
    """One new token, no window: the decode call's result."""
    from fp8_e4m3_paged_gb300.device_problem import DeviceProblem
    from synth import make_dense

    p = make_dense(name="d128", B=4, q=1, Hq=16, Hkv=4, D=128, page_size=16, lens=[700, 2000, 130, 1025], seed=8)
    dp = DeviceProblem(p)
    old = dp.run().clone()
    from fp8_e4m3_paged_gb300 import binding as B

    plan = B.fp8kv_attn_chunk_plan(B.make_chunk_desc(
        batch=4, total_q=4, max_q=1, num_q_heads=16, num_kv_heads=4, head_dim=128, page_size=16,
        max_kv_len=int(p.max_kv_len), max_blocks=int(p.block_table.shape[1]), num_kv_blocks=int(p.k_cache.shape[0])))
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.zeros(4, 16, 128, dtype=torch.float16, device="cuda")
    args = B.make_chunk_args(q=dp.q.view(4, 16, 128), k_cache=dp.k_caches[0], v_cache=dp.v_caches[0], out=out,
                             workspace=ws, softmax_scale=p.softmax_scale, k_scale=p.k_scale, v_scale=p.v_scale,
                             block_table=dp.block_table, cu_q=torch.arange(5, dtype=torch.int32, device="cuda"),
                             kv_len=dp.row_len.view(4).contiguous())
    B.ChunkCall(plan, args).run(torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    # Both round their sum once (half an fp16 step, 2^-11 of it); this call also rounds each probability to fp16, which
    # moves the sum by at most 2^-11 of sum_j w_j |v_j|; 2^-14 of that covers the FP32 logits, weights and sums.
    import oracle

    cond = torch.from_numpy(oracle.attention_abs(p)).view(4, 16, 128).cuda()
    a, b = out.double(), old.view(4, 16, 128).double()
    bound = (a.abs() + b.abs()) * 2.0 ** -11 + cond * (2.0 ** -11 + 2.0 ** -14)
    assert float(((a - b).abs() / bound).max()) <= 1.0


def test_workspace_and_device_of_tensors():
    from fp8_e4m3_paged_gb300 import binding as B

    c = CASES["ragged"]
    r = Run(c, 2, 3)
    r.args.workspace_bytes = r.plan.workspace_bytes - 1
    with pytest.raises(B.Fp8kvError) as e:
        r()
    assert e.value.code == B.EWORKSPACE


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_nan_logits_outweigh_infinite_values(D, dtype):
    """A row that is NaN for its logits (a NaN K code, a NaN query) stays NaN where it also sees an infinite V code."""
    for requests in ([(4, 90), (3, 40)], [(150, 170)]):
        c = Case(requests, Hq=4, Hkv=2, D=D, fmt="e5m2", k_scale=0.001, dtype=dtype, seed=6)
        n, kv = c.requests[0]

        def put(cache, t, g, d, code):
            cache[c.table[0, t // c.page].long(), t % c.page, g, d] = code

        put(c.v, 5, 0, 9, 0x7C)             # +inf, seen by every row of KV head 0
        put(c.v, 5, 0, 10, 0xFC)            # -inf
        put(c.k, kv - 2, 0, 7, 0x7F)        # NaN, seen by the last two rows of KV head 0
        c.q[0, 1, 3] = float("nan")         # one query of KV head 0
        ref = c.reference()
        assert torch.isnan(ref[0][n - 2:n, :2]).all() and torch.isnan(ref[0][0, 1]).all()
        assert torch.isinf(ref[0][1, 0, 9:11]).all()
        for kernel, splits in kernels(c):
            check(Run(c, kernel, splits)(), c, ref)


@pytest.mark.parametrize("name", ["ragged", "wide", "dead_rows", "dead_rows_many", "window_decode"])
def test_a_nan_scale_reaches_every_row_that_sees_something(name):
    """Device scales are not known on the host: a NaN must not become finite weights, nor reach rows that see nothing."""
    c = CASES[name]
    sees = torch.cat([torch.arange(kv - n, kv) >= 0 for n, kv in c.requests])
    for kernel, splits in kernels(c):
        for i in range(2):  # of K, of V
            r = Run(c, kernel, splits, device_scales=True)
            r.scales[i].fill_(float("nan"))
            got = r()[:int(c.cu[-1])]
            assert torch.isnan(got[sees]).all() and (got[~sees] == 0).all()


def test_long_contexts():
    """Sums cut at 32768 positions: the bound on their truncation is that of such a sum, whatever the context."""
    c = Case([(1, 140000), (2, 70001)], Hq=2, Hkv=1, D=64, page=64)
    out, tol, cond = c.reference()
    for b, (n, kv) in enumerate(c.requests):  # the reference counts a truncation for every K16 step of the context
        rows = slice(int(c.cu[b]), int(c.cu[b]) + n)
        tol[rows] -= (kv - 32768) / 16 * 2.0 ** -23 * cond[rows]
    for kernel, splits in [(0, 0), (1, 1), (1, 2), (2, 1), (2, 9)]:
        check(Run(c, kernel, splits)(), c, (out, tol, cond))


@pytest.mark.parametrize("name", ["decode", "decode_gqa8", "decode_group1", "decode_group12", "drafts", "window_decode",
                                  "ragged", "long"])
def test_the_stream_kernel_keeps_two_halves_of_each_probability(name):
    """A probability as two fp16 numbers: 2^-22 of its own value, where one leaves 2^-11."""
    c = CASES[name]
    out, tol, cond = c.reference()
    used = int(c.cu[-1])
    for splits in (0, 1, 3, 11):
        got = Run(c, 1, splits)()
        worst = ((got - out).abs() / (tol + 2.0 ** -21 * cond))[:used].max()
        assert worst <= 1.0, f"{splits} partitions: {float(worst):.3f} of the bound"


@pytest.mark.parametrize("cu,max_q,becomes", [
    # new tokens past max_q are not computed; the others are the last ones of the context
    ([0, 4, 7], 3, [(0, 3, 90), (4, 3, 60)]),
    ([0, 4, 7], 2, [(0, 2, 90), (4, 2, 60)]),
    # request 0 is empty, request 1 begins at row 0 and has max_q tokens
    ([0, -3, 7], 4, [(0, 0, 90), (0, 4, 60)]),
    ([0, -3, 7], 7, [(0, 0, 90), (0, 7, 60)]),
    # a decrease: request 1 is empty
    ([0, 4, 2], 4, [(0, 4, 90), (4, 0, 60)]),
    ([0, 4, 100], 4, [(0, 4, 90), (4, 3, 60)]),
    ([-9, 4, 7], 4, [(0, 4, 90), (4, 3, 60)]),
])
def test_clamped_lengths_compute_what_the_header_says(cu, max_q, becomes):
    """Rows, new tokens and positions that the clamped lengths leave: those rows right, every other row untouched."""
    c = Case([(4, 90), (3, 60)], Hq=4, Hkv=2, D=128)
    for kernel, splits in [(1, 0), (1, 1), (1, 11), (2, 0), (2, 1), (2, 2)]:
        r = Run(c, kernel, splits, max_q=max_q)
        r.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        got = r()
        assert r.status() == r.B.STATUS_BAD_LEN
        written = torch.zeros(c.total, dtype=torch.bool)
        for b, (row0, n, kv) in enumerate(becomes):
            d = copy.copy(c)
            d.requests = [(0, kv) if x != b else (n, kv) for x in range(2)]
            d.cu = np.array([row0] * (b + 1) + [row0 + n] * (2 - b), dtype=np.int32)
            out, tol, cond = d.reference()
            rows = slice(row0, row0 + n)
            assert ((got[rows] - out[rows]).abs() <= tol[rows] + P_ERR * cond[rows]).all()
            written[rows] = True
        assert (got[~written] == 7.0).all()


def test_rows_before_the_first_request_are_left():
    c = Case([(4, 90), (3, 60)], Hq=4, Hkv=2, D=128)
    d = copy.copy(c)
    d.requests, d.cu = [(2, 90), (3, 60)], np.array([2, 4, 7], dtype=np.int32)
    out, tol, cond = d.reference()
    for kernel, splits in kernels(c):
        r = Run(c, kernel, splits)
        r.cu[0] = 2
        got = r()
        assert r.status() == 0 and (got[:2] == 7.0).all()
        assert ((got - out).abs() <= tol + P_ERR * cond)[2:].all()


def _minus_infinite_logits(requests, D):
    """E5M2 case whose request 0 has a logit of -inf at every position but the last two, for KV head 0."""
    c = Case(requests, Hq=4, Hkv=2, D=D, fmt="e5m2", k_scale=0.001, seed=9)
    c.q[:, :, 3] = c.q[:, :, 3].abs() + 0.5
    n, kv = c.requests[0]
    t = torch.arange(kv - 2)
    c.k[c.table[0].long()[t // c.page], t % c.page, 0, 3] = 0xFC
    return c, n


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_whose_logits_are_all_minus_infinity_are_zero(D):
    """Infinite K codes: a sum of weights of 0 gives +0, as in the decode path's combine."""
    for requests in ([(4, 90), (1, 40)], [(150, 300)]):
        c, n = _minus_infinite_logits(requests, D)
        ref = c.reference()
        assert (ref[0][:n - 2, :2] == 0).all() and (ref[0][n - 2:n, :2] != 0).any()
        # The reference has no bound for logits beside infinite codes.  The last rows have one or two finite logits: their
        # FP32 errors, (D/16 + 16) 2^-23 of a = sum |q k| <= 13 (D = 256: 256 * 0.64 * 256^-0.5 = 10), move the output by
        # at most twice that of cond: below 2^-13
        ref[1][:n, :2] = 2.0 ** -11 * ref[0][:n, :2].abs() + 2.0 ** -13 * ref[2][:n, :2] + 2.0 ** -25
        for kernel, splits in kernels(c):
            got = Run(c, kernel, splits)()
            assert not torch.signbit(got[:n - 2, :2]).any()
            check(got, c, ref)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_nonfinite_values_of_weight_zero_do_not_depend_on_partitions(D):
    """An infinite V code at a position whose logit is -inf: it reaches the rows that have other positions to see, also
    where its partition holds nothing else for them; a row without any stays +0."""
    for requests in ([(4, 90), (1, 40)], [(150, 300)], [(1, 700)]):
        c, n = _minus_infinite_logits(requests, D)
        clean = c.reference()[0]
        c.v[c.table[0, 0].long(), 2, 0, 8] = 0x7C
        c.v[c.table[0, 0].long(), 3, 0, 9] = 0x7F
        dead = torch.arange(n) < n - 2
        for kernel, splits in kernels(c) + [(1, 8), (2, 2)]:
            got = Run(c, kernel, splits)()[:n, :2]
            assert (got[dead] == 0).all()
            assert (got[~dead, :, 8] == float("inf")).all() and torch.isnan(got[~dead, :, 9]).all()
            others = [d for d in range(D) if d not in (8, 9)]
            assert torch.isfinite(got[..., others]).all()
            assert ((got - clean[:n, :2])[..., others].abs() <= 2.0 ** -6 * (1 + clean[:n, :2][..., others].abs())).all()


@pytest.mark.parametrize("negative", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_logits_past_the_integers_of_32_bits(D, negative):
    """Logits whose neighbours in FP32 are further apart than the softmax resolves.  Every V row is the same, so any
    weights give that row: a probability that overflows, or a sum that vanishes, would show."""
    for power in (10, 20, 22, 23, 24, 25, 26, 27, 28, 30, 34, 50):
        for requests in ([(4, 300), (1, 90)], [(150, 300)]):
            c = Case(requests, Hq=4, Hkv=2, D=D, dtype=torch.bfloat16, k_scale=1.0, v_scale=0.5,
                     softmax_scale=-0.7 if negative else 0.7, seed=power)
            # K: 1 and a small number; q: 2^power and, for the second, about its unit in the last place
            g = torch.Generator().manual_seed(power)
            small = torch.randint(0, 17, c.k.shape[:3], generator=g).float()
            k = torch.zeros(c.k.shape)
            k[..., 0], k[..., 1] = 1.0, small
            c.k = k.to(torch.float8_e4m3fn).view(torch.uint8)
            c.v[:] = c.v[1, 0, :, :][None, None]
            c.v[c.v == POISON["e4m3"]] = 0x38
            c.q[:] = 0
            c.q[..., 0] = 2.0 ** power
            c.q[..., 1] = torch.randint(0, 9, c.q.shape[:2], generator=g) * 2.0 ** (power - 24)
            v = decode_table("e4m3")[c.v[1, 0].long()] * 0.5
            want = v.repeat_interleave(2, 0)[None].expand(c.total, -1, -1)
            for kernel, splits in kernels(c):
                got = Run(c, kernel, splits)()
                # rounding of the output and of the probabilities, and 2^-12 for sums and vanishing ones
                assert ((got - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12)).all(), (power, kernel)


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("splits", [0, 1, 2, 7])
def test_plans_for_far_longer_contexts(kernel, splits):
    """Partitions that only the planned bound asks for stay empty; parity as with the exact plan."""
    c = Case([(3, 400), (1, 65), (9, 1000), (1, 0)], Hq=4, Hkv=2, D=64, page=64)
    d = copy.copy(c)
    d.cols = 1 << 14
    d.table = torch.zeros(len(c.requests), d.cols, dtype=torch.int32)
    d.table[:, :c.cols] = c.table
    exact, wide = Run(c, kernel, splits or 1), Run(d, kernel, splits, max_kv_len=1 << 20)
    assert wide.plan.num_splits >= 16 > exact.plan.num_splits
    got = wide()
    check(got, c)
    if splits:
        assert wide.plan.min_splits == splits
        a, b = exact(), got  # the same partitions, perhaps joined in another order
        assert ((a - b).abs() <= a.abs() * 2.0 ** -9 + 2.0 ** -20).all()
