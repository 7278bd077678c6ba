"""Selection of cached positions by their weights (fp8kv_attn_cache_select) and the move of cache rows
(fp8kv_attn_cache_move) against their definitions on the host: every output is a whole number or a byte, and equal.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_e4m3_paged_gb300 import build_lib

    build_lib.build()
    from fp8_e4m3_paged_gb300 import binding

    return binding


def stream():
    return torch.cuda.current_stream().cuda_stream


# ---------------------------------------------------------------- selection

def chosen(weights, n, budget, sinks, recent):
    """Positions that stay, from the definition; weights: float32 [heads][positions] of one list."""
    if n <= budget:
        return np.arange(n)
    w = weights[0, :n].copy()
    for x in weights[1:, :n]:
        w = w + x  # float32, head after head
    lo, hi, m = sinks, n - recent, budget - sinks - recent
    mid = w[lo:hi].astype(np.float64)
    order = np.lexsort((np.arange(lo, hi), -np.nan_to_num(mid, nan=0.0, posinf=1e300, neginf=-1e300), np.isnan(mid)))
    return np.concatenate([np.arange(sinks), np.sort(lo + order[:m]), np.arange(hi, n)])


def select(B, score, lens, budget, sinks, recent, joint, spread=False, on=None):
    b, hkv, width = score.shape
    lists = 1 if joint else hkv
    x = torch.from_numpy(score).cuda()
    entries = max(1, min(budget, width))
    keep = torch.full((b, lists, entries), -7, dtype=torch.int32, device="cuda")
    if spread:
        wide = torch.full((b, hkv + 1, width + 5), 1e30, device="cuda")
        wide[:, :hkv, 3:3 + width] = x
        x = wide[:, :hkv, 3:3 + width]
        keep = torch.full((b, lists + 2, entries + 3), -7, dtype=torch.int32, device="cuda")[:, 1:1 + lists, :entries]
    n_keep = torch.full((b,), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv_len = torch.tensor(lens, dtype=torch.int32).cuda()
    args = B.make_cache_select_args(score=x, kv_len=kv_len, budget=budget, sinks=sinks, recent=recent, keep=keep,
                                    n_keep=n_keep, status=status)
    torch.cuda.synchronize()
    B.fp8kv_attn_cache_select(args, stream() if on is None else on.cuda_stream)
    torch.cuda.synchronize()
    return keep.cpu().numpy(), n_keep.cpu().numpy(), int(status.item())


def check_select(B, score, lens, budget, sinks=0, recent=0, joint=False, **kw):
    keep, n_keep, status = select(B, score, lens, budget, sinks, recent, joint, **kw)
    assert status == 0
    for b, n in enumerate(lens):
        assert n_keep[b] == min(n, budget)
        for l in range(keep.shape[1]):
            want = chosen(score[b] if joint else score[b, l:l + 1], n, budget, sinks, recent)
            assert (keep[b, l, :len(want)] == want).all(), (b, l)
            assert (keep[b, l, len(want):] == -7).all(), "entries behind the list were written"


def weights(b, hkv, width, seed, kind="spread"):
    r = np.random.default_rng(seed)
    if kind == "spread":
        return (r.random((b, hkv, width)) ** 6 * 20).astype(np.float32)
    if kind == "few":  # ties everywhere
        return r.integers(-2, 3, (b, hkv, width)).astype(np.float32) / 4
    if kind == "zero":
        return np.where(r.random((b, hkv, width)) < 0.5, 0.0, -0.0).astype(np.float32)
    if kind == "near":  # differ in their last bits
        return (1.0 + r.integers(0, 64, (b, hkv, width)) * 2.0 ** -23).astype(np.float32)
    x = r.standard_normal((b, hkv, width)).astype(np.float32)
    pick = r.random(x.shape)
    for lo, v in ((0.0, np.nan), (0.1, np.inf), (0.15, -np.inf), (0.2, 1e-42), (0.25, -1e-42), (0.3, 3e38)):
        x[(pick >= lo) & (pick < lo + 0.05)] = v
    x[x.shape[0] // 2, 0, ::2] = -np.nan
    return x


@pytest.mark.parametrize("kind", ["spread", "few", "zero", "near", "any"])
@pytest.mark.parametrize("joint", [False, True])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 0, 1), (1, 1, 0), (7, 2, 3), (100, 4, 16), (100, 0, 0),
                                                 (100, 60, 40), (333, 1, 332), (4096, 4, 1)])
def test_select(B, kind, joint, budget, sinks, recent):
    lens = [0, 1, 2, budget - 1, budget, budget + 1, 333, 1000, 6001]
    score = weights(len(lens), 2, 6001, budget, kind)
    if joint and kind == "any":
        score = np.clip(score, -1e37, 1e37)  # sums of infinities of both signs are a matter of another test
    check_select(B, score, lens, budget, sinks, recent, joint)


@pytest.mark.parametrize("hkv,width,budget,joint", [(1, 40000, 4000, False), (1, 131072, 16384, False),
                                                    (8, 70001, 3001, True), (3, 33000, 32999, False),
                                                    (2, 500000, 100000, False), (2, 420001, 5, True)])
def test_select_long(B, hkv, width, budget, joint):
    """Lists over several CTAs, and longer than their shared memory takes."""
    for kind in ("spread", "few"):
        check_select(B, weights(2, hkv, width, 5, kind), [width, width - 4099], budget, min(4, budget), min(budget // 4, 300), joint)


@pytest.mark.parametrize("width", [1001, 5002, 20003, 33001, 420003])
def test_select_cut_among_nans(B, width):
    """More positions wanted than have a number: the first NaNs stay too, up to the end of runs of any length."""
    r = np.random.default_rng(width)
    score = r.random((2, 1, width)).astype(np.float32)
    score[r.random(score.shape) < 0.7] = np.nan
    score[:, :, 1::7] = -np.inf
    lens = [width, width - 3]
    check_select(B, score, lens, width // 2, 1, 2)
    check_select(B, score, lens, width - 4, 0, 0)
    check_select(B, np.full_like(score, np.nan), lens, width - 5, 0, 1)


def test_more_lists_than_room(B):
    """Lists whose keys leave room for one CTA on an SM, more of them than SMs."""
    check_select(B, weights(20, 9, 24000, 8), [24000 - 997 * i for i in range(20)], 1000, 4, 64)


def test_select_sums_head_after_head(B):
    """The joint weight is the FP32 sum in the order of the heads: 1e8 + 1 - 1e8 is not 1."""
    score = np.zeros((1, 3, 64), dtype=np.float32)
    score[0, 0, 10], score[0, 1, 10], score[0, 2, 10] = 1e8, 1.0, -1e8
    score[0, 0, 40] = 0.5
    keep, _, _ = select(B, score, [64], 1, 0, 0, True)
    assert keep[0, 0, 0] == 40
    score[0, 0, 20], score[0, 1, 20] = np.inf, -np.inf  # a NaN: below all
    keep, _, _ = select(B, score, [64], 63, 0, 0, True)
    assert (keep[0, 0] == np.delete(np.arange(64), 20)).all()


def test_select_strides_streams_and_lengths(B):
    score = weights(5, 4, 3000, 1)
    s = torch.cuda.Stream()
    for joint in (False, True):
        check_select(B, score, [3000, 10, 2999, 500, 1500], 400, 4, 30, joint, spread=True, on=s)
    keep, n_keep, status = select(B, score, [-5, 3001, 1 << 30, 100, 3000], 400, 4, 30, False)
    assert status == B.STATUS_BAD_LEN and n_keep.tolist() == [0, 400, 400, 100, 400]
    want = chosen(score[1, 2:3], 3000, 400, 4, 30)
    assert (keep[1, 2] == want).all() and (keep[0] == -7).all()


def test_select_many_lists(B):
    check_select(B, weights(300, 3, 257, 2), [i % 258 for i in range(300)], 64, 2, 9)


def test_select_replay(B):
    """A captured call on other weights and lengths."""
    score = torch.from_numpy(weights(3, 2, 9000, 3)).cuda()
    lens = torch.tensor([9000, 100, 5000], dtype=torch.int32).cuda()
    keep = torch.full((3, 2, 700), -7, dtype=torch.int32, device="cuda")
    n_keep = torch.zeros(3, dtype=torch.int32, device="cuda")
    args = B.make_cache_select_args(score=score, kv_len=lens, budget=700, sinks=3, recent=50, keep=keep, n_keep=n_keep)
    B.fp8kv_attn_cache_select(args, stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.fp8kv_attn_cache_select(args, stream())
    other = weights(3, 2, 9000, 4, "few")
    score.copy_(torch.from_numpy(other))
    lens.copy_(torch.tensor([701, 8000, 650], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    for b, n in enumerate((701, 8000, 650)):
        for h in range(2):
            want = chosen(other[b, h:h + 1], n, 700, 3, 50)
            assert (keep[b, h, :len(want)].cpu().numpy() == want).all()


# ---------------------------------------------------------------- move

class Pool:
    """Random pages and tables of a few requests."""

    def __init__(self, b, columns, page, hkv, d, seed=0, fmt=0, fresh=0, interleaved=False):
        g = torch.Generator().manual_seed(seed)
        self.page, self.hkv, self.fmt = page, hkv, fmt
        blocks = 1 + b * (columns + fresh)
        size = 2 if fmt == 2 else 1
        kind = torch.int16 if size == 2 else torch.uint8
        top = 1 << 8 * size
        shape = (blocks, page, hkv, d)
        self.k, self.v = (torch.randint(0, top, shape, generator=g).sub(top // 2 if size == 2 else 0).to(kind)
                          for _ in "kv")
        order = (1 + torch.randperm(blocks - 1, generator=g)).to(torch.int32).view(b, columns + fresh)
        self.table = order[:, :columns].contiguous()
        self.target = order[:, columns:].contiguous() if fresh else None
        self.dk, self.dv = self.k.cuda(), self.v.cuda()
        if interleaved:
            both = torch.zeros((blocks, page, 2, hkv, d + 16 // size), dtype=kind, device="cuda")
            both[:, :, 0, :, :d], both[:, :, 1, :, :d] = self.dk, self.dv
            self.dk, self.dv = both[:, :, 0, :, :d], both[:, :, 1, :, :d]

    def expected(self, src, count, first, skip=lambda b, l, k: False):
        """Both caches afterwards: every row read before any is written."""
        out = [self.k.clone(), self.v.clone()]
        to = self.table if self.target is None else self.target
        P = self.page
        for b in range(src.shape[0]):
            for h in range(self.hkv):
                l = h if src.shape[1] > 1 else 0
                for k in range(count[b]):
                    s = int(src[b, l, k])
                    if skip(b, l, k) or (self.target is None and s < k):
                        continue
                    at, new = first[b] + s, first[b] + k
                    old_blk, new_blk = int(self.table[b, at // P]), int(to[b, new // P])
                    out[0][new_blk, new % P, h] = self.k[old_blk, at % P, h]
                    out[1][new_blk, new % P, h] = self.v[old_blk, at % P, h]
        return out

    def args(self, B, src, count, first=None, **kw):
        dev = lambda t: None if t is None else (torch.as_tensor(t, dtype=torch.int32).cuda())  # noqa: E731
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # (kept: an argument block holds addresses only)
        self.kept = dict(block_table=dev(self.table), src=dev(src).contiguous(), count=dev(count), first=dev(first),
                         dst_table=dev(self.target))
        return B.make_cache_move_args(k_cache=self.dk, v_cache=self.dv, status=self.status, kv_format=self.fmt,
                                      **self.kept, **kw)

    def check(self, B, src, count, first=None, status=0, skip=lambda b, l, k: False, on=None):
        want = self.expected(src, count, [0] * len(count) if first is None else first, skip)
        args = self.args(B, src, count, first)
        torch.cuda.synchronize()
        B.fp8kv_attn_cache_move(args, stream() if on is None else on.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(self.dk.cpu(), want[0]) and torch.equal(self.dv.cpu(), want[1])
        assert int(self.status.item()) == status


def rising(b, lists, n, width, seed):
    """Increasing lists of n of `width` positions."""
    r = np.random.default_rng(seed)
    return torch.from_numpy(np.stack([[np.sort(r.choice(width, n, replace=False)) for _ in range(lists)]
                                      for _ in range(b)]).astype(np.int32))


@pytest.mark.parametrize("page,hkv,d,fmt", [(16, 2, 128, 0), (1, 1, 64, 1), (7, 3, 16, 0), (1728, 2, 256, 0), (16, 2, 128, 2),
                                            (5, 1, 1024, 2), (64, 8, 128, 0)])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("n,width", [(1, 1), (5, 40), (300, 500), (1500, 1600)])
@pytest.mark.parametrize("fresh", [False, True])
def test_move(B, page, hkv, d, fmt, per_head, n, width, fresh):
    if n * hkv * d > 1 << 20:
        n, width = n // 4, width // 4
    cols = -(-width // page)
    p = Pool(3, cols, page, hkv, d, seed=n, fmt=fmt, fresh=-(-n // page) if fresh else 0)
    src = rising(3, hkv if per_head else 1, n, width, n + d)
    p.check(B, src, [n, 0, n // 2])


@pytest.mark.parametrize("hkv,d,n", [(1, 128, 9001), (2, 256, 3100)])
def test_move_many_rounds(B, hkv, d, n):
    """Lists longer than a round of a cluster, most rows moving into rows that move on."""
    p = Pool(2, -(-(n + 900) // 16), 16, hkv, d, seed=1)
    src = rising(2, 1, n, n + 900, 3)
    p.check(B, src, [n, n - 1])


def test_move_by_one(B):
    """Every row one to the front: each new place is the next row's old one."""
    n = 5000
    p = Pool(1, -(-(n + 1) // 16), 16, 1, 128, seed=2)
    p.check(B, torch.arange(1, n + 1, dtype=torch.int32).view(1, 1, n), [n])


def test_move_any_order(B):
    """Sources in any order, some of them twice, none before its new place; the others are refused."""
    r = np.random.default_rng(4)
    n, width = 2100, 4000
    src = np.maximum(r.integers(0, width, n), np.arange(n)).astype(np.int32)
    p = Pool(1, -(-width // 16), 16, 2, 128, seed=3)
    p.check(B, torch.from_numpy(src).view(1, 1, n), [n])
    src[5], src[1700], src[9] = 4, 3, -2
    p = Pool(1, -(-width // 16), 16, 2, 128, seed=4)
    p.check(B, torch.from_numpy(src).view(1, 1, n), [n], status=B.STATUS_BAD_ENTRIES)
    # to other pages everything but a negative source is taken
    p = Pool(1, -(-width // 16), 16, 2, 128, seed=5, fresh=-(-n // 16))
    p.check(B, torch.from_numpy(src).view(1, 1, n), [n], status=B.STATUS_BAD_ENTRIES, skip=lambda b, l, k: k == 9)


def test_move_accepted_paths(B):
    """Paths of drafted trees behind contexts of any length, on a stream of their own."""
    r = np.random.default_rng(5)
    b, cols, page = 40, 6, 16
    src = np.stack([[np.concatenate([[0], np.sort(r.choice(np.arange(1, 26), 6, replace=False))])] for _ in range(b)])
    count = r.integers(0, 8, b).tolist()
    first = r.integers(0, cols * page - 26, b).tolist()
    p = Pool(b, cols, page, 4, 128, seed=6)
    p.check(B, torch.from_numpy(src.astype(np.int32)), count, first, on=torch.cuda.Stream())


def test_move_interleaved_caches(B):
    for fresh in (0, 40):
        p = Pool(2, 70, 16, 2, 128, seed=7, fresh=fresh, interleaved=True)
        p.check(B, rising(2, 2, 600, 1100, 8), [600, 77])


@pytest.mark.parametrize("fresh", [0, 3])
def test_move_past_32_bits(B, fresh):
    """Pages 600 MB apart: byte offsets up to 6 GB."""
    p = Pool(2, 5, 16, 2, 128, seed=16, fresh=fresh)
    blocks, far = p.k.shape[0], (600 << 20) // 128 * 128
    pool = torch.empty(blocks * far, dtype=torch.uint8, device="cuda")
    assert pool.numel() > 1 << 32
    p.dk = pool.as_strided((blocks, 16, 2, 128), (far, 256, 128, 1))
    p.dv = pool.as_strided((blocks, 16, 2, 128), (far, 256, 128, 1), 4096)
    p.dk.copy_(p.k)
    p.dv.copy_(p.v)
    p.check(B, rising(2, 2, 48, 80, 17), [48, 31])


def test_two_streams_at_once(B):
    """Selections and moves in flight on streams of their own."""
    score = weights(3, 2, 20000, 21)
    x, lens = torch.from_numpy(score).cuda(), torch.tensor([20000, 9000, 100], dtype=torch.int32).cuda()
    outs = [(torch.full((3, 2, 500), -7, dtype=torch.int32, device="cuda"),
             torch.zeros(3, dtype=torch.int32, device="cuda")) for _ in range(2)]
    chosen_by = [B.make_cache_select_args(score=x, kv_len=lens, budget=500, sinks=i, recent=9, keep=keep, n_keep=n)
                 for i, (keep, n) in enumerate(outs)]
    pools = [Pool(2, 70, 16, 2, 128, seed=22 + i) for i in range(2)]
    lists = [rising(2, 2, 600, 1100, 24 + i) for i in range(2)]
    moved = [p.args(B, src, [600, 77 + i]) for i, (p, src) in enumerate(zip(pools, lists))]
    want = [p.expected(src, [600, 77 + i], [0, 0]) for i, (p, src) in enumerate(zip(pools, lists))]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for i in range(2):
        B.fp8kv_attn_cache_select(chosen_by[i], streams[i].cuda_stream)
        B.fp8kv_attn_cache_move(moved[i], streams[2 + i].cuda_stream)
    torch.cuda.synchronize()
    for i, (keep, n_keep) in enumerate(outs):
        assert n_keep.tolist() == [500, 500, 100]
        for b, n in enumerate((20000, 9000, 100)):
            for h in range(2):
                line = chosen(score[b, h:h + 1], n, 500, i, 9)
                assert (keep[b, h, :len(line)].cpu().numpy() == line).all()
        assert torch.equal(pools[i].dk.cpu(), want[i][0]) and torch.equal(pools[i].dv.cpu(), want[i][1])


def test_move_bad_places(B):
    """Positions outside the table and blocks out of range are not moved; counts are clamped."""
    src = rising(2, 1, 100, 200, 9)
    src[0, 0, 99] = 5000
    src[0, 0, 98] = (1 << 31) - 1
    p = Pool(2, 13, 16, 2, 128, seed=8)
    hidden = p.table.clone()
    p.table[1, 3] = -4
    p.table[0, 11] = 1 << 20

    def skip(b, l, k):
        s = int(src[b, l, k])
        if b == 0 and s >= 13 * 16:
            return True
        return any(int(hidden[b, x // 16]) != int(p.table[b, x // 16]) for x in (s, k))

    p.check(B, src, [100, 100], status=B.STATUS_BAD_BLOCK, skip=skip)
    p = Pool(2, 13, 16, 2, 128, seed=8)
    want = p.expected(src[:, :, :90], [90, 0], [0, 0])
    B.fp8kv_attn_cache_move(p.args(B, src[:, :, :90], [1000, -3]), stream())
    torch.cuda.synchronize()
    assert torch.equal(p.dk.cpu(), want[0]) and torch.equal(p.dv.cpu(), want[1])
    assert int(p.status.item()) == B.STATUS_BAD_LEN
    # before position 0
    p = Pool(1, 4, 16, 1, 64, seed=9)
    p.check(B, torch.arange(1, 21, dtype=torch.int32).view(1, 1, 20), [20], [-5], status=B.STATUS_BAD_BLOCK,
            skip=lambda b, l, k: k < 5)


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("fresh", [0, 60])
def test_move_weights(B, per_head, fresh):
    p = Pool(3, 70, 16, 2, 64, seed=10, fresh=fresh)
    n = 900
    src = rising(3, 2 if per_head else 1, n, 1100, 11)
    r = np.random.default_rng(12)
    score = r.random((3, 2, 1100)).astype(np.float32)
    x = torch.from_numpy(score).cuda()
    out = torch.full((3, 3, 1200), -1.0, device="cuda")[:, :2, :1100]
    count = [n, 5, 0]
    want = p.expected(src, count, [0, 0, 0])
    B.fp8kv_attn_cache_move(p.args(B, src, count, score=x, score_out=out), stream())
    torch.cuda.synchronize()
    assert torch.equal(p.dk.cpu(), want[0]) and int(p.status.item()) == 0
    expect = np.full((3, 2, 1100), -1.0, dtype=np.float32)
    for b in range(3):
        for h in range(2):
            line = src[b, h if per_head else 0, :count[b]].numpy()
            expect[b, h, :count[b]] = score[b, h, line]
    assert (out.cpu().numpy() == expect).all()
    # past the weights' row
    short = torch.full((3, 2, 500), -1.0, device="cuda")
    B.fp8kv_attn_cache_move(p.args(B, src, count, score=x[:, :, :500].contiguous(), score_out=short), stream())
    torch.cuda.synchronize()
    assert int(p.status.item()) == B.STATUS_BAD_LEN


def test_move_replay(B):
    p = Pool(2, 40, 16, 2, 128, seed=13)
    src = rising(2, 1, 300, 600, 14).cuda()
    count = torch.tensor([300, 100], dtype=torch.int32).cuda()
    table = p.table.cuda()
    args = B.make_cache_move_args(k_cache=p.dk, v_cache=p.dv, block_table=table, src=src, count=count)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.fp8kv_attn_cache_move(args, stream())
    other = rising(2, 1, 300, 600, 15)
    src.copy_(other)
    count.copy_(torch.tensor([17, 299], dtype=torch.int32))
    want = p.expected(other, [17, 299], [0, 0])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.dk.cpu(), want[0]) and torch.equal(p.dv.cpu(), want[1])


def test_move_nothing(B):
    p = Pool(1, 2, 16, 1, 64)
    p.check(B, torch.zeros(1, 1, 0, dtype=torch.int32), [0])


def test_move_units_that_leave_a_wave_empty(B):
    """More units than half of the GPU's CTAs, in shorter CTAs to other pages; in place one each."""
    for fresh in (0, 30):
        p = Pool(22, 38, 16, 8, 256, seed=18, fresh=fresh)
        p.check(B, rising(22, 8, 470, 600, 19), [470 - 13 * i for i in range(22)])


def test_move_weights_between_views(B):
    """Weights from and to rows of one buffer in turn; views that share a place are refused."""
    p = Pool(3, 20, 16, 2, 64, seed=30)
    src = rising(3, 2, 200, 300, 31)
    both = torch.rand((3, 2, 2, 300), generator=torch.Generator().manual_seed(32)).cuda()
    want = both.cpu()
    for b in range(3):
        for h in range(2):
            want[b, 1, h, :200] = want[b, 0, h, src[b, h].long()]
    B.fp8kv_attn_cache_move(p.args(B, src, [200, 200, 200], score=both[:, 0], score_out=both[:, 1]), stream())
    torch.cuda.synchronize()
    assert torch.equal(both.cpu(), want)
    line = torch.rand(3 * 2 * 300 + 50, device="cuda")
    for k in (0, 1, 50):
        with pytest.raises(B.Fp8kvError) as e:
            B.fp8kv_attn_cache_move(p.args(B, src, [200, 200, 200], score=line[:1800].view(3, 2, 300),
                                           score_out=line[k:k + 1800].view(3, 2, 300)), stream())
        assert e.value.code == B.EINVAL
