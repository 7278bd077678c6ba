"""Host-side tests of the tree attention, the gathered weights, the selection and the move of cached positions (no GPU
needed): struct layouts, plans, refusals of the library and of the binding.  Calls are made only with arguments that the
host-side validation rejects, or with nothing to do, so no kernel is launched.
"""

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # aligned, never dereferenced on the host


@pytest.fixture(scope="module")
def B():
    from fp8_e4m3_paged_gb300 import build_lib

    build_lib.build()
    from fp8_e4m3_paged_gb300 import binding

    return binding


def test_struct_layouts_match_the_header(B, tmp_path):
    """Size and field offsets of every struct, as a C compiler sees them."""
    structs = {"fp8kv_chunk_plan_t": B.ChunkPlan, "fp8kv_tree_args": B.TreeArgs,
               "fp8kv_cache_score_plan_t": B.CacheScorePlan, "fp8kv_cache_score_args": B.CacheScoreArgs,
               "fp8kv_cache_select_args": B.CacheSelectArgs, "fp8kv_cache_move_args": B.CacheMoveArgs}
    lines = ['#include <stdio.h>', '#include "fp8kv_attn.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for cls in structs.values():
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def _desc(B, **kw):
    base = dict(batch=3, total_q=100, max_q=64, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
                max_kv_len=4000, max_blocks=250, num_kv_blocks=900, num_sms=152)
    base.update(kw)
    return B.make_chunk_desc(**base)


BAD_SHAPES = [
    (dict(batch=-1), -1), (dict(total_q=-1), -1), (dict(max_q=0), -1), (dict(num_q_heads=7), -1),
    (dict(num_kv_heads=0), -1), (dict(page_size=0), -1), (dict(max_kv_len=-1), -1), (dict(max_blocks=249), -1),
    (dict(num_kv_blocks=0), -1), (dict(dtype=2), -1), (dict(kv_format=3), -1), (dict(num_splits=-1), -1),
    (dict(kernel=3), -1), (dict(num_sms=-1), -1), (dict(kv_format=2), -2), (dict(head_dim=96), -2),
]


def _rejects(B, call, code):
    with pytest.raises(B.Fp8kvError) as e:
        call()
    assert e.value.code == code


# ---------------------------------------------------------------- tree attention

@pytest.mark.parametrize("kw,code", BAD_SHAPES + [(dict(total_q=2000, max_q=1025), -2), (dict(sinks=1), -1)])
def test_tree_plan_rejects(B, kw, code):
    _rejects(B, lambda: B.fp8kv_attn_tree_plan(_desc(B, **kw)), code)


def test_tree_plan(B):
    p = B.fp8kv_attn_tree_plan(_desc(B))
    assert p.tree == 1 and p.revision == B.REVISION and p.workspace_bytes % 256 == 0
    assert B.fp8kv_attn_chunk_plan(_desc(B)).tree == 0
    assert B.fp8kv_attn_tree_plan(_desc(B, total_q=2000, max_q=1024)).max_q == 1024
    assert B.fp8kv_attn_tree_plan(_desc(B, total_q=5, max_q=4000)).max_q == 5  # no tree has more nodes than there are rows
    # a window that reaches back over every context is none
    assert B.fp8kv_attn_tree_plan(_desc(B, window=4000, sinks=4)).window == 0
    # no FP32 sum over more than 32768 positions, whoever chose the partitions
    for batch in (1, 2, 16, 100):
        for kernel, most in ((B.CHUNK_TILE, 32768), (B.CHUNK_STREAM, 65536)):
            for splits in (0, 1):
                n = 1 << 20
                p = B.fp8kv_attn_tree_plan(_desc(B, batch=batch, total_q=64 * batch, max_kv_len=n, max_blocks=n // 16,
                                                 kernel=kernel, num_splits=splits))
                assert p.num_splits * min(p.max_part, most) >= n or p.per_head > 0
                if p.per_head > 0:
                    assert p.per_head * p.num_kv_heads <= 152 + batch * p.num_kv_heads and p.num_splits >= p.per_head
                rows = p.num_splits * p.total_q * p.num_q_heads if p.num_splits > 1 else 0
                if kernel == B.CHUNK_TILE:
                    assert p.ml_offset >= p.partial_offset + rows * 128 * 4 and p.workspace_bytes >= p.ml_offset + rows * 8


def test_tree_plan_null(B):
    d = _desc(B)
    assert B.lib.fp8kv_attn_tree_plan(None, ctypes.byref(B.ChunkPlan())) == B.EINVAL
    assert B.lib.fp8kv_attn_tree_plan(ctypes.byref(d), None) == B.EINVAL


def _tree_args(B, plan, **kw):
    a = B.TreeArgs()
    c = a.chunk
    for f in ("q", "out", "k_cache", "v_cache", "block_table", "cu_q", "kv_len", "workspace"):
        setattr(c, f, FAKE)
    c.q_stride_token, c.q_stride_head = 1024, 128
    c.out_stride_token, c.out_stride_head = 1024, 128
    c.k_stride_block, c.k_stride_token, c.k_stride_head = 4096, 256, 128
    c.v_stride_block, c.v_stride_token, c.v_stride_head = 4096, 256, 128
    c.block_table_stride = 250
    c.softmax_scale = c.k_scale = c.v_scale = 1.0
    c.workspace_bytes = plan.workspace_bytes
    a.mask, a.mask_stride, a.depth = FAKE, 2, FAKE
    for k, v in kw.items():
        setattr(c if hasattr(c, k) else a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(mask=None), -1), (dict(mask=FAKE + 2), -1), (dict(mask_stride=1), -1), (dict(mask_stride=-4), -1),
    (dict(q=None), -1), (dict(q=FAKE + 8), -1), (dict(out=None), -1), (dict(k_cache=FAKE + 4), -1),
    (dict(block_table=None), -1), (dict(block_table_stride=249), -1), (dict(cu_q=None), -1), (dict(kv_len=FAKE + 1), -1),
    (dict(workspace=None), -1), (dict(workspace=FAKE + 64), -1), (dict(workspace_bytes=0), -3),
    (dict(q_stride_token=1020), -1), (dict(k_stride_head=8), -1), (dict(out_stride_head=64), -1),
    (dict(softmax_scale=float("nan")), -1), (dict(v_scale=float("inf")), -1),
])
def test_tree_rejects(B, kw, code):
    plan = B.fp8kv_attn_tree_plan(_desc(B))
    _rejects(B, lambda: B.fp8kv_attn_tree(plan, _tree_args(B, plan, **kw)), code)


def test_tree_rejects_other_plans(B):
    plan = B.fp8kv_attn_tree_plan(_desc(B))
    chunk = B.fp8kv_attn_chunk_plan(_desc(B))
    _rejects(B, lambda: B.fp8kv_attn_tree(chunk, _tree_args(B, plan, workspace_bytes=1 << 30)), -1)
    _rejects(B, lambda: B.fp8kv_attn_chunk(plan, _tree_args(B, plan).chunk), -1)
    plan.revision += 1
    _rejects(B, lambda: B.fp8kv_attn_tree(plan, _tree_args(B, plan)), -4)
    # a window needs depths
    plan = B.fp8kv_attn_tree_plan(_desc(B, window=100))
    _rejects(B, lambda: B.fp8kv_attn_tree(plan, _tree_args(B, plan, depth=None)), -1)
    _rejects(B, lambda: B.fp8kv_attn_tree(plan, _tree_args(B, plan, depth=FAKE + 2)), -1)
    assert B.lib.fp8kv_attn_tree(ctypes.byref(plan), None, None) == B.EINVAL
    assert B.lib.fp8kv_attn_tree(None, ctypes.byref(_tree_args(B, plan)), None) == B.EINVAL


def test_tree_nothing_to_do(B):
    for kw in (dict(batch=0, total_q=0), dict(total_q=0)):
        plan = B.fp8kv_attn_tree_plan(_desc(B, **kw))
        a = B.TreeArgs()
        a.chunk.workspace, a.chunk.workspace_bytes = FAKE, plan.workspace_bytes
        B.fp8kv_attn_tree(plan, a)


# ---------------------------------------------------------------- gathered weights

@pytest.mark.parametrize("kw,code", BAD_SHAPES + [
    (dict(window=100), -2), (dict(sinks=1), -1), (dict(kernel=1, max_q=65), -2),
    (dict(max_kv_len=(1 << 26) + 1, max_blocks=1 << 23), -2), (dict(batch=40000, total_q=40000, max_q=1), -2),
    (dict(num_splits=65536), -1),
])
def test_score_plan_rejects(B, kw, code):
    _rejects(B, lambda: B.fp8kv_attn_cache_score_plan(_desc(B, **kw)), code)


def test_score_plan(B):
    for kw in (dict(max_q=1), dict(max_q=4), dict(max_q=64), dict(max_q=3000, total_q=5000), dict(batch=64, total_q=64, max_q=1),
               dict(max_kv_len=1 << 26, max_blocks=1 << 22), dict(max_kv_len=1 << 26, max_blocks=1 << 22, num_sms=65535),
               dict(max_kv_len=1 << 26, max_blocks=1 << 22, max_q=4, batch=1), dict(max_kv_len=0, max_blocks=0),
               dict(max_kv_len=1 << 20, max_blocks=1 << 16, batch=256, total_q=256, max_q=1, num_q_heads=32, num_kv_heads=8), dict(num_splits=7),
               dict(head_dim=256, max_q=40), dict(batch=0, total_q=0), dict(num_kv_heads=8, num_sms=4),
               dict(num_kv_heads=8, num_sms=4, batch=0, total_q=0, kernel=2),
               dict(max_kv_len=1 << 26, max_blocks=1 << 22, max_q=1, num_splits=1, kernel=1)):
        p = B.fp8kv_attn_cache_score_plan(_desc(B, **kw))
        rows = p.max_q * p.group
        pairs = p.batch * p.num_kv_heads
        if "kernel" not in kw and rows <= 16 and pairs * p.max_kv_len * 64 <= 1 << 32:
            assert p.kernel == B.CHUNK_STREAM
        if p.kernel == B.CHUNK_STREAM:  # FP32 sums, whoever chose the partitions
            assert p.stat_part <= 65536 and p.num_splits * p.stat_part >= p.max_kv_len
        assert "kernel" in kw or p.kernel == B.CHUNK_TILE or rows <= 256 and 4 * pairs * p.max_kv_len * p.vectors <= 1 << 32
        assert -(-p.max_kv_len // p.col_part) <= 65535 and 1 <= p.num_splits <= 65535
        keep = pairs * p.max_kv_len * (p.vectors if p.kernel == B.CHUNK_STREAM else p.row_groups if p.row_groups > 1 else 0)
        assert p.ml_offset >= p.partial_offset + 4 * keep
        assert p.workspace_bytes >= p.ml_offset + 8 * p.num_splits * p.total_q * p.num_q_heads
        if p.kernel == B.CHUNK_STREAM:
            assert p.vectors >= rows and (p.vectors in (4, 8) or p.vectors % 16 == 0)
        assert p.per_head > 0 or p.num_splits * p.stat_part >= p.max_kv_len
        # positions whose sums meet in shared memory
        assert p.kernel == B.CHUNK_STREAM or rows <= 128 or p.per_head > 0 or p.col_part <= 2048
    assert B.lib.fp8kv_attn_cache_score_plan(None, ctypes.byref(B.CacheScorePlan())) == B.EINVAL
    assert B.lib.fp8kv_attn_cache_score_plan(ctypes.byref(_desc(B)), None) == B.EINVAL


def _score_args(B, plan, **kw):
    a = B.CacheScoreArgs()
    for f in ("q", "k_cache", "block_table", "cu_q", "kv_len", "workspace", "score"):
        setattr(a, f, FAKE)
    a.score_in = FAKE * 2
    a.q_stride_token, a.q_stride_head = 1024, 128
    a.k_stride_block, a.k_stride_token, a.k_stride_head = 4096, 256, 128
    a.block_table_stride = 250
    a.score_stride_req, a.score_stride_head = 8000, 4000
    a.score_in_stride_req, a.score_in_stride_head = 8000, 4000
    a.softmax_scale = a.k_scale = a.decay = 1.0
    a.workspace_bytes = plan.workspace_bytes
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(q=FAKE + 8), -1), (dict(k_cache=None), -1), (dict(k_cache=FAKE + 8), -1),
    (dict(block_table=None), -1), (dict(block_table_stride=249), -1), (dict(cu_q=None), -1), (dict(kv_len=None), -1),
    (dict(score=None), -1), (dict(score=FAKE + 2), -1), (dict(score_in=FAKE + 1), -1), (dict(score_stride_head=3999), -1),
    (dict(score_stride_req=-8), -1), (dict(score_in_stride_head=-1), -1), (dict(score_in=FAKE, score_in_stride_req=9000), -1),
    (dict(softmax_scale=float("inf")), -1), (dict(decay=float("nan")), -1), (dict(k_scale=float("nan")), -1),
    (dict(k_scale_dev=FAKE + 2), -1), (dict(q_stride_head=4), -1), (dict(k_stride_token=8), -1),
    (dict(workspace=None), -1), (dict(workspace=FAKE + 16), -1), (dict(workspace_bytes=0), -3),
])
def test_score_rejects(B, kw, code):
    for max_q in (1, 64):
        plan = B.fp8kv_attn_cache_score_plan(_desc(B, max_q=max_q))
        _rejects(B, lambda: B.fp8kv_attn_cache_score(plan, _score_args(B, plan, **kw)), code)


def test_score_stale_plan_and_nothing_to_do(B):
    plan = B.fp8kv_attn_cache_score_plan(_desc(B))
    plan.revision += 1
    _rejects(B, lambda: B.fp8kv_attn_cache_score(plan, _score_args(B, plan)), -4)
    assert B.lib.fp8kv_attn_cache_score(ctypes.byref(plan), None, None) == B.EINVAL
    for kw in (dict(batch=0, total_q=0), dict(total_q=0), dict(max_kv_len=0, max_blocks=0)):
        plan = B.fp8kv_attn_cache_score_plan(_desc(B, **kw))
        a = B.CacheScoreArgs()
        a.workspace, a.workspace_bytes = FAKE, plan.workspace_bytes
        B.fp8kv_attn_cache_score(plan, a)


# ---------------------------------------------------------------- selection, move

def _select_args(B, **kw):
    a = B.CacheSelectArgs()
    a.batch, a.num_kv_heads, a.lists, a.max_len = 3, 2, 2, 1000
    a.budget, a.sinks, a.recent = 100, 4, 10
    a.score = a.kv_len = a.keep = FAKE
    a.n_keep = FAKE << 20
    a.score_stride_req, a.score_stride_head = 2000, 1000
    a.keep_stride_req, a.keep_stride_list = 200, 100
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -1), (dict(num_kv_heads=0), -1), (dict(lists=3), -1), (dict(lists=0), -1), (dict(max_len=-1), -1),
    (dict(budget=0), -1), (dict(sinks=-1), -1), (dict(recent=-1), -1), (dict(sinks=50, recent=51), -1),
    (dict(sinks=1 << 30, recent=1 << 30, budget=(1 << 31) - 1), -1), (dict(score=None), -1), (dict(score=FAKE + 2), -1),
    (dict(kv_len=None), -1), (dict(keep=None), -1), (dict(keep=FAKE + 1), -1), (dict(n_keep=None), -1),
    (dict(status=FAKE + 2), -1), (dict(score_stride_req=-1), -1), (dict(keep_stride_list=99), -1),
    (dict(keep_stride_req=150), -1), (dict(num_kv_heads=65536, lists=1), -2), (dict(max_len=(1 << 30) + 1), -2),
    (dict(batch=1 << 28, lists=1, num_kv_heads=1, keep_stride_req=100), -2),
    # the lengths are read while the numbers kept are written
    (dict(n_keep=FAKE), -1), (dict(n_keep=FAKE + 8), -1), (dict(n_keep=FAKE - 8), -1),
    (dict(n_keep=FAKE, batch=1, lists=1, num_kv_heads=1), -1),
])
def test_select_rejects(B, kw, code):
    _rejects(B, lambda: B.fp8kv_attn_cache_select(_select_args(B, **kw)), code)


def _move_args(B, **kw):
    a = B.CacheMoveArgs()
    a.batch, a.num_kv_heads, a.lists, a.max_count, a.head_dim, a.page_size = 3, 2, 2, 100, 128, 16
    a.max_blocks, a.num_kv_blocks = 20, 100
    a.k_cache = a.v_cache = a.block_table = a.src = a.count = FAKE
    a.kc_stride_block, a.kc_stride_token, a.kc_stride_head = 4096, 256, 128
    a.vc_stride_block, a.vc_stride_token, a.vc_stride_head = 4096, 256, 128
    a.block_table_stride, a.dst_table_stride = 20, 20
    a.src_stride_req, a.src_stride_list = 200, 100
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -1), (dict(num_kv_heads=0), -1), (dict(lists=3), -1), (dict(max_count=-1), -1), (dict(head_dim=8), -1),
    (dict(head_dim=1040), -1), (dict(head_dim=24), -1), (dict(page_size=0), -1), (dict(max_blocks=0), -1),
    (dict(num_kv_blocks=0), -1), (dict(kv_format=3), -1), (dict(kv_format=-1), -1), (dict(k_cache=None), -1),
    (dict(v_cache=FAKE + 8), -1), (dict(kc_stride_token=8), -1), (dict(vc_stride_head=-16), -1), (dict(block_table=None), -1),
    (dict(block_table_stride=19), -1), (dict(dst_table=FAKE * 2, dst_max_blocks=0), -1),
    (dict(dst_table=FAKE * 2, dst_max_blocks=9, dst_table_stride=8), -1),
    (dict(dst_table=FAKE + 2, dst_max_blocks=1, dst_table_stride=1), -1), (dict(dst_table=FAKE, dst_max_blocks=20), -1),
    (dict(src=None), -1), (dict(src=FAKE + 2), -1), (dict(count=None), -1), (dict(first=FAKE + 1), -1), (dict(status=FAKE + 2), -1),
    (dict(src_stride_list=-1), -1), (dict(score=FAKE), -1), (dict(score_out=FAKE), -1),
    (dict(score=FAKE, score_out=FAKE, max_len=10, score_out_stride_req=20, score_out_stride_head=10), -1),
    (dict(score=FAKE, score_out=FAKE * 2, max_len=0), -1),
    (dict(score=FAKE, score_out=FAKE * 2, max_len=10, score_out_stride_req=20, score_out_stride_head=9), -1),
    (dict(num_kv_heads=65536, lists=1), -2), (dict(max_count=(1 << 30) + 1), -2),
])
def test_move_rejects(B, kw, code):
    _rejects(B, lambda: B.fp8kv_attn_cache_move(_move_args(B, **kw)), code)


def test_select_and_move_nothing_to_do(B):
    B.fp8kv_attn_cache_select(_select_args(B, batch=0, score=None, kv_len=None, keep=None, n_keep=None))
    B.fp8kv_attn_cache_move(_move_args(B, batch=0, k_cache=None, src=None))
    B.fp8kv_attn_cache_move(_move_args(B, max_count=0, k_cache=None, src=None))
    assert B.lib.fp8kv_attn_cache_select(None, None) == B.EINVAL
    assert B.lib.fp8kv_attn_cache_move(None, None) == B.EINVAL


# ---------------------------------------------------------------- binding

def _tensors():
    import torch

    t = dict(q=torch.zeros(5, 4, 128, dtype=torch.float16), out=torch.zeros(5, 4, 128, dtype=torch.float16),
             cache=torch.zeros(9, 16, 2, 128, dtype=torch.uint8), ws=torch.zeros(4096, dtype=torch.uint8),
             table=torch.zeros(3, 4, dtype=torch.int32), cu=torch.zeros(4, dtype=torch.int32),
             n=torch.zeros(3, dtype=torch.int32), mask=torch.zeros(5, 2, dtype=torch.int32),
             score=torch.zeros(3, 2, 64), keep=torch.zeros(3, 2, 10, dtype=torch.int32))
    return torch, t


def test_binding_checks_tree(B):
    torch, t = _tensors()
    base = dict(q=t["q"], k_cache=t["cache"], v_cache=t["cache"], out=t["out"], workspace=t["ws"], softmax_scale=1.0,
                block_table=t["table"], cu_q=t["cu"], kv_len=t["n"], mask=t["mask"], depth=torch.zeros(5, dtype=torch.int32))
    a = B.make_tree_args(**base)
    assert a.words == 2 and a.mask_stride == 2
    wide = torch.zeros(5, 7, dtype=torch.int32)[:, :2]
    assert B.make_tree_args(**{**base, "mask": wide}).mask_stride == 7
    for bad in (dict(mask=t["mask"].long()), dict(mask=t["mask"][:4]), dict(mask=t["mask"].t().contiguous().t()[:, ::1].t()),
                dict(mask=t["mask"][0]), dict(depth=torch.zeros(4, dtype=torch.int32)), dict(depth=torch.zeros(5)),
                dict(out=t["out"][:4]), dict(q=t["q"].float())):
        with pytest.raises(ValueError):
            B.make_tree_args(**{**base, **bad})
    # fewer words than the plan's nodes take, other sizes than the plan's
    plan = B.fp8kv_attn_tree_plan(_desc(B, total_q=100, max_q=65, num_q_heads=4, max_kv_len=60, max_blocks=4, num_kv_blocks=9))
    with pytest.raises(ValueError):
        B.fp8kv_attn_tree(plan, a)
    plan = B.fp8kv_attn_tree_plan(_desc(B, total_q=5, max_q=5, num_q_heads=8, max_kv_len=60, max_blocks=4, num_kv_blocks=9))
    with pytest.raises(ValueError):
        B.fp8kv_attn_tree(plan, a)


def test_binding_checks_score(B):
    torch, t = _tensors()
    base = dict(q=t["q"], k_cache=t["cache"], workspace=t["ws"], softmax_scale=1.0, block_table=t["table"], cu_q=t["cu"],
                kv_len=t["n"], score=t["score"], score_in=t["score"])
    a = B.make_cache_score_args(**base)
    assert a.positions == 64 and a.score_in == a.score
    for bad in (dict(score=t["score"].double()), dict(score=t["score"][:2]), dict(score=t["score"][:, :1]),
                dict(score=t["score"][..., ::2]), dict(score_in=t["score"][..., :60]), dict(score_in=t["score"].half()),
                dict(kv_len=t["n"].long()), dict(cu_q=t["n"]), dict(q=t["q"][..., :64]), dict(k_scale_dev=torch.zeros(2))):
        with pytest.raises(ValueError):
            B.make_cache_score_args(**{**base, **bad})
    for over in (dict(max_kv_len=65, max_blocks=4 + 1), dict(batch=4), dict(total_q=6), dict(num_kv_heads=4)):
        d = dict(total_q=5, max_q=1, num_q_heads=4, max_kv_len=60, max_blocks=4, num_kv_blocks=9)
        plan = B.fp8kv_attn_cache_score_plan(_desc(B, **{**d, **over}))
        with pytest.raises(ValueError):
            B.fp8kv_attn_cache_score(plan, a)


def test_binding_checks_select_and_move(B):
    torch, t = _tensors()
    base = dict(score=t["score"], kv_len=t["n"], budget=10, keep=t["keep"], n_keep=t["n"].clone())
    a = B.make_cache_select_args(**base)
    assert (a.batch, a.num_kv_heads, a.lists, a.max_len) == (3, 2, 2, 64)
    assert B.make_cache_select_args(**{**base, "keep": t["keep"][:, :1]}).lists == 1
    for bad in (dict(budget=11), dict(keep=t["keep"].long()), dict(keep=t["keep"][:2]), dict(keep=t["keep"][..., ::2], budget=5),
                dict(kv_len=t["n"][:2]), dict(score=t["score"].half()), dict(score=t["score"][..., ::2]),
                dict(status=torch.zeros(2, dtype=torch.int32)), dict(n_keep=t["n"].long()),
                dict(keep=torch.zeros(3, 3, 10, dtype=torch.int32))):
        with pytest.raises(ValueError):
            B.make_cache_select_args(**{**base, **bad})
    base = dict(k_cache=t["cache"], v_cache=t["cache"].clone(), block_table=t["table"], src=t["keep"], count=t["n"])
    a = B.make_cache_move_args(**base)
    assert (a.batch, a.lists, a.max_count, a.num_kv_heads, a.head_dim, a.kc_stride_token) == (3, 2, 10, 2, 128, 256)
    wide = torch.zeros(9, 16, 2, 128, dtype=torch.bfloat16)
    a = B.make_cache_move_args(**{**base, "k_cache": wide, "v_cache": wide.clone(), "kv_format": B.KV_BF16})
    assert a.kc_stride_token == 512 and a.head_dim == 128
    for bad in (dict(k_cache=wide), dict(v_cache=t["cache"][:8]), dict(kv_format=B.KV_BF16), dict(src=t["keep"].long()),
                dict(src=t["keep"][:2]), dict(src=torch.zeros(3, 3, 10, dtype=torch.int32)), dict(count=t["n"][:2]),
                dict(first=t["n"].long()), dict(dst_table=t["table"][:2]), dict(dst_table=t["table"].long()),
                dict(score=t["score"]), dict(score_out=t["score"]), dict(score=t["score"], score_out=t["score"][..., :60]),
                dict(score=t["score"][:2], score_out=t["score"][:2]), dict(block_table=t["table"].expand(3, 4).t())):
        with pytest.raises(ValueError):
            B.make_cache_move_args(**{**base, **bad})


# ---------------------------------------------------------------- weights that share places

def test_meet(tmp_path):
    """Whether rows of two arrays share a place, against all pairs of them."""
    import numpy as np

    r = np.random.default_rng(11)
    L, cases = 8, []
    for _ in range(4000):
        x, y = ([int(r.integers(1, 6)), int(r.integers(0, 90)), int(r.integers(1, 5)), int(r.integers(0, 60))] for _ in "xy")
        kind = r.integers(0, 4)
        if kind == 1:  # the same strides
            y[1], y[3] = x[1], x[3]
        elif kind == 2:  # rows of one buffer in turn
            x[3], x[1] = 2 * L, 2 * L * x[2]
            y[1:] = x[1:]
        elif kind == 3:
            y[1] = x[1]
        cases.append((*x, *y, int(r.integers(-400, 400)) if kind != 2 else int(r.choice([-L - 1, -L, L, L - 1, L + 1, 0, 5 * L]))))
    src = tmp_path / "meet.cpp"
    src.write_text("""#include <cstdio>
#include "output_layout.h"
int main() {
  long long a[9];
  while (true) {
    for (auto& x : a)
      if (std::scanf("%lld", &x) != 1) return 0;
    std::printf("%d\\n", fp8kv::meet({a[0], a[1], a[2], a[3]}, {a[4], a[5], a[6], a[7]}, 8, a[8]));
  }
}
""")
    exe = tmp_path / "meet"
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "fp8_e4m3_paged_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    got = [x == "1" for x in subprocess.run([str(exe)], input=text, check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for c in cases:
        starts = [(np.arange(c[i])[:, None] * c[i + 1] + np.arange(c[i + 2])[None] * c[i + 3]).ravel() for i in (0, 4)]
        want.append(bool((np.abs(starts[1][None] + c[8] - starts[0][:, None]) < L).any()))
    assert got == want and 500 < sum(want) < len(want) - 500


SHARED = [  # (first places in floats, strides by request and head) of the weights read, and of those written; rows of 10
    ((0, 20, 10), (5, 20, 10)),     # some elements on
    ((5, 20, 10), (0, 20, 10)),     # ... back
    ((0, 20, 10), (59, 20, 10)),    # the last one
    ((0, 40, 10), (10, 40, 10)),    # another head's row of the same buffer
    ((0, 40, 20), (15, 40, 20)),    # rows in turn, too near
    ((0, 20, 10), (0, 40, 20)),     # the same rows, other strides
    ((0, 0, 0), (9, 30, 10)),       # one row for all
]
APART = [
    ((0, 20, 10), (60, 20, 10)),
    ((60, 20, 10), (0, 20, 10)),
    ((0, 40, 20), (10, 40, 20)),    # rows in turn
    ((0, 40, 10), (20, 40, 10)),    # requests in turn
    ((0, 100, 10), (20, 100, 40)),  # other strides
    ((0, 0, 0), (10, 30, 10)),
]


@pytest.mark.parametrize("read,written", SHARED)
def test_weights_that_share_places_are_refused(B, read, written):
    at = 4 * read[0] + FAKE, 4 * written[0] + FAKE
    kw = dict(score=at[0], score_out=at[1], max_len=10, score_stride_req=read[1], score_stride_head=read[2],
              score_out_stride_req=written[1], score_out_stride_head=written[2])
    _rejects(B, lambda: B.fp8kv_attn_cache_move(_move_args(B, **kw)), -1)
    for max_q in (1, 64):
        plan = B.fp8kv_attn_cache_score_plan(_desc(B, max_q=max_q, max_kv_len=10))
        kw = dict(score_in=at[0], score=at[1], score_in_stride_req=read[1], score_in_stride_head=read[2],
                  score_stride_req=written[1], score_stride_head=written[2])
        _rejects(B, lambda: B.fp8kv_attn_cache_score(plan, _score_args(B, plan, **kw)), -1)


@pytest.mark.parametrize("read,written", APART)
def test_weights_beside_each_other_are_taken(B, tmp_path, read, written):
    """Views of one buffer whose rows share no place.  (The check itself: a call that passes it would launch.)"""
    src = tmp_path / "apart.cpp"
    src.write_text(f"""#include "output_layout.h"
int main() {{
  return fp8kv::meet({{3, {read[1]}, 2, {read[2]}}}, {{3, {written[1]}, 2, {written[2]}}}, 10, {written[0] - read[0]});
}}
""")
    exe = tmp_path / "apart"
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "fp8_e4m3_paged_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    assert subprocess.run([str(exe)]).returncode == 0
