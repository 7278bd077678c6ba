"""Host-side tests of the chunk attention, cache read and calibration calls
(no GPU needed): struct layouts, plans, refusals.  Calls are made only with
arguments that the host-side validation rejects, or with nothing to do, so
no kernel is launched.
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
    """Size and field offsets of every new struct, as a C compiler sees them."""
    structs = {"fp8kv_chunk_desc": B.ChunkDesc, "fp8kv_chunk_plan_t": B.ChunkPlan, "fp8kv_chunk_args": B.ChunkArgs,
               "fp8kv_cache_read_args": B.CacheReadArgs, "fp8kv_calibrate_args": B.CalibrateArgs}
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


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -1), (dict(total_q=-1), -1), (dict(max_q=0), -1), (dict(num_q_heads=0), -1),
    (dict(num_q_heads=7), -1), (dict(num_kv_heads=0), -1), (dict(page_size=0), -1), (dict(max_kv_len=-1), -1),
    (dict(max_blocks=249), -1), (dict(num_kv_blocks=0), -1), (dict(window=-1), -1), (dict(sinks=-1, window=5), -1),
    (dict(sinks=4), -1), (dict(dtype=2), -1), (dict(kv_format=3), -1), (dict(kv_format=-1), -1),
    (dict(num_splits=-1), -1), (dict(num_splits=1 << 17), -1), (dict(kernel=3), -1), (dict(num_sms=-1), -1),
    (dict(kv_format=2), -2), (dict(head_dim=96), -2), (dict(head_dim=0), -2),
    (dict(kernel=1, max_q=300000, total_q=1 << 20), -2),
    (dict(max_q=(1 << 24) + 1), -2), (dict(total_q=(1 << 30) + 1), -2),
    (dict(max_kv_len=(1 << 30) + 1, max_blocks=(1 << 27)), -2),
    (dict(num_q_heads=1 << 17, num_kv_heads=1 << 17), -2),
])
def test_chunk_plan_rejects(B, kw, code):
    with pytest.raises(B.Fp8kvError) as e:
        B.fp8kv_attn_chunk_plan(_desc(B, **kw))
    assert e.value.code == code


def test_chunk_plan_null(B):
    d = _desc(B)
    assert B.lib.fp8kv_attn_chunk_plan(None, ctypes.byref(B.ChunkPlan())) == B.EINVAL
    assert B.lib.fp8kv_attn_chunk_plan(ctypes.byref(d), None) == B.EINVAL


def test_chunk_plan_workspace_and_windows(B):
    for S in (1, 2, 7):
        p = B.fp8kv_attn_chunk_plan(_desc(B, num_splits=S))
        n = S * 100 * 8 if S > 1 else 0
        assert p.num_splits == S and p.revision == B.REVISION
        assert p.partial_offset >= 4 and p.ml_offset >= p.partial_offset + n * 128 * 4
        assert p.workspace_bytes >= max(256, p.ml_offset + n * 8) and p.workspace_bytes % 256 == 0
    # a window that reaches back over every context is none
    assert B.fp8kv_attn_chunk_plan(_desc(B, window=4000, sinks=4)).window == 0
    p = B.fp8kv_attn_chunk_plan(_desc(B, window=3999, sinks=1 << 30))
    assert p.window == 3999 and p.sinks == 4000
    # no request has more new tokens than there are rows
    assert B.fp8kv_attn_chunk_plan(_desc(B, total_q=5)).max_q == 5
    assert B.fp8kv_attn_chunk_plan(_desc(B, batch=0, total_q=0)).workspace_bytes >= 4
    assert B.fp8kv_attn_chunk_plan(_desc(B, max_q=4)).kernel == B.CHUNK_STREAM


@pytest.mark.parametrize("kw,kernel", [
    (dict(max_q=1), 1), (dict(max_q=4), 1),                       # up to 16 query vectors per KV head
    (dict(max_q=8, max_kv_len=500), 1),                           # 32 on few positions
    (dict(max_q=8, window=300), 1),
    (dict(max_q=8), 2),                                           # 32 on 4000 positions
    (dict(max_q=8, max_kv_len=500, head_dim=256), 1),
    (dict(max_q=8, max_kv_len=2000, head_dim=256), 2),
    (dict(batch=64, total_q=512, max_q=8, max_kv_len=1000), 2),   # ... of many requests
    (dict(batch=64, total_q=512, max_q=8, max_kv_len=500), 1),
    (dict(batch=64, total_q=1024, max_q=16, max_kv_len=500), 2),
    (dict(batch=1, max_q=100, max_kv_len=500), 1),                # 400 of one request
    (dict(batch=0, total_q=0), 1),
])
def test_chunk_plan_chooses_a_kernel(B, kw, kernel):
    assert B.fp8kv_attn_chunk_plan(_desc(B, **kw)).kernel == kernel


def test_chunk_plan_partitions(B):
    def splits(**kw):
        return B.fp8kv_attn_chunk_plan(_desc(B, **kw)).num_splits

    long = dict(batch=1, total_q=2048, max_q=2048, num_q_heads=32, num_kv_heads=8, max_kv_len=32048, max_blocks=2003)
    assert splits(**long) == 4                       # 256 CTAs: 7 waves of a quarter, not 2 whole ones
    assert splits(**dict(long, num_sms=256)) == 1    # one full wave
    # no FP32 sum of the tile kernel over more than 32768 positions
    assert splits(**dict(long, max_kv_len=200000, max_blocks=12500)) >= 7
    # stream kernel: two CTAs per SM, four where each keeps 512 positions
    one = dict(max_q=1, num_q_heads=32, num_kv_heads=8)
    assert splits(batch=16, total_q=16, **dict(one, max_kv_len=300)) == 2
    assert splits(batch=32, total_q=32, **dict(one, max_kv_len=500)) == 1
    assert splits(batch=32, total_q=32, **dict(one, max_kv_len=2000)) == 2
    assert splits(batch=1, total_q=1, **dict(one, max_kv_len=2000)) == 8     # a cluster
    # whatever the sizes, a grid that can be launched
    for sms in (1, 65535):
        for kernel in (1, 2):
            p = B.fp8kv_attn_chunk_plan(_desc(B, batch=1, max_q=1, num_sms=sms, kernel=kernel, max_kv_len=1 << 30,
                                              max_blocks=1 << 26))
            assert 1 <= p.num_splits <= 65535


@pytest.mark.parametrize("kw", [
    dict(num_sms=65536), dict(batch=1 << 30, num_kv_heads=8, max_q=1), dict(batch=(1 << 31) - 1, kernel=1),
])
def test_chunk_plan_refuses_grids(B, kw):
    with pytest.raises(B.Fp8kvError) as e:
        B.fp8kv_attn_chunk_plan(_desc(B, **kw))
    assert e.value.code == -2


def _args(B, plan, **kw):
    a = B.ChunkArgs()
    a.q = a.out = a.k_cache = a.v_cache = a.block_table = a.cu_q = a.kv_len = FAKE
    a.q_stride_token = a.out_stride_token = 1024
    a.q_stride_head = a.out_stride_head = 128
    a.k_stride_block = a.v_stride_block = 4096
    a.k_stride_token = a.v_stride_token = 256
    a.k_stride_head = a.v_stride_head = 128
    a.block_table_stride = plan.max_blocks
    a.softmax_scale = a.k_scale = a.v_scale = 1.0
    a.workspace, a.workspace_bytes = FAKE, plan.workspace_bytes
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(out=0), dict(k_cache=0), dict(v_cache=0), dict(block_table=0), dict(cu_q=0), dict(kv_len=0),
    dict(workspace=0), dict(q=FAKE + 8), dict(out=FAKE + 2), dict(k_cache=FAKE + 1), dict(workspace=FAKE + 16),
    dict(cu_q=FAKE + 2), dict(q_stride_token=1020), dict(q_stride_head=-8), dict(out_stride_head=4),
    dict(k_stride_token=250), dict(v_stride_block=-16), dict(block_table_stride=249),
    dict(softmax_scale=float("nan")), dict(k_scale=float("inf")), dict(v_scale=float("nan")),
])
def test_chunk_rejects_arguments(B, kw):
    plan = B.fp8kv_attn_chunk_plan(_desc(B))
    assert B.lib.fp8kv_attn_chunk(ctypes.byref(plan), ctypes.byref(_args(B, plan, **kw)), None) == B.EINVAL


def test_outputs_in_one_place_are_refused(B):
    """A zero stride would write several rows (heads) to one place; inputs may have one."""
    plan = B.fp8kv_attn_chunk_plan(_desc(B))
    for kw in (dict(out_stride_token=0), dict(out_stride_head=0)):
        assert B.lib.fp8kv_attn_chunk(ctypes.byref(plan), ctypes.byref(_args(B, plan, **kw)), None) == B.EINVAL
    for kw in (dict(ko_stride_token=0), dict(vo_stride_token=0), dict(ko_stride_head=0), dict(vo_stride_head=0)):
        assert B.lib.fp8kv_attn_cache_read(ctypes.byref(_read(B, **kw)), None) == B.EINVAL


def test_more_heads_than_a_row_can_count_are_refused(B):
    assert B.lib.fp8kv_attn_cache_read(ctypes.byref(_read(B, num_kv_heads=65536)), None) == -2
    assert B.lib.fp8kv_attn_cache_calibrate(ctypes.byref(_cal(B, num_kv_heads=65536)), None) == -2


def test_chunk_plan_and_workspace_checks(B):
    plan = B.fp8kv_attn_chunk_plan(_desc(B))
    assert B.lib.fp8kv_attn_chunk(None, ctypes.byref(_args(B, plan)), None) == B.EINVAL
    assert B.lib.fp8kv_attn_chunk(ctypes.byref(plan), None, None) == B.EINVAL
    a = _args(B, plan, workspace_bytes=plan.workspace_bytes - 1)
    assert B.lib.fp8kv_attn_chunk(ctypes.byref(plan), ctypes.byref(a), None) == B.EWORKSPACE
    plan.revision += 1
    assert B.lib.fp8kv_attn_chunk(ctypes.byref(plan), ctypes.byref(_args(B, plan)), None) == B.EVERSION
    # nothing to do: no pointers needed but the workspace
    for kw in (dict(batch=0), dict(total_q=0)):
        plan = B.fp8kv_attn_chunk_plan(_desc(B, **kw))
        a = _args(B, plan, q=0, out=0, k_cache=0, v_cache=0, cu_q=0, kv_len=0, block_table=0)
        assert B.lib.fp8kv_attn_chunk(ctypes.byref(plan), ctypes.byref(a), None) == B.OK


def _read(B, **kw):
    a = B.CacheReadArgs()
    a.batch, a.total, a.num_kv_heads, a.head_dim, a.page_size, a.max_blocks, a.num_kv_blocks = 2, 9, 2, 128, 16, 4, 9
    a.k_cache = a.v_cache = a.block_table = a.cu_len = a.k_out = FAKE
    a.v_out = FAKE + (1 << 20)
    a.kc_stride_block = a.vc_stride_block = 4096
    a.kc_stride_token = a.vc_stride_token = 256
    a.kc_stride_head = a.vc_stride_head = a.ko_stride_head = a.vo_stride_head = 128
    a.ko_stride_token = a.vo_stride_token = 256
    a.block_table_stride = 4
    a.k_scale = a.v_scale = 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(batch=-1), dict(total=-1), dict(num_kv_heads=0), dict(head_dim=24), dict(head_dim=0), dict(head_dim=1040),
    dict(page_size=0), dict(max_blocks=0), dict(num_kv_blocks=0), dict(dtype=3), dict(kv_format=2), dict(k_cache=0),
    dict(v_cache=FAKE + 8), dict(k_out=0), dict(v_out=FAKE + 2), dict(block_table=0), dict(cu_len=0),
    dict(start=FAKE + 1), dict(kc_stride_token=8), dict(vc_stride_head=-16), dict(ko_stride_token=4),
    dict(vo_stride_head=-8), dict(block_table_stride=3), dict(k_scale=float("nan")), dict(v_scale=float("inf")),
])
def test_cache_read_rejects(B, kw):
    assert B.lib.fp8kv_attn_cache_read(ctypes.byref(_read(B, **kw)), None) == B.EINVAL


def test_cache_read_nothing_to_do(B):
    assert B.lib.fp8kv_attn_cache_read(None, None) == B.EINVAL
    for kw in (dict(batch=0), dict(total=0)):
        assert B.lib.fp8kv_attn_cache_read(ctypes.byref(_read(B, k_cache=0, k_out=0, **kw)), None) == B.OK


def _cal(B, **kw):
    a = B.CalibrateArgs()
    a.num_tokens, a.num_kv_heads, a.head_dim = 5, 2, 128
    a.k = a.v = a.k_scale = FAKE
    a.v_scale = FAKE + 4
    a.k_stride_token = a.v_stride_token = 256
    a.k_stride_head = a.v_stride_head = 128
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(num_tokens=-1), dict(num_kv_heads=0), dict(head_dim=8), dict(head_dim=1040), dict(dtype=2),
    dict(kv_format=2), dict(k=0), dict(v=FAKE + 8), dict(k_stride_token=4), dict(v_stride_head=-8),
    dict(k_scale=0), dict(v_scale=0), dict(v_scale=FAKE), dict(k_scale=FAKE + 2), dict(slot_mapping=FAKE + 4),
])
def test_calibrate_rejects(B, kw):
    assert B.lib.fp8kv_attn_cache_calibrate(ctypes.byref(_cal(B, **kw)), None) == B.EINVAL


def test_calibrate_nothing_to_do(B):
    assert B.lib.fp8kv_attn_cache_calibrate(None, None) == B.EINVAL
    assert B.lib.fp8kv_attn_cache_calibrate(ctypes.byref(_cal(B, num_tokens=0, k=0, v=0, k_scale=0)), None) == B.OK


def test_binding_refuses_tensors_that_do_not_fit(B):
    """What the struct cannot carry is checked where it is filled."""
    import torch

    q = torch.zeros(4, 8, 64, dtype=torch.float16)
    cache = torch.zeros(5, 16, 2, 64, dtype=torch.uint8)
    good = dict(q=q, out=torch.zeros_like(q), k_cache=cache, v_cache=cache, workspace=torch.zeros(256, dtype=torch.uint8),
                softmax_scale=1.0, block_table=torch.zeros(2, 3, dtype=torch.int32),
                cu_q=torch.zeros(3, dtype=torch.int32), kv_len=torch.zeros(2, dtype=torch.int32))
    B.make_chunk_args(**good)
    for bad in (dict(q=q.float()), dict(out=q.bfloat16()), dict(out=q[:3]), dict(q=q.transpose(1, 2)),
                dict(k_cache=cache.float()), dict(v_cache=cache[0]), dict(cu_q=torch.zeros(2, dtype=torch.int32)),
                dict(kv_len=torch.zeros(2, dtype=torch.int64)), dict(block_table=torch.zeros(2, 3)),
                dict(k_scale_dev=torch.zeros(2))):
        with pytest.raises(ValueError):
            B.make_chunk_args(**{**good, **bad})
    k = torch.zeros(5, 2, 64, dtype=torch.float16)
    one = torch.ones(1)
    B.make_calibrate_args(k=k, v=k, k_scale=one, v_scale=one)
    for bad in (dict(k=k.float()), dict(v=k[:2]), dict(k_scale=one.double()), dict(v_scale=None),
                dict(slot_mapping=torch.zeros(5, dtype=torch.int32))):
        with pytest.raises(ValueError):
            B.make_calibrate_args(**{**dict(k=k, v=k, k_scale=one, v_scale=one), **bad})
    table, cu = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    good = dict(k_cache=cache, v_cache=cache, block_table=table, cu_len=cu, k_out=k, v_out=k)
    B.make_cache_read_args(**good)
    for bad in (dict(k_out=k.double()), dict(v_out=k.bfloat16()), dict(k_out=k[:, :1]), dict(cu_len=cu[:2]),
                dict(start=cu), dict(block_table=table.long())):
        with pytest.raises(ValueError):
            B.make_cache_read_args(**{**good, **bad})


def _table_calls(B):
    """Both calls that take a block table, as functions of it."""
    import torch

    q = torch.zeros(4, 8, 64, dtype=torch.float16)
    cache = torch.zeros(5, 16, 2, 64, dtype=torch.uint8)
    k = torch.zeros(5, 2, 64, dtype=torch.float16)

    def ints(n):
        return torch.zeros(n, dtype=torch.int32)

    return [lambda t: B.make_chunk_args(q=q, out=torch.zeros_like(q), k_cache=cache, v_cache=cache,
                                        workspace=torch.zeros(256, dtype=torch.uint8), softmax_scale=1.0, block_table=t,
                                        cu_q=ints(t.shape[0] + 1), kv_len=ints(t.shape[0])),
            lambda t: B.make_cache_read_args(k_cache=cache, v_cache=cache, block_table=t, cu_len=ints(t.shape[0] + 1),
                                             k_out=k, v_out=torch.zeros_like(k))]


def test_binding_keeps_a_block_table_inside_its_storage(B):
    """Rows of the table as the call reads them: address + request * stride, inside of the tensor for every request."""
    import torch

    base = torch.arange(24, dtype=torch.int32)
    for call in _table_calls(B):
        for t in (base[:3].view(1, 3).expand(2, -1),          # one row for all requests
                  base.as_strided((3, 4), (2, 1)),             # rows that overlap
                  base[:1].view(1, 1).expand(5, -1)):
            with pytest.raises(ValueError):
                call(t)
        for t in (base.view(4, 6), base.view(4, 6)[:, :5], base.view(4, 6)[::2], base.view(1, 24), base.view(24, 1),
                  base[:6].view(1, 6).expand(1, -1), base.as_strided((1, 6), (0, 1)), base.view(4, 6)[:0]):
            a = call(t)
            assert a.block_table_stride >= t.shape[1]
            if t.shape[0] == 0:
                continue
            end = a.block_table + 4 * ((t.shape[0] - 1) * a.block_table_stride + t.shape[1])
            assert end <= base.data_ptr() + 4 * base.numel()
            for b in range(t.shape[0]):
                at = (a.block_table - base.data_ptr()) // 4 + b * a.block_table_stride
                assert base[at:at + t.shape[1]].tolist() == t[b].tolist()
        with pytest.raises(ValueError):
            call(base.view(6, 4).t())                          # columns not contiguous


def test_binding_compares_plan_and_tensors(B, monkeypatch):
    """A plan made for other sizes than the tensors' would read or write outside of them."""
    import torch

    def call(**kw):
        n = dict(B=2, rows=4, Hq=8, Hkv=2, D=64, page=16, blocks=5, v_blocks=5, v_page=16, v_heads=2, cols=3,
                 dtype=torch.float16)
        n.update(kw)
        q = torch.zeros(n["rows"], n["Hq"], n["D"], dtype=n["dtype"])
        return B.make_chunk_args(
            q=q, out=torch.zeros_like(q), k_cache=torch.zeros(n["blocks"], n["page"], n["Hkv"], 64, dtype=torch.uint8),
            v_cache=torch.zeros(n["v_blocks"], n["v_page"], n["v_heads"], 64, dtype=torch.uint8),
            workspace=torch.zeros(256, dtype=torch.uint8), softmax_scale=1.0,
            block_table=torch.zeros(n["B"], n["cols"], dtype=torch.int32),
            cu_q=torch.zeros(n["B"] + 1, dtype=torch.int32), kv_len=torch.zeros(n["B"], dtype=torch.int32))

    launched = []
    monkeypatch.setattr(B.lib, "fp8kv_attn_chunk", lambda *a: launched.append(a) or B.OK)
    plan = B.fp8kv_attn_chunk_plan(_desc(B, batch=2, total_q=4, max_q=4, head_dim=64, max_kv_len=48, max_blocks=3,
                                         num_kv_blocks=5))
    for kw in (dict(v_page=8), dict(v_heads=1), dict(D=128)):      # tensors that do not belong together
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(B=1), dict(rows=3), dict(Hq=4), dict(Hkv=1, v_heads=1), dict(page=8, v_page=8), dict(blocks=4),
               dict(v_blocks=2), dict(cols=2), dict(dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            B.ChunkCall(plan, call(**kw)).run(0)
    assert not launched
    for kw in ({}, dict(B=3), dict(rows=9), dict(blocks=7, v_blocks=6), dict(cols=4)):
        B.ChunkCall(plan, call(**kw)).run(0)
    assert len(launched) == 5
    B.fp8kv_attn_chunk(plan, _args(B, plan), 0)                    # a struct filled by hand
    assert len(launched) == 6


def test_device_words_off_their_boundary_are_refused(B):
    """Device scales and the status word: a misaligned access would fault."""
    plan = B.fp8kv_attn_chunk_plan(_desc(B))
    for kw in (dict(k_scale_dev=FAKE + 2), dict(v_scale_dev=FAKE + 1)):
        assert B.lib.fp8kv_attn_chunk(ctypes.byref(plan), ctypes.byref(_args(B, plan, **kw)), None) == B.EINVAL
        assert B.lib.fp8kv_attn_cache_read(ctypes.byref(_read(B, **kw)), None) == B.EINVAL
    assert B.lib.fp8kv_attn_cache_read(ctypes.byref(_read(B, status=FAKE + 2)), None) == B.EINVAL


@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("kernel,chains", [(1, 4), (2, 1)])  # FP32 sums of a partition: one per warp, one
def test_no_sum_over_more_than_32768_positions(B, kernel, chains, head_dim):
    """Whatever the batch, the bound of the lengths or the partitions asked for."""
    for n in (32768, 32769, 131072, 131073, 262144, 1 << 20, 1 << 30):
        for batch in (1, 64):
            for splits in (0, 1, 2, 7):
                p = B.fp8kv_attn_chunk_plan(_desc(
                    B, batch=batch, total_q=batch, max_q=1, num_q_heads=32, num_kv_heads=8, head_dim=head_dim,
                    max_kv_len=n, max_blocks=-(-n // 16), kernel=kernel, num_splits=splits))
                per = -(-n // p.num_splits)
                per = -(-per // (64 if kernel == 1 else 128)) * (64 if kernel == 1 else 128)
                assert per <= chains * 32768
                if splits and n <= splits * chains * 16384:  # no more than it takes
                    assert p.num_splits == splits
    # a window bounds the sums by itself
    p = B.fp8kv_attn_chunk_plan(_desc(B, max_kv_len=1 << 30, max_blocks=1 << 26, window=4096, sinks=4, kernel=kernel,
                                      num_splits=1))
    assert p.num_splits == 1


def test_overlapping_outputs_are_refused(B):
    """Rows or heads that share elements: what those would hold depends on timing."""
    plan = B.fp8kv_attn_chunk_plan(_desc(B))
    for st, sh in ((1024, 8), (1024, 120), (1016, 128), (64, 1024), (128, 12792), (256, 384), (8, 8)):
        a = _args(B, plan, out_stride_token=st, out_stride_head=sh)
        assert B.lib.fp8kv_attn_chunk(ctypes.byref(plan), ctypes.byref(a), None) == B.EINVAL
    for kw in (dict(ko_stride_head=120), dict(vo_stride_head=120), dict(ko_stride_token=248), dict(vo_stride_token=128)):
        assert B.lib.fp8kv_attn_cache_read(ctypes.byref(_read(B, **kw)), None) == B.EINVAL


def test_every_layout_without_overlap_is_taken(tmp_path):
    """The check itself against a list of every row's and head's first element, interleaved layouts among them."""
    import random

    rng = random.Random(5)
    D = 128
    cases = [(100, 1024, 8, 8), (100, 64, 8, 1024), (100, 1024, 8, 128), (100, 1000, 8, 128), (100, 128, 8, 12800),
             (100, 128, 8, 12792), (3, 384, 2, 256), (3, 256, 2, 384), (2, 256, 2, 384), (100, 256, 2, 128),
             (100, 256, 2, 384), (4, 640, 3, 384), (1, 0, 8, 128), (1, 0, 8, 120), (100, 128, 1, 0), (100, 120, 1, 0),
             (100, 1 << 62, 8, 128), (100, 1 << 62, 8, 1 << 62)]
    cases += [(rng.randint(1, 9), 8 * rng.randint(0, 80), rng.randint(1, 5), 8 * rng.randint(0, 80))
              for _ in range(3000)]
    src = tmp_path / "layout.cpp"
    src.write_text("""#include <cstdio>
#include "output_layout.h"
int main() {
  long long r, s, h, t;
  while (std::scanf("%lld %lld %lld %lld", &r, &s, &h, &t) == 4)
    std::printf("%d\\n", fp8kv::apart(r, s, h, t, 128));
}
""")
    exe = tmp_path / "layout"
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "fp8_e4m3_paged_gb300", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    got = [x == "1" for x in subprocess.run([str(exe)], input=text, check=True, capture_output=True,
                                            text=True).stdout.split()]
    want = []
    for rows, st, heads, sh in cases:
        at = sorted(r * st + h * sh for r in range(rows) for h in range(heads))
        want.append(all(b - a >= D for a, b in zip(at, at[1:])))
    assert got == want and 300 < sum(want) < len(want) - 300


def test_binding_refuses_tensors_on_several_devices(B, monkeypatch):
    """Tensors of two GPUs in one call: a kernel would fault on the other's memory.  (No GPU here: tensors that say so.)"""
    import torch

    class Elsewhere(torch.Tensor):
        where = "cuda:1"

        @property
        def device(self):
            return torch.device(self.where)

    class There(Elsewhere):
        where = "cuda:0"

    q = torch.zeros(4, 8, 64, dtype=torch.float16)
    k = torch.zeros(5, 2, 64, dtype=torch.float16)
    cache = torch.zeros(5, 16, 2, 64, dtype=torch.uint8)
    i = torch.zeros(3, dtype=torch.int32)
    one = torch.ones(1)
    calls = [(B.make_chunk_args, dict(q=q, out=q.clone(), k_cache=cache, v_cache=cache, softmax_scale=1.0, cu_q=i,
                                      workspace=torch.zeros(256, dtype=torch.uint8), kv_len=i[:2],
                                      block_table=torch.zeros(2, 3, dtype=torch.int32), k_scale_dev=one,
                                      v_scale_dev=one)),
             (B.make_cache_read_args, dict(k_cache=cache, v_cache=cache, cu_len=i, start=i[:2], k_out=k, v_out=k.clone(),
                                           block_table=torch.zeros(2, 3, dtype=torch.int32), k_scale_dev=one,
                                           v_scale_dev=one, status=i[:1])),
             (B.make_calibrate_args, dict(k=k, v=k, k_scale=one, v_scale=one.clone(),
                                          slot_mapping=torch.zeros(5, dtype=torch.int64)))]
    for make, good in calls:
        tensors = [n for n, t in good.items() if isinstance(t, torch.Tensor)]
        make(**good)
        make(**{n: t.as_subclass(There) if n in tensors else t for n, t in good.items()})
        make(**{n: t.as_subclass(There) if n == tensors[0] else t for n, t in good.items()})  # the others on the host
        for other in tensors[1:]:
            with pytest.raises(ValueError, match="several devices"):
                make(**{n: t.as_subclass(There if n != other else Elsewhere) if n in tensors else t
                        for n, t in good.items()})


def test_a_loose_bound_of_new_tokens_is_taken(B):
    """max_q only counts up to the rows that there are, also for the sizes that grids and packed rows allow."""
    p = B.fp8kv_attn_chunk_plan(_desc(B, kernel=1, max_q=1 << 24, num_q_heads=32, num_kv_heads=1))
    assert p.max_q == 100
    p = B.fp8kv_attn_chunk_plan(_desc(B, max_q=1 << 24, num_q_heads=128, num_kv_heads=1))
    assert p.max_q == 100


def test_further_partitions_wait_for_contexts_that_need_them(B):
    """A bound far above the lengths: the partitions that the sum limit adds are not forced on short contexts."""
    one = dict(batch=64, total_q=64, max_q=1, num_q_heads=32, num_kv_heads=8, max_kv_len=1 << 20, max_blocks=1 << 16)
    p = B.fp8kv_attn_chunk_plan(_desc(B, **one))
    assert p.min_splits == 1 and p.num_splits == 16
    p = B.fp8kv_attn_chunk_plan(_desc(B, **one, num_splits=3))
    assert p.min_splits == 3 and p.num_splits == 16
    p = B.fp8kv_attn_chunk_plan(_desc(B, **one, num_splits=20))
    assert p.min_splits == p.num_splits == 20
    for bad in (0, 21):
        p.min_splits = bad
        assert B.lib.fp8kv_attn_chunk(ctypes.byref(p), ctypes.byref(_args(B, p)), None) == B.EINVAL
