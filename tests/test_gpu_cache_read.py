"""GPU parity of the cache read and the scale calibration, and a run of all
cache operators together.

Both compute one correctly rounded FP32 operation per element, so results are
compared bit for bit with the same operation in torch (the product of two
FP32 values is exact in 64 bits; rounding it to FP32 and then to the output
type is the definition).
"""

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


def _read(lens, starts, Hkv, D, page, dtype, fmt, *, spread=False, device_scales=False, seed=0, bad=False):
    from fp8_e4m3_paged_gb300 import binding as B

    g = torch.Generator().manual_seed(seed)
    n = len(lens)
    cols = max(1, -(-max([a + b for a, b in zip(lens, starts)]) // page))
    blocks = n * cols + 1
    k, v = (torch.randint(0, 256, (blocks, page, Hkv, D), generator=g, dtype=torch.uint8) for _ in "kv")
    table = (1 + torch.randperm(n * cols, generator=g)).to(torch.int32).view(n, cols)
    cu = torch.tensor([3] + [3 + sum(lens[:i + 1]) for i in range(n)], dtype=torch.int32)
    total = int(cu[-1]) + 4
    ks, vs = 0.37, -1.9
    shape = (total, Hkv + 1, D + 8) if spread else (total, Hkv, D)
    outs = [torch.full(shape, 5.0, dtype=dtype, device="cuda") for _ in "kv"]
    views = [o[:, :Hkv, :D] for o in outs]
    if bad:
        table[0, 0] = blocks
    dev = [x.cuda() for x in (k, v, table, cu, torch.tensor(starts, dtype=torch.int32))]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sc = dict(k_scale=ks, v_scale=vs)
    if device_scales:
        sc = dict(k_scale_dev=torch.tensor([ks], device="cuda"), v_scale_dev=torch.tensor([vs], device="cuda"))
    a = B.make_cache_read_args(k_cache=dev[0], v_cache=dev[1], block_table=dev[2], cu_len=dev[3], start=dev[4],
                               k_out=views[0], v_out=views[1], status=status,
                               kv_format=B.KV_E4M3 if fmt == "e4m3" else B.KV_E5M2, **sc)
    B.fp8kv_attn_cache_read(a, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    tab = decode_table(fmt).float()
    for cache, scale, out, view in ((k, ks, outs[0], views[0]), (v, vs, outs[1], views[1])):
        want = torch.full((total, Hkv, D), 5.0, dtype=dtype)
        for b in range(n):
            t = torch.arange(starts[b], starts[b] + lens[b])
            blk = table[b].long()[t // page]
            x = tab[cache[blk.clamp(max=blocks - 1), t % page].long()] * torch.tensor(scale, dtype=torch.float32)
            x = torch.where((blk < blocks)[:, None, None], x, 0.0)
            want[int(cu[b]):int(cu[b]) + lens[b]] = x.to(dtype)
        got = view.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        fine = ~torch.isnan(want)
        bits = torch.int32 if dtype == torch.float32 else torch.int16
        assert torch.equal(got.contiguous().view(bits)[fine], want.view(bits)[fine])
        if spread:
            assert (out[:, Hkv:] == 5.0).all() and (out[:, :, D:] == 5.0).all()
    return int(status.item())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("lens,starts,Hkv,D,page", [
    ([1], [0], 1, 16, 1),
    ([5, 0, 130, 1], [0, 7, 3, 99], 2, 128, 16),
    ([300, 17], [1, 1000], 8, 64, 7),
    ([70, 33], [13, 0], 1, 256, 1728),
    ([9, 2], [0, 5], 3, 80, 4),
    ([6], [2], 20, 1024, 3),
])
def test_read_bit_for_bit(lens, starts, Hkv, D, page, dtype, fmt):
    assert _read(lens, starts, Hkv, D, page, dtype, fmt) == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_read_strides_scales_and_many_requests(dtype):
    assert _read([5, 40, 3], [0, 9, 1], 2, 128, 16, dtype, "e4m3", spread=True, device_scales=True) == 0
    assert _read([(i * 7) % 5 for i in range(140)], [i % 11 for i in range(140)], 1, 64, 4, dtype, "e5m2") == 0


def test_read_bad_block_gives_zero_rows():
    from fp8_e4m3_paged_gb300 import binding as B

    assert _read([40, 3], [0, 2], 2, 64, 16, torch.float16, "e4m3", bad=True) == B.STATUS_BAD_BLOCK


def test_read_bad_lengths_stay_in_bounds():
    """A cu_len that decreases or leaves [0, total]: flagged, nothing outside of the rows is written."""
    from fp8_e4m3_paged_gb300 import binding as B

    k = torch.zeros(4, 16, 2, 64, dtype=torch.uint8, device="cuda")
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    for cu in ([0, 20, 10], [-5, 3, 9], [0, 5, 1000], [0, 40, 9]):
        pool = torch.full((30, 2, 64), 5.0, dtype=torch.float16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        a = B.make_cache_read_args(k_cache=k, v_cache=k, block_table=table,
                                   cu_len=torch.tensor(cu, dtype=torch.int32, device="cuda"), k_out=pool[10:20],
                                   v_out=pool[10:20], status=status)
        B.fp8kv_attn_cache_read(a, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert int(status.item()) & B.STATUS_BAD_LEN, cu
        assert (pool[:10] == 5.0).all() and (pool[20:] == 5.0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("N,Hkv,D", [(1, 1, 16), (64, 8, 128), (777, 3, 80), (5000, 2, 256)])
def test_calibrate(N, Hkv, D, dtype, fmt):
    from fp8_e4m3_paged_gb300 import binding as B

    fmax = 448.0 if fmt == "e4m3" else 57344.0
    g = torch.Generator().manual_seed(N)
    k, v = (torch.randn(N, Hkv, D, generator=g).mul_(3).to(dtype) for _ in "kv")
    k.view(-1)[N % 7] = -float(torch.finfo(dtype).max)
    v.view(-1)[-1] = float("inf")
    v.view(-1)[0] = float("nan")
    slots = torch.arange(N, dtype=torch.int64)
    slots[N // 2::3] = -1
    for spread in (False, True):
        for sl in (None, slots):
            kd, vd = k.cuda(), v.cuda()
            if spread:
                w = torch.full((N, Hkv + 1, 2 * D), 60000.0, dtype=dtype, device="cuda")
                w[:, :Hkv, :D], w[:, :Hkv, D:] = kd, vd
                kd, vd = w[:, :Hkv, :D], w[:, :Hkv, D:]
            for start in (1e-6, 1e30):
                ks, vs = (torch.tensor([start], device="cuda") for _ in "kv")
                a = B.make_calibrate_args(k=kd, v=vd, k_scale=ks, v_scale=vs,
                                          slot_mapping=None if sl is None else sl.cuda(),
                                          kv_format=B.KV_E4M3 if fmt == "e4m3" else B.KV_E5M2)
                for _ in range(2):
                    B.fp8kv_attn_cache_calibrate(a, torch.cuda.current_stream().cuda_stream)
                torch.cuda.synchronize()
                for x, s in ((k, ks), (v, vs)):
                    x = x.float() if sl is None else x[sl >= 0].float()
                    x = x[torch.isfinite(x)].abs()
                    top = x.max() / torch.tensor(fmax) if x.numel() else torch.tensor(0.0)
                    assert float(s.cpu()) == max(float(torch.tensor(start)), float(top))


def test_calibrate_write_attend_read():
    """A prompt and two single tokens through one layer: calibrate, write, attend, read back."""
    from fp8_e4m3_paged_gb300 import binding as B

    s = torch.cuda.current_stream().cuda_stream
    g = torch.Generator().manual_seed(1)
    T, Hq, Hkv, D, page, window, sinks = 150, 8, 2, 128, 16, 40, 3
    k, v = (torch.randn(T + 2, Hkv, D, generator=g).half().cuda() for _ in "kv")
    q = torch.randn(T + 2, Hq, D, generator=g).half().cuda()
    cols = -(-(T + 2) // page)
    table = torch.randperm(cols, generator=g).to(torch.int32).view(1, cols).cuda()
    kc, vc = (torch.full((cols, page, Hkv, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.full((1,), 1e-6, device="cuda") for _ in "kv")
    out = torch.zeros_like(q)
    pos = torch.arange(T + 2, device="cuda")
    slots = (table[0].long()[pos // page] * page + pos % page).contiguous()
    for a, b in ((0, T), (T, T + 1), (T + 1, T + 2)):
        if a == 0:
            B.fp8kv_attn_cache_calibrate(B.make_calibrate_args(k=k[a:b], v=v[a:b], k_scale=ks, v_scale=vs), s)
        B.fp8kv_attn_cache_write(B.make_cache_write_args(
            k=k[a:b], v=v[a:b], slot_mapping=slots[a:b], k_cache=kc, v_cache=vc, page_size=page, k_scale_dev=ks,
            v_scale_dev=vs), s)
        plan = B.fp8kv_attn_chunk_plan(B.make_chunk_desc(
            batch=1, total_q=b - a, max_q=b - a, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=D, page_size=page,
            max_kv_len=b, max_blocks=cols, num_kv_blocks=cols, window=window, sinks=sinks))
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        B.fp8kv_attn_chunk(plan, B.make_chunk_args(
            q=q[a:b], k_cache=kc, v_cache=vc, out=out[a:b], workspace=ws, softmax_scale=D ** -0.5, block_table=table,
            cu_q=torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
            kv_len=torch.tensor([b], dtype=torch.int32, device="cuda"), k_scale_dev=ks, v_scale_dev=vs), s)
        torch.cuda.synchronize()
        assert int(ws[:4].view(torch.int32).item()) == 0
    ko, vo = (torch.zeros(T + 2, Hkv, D, dtype=torch.float32, device="cuda") for _ in "kv")
    B.fp8kv_attn_cache_read(B.make_cache_read_args(
        k_cache=kc, v_cache=vc, block_table=table, cu_len=torch.tensor([0, T + 2], dtype=torch.int32, device="cuda"),
        k_out=ko, v_out=vo, k_scale_dev=ks, v_scale_dev=vs), s)
    torch.cuda.synchronize()
    # half a step of e4m3 (2^-4) of each value, or of its subnormal quantum 2^-9 (times the scale); the last two rows
    # may saturate
    for x, y, sc in ((k, ko, ks), (v, vo, vs)):
        step = torch.maximum(x.float().abs() * 2.0 ** -4, sc * 2.0 ** -10)
        assert bool(((y - x.float()).abs()[:T] <= step[:T] * (1 + 2.0 ** -20)).all())
    # the attention over what was read back, in 64 bits
    at = torch.arange(T + 2, device="cuda")
    sees = (at[None] <= at[:, None]) & ((at[:, None] - at[None] < window) | (at[None] < sinks))
    kd, vd = (x.double().repeat_interleave(Hq // Hkv, 1).transpose(0, 1) for x in (ko, vo))
    z = torch.matmul(q.double().transpose(0, 1), kd.transpose(1, 2)) * D ** -0.5
    w = torch.softmax(z.masked_fill(~sees, -float("inf")), -1)
    ref = (w @ vd).transpose(0, 1)
    cond = (w @ vd.abs()).transpose(0, 1)
    # output rounding, probabilities as fp16 (2^-11 each), 2^-14 for the FP32 logits and sums
    assert float(((out.double() - ref).abs() / (ref.abs() * 2.0 ** -11 + cond * (2.0 ** -11 + 2.0 ** -14))).max()) <= 1.0


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_read_positions_outside_of_the_table_give_zero_rows(dtype):
    """Rows before position 0 or past the table: +0.0 whatever the scale's sign, flagged; the others as ever."""
    from fp8_e4m3_paged_gb300 import binding as B

    g = torch.Generator().manual_seed(2)
    k, v = (torch.randint(1, 120, (9, 16, 2, 64), generator=g, dtype=torch.uint8) for _ in "kv")
    table = torch.randperm(8, generator=g).to(torch.int32).view(2, 4)
    for start in ([-3, 60], [-(2 ** 31), 2 ** 31 - 5], [0, 0]):
        lens = [10, 9]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ko, vo = (torch.full((19, 2, 64), 5.0, dtype=dtype, device="cuda") for _ in "kv")
        B.fp8kv_attn_cache_read(B.make_cache_read_args(
            k_cache=k.cuda(), v_cache=v.cuda(), block_table=table.cuda(), k_out=ko, v_out=vo, k_scale=-0.5, v_scale=2.0,
            cu_len=torch.tensor([0, 10, 19], dtype=torch.int32, device="cuda"),
            start=torch.tensor(start, dtype=torch.int32, device="cuda"), status=status),
            torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert int(status.item()) == (0 if start == [0, 0] else B.STATUS_BAD_BLOCK)
        tab = decode_table("e4m3")
        for cache, scale, out in ((k, -0.5, ko.cpu()), (v, 2.0, vo.cpu())):
            for b in range(2):
                for i in range(lens[b]):
                    t, got = start[b] + i, out[10 * b + i]
                    if 0 <= t < 64:
                        assert torch.equal(got, (tab[cache[table[b, t // 16].long(), t % 16].long()] * scale).to(dtype))
                    else:
                        assert (got == 0).all() and not torch.signbit(got).any()
