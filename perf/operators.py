"""The operators around a quantised paged cache, as cases to measure.

Four operators: attention of a ragged batch of new tokens over the paged FP8
cache ("attention" with window 0), the same with a sliding window and a few
first tokens that stay visible ("attention" with a window), reading rows back
out of the cache ("read"), and the running scale of the rows about to be
written ("calibrate").  With ``own`` false, ``run`` computes them with
elementary torch operations in 32 bits; with ``own`` true it makes the calls
of this package.
"""

import torch

own = False

#: largest finite value of each cache format
_FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _attention(name, **kw):
    return dict(name=name, op="attention", **kw)


def listed():
    return [
        # The first step after a short prompt: one new token, one request, all of its context visible.
        _attention("chunk_one_token", batch=1, q_lo=1, q_hi=1, ctx_lo=611, ctx_hi=611, heads=6, kv_heads=1,
                   dim=256, page=16, window=0, sinks=0, dtype="f16", fmt="e4m3"),
        # A continuous batch: decoding requests beside requests in the middle of their prompt.
        _attention("chunk_mixed_batch", batch=16, q_lo=1, q_hi=509, ctx_lo=100, ctx_hi=8000, heads=32, kv_heads=8,
                   dim=128, page=16, window=0, sinks=0, dtype="bf16", fmt="e4m3"),
        # One piece of a long prompt: 2048 new tokens on 30000 that are already cached.
        _attention("chunk_long_prompt", batch=1, q_lo=2048, q_hi=2048, ctx_lo=30000, ctx_hi=30000, heads=32,
                   kv_heads=8, dim=128, page=16, window=0, sinks=0, dtype="f16", fmt="e4m3"),
        # Wide heads, one KV head, big pages: 1000 new tokens on 8192.
        _attention("chunk_wide_heads", batch=1, q_lo=1000, q_hi=1000, ctx_lo=8192, ctx_hi=8192, heads=6, kv_heads=1,
                   dim=256, page=3296, window=0, sinks=0, dtype="f16", fmt="e4m3"),
        # One decode step of a batch of 64 in a windowed layer.
        _attention("window_decode_batch", batch=64, q_lo=1, q_hi=1, ctx_lo=512, ctx_hi=65536, heads=32, kv_heads=8,
                   dim=128, page=16, window=4096, sinks=4, dtype="f16", fmt="e4m3"),
        # One decode step of one long request in a windowed layer (latency).
        _attention("window_decode_one", batch=1, q_lo=1, q_hi=1, ctx_lo=131071, ctx_hi=131071, heads=16, kv_heads=2,
                   dim=128, page=4, window=1024, sinks=4, dtype="bf16", fmt="e4m3"),
        # A whole prompt through a windowed layer.
        _attention("window_prompt", batch=1, q_lo=8192, q_hi=8192, ctx_lo=0, ctx_hi=0, heads=32, kv_heads=8,
                   dim=128, page=16, window=1024, sinks=4, dtype="bf16", fmt="e4m3"),
        # Checking drafts in a windowed layer with narrow heads and the older cache format.
        _attention("window_drafts", batch=7, q_lo=3, q_hi=8, ctx_lo=100, ctx_hi=20000, heads=8, kv_heads=2,
                   dim=64, page=16, window=500, sinks=1, dtype="f16", fmt="e5m2"),
        # Taking the prefixes of four requests out of the cache.
        dict(name="read_prefixes", op="read", batch=4, len_lo=1001, len_hi=60000, kv_heads=8, dim=128, page=16,
             dtype="f16", fmt="e4m3"),
        # A few short ones, one wide KV head, big pages.
        dict(name="read_short", op="read", batch=3, len_lo=5, len_hi=130, kv_heads=1, dim=256, page=1728,
             dtype="bf16", fmt="e5m2"),
        # The scales of a long prompt's rows.
        dict(name="calibrate_prompt", op="calibrate", tokens=65536, kv_heads=8, dim=128, dtype="f16", fmt="e4m3"),
        # The scales of one decode step's rows.
        dict(name="calibrate_step", op="calibrate", tokens=64, kv_heads=8, dim=128, dtype="bf16", fmt="e4m3"),
    ]


def _log_between(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("chunk", "chunk", "window", "window", "read", "calibrate"))
    fmt = rng.choice(("e4m3", "e4m3", "e5m2"))
    page = rng.choice((1, 4, 16, 16, 64, 1728, 3296))
    dtype = rng.choice(("f16", "bf16"))
    kv_heads, group, dim = rng.choice(((1, 6, 256), (1, 8, 128), (2, 1, 128), (2, 12, 128), (8, 4, 128), (8, 5, 128),
                                       (2, 4, 64), (8, 1, 64), (2, 2, 256)))
    if op == "calibrate":
        return dict(op=op, tokens=_log_between(rng, 1, 65536), kv_heads=kv_heads, dim=dim, dtype=dtype, fmt=fmt)
    if op == "read":
        hi = _log_between(rng, 1, 40000)
        return dict(op=op, batch=_log_between(rng, 1, 5), len_lo=rng.randint(max(0, hi // 50), hi), len_hi=hi,
                    kv_heads=kv_heads, dim=dim, page=page, dtype=rng.choice(("f16", "bf16", "f32")), fmt=fmt)
    while True:
        batch = _log_between(rng, 1, 48)
        q_hi = 1 if rng.random() < 0.4 else _log_between(rng, 1, 6000)
        q_lo = q_hi if batch == 1 else rng.randint(1, q_hi)
        ctx_hi = _log_between(rng, 1, 60000) - 1
        ctx_lo = ctx_hi if batch == 1 else rng.randint(ctx_hi // 20, ctx_hi)
        window = _log_between(rng, 16, 5000) if op == "window" else 0
        case = dict(op="attention", batch=batch, q_lo=q_lo, q_hi=q_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                    heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page, window=window,
                    sinks=rng.randint(0, 8) if window else 0, dtype=dtype, fmt=fmt)
        spread = _spread_of(case)
        # no dearer than the listed ones: scores, gathered rows and the pool
        if (batch * kv_heads * group * q_hi * spread <= 1.0e9 and batch * spread * kv_heads * dim <= 2.5e8
                and batch * ctx_hi * kv_heads * dim <= 5e8 and 4 * work(case)["flops"] <= 1e12):
            return case


def _lengths(lo, hi, n):
    """n lengths between lo and hi, spread over their logarithm, out of order."""
    if n == 1:
        return [hi]
    got = [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]
    step = next(s for s in (5, 7, 3, 1) if n % s or s == 1)
    return [got[(i * step) % n] for i in range(n)]


def _spread_of(case):
    """The most positions that one request's new tokens see together."""
    longest = case["ctx_hi"] + case["q_hi"]
    return min(longest, case["sinks"] + case["window"] + case["q_hi"] - 1) if case["window"] else longest


def _requests(case):
    """(new tokens, length with them) of each request."""
    n = case["batch"]
    new = _lengths(case["q_lo"], case["q_hi"], n)
    ctx = list(reversed(_lengths(case["ctx_lo"], case["ctx_hi"], n)))
    return [(a, a + b) for a, b in zip(new, ctx)]


def work(case):
    if case["op"] == "calibrate":
        return {"bytes": 2 * 2 * case["tokens"] * case["kv_heads"] * case["dim"] + 8, "flops": 0}
    if case["op"] == "read":
        size = {"f16": 2, "bf16": 2, "f32": 4}[case["dtype"]]
        n = sum(_lengths(case["len_lo"], case["len_hi"], case["batch"]))
        return {"bytes": 2 * (1 + size) * n * case["kv_heads"] * case["dim"], "flops": 0}
    W, S = case["window"], case["sinks"]
    pairs = tokens = rows = 0
    for new, kv in _requests(case):
        first = kv - new
        rows += new
        if W == 0:
            pairs += new * first + new * (new + 1) // 2
            tokens += kv
            continue
        for p in (first + i for i in range(new)):
            low = max(0, p - W + 1)
            pairs += p + 1 - low + min(S, low)
        low = max(0, first - W + 1)
        tokens += kv - low + min(S, low)
    return {"bytes": 2 * 2 * rows * case["heads"] * case["dim"] + 2 * tokens * case["kv_heads"] * case["dim"],
            "flops": 4 * pairs * case["heads"] * case["dim"]}


def _bytes(shape, fmt, scale, gen):
    """Cache bytes of normally distributed values over `scale`."""
    kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    flat = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for piece in flat.view(-1).split(1 << 28):
        x = torch.randn(piece.numel(), device="cuda", generator=gen).div_(scale).clamp_(-_FMAX[fmt], _FMAX[fmt])
        piece.copy_(x.to(kind).view(torch.uint8))
    return flat


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lengths):
    total = [0]
    for n in lengths:
        total.append(total[-1] + n)
    return total


def _pool(case, longest, gen):
    """K and V pages, and a table that hands a request its pages in any order."""
    page, n = case["page"], len(longest)
    columns = max(1, -(-max(longest) // page))
    blocks = n * columns
    # rows as they lie side by side in memory: a token's KV heads, then the next token
    scale = torch.tensor(6.0 / _FMAX[case["fmt"]], dtype=torch.float32).item()
    state = {c: _bytes((blocks + 1, page, case["kv_heads"], case["dim"]), case["fmt"], scale, gen) for c in ("k", "v")}
    order = torch.randperm(blocks, device="cuda", generator=gen).to(torch.int32) + 1
    state["table"] = order.view(n, columns).contiguous()
    state["k_scale"] = state["v_scale"] = scale
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = _TYPES[case["dtype"]]
    state = {"case": case, "op": case["op"]}
    if case["op"] == "calibrate":
        shape = (case["tokens"], case["kv_heads"], case["dim"])
        for c in ("k", "v"):
            x = torch.randn(shape, device="cuda", generator=gen)
            x[..., 0] *= 8  # a column of outliers
            state[c] = x.to(dtype)
            # what earlier batches left: lower than this batch needs for K, higher for V
            state[c + "_scale"] = torch.full((1,), {"k": 1e-4, "v": 1.0}[c] * (448.0 / _FMAX[case["fmt"]]) *
                                             (1.0 + seed % 97 / 128), dtype=torch.float32, device="cuda")
    elif case["op"] == "read":
        lengths = _lengths(case["len_lo"], case["len_hi"], case["batch"])
        first = [37 * (i + 1) % 101 for i in range(case["batch"])]
        state.update(_pool(case, [a + b for a, b in zip(first, lengths)], gen))
        state["cu"], state["first"] = _ints(_starts(lengths)), _ints(first)
        shape = (sum(lengths), case["kv_heads"], case["dim"])
        state["out_k"], state["out_v"] = (torch.zeros(shape, dtype=dtype, device="cuda") for _ in "kv")
    else:
        requests = _requests(case)
        state.update(_pool(case, [kv for _, kv in requests], gen))
        rows = sum(new for new, _ in requests)
        state["cu"], state["kv_len"] = _ints(_starts([new for new, _ in requests])), _ints([kv for _, kv in requests])
        shape = (rows, case["heads"], case["dim"])
        state["q"] = (torch.randn(shape, device="cuda", generator=gen) * 1.5).to(dtype)
        state["out"] = torch.zeros(shape, dtype=dtype, device="cuda")
        state["softmax_scale"] = case["dim"] ** -0.5
    state["handle"] = _handle(state) if own else None
    return state


def _handle(state):
    """The plan, workspace and argument block that a program keeps for its buffers."""
    import fp8_e4m3_paged_gb300 as lib

    case = state["case"]
    fmt = {"e4m3": lib.KV_E4M3, "e5m2": lib.KV_E5M2}[case["fmt"]]
    if state["op"] == "calibrate":
        return lib.make_calibrate_args(k=state["k"], v=state["v"], k_scale=state["k_scale"],
                                       v_scale=state["v_scale"], kv_format=fmt)
    if state["op"] == "read":
        return lib.make_cache_read_args(
            k_cache=state["k"], v_cache=state["v"], block_table=state["table"], cu_len=state["cu"],
            start=state["first"], k_out=state["out_k"], v_out=state["out_v"], k_scale=state["k_scale"],
            v_scale=state["v_scale"], kv_format=fmt)
    plan = lib.fp8kv_attn_chunk_plan(lib.make_chunk_desc(
        batch=case["batch"], total_q=state["q"].shape[0], max_q=case["q_hi"], num_q_heads=case["heads"],
        num_kv_heads=case["kv_heads"], head_dim=case["dim"], page_size=case["page"],
        max_kv_len=max(kv for _, kv in _requests(case)), max_blocks=state["table"].shape[1],
        num_kv_blocks=state["k"].shape[0], window=case["window"], sinks=case["sinks"],
        dtype=lib.DTYPE_F16 if case["dtype"] == "f16" else lib.DTYPE_BF16, kv_format=fmt))
    workspace = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    args = lib.make_chunk_args(
        q=state["q"], k_cache=state["k"], v_cache=state["v"], out=state["out"], workspace=workspace,
        softmax_scale=state["softmax_scale"], k_scale=state["k_scale"], v_scale=state["v_scale"],
        block_table=state["table"], cu_q=state["cu"], kv_len=state["kv_len"])
    return lib.ChunkCall(plan, args), workspace


def run(state):
    if own:
        return _run_own(state)
    return {"attention": _plain_attention, "read": _plain_read, "calibrate": _plain_calibrate}[state["op"]](state)


def _run_own(state):
    import fp8_e4m3_paged_gb300 as lib

    stream = torch.cuda.current_stream().cuda_stream
    if state["op"] == "calibrate":
        lib.fp8kv_attn_cache_calibrate(state["handle"], stream)
        return state["k_scale"], state["v_scale"]
    if state["op"] == "read":
        lib.fp8kv_attn_cache_read(state["handle"], stream)
        return state["out_k"], state["out_v"]
    state["handle"][0].run(stream)
    return state["out"]


# ------------------------------------------------------------------ plain forms


def _rows(state, cache, request, position):
    """FP32 values of cache rows at the positions of the requests (any shape), [..., kv head, d]."""
    page = state["case"]["page"]
    kind = torch.float8_e4m3fn if state["case"]["fmt"] == "e4m3" else torch.float8_e5m2
    block = state["table"][request, position // page].long()
    return state[cache][block, position % page].view(kind).float()


def _owner(cu, n):
    """Request and place in it of each of the n rows."""
    row = torch.arange(n, device="cuda")
    request = torch.searchsorted(cu.long(), row, right=True) - 1
    return request, row - cu.long()[request]


def _plain_attention(state):
    case, W, S = state["case"], state["case"]["window"], state["case"]["sinks"]
    B, H, Hkv, D, nq = case["batch"], case["heads"], case["kv_heads"], case["dim"], case["q_hi"]
    cu, kv = state["cu"].long(), state["kv_len"].long()
    new = cu[1:] - cu[:-1]
    # positions that the requests' new tokens can see: first ones that stay, then the rest
    j = torch.arange(_spread_of(case), device="cuda")
    if W:
        low = (kv - new - W + 1).clamp(min=0)
        position = torch.where(j < S, j, (low.clamp(min=S)[:, None] + j - S))
    else:
        position = j.expand(B, -1)
    inside = position < kv[:, None]
    index = torch.where(inside, position, 0)
    request = torch.arange(B, device="cuda")[:, None]
    k = _rows(state, "k", request, index).permute(0, 2, 1, 3)  # [B, kv head, J, D]
    v = _rows(state, "v", request, index).permute(0, 2, 1, 3)
    i = torch.arange(nq, device="cuda")
    place = (cu[:-1, None] + i).clamp(max=state["q"].shape[0] - 1)
    q = state["q"][place].float().view(B, nq, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)
    at = (kv - new)[:, None] + i  # position of each new token, [B, nq]
    sees = inside[:, None, :] & (position[:, None, :] <= at[:, :, None])
    if W:
        sees &= (at[:, :, None] - position[:, None, :] < W) | (position[:, None, :] < S)
    z = torch.matmul(q.reshape(B, Hkv, -1, D), k.transpose(2, 3)).view(B, Hkv, H // Hkv, nq, -1)
    z = z.mul_(state["softmax_scale"] * state["k_scale"]).masked_fill_(~sees[:, None, None], float("-inf"))
    z = z.sub_(z.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, Hkv, -1, z.shape[-1]), v).view(B, Hkv, H // Hkv, nq, D)
    o = (o * state["v_scale"] / total).permute(0, 3, 1, 2, 4).reshape(B, nq, H, D)
    request, place = _owner(state["cu"], state["q"].shape[0])
    return o[request, place].to(state["q"].dtype)


def _plain_read(state):
    request, place = _owner(state["cu"], state["out_k"].shape[0])
    position = state["first"].long()[request] + place
    return tuple((_rows(state, c, request, position) * state[c + "_scale"]).to(state["out_" + c].dtype) for c in "kv")


def _plain_calibrate(state):
    fmax = _FMAX[state["case"]["fmt"]]
    return tuple(torch.maximum(state[c + "_scale"], state[c].float().abs().amax() / fmax) for c in "kv")


# ------------------------------------------------------------------ from the definition, in 64 bits


def _values(fmt):
    """The 256 values of a cache format, from its definition."""
    bits, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    got = []
    for code in range(256):
        e, m = (code & 127) >> bits, code & ((1 << bits) - 1)
        x = m * 2.0 ** (1 - bias - bits) if e == 0 else (1 + m / (1 << bits)) * 2.0 ** (e - bias)
        got.append(-x if code > 127 else x)
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def _line(state, cache, request, first, last, head, values):
    """Rows first..last-1 of one request and head, in 64 bits."""
    t = torch.arange(first, last, device="cuda")
    flat = state[cache].view(-1, *state[cache].shape[2:])
    P = state["case"]["page"]
    return values[flat[state["table"][request].long()[t // P] * P + t % P, head].long()]


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "calibrate":
        return tuple(torch.stack([state[c].double().abs().flatten().max() / _FMAX[case["fmt"]],
                                  state[c + "_scale"].double()[0]]).max().view(1) for c in "kv")
    values = _values(case["fmt"])
    if case["op"] == "read":
        cu, first = state["cu"].tolist(), state["first"].tolist()
        return tuple(torch.cat([torch.stack([
            _line(state, c, b, first[b], first[b] + cu[b + 1] - cu[b], h, values) * state[c + "_scale"]
            for h in range(case["kv_heads"])], 1) for b in range(case["batch"])]) for c in "kv")
    if work(case)["flops"] > 2.5e12:
        return None
    W, S, G = case["window"], case["sinks"], case["heads"] // case["kv_heads"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (new, kv) in enumerate(_requests(case)):
        for h in range(case["kv_heads"]):
            for a in range(0, new, 512):  # a few new tokens at a time
                n = min(512, new - a)
                start = kv - new + a
                low = max(0, start - W + 1) if W else 0
                keep = min(S, low)
                K, V = (torch.cat([_line(state, c, b, 0, keep, h, values),
                                   _line(state, c, b, low, start + n, h, values)]) for c in "kv")
                t = torch.cat([torch.arange(keep, device="cuda"), torch.arange(low, start + n, device="cuda")])
                at = torch.arange(start, start + n, device="cuda")[:, None]
                hidden = t > at
                if W:
                    hidden |= (t <= at - W) & (t >= S)
                heads = slice(h * G, (h + 1) * G)
                q = state["q"][row + a:row + a + n, heads].double().transpose(0, 1)
                z = (q @ K.T) * (state["softmax_scale"] * state["k_scale"])
                w = torch.softmax(z.masked_fill(hidden, -float("inf")), -1)
                out[row + a:row + a + n, heads] = (w @ V).transpose(0, 1) * state["v_scale"]
        row += new
    return out
