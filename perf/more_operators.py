"""What happens around the cache between two steps, as cases to measure.

Four operators: attention of trees of drafted tokens over the paged FP8 cache
("tree"), the attention weight that each cached position has gathered
("score"), the choice of the positions that stay in the cache ("select"), and
the move of rows within it ("move": the accepted path of a tree to the front
of its place, the positions that stay to the front of theirs).  With ``own``
false, ``run`` computes them with elementary torch operations in 32 bits; with
``own`` true it makes the calls of this package.
"""

import functools

import torch

own = False

#: largest finite value of each cache format
_FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
_KINDS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _tree(name, **kw):
    return dict(name=name, op="tree", **kw)


def _score(name, **kw):
    return dict(name=name, op="score", **kw)


def listed():
    return [
        # One request checks a tree of 26 drafts a little behind its prompt (latency).
        _tree("tree_one", batch=1, q_lo=26, q_hi=26, ctx_lo=611, ctx_hi=611, heads=6, kv_heads=1, dim=256, page=16,
              window=0, sinks=0, dtype="f16", fmt="e4m3"),
        # A batch whose requests check trees of 9 to 64 drafts.
        _tree("tree_batch", batch=16, q_lo=9, q_hi=64, ctx_lo=100, ctx_hi=8000, heads=32, kv_heads=8, dim=128, page=16,
              window=0, sinks=0, dtype="bf16", fmt="e4m3"),
        # One long context and a tree of 64.
        _tree("tree_long", batch=1, q_lo=64, q_hi=64, ctx_lo=131008, ctx_hi=131008, heads=16, kv_heads=2, dim=128,
              page=16, window=0, sinks=0, dtype="f16", fmt="e4m3"),
        # The weights of one decode step of a batch, added to what earlier steps left.
        _score("score_step", batch=64, q_lo=1, q_hi=1, ctx_lo=512, ctx_hi=16000, heads=32, kv_heads=8, dim=128,
               page=16, fresh=False, dtype="f16", fmt="e4m3"),
        # The same of one request (latency).
        _score("score_one", batch=1, q_lo=1, q_hi=1, ctx_lo=4001, ctx_hi=4001, heads=16, kv_heads=2, dim=128, page=4,
               fresh=False, dtype="bf16", fmt="e4m3"),
        # What the last 32 tokens of long prompts look at: the choice of what to keep of a prompt.
        _score("score_last_rows", batch=4, q_lo=32, q_hi=32, ctx_lo=8000, ctx_hi=60000, heads=32, kv_heads=8, dim=128,
               page=16, fresh=True, dtype="bf16", fmt="e4m3"),
        # What every token of a prompt looks at.
        _score("score_prompt", batch=1, q_lo=8192, q_hi=8192, ctx_lo=0, ctx_hi=0, heads=32, kv_heads=8, dim=128,
               page=16, fresh=True, dtype="f16", fmt="e4m3"),
        # A batch's choice, a list for each KV head.
        dict(name="select_heads", op="select", batch=16, len_lo=1000, len_hi=40000, kv_heads=8, joint=False,
             budget=4096, sinks=4, recent=256),
        # One long context's choice, one list for all KV heads.
        dict(name="select_joint", op="select", batch=1, len_lo=131072, len_hi=131072, kv_heads=8, joint=True,
             budget=16384, sinks=4, recent=1024),
        # The kept rows of a batch to pages of their own, a list for each KV head, the weights with them.
        dict(name="move_kept", op="move", batch=8, how="kept", len_lo=8000, len_hi=30000, count=4096, kv_heads=8,
             dim=128, page=16, fmt="e4m3"),
        # First tokens and the last ones to the front of the pages that they are in.
        dict(name="move_recent", op="move", batch=16, how="recent", len_lo=4200, len_hi=20000, count=2052, kv_heads=8,
             dim=128, page=16, fmt="e4m3"),
        # The accepted path of each request's tree.
        dict(name="move_accepted", op="move", batch=64, how="accepted", len_lo=500, len_hi=4000, count=5, kv_heads=8,
             dim=128, page=16, fmt="e4m3"),
    ]


def _log_between(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("tree", "tree", "score", "score", "select", "move"))
    fmt = rng.choice(("e4m3", "e4m3", "e5m2"))
    page = rng.choice((1, 4, 16, 16, 64, 1728, 3296))
    dtype = rng.choice(("f16", "bf16"))
    kv_heads, group, dim = rng.choice(((1, 6, 256), (1, 8, 128), (2, 1, 128), (2, 12, 128), (8, 4, 128), (8, 5, 128),
                                       (2, 4, 64), (8, 1, 64), (2, 2, 256)))
    if op == "select":
        while True:
            hi = _log_between(rng, 1, 131072)
            case = dict(op=op, batch=_log_between(rng, 1, 32), len_lo=rng.randint(hi // 20, hi), len_hi=hi,
                        kv_heads=kv_heads, joint=rng.random() < 0.4, budget=_log_between(rng, 1, 20000), sinks=0,
                        recent=0)
            case["sinks"] = rng.randint(0, min(8, case["budget"]))
            case["recent"] = rng.randint(0, (case["budget"] - case["sinks"]) // 2)
            if case["batch"] == 1:
                case["len_lo"] = hi
            if case["batch"] * hi * kv_heads <= 5.2e6:
                return case
    if op == "move":
        while True:
            how = rng.choice(("kept", "recent", "accepted"))
            count = _log_between(rng, 1, 16 if how == "accepted" else 8000)
            hi = _log_between(rng, 1, 15) * count + 200
            case = dict(op=op, batch=_log_between(rng, 1, 48), how=how, len_lo=0, len_hi=hi, count=count,
                        kv_heads=kv_heads, dim=dim, page=page, fmt=fmt)
            case["len_lo"] = hi if case["batch"] == 1 else rng.randint(min(2 * count + 150, hi), hi)
            most = case["batch"] * (_columns(case) + _fresh_columns(case)) * page * kv_heads * dim
            behind = how != "recent" or case["len_lo"] >= 2 * count  # the last ones lie behind their new places
            if behind and work(case)["bytes"] <= 1.3e8 and most <= 3.4e8:
                return case
    while True:
        batch = _log_between(rng, 1, 48)
        most_q = 160 if op == "tree" else 1 if rng.random() < 0.4 else _log_between(rng, 1, 6000)
        q_hi = _log_between(rng, 1, most_q)
        q_lo = q_hi if batch == 1 else rng.randint(1, q_hi)
        ctx_hi = _log_between(rng, 1, 60000) - 1
        ctx_lo = ctx_hi if batch == 1 else rng.randint(ctx_hi // 20, ctx_hi)
        case = dict(op=op, batch=batch, q_lo=q_lo, q_hi=q_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, heads=kv_heads * group,
                    kv_heads=kv_heads, dim=dim, page=page, dtype=dtype, fmt=fmt)
        if op == "tree":
            case["window"] = _log_between(rng, 200, 5000) if rng.random() < 0.35 else 0
            case["sinks"] = rng.randint(0, 8) if case["window"] else 0
        else:
            case["fresh"] = rng.random() < 0.5
        spread = _spread_of(case)
        # no dearer than the listed ones: scores, gathered rows and the pool
        if (batch * kv_heads * group * q_hi * spread <= 1.0e9 and batch * spread * kv_heads * dim <= 2.5e8
                and batch * ctx_hi * kv_heads * dim <= 5e8 and work(case)["flops"] <= 1.2e11):
            return case


def _lengths(lo, hi, n):
    """n lengths between lo and hi, spread over their logarithm, out of order."""
    if n == 1:
        return [hi]
    got = [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]
    step = next(s for s in (5, 7, 3, 1) if n % s or s == 1)
    return [got[(i * step) % n] for i in range(n)]


def _requests(case):
    """(new tokens, length with them) of each request."""
    n = case["batch"]
    new = _lengths(case["q_lo"], case["q_hi"], n)
    ctx = list(reversed(_lengths(case["ctx_lo"], case["ctx_hi"], n)))
    return [(a, a + b) for a, b in zip(new, ctx)]


def _spread_of(case):
    """The most positions that one request's new tokens see together."""
    longest, window = case["ctx_hi"] + case["q_hi"], case.get("window", 0)
    return min(longest, case["sinks"] + window - 1 + case["q_hi"]) if window else longest


def _columns(case):
    return -(-case["len_hi"] // case["page"])


def _fresh_columns(case):
    """Pages of a request's own that its kept rows go to (0: they stay in the pages that they are in)."""
    return -(-case["count"] // case["page"]) if case["how"] == "kept" else 0


def work(case):
    if case["op"] == "select":
        lengths = _lengths(case["len_lo"], case["len_hi"], case["batch"])
        lists = 1 if case["joint"] else case["kv_heads"]
        return {"bytes": sum(4 * case["kv_heads"] * n + 4 * lists * min(n, case["budget"]) for n in lengths), "flops": 0}
    if case["op"] == "move":
        rows = case["batch"] * case["kv_heads"] * case["count"]
        lists = case["batch"] * case["count"] * (case["kv_heads"] if case["how"] == "kept" else 1)
        weights = 8 * rows if case["how"] == "kept" else 0
        return {"bytes": 2 * 2 * rows * case["dim"] + 4 * lists + weights, "flops": 0}
    W, S, tree = case.get("window", 0), case.get("sinks", 0), case["op"] == "tree"
    pairs = tokens = rows = masks = 0
    for new, kv in _requests(case):
        first = kv - new
        rows += new
        masks += 4 * new * -(-new // 32)
        low = max(0, first - W + 1) if W else 0
        seen = first - low + min(S, low)
        tokens += seen + new
        # of a tree a drafted token sees itself at least, else the new tokens up to itself
        pairs += new * seen + (new if tree else new * (new + 1) // 2)
    q = 2 * rows * case["heads"] * case["dim"]
    cached = tokens * case["kv_heads"] * case["dim"]
    if tree:
        return {"bytes": 2 * q + 2 * cached + masks, "flops": 4 * pairs * case["heads"] * case["dim"]}
    scores = 4 * tokens * case["kv_heads"] * (1 if case["fresh"] else 2)
    return {"bytes": q + cached + scores, "flops": 2 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ inputs


def _bytes(shape, fmt, scale, gen):
    """Cache bytes of normally distributed values over `scale`."""
    flat = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for piece in flat.view(-1).split(1 << 28):
        x = torch.randn(piece.numel(), device="cuda", generator=gen).div_(scale).clamp_(-_FMAX[fmt], _FMAX[fmt])
        piece.copy_(x.to(_KINDS[fmt]).view(torch.uint8))
    return flat


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lengths):
    total = [0]
    for n in lengths:
        total.append(total[-1] + n)
    return total


def _pool(case, columns, gen, which="kv"):
    """K and V pages (and some for the kept rows), and a table that hands a request its pages in any order."""
    n = case["batch"]
    # rows as they lie side by side in memory: a token's KV heads, then the next token
    scale = torch.tensor(6.0 / _FMAX[case["fmt"]], dtype=torch.float32).item()
    shape = (n * columns + 1, case["page"], case["kv_heads"], case["dim"])
    state = {c: _bytes(shape, case["fmt"], scale, gen) for c in which}
    order = torch.randperm(n * columns, device="cuda", generator=gen).to(torch.int32) + 1
    state["table"] = order.view(n, columns).contiguous()
    state["k_scale"] = state["v_scale"] = scale
    return state


def _trees(sizes, seed):
    """Masks (a word for 32 nodes) and depths of random trees: each node sees its ancestors and itself."""
    gen = torch.Generator().manual_seed(seed)
    words = -(-max(sizes) // 32)
    masks, depths = [], []
    for n in sizes:
        pick = torch.rand(n, generator=gen).tolist()
        sees, depth = [1], [0]
        for i in range(1, n):
            # a node's children follow it by a factor of two to eight: trees that widen
            low, high = (i - 1) // 8, (i - 1) // 2
            parent = low + int(pick[i] * (high - low + 1))
            sees.append(sees[parent] | 1 << i)
            depth.append(depth[parent] + 1)
        masks += [[(s >> 32 * w) & 0xFFFFFFFF for w in range(words)] for s in sees]
        depths += depth
    masks = torch.tensor(masks, dtype=torch.int64, device="cuda")
    return torch.where(masks >= 1 << 31, masks - (1 << 32), masks).to(torch.int32), _ints(depths)


def _gathered(shape, gen):
    """Weights that positions have gathered: a few large ones, most of them small."""
    return torch.rand(shape, device="cuda", generator=gen).pow_(6).mul_(20.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"case": case, "op": case["op"]}
    if case["op"] == "select":
        lengths = _lengths(case["len_lo"], case["len_hi"], case["batch"])
        lists = 1 if case["joint"] else case["kv_heads"]
        state["kv_len"] = _ints(lengths)
        state["score"] = _gathered((case["batch"], case["kv_heads"], case["len_hi"]), gen)
        state["keep"] = torch.zeros(case["batch"], lists, case["budget"], dtype=torch.int32, device="cuda")
        state["n_keep"] = torch.zeros(case["batch"], dtype=torch.int32, device="cuda")
    elif case["op"] == "move":
        state.update(_move_inputs(case, gen))
    else:
        _attention_inputs(state, case, seed, gen)
    state["handle"] = _handle(state) if own else None
    return state


def _attention_inputs(state, case, seed, gen):
    requests = _requests(case)
    columns = max(1, -(-max(kv for _, kv in requests) // case["page"]))
    state.update(_pool(case, columns, gen, "kv" if case["op"] == "tree" else "k"))
    rows = sum(new for new, _ in requests)
    state["cu"], state["kv_len"] = _ints(_starts([new for new, _ in requests])), _ints([kv for _, kv in requests])
    shape = (rows, case["heads"], case["dim"])
    state["q"] = (torch.randn(shape, device="cuda", generator=gen) * 1.5).to(_TYPES[case["dtype"]])
    state["softmax_scale"] = case["dim"] ** -0.5
    if case["op"] == "tree":
        state["out"] = torch.zeros(shape, dtype=_TYPES[case["dtype"]], device="cuda")
        state["mask"], state["depth"] = _trees([new for new, _ in requests], seed)
        return
    shape = (case["batch"], case["kv_heads"], max(kv for _, kv in requests))
    state["before"] = None if case["fresh"] else _gathered(shape, gen)
    state["decay"] = 0.96875
    state["score"] = torch.zeros(shape, device="cuda")


def _move_inputs(case, gen):
    n, count = case["batch"], case["count"]
    lengths = _lengths(case["len_lo"], case["len_hi"], n)
    columns, fresh = _columns(case), _fresh_columns(case)
    got = _pool(case, columns + fresh, gen)
    got["target"] = got["table"][:, columns:].contiguous() if fresh else None
    got["table"] = got["table"][:, :columns].contiguous()
    lists = case["kv_heads"] if case["how"] == "kept" else 1
    kv = _ints(lengths)[:, None, None]
    got["first"], got["count"] = None, _ints([min(count, x) for x in lengths])
    if case["how"] == "recent":
        # a few first tokens, then the last ones, which all lie behind the place that they go to
        sinks = min(4, count)
        i = torch.arange(count, device="cuda")
        src = torch.where(i < sinks, i, kv - count + i)
    elif case["how"] == "accepted":
        # root, then nodes of a path: all behind the place that the path goes to
        step = 1 + torch.rand((n, lists, count), device="cuda", generator=gen).mul_(4).int()
        src = count - 1 + step.cumsum(-1)
        src[..., 0] = 0
        got["first"] = _ints([max(0, x - count - 5 * count) for x in lengths])
        got["count"] = _ints([min(count, 1 + 3 * b % 7) for b in range(n)])
    else:
        # the positions with the largest of random weights, in order
        weight = torch.rand((n, lists, case["len_hi"]), device="cuda", generator=gen)
        weight = torch.where(torch.arange(case["len_hi"], device="cuda") < kv, weight, -1.0)
        src = weight.topk(count, -1).indices.sort(-1).values
        got["score"] = _gathered((n, case["kv_heads"], case["len_hi"]), gen)
        got["score_out"] = torch.zeros_like(got["score"])
    got["src"] = src.to(torch.int32).contiguous()
    return got


def _handle(state):
    """The plan, workspace and argument block that a program keeps for its buffers."""
    import fp8_e4m3_paged_gb300 as lib

    case = state["case"]
    if state["op"] == "select":
        return lib.make_cache_select_args(score=state["score"], kv_len=state["kv_len"], budget=case["budget"],
                                          sinks=case["sinks"], recent=case["recent"], keep=state["keep"],
                                          n_keep=state["n_keep"])
    if state["op"] == "move":
        return lib.make_cache_move_args(
            k_cache=state["k"], v_cache=state["v"], block_table=state["table"], src=state["src"],
            count=state["count"], first=state["first"], dst_table=state["target"], score=state.get("score"),
            score_out=state.get("score_out"))
    desc = lib.make_chunk_desc(
        batch=case["batch"], total_q=state["q"].shape[0], max_q=case["q_hi"], num_q_heads=case["heads"],
        num_kv_heads=case["kv_heads"], head_dim=case["dim"], page_size=case["page"],
        max_kv_len=max(kv for _, kv in _requests(case)), max_blocks=state["table"].shape[1],
        num_kv_blocks=state["k"].shape[0], window=case.get("window", 0), sinks=case.get("sinks", 0),
        dtype=lib.DTYPE_F16 if case["dtype"] == "f16" else lib.DTYPE_BF16,
        kv_format={"e4m3": lib.KV_E4M3, "e5m2": lib.KV_E5M2}[case["fmt"]])
    same = dict(q=state["q"], k_cache=state["k"], softmax_scale=state["softmax_scale"], k_scale=state["k_scale"],
                block_table=state["table"], cu_q=state["cu"], kv_len=state["kv_len"])
    if state["op"] == "tree":
        plan = lib.fp8kv_attn_tree_plan(desc)
        workspace = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        args = lib.make_tree_args(v_cache=state["v"], v_scale=state["v_scale"], out=state["out"], workspace=workspace,
                                  mask=state["mask"], depth=state["depth"], **same)
        return lib.TreeCall(plan, args), workspace
    plan = lib.fp8kv_attn_cache_score_plan(desc)
    workspace = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    args = lib.make_cache_score_args(score_in=state["before"], score=state["score"], decay=state["decay"],
                                     workspace=workspace, **same)
    return lib.CacheScoreCall(plan, args), workspace


def run(state):
    if own:
        return _run_own(state)
    return {"tree": _plain_tree, "score": _plain_score, "select": _plain_select, "move": _plain_move}[state["op"]](state)


def _moved(state):
    """What a move leaves: both caches as the values that they hold, and the weights."""
    kind = _KINDS[state["case"]["fmt"]]
    out = [state["k"].view(kind), state["v"].view(kind)]
    return out + [state["score_out"]] if "score_out" in state else out


def _run_own(state):
    import fp8_e4m3_paged_gb300 as lib

    stream = torch.cuda.current_stream().cuda_stream
    if state["op"] == "select":
        lib.fp8kv_attn_cache_select(state["handle"], stream)
        return state["keep"], state["n_keep"]
    if state["op"] == "move":
        lib.fp8kv_attn_cache_move(state["handle"], stream)
        return _moved(state)
    state["handle"][0].run(stream)
    return state["out"] if state["op"] == "tree" else state["score"]


# ------------------------------------------------------------------ plain forms


def _rows(state, cache, request, position):
    """FP32 values of cache rows at the positions of the requests (any shape), [..., kv head, d]."""
    page = state["case"]["page"]
    block = state["table"][request, position // page].long()
    return state[cache][block, position % page].view(_KINDS[state["case"]["fmt"]]).float()


def _owner(cu, n):
    """Request and place in it of each of the n rows."""
    row = torch.arange(n, device="cuda")
    request = torch.searchsorted(cu.long(), row, right=True) - 1
    return request, row - cu.long()[request]


def _plain_logits(state, position, sees):
    """Logits of all new tokens over the positions [B, J], -inf where not seen: [B, kv head, group, new token, J]."""
    case = state["case"]
    B, H, Hkv, D, nq = case["batch"], case["heads"], case["kv_heads"], case["dim"], case["q_hi"]
    request = torch.arange(B, device="cuda")[:, None]
    k = _rows(state, "k", request, position).permute(0, 2, 1, 3)  # [B, kv head, J, D]
    place = (state["cu"].long()[:-1, None] + torch.arange(nq, device="cuda")).clamp(max=state["q"].shape[0] - 1)
    q = state["q"][place].float().view(B, nq, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)
    z = torch.matmul(q.reshape(B, Hkv, -1, D), k.transpose(2, 3)).view(B, Hkv, H // Hkv, nq, -1)
    z = z.mul_(state["softmax_scale"] * state["k_scale"])
    return z.masked_fill_(~sees[:, None, None], float("-inf"))


def _plain_tree(state):
    case, W, S = state["case"], state["case"]["window"], state["case"]["sinks"]
    B, H, Hkv, D, nq = case["batch"], case["heads"], case["kv_heads"], case["dim"], case["q_hi"]
    cu, kv = state["cu"].long(), state["kv_len"].long()
    base = kv - (cu[1:] - cu[:-1])
    # positions that the requests' new tokens can see: first ones that stay, then the rest
    j = torch.arange(_spread_of(case), device="cuda")
    if W:
        low = (base - W + 1).clamp(min=0)
        position = torch.where(j < S, j, (low.clamp(min=S)[:, None] + j - S))
    else:
        position = j.expand(B, -1)
    inside = position < kv[:, None]
    position = torch.where(inside, position, 0)
    place = (cu[:-1, None] + torch.arange(nq, device="cuda")).clamp(max=state["q"].shape[0] - 1)
    words = state["mask"][place]  # [B, nq, words]
    node = (position - base[:, None]).clamp(min=0, max=32 * words.shape[2] - 1)
    drawn = node[:, None, :].expand(-1, nq, -1)
    bit = torch.gather(words, 2, drawn >> 5) >> (drawn & 31) & 1
    context = (position < base[:, None])[:, None, :].expand(-1, nq, -1)
    if W:
        at = base[:, None] + state["depth"].long()[place]
        near = (at[:, :, None] - position[:, None, :] < W) | (position[:, None, :] < S)
        sees = torch.where(context, near, bit.bool())
    else:
        sees = context | bit.bool()
    z = _plain_logits(state, position, sees & inside[:, None, :])
    z = z.sub_(z.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = z.sum(-1, keepdim=True)
    v = _rows(state, "v", torch.arange(B, device="cuda")[:, None], position).permute(0, 2, 1, 3)
    o = torch.matmul(z.view(B, Hkv, -1, z.shape[-1]), v).view(B, Hkv, H // Hkv, nq, D)
    o = (o * state["v_scale"] / total).permute(0, 3, 1, 2, 4).reshape(B, nq, H, D)
    request, place = _owner(state["cu"], state["q"].shape[0])
    return o[request, place].to(state["q"].dtype)


def _plain_score(state):
    case, nq = state["case"], state["case"]["q_hi"]
    cu, kv = state["cu"].long(), state["kv_len"].long()
    new = cu[1:] - cu[:-1]
    t, i = torch.arange(state["score"].shape[2], device="cuda"), torch.arange(nq, device="cuda")
    inside = t < kv[:, None]
    at = torch.where(i < new[:, None], (kv - new)[:, None] + i, -1)  # position of each new token, [B, nq]
    z = _plain_logits(state, torch.where(inside, t, 0), t <= at[:, :, None])
    z = z.sub_(z.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    z = z.div_(z.sum(-1, keepdim=True).clamp(min=1e-30))
    got = z.sum((2, 3))
    if state["before"] is not None:
        got = got + torch.where(t < (kv - new)[:, None], 1.0, 0.0)[:, None] * state["before"] * state["decay"]
    return torch.where(inside[:, None], got, state["score"])


def _plain_select(state):
    case, kv = state["case"], state["kv_len"].long()[:, None, None]
    weight = state["score"]
    if case["joint"]:
        weight = functools.reduce(torch.add, weight.unbind(1))[:, None]  # head after head
    t = torch.arange(weight.shape[2], device="cuda")
    stays = (t < case["sinks"]) | (t >= kv - case["recent"])
    weight = torch.where(stays, float("inf"), weight).masked_fill(t >= kv, -1.0)
    order = torch.sort(weight, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, t.expand_as(order).contiguous())
    kept = (rank < case["budget"]) & (t < kv)
    to = torch.where(kept, kept.long().cumsum(-1) - 1, case["budget"])
    keep = torch.cat([state["keep"], torch.zeros_like(state["keep"][..., :1])], -1)
    keep = keep.scatter(-1, to, t.to(torch.int32).expand_as(to))[..., :-1]
    return keep.contiguous(), kept[:, 0].sum(-1).to(torch.int32)


def _plain_move(state):
    case, page = state["case"], state["case"]["page"]
    src = state["src"].long().expand(-1, case["kv_heads"], -1)  # [B, kv head, row]
    b = torch.arange(case["batch"], device="cuda")[:, None, None]
    h = torch.arange(case["kv_heads"], device="cuda")[None, :, None]
    i = torch.arange(src.shape[2], device="cuda")
    first = torch.zeros_like(state["count"]) if state["first"] is None else state["first"]
    first = first.long()[:, None, None]
    live = (i < state["count"].long()[:, None, None]).expand_as(src)
    b, h, at, to = (x.expand_as(src)[live] for x in (b, h, first + src, first + i))
    target = state["table"] if state["target"] is None else state["target"]
    old, new = state["table"][b, at // page].long(), target[b, to // page].long()
    k, v = (state[c][old, at % page, h] for c in "kv")
    state["k"][new, to % page, h] = k
    state["v"][new, to % page, h] = v
    if "score_out" in state:
        state["score_out"][b, h, to] = state["score"][b, h, at]
    return _moved(state)


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


def _line(state, cache, request, positions, head, values):
    """Rows of one request and head, in 64 bits."""
    flat = state[cache].view(-1, *state[cache].shape[2:])
    P = state["case"]["page"]
    return values[flat[state["table"][request].long()[positions // P] * P + positions % P, head].long()]


def _exact_tree(state, case, values):
    W, S, G = case["window"], case["sinks"], case["heads"] // case["kv_heads"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    words, depth = state["mask"].tolist(), state["depth"].tolist()
    row = 0
    for b, (new, kv) in enumerate(_requests(case)):
        base = kv - new
        low = max(0, base - W + 1) if W else 0
        t = torch.cat([torch.arange(min(S, low), device="cuda"), torch.arange(low, kv, device="cuda")])
        nodes = torch.tensor([[words[row + i][n // 32] >> (n % 32) & 1 for n in range(new)] for i in range(new)],
                             dtype=torch.bool, device="cuda")
        at = base + torch.tensor(depth[row:row + new], device="cuda")[:, None]
        hidden = torch.zeros(new, t.numel(), dtype=torch.bool, device="cuda")
        if W:
            hidden |= (t <= at - W) & (t >= S)
        hidden[:, t.numel() - new:] = ~nodes
        for h in range(case["kv_heads"]):
            K, V = (_line(state, c, b, t, h, values) for c in "kv")
            q = state["q"][row:row + new, h * G:(h + 1) * G].double().transpose(0, 1)
            z = (q @ K.T) * (state["softmax_scale"] * state["k_scale"])
            w = torch.softmax(z.masked_fill(hidden, -float("inf")), -1)
            out[row:row + new, h * G:(h + 1) * G] = (w @ V).transpose(0, 1) * state["v_scale"]
        row += new
    return out


def _exact_score(state, case, values):
    out, G, row = state["score"].double(), case["heads"] // case["kv_heads"], 0
    for b, (new, kv) in enumerate(_requests(case)):
        t = torch.arange(kv, device="cuda")
        for h in range(case["kv_heads"]):
            K = _line(state, "k", b, t, h, values)
            total = torch.zeros(kv, dtype=torch.float64, device="cuda")
            if state["before"] is not None:
                total[:kv - new] = state["before"][b, h, :kv - new].double() * state["decay"]
            for a in range(0, new, 512):  # a few new tokens at a time
                n = min(512, new - a)
                q = state["q"][row + a:row + a + n, h * G:(h + 1) * G].double()
                z = torch.einsum("ngd,td->gnt", q, K) * (state["softmax_scale"] * state["k_scale"])
                at = kv - new + a + torch.arange(n, device="cuda")[:, None]
                total += torch.softmax(z.masked_fill(t > at, -float("inf")), -1).sum((0, 1))
            out[b, h, :kv] = total
        row += new
    return out


def _exact_move(state, case, values):
    src, count, P = state["src"].tolist(), state["count"].tolist(), case["page"]
    first = [0] * case["batch"] if state["first"] is None else state["first"].tolist()
    table = state["table"].tolist()
    target = table if state["target"] is None else state["target"].tolist()
    old = [state[c].view(-1, case["kv_heads"], case["dim"]) for c in "kv"]
    new = [x.clone() for x in old]
    score = state["score_out"].double() if "score_out" in state else None
    for b in range(case["batch"]):
        n, f = count[b], first[b]
        to = torch.tensor([target[b][(f + i) // P] * P + (f + i) % P for i in range(n)], device="cuda")
        for h in range(case["kv_heads"]):
            line = src[b][h % len(src[b])][:n]
            at = torch.tensor([table[b][(f + s) // P] * P + (f + s) % P for s in line], device="cuda")
            for x, y in zip(old, new):
                y[to, h] = x[at, h]
            if score is not None:
                score[b, h, f:f + n] = state["score"][b, h, f + torch.tensor(line, device="cuda")].double()
    out = [values[x.long()].view(state["k"].shape) for x in new]
    return out + [score] if score is not None else out


def exact(case, seed):
    if case["op"] == "select":
        return None  # whole numbers
    state = prepare(case, seed)
    values = _values(case["fmt"])
    if case["op"] == "move":
        return _exact_move(state, case, values)
    if work(case)["flops"] > 2.5e12:
        return None
    return (_exact_tree if case["op"] == "tree" else _exact_score)(state, case, values)
