"""What a serving step does around its projections before the key/value cache is read, as cases to
measure: block tables, positions and slots from the requests' lengths, the root-mean-square norm with
the residual's addition (fp16 or 8-bit output), the norm and rotation of query and key heads, and
attention over whole packed prompts.

``run`` computes them in elementary torch operations in fp32 (``own`` false) or through the
package's entry points (``own`` true), on the same inputs.
"""
import math

import torch

own = False

BLOCK = 64  # tokens of a cache block
E4M3 = torch.float8_e4m3fn
TYPES = {"f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # 16 users, one token each: what every decode step begins with
        {"name": "plan_step", "op": "plan", "seqs": 16, "prompts": 0, "prompt_max": 1, "ended": 0, "cached_max": 8192, "pad": 0},
        # a step that takes in prompts of up to 2048 tokens beside running users, while a few end
        {"name": "plan_prompts", "op": "plan", "seqs": 64, "prompts": 16, "prompt_max": 2048, "ended": 5, "cached_max": 32768, "pad": 517},
        # thousands of short conversations
        {"name": "plan_many", "op": "plan", "seqs": 4096, "prompts": 100, "prompt_max": 300, "ended": 200, "cached_max": 2048, "pad": 0},
        # one user's token between two layers: latency
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 5120, "x": "f16", "residual": "f16", "weight": True, "offset": 0.0,
         "codes": 0, "y": True},
        # a middling batch, the projection's fp32 output on an fp32 stream, 8-bit output with a scale for each 128 columns
        {"name": "norm_codes", "op": "norm", "rows": 777, "cols": 5120, "x": "f32", "residual": "f32", "weight": True, "offset": 1.0,
         "codes": 128, "y": False},
        # a batch of prompts between two layers
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "cols": 5120, "x": "f16", "residual": "f16", "weight": True, "offset": 0.0,
         "codes": 0, "y": True},
        # 16 users' new query and key heads
        {"name": "rotary_step", "op": "rotary", "rows": 16, "heads": 40, "kv_heads": 8, "dim": 128, "rot": 128, "norm": True,
         "interleaved": False, "positions": 131072, "pad": 0},
        # the same for a batch of prompts
        {"name": "rotary_prompt", "op": "rotary", "rows": 6827, "heads": 40, "kv_heads": 8, "dim": 128, "rot": 128, "norm": True,
         "interleaved": False, "positions": 131072, "pad": 0},
        # one user's short question: latency
        {"name": "prompt_short", "op": "prompt", "seqs": 1, "len_min": 61, "len_max": 61, "heads": 40, "kv_heads": 8, "dim": 128,
         "cap": 0.0, "causal": True, "pad": 0},
        # sixteen prompts of ragged lengths in one call
        {"name": "prompt_packed", "op": "prompt", "seqs": 16, "len_min": 33, "len_max": 2048, "heads": 40, "kv_heads": 8, "dim": 128,
         "cap": 0.0, "causal": True, "pad": 0},
        # smaller heads and capped scores, as ragged
        {"name": "prompt_capped", "op": "prompt", "seqs": 5, "len_min": 777, "len_max": 2500, "heads": 32, "kv_heads": 4, "dim": 64,
         "cap": 30.0, "causal": True, "pad": 0},
        # one long document
        {"name": "prompt_long", "op": "prompt", "seqs": 1, "len_min": 8192, "len_max": 8192, "heads": 40, "kv_heads": 8, "dim": 128,
         "cap": 0.0, "causal": True, "pad": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "norm", "rotary", "prompt", "prompt"])
    if op == "plan":
        seqs = _log(rng, 1, 4096)
        most = _log(rng, 1, max(1, min(4096, 32768 // seqs)))
        return {"op": op, "seqs": seqs, "prompts": rng.randrange(0, seqs + 1), "prompt_max": most, "ended": rng.randrange(0, seqs // 4 + 1),
                "cached_max": _log(rng, 1, min(32768, 8388608 // seqs)), "pad": rng.choice([0, rng.randrange(1, 300)])}
    if op == "norm":
        codes = rng.choice([0, 0, -1, 128])
        cols = _log(rng, 64, 17408)
        cols = max(128, cols // 128 * 128) if codes == 128 else max(8, cols // 8 * 8)
        return {"op": op, "rows": _log(rng, 1, min(8192, 8192 * 5120 // cols)), "cols": cols, "x": rng.choice(["f16", "f16", "f32"]),
                "residual": rng.choice(["f16", "f16", "f32", ""]), "weight": rng.random() < 0.85, "offset": rng.choice([0.0, 1.0]),
                "codes": codes, "y": codes == 0 or rng.random() < 0.5}
    if op == "rotary":
        kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        return {"op": op, "rows": _log(rng, 1, 8192), "heads": kv * rng.choice([1, 2, 4, 5]), "kv_heads": kv, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2, 16]), "norm": rng.random() < 0.6, "interleaved": rng.random() < 0.3,
                "positions": _log(rng, 1000, 131072), "pad": rng.choice([0, rng.randrange(1, 100)])}
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = min(40, kv * rng.choice([1, 2, 4, 5, 8])) // kv * kv
    most = _log(rng, 1, 8192)
    causal = rng.random() < 0.85
    most = most if causal else min(most, 5000)
    seqs = min(_log(rng, 1, 64), max(1, 32768 // most), max(1, 8192 * 8192 * 40 // (heads * most * most * (1 if causal else 2))))
    return {"op": op, "seqs": seqs, "len_min": max(1, most // rng.randrange(1, 9)), "len_max": most, "heads": heads, "kv_heads": kv,
            "dim": rng.choice([64, 128]), "cap": rng.choice([0.0, 0.0, 0.0, 30.0]), "causal": causal,
            "pad": rng.choice([0, 0, rng.randrange(1, 200)])}


def _lens(case):
    """Tokens of each prompt, spread evenly between the case's two bounds."""
    n, lo, hi = case["seqs"], case["len_min"], case["len_max"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _requests(case):
    """New and cached tokens of each sequence of a plan: prompts, running ones and ended ones (-1) mixed."""
    n, tokens, cached = case["seqs"], [], []
    for i in range(n):
        at = i * 7919 % n
        prompt, ended = at < case["prompts"], n - 1 - at < case["ended"]
        tokens.append(-1 if ended else 1 + (at * 104729 + 13) % case["prompt_max"] if prompt else 1)
        cached.append(0 if prompt and at % 3 and not ended else 1 + (i * 15485863 + 7) % case["cached_max"])
    return tokens, cached


def _blocks(tokens):
    return (tokens + BLOCK - 1) // BLOCK


def work(case):
    op = case["op"]
    if op == "plan":
        tokens, cached = _requests(case)
        rows = sum(max(t, 0) for t in tokens) + case["pad"]
        new = sum(_blocks(c + t) - _blocks(c) for t, c in zip(tokens, cached) if t > 0)
        gone = sum(_blocks(c) for t, c in zip(tokens, cached) if t < 0)
        begun = sum(1 for t, c in zip(tokens, cached) if t > 0 and c % BLOCK)
        return {"bytes": 16 * case["seqs"] + 8 * rows + 8 * (new + gone) + 4 * begun, "flops": 0}
    if op == "norm":
        size = {"f16": 2, "f32": 4, "": 0}
        each = size[case["x"]] + 2 * size[case["residual"]] + (2 if case["y"] else 0) + (1 if case["codes"] else 0)
        groups = 0 if not case["codes"] else 1 if case["codes"] < 0 else case["cols"] // case["codes"]
        return {"bytes": case["rows"] * (case["cols"] * each + 4 * groups) + (2 * case["cols"] if case["weight"] else 0),
                "flops": 5 * case["rows"] * case["cols"]}
    if op == "rotary":
        width = (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": case["rows"] * (4 * width + 4 * case["rot"] + 4), "flops": case["rows"] * width * 8}
    h, kv, d, lens = case["heads"], case["kv_heads"], case["dim"], _lens(case)
    seen = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens) * h
    return {"bytes": sum(lens) * (4 * h * d + 4 * kv * d + 4 * h), "flops": 4 * seen * d}


# --------------------------------------------------------------------------- inputs


def _cumulative(counts):
    return torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _plan_inputs(case, gen):
    tokens, cached = _requests(case)
    n, rows = case["seqs"], sum(max(t, 0) for t in tokens) + case["pad"]
    max_pages = max(_blocks(c + max(t, 0)) for t, c in zip(tokens, cached)) + 1
    held = sum(_blocks(c) for c in cached)
    new = sum(_blocks(c + t) - _blocks(c) for t, c in zip(tokens, cached) if t > 0)
    n_pages = held + new + 11
    pages = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    # a sequence's first blocks hold its cached tokens; what lies behind them is left from before
    slot = torch.arange(max_pages, device="cuda")
    have = torch.tensor([_blocks(c) for c in cached], device="cuda")
    at = _cumulative([_blocks(c) for c in cached])[:-1, None] + slot[None, :]
    real = slot[None, :] < have[:, None]
    table = torch.where(real, pages[torch.where(real, at, 0).long()], -7).to(torch.int32).contiguous()
    free = torch.full((n_pages,), -9, dtype=torch.int32, device="cuda")
    free[:n_pages - held] = pages[held:]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def empty(k):
        return torch.empty((k,), dtype=torch.int32, device="cuda")

    return {"tokens": ints(tokens), "cached": ints(cached), "table": table, "free": free, "count": ints([n_pages - held]), "n_pages": n_pages,
            "rows": rows, "max_rows": max(1, max(tokens)), "left": empty(1), "kv_len": empty(n), "q_start": empty(n + 1),
            "position": empty(rows), "slot": empty(rows), "served": empty(1)}


def _norm_inputs(case, gen):
    r, c = case["rows"], case["cols"]
    x = torch.randn((r, c), generator=gen, device="cuda")
    s = {"x": x.to(TYPES[case["x"]]), "residual": None, "sum": None, "weight": None, "y": None, "codes": None, "scales": None}
    if case["residual"]:
        # the stream between layers: a few channels far larger than the others
        loud = 1.0 + 40.0 * (torch.rand((c,), generator=gen, device="cuda") < 0.004)
        s["residual"] = (3.0 * torch.randn((r, c), generator=gen, device="cuda") * loud).to(TYPES[case["residual"]])
        s["sum"] = torch.empty_like(s["residual"])
    if case["weight"]:
        s["weight"] = ((1.0 - case["offset"]) + 0.2 * torch.randn((c,), generator=gen, device="cuda")).half()
    if case["y"]:
        s["y"] = torch.empty((r, c), dtype=torch.float16, device="cuda")
    if case["codes"]:
        s["codes"] = torch.empty((r, c), dtype=E4M3, device="cuda")
        s["scales"] = torch.empty((r, 1 if case["codes"] < 0 else c // case["codes"]), device="cuda")
    return s


def _rotary_inputs(case, gen):
    h, kv, d, n = case["heads"], case["kv_heads"], case["dim"], case["rows"] + case["pad"]
    qkv = torch.randn((n, (h + 2 * kv) * d), generator=gen, device="cuda")
    qkv *= torch.exp(0.5 * torch.randn((n, 1), generator=gen, device="cuda"))
    # positions of several users' rows, one behind the other; padding rows at the end have none
    first = torch.randint(0, case["positions"], (1 + n // 64,), generator=gen, device="cuda")
    i = torch.arange(n, device="cuda")
    position = ((first[i // 64] + i) % case["positions"]).to(torch.int32)
    position[case["rows"]:] = -1
    angle = torch.arange(case["positions"], device="cuda").double()[:, None] * 1e6 ** (
        -torch.arange(0, case["rot"], 2, device="cuda").double() / case["rot"])
    s = {"qk": qkv.half()[:, :(h + kv) * d], "position": position, "cos_sin": torch.cat([torch.cos(angle), torch.sin(angle)], 1).float(),
         "out": torch.zeros((n, (h + kv) * d), dtype=torch.float16, device="cuda"), "q_weight": None, "k_weight": None}
    if case["norm"]:
        s["q_weight"], s["k_weight"] = (1.0 + 0.2 * torch.randn((2, d), generator=gen, device="cuda")).half()
    return s


def _prompt_inputs(case, gen):
    h, kv, d, lens = case["heads"], case["kv_heads"], case["dim"], _lens(case)
    n = sum(lens) + case["pad"]
    # rows of a fused projection: queries, keys and values are column ranges of one matrix
    qkv = torch.randn((n, (h + 2 * kv) * d), generator=gen, device="cuda")
    qkv[:, :h * d] *= 2.0
    qkv[:, (h + kv) * d:] *= 0.5
    qkv = qkv.half()
    return {"q": qkv[:, :h * d], "k": qkv[:, h * d:(h + kv) * d], "v": qkv[:, (h + kv) * d:], "q_start": _cumulative(lens),
            "counts": torch.tensor(lens, dtype=torch.int32, device="cuda"), "max_rows": max(lens), "scale": 1.0 / math.sqrt(d),
            "out": torch.zeros((n, h * d), dtype=torch.float16, device="cuda"), "lse": torch.zeros((n, h), device="cuda")}


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"case": case, **{"plan": _plan_inputs, "norm": _norm_inputs, "rotary": _rotary_inputs, "prompt": _prompt_inputs}[case["op"]](case, gen)}


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import trellis_quantized_linear_gb300 as tql
        tql.build()
        tql.exl3_init(torch.cuda.current_device())
        if case["op"] == "plan":
            s["batch"] = tql.Exl3Kv8Batch(s["table"], s["kv_len"], s["q_start"], s["rows"], s["max_rows"])
    return s


# --------------------------------------------------------------------------- plain forms


def _plan_plain(s):
    tokens, cached, table = s["tokens"].long(), s["cached"].long(), s["table"]
    n, width, rows = tokens.numel(), table.shape[1], s["rows"]
    ended, grows = tokens < 0, tokens > 0
    have = (cached + BLOCK - 1) // BLOCK
    column = torch.arange(width, device="cuda")
    # ended sequences give their pages back, in their order, on top of the free ones
    gone = (column[None, :] < have[:, None]) & ended[:, None]
    rank = gone.flatten().long().cumsum(0) - 1
    spare = s["free"].numel()  # an entry that takes what is not given back
    free = torch.nn.functional.pad(s["free"], (0, 1))
    free[torch.where(gone.flatten(), s["count"] + rank, spare)] = torch.where(gone.flatten(), table.flatten(), -1)
    count = s["count"][0] + gone.sum()
    # sequences are served in their order as long as pages and rows last
    add = torch.where(grows, tokens, 0)
    need = torch.where(grows, (cached + add + BLOCK - 1) // BLOCK - have, 0)
    fits = (need.cumsum(0) <= count) & (add.cumsum(0) <= rows) & (add <= s["max_rows"]) & (cached + add <= width * BLOCK)
    served = fits.long().cumprod(0)
    add, need = add * served, need * served
    ends, page_ends = add.cumsum(0), need.cumsum(0)
    s["kv_len"].copy_(torch.where(ended, 0, cached + add))
    s["q_start"][0] = 0
    s["q_start"][1:] = ends
    new = (column[None, :] >= have[:, None]) & (column[None, :] < (have + need)[:, None])
    from_top = page_ends[:, None] - need[:, None] + column[None, :] - have[:, None]
    table.copy_(torch.where(new, free[torch.where(new, count - 1 - from_top, 0)], table))
    s["free"].copy_(free[:spare])
    s["left"][0] = count - page_ends[-1]
    s["served"][0] = served.sum()
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(ends, row, right=True).clamp(max=n - 1)
    at = cached[seq] + row - (ends - add)[seq]
    real = row < ends[-1]
    at = torch.where(real, at, 0)
    s["position"].copy_(torch.where(real, at, -1))
    s["slot"].copy_(torch.where(real, table[seq, at // BLOCK].long() * BLOCK + at % BLOCK, -1))
    return {k: s[k] for k in ("kv_len", "q_start", "table", "free", "left", "served", "position", "slot")}


def _norm_plain(s):
    c = s["case"]
    h = s["x"].float()
    got = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        got["sum"] = h.to(s["residual"].dtype)
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6)
    if s["weight"] is not None:
        y = y * (s["weight"].float() + c["offset"])
    if c["y"]:
        got["y"] = y.half()
    if c["codes"]:
        g = y.view(c["rows"], s["scales"].shape[1], -1)
        scale = (g.abs().amax(2, keepdim=True) / 448.0).clamp(min=2.0 ** -40)
        got["codes"] = (g / scale).clamp(-448.0, 448.0).to(E4M3).view(c["rows"], -1)
        got["scales"] = scale[:, :, 0]
    return got


def _rotary_plain(s):
    c = s["case"]
    h, kv, d, rot = c["heads"], c["kv_heads"], c["dim"], c["rot"]
    x = s["qk"].float().view(-1, h + kv, d)
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + 1e-6)
        w = torch.stack([s["q_weight"], s["k_weight"]]).float()
        x = x * w[(torch.arange(h + kv, device="cuda") >= h).long()]
    there = s["position"] >= 0
    angles = s["cos_sin"][torch.where(there, s["position"], 0).long()][:, None, :]
    cos, sin = angles[..., :rot // 2], angles[..., rot // 2:]
    turned = x[..., :rot]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if c["interleaved"] else (turned[..., :rot // 2], turned[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(2) if c["interleaved"] else torch.cat([a, b], -1)
    y = torch.cat([turned, x[..., rot:]], -1).flatten(1).half()
    return {"out": torch.where(there[:, None], y, s["out"])}


def _prompt_plain(s):
    c = s["case"]
    n, h, kv, d, most = c["seqs"], c["heads"], c["kv_heads"], c["dim"], s["max_rows"]
    slot = torch.arange(most, device="cuda")
    real = slot[None, :] < s["counts"][:, None]
    at = torch.where(real, s["q_start"][:-1, None] + slot[None, :], 0).long()
    q = s["q"].float()[at].view(n, most, kv, h // kv, d).permute(0, 2, 3, 1, 4)
    k = s["k"].float()[at].view(n, most, kv, d).transpose(1, 2)
    v = torch.where(real[:, :, None], s["v"].float()[at], 0.0).view(n, most, kv, d).transpose(1, 2)
    x = torch.matmul(q.reshape(n, kv, -1, d), k.transpose(2, 3)) * s["scale"]
    if c["cap"] > 0:
        x = c["cap"] * torch.tanh(x / c["cap"])
    seen = real[:, None, :]
    if c["causal"]:
        seen = seen & (slot[None, None, :] <= slot[None, :, None])
    x = x.view(n, kv, h // kv, most, most).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul((p / total).view(n, kv, -1, most), v).view(n, kv, h // kv, most, d).permute(0, 3, 1, 2, 4).reshape(n, most, h * d)
    lse = (torch.log(total) + top)[..., 0].permute(0, 3, 1, 2).reshape(n, most, h)
    s["out"][at[real]] = o[real].half()
    s["lse"][at[real]] = lse[real]
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"plan": _plan_plain, "norm": _norm_plain, "rotary": _rotary_plain, "prompt": _prompt_plain}[op](s)
    import trellis_quantized_linear_gb300 as tql
    if op == "plan":
        tql.exl3_kv8_plan(s["batch"], s["tokens"], s["cached"], s["free"], s["count"], s["left"], s["n_pages"], s["position"], s["slot"],
                          s["served"])
        return {k: s[k] for k in ("kv_len", "q_start", "table", "free", "left", "served", "position", "slot")}
    if op == "norm":
        tql.exl3_rms_norm(s["x"], s["y"], weight=s["weight"], residual=s["residual"], residual_out=s["sum"], eps=1e-6,
                          weight_offset=c["offset"], codes=s["codes"], scales=s["scales"])
        return {k: s[k] for k in ("sum", "y", "codes", "scales") if s[k] is not None}
    if op == "rotary":
        tql.exl3_qk_rotary(s["qk"], s["out"], c["heads"], c["kv_heads"], c["dim"], s["position"], s["cos_sin"], interleaved=c["interleaved"],
                           q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6)
        return {"out": s["out"]}
    tql.exl3_prompt_attention(s["q"], s["k"], s["v"], c["heads"], c["kv_heads"], c["dim"], s["q_start"], s["scale"], s["out"],
                              softcap=c["cap"], causal=c["causal"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    return {"plan": _exact_plan, "norm": _exact_norm, "rotary": _exact_rotary, "prompt": _exact_prompt}[case["op"]](case, _inputs(case, seed))


def _exact_plan(case, s):
    """One sequence, page and row after the other."""
    tokens, cached = _requests(case)
    table, stack, width = s["table"].tolist(), s["free"].tolist(), s["table"].shape[1]
    top = int(s["count"])
    for t, c, line in zip(tokens, cached, table):
        if t < 0:
            for page in line[:_blocks(c)]:
                stack[top] = page
                top += 1
    kv_len, q_start, position, slot, served, stopped = [], [0], [], [], 0, False
    for t, c, line in zip(tokens, cached, table):
        need = _blocks(c + t) - _blocks(c) if t > 0 else 0
        if need > top or len(position) + t > s["rows"] or t > s["max_rows"] or c + t > width * BLOCK:
            stopped = True
        if stopped and t > 0:
            t = need = 0
        served += not stopped
        for i in range(need):
            top -= 1
            line[_blocks(c) + i] = stack[top]
        for i in range(c, c + t):
            position.append(i)
            slot.append(line[i // BLOCK] * BLOCK + i % BLOCK)
        kv_len.append(0 if t < 0 else c + t)
        q_start.append(len(position))
    rest = [-1] * (s["rows"] - len(position))
    got = {"kv_len": kv_len, "q_start": q_start, "table": table, "free": stack, "left": [top], "served": [served], "position": position + rest,
           "slot": slot + rest}
    return {k: torch.tensor(v, dtype=torch.int64) for k, v in got.items()}


_VALUES = None


def _nearest(x):
    """Nearest E4M3 value, ties to the even code, of numbers within +-448."""
    global _VALUES
    if _VALUES is None:
        c = torch.arange(127, device="cuda")
        _VALUES = torch.where(c < 8, c * 2.0 ** -9, (1.0 + (c % 8) / 8.0) * 2.0 ** (c // 8 - 7.0)).double()
    a = x.abs().clamp(max=448.0)
    up = torch.searchsorted(_VALUES, a.contiguous()).clamp(max=126)
    down = (up - 1).clamp(min=0)
    du, dd = _VALUES[up] - a, a - _VALUES[down]
    code = torch.where((du < dd) | ((du == dd) & (up % 2 == 0)), up, down)
    return torch.copysign(_VALUES[code], x)


def _exact_norm(case, s):
    got = {}
    h = s["x"].double()
    if s["residual"] is not None:
        got["sum"] = h = h + s["residual"].double()
    y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["cols"] + 1e-6)
    if s["weight"] is not None:
        y = y * (case["offset"] + s["weight"].double())
    if case["y"]:
        got["y"] = y
    if case["codes"]:
        groups = y.unflatten(1, (s["scales"].shape[1], -1))
        got["scales"] = torch.clamp(groups.abs().max(2).values / 448.0, min=2.0 ** -40)
        got["codes"] = _nearest(groups / got["scales"][:, :, None]).flatten(1)
    return got


def _exact_rotary(case, s):
    """As complex numbers turned by cos + i sin."""
    out, half = s["out"].double(), case["rot"] // 2
    r = case["rows"]
    table = s["cos_sin"][s["position"][:r].long()].double()
    turn = torch.complex(table[:, :half], table[:, half:])
    for h in range(case["heads"] + case["kv_heads"]):
        x = s["qk"][:r, h * case["dim"]:(h + 1) * case["dim"]].double()
        if case["norm"]:
            w = s["q_weight"] if h < case["heads"] else s["k_weight"]
            x = x / torch.sqrt(x.pow(2).sum(1, keepdim=True) / case["dim"] + 1e-6) * w.double()
        pair = x[:, :2 * half].reshape(r, half, 2) if case["interleaved"] else x[:, :2 * half].reshape(r, 2, half).transpose(1, 2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z.reshape(r, -1) if case["interleaved"] else z.transpose(1, 2).reshape(r, -1)
        out[:r, h * case["dim"]:(h + 1) * case["dim"]] = torch.cat([z, x[:, 2 * half:]], 1)
    return {"out": out}


def _exact_prompt(case, s):
    d, kv = case["dim"], case["kv_heads"]
    g = case["heads"] // kv
    out, lse = s["out"].double(), s["lse"].double()
    r0 = 0
    for n in _lens(case):
        later = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
        for h in range(case["heads"]):
            q, k, v = (t[r0:r0 + n, i * d:(i + 1) * d].double() for t, i in ((s["q"], h), (s["k"], h // g), (s["v"], h // g)))
            x = q @ k.t() * s["scale"]
            if case["cap"] > 0:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case["causal"]:
                x[later] = -math.inf
            lse[r0:r0 + n, h] = torch.logsumexp(x, 1)
            out[r0:r0 + n, h * d:(h + 1) * d] = torch.softmax(x, 1) @ v
        r0 += n
    return {"out": out, "lse": lse}
