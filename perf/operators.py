"""The serving operators around the trellis-quantized linear layer, as cases to measure:
an 8-bit paged key/value cache (append, attention over it, accumulated attention weight,
eviction by that weight) and the adjustment of the masked logits before a token is chosen.

``run`` computes them in elementary torch operations in fp32 (``own`` false) or through the
package's entry points (``own`` true), on the same inputs.

The cache holds E4M3 codes in blocks (pages) of 64 tokens, n_pages x kv_heads x 64 x dim, with one
power-of-two scale for each block and head, keys and values apart.
"""
import math

import torch

own = False

BLOCK = 64
E4M3 = torch.float8_e4m3fn
VOCAB, LOGITS_LD = 248077, 248192  # decodable tokens, aligned logits width


def listed():
    return [
        # one user's next token after a short prompt: latency
        {"name": "attend_one", "op": "attend", "seqs": 1, "rows": 1, "len_min": 777, "len_max": 777,
         "heads": 32, "kv_heads": 8, "dim": 128, "cap": 0.0},
        # a serving batch of 16 users at ragged lengths, capped scores, five query heads to a key head
        {"name": "attend_batch", "op": "attend", "seqs": 16, "rows": 1, "len_min": 61, "len_max": 8192,
         "heads": 40, "kv_heads": 8, "dim": 128, "cap": 30.0},
        # two long documents, next token of each: the cache stream
        {"name": "attend_long", "op": "attend", "seqs": 2, "rows": 1, "len_min": 98765, "len_max": 131072,
         "heads": 40, "kv_heads": 8, "dim": 128, "cap": 0.0},
        # a 2048-token prefill chunk behind 6144 cached tokens
        {"name": "attend_chunk", "op": "attend", "seqs": 1, "rows": 2048, "len_min": 8192, "len_max": 8192,
         "heads": 40, "kv_heads": 8, "dim": 128, "cap": 0.0},
        # the new token of each of 16 users into their last blocks
        {"name": "append_token", "op": "append", "seqs": 16, "rows": 1, "len_min": 1, "len_max": 128,
         "kv_heads": 8, "dim": 128},
        # four prefill chunks, starting inside blocks that already hold tokens
        {"name": "append_chunk", "op": "append", "seqs": 4, "rows": 2048, "len_min": 2048, "len_max": 2143,
         "kv_heads": 8, "dim": 128},
        # the weight that 16 users' new tokens give to what each has cached
        {"name": "weigh_token", "op": "weigh", "seqs": 16, "rows": 1, "len_min": 61, "len_max": 8192,
         "heads": 40, "kv_heads": 8, "dim": 128, "cap": 0.0},
        # the same for a whole prefill chunk: the weights that choose what a long prompt keeps
        {"name": "weigh_chunk", "op": "weigh", "seqs": 1, "rows": 2048, "len_min": 8192, "len_max": 8192,
         "heads": 40, "kv_heads": 8, "dim": 128, "cap": 0.0},
        # one user's cache cut back a little past its budget
        {"name": "evict_small", "op": "evict", "seqs": 1, "len_min": 1100, "len_max": 1100, "budget": 1000,
         "recent": 128, "kv_heads": 8, "dim": 128},
        # eight long prompts cut to 4096 tokens each
        {"name": "evict_large", "op": "evict", "seqs": 8, "len_min": 9001, "len_max": 32768, "budget": 4096,
         "recent": 512, "kv_heads": 8, "dim": 128},
        # one user's logits with a short history
        {"name": "adjust_one", "op": "adjust", "rows": 1, "vocab": VOCAB, "ld": LOGITS_LD, "history": 700, "biases": 20,
         "grammar": True},
        # 64 users' logits with long histories
        {"name": "adjust_batch", "op": "adjust", "rows": 64, "vocab": VOCAB, "ld": LOGITS_LD, "history": 8192, "biases": 300,
         "grammar": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "weigh", "weigh", "evict", "adjust"])
    if op == "adjust":
        vocab = rng.randrange(1000, VOCAB + 1)
        return {"op": op, "rows": _log(rng, 1, 64), "vocab": vocab, "ld": (vocab + 127) // 128 * 128,
                "history": _log(rng, 1, 8192), "biases": rng.randrange(0, 300), "grammar": rng.random() < 0.7}
    dim, kv = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8])
    case = {"op": op, "seqs": _log(rng, 1, 16), "kv_heads": kv, "dim": dim}
    if op == "append":
        rows = _log(rng, 1, 2048)
        case["seqs"] = min(case["seqs"], max(1, 8192 // rows))
        return {**case, "rows": rows, "len_min": rows, "len_max": rows + rng.randrange(0, 128)}
    if op == "evict":
        most = _log(rng, 200, 32768)
        case["seqs"] = min(case["seqs"], 8)
        budget = _log(rng, 64, max(64, min(4096, most - 1)))
        return {**case, "len_min": max(1, most // rng.randrange(1, 4)), "len_max": most, "budget": budget,
                "recent": rng.randrange(0, budget // 2 + 1)}
    case["heads"] = kv * rng.choice([1, 2, 4, 5, 8])
    case["cap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
    if rng.random() < 0.6:  # single tokens, or a few speculated ones
        case["rows"] = rng.choice([1, 1, 1, 2, 4])
        most = _log(rng, 1, 131072)
        case["seqs"] = min(case["seqs"], max(1, 200000 // most))
    else:  # chunks
        case["rows"] = _log(rng, 5, 2048)
        most = case["rows"] + _log(rng, 1, 6144)
        case["heads"] = min(case["heads"], kv * max(1, 40 // kv))
        case["seqs"] = min(case["seqs"], max(1, 2048 // case["rows"]))
    least = max(case["rows"], 1)
    return {**case, "len_min": min(max(least, most // rng.randrange(1, 5)), max(least, most)), "len_max": max(least, most)}


def _lens(case):
    """Cached tokens of each sequence, spread evenly between the case's two bounds."""
    n, lo, hi = case["seqs"], case["len_min"], case["len_max"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _counts(case):
    """Rows of each sequence in this call: the case's, and fewer for every second sequence of a chunk."""
    r = case.get("rows", 0)
    return [r if i % 2 == 0 or r < 5 else r - r // 3 for i in range(case["seqs"])]


def work(case):
    op = case["op"]
    if op == "adjust":
        m, n = case["rows"], case["vocab"]
        b = m * (8 * n + 4 * case["history"] + 8 * case["biases"] + 4) + (m * ((n + 31) // 32) * 4 if case["grammar"] else 0)
        return {"bytes": b, "flops": 6 * m * n}
    kv, d, lens, counts = case["kv_heads"], case["dim"], _lens(case), _counts(case)
    blocks = sum((x + BLOCK - 1) // BLOCK for x in lens)
    if op == "append":
        new = sum(counts)
        touched = sum((x + BLOCK - 1) // BLOCK - (x - c) // BLOCK for x, c in zip(lens, counts))
        return {"bytes": 2 * kv * (new * d * 3 + touched * 4), "flops": 4 * kv * new * d}
    if op == "evict":
        kept = sum(min(x, case["budget"]) for x in lens)
        return {"bytes": kv * (4 * sum(lens) + kept * (4 * d + 4 + 4)), "flops": kv * (4 * sum(lens) + 2 * kept * d)}
    h, rows = case["heads"], sum(counts)
    seen = sum(c * (x - c) + c * (c + 1) // 2 for x, c in zip(lens, counts)) * h  # scores under the causal mask
    if op == "attend":
        return {"bytes": kv * (2 * sum(lens) * d + 8 * blocks) + rows * h * (4 * d + 4), "flops": 4 * seen * d}
    return {"bytes": kv * (sum(lens) * (d + 8) + 4 * blocks) + rows * h * (2 * d + 4), "flops": 2 * seen * d}


# --------------------------------------------------------------------------- inputs


def _block_exponent(amax):
    """Smallest e >= -32 with amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, (x - 9 + (m > 0.875).int()).clamp(-32, 8), torch.full_like(x, -32))


def _pow2(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _to_codes(x, e):
    return (x * _pow2(-e)).clamp(-448.0, 448.0).to(E4M3)


def _quantized(gen, shape, gain):
    """Codes and scales of a cache with values of every magnitude that heads have."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= gain * torch.exp(0.5 * torch.randn((shape[0], shape[1], 1, 1), generator=gen, device="cuda"))
    e = _block_exponent(x.abs().amax((2, 3)))
    return _to_codes(x, e[:, :, None, None]), _pow2(e)


def _cumulative(counts):
    t = torch.tensor([0] + counts, dtype=torch.int32)
    return t.cumsum(0).to(torch.int32).cuda()


def _cache_inputs(case, gen):
    lens, counts, kv, d = _lens(case), _counts(case), case["kv_heads"], case["dim"]
    # an evicted sequence moves to `extra` new pages at the end of the pool
    max_pages = max((x + BLOCK - 1) // BLOCK for x in lens)
    n_src = case["seqs"] * max_pages
    new_pages = (case["budget"] + BLOCK - 1) // BLOCK if case["op"] == "evict" else 0
    n_pages = n_src + case["seqs"] * new_pages
    k, ks = _quantized(gen, (n_pages, kv, BLOCK, d), 1.0)
    v, vs = _quantized(gen, (n_pages, kv, BLOCK, d), 0.5)
    perm = torch.randperm(n_src, generator=gen, device="cuda").to(torch.int32)
    s = {"case": case, "k": k, "v": v, "ks": ks, "vs": vs, "table": perm.view(case["seqs"], max_pages).contiguous(),
         "kv_len": torch.tensor(lens, dtype=torch.int32, device="cuda"), "q_start": _cumulative(counts),
         "counts": torch.tensor(counts, dtype=torch.int32, device="cuda"), "weight": None, "n_src": n_src,
         "max_rows": max(counts), "total": sum(counts)}
    if case["op"] == "evict":
        # attention weights: most tokens hardly ever attended, a few heavily, many exactly alike
        u = torch.rand((n_pages, kv, BLOCK), generator=gen, device="cuda")
        s["weight"] = torch.where(u < 0.2, torch.zeros_like(u), torch.exp(-6.0 * torch.rand(u.shape, generator=gen, device="cuda")))
        s["weight"] = torch.where((u > 0.2) & (u < 0.4), (s["weight"] * 16).floor() / 16, s["weight"])
        s["dst"] = (n_src + torch.arange(case["seqs"] * new_pages, device="cuda", dtype=torch.int32)).view(case["seqs"], new_pages)
        s["kept"] = torch.empty((case["seqs"], kv, case["budget"]), dtype=torch.int32, device="cuda")
        s["new_len"] = torch.empty((case["seqs"],), dtype=torch.int32, device="cuda")
    elif case["op"] == "append":
        # rows of a fused projection: keys and values are column ranges of one matrix
        kvx = torch.randn((s["total"], 2 * kv * d), generator=gen, device="cuda")
        kvx *= torch.exp(0.7 * torch.randn((s["total"], 1), generator=gen, device="cuda"))
        kvx = kvx.half()
        s["new_k"], s["new_v"] = kvx[:, :kv * d], kvx[:, kv * d:]
    else:
        h = case["heads"]
        s["scale"] = 1.0 / math.sqrt(d)
        qx = 2.0 * torch.randn((s["total"], (h + 2 * kv) * d), generator=gen, device="cuda")
        s["q"] = qx.half()[:, :h * d]
        if case["op"] == "attend":
            s["out"] = torch.empty((s["total"], h * d), dtype=torch.float16, device="cuda")
            s["lse"] = torch.empty((s["total"], h), dtype=torch.float32, device="cuda")
        else:
            s["weight"] = torch.rand((n_pages, kv, BLOCK), generator=gen, device="cuda")
            s["lse"] = _attend_plain({**s, "case": {**case, "op": "attend"}}, only_lse=True)
    return s


def _logit_inputs(case, gen):
    m, n, ld = case["rows"], case["vocab"], case["ld"]

    def per_row(lo, hi):
        return lo + (hi - lo) * torch.rand((m,), generator=gen, device="cuda")

    logits = 3.0 * torch.randn((m, ld), generator=gen, device="cuda")
    logits[:, n:] = -math.inf
    # histories of different lengths in which a few tokens come often
    lens = [max(1, case["history"] - (case["history"] // 3) * (i % 3)) for i in range(m)]
    total = sum(lens)
    u = torch.rand((total,), generator=gen, device="cuda")
    history = (n * u * u * u).to(torch.int32).clamp(max=n - 1)
    s = {"case": case, "logits": logits, "out": torch.empty_like(logits), "argmax": torch.empty((m,), dtype=torch.int32, device="cuda"),
         "history": history, "history_start": _cumulative(lens),
         "generated_from": torch.tensor([x // 2 for x in lens], dtype=torch.int32, device="cuda"),
         "repetition": per_row(1.0, 1.5), "presence": per_row(0.0, 1.0), "frequency": per_row(0.0, 0.5),
         "bias_id": None, "bias_value": None, "bias_start": None, "allowed": None}
    if case["biases"]:
        ids = torch.rand((m, n), generator=gen, device="cuda").topk(case["biases"], dim=1).indices
        s["bias_id"] = ids.to(torch.int32).reshape(-1)
        s["bias_value"] = 4.0 * torch.randn((m * case["biases"],), generator=gen, device="cuda")
        s["bias_start"] = _cumulative([case["biases"]] * m)
    if case["grammar"]:
        s["allowed"] = torch.randint(-2**31, 2**31, (m, (n + 31) // 32), generator=gen, device="cuda").to(torch.int32)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = _logit_inputs(case, gen) if case["op"] == "adjust" else _cache_inputs(case, gen)
    if own:
        import trellis_quantized_linear_gb300 as tql
        tql.build()
        tql.exl3_init(torch.cuda.current_device())
        if case["op"] != "adjust":
            s["cache"] = tql.Exl3Kv8Cache(s["k"], s["v"], s["ks"], s["vs"], s["weight"])
            s["batch"] = tql.Exl3Kv8Batch(s["table"], s["kv_len"], s["q_start"], s["total"], s["max_rows"])
        if case["op"] == "attend":
            n = tql.exl3_kv8_attention_workspace_bytes(s["cache"], s["batch"], case["heads"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------- plain forms


def _dense(codes, scales, table):
    """Values of the pages in `table`, seqs x kv_heads x tokens x dim, fp32."""
    x = codes.view(torch.uint8)[table.long()].view(E4M3).float() * scales[table.long()][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _row_index(s):
    """For each sequence and row slot: the row of the call (0 where there is none), and whether there is one."""
    slot = torch.arange(s["max_rows"], device="cuda")
    real = slot[None, :] < s["counts"][:, None]
    return torch.where(real, s["q_start"][:-1, None] + slot[None, :], 0).long(), real


def _scores(s):
    """Capped, masked scores seqs x kv_heads x group x row slots x tokens, and what is seen."""
    c = s["case"]
    kv, d, g = c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    at, real = _row_index(s)
    q = s["q"].float()[at].view(c["seqs"], s["max_rows"], kv, g, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k = _dense(s["k"], s["ks"], s["table"])
    limit = s["kv_len"][:, None] - s["counts"][:, None] + torch.arange(s["max_rows"], device="cuda")[None, :] + 1
    pos = torch.arange(k.shape[2], device="cuda")
    seen = (pos[None, None, :] < limit[:, :, None]) & real[:, :, None]
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    if c["cap"] > 0:
        x = c["cap"] * torch.tanh(x / c["cap"])
    x = x.view(c["seqs"], kv, g, s["max_rows"], -1)
    seen = seen[:, None, None]
    return x.masked_fill(~seen, -math.inf), at, real


def _attend_plain(s, only_lse=False):
    c = s["case"]
    x, at, real = _scores(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0].permute(0, 3, 1, 2).reshape(c["seqs"], s["max_rows"], c["heads"])[real]
    if only_lse:
        return lse.contiguous()
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    cached = torch.arange(x.shape[-1], device="cuda")[None, :] < s["kv_len"][:, None]
    v = torch.where(cached[:, None, :, None], _dense(s["v"], s["vs"], s["table"]), 0.0)
    o = torch.matmul(p.flatten(2, 3), v).view(c["seqs"], c["kv_heads"], -1, s["max_rows"], c["dim"])
    o = o.permute(0, 3, 1, 2, 4).reshape(c["seqs"], s["max_rows"], c["heads"] * c["dim"])[real]
    return {"out": o.half(), "lse": lse}


def _weigh_plain(s):
    c = s["case"]
    x, at, real = _scores(s)
    lse = s["lse"][at].view(c["seqs"], s["max_rows"], c["kv_heads"], -1).permute(0, 2, 3, 1)
    lse = torch.where(lse == -math.inf, math.inf, lse)
    add = torch.exp(x - lse[..., None]).sum((2, 3))  # seqs x kv_heads x tokens
    add = add.view(c["seqs"], c["kv_heads"], -1, BLOCK).permute(0, 2, 1, 3).flatten(0, 1)
    t = s["table"].long().flatten()
    s["weight"][t] = s["weight"][t] + add
    return {"weight": s["weight"]}


def _append_plain(s):
    c = s["case"]
    kv, d, n = c["kv_heads"], c["dim"], c["seqs"]
    at, real = _row_index(s)
    tokens = s["table"].shape[1] * BLOCK
    first = s["kv_len"] - s["counts"]
    pos = torch.arange(tokens, device="cuda")
    slot = pos[None, :] - first[:, None]  # row slot that a cached token comes from
    new = (slot >= 0) & (slot < s["counts"][:, None])
    old = pos[None, :] < first[:, None]
    row = at.gather(1, slot.clamp(0, s["max_rows"] - 1).long())
    t = s["table"].long().flatten()

    def blocks(x):
        return x.view(n, -1, BLOCK, kv, d).transpose(2, 3).flatten(0, 1)

    new_b, old_b = new.view(-1, 1, BLOCK, 1), old.view(-1, 1, BLOCK, 1)
    touched = new_b.any(2, keepdim=True)
    for codes, scales, rows in ((s["k"], s["ks"], s["new_k"]), (s["v"], s["vs"], s["new_v"])):
        x = blocks(rows.float()[row])
        amax = torch.where(new_b & torch.isfinite(x), x.abs(), 0.0).amax((2, 3), keepdim=True)
        need = _block_exponent(amax)
        had = torch.frexp(scales[t])[1][:, :, None, None] - 1
        e = torch.where(old_b.any(2, keepdim=True), torch.maximum(had, need), need)
        was = codes.view(torch.uint8)[t].view(E4M3)
        again = (was.float() * _pow2(had - e)).to(E4M3)
        got = torch.where(new_b, _to_codes(x, e).view(torch.uint8), torch.where(old_b, again.view(torch.uint8), was.view(torch.uint8)))
        codes.view(torch.uint8)[t] = torch.where(touched, got, was.view(torch.uint8))
        scales[t] = torch.where(touched, _pow2(e), scales[t][:, :, None, None])[..., 0, 0]
    return {"k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"]}


def _evict_plain(s):
    c = s["case"]
    n, kv, d, budget = c["seqs"], c["kv_heads"], c["dim"], c["budget"]
    t = s["table"].long()
    w = s["weight"][t].permute(0, 2, 1, 3).flatten(2, 3)  # seqs x kv_heads x tokens
    tokens = w.shape[2]
    pos = torch.arange(tokens, device="cuda")
    length = s["kv_len"][:, None, None]
    key = torch.where(torch.isnan(w), -math.inf, w)
    # a rank for each token: the recent ones, then the others by weight, then what is not cached
    level = (pos >= length - c["recent"]).int() + (pos < length).int() - (pos >= length).int()
    by_weight = torch.sort(key, dim=2, descending=True, stable=True).indices
    by_level = torch.sort(level.expand_as(key).gather(2, by_weight), dim=2, descending=True, stable=True).indices
    first = by_weight.gather(2, by_level)[:, :, :budget]
    if first.shape[2] < budget:
        first = torch.nn.functional.pad(first, (0, budget - first.shape[2]), value=tokens)
    new_len = s["kv_len"].clamp(max=budget)
    first = torch.where(torch.arange(budget, device="cuda") < new_len[:, None, None], first, tokens)
    kept = torch.sort(first, dim=2).values
    real = kept < tokens
    s["kept"].copy_(torch.where(real, kept, -1))
    s["new_len"].copy_(new_len)
    pages = s["dst"].shape[1]
    src = torch.nn.functional.pad(torch.where(real, kept, 0), (0, pages * BLOCK - budget))
    real = torch.nn.functional.pad(real, (0, pages * BLOCK - budget))
    page = t[:, None, :].expand(n, kv, -1).gather(2, src // BLOCK)
    head = torch.arange(kv, device="cuda")[None, :, None]
    to = s["dst"].long().flatten()

    def blocks(x):
        return x.view((n, kv, pages, BLOCK) + x.shape[3:]).transpose(1, 2).flatten(0, 1)

    written = blocks(real)
    held = written.any(2)
    for codes, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        x = codes.view(torch.uint8)[page, head, src % BLOCK].view(E4M3).float()
        had = torch.frexp(scales[page, head])[1] - 1
        e = torch.where(real, had, -64).view(n, kv, pages, BLOCK).amax(3)
        moved = (x * _pow2(had - e.repeat_interleave(BLOCK, 2))[..., None]).to(E4M3).view(torch.uint8)
        codes.view(torch.uint8)[to] = torch.where(written[..., None], blocks(moved), codes.view(torch.uint8)[to])
        scales[to] = torch.where(held, _pow2(e.transpose(1, 2).flatten(0, 1)), scales[to])
    s["weight"][to] = torch.where(written, blocks(s["weight"][page, head, src % BLOCK]), s["weight"][to])
    new = s["n_src"]
    return {"kept": s["kept"], "new_len": s["new_len"], "k": s["k"][new:], "v": s["v"][new:], "k_scale": s["ks"][new:],
            "v_scale": s["vs"][new:], "weight": s["weight"][new:]}


def _adjust_plain(s):
    c = s["case"]
    m, n = c["rows"], c["vocab"]
    lens = (s["history_start"][1:] - s["history_start"][:-1]).long()
    row = torch.repeat_interleave(torch.arange(m, device="cuda"), lens, output_size=s["history"].numel())
    place = torch.arange(s["history"].numel(), device="cuda") - s["history_start"][row]
    at = row * n + s["history"].long()
    one = torch.ones_like(at, dtype=torch.int32)
    seen = torch.zeros(m * n, dtype=torch.int32, device="cuda").index_add_(0, at, one).view(m, n) > 0
    made = (place >= s["generated_from"][row]).int()
    count = torch.zeros(m * n, dtype=torch.int32, device="cuda").index_add_(0, at, made).view(m, n).float()
    x, rep = s["logits"][:, :n], s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - (s["frequency"][:, None] * count + torch.where(count > 0, s["presence"][:, None], 0.0))
    if s["bias_id"] is not None:
        lens = (s["bias_start"][1:] - s["bias_start"][:-1]).long()
        row = torch.repeat_interleave(torch.arange(m, device="cuda"), lens, output_size=s["bias_id"].numel())
        bias = torch.zeros((m, n), device="cuda")
        bias[row, s["bias_id"].long()] = s["bias_value"]
        x = x + bias
    if s["allowed"] is not None:
        token = torch.arange(n, device="cuda")
        bit = (s["allowed"][:, token // 32] >> (token % 32)) & 1
        x = torch.where(bit == 1, x, -math.inf)
    best = x.amax(1, keepdim=True)
    index = torch.where(x == best, torch.arange(n, device="cuda"), n).amin(1)
    s["out"][:, :n] = x
    s["argmax"].copy_(torch.where(best[:, 0] == -math.inf, -1, index))
    return {"logits": s["out"][:, :n], "argmax": s["argmax"]}


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"attend": _attend_plain, "append": _append_plain, "weigh": _weigh_plain, "evict": _evict_plain,
                "adjust": _adjust_plain}[op](s)
    import trellis_quantized_linear_gb300 as tql
    if op == "attend":
        tql.exl3_kv8_attention(s["cache"], s["batch"], s["q"], c["heads"], s["scale"], s["out"], s["workspace"],
                               softcap=c["cap"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "append":
        tql.exl3_kv8_append(s["cache"], s["batch"], s["new_k"], s["new_v"])
        return {"k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if op == "weigh":
        tql.exl3_kv8_weigh(s["cache"], s["batch"], s["q"], c["heads"], s["scale"], s["lse"], softcap=c["cap"])
        return {"weight": s["weight"]}
    if op == "evict":
        tql.exl3_kv8_evict(s["cache"], s["batch"], s["dst"], c["budget"], c["recent"], s["kept"], s["new_len"])
        new = s["n_src"]
        return {"kept": s["kept"], "new_len": s["new_len"], "k": s["k"][new:], "v": s["v"][new:], "k_scale": s["ks"][new:],
                "v_scale": s["vs"][new:], "weight": s["weight"][new:]}
    tql.exl3_logits_adjust(s["logits"], c["vocab"], s["out"], s["argmax"], history=s["history"], history_start=s["history_start"],
                           generated_from=s["generated_from"], repetition=s["repetition"], presence=s["presence"],
                           frequency=s["frequency"], bias_id=s["bias_id"], bias_value=s["bias_value"],
                           bias_start=s["bias_start"], allowed=s["allowed"])
    return {"logits": s["out"][:, :c["vocab"]], "argmax": s["argmax"]}


# --------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "adjust":
        return _exact_adjust(case, _logit_inputs(case, gen))
    s = _cache_inputs(case, gen)
    return {"attend": _exact_attention, "weigh": _exact_attention, "append": _exact_append, "evict": _exact_evict}[case["op"]](case, s)


def _sequence(s, codes, scales, i, h, length):
    """One sequence's cached values of one head, token by token, fp64."""
    pages = s["table"][i, :(length + BLOCK - 1) // BLOCK].long()
    x = codes.view(torch.uint8)[pages, h].view(E4M3).double() * scales[pages, h].double()[:, None, None]
    return x.reshape(-1, x.shape[-1])[:length]


def _exact_attention(case, s):
    d, kv = case["dim"], case["kv_heads"]
    g, weigh = case["heads"] // kv, case["op"] == "weigh"
    out = torch.zeros((s["total"], case["heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((s["total"], case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    weight = None if s["weight"] is None else s["weight"].double()
    r0 = 0
    for i, (length, rows) in enumerate(zip(_lens(case), _counts(case))):
        last = torch.arange(rows, device="cuda") + (length - rows)  # the last position that each row sees
        hidden = torch.arange(length, device="cuda")[None, :] > last[:, None]
        for h in range(kv):
            key = _sequence(s, s["k"], s["ks"], i, h, length)
            q = s["q"][r0:r0 + rows, h * g * d:(h + 1) * g * d].double().reshape(rows, g, d)
            x = torch.einsum("rgd,td->grt", q, key) * s["scale"]
            if case["cap"] > 0:
                x = case["cap"] * torch.tanh(x / case["cap"])
            x[:, hidden] = -math.inf
            if weigh:
                p = torch.exp(x - s["lse"][r0:r0 + rows, h * g:(h + 1) * g].double().t()[:, :, None]).sum((0, 1))
                page = s["table"][i, :(length + BLOCK - 1) // BLOCK].long()
                grown = torch.zeros(page.numel() * BLOCK, dtype=torch.float64, device="cuda")
                grown[:length] = p
                weight[page, h] += grown.view(-1, BLOCK)
            else:
                lse[r0:r0 + rows, h * g:(h + 1) * g] = torch.logsumexp(x, 2).t()
                value = _sequence(s, s["v"], s["vs"], i, h, length)
                out[r0:r0 + rows, h * g:(h + 1) * g] = torch.einsum("grt,td->rgd", torch.softmax(x, 2), value)
        r0 += rows
    return {"weight": weight} if weigh else {"out": out.reshape(s["total"], -1), "lse": lse}


def _exact_exponent(a):
    """Smallest e in -32 .. 8 with a <= 448 * 2^e, by trying each."""
    e = torch.full_like(a, 8.0)
    for x in range(7, -33, -1):
        e = torch.where(a <= 448.0 * 2.0 ** x, float(x), e)
    return e


def _exact_pow2(e):
    return ((e.round().long() + 1023) << 52).view(torch.float64)


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


def _exact_append(case, s):
    got = {}
    d = case["dim"]
    for name, codes, scales, rows in (("k", s["k"], s["ks"], s["new_k"]), ("v", s["v"], s["vs"], s["new_v"])):
        value, scale = codes.double(), scales.double()
        r0 = 0
        for i, (length, n) in enumerate(zip(_lens(case), _counts(case))):
            for b in range((length - n) // BLOCK, (length + BLOCK - 1) // BLOCK):
                page = int(s["table"][i, b])
                a = max(length - n, b * BLOCK)
                z = min(length, (b + 1) * BLOCK)
                x = rows[r0 + a - (length - n):r0 + z - (length - n)].double().view(z - a, -1, d).transpose(0, 1)
                e = _exact_exponent(x.abs().amax((1, 2)))
                if a > b * BLOCK:  # older tokens share the block
                    e = torch.maximum(e, torch.log2(scale[page]).round())
                    value[page, :, :a - b * BLOCK] = _nearest(value[page, :, :a - b * BLOCK] * (scale[page] * _exact_pow2(-e))[:, None, None])
                value[page, :, a - b * BLOCK:z - b * BLOCK] = _nearest(x * _exact_pow2(-e)[:, None, None])
                scale[page] = _exact_pow2(e)
            r0 += n
        got[name], got[name + "_scale"] = value, scale
    return got


def _exact_evict(case, s):
    kv, budget, new = case["kv_heads"], case["budget"], s["n_src"]
    kept = torch.full((case["seqs"], kv, budget), -1, dtype=torch.int64)
    got = {"k": s["k"][new:].double(), "v": s["v"][new:].double(), "k_scale": s["ks"][new:].double(),
           "v_scale": s["vs"][new:].double(), "weight": s["weight"][new:].double()}
    table = s["table"].long().cpu()
    for i, length in enumerate(_lens(case)):
        for h in range(kv):
            pages = s["table"][i].long()
            w = s["weight"][pages, h].reshape(-1)[:length].cpu().numpy()
            early = max(0, length - case["recent"])
            order = sorted(range(early), key=lambda t: (-w[t], t))[:max(0, min(length, budget) - (length - early))]
            keep = torch.tensor(sorted(order) + list(range(early, length)))
            kept[i, h, :keep.numel()] = keep
            for b in range((keep.numel() + BLOCK - 1) // BLOCK):
                at = keep[b * BLOCK:(b + 1) * BLOCK]
                p, o = table[i, at // BLOCK].cuda(), (at % BLOCK).cuda()
                page = int(s["dst"][i, b]) - new
                for name, codes, scales in (("k", s["k"], s["ks"]), ("v", s["v"], s["vs"])):
                    from_scale = scales[p, h].double()
                    x = codes.view(torch.uint8)[p, h, o].view(E4M3).double() * from_scale[:, None]
                    got[name + "_scale"][page, h] = from_scale.max()
                    got[name][page, h, :at.numel()] = _nearest(x / from_scale.max())
                got["weight"][page, h, :at.numel()] = s["weight"][p, h, o].double()
    return {"kept": kept.cuda(), "new_len": s["kv_len"].clamp(max=budget).long(), **got}


def _exact_adjust(case, s):
    n = case["vocab"]
    x = s["logits"][:, :n].double()
    starts = s["history_start"].tolist()
    for r in range(case["rows"]):
        past = s["history"][starts[r]:starts[r + 1]].long()
        made = torch.bincount(past[int(s["generated_from"][r]):], minlength=n).double()
        for_any = torch.bincount(past, minlength=n) > 0
        rep = s["repetition"][r].double()
        x[r] = torch.where(for_any, torch.where(x[r] > 0, x[r] / rep, x[r] * rep), x[r])
        x[r] -= s["frequency"][r].double() * made + s["presence"][r].double() * (made > 0)
        if s["bias_id"] is not None:
            a, z = int(s["bias_start"][r]), int(s["bias_start"][r + 1])
            x[r, s["bias_id"][a:z].long()] += s["bias_value"][a:z].double()
        if s["allowed"] is not None:
            words = s["allowed"][r].cpu().numpy().view("uint32")
            bits = ((words[:, None] >> torch.arange(32).numpy()) & 1).reshape(-1)[:n]
            x[r, torch.from_numpy(bits).cuda() == 0] = -math.inf
    top = x.max(1)
    return {"logits": x, "argmax": torch.where(top.values == -math.inf, -1, top.indices)}
