"""Plain 64-bit implementations of the serving operators (include/exl3.h), on
numpy arrays and one sequence, head and token at a time where that is simplest.
Nothing here comes from the library."""
import numpy as np

BLOCK = 64


def e4m3_values():
    """Value of each of the 256 E4M3 codes."""
    c = np.arange(256)
    exp, man = (c >> 3) & 15, c & 7
    v = np.where(exp == 0, man * 2.0 ** -9, (1 + man / 8.0) * 2.0 ** (exp - 7.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


VALUES = e4m3_values()
POSITIVE = VALUES[:127]


def nearest_code(x):
    """E4M3 code nearest to x, ties to the even code, saturating; NaN to 127."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    up = np.minimum(np.searchsorted(POSITIVE, a), 126)
    down = np.maximum(up - 1, 0)
    du, dd = POSITIVE[up] - a, a - POSITIVE[down]
    code = np.where((du < dd) | ((du == dd) & (up % 2 == 0)), up, down)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def block_exponent(values):
    v = np.abs(np.asarray(values, dtype=np.float64)).ravel()
    a = v[np.isfinite(v)].max(initial=0.0)
    return next(e for e in range(-32, 9) if a <= 448.0 * 2.0 ** e)


def append(codes, scales, table, kv_len, counts, rows):
    """codes n_pages x heads x 64 x D (uint8) and scales in place; rows R x heads x D."""
    r0 = 0
    for s, (length, n) in enumerate(zip(kv_len, counts)):
        first = length - n
        for b in range(max(first, 0) // BLOCK, -(-length // BLOCK)):
            page, a, z = table[s][b], max(first, b * BLOCK), min(length, (b + 1) * BLOCK)
            if z <= a:
                continue
            for h in range(codes.shape[1]):
                x = rows[r0 + a - first:r0 + z - first, h].astype(np.float64)
                e = block_exponent(x)
                old = a - b * BLOCK
                if old:
                    was = int(np.log2(scales[page, h]))
                    e = max(e, was)
                    if e != was:
                        codes[page, h, :old] = nearest_code(VALUES[codes[page, h, :old]] * 2.0 ** (was - e))
                codes[page, h, old:z - b * BLOCK] = nearest_code(x * 2.0 ** -e)
                scales[page, h] = 2.0 ** e
        r0 += n


def cached(codes, scales, table_row, length, h):
    pages = np.asarray(table_row[:-(-length // BLOCK)], dtype=np.int64)
    x = VALUES[codes[pages, h]] * scales[pages, h][:, None, None].astype(np.float64)
    return x.reshape(-1, codes.shape[3])[:length]


def attention(k, ks, v, vs, table, kv_len, counts, q, scale, cap, causal):
    """q R x H x D (any float). Returns out, lse, and for tolerances: sum p |v| per
    output, the largest |score| sum of products per row and head."""
    R, H, D = q.shape
    G = H // k.shape[1]
    out, mag = np.zeros((R, H, D)), np.zeros((R, H, D))
    lse, sabs = np.full((R, H), -np.inf), np.zeros((R, H))
    r0 = 0
    for s, (length, n) in enumerate(zip(kv_len, counts)):
        for h in range(H):
            kx, vx = cached(k, ks, table[s], length, h // G), cached(v, vs, table[s], length, h // G)
            for i in range(n):
                seen = max(0, min(length, length - n + i + 1)) if causal else length
                if seen == 0:
                    continue
                qi = q[r0 + i, h].astype(np.float64)
                x = kx[:seen] @ qi * scale
                sabs[r0 + i, h] = (np.abs(kx[:seen]) @ np.abs(qi)).max() * abs(scale)
                if cap > 0:
                    x = cap * np.tanh(x / cap)
                top = x.max()
                p = np.exp(x - top)
                lse[r0 + i, h] = top + np.log(p.sum())
                p /= p.sum()
                out[r0 + i, h], mag[r0 + i, h] = p @ vx[:seen], p @ np.abs(vx[:seen])
        r0 += n
    return out, lse, mag, sabs


def weigh(k, ks, table, kv_len, counts, q, lse, scale, cap, causal, max_tokens):
    """Added weight per sequence, head and token, and the same sum of exp(s) times each row's |score| bound."""
    R, H, D = q.shape
    Hk = k.shape[1]
    G = H // Hk
    add, bound = np.zeros((len(kv_len), Hk, max_tokens)), np.zeros((len(kv_len), Hk, max_tokens))
    r0 = 0
    for s, (length, n) in enumerate(zip(kv_len, counts)):
        for h in range(H):
            kx = cached(k, ks, table[s], length, h // G)
            for i in range(n):
                seen = max(0, min(length, length - n + i + 1)) if causal else length
                if seen == 0 or lse[r0 + i, h] == -np.inf:
                    continue
                qi = q[r0 + i, h].astype(np.float64)
                x = kx[:seen] @ qi * scale
                sabs = np.abs(kx[:seen]) @ np.abs(qi) * abs(scale)
                if cap > 0:
                    x = cap * np.tanh(x / cap)
                p = np.exp(x - lse[r0 + i, h])
                add[s, h // G, :seen] += p
                bound[s, h // G, :seen] += p * (sabs + abs(lse[r0 + i, h]) + 1)
        r0 += n
    return add, bound


def evict_choice(weights, length, budget, recent):
    """Positions kept of one sequence and head; weights in position order."""
    early = max(0, length - recent)
    key = [(-np.inf if np.isnan(w) else w) for w in weights[:early].astype(np.float64)]
    order = sorted(range(early), key=lambda t: (-key[t], t))
    return sorted(order[:max(0, min(length, budget) - (length - early))]) + list(range(early, length))


def adjust(logits, history, generated_from, rep, pres, freq, biases, allowed, dtype):
    """One row, in `dtype` (np.float32: every operation rounded by itself)."""
    n = logits.shape[0]
    x = logits.astype(dtype)
    ok = [(i, t) for i, t in enumerate(history) if 0 <= t < n]
    seen = np.zeros(n, dtype=bool)
    seen[[t for _, t in ok]] = True
    count = np.bincount([t for i, t in ok if i >= generated_from], minlength=n).astype(dtype)
    rep, pres, freq = dtype(rep), dtype(pres), dtype(freq)
    with np.errstate(invalid="ignore"):
        x = np.where(seen, np.where(x > 0, x / rep, x * rep), x)
        x = np.where(count > 0, x - (freq * count + pres), x)
        total = np.zeros(n, dtype=dtype)
        for t, b in biases:
            if 0 <= t < n:
                total[t] += dtype(b)
        x = x + total
    if allowed is not None:
        x = np.where(allowed, x, dtype(-np.inf))
    c = np.where(np.isnan(x), -np.inf, x)
    return x, (-1 if c.max() == -np.inf else int(np.argmax(c)))
