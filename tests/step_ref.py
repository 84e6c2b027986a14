"""Plain 64-bit implementations of the step operators (include/exl3.h), on numpy arrays
and one sequence, row and head at a time where that is simplest. Nothing here comes from
the library."""
import numpy as np

from serving_ref import BLOCK, nearest_code


def blocks(tokens):
    return -(-tokens // BLOCK)


def plan(tokens, cached, table, stack, count, n_pages, rows, max_rows):
    """(kv_len, q_start, position, slot, served, left, whether something was out of range);
    table and stack in place."""
    width, bad = table.shape[1], False
    if not 0 <= count <= len(stack):
        count, bad = min(max(count, 0), len(stack)), True
    valid = [0 <= c <= width * BLOCK for c in cached]
    for s, t in enumerate(tokens):
        if t < 0 and valid[s]:
            for b in range(blocks(int(cached[s]))):
                if count < len(stack):
                    stack[count] = table[s, b]
                    count += 1
                else:
                    bad = True
    kv_len, q_start, position, slot, served, stopped = [], [0], [], [], 0, False
    for s, (t, c) in enumerate(zip(tokens, cached)):
        t, c = int(t), int(c)
        bad |= not valid[s]
        new = max(t, 0)
        need = blocks(c + new) - blocks(c) if new and valid[s] else 0
        stopped |= not valid[s] or new > max_rows or c + new > width * BLOCK or need > count or len(position) + new > rows
        if stopped:
            new = need = 0
        served += not stopped
        for b in range(blocks(c), blocks(c) + need):
            count -= 1
            page = stack[count]
            if not 0 <= page < n_pages:
                page, bad = -1, True
            table[s, b] = page
        for i in range(c, c + new):
            page = table[s, i // BLOCK]
            ok = 0 <= page < n_pages
            bad |= not ok
            position.append(i)
            slot.append(page * BLOCK + i % BLOCK if ok else -1)
        kv_len.append(0 if t < 0 or not valid[s] else c + new)
        q_start.append(len(position))
    rest = [-1] * (rows - len(position))
    return kv_len, q_start, position + rest, slot + rest, served, count, bad


def rms_norm(x, residual, weight, offset, eps):
    """(h, y) in 64 bits."""
    h = x.astype(np.float64)
    if residual is not None:
        h = h + residual.astype(np.float64)
    with np.errstate(all="ignore"):
        y = h / np.sqrt((h * h).sum(1, keepdims=True) / h.shape[1] + eps)
        if weight is not None:
            y = y * (weight.astype(np.float64) + offset)
    return h, y


def scales(y, group):
    """Scale of each group of columns, from its finite values."""
    g = np.abs(y.reshape(y.shape[0], -1, group))
    return np.maximum(np.where(np.isfinite(g), g, 0.0).max(2) / 448.0, 2.0 ** -40)


def codes(y, scale, group):
    """E4M3 codes of y / scale."""
    with np.errstate(invalid="ignore"):
        return nearest_code(y / np.repeat(scale, group, 1))


def rotary(x, heads_q, heads_k, dim, position, cos_sin, interleaved, q_weight, k_weight, eps, offset):
    """x rows x (heads * dim); rows without a position in the table are left as they are."""
    out = x.astype(np.float64).copy()
    rot = cos_sin.shape[1]
    c, s = cos_sin[:, :rot // 2].astype(np.float64), cos_sin[:, rot // 2:].astype(np.float64)
    for r, p in enumerate(position):
        if not 0 <= p < len(cos_sin):
            continue
        for h in range(heads_q + heads_k):
            v = x[r, h * dim:(h + 1) * dim].astype(np.float64)
            w = q_weight if h < heads_q else k_weight
            if w is not None:
                v = v / np.sqrt((v * v).sum() / dim + eps) * (w.astype(np.float64) + offset)
            y = v.copy()
            for i in range(rot // 2):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
                y[a] = v[a] * c[p, i] - v[b] * s[p, i]
                y[b] = v[b] * c[p, i] + v[a] * s[p, i]
            out[r, h * dim:(h + 1) * dim] = y
    return out


def prompt_attention(q, k, v, q_start, heads, kv_heads, dim, scale, cap, causal):
    """(out, lse) of the rows of the sequences, NaN elsewhere. Only what a row sees is
    touched: infinities and NaN elsewhere leave no trace."""
    rows, g = q.shape[0], heads // kv_heads
    out, lse = np.full((rows, heads * dim), np.nan), np.full((rows, heads), np.nan)
    q, k, v = (a.astype(np.float64) for a in (q, k, v))
    for a, z in zip(q_start[:-1], q_start[1:]):
        n = z - a
        if n <= 0:
            continue
        for h in range(heads):
            qs, ks, vs = q[a:z, h * dim:(h + 1) * dim], k[a:z, h // g * dim:(h // g + 1) * dim], v[a:z, h // g * dim:(h // g + 1) * dim]
            with np.errstate(all="ignore"):
                x = qs @ ks.T * scale
                if cap > 0:
                    x = cap * np.tanh(x / cap)
                if causal:
                    x[np.triu_indices(n, 1)] = -np.inf
                top = x.max(1, keepdims=True)
                p = np.exp(x - top)
                total = p.sum(1, keepdims=True)
                p /= total
                o = p @ np.where(np.isfinite(vs), vs, 0.0)
                for t, d in zip(*np.nonzero(~np.isfinite(vs))):
                    seen = slice(t, None) if causal else slice(None)
                    o[seen, d] += vs[t, d]
            out[a:z, h * dim:(h + 1) * dim] = o
            lse[a:z, h] = np.log(total[:, 0]) + top[:, 0]
    return out, lse
