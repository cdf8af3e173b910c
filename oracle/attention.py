"""fp64 oracle of the attention step between q|k|v and o: page assignment, head
norms with rotary positions, attention of one token over a paged cache.  Written
from the definitions, one request, row and head at a time."""
from __future__ import annotations

import math

import numpy as np


def kv_assign(lens, n_new, page_size, table, free_pages, n_free, max_rows):
    """One step of the page bookkeeping, played through with a list as the stack.  Returns a dict of the outputs
    (copies), or None when the step is refused (a length that is negative or does not fit the table, too many
    rows, not enough pages, a free count outside the list)."""
    lens, n_new = [int(v) for v in lens], [int(v) for v in n_new]
    table, free_pages = np.array(table, np.int64), np.array(free_pages, np.int64)
    width, n_pages = table.shape[1], free_pages.size
    pages = lambda tokens: (tokens + page_size - 1) // page_size
    if not 0 <= n_free <= n_pages:
        return None
    if any(l < 0 or l + max(a, 0) > width * page_size for l, a in zip(lens, n_new)):
        return None
    if sum(max(a, 0) for a in n_new) > max_rows:
        return None
    stack = list(free_pages[:n_free])
    for b, (l, a) in enumerate(zip(lens, n_new)):
        if a < 0:
            stack.extend(table[b, :pages(l)])
    if len(stack) > n_pages:
        return None
    if sum(pages(l + a) - pages(l) for l, a in zip(lens, n_new) if a >= 0) > len(stack):
        return None
    released = stack[n_free:]
    cu, positions, slots, lens_out = [0], [], [], []
    for b, (l, a) in enumerate(zip(lens, n_new)):
        if a < 0:
            lens_out.append(0)
            cu.append(cu[-1])
            continue
        for j in range(pages(l), pages(l + a)):
            table[b, j] = stack.pop()
        for pos in range(l, l + a):
            page = table[b, pos // page_size]
            positions.append(pos)
            slots.append(page * page_size + pos % page_size if 0 <= page < n_pages else -1)
        lens_out.append(l + a)
        cu.append(cu[-1] + a)
    for i in range(n_free, len(stack)):          # released pages that nobody took
        free_pages[i] = released[i - n_free]
    pad = [-1] * (max_rows - len(slots))
    return {"block_table": table, "free_pages": free_pages, "lens_out": np.array(lens_out),
            "n_free_out": len(stack), "cu_rows": np.array(cu), "positions": np.array(positions + pad),
            "slots": np.array(slots + pad)}


def head_norm(x, gamma, eps):
    """x [..., D] * gamma / sqrt(mean(x^2) + eps); gamma None: x."""
    x = np.asarray(x, np.float64)
    if gamma is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(gamma, np.float64)


def rotate(x, position, inv_freq, factor=1.0, interleaved=False):
    """One head [D] at one position: the pairs of its first 2 * len(inv_freq) entries turned by
    position * inv_freq[i] and multiplied by factor.  Angles by math.fmod of the fp64 product."""
    x, y = np.asarray(x, np.float64), np.array(x, np.float64)
    half = len(inv_freq)
    for i, f in enumerate(inv_freq):
        a = math.fmod(float(position) * float(f), 2.0 * math.pi)
        j, k = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[j] = factor * (x[j] * math.cos(a) - x[k] * math.sin(a))
        y[k] = factor * (x[j] * math.sin(a) + x[k] * math.cos(a))
    return y


def pair_size(x, rot, interleaved=False):
    """For each entry of a head, the length of its pair (its own size where it is not rotated)."""
    x, y = np.asarray(x, np.float64), np.abs(np.array(x, np.float64))
    half = rot // 2
    for i in range(half):
        j, k = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[j] = y[k] = math.hypot(x[j], x[k])
    return y


def attend(q, keys, values, scale):
    """q [D] over keys, values [n][D]: the output, the log of the sum of exponentials, sum_j p_j |v_j| and
    max_j scale * sum_i |q_i k_ji| (the sizes that rounding errors are relative to)."""
    q, keys, values = (np.asarray(a, np.float64) for a in (q, keys, values))
    if len(keys) == 0:
        z = np.zeros(q.shape)
        return z, -math.inf, z, 0.0
    s = scale * (keys @ q)
    top = s.max()
    if top == -math.inf:
        z = np.zeros(q.shape)
        return z, -math.inf, z, 0.0
    e = np.exp(s - top)
    total = e.sum()
    return (e @ values) / total, top + math.log(total), (e @ np.abs(values)) / total, \
        abs(scale) * float((np.abs(keys) @ np.abs(q)).max())


def paged_attention(q, k_pool, v_pool, lens, table, scale, cu_rows=None):
    """q [rows][Hq][D], pools [pages][page][Hk][D]: {row: (out [Hq][D], lse [Hq], size [Hq][D], score size [Hq])}."""
    n_pages, page_size, n_kv, _ = k_pool.shape
    group = q.shape[1] // n_kv
    out = {}
    for b, length in enumerate(int(l) for l in lens):
        row = b
        if cu_rows is not None:
            if cu_rows[b] >= cu_rows[b + 1]:
                continue
            row = int(cu_rows[b + 1]) - 1
        where = [(int(table[b][j // page_size]), j % page_size) for j in range(length)]
        where = [(p, t) for p, t in where if 0 <= p < n_pages]
        pages, offs = (np.array([w[i] for w in where], np.int64) for i in (0, 1))
        heads = []
        for h in range(q.shape[1]):
            heads.append(attend(q[row, h], k_pool[pages, offs, h // group], v_pool[pages, offs, h // group], scale))
        out[row] = tuple(np.array([x[i] for x in heads]) for i in range(4))
    return out
