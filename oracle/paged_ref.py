"""Plain fp64 CPU oracle of the norm + rotation of queries and keys and of the paged key/value
cache (test infrastructure only, like attention_ref; shares no code with the CUDA path).

Every function is pinned by CPU tests against closed forms, finite differences, torch autograd or
the attention oracle (tests/test_norm_rope.py, tests/test_paged.py).
"""
from __future__ import annotations

import numpy as np


def rope_table(rows: int, rot: int, base: float = 10000.0) -> np.ndarray:
    """[rows, 2, rot/2]: cos and sin of p * base^(-2i/rot)."""
    ang = np.arange(rows)[:, None] * base ** (-np.arange(0, rot, 2) / max(rot, 1))[None]
    return np.stack([np.cos(ang), np.sin(ang)], 1)


def rotated_pairs(rot: int, interleaved: bool):
    """Index lists (a, b) of the rotated pairs."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(y, rope, positions, interleaved, back=False):
    """y [..., heads, d] turned by the angles of positions [...]; back: by their negatives."""
    if rope is None:
        return y.copy()
    cos, sin = (rope[positions, n][..., None, :] for n in (0, 1))
    if back:
        sin = -sin
    a, b = rotated_pairs(2 * rope.shape[2], interleaved)
    out = y.copy()
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., b] * cos + y[..., a] * sin
    return out


def norm_rope(x, w, rope, positions, interleaved, eps):
    """x [..., heads, d] normalised per row, weighted (w None: 1) and rotated."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotate(x * r * (1.0 if w is None else w), rope, positions, interleaved)


def norm_rope_backward(g, x, w, rope, positions, interleaved, eps):
    """(dx, dw) from g, the gradient of norm_rope's result."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    dy = rotate(g, rope, positions, interleaved, back=True)
    u = dy * (1.0 if w is None else w)
    dx = r * (u - xh * (u * xh).mean(-1, keepdims=True))
    return dx, (dy * xh).reshape(-1, x.shape[-1]).sum(0)


def plan(cached, new, table, free, page_size, cols, max_tokens):
    """One step's pages and slots, request by request: dict of lens, cu, slots, positions, req, table,
    free (the list of free pages, last one the top), status (bits 1 no pages, 2 row full, 4 too many
    tokens, 8 bad input); on a non-zero status everything stays."""
    R = len(cached)
    out = {"lens": list(cached), "cu": [0] * (R + 1), "slots": [], "positions": [], "req": [],
           "table": [list(r) for r in table], "free": list(free), "status": 0}
    bits = 0
    bad = [not (0 <= c <= cols * page_size and n >= -1) for c, n in zip(cached, new)]
    if any(bad):
        bits |= 8
    stack = list(free)
    pages = lambda n: -(-n // page_size)  # noqa: E731
    for b in range(R):
        if new[b] == -1 and not bad[b]:
            stack += out["table"][b][:pages(cached[b])]
    want = tokens = 0
    for b in range(R):
        if new[b] < 0 or bad[b]:
            continue
        if cached[b] + new[b] > cols * page_size:
            bits |= 2
            continue
        want += pages(cached[b] + new[b]) - pages(cached[b])
        tokens += new[b]
    bits |= (1 if want > len(stack) else 0) | (4 if tokens > max_tokens else 0)
    out["status"] = bits
    if bits == 0:
        out["free"] = stack
        for b in range(R):
            if new[b] == -1:
                out["lens"][b] = 0
            else:
                for p in range(pages(cached[b]), pages(cached[b] + new[b])):
                    out["table"][b][p] = stack.pop()
                for j in range(cached[b], cached[b] + new[b]):
                    out["slots"].append(out["table"][b][j // page_size] * page_size + j % page_size)
                    out["positions"].append(j)
                    out["req"].append(b)
                out["lens"][b] = cached[b] + new[b]
            out["cu"][b + 1] = len(out["slots"])
    pad = max_tokens - len(out["slots"])
    out["slots"] += [-1] * pad
    out["positions"] += [0] * pad
    out["req"] += [-1] * pad
    return out


def gather(cache, table_row, length, head, page_size):
    """[length, d] rows of one kv head of cache [pages, page_size, Hk, d]."""
    j = np.arange(length)
    return cache[np.asarray(table_row)[j // page_size], j % page_size, head]


def decode_row(q, k, v, scale):
    """(o [d], lse) of one query over keys k, v [n, d]; no key: zeros and -inf."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), -np.inf
    s = scale * (k @ q)
    m = s.max()
    p = np.exp(s - m)
    return (p @ v) / p.sum(), m + np.log(p.sum())


def paged_decode(q, k_cache, v_cache, table, lens, req, scale):
    """o [T, Hq, d], lse [T, Hq]; rows with req < 0 are NaN (left as they were)."""
    T, Hq, d = q.shape
    ps, Hk = k_cache.shape[1], k_cache.shape[2]
    o, lse = np.full((T, Hq, d), np.nan), np.full((T, Hq), np.nan)
    for t in range(T):
        if req[t] < 0:
            continue
        for h in range(Hq):
            hk = h // (Hq // Hk)
            k, v = (gather(c, table[req[t]], lens[t], hk, ps) for c in (k_cache, v_cache))
            o[t, h], lse[t, h] = decode_row(q[t, h], k, v, scale)
    return o, lse
