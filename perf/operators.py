"""The operators around a paged key/value cache and in front of the attention kernels, as
measured cases: per-head norm + rotation of queries and keys (forward and backward), the same
step writing a paged cache, the plan of a serving step (block tables and slots), and the
attention of one new token per request over the paged cache.

``own`` selects what ``run`` does: the operators in plain torch (False), or the calls that a
user makes of ``io_aware_exact_22_b200.fa`` (True).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # training, the multi-head benchmark shape (d = 64): latency and a short stream
        {"name": "norm-rope B4 H16 N1024 d64", "op": "rope", "B": 4, "N": 1024, "Hq": 16, "Hk": 16, "d": 64,
         "rot": 64, "inter": False, "fused": False, "pos": False},
        # training, the long-sequence benchmark shape
        {"name": "norm-rope B1 H32 N16384 d128", "op": "rope", "B": 1, "N": 16384, "Hq": 32, "Hk": 32, "d": 128,
         "rot": 128, "inter": False, "fused": True, "pos": False},
        # its gradient at the backward benchmark's shape
        {"name": "norm-rope bwd B2 H16 N4096 d128", "op": "rope_bwd", "B": 2, "N": 4096, "Hq": 16, "Hk": 16, "d": 128,
         "rot": 128, "inter": False, "fused": True, "pos": False},
        # gradient with shared key heads, an odd length, packed positions, half of the head rotated in pairs
        {"name": "norm-rope bwd B3 Hq8 Hk2 N1001 d64", "op": "rope_bwd", "B": 3, "N": 1001, "Hq": 8, "Hk": 2, "d": 64,
         "rot": 32, "inter": True, "fused": True, "pos": True},
        # a decode step's append: a few requests, one token each
        {"name": "append 8 tokens Hq32 Hk8 d128", "op": "append", "T": 8, "pad": 0, "Hq": 32, "Hk": 8, "d": 128,
         "rot": 128, "inter": False, "fp8": False, "ps": 16, "pages": 512},
        # a chunk of prompts written to an E4M3 cache, padded to the graph's size
        {"name": "append 4099 tokens Hq32 Hk4 d128 E4M3", "op": "append", "T": 4099, "pad": 93, "Hq": 32, "Hk": 4,
         "d": 128, "rot": 128, "inter": False, "fp8": True, "ps": 64, "pages": 200},
        # plan of a decode step: every request grows by one token
        {"name": "plan 16 requests decode", "op": "plan", "R": 16, "maxlen": 4096, "chunk": 1, "gone": 0, "ps": 16},
        # plan of a mixed step: prompts' chunks, decoding and finished requests
        {"name": "plan 1000 requests mixed", "op": "plan", "R": 1000, "maxlen": 6000, "chunk": 301, "gone": 9, "ps": 32},
        # one request, a short context: latency
        {"name": "decode 1 x 300 H16 d64", "op": "decode", "T": 1, "lo": 300, "hi": 300, "Hq": 16, "Hk": 16, "d": 64,
         "ps": 16, "fp8": False},
        # an ordinary ragged batch over shared key heads, one request without a token in the cache
        {"name": "decode 32 x 0-4096 Hq32 Hk8 d128", "op": "decode", "T": 32, "lo": 0, "hi": 4096, "Hq": 32, "Hk": 8,
         "d": 128, "ps": 16, "fp8": False},
        # two long contexts: the work has to be split over the length
        {"name": "decode 2 x 131071 Hq32 Hk4 d128", "op": "decode", "T": 2, "lo": 131001, "hi": 131071, "Hq": 32,
         "Hk": 4, "d": 128, "ps": 64, "fp8": False},
        # a large batch over an E4M3 cache
        {"name": "decode 64 x 1024-8192 Hq64 Hk8 d128 E4M3", "op": "decode", "T": 64, "lo": 1024, "hi": 8192, "Hq": 64,
         "Hk": 8, "d": 128, "ps": 32, "fp8": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "plan", "decode", "decode"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 8, 16])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if op in ("rope", "rope_bwd"):
        B = rng.randint(1, 4)
        most = (1 << 26) // (B * Hk * (g + 1) * d)  # elements of q and k: the long-sequence shape's at most
        return {"op": op, "B": B, "N": _log(rng, 1, min(16384, most)), "Hq": Hk * g, "Hk": Hk, "d": d,
                "rot": rng.choice([0, 16, 32, 48, d // 2, d, d, d][0 if d == 128 else 1:]), "inter": rng.random() < 0.4,
                "fused": rng.random() < 0.5, "pos": rng.random() < 0.5}
    if op == "append":
        T = _log(rng, 1, 8192)
        ps = rng.choice([1, 8, 16, 20, 32, 64, 128, 256])
        return {"op": op, "T": T, "pad": rng.choice([0, 0, rng.randint(1, 100)]), "Hq": Hk * g, "Hk": Hk, "d": d,
                "rot": rng.choice([32, d // 2, d, d, d]), "inter": rng.random() < 0.4, "fp8": rng.random() < 0.5,
                "ps": ps, "pages": T // ps + rng.randint(2, 40)}
    if op == "plan":
        R = _log(rng, 1, 1500)
        return {"op": op, "R": R, "maxlen": _log(rng, 40, 8000), "chunk": _log(rng, 1, min(2000, 100000 // R + 1)),
                "gone": rng.choice([0, 0, 3, 8]), "ps": rng.choice([1, 16, 16, 24, 32, 64, 128])}
    fp8 = rng.random() < 0.4
    T = _log(rng, 1, 128)
    ps = rng.choice([1, 8, 16, 20, 32, 64, 128, 256])
    most = (1 << 28) // (T * Hk * d)  # keys of a request: the plain form's padded copy stays within 2 GB
    hi = _log(rng, 1, max(1, min(65536, most)))
    return {"op": op, "T": T, "lo": rng.choice([0, hi // 2, hi]), "hi": hi, "Hq": Hk * g, "Hk": Hk, "d": d, "ps": ps,
            "fp8": fp8}


def _lens(c):
    """The context lengths of a decode case: spread evenly over its range, whatever the seed."""
    T = c["T"]
    return [c["lo"] + (c["hi"] - c["lo"]) * i // max(1, T - 1) for i in range(T)] if T > 1 else [c["hi"]]


def _plan_lens(c):
    """Cached and new tokens of a plan case's requests: lengths spread over the range, every
    `gone`-th request finished (-1), every third of the others a prompt's chunk, the rest one
    token.  With chunk 1 every request grows by one token."""
    R, i = c["R"], np.arange(c["R"])
    cached = (i * 2654435761 % (c["maxlen"] + 1)).astype(np.int64)
    new = np.where(i % 3 == 0, 1 + (i * 40503) % c["chunk"], 1)
    if c["gone"]:
        new[i % c["gone"] == c["gone"] - 1] = -1
    return cached, new


# ------------------------------------------------------------------ inputs
def _rope_table(rows, rot):
    """cos and sin of position * 10000^(-2i/rot), fp32 [rows, 2, rot/2], from 64-bit angles."""
    if rot == 0:
        return None
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * inv[None]
    return torch.stack([ang.cos(), ang.sin()], 1).float().contiguous()


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _weight(g, d):
    return (1 + 0.2 * _randn(g, d)).bfloat16()


def _cache(g, pages, ps, Hk, d, fp8):
    """A cache in use: every slot holds some earlier token's values."""
    def one():
        if not fp8:
            return torch.randn(pages, ps, Hk, d, generator=g, device=DEV, dtype=torch.bfloat16)
        return (64 * torch.randn(pages, ps, Hk, d, generator=g, device=DEV, dtype=torch.bfloat16)).clamp(-448, 448).to(
            torch.float8_e4m3fn)
    return one(), one()


def _descales(g, Hk, fp8):
    if not fp8:
        return None, None
    return tuple((1 + 0.2 * torch.rand(Hk, generator=g, device=DEV)) / 64 for _ in range(2))


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + 17)
    s = {"c": c, "op": op}
    if op in ("rope", "rope_bwd"):
        B, N, Hq, Hk, d = c["B"], c["N"], c["Hq"], c["Hk"], c["d"]
        if c["fused"]:  # q, k as a projection of q, k and v leaves them
            x = _randn(g, B, N, Hq + 2 * Hk, d).bfloat16()
            s["q"], s["k"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
        else:
            s["q"], s["k"] = _randn(g, B, N, Hq, d).bfloat16(), _randn(g, B, N, Hk, d).bfloat16()
        s["wq"], s["wk"] = _weight(g, d), _weight(g, d)
        s["pos"] = None
        rows = N
        if c["pos"]:  # sequences packed into the rows: positions start again inside a row
            rows = max(2, N // 2 + 1)
            start = torch.randint(0, rows, (B, 1), generator=g, device=DEV)
            s["pos"] = ((start + torch.arange(N, device=DEV)[None]) % rows).int()
        s["rope"] = _rope_table(rows, c["rot"])
        if op == "rope":
            s["q_out"] = torch.empty(B, Hq, N, d, device=DEV, dtype=torch.bfloat16)
            s["k_out"] = torch.empty(B, Hk, N, d, device=DEV, dtype=torch.bfloat16)
        else:
            s["gq"], s["gk"] = _randn(g, B, Hq, N, d).bfloat16(), _randn(g, B, Hk, N, d).bfloat16()
    elif op == "append":
        T, Hq, Hk, d = c["T"], c["Hq"], c["Hk"], c["d"]
        n = T + c["pad"]
        x = _randn(g, n, Hq + 2 * Hk, d).bfloat16()
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
        s["wq"], s["wk"] = _weight(g, d), _weight(g, d)
        s["rope"] = _rope_table(40000, c["rot"])
        s["pos"] = torch.randint(0, 40000, (n,), generator=g, device=DEV).int()
        s["slots"] = torch.randperm(c["pages"] * c["ps"], generator=g, device=DEV)[:n].contiguous()
        s["slots"] = torch.cat([s["slots"][:T], torch.full((c["pad"],), -1, device=DEV, dtype=torch.int64)])
        s["kd"], s["vd"] = _descales(g, Hk, c["fp8"])
        s["kc"], s["vc"] = _cache(g, c["pages"], c["ps"], Hk, d, c["fp8"])
        s["q_out"] = torch.zeros(n, Hq, d, device=DEV, dtype=torch.bfloat16)
    elif op == "plan":
        cached, new = _plan_lens(c)
        R, ps = c["R"], c["ps"]
        order = torch.randperm(R, generator=g, device=DEV)
        s["cached"] = torch.from_numpy(cached).to(DEV)[order].int()
        s["new"] = torch.from_numpy(new).to(DEV)[order].int()
        maxp = (c["maxlen"] + c["chunk"] + ps) // ps + 1
        used = (cached + ps - 1) // ps
        want = (cached + np.maximum(new, 0) + ps - 1) // ps - used
        pool = int(used.sum() + want.sum()) + 10
        pages = torch.randperm(pool, generator=g, device=DEV).int()
        used = ((s["cached"] + ps - 1) // ps).long()
        first = torch.cumsum(used, 0) - used
        j = torch.arange(maxp, device=DEV)[None]
        s["table"] = torch.where(j < used[:, None], pages[(first[:, None] + j).clamp(max=pool - 1)], -1).int()
        n_used = int(used.sum())
        s["free"] = torch.cat([pages[n_used:], torch.full((n_used,), -1, device=DEV, dtype=torch.int32)])
        s["n_free"] = torch.tensor([pool - n_used], device=DEV, dtype=torch.int32)
        s["tokens"] = int(np.maximum(new, 0).sum()) + R // 8
        for name, size, kind in (("lens", R, torch.int32), ("cu", R + 1, torch.int32), ("slots", s["tokens"], torch.int64),
                                 ("pos", s["tokens"], torch.int32), ("req", s["tokens"], torch.int32),
                                 ("n_free_out", 1, torch.int32), ("status", 1, torch.int32)):
            s[name] = torch.empty(size, device=DEV, dtype=kind)
    else:
        T, Hq, Hk, d, ps = c["T"], c["Hq"], c["Hk"], c["d"], c["ps"]
        lens = np.array(_lens(c))
        order = torch.randperm(T, generator=g, device=DEV)
        s["lens"] = torch.from_numpy(lens).to(DEV)[order].int()
        need = (lens + ps - 1) // ps
        maxp, pool = max(1, int(need.max())), int(need.sum()) + 3
        used = ((s["lens"] + ps - 1) // ps).long()
        first = torch.cumsum(used, 0) - used
        pages = torch.randperm(pool, generator=g, device=DEV).int()
        j = torch.arange(maxp, device=DEV)[None]
        s["table"] = torch.where(j < used[:, None], pages[(first[:, None] + j).clamp(max=pool - 1)], -1).int()
        s["kc"], s["vc"] = _cache(g, pool, ps, Hk, d, c["fp8"])
        s["kd"], s["vd"] = _descales(g, Hk, c["fp8"])
        s["q"] = _randn(g, T, Hq, d).bfloat16()
        s["out"] = torch.empty(T, Hq, d, device=DEV, dtype=torch.bfloat16)
        s["lse"] = torch.empty(T, Hq, device=DEV, dtype=torch.float32)
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(y, rope, pos, inter, back=False):
    """y [..., heads, d] rotated by the table rows of pos [...] (back: by the negative angles)."""
    if rope is None:
        return y
    half = rope.shape[-1]
    t = rope[pos.long()].to(y.dtype)
    cos, sin = t[..., None, 0, :], t[..., None, 1, :]
    if back:
        sin = -sin
    r = y[..., :2 * half]
    if inter:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, y[..., 2 * half:]], -1)


EPS = 1e-6


def _norm_rope(x, w, rope, pos, inter):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return _rotate(x * r * w.float(), rope, pos, inter)


def _norm_rope_bwd(go, x, w, rope, pos, inter):
    x, go = x.float(), go.transpose(1, 2).float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    dy = _rotate(go, rope, pos, inter, back=True)
    dw = (dy * xh).double().sum((0, 1, 2)).float()
    u = dy * w.float()
    dx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
    return dx.bfloat16(), dw


def _positions(s):
    x = s["q"]
    if s["pos"] is not None:
        return s["pos"]
    return torch.arange(x.shape[1], device=DEV)[None].expand(x.shape[0], -1)


def _store(cache, slots, x, descale):
    """x [n, Hk, d] written at the tokens' slots (slot -1: nothing written)."""
    if descale is not None:
        x = (x / descale[:, None]).clamp(-448, 448)
    pages, ps, Hk, d = cache.shape
    old = cache.reshape(pages * ps, Hk, d)
    kind = torch.uint8 if cache.dtype == torch.float8_e4m3fn else cache.dtype
    new = torch.cat([old.view(kind), old[:1].view(kind)])  # the last row takes the skipped tokens
    new[torch.where(slots < 0, pages * ps, slots)] = x.to(cache.dtype).view(kind)
    return new[:-1].view(cache.dtype).view(cache.shape)


def _plan(s):
    ps, cached, new = s["c"]["ps"], s["cached"].long(), s["new"].long()
    table, free = s["table"], s["free"]
    R, maxp = table.shape
    cap = free.shape[0]
    n0 = s["n_free"].long()
    used = (cached + ps - 1) // ps
    gone = new < 0
    grow = new.clamp(min=0)
    want = torch.where(gone, 0, (cached + grow + ps - 1) // ps - used)
    back = torch.where(gone, used, 0)
    j = torch.arange(maxp, device=DEV)[None]
    # released pages go on the stack in order of request and page
    at = n0 + (torch.cumsum(back, 0) - back)[:, None] + j
    stack = torch.cat([free, free[:1]])
    stack.scatter_(0, torch.where(j < back[:, None], at, cap).flatten(), table.flatten())
    stack = stack[:cap]
    avail = n0 + back.sum()
    total, tokens = want.sum(), grow.sum()
    bits = ((total > avail).int() + 2 * (torch.where(gone, 0, cached + grow) > maxp * ps).any().int()
            + 4 * (tokens > s["tokens"]).int())
    ok = bits == 0
    # wanted pages come off its top in the same order
    order = (torch.cumsum(want, 0) - want)[:, None] + j - used[:, None]
    fresh = (j >= used[:, None]) & (j < (used + want)[:, None]) & ok
    table = torch.where(fresh, stack[(avail - 1 - order).clamp(0, cap - 1)], table)
    cu = torch.cat([torch.zeros(1, device=DEV, dtype=torch.int64), torch.cumsum(grow, 0)])
    cu = torch.where(ok, cu, 0)
    t = torch.arange(s["tokens"], device=DEV)
    req = (t[:, None] >= cu[None, 1:]).sum(1)
    live = req < R
    req = req.clamp(max=R - 1)
    pos = cached[req] + t - cu[req]
    page = table[req, (pos // ps).clamp(max=maxp - 1)].long()
    return {"lens": torch.where(ok, torch.where(gone, 0, cached + grow), cached).int(), "cu": cu.int(),
            "slots": torch.where(live, page * ps + pos % ps, -1), "pos": torch.where(live, pos, 0).int(),
            "req": torch.where(live, req, -1).int(), "table": table, "free": torch.where(ok, stack, free),
            "n_free": torch.where(ok, avail - total, n0).int(), "status": bits.int().reshape(1)}


def _gather(cache, table, descale):
    """[T, keys, Hk, d] fp32 of the pages that the table names."""
    kind = torch.uint8 if cache.dtype == torch.float8_e4m3fn else cache.dtype
    x = cache.view(kind)[table.long().clamp(min=0)].view(cache.dtype).float().flatten(1, 2)
    return x if descale is None else x * descale[:, None]


def _decode(s):
    T, Hq, d = s["q"].shape
    Hk = s["kc"].shape[2]
    q = s["q"].float().view(T, Hk, Hq // Hk, d)
    k = _gather(s["kc"], s["table"], s["kd"]).permute(0, 2, 3, 1)
    sc = (q @ k) * d ** -0.5
    del k
    n = sc.shape[-1]
    seen = (torch.arange(n, device=DEV)[None] < s["lens"][:, None])[:, None, None]
    sc = torch.where(seen, sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    v = _gather(s["vc"], s["table"], s["vd"]).permute(0, 2, 1, 3)
    o = (p @ v) / torch.where(l > 0, l, 1.0)
    return {"o": o.view(T, Hq, d).bfloat16(), "lse": (m + torch.log(l)).view(T, Hq)}


def run(s):
    op, c = s["op"], s["c"]
    if own:
        from io_aware_exact_22_b200 import fa
        if op == "rope":
            q, k = fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["rope"], positions=s["pos"], eps=EPS,
                                   interleaved=c["inter"], q_out=s["q_out"], k_out=s["k_out"])
            return {"q": q, "k": k}
        if op == "rope_bwd":
            dq, dk, dwq, dwk = fa.qk_norm_rope_backward(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["rope"],
                                                        positions=s["pos"], eps=EPS, interleaved=c["inter"])
            return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
        if op == "append":
            q = fa.paged_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["rope"], s["pos"], s["slots"], s["kc"],
                                s["vc"], eps=EPS, interleaved=c["inter"], k_descale=s["kd"], v_descale=s["vd"],
                                q_out=s["q_out"])
            return {"q": q, "k": s["kc"], "v": s["vc"]}
        if op == "plan":
            fa.paged_plan(s["cached"], s["new"], s["table"], s["free"], s["n_free"], c["ps"], s["lens"], s["cu"],
                          s["slots"], s["pos"], s["req"], s["n_free_out"], s["status"])
            return {"lens": s["lens"], "cu": s["cu"], "slots": s["slots"], "pos": s["pos"], "req": s["req"],
                    "table": s["table"], "free": s["free"], "n_free": s["n_free_out"], "status": s["status"]}
        o, lse = fa.paged_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], k_descale=s["kd"], v_descale=s["vd"],
                                 out=s["out"], lse=s["lse"])
        return {"o": o, "lse": lse}
    if op == "rope":
        pos = _positions(s)
        return {n: _norm_rope(s[n], s["w" + n], s["rope"], pos, c["inter"]).transpose(1, 2).bfloat16().contiguous()
                for n in ("q", "k")}
    if op == "rope_bwd":
        pos = _positions(s)
        dq, dwq = _norm_rope_bwd(s["gq"], s["q"], s["wq"], s["rope"], pos, c["inter"])
        dk, dwk = _norm_rope_bwd(s["gk"], s["k"], s["wk"], s["rope"], pos, c["inter"])
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if op == "append":
        q = _norm_rope(s["q"], s["wq"], s["rope"], s["pos"], c["inter"]).bfloat16()
        q = torch.where((s["slots"] < 0)[:, None, None], s["q_out"], q)
        k = _norm_rope(s["k"], s["wk"], s["rope"], s["pos"], c["inter"])
        return {"q": q, "k": _store(s["kc"], s["slots"], k, s["kd"]),
                "v": _store(s["vc"], s["slots"], s["v"].float(), s["vd"])}
    if op == "plan":
        return _plan(s)
    return _decode(s)


def work(case):
    c, op = case, case["op"]
    if op in ("rope", "rope_bwd"):
        rows = c["B"] * c["N"] * (c["Hq"] + c["Hk"])
        table = 4 * c["rot"] * c["N"] + (4 * c["B"] * c["N"] if c["pos"] else 0)
        return {"bytes": (4 if op == "rope" else 6) * rows * c["d"] + table,
                "flops": (10 if op == "rope" else 22) * rows * c["d"]}
    if op == "append":
        T, Hq, Hk, d = c["T"], c["Hq"], c["Hk"], c["d"]
        return {"bytes": 2 * T * (Hq + 2 * Hk) * d + 2 * T * Hq * d + (1 if c["fp8"] else 2) * 2 * T * Hk * d
                + T * (4 * c["rot"] + 12), "flops": 10 * T * (Hq + 2 * Hk) * d}
    if op == "plan":
        cached, new = _plan_lens(c)
        ps = c["ps"]
        used = (cached + ps - 1) // ps
        want = np.where(new < 0, 0, (cached + np.maximum(new, 0) + ps - 1) // ps - used)
        back = np.where(new < 0, used, 0)
        t = int(np.maximum(new, 0).sum())
        return {"bytes": 16 * (t + c["R"] // 8) + 16 * c["R"] + 8 * int(want.sum()) + 8 * int(back.sum()), "flops": 0}
    n = sum(_lens(c))
    b = 1 if c["fp8"] else 2
    return {"bytes": 2 * b * n * c["Hk"] * c["d"] + 4 * (n // c["ps"]) + c["T"] * c["Hq"] * (4 * c["d"] + 4),
            "flops": 4 * n * c["Hq"] * c["d"]}


# ------------------------------------------------------------------ from the definition, in 64 bits
def _rows64(x, w, cos, sin, pairs):
    """Norm and rotation of rows x [rows, heads, d] fp64; cos, sin [rows, rot/2]; pairs: two index
    lists (a, b) of the rotated elements.  Written with a rotation matrix applied to the pairs."""
    y = x / torch.sqrt(torch.mean(x ** 2, dim=2, keepdim=True) + EPS) * w
    if cos is None:
        return y
    a, b = pairs
    out = y.clone()
    turn = torch.stack([torch.stack([cos, -sin], -1), torch.stack([sin, cos], -1)], -2)  # [rows, rot/2, 2, 2]
    both = torch.stack([y[:, :, a], y[:, :, b]], -1)  # [rows, heads, rot/2, 2]
    both = (turn[:, None] * both[..., None, :]).sum(-1)
    out[:, :, a], out[:, :, b] = both[..., 0], both[..., 1]
    return out


def _pairs64(rot, inter):
    i = torch.arange(rot // 2, device=DEV)
    return (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op in ("rope", "rope_bwd"):
        B, N = c["B"], c["N"]
        pos = (s["pos"].long() if s["pos"] is not None else torch.arange(N, device=DEV).repeat(B, 1)).reshape(-1)
        t = None if s["rope"] is None else s["rope"].double()[pos]
        cos, sin = (None, None) if t is None else (t[:, 0], t[:, 1])
        pairs = _pairs64(c["rot"], c["inter"])
        out = {}
        for n in ("q", "k"):
            x = s[n].double().reshape(B * N, -1, c["d"])
            w = s["w" + n].double()
            if op == "rope":
                y = _rows64(x, w, cos, sin, pairs)
                out[n] = y.view(B, N, -1, c["d"]).permute(0, 2, 1, 3).contiguous()
            else:  # the forward's gradient by differentiation
                go = s["g" + n].double().permute(0, 2, 1, 3).reshape(B * N, -1, c["d"])
                dw = torch.zeros(c["d"], device=DEV, dtype=torch.float64)
                dx = torch.empty_like(x)
                for r in range(0, B * N, 4096):
                    e = slice(r, r + 4096)
                    xr, wr = x[e].clone().requires_grad_(), w.clone().requires_grad_()
                    y = _rows64(xr, wr, None if cos is None else cos[e], None if sin is None else sin[e], pairs)
                    dx[e], part = torch.autograd.grad(y, (xr, wr), go[e])
                    dw += part
                out["d" + n], out["dw" + n] = dx.view(B, N, -1, c["d"]), dw
        return out
    if op == "append":
        T, n = c["T"], c["T"] + c["pad"]
        t = s["rope"].double()[s["pos"].long()]
        pairs = _pairs64(c["rot"], c["inter"])
        q = _rows64(s["q"].double(), s["wq"].double(), t[:, 0], t[:, 1], pairs)
        k = _rows64(s["k"].double(), s["wk"].double(), t[:, 0], t[:, 1], pairs)
        q[T:] = s["q_out"][T:].double()
        out = {"q": q}
        for name, x in (("k", k), ("v", s["v"].double())):
            cache = s[name + "c"].float().double().view(-1, c["Hk"], c["d"])
            x = x[:T] if not c["fp8"] else (x[:T] / s[name + "d"].double()[None, :, None]).clamp(-448, 448)
            cache[s["slots"][:T]] = x
            out[name] = cache.view(s[name + "c"].shape)
        return out
    if op == "plan":
        return None
    T, Hq, d = s["q"].shape
    Hk, ps = c["Hk"], c["ps"]
    o = torch.zeros(T, Hq, d, device=DEV, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, device=DEV, dtype=torch.float64)
    for t in range(T):
        n = int(s["lens"][t])
        if n == 0:
            continue
        j = torch.arange(n, device=DEV)
        page, at = s["table"][t].long()[j // ps], j % ps
        for h in range(Hk):
            kind = torch.uint8 if c["fp8"] else torch.bfloat16
            k, v = (x[:, :, h].view(kind)[page, at].view(x.dtype).double() for x in (s["kc"], s["vc"]))
            if c["fp8"]:
                k, v = k * s["kd"][h].double(), v * s["vd"][h].double()
            for r in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
                x = (k * s["q"][t, r].double()).sum(1) / math.sqrt(d)
                lse[t, r] = torch.logsumexp(x, 0)
                o[t, r] = (torch.exp(x - lse[t, r])[:, None] * v).sum(0)
    return {"o": o, "lse": lse}
