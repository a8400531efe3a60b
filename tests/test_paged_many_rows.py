"""Decode with more (row, kv heads) groups than CTAs, against fp64 on the GPU.  The kernel then keeps one header of a
divided group per CTA, and the join has a block for each; with fewer groups (tests/test_paged.py) a header
and a block belong to each group.

Tolerance as in test_paged.py: E = 4 d u A + 4 n u, and 2^-20 for the exponential and P's terms.
"""
import math

import pytest
import torch

from io_aware_exact_22_b200 import fa

OK = 0
U = 2.0 ** -24


def _problem(lens, ps, Hk, d, fp8, seed):
    """Caches with the rows' pages in random order and NaN in what no key uses, block table, fp64 keys and values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    pages = torch.randperm(sum(need) + 3, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(1, *need)), -1, dtype=torch.int32, device="cuda")
    free = torch.ones(len(pages) * ps, dtype=torch.bool, device="cuda")
    at = 0
    for t, n in enumerate(lens):
        mine = pages[at:at + need[t]]
        at += need[t]
        table[t, :need[t]] = mine
        slots = (mine.long()[:, None] * ps + torch.arange(ps, device="cuda")).flatten()
        free[slots[:n]] = False
    out = []
    for _ in range(2):
        c = torch.randn(len(pages) * ps, Hk, d, generator=g, device="cuda")
        c = (64 * c).clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else c.bfloat16()
        if fp8:
            c.view(torch.uint8)[free] = 0x7f
        else:
            c[free] = math.nan
        out.append(c.view(len(pages), ps, Hk, d))
    return out[0], out[1], table


def _check(q, kc, vc, table, lens, req, o, lse, scale, kd, vd):
    T, Hq, d = q.shape
    ps, Hk = kc.shape[1], kc.shape[2]
    for t in range(T):
        r, n = req[t], lens[t]
        if r < 0:
            assert (o[t] == 9).all() and (lse[t] == 9).all(), t
            continue
        if n == 0:
            assert (o[t] == 0).all() and (lse[t] == -math.inf).all(), t
            continue
        j = torch.arange(n, device="cuda")
        page = table[r].long()[j // ps]
        k, v = (c.view(torch.uint8)[page, j % ps].view(c.dtype).double() if kd is not None else c[page, j % ps].double()
                for c in (kc, vc))
        if kd is not None:
            k, v = k * kd.double()[:, None], v * vd.double()[:, None]
        x = q[t].double().view(Hk, Hq // Hk, d)
        s = torch.einsum("hgd,nhd->hgn", x, k) * scale
        A = (torch.einsum("hgd,nhd->hgn", x.abs(), k.abs()) * scale).amax(-1, keepdim=True)
        want_l = torch.logsumexp(s, -1, keepdim=True)
        p = torch.exp(s - want_l)
        want, mag = torch.einsum("hgn,nhd->hgd", p, v), torch.einsum("hgn,nhd->hgd", p, v.abs())
        E = 4 * d * U * A + 2.0 ** -20 + 4 * n * U
        assert ((o[t].double().view_as(want) - want).abs() <= 2.0 ** -8 * want.abs() + E * mag).all(), t
        assert ((lse[t].double().view_as(want_l) - want_l).abs() <= E + 2.0 ** -22 * want_l.abs()).all(), t


def _ragged(rng, T):  # 0 to 300 keys, every seventh row without a key
    return [0 if t % 7 == 3 else n for t, n in enumerate(torch.randint(1, 301, (T,), generator=rng).tolist())]


def _one_long(rng, T):
    lens = torch.randint(0, 25, (T,), generator=rng).tolist()
    lens[T // 2] = 60011
    return lens


def _few(rng, T):  # fewer tiles than CTAs
    return [n if t % 100 == 50 else 0 for t, n in enumerate(torch.randint(1, 90, (T,), generator=rng).tolist())]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape,T,Hq,Hk,ps", [
    (_ragged, 300, 16, 8, 16), (_ragged, 300, 24, 1, 20), (_ragged, 130, 66, 22, 1), (_one_long, 300, 8, 8, 64),
    (_one_long, 250, 48, 2, 16), (_few, 1500, 16, 8, 32), (_few, 700, 20, 1, 16)])
def test_more_groups_than_ctas(cuda_ok, shape, T, Hq, Hk, ps, d, fp8):
    rng = torch.Generator().manual_seed(T + Hq)
    lens = shape(rng, T)
    kc, vc, table = _problem(lens, ps, Hk, d, fp8, T)
    # the kernel reads kv heads of less than 256 bytes side by side and runs 3 CTAs per SM at most
    side = max(h for h in (1, 2, 4) if h * d * (1 if fp8 else 2) <= 256 and Hk % h == 0)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert T * (Hk // side) * (-(-(Hq // Hk) // 16)) > 3 * sms
    req = [-1 if t % 11 == 5 and t != T // 2 else t for t in range(T)]
    req[0], lens[0] = T // 2, min(lens[0], lens[T // 2])  # two rows of one request
    q = torch.randn(T, Hq, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    kd, vd = (0.01 + 0.02 * torch.rand(2, Hk, generator=torch.Generator().manual_seed(2)).cuda()) if fp8 else (None, None)
    nbytes = fa.fa_paged_decode_workspace_bytes(T, Hq, Hk, d)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    first = None
    for fill in ("zeros", "headers", "ones"):
        ws = torch.full((nbytes,), 0xff if fill == "ones" else 0, dtype=torch.uint8, device="cuda")
        if fill == "headers":  # what an earlier call may have left: (row, group, first and last CTA)
            ws.view(torch.int32)[:4 * 3 * sms] = ints([[t % T, 0, t, min(t + 1, 3 * sms - 1)] for t in range(3 * sms)]).flatten()
        o = torch.full((T, Hq, d), 9.0, device="cuda", dtype=torch.bfloat16)
        lse = torch.full((T, Hq), 9.0, device="cuda")
        fa.paged_decode(q, kc, vc, table, ints(lens), req=ints(req), k_descale=kd, v_descale=vd, out=o, lse=lse, workspace=ws)
        assert fa.fa_get_device_status() == OK
        if first is None:
            first = o, lse
            _check(q, kc, vc, table, lens, req, o, lse, d ** -0.5, kd, vd)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
