"""Norm + rotation at sizes where a run of lanes takes several heads and several units, against fp64 on the GPU: the
rings in shared memory wrap and are filled again, a unit goes from q's heads to k's and v's, the last unit of a
token is a short one, and a warp of the backward goes from unit to unit.  (Heads per unit, units per warp:
in the cases' comments.)

Tolerances as in test_norm_rope.py: 2^-20 of |y_a| + |y_b| forward, 2^-19 of the terms' magnitudes backward,
half a bf16 step; dw: a lane adds its rows one after another, at most twice the mean over the 592 x 4 warps'
rows and a unit of 35 heads, then 64 sums at most.
"""
import pytest
import torch

from io_aware_exact_22_b200 import fa

OK, DEVICE_CHECK = 0, 5
EPS = 1e-5
U = 2.0 ** -24


def _turn(y, rope, pos, inter, back=False, size=False):
    """y [n, heads, d] fp64 turned by the angles of pos [n]; size: the sum of the terms' magnitudes."""
    if rope is None:
        return y.abs() if size else y
    half = rope.shape[2]
    t = rope.double()[pos.long()]
    c, s = t[:, None, 0], (-t[:, None, 1] if back else t[:, None, 1])
    i = torch.arange(half, device=y.device)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
    out = y.clone()
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    if size:
        out = y.abs()
        out[..., a] = out[..., b] = y[..., a].abs() + y[..., b].abs()
    return out


def _inputs(tokens, heads, d, rot, seed, bad):
    """Rows of a fused projection [tokens, heads, d], weights, table, positions; `bad`: the tokens whose position
    lies outside the table."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, heads, d, generator=g, device="cuda").bfloat16()
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16() for _ in range(2))
    rope = fa.rope_table(3000, rot) if rot else None
    pos = torch.randint(0, 3000, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    for i, n in enumerate(bad):
        pos[n] = -1 if i % 2 else 3000
    return x, wq, wk, rope, pos


def _check_rows(got, x, w, rope, pos, inter):
    """got [n, heads, d]: norm + rotation of x's rows, in chunks."""
    for n in range(0, x.shape[0], 2048):
        y = x[n:n + 2048].double()
        y = y / (y.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
        p = pos[n:n + 2048]
        want = _turn(y, rope, p, inter)
        lim = 2.0 ** -8 * want.abs() + 2.0 ** -20 * _turn(y, rope, p, inter, size=True)
        assert ((got[n:n + 2048].double() - want).abs() <= lim).all(), n


def _good(tokens, bad):
    keep = torch.ones(tokens, dtype=torch.bool, device="cuda")
    keep[list(bad)] = False
    return keep


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,inter", [
    (4, 1024, 16, 16, 64, 64, False),    # 8 heads per unit, 4 units per token
    (1, 4100, 24, 7, 128, 64, True),     # 16, then 15: from q to k inside the second
    (2, 9001, 32, 5, 64, 48, False),     # all 37, one wave
    (1, 16384, 32, 32, 128, 128, False),  # 16, many waves
    (2, 1025, 41, 9, 128, 0, False)])    # 13, the last of four units 11
def test_forward(cuda_ok, B, N, Hq, Hk, d, rot, inter):
    bad = (5, B * N - 3) if rot else ()
    x, wq, wk, rope, pos = _inputs(B * N, Hq + 2 * Hk, d, rot, N, bad)
    x4 = x.view(B, N, -1, d)
    qo, ko = (torch.full((B, H, N, d), 9.0, device="cuda", dtype=torch.bfloat16) for H in (Hq, Hk))
    fa.qk_norm_rope(x4[:, :, :Hq], x4[:, :, Hq:Hq + Hk], wq, wk, rope, pos.view(B, N) if rot else None, eps=EPS,
                    interleaved=inter, q_out=qo, k_out=ko)
    assert fa.fa_get_device_status() == (DEVICE_CHECK if bad else OK)
    keep = _good(B * N, bad)
    for out, rows, w in ((qo, x[:, :Hq], wq), (ko, x[:, Hq:Hq + Hk], wk)):
        out = out.transpose(1, 2).reshape(B * N, -1, d)
        assert (out[~keep] == 9).all()
        _check_rows(out[keep], rows[keep], w, rope, pos[keep], inter)


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,inter", [
    (2, 4096, 16, 16, 128, 128, False),  # 16 heads per unit, two units per warp
    (1, 8191, 32, 5, 128, 64, True),     # 32 and 5; two and five units
    (3, 5001, 13, 1, 64, 48, False),     # 13 and 1; one and four
    (1, 20001, 35, 5, 64, 64, False),    # 12 (a token's last unit 11) and 5; four and seven
    (1, 16383, 35, 5, 128, 0, False)])   # the same; seven and eleven
def test_backward(cuda_ok, B, N, Hq, Hk, d, rot, inter):
    T = B * N
    bad = (7, T - 2) if rot else ()
    x, wq, wk, rope, pos = _inputs(T, Hq + 2 * Hk, d, rot, N + 1, bad)
    x4 = x.view(B, N, -1, d)
    gen = torch.Generator(device="cuda").manual_seed(N)
    gq, gk = (torch.randn(B, H, N, d, generator=gen, device="cuda").bfloat16() for H in (Hq, Hk))
    dx = torch.full((B, N, Hq + Hk + 1, d), 7.0, device="cuda", dtype=torch.bfloat16)
    args = (gq, gk, x4[:, :, :Hq], x4[:, :, Hq:Hq + Hk], wq, wk, rope, pos.view(B, N) if rot else None)
    _, _, dwq, dwk = fa.qk_norm_rope_backward(*args, eps=EPS, interleaved=inter, dq=dx[:, :, :Hq], dk=dx[:, :, Hq:Hq + Hk])
    assert fa.fa_get_device_status() == (DEVICE_CHECK if bad else OK)
    keep = _good(T, bad)
    dx = dx.view(T, -1, d)
    assert (dx[:, -1] == 7).all() and (dx[~keep] == 7).all()
    depth = 2 * T * (Hq + Hk) / (592 * 4 * (512 // d)) + 35 + 64
    for rows, g, w, got, dw in ((x[:, :Hq], gq, wq, dx[:, :Hq], dwq), (x[:, Hq:Hq + Hk], gk, wk, dx[:, Hq:Hq + Hk], dwk)):
        g = g.transpose(1, 2).reshape(T, -1, d)[keep]
        rows, got, p = rows[keep], got[keep], pos[keep]
        total, size_dw = torch.zeros(2, d, device="cuda", dtype=torch.float64)
        for n in range(0, rows.shape[0], 2048):
            y, go, e = rows[n:n + 2048].double(), g[n:n + 2048].double(), p[n:n + 2048]
            r = 1 / (y.square().mean(-1, keepdim=True) + EPS).sqrt()
            xh, wd = y * r, w.double()
            dy, size_dy = _turn(go, rope, e, inter, back=True), _turn(go, rope, e, inter, back=True, size=True)
            want = r * (dy * wd - xh * (dy * wd * xh).mean(-1, keepdim=True))
            size = r * (size_dy * wd.abs() + xh.abs() * (size_dy * wd.abs() * xh.abs()).mean(-1, keepdim=True))
            assert ((got[n:n + 2048].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * size).all(), n
            total += (dy * xh).sum((0, 1))
            size_dw += (size_dy * xh.abs()).sum((0, 1))
        assert ((dw.double() - total).abs() <= (depth * U + 2.0 ** -20) * size_dw).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter,fp8,heads_outer", [
    (4100, 32, 4, 128, 128, False, False, True),  # 20 heads per unit: from q to k to v in the second
    (4100, 32, 4, 128, 128, False, True, False),
    (4100, 31, 4, 128, 64, True, True, True),     # 20, then 19
    (9000, 20, 20, 64, 64, True, False, False),   # 30: from q to k in the first, from k to v in the second
    (9000, 20, 20, 64, 32, False, True, True)])
def test_append(cuda_ok, T, Hq, Hk, d, rot, inter, fp8, heads_outer):
    bad = (11, T - 4)
    x, wq, wk, rope, pos = _inputs(T, Hq + 2 * Hk, d, rot, T, bad)
    ps = 16
    pages = T // ps + 9
    g = torch.Generator(device="cuda").manual_seed(1)
    slots = torch.randperm(pages * ps, generator=g, device="cuda")[:T].contiguous()
    skipped = torch.rand(T, generator=g, device="cuda") < 0.05
    skipped[list(bad)] = False
    slots[skipped] = -1
    kind, fill = (torch.float8_e4m3fn, 0x31) if fp8 else (torch.bfloat16, 3.0)
    as_bits = (lambda c: c.view(torch.uint8)) if fp8 else (lambda c: c)
    kc, vc = (torch.empty(pages, Hk, ps, d, dtype=kind, device="cuda").transpose(1, 2) if heads_outer else
              torch.empty(pages, ps, Hk, d, dtype=kind, device="cuda") for _ in range(2))
    as_bits(kc).fill_(fill)
    as_bits(vc).fill_(fill)
    kd, vd = (0.01 + 0.02 * torch.rand(2, Hk, generator=g, device="cuda")) if fp8 else (None, None)
    qo = torch.full((T, Hq, d), 9.0, device="cuda", dtype=torch.bfloat16)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    fa.paged_append(q, k, v, wq, wk, rope, pos, slots, kc, vc, eps=EPS, interleaved=inter, k_descale=kd, v_descale=vd,
                    q_out=qo)
    assert fa.fa_get_device_status() == DEVICE_CHECK
    keep = _good(T, bad) & ~skipped
    assert (qo[~keep] == 9).all()
    _check_rows(qo[keep], q[keep], wq, rope, pos[keep], inter)
    at = slots[keep]
    gk, gv = as_bits(kc)[at // ps, at % ps], as_bits(vc)[at // ps, at % ps]
    if fp8:
        y = k[keep].double()
        y = y / (y.square().mean(-1, keepdim=True) + EPS).sqrt() * wk.double()
        f = kd.double()[:, None]
        want, size = _turn(y, rope, pos[keep], inter) / f, _turn(y, rope, pos[keep], inter, size=True) / f
        want = want.clamp(-448, 448)
        lim = (2.0 ** -4 * want.abs()).clamp(min=2.0 ** -10) + 2.0 ** -20 * size
        assert ((gk.view(kind).double() - want).abs() <= lim).all()
        code = (v[keep].float() / vd[:, None]).clamp(-448, 448).to(kind)
        assert torch.equal(gv, code.view(torch.uint8))
    else:
        _check_rows(gk, k[keep], wk, rope, pos[keep], inter)
        assert torch.equal(gv, v[keep])
    rest = torch.ones(pages * ps, dtype=torch.bool, device="cuda")
    rest[at] = False
    rest = rest.nonzero()[:, 0]
    for c in (kc, vc):  # other slots are as they were
        assert (as_bits(c)[rest // ps, rest % ps] == fill).all()


def test_workspace_size_does_not_shrink_as_the_problem_grows():
    n = fa.fa_qk_norm_rope_bwd_workspace_bytes
    for d in (64, 128):
        for Hq, Hk in ((1, 0), (16, 16), (32, 8), (35, 5)):
            sizes = [n(1, N, Hq, Hk, d) for N in (1, 5, 100, 1000, 2368, 2372, 4096, 4100, 16384, 100000)]
            assert sizes == sorted(sizes) and sizes[0] > 0
    assert n(1, 2368, 16, 16, 128) <= n(2, 4096, 16, 16, 128) and n(1, 100, 8, 2, 64) <= n(1, 100, 32, 8, 64)


@pytest.mark.gpu
def test_one_workspace_serves_shorter_sequences(cuda_ok):
    # sized for the longest of them, handed to all
    H, d = 16, 128
    ws = torch.full((fa.fa_qk_norm_rope_bwd_workspace_bytes(1, 2372, H, H, d),), 0xff, dtype=torch.uint8, device="cuda")
    for N in (2372, 2368, 700, 1):
        q, k, gq, gk = (torch.randn(*s, d, device="cuda").bfloat16() for s in ((1, N, H), (1, N, H), (1, H, N), (1, H, N)))
        want = fa.qk_norm_rope_backward(gq, gk, q, k, None, None, None)
        got = fa.qk_norm_rope_backward(gq, gk, q, k, None, None, None, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
