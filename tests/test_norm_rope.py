"""Norm + rotation of queries and keys (fa_qk_norm_rope, fa_qk_norm_rope_bwd) against fp64.

Tolerances.  u = 2^-24.  The squares' sum is 8 products in a lane and 4 levels over lanes: relative
error below 13 u, half of it in r; rsqrtf adds 2 ulp (4 u), x r w two roundings, the rotation two
more of the sum of its terms' magnitudes: below 2^-20 (16 u) of |y_a| + |y_b|.  The bf16 store moves
a value by at most half a step, 2^-8 of it.  The backward's chain is twice as long (the rotation,
the weight, the mean over the row, the last difference): 2^-19 of its terms' magnitudes.  dw is an
fp32 sum: (depth of the longest chain of additions) u + 2^-20 of the sum of the terms' magnitudes.
"""
import math

import numpy as np
import pytest
import torch

from io_aware_exact_22_b200 import fa
from oracle import paged_ref as ref
from tests._helpers import f64

OK, INVALID, UNSUPPORTED = 0, 1, 2
A16 = 0x10000  # fake, aligned, never dereferenced
U = 2.0 ** -24


# ------------------------------------------------------------------ the oracle
def test_oracle_rotation_keeps_pair_norms_and_composes():
    rng = np.random.default_rng(0)
    y = rng.standard_normal((5, 3, 64))
    rope = ref.rope_table(20, 32)
    for inter in (False, True):
        pos = np.array([0, 3, 5, 7, 9])
        z = ref.rotate(y, rope, pos, inter)
        a, b = ref.rotated_pairs(32, inter)
        assert np.allclose(z[..., a] ** 2 + z[..., b] ** 2, y[..., a] ** 2 + y[..., b] ** 2)
        assert np.array_equal(z[0], y[0]) and np.array_equal(z[..., 32:], y[..., 32:])
        assert np.allclose(ref.rotate(z, rope, pos, inter, back=True), y)
        assert np.allclose(ref.rotate(ref.rotate(y, rope, pos, inter), rope, pos, inter), ref.rotate(y, rope, 2 * pos, inter))
    # scores depend on the distance alone
    q, k = rng.standard_normal((2, 1, 1, 64))
    at = lambda x, p: ref.rotate(x, rope, np.array([p]), False)[0, 0]  # noqa: E731
    assert math.isclose(at(q, 9) @ at(k, 4), at(q, 15) @ at(k, 10), rel_tol=1e-9)


@pytest.mark.parametrize("inter", [False, True])
def test_oracle_gradient_against_autograd_and_differences(inter):
    rng = np.random.default_rng(1)
    x, g, w = rng.standard_normal((4, 2, 16)), rng.standard_normal((4, 2, 16)), rng.standard_normal(16)
    rope, pos = ref.rope_table(9, 16), np.array([0, 8, 2, 2])
    dx, dw = ref.norm_rope_backward(g, x, w, rope, pos, inter, 1e-3)
    f = lambda x, w: (g * ref.norm_rope(x, w, rope, pos, inter, 1e-3)).sum()  # noqa: E731
    h = 1e-6
    for i in [(0, 0, 0), (1, 1, 7), (3, 0, 15)]:
        e = np.zeros_like(x)
        e[i] = h
        assert math.isclose((f(x + e, w) - f(x - e, w)) / (2 * h), dx[i], rel_tol=1e-6, abs_tol=1e-8)
    for i in (0, 9):
        e = np.zeros_like(w)
        e[i] = h
        assert math.isclose((f(x, w + e) - f(x, w - e)) / (2 * h), dw[i], rel_tol=1e-6, abs_tol=1e-8)
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = tx * torch.rsqrt((tx * tx).mean(-1, keepdim=True) + 1e-3) * tw
    t = torch.tensor(rope)[torch.tensor(pos)]
    a, b = (torch.tensor(n) for n in ref.rotated_pairs(16, inter))
    ya, yb = y[..., a], y[..., b]
    out = torch.empty_like(y)
    out[..., a] = ya * t[:, None, 0] - yb * t[:, None, 1]
    out[..., b] = yb * t[:, None, 0] + ya * t[:, None, 1]
    gx, gw = torch.autograd.grad((torch.tensor(g) * out).sum(), (tx, tw))
    assert np.allclose(gx.numpy(), dx) and np.allclose(gw.numpy(), dw)


def test_table_matches_the_oracle():
    t = fa.rope_table(50, 48, device="cpu")
    assert t.dtype is torch.float32 and t.shape == (50, 2, 24)
    assert np.abs(f64(t) - ref.rope_table(50, 48)).max() <= U


# ------------------------------------------------------------------ refusals
def _fwd(**kw):
    a = dict(q=A16, k=A16, wq=A16, wk=A16, rope=A16, rows=128, rot=64, inter=0, pos=None, pos_sb=0, qo=A16, ko=A16, B=1,
             N=128, Hq=2, Hk=1, d=64, qs=(8192, 128, 64), ks=(8192, 64, 64), eps=1e-6)
    a.update(kw)
    return fa.fa_qk_norm_rope(a["q"], a["k"], a["wq"], a["wk"], a["rope"], a["rows"], a["rot"], a["inter"], a["pos"],
                              a["pos_sb"], a["qo"], a["ko"], a["B"], a["N"], a["Hq"], a["Hk"], a["d"], a["qs"], a["ks"],
                              a["eps"], 0)


def _bwd(**kw):
    a = dict(gq=A16, gk=A16, q=A16, k=A16, wq=A16, wk=A16, rope=A16, rows=128, rot=64, inter=0, pos=None, pos_sb=0,
             dq=A16, dk=A16, dwq=A16, dwk=A16, ws=A16, wsb=1 << 40, B=1, N=128, Hq=2, Hk=1, d=64, qs=(8192, 128, 64),
             ks=(8192, 64, 64), dqs=(8192, 128, 64), dks=(8192, 64, 64), eps=1e-6)
    a.update(kw)
    return fa.fa_qk_norm_rope_bwd(a["gq"], a["gk"], a["q"], a["k"], a["wq"], a["wk"], a["rope"], a["rows"], a["rot"],
                                  a["inter"], a["pos"], a["pos_sb"], a["dq"], a["dk"], a["dwq"], a["dwk"], a["ws"],
                                  a["wsb"], a["B"], a["N"], a["Hq"], a["Hk"], a["d"], a["qs"], a["ks"], a["dqs"],
                                  a["dks"], a["eps"], 0)


REFUSALS = [
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(q=A16 + 8), INVALID), (dict(k=A16 + 2), INVALID),
    (dict(wq=A16 + 8), INVALID), (dict(rope=0), INVALID), (dict(rope=A16 + 4), INVALID), (dict(rows=0), INVALID),
    (dict(rows=127), INVALID), (dict(pos=A16 + 2), INVALID),
    (dict(rot=-16), INVALID), (dict(rot=80), INVALID), (dict(rot=8), UNSUPPORTED), (dict(rot=2), UNSUPPORTED),
    (dict(inter=2), INVALID), (dict(d=32, rot=0), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hk=-1), INVALID),
    (dict(qs=(8192, 128, 60)), INVALID), (dict(qs=(8192, 4, 64)), INVALID), (dict(B=2, ks=(8190, 64, 64)), INVALID),
    (dict(B=2, qs=(1 << 60, 128, 64)), INVALID), (dict(B=1 << 16, N=1 << 16), INVALID),
]


@pytest.mark.parametrize("kw,code", REFUSALS + [(dict(qo=0), INVALID), (dict(ko=A16 + 4), INVALID)])
def test_forward_refuses(kw, code):
    assert _fwd(**kw) == code


@pytest.mark.parametrize("kw,code", REFUSALS + [
    (dict(gq=0), INVALID), (dict(gk=A16 + 8), INVALID), (dict(dq=0), INVALID), (dict(dk=A16 + 2), INVALID),
    (dict(dwq=A16 + 2), INVALID), (dict(dqs=(8192, 128, 4)), INVALID), (dict(dks=(8192, 63, 64)), INVALID),
    (dict(ws=0), INVALID), (dict(ws=A16 + 16), INVALID), (dict(wsb=64), INVALID)])
def test_backward_refuses(kw, code):
    assert _bwd(**kw) == code


@pytest.mark.parametrize("kw", [dict(N=0), dict(B=0), dict(Hq=0, Hk=0)])
def test_empty_problem_is_a_no_op(kw):
    assert _fwd(**kw) == OK
    assert _bwd(dwq=0, dwk=0, **kw) == OK


def test_workspace_size():
    n = fa.fa_qk_norm_rope_bwd_workspace_bytes
    assert n(0, 5, 2, 1, 64) == n(1, 5, 0, 0, 64) == n(1, 5, 2, 1, 80) == n(1, -5, 2, 1, 64) == 0
    assert n(1, 5, 2, 1, 64) % (2 * 64 * 4) == 0
    assert 0 < n(1, 1, 1, 1, 128) <= n(4, 16384, 32, 8, 128) <= 148 * 4 * 2 * 128 * 4


def test_binding_refuses():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(x, x, None, None, None)  # not on the GPU


# ------------------------------------------------------------------ on the GPU
def _case(B, N, Hq, Hk, d, rot, fused, pos, seed, weights=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    if fused:
        x = rnd(B, N, Hq + 2 * Hk, d).cuda()
        q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    else:
        q, k = rnd(B, N, Hq, d).cuda(), rnd(B, N, Hk, d).cuda()
    wq, wk = ((rnd(d) * 0.2 + 1).cuda(), (rnd(d) * 0.2 + 1).cuda()) if weights else (None, None)
    rows = N + 7
    rope = fa.rope_table(rows, rot) if rot else None
    positions = None
    if pos == "batch":
        positions = torch.randint(0, rows, (B, N), generator=g, dtype=torch.int32).cuda()
    elif pos == "shared":
        positions = torch.randint(0, rows, (N,), generator=g, dtype=torch.int32).cuda()
    return q, k, wq, wk, rope, positions


def _pos(positions, B, N):
    if positions is None:
        return np.broadcast_to(np.arange(N), (B, N))
    return np.broadcast_to(positions.cpu().numpy(), (B, N))


def _abs_pair(y, rope, pos, inter):
    """|y_a| + |y_b| at both elements of each pair, |y| elsewhere."""
    if rope is None:
        return np.abs(y)
    out = np.abs(y)
    a, b = ref.rotated_pairs(2 * rope.shape[2], inter)
    out[..., a] = out[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out


def _w(w):
    return None if w is None else f64(w)


CASES = [  # B, N, Hq, Hk, d, rot, fused, pos, inter
    (1, 1, 1, 1, 64, 64, False, None, False), (1, 1, 1, 1, 128, 128, False, None, True),
    (2, 17, 3, 1, 128, 128, True, "batch", False), (2, 17, 3, 1, 128, 128, True, "batch", True),
    (3, 33, 8, 2, 64, 32, True, "shared", True), (1, 40, 5, 5, 64, 16, True, None, False),
    (1, 65, 7, 7, 128, 48, False, "batch", False), (2, 5, 64, 4, 128, 64, True, None, True),
    (1, 9, 4, 2, 64, 0, False, None, False), (1, 700, 3, 2, 64, 48, True, "batch", False),
    (1, 6, 4, 0, 128, 128, False, None, False), (1, 6, 0, 4, 128, 128, False, None, False),
    (1, 5000, 2, 1, 64, 64, True, None, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,fused,pos,inter", CASES)
def test_forward(cuda_ok, B, N, Hq, Hk, d, rot, fused, pos, inter):
    q, k, wq, wk, rope, positions = _case(B, N, Hq, Hk, d, rot, fused, pos, N)
    qo, ko = fa.qk_norm_rope(q, k, wq, wk, rope, positions, eps=1e-5, interleaved=inter)
    assert fa.fa_get_device_status() == OK
    table = None if rope is None else f64(rope)
    p = _pos(positions, B, N)
    for x, w, got in ((q, wq, qo), (k, wk, ko)):
        want = ref.norm_rope(f64(x), _w(w), table, p, inter, 1e-5)
        size = _abs_pair(ref.norm_rope(f64(x), _w(w), None, p, inter, 1e-5), table, p, inter)
        err = np.abs(f64(got).transpose(0, 2, 1, 3) - want)
        assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size).all()


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,fused,pos,inter", CASES)
def test_backward(cuda_ok, B, N, Hq, Hk, d, rot, fused, pos, inter):
    q, k, wq, wk, rope, positions = _case(B, N, Hq, Hk, d, rot, fused, pos, N + 1)
    g = torch.Generator().manual_seed(7)
    gq, gk = (torch.randn(B, H, N, d, generator=g).bfloat16().cuda() for H in (Hq, Hk))
    dx = torch.full((B, N, Hq + Hk + 1, d), 7.0, device="cuda", dtype=torch.bfloat16)  # views, and a column not theirs
    dq, dk = dx[:, :, :Hq], dx[:, :, Hq:Hq + Hk]
    got = fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, rope, positions, eps=1e-5, interleaved=inter, dq=dq, dk=dk)
    assert fa.fa_get_device_status() == OK
    assert (dx[:, :, -1] == 7).all()
    table = None if rope is None else f64(rope)
    p = _pos(positions, B, N)
    depth = (Hq + Hk) * math.ceil(B * N * (Hq + Hk) / 4736) + 64
    for x, go, w, gx, gw in ((q, gq, wq, got[0], got[2]), (k, gk, wk, got[1], got[3])):
        x, go = f64(x), f64(go).transpose(0, 2, 1, 3)
        want, dw = ref.norm_rope_backward(go, x, _w(w), table, p, inter, 1e-5)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
        size_dy = _abs_pair(go, table, p, inter)
        size_u = size_dy * np.abs(_w(w))
        size = r * (size_u + np.abs(x * r) * (size_u * np.abs(x * r)).mean(-1, keepdims=True))
        assert (np.abs(f64(gx) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size).all()
        terms = (size_dy * np.abs(x * r)).reshape(-1, d).sum(0)
        assert (np.abs(f64(gw) - dw) <= (depth * U + 2.0 ** -20) * terms).all()


@pytest.mark.gpu
def test_backward_against_differences_of_the_forward(cuda_ok):
    # <g, f(x + h v) - f(x - h v)> / 2h: f on the GPU against the formula at the same points (f's bf16
    # rounding moves each output by 2^-8 of its size, which the sum over 64 k elements with random
    # signs averages out: 5 sigma, sigma^2 = sum (g f 2^-8)^2 / 3 per evaluation, two of them, over
    # 2h), and at a small step the formula's against the GPU's <dx, v>
    q, k, wq, wk, rope, _ = _case(1, 256, 2, 2, 128, 128, False, None, 3)
    g = torch.Generator().manual_seed(11)
    gq = torch.randn(1, 2, 256, 128, generator=g).bfloat16().cuda()
    gk = torch.zeros_like(gq)
    v = torch.randn(q.shape, generator=g).cuda()
    dq = fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, rope)[0]
    h = 0.25
    up, down = (q.float() + h * v).bfloat16(), (q.float() - h * v).bfloat16()
    a, b = (fa.qk_norm_rope(x, k, wq, wk, rope)[0].double() for x in (up, down))
    table, p = f64(rope), np.arange(256)[None]
    fu, fd = (ref.norm_rope(f64(x), f64(wq), table, p, False, 1e-6).transpose(0, 2, 1, 3) for x in (up, down))
    gd = f64(gq)
    quotient = float((gq.double() * (a - b)).sum()) / (2 * h)
    sigma = math.sqrt(((gd * fu * 2.0 ** -8) ** 2 / 3).sum() + ((gd * fd * 2.0 ** -8) ** 2 / 3).sum()) / (2 * h)
    assert abs(quotient - (gd * (fu - fd)).sum() / (2 * h)) <= 5 * sigma
    h = 1e-4
    x = f64(q)
    vd = v.double().cpu().numpy()
    fu, fd = (ref.norm_rope(x + s * h * vd, f64(wq), table, p, False, 1e-6).transpose(0, 2, 1, 3) for s in (1, -1))
    exact = (gd * (fu - fd)).sum() / (2 * h)
    assert abs((f64(dq) * vd).sum() - exact) <= 5 * math.sqrt(((f64(dq) * vd * 2.0 ** -8) ** 2 / 3).sum()) + 1e-4


@pytest.mark.gpu
def test_without_weights_and_repeatable(cuda_ok):
    q, k, _, _, rope, positions = _case(2, 333, 4, 2, 64, 64, True, "batch", 5, weights=False)
    one = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    a, b = fa.qk_norm_rope(q, k, None, None, rope, positions), fa.qk_norm_rope(q, k, one, one, rope, positions)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    first = fa.qk_norm_rope_backward(a[0], a[1], q, k, None, None, rope, positions)
    for _ in range(3):
        again = fa.qk_norm_rope_backward(a[0], a[1], q, k, one, one, rope, positions)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.gpu
def test_position_outside_the_table_is_reported_and_skipped(cuda_ok):
    q, k, wq, wk, rope, _ = _case(1, 8, 2, 1, 64, 64, False, None, 5)
    positions = torch.tensor([0, 1, rope.shape[0], 3, -1, 5, 6, 7], dtype=torch.int32, device="cuda")
    qo = torch.full((1, 2, 8, 64), 9.0, device="cuda", dtype=torch.bfloat16)
    fa.qk_norm_rope(q, k, wq, wk, rope, positions, q_out=qo)
    assert fa.fa_get_device_status() == 5 and fa.fa_get_device_status() == OK
    good = [0, 1, 3, 5, 6, 7]
    want, _ = fa.qk_norm_rope(q, k, wq, wk, rope, positions.clamp(0, 8))
    assert torch.equal(qo[:, :, good], want[:, :, good]) and (qo[:, :, [2, 4]] == 9).all()
    gq, gk = qo * 0 + 1, torch.ones(1, 1, 8, 64, device="cuda", dtype=torch.bfloat16)
    dq = torch.full_like(q, 9.0)
    _, _, dwq, _ = fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, rope, positions, dq=dq)
    assert fa.fa_get_device_status() == 5
    assert (dq[:, [2, 4]] == 9).all()
    part = fa.qk_norm_rope_backward(gq[:, :, good].contiguous(), gk[:, :, good].contiguous(), q[:, good], k[:, good], wq, wk,
                                    rope, positions[good].contiguous())
    assert torch.equal(dq[:, good], part[0]) and (dwq - part[2]).abs().max() <= 1e-4
    assert fa.fa_get_device_status() == OK


@pytest.mark.gpu
def test_zero_rows_and_empty_problem(cuda_ok):
    x = torch.zeros(1, 4, 2, 128, device="cuda", dtype=torch.bfloat16)
    rope = fa.rope_table(4, 128)
    qo, ko = fa.qk_norm_rope(x, x, None, None, rope)
    assert (qo == 0).all() and (ko == 0).all()
    got = fa.qk_norm_rope_backward(qo + 1, ko + 1, x, x, None, None, rope)
    assert all(torch.isfinite(t.float()).all() for t in got)
    e = torch.empty(2, 0, 3, 64, device="cuda", dtype=torch.bfloat16)
    qo, ko = fa.qk_norm_rope(e, e, None, None, None)
    assert qo.shape == (2, 3, 0, 64)
    _, _, dwq, dwk = fa.qk_norm_rope_backward(qo, ko, e, e, None, None, None)
    torch.cuda.synchronize()
    assert (dwq == 0).all() and (dwk == 0).all()


@pytest.mark.gpu
def test_infinite_and_nan_rows_stay_in_their_rows(cuda_ok):
    q, k, wq, wk, rope, _ = _case(1, 16, 3, 2, 128, 64, True, None, 9)
    clean = fa.qk_norm_rope(q, k, wq, wk, rope)
    q2 = q.clone()
    q2[0, 3, 1, 5], q2[0, 7, 2, 0] = math.nan, math.inf
    qo, ko = fa.qk_norm_rope(q2, k, wq, wk, rope)
    hit = torch.zeros(1, 3, 16, dtype=torch.bool, device="cuda")
    hit[0, 1, 3] = hit[0, 2, 7] = True
    assert torch.equal(qo[~hit], clean[0][~hit]) and torch.equal(ko, clean[1])
    assert torch.isnan(qo[0, 1, 3]).all()
    g = torch.ones_like(qo)
    a = fa.qk_norm_rope_backward(g, torch.ones_like(ko), q, k, wq, wk, rope)
    b = fa.qk_norm_rope_backward(g, torch.ones_like(ko), q2, k, wq, wk, rope)
    keep = ~hit.transpose(1, 2)
    assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1], b[1]) and torch.equal(a[3], b[3])


@pytest.mark.gpu
def test_on_a_side_stream_and_captured(cuda_ok):
    q, k, wq, wk, rope, _ = _case(1, 100, 4, 2, 64, 64, False, None, 21)
    gq, gk = torch.randn(1, 4, 100, 64, device="cuda").bfloat16(), torch.randn(1, 2, 100, 64, device="cuda").bfloat16()
    want = fa.qk_norm_rope(q, k, wq, wk, rope) + fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, rope)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = fa.qk_norm_rope(q, k, wq, wk, rope) + fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, rope)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.qk_norm_rope(q, k, wq, wk, rope) + fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, rope)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    q2 = q.clone()
    q.copy_(torch.randn_like(q))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], fa.qk_norm_rope(q, k, wq, wk, rope)[0]) and not torch.equal(q, q2)


@pytest.mark.gpu
def test_training_step_through_attention(cuda_ok):
    # projection's output -> norm + rotation -> forward -> backward -> its gradient, against fp64
    # autograd of the whole chain.  The chain rounds q, k (2^-8), P and dS (2^-8) and dq, dk (2^-8): the
    # attention's own contract holds its gradients to rel-L2 1e-2, each rounding adds 2^-8 / sqrt(3)
    # of it in the root mean square, and the norm's gradient is a projection (it does not stretch
    # more than r |w|): 2e-2 in all.
    B, N, H, d = 1, 200, 2, 64
    q, k, wq, wk, rope, _ = _case(B, N, H, H, d, 64, False, None, 31)
    v, do = (torch.randn(B, H, N, d, generator=torch.Generator().manual_seed(s)).bfloat16().cuda() for s in (1, 2))
    qr, kr = fa.qk_norm_rope(q, k, wq, wk, rope)
    o, lse = fa.forward(qr, kr, v, True)
    gq, gk, _ = fa.backward(qr, kr, v, o, do, lse, True)
    got = fa.qk_norm_rope_backward(gq, gk, q, k, wq, wk, rope)
    leaves = [t.double().cpu().requires_grad_() for t in (q, k, wq, wk)]
    t = rope.double().cpu()

    def turn(x, w):
        y = (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w).transpose(1, 2)
        c, s = t[:N, 0], t[:N, 1]
        a, b = y[..., :32], y[..., 32:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    a, b = turn(leaves[0], leaves[2]), turn(leaves[1], leaves[3])
    sc = (a @ b.transpose(-1, -2)) * d ** -0.5
    sc = sc.masked_fill(~torch.ones(N, N, dtype=torch.bool).tril(), -math.inf)
    loss = (sc.softmax(-1) @ v.double().cpu() * do.double().cpu()).sum()
    for g, w in zip(got, torch.autograd.grad(loss, leaves)):
        assert np.linalg.norm(f64(g) - w.numpy()) <= 2e-2 * np.linalg.norm(w.numpy())
