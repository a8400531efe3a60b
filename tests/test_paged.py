"""The paged key/value cache: fa_paged_plan, fa_paged_append, fa_paged_decode against fp64.

Tolerances.  u = 2^-24.  Decode: a score is a sum of d products in fp32 (in the matrix unit, d / 16
steps): error below 2 d u of the sum of the products' magnitudes, A = max_j scale sum |q K_j|; the
base-2 exponential adds 2^-22 and the split of P into two bf16 terms leaves 2^-16 of it (one fp16
term with an E4M3 cache: 2^-11); P V over n keys is an fp32 sum of n terms and l one of n: 2 n u.  So
O is off by at most E sum_j p_j |v_j|, E = 2 (2 d u A) + 2^-15 (2^-11 + 2^-15) + 4 n u, and half a bf16
step, 2^-8 of it; LSE by E + 2^-22 |LSE|.  Append: as fa_qk_norm_rope (tests/test_norm_rope.py); an
E4M3 store moves a code's value by at most half a step, 2^-4 of it or 2^-10 (half of the smallest).
"""
import math

import numpy as np
import pytest
import torch

import oracle
from io_aware_exact_22_b200 import fa
from oracle import paged_ref as ref
from tests._helpers import f64

OK, INVALID, UNSUPPORTED, DEVICE_CHECK = 0, 1, 2, 5
A16 = 0x10000  # fake, aligned, never dereferenced
U = 2.0 ** -24


# ------------------------------------------------------------------ the oracle
def test_oracle_decode_is_the_last_row_of_causal_attention():
    rng = np.random.default_rng(0)
    n, d = 37, 64
    q, k, v = (rng.standard_normal((1, 1, n, d)) for _ in range(3))
    o, lse = oracle.attention_forward(q, k, v, 0.1, True)
    pages = rng.permutation(9)[:5]
    kc, vc = rng.standard_normal((2, 9, 8, 1, d))
    for j in range(n):
        kc[pages[j // 8], j % 8, 0], vc[pages[j // 8], j % 8, 0] = k[0, 0, j], v[0, 0, j]
    got, gl = ref.paged_decode(q[0, 0, -1][None, None], kc, vc, [list(pages)], [n], [0], 0.1)
    assert np.allclose(got[0, 0], o[0, 0, -1]) and np.allclose(gl[0, 0], lse[0, 0, -1])


def test_oracle_plan_small_by_hand():
    # page size 4, stack 5 7 9 (top 9): request 0 holds 3 tokens on page 2 and adds 3 (one page: the top),
    # request 1 ends and returns pages 1, 3, request 2 is new with 5 tokens (two pages)
    got = ref.plan([3, 8, 0], [3, -1, 5], [[2, -1, -1], [1, 3, -1], [-1, -1, -1]], [5, 7, 9], 4, 3, 10)
    assert got["status"] == 0 and got["free"] == [5, 7] and got["lens"] == [6, 0, 5] and got["cu"] == [0, 3, 3, 8]
    assert got["table"] == [[2, 3, -1], [1, 3, -1], [1, 9, -1]]
    assert got["slots"] == [11, 12, 13, 4, 5, 6, 7, 36, -1, -1]
    assert got["positions"] == [3, 4, 5, 0, 1, 2, 3, 4, 0, 0] and got["req"] == [0, 0, 0, 2, 2, 2, 2, 2, -1, -1]
    assert ref.plan([3], [6], [[2, -1]], [], 4, 2, 10)["status"] == 2 | 0
    assert ref.plan([3], [5], [[2, -1]], [], 4, 2, 4)["status"] == 1 | 4
    assert ref.plan([9], [5], [[2, -1]], [], 4, 2, 9)["status"] == 8


# ------------------------------------------------------------------ refusals
def _plan(**kw):
    a = dict(cached=A16, new=A16, table=A16, ts=8, cols=8, free=A16, pool=64, fc=A16, ps=16, R=4, most=16, lens=A16,
             cu=A16, slots=A16, pos=A16, req=A16, fco=A16, st=A16)
    a.update(kw)
    return fa.fa_paged_plan(a["cached"], a["new"], a["table"], a["ts"], a["cols"], a["free"], a["pool"], a["fc"], a["ps"],
                            a["R"], a["most"], a["lens"], a["cu"], a["slots"], a["pos"], a["req"], a["fco"], a["st"], 0)


@pytest.mark.parametrize("kw,code", [
    *((dict([(n, 0)]), INVALID) for n in ("cached", "new", "table", "free", "fc", "lens", "cu", "slots", "pos", "req",
                                          "fco", "st")),
    (dict(cached=A16 + 2), INVALID), (dict(slots=A16 + 4), INVALID), (dict(ps=0), INVALID), (dict(R=-1), INVALID),
    (dict(most=-1), INVALID), (dict(cols=-1), INVALID), (dict(pool=-1), INVALID), (dict(ts=7), INVALID),
    (dict(R=fa.PLAN_MAX_REQUESTS + 1), UNSUPPORTED), (dict(cols=1 << 20, ts=1 << 20, ps=1 << 12), INVALID),
    (dict(most=fa.PAGED_MAX_LEN + 1), INVALID), (dict(pool=fa.PAGED_MAX_LEN + 1), INVALID), (dict(cols=1, ts=1, ps=fa.PAGED_MAX_LEN + 1), INVALID)])
def test_plan_refuses(kw, code):
    assert _plan(**kw) == code


def _append(**kw):
    a = dict(q=A16, k=A16, v=A16, wq=A16, wk=A16, rope=A16, rows=128, rot=64, inter=0, pos=A16, slots=A16, qo=A16, kc=A16,
             vc=A16, fp8=0, kd=None, vd=None, pages=4, ps=16, T=8, Hq=4, Hk=2, d=64, qs=(256, 64), ks=(128, 64),
             vs=(128, 64), cs=(2048, 128, 64), eps=1e-6)
    a.update(kw)
    return fa.fa_paged_append(a["q"], a["k"], a["v"], a["wq"], a["wk"], a["rope"], a["rows"], a["rot"], a["inter"],
                              a["pos"], a["slots"], a["qo"], a["kc"], a["vc"], a["fp8"], a["kd"], a["vd"], a["pages"],
                              a["ps"], a["T"], a["Hq"], a["Hk"], a["d"], a["qs"], a["ks"], a["vs"], a["cs"], a["eps"], 0)


@pytest.mark.parametrize("kw,code", [
    *((dict([(n, 0)]), INVALID) for n in ("q", "k", "v", "rope", "pos", "slots", "qo", "kc", "vc", "rows", "pages", "ps")),
    (dict(kc=A16 + 8), INVALID), (dict(slots=A16 + 4), INVALID), (dict(fp8=2), INVALID), (dict(kd=A16), INVALID),
    (dict(fp8=1, vd=A16 + 2), INVALID), (dict(fp8=1, cs=(2048, 128, 72)), INVALID), (dict(cs=(2044, 128, 64)), INVALID), (dict(cs=(-2048, 128, 64)), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(rot=66), INVALID), (dict(T=-1), INVALID),
    (dict(qs=(255, 64)), INVALID), (dict(vs=(128, 4)), INVALID), (dict(eps=-1.0), INVALID), (dict(T=0), OK)])
def test_append_refuses(kw, code):
    assert _append(**kw) == code


def _dec(**kw):
    a = dict(q=A16, kc=A16, vc=A16, fp8=0, kd=None, vd=None, table=A16, ts=8, rows=8, cols=8, lens=A16, req=None, o=A16,
             lse=A16, ws=A16, wsb=1 << 40, pages=64, ps=16, T=8, Hq=4, Hk=2, d=64, qs=(256, 64), cs=(2048, 128, 64),
             scale=0.125)
    a.update(kw)
    return fa.fa_paged_decode(a["q"], a["kc"], a["vc"], a["fp8"], a["kd"], a["vd"], a["table"], a["ts"], a["rows"],
                              a["cols"], a["lens"], a["req"], a["o"], a["lse"], a["ws"], a["wsb"], a["pages"], a["ps"],
                              a["T"], a["Hq"], a["Hk"], a["d"], a["qs"], a["cs"], a["scale"], 0)


@pytest.mark.parametrize("kw,code", [
    *((dict([(n, 0)]), INVALID) for n in ("q", "kc", "vc", "table", "lens", "o", "lse", "ws", "pages", "ps", "Hk")),
    (dict(q=A16 + 8), INVALID), (dict(lse=A16 + 2), INVALID), (dict(lens=A16 + 1), INVALID), (dict(req=A16 + 2), INVALID),
    (dict(ws=A16 + 16), INVALID), (dict(wsb=1000), INVALID), (dict(Hq=3), INVALID), (dict(d=80), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(T=-1), INVALID),
    (dict(rows=7), INVALID), (dict(ts=7), INVALID), (dict(kd=A16), INVALID), (dict(fp8=3), INVALID),
    (dict(cs=(2048, 100, 64)), INVALID), (dict(cs=(2048, -128, 64)), INVALID), (dict(qs=(256, 63)), INVALID),
    (dict(cols=1 << 20, ts=1 << 20, ps=1 << 11), INVALID), (dict(T=0), OK), (dict(Hq=0), OK)])
def test_decode_refuses(kw, code):
    assert _dec(**kw) == code


def test_decode_workspace_does_not_grow_with_the_lengths():
    n = fa.fa_paged_decode_workspace_bytes
    assert n(0, 8, 8, 64) == n(4, 0, 0, 64) == n(4, 8, 8, 96) == 0
    assert 0 < n(1, 8, 8, 64) <= n(1, 8, 8, 128) == n(500, 64, 8, 128) < 16 << 20


# ------------------------------------------------------------------ plan on the GPU
def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _state(lens, ps, cols, spare, seed):
    """Block table (random pages, -1 elsewhere) and stack of the free pages."""
    rng = np.random.default_rng(seed)
    need = [-(-n // ps) for n in lens]
    pages = rng.permutation(sum(need) + spare).tolist()
    table = []
    for n in need:
        table.append([pages.pop() for _ in range(n)] + [-1] * (cols - n))
    return table, pages


def _run_plan(cached, new, table, free, ps, most, pool=None):
    R, cols = len(cached), len(table[0]) if table else 3
    pool = len(free) + sum(-(-max(c, 0) // ps) for c in cached) + 2 if pool is None else pool
    t = dict(cached=_ints(cached), new=_ints(new),
             table=_ints(table) if R else torch.empty(0, cols, dtype=torch.int32, device="cuda"),
             free=_ints(free + [-7] * (pool - len(free))), count=_ints([len(free)]))
    o = {n: torch.full((k,), -99, dtype=torch.int64 if n == "slots" else torch.int32, device="cuda")
         for n, k in (("lens", R), ("cu", R + 1), ("slots", most), ("positions", most), ("req", most), ("fco", 1), ("st", 1))}
    fa.paged_plan(t["cached"], t["new"], t["table"], t["free"], t["count"], ps, o["lens"], o["cu"], o["slots"],
                  o["positions"], o["req"], o["fco"], o["st"])
    return t, o


def _check_plan(cached, new, table, free, ps, most):
    cols = len(table[0]) if table else 3
    want = ref.plan(cached, new, table, free, ps, cols, most)
    t, o = _run_plan(cached, new, table, free, ps, most)
    assert o["st"].item() == want["status"]
    for n in ("lens", "cu", "slots", "positions", "req"):
        assert o[n].tolist() == want[n], n
    assert t["table"].tolist() == want["table"]
    n = o["fco"].item()
    assert n == len(want["free"]) and t["free"][:n].tolist() == want["free"]
    return want


@pytest.mark.gpu
@pytest.mark.parametrize("R,maxlen,chunk,gone,ps,extra", [
    (1, 0, 1, 0, 16, 0), (1, 40, 1, 0, 1, 3), (16, 300, 1, 0, 16, 0), (33, 90, 40, 5, 24, 7), (31, 500, 9, 2, 7, 1),
    (1023, 60, 3, 4, 16, 100), (1025, 60, 3, 4, 16, 100), (2500, 20, 2, 3, 4, 9), (70, 700, 700, 6, 64, 40),
    (3, 0, 30000, 0, 16, 5), (5, 10, 1, 1, 8, 4), (50, 20000, 2, 2, 1, 3), (fa.PLAN_MAX_REQUESTS, 3, 1, 3, 2, 0)])
def test_plan(cuda_ok, R, maxlen, chunk, gone, ps, extra):
    rng = np.random.default_rng(R + ps)
    cached = rng.integers(0, maxlen + 1, R).tolist()
    new = rng.integers(0, chunk + 1, R).tolist()
    for b in range(R):
        if gone and b % gone == gone - 1:
            new[b] = -1
    cols = max(1, -(-(maxlen + chunk) // ps))
    table, free = _state(cached, ps, cols, max(1, sum(max(n, 0) for n in new) // ps + R), R)
    want = _check_plan(cached, new, table, free, ps, sum(max(n, 0) for n in new) + extra)
    assert want["status"] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("cached,new,spare,most,status", [
    ([5, 16], [1, 1], 0, 8, fa.PLAN_NO_PAGES), ([5, 16], [1, 33], 9, 80, fa.PLAN_ROW_FULL),
    ([5, 16], [1, 20], 9, 20, fa.PLAN_TOO_MANY_TOKENS), ([5, 16], [1, 17], 0, 2, fa.PLAN_NO_PAGES | fa.PLAN_TOO_MANY_TOKENS),
    ([5, 16], [-2, 1], 4, 8, fa.PLAN_BAD_INPUT), ([5, 16, 3], [2**31 - 1, 1, 2**31 - 1], 4, 8, fa.PLAN_ROW_FULL)])
def test_plan_that_cannot_be_made_changes_nothing(cuda_ok, cached, new, spare, most, status):
    table, free = _state(cached, 16, 3, spare, 3)
    assert _check_plan(cached, new, table, free, 16, most)["status"] == status


@pytest.mark.gpu
def test_plan_refuses_what_the_device_holds_wrong(cuda_ok):
    table, free = _state([5, 16], 16, 3, 4, 3)
    for cached, count in (([-1, 16], None), ([49, 16], None), ([5, 16], -3), ([5, 16], 100)):
        t = _ints(table)
        fp = _ints(free + [-1] * 2)
        n = _ints([len(free) if count is None else count])
        lens, cu, fco, st = (torch.empty(k, dtype=torch.int32, device="cuda") for k in (2, 3, 1, 1))
        slots, pos, req = torch.empty(8, dtype=torch.int64, device="cuda"), _ints([5] * 8), _ints([5] * 8)
        fa.paged_plan(_ints(cached), _ints([1, -1]), t, fp, n, 16, lens, cu, slots, pos, req, fco, st)
        assert st.item() == fa.PLAN_BAD_INPUT
        assert t.tolist() == table and fp.tolist() == free + [-1] * 2 and lens.tolist() == cached
        assert fco.item() == n.item() and (slots == -1).all() and (req == -1).all() and cu.tolist() == [0, 0, 0]


@pytest.mark.gpu
def test_plan_without_requests_or_tokens(cuda_ok):
    _check_plan([], [], [], [4, 5], 16, 5)
    table, free = _state([5, 16], 16, 3, 2, 3)
    _check_plan([5, 16], [0, -1], table, free, 16, 0)


@pytest.mark.gpu
def test_plan_in_place_over_many_steps_captured(cuda_ok):
    # lens is cached, free_count_out is free_count: one captured graph, replayed, against the oracle
    R, ps, cols, most = 40, 8, 30, 200
    rng = np.random.default_rng(5)
    table, free = _state([0] * R, ps, cols, 220, 1)
    lens = [0] * R
    t = dict(cached=_ints(lens), new=_ints([0] * R), table=_ints(table), free=_ints(free), n=_ints([len(free)]),
             cu=_ints([0] * (R + 1)), slots=torch.zeros(most, dtype=torch.int64, device="cuda"), pos=_ints([0] * most),
             req=_ints([0] * most), st=_ints([0]))

    def step():
        fa.paged_plan(t["cached"], t["new"], t["table"], t["free"], t["n"], ps, t["cached"], t["cu"], t["slots"], t["pos"],
                      t["req"], t["n"], t["st"])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(25):
        new = np.where(rng.random(R) < 0.15, -1, rng.integers(0, 9, R)).tolist()
        want = ref.plan(lens, new, table, free, ps, cols, most)
        t["new"].copy_(_ints(new))
        graph.replay()
        torch.cuda.synchronize()
        assert t["st"].item() == want["status"]
        lens, table, free = want["lens"], want["table"], want["free"]
        assert t["cached"].tolist() == lens and t["slots"].tolist() == want["slots"] and t["cu"].tolist() == want["cu"]
        assert t["pos"].tolist() == want["positions"] and t["req"].tolist() == want["req"]
        n = t["n"].item()
        assert t["free"][:n].tolist() == free
        live = [r[:-(-k // ps)] for r, k in zip(table, lens)]
        assert [r[:len(w)] for r, w in zip(t["table"].tolist(), live)] == live
        flat = sum(live, []) + free
        assert sorted(flat) == list(range(220))  # every page is in one place


@pytest.mark.gpu
def test_plan_on_a_whole_cluster_captured_and_on_a_side_stream(cuda_ok):
    # 3000 requests are a full cluster: one captured step, replayed from the same start, and the call on another stream
    R, ps = 3000, 16
    rng = np.random.default_rng(8)
    cached, new = rng.integers(0, 200, R).tolist(), rng.integers(-1, 9, R).tolist()
    table, free = _state(cached, ps, 14, 2000, 4)
    most = sum(max(n, 0) for n in new) + 5
    want = ref.plan(cached, new, table, free, ps, 14, most)
    assert want["status"] == 0
    t0, f0 = _ints(table), _ints(free + [-7] * 45000)
    t, f, c, n, count = t0.clone(), f0.clone(), _ints(cached), _ints(new), _ints([len(free)])
    o = {k: torch.full((m,), -99, dtype=torch.int64 if k == "slots" else torch.int32, device="cuda")
         for k, m in (("lens", R), ("cu", R + 1), ("slots", most), ("positions", most), ("req", most), ("fco", 1), ("st", 1))}
    step = lambda: fa.paged_plan(c, n, t, f, count, ps, o["lens"], o["cu"], o["slots"], o["positions"], o["req"],  # noqa: E731
                                 o["fco"], o["st"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for replay in range(3):  # the side stream's result first, then the replays'
        if replay:
            t.copy_(t0)
            f.copy_(f0)
            graph.replay()
        torch.cuda.synchronize()
        assert o["st"].item() == 0 and t.tolist() == want["table"]
        for k in ("lens", "cu", "slots", "positions", "req"):
            assert o[k].tolist() == want[k], k
            o[k].fill_(-99)
        m = o["fco"].item()
        assert m == len(want["free"]) and f[:m].tolist() == want["free"]


# ------------------------------------------------------------------ append on the GPU
def _e4m3(x):
    return torch.from_numpy(oracle.e4m3_decode(x.view(torch.uint8).cpu().numpy()))


def _values(cache, fp8):
    return _e4m3(cache).double().numpy() if fp8 else f64(cache)


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter,fp8,ps,layout", [
    (1, 1, 1, 64, 64, False, False, 16, "plain"), (8, 32, 8, 128, 128, False, False, 16, "plain"),
    (33, 7, 7, 128, 64, True, True, 1, "heads"), (50, 6, 2, 64, 32, True, False, 20, "joint"),
    (300, 3, 1, 128, 0, False, True, 64, "joint"), (17, 16, 1, 64, 48, False, True, 256, "plain"),
    (65, 0, 4, 128, 128, False, False, 8, "heads"), (9, 4, 0, 64, 64, False, False, 8, "plain")])
def test_append(cuda_ok, T, Hq, Hk, d, rot, inter, fp8, ps, layout):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, Hq + 2 * Hk, d, generator=g).bfloat16().cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    wq, wk = ((torch.randn(d, generator=g) * 0.2 + 1).bfloat16().cuda() for _ in range(2))
    rope = fa.rope_table(5000, rot) if rot else None
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32).cuda()
    pages = T // ps + 3
    slots = torch.randperm(pages * ps, generator=g)[:T].cuda()
    skipped = torch.rand(T, generator=g).cuda() < (0.2 if T > 1 else 0)
    slots[skipped] = -1
    kind = torch.uint8 if fp8 else torch.bfloat16
    fill = 0x31 if fp8 else 3.0
    if layout == "heads":
        kc, vc = (torch.full((pages, Hk, ps, d), fill, dtype=kind, device="cuda").transpose(1, 2) for _ in range(2))
    elif layout == "joint":
        both = torch.full((pages, 2, ps, Hk, d), fill, dtype=kind, device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    else:
        kc, vc = (torch.full((pages, ps, Hk, d), fill, dtype=kind, device="cuda") for _ in range(2))
    kd, vd = ((torch.rand(Hk, generator=g) * 0.02 + 0.01).cuda() for _ in range(2)) if fp8 else (None, None)
    qo = torch.full((T, Hq, d), 9.0, device="cuda", dtype=torch.bfloat16)
    fa.paged_append(q, k, v, wq, wk, rope, pos, slots, kc, vc, eps=1e-5, interleaved=inter, k_descale=kd, v_descale=vd,
                    q_out=qo)
    assert fa.fa_get_device_status() == OK
    table, p = None if rope is None else f64(rope), pos.cpu().numpy()
    size = lambda y: np.abs(y) + np.abs(y).max(-1, keepdims=True)  # noqa: E731  at least |y_a| + |y_b|
    live = ~skipped.cpu().numpy()
    want = ref.norm_rope(f64(q), f64(wq), table, p, inter, 1e-5)
    flat = size(ref.norm_rope(f64(q), f64(wq), None, p, inter, 1e-5))
    assert (np.abs(f64(qo) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * flat)[live].all()
    assert (qo[skipped] == 9).all()
    want = ref.norm_rope(f64(k), f64(wk), table, p, inter, 1e-5)
    flat = size(ref.norm_rope(f64(k), f64(wk), None, p, inter, 1e-5))
    at = slots[~skipped].cpu().numpy()
    got_k, got_v = (_values(c, fp8)[at // ps, at % ps] for c in (kc, vc))
    if fp8:
        want, flat = (np.clip(z / f64(kd)[None, :, None], -448, 448) for z in (want, flat))
        lim = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 2.0 ** -20 * flat
        assert (np.abs(got_k - want[live]) <= lim[live]).all()
        code = (v.float() / vd[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(vc.view(torch.uint8)[slots[~skipped] // ps, slots[~skipped] % ps], code[~skipped])
    else:
        assert (np.abs(got_k - want[live]) <= 2.0 ** -8 * np.abs(want[live]) + 2.0 ** -20 * flat[live]).all()
        assert torch.equal(vc[slots[~skipped] // ps, slots[~skipped] % ps], v[~skipped])
    rest = torch.ones(pages * ps, dtype=torch.bool, device="cuda")
    rest[slots[~skipped]] = False
    rest = rest.nonzero()[:, 0]
    for c in (kc, vc):  # other slots are as they were
        assert (c[rest // ps, rest % ps] == fill).all()


@pytest.mark.gpu
def test_append_slot_or_position_outside_is_reported_and_skipped(cuda_ok):
    x = torch.randn(4, 3, 64, device="cuda").bfloat16()
    rope = fa.rope_table(10, 64)
    for slots, pos in (([0, 32, 2, 3], [0, 1, 2, 3]), ([0, 2**40, 2, 3], [0, 1, 2, 3]), ([0, 1, 2, 3], [0, 10, 2, 3]),
                       ([0, 1, 2, 3], [0, -1, 2, 3])):
        kc, vc = torch.zeros(2, 2, 16, 1, 64, device="cuda", dtype=torch.bfloat16)
        qo = torch.full((4, 1, 64), 9.0, device="cuda", dtype=torch.bfloat16)
        fa.paged_append(x[:, :1], x[:, 1:2], x[:, 2:], None, None, rope, _ints(pos),
                        torch.tensor(slots, device="cuda"), kc, vc, q_out=qo)
        assert fa.fa_get_device_status() == DEVICE_CHECK and fa.fa_get_device_status() == OK
        assert (qo[1] == 9).all() and (kc[0, 1] == 0).all() and (vc[0, 4:] == 0).all()
        assert torch.equal(vc[0, [0, 2, 3], 0], x[[0, 2, 3], 2])


@pytest.mark.gpu
def test_append_e4m3_saturates_and_keeps_nan(cuda_ok):
    v = torch.tensor([math.inf, -math.inf, math.nan, 1e30, -1e30, 448.0, 464.0, 2.0 ** -9], device="cuda")
    v = v.repeat(8)[None, None].bfloat16()
    kc, vc = torch.zeros(2, 1, 1, 1, 64, device="cuda", dtype=torch.float8_e4m3fn)
    fa.paged_append(v * 0, torch.ones_like(v), v, None, None, None, None, torch.zeros(1, dtype=torch.int64, device="cuda"),
                    kc, vc)
    got = _e4m3(vc).reshape(8, 8)
    assert torch.equal(got[:, [0, 1, 3, 4, 5, 6, 7]],
                       torch.tensor([448, -448, 448, -448, 448, 448, 2.0 ** -9]).to(got.dtype).expand(8, 7))
    assert torch.isnan(got[:, 2]).all()


@pytest.mark.gpu
def test_append_e4m3_rounds_the_quotient(cuda_ok):
    # codes equal the cast of the fp32 quotient, on rounding borders too: every bf16 value from 2^-12 to
    # 2^11, both signs, over factors that are powers of two, odd integers (exact ties among the
    # quotients), reciprocals, tiny and huge
    x = torch.arange(0x3980, 0x4500, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.cat([x, -x]).cuda()
    T = x.numel() // 64
    x = x[:T * 64].reshape(T, 1, 64)
    for f in (0.25, 1.0, 3.0, 5.0, 7.0, 0.1, 1 / 3, 0.7, 0.0123, 448.0 / 3, 2.0 ** -120, 1e-38, 1e-40, 3e35):
        kc, vc = torch.zeros(2, T, 1, 1, 64, device="cuda", dtype=torch.float8_e4m3fn)
        d = torch.tensor([f], device="cuda")
        fa.paged_append(x, x, x, None, None, None, None, torch.arange(T, device="cuda"), kc, vc, v_descale=d)
        want = (x.float() / d).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(vc[:, 0].view(torch.uint8), want.view(torch.uint8)), f


# ------------------------------------------------------------------ decode on the GPU
def _pool(lens, ps, Hk, d, fp8, seed, cols=None, poison=True):
    """Caches whose unused slots and pages are NaN, block table with -1 past a row's pages, and fp64
    values of both caches."""
    g = torch.Generator().manual_seed(seed)
    table, _ = _state(lens, ps, cols or max([1] + [-(-n // ps) for n in lens]), 3, seed)
    used = sum(-(-n // ps) for n in lens)
    pages = used + 3
    out = []
    for _ in range(2):
        c = torch.randn(pages, ps, Hk, d, generator=g)
        c = (64 * c).clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else c.bfloat16()
        keep = torch.zeros(pages, ps, dtype=torch.bool)
        for row, n in zip(table, lens):
            for j in range(0, n, ps):
                keep[row[j // ps], :min(ps, n - j)] = True
        if poison:
            if fp8:
                c.view(torch.uint8)[~keep] = 0x7f
            else:
                c[~keep] = math.nan
        out.append(c)
    kc, vc = (c.cuda() for c in out)
    return kc, vc, table


def _check_decode(q, kc, vc, table, lens, req, o, lse, scale, fp8=False, kd=None, vd=None):
    T, Hq, d = q.shape
    k, v = (np.nan_to_num(_values(c, fp8)) for c in (kc, vc))
    if kd is not None:
        k, v = k * f64(kd)[:, None], v * f64(vd)[:, None]
    ps, Hk = kc.shape[1], kc.shape[2]
    q64, o64, l64 = f64(q), f64(o), f64(lse)
    for t in range(T):
        if req[t] < 0:
            continue
        n = lens[t]
        for hk in range(Hk):
            rows = slice(hk * (Hq // Hk), (hk + 1) * (Hq // Hk))
            kk, vv = (ref.gather(c, table[req[t]], n, hk, ps) for c in (k, v))
            for h in range(rows.start, rows.stop):
                wo, wl = ref.decode_row(q64[t, h], kk, vv, scale)
                if n == 0:
                    assert (o64[t, h] == 0).all() and l64[t, h] == -np.inf
                    continue
                A = scale * (np.abs(kk) @ np.abs(q64[t, h])).max()
                E = 4 * d * U * A + 2.0 ** -15 + (2.0 ** -11 if fp8 else 0) + 4 * n * U
                mag = np.exp(scale * (kk @ q64[t, h]) - wl) @ np.abs(vv)
                assert (np.abs(o64[t, h] - wo) <= 2.0 ** -8 * np.abs(wo) + E * mag).all(), (t, h)
                assert abs(l64[t, h] - wl) <= E + 2.0 ** -22 * abs(wl), (t, h)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,Hq,Hk,d,ps", [
    ([1], 1, 1, 64, 16), ([1], 1, 1, 128, 1), ([2, 0, 1], 4, 2, 128, 16), ([0, 0], 8, 8, 64, 8),
    ([15, 16, 17, 63, 64, 65, 127, 128, 129], 8, 2, 64, 16), ([15, 16, 17, 63, 64, 65, 127, 128, 129], 6, 2, 128, 20),
    ([300], 16, 16, 64, 16), ([4097], 8, 1, 128, 64), ([5000, 1], 7, 1, 64, 256), ([1000, 33, 0, 2], 5, 1, 128, 32),
    ([777, 600], 16, 1, 128, 8), ([513, 20], 24, 1, 64, 16), ([100, 2000], 33, 1, 128, 32), ([70] * 60, 9, 3, 64, 16),
    ([900, 3, 77], 32, 2, 128, 7), (list(range(130)), 2, 1, 64, 32)])
def test_decode(cuda_ok, lens, Hq, Hk, d, ps, fp8):
    kc, vc, table = _pool(lens, ps, Hk, d, fp8, len(lens) + ps)
    g = torch.Generator().manual_seed(d + ps)
    q = torch.randn(len(lens), Hq, d, generator=g).bfloat16().cuda()
    kd, vd = ((torch.rand(Hk, generator=g) * 0.02 + 0.01).cuda() for _ in range(2)) if fp8 else (None, None)
    o, lse = fa.paged_decode(q, kc, vc, _ints(table), _ints(lens), k_descale=kd, v_descale=vd)
    assert fa.fa_get_device_status() == OK
    _check_decode(q, kc, vc, table, lens, range(len(lens)), o, lse, d ** -0.5, fp8, kd, vd)
    again = fa.paged_decode(q, kc, vc, _ints(table), _ints(lens), k_descale=kd, v_descale=vd)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.gpu
def test_decode_rows_that_share_requests_and_padded_rows(cuda_ok):
    # a chunk of 3 tokens of request 1 (each sees itself and what is before it), single tokens of requests
    # 2 and 0, two padded rows whose results stay, strided q
    lens0, ps = [40, 100, 7], 16
    kc, vc, table = _pool(lens0, ps, 2, 64, False, 3)
    req, lens = [1, 1, -1, 1, 2, 0, -1], [98, 99, 77, 100, 7, 40, -5]
    x = torch.randn(7, 12, 64, device="cuda").bfloat16()
    q = x[:, 2:8]
    o = torch.full((7, 6, 64), 9.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((7, 6), 9.0, device="cuda")
    fa.paged_decode(q, kc, vc, _ints(table), _ints(lens), scale=0.3, req=_ints(req), out=o, lse=lse)
    assert fa.fa_get_device_status() == OK
    _check_decode(q, kc, vc, table, lens, req, o, lse, 0.3)
    assert (o[[2, 6]] == 9).all() and (lse[[2, 6]] == 9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_cache_layouts(cuda_ok, fp8):
    lens, ps = [50, 21], 16
    kc, vc, table = _pool(lens, ps, 4, 128, fp8, 3)
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    heads = [c.view(torch.uint8 if fp8 else torch.bfloat16).transpose(1, 2).contiguous().transpose(1, 2) for c in (kc, vc)]
    joint = torch.stack([c.view(torch.uint8 if fp8 else torch.bfloat16) for c in (kc, vc)], 1)
    wide = torch.full((2, 9), -1, dtype=torch.int32, device="cuda")
    wide[:, :len(table[0])] = _ints(table)
    for a, b, t in ((*heads, _ints(table)), (joint[:, 0], joint[:, 1], wide), (kc, vc, wide[:, :len(table[0])])):
        o, lse = fa.paged_decode(q, a, b, t, _ints(lens))
        _check_decode(q, a, b, table, lens, range(2), o, lse, 128 ** -0.5, fp8)
    assert fa.fa_get_device_status() == OK


@pytest.mark.gpu
def test_decode_offsets_past_32_bits(cuda_ok):
    # pages 512 M elements apart: 10 pages of one 5 GB buffer, K at its start, V in its second half page
    step = 1 << 29
    buf = torch.zeros(10 * step, dtype=torch.uint8, device="cuda")
    kc = buf.as_strided((10, 16, 2, 64), (step, 128, 64, 1))
    vc = buf.as_strided((10, 16, 2, 64), (step, 128, 64, 1), step // 2)
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = ((32 * torch.randn(10, 16, 2, 64, generator=g, device="cuda")).to(torch.float8_e4m3fn) for _ in range(2))
    kc.copy_(k.view(torch.uint8))
    vc.copy_(v.view(torch.uint8))
    q = torch.randn(1, 4, 64, device="cuda").bfloat16()
    table, lens = _ints([[9, 0, 8, 4, 7]]), _ints([75])
    d = torch.full((2,), 0.02, device="cuda")
    want = fa.paged_decode(q, k, v, table, lens, k_descale=d, v_descale=d)
    got = fa.paged_decode(q, kc, vc, table, lens, k_descale=d, v_descale=d)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and fa.fa_get_device_status() == OK
    # and the append to its far end
    x = torch.randn(1, 8, 64, device="cuda").bfloat16()
    slot = torch.tensor([9 * 16 + 15], device="cuda")
    fa.paged_append(x[:, :4], x[:, 4:6], x[:, 6:], None, None, None, None, slot, kc, vc, k_descale=d, v_descale=d)
    fa.paged_append(x[:, :4], x[:, 4:6], x[:, 6:], None, None, None, None, slot, k, v, k_descale=d, v_descale=d)
    assert torch.equal(kc[9, 15], k.view(torch.uint8)[9, 15]) and torch.equal(vc[9, 15], v.view(torch.uint8)[9, 15])


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_large_scores_equal_keys_and_special_values(cuda_ok, fp8):
    lens, ps, d = [200, 130, 90], 16, 64
    kc, vc, table = _pool(lens, ps, 1, d, fp8, 8)
    q = torch.randn(3, 2, d, device="cuda").bfloat16()
    o, lse = fa.paged_decode(q * 1024, kc, vc, _ints(table), _ints(lens), scale=0.01)  # one key takes it all
    _check_decode(q * 1024, kc, vc, table, lens, range(3), o, lse, 0.01, fp8)
    o, lse = fa.paged_decode(q * 0, kc, vc, _ints(table), _ints(lens))  # equal scores: the mean
    _check_decode(q * 0, kc, vc, table, lens, range(3), o, lse, 0.125, fp8)
    # a NaN key and an infinite value reach their own row alone
    kind = (lambda c: c.view(torch.uint8)) if fp8 else (lambda c: c)
    k2, v2 = kc.clone(), vc.clone()
    kind(k2)[table[1][2], 3] = 0x7f if fp8 else math.nan
    a, b = fa.paged_decode(q, kc, vc, _ints(table), _ints(lens)), fa.paged_decode(q, k2, v2, _ints(table), _ints(lens))
    assert torch.isnan(b[0][1]).all() and torch.isnan(b[1][1]).all()
    assert torch.equal(a[0][[0, 2]], b[0][[0, 2]]) and torch.equal(a[1][[0, 2]], b[1][[0, 2]])
    if not fp8:
        v2[table[2][0], 5, 0, 7] = math.inf
        c = fa.paged_decode(q, kc, v2, _ints(table), _ints(lens))
        assert torch.equal(c[0][:2], a[0][:2]) and not torch.isfinite(c[0][2, :, 7]).any()
        assert torch.equal(c[0][2, :, :7], a[0][2, :, :7]) and torch.equal(c[1], a[1])
    assert fa.fa_get_device_status() == OK


@pytest.mark.gpu
def test_decode_bad_device_values_are_reported_and_leave_other_rows(cuda_ok):
    lens, ps = [70, 40, 90], 16
    kc, vc, table = _pool(lens, ps, 2, 64, False, 5)
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    want = fa.paged_decode(q, kc, vc, _ints(table), _ints(lens))
    assert fa.fa_get_device_status() == OK
    for page, n, r in ((10 ** 6, 40, 1), (-1, 40, 1), (None, 97, 1), (None, -3, 1), (None, 40, 3), (None, 2 ** 31 - 1, 1)):
        t = [list(row) for row in table]
        if page is not None:
            t[1][1] = page
        got = fa.paged_decode(q, kc, vc, _ints(t), _ints([70, n, 90]), req=_ints([0, r, 2]))
        assert fa.fa_get_device_status() == DEVICE_CHECK
        assert torch.equal(got[0][[0, 2]], want[0][[0, 2]]) and torch.equal(got[1][[0, 2]], want[1][[0, 2]])
    assert fa.fa_get_device_status() == OK


@pytest.mark.gpu
def test_decode_captured_with_lengths_that_change_and_on_a_side_stream(cuda_ok):
    ps, d = 16, 128
    full = [600, 300, 40, 1200]
    kc, vc, table = _pool(full, ps, 2, d, False, 9, poison=False)
    t = _ints(table)
    q = torch.randn(4, 8, d, device="cuda").bfloat16()
    lens = _ints(full)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = fa.paged_decode(q, kc, vc, t, lens)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.paged_decode(q, kc, vc, t, lens)
    for new in (full, [1, 0, 40, 1199], [0, 0, 0, 0], [599, 300, 1, 64]):
        lens.copy_(_ints(new))
        graph.replay()
        want = fa.paged_decode(q, kc, vc, t, _ints(new))
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        if new is full:
            assert torch.equal(side[0], o) and torch.equal(side[1], lse)
    assert fa.fa_get_device_status() == OK


@pytest.mark.gpu
def test_two_decodes_at_once_with_workspaces_of_their_own(cuda_ok):
    full = [3000, 17, 900]
    kc, vc, table = _pool(full, 16, 2, 128, False, 9)
    t, lens = _ints(table), _ints(full)
    qs = [torch.randn(3, 8, 128, device="cuda").bfloat16() for _ in range(2)]
    want = [fa.paged_decode(q, kc, vc, t, lens) for q in qs]
    nbytes = fa.fa_paged_decode_workspace_bytes(3, 8, 2, 128)
    ws = [torch.full((nbytes,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got.append(fa.paged_decode(qs[i], kc, vc, t, lens, workspace=ws[i]))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_binding_refuses(cuda_ok):
    kc, vc, table = _pool([40], 16, 2, 64, False, 1)
    q, t, n = torch.zeros(1, 4, 64, device="cuda", dtype=torch.bfloat16), _ints(table), _ints([40])
    for call in (lambda: fa.paged_decode(q.float(), kc, vc, t, n), lambda: fa.paged_decode(q, kc, vc.float(), t, n),
                 lambda: fa.paged_decode(q, kc, vc[:1], t, n), lambda: fa.paged_decode(q, kc, vc, t, n.long()),
                 lambda: fa.paged_decode(q, kc, vc, t.cpu(), n), lambda: fa.paged_decode(q[:, :3], kc, vc, t, n),
                 lambda: fa.paged_decode(q, kc, vc, t, n, workspace=torch.empty(1 << 24, dtype=torch.uint8)),
                 lambda: fa.paged_decode(q, kc, vc, t, n, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
                 lambda: fa.paged_decode(q, kc, vc, t, n, k_descale=torch.ones(2, device="cuda")),
                 lambda: fa.paged_decode(q, kc, vc, t, n, out=torch.empty_like(q[:, :2])),
                 lambda: fa.paged_append(q, kc[0, :1], kc[0, :1], None, None, None, None, n, kc, vc),
                 lambda: fa.paged_append(q, kc[0, :1], kc[0, :1], None, None, None, None, n.long(),
                                         kc[:1].expand(4, -1, -1, -1), vc[:1].expand(4, -1, -1, -1)),
                 lambda: fa.paged_append(q, kc[0, :2], kc[0, :2], None, None, None, None, n.long(), kc, vc)):
        with pytest.raises((ValueError, fa.FAError)):
            call()
    with pytest.raises(fa.FAError):
        fa.paged_decode(q, kc, vc, t, n, scale=-1.0)
    with pytest.raises(ValueError):
        fa.paged_decode(q[:, :, :0], kc, vc, t, n)
    x = q[:, :2]
    with pytest.raises(ValueError):
        fa.paged_append(q, x, x, None, None, None, None, n.long(), kc, kc)
    with pytest.raises(TypeError):
        fa.paged_decode(q, kc, vc, t, [40])
    with pytest.raises(fa.FAError):
        fa.paged_decode(q, kc, vc, torch.empty(0, 3, dtype=torch.int32, device="cuda"), n)


# ------------------------------------------------------------------ together
@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_serving_steps(cuda_ok, fp8):
    """Prompts in chunks, single tokens, requests that end and begin, over one small pool: plan -> append ->
    decode in one captured graph whose sizes are padded, checked each step against fp64 attention over
    every request's whole history (as the cache holds it)."""
    R, ps, cols, most, Hq, Hk, d = 6, 8, 12, 24, 4, 2, 64
    pool = 30
    rng = np.random.default_rng(2)
    g = torch.Generator(device="cuda").manual_seed(3)
    z = lambda n, kind=torch.int32: torch.zeros(n, dtype=kind, device="cuda")  # noqa: E731
    lens, new, table, free, count = z(R), z(R), z((R, cols)) - 1, torch.arange(pool, dtype=torch.int32, device="cuda"), z(1) + pool
    cu, slots, pos, req, st = z(R + 1), z(most, torch.int64), z(most), z(most), z(1)
    x = torch.zeros(most, Hq + 2 * Hk, d, device="cuda", dtype=torch.bfloat16)
    kind = torch.uint8 if fp8 else torch.bfloat16
    kc, vc = torch.zeros(2, pool, ps, Hk, d, device="cuda", dtype=kind)
    kd, vd = (torch.tensor([0.02, 0.03], device="cuda"), torch.tensor([0.025, 0.02], device="cuda")) if fp8 else (None, None)
    w = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).bfloat16()
    rope = fa.rope_table(cols * ps, d)
    q, o, lse = z((most, Hq, d), torch.bfloat16), z((most, Hq, d), torch.bfloat16), z((most, Hq), torch.float32)

    def step():
        fa.paged_plan(lens, new, table, free, count, ps, lens, cu, slots, pos, req, count, st)
        fa.paged_append(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], w, w, rope, pos, slots, kc, vc, k_descale=kd,
                        v_descale=vd, q_out=q)
        fa.paged_decode(q, kc, vc, table, pos + 1, req=req, k_descale=kd, v_descale=vd, out=o, lse=lse)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    keys, values, length = [[] for _ in range(R)], [[] for _ in range(R)], [0] * R
    for i in range(30):
        n = [int(rng.integers(3, 9)) if length[b] == 0 else -1 if length[b] > 60 else int(rng.integers(0, 3)) for b in range(R)]
        while sum(max(a, 0) for a in n) > most:
            n[int(np.argmax(n))] -= 1
        new.copy_(torch.tensor(n, dtype=torch.int32))
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        graph.replay()
        assert fa.fa_get_device_status() == OK and st.item() == 0
        kall, vall = ref.norm_rope(f64(x[:, Hq:Hq + Hk]), f64(w), f64(rope), pos.cpu().numpy(), False, 1e-6), f64(x[:, Hq + Hk:])
        t = 0
        hist_k, hist_v = (_values(c, fp8) for c in (kc, vc))
        tab = table.cpu().numpy()
        for b in range(R):
            if n[b] < 0:
                keys[b], values[b], length[b] = [], [], 0
                continue
            for _ in range(n[b]):
                keys[b].append(kall[t])
                values[b].append(vall[t])
                length[b] += 1
                assert req[t].item() == b and pos[t].item() == length[b] - 1
                t += 1
            for j in range(length[b]):  # the cache holds the whole history, to its type's precision
                half, floor = (2.0 ** -4, 2.0 ** -10) if fp8 else (2.0 ** -8, 0)
                for hist, want, f in ((hist_k, keys[b][j], kd), (hist_v, values[b][j], vd)):
                    want = want if f is None else np.clip(want / f64(f)[:, None], -448, 448)
                    got = hist[tab[b, j // ps], j % ps]
                    assert (np.abs(got - want) <= np.maximum(half * np.abs(want), floor) + 2.0 ** -18 * np.abs(want).max()).all()
        assert lens.tolist() == length and (req[t:] == -1).all()
        _check_decode(q, kc, vc, tab, (pos + 1).tolist(), req.tolist(), o, lse, d ** -0.5, fp8, kd, vd)
