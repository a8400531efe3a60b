"""Precision of the paged decode, on problems whose terms cancel: the values of a row's keys are chosen so
that sum_j p_j V_j nearly vanishes, so that the rounding of O does not hide what becomes of P.

Tolerance of `cancelling`.  Scores are one product each, exact in fp32, of base-2 size below 0.12, and 5
keys at most fall into one step of the matrix unit.  Relative error of p_j: the scale and its product,
2 u 0.12; the difference to the reference, u 0.12 (E4M3: it carries the power 2^7, u 8 in the reference
and as much in the difference, u = 2^-24); the exponential 2^-22; the terms that P is split into, 2^-23
(three of bf16) or 2^-22 (two of fp16): together below 2^-21 (bf16) and 2^-20 (E4M3).  The matrix unit
may cut each of 5 products and the sum to 24 bits of the largest, which is at most half of
mag = sum p_j |V_j|: 6 2^-23 / 2 mag, below 2^-21.4.  The factors to 1 / l and the store are relative
to O, which is near zero: 2^-8 of it and 2^-20 more.  So |error| <= 2^-20 mag (bf16), 2^-19 mag (E4M3), and
2^-8 |O|.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from io_aware_exact_22_b200 import fa
from oracle import paged_ref as ref
from tests._helpers import f64

OK = 0
SCALE = 2.0 ** -6


def _round_bf16(x):
    return float(torch.tensor(x, dtype=torch.float64).bfloat16())


E4M3_VALUES = np.unique([oracle.e4m3_decode(np.array([c], dtype=np.uint8))[0] for c in range(256) if c & 0x7f != 0x7f])


def _round_e4m3(x):
    return float(E4M3_VALUES[np.abs(E4M3_VALUES - x).argmin()])


def cancelling(T, g, d, fp8, seed):
    """q [T, g, d] bf16, k, v [T, n, d] fp64 of one kv head, values of the cache's type: the column c of V
    makes sum_j p_j V_jc nearly zero for the query head c % g."""
    rng = np.random.default_rng(seed)
    n = 5 if fp8 else 3
    q = np.zeros((T, g, d))
    k, v = np.zeros((2, T, n, d))
    q[:, :, 0] = rng.integers(128, 256, (T, g)) / 128 * rng.choice([-1, 1], (T, g))  # bf16 values in [1, 2)
    k[:, :, 0] = rng.integers(8, 16, (T, n)) / 8 * rng.choice([-1, 1], (T, n))       # E4M3 values in [1, 2)
    to = _round_e4m3 if fp8 else _round_bf16
    for t in range(T):
        p = np.exp(SCALE * np.outer(q[t, :, 0], k[t, :, 0]))  # [g, n]
        for c in range(d):
            w, total = p[c % g], 0.0
            v[t, 0, c] = to(rng.uniform(200, 256) if fp8 else rng.uniform(1, 2))
            for j in range(1, n):
                total += w[j - 1] * v[t, j - 1, c]
                v[t, j, c] = to(-total / w[j])
    return q, k, v


def test_the_problem_shows_the_split_of_p():
    # with exact arithmetic but for P's terms: three bf16 terms and two fp16 terms pass, one fewer do not
    def cut(p, kind, terms):
        kept = np.zeros_like(p)
        for _ in range(terms):
            kept += torch.from_numpy(p - kept).to(kind).double().numpy()
        return kept

    for fp8, kind, terms, tol in ((False, torch.bfloat16, 3, 2.0 ** -20), (True, torch.float16, 2, 2.0 ** -19)):
        q, k, v = cancelling(16, 4, 64, fp8, 3)
        worst = []
        for m in (terms, terms - 1):
            over = 0.0
            for t in range(16):
                p = np.exp(SCALE * q[t, :, 0:1] * k[t, :, 0])
                mag, want = p @ np.abs(v[t]), p @ v[t]
                assert (np.abs(want) <= 2.0 ** -11 * mag)[np.arange(64) % 4, np.arange(64)].all()
                over = max(over, ((np.abs(cut(p, kind, m) @ v[t] - want) - 2.0 ** -8 * np.abs(want)) / mag).max())
            worst.append(over)
        assert worst[0] < tol / 8 and worst[1] > 2 * tol, worst


@pytest.mark.gpu
@pytest.mark.parametrize("d,g", [(64, 4), (64, 12), (128, 4), (128, 16)])
@pytest.mark.parametrize("fp8", [False, True])
def test_probabilities_keep_fp32_precision(cuda_ok, fp8, d, g):
    T, ps = 24, 16
    q, k, v = cancelling(T, g, d, fp8, d + g)
    n = k.shape[1]
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kc, vc = torch.zeros(2, T, ps, 1, d, dtype=torch.float32)
    kc[:, :n, 0], vc[:, :n, 0] = torch.from_numpy(k).float(), torch.from_numpy(v).float()
    kc, vc = kc.to(kind).cuda(), vc.to(kind).cuda()
    assert np.array_equal(vc.float().double().cpu().numpy()[:, :n, 0], v)  # nothing was rounded
    table = torch.arange(T, dtype=torch.int32, device="cuda")[:, None]
    lens = torch.full((T,), n, dtype=torch.int32, device="cuda")
    o, lse = fa.paged_decode(torch.from_numpy(q).bfloat16().cuda(), kc, vc, table, lens, scale=SCALE)
    assert fa.fa_get_device_status() == OK
    o, lse = f64(o), f64(lse)
    tol = 2.0 ** -19 if fp8 else 2.0 ** -20
    for t in range(T):
        for h in range(g):
            want, wl = ref.decode_row(q[t, h], k[t], v[t], SCALE)
            mag = np.exp(SCALE * (k[t] @ q[t, h]) - wl) @ np.abs(v[t])
            assert (np.abs(o[t, h] - want) <= 2.0 ** -8 * np.abs(want) + tol * mag).all(), (t, h)
            assert abs(lse[t, h] - wl) <= 2.0 ** -19, (t, h)

def _cache(lens, ps, d, seed):
    """Block table and bf16 caches of one kv head, pages in random order, what no key uses NaN."""
    rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    pages = rng.permutation(sum(need)).tolist()
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    kc, vc = (torch.randn(sum(need), ps, 1, d, generator=g).bfloat16() for _ in range(2))
    for t, n in enumerate(lens):
        mine = [pages.pop() for _ in range(need[t])]
        table[t, :need[t]] = torch.tensor(mine, dtype=torch.int32)
        if n % ps:
            kc[mine[-1], n % ps:] = vc[mine[-1], n % ps:] = math.nan
    return table.cuda(), kc.cuda(), vc.cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("equal", [True, False])
@pytest.mark.parametrize("d,g,lens", [(64, 2, [1, 5, 200]), (128, 12, [3, 90, 17]), (128, 4, [20000, 2, 700])])
def test_infinite_values_are_as_the_formula_has_them(cuda_ok, d, g, lens, equal):
    # every key has a positive probability (equal scores: a power of two), so a column with +inf is +inf, with
    # -inf -inf, with both NaN; the others are as without them
    T, ps = len(lens), 16
    table, kc, vc = _cache(lens, ps, d, 7)
    q = torch.randn(T, g, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda() * (0 if equal else 1)
    args = (table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    clean, lse = fa.paged_decode(q, kc, vc, *args)
    for t, n in enumerate(lens):
        first, last = table[t, 0].item(), table[t, (n - 1) // ps].item()
        vc[first, 0, 0, 3] = math.inf
        vc[last, (n - 1) % ps, 0, 8] = -math.inf
        vc[last, (n - 1) % ps, 0, d - 1] = math.inf
        if n > 1:
            vc[first, 0, 0, d - 1] = -math.inf
    got, l2 = fa.paged_decode(q, kc, vc, *args)
    assert fa.fa_get_device_status() == OK and torch.equal(lse, l2)
    keep = [c for c in range(d) if c not in (3, 8, d - 1)]
    assert torch.equal(got[:, :, keep], clean[:, :, keep])
    assert (got[:, :, 3] == math.inf).all() and (got[:, :, 8] == -math.inf).all()
    for t, n in enumerate(lens):
        assert torch.isnan(got[t, :, d - 1]).all() if n > 1 else (got[t, :, d - 1] == math.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d,g", [(64, 2), (128, 12)])
@pytest.mark.parametrize("small", [2.0 ** -12, 2.0 ** -20])
def test_a_large_channel_of_q_leaves_the_small_ones_exact(cuda_ok, d, g, small):
    # E4M3 cache, one channel of q 2^22 or 2^30 times the others, which meets keys that are 0 there.  Tolerance
    # as in test_paged.py, E = 4 d u A + 4 n u with 2^-20 for the exponential and P; q's elements
    # lie above 2^-32 of the largest and are exact
    n, ps, T = 40, 16, 3
    rng = torch.Generator().manual_seed(d)
    table, kc, vc = _cache([n] * T, ps, d, 4)
    kc, vc = ((64 * c.float()).clamp(-448, 448).nan_to_num(0.0).to(torch.float8_e4m3fn) for c in (kc, vc))
    kc.view(torch.uint8)[..., 5] = 0
    q = ((1 + torch.rand(T, g, d, generator=rng)) * small).bfloat16()
    q[..., 5] = 1024.0
    scale = 2.0 ** -8 / small
    o, lse = fa.paged_decode(q.cuda(), kc, vc, table, torch.full((T,), n, dtype=torch.int32, device="cuda"), scale=scale)
    assert fa.fa_get_device_status() == OK
    k, v = (c.float().double().cpu().numpy() for c in (kc, vc))
    q64, o, lse, tab = f64(q), f64(o), f64(lse), table.cpu().numpy()
    for t in range(T):
        kk, vv = (ref.gather(c, tab[t], n, 0, ps) for c in (k, v))
        for h in range(g):
            want, wl = ref.decode_row(q64[t, h], kk, vv, scale)
            E = 4 * d * 2.0 ** -24 * scale * (np.abs(kk) @ np.abs(q64[t, h])).max() + 2.0 ** -20 + 4 * n * 2.0 ** -24
            mag = np.exp(scale * (kk @ q64[t, h]) - wl) @ np.abs(vv)
            assert (np.abs(o[t, h] - want) <= 2.0 ** -8 * np.abs(want) + E * mag).all(), (t, h)
            assert abs(lse[t, h] - wl) <= E + 2.0 ** -22 * abs(wl), (t, h)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_long_sums_are_not_cut(cuda_ok, fp8):
    # The scores of 16 keys, 1025 times over: with values of v, and -1024 v the last time.  O is 0 then, every
    # p is off by the same wherever its score comes, and what the kernel gives is the error of its sums alone.
    # In units of |v| sum p / l = |v|: 888 rows, two for each of 444 CTAs, so that a warp adds up a quarter of
    # a row in 128 tiles of 32 keys.  Added with rounding, a tile costs u = 2^-24 of the warp's sum so far, half
    # of a quarter on average: 64 u for the four warps.  Within a tile, 4 (E4M3) or 6 (bf16) steps of the matrix
    # unit may each cut 2 u off the tile's own sum: 12 u over all tiles, and as much for the large last one.
    # Below 128 u = 2^-17.  (Where each step is cut against the long sum, 512 or 768 steps lose about u
    # of it each: 256 to 384 u.)
    T, g, d, ps, n = 888, 4, 64, 16, 16 * 1025
    rng = np.random.default_rng(6)
    k0 = rng.integers(8, 16, ps) / 8 * rng.choice([-1, 1], ps)
    v0 = rng.choice([-0.25, 0.25], d)
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kc, vc = torch.zeros(2, n // ps, ps, 1, d)
    kc[..., 0] = torch.from_numpy(k0).float()[:, None]
    vc[:] = torch.from_numpy(v0).float()
    vc[-1] *= -1024
    q = torch.zeros(T, g, d)
    q[..., 0] = torch.from_numpy(rng.integers(128, 256, (T, g)) / 128)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    o, lse = fa.paged_decode(q.bfloat16().cuda(), kc.to(kind).cuda(), vc.to(kind).cuda(), ints([list(range(n // ps))]),
                             ints([n] * T), req=ints([0] * T), scale=SCALE)
    assert fa.fa_get_device_status() == OK
    assert o.double().abs().max().item() <= 2.0 ** -17 * 0.25
    want = np.log(1025 * np.exp(SCALE * f64(q[..., 0])[..., None] * k0).sum(-1))
    # l: a lane adds up 512 terms (u of its sum each, half of it on average: 256 u = 2^-16), then 7 sums
    assert np.abs(f64(lse) - want).max() <= 2.0 ** -15
