"""Layouts of the paged cache's tensors as the binding takes them."""
import pytest
import torch

from io_aware_exact_22_b200 import fa

OK = 0


@pytest.mark.gpu
@pytest.mark.parametrize("pages,ps,Hk", [(5, 16, 1), (1, 16, 2), (7, 1, 2), (1, 1, 1)])
def test_strides_of_one_element_dimensions_do_not_count(cuda_ok, pages, ps, Hk):
    # one head, one page, or pages of one token: K and V may then have different strides there (as a
    # transposed and a plain tensor do) and lie alike all the same
    d, T = 64, min(4, pages * ps)
    rnd = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    kc, vc = rnd(pages, ps, Hk, d), rnd(pages, ps, Hk, d)
    strides = [s if n > 1 else s + 8 * (i + 1) for i, (s, n) in enumerate(zip(kc.stride(), kc.shape))]
    other = kc.clone().as_strided(kc.shape, strides)
    assert torch.equal(other, kc) and other.stride() != vc.stride()
    n = pages * ps
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = rnd(1, 2 * Hk, d)
    want, got = (fa.paged_decode(q, c, vc, table, lens) for c in (kc, other))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    x = rnd(T, 4 * Hk, d)
    slots = torch.arange(T, device="cuda")
    v2 = vc.clone()
    for c, v in ((kc, vc), (other, v2)):
        fa.paged_append(x[:, :2 * Hk], x[:, 2 * Hk:3 * Hk], x[:, 3 * Hk:], None, None, None, None, slots, c, v)
    assert torch.equal(other, kc) and torch.equal(v2, vc)
    assert fa.fa_get_device_status() == OK


@pytest.mark.gpu
def test_different_strides_are_refused(cuda_ok):
    kc = torch.zeros(4, 2, 16, 64, device="cuda", dtype=torch.bfloat16).transpose(1, 2)
    vc = torch.zeros(4, 16, 2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.paged_decode(torch.zeros(1, 2, 64, device="cuda", dtype=torch.bfloat16), kc, vc,
                        torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda"))


@pytest.mark.gpu
def test_new_outputs_take_torchs_fill_of_uninitialised_memory(cuda_ok):
    # as forward's do: with torch's deterministic fill, rows that a call leaves as they were are NaN
    d = 64
    kc, vc = torch.randn(2, 4, 16, 2, d, device="cuda").bfloat16()
    q, x = torch.randn(40, 4, d, device="cuda").bfloat16(), torch.randn(1, 40, 6, d, device="cuda").bfloat16()
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    ints = lambda v: torch.full((40,), v, dtype=torch.int32, device="cuda")  # noqa: E731
    for shape in ((40, 4, d), (1, 4, 40, d), (1, 2, 40, d), (1, 40, 4, d), (1, 40, 2, d)):  # blocks that are handed out again
        torch.full(shape, 5.0, device="cuda", dtype=torch.bfloat16)
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        assert torch.utils.deterministic.fill_uninitialized_memory
        o, lse = fa.paged_decode(q, kc, vc, table, ints(3), req=ints(-1))
        qo = fa.paged_append(q, x[0, :, :2], x[0, :, :2], None, None, None, None, ints(-1).long(), kc, vc)
        rope = fa.rope_table(8, d)
        a, b = fa.qk_norm_rope(x[:, :, :4], x[:, :, 4:], None, None, rope, ints(9))  # no position is in the table
        dq, dk, _, _ = fa.qk_norm_rope_backward(a, b, x[:, :, :4], x[:, :, 4:], None, None, rope, ints(9))
    finally:
        torch.use_deterministic_algorithms(before)
    assert fa.fa_get_device_status() == 5  # the positions
    for t in (o, lse, qo, a, b, dq, dk):
        assert torch.isnan(t).all()
