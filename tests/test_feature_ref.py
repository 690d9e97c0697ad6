"""The 64-bit implementations the operator tests compare with: closed forms, gradients against central
differences, and the checkpoint's arithmetic on hand-worked blocks."""
import pytest
import torch

import feature_ref as R


def _inputs(n, L, C, seed=0):
    g = torch.Generator().manual_seed(seed)
    f = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    return f(n, (L + 1) ** 2, C) + 0.3, 1 + 0.2 * f(L + 1, C), f(C), f(n, (L + 1) ** 2, C)


def test_norm_has_unit_groups_and_commutes_with_row_rotations():
    h, w, b, _ = _inputs(3, 2, 8)
    y, mean, rstd = R.norm(h, torch.ones_like(w), None, 2, 0.0 + 1e-300)
    assert torch.allclose(y[:, 0].mean(-1), torch.zeros(3, dtype=torch.float64), atol=1e-14)
    for rows in R.degrees(2):
        assert torch.allclose(y[:, rows].pow(2).mean((1, 2)), torch.ones(3, dtype=torch.float64))
    q = torch.linalg.qr(torch.randn(5, 5, dtype=torch.float64))[0]
    t = h.clone()
    t[:, 4:9] = torch.einsum("ab,nbc->nac", q, h[:, 4:9])
    a, c = R.norm(h, w, b, 2, 1e-5)[0], R.norm(t, w, b, 2, 1e-5)[0]
    assert torch.allclose(c[:, 4:9], torch.einsum("ab,nbc->nac", q, a[:, 4:9]))


@pytest.mark.parametrize("L,C", [(0, 7), (2, 5)])
def test_norm_gradient_formula_matches_autograd_and_differences(L, C):
    h, w, b, g = _inputs(4, L, C)
    t = [v.clone().requires_grad_() for v in (h, w, b)]
    (g * R.norm(*t, L, 1e-5)[0]).sum().backward()
    _, mean, rstd = R.norm(h, w, b, L, 1e-5)
    for got, want in zip(R.norm_backward(h, w, mean, rstd, g, L), t):
        assert torch.allclose(got, want.grad, rtol=1e-11, atol=1e-12)
    for k in range(3):
        dirn = torch.randn(t[k].shape, dtype=torch.float64)
        at = lambda s: (g * R.norm(*[v + s * dirn if i == k else v for i, v in enumerate((h, w, b))], L, 1e-5)[0]).sum()
        diff = (at(1e-5) - at(-1e-5)) / 2e-5
        assert torch.allclose(diff, (t[k].grad * dirn).sum(), rtol=1e-7)


def test_checkpoint_blocks_worked_by_hand():
    x = torch.zeros(1, 40)
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 1.0, -1.999, 0.0078125, 0.0234375  # e = 0, unit 1/64
    x[0, 32] = 2.0 ** -130                                                 # below the smallest exponent
    val, code, byte = R.coded(x)
    assert code[0, :4].tolist() == [64, -127, 0, 2] and byte.tolist() == [[127, 7]]  # 0.5 to 0, 1.5 to 2: half to even
    assert val[0, :4].tolist() == [1.0, -127 / 64, 0.0, 2 / 64] and val[0, 32] == 0
    x[0, 33] = float("inf")
    val, _, byte = R.coded(x)
    assert byte[0, 1] == 255 and torch.isnan(val[0, 32:]).all() and torch.isfinite(val[0, :32]).all()


def test_embedding_gradient_is_the_transpose_of_the_lookup():
    tok = torch.tensor([2, -1, 0, 2, 9], dtype=torch.int32)
    table, g = torch.randn(4, 3, dtype=torch.float64), torch.randn(5, 4, 3, dtype=torch.float64)
    out = R.embedding(tok, table, 1.5, 1)
    grad, _ = R.embedding_backward(tok, g, 4, 1.5)
    assert torch.allclose((out * g).sum(), (grad * table).sum())
    assert (out[1] == 0).all() and (out[4] == 0).all() and (grad[1] == 0).all() and (grad[3] == 0).all()
