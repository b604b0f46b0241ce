"""Pins of the 64-bit reference that the GPU tests of the token-sequence operators compare with:
library routines, automatic differentiation and central differences (no GPU needed)."""
import math

import pytest
import torch

from token_reference import dequantise, norm_rope, quantise, rotate, visible, window_attention


def _qkv(B, nh, nkv, nq, nk, d, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return rn(B, nh, nq, d), rn(B, nkv, nk, d), rn(B, nkv, nk, d), rn(B, nh, nq, d)


@pytest.mark.parametrize("left,right,sinks,nq", [(-1, 0, 0, 12), (3, 0, 2, 12), (2, 1, 0, 12), (-1, -1, 0, 12),
                                                 (3, 0, 1, 5), (0, 0, 0, 12)])
def test_attention_is_the_library_s_with_a_mask(left, right, sinks, nq):
    q, k, v, do = _qkv(2, 4, 2, nq, 12, 8, 1)
    for t in (q, k, v):
        t.requires_grad_()
    mask = visible(nq, 12, 12, left, right, sinks, "cpu")
    kk, vv = (t.repeat_interleave(2, 1) for t in (k, v))
    o = torch.nn.functional.scaled_dot_product_attention(q, kk, vv, attn_mask=mask, scale=0.3)
    gq, gk, gv = torch.autograd.grad(o, (q, k, v), do)
    r = window_attention(q.detach(), k.detach(), v.detach(), None, left, right, sinks, 0.3, do)
    for name, want in (("o", o), ("dq", gq), ("dk", gk), ("dv", gv)):
        assert torch.allclose(r[name], want, atol=1e-12), name


def test_visible_by_its_words():
    ok = visible(3, 5, 5, 1, 0, 1, "cpu")  # queries at positions 2, 3, 4
    assert ok.tolist() == [[True, True, True, False, False], [True, False, True, True, False],
                           [True, False, False, True, True]]
    assert not visible(4, 2, 2, -1, 0, 0, "cpu")[:2].any()  # rows in front of position 0
    assert not visible(4, 4, 2, -1, 0, 0, "cpu")[2:].any()  # rows of padding


def test_rows_that_see_nothing_and_padding_that_holds_nan():
    q, k, v, do = _qkv(1, 1, 1, 6, 4, 8, 3)
    k[:, :, 3:], v[:, :, 3:], q[:, :, 5:], do[:, :, :2] = (math.nan,) * 4
    r = window_attention(q, k, v, [3], -1, 0, 0, 0.5, do)
    assert (r["o"][0, 0, [0, 1, 5]] == 0).all() and (r["lse"][0, 0, [0, 1, 5]] == -math.inf).all()
    assert all(torch.isfinite(r[n]).all() for n in ("o", "dq", "dk", "dv"))
    assert (r["dk"][0, 0, 3:] == 0).all() and (r["dq"][0, 0, [0, 1, 5]] == 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradients_by_differences(interleaved):
    g = torch.Generator().manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, do, angle = rn(2, 3, 4, 32), rn(32), rn(2, 3, 4, 32), rn(10, 8)
    pos = torch.tensor([[0, 9, 3, 3], [1, 2, 8, 0]])
    f = lambda x, w: (norm_rope(x, w, angle.cos(), angle.sin(), pos, interleaved, 1e-3)[0] * do).sum()  # noqa: E731
    dx, _, dw, _ = norm_rope(x, w, angle.cos(), angle.sin(), pos, interleaved, 1e-3, do)
    h = 1e-5
    for _ in range(4):
        tx, tw = rn(2, 3, 4, 32), rn(32)
        diff = (f(x + h * tx, w + h * tw) - f(x - h * tx, w - h * tw)) / (2 * h)
        assert abs(diff - (dx * tx).sum() - (dw * tw).sum()) < 1e-6


def test_rotation_keeps_lengths_and_turns_by_the_difference_of_positions():
    g = torch.Generator().manual_seed(6)
    a, b = (torch.randn(1, 16, generator=g, dtype=torch.float64) for _ in range(2))
    freq = torch.rand(8, generator=g, dtype=torch.float64)
    at = lambda x, p: rotate(x, (p * freq).cos()[None], (p * freq).sin()[None], False)  # noqa: E731
    assert torch.allclose(at(a, 7).norm(), a.norm())
    assert torch.allclose((at(a, 7) * at(b, 4)).sum(), (at(a, 13) * at(b, 10)).sum())


def test_quantised_values():
    x = torch.tensor([7.0, -7.0, 0.5, -0.5, 1.5, 2.5, 3.25, 0.0] * 8)
    codes, scales = quantise(x)
    assert codes.shape == (32,) and scales.tolist() == [1.0, 1.0]
    assert dequantise(codes, scales).tolist() == [7.0, -7.0, 0.0, 0.0, 2.0, 2.0, 3.0, 0.0] * 8
    codes, scales = quantise(torch.zeros(64))
    assert (codes == 0x88).all() and (scales == 0).all()
