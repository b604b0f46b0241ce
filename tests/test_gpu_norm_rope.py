"""psa_qk_norm_rope_fwd / _bwd against their 64-bit form."""
import pytest
import torch

from token_reference import norm_rope, within
from vision_transformer_attention_psapackqkv_gb300 import binding as B

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _case(Bn, nh, nkv, N, d, rot, dtype, seed, max_pos=64, packed=False, positions=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if packed:  # views of a projection's output [B, N, heads of q | k | v, d]
        x = rn(Bn, N, nh + 2 * nkv, d).to(dtype).transpose(1, 2)
        q, k = x[:, :nh], x[:, nh:nh + nkv]
    else:
        q, k = rn(Bn, nh, N, d).to(dtype), rn(Bn, nkv, N, d).to(dtype)
    angle = rn(max_pos, rot // 2) * 3
    cos, sin = (angle.cos().contiguous(), angle.sin().contiguous()) if rot else (None, None)
    pos = torch.randint(0, max_pos, (Bn, N), generator=g, device="cuda", dtype=torch.int32) if positions else None
    return dict(q=q, k=k, wq=1 + 0.3 * rn(d), wk=1 + 0.3 * rn(d), cos=cos, sin=sin, pos=pos,
                gq=rn(Bn, nh, N, d).to(dtype), gk=rn(Bn, nkv, N, d).to(dtype))


def _positions(c):
    Bn, _, N, _ = c["q"].shape
    return c["pos"] if c["pos"] is not None else torch.arange(N, device="cuda").expand(Bn, -1)


def _forward(c, inter, eps=1e-5):
    p = B.norm_rope_of(c["q"], c["k"], c["cos"], eps, inter)
    q, k = (torch.full(c[n].shape, 7.0, dtype=c[n].dtype, device="cuda") for n in "qk")
    B.psa_qk_norm_rope_fwd(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], c["pos"], q, k, p)
    return q, k


def _backward(c, inter, eps=1e-5):
    p = B.norm_rope_of(c["q"], c["k"], c["cos"], eps, inter)
    new = lambda t: torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda")  # noqa: E731
    dq, dk, dwq, dwk = new(c["q"]), new(c["k"]), new(c["cos"][0].new_zeros(p.head_dim) if c["cos"] is not None
                                                     else torch.zeros(p.head_dim, device="cuda")), \
        torch.full((p.head_dim,), 7.0, device="cuda")
    ws = torch.full((B.psa_qk_norm_rope_bwd_workspace_size(p),), 0xAB, dtype=torch.uint8, device="cuda")
    B.psa_qk_norm_rope_bwd(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], c["pos"], c["gq"], c["gk"], dq, dk,
                           dwq, dwk, ws, p)
    return dq, dk, dwq, dwk


CASES = [(1, 1, 1, 1, 64, 64), (2, 4, 2, 7, 128, 128), (1, 5, 1, 33, 64, 32), (3, 3, 3, 17, 128, 64),
         (2, 8, 2, 300, 32, 32), (1, 2, 1, 5, 128, 16), (2, 2, 1, 9, 64, 0), (64, 32, 8, 1, 128, 128),
         (1, 40, 8, 1300, 128, 96)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Bn,nh,nkv,N,d,rot", CASES)
def test_forward_and_backward(Bn, nh, nkv, N, d, rot, interleaved, dtype):
    c = _case(Bn, nh, nkv, N, d, rot, dtype, N + d + rot, packed=N % 2 == 1)
    eps = 2.0 ** -16  # the same number in fp32
    q, k = _forward(c, interleaved, eps)
    dq, dk, dwq, dwk = _backward(c, interleaved, eps)
    for x, w, y, g, dx, dw, what in ((c["q"], c["wq"], q, c["gq"], dq, dwq, "q"),
                                     (c["k"], c["wk"], k, c["gk"], dk, dwk, "k")):
        within(y, *norm_rope(x, w, c["cos"], c["sin"], _positions(c), interleaved, eps, half=HALF[dtype]), what)
        rdx, tdx, rdw, tdw = norm_rope(x, w, c["cos"], c["sin"], _positions(c), interleaved, eps, g, HALF[dtype])
        within(dx, rdx, tdx, "d" + what)
        within(dw, rdw, tdw, "dw" + what)


def test_without_weights_and_positions():
    c = _case(2, 4, 2, 40, 64, 64, torch.bfloat16, 3, positions=False)
    c["wq"] = c["wk"] = None
    eps = 2.0 ** -16
    q, k = _forward(c, False, eps)
    within(q, *norm_rope(c["q"], None, c["cos"], c["sin"], _positions(c), False, eps), "q")
    p = B.norm_rope_of(c["q"], c["k"], c["cos"], eps)
    dq, dk = torch.empty_like(c["q"]), torch.empty_like(c["k"])
    ws = torch.empty(B.psa_qk_norm_rope_bwd_workspace_size(p), dtype=torch.uint8, device="cuda")
    B.psa_qk_norm_rope_bwd(c["q"], c["k"], None, None, c["cos"], c["sin"], None, c["gq"], c["gk"], dq, dk, None, None,
                           ws, p)
    rdx, tdx, _, _ = norm_rope(c["q"], None, c["cos"], c["sin"], _positions(c), False, eps, c["gq"])
    within(dq, rdx, tdx, "dq")


def test_padding_is_left_as_it_was_and_gets_no_gradient():
    c = _case(2, 4, 2, 12, 64, 64, torch.bfloat16, 4)
    pad = torch.zeros(2, 12, dtype=torch.bool, device="cuda")
    pad[0, 3:], pad[1, 7] = True, True
    whole = _forward(c, False), _backward(c, False)
    c["pos"][pad] = -1
    c["pos"][1, 7] = 64  # the first position past the table
    for n in ("q", "k", "gq", "gk"):
        c[n].transpose(1, 2)[pad] = float("nan")
    q, k = _forward(c, False)
    dq, dk, dwq, dwk = _backward(c, False)
    for y, was in ((q, whole[0][0]), (k, whole[0][1])):
        assert (y.transpose(1, 2)[pad] == 7.0).all()
        assert torch.equal(y.transpose(1, 2)[~pad], was.transpose(1, 2)[~pad])
    for dx, was in ((dq, whole[1][0]), (dk, whole[1][1])):
        assert (dx.transpose(1, 2)[pad] == 0).all()
        assert torch.equal(dx.transpose(1, 2)[~pad], was.transpose(1, 2)[~pad])
    assert torch.isfinite(dwq).all() and torch.isfinite(dwk).all()


def test_in_place_and_reruns_are_bitwise_identical():
    c = _case(2, 8, 2, 500, 128, 128, torch.bfloat16, 5, packed=True)
    q, k = _forward(c, False)
    first, second = _backward(c, False), _backward(c, False)
    assert all(torch.equal(x, y) for x, y in zip(first, second))
    p = B.norm_rope_of(c["q"], c["k"], c["cos"], 1e-5)
    ws = torch.empty(B.psa_qk_norm_rope_bwd_workspace_size(p), dtype=torch.uint8, device="cuda")
    dwq, dwk = torch.empty(128, device="cuda"), torch.empty(128, device="cuda")
    gq, gk = c["gq"].clone(), c["gk"].clone()
    B.psa_qk_norm_rope_bwd(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], c["pos"], gq, gk, gq, gk, dwq, dwk,
                           ws, p)
    assert torch.equal(gq, first[0]) and torch.equal(gk, first[1]) and torch.equal(dwq, first[2])
    B.psa_qk_norm_rope_fwd(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], c["pos"], c["q"], c["k"], p)
    assert torch.equal(c["q"], q) and torch.equal(c["k"], k)


def test_on_another_stream():
    c = _case(1, 8, 2, 64, 128, 128, torch.bfloat16, 6)
    want = _forward(c, True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    p = B.norm_rope_of(c["q"], c["k"], c["cos"], 1e-5, True)
    q, k = torch.empty_like(c["q"]), torch.empty_like(c["k"])
    B.psa_qk_norm_rope_fwd(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], c["pos"], q, k, p, s)
    s.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_eps_zero_with_odd_heads_and_padding(dtype):
    """Without eps, rows that are not there (past the last head, the last token, padding) have no
    norm to divide by: they must not reach the weights' gradients."""
    c = _case(2, 5, 1, 7, 64, 32, dtype, 9)
    pad = torch.zeros(2, 7, dtype=torch.bool, device="cuda")
    pad[0, 2], pad[1, 5:] = True, True
    for n in ("gq", "gk"):
        c[n].transpose(1, 2)[pad] = 0
    dq, dk, dwq, dwk = _backward(c, False, 0.0)
    for x, w, g, dx, dw, what in ((c["q"], c["wq"], c["gq"], dq, dwq, "q"), (c["k"], c["wk"], c["gk"], dk, dwk, "k")):
        rdx, tdx, rdw, tdw = norm_rope(x, w, c["cos"], c["sin"], c["pos"], False, 0.0, g, HALF[dtype])
        within(dx, rdx, tdx, "d" + what)
        within(dw, rdw, tdw, "dw" + what)
    c["pos"][pad] = -1
    padded = _backward(c, False, 0.0)
    for dx, was in ((padded[0], dq), (padded[1], dk)):
        assert (dx.transpose(1, 2)[pad] == 0).all()
        assert torch.equal(dx.transpose(1, 2)[~pad], was.transpose(1, 2)[~pad])
    assert torch.equal(padded[2], dwq) and torch.equal(padded[3], dwk)


# tokens and heads at which the forward takes 1, 4 and 8 heads a group, by type, the backward 4 and 8
# (neither divides 23 or 3) and, with very many heads, 9
MANY = [(1, 23, 3, 1400, 128, 96), (1, 23, 3, 2900, 128, 64), (1, 23, 3, 6100, 128, 128), (2, 23, 3, 6100, 64, 32),
        (1, 2501, 3, 2, 64, 32)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Bn,nh,nkv,N,d,rot", MANY)
def test_many_tokens_of_heads_that_fill_no_group(Bn, nh, nkv, N, d, rot, interleaved, dtype):
    """Views of a packed projection with padding among the tokens, then in place."""
    c = _case(Bn, nh, nkv, N, d, rot, dtype, N + d, packed=True)
    pad = torch.rand(Bn, N, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") < 0.1
    eps = 2.0 ** -16
    real = c["pos"].clone()
    c["pos"][pad] = torch.where(torch.arange(int(pad.sum()), device="cuda") % 2 == 0, -3, 64).int()
    for n in ("gq", "gk"):
        c[n].transpose(1, 2)[pad] = 0  # what the reference sums; the kernels do not read them
    q, k = _forward(c, interleaved, eps)
    dq, dk, dwq, dwk = _backward(c, interleaved, eps)
    for x, w, y, g, dx, dw, what in ((c["q"], c["wq"], q, c["gq"], dq, dwq, "q"),
                                     (c["k"], c["wk"], k, c["gk"], dk, dwk, "k")):
        ref, tol = norm_rope(x, w, c["cos"], c["sin"], real, interleaved, eps, half=HALF[dtype])
        within(y.transpose(1, 2)[~pad], ref.transpose(1, 2)[~pad], tol.transpose(1, 2)[~pad], what)
        assert (y.transpose(1, 2)[pad] == 7.0).all()
        rdx, tdx, rdw, tdw = norm_rope(x, w, c["cos"], c["sin"], real, interleaved, eps, g, HALF[dtype])
        within(dx, rdx, tdx, "d" + what)
        assert (dx.transpose(1, 2)[pad] == 0).all()
        within(dw, rdw, tdw, "dw" + what)
    # the same tokens a few at a time
    few = {n: c[n][:, :, :9] for n in "qk"} | {n: c[n] for n in ("wq", "wk", "cos", "sin")} | \
        {"pos": c["pos"][:, :9].contiguous()}
    for y, was in zip(_forward(few, interleaved, eps), (q, k)):
        assert torch.equal(y, was[:, :, :9])
    was = c["q"].clone(), c["k"].clone()
    p = B.norm_rope_of(c["q"], c["k"], c["cos"], eps, interleaved)
    B.psa_qk_norm_rope_fwd(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], c["pos"], c["q"], c["k"], p)
    for y, x, before in ((q, c["q"], was[0]), (k, c["k"], was[1])):
        assert torch.equal(x.transpose(1, 2)[~pad], y.transpose(1, 2)[~pad])
        assert torch.equal(x.transpose(1, 2)[pad], before.transpose(1, 2)[pad])
