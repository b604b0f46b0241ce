"""psa_qk_norm_rope_axes_fwd / _bwd: the one-axis 64-bit form on each token's own angles."""
import itertools

import pytest
import torch

from token_reference import HALF, U, norm_rope, rotate, within
from vision_transformer_attention_psapackqkv_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 2.0 ** -16  # the same number in fp32


def _case(Bn, nh, nkv, N, d, sections, dtype, seed, grid=None, max_pos=50, packed=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rn(Bn, N, nh + 2 * nkv, d).to(dtype).transpose(1, 2)
    q, k = x[:, :nh], x[:, nh:nh + nkv]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    half = sum(sections)
    angle = rn(max_pos, half) * 3
    cos, sin = (angle.cos().contiguous(), angle.sin().contiguous()) if half else (None, None)
    pos = None
    if grid is None:
        pos = torch.randint(0, max_pos, (len(sections), Bn, N), generator=g, device="cuda", dtype=torch.int32)
    return dict(q=q, k=k, wq=1 + 0.3 * rn(d), wk=1 + 0.3 * rn(d), cos=cos, sin=sin, pos=pos, sections=sections, grid=grid,
                gq=rn(Bn, nh, N, d).to(dtype), gk=rn(Bn, nkv, N, d).to(dtype))


def _by_hand(sections, alternate):
    """The axis of each pair: sections in turn, or round after round one pair of every axis that has some."""
    left, out = list(sections), []
    while sum(left):
        for a in range(len(left)):
            take = left[a] if not alternate else min(1, left[a])
            out += [a] * take
            left[a] -= take
    return out


def _own_tables(c, alternate):
    """Each token's angles: tables [B N, pairs] and positions into them."""
    Bn, _, N, _ = c["q"].shape
    own = torch.arange(Bn * N, device="cuda").view(Bn, N)
    if c["cos"] is None:
        return None, None, own
    if c["pos"] is None:
        cells = torch.tensor(list(itertools.product(*map(range, c["grid"]))), device="cuda").T  # [axes, N]
        at = cells[:, None].expand(-1, Bn, -1)
    else:
        at = c["pos"].long()
    col = [(t[:, i][at[a]]).flatten() for t in (c["cos"], c["sin"]) for i, a in enumerate(_by_hand(c["sections"], alternate))]
    half = len(col) // 2
    return torch.stack(col[:half], 1), torch.stack(col[half:], 1), own


def _problem(c, inter, alternate, normalize=True, eps=EPS):
    return B.rope_axes_of(c["q"], c["k"], c["cos"], c["sections"], eps, inter, alternate, c["grid"], normalize)


def _forward(c, inter, alternate, normalize=True, eps=EPS):
    q, k = (torch.full(c[n].shape, 7.0, dtype=c[n].dtype, device="cuda") for n in "qk")
    B.psa_qk_norm_rope_axes_fwd(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], c["pos"], q, k,
                                _problem(c, inter, alternate, normalize, eps))
    return q, k


def _backward(c, inter, alternate, normalize=True, weights=True, eps=EPS):
    p = _problem(c, inter, alternate, normalize, eps)
    d = p.rope.head_dim
    dq, dk = (torch.full(c[n].shape, 7.0, dtype=c[n].dtype, device="cuda") for n in "qk")
    dwq, dwk = (torch.full((d,), 7.0, device="cuda") for _ in range(2)) if weights else (None, None)
    ws = torch.full((B.psa_qk_norm_rope_bwd_workspace_size(p.rope),), 0xAB, dtype=torch.uint8, device="cuda")
    B.psa_qk_norm_rope_axes_bwd(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], c["pos"], c["gq"], c["gk"], dq, dk,
                                dwq, dwk, ws, p)
    return dq, dk, dwq, dwk


# B, nh, nkv, N, d, sections, grid; head counts and lengths at which a group takes one, four, eight heads
CASES = [(1, 1, 1, 1, 64, (32,), None), (2, 4, 2, 7, 128, (16, 24, 24), None), (1, 5, 1, 33, 64, (15, 1), None),
         (3, 3, 3, 24, 128, (10, 11, 11), (2, 3, 4)), (2, 8, 2, 300, 32, (8, 8), (15, 20)), (1, 2, 1, 50, 128, (0, 3, 5), (1, 50, 1)),
         (2, 2, 1, 9, 64, (0, 0), (3, 3)), (1, 4, 1, 210, 64, (8, 8, 8, 8), (2, 3, 5, 7)), (64, 32, 8, 1, 128, (16, 24, 24), None),
         (1, 40, 8, 1300, 128, (16, 32), None), (1, 23, 3, 6100, 128, (64, 0), None), (2, 23, 3, 2450, 64, (2, 7, 7), (49, 50, 1))]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("alternate", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("Bn,nh,nkv,N,d,sections,grid", CASES)
def test_forward_and_backward(Bn, nh, nkv, N, d, sections, grid, inter, alternate, dtype):
    c = _case(Bn, nh, nkv, N, d, sections, dtype, N + d, grid, packed=N % 2 == 1)
    cos, sin, own = _own_tables(c, alternate)
    q, k = _forward(c, inter, alternate)
    dq, dk, dwq, dwk = _backward(c, inter, alternate)
    for x, w, y, g, dx, dw, what in ((c["q"], c["wq"], q, c["gq"], dq, dwq, "q"), (c["k"], c["wk"], k, c["gk"], dk, dwk, "k")):
        within(y, *norm_rope(x, w, cos, sin, own, inter, EPS, half=HALF[dtype]), what)
        rdx, tdx, rdw, tdw = norm_rope(x, w, cos, sin, own, inter, EPS, g, HALF[dtype])
        within(dx, rdx, tdx, "d" + what)
        within(dw, rdw, tdw, "dw" + what)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("Bn,nh,nkv,N,d,sections,grid", [CASES[1], CASES[3], CASES[4], CASES[9]])
def test_without_norms(Bn, nh, nkv, N, d, sections, grid, weighted, inter, dtype):
    """y = R (w o x), dx = w o R^T g, dw = sum of x o R^T g; without weights' gradients x is not read."""
    c = _case(Bn, nh, nkv, N, d, sections, dtype, N + d + 1, grid, packed=True)
    if not weighted:
        c["wq"] = c["wk"] = None
    cos, sin, own = _own_tables(c, True)
    co, si = cos.double()[own][:, None], sin.double()[own][:, None]
    # The bound goes by |c a| + |s b|, as c a - s b rounds twice on numbers up to that, w o x and w o c once
    # more each.  Of a rotation of magnitudes by -|s| and by +|s| one has that sum in the pair's first
    # channel, the other in its second, and the remaining two (|c b| - |s a| and |c a| - |s b|) count with
    # their magnitude: with their sign, they took |s a| out of the second channel's bound again.
    mags = lambda t: rotate(t.abs(), co.abs(), -si.abs(), inter).abs() + rotate(t.abs(), co.abs(), si.abs(), inter).abs()  # noqa: E731
    q, k = _forward(c, inter, True, False)
    dq, dk, dwq, dwk = _backward(c, inter, True, False)
    for x, w, y, g, dx, dw, what in ((c["q"], c["wq"], q, c["gq"], dq, dwq, "q"), (c["k"], c["wk"], k, c["gk"], dk, dwk, "k")):
        wd = torch.ones(d, dtype=torch.float64, device="cuda") if w is None else w.double()
        ref = rotate(x.double() * wd, co, si, inter)
        within(y, ref, HALF[dtype] * ref.abs() + 8 * U * mags(x.double() * wd), what)
        gy, gm = rotate(g.double(), co, si, inter, back=True), mags(g.double())
        within(dx, gy * wd, HALF[dtype] * (gy * wd).abs() + 8 * U * gm * wd.abs(), "d" + what)
        rdw, size = (gy * x.double()).sum((0, 1, 2)), (gm * x.double().abs()).sum((0, 1, 2))
        within(dw, rdw, (8 + x.shape[0] * x.shape[1] * N + 64) * U * size, "dw" + what)
    c["q"], c["k"] = torch.full_like(c["q"], float("nan")), torch.full_like(c["k"], float("inf"))
    again = _backward(c, inter, True, False, weights=False)
    assert torch.equal(again[0], dq) and torch.equal(again[1], dk)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
def test_one_axis_is_the_plain_rotation_bit_for_bit(inter, dtype):
    c = _case(2, 8, 2, 700, 128, (48,), dtype, 3, packed=True)
    p = B.norm_rope_of(c["q"], c["k"], c["cos"], EPS, inter)
    q, k, dq, dk = (torch.empty(c[n].shape, dtype=dtype, device="cuda") for n in "qkqk")
    dwq, dwk = torch.empty(128, device="cuda"), torch.empty(128, device="cuda")
    ws = torch.empty(B.psa_qk_norm_rope_bwd_workspace_size(p), dtype=torch.uint8, device="cuda")
    args = (c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], c["pos"][0].contiguous())
    B.psa_qk_norm_rope_fwd(*args, q, k, p)
    B.psa_qk_norm_rope_bwd(*args, c["gq"], c["gk"], dq, dk, dwq, dwk, ws, p)
    want = (q, k, dq, dk, dwq, dwk)
    # as one axis, and as three that stand at the same place
    for sections in ((48,), (13, 30, 5)):
        three = dict(c, sections=sections, pos=c["pos"][:1].repeat(len(sections), 1, 1))
        got = _forward(three, inter, True) + _backward(three, inter, True)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_padding_on_any_axis():
    c = _case(2, 4, 2, 30, 64, (8, 12, 12), BF16, 4)
    whole = _forward(c, False, False) + _backward(c, False, False)
    pad = torch.zeros(2, 30, dtype=torch.bool, device="cuda")
    for i, (b, n, bad) in enumerate([(0, 3, -1), (0, 9, 50), (1, 0, -2 ** 31), (1, 17, 2 ** 31 - 1), (1, 29, -1)]):
        c["pos"][i % 3, b, n] = bad
        pad[b, n] = True
    for n in ("q", "k", "gq", "gk"):
        c[n].transpose(1, 2)[pad] = float("nan")
    got = _forward(c, False, False) + _backward(c, False, False)
    for i, (x, was) in enumerate(zip(got[:4], whole[:4])):
        assert (x.transpose(1, 2)[pad] == (7.0 if i < 2 else 0.0)).all()
        assert torch.equal(x.transpose(1, 2)[~pad], was.transpose(1, 2)[~pad])
    assert torch.isfinite(got[4]).all() and torch.isfinite(got[5]).all()


def test_in_place_on_another_stream_and_replayed():
    c = _case(2, 8, 2, 600, 128, (16, 24, 24), BF16, 5, grid=(6, 10, 10), packed=True)
    want = _forward(c, False, True)
    first, second = _backward(c, False, True), _backward(c, False, True)
    assert all(torch.equal(x, y) for x, y in zip(first, second))
    p = _problem(c, False, True)
    gq, gk = c["gq"].clone(), c["gk"].clone()
    dwq, dwk = torch.empty(128, device="cuda"), torch.empty(128, device="cuda")
    ws = torch.empty(B.psa_qk_norm_rope_bwd_workspace_size(p.rope), dtype=torch.uint8, device="cuda")
    args = (c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.psa_qk_norm_rope_axes_bwd(*args, gq, gk, gq, gk, dwq, dwk, ws, p)
        B.psa_qk_norm_rope_axes_fwd(*args, c["q"], c["k"], p)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip((gq, gk, dwq, dwk, c["q"], c["k"]), first + want):
        assert torch.equal(x, y)


def test_gradients_against_differences():
    """<g, y(x + h e) - y(x - h e)> / 2 h in fp32, against the backward's <dx, e>."""
    c = _case(1, 2, 1, 60, 64, (8, 12, 12), F32, 6, grid=(3, 4, 5))
    dq, dk, dwq, dwk = _backward(c, False, True)
    h = 2.0 ** -6
    for name, dx in (("q", dq), ("k", dk), ("wq", dwq), ("wk", dwk)):
        e = torch.randn(c[name].shape, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")
        out = []
        for sign in (1, -1):
            q, k = _forward(dict(c, **{name: c[name] + sign * h * e}), False, True)
            out.append((q.double() * c["gq"].double()).sum() + (k.double() * c["gk"].double()).sum())
        got, want = (out[0] - out[1]) / (2 * h), (dx.double() * e.double()).sum()
        # the rows' third derivative times h^2 / 6 and the forward's roundings over 2 h: both far below 1 % of
        # the derivative's own spread, |dx| |e| / sqrt(n) per entry
        assert abs(got - want) < 0.01 * dx.double().norm() * e.double().norm() / e.numel() ** 0.5, (name, got, want)


def test_refusals_of_the_binding():
    c = _case(1, 2, 1, 12, 64, (8, 12, 12), BF16, 8)
    for sections, grid in (((8, 12), None), ((8, 12, 13), None), ((8, 8, 8, 4, 4), None), ((40, -8), None),
                           ((8, 12, 12), (2, 6)), ((8, 12, 12), (2, 3, 3)), ((8, 12, 12), (12, 1, 0))):
        with pytest.raises(ValueError):
            B.rope_axes_of(c["q"], c["k"], c["cos"], sections, grid=grid)
    with pytest.raises(B.PsaError):  # neither positions nor a grid
        _forward(dict(c, pos=None), False, False)
    with pytest.raises(ValueError):
        _forward(dict(c, pos=c["pos"][0]), False, False)
