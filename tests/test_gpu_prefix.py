"""Attention behind a shared prefix against its 64-bit form: each sequence's keys are the prefix' and
its own, side by side."""
import math

import pytest
import torch

from token_reference import U, window_attention, within
from vision_transformer_attention_psapackqkv_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def _case(Bn, nh, nkv, nq, P, nk, d, seed=1):
    rn = lambda i, *s: _randn(seed + i, *s).to(BF16)  # noqa: E731
    return dict(q=rn(0, Bn, nh, nq, d), kp=rn(1, 1, nkv, P, d), vp=rn(2, 1, nkv, P, d), k=rn(3, Bn, nkv, nk, d),
                v=rn(4, Bn, nkv, nk, d))


def _prompts(c, lens, scale, lse=True, ws=None):
    p = B.prefix_of(c["q"], c["kp"], c["k"])
    o = torch.full_like(c["q"], 7.0)
    l = torch.full(o.shape[:3], 7.0, device="cuda") if lse else None
    if ws is None:
        ws = torch.full((B.psa_prefix_attn_workspace_size(p),), 0xFF, dtype=torch.uint8, device="cuda")
    B.psa_prefix_attn_fwd(c["q"], c["kp"], c["vp"], c["k"], c["v"], _i32(lens), o, l, ws, p, scale)
    return o, l


def _decode(c, lens, scale):
    p = B.prefix_of(c["q"], c["kp"], c["k"])
    o = torch.full_like(c["q"], 7.0)
    ws = torch.full((B.psa_prefix_attn_workspace_size(p),), 0xFF, dtype=torch.uint8, device="cuda")
    B.psa_prefix_attn_decode(c["q"], c["kp"], c["vp"], c["k"], c["v"], _i32(lens), o, ws, p, scale)
    return o


def _reference(c, lens, scale):
    """window_attention's o, lse and bounds over prefix and own keys."""
    Bn, P = c["q"].shape[0], c["kp"].shape[2]
    k, v = (torch.cat([c[a].expand(Bn, -1, -1, -1), c[b]], 2) for a, b in (("kp", "k"), ("vp", "v")))
    return window_attention(c["q"], k, v, None if lens is None else [P + max(0, n) for n in lens], -1, 0, 0, scale)


def _pad(c, lens, off):
    """What padding holds plays no part."""
    for b, n in enumerate(lens or []):
        n = max(0, n)
        c["k"][b, :, n:], c["v"][b, :, n:] = math.nan, math.inf
        if off is not None:
            c["q"][b, :, max(0, n - off):] = math.nan


HEADS = [(4, 2), (1, 1), (5, 1), (24, 3), (32, 8)]
# B, nq, P, nk, lens
PROMPTS = [(1, 1, 1, 1, None), (3, 5, 40, 9, [9, 5, 4]), (16, 3, 129, 3, [3, 2, 1, 0] * 4), (2, 77, 500, 77, [77, 30]),
           (1, 130, 256, 200, None), (3, 128, 128, 128, [128, 0, -5]), (2, 300, 1111, 300, [299, 300]), (5, 33, 2000, 64, [64, 40, 33, 31, 1])]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh,nkv", HEADS)
@pytest.mark.parametrize("Bn,nq,P,nk,lens", PROMPTS)
def test_prompts(Bn, nq, P, nk, lens, nh, nkv, d):
    c = _case(Bn, nh, nkv, nq, P, nk, d)
    scale = d ** -0.5
    r = _reference(c, lens, scale)
    valid = torch.ones(Bn, nq, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens or []):
        valid[b] = torch.arange(nq, device="cuda") + nk - nq < n
    _pad(c, lens, nk - nq)
    o, lse = _prompts(c, lens, scale)
    rows = valid[:, None, :].expand(-1, nh, -1)
    within(o[rows], r["o"][rows], r["o_tol"][rows], "o")
    # parts and own keys are joined in fp32: one term more of lse's bound
    within(lse[rows], r["lse"][rows], r["lse_tol"][rows] + 8 * U * (1 + r["lse"][rows].abs()), "lse")
    assert (o[~rows] == 0).all() and (lse[~rows] == -math.inf).all()
    again, none = _prompts(c, lens, scale, lse=False)
    assert none is None and torch.equal(o, again)


@pytest.mark.parametrize("nh,nkv", [(4, 2), (1, 1), (6, 1), (32, 8)])
@pytest.mark.parametrize("lens", [[300, 1, 0, 37, 300, 128, 129, 5, 0], [0] * 9, [-1] * 8 + [1], [0, 300] * 4 + [16], [1] * 9])
def test_row_tiles_of_padding_are_left_out(lens, nh, nkv):
    """Whatever the lengths leave of the row tiles: the same as without lengths, where there is something."""
    c, scale = _case(9, nh, nkv, 300, 2300, 300, 64, 21), 0.125
    whole, whole_lse = _prompts(c, None, scale)
    _pad(c, lens, 0)
    o, lse = _prompts(c, lens, scale)
    assert torch.equal(o, _prompts(c, lens, scale)[0])
    for b, n in enumerate(lens):
        n = max(0, n)
        assert (o[b, :, n:] == 0).all() and (lse[b, :, n:] == -math.inf).all()
        # the prefix' pieces fall differently: sums in another order, P and the result rounded alike
        assert ((o[b, :, :n].float() - whole[b, :, :n].float()).abs() <= 2.0 ** -7 * whole[b, :, :n].float().abs() + 2.0 ** -9).all()
        assert ((lse[b, :, :n] - whole_lse[b, :, :n]).abs() <= 1e-5).all()


@pytest.mark.parametrize("Bn,nq,nh,nkv,P,d", [(16, 77, 32, 8, 1000, 128), (8, 200, 32, 8, 700, 64), (16, 48, 32, 8, 1500, 128),
                                              (3, 33, 24, 3, 2000, 64), (5, 1, 8, 2, 300, 64), (16, 400, 8, 1, 260, 64)])
def test_lengths_that_are_all_full(Bn, nq, nh, nkv, P, d):
    """The rows are cut as without lengths then, and the work is dealt alike: the same bits."""
    c = _case(Bn, nh, nkv, nq, P, nq, d, 51)
    o, lse = _prompts(c, [nq] * Bn, 0.1)
    whole, whole_lse = _prompts(c, None, 0.1)
    assert torch.equal(o, whole) and torch.equal(lse, whole_lse)


@pytest.mark.parametrize("lens", [[400, 1, 0, 37] * 4, [400] * 15 + [399], [64] * 16, [130, 250] * 8, [0] * 15 + [400], list(range(10, 394, 24))])
def test_hundreds_of_row_tiles(lens):
    """More row tiles than the threads that count those in use, whichever way the rows are cut."""
    Bn, nh, nkv, nq, P, d, scale = 16, 8, 1, 400, 260, 64, 0.125
    c = _case(Bn, nh, nkv, nq, P, nq, d, 61)
    r = _reference(c, lens, scale)
    _pad(c, lens, 0)
    o, lse = _prompts(c, lens, scale)
    for b, n in enumerate(lens):
        within(o[b, :, :n], r["o"][b, :, :n], r["o_tol"][b, :, :n], "o")
        want = r["lse"][b, :, :n]
        within(lse[b, :, :n], want, r["lse_tol"][b, :, :n] + 8 * U * (1 + want.abs()), "lse")
        assert (o[b, :, n:] == 0).all() and (lse[b, :, n:] == -math.inf).all()


@pytest.mark.parametrize("nh,nkv", [(4, 2), (1, 1)])
@pytest.mark.parametrize("Bn,nq,nk", [(257, 3, 5), (700, 7, 7)])
def test_many_prompts(Bn, nq, nk, nh, nkv):
    """More sequences than the lengths that the kernel keeps at hand; a length in ten is of padding alone."""
    c, scale = _case(Bn, nh, nkv, nq, 300, nk, 64, 71), 0.125
    lens = [(b * 7919) % (nk + 1) if b % 10 else -b for b in range(Bn)]
    r = _reference(c, lens, scale)
    valid = (torch.arange(nq, device="cuda") + nk - nq)[None] < _i32(lens)[:, None]
    _pad(c, lens, nk - nq)
    o, lse = _prompts(c, lens, scale)
    rows = valid[:, None, :].expand(-1, nh, -1)
    within(o[rows], r["o"][rows], r["o_tol"][rows], "o")
    within(lse[rows], r["lse"][rows], r["lse_tol"][rows] + 8 * U * (1 + r["lse"][rows].abs()), "lse")
    assert (o[~rows] == 0).all() and (lse[~rows] == -math.inf).all()


# B, P, rows, lens
STEPS = [(1, 1, 1, [1]), (2, 40, 9, [0, 9]), (4, 128, 30, [30, 1, 0, -1]), (7, 129, 200, [200, 0, 17, 16, -3, 15, 300]),
         (33, 1000, 50, [50, 49, 3] * 11), (3, 4500, 700, [700, 350, 1]), (130, 300, 20, [20, -1, 7, 0, 11] * 26), (1, 9000, 5, [5])]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh,nkv", HEADS + [(160, 1)])
@pytest.mark.parametrize("Bn,P,rows,lens", STEPS)
def test_single_tokens(Bn, P, rows, lens, nh, nkv, d):
    if Bn * nh > 1100:
        nh, nkv = max(1, 1024 // Bn // nkv) * nkv, nkv
    c = _case(Bn, nh, nkv, 1, P, rows, d)
    scale = d ** -0.5
    ref, tol = (torch.zeros(c["q"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for n in sorted(set(lens)):
        at = [b for b, x in enumerate(lens) if x == n]
        if n < 0:
            continue
        m = min(n, rows)
        # the query stands at the last position: behind the prefix, or on its last one's place
        sub = dict(c, q=c["q"][at], k=c["k"][at][:, :, :m], v=c["v"][at][:, :, :m])
        k, v = (torch.cat([sub[a].expand(len(at), -1, -1, -1), sub[b]], 2) for a, b in (("kp", "k"), ("vp", "v")))
        r = window_attention(sub["q"], k, v, None, -1, 0, 0, scale)
        ref[at], tol[at] = r["o"], r["o_tol"]
    _pad(c, lens, None)
    o = _decode(c, lens, scale)
    within(o, ref, tol, "o")
    assert torch.equal(o, _decode(c, lens, scale))


@pytest.mark.parametrize("rows", [15, 16, 17, 20, 31, 32])
def test_single_tokens_over_short_caches(rows):
    c, lens, scale = _case(5, 6, 2, 1, 130, rows, 64, 81), [rows, rows - 1, 1, 16, 17], 0.125
    o = _decode(c, lens, scale)
    for b, n in enumerate(lens):
        k, v = (torch.cat([c[a], c[x][b:b + 1, :, :min(n, rows)]], 2) for a, x in (("kp", "k"), ("vp", "v")))
        r = window_attention(c["q"][b:b + 1], k, v, None, -1, 0, 0, scale)
        within(o[b:b + 1], r["o"], r["o_tol"], b)


def test_strided_views_and_two_calls_at_once():
    """A packed projection's queries, a prefix in the first rows of a longer cache, two streams with a
    workspace each."""
    Bn, nh, nkv, nq, P, d, scale = 6, 8, 2, 20, 700, 128, 0.1
    packed = _randn(5, Bn, nq, nh + 2 * nkv, d).to(BF16).transpose(1, 2)
    long = _randn(6, 1, 1000, 2 * nkv, d).to(BF16).transpose(1, 2)
    c = dict(q=packed[:, :nh], k=packed[:, nh:nh + nkv], v=packed[:, nh + nkv:], kp=long[:, :nkv, :P], vp=long[:, nkv:, :P])
    lens = [20, 1, 7, 20, 13, 0]
    want = _prompts({n: t.contiguous() for n, t in c.items()}, lens, scale)
    one = dict(c, q=c["q"][:, :, :1])
    want1 = _decode({n: t.contiguous() for n, t in one.items()}, lens, scale)
    torch.cuda.synchronize()
    outs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        with torch.cuda.stream(s):
            p, p1 = B.prefix_of(c["q"], c["kp"], c["k"]), B.prefix_of(one["q"], c["kp"], c["k"])
            out = torch.full((Bn, nq, nh, d), 7.0, dtype=BF16, device="cuda").transpose(1, 2)
            out1, lse = torch.full_like(out[:, :, :1], 7.0), torch.empty(Bn, nh, nq, device="cuda")
            ws = torch.empty(B.psa_prefix_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
            ws1 = torch.empty(B.psa_prefix_attn_workspace_size(p1), dtype=torch.uint8, device="cuda")
            for _ in range(20):
                B.psa_prefix_attn_fwd(c["q"], c["kp"], c["vp"], c["k"], c["v"], _i32(lens), out, lse, ws, p, scale)
                B.psa_prefix_attn_decode(one["q"], c["kp"], c["vp"], c["k"], c["v"], _i32(lens), out1, ws1, p1, scale)
            outs.append((out, lse, out1))
    torch.cuda.synchronize()
    for out, lse, out1 in outs:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(out1, want1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh,nkv", [(4, 2), (40, 2)])
def test_maxima_that_move_between_parts_and_tiles(nh, nkv, d):
    """Scores that rise or fall by far more than 2^8 along the prefix, into the own keys."""
    P, Bn, scale = 3000, 3, 0.5
    u = _randn(41, d)
    u /= u.norm()
    c = _case(Bn, nh, nkv, 1, P, 40, d, 7)
    c["q"] = (_randn(42, Bn, nh, 1, d) * 0.3 + torch.tensor([8.0, -8.0, 0.0], device="cuda")[:, None, None, None] * u).to(BF16)
    c["kp"] = (0.3 * _randn(43, 1, nkv, P, d) + torch.linspace(-20, 20, P, device="cuda")[:, None] * u).to(BF16)
    lens = [40, 3, 0]
    for b, n in enumerate(lens):
        sub = [torch.cat([c[a], c[x][b:b + 1, :, :n]], 2) for a, x in (("kp", "k"), ("vp", "v"))]
        r = window_attention(c["q"][b:b + 1], *sub, None, -1, 0, 0, scale)
        within(_decode(c, lens, scale)[b:b + 1], r["o"], r["o_tol"], b)


def test_a_nan_that_is_seen_stays_one():
    c = _case(3, 4, 2, 1, 600, 50, 64, 9)
    clean = _decode(c, [50, 20, 0], 0.2)
    c["kp"][0, 1, 300, 5] = math.nan
    o = _decode(c, [50, 20, 0], 0.2)
    assert o[:, 2:].isnan().all() and torch.equal(o[:, :2], clean[:, :2])
    c["kp"][0, 1, 300, 5] = 0
    clean = _decode(c, [50, 20, 0], 0.2)
    c["k"][0, 0, 7, 1] = math.nan
    o = _decode(c, [50, 20, 0], 0.2)
    assert o[0, :2].isnan().all() and torch.equal(o[0, 2:], clean[0, 2:]) and torch.equal(o[1:], clean[1:])
    many = _case(2, 4, 2, 40, 600, 40, 64, 9)
    want = _prompts(many, None, 0.2)
    many["q"][1, 3, 17, 0] = math.nan
    o, lse = _prompts(many, None, 0.2)
    assert o[1, 3, 17].isnan().all() and lse[1, 3, 17].isnan()
    keep = torch.ones(2, 4, 40, dtype=torch.bool, device="cuda")
    keep[1, 3, 17] = False
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


def test_replayed():
    c, lens = _case(5, 8, 2, 1, 900, 64, 128, 11), [64, 3, 0, -1, 20]
    want = _decode(c, lens, 0.1)
    p, o, l = B.prefix_of(c["q"], c["kp"], c["k"]), torch.empty_like(c["q"]), _i32([1] * 5)
    ws = torch.empty(B.psa_prefix_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        B.psa_prefix_attn_decode(c["q"], c["kp"], c["vp"], c["k"], c["v"], l, o, ws, p, 0.1)
    l.copy_(_i32(lens))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)
