"""The operators of images, shared prompts and thinned caches run together, as they are used: many
questions about one video, a cache that is kept at its length, and a training step over two axes."""
import math

import pytest
import torch

from token_reference import norm_rope, window_attention, within
from vision_transformer_attention_psapackqkv_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPS = 2.0 ** -18


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(rows, pairs):
    freq = 1e4 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    return angle.cos().float().contiguous(), angle.sin().float().contiguous()


def _turn(x, weights, cos, sin, positions=None, grid=None):
    """q and k of a projection's output [B, N, heads of q | k | v, d], normed and rotated; v as it is."""
    q, k, v = x
    p = B.rope_axes_of(q, k, cos, (16, 24, 24), EPS, alternate=True, grid=grid)
    oq, ok = (torch.empty(t.shape, dtype=BF16, device="cuda") for t in (q, k))
    B.psa_qk_norm_rope_axes_fwd(q, k, *weights, cos, sin, positions, oq, ok, p)
    return oq, ok, v


def _split(packed, nh, nkv):
    x = packed.transpose(1, 2)
    return x[:, :nh], x[:, nh:nh + nkv], x[:, nh + nkv:]


def test_questions_about_a_video():
    """The video's tokens go through the layer once; a batch of questions is read behind them, then answered
    token by token from one captured graph, each step through rotation, cache and attention."""
    nh, nkv, d, Bn, longest, steps, scale = 8, 2, 128, 5, 20, 6, 128 ** -0.5
    grid = (3, 8, 9)
    P = math.prod(grid)
    cos, sin = _tables(256, 64)
    weights = 1 + 0.1 * _randn(1, d), 1 + 0.1 * _randn(2, d)
    # the video, in raster order
    _, kp, vp = _turn(_split(_randn(3, 1, P, nh + 2 * nkv, d).to(BF16), nh, nkv), weights, cos, sin, grid=grid)
    # the questions: text stands at one position on all axes, behind the video's largest
    lens, rows = [20, 7, 13, 1, 20], longest + steps
    packed = _randn(4, Bn, rows, nh + 2 * nkv, d).to(BF16)
    where = (max(grid) + torch.arange(rows, device="cuda")).int().expand(3, Bn, -1)
    q, k, v = _turn(_split(packed, nh, nkv), weights, cos, sin, where.contiguous())
    for x, w, y, heads in ((packed.transpose(1, 2)[:, :nh], weights[0], q, nh), (packed.transpose(1, 2)[:, nh:nh + nkv], weights[1], k, nkv)):
        within(y, *norm_rope(x, w, cos, sin, where[0], False, EPS), "rotation of text")
    o, lse = torch.empty(Bn, nh, longest, d, dtype=BF16, device="cuda"), torch.empty(Bn, nh, longest, device="cuda")
    p = B.prefix_of(q[:, :, :longest], kp, k[:, :, :longest])
    ws = torch.empty(B.psa_prefix_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
    B.psa_prefix_attn_fwd(q[:, :, :longest], kp, vp, k[:, :, :longest], v[:, :, :longest], _i32(lens), o, lse, ws, p, scale)
    both = [torch.cat([a.expand(Bn, -1, -1, -1), b], 2) for a, b in ((kp, k), (vp, v))]

    def check(out, b, i):
        r = window_attention(q[b:b + 1, :, i:i + 1], *(t[b:b + 1, :, :P + i + 1] for t in both), None, -1, 0, 0, scale)
        within(out, r["o"], r["o_tol"], (b, i))

    for b, n in enumerate(lens):
        assert (o[b, :, n:] == 0).all()
        check(o[b:b + 1, :, n - 1:n], b, n - 1)

    # answers: question b's next token is its row lens[b] + step of `packed`
    cache = [torch.full((Bn, nkv, rows, d), math.nan, dtype=BF16, device="cuda") for _ in range(2)]
    B.psa_kv_append(k[:, :, :longest].contiguous(), v[:, :, :longest].contiguous(), _i32([0] * Bn), _i32(lens), *cache)
    x = torch.empty(Bn, 1, nh + 2 * nkv, d, dtype=BF16, device="cuda")
    at, now = torch.zeros(3, Bn, 1, dtype=torch.int32, device="cuda"), _i32(lens)
    length, out = now + 1, torch.empty(Bn, nh, 1, d, dtype=BF16, device="cuda")
    x.copy_(packed[:, :1])
    p1 = B.prefix_of(out, kp, cache[0])
    ws1 = torch.empty(B.psa_prefix_attn_workspace_size(p1), dtype=torch.uint8, device="cuda")
    nq, nk = torch.empty_like(out), torch.empty(Bn, nkv, 1, d, dtype=BF16, device="cuda")
    rope = B.rope_axes_of(nq, nk, cos, (16, 24, 24), EPS, alternate=True)
    xq, xk, xv = _split(x, nh, nkv)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        B.psa_qk_norm_rope_axes_fwd(xq, xk, *weights, cos, sin, at, nq, nk, rope)
        B.psa_kv_append(nk, xv, now, None, *cache)
        B.psa_prefix_attn_decode(nq, kp, vp, *cache, length, out, ws1, p1, scale)
    for s in range(steps):
        rows_now = [n + s for n in lens]
        x.copy_(torch.stack([packed[b, i] for b, i in enumerate(rows_now)])[:, None])
        at.copy_((max(grid) + _i32(rows_now))[None, :, None].expand(3, -1, -1))
        now.copy_(_i32(rows_now))
        length.copy_(now + 1)
        graph.replay()
        torch.cuda.synchronize()
        for b, i in enumerate(rows_now):
            assert torch.equal(nq[b, :, 0], q[b, :, i])  # the same row, alone and among others
            check(out[b:b + 1], b, i)


def test_a_cache_that_keeps_its_length():
    """A prompt's keys are weighed, cut to `keep`, and each further token pushes one out: the rows that stay, their
    places, weights and positions are those of the definition, and attention over them is."""
    Bn, nh, nkv, d, N, keep, sinks, recent, steps = 2, 8, 2, 64, 300, 120, 4, 16, 12
    scale, rows = 0.3, 301
    lens = [300, 211]
    q, k, v = _randn(1, Bn, nh, N, d).to(BF16), _randn(2, Bn, nkv, N, d).to(BF16), _randn(3, Bn, nkv, N, d).to(BF16)
    win = B.window_of(q, k)
    o, lse = torch.empty_like(q), torch.empty(Bn, nh, N, device="cuda")
    length = _i32(lens)
    B.psa_window_attn_fwd(q, k, v, length, o, lse, win, scale)
    weights = torch.zeros(Bn, nkv, rows, device="cuda")
    first = torch.zeros(Bn, nkv, N, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    B.psa_window_attn_weights(q, k, length, lse, first, ws, win, scale)
    weights[:, :, :N] = first
    for b, n in enumerate(lens):  # every query spreads a weight of one
        assert (weights[b].sum(-1) - n * nh / nkv).abs().max() < 1e-3 * n and (weights[b, :, n:] == 0).all()
    cache = [torch.full((Bn, nkv, rows, d), math.nan, dtype=BF16, device="cuda") for _ in range(2)]
    B.psa_kv_append(k, v, _i32([0, 0]), length, *cache)
    positions = torch.arange(rows, device="cuda", dtype=torch.int32).expand(Bn, nkv, -1).contiguous()
    spare = torch.zeros_like(length)
    p = B.evict_of(cache[0], keep, sinks, recent)
    assert B.psa_kv_evict_workspace_size(p) <= ws.numel()
    # a second account in 64 bits of the same fp32 weights: {position: weight} for each list
    book = [[{i: (k[b, h, i], v[b, h, i]) for i in range(lens[b])} for h in range(nkv)] for b in range(Bn)]

    def evict(next_position):
        nonlocal length, spare
        before_w, before_p = weights.clone(), positions.clone()
        B.psa_kv_evict(weights, positions, length, *cache, weights, positions, spare, ws, p)
        for b in range(Bn):
            n = int(length[b])
            for h in range(nkv):
                rank = sorted(range(n), key=lambda r: (0 if before_p[b, h, r] < sinks or before_p[b, h, r] >= next_position[b] - recent
                                                       else 1, -float(before_w[b, h, r]) if not (before_p[b, h, r] < sinks or before_p[b, h, r] >= next_position[b] - recent) else 0, r))
                stay = sorted(int(before_p[b, h, r]) for r in rank[:keep])
                assert sorted(positions[b, h, :keep].tolist()) == stay
                for r in range(0, keep, 7):
                    pos = int(positions[b, h, r])
                    assert torch.equal(cache[0][b, h, r], book[b][h][pos][0]) and torch.equal(cache[1][b, h, r], book[b][h][pos][1])
                assert (weights[b, h, keep:n] == 0).all()
        length, spare = spare, length

    evict(lens)
    at = list(lens)
    for s in range(steps):
        nq, nk, nv = (_randn(10 + 3 * s + i, Bn, h, 1, d).to(BF16) for i, h in enumerate((nh, nkv, nkv)))
        B.psa_kv_append(nk, nv, length, None, *cache)
        for b in range(Bn):
            positions[b, :, int(length[b])] = at[b]
            for h in range(nkv):
                book[b][h][at[b]] = (nk[b, h, 0], nv[b, h, 0])
            at[b] += 1
        length += 1
        step = B.window_of(nq, cache[0])
        before, out = weights.clone(), torch.empty_like(nq)
        ws2 = torch.empty(B.psa_window_attn_decode_weights_workspace_size(step), dtype=torch.uint8, device="cuda")
        B.psa_window_attn_decode_weights(nq, *cache, length, out, weights, ws2, step, scale)
        for b in range(Bn):
            n = int(length[b])
            kk, vv = (torch.stack([torch.stack([book[b][h][int(i)][c] for i in positions[b, h, :n]]) for h in range(nkv)])[None] for c in (0, 1))
            r = window_attention(nq[b:b + 1], kk, vv, None, -1, 0, 0, scale)
            within(out[b:b + 1], r["o"], r["o_tol"], (s, b))
            added = (weights[b, :, :n] - before[b, :, :n]).sum(-1)
            assert (added - nh / nkv).abs().max() < 1e-3
        evict(at)
        assert length.tolist() == [keep] * Bn


def test_training_step_over_a_feature_map():
    """Two axes, norms, attention both ways over a 12 x 15 map, and the gradients back to the projection's
    output, against the 64-bit chain by differences of each operator on what the one before gave."""
    Bn, nh, nkv, d, grid, scale = 2, 4, 2, 64, (12, 15), 0.125
    N = math.prod(grid)
    cos, sin = _tables(15, 32)
    packed = _randn(1, Bn, N, nh + 2 * nkv, d).to(BF16)
    wq, wk = 1 + 0.1 * _randn(2, d), 1 + 0.1 * _randn(3, d)
    do = _randn(4, Bn, N, nh, d).to(BF16).transpose(1, 2)
    q0, k0, v = _split(packed, nh, nkv)
    p = B.rope_axes_of(q0, k0, cos, (16, 16), EPS, grid=grid)
    q, k = (torch.empty(t.shape, dtype=BF16, device="cuda") for t in (q0, k0))
    B.psa_qk_norm_rope_axes_fwd(q0, k0, wq, wk, cos, sin, None, q, k, p)
    win = B.window_of(q, k, -1, -1)
    o, lse = torch.empty(Bn, nh, N, d, dtype=BF16, device="cuda"), torch.empty(Bn, nh, N, device="cuda")
    B.psa_window_attn_fwd(q, k, v, None, o, lse, win, scale)
    grad = torch.empty_like(packed)
    gq0, gk0, gv = _split(grad, nh, nkv)
    gq, gk = torch.empty_like(q), torch.empty_like(k)
    ws = torch.empty(max(B.psa_window_attn_bwd_workspace_size(win), B.psa_qk_norm_rope_bwd_workspace_size(p.rope)),
                     dtype=torch.uint8, device="cuda")
    dwq, dwk = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    B.psa_window_attn_bwd(q, k, v, o, do, lse, None, gq, gk, gv, ws, win, scale)
    B.psa_qk_norm_rope_axes_bwd(q0, k0, wq, wk, cos, sin, None, gq, gk, gq0, gk0, dwq, dwk, ws, p)
    y, x = torch.meshgrid(*(torch.arange(g, device="cuda") for g in grid), indexing="ij")
    own = [torch.cat([t[y.flatten()][:, :16], t[x.flatten()][:, 16:]], 1) for t in (cos, sin)]  # each cell's angles
    cells = torch.arange(N, device="cuda").expand(Bn, -1)
    within(q, *norm_rope(q0, wq, *own, cells, False, EPS), "q")
    within(k, *norm_rope(k0, wk, *own, cells, False, EPS), "k")
    r = window_attention(q, k, v, None, -1, -1, 0, scale, do)
    for name, t in (("o", o), ("lse", lse), ("dq", gq), ("dk", gk), ("dv", gv)):
        within(t, r[name], r[name + "_tol"], name)
    for x0, w, g, dx, dw in ((q0, wq, gq, gq0, dwq), (k0, wk, gk, gk0, dwk)):
        rdx, tdx, rdw, tdw = norm_rope(x0, w, *own, cells, False, EPS, g)
        within(dx, rdx, tdx, "dx")
        within(dw, rdw, tdw, "dw")
