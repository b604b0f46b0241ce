"""The token-sequence operators run together, as a layer uses them: a training step from one
projection's output, and decoding through a cache that agrees with the forward over the whole
sequence."""
import pytest
import torch

from token_reference import dequantise, norm_rope, quantise, window_attention, within
from vision_transformer_attention_psapackqkv_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPS = 2.0 ** -18


def _layer(Bn, nh, nkv, N, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    packed = rn(Bn, N, nh + 2 * nkv, d).to(BF16)
    freq = 1e4 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") / (d // 2))
    angle = torch.arange(N, dtype=torch.float64, device="cuda")[:, None] * freq
    x = packed.transpose(1, 2)
    return dict(packed=packed, q=x[:, :nh], k=x[:, nh:nh + nkv], v=x[:, nh + nkv:], wq=1 + 0.1 * rn(d),
                wk=1 + 0.1 * rn(d), cos=angle.cos().float().contiguous(), sin=angle.sin().float().contiguous(),
                do=rn(Bn, N, nh, d).to(BF16).transpose(1, 2))


@pytest.mark.parametrize("d", [64, 128])
def test_training_step(d):
    Bn, nh, nkv, N, left, sinks = 2, 4, 2, 200, 90, 3
    c = _layer(Bn, nh, nkv, N, d, 1)
    p = B.norm_rope_of(c["q"], c["k"], c["cos"], EPS)
    q, k = (torch.empty(t.shape, dtype=BF16, device="cuda") for t in (c["q"], c["k"]))
    win = B.window_of(q, k, left, 0, sinks)
    scale = d ** -0.5
    out = torch.empty(Bn, N, nh, d, dtype=BF16, device="cuda").transpose(1, 2)  # what the next projection reads
    lse = torch.empty(Bn, nh, N, device="cuda")
    B.psa_qk_norm_rope_fwd(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], None, q, k, p)
    B.psa_window_attn_fwd(q, k, c["v"], None, out, lse, win, scale)
    grad = torch.empty_like(c["packed"])  # the projection's gradient, written in place as views
    gx = grad.transpose(1, 2)
    gq, gk = torch.empty_like(q), torch.empty_like(k)
    ws = torch.empty(max(B.psa_window_attn_bwd_workspace_size(win), B.psa_qk_norm_rope_bwd_workspace_size(p)),
                     dtype=torch.uint8, device="cuda")
    dwq, dwk = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    B.psa_window_attn_bwd(q, k, c["v"], out, c["do"], lse, None, gq, gk, gx[:, nh + nkv:], ws, win, scale)
    B.psa_qk_norm_rope_bwd(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], None, gq, gk, gx[:, :nh],
                           gx[:, nh:nh + nkv], dwq, dwk, ws, p)
    # each operator against its 64-bit form on what the one before it gave
    pos = torch.arange(N, device="cuda").expand(Bn, -1)
    within(q, *norm_rope(c["q"], c["wq"], c["cos"], c["sin"], pos, False, EPS), "q")
    within(k, *norm_rope(c["k"], c["wk"], c["cos"], c["sin"], pos, False, EPS), "k")
    r = window_attention(q, k, c["v"], None, left, 0, sinks, scale, c["do"])
    for name, x in (("o", out), ("lse", lse), ("dq", gq), ("dk", gk), ("dv", gx[:, nh + nkv:])):
        within(x, r[name], r[name + "_tol"], name)
    for x, w, g, dx, dw in ((c["q"], c["wq"], gq, gx[:, :nh], dwq), (c["k"], c["wk"], gk, gx[:, nh:nh + nkv], dwk)):
        rdx, tdx, rdw, tdw = norm_rope(x, w, c["cos"], c["sin"], pos, False, EPS, g)
        within(dx, rdx, tdx, "dx")
        within(dw, rdw, tdw, "dw")


@pytest.mark.parametrize("kv4", [False, True])
def test_decoding_through_a_cache(kv4):
    """A prompt goes into the cache, then tokens one at a time from one captured graph."""
    Bn, nh, nkv, d, rows, left, sinks, scale = 3, 8, 2, 128, 96, 40, 2, 128 ** -0.5
    prompt, steps = [50, 61, 17], 20
    N = max(prompt) + steps
    c = _layer(Bn, nh, nkv, N, d, 2)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    p = B.norm_rope_of(c["q"], c["k"], c["cos"], EPS)
    q, k = (torch.empty(t.shape, dtype=BF16, device="cuda") for t in (c["q"], c["k"]))
    B.psa_qk_norm_rope_fwd(c["q"], c["k"], c["wq"], c["wk"], c["cos"], c["sin"], None, q, k, p)
    v = c["v"]
    if kv4:
        cache = tuple(torch.zeros(Bn, nkv, rows, n, dtype=t, device="cuda") for n, t in ((d // 2, torch.uint8), (d // 32, BF16)) * 2)
        append = lambda *a: B.psa_kv4_append(*a, *cache)  # noqa: E731
    else:
        cache = tuple(torch.full((Bn, nkv, rows, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
        append = lambda *a: B.psa_kv_append(*a, *cache)  # noqa: E731
    append(k, v, i32([0] * Bn), i32(prompt))

    # one step: the new token's projection -> norms and rotation -> cache -> attention
    x = torch.empty(Bn, 1, nh + 2 * nkv, d, dtype=BF16, device="cuda")
    xt, pos, lens = x.transpose(1, 2), i32(prompt), i32(prompt) + 1
    nq, nk = torch.empty(Bn, nh, 1, d, dtype=BF16, device="cuda"), torch.empty(Bn, nkv, 1, d, dtype=BF16, device="cuda")
    o = torch.empty_like(nq)
    p1 = B.norm_rope_of(nq, nk, c["cos"], EPS)
    win = B.window_of(nq, cache[0], left, 0, sinks)
    ws = torch.empty(B.psa_window_attn_decode_workspace_size(win), dtype=torch.uint8, device="cuda")

    def step():
        B.psa_qk_norm_rope_fwd(xt[:, :nh], xt[:, nh:nh + nkv], c["wq"], c["wk"], c["cos"], c["sin"], pos[:, None], nq,
                               nk, p1)
        append(nk, xt[:, nh + nkv:], pos, None)
        if kv4:
            B.psa_window_attn_decode_kv4(nq, *cache, lens, o, ws, win, scale)
        else:
            B.psa_window_attn_decode(nq, *cache, lens, o, ws, win, scale)

    graph = torch.cuda.CUDAGraph()
    x.copy_(c["packed"][:, :1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pass
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        step()
    seen_k, seen_v = (dequantise(*quantise(t)) if kv4 else t for t in (k, v))
    for s in range(steps):
        at = [n + s for n in prompt]
        for b, i in enumerate(at):
            x[b, 0] = c["packed"][b, i]
        pos.copy_(i32(at))
        lens.copy_(i32(at) + 1)
        graph.replay()
        torch.cuda.synchronize()
        for b, i in enumerate(at):
            assert torch.equal(nq[b, :, 0], q[b, :, i])  # the same row, alone and in the prompt
            r = window_attention(q[b:b + 1, :, i:i + 1], seen_k[b:b + 1, :, :i + 1], seen_v[b:b + 1, :, :i + 1], None,
                                 left, 0, sinks, scale)
            within(o[b:b + 1], r["o"], r["o_tol"], (s, b))
    for b, n in enumerate(prompt):  # rows behind the sequence are as they were
        if not kv4:
            assert torch.equal(cache[0][b, :, :n + steps], k[b, :, :n + steps])
            assert torch.isnan(cache[0][b, :, n + steps:]).all()
        else:
            assert (cache[0][b, :, n + steps:] == 0).all() and (cache[3][b, :, n + steps:] == 0).all()
