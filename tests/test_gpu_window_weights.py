"""psa_window_attn_weights: column sums of the probabilities against their 64-bit form."""
import math

import pytest
import torch

from token_reference import U, visible, within
from vision_transformer_attention_psapackqkv_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _reference(q, k, lens, lse, left, right, sinks, scale):
    """Sums over each key/value head's query heads and all queries, from the lse given, and a bound."""
    Bn, nh, nq, d = q.shape
    nkv, nk = k.shape[1:3]
    group = nh // nkv
    out, tol = (torch.zeros(Bn, nkv, nk, dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(Bn):
        n = nk if lens is None else max(0, min(lens[b], nk))
        ok = visible(nq, nk, n, left, right, sinks, "cuda")
        rows = ok.any(1)
        for h in range(nh):
            qq, kk = q[b, h].double()[rows], torch.where(ok.any(0)[:, None], k[b, h // group].double(), 0.0)
            l = lse[b, h].double()[rows, None]
            p = torch.where(ok[rows], torch.exp(qq @ kk.T * scale - l), 0.0)
            if not rows.any():
                continue
            # the argument of the exponential: d products, the scale, lse times log2(e) (rounded) and the sum of
            # the two; the exponential; then a sum of positive terms
            big = float((qq.abs() @ kk.abs().T * scale).max())
            ex = U * ((d + 4) * big + 4 * float(l.abs().max()) + 32)
            out[b, h // group] += p.sum(0)
            tol[b, h // group] += p.sum(0) * (ex + (nq * group + 64) * U)
    return out, tol


def _run(q, k, lens, lse, weights, win, scale):
    ws = torch.full((B.psa_window_attn_weights_workspace_size(win),), 0xFF, dtype=torch.uint8, device="cuda")
    l = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    B.psa_window_attn_weights(q, k, l, lse, weights, ws, win, scale)
    return weights


# B, nq, nk, lens, left, right, sinks
CASES = [(1, 1, 1, None, -1, 0, 0), (2, 1, 77, [77, 30], -1, 0, 0), (1, 5, 5, None, 1, 1, 0), (3, 32, 700, [700, 690, 500], -1, 0, 0),
         (2, 77, 300, None, 100, 0, 3), (2, 128, 128, [128, 1], -1, 0, 0), (1, 129, 129, None, -1, -1, 0), (2, 256, 256, None, -1, 0, 0),
         (2, 400, 400, [400, 133], 60, 60, 4), (1, 500, 1100, None, 255, 0, 130), (3, 1000, 1000, [1000, 0, -3], -1, 0, 0),
         (1, 2100, 2100, None, 1023, 0, 4), (2, 300, 300, None, 0, 0, 1), (1, 40, 30, None, -1, 0, 0), (1, 600, 450, [445], 20, 5, 2)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh,nkv", [(4, 2), (1, 1), (5, 1), (24, 3), (160, 1)])
@pytest.mark.parametrize("Bn,nq,nk,lens,left,right,sinks", CASES)
def test_weights(Bn, nq, nk, lens, left, right, sinks, nh, nkv, d):
    q, k, v = _randn(1, Bn, nh, nq, d).to(BF16), _randn(2, Bn, nkv, nk, d).to(BF16), _randn(3, Bn, nkv, nk, d).to(BF16)
    before = torch.rand(Bn, nkv, nk, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    scale, off = d ** -0.5, nk - nq
    win = B.window_of(q, k, left, right, sinks)
    for b, n in enumerate(lens or []):  # what padding holds plays no part
        n = max(0, n)
        q[b, :, max(0, n - off):], k[b, :, n:], v[b, :, n:], before[b, :, n:] = math.nan, math.inf, math.nan, math.inf
    if off < 0:
        q[:, :, :-off] = math.nan
    o, lse = torch.empty_like(q), torch.empty(Bn, nh, nq, device="cuda")
    l32 = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    B.psa_window_attn_fwd(q, k, v, l32, o, lse, win, scale)
    want, tol = _reference(q, k, lens, lse, left, right, sinks, scale)
    w = _run(q, k, lens, lse, before.clone(), win, scale)
    total = before.double() + want
    within(w, total, torch.where(total.isfinite(), tol + U * total, 0.0), "weights")
    assert torch.equal(w, _run(q, k, lens, lse, before.clone(), win, scale))


def test_a_prompt_in_chunks_adds_up_to_the_whole():
    """Each query's probabilities sum to one, whatever part of the prompt it comes with."""
    N, nh, nkv, d = 1500, 8, 2, 128
    packed = _randn(5, 1, N, nh + 2 * nkv, d).to(BF16).transpose(1, 2)
    q, k, v = packed[:, :nh], packed[:, nh:nh + nkv], packed[:, nh + nkv:]
    lse, o = torch.empty(1, nh, N, device="cuda"), torch.empty(q.shape, dtype=BF16, device="cuda")
    B.psa_window_attn_fwd(q, k, v, None, o, lse, B.window_of(q, k), 0.09)
    whole = _run(q, k, None, lse, torch.zeros(1, nkv, N, device="cuda"), B.window_of(q, k), 0.09)
    parts = torch.zeros(1, nkv, N, device="cuda")
    for a, b in ((0, 700), (700, 701), (701, 730), (730, 1500)):
        w = torch.zeros(1, nkv, b, device="cuda")
        qc, kc = q[:, :, a:b], k[:, :, :b]
        parts[:, :, :b] += _run(qc, kc, None, lse[:, :, a:b].contiguous(), w, B.window_of(qc, kc), 0.09)
    want, tol = _reference(q, k, None, lse, -1, 0, 0, 0.09)
    within(whole, want, tol, "whole")
    within(parts, want, 2 * tol, "parts")
    assert abs(float(whole.sum()) - N * nh) < 1e-4 * N * nh


def test_many_lists_and_long_parts():
    """More units than CTAs several times over, and key tiles whose queries are cut into parts."""
    for Bn, nh, nkv, nq, nk, left, sinks in ((40, 4, 4, 200, 200, -1, 0), (64, 12, 12, 40, 200, -1, 0), (1, 16, 1, 3100, 3100, 63, 16), (1, 2, 1, 6000, 6000, -1, 0)):
        q, k = _randn(6, Bn, nh, nq, 64).to(BF16), _randn(7, Bn, nkv, nk, 64).to(BF16)
        win, lse = B.window_of(q, k, left, 0, sinks), torch.empty(Bn, nh, nq, device="cuda")
        B.psa_window_attn_fwd(q, k, k, None, torch.empty_like(q), lse, win, 0.2)
        want, tol = _reference(q, k, None, lse, left, 0, sinks, 0.2)
        first = _run(q, k, None, lse, torch.zeros(Bn, nkv, nk, device="cuda"), win, 0.2)
        within(first, want, tol, (Bn, nq))
        for _ in range(10):
            assert torch.equal(first, _run(q, k, None, lse, torch.zeros(Bn, nkv, nk, device="cuda"), win, 0.2))


def test_replayed_on_another_stream():
    q, k = _randn(8, 2, 8, 300, 128).to(BF16), _randn(9, 2, 2, 300, 128).to(BF16)
    win, lse = B.window_of(q, k), torch.empty(2, 8, 300, device="cuda")
    B.psa_window_attn_fwd(q, k, k, None, torch.empty_like(q), lse, win, 0.1)
    want = _run(q, k, None, lse, torch.zeros(2, 2, 300, device="cuda"), win, 0.1)
    w, ws = torch.zeros(2, 2, 300, device="cuda"), torch.empty(B.psa_window_attn_weights_workspace_size(win), dtype=torch.uint8, device="cuda")
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        B.psa_window_attn_weights(q, k, None, lse, w, ws, win, 0.1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, want)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, want + want)
