"""psa_window_attn_fwd / _bwd against their 64-bit form: masks, ragged sizes, shared heads, strides,
padding, and rows that see nothing."""
import math

import pytest
import torch

from token_reference import window_attention, within
from vision_transformer_attention_psapackqkv_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _inputs(Bn, nh, nkv, nq, nk, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    return rn(Bn, nh, nq, d), rn(Bn, nkv, nk, d), rn(Bn, nkv, nk, d), rn(Bn, nh, nq, d)


def _seven(t):
    return torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda")


def _fwd(q, k, v, lens, left, right, sinks, scale, stream=None):
    win = B.window_of(q, k, left, right, sinks)
    o, lse = _seven(q), torch.full(q.shape[:3], 7.0, device="cuda")
    B.psa_window_attn_fwd(q, k, v, lens, o, lse, win, scale, stream)
    return o, lse


def _bwd(q, k, v, o, do, lse, lens, left, right, sinks, scale):
    win = B.window_of(q, k, left, right, sinks)
    dq, dk, dv = _seven(q), _seven(k), _seven(v)
    ws = torch.full((B.psa_window_attn_bwd_workspace_size(win),), 0xFF, dtype=torch.uint8, device="cuda")
    B.psa_window_attn_bwd(q, k, v, o, do, lse, lens, dq, dk, dv, ws, win, scale)
    return dq, dk, dv


def _check(q, k, v, do, lens, left, right, sinks, scale):
    dtype = q.dtype
    lens_t = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = _fwd(q, k, v, lens_t, left, right, sinks, scale)
    dq, dk, dv = _bwd(q, k, v, o, do, lse, lens_t, left, right, sinks, scale)
    r = window_attention(q, k, v, lens, left, right, sinks, scale, do, 2.0 ** -8 if dtype == BF16 else 2.0 ** -24,
                         dtype == F32)
    for name, x in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(x, r[name], r[name + "_tol"], name)
    assert B.psa_get_last_device_error() == B.PSA_OK


# n_q, n_k, left, right, sinks
MASKS = [(1, 1, -1, 0, 0), (2, 2, 0, 0, 0), (65, 65, -1, 0, 0), (127, 127, 30, 0, 4), (128, 128, -1, -1, 0),
         (129, 129, 63, 0, 1), (200, 200, 17, 20, 3), (257, 257, 40, 0, 130), (400, 400, 60, 60, 4),
         (385, 385, 128, 0, 0), (1, 300, -1, 0, 0), (70, 300, 90, 0, 8), (130, 513, 1, 0, 129), (90, 40, -1, 0, 0),
         (300, 130, 20, 5, 2), (640, 640, 255, 0, 64)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nk,left,right,sinks", MASKS)
def test_masks_and_sizes(nq, nk, left, right, sinks, d, dtype):
    q, k, v, do = _inputs(2, 4, 2, nq, nk, d, dtype, nq + nk + d)
    _check(q, k, v, do, None, left, right, sinks, d ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,left,sinks,lens", [(300, -1, 0, [300, 0, 1, 129]), (260, 50, 4, [128, 127, 260, 3]),
                                               (129, 200, 0, [129, 64, 500, -7])])
def test_padded_batches_whose_padding_holds_nan(n, left, sinks, lens, d, dtype):
    q, k, v, do = _inputs(4, 4, 1, n, n, d, dtype, n + d)
    for b, m in enumerate(lens):
        for t in (q, k, v, do):
            t[b, :, max(0, min(m, n)):] = math.nan
    _check(q, k, v, do, lens, left, 0, sinks, d ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_chunk_behind_a_prefix_in_a_padded_batch(dtype):
    q, k, v, do = _inputs(3, 2, 2, 100, 350, 64, dtype, 8)
    lens = [350, 300, 240]  # the last sequence ends in front of the chunk
    for b, m in enumerate(lens):
        k[b, :, m:], v[b, :, m:] = math.nan, math.inf
        q[b, :, max(0, m - 250):], do[b, :, max(0, m - 250):] = math.nan, math.nan
    _check(q, k, v, do, lens, 100, 0, 2, 0.2)


@pytest.mark.parametrize("nh,nkv", [(8, 8), (8, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_short_sequences_in_a_padded_batch(nh, nkv, d):
    """Several units per CTA, each of one or two tiles that a sequence ends in."""
    Bn, n = 90, 140
    q, k, v, do = _inputs(Bn, nh, nkv, n, n, d, BF16, 19)
    lens = [(37 * b) % (n + 1) for b in range(Bn)]
    for b, m in enumerate(lens):
        for t in (q, k, v, do):
            t[b, :, m:] = math.nan
    _check(q, k, v, do, lens, 100, 0, 3, 0.1)


@pytest.mark.parametrize("nh,nkv", [(1, 1), (5, 1), (8, 8), (6, 2), (7, 7), (16, 1), (40, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_heads(nh, nkv, d):
    q, k, v, do = _inputs(1, nh, nkv, 140, 140, d, BF16, nh)
    _check(q, k, v, do, None, 77, 0, 1, 0.1)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_views(dtype):
    """q, k, v as parts of one projection's output, the keys as the front of a longer cache."""
    Bn, n, nh, nkv, d = 2, 150, 4, 2, 128
    g = torch.Generator(device="cuda").manual_seed(11)
    packed = torch.randn(Bn, n, nh + 2 * nkv, d, generator=g, device="cuda").to(dtype).transpose(1, 2)
    q, k, v = packed[:, :nh], packed[:, nh:nh + nkv], packed[:, nh + nkv:]
    cache = torch.full((nkv, Bn, 200, 2 * d), math.nan, dtype=dtype, device="cuda")
    kc = cache.transpose(0, 1)[:, :, :n, d:]
    kc.copy_(k)
    do = torch.randn(Bn, n, nh, d, generator=g, device="cuda").to(dtype).transpose(1, 2)
    _check(q, kc, v, do, None, 33, 0, 2, 0.08)
    win = B.window_of(q, kc, 33, 0, 2)
    dense = _fwd(q.contiguous(), k.contiguous(), v.contiguous(), None, 33, 0, 2, 0.08)
    out = torch.full((Bn, n, nh + 1, d), 7.0, dtype=dtype, device="cuda")  # a view as the output
    B.psa_window_attn_fwd(q, kc, v, None, out.transpose(1, 2)[:, :nh], None, win, 0.08)
    assert torch.equal(out[:, :, :nh].transpose(1, 2), dense[0]) and (out[:, :, nh] == 7.0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_growing_scores(d):
    """Row maxima that jump by far more than 2^8 from key tile to key tile, in both directions."""
    q, k, v, do = _inputs(1, 2, 1, 520, 520, d, BF16, 12)
    u = torch.randn(d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    u /= u.norm()
    ramp = torch.linspace(-20, 20, 520, device="cuda")[:, None] * u
    k = (k.float() * 0.3 + ramp).to(BF16)
    q = (q.float() * 0.3 + 8 * u).to(BF16)
    for kk in (k, k.flip(2).contiguous()):
        o, lse = _fwd(q, kk, v, None, -1, 0, 0, 0.5)
        r = window_attention(q, kk, v, None, -1, 0, 0, 0.5)
        within(o, r["o"], r["o_tol"], "o")
        within(lse, r["lse"], r["lse_tol"], "lse")


def test_a_long_sequence_s_rows():
    """One head of 8192 positions with a window: sampled rows, whole gradients' sums."""
    n, d, scale = 8192, 128, 128 ** -0.5
    q, k, v, do = _inputs(1, 2, 1, n, n, d, BF16, 13)
    o, lse = _fwd(q, k, v, None, 1023, 0, 4, scale)
    dq, dk, dv = _bwd(q, k, v, o, do, lse, None, 1023, 0, 4, scale)
    r = window_attention(q, k, v, None, 1023, 0, 4, scale, do)
    for name, x in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(x, r[name], r[name + "_tol"], name)


def test_reruns_are_bitwise_identical():
    q, k, v, do = _inputs(2, 8, 2, 700, 700, 128, BF16, 14)
    runs = []
    for _ in range(3):
        o, lse = _fwd(q, k, v, None, 200, 0, 4, 0.1)
        runs.append((o, lse) + _bwd(q, k, v, o, do, lse, None, 200, 0, 4, 0.1))
    for again in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(runs[0], again))


@pytest.mark.parametrize("d", [64, 128])
def test_many_runs_of_a_long_sequence_agree(d):
    """Long runs of tiles per thread block, again and again: threads of a block that drift apart by a
    tile must not meet one another's barriers (a wait that gives up shows as a device error)."""
    n, scale = 16384, d ** -0.5
    q, k, v, do = _inputs(1, 16, 2, n, n, d, BF16, 20)
    first = None
    for _ in range(40):
        o, lse = _fwd(q, k, v, None, -1, 0, 0, scale)
        got = (o, lse) + _bwd(q, k, v, o, do, lse, None, -1, 0, 0, scale)
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(first, got))
    assert B.psa_get_last_device_error() == B.PSA_OK


def test_graph_replays_on_new_inputs_and_another_stream():
    q, k, v, do = _inputs(2, 4, 2, 333, 333, 64, BF16, 15)
    lens = torch.tensor([333, 200], dtype=torch.int32, device="cuda")
    win = B.window_of(q, k, 100, 0, 2)
    o, lse = _seven(q), torch.empty(q.shape[:3], device="cuda")
    dq, dk, dv = _seven(q), _seven(k), _seven(v)
    ws = torch.empty(B.psa_window_attn_bwd_workspace_size(win), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        B.psa_window_attn_fwd(q, k, v, lens, o, lse, win, 0.1, stream)
        B.psa_window_attn_bwd(q, k, v, o, do, lse, lens, dq, dk, dv, ws, win, 0.1, stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    new = _inputs(2, 4, 2, 333, 333, 64, BF16, 16)
    for t, x in zip((q, k, v, do), new):
        t.copy_(x)
    lens.copy_(torch.tensor([150, 333], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (o, lse, dq, dk, dv)]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, (o, lse, dq, dk, dv)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,left,right,lens,rows", [(1, -1, 0, None, "all"), (200, 0, 0, None, "all"), (2, 0, 0, None, "all"),
                                                    (150, 3, 0, [1, 1], "all"), (300, -1, 0, None, [0]),
                                                    (200, 0, 5, None, [199]), (2, 0, 1, None, [1]),
                                                    (260, 0, 300, [260, 131], [[259], [130]])])
def test_rows_that_see_one_key_pass_no_gradient(n, left, right, lens, rows, dtype):
    """Their probability is 1 whatever the score: exactly 0, not what is left of dP - delta."""
    q, k, v, do = _inputs(2, 4, 2, n, n, 128, dtype, 21)
    lens_t = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = _fwd(q, k, v, lens_t, left, right, 0, 0.3)
    dq, dk, dv = _bwd(q, k, v, o, do, lse, lens_t, left, right, 0, 0.3)
    if rows == "all":
        assert (dq == 0).all() and (dk == 0).all() and (dv[:, :, 0] != 0).any()
    else:
        for b in range(2):
            one = rows[b] if isinstance(rows[0], list) else rows
            m = n if lens is None else lens[b]
            assert (dq[b, :, one] == 0).all()
            assert all((dq[b, :, i] != 0).any() for i in range(m) if i not in one)
    _check(q, k, v, do, lens, left, right, 0, 0.3)


def test_a_window_as_wide_as_the_sequence_is_no_window():
    q, k, v, _ = _inputs(1, 2, 2, 200, 200, 64, BF16, 17)
    a = _fwd(q, k, v, None, -1, 0, 0, 0.1)
    b = _fwd(q, k, v, None, 2 ** 31 - 1, 0, 2 ** 31 - 1, 0.1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_causal_attention_next_to_flash_attn2():
    """Without any limit the operator is the framework's own attention."""
    q, k, v, _ = _inputs(1, 3, 3, 300, 300, 64, BF16, 18)
    o, lse = _fwd(q, k, v, None, -1, -1, 0, 0.125)
    o2, lse2 = torch.empty_like(q[0]), torch.empty(3, 300, device="cuda")
    B.flash_attn2_fwd(q[0], k[0], v[0], o2, lse2, 0.125)
    r = window_attention(q, k, v, None, -1, -1, 0, 0.125)
    within(o[0], o2, 2 * r["o_tol"][0], "o")
    within(lse[0], lse2, 2 * r["lse_tol"][0], "lse")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_nan_in_a_query_stays_in_its_row(dtype):
    q, k, v, _ = _inputs(1, 2, 1, 150, 150, 64, dtype, 31)
    o, lse = _fwd(q, k, v, None, -1, 0, 0, 0.2)
    q[0, 1, 70, 3] = math.nan
    o2, lse2 = _fwd(q, k, v, None, -1, 0, 0, 0.2)
    assert o2[0, 1, 70].isnan().all() and lse2[0, 1, 70].isnan()
    keep = torch.ones(2, 150, dtype=torch.bool, device="cuda")
    keep[1, 70] = False
    assert torch.equal(o2[0, 0], o[0, 0]) and o2[0][keep].isfinite().all() and lse2[0][keep].isfinite().all()


@pytest.mark.parametrize("Bn,nh,nkv,n,d,left,right,sinks,lens", [(3, 8, 8, 420, 64, 60, 60, 4, [420, 1, 333]),
                                                              (2, 32, 4, 260, 64, -1, 0, 0, None),
                                                              (2, 6, 3, 700, 128, 99, 0, 3, [700, 650])])
def test_fp32_of_many_heads(Bn, nh, nkv, n, d, left, right, sinks, lens):
    """More rows than the tiles for few of them take, on both sides or on the queries' alone."""
    _check(*_inputs(Bn, nh, nkv, n, n, d, F32, 41), lens, left, right, sinks, 0.2)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("right", [-1, 30])
@pytest.mark.parametrize("nq,nk", [(300, 130), (131, 3), (260, 259)])
def test_rows_in_front_of_position_0_see_nothing(nq, nk, right, dtype):
    """More queries than keys, and a window that looks ahead."""
    q, k, v, do = _inputs(1, 2, 2, nq, nk, 64, dtype, 51)
    front, half = slice(0, nq - nk), 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    r = window_attention(q, k, v, None, -1, right, 0, 0.2, do, half, dtype == F32)
    q[:, :, front], do[:, :, front] = math.nan, math.inf
    o, lse = _fwd(q, k, v, None, -1, right, 0, 0.2)
    dq, dk, dv = _bwd(q, k, v, o, do, lse, None, -1, right, 0, 0.2)
    assert (o[:, :, front] == 0).all() and (lse[:, :, front] == -math.inf).all() and (dq[:, :, front] == 0).all()
    for name, x in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(x, r[name], r[name + "_tol"], name)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Bn,n,left,right,sinks,lens", [(32, 2, -1, 0, 0, None), (8, 8, -1, 0, 0, None), (4, 5, -1, -1, 0, None),
                                                        (1, 300, 1, 0, 0, None), (2, 300, 4, 3, 0, [300, 131]),
                                                        (1, 300, 0, 0, 1, None), (2, 260, 1, 2, 4, [260, 7]),
                                                        (1, 130, 7, 0, 0, None)])
def test_gradients_of_rows_that_see_few_keys(Bn, n, left, right, sinks, lens, d):
    """Up to eight keys: dP - delta may be small next to delta, so that delta is to be as exact as dP,
    not as o, whose rounding to bf16 is of delta's size.  Roundings of P, dS and the outputs to bf16
    are counted, and fp32 sums of products; no rounding of o."""
    nh, nkv, scale, half, u = 4, 2, d ** -0.5, 2.0 ** -8, 2.0 ** -24
    q, k, v, do = _inputs(Bn, nh, nkv, n, n, d, BF16, 71 + n)
    lens_t = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = _fwd(q, k, v, lens_t, left, right, sinks, scale)
    dq, dk, dv = _bwd(q, k, v, o, do, lse, lens_t, left, right, sinks, scale)
    p = torch.arange(n, device="cuda")[:, None] + torch.zeros(n, dtype=torch.int64, device="cuda")
    j = p.T
    for b in range(Bn):
        m = n if lens is None else lens[b]
        ok = (p < m) & (j < m)
        ok &= (j >= p - left) | (j < sinks) if left >= 0 else ok
        ok &= j <= p + right if right >= 0 else ok
        assert ok.sum(1).max() <= 8
        for hk in range(nkv):
            dk64 = torch.zeros(n, d, dtype=torch.float64, device="cuda")
            dk_tol = torch.zeros_like(dk64)
            for h in range(hk * nh // nkv, (hk + 1) * nh // nkv):
                qq, kk, vv, g = (t.double() for t in (q[b, h], k[b, hk], v[b, hk], do[b, h]))
                x = torch.where(ok, qq @ kk.T * scale, -math.inf)
                prob = torch.softmax(x, 1).nan_to_num(0.0)
                dp, dpm = g @ vv.T, g.abs() @ vv.abs().T
                ds = prob * (dp - (prob * dp).sum(1, keepdim=True))
                # P in fp32: the scores' sums of d products, the exponent's rounding and the lse's, ex2
                ex = u * ((d + 4) * float((qq.abs() @ kk.abs().T).max()) * scale + 64)
                every = (prob * dpm).sum(1, keepdim=True)  # magnitudes of delta's terms
                ds_err = half * ds.abs() + prob * (((d + 16) * u + 2 * ex) * (dpm + every))
                within(dq[b, h], scale * ds @ kk, half * (scale * ds @ kk).abs() + scale * (ds_err + 16 * u * ds.abs()) @ kk.abs(), "dq")
                dk64 += scale * ds.T @ qq
                dk_tol += scale * (ds_err + 64 * u * ds.abs()).T @ qq.abs()
            within(dk[b, hk], dk64, half * dk64.abs() + dk_tol, "dk")
