"""Attention weights kept along with decoding steps, and the eviction of the rows that have least."""
import math

import pytest
import torch

from token_reference import U, visible, window_attention, within
from vision_transformer_attention_psapackqkv_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(seed, *shape):
    return torch.randn(*shape, generator=_gen(seed), device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ weights of a decoding step
def _probabilities(q, k, lens, left, sinks, scale):
    """Sums over each key/value head's query heads in 64 bits, and a bound on fp32's error."""
    Bn, nh, _, d = q.shape
    nkv, rows = k.shape[1:3]
    group = nh // nkv
    out, tol = (torch.zeros(Bn, nkv, rows, dtype=torch.float64, device="cuda") for _ in range(2))
    for b, n in enumerate(lens):
        n = max(0, min(n, rows))
        if n == 0:
            continue
        ok = visible(1, n, n, left, 0, sinks, "cuda")
        for h in range(nh):
            qq, kk = q[b, h].double(), k[b, h // group, :n].double()
            kk = torch.where(ok.T, kk, 0.0)
            p = torch.softmax(torch.where(ok, qq @ kk.T * scale, -math.inf), 1)[0]
            # a score's error moves a probability by its share of that, twice (the key's own, and the sum's)
            ex = U * ((d + 4) * float((qq.abs() @ kk.abs().T * scale).max()) + 32)
            out[b, h // group, :n] += p
            tol[b, h // group, :n] += p * (2 * ex + (n + 16 + group) * U)
    return out, tol


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh,nkv", [(4, 2), (1, 1), (17, 1), (40, 8), (12, 4)])
@pytest.mark.parametrize("lens,rows,left,sinks", [([1], 1, -1, 0), ([0, 1, 2, 17], 40, -1, 0), ([16, 15, 33, -4], 33, 7, 2),
                                                  ([300, 129, 500, 64], 300, -1, 0), ([1000, 999, 5, 130], 1001, 63, 4),
                                                  ([700, 350], 700, 100, 130), ([2000], 2100, 0, 1), ([5000, 4099], 5000, 4095, 16)])
def test_decode_weights(lens, rows, left, sinks, nh, nkv, d):
    Bn = len(lens)
    q = _randn(1, Bn, nh, 1, d).to(BF16)
    k, v = _randn(2, Bn, nkv, rows, d).to(BF16), _randn(3, Bn, nkv, rows, d).to(BF16)
    before = torch.rand(Bn, nkv, rows, generator=_gen(4), device="cuda") * 3
    scale = d ** -0.5
    want, tol = _probabilities(q, k, lens, left, sinks, scale)
    seen = torch.zeros(Bn, rows, dtype=torch.bool, device="cuda")
    o, o_tol = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        n = max(0, min(n, rows))
        if n:
            seen[b, :n] = visible(1, n, n, left, 0, sinks, "cuda")[0]
            r = window_attention(q[b:b + 1], k[b:b + 1, :, :n], v[b:b + 1, :, :n], None, left, 0, sinks, scale)
            o[b], o_tol[b] = r["o"][0], r["o_tol"][0]
        k[b, :, ~seen[b]], v[b, :, ~seen[b]] = math.nan, math.inf  # what is not seen plays no part
    win = B.window_of(q, k, left, 0, sinks)
    got = []
    for _ in range(2):
        w, out = before.clone(), torch.full_like(q, 7.0)
        ws = torch.full((B.psa_window_attn_decode_weights_workspace_size(win),), 0xFF, dtype=torch.uint8, device="cuda")
        B.psa_window_attn_decode_weights(q, k, v, _i32(lens), out, w, ws, win, scale)
        got.append((out, w))
    out, w = got[0]
    within(out, o, o_tol, "o")
    # adding to what was there rounds once more
    within(w, before.double() + want, tol + U * (before.double() + want), "weights")
    assert torch.equal(w.transpose(0, 1)[:, ~seen], before.transpose(0, 1)[:, ~seen])
    assert torch.equal(out, got[1][0]) and torch.equal(w, got[1][1])


def test_decode_weights_of_a_strided_cache_and_sums_to_the_heads():
    Bn, nh, nkv, rows, d = 2, 8, 2, 500, 128
    q = _randn(5, Bn, nh, 1, d).to(BF16)
    packed = _randn(6, Bn, rows, 2 * nkv, d).to(BF16).transpose(1, 2)
    k, v = packed[:, :nkv], packed[:, nkv:]
    win = B.window_of(q, k)
    ws = torch.empty(B.psa_window_attn_decode_weights_workspace_size(win), dtype=torch.uint8, device="cuda")
    w, o = torch.zeros(Bn, nkv, rows, device="cuda"), torch.empty_like(q)
    lens = [500, 123]
    for _ in range(3):
        B.psa_window_attn_decode_weights(q, k, v, _i32(lens), o, w, ws, win, 0.1)
    want, tol = _probabilities(q, k, lens, -1, 0, 0.1)
    within(w, 3 * want, 3 * tol + 6 * U * want, "weights")
    assert ((w.sum(-1) - 3 * nh / nkv).abs() < 1e-4).all()


@pytest.mark.parametrize("rows", [15, 16, 17, 20, 31, 32])
@pytest.mark.parametrize("left,sinks", [(-1, 0), (5, 3)])
def test_decode_weights_over_short_caches(rows, left, sinks):
    """A last block that reaches back into the one before it, in caches that end inside their second block."""
    nh, nkv, d, scale, lens = 6, 2, 64, 0.125, [rows, rows - 1, 1, 16, 17]
    q, k = _randn(31, 5, nh, 1, d).to(BF16), _randn(32, 5, nkv, rows, d).to(BF16)
    v = _randn(33, 5, nkv, rows, d).to(BF16)
    want, tol = _probabilities(q, k, lens, left, sinks, scale)
    win = B.window_of(q, k, left, 0, sinks)
    ws = torch.full((B.psa_window_attn_decode_weights_workspace_size(win),), 0xFF, dtype=torch.uint8, device="cuda")
    w, o = torch.zeros(5, nkv, rows, device="cuda"), torch.full_like(q, 7.0)
    B.psa_window_attn_decode_weights(q, k, v, _i32(lens), o, w, ws, win, scale)
    within(w, want, tol + U * want, "weights")
    for b, n in enumerate(lens):
        n = min(n, rows)
        r = window_attention(q[b:b + 1], k[b:b + 1, :, :n], v[b:b + 1, :, :n], None, left, 0, sinks, scale)
        within(o[b:b + 1], r["o"], r["o_tol"], "o")
        assert (w[b, :, n:] == 0).all()


def test_a_nan_among_the_scores_shows_in_the_weights():
    q, k, v = _randn(7, 2, 4, 1, 64).to(BF16), _randn(8, 2, 2, 90, 64).to(BF16), _randn(9, 2, 2, 90, 64).to(BF16)
    k[0, 1, 40, 3] = math.nan
    win = B.window_of(q, k)
    ws = torch.empty(B.psa_window_attn_decode_weights_workspace_size(win), dtype=torch.uint8, device="cuda")
    w, o = torch.zeros(2, 2, 90, device="cuda"), torch.empty_like(q)
    B.psa_window_attn_decode_weights(q, k, v, _i32([90, 90]), o, w, ws, win, 0.2)
    assert w[0, 1].isnan().all() and o[0, 2:].isnan().all()
    assert w[0, 0].isfinite().all() and w[1].isfinite().all() and o[1].isfinite().all()


# ------------------------------------------------------------------ eviction
def _by_hand(w, pos, n, keep, sinks, recent):
    """Rows that stay, in their places afterwards."""
    w, pos = w[:n].cpu().tolist(), pos[:n].cpu().tolist()
    count, newest = min(n, keep), max(pos, default=0)

    def order(r):
        if pos[r] < sinks or pos[r] > newest - recent:
            return (0, 0.0, r)
        return (1, 0.0, r) if math.isnan(w[r]) else (2, -w[r], r)

    stay = set(sorted(range(n), key=order)[:count])
    gaps, come = [r for r in range(count) if r not in stay], sorted(r for r in stay if r >= count)
    place = list(range(count))
    for g, r in zip(gaps, come):
        place[g] = r
    return place


def _evict(c, keep, sinks, recent, in_place=False):
    """Runs it on copies; returns k, v, weights, positions, lens afterwards."""
    k, v = c["k"].clone(memory_format=torch.preserve_format), c["v"].clone(memory_format=torch.preserve_format)
    w, pos = c["w"].clone(), c["pos"].clone()
    w_out, pos_out = (w, pos) if in_place else (torch.full_like(w, 7.0), torch.full_like(pos, 7))
    lens_out = torch.full_like(c["lens"], 7)
    p = B.evict_of(k, keep, sinks, recent)
    ws = torch.full((B.psa_kv_evict_workspace_size(p),), 0xFF, dtype=torch.uint8, device="cuda")
    B.psa_kv_evict(w, pos, c["lens"], k, v, w_out, pos_out, lens_out, ws, p)
    if not in_place:
        assert torch.equal(w.view(torch.int32), c["w"].view(torch.int32)) and torch.equal(pos, c["pos"])
    return k, v, w_out, pos_out, lens_out


def _case(lens, rows, nkv, d, dtype, seed, kind="spread", strided=False):
    Bn = len(lens)
    shape = (Bn, rows, nkv, d) if strided else (Bn, nkv, rows, d)
    k, v = _randn(seed, *shape).to(dtype), _randn(seed + 1, *shape).to(dtype)
    if strided:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    w = torch.exp(2 * _randn(seed + 2, Bn, nkv, rows))
    if kind == "ties":  # many equal ones, both zeros among them
        w = (w * 2).round() / 2 * torch.where(_randn(seed + 3, Bn, nkv, rows) > 0, 1.0, -1.0) * (w < 2)
    elif kind == "equal":
        w = torch.full_like(w, 0.25)
    elif kind == "strange":
        pick = torch.randint(0, 6, w.shape, generator=_gen(seed + 4), device="cuda")
        for i, x in enumerate((math.nan, math.inf, -math.inf, 1e-40)):
            w = torch.where(pick == i, x, w)
    pos = torch.rand(Bn, nkv, rows, generator=_gen(seed + 5), device="cuda").argsort(-1)
    for b, n in enumerate(lens):  # positions 0 .. n - 1 in any order, then anything
        n = max(0, min(n, rows))
        pos[b, :, :n] = torch.rand(nkv, n, generator=_gen(seed + 6 + b), device="cuda").argsort(-1)
    return dict(k=k, v=v, w=w, pos=pos.int().contiguous(), lens=_i32(lens))


def _check(c, keep, sinks, recent, got, in_place):
    k, v, w, pos, lens = got
    was_w, was_pos = (c["w"], c["pos"]) if in_place else (torch.full_like(c["w"], 7.0), torch.full_like(c["pos"], 7))
    Bn, nkv, rows, d = k.shape
    for b in range(Bn):
        n = max(0, min(int(c["lens"][b]), rows))
        count = min(n, keep)
        assert int(lens[b]) == count
        for h in range(nkv):
            place = torch.tensor(_by_hand(c["w"][b, h], c["pos"][b, h], n, keep, sinks, recent), dtype=torch.long, device="cuda")
            bits = lambda t: t.contiguous().view(torch.int32)  # noqa: E731
            assert torch.equal(pos[b, h, :count], c["pos"][b, h, place]), (b, h)
            assert torch.equal(bits(w[b, h, :count]), bits(c["w"][b, h, place]))
            assert (w[b, h, count:n] == 0).all()
            assert torch.equal(bits(w[b, h, n:]), bits(was_w[b, h, n:])) and torch.equal(pos[b, h, count:], was_pos[b, h, count:])
            for x, old in ((k, c["k"]), (v, c["v"])):
                assert torch.equal(x[b, h, :count], old[b, h, place]) and torch.equal(x[b, h, count:], old[b, h, count:])


@pytest.mark.parametrize("rows,keep", [(700, 300), (700, 690), (50000, 20000)])
@pytest.mark.parametrize("same", ["weights", "positions"])
def test_one_of_the_lists_in_place(rows, keep, same):
    """Weights written where they were read and positions elsewhere, or the other way round."""
    c = _case([rows, rows - 300], rows, 2, 64, BF16, 19, "ties")
    want = _evict(c, keep, 4, 32)
    k, v, w, pos = (c[n].clone() for n in ("k", "v", "w", "pos"))
    w_out = w if same == "weights" else torch.full_like(w, 7.0)
    pos_out = pos if same == "positions" else torch.full_like(pos, 7)
    p, lens_out = B.evict_of(k, keep, 4, 32), torch.full_like(c["lens"], 7)
    ws = torch.full((B.psa_kv_evict_workspace_size(p),), 0xFF, dtype=torch.uint8, device="cuda")
    B.psa_kv_evict(w, pos, c["lens"], k, v, w_out, pos_out, lens_out, ws, p)
    for b, n in enumerate(c["lens"].tolist()):
        count = min(n, keep)
        assert torch.equal(w_out[b, :, :n], want[2][b, :, :n]) and torch.equal(pos_out[b, :, :count], want[3][b, :, :count])
    assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and torch.equal(lens_out, want[4])


# lens, rows, keep, sinks, recent: one kernel and two, threads by length, lists that end anywhere
CUTS = [([5], 5, 4, 0, 0), ([1, 0, 3, -2], 3, 1, 1, 0), ([40, 33, 7, 39], 40, 32, 4, 8), ([41, 40], 41, 8, 0, 0),
        ([1000, 999, 3, 500], 1000, 500, 4, 64), ([300], 300, 299, 2, 5), ([2049, 2048], 2049, 2048, 4, 64),
        ([4097, 2222], 4100, 1025, 0, 1024), ([9000, 8999], 9000, 4500, 4500, 0), ([5000], 6000, 5500, 1, 1),
        ([5000], 5000, 7000, 1, 1)]


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "strange"])
@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, BF16), (64, F32), (128, F32)])
@pytest.mark.parametrize("lens,rows,keep,sinks,recent", CUTS)
def test_evict(lens, rows, keep, sinks, recent, d, dtype, kind):
    strided = rows % 2 == 0
    c = _case(lens, rows, 3, d, dtype, rows + keep, kind, strided)
    for in_place in (False, True):
        _check(c, keep, sinks, recent, _evict(c, keep, sinks, recent, in_place), in_place)


@pytest.mark.parametrize("rows", [1024, 1025, 8192, 8193, 40960, 40961])
def test_lists_at_the_lengths_where_threads_and_places_change(rows):
    c = _case([rows, rows - 5], rows, 1, 64, BF16, 18, "ties" if rows % 2 else "spread")
    _check(c, rows // 3, 2, rows // 9, _evict(c, rows // 3, 2, rows // 9, True), True)


def test_lists_longer_than_shared_memory():
    c = _case([100001, 60000, 49153], 100001, 1, 64, BF16, 11)
    _check(c, 30000, 4, 1000, _evict(c, 30000, 4, 1000), False)
    c["w"] = (c["w"] * 4).round()
    _check(c, 99999, 4, 0, _evict(c, 99999, 4, 0, True), True)


def test_positions_that_are_not_distinct_or_not_there():
    """More rows than `keep` may claim to be safe: the lower ones of them stay."""
    c = _case([200, 150], 200, 2, 64, BF16, 12)
    c["pos"][:] = 3
    _check(c, 20, 5, 2, _evict(c, 20, 5, 2), False)
    c["pos"][:] = -2 ** 31
    _check(c, 20, 0, 7, _evict(c, 20, 0, 7), False)
    c["pos"][:] = torch.where(torch.arange(200, device="cuda") % 3 == 0, 2 ** 31 - 1, -2 ** 31).int()
    _check(c, 90, 0, 90, _evict(c, 90, 0, 90), False)


def test_caches_beyond_32_bit_offsets():
    rows, nkv = 1 << 20, 2
    k = torch.zeros(9, nkv, rows, 128, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    assert k[8].storage_offset() > 2 ** 31 - 1
    n, keep = rows - 3, rows - 103
    k[8], v[8] = _randn(13, nkv, rows, 128).to(BF16), _randn(14, nkv, rows, 128).to(BF16)
    w = torch.zeros(9, nkv, rows, device="cuda")
    w[8] = torch.rand(nkv, rows, generator=_gen(15), device="cuda")
    pos = torch.arange(rows, dtype=torch.int32, device="cuda").expand(9, nkv, -1).contiguous()
    lens, lens_out = _i32([5] * 8 + [n]), _i32([0] * 9)
    old = k[8].clone(), v[8].clone()
    p = B.evict_of(k, keep, 4, 32)
    ws = torch.empty(B.psa_kv_evict_workspace_size(p), dtype=torch.uint8, device="cuda")
    pos_out, w_out = pos.clone(), w.clone()
    B.psa_kv_evict(w, pos, lens, k, v, w_out, pos_out, lens_out, ws, p)
    assert lens_out.tolist() == [5] * 8 + [keep]
    for h in range(nkv):
        at = pos_out[8, h, :keep].long()  # positions are the old rows
        assert torch.equal(k[8, h, :keep], old[0][h, at]) and torch.equal(v[8, h, :keep], old[1][h, at])
        gone = torch.ones(n, dtype=torch.bool, device="cuda")
        gone[at] = False
        assert int(gone.sum()) == 100 and w[8, h, :n][gone].max() <= w_out[8, h, :keep].min().clamp(min=float(w[8, h, :n][gone].max()))
        assert int((at != torch.arange(keep, device="cuda")).sum()) <= 100
    assert (k[:8] == 0).all()


def test_which_rows_of_a_long_cache_stay():
    """Lists of 2^20 rows behind 32-bit offsets, with weights that are equal here and there: every output
    against a stable sort."""
    rows, nkv, b, sinks, recent = 1 << 20, 2, 8, 4, 32
    n, keep = rows - 3, rows - 103
    w = torch.rand(9, nkv, rows, generator=_gen(25), device="cuda")
    pos = torch.arange(rows, dtype=torch.int32, device="cuda").expand(9, nkv, -1).contiguous()
    pos[b, 1] = pos[b, 1].flip(0) - 3  # (the newest tokens in the first rows)
    k = torch.zeros(9, nkv, rows, 64, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    k[b], v[b] = _randn(26, nkv, rows, 64).to(BF16), _randn(27, nkv, rows, 64).to(BF16)
    assert k[b, 1].storage_offset() + k[b, 1].numel() > 2 ** 30 and k.numel() * 2 > 2 ** 31
    old = k[b].clone(), v[b].clone()
    lens, lens_out = _i32([5] * 8 + [n]), _i32([7] * 9)
    p = B.evict_of(k, keep, sinks, recent)
    ws = torch.full((B.psa_kv_evict_workspace_size(p),), 0xFF, dtype=torch.uint8, device="cuda")
    w_out, pos_out = torch.full_like(w, 7.0), torch.full_like(pos, 7)
    B.psa_kv_evict(w, pos, lens, k, v, w_out, pos_out, lens_out, ws, p)
    assert lens_out.tolist() == [5] * 8 + [keep]
    assert torch.equal(w_out[:b, :, :5], w[:b, :, :5]) and (w_out[:b, :, 5:] == 7).all() and (k[:b] == 0).all()
    for h in range(nkv):
        safe = (pos[b, h, :n] < sinks) | (pos[b, h, :n] > pos[b, h, :n].max() - recent)
        order = torch.where(safe, math.inf, w[b, h, :n]).sort(descending=True, stable=True).indices
        stays = torch.zeros(n, dtype=torch.bool, device="cuda")
        stays[order[:keep]] = True
        place = torch.arange(keep, device="cuda")
        place[~stays[:keep]] = keep + stays[keep:].nonzero()[:, 0]
        assert torch.equal(pos_out[b, h, :keep], pos[b, h, place]) and (pos_out[b, h, keep:] == 7).all()
        assert torch.equal(w_out[b, h, :keep], w[b, h, place])
        assert (w_out[b, h, keep:n] == 0).all() and (w_out[b, h, n:] == 7).all()
        for x, was in ((k, old[0]), (v, old[1])):
            assert torch.equal(x[b, h, :keep], was[h, place]) and torch.equal(x[b, h, keep:], was[h, keep:])


def test_on_another_stream_and_replayed():
    c = _case([900, 700], 900, 4, 128, BF16, 16)
    want = _evict(c, 400, 4, 50)
    k, v = c["k"].clone(), c["v"].clone()
    w_out, pos_out, lens_out = torch.full_like(c["w"], 7.0), torch.full_like(c["pos"], 7), torch.zeros_like(c["lens"])
    p = B.evict_of(k, 400, 4, 50)
    ws = torch.empty(B.psa_kv_evict_workspace_size(p), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.psa_kv_evict(c["w"], c["pos"], c["lens"], k, v, w_out, pos_out, lens_out, ws, p)
    for _ in range(2):  # sources are not written to: a second run moves the same rows again
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((k, v, w_out, pos_out, lens_out), want):
            assert torch.equal(x, y)


def test_refusals_of_the_binding():
    c = _case([9], 9, 1, 64, BF16, 17)
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")

    def call(keep=4, sinks=0, recent=0, ws=ws, **other):
        a = dict(weights=c["w"], positions=c["pos"], lens=c["lens"], k_cache=c["k"], v_cache=c["v"],
                 weights_out=c["w"].clone(), positions_out=c["pos"].clone(), lens_out=c["lens"].clone()) | other
        B.psa_kv_evict(**a, workspace=ws, p=B.evict_of(c["k"], keep, sinks, recent))

    call()
    for bad in (dict(keep=0), dict(keep=-3), dict(sinks=5), dict(recent=2 ** 40), dict(sinks=3, recent=2), dict(lens_out=c["lens"]),
                dict(ws=ws[:16])):
        with pytest.raises(B.PsaError):
            call(**bad)
    for bad in (dict(weights=None), dict(weights=c["w"][:, :, :8]), dict(positions=None), dict(v_cache=c["v"][:, :, :8]),
                dict(weights_out=c["w"].transpose(0, 1).expand(1, 1, 9)[:, :, ::2])):
        with pytest.raises((ValueError, B.PsaError)):
            call(**bad)
    with pytest.raises(TypeError):
        call(positions=c["pos"].long())
