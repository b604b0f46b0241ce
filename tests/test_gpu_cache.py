"""Single-token attention over a bf16 cache and over a 4-bit cache, and what fills and reads the
caches."""
import math

import pytest
import torch

from token_reference import dequantise, quantise, window_attention, within
from vision_transformer_attention_psapackqkv_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(seed, *shape):
    return torch.randn(*shape, generator=_gen(seed), device="cuda")


def _reference(q, k, v, lens, left, sinks, scale, kv4=False):
    """Row by row: the query of sequence b is the last of its lens[b] positions."""
    o, tol = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for b, n in enumerate(lens):
        n = max(0, min(n, k.shape[2]))
        if n == 0:
            continue
        r = window_attention(q[b:b + 1], k[b:b + 1, :, :n], v[b:b + 1, :, :n], None, left, 0, sinks, scale)
        o[b], tol[b] = r["o"][0], r["o_tol"][0]
    return o, tol


def _decode(q, k, v, lens, left, sinks, scale):
    win = B.window_of(q, k, left, 0, sinks)
    o = torch.full_like(q, 7.0)
    ws = torch.full((B.psa_window_attn_decode_workspace_size(win),), 0xFF, dtype=torch.uint8, device="cuda")
    B.psa_window_attn_decode(q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), o, ws, win, scale)
    return o


def _decode4(q, cache, lens, left, sinks, scale):
    win = B.window_of(q, cache[0], left, 0, sinks)
    o = torch.full_like(q, 7.0)
    ws = torch.full((B.psa_window_attn_decode_workspace_size(win),), 0xFF, dtype=torch.uint8, device="cuda")
    B.psa_window_attn_decode_kv4(q, *cache, torch.tensor(lens, dtype=torch.int32, device="cuda"), o, ws, win, scale)
    return o


# lens, cache rows, left, sinks
LENGTHS = [([1], 1, -1, 0), ([0, 1, 2, 17], 40, -1, 0), ([16, 15, 33, -4], 33, 7, 2), ([300, 129, 500, 64], 300, -1, 0),
           ([1000, 999, 5, 130], 1001, 63, 4), ([700, 350], 700, 100, 130), ([2000], 2100, 0, 0), ([2000], 2100, 0, 1),
           ([5000, 4097], 5000, -1, 0), ([5000, 4099], 5000, 4095, 16)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh,nkv", [(4, 2), (1, 1), (17, 1), (40, 8)])
@pytest.mark.parametrize("lens,rows,left,sinks", LENGTHS)
def test_decode(lens, rows, left, sinks, nh, nkv, d):
    Bn = len(lens)
    q = _randn(1, Bn, nh, 1, d).to(BF16)
    k, v = _randn(2, Bn, nkv, rows, d).to(BF16), _randn(3, Bn, nkv, rows, d).to(BF16)
    scale = d ** -0.5
    ref = _reference(q, k, v, lens, left, sinks, scale)
    for b, n in enumerate(lens):  # what lies behind a sequence, or between sinks and window, plays no part
        n = max(0, min(n, rows))
        k[b, :, n:], v[b, :, n:] = math.nan, math.inf
        if left >= 0:
            k[b, :, sinks:max(sinks, n - 1 - left)], v[b, :, sinks:max(sinks, n - 1 - left)] = math.inf, math.nan
    o = _decode(q, k, v, lens, left, sinks, scale)
    within(o, *ref, "o")
    assert torch.equal(o, _decode(q, k, v, lens, left, sinks, scale))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh,nkv", [(4, 2), (1, 1), (17, 1), (40, 8)])
@pytest.mark.parametrize("lens,rows,left,sinks", LENGTHS)
def test_decode_kv4(lens, rows, left, sinks, nh, nkv, d):
    Bn = len(lens)
    q = _randn(1, Bn, nh, 1, d).to(BF16)
    cache = quantise(_randn(2, Bn, nkv, rows, d)) + quantise(_randn(3, Bn, nkv, rows, d))
    scale = d ** -0.5
    k, v = dequantise(*cache[:2]), dequantise(*cache[2:])
    o, tol = _reference(q, k, v, lens, left, sinks, scale)
    for b, n in enumerate(lens):
        n = max(0, min(n, rows))
        cache[1][b, :, n:], cache[3][b, :, n:] = math.nan, math.inf
        cache[0][b, :, n:], cache[2][b, :, n:] = 0xFF, 0x0F
    got = _decode4(q, cache, lens, left, sinks, scale)
    within(got, o, tol, "o")
    assert torch.equal(got, _decode4(q, cache, lens, left, sinks, scale))


def test_every_code_and_a_cache_of_strange_scales():
    """All sixteen codes (an append writes fifteen), scales from tiny to large."""
    d, rows = 128, 64
    codes = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8).repeat(rows * d // 512).view(1, 1, rows, d // 2)
    scales = (2.0 ** torch.randint(-30, 3, (1, 1, rows, d // 32), generator=_gen(4), device="cuda")).to(BF16)
    q = _randn(5, 1, 4, 1, d).to(BF16)
    cache = (codes, scales, codes.flip(2).contiguous(), scales.flip(2).contiguous())
    o, tol = _reference(q, dequantise(*cache[:2]), dequantise(*cache[2:]), [rows], -1, 0, 0.05)
    within(_decode4(q, cache, [rows], -1, 0, 0.05), o, tol, "o")


def test_a_cache_beyond_32_bit_offsets():
    """The last sequence's rows lie more than 2^31 elements behind the cache's first."""
    nkv, rows, d = 2, 1 << 20, 128
    k = torch.zeros(9, nkv, rows, d, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    assert k[8].storage_offset() > 2 ** 31 - 1
    q = _randn(6, 9, 4, 1, d).to(BF16)
    n = rows - 3
    k[8, :, n - 700:n], v[8, :, n - 700:n] = _randn(7, nkv, 700, d).to(BF16), _randn(8, nkv, 700, d).to(BF16)
    o = _decode(q, k, v, [1] * 8 + [n], 699, 0, 0.09)
    r = window_attention(q[8:], k[8:, :, n - 700:n], v[8:, :, n - 700:n], None, 699, 0, 0, 0.09)
    within(o[8:], r["o"], r["o_tol"], "o")
    assert (o[:8] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,rows,starts,counts", [(1, 9, [8, 0], None), (5, 40, [0, 33], [5, 3]),
                                                  (70, 64, [-6, 10], None), (200, 300, [99, 7], [200, 0])])
def test_append_and_read(N, rows, starts, counts, d, dtype):
    Bn, nkv = 2, 3
    packed = (_randn(9, Bn, N, 2 * nkv, d) * torch.exp(_randn(10, d))).to(dtype).transpose(1, 2)
    k, v = packed[:, :nkv], packed[:, nkv:]
    k[0, 0, 0], v[1, 2, N - 1] = 0.0, 1e30
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    ct = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    kc, vc = (_randn(s, Bn, nkv, rows, d).to(dtype) for s in (11, 12))
    cache = quantise(_randn(13, Bn, nkv, rows, d)) + quantise(_randn(14, Bn, nkv, rows, d))
    want, want4 = [kc.clone(), vc.clone()], [t.clone() for t in cache]
    new4 = quantise(k) + quantise(v)
    for b in range(Bn):
        for n in range(N if counts is None else counts[b]):
            r = starts[b] + n
            if not 0 <= r < rows:
                continue
            want[0][b, :, r], want[1][b, :, r] = k[b, :, n], v[b, :, n]
            for t, x in zip(want4, new4):
                t[b, :, r] = x[b, :, n]
    B.psa_kv_append(k, v, st, ct, kc, vc)
    B.psa_kv4_append(k, v, st, ct, *cache)
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    assert all(torch.equal(a, b) for a, b in zip(cache, want4))
    ko, vo = (torch.full((Bn, nkv, rows, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    B.psa_kv4_read(*cache, ko, vo)
    assert torch.equal(ko, dequantise(*cache[:2]).to(dtype)) and torch.equal(vo, dequantise(*cache[2:]).to(dtype))
    few = torch.full((Bn, rows + 2, nkv, d), 7.0, dtype=dtype, device="cuda")  # the first rows, into a view
    front = few[:, 1:rows].transpose(1, 2)
    B.psa_kv4_read(*cache, front, vo[:, :, :rows - 1])
    assert torch.equal(front, ko[:, :, :rows - 1]) and (few[:, 0] == 7.0).all() and (few[:, rows:] == 7.0).all()


def test_quotients_near_ties():
    """Codes of many values, exact ties and their neighbours among them, and of scales from the
    smallest to the largest, against the division of the format's definition."""
    x = _randn(16, 1, 2, 8192, 128) * torch.exp2(torch.randint(-140, 120, (1, 2, 8192, 1), generator=_gen(17), device="cuda").float())
    top = x[..., :32].abs().amax(-1, keepdim=True)
    scale = (top * torch.full_like(top, 1 / 7)).to(BF16).float()
    half = (torch.randint(-7, 7, (1, 2, 8192, 16), generator=_gen(18), device="cuda") + 0.5) * scale  # exact
    x[..., 1:17] = torch.where(x[..., 1:17].abs() <= x[..., :32].abs().amax(-1, keepdim=True), half, x[..., 1:17])
    bits = x[..., 9:17].contiguous().view(torch.int32)
    x[..., 9:17] = (bits + torch.randint(-1, 2, bits.shape, generator=_gen(19), device="cuda", dtype=torch.int32)).view(torch.float32)
    x = torch.where(torch.isfinite(x), x, 1.0)
    cache = tuple(torch.zeros(1, 2, 8192, n, dtype=t, device="cuda") for n, t in ((64, torch.uint8), (4, BF16)) * 2)
    B.psa_kv4_append(x, -x, torch.zeros(1, dtype=torch.int32, device="cuda"), None, *cache)
    for got, want in zip(cache, quantise(x) + quantise(-x)):
        assert torch.equal(got, want)


def test_values_that_are_not_finite_do_not_read_back_as_finite():
    k = _randn(15, 1, 1, 4, 64)
    k[0, 0, 1, 3], k[0, 0, 2, 40] = math.nan, math.inf
    cache = tuple(torch.zeros(1, 1, 4, n, dtype=t, device="cuda") for n, t in ((32, torch.uint8), (2, BF16)) * 2)
    B.psa_kv4_append(k, k, torch.zeros(1, dtype=torch.int32, device="cuda"), None, *cache)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    B.psa_kv4_read(*cache, ko, vo)
    assert torch.isfinite(ko[0, 0, [0, 3]]).all()
    assert not torch.isfinite(ko[0, 0, 1, :32]).any() and torch.isfinite(ko[0, 0, 1, 32:]).all()
    assert not torch.isfinite(ko[0, 0, 2, 32:]).any() and torch.isfinite(ko[0, 0, 2, :32]).all()


@pytest.mark.parametrize("rows", [20, 40, 3000])
def test_a_nan_that_is_seen_stays_one(rows):
    """One among the scores, or the query's own: not the zeros of a row that sees nothing."""
    d = 64
    q = _randn(31, 2, 4, 1, d).to(BF16)
    k, v = _randn(32, 2, 2, rows, d).to(BF16), _randn(33, 2, 2, rows, d).to(BF16)
    lens = [rows, rows - 3]
    clean = _decode(q, k, v, lens, -1, 0, 0.2)
    cache = quantise(k) + quantise(v)
    clean4 = _decode4(q, cache, lens, -1, 0, 0.2)
    k[0, 1, rows // 2, 5] = math.nan
    cache[1][0, 1, rows // 2, 0] = math.nan
    for o, was in ((_decode(q, k, v, lens, -1, 0, 0.2), clean), (_decode4(q, cache, lens, -1, 0, 0.2), clean4)):
        assert o[0, 2:].isnan().all()
        assert torch.equal(o[0, :2], was[0, :2]) and torch.equal(o[1], was[1])
    q[1, 3, 0, 0] = math.nan
    for o, was in ((_decode(q, k, v, lens, -1, 0, 0.2), clean), (_decode4(q, cache, lens, -1, 0, 0.2), clean4)):
        # (head 2 shares its products with head 3, and the steps at which maxima move)
        assert o[1, 3].isnan().all() and torch.equal(o[1, :2], was[1, :2]) and o[1, 2].isfinite().all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh", [4, 24])
@pytest.mark.parametrize("size", [10.0, 100.0, 1000.0])
def test_4_bit_scores_of_large_one_signed_queries(size, nh, d):
    """Half of a query's channels are large and of one sign, and meet one large code in every group, so
    that all keys' scores are large and alike; what tells them apart is in the other half."""
    Bn, rows, G = 32, 8, d // 32
    large = torch.arange(d, device="cuda") % 32 < 16
    q = torch.where(large, size, 0.1 * _randn(51, Bn, nh, 1, d)).to(BF16)
    k = torch.where(large, 0.0, (7 * _randn(52, Bn, 1, rows, d)).round().clamp(-7, 7)).unflatten(-1, (G, 32))
    k.scatter_(-1, torch.randint(0, 16, (Bn, 1, rows, G, 1), generator=_gen(53), device="cuda"), 7.0)
    step = 1.0 + torch.randint(0, 2, (Bn, 1, rows, 1, 1), generator=_gen(54), device="cuda")
    k = (k * torch.cat([step, 3 - step] * (G // 2), 3)).flatten(-2)
    cache = quantise(k) + quantise(_randn(55, Bn, 1, rows, d))
    assert torch.equal(dequantise(*cache[:2]), k.double())
    lens, scale = [rows] * Bn, d ** -0.5
    within(_decode4(q, cache, lens, -1, 0, scale), *_reference(q, k, dequantise(*cache[2:]), lens, -1, 0, scale), "o")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh", [4, 24])
@pytest.mark.parametrize("e", [4, 12, 40])
def test_4_bit_scores_of_groups_of_unlike_sizes(e, nh, d):
    """Channels that are large in the queries are small in the keys, and the other way round."""
    rows, lens, scale = 600, [600, 391], d ** -0.5
    up = torch.where(torch.arange(d, device="cuda") // 32 % 2 == 0, 2.0 ** e, 2.0 ** -e)
    q = (_randn(61, 2, nh, 1, d) * up).to(BF16)
    cache = quantise(_randn(62, 2, 2, rows, d) / up) + quantise(_randn(63, 2, 2, rows, d))
    within(_decode4(q, cache, lens, -1, 0, scale),
           *_reference(q, dequantise(*cache[:2]), dequantise(*cache[2:]), lens, -1, 0, scale), "o")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh,nkv", [(4, 2), (40, 2)])
def test_maxima_that_jump_from_block_to_block(nh, nkv, d):
    """Scores that rise, or fall, by far more than 2^8 along the cache, in bf16 and in 4 bits."""
    rows, scale = 900, 0.5
    u = _randn(41, d)
    u /= u.norm()
    q = (_randn(42, 2, nh, 1, d) * 0.3 + 8 * u).to(BF16)
    ramp = torch.linspace(-20, 20, rows, device="cuda")[:, None] * u
    k, v = _randn(43, 2, nkv, rows, d) * 0.3 + ramp, _randn(44, 2, nkv, rows, d).to(BF16)
    k[1] = k[1].flip(1)
    k = k.to(BF16)
    lens = [rows, rows - 17]
    within(_decode(q, k, v, lens, -1, 0, scale), *_reference(q, k, v, lens, -1, 0, scale), "o")
    cache = quantise(k) + quantise(v)
    within(_decode4(q, cache, lens, -1, 0, scale),
           *_reference(q, dequantise(*cache[:2]), dequantise(*cache[2:]), lens, -1, 0, scale), "o4")
