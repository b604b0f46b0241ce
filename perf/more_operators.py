"""Operators of a transformer over images and video and of the caches that serve it: the calls that
are measured, their plain forms in elementary torch operations, and their values in 64 bits.

  axes     norms of queries and keys for each head with a position rotation whose channels turn with
           several axes (time, height, width)  (psa_qk_norm_rope_axes_fwd / _bwd)
  prefix   attention of a batch whose sequences share a long prefix, which is read once for all
           (psa_prefix_attn_fwd, and psa_prefix_attn_decode for single tokens)
  evict    attention weights summed for each key of a cache (psa_window_attn_weights over a prompt,
           psa_window_attn_decode_weights along with a decoding step) and the eviction of the keys
           that have least of them (psa_kv_evict)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoding step of 64 sequences behind images: a latency-bound call
        dict(name="axes_step", op="axes_fwd", dtype="bf16", B=64, nh=32, nkv=8, N=1, d=128, rot=128, sections="16,24,24",
             alternate=True, grid="", table=4096, norm=True),
        # a long video clip, 16 frames of 32 x 32 patches, positions from the grid itself
        dict(name="axes_video", op="axes_fwd", dtype="bf16", B=1, nh=32, nkv=8, N=16384, d=128, rot=128,
             sections="16,24,24", alternate=False, grid="16,32,32", table=32, norm=True),
        # training on images and their captions, odd length, explicit positions
        dict(name="axes_train", op="axes_bwd", dtype="bf16", B=4, nh=16, nkv=16, N=2301, d=64, rot=64, sections="8,12,12",
             alternate=True, grid="", table=2304, norm=True),
        # 20 x 20 feature maps in fp32, two axes, no norms, neighbouring channels turned, training
        dict(name="axes_map_f32", op="axes_bwd", dtype="f32", B=16, nh=4, nkv=4, N=400, d=64, rot=64, sections="16,16",
             alternate=False, grid="20,20", table=20, norm=False),
        # 64 users' decoding step over one long document
        dict(name="prefix_decode_batch", op="prefix_decode", dtype="bf16", B=64, nh=32, nkv=8, P=16384, Nq=1, Nk=1024,
             d=128, ragged=True),
        # a few samples of one answer behind a short odd prompt: a latency-bound call
        dict(name="prefix_decode_few", op="prefix_decode", dtype="bf16", B=4, nh=8, nkv=2, P=2001, Nq=1, Nk=100, d=64,
             ragged=True),
        # questions of unequal lengths about one video
        dict(name="prefix_questions", op="prefix_fwd", dtype="bf16", B=16, nh=32, nkv=8, P=8192, Nq=77, Nk=77, d=128,
             ragged=True),
        # what the keys of two prompts got, before the first eviction
        dict(name="weights_prompt", op="weights", dtype="bf16", B=2, nh=16, nkv=4, Nq=4096, Nk=4096, d=128, left=-1,
             right=0, sinks=0, ragged=False),
        # the same from the last 32 queries of a long prompt alone
        dict(name="weights_last_queries", op="weights", dtype="bf16", B=1, nh=32, nkv=8, Nq=32, Nk=16001, d=128, left=-1,
             right=0, sinks=0, ragged=False),
        # a decoding step of 16 sequences that keeps account
        dict(name="decode_weights", op="decode_weights", dtype="bf16", B=16, nh=32, nkv=8, Nk=8192, d=128, left=-1,
             sinks=0, ragged=True),
        # caches that have grown to their limit are cut to half
        dict(name="evict_half", op="evict", dtype="bf16", B=8, nkv=8, Nk=16384, d=128, keep=8192, sinks=4, recent=512,
             ragged=True),
        # each step evicts one key for the one that came
        dict(name="evict_one", op="evict", dtype="bf16", B=32, nkv=8, Nk=2049, d=128, keep=2048, sinks=4, recent=64,
             ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes_fwd", "axes_bwd", "prefix_decode", "prefix_decode", "prefix_fwd", "weights", "weights",
                     "decode_weights", "evict", "evict"])
    d = rng.choice([64, 128])
    nkv = rng.choice([1, 2, 4, 8])
    nh = nkv * rng.choice([1, 2, 4, 5, 8])
    ragged = rng.random() < 0.5
    if op.startswith("axes"):
        B = rng.choice([1, 2, 3, 8])
        rot = rng.choice([32, d // 2, d])
        axes = rng.choice([2, 3])
        cuts = sorted(rng.sample(range(1, rot // 2), axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [rot // 2])]
        most = max(1, 600000 // (B * (nh + nkv)))
        if rng.random() < 0.5:
            grid = [max(1, _log(rng, 1, 40)) for _ in range(axes)]
            while math.prod(grid) > min(most, 16384):
                grid = [max(1, g * 3 // 4) for g in grid]
            N, table = math.prod(grid), max(grid) + rng.randrange(30)
        else:
            grid, N = [], min(_log(rng, 1, 16384), most)
            table = N + rng.randrange(5000)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, nh=nh, nkv=nkv, N=N, d=d, rot=rot,
                    sections=",".join(map(str, sections)), alternate=rng.random() < 0.5, grid=",".join(map(str, grid)),
                    table=table, norm=rng.random() < 0.7)
    if op == "prefix_decode":
        B = rng.choice([1, 2, 5, 16, 40, 64, 100])
        P = min(_log(rng, 1, 32768), (1 << 25) // (B * nh))
        Nk = min(_log(rng, 1, 2048), (1 << 19) // (B * nkv))
        return dict(op=op, dtype="bf16", B=B, nh=nh, nkv=nkv, P=P, Nq=1, Nk=Nk, d=d, ragged=ragged)
    if op == "prefix_fwd":
        B, Nq = rng.choice([1, 3, 8, 16]), _log(rng, 1, 400)
        P = min(_log(rng, 1, 16384), max(1, (1 << 28) // (B * nh * Nq)))
        return dict(op=op, dtype="bf16", B=B, nh=nh, nkv=nkv, P=P, Nq=Nq, Nk=Nq + rng.choice([0, 0, rng.randrange(200)]),
                    d=d, ragged=ragged)
    left, sinks = rng.choice([-1, -1, _log(rng, 1, 4096)]), rng.choice([0, 1, 4, 130])
    if op == "weights":
        B, Nk = rng.choice([1, 2, 3]), _log(rng, 1, 16384)
        Nq = rng.choice([Nk, min(Nk, _log(rng, 1, 64))])
        while B * nh * Nq * Nk > (1 << 28) and Nk > 16:
            B, Nk = max(1, B // 2), Nk * 3 // 4
            Nq = min(Nq, Nk)
        return dict(op=op, dtype="bf16", B=B, nh=nh, nkv=nkv, Nq=Nq, Nk=Nk, d=d, left=left, right=rng.choice([0, 0, 25]),
                    sinks=sinks, ragged=ragged)
    if op == "decode_weights":
        B = rng.choice([1, 3, 8, 16])
        Nk = min(_log(rng, 1, 32768), (1 << 20) // (B * nkv))
        return dict(op=op, dtype="bf16", B=B, nh=nh, nkv=nkv, Nk=Nk, d=d, left=left, sinks=sinks, ragged=ragged)
    B = rng.choice([1, 2, 8, 32])
    Nk = min(_log(rng, 8, 65536), (1 << 20) // (B * nkv))
    keep = rng.choice([max(1, Nk - 1), max(1, Nk // 2), max(1, Nk // 4 + rng.randrange(Nk // 2))])
    sinks = min(sinks, keep // 2)
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, nkv=nkv, Nk=Nk, d=d, keep=keep, sinks=sinks,
                recent=rng.choice([0, (keep - sinks) // 8, keep - sinks]), ragged=ragged)


def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _lens(c, n):
    """Valid lengths of the batch's sequences: the longest is whole, the others fall off unevenly."""
    if not c["ragged"]:
        return [n] * c["B"]
    return [max(1, n - (b * (2 * n // 7 + 1)) % (3 * n // 4 + 1)) for b in range(c["B"])]


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(nq, nk, length, left, right, sinks):
    """Numbers of visible (query, key) pairs and of keys that some query sees, one sequence."""
    p = torch.arange(nq, dtype=torch.int64) + (nk - nq)
    p = p[(p >= 0) & (p < length)]
    if p.numel() == 0:
        return 0, 0
    hi = torch.full_like(p, length - 1) if right < 0 else (p + right).clamp(max=length - 1)
    lo = torch.zeros_like(p) if left < 0 else (p - left).clamp(min=0)
    first = torch.minimum(lo, hi + 1).clamp(max=sinks)  # sinks in front of the window
    return int(((hi - lo + 1).clamp(min=0) + first).sum()), int(hi.max()) + 1 - int(lo.min()) + min(sinks, int(lo.min()))


def work(c):
    e, d, B = 2 if c["dtype"] == "bf16" else 4, c["d"], c["B"]
    if c["op"].startswith("axes"):
        rows = B * c["N"] * (c["nh"] + c["nkv"])
        small = min(c["table"], B * c["N"]) * c["rot"] * 4 + (0 if c["grid"] else 4 * len(_ints(c["sections"])) * B * c["N"])
        if c["op"] == "axes_fwd":
            return {"bytes": rows * d * e * 2 + small, "flops": rows * d * 8}
        # without norms the inputs play no part in their gradients
        return {"bytes": rows * d * e * (3 if c["norm"] else 2) + small, "flops": rows * d * 16}
    if c["op"].startswith("prefix"):
        shared, rows = 2 * c["P"] * c["nkv"] * d * e, B * c["Nq"] * c["nh"] * d * e
        pairs, keys, valid = 0, 0, 0
        for n in _lens(c, c["Nk"]):
            a, b = (n, n) if c["op"] == "prefix_decode" else _pairs(c["Nq"], c["Nk"], n, -1, 0, 0)
            pairs, keys = pairs + a, keys + b
            valid += 1 if c["op"] == "prefix_decode" else max(0, min(c["Nq"], n - (c["Nk"] - c["Nq"])))
        lse = 0 if c["op"] == "prefix_decode" else B * c["Nq"] * c["nh"] * 4
        return {"bytes": shared + 2 * rows + 2 * keys * c["nkv"] * d * e + lse,
                "flops": 4 * d * c["nh"] * (pairs + valid * c["P"])}
    if c["op"] == "weights":
        pairs = keys = valid = 0
        for n in _lens(c, c["Nk"]):
            a, b = _pairs(c["Nq"], c["Nk"], n, c["left"], c["right"], c["sinks"])
            pairs, keys = pairs + a, keys + b
            valid += max(0, min(c["Nq"], n - (c["Nk"] - c["Nq"])))
        return {"bytes": valid * c["nh"] * (d * e + 4) + keys * c["nkv"] * (d * e + 8), "flops": 2 * d * c["nh"] * pairs}
    if c["op"] == "decode_weights":
        keys = sum(_pairs(1, n, n, c["left"], 0, c["sinks"])[1] for n in _lens(c, c["Nk"]))
        return {"bytes": keys * c["nkv"] * (2 * d * e + 8) + 2 * B * c["nh"] * d * e, "flops": 4 * d * c["nh"] * keys}
    total = 0
    for n in _lens(c, c["Nk"]):
        kept, safe = min(n, c["keep"]), c["sinks"] + c["recent"]
        tail = n - kept
        # rows behind the first `kept` that stay: the recent ones, and their share of the others
        moved = min(c["recent"], tail) + max(0, tail - c["recent"]) * (kept - safe) / max(1, n - safe) if tail else 0
        total += c["nkv"] * (8 * n + 8 * kept + 4 * tail + moved * 4 * d * e)
    return {"bytes": total, "flops": 0}


# ------------------------------------------------------------------ inputs
def _axes_inputs(c, gen):
    B, nh, nkv, N, d, dt = c["B"], c["nh"], c["nkv"], c["N"], c["d"], DTYPES[c["dtype"]]
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    # the projection's output, [B, N, heads of q | k | v, d], of which q and k are views
    packed = (rn(B, N, nh + 2 * nkv, d) * 1.5).to(dt).transpose(1, 2)
    half, sections = c["rot"] // 2, _ints(c["sections"])
    freq = 1e4 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(c["table"], dtype=torch.float64, device="cuda")[:, None] * freq
    w = lambda: 1 + 0.2 * rn(d) if c["norm"] else None  # noqa: E731
    s = dict(c=c, q=packed[:, :nh], k=packed[:, nh:nh + nkv], wq=w(), wk=w(), cos=angle.cos().float().contiguous(),
             sin=angle.sin().float().contiguous(), eps=1e-6, pos=None, sections=sections, grid=_ints(c["grid"]))
    if not s["grid"]:
        s["pos"] = torch.randint(0, c["table"], (len(sections), B, N), generator=gen, device="cuda", dtype=torch.int32)
    if c["op"] == "axes_bwd":
        s["gq"], s["gk"] = rn(B, nh, N, d).to(dt), rn(B, nkv, N, d).to(dt)
    return s


def _prefix_inputs(c, gen):
    B, nh, nkv, d = c["B"], c["nh"], c["nkv"], c["d"]
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    return dict(c=c, q=rn(B, nh, c["Nq"], d), kp=rn(1, nkv, c["P"], d), vp=rn(1, nkv, c["P"], d),
                k=rn(B, nkv, c["Nk"], d), v=rn(B, nkv, c["Nk"], d), scale=d ** -0.5,
                lens=torch.tensor(_lens(c, c["Nk"]), dtype=torch.int32, device="cuda"))


def _weights_inputs(c, gen):
    B, nh, nkv, d = c["B"], c["nh"], c["nkv"], c["d"]
    Nq = c.get("Nq", 1)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    s = dict(c=c, q=rn(B, nh, Nq, d), k=rn(B, nkv, c["Nk"], d), scale=d ** -0.5,
             lens=torch.tensor(_lens(c, c["Nk"]), dtype=torch.int32, device="cuda"),
             weights=torch.rand(B, nkv, c["Nk"], generator=gen, device="cuda"))
    if c["op"] == "decode_weights":
        s["v"] = rn(B, nkv, c["Nk"], d)
        return s
    see = _mask(c, s["lens"])  # what the forward left behind
    x = _scores(s["q"], s["k"], s["scale"], see)
    s["lse"] = torch.logsumexp(x.double() if x.numel() < 1 << 27 else x, -1).float().flatten(1, 2)
    return s


def _evict_inputs(c, gen):
    B, nkv, L, d, dt = c["B"], c["nkv"], c["Nk"], c["d"], DTYPES[c["dtype"]]
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    rows = torch.arange(L, device="cuda")
    # rows have been moved by earlier evictions: each position stands somewhere, the newest ones behind
    lens = torch.tensor(_lens(c, L), device="cuda")[:, None, None]
    old = min(c["keep"], L)
    mixed = torch.rand(B, nkv, old, generator=gen, device="cuda")
    mixed = mixed.masked_fill(rows[:old] >= lens, 2).argsort(-1)
    positions = torch.cat([mixed, rows[old:].expand(B, nkv, -1)], -1)
    return dict(c=c, k=rn(B, nkv, L, d).to(dt), v=rn(B, nkv, L, d).to(dt), weights=torch.exp(2 * rn(B, nkv, L)),
                positions=positions.int().contiguous(), lens=lens.flatten().int(),
                weights_out=torch.zeros(B, nkv, L, device="cuda"),
                positions_out=torch.zeros(B, nkv, L, dtype=torch.int32, device="cuda"),
                lens_out=torch.zeros(B, dtype=torch.int32, device="cuda"))


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if c["op"].startswith("axes"):
        return _axes_inputs(c, gen)
    if c["op"].startswith("prefix"):
        return _prefix_inputs(c, gen)
    return _evict_inputs(c, gen) if c["op"] == "evict" else _weights_inputs(c, gen)


# ------------------------------------------------------------------ plain forms
def _axis_of_pairs(sections, alternate):
    """Which axis each pair of channels turns with: the axes' sections one behind the other, or the
    axes in turn for as long as each has pairs left."""
    if not alternate:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    order = [(i, a) for a, n in enumerate(sections) for i in range(n)]
    return [a for _, a in sorted(order)]


def _positions(s):
    """[axes, B or 1, N]"""
    if s["pos"] is not None:
        return s["pos"].long()
    n, out = torch.arange(s["c"]["N"], device="cuda"), []
    for extent in reversed(s["grid"]):
        out.append(n % extent)
        n = n // extent
    return torch.stack(out[::-1])[:, None]


def _angles(s, sign):
    """cos and sin of each row's angles, [B or 1, 1, N, rot / 2]."""
    axis = torch.tensor(_axis_of_pairs(s["sections"], s["c"]["alternate"]), device="cuda")
    at = _positions(s)[axis].movedim(0, -1)  # [B or 1, N, rot / 2]
    cos, sin = (t.gather(0, at.flatten(0, 1)).view(at.shape)[:, None] for t in (s["cos"], s["sin"]))
    return cos, sign * sin


def _pairwise(c):
    """Whether neighbouring channels are pairs (the feature maps of fp32), or those half a rotation apart."""
    return c["dtype"] == "f32"


def _rotate(x, cos, sin, c):
    rot = c["rot"]
    r, rest = x[..., :rot], x[..., rot:]
    if _pairwise(c):
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([r, rest], -1)


def _axes_fwd(s):
    cos, sin = _angles(s, 1)

    def one(x, w):
        y = x.float()
        if s["c"]["norm"]:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w
        return _rotate(y, cos, sin, s["c"]).to(x.dtype)

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _axes_bwd(s):
    cos, sin = _angles(s, -1)

    def one(x, w, g):
        gy = _rotate(g.float(), cos, sin, s["c"])
        if not s["c"]["norm"]:
            return (gy.to(x.dtype),)
        x32 = x.float()
        r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + s["eps"])
        xh, gx = x32 * r, gy * w
        dx = r * (gx - xh * (gx * xh).mean(-1, keepdim=True))
        return dx.to(x.dtype), (gy * xh).double().sum((0, 1, 2)).float()

    return one(s["q"], s["wq"], s["gq"]) + one(s["k"], s["wk"], s["gk"])


def _mask(c, lens):
    """What each query sees of its own keys, [B, 1, 1, nq, nk]."""
    nq, nk = c.get("Nq", 1), c["Nk"]
    j = torch.arange(nk, device="cuda")[None, None]
    if c["op"] in ("decode_weights", "prefix_decode"):  # the query is the sequence's last token
        p = lens.long()[:, None, None] - 1
    else:
        p = torch.arange(nq, device="cuda")[None, :, None] + (nk - nq)
    see = (j < lens[:, None, None]) & (p < lens[:, None, None]) & (p >= 0)
    left, right = c.get("left", -1), c.get("right", 0)
    if left >= 0:
        see = see & ((j >= p - left) | (j < c["sinks"]))
    if right >= 0:
        see = see & (j <= p + right)
    return see[:, None, None]


def _scores(q, k, scale, see):
    """[B, kv heads, group, nq, nk] in 32 bits, -inf where masked."""
    x = q.float().unflatten(1, (k.shape[1], -1)) @ k.float()[:, :, None].mT
    return (x * scale).masked_fill(~see, -math.inf)


def _prefix(s):
    c, nkv = s["c"], s["c"]["nkv"]
    own_keys = _scores(s["q"], s["k"], s["scale"], _mask(c, s["lens"]))
    at = torch.arange(c["Nq"], device="cuda") + c["Nk"] - c["Nq"]
    if c["op"] == "prefix_decode":  # the query is each sequence's last token
        at = s["lens"][:, None] - 1
    valid = (at < s["lens"][:, None])[:, None, None, :, None]
    # all sequences' queries of a key/value head against the prefix at once
    rows = s["q"].float().unflatten(1, (nkv, -1)).transpose(0, 1).flatten(1, 3)
    shared = (rows @ s["kp"][0].float().mT * s["scale"]).unflatten(1, (c["B"], -1, c["Nq"])).transpose(0, 1)
    m = torch.maximum(shared.amax(-1, keepdim=True), own_keys.amax(-1, keepdim=True))
    a, b = torch.exp(shared - m), torch.exp(own_keys - m)
    total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
    o = (a.transpose(0, 1).flatten(1, 3) @ s["vp"][0].float()).unflatten(1, (c["B"], -1, c["Nq"])).transpose(0, 1)
    o = torch.where(valid, (o + b @ s["v"].float()[:, :, None]) / total, 0).flatten(1, 2).to(s["q"].dtype)
    if c["op"] == "prefix_decode":
        return o
    return o, torch.where(valid, m + torch.log(total), -math.inf).flatten(1, 2).squeeze(-1)


def _weights(s):
    x = _scores(s["q"], s["k"], s["scale"], _mask(s["c"], s["lens"]))
    lse = s["lse"].unflatten(1, (s["c"]["nkv"], -1))[..., None]
    s["weights"] += torch.exp(x - torch.where(lse == -math.inf, 0, lse)).sum((2, 3))
    return s["weights"]


def _decode_weights(s):
    x = _scores(s["q"], s["k"], s["scale"], _mask(s["c"], s["lens"]))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    s["weights"] += p.sum((2, 3))
    return (p @ s["v"].float()[:, :, None]).flatten(1, 2).to(s["q"].dtype), s["weights"]


def _evict(s):
    c, L, lens = s["c"], s["c"]["Nk"], s["lens"].long()[:, None, None]
    row = torch.arange(L, device="cuda")[None, None]
    there, pos = row < lens, s["positions"].long()
    newest = pos.masked_fill(~there, -1).amax(-1, keepdim=True)
    safe = (pos < c["sinks"]) | (pos > newest - c["recent"])
    key = s["weights"].masked_fill(safe, math.inf).masked_fill(~there, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    count = lens.clamp(max=c["keep"])
    kept = torch.zeros_like(there.expand_as(pos)).scatter(-1, order, (row < count).expand_as(pos))
    hole, mover = ~kept & (row < count), kept & (row >= count)
    movers = torch.sort((~mover).int(), dim=-1, stable=True).indices  # those that move come first, in order
    src = torch.where(hole, movers.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), row)
    most = min(c["keep"], L)
    src, to = src[..., :most], (row < count)[..., :most]
    for name in ("k", "v"):
        part = s[name][:, :, :most]
        part.copy_(torch.where(to[..., None], s[name].gather(2, src[..., None].expand(-1, -1, -1, c["d"])), part))
    for name in ("weights", "positions"):
        part = s[name + "_out"][..., :most]
        part.copy_(torch.where(to, s[name].gather(-1, src), part))
    s["weights_out"].masked_fill_((row >= count) & there, 0)
    s["lens_out"].copy_(count.flatten())
    return s["k"], s["v"], s["weights_out"], s["positions_out"], s["lens_out"]


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["c"]["op"]
    if own:
        return _own(s)
    if op == "axes_fwd":
        return _axes_fwd(s)
    if op == "axes_bwd":
        return _axes_bwd(s)
    if op.startswith("prefix"):
        return _prefix(s)
    if op == "weights":
        return _weights(s)
    return _decode_weights(s) if op == "decode_weights" else _evict(s)


def _own(s):
    from vision_transformer_attention_psapackqkv_gb300 import binding as B

    c, op = s["c"], s["c"]["op"]
    room = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    if op.startswith("axes"):
        p = B.rope_axes_of(s["q"], s["k"], s["cos"], s["sections"], eps=s["eps"], interleaved=_pairwise(c),
                           alternate=c["alternate"], grid=s["grid"] or None, normalize=c["norm"])
        args = (s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"])
        new = lambda x: torch.empty(x.shape, dtype=x.dtype, device=x.device)  # noqa: E731
        q, k = new(s["q"]), new(s["k"])
        if op == "axes_fwd":
            B.psa_qk_norm_rope_axes_fwd(*args, q, k, p)
            return q, k
        dwq, dwk = (torch.empty_like(s["wq"]), torch.empty_like(s["wk"])) if c["norm"] else (None, None)
        B.psa_qk_norm_rope_axes_bwd(*args, s["gq"], s["gk"], q, k, dwq, dwk,
                                    room(B.psa_qk_norm_rope_bwd_workspace_size(p.rope)), p)
        return (q, dwq, k, dwk) if c["norm"] else (q, k)
    if op.startswith("prefix"):
        p = B.prefix_of(s["q"], s["kp"], s["k"])
        o, ws = torch.empty_like(s["q"]), room(B.psa_prefix_attn_workspace_size(p))
        if op == "prefix_decode":
            B.psa_prefix_attn_decode(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["lens"], o, ws, p, s["scale"])
            return o
        lse = torch.empty(o.shape[:3], dtype=torch.float32, device="cuda")
        B.psa_prefix_attn_fwd(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["lens"], o, lse, ws, p, s["scale"])
        return o, lse
    if op == "weights":
        win = B.window_of(s["q"], s["k"], c["left"], c["right"], c["sinks"])
        B.psa_window_attn_weights(s["q"], s["k"], s["lens"], s["lse"], s["weights"],
                                  room(B.psa_window_attn_weights_workspace_size(win)), win, s["scale"])
        return s["weights"]
    if op == "decode_weights":
        win = B.window_of(s["q"], s["k"], c["left"], 0, c["sinks"])
        o = torch.empty_like(s["q"])
        B.psa_window_attn_decode_weights(s["q"], s["k"], s["v"], s["lens"], o, s["weights"],
                                         room(B.psa_window_attn_decode_weights_workspace_size(win)), win, s["scale"])
        return o, s["weights"]
    p = B.evict_of(s["k"], c["keep"], c["sinks"], c["recent"])
    B.psa_kv_evict(s["weights"], s["positions"], s["lens"], s["k"], s["v"], s["weights_out"], s["positions_out"],
                   s["lens_out"], room(B.psa_kv_evict_workspace_size(p)), p)
    return s["k"], s["v"], s["weights_out"], s["positions_out"], s["lens_out"]


# ------------------------------------------------------------------ values in 64 bits
def _exact_axes(c, s):
    half = c["rot"] // 2
    left, turn_of, axes = list(s["sections"]), [], len(s["sections"])
    if c["alternate"]:
        while sum(left):
            for a in range(axes):
                if left[a]:
                    left[a] -= 1
                    turn_of.append(a)
    else:
        for a in range(axes):
            turn_of += [a] * left[a]
    cos, sin = (torch.empty(c["B"], c["N"], half, dtype=torch.float64, device="cuda") for _ in range(2))
    n = torch.arange(c["N"], device="cuda")
    for i, a in enumerate(turn_of):
        if s["pos"] is None:
            inner = math.prod(s["grid"][a + 1:])
            at = (n // inner % s["grid"][a]).expand(c["B"], -1)
        else:
            at = s["pos"][a].long()
        cos[..., i], sin[..., i] = s["cos"][:, i].double()[at], s["sin"][:, i].double()[at]
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if _pairwise(c) else (i, i + half)
    if c["op"] == "axes_bwd":
        sin = -sin

    def turn(x):  # [B, N, d]
        y = x.clone()
        y[..., first] = cos * x[..., first] - sin * x[..., second]
        y[..., second] = sin * x[..., first] + cos * x[..., second]
        return y

    def heads(x, w, g):
        out, dw = torch.empty(x.shape, dtype=torch.float64, device="cuda"), 0.0
        for h in range(x.shape[1]):
            a = x[:, h].double()
            if not c["norm"]:
                out[:, h] = turn(a if g is None else g[:, h].double())
                continue
            size = torch.sqrt((a * a).sum(-1, keepdim=True) / c["d"] + s["eps"])
            if g is None:
                out[:, h] = turn(w.double() * a / size)
                continue
            gy = turn(g[:, h].double())
            dw = dw + (gy * a / size).sum((0, 1))
            gw = gy * w.double()
            out[:, h] = gw / size - a * (gw * a).sum(-1, keepdim=True) / (c["d"] * size ** 3)
        return (out,) if g is None or not c["norm"] else (out, dw)

    return heads(s["q"], s["wq"], s.get("gq")) + heads(s["k"], s["wk"], s.get("gk"))


def _exact_prefix(c, s):
    group = c["nh"] // c["nkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(c, c["Nk"])):
        if c["op"] == "prefix_decode":
            at = torch.tensor([n - 1], device="cuda")
        else:
            at = torch.arange(c["Nq"], device="cuda") + c["Nk"] - c["Nq"]
        rows = at < n
        if not rows.any():
            continue
        at = at[rows]
        for h in range(c["nh"]):
            k = torch.cat([s["kp"][0, h // group], s["k"][b, h // group, :n]]).double()
            v = torch.cat([s["vp"][0, h // group], s["v"][b, h // group, :n]]).double()
            x = s["q"][b, h, rows].double() @ k.T * s["scale"]
            j = torch.arange(k.shape[0], device="cuda")
            e = torch.where(j[None] - c["P"] <= at[:, None], torch.exp(x - x.max()), 0.0)
            o[b, h, rows] = e @ v / e.sum(1, keepdim=True)
            lse[b, h, rows] = x.max() + torch.log(e.sum(1))
    return o if c["op"] == "prefix_decode" else (o, lse)


def _exact_weights(c, s):
    group, total = c["nh"] // c["nkv"], s["weights"].double()
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(c, c["Nk"])):
        if c["op"] == "decode_weights":
            at = torch.tensor([n - 1], device="cuda")
        else:
            at = torch.arange(c["Nq"], device="cuda") + c["Nk"] - c["Nq"]
        rows = torch.nonzero(at < n)[:, 0]
        j = torch.arange(n, device="cuda")[None]
        for h in range(c["nh"]):
            k = s["k"][b, h // group, :n].double()
            for part in rows.split(2048):
                p = at[part][:, None]
                ok = torch.ones(len(part), n, dtype=torch.bool, device="cuda")
                if c["left"] >= 0:
                    ok &= (p - j <= c["left"]) | (j < c["sinks"])
                if c.get("right", 0) >= 0:
                    ok &= j - p <= c.get("right", 0)
                x = s["q"][b, h, part].double() @ k.T * s["scale"]
                if c["op"] == "decode_weights":
                    e = torch.where(ok, torch.exp(x - x[ok].max()), 0.0)
                    e = e / e.sum()
                    o[b, h] = e @ s["v"][b, h // group, :n].double()
                else:
                    e = torch.where(ok, torch.exp(x - s["lse"][b, h, part].double()[:, None]), 0.0)
                total[b, h // group, :n] += e.sum(0)
    return total if c["op"] == "weights" else (o, total)


def _exact_evict(c, s):
    """Head by head: sort, drop, and let the kept rows from behind fill the gaps in their order."""
    k, v = s["k"].double(), s["v"].double()
    w_out, lens = s["weights_out"].double(), _lens(c, c["Nk"])
    for b, n in enumerate(lens):
        for h in range(c["nkv"]):
            w, pos = s["weights"][b, h, :n].cpu().tolist(), s["positions"][b, h, :n].cpu().tolist()
            newest, count = max(pos), min(n, c["keep"])
            best = sorted(range(n), key=lambda r: (-math.inf if pos[r] < c["sinks"] or pos[r] > newest - c["recent"] else -w[r], r))
            stay = set(best[:count])
            gaps = [r for r in range(count) if r not in stay]
            come = sorted(r for r in stay if r >= count)
            place = list(range(count))
            for g, r in zip(gaps, come):
                place[g] = r
            at = torch.tensor(place, device="cuda")
            k[b, h, :count], v[b, h, :count] = s["k"][b, h, at].double(), s["v"][b, h, at].double()
            w_out[b, h, :count], w_out[b, h, count:n] = s["weights"][b, h, at].double(), 0
    return k, v, w_out, None, None


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"].startswith("axes"):
        return _exact_axes(c, s)
    if c["op"].startswith("prefix"):
        return _exact_prefix(c, s)
    return _exact_evict(c, s) if c["op"] == "evict" else _exact_weights(c, s)
