"""The language-model operators next to the attention path: the calls that are measured, their
plain forms in elementary torch operations, and their values in 64 bits.

  norm_rope      norms of queries and keys for each head with the position rotation, one pass
                 (psa_qk_norm_rope_fwd / _bwd)
  window         attention in which a query sees a sliding window of keys and the first few ones
                 (psa_window_attn_fwd / _bwd), and its single-token form over a cache
                 (psa_window_attn_decode)
  kv4            the same single-token form over a cache held in 4 bits
                 (psa_window_attn_decode_kv4), and what fills and reads that cache
                 (psa_kv4_append / psa_kv4_read)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoding step of 64 sequences at far, unequal positions: a latency-bound call
        dict(name="norm_rope_step", op="norm_rope_fwd", dtype="bf16", B=64, nh=32, nkv=8, N=1, d=128,
             rot=128, interleaved=False, max_pos=32768, scattered=True),
        # two long prompts, q and k read from the packed projection in place
        dict(name="norm_rope_prompt", op="norm_rope_fwd", dtype="bf16", B=2, nh=32, nkv=8, N=8192, d=128,
             rot=128, interleaved=False, max_pos=8192, scattered=False),
        # training, odd length, half of the channels rotated in neighbouring pairs
        dict(name="norm_rope_train", op="norm_rope_bwd", dtype="bf16", B=4, nh=16, nkv=16, N=2047, d=64,
             rot=32, interleaved=True, max_pos=2048, scattered=False),
        # a 20 x 20 feature map as a sequence: both directions visible, a few register tokens, fp32
        dict(name="window_map_f32", op="window_fwd", dtype="f32", B=4, nh=4, nkv=4, Nq=400, Nk=400, d=64,
             left=60, right=60, sinks=4, ragged=False),
        # a long prompt through a sliding window with its first tokens kept
        dict(name="window_prompt", op="window_fwd", dtype="bf16", B=1, nh=32, nkv=8, Nq=8192, Nk=8192, d=128,
             left=1023, right=0, sinks=4, ragged=False),
        # a padded batch of odd length without a window: the whole causal triangle
        dict(name="window_causal_ragged", op="window_fwd", dtype="bf16", B=2, nh=16, nkv=2, Nq=4097, Nk=4097,
             d=128, left=-1, right=0, sinks=0, ragged=True),
        # training on sequences of 4096
        dict(name="window_train", op="window_bwd", dtype="bf16", B=2, nh=16, nkv=4, Nq=4096, Nk=4096, d=128,
             left=1023, right=0, sinks=4, ragged=False),
        # a small, padded training batch of odd length, no shared heads
        dict(name="window_train_ragged", op="window_bwd", dtype="bf16", B=3, nh=8, nkv=8, Nq=1000, Nk=1000,
             d=64, left=255, right=0, sinks=8, ragged=True),
        # a decoding step of 32 sequences of unequal lengths
        dict(name="decode_batch", op="decode", dtype="bf16", B=32, nh=32, nkv=8, Nk=8192, d=128,
             left=4095, sinks=4, ragged=True),
        # a chunk of prompts goes into the 4-bit cache and is read back for the next chunk
        dict(name="kv4_store", op="kv4_store", dtype="bf16", B=4, nkv=8, N=2048, Nk=4096, d=128, ragged=True),
        # a decoding step over long 4-bit caches, every key visible
        dict(name="kv4_decode_long", op="kv4_decode", dtype="bf16", B=16, nh=32, nkv=8, Nk=32768, d=128,
             left=-1, sinks=0, ragged=True),
        # one sequence, a short window: a latency-bound call
        dict(name="kv4_decode_one", op="kv4_decode", dtype="bf16", B=1, nh=16, nkv=4, Nk=2000, d=64,
             left=1023, sinks=4, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope_fwd", "norm_rope_bwd", "window_fwd", "window_fwd", "window_bwd", "decode",
                     "kv4_store", "kv4_decode"])
    d = rng.choice([64, 128])
    nkv = rng.choice([1, 2, 4, 8])
    nh = nkv * rng.choice([1, 2, 4, 5, 8])
    B = rng.choice([1, 2, 3, 4])
    ragged = rng.random() < 0.5
    sinks = rng.choice([0, 1, 4, 16, 130])
    if op.startswith("norm_rope"):
        N = min(_log(rng, 1, 8192), 600000 // (B * (nh + nkv)))
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, nh=nh, nkv=nkv, N=N, d=d,
                    rot=rng.choice([32, d // 2, d]), interleaved=rng.random() < 0.5,
                    max_pos=N + rng.randrange(5000), scattered=ragged)
    if op in ("window_fwd", "window_bwd"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        most = 8192 if dtype == "bf16" else 600
        Nk = _log(rng, 1, most)
        while B * nh * Nk * Nk > (1 << 29) and Nk > 16:
            B, Nk = max(1, B // 2), Nk * 3 // 4
        # a chunk behind a prefix, or the sequence itself
        Nq = Nk if op == "window_bwd" or ragged or rng.random() < 0.7 else max(1, Nk - rng.randrange(Nk))
        left = rng.choice([-1, _log(rng, 1, 4096)])
        return dict(op=op, dtype=dtype, B=B, nh=nh, nkv=nkv, Nq=Nq, Nk=Nk, d=d, left=left,
                    right=rng.choice([0, 0, 0, 37]), sinks=sinks, ragged=ragged)
    if op == "kv4_store":
        N = _log(rng, 1, 4096)
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), B=B, nkv=nkv, N=N, Nk=N + rng.randrange(1, 1000),
                    d=d, ragged=ragged)
    B = rng.choice([1, 3, 8, 16])
    Nk = min(_log(rng, 1, 32768), (1 << 20 if op == "decode" else 1 << 22) // (B * nkv))
    return dict(op=op, dtype="bf16", B=B, nh=nh, nkv=nkv, Nk=Nk, d=d, left=rng.choice([-1, _log(rng, 1, 8192)]),
                sinks=sinks, ragged=ragged)


def _lens(c, n):
    """Valid lengths of the batch's sequences: the longest is whole, the others fall off unevenly."""
    if not c["ragged"]:
        return [n] * c["B"]
    return [max(1, n - (b * (2 * n // 7 + 1)) % (3 * n // 4 + 1)) for b in range(c["B"])]


# ------------------------------------------------------------------ what a pass cannot do without
def _visible(nq, nk, length, left, right, sinks):
    """Numbers of visible (query, key) pairs and of keys that some query sees, one sequence."""
    p = torch.arange(nq, dtype=torch.int64) + (nk - nq)
    p = p[(p >= 0) & (p < length)]
    if p.numel() == 0:
        return 0, 0
    hi = torch.full_like(p, length - 1) if right < 0 else (p + right).clamp(max=length - 1)
    lo = torch.zeros_like(p) if left < 0 else (p - left).clamp(min=0)
    first = torch.minimum(lo, hi + 1).clamp(max=sinks)  # sinks in front of the window
    pairs = (hi - lo + 1).clamp(min=0) + first
    keys = int(hi.max()) + 1 - int(lo.min()) + min(sinks, int(lo.min()))
    return int(pairs.sum()), keys


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    d, B = c["d"], c["B"]
    if c["op"].startswith("norm_rope"):
        rows = B * c["N"] * (c["nh"] + c["nkv"])
        table = min(c["max_pos"], B * c["N"] if c["scattered"] else c["N"]) * c["rot"] * 4
        if c["op"] == "norm_rope_fwd":
            return {"bytes": rows * d * e * 2 + table, "flops": rows * d * 8}
        return {"bytes": rows * d * e * 3 + table, "flops": rows * d * 16}
    if c["op"] in ("window_fwd", "window_bwd"):
        pairs = keys = valid = 0
        for n in _lens(c, c["Nk"]):
            a, b = _visible(c["Nq"], c["Nk"], n, c["left"], c["right"], c["sinks"])
            pairs, keys = pairs + a, keys + b
            valid += max(0, min(c["Nq"], n - (c["Nk"] - c["Nq"])))
        # rows read where they are valid, written everywhere; keys read where some query sees them
        q_in, q_out = valid * c["nh"] * d * e, B * c["Nq"] * c["nh"] * d * e
        k_in, k_out = keys * c["nkv"] * d * e, B * c["Nk"] * c["nkv"] * d * e
        if c["op"] == "window_fwd":
            return {"bytes": q_in + q_out + 2 * k_in + B * c["Nq"] * c["nh"] * 4, "flops": 4 * d * c["nh"] * pairs}
        return {"bytes": 3 * q_in + q_out + 2 * k_in + 2 * k_out + valid * c["nh"] * 4, "flops": 10 * d * c["nh"] * pairs}
    if c["op"] == "kv4_store":
        n = sum(_lens(c, c["N"])) * c["nkv"]
        packed = d // 2 + d // 32 * 2
        return {"bytes": 2 * (n * d * e + n * packed + B * c["nkv"] * c["Nk"] * (packed + d * e)), "flops": 2 * 4 * n * d}
    keys = sum(_visible(1, n, n, c["left"], 0, c["sinks"])[1] for n in _lens(c, c["Nk"]))
    row = d * 2 if c["op"] == "decode" else d // 2 + d // 32 * 2
    return {"bytes": 2 * keys * c["nkv"] * row + 2 * B * c["nh"] * d * 2, "flops": 4 * d * c["nh"] * keys}


# ------------------------------------------------------------------ inputs
def _norm_rope_inputs(c, gen):
    B, nh, nkv, N, d, dt = c["B"], c["nh"], c["nkv"], c["N"], c["d"], DTYPES[c["dtype"]]
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    # the projection's output, [B, N, heads of q | k | v, d], of which q and k are views
    packed = (rn(B, N, nh + 2 * nkv, d) * 1.5).to(dt).transpose(1, 2)
    half = c["rot"] // 2
    freq = 1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(c["max_pos"], dtype=torch.float64, device="cuda")[:, None] * freq
    s = dict(c=c, q=packed[:, :nh], k=packed[:, nh:nh + nkv], wq=1 + 0.2 * rn(d), wk=1 + 0.2 * rn(d),
             cos=angle.cos().float().contiguous(), sin=angle.sin().float().contiguous(), eps=1e-6, pos=None)
    if c["scattered"]:
        s["pos"] = torch.randint(0, c["max_pos"], (B, N), generator=gen, device="cuda", dtype=torch.int32)
    if c["op"] == "norm_rope_bwd":
        s["gq"], s["gk"] = rn(B, nh, N, d).to(dt), rn(B, nkv, N, d).to(dt)
    return s


def _window_inputs(c, gen):
    B, nh, nkv, d, dt = c["B"], c["nh"], c["nkv"], c["d"], DTYPES[c["dtype"]]
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dt)  # noqa: E731
    s = dict(c=c, q=rn(B, nh, c["Nq"], d), k=rn(B, nkv, c["Nk"], d), v=rn(B, nkv, c["Nk"], d), scale=d ** -0.5,
             lens=None)
    if c["ragged"]:
        s["lens"] = torch.tensor(_lens(c, c["Nk"]), dtype=torch.int32, device="cuda")
    if c["op"] == "window_bwd":
        s["do"] = rn(B, nh, c["Nq"], d)
        s["o"], s["lse"] = _window_fwd(s)
    return s


def _quantise(x):
    """[..., d] -> (codes [..., d // 2] uint8, scales [..., d // 32] bf16) of the 4-bit cache.

    A group of 32 channels has one scale, the largest magnitude / 7 rounded to bf16; a code is the
    nearest whole multiple of it (ties to even, -7 .. 7) plus 8.  The code of channel 32 g + 4 a + i
    is nibble (a * groups + g) * 4 + i of its row, low nibbles first."""
    groups = x.shape[-1] // 32
    x = x.float().unflatten(-1, (groups, 32))
    scale = (x.abs().amax(-1) / 7).to(torch.bfloat16)
    step = scale.float()[..., None]
    n = torch.where(step > 0, torch.round(x / torch.where(step > 0, step, 1)), 0).clamp(-7, 7) + 8
    n = n.to(torch.uint8).unflatten(-1, (8, 4)).transpose(-3, -2).flatten(-3)
    return n[..., 0::2] | (n[..., 1::2] << 4), scale


def _dequantise(codes, scales):
    groups = scales.shape[-1]
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (8, groups, 4)).transpose(-3, -2)
    return ((n.flatten(-2).float() - 8) * scales.float()[..., None]).flatten(-2)


def _decode_inputs(c, gen):
    B, nh, nkv, L, d = c["B"], c["nh"], c["nkv"], c["Nk"], c["d"]
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    s = dict(c=c, q=rn(B, nh, 1, d).to(torch.bfloat16), scale=d ** -0.5,
             lens=torch.tensor(_lens(c, L), dtype=torch.int32, device="cuda"),
             o=torch.empty(B, nh, 1, d, dtype=torch.bfloat16, device="cuda"))
    k, v = rn(B, nkv, L, d).to(torch.bfloat16), rn(B, nkv, L, d).to(torch.bfloat16)
    if c["op"] == "decode":
        s["k"], s["v"] = k, v
    else:
        (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _quantise(k), _quantise(v)
    return s


def _store_inputs(c, gen):
    B, nkv, N, L, d, dt = c["B"], c["nkv"], c["N"], c["Nk"], c["d"], DTYPES[c["dtype"]]
    # heads of unlike sizes, a few large channels, as keys have them
    size = torch.exp(torch.randn(nkv, 1, d, generator=gen, device="cuda"))
    k, v = ((torch.randn(B, nkv, N, d, generator=gen, device="cuda") * size).to(dt) for _ in range(2))
    lens = torch.tensor(_lens(c, N), dtype=torch.int32, device="cuda")
    old = torch.randn(B, nkv, L, d, generator=gen, device="cuda")
    (kc, ks), (vc, vs) = _quantise(old), _quantise(-old)
    out = lambda: torch.empty(B, nkv, L, d, dtype=dt, device="cuda")  # noqa: E731
    starts = torch.tensor([(L - n) * (b % 3) // 2 for b, n in enumerate(_lens(c, N))], dtype=torch.int32, device="cuda")
    return dict(c=c, k=k, v=v, counts=lens, starts=starts, kc=kc, ks=ks, vc=vc, vs=vs, ko=out(), vo=out())


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if c["op"].startswith("norm_rope"):
        return _norm_rope_inputs(c, gen)
    if c["op"] in ("window_fwd", "window_bwd"):
        return _window_inputs(c, gen)
    return _store_inputs(c, gen) if c["op"] == "kv4_store" else _decode_inputs(c, gen)


# ------------------------------------------------------------------ plain forms
def _angles(s, sign):
    """cos and sin of each row's angles, [B or 1, 1, N, rot / 2]."""
    c = s["c"]
    pos = s["pos"] if s["pos"] is not None else torch.arange(c["N"], device="cuda")[None]
    return s["cos"][pos.long()][:, None], sign * s["sin"][pos.long()][:, None]


def _rotate(x, cos, sin, c):
    rot = c["rot"]
    r, rest = x[..., :rot], x[..., rot:]
    if c["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([r, rest], -1)


def _norm_rope_fwd(s):
    cos, sin = _angles(s, 1)

    def one(x, w):
        x32 = x.float()
        y = x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + s["eps"]) * w
        return _rotate(y, cos, sin, s["c"]).to(x.dtype)

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _norm_rope_bwd(s):
    cos, sin = _angles(s, -1)

    def one(x, w, g):
        x32 = x.float()
        r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + s["eps"])
        xh, gy = x32 * r, _rotate(g.float(), cos, sin, s["c"])
        gx = gy * w
        dx = r * (gx - xh * (gx * xh).mean(-1, keepdim=True))
        return dx.to(x.dtype), (gy * xh).double().sum((0, 1, 2)).float()

    (dq, dwq), (dk, dwk) = one(s["q"], s["wq"], s["gq"]), one(s["k"], s["wk"], s["gk"])
    return dq, dk, dwq, dwk


def _mask(nq, nk, left, right, sinks, lens):
    """What each query sees, [B or 1, 1, 1, nq, nk]."""
    p = torch.arange(nq, device="cuda")[:, None] + (nk - nq)
    j = torch.arange(nk, device="cuda")[None]
    see = torch.ones(nq, nk, dtype=torch.bool, device="cuda")
    if left >= 0:
        see &= (j >= p - left) | (j < sinks)
    if right >= 0:
        see &= j <= p + right
    see = (see & (p >= 0))[None]
    if lens is not None:
        see = see & (j < lens[:, None, None]) & (p < lens[:, None, None])
    return see[:, None, None]


def _scores(q, k, scale, see):
    """[B, kv heads, group, nq, nk] in 32 bits, -inf where masked."""
    q = q.float().unflatten(1, (k.shape[1], -1))
    return ((q @ k.float()[:, :, None].mT) * scale).masked_fill(~see, -math.inf)


def _window_fwd(s):
    c = s["c"]
    see = _mask(c["Nq"], c["Nk"], c["left"], c["right"], c["sinks"], s["lens"])
    x = _scores(s["q"], s["k"], s["scale"], see)
    m = x.amax(-1, keepdim=True)
    base = torch.where(m == -math.inf, 0, m)
    x = torch.exp(x - base)
    l = x.sum(-1, keepdim=True)
    o = (x @ s["v"].float()[:, :, None]) / torch.where(l == 0, 1, l)
    return o.flatten(1, 2).to(s["q"].dtype), (base + torch.log(l)).flatten(1, 2).squeeze(-1)


def _window_bwd(s):
    c, dt = s["c"], s["q"].dtype
    see = _mask(c["Nq"], c["Nk"], c["left"], c["right"], c["sinks"], s["lens"])
    p = _scores(s["q"], s["k"], s["scale"], see)
    lse = s["lse"].unflatten(1, (c["nkv"], -1))[..., None]
    p = torch.exp(p - torch.where(lse == -math.inf, 0, lse))
    q, do = (t.float().unflatten(1, (c["nkv"], -1)) for t in (s["q"], s["do"]))
    dv = (p.mT @ do).sum(2)
    ds = do @ s["v"].float()[:, :, None].mT
    ds = p * (ds - (p * ds).sum(-1, keepdim=True)) * s["scale"]
    dq = (ds @ s["k"].float()[:, :, None]).flatten(1, 2)
    return dq.to(dt), (ds.mT @ q).sum(2).to(dt), dv.to(dt)


def _decode_over(s, k, v):
    c, lens = s["c"], s["lens"].long()[:, None]
    j = torch.arange(c["Nk"], device="cuda")[None]
    see = j < lens
    if c["left"] >= 0:
        see &= (j >= lens - 1 - c["left"]) | (j < c["sinks"])
    x = _scores(s["q"], k, s["scale"], see[:, None, None, None])
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = (p @ v.float()[:, :, None]) / p.sum(-1, keepdim=True)
    return o.flatten(1, 2).to(s["q"].dtype)


def _store(s):
    c = s["c"]
    row = torch.arange(c["Nk"], device="cuda")[None] - s["starts"].long()[:, None]
    new = ((row >= 0) & (row < s["counts"][:, None]))[:, None, :, None]
    row = row.clamp(0, c["N"] - 1)[:, None, :, None]

    def one(x, codes, scales):
        nc, ns = _quantise(x)
        codes = torch.where(new, nc.gather(2, row.expand(-1, c["nkv"], -1, nc.shape[-1])), codes)
        scales = torch.where(new, ns.gather(2, row.expand(-1, c["nkv"], -1, ns.shape[-1])), scales)
        return _dequantise(codes, scales).to(x.dtype)

    return one(s["k"], s["kc"], s["ks"]), one(s["v"], s["vc"], s["vs"])


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["c"]["op"]
    if own:
        return _own(s)
    if op == "norm_rope_fwd":
        return _norm_rope_fwd(s)
    if op == "norm_rope_bwd":
        return _norm_rope_bwd(s)
    if op == "window_fwd":
        return _window_fwd(s)
    if op == "window_bwd":
        return _window_bwd(s)
    if op == "decode":
        return _decode_over(s, s["k"], s["v"])
    if op == "kv4_decode":
        return _decode_over(s, _dequantise(s["kc"], s["ks"]), _dequantise(s["vc"], s["vs"]))
    return _store(s)


def _own(s):
    from vision_transformer_attention_psapackqkv_gb300 import binding as B

    c, op = s["c"], s["c"]["op"]
    if op.startswith("norm_rope"):
        p = B.norm_rope_of(s["q"], s["k"], s["cos"], eps=s["eps"], interleaved=c["interleaved"])
        args = (s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"])
        new = lambda x: torch.empty(x.shape, dtype=x.dtype, device=x.device)  # noqa: E731
        q, k = new(s["q"]), new(s["k"])
        if op == "norm_rope_fwd":
            B.psa_qk_norm_rope_fwd(*args, q, k, p)
            return q, k
        dwq, dwk = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
        ws = torch.empty(B.psa_qk_norm_rope_bwd_workspace_size(p), dtype=torch.uint8, device="cuda")
        B.psa_qk_norm_rope_bwd(*args, s["gq"], s["gk"], q, k, dwq, dwk, ws, p)
        return q, k, dwq, dwk
    if op == "kv4_store":
        cache = (s["kc"], s["ks"], s["vc"], s["vs"])
        B.psa_kv4_append(s["k"], s["v"], s["starts"], s["counts"], *cache)
        B.psa_kv4_read(*cache, s["ko"], s["vo"])
        return s["ko"], s["vo"]
    if op in ("window_fwd", "window_bwd"):
        win = B.window_of(s["q"], s["k"], c["left"], c["right"], c["sinks"])
        if op == "window_fwd":
            o = torch.empty_like(s["q"])
            lse = torch.empty(o.shape[:3], dtype=torch.float32, device="cuda")
            B.psa_window_attn_fwd(s["q"], s["k"], s["v"], s["lens"], o, lse, win, s["scale"])
            return o, lse
        dq, dk, dv = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
        ws = torch.empty(B.psa_window_attn_bwd_workspace_size(win), dtype=torch.uint8, device="cuda")
        B.psa_window_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["lens"], dq, dk, dv, ws, win,
                              s["scale"])
        return dq, dk, dv
    if op == "decode":
        win = B.window_of(s["q"], s["k"], c["left"], 0, c["sinks"])
        ws = torch.empty(B.psa_window_attn_decode_workspace_size(win), dtype=torch.uint8, device="cuda")
        B.psa_window_attn_decode(s["q"], s["k"], s["v"], s["lens"], s["o"], ws, win, s["scale"])
        return s["o"]
    win = B.window_of(s["q"], s["kc"], c["left"], 0, c["sinks"])
    ws = torch.empty(B.psa_window_attn_decode_workspace_size(win), dtype=torch.uint8, device="cuda")
    B.psa_window_attn_decode_kv4(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["lens"], s["o"], ws, win, s["scale"])
    return s["o"]


# ------------------------------------------------------------------ values in 64 bits
def _sees(p, j, length, left, right, sinks):
    ok = (p >= 0) & (p < length) & (j < length)
    if right >= 0:
        ok = ok & (j - p <= right)
    if left >= 0:
        ok = ok & ((p - j <= left) | (j < sinks))
    return ok


def _attend64(q, k, v, p, length, left, right, sinks, scale):
    """Rows of one query head: output, log of the sum, probabilities, in 64 bits."""
    ok = _sees(p[:, None], torch.arange(k.shape[0], device="cuda")[None], length, left, right, sinks)
    x = torch.einsum("id,jd->ij", q, k) * scale
    top = torch.where(ok, x, -1e300).max(1, keepdim=True).values
    e = torch.where(ok, torch.exp(torch.where(ok, x - top, 0.0)), 0.0)
    total = e.sum(1, keepdim=True)
    some = total > 0
    prob = torch.where(some, e / torch.where(some, total, 1.0), 0.0)
    lse = torch.where(some, top + torch.log(torch.where(some, total, 1.0)), -math.inf)
    return torch.einsum("ij,jd->id", prob, v), lse[:, 0], prob


def _turn64(c, s, back):
    """Each position's rotation in 64 bits as pairs of channels: their indexes, cos and sin."""
    half = c["rot"] // 2
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    at = s["pos"].long() if s["pos"] is not None else torch.arange(c["N"], device="cuda").expand(c["B"], -1)
    cos, sin = s["cos"].double()[at], s["sin"].double()[at]  # [B, N, half]
    return first, second, cos, -sin if back else sin


def _exact_norm_rope(c, s):
    first, second, cos, sin = _turn64(c, s, c["op"] == "norm_rope_bwd")

    def turn(x):  # [B, N, d]
        y = x.clone()
        y[..., first] = cos * x[..., first] - sin * x[..., second]
        y[..., second] = sin * x[..., first] + cos * x[..., second]
        return y

    def heads(x, w, g):
        w = w.double()
        out, dw = torch.empty(x.shape, dtype=torch.float64, device="cuda"), torch.zeros_like(w)
        for h in range(x.shape[1]):
            a = x[:, h].double()
            size = torch.sqrt((a * a).sum(-1, keepdim=True) / c["d"] + s["eps"])
            if g is None:
                out[:, h] = turn(w * a / size)
                continue
            gy = turn(g[:, h].double())
            dw += (gy * a / size).sum((0, 1))
            gw = gy * w
            out[:, h] = gw / size - a * (gw * a).sum(-1, keepdim=True) / (c["d"] * size ** 3)
        return out, dw

    (q, dwq), (k, dwk) = heads(s["q"], s["wq"], s.get("gq")), heads(s["k"], s["wk"], s.get("gk"))
    return (q, k) if c["op"] == "norm_rope_fwd" else (q, k, dwq, dwk)


def _exact_window(c, s):
    lens, group = _lens(c, c["Nk"]), c["nh"] // c["nkv"]
    f64 = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(s["q"].shape, **f64), torch.zeros(s["q"].shape[:3], **f64)
    dk, dv = torch.zeros(s["k"].shape, **f64), torch.zeros(s["k"].shape, **f64)
    for b in range(c["B"]):
        for h in range(c["nh"]):
            k, v = s["k"][b, h // group].double(), s["v"][b, h // group].double()
            for i in range(0, c["Nq"], 2048):
                rows = slice(i, min(i + 2048, c["Nq"]))
                q = s["q"][b, h, rows].double()
                p = torch.arange(rows.start, rows.stop, device="cuda") + c["Nk"] - c["Nq"]
                out, l, prob = _attend64(q, k, v, p, lens[b], c["left"], c["right"], c["sinks"], s["scale"])
                if c["op"] == "window_fwd":
                    o[b, h, rows], lse[b, h, rows] = out, l
                    continue
                g = s["do"][b, h, rows].double()
                dv[b, h // group] += prob.T @ g
                dx = prob * (g @ v.T - (g * out).sum(1, keepdim=True)) * s["scale"]
                o[b, h, rows] = dx @ k
                dk[b, h // group] += dx.T @ q
    return (o, lse) if c["op"] == "window_fwd" else (o, dk, dv)


def _unpack64(codes, scales):
    """Channel by channel: the value that its nibble and its group's scale stand for."""
    groups = scales.shape[-1]
    out = torch.empty(*scales.shape[:-1], groups * 32, dtype=torch.float64, device="cuda")
    for ch in range(groups * 32):
        g, a, i = ch // 32, ch % 32 // 4, ch % 4
        nibble = (a * groups + g) * 4 + i
        out[..., ch] = ((codes[..., nibble // 2] >> (4 * (nibble % 2))) & 15).double() - 8
        out[..., ch] *= scales[..., g].double()
    return out


def _exact_decode(c, s):
    group = c["nh"] // c["nkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(c, c["Nk"])):
        p = torch.tensor([n - 1], device="cuda")
        for h in range(c["nkv"]):
            if c["op"] == "decode":
                k, v = s["k"][b, h, :n].double(), s["v"][b, h, :n].double()
            else:
                k, v = _unpack64(s["kc"][b, h, :n], s["ks"][b, h, :n]), _unpack64(s["vc"][b, h, :n], s["vs"][b, h, :n])
            heads = slice(h * group, (h + 1) * group)
            out[b, heads, 0] = _attend64(s["q"][b, heads, 0].double(), k, v, p.expand(group), n, c["left"], 0,
                                         c["sinks"], s["scale"])[0]
    return out


def _exact_store(c, s):
    def one(x, codes, scales):
        out = _unpack64(codes, scales)
        for b, (start, n) in enumerate(zip(s["starts"].tolist(), s["counts"].tolist())):
            a = x[b, :, :n].double()
            for g in range(c["d"] // 32):
                part = a[..., 32 * g:32 * g + 32]
                # the scale is held in bf16 by the format, made from a quotient in fp32
                step = (part.abs().amax(-1, keepdim=True).float() / 7).to(torch.bfloat16).double()
                n7 = torch.where(step > 0, (part / torch.where(step > 0, step, 1.0)).round(), 0.0).clamp(-7, 7)
                out[b, :, start:start + n, 32 * g:32 * g + 32] = n7 * step
        return out

    return one(s["k"], s["kc"], s["ks"]), one(s["v"], s["vc"], s["vs"])


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"].startswith("norm_rope"):
        return _exact_norm_rope(c, s)
    if c["op"] in ("window_fwd", "window_bwd"):
        return _exact_window(c, s)
    return _exact_store(c, s) if c["op"] == "kv4_store" else _exact_decode(c, s)
