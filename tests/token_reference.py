"""Plain 64-bit forms of the token-sequence operators, one query row's definition at a time in
tensor notation, together with the sums of magnitudes that the tests' tolerances are made of.

Tolerances count roundings.  A value rounded to bf16 is off by at most 2^-8 of itself, to fp32 by
U = 2^-24; a sum of products of n terms in fp32 by at most n U times the sum of the terms' magnitudes."""
import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def visible(n_q, n_k, length, left, right, sinks, device):
    p = torch.arange(n_q, device=device)[:, None] + (n_k - n_q)
    j = torch.arange(n_k, device=device)[None, :]
    ok = (p >= 0) & (p < length) & (j < length)
    if right >= 0:
        ok &= j <= p + right
    if left >= 0:
        ok &= (j >= p - left) | (j < sinks)
    return ok


def _clean(x, rows):
    """Rows from `rows` on are padding: whatever they hold plays no part."""
    x = x.double().clone()
    x[rows:] = 0
    return x


def window_attention(q, k, v, lens, left, right, sinks, scale, do=None, half=2.0 ** -8, fp32_only=False):
    """Everything about the forward and (with do) the backward, all in float64 [B, heads, ...]:
    o, lse, dq, dk, dv and a bound for each (o_tol, lse_tol, dq_tol, dk_tol, dv_tol) on how far an
    implementation may be off that holds P and dS in a type of rounding error `half` (fp32_only: not
    rounded), everything else in fp32, takes delta from an o that is itself within o_tol, and rounds
    its outputs once to the type of `half`."""
    B, nh, nq, d = q.shape
    nkv, nk = k.shape[1:3]
    group, off, dev = nh // nkv, nk - nq, q.device
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)  # noqa: E731
    r = {n: z(B, nh, nq, d) for n in ("o", "o_tol", "dq", "dq_tol")}
    r |= {n: z(B, nkv, nk, d) for n in ("dk", "dk_tol", "dv", "dv_tol")}
    r["lse"], r["lse_tol"] = z(B, nh, nq), z(B, nh, nq)
    hp = U if fp32_only else half  # rounding of P and dS
    for b in range(B):
        n = nk if lens is None else max(0, min(int(lens[b]), nk))
        ok = visible(nq, nk, n, left, right, sinks, dev)
        for h in range(nh):
            qq, kk, vv = (_clean(t, m) for t, m in ((q[b, h], max(0, n - off)), (k[b, h // group], n),
                                                    (v[b, h // group], n)))
            x = torch.where(ok, qq @ kk.T * scale, -math.inf)
            lse = torch.logsumexp(x, 1)
            p = torch.where(ok, torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
            o = p @ vv
            # scores in fp32: a product of d terms, the scale, the exponential's argument; the
            # exponential itself within a few units in the last place, or 2^-21 of ex2.approx
            big = (qq.abs() @ kk.abs().T * scale).max() if nq and nk else torch.tensor(0.0)
            ex = U * ((d + 4) * float(big) + 32)
            mag = p @ vv.abs()
            o_tol = half * o.abs() + (hp + 2 * ex + (nk + 8) * U) * mag
            r["o"][b, h], r["o_tol"][b, h], r["lse"][b, h] = o, o_tol, lse
            r["lse_tol"][b, h] = ex + (nk + 8) * U + U * torch.where(lse == -math.inf, 0.0, lse).abs()
            if do is None:
                continue
            g = _clean(do[b, h], max(0, n - off))
            g[~ok.any(1)] = 0  # rows that see nothing
            dp, dpm = g @ vv.T, g.abs() @ vv.abs().T
            delta = (g * o).sum(1, keepdim=True)
            ds = p * (dp - delta)
            delta_err = (g.abs() * (o_tol + (d + 2) * U * o.abs())).sum(1, keepdim=True)
            ds_err = hp * ds.abs() + p * (delta_err + (d + 4) * U * dpm + (2 * ex + 8 * U) * (dp - delta).abs())
            dq, dv, dk = scale * ds @ kk, p.T @ g, scale * ds.T @ qq
            r["dq"][b, h] = dq
            r["dq_tol"][b, h] = half * dq.abs() + scale * (ds_err + (nk + 8) * U * ds.abs()) @ kk.abs()
            r["dk"][b, h // group] += dk
            r["dv"][b, h // group] += dv
            r["dk_tol"][b, h // group] += scale * (ds_err + (nq * group + 8) * U * ds.abs()).T @ qq.abs()
            r["dv_tol"][b, h // group] += ((hp + 2 * ex + (nq * group + 8) * U) * p).T @ g.abs()
    r["dk_tol"] += half * r["dk"].abs()
    r["dv_tol"] += half * r["dv"].abs()
    return r


def within(x, ref, tol, what):
    """|x - ref| <= tol everywhere (a hair for the fp64 reference itself); infinities equal."""
    x, ref, tol = x.double(), ref.double(), tol.double()
    same = x == ref
    off = torch.where(same, 0.0, (x - ref).abs())
    bad = ~(same | (off <= tol * (1 + 1e-9) + 1e-30))
    assert not bad.any(), (what, int(bad.sum()), float((off / tol.clamp(min=1e-300))[bad].max()),
                           bad.nonzero()[:4].tolist())


def rotate(x, cos, sin, interleaved, back=False):
    """x [..., N, d] turned by cos, sin [..., N, rot / 2]."""
    half = cos.shape[-1]
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    s = -sin if back else sin
    y = x.clone()
    y[..., a] = cos * x[..., a] - s * x[..., b]
    y[..., b] = s * x[..., a] + cos * x[..., b]
    return y


def norm_rope(x, w, cos, sin, positions, interleaved, eps, g=None, half=2.0 ** -8):
    """One of q and k: [B, heads, N, d]; positions [B, N], valid ones only.  Without g: y and its
    bound; with the output's gradient g: dx, its bound, dw and its bound."""
    B, H, N, d = x.shape
    x, dev = x.double(), x.device
    w = torch.ones(d, dtype=torch.float64, device=dev) if w is None else w.double()
    if cos is None:
        c = s = torch.zeros(B, 1, N, 0, dtype=torch.float64, device=dev)
    else:
        c, s = (t.double()[positions.long()][:, None] for t in (cos, sin))
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    few = (d + 24) * U  # the mean of d squares, the root, and a handful of products
    mags = lambda t: rotate(t.abs(), c.abs(), -s.abs(), interleaved).abs() + rotate(t.abs(), c.abs(), s.abs(), interleaved).abs()  # noqa: E731
    if g is None:
        y = x * r * w
        out = rotate(y, c, s, interleaved)
        return out, half * out.abs() + few * mags(y)
    g = g.double()
    gy, gm = rotate(g, c, s, interleaved, back=True), mags(g)
    xh, gw = x * r, gy * w
    back = (gw * xh).mean(-1, keepdim=True)
    dx = r * (gw - xh * back)
    size = r * (gm * w.abs() + xh.abs() * (gm * w.abs() * xh.abs()).mean(-1, keepdim=True))
    dw, dwm = (gy * xh).sum((0, 1, 2)), (gm * xh.abs()).sum((0, 1, 2))
    return dx, half * dx.abs() + 2 * few * size, dw, (few + (B * H * N + 64) * U) * dwm


def quantise(x):
    """codes [..., d / 2] uint8 and scales [..., d / 32] bf16 of the 4-bit cache, channel by channel."""
    d = x.shape[-1]
    groups, x = d // 32, x.float()
    codes = torch.zeros(*x.shape[:-1], d // 2, dtype=torch.uint8, device=x.device)
    scales = torch.zeros(*x.shape[:-1], groups, dtype=torch.bfloat16, device=x.device)
    for g in range(groups):
        part = x[..., 32 * g:32 * g + 32]
        top = part.abs().amax(-1)
        sc = (top * torch.full_like(top, 1 / 7)).to(torch.bfloat16)
        scales[..., g] = sc
        step = sc.float()
        for e in range(32):
            n = torch.where(step > 0, torch.round(part[..., e] / torch.where(step > 0, step, 1.0)), 0.0)
            nibble = ((e // 4) * groups + g) * 4 + e % 4
            codes[..., nibble // 2] |= (n.clamp(-7, 7) + 8).to(torch.uint8) << (4 * (nibble % 2))
    return codes, scales


def dequantise(codes, scales):
    groups = scales.shape[-1]
    out = torch.zeros(*scales.shape[:-1], 32 * groups, dtype=torch.float64, device=codes.device)
    for c in range(32 * groups):
        nibble = ((c % 32 // 4) * groups + c // 32) * 4 + c % 4
        out[..., c] = ((codes[..., nibble // 2] >> (4 * (nibble % 2))) & 15).double() - 8
        out[..., c] *= scales[..., c // 32].double()
    return out
