"""Host-side checks of the entry points for positions of several axes, shared prefixes, attention weights
and eviction (no GPU needed): what they refuse, with the documented status codes, before anything is
launched, and the sizes of their workspaces."""
import ctypes

import pytest

INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 3
P = ctypes.c_void_p
A, B8, MIS = P(0x10000), P(0x20000), P(0x10008)  # placeholders, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from vision_transformer_attention_psapackqkv_gb300 import _build, binding

    _build.build()
    return binding.load()


def _no_device():
    import torch

    return not torch.cuda.is_available()


placeholder_only = pytest.mark.skipif(not _no_device(), reason="placeholder pointers are for GPU-less hosts")


def _rows(heads=4, N=16, d=64, ptr=0x10000, **strides):
    from vision_transformer_attention_psapackqkv_gb300.binding import PsaRows

    s = dict(b=heads * N * d, h=N * d, n=d) | strides
    return PsaRows(ptr, s["b"], s["h"], s["n"])


def _axes(axes=3, sections=(8, 12, 12), grid=(2, 2, 4, 0), normalize=1, of_pair=None, **rope):
    from vision_transformer_attention_psapackqkv_gb300.binding import PsaNormRope, PsaRopeAxes

    r = dict(B=2, nh=4, nkv=2, N=16, d=64, dtype=1, rot=64, inter=0, max_pos=16, eps=1e-6) | rope
    of = of_pair or [a for a, n in enumerate(sections) for _ in range(n)]
    return PsaRopeAxes(PsaNormRope(*r.values()), axes, (ctypes.c_int * 4)(*grid), normalize, (ctypes.c_ubyte * 64)(*of))


def _window(B=2, nh=4, nkv=2, nq=16, nk=16, d=64, dtype=1, left=-1, right=0, sinks=0):
    from vision_transformer_attention_psapackqkv_gb300.binding import PsaWindow

    return PsaWindow(B, nh, nkv, nq, nk, d, dtype, left, right, sinks)


def _prefix(B=2, nh=4, nkv=2, nq=16, P=100, nk=16, d=64, dtype=1):
    from vision_transformer_attention_psapackqkv_gb300.binding import PsaPrefix

    return PsaPrefix(B, nh, nkv, nq, P, nk, d, dtype)


def _evict(B=2, nkv=2, max_len=16, d=64, dtype=1, keep=8, sinks=2, recent=4):
    from vision_transformer_attention_psapackqkv_gb300.binding import PsaEvict

    return PsaEvict(B, nkv, max_len, d, dtype, keep, sinks, recent)


KV = dict(heads=2)


@placeholder_only
def test_axes_refusals(lib):
    def fwd(p=_axes(), q=_rows(), k=_rows(**KV), qw=A, cos=A, sin=A, pos=None, qo=_rows(), ko=_rows(**KV)):
        return lib.psa_qk_norm_rope_axes_fwd(q, k, qw, A, cos, sin, pos, qo, ko, p, None)

    assert fwd(p=_axes(axes=0)) == INVALID
    assert fwd(p=_axes(axes=5)) == INVALID
    assert fwd(p=_axes(normalize=2)) == INVALID
    assert fwd(p=_axes(axes=2)) == INVALID                          # a pair turns with an axis that is not there
    assert fwd(p=_axes(of_pair=[0] * 31 + [3])) == INVALID
    assert fwd(p=_axes(grid=(2, 2, 3, 0))) == INVALID               # 12 cells, 16 tokens
    assert fwd(p=_axes(grid=(2, 2, 8, 0))) == INVALID
    assert fwd(p=_axes(grid=(2, -2, -4, 0))) == INVALID
    assert fwd(p=_axes(grid=(0, 0, 0, 0))) == INVALID
    assert fwd(p=_axes(grid=(2, 2, 4, 0), max_pos=3)) == INVALID    # an extent past the tables
    assert fwd(p=_axes(grid=(2 ** 30, 2 ** 30, 16, 0), max_pos=2 ** 30)) == INVALID
    assert fwd(p=_axes(rot=24)) == INVALID
    assert fwd(p=_axes(rot=80)) == INVALID
    assert fwd(p=_axes(d=96, rot=64)) == UNSUPPORTED
    assert fwd(cos=None) == INVALID
    assert fwd(q=_rows(ptr=0)) == INVALID
    assert fwd(ko=_rows(ptr=0x10008, **KV)) == ALIGNMENT
    assert fwd(cos=MIS) == ALIGNMENT
    assert fwd(pos=P(0x10002)) == ALIGNMENT
    assert fwd(qw=P(0x10001)) == ALIGNMENT
    ws = lib.psa_qk_norm_rope_bwd_workspace_size(_axes().rope)

    def bwd(p=_axes(), dq=_rows(), gk=_rows(**KV), dw=A, ws_ptr=A, ws_bytes=ws):
        return lib.psa_qk_norm_rope_axes_bwd(_rows(), _rows(**KV), None, None, A, A, None, _rows(), gk, dq, _rows(**KV),
                                             dw, None, ws_ptr, ws_bytes, p, None)

    assert bwd(p=_axes(axes=0)) == INVALID
    assert bwd(ws_ptr=None) == INVALID
    assert bwd(ws_bytes=ws - 1) == INVALID
    assert bwd(ws_ptr=MIS) == ALIGNMENT
    assert bwd(dw=P(0x10002)) == ALIGNMENT
    assert bwd(dq=_rows(n=32)) == INVALID
    assert bwd(gk=_rows(b=0, **KV)) == INVALID                      # a broadcast gradient


@placeholder_only
def test_prefix_refusals(lib):
    size = lib.psa_prefix_attn_workspace_size
    for bad in (_prefix(nq=0), _prefix(P=0), _prefix(nk=8), _prefix(nh=3), _prefix(d=32), _prefix(dtype=0), _prefix(B=40000),
                _prefix(B=8000, nh=8, nq=5000, nk=5000)):
        assert size(bad) == 0
    shared = _rows(heads=2, N=100, b=-7)  # the stride of its single sequence is not read

    def fwd(p=_prefix(), q=_rows(), kp=shared, k=_rows(**KV), lens=None, o=_rows(), lse=None, ws=A, more=0, scale=0.1):
        return lib.psa_prefix_attn_fwd(q, kp, shared, k, _rows(**KV), lens, o, lse, ws, size(p) + more, p, scale, None)

    assert fwd(p=_prefix(P=0)) == INVALID
    assert fwd(p=_prefix(nq=17)) == INVALID                        # more queries than own keys
    assert fwd(p=_prefix(nkv=3)) == INVALID
    assert fwd(p=_prefix(dtype=0)) == UNSUPPORTED
    assert fwd(p=_prefix(dtype=2)) == INVALID
    assert fwd(p=_prefix(d=256)) == UNSUPPORTED
    assert fwd(p=_prefix(P=2 ** 28 + 1)) == UNSUPPORTED
    assert fwd(scale=0.0) == INVALID
    assert fwd(ws=None) == INVALID
    assert fwd(more=-1) == INVALID
    assert fwd(ws=MIS) == ALIGNMENT
    assert fwd(kp=_rows(ptr=0, heads=2, N=100)) == INVALID
    assert fwd(kp=_rows(heads=2, N=100, n=72, h=7200, ptr=0x10008)) == ALIGNMENT
    assert fwd(kp=_rows(heads=2, N=100, h=64)) == INVALID          # heads overlap
    assert fwd(lse=P(0x10002)) == ALIGNMENT
    one = _prefix(nq=1)

    def decode(p=one, q=_rows(N=1), lens=A, ws=A, more=0, kp=shared):
        return lib.psa_prefix_attn_decode(q, kp, shared, _rows(**KV), _rows(**KV), lens, _rows(N=1), ws, size(p) + more, p, 0.1, None)

    assert decode(p=_prefix()) == INVALID                          # not single tokens
    assert decode(lens=None) == INVALID
    assert decode(lens=P(0x10002)) == ALIGNMENT
    assert decode(more=-1) == INVALID
    assert decode(q=_rows(N=1, ptr=0x10004)) == ALIGNMENT


@placeholder_only
def test_weights_refusals(lib):
    size = lib.psa_window_attn_weights_workspace_size
    assert size(_window()) > 0 and size(_window(d=32)) == 0

    def call(w=_window(), q=_rows(), k=_rows(**KV), lens=None, lse=A, weights=A, ws=A, more=0, scale=0.1):
        return lib.psa_window_attn_weights(q, k, lens, lse, weights, ws, size(w) + more, w, scale, None)

    assert call(w=_window(nq=0)) == INVALID
    assert call(w=_window(dtype=0)) == UNSUPPORTED
    assert call(w=_window(d=32)) == UNSUPPORTED
    assert call(lse=None) == INVALID
    assert call(weights=None) == INVALID
    assert call(ws=None) == INVALID
    assert call(more=-1) == INVALID
    assert call(scale=float("inf")) == INVALID
    assert call(k=_rows(ptr=0, **KV)) == INVALID
    assert call(lse=P(0x10002)) == ALIGNMENT
    assert call(weights=P(0x10002)) == ALIGNMENT
    assert call(lens=P(0x10001)) == ALIGNMENT
    assert call(ws=MIS) == ALIGNMENT
    step = lib.psa_window_attn_decode_weights_workspace_size
    one = _window(nq=1)
    assert step(_window()) == 0 and step(one) > lib.psa_window_attn_decode_workspace_size(one)
    # by what a step can see, not by how long the cache is
    assert step(_window(B=1, nq=1, nk=2 ** 24, left=1000, sinks=16)) < 1 << 20

    def decode(w=one, q=_rows(N=1), lens=A, o=_rows(N=1), weights=A, ws=A, more=0):
        return lib.psa_window_attn_decode_weights(q, _rows(**KV), _rows(**KV), lens, o, weights, ws, step(w) + more, w, 0.1, None)

    assert decode(w=_window(nq=2)) == INVALID
    assert decode(w=_window(nq=1, dtype=0)) == UNSUPPORTED
    assert decode(lens=None) == INVALID
    assert decode(weights=None) == INVALID
    assert decode(weights=P(0x10002)) == ALIGNMENT
    assert decode(more=-1) == INVALID
    many = _window(nq=1, B=1, nh=5000, nkv=1)
    assert step(many) == 0 and decode(w=many, q=_rows(heads=5000, N=1), o=_rows(heads=5000, N=1)) in (INVALID, UNSUPPORTED)


@placeholder_only
def test_evict_refusals(lib):
    size = lib.psa_kv_evict_workspace_size
    assert size(_evict()) > 0

    def call(p=_evict(), w=A, pos=A, lens=A, k=_rows(**KV), v=_rows(**KV), w_out=A, pos_out=A, lens_out=B8, ws=A, more=0):
        return lib.psa_kv_evict(w, pos, lens, k, v, w_out, pos_out, lens_out, ws, size(p) + more, p, None)

    for bad in (dict(keep=0), dict(sinks=-1), dict(recent=-1), dict(sinks=5), dict(recent=2 ** 31 - 1, sinks=2 ** 31 - 1), dict(B=0),
                dict(max_len=0), dict(dtype=3), dict(nkv=-1)):
        assert size(_evict(**bad)) == 0 and call(p=_evict(**bad)) == INVALID
    for bad in (dict(d=32), dict(max_len=2 ** 24 + 1), dict(B=40000)):
        assert size(_evict(**bad)) == 0 and call(p=_evict(**bad)) == UNSUPPORTED
    for name in ("w", "pos", "lens", "w_out", "pos_out", "lens_out", "ws"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: P(0x30002)}) == ALIGNMENT
    assert call(lens_out=A) == INVALID                              # lens itself
    assert call(more=-1) == INVALID
    assert call(k=_rows(ptr=0, **KV)) == INVALID
    assert call(v=_rows(ptr=0x10004, **KV)) == ALIGNMENT
    assert call(v=_rows(n=0, **KV)) == INVALID
