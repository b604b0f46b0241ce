"""Host-side checks of the token-sequence entry points (no GPU needed): views, problems and
workspaces that they refuse, with the documented status codes, before anything is launched."""
import ctypes

import pytest

INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 3
P = ctypes.c_void_p
A, MIS = P(0x10000), P(0x10008)  # placeholders, never dereferenced


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


def _window(B=2, nh=4, nkv=2, nq=16, nk=16, d=64, dtype=1, left=-1, right=0, sinks=0):
    from vision_transformer_attention_psapackqkv_gb300.binding import PsaWindow

    return PsaWindow(B, nh, nkv, nq, nk, d, dtype, left, right, sinks)


def _norm(B=2, nh=4, nkv=2, N=16, d=64, dtype=1, rot=64, inter=0, max_pos=16, eps=1e-6):
    from vision_transformer_attention_psapackqkv_gb300.binding import PsaNormRope

    return PsaNormRope(B, nh, nkv, N, d, dtype, rot, inter, max_pos, eps)


def _cache(B=2, nkv=2, N=4, max_len=16, d=64, dtype=1):
    from vision_transformer_attention_psapackqkv_gb300.binding import PsaCache

    return PsaCache(B, nkv, N, max_len, d, dtype)


KV = dict(heads=2)


@placeholder_only
def test_window_forward_refusals(lib):
    f = lib.psa_window_attn_fwd

    def call(q=_rows(), k=_rows(**KV), v=_rows(**KV), lens=None, o=_rows(), lse=None, w=_window(), scale=0.1):
        return f(q, k, v, lens, o, lse, w, scale, None)

    assert call(q=_rows(ptr=0)) == INVALID
    assert call(o=_rows(ptr=0)) == INVALID
    assert call(w=_window(nh=3, nkv=2)) == INVALID
    assert call(w=_window(nq=0)) == INVALID
    assert call(w=_window(nk=-1)) == INVALID
    assert call(w=_window(B=0)) == INVALID
    assert call(w=_window(sinks=-1)) == INVALID
    assert call(w=_window(dtype=2)) == INVALID
    assert call(scale=0.0) == INVALID
    assert call(scale=float("nan")) == INVALID
    for d in (32, 96, 256):
        assert call(w=_window(d=d)) == UNSUPPORTED
    assert call(w=_window(B=40000)) == UNSUPPORTED
    assert call(k=_rows(ptr=0x10008, **KV)) == ALIGNMENT
    assert call(v=_rows(n=68, **KV)) == INVALID             # then a head's rows run into the next head's
    assert call(v=_rows(n=68, h=68 * 16, b=68 * 32, **KV)) == ALIGNMENT  # 136-byte rows
    assert call(q=_rows(n=32)) == INVALID                   # rows overlap
    assert call(q=_rows(b=0)) == INVALID                    # broadcast batch
    assert call(q=_rows(h=-64)) == INVALID
    assert call(lens=P(0x10002)) == ALIGNMENT
    assert call(lse=P(0x10001)) == ALIGNMENT


@placeholder_only
def test_strides_of_single_entries_are_not_read(lib):
    # passes every check of the views and stops at the last one, the misaligned lse
    w = _window(B=1, nh=1, nkv=1)
    one = _rows(heads=1, b=-5, h=3)
    assert lib.psa_window_attn_fwd(one, one, one, None, one, P(0x10001), w, 0.1, None) == ALIGNMENT


@placeholder_only
def test_window_backward_refusals(lib):
    ws = lib.psa_window_attn_bwd_workspace_size(_window())
    assert ws >= 2 * 4 * 16 * 4
    assert lib.psa_window_attn_bwd_workspace_size(_window(d=48)) == 0

    def call(lse=A, dk=_rows(**KV), ws_ptr=A, ws_bytes=ws, w=_window(), do=_rows()):
        return lib.psa_window_attn_bwd(_rows(), _rows(**KV), _rows(**KV), _rows(), do, lse, None, _rows(), dk,
                                       _rows(**KV), ws_ptr, ws_bytes, w, 0.1, None)

    assert call(lse=None) == INVALID
    assert call(ws_ptr=None) == INVALID
    assert call(ws_bytes=ws - 1) == INVALID
    assert call(ws_ptr=MIS) == ALIGNMENT
    assert call(dk=_rows(ptr=0x10004, **KV)) == ALIGNMENT
    assert call(do=_rows(ptr=0)) == INVALID
    assert call(w=_window(d=32)) == UNSUPPORTED


@placeholder_only
def test_decode_refusals(lib):
    w = _window(nq=1, nk=512)
    ws = lib.psa_window_attn_decode_workspace_size(w)
    assert ws > 0
    assert lib.psa_window_attn_decode_workspace_size(_window(nq=2)) == 0
    q, kv = _rows(N=1), _rows(N=512, **KV)

    def call(q=q, k=kv, lens=A, o=q, ws_ptr=A, ws_bytes=ws, w=w, scale=0.1):
        return lib.psa_window_attn_decode(q, k, kv, lens, o, ws_ptr, ws_bytes, w, scale, None)

    assert call(lens=None) == INVALID
    assert call(ws_ptr=None) == INVALID
    assert call(ws_bytes=ws - 1) == INVALID
    assert call(w=_window(nq=2, nk=512)) == INVALID
    assert call(w=_window(nq=1, nk=512, dtype=0)) == UNSUPPORTED
    assert call(w=_window(nq=1, nk=512, d=96)) == UNSUPPORTED
    assert call(k=_rows(N=512, ptr=0x10008, **KV)) == ALIGNMENT
    assert call(o=_rows(N=1, ptr=0)) == INVALID
    assert call(scale=-1.0) == INVALID

    def call4(kc=A, ks=A, lens=A, w=w):
        return lib.psa_window_attn_decode_kv4(q, kc, ks, A, A, lens, q, A, ws, w, 0.1, None)

    assert call4(kc=None) == INVALID
    assert call4(ks=MIS) == ALIGNMENT
    assert call4(lens=None) == INVALID
    assert call4(w=_window(nq=1, nk=512, dtype=0)) == UNSUPPORTED


@placeholder_only
def test_cache_refusals(lib):
    r, c = _rows(N=4, **KV), _rows(N=16, **KV)
    assert lib.psa_kv_append(r, r, None, None, c, c, _cache(), None) == INVALID
    assert lib.psa_kv_append(r, r, A, None, c, c, _cache(N=0), None) == INVALID
    assert lib.psa_kv_append(r, r, A, None, c, c, _cache(d=32), None) == UNSUPPORTED
    assert lib.psa_kv_append(r, r, A, P(0x10001), c, c, _cache(), None) == ALIGNMENT
    assert lib.psa_kv_append(r, r, A, None, _rows(N=16, n=60, **KV), c, _cache(), None) == INVALID
    assert lib.psa_kv4_append(r, r, None, None, A, A, A, A, _cache(), None) == INVALID
    assert lib.psa_kv4_append(r, r, A, None, A, None, A, A, _cache(), None) == INVALID
    assert lib.psa_kv4_append(r, r, A, None, A, A, MIS, A, _cache(), None) == ALIGNMENT
    assert lib.psa_kv4_append(r, r, A, None, A, A, A, A, _cache(max_len=0), None) == INVALID
    assert lib.psa_kv4_read(A, A, A, A, r, r, _cache(N=17), None) == INVALID
    assert lib.psa_kv4_read(A, A, A, MIS, r, r, _cache(), None) == ALIGNMENT
    assert lib.psa_kv4_read(A, A, A, A, r, _rows(N=4, ptr=0, **KV), _cache(), None) == INVALID


@placeholder_only
def test_norm_rope_refusals(lib):
    def call(q=_rows(), k=_rows(**KV), cos=A, sin=A, pos=None, qo=_rows(), p=_norm()):
        return lib.psa_qk_norm_rope_fwd(q, k, None, None, cos, sin, pos, qo, _rows(**KV), p, None)

    assert call(q=_rows(ptr=0)) == INVALID
    assert call(cos=None) == INVALID
    assert call(sin=MIS) == ALIGNMENT
    assert call(pos=P(0x10002)) == ALIGNMENT
    assert call(qo=_rows(n=72)) == INVALID
    assert call(p=_norm(rot=24)) == INVALID
    assert call(p=_norm(rot=80)) == INVALID
    assert call(p=_norm(rot=-16)) == INVALID
    assert call(p=_norm(inter=2)) == INVALID
    assert call(p=_norm(max_pos=0)) == INVALID
    assert call(p=_norm(max_pos=15)) == INVALID             # rows without positions run past the table
    assert call(p=_norm(eps=float("inf"))) == INVALID
    assert call(p=_norm(eps=-1e-6)) == INVALID
    assert call(p=_norm(nkv=0)) == INVALID
    assert call(p=_norm(d=256)) == UNSUPPORTED
    assert call(p=_norm(d=16, rot=16)) == UNSUPPORTED
    ws = lib.psa_qk_norm_rope_bwd_workspace_size(_norm())
    assert ws > 0 and lib.psa_qk_norm_rope_bwd_workspace_size(_norm(N=0)) == 0
    q, k = _rows(), _rows(**KV)

    def back(dq_out=q, dw=None, ws_ptr=A, ws_bytes=ws):
        return lib.psa_qk_norm_rope_bwd(q, k, None, None, A, A, None, dq_out, k, q, k, dw, None, ws_ptr, ws_bytes,
                                        _norm(), None)

    assert back(dq_out=_rows(ptr=0)) == INVALID
    assert back(dw=P(0x10001)) == ALIGNMENT
    assert back(ws_ptr=None) == INVALID
    assert back(ws_bytes=ws - 4) == INVALID


def test_binding_refuses_on_the_host():
    import torch

    from vision_transformer_attention_psapackqkv_gb300 import binding as B

    q, k = torch.zeros(1, 4, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    win = B.window_of(q, k, 3, 0, 1)
    assert (win.num_heads, win.num_kv_heads, win.n_q, win.n_k, win.window_left, win.sinks) == (4, 2, 8, 8, 3, 1)
    with pytest.raises(ValueError, match="CUDA device"):
        B.psa_window_attn_fwd(q, k, k, None, q, None, win, 0.1)
    with pytest.raises(ValueError, match="shape"):
        B.psa_window_attn_fwd(q, k[:, :, :4], k, None, q, None, win, 0.1)
    with pytest.raises(TypeError, match="expected torch.bfloat16"):
        B.psa_window_attn_fwd(q, k.float(), k, None, q, None, win, 0.1)
    with pytest.raises(ValueError, match="contiguous"):
        B.psa_window_attn_fwd(q.transpose(2, 3).contiguous().transpose(2, 3), k, k, None, q, None, win, 0.1)
    with pytest.raises(TypeError, match="lens"):
        B.psa_window_attn_fwd(q, k, k, torch.zeros(1, dtype=torch.int64), q, None, win, 0.1)
    with pytest.raises(TypeError, match="unsupported dtype"):
        B.window_of(q.half(), k.half())
    cos = torch.zeros(8, 32)
    p = B.norm_rope_of(q, k, cos)
    assert (p.rotary_dim, p.max_pos, p.N) == (64, 8, 8)
    with pytest.raises(ValueError, match="sin"):
        B.psa_qk_norm_rope_fwd(q, k, None, None, cos, cos[:4], None, q, k, p)
    with pytest.raises(ValueError, match="k_scales"):
        B.psa_kv4_append(k, k, torch.zeros(1, dtype=torch.int32), None, torch.zeros(1, 2, 8, 32, dtype=torch.uint8),
                         torch.zeros(1, 2, 8, 4, dtype=torch.bfloat16), torch.zeros(1, 2, 8, 32, dtype=torch.uint8),
                         torch.zeros(1, 2, 8, 2, dtype=torch.bfloat16))


def test_windows_wider_than_an_int():
    """A limit that no C int holds is no limit, not what is left of its lower bits."""
    import torch

    from vision_transformer_attention_psapackqkv_gb300 import binding as B

    q = torch.zeros(1, 2, 8, 64)
    win = B.window_of(q, q, 2 ** 32, 2 ** 40, 2 ** 33 + 1)
    assert (win.window_left, win.window_right, win.sinks) == (8, 8, 8)
    win = B.window_of(q, q, -2 ** 32, -2 ** 33, 0)
    assert (win.window_left, win.window_right, win.sinks) == (-1, -1, 0)
    assert B.window_of(q, q, 0, 0, -2 ** 32).sinks == -1  # refused by the calls


def test_tensors_of_another_type_than_the_problem_s():
    """A problem made for fp32 rows reads twice the bytes of bf16 ones: past their end."""
    import torch

    from vision_transformer_attention_psapackqkv_gb300 import binding as B

    t = {torch.float32: (torch.zeros(1, 4, 8, 64), torch.zeros(1, 2, 8, 64))}
    t[torch.bfloat16] = tuple(x.bfloat16() for x in t[torch.float32])
    cos, w, ws = torch.zeros(8, 32), torch.zeros(64), torch.zeros(1 << 20, dtype=torch.uint8)
    lse, lens, u8 = torch.zeros(1, 4, 8), torch.zeros(1, dtype=torch.int32), torch.uint8
    cache = tuple(torch.zeros(1, 2, 8, n, dtype=e) for n, e in ((32, u8), (2, torch.bfloat16)) * 2)
    for mine, other in ((torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)):
        q, k = t[mine]
        q1, p = q[:, :, :1], B.norm_rope_of(*t[other], cos)
        win, win1 = B.window_of(*t[other]), B.window_of(t[other][0][:, :, :1], t[other][1])
        for call in (lambda: B.psa_qk_norm_rope_fwd(q, k, w, w, cos, cos, None, q, k, p),
                     lambda: B.psa_qk_norm_rope_bwd(q, k, w, w, cos, cos, None, q, k, q, k, w, w, ws, p),
                     lambda: B.psa_window_attn_fwd(q, k, k, None, q, None, win, 0.1),
                     lambda: B.psa_window_attn_bwd(q, k, k, q, q, lse, None, q, k, k, ws, win, 0.1),
                     lambda: B.psa_window_attn_decode(q1, k, k, lens, q1, ws, win1, 0.1),
                     lambda: B.psa_window_attn_decode_kv4(q1, *cache, lens, q1, ws, win1, 0.1)):
            with pytest.raises(TypeError, match="problem"):
                call()


def test_rows_past_the_range_of_an_int():
    """More rows than a C int counts are refused, not taken for what is left of their lower bits."""
    import torch

    from vision_transformer_attention_psapackqkv_gb300 import binding as B

    one = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    k, cache, st = one.expand(1, 1, 2 ** 32 + 1, 64), torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    kv4 = tuple(torch.zeros(1, 1, 8, n, dtype=e) for n, e in ((32, torch.uint8), (2, torch.bfloat16)) * 2)
    for call in (lambda: B.psa_kv_append(k, k, st, None, cache, cache), lambda: B.psa_kv4_append(k, k, st, None, *kv4),
                 lambda: B.psa_kv4_read(*kv4, k, k)):
        with pytest.raises(ValueError, match="shape"):
            call()
    long = cache.expand(1, 1, 8, 64)[:, :, :1].expand(1, 1, 2 ** 32 + 8, 64)
    with pytest.raises(ValueError, match="shape"):
        B.psa_window_attn_fwd(cache, long, long, None, cache, None, B.window_of(cache, long), 0.1)
    with pytest.raises(ValueError, match="shape"):
        B.psa_qk_norm_rope_fwd(k, k, None, None, None, None, None, k, k, B.norm_rope_of(k, k, None))
