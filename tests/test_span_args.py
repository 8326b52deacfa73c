"""The span attentions' and the norm and rotation's argument checks and workspace queries, without a GPU."""

import ctypes

import numpy as np
import pytest

from oracle import attention as oa


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_lightning_b200 import build
    build.build()
    from sparse_attention_indexer_lightning_b200 import _lib
    return _lib.load_library()


D = ctypes.c_void_p(16)


def window(lib, q=D, latent=D, start=D, lens=D, B=1, T=4, H=16, d=576, dv=512, n=100, max_q=4, w=64, align=1, sink=4,
           scale=0.04, dt=1, out=D, ws=None, wsb=0):
    return lib.ls_window_attention(q, latent, start, lens, None, B, T, H, d, dv, n, max_q, w, align, sink, scale, dt,
                                   out, None, ws, wsb, None)


def tree(lib, mask=D, words=1, q=D, B=1, T=4, H=16, d=576, n=100, max_q=4, max_ctx=0, w=0, align=1, sink=0,
         scale=0.04, dt=1, ws=None, wsb=0):
    return lib.ls_tree_attention(q, D, D, D, None, mask, words, B, T, H, d, 512, n, max_q, max_ctx, w, align, sink,
                                 scale, dt, D, None, ws, wsb, None)


def test_span_refusals(lib):
    for kw in (dict(B=-1), dict(T=-1), dict(H=0), dict(H=1025), dict(max_q=-1), dict(w=0), dict(w=-1), dict(align=0),
               dict(sink=-1), dict(w=1 << 30), dict(T=1 << 22, H=1024), dict(dt=2), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(n=0), dict(n=1 << 31), dict(q=None), dict(latent=None),
               dict(start=None), dict(lens=None), dict(out=None), dict(q=ctypes.c_void_p(24)),
               dict(latent=ctypes.c_void_p(8)), dict(out=ctypes.c_void_p(4)),
               dict(B=1 << 20, T=1 << 20, H=1024, max_q=1 << 20)):
        assert window(lib, **kw) == 1, kw
    assert window(lib, d=512) == 3 and window(lib, dv=576) == 3
    assert window(lib, T=0) == 0 and window(lib, B=0) == 0 and window(lib, max_q=0) == 0
    for kw in (dict(mask=None), dict(words=0), dict(words=-1), dict(words=(1 << 20) + 1), dict(w=-1), dict(align=0),
               dict(n=0), dict(q=None)):
        assert tree(lib, **kw) == 1, kw
    assert tree(lib, d=128) == 3
    assert tree(lib, T=0) == 0


def test_span_workspaces(lib):
    """Few query rows over a long axis are split and need a workspace; query rows that fill the machine do not."""
    need = lib.ls_tree_attention_workspace_size(1, 16, 128, 16, 40000, 32768, 0, 1, 0)
    assert need >= 2 * 16 * 128 * 513 * 4
    assert tree(lib, T=16, H=128, n=40000, max_q=16, max_ctx=32768, ws=D, wsb=need - 1) == 2
    assert tree(lib, T=16, H=128, n=40000, max_q=16, max_ctx=32768, ws=None, wsb=need) == 1
    assert lib.ls_window_attention_workspace_size(1, 4096, 128, 4096, 512, 1, 4) == 0
    assert lib.ls_window_attention_workspace_size(0, 16, 128, 16, 512, 1, 4) == 0
    assert lib.ls_window_attention_workspace_size(1, 16, 128, 16, 0, 1, 4) == 0
    # max_q above T changes nothing: a sequence has at most T tokens
    assert (lib.ls_window_attention_workspace_size(1, 4, 16, 4, 512, 1, 4)
            == lib.ls_window_attention_workspace_size(1, 4, 16, 1000, 512, 1, 4))


def rows(lib, **kw):
    from sparse_attention_indexer_lightning_b200._lib import NormRows
    v = dict(x=16, x_stride=512, heads=4, norm=1, weight=None, bias=None, out=16, scale=16, slots=None, out_rows=0)
    v.update(kw)
    return NormRows(**v)


def norm(lib, q=None, k=None, pos=D, f=D, T=4, d=128, nd=128, rope=64, off=0, eps=1e-6, dt=0):
    return lib.ls_norm_rope(None if q is None else ctypes.byref(q), None if k is None else ctypes.byref(k), pos, f, T, d,
                            nd, rope, off, 0, eps, dt, None)


def test_norm_refusals(lib):
    for kw in (dict(T=-1), dict(d=0), dict(d=100), dict(d=1032), dict(rope=63), dict(rope=258), dict(rope=64, off=65),
               dict(off=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(dt=2), dict(nd=0), dict(nd=100),
               dict(nd=136), dict(pos=None), dict(f=None)):
        assert norm(lib, rows(lib, x_stride=8192), **kw) == 1, kw
    for kw in (dict(heads=0), dict(heads=5000), dict(norm=3), dict(x_stride=500), dict(x_stride=504), dict(x=None),
               dict(out=None), dict(x=8), dict(out=24), dict(slots=16, out_rows=-1)):
        assert norm(lib, rows(lib, **kw)) == 1, kw
        assert norm(lib, None, rows(lib, **kw)) == 1, kw
    assert norm(lib, rows(lib, scale=None), dt=1) == 1
    assert norm(lib, rows(lib), T=0) == 0 and norm(lib) == 0


def test_window_oracle_by_hand():
    """The windows that the definition gives, written out."""
    assert oa.window_rows(5, 3, 1, 0) == [3, 4, 5]
    assert oa.window_rows(5, 3, 1, 2) == [0, 1, 3, 4, 5]
    assert oa.window_rows(1, 3, 1, 4) == [0, 1]
    assert oa.window_rows(-1, 3, 1, 4) == []
    assert oa.window_rows(9, 1, 4, 1) == [0, 8, 9]
    assert oa.window_rows(7, 1, 4, 0) == [4, 5, 6, 7]
    assert oa.window_rows(9, 3, 4, 0) == [4, 5, 6, 7, 8, 9]


def test_norm_oracle_by_hand():
    x = np.zeros((1, 1, 8))
    x[0, 0] = [3.0, 4.0, 0, 0, 1.0, 2.0, 3.0, 4.0]
    y = oa.norm_rope(x, [0], [1.0], "rms", 4, None, None, 0.0, 4, True)
    assert np.allclose(y[0, 0, :4], np.array([3, 4, 0, 0]) / 2.5) and np.array_equal(y[0, 0, 4:], x[0, 0, 4:])
    y = oa.norm_rope(x, [1], [np.pi / 2, 0.0], "none", 8, None, None, 0.0, 4, True)
    assert np.allclose(y[0, 0, 4:], [-2, 1, 3, 4])
    y = oa.norm_rope(x, [1], [np.pi / 2, 0.0], "none", 8, None, None, 0.0, 4, False)
    assert np.allclose(y[0, 0, 4:], [-3, 2, 1, 4])


def test_bindings_refuse_host_tensors():
    import torch

    import sparse_attention_indexer_lightning_b200 as ls
    q = torch.zeros(2, 16, 576, dtype=torch.bfloat16)
    lat, i32 = torch.zeros(9, 576, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: ls.ls_window_attention(q, lat, i32, i32[:1]),
                 lambda: ls.ls_tree_attention(q, lat, i32, i32[:1], torch.zeros(2, 1, dtype=torch.int64)),
                 lambda: ls.ls_norm_rope(q, None, torch.zeros(2, dtype=torch.int64), torch.ones(32)),
                 lambda: ls.ls_norm_rope()):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ls.ls_tree_attention(q, lat, i32, i32[:1], None)
