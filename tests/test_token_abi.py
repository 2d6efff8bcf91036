"""Host checks of the token log-prob and gradient-norm entry points (no
pointer is dereferenced: fake addresses, no GPU)."""
import ctypes
import math

import pytest

import grad_row_online_gb300 as g
from test_abi import FAKE, lib  # noqa: F401  (the built library)


def _fwd(lib, dt=1, B=2, T=3, V=100, sb=300, st=100, logits=FAKE, ids=FAKE, mask=FAKE, temp=1.0,
         k=0, lp=FAKE, ent=None, stats=None, ti=None, tl=None, status=None):
    return lib.grpo_token_logps(logits, dt, B, T, V, sb, st, ids, mask, temp, k, lp, ent, stats,
                                ti, tl, status, None)


def test_token_logps_rejects_bad_arguments(lib):  # noqa: F811
    assert _fwd(lib, dt=3) == 3
    assert _fwd(lib, dt=-1) == 3
    for kw in (dict(B=-1), dict(T=-1), dict(V=0), dict(V=1 << 31), dict(T=(1 << 30) + 1),
               dict(B=1 << 20, T=1 << 20), dict(sb=-1), dict(st=-1), dict(sb=1 << 62)):
        assert _fwd(lib, **kw) == 2, kw
    for t in (0.0, -1.0, math.nan, math.inf, 1e-45, 4.1e-39):
        assert _fwd(lib, temp=t) == 6, t
    assert _fwd(lib, k=-1) == 6
    assert _fwd(lib, k=33, ti=FAKE, tl=FAKE) == 6
    assert _fwd(lib, V=4, k=5, ti=FAKE, tl=FAKE) == 6
    assert _fwd(lib, logits=None) == 1
    assert _fwd(lib, ids=None) == 1
    assert _fwd(lib, k=2, ti=FAKE) == 1
    assert _fwd(lib, k=2, tl=FAKE) == 1
    for kw in (dict(logits=FAKE + 1), dict(logits=FAKE + 2, dt=0), dict(ids=FAKE + 4),
               dict(lp=FAKE + 2), dict(ent=FAKE + 1), dict(stats=FAKE + 2),
               dict(k=1, ti=FAKE + 4, tl=FAKE), dict(k=1, ti=FAKE, tl=FAKE + 2),
               dict(status=FAKE + 16)):
        assert _fwd(lib, **kw) == 4, kw
    assert _fwd(lib, B=0, logits=None, ids=None) == 0  # nothing to do
    assert _fwd(lib, T=0) == 0


def _bwd(lib, dt=1, B=2, T=3, V=100, sb=300, st=100, logits=FAKE, ids=FAKE, mask=None, stats=FAKE,
         ent=None, dl=FAKE, dh=None, temp=1.0, grad=2 * FAKE, gsb=300, gst=100, flags=0,
         status=None):
    return lib.grpo_token_logps_grad(logits, dt, B, T, V, sb, st, ids, mask, stats, ent, dl, dh,
                                     temp, grad, gsb, gst, flags, status, None)


def test_token_logps_grad_rejects_bad_arguments(lib):  # noqa: F811
    assert _bwd(lib, dt=7) == 3
    for kw in (dict(B=-1), dict(V=0), dict(sb=-1), dict(gsb=-1), dict(gst=-5), dict(gst=99),
               dict(gsb=299), dict(gsb=100, gst=100), dict(gst=0), dict(gsb=0),
               dict(grad=FAKE, gsb=600), dict(grad=FAKE, sb=0)):
        assert _bwd(lib, **kw) == 2, kw
    for t in (0.0, math.nan, -2.0):
        assert _bwd(lib, temp=t) == 6
    for f in (1, 4, 1 << 31):
        assert _bwd(lib, flags=f) == 6
    for kw in (dict(dl=None), dict(logits=None), dict(stats=None), dict(grad=None), dict(ids=None),
               dict(dh=FAKE)):
        assert _bwd(lib, **kw) == 1, kw
    for kw in (dict(logits=FAKE + 1), dict(grad=FAKE + 1), dict(ids=FAKE + 4), dict(stats=FAKE + 2),
               dict(dl=FAKE + 2), dict(dh=FAKE + 1, ent=FAKE), dict(dh=FAKE, ent=FAKE + 2),
               dict(status=FAKE + 8)):
        assert _bwd(lib, **kw) == 4, kw
    assert _bwd(lib, B=0) == 0
    # a [T, B, V] order is not an overlap, and a single row has any stride
    assert _bwd(lib, T=0, gsb=100, gst=200) == 0
    assert _bwd(lib, B=1, T=0, gsb=0, gst=0) == 0


def _clip(lib, ptrs=(FAKE, 2 * FAKE), outs=None, numels=(10, 20), dtypes=(0, 1), n=2, max_norm=1.0,
          eps=1e-6, scale=1.0, flags=0, out2=FAKE, ws=FAKE, ws_bytes=None):
    arr = lambda t, v: None if v is None else (t * len(v))(*v)
    need = lib.grpo_clip_workspace_size(max(n, 0)) if ws_bytes is None else ws_bytes
    return lib.grpo_clip_grad_norm(arr(ctypes.c_void_p, ptrs), arr(ctypes.c_void_p, outs),
                                   arr(ctypes.c_int64, numels), arr(ctypes.c_int32, dtypes), n,
                                   max_norm, eps, scale, flags, out2, ws, need, None)


def test_clip_grad_norm_rejects_bad_arguments(lib):  # noqa: F811
    assert _clip(lib, n=-1) == 2
    assert _clip(lib, n=(1 << 20) + 1) == 2
    assert _clip(lib, numels=(10, -1)) == 2
    assert _clip(lib, numels=(1 << 40, 1)) == 2
    assert _clip(lib, dtypes=(0, 3)) == 3
    assert _clip(lib, dtypes=(-1, 0)) == 3
    for kw in (dict(max_norm=-1.0), dict(max_norm=math.nan), dict(eps=-1.0), dict(eps=math.inf),
               dict(eps=math.nan), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
               dict(scale=math.nan), dict(flags=2), dict(flags=1, outs=(FAKE, FAKE))):
        assert _clip(lib, **kw) == 6, kw
    for kw in (dict(ptrs=None), dict(numels=None), dict(dtypes=None), dict(out2=None),
               dict(ws=None), dict(ptrs=(FAKE, None)), dict(outs=(None, FAKE))):
        assert _clip(lib, **kw) == 1, kw
    for kw in (dict(ptrs=(FAKE + 2, FAKE)), dict(ptrs=(FAKE, FAKE + 1)), dict(out2=FAKE + 2),
               dict(outs=(FAKE + 2, FAKE)), dict(ws=FAKE + 128)):
        assert _clip(lib, **kw) == 4, kw
    assert _clip(lib, ws_bytes=16) == 7
    assert lib.grpo_clip_workspace_size(-1) == 0
    assert lib.grpo_clip_workspace_size(1) % 256 == 0
    assert lib.grpo_clip_workspace_size(5000) > lib.grpo_clip_workspace_size(5)


def test_wrappers_check_before_the_library(lib):  # noqa: F811
    import torch
    x = torch.zeros((2, 3, 10))
    ids = torch.zeros((2, 3), dtype=torch.int64)
    with pytest.raises(ValueError):  # a host tensor
        g.grpo_token_logps(x, ids)
    with pytest.raises(ValueError):
        g.grpo_token_logps_grad(x, ids, None, torch.zeros((2, 2, 3)), grad_logps=x[..., 0])
    for bad in ([x], [None], ["x"]):
        with pytest.raises(ValueError):
            g.grpo_clip_grad_norm(bad, 1.0)
    for bad in (None, 3, x.double(), x.long(), x[0, 0]):
        with pytest.raises(ValueError):
            g.grpo_token_logps(bad, ids)
    with pytest.raises(TypeError):
        g.grpo_clip_grad_norm([x], "one")
    with pytest.raises(TypeError):
        g.native().token_logps(x)
