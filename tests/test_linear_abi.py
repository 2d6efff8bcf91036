"""Host checks of the head's and the embedding's entry points (no pointer is
dereferenced: fake addresses, no GPU)."""
import math

import pytest
import torch

import grad_row_online_gb300 as g
from test_abi import FAKE, lib  # noqa: F401  (the built library)

BIG = 1 << 60  # bytes of workspace, more than any call needs


def _fwd(lib, dt=1, B=2, T=3, K=64, sb=192, st=64, h=FAKE, W=2 * FAKE, V=100, sv=64, ids=FAKE,
         mask=FAKE, temp=1.0, lp=FAKE, ent=None, stats=None, status=None, ws=FAKE, ws_bytes=BIG):
    return lib.grpo_linear_logps(h, dt, B, T, K, sb, st, W, V, sv, ids, mask, temp, lp, ent, stats,
                                 status, ws, ws_bytes, None)


SHAPES = [dict(B=-1), dict(T=-1), dict(K=0), dict(V=0), dict(K=(1 << 20) + 1, sv=1 << 21), dict(V=1 << 31),
          dict(V=(1 << 31) - 1), dict(B=1 << 20, T=1 << 20), dict(B=(1 << 31) - 1, T=1), dict(sb=-1), dict(st=-1),
          dict(sb=1 << 62), dict(sv=63), dict(sv=0), dict(sv=-64), dict(sv=(1 << 36) + 64),
          dict(B=1 << 24, V=1 << 26), dict(V=1 << 30, K=1 << 16, sv=1 << 16)]


def test_linear_logps_rejects_bad_arguments(lib):  # noqa: F811
    for dt in (3, -1):
        assert _fwd(lib, dt=dt) == 3
    for kw in SHAPES:
        assert _fwd(lib, **kw) == 2, kw
    for t in (0.0, -1.0, math.nan, math.inf, 1e-45, 4.1e-39):
        assert _fwd(lib, temp=t) == 6, t
    for kw in (dict(h=None), dict(W=None), dict(ids=None), dict(ws=None)):
        assert _fwd(lib, **kw) == 1, kw
    for kw in (dict(h=FAKE + 1), dict(h=FAKE + 2, dt=0), dict(W=FAKE + 1), dict(ids=FAKE + 4), dict(lp=FAKE + 2),
               dict(ent=FAKE + 1), dict(stats=FAKE + 2), dict(status=FAKE + 16), dict(ws=FAKE + 128)):
        assert _fwd(lib, **kw) == 4, kw
    assert _fwd(lib, ws_bytes=4096) == 7
    assert _fwd(lib, B=0, h=None, W=None, ids=None, ws=None) == 0
    assert _fwd(lib, T=0) == 0


def _bwd(lib, dt=1, B=2, T=3, K=64, sb=192, st=64, h=FAKE, W=2 * FAKE, V=100, sv=64, ids=FAKE, mask=FAKE,
         stats=FAKE, ent=None, dl=FAKE, dh=None, temp=1.0, gh=3 * FAKE, gsb=192, gst=64, gw=4 * FAKE, wdt=1,
         gsv=64, add=None, asv=64, flags=0, status=None, ws=FAKE, ws_bytes=BIG):
    return lib.grpo_linear_logps_grad(h, dt, B, T, K, sb, st, W, V, sv, ids, mask, stats, ent, dl, dh, temp, gh, gsb,
                                      gst, gw, wdt, gsv, add, asv, flags, status, ws, ws_bytes, None)


def test_linear_logps_grad_rejects_bad_arguments(lib):  # noqa: F811
    for kw in (dict(dt=3), dict(wdt=2), dict(wdt=5), dict(dt=0, wdt=1)):
        assert _bwd(lib, **kw) == 3, kw
    for kw in SHAPES + [dict(gsb=-1), dict(gst=63), dict(gsb=191), dict(gst=0), dict(gsv=63), dict(gsv=-1),
                        dict(add=5 * FAKE, asv=63), dict(add=4 * FAKE, asv=128)]:
        assert _bwd(lib, **kw) == 2, kw
    for t in (0.0, math.nan, -2.0):
        assert _bwd(lib, temp=t) == 6
    for f in (1, 4, 1 << 31):
        assert _bwd(lib, flags=f) == 6
    for kw in (dict(gh=None, gw=None), dict(gw=None, add=FAKE), dict(dl=None), dict(h=None), dict(W=None),
               dict(stats=None), dict(ids=None), dict(dh=FAKE), dict(ws=None)):
        assert _bwd(lib, **kw) == 1, kw
    for kw in (dict(h=FAKE + 1), dict(W=FAKE + 1), dict(gh=FAKE + 1), dict(gw=FAKE + 1), dict(gw=FAKE + 2, wdt=0),
               dict(add=FAKE + 1), dict(ids=FAKE + 4), dict(stats=FAKE + 2), dict(dl=FAKE + 2),
               dict(dh=FAKE + 1, ent=FAKE), dict(dh=FAKE, ent=FAKE + 2), dict(status=FAKE + 8), dict(ws=FAKE + 64)):
        assert _bwd(lib, **kw) == 4, kw
    assert _bwd(lib, ws_bytes=4096) == 7
    assert _bwd(lib, B=0, gw=None) == 0  # nothing to do


def test_workspace_sizes(lib):  # noqa: F811
    size = lib.grpo_linear_workspace_size
    assert size(FAKE, 3, 1, 1, 64, 100, 64, 0) == 0 and size(FAKE, 1, 1, 1, 0, 100, 64, 0) == 0
    aligned, shifted = size(FAKE, 1, 8, 64, 64, 10000, 64, 0), size(FAKE + 2, 1, 8, 64, 64, 10000, 64, 0)
    assert shifted >= aligned + 2 * 64 * 10000
    # no room for the logits: 65536 x 151936 of them
    assert size(FAKE, 1, 64, 1024, 2048, 151936, 2048, 0) < 2 * 65536 * 151936 / 10
    assert size(FAKE, 1, 64, 1024, 2048, 151936, 2048, 1) < 2 * 65536 * 151936 / 10
    assert lib.grpo_embed_workspace_size(-1, 64, 100) == 0
    assert lib.grpo_embed_workspace_size(10, 64, 0) == 0
    assert lib.grpo_embed_workspace_size(10, 64, 100) % 256 == 0
    # no tokens: what the calls without any take
    assert lib.grpo_embed_workspace_size(0, 64, 100) % 256 == 0 < lib.grpo_embed_workspace_size(0, 64, 100)
    for backward in (0, 1):
        for dt in (0, 1, 2):
            assert size(FAKE, dt, 0, 5, 64, 100, 64, backward) > 0 and size(FAKE, dt, 1, 1, 1, 1, 1, backward) > 0


def _embed(lib, dt=1, V=100, K=64, sv=64, W=FAKE, ids=FAKE, mask=None, B=2, T=3, scale=1.0, out=2 * FAKE, sb=192,
           st=64, status=None):
    return lib.grpo_embed_tokens(W, dt, V, K, sv, ids, mask, B, T, scale, out, sb, st, status, None)


def test_embed_tokens_rejects_bad_arguments(lib):  # noqa: F811
    assert _embed(lib, dt=7) == 3
    for kw in (dict(V=0), dict(K=0), dict(sv=63), dict(B=-1), dict(T=-1), dict(B=1 << 20, T=1 << 20), dict(st=63),
               dict(sb=0), dict(sb=-1), dict(V=1 << 31)):
        assert _embed(lib, **kw) == 2, kw
    for s in (math.nan, math.inf):
        assert _embed(lib, scale=s) == 6
    for kw in (dict(W=None), dict(ids=None), dict(out=None)):
        assert _embed(lib, **kw) == 1
    for kw in (dict(W=FAKE + 1), dict(out=FAKE + 2, dt=0), dict(ids=FAKE + 4), dict(status=FAKE + 8)):
        assert _embed(lib, **kw) == 4
    assert _embed(lib, B=0, W=None, ids=None, out=None) == 0


def _embed_grad(lib, dt=1, B=2, T=3, K=64, sb=192, st=64, grad=FAKE, ids=FAKE, mask=None, V=100, scale=1.0, add=None,
                asv=64, gw=2 * FAKE, wdt=1, osv=64, status=None, ws=FAKE, ws_bytes=BIG):
    return lib.grpo_embed_tokens_grad(grad, dt, B, T, K, sb, st, ids, mask, V, scale, add, asv, gw, wdt, osv, status,
                                      ws, ws_bytes, None)


def test_embed_tokens_grad_rejects_bad_arguments(lib):  # noqa: F811
    for kw in (dict(dt=7), dict(wdt=2), dict(dt=0, wdt=1)):
        assert _embed_grad(lib, **kw) == 3
    for kw in (dict(V=0), dict(K=0), dict(osv=63), dict(B=-1), dict(T=-1), dict(B=1 << 20, T=1 << 20), dict(st=-1),
               dict(sb=-1), dict(add=FAKE, asv=63), dict(add=2 * FAKE, asv=128)):
        assert _embed_grad(lib, **kw) == 2, kw
    assert _embed_grad(lib, scale=math.nan) == 6
    for kw in (dict(grad=None), dict(ids=None), dict(gw=None), dict(ws=None)):
        assert _embed_grad(lib, **kw) == 1
    for kw in (dict(grad=FAKE + 1), dict(gw=FAKE + 2, wdt=0), dict(add=FAKE + 1), dict(ids=FAKE + 4),
               dict(status=FAKE + 8), dict(ws=FAKE + 8)):
        assert _embed_grad(lib, **kw) == 4
    assert _embed_grad(lib, ws_bytes=100) == 7


def test_wrappers_check_before_the_library(lib):  # noqa: F811
    h, W, ids = torch.zeros((6, 8)), torch.zeros((10, 8)), torch.zeros(6, dtype=torch.int64)
    f = torch.zeros(6)
    for bad in (h, None, 3, h.double(), h.long(), h[0]):  # a host tensor, no tensor, other types
        with pytest.raises(ValueError):
            g.grpo_linear_logps(bad, W, ids)
        with pytest.raises(ValueError):
            g.grpo_linear_logps_grad(bad, W, ids, None, f, grad_logps=f)
        with pytest.raises(ValueError):
            g.grpo_embed_tokens(bad, ids)
        with pytest.raises(ValueError):
            g.grpo_embed_tokens_grad(bad, ids, 10)
    with pytest.raises(TypeError):
        g.native().linear_logps(h)
    with pytest.raises(TypeError):
        g.native().embed_tokens_grad(h, ids)
