"""CPU checks of the norm, checkpoint and embedding entry points: every bad argument is refused before a GPU is
touched, by the library and by the binding."""
import ctypes

import pytest
import torch

import atomistic_cell_list_b200 as e2f

OK, INVALID, UNSUPPORTED, ALIGN = 0, 1, 2, 4


def _v(p):
    return None if p is None else ctypes.c_void_p(p)


def _norm(cfg, **kw):
    a = dict(n=4, x=16, xs=None, res=None, w=32, b=48, sum=None, y=64, mean=4, rstd=4, codes=None, scales=None)
    a.update(kw)
    return e2f.lib().e2f_layer_norm(ctypes.byref(cfg), a["n"], *[_v(a[k]) for k in (
        "x", "xs", "res", "w", "b", "sum", "y", "mean", "rstd", "codes", "scales")], None)


def _norm_bwd(cfg, **kw):
    a = dict(n=4, x=16, xs=None, w=32, mean=4, rstd=4, gy=64, skip=None, gx=80, gw=96, gb=112, ws=256, wsb=1 << 24)
    a.update(kw)
    return e2f.lib().e2f_layer_norm_backward(ctypes.byref(cfg), a["n"], *[_v(a[k]) for k in (
        "x", "xs", "w", "mean", "rstd", "gy", "skip", "gx", "gw", "gb", "ws")], a["wsb"], None)


@pytest.mark.parametrize("cfg,code", [((5, 16), UNSUPPORTED), ((-1, 16), INVALID), ((0, 0), INVALID),
                                      ((0, 16385), UNSUPPORTED)])
def test_norm_shapes(cfg, code):
    c = e2f.make_norm_cfg(*cfg)
    assert _norm(c) == code and _norm_bwd(c) == code
    assert e2f.e2f_layer_norm_backward_workspace_size(4, c) == 0


@pytest.mark.parametrize("eps", [0.0, -1.0, float("nan"), float("inf")])
def test_norm_eps(eps):
    assert _norm(e2f.make_norm_cfg(0, 16, eps=eps)) == INVALID


def test_norm_arguments():
    c, q = e2f.make_norm_cfg(2, 16), e2f.make_norm_cfg(2, 16, "mxi8")
    assert _norm(e2f.e2f_norm_cfg(2, 16, 1e-5, 3, 0)) == UNSUPPORTED
    assert _norm(e2f.e2f_norm_cfg(2, 16, 1e-5, 0, 2)) == UNSUPPORTED
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(n=-1), dict(n=1 << 31), dict(res=128), dict(sum=128),
               dict(codes=128), dict(scales=128), dict(y=16), dict(res=128, sum=128), dict(res=128, sum=64),
               dict(res=64, sum=128)):
        assert _norm(c, **kw) == INVALID, kw
    for kw in (dict(x=8), dict(w=8), dict(b=8), dict(y=8), dict(res=8, sum=128), dict(res=128, sum=8),
               dict(codes=8, scales=1)):
        assert _norm(c, **kw) == ALIGN, kw
    assert _norm(q) == INVALID                                  # no scales
    assert _norm(q, xs=1, res=128, sum=144) == UNSUPPORTED      # a checkpoint is not added to
    assert _norm(q, xs=1, codes=128, scales=1) == UNSUPPORTED
    assert _norm(c, n=0) == OK and _norm(c, n=0, x=None, y=None) == OK


def test_norm_backward_arguments():
    c, q = e2f.make_norm_cfg(2, 16), e2f.make_norm_cfg(2, 16, "mxi8")
    need = e2f.e2f_layer_norm_backward_workspace_size(4, c)
    assert need > 0
    for kw in (dict(x=None), dict(w=None), dict(mean=None), dict(rstd=None), dict(gy=None), dict(gx=None),
               dict(ws=None), dict(wsb=need - 1), dict(n=-1)):
        assert _norm_bwd(c, **kw) == INVALID, kw
    for kw in (dict(x=8), dict(w=8), dict(gy=8), dict(skip=8), dict(gx=8), dict(gw=8), dict(gb=8), dict(ws=128)):
        assert _norm_bwd(c, **kw) == ALIGN, kw
    assert _norm_bwd(q) == INVALID
    assert _norm_bwd(c, n=0, gw=None, gb=None) == OK


def test_checkpoint_arguments():
    f, g = e2f.lib().e2f_checkpoint_store, e2f.lib().e2f_checkpoint_load
    for rows, C, x, c, s, dt, code in ((4, 8, 16, 32, 1, 0, None), (-1, 8, 16, 32, 1, 0, INVALID),
                                       (4, 0, 16, 32, 1, 0, INVALID), (4, 8, None, 32, 1, 0, INVALID),
                                       (4, 8, 16, None, 1, 0, INVALID), (4, 8, 16, 32, None, 1, INVALID),
                                       (4, 8, 8, 32, 1, 0, ALIGN), (4, 8, 16, 8, 1, 0, ALIGN),
                                       (4, 8, 16, 32, 1, 2, UNSUPPORTED), (1 << 62, 8, 16, 32, 1, 0, INVALID),
                                       (0, 8, None, None, None, 0, OK)):
        if code is None:
            continue
        assert f(_v(x), dt, rows, C, _v(c), _v(s), None) == code
        assert g(_v(c), _v(s), rows, C, dt, _v(x), None) == code


def _embed(cfg, **kw):
    a = dict(tok=4, n=4, table=16, out=32, ws=None, wsb=0)
    a.update(kw)
    return e2f.lib().e2f_embedding(ctypes.byref(cfg), _v(a["tok"]), a["n"], _v(a["table"]), _v(a["out"]), _v(a["ws"]),
                                   a["wsb"], None)


def _embed_bwd(cfg, **kw):
    a = dict(tok=4, n=4, g=16, out=32, ws=256, wsb=1 << 24)
    a.update(kw)
    return e2f.lib().e2f_embedding_backward(ctypes.byref(cfg), _v(a["tok"]), a["n"], _v(a["g"]), _v(a["out"]),
                                            _v(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("cfg,code", [((0, 16), INVALID), ((-1, 16), INVALID), ((9, 0), INVALID),
                                      ((9, 16385), UNSUPPORTED), ((9, 16, 5), UNSUPPORTED), ((9, 16, -1), INVALID),
                                      ((9, 16, 0, float("nan")), INVALID), ((9, 16, 0, 1.0, "mxi8"), UNSUPPORTED),
                                      ((9, 16, 0, 1.0, "f32", "mxi8"), UNSUPPORTED)])
def test_embedding_shapes(cfg, code):
    c = e2f.make_embed_cfg(*cfg)
    assert _embed(c) == code and _embed_bwd(c) == code
    assert e2f.e2f_embedding_backward_workspace_size(4, c) == 0


def test_embedding_arguments():
    c = e2f.make_embed_cfg(9, 16, 2)
    need = e2f.e2f_embedding_backward_workspace_size(4, c)
    assert need > 0
    for kw in (dict(tok=None), dict(table=None), dict(out=None), dict(n=-1), dict(n=1 << 31), dict(ws=256, wsb=255)):
        assert _embed(c, **kw) == INVALID, kw
    for kw in (dict(table=8), dict(out=8), dict(ws=128, wsb=256)):
        assert _embed(c, **kw) == ALIGN, kw
    for kw in (dict(tok=None), dict(g=None), dict(out=None), dict(n=-1), dict(ws=None), dict(wsb=need - 1)):
        assert _embed_bwd(c, **kw) == INVALID, kw
    for kw in (dict(g=8), dict(out=8), dict(ws=128)):
        assert _embed_bwd(c, **kw) == ALIGN, kw
    assert _embed(c, n=0, tok=None, table=None, out=None) == OK


def test_binding_refuses_tensors_of_another_kind():
    c = e2f.make_norm_cfg(1, 16, "f32", "f32")
    x, w = torch.zeros(3, 4, 16), torch.ones(2, 16)
    for bad in (x, x[:, :3], x.double(), x.transpose(1, 2), x[..., ::2], torch.zeros(())):
        with pytest.raises(ValueError):
            e2f.e2f_layer_norm(c, bad, w)      # on the CPU, or of another shape, type or order
    with pytest.raises(ValueError):
        e2f.e2f_layer_norm_backward(c, x, w, x, x, x)
    with pytest.raises(ValueError):
        e2f.e2f_checkpoint_store(x.double())
    with pytest.raises(ValueError):
        e2f.e2f_checkpoint_load(torch.zeros(3, 16, dtype=torch.int8), torch.zeros(3, 1, dtype=torch.uint8), "mxi8")
    with pytest.raises(ValueError):
        e2f.e2f_embedding(e2f.make_embed_cfg(9, 16), torch.zeros(3, dtype=torch.int64), torch.zeros(9, 16))
    with pytest.raises(KeyError):
        e2f.make_norm_cfg(1, 16, "f16")


@pytest.mark.parametrize("V,C", [(100, 128), (256, 1024), (256, 16384), (5, 16383), (9, 1), (2, 33), (300, 128),
                                 (70000, 1024), (257, 16384)])
def test_workspaces_of_the_table_gradient_do_not_shrink_with_more_atoms(V, C):
    """One workspace, made for the largest batch, serves every smaller one."""
    c = e2f.make_embed_cfg(V, C)
    steps = [1, 63, 64, 65, 511, 512, 513, 18943, 18944, 18945, 19000, 30000, 37888, 37889, 606207, 606208, 606209]
    steps += [t * b + d for t in (64, 128, 256, 512, 1024, 2048) for b in (2, 37, 74, 148, 296) for d in (-1, 0, 1)]
    sizes = [e2f.e2f_embedding_backward_workspace_size(n, c) for n in sorted(steps)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("V,C", [(256, 128), (256, 1024), (256, 8192), (256, 16384), (100, 8191), (2, 16384)])
@pytest.mark.parametrize("n", [600, 19000, 100000, 600000])
def test_workspace_of_the_table_gradient_is_no_larger_than_what_it_sums(V, C, n):
    """The tiles' partial sums take no more than 16 MB or the degree-0 rows of grad_out that they are made of, nor
    more than 160 MB or a share V / 2048 of those rows (beside them at most 64 bytes an atom: flags and alignment)."""
    need = e2f.e2f_embedding_backward_workspace_size(n, e2f.make_embed_cfg(V, C))
    rows = 4 * (n + 2048) * C
    assert need <= min(max(2 ** 24, rows), max(160e6, rows * V / 2048)) + 64 * n + 4096
