"""e2f_layer_norm and e2f_layer_norm_backward against the plain 64-bit implementation, element by element within
the rounding bounds of tests/feature_ref.py, on every input and output type, from one row to long odd ones."""
import subprocess
import sys

import pytest
import torch

import atomistic_cell_list_b200 as e2f
import feature_ref as R

pytestmark = pytest.mark.gpu

EPS = 1e-5
# (n, L, C): every lane layout (a few lanes per row up to several vectors per lane, odd channel counts, long rows)
SHAPES = [(1, 0, 1), (1, 0, 16), (64, 2, 16), (5, 4, 16), (7, 1, 20), (3, 3, 31), (50, 4, 32), (9, 2, 33), (40, 4, 64),
          (11, 1, 48), (6, 4, 100), (300, 4, 128), (1, 4, 128), (13, 0, 128), (17, 3, 128), (1025, 0, 130),
          (23, 2, 200), (700, 1, 256), (6, 4, 252), (10, 4, 255), (4, 4, 256), (4, 2, 260), (19, 0, 257),
          (30, 0, 1000), (5, 1, 1001), (7, 0, 4096), (3, 0, 8190), (2, 0, 16384), (2, 4, 1024), (2, 0, 16381)]

# enough nodes that every warp takes several units, at each degree's layout
LONG = [(6000, 4, 128), (9000, 2, 64), (3000, 4, 256), (20000, 1, 16), (5000, 3, 36), (6000, 2, 101), (3000, 1, 255),
        (5000, 0, 1001), (1500, 0, 5001), (30000, 0, 33), (3000, 0, 2048), (700, 0, 8190), (400, 1, 300)]


def _x(n, L, C, dtype, seed=0, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, (L + 1) ** 2, C, generator=g)
    x[:, 0] += offset
    x *= torch.exp(torch.randn(n, 1, 1, generator=g))
    w = 1 + 0.2 * torch.randn(L + 1, C, generator=g)
    b = torch.randn(C, generator=g)
    r = torch.randn(n, (L + 1) ** 2, C, generator=g)
    return x.to(R.DT[dtype]), w, b, r


def _within(got, want, bound, what):
    d = (got.cpu().double() - want).abs()
    assert (d <= bound).all(), f"{what}: {float((d / bound).max()):.2f} of the bound"


def _check_forward(cfg_types, f, h, w, b, L):
    xt, yt = cfg_types
    hd, wd, bd = h.double(), w.double(), None if b is None else b.double()
    y, mean, rstd = R.norm(hd, wd, bd, L, float(torch.tensor(EPS)))
    by, bm, br = R.norm_bound(hd, wd, bd, L, EPS, yt)
    _within(f["y"], y, by, "y")
    _within(f["mean"], mean, bm, "mean")
    _within(f["rstd"], rstd, br * rstd, "rstd")


@pytest.mark.parametrize("yt", ["f32", "bf16"])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("n,L,C", SHAPES)
def test_forward(n, L, C, xt, yt):
    x, w, b, _ = _x(n, L, C, xt, seed=n + C)
    f = e2f.e2f_layer_norm(e2f.make_norm_cfg(L, C, xt, yt, EPS), x.cuda(), w.cuda(), b.cuda())
    _check_forward((xt, yt), f, x, w, b, L)


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("n,L,C", SHAPES)
def test_residual_and_checkpoint(n, L, C, xt):
    """The stored sum is the fp32 sum rounded once; the norm and the checkpoint are of the stored sum."""
    x, w, b, r = _x(n, L, C, xt, seed=n + C + 1)
    cfg = e2f.make_norm_cfg(L, C, xt, "f32", EPS)
    f = e2f.e2f_layer_norm(cfg, x.cuda(), w.cuda(), None, residual=r.cuda(), checkpoint=True)
    h = (x.float() + r).to(x.dtype)
    assert torch.equal(f["sum"].cpu(), h)
    _check_forward((xt, "f32"), f, h, w, None, L)
    _, code, byte = R.coded(h[:40])
    assert torch.equal(f["codes"][:40].cpu(), code) and torch.equal(f["scales"][:40].cpu(), byte)
    only = e2f.e2f_layer_norm(cfg, f["sum"], w.cuda(), None, checkpoint=True, stats=False)
    assert torch.equal(only["codes"], f["codes"]) and torch.equal(only["y"], f["y"]) and "mean" not in only


@pytest.mark.parametrize("yt", ["f32", "bf16"])
@pytest.mark.parametrize("n,L,C", SHAPES)
def test_forward_from_a_checkpoint(n, L, C, yt):
    x, w, b, _ = _x(n, L, C, "f32", seed=n + C + 2)
    val, code, byte = R.coded(x)
    f = e2f.e2f_layer_norm(e2f.make_norm_cfg(L, C, "mxi8", yt, EPS), code.cuda(), w.cuda(), b.cuda(),
                           x_scales=byte.cuda())
    _check_forward(("mxi8", yt), f, val, w, b, L)


@pytest.mark.parametrize("xt", ["f32", "bf16", "mxi8"])
@pytest.mark.parametrize("n,L,C", SHAPES)
def test_backward(n, L, C, xt):
    x, w, b, skip = _x(n, L, C, "f32" if xt == "mxi8" else xt, seed=n + C + 3)
    gy = torch.randn(x.shape, generator=torch.Generator().manual_seed(5))
    h, dev, scales = x.double(), x.cuda(), None
    if xt == "mxi8":
        h, code, byte = R.coded(x)
        dev, scales = code.cuda(), byte.cuda()
    _, mean, rstd = (t.float() for t in R.norm(h, w.double(), None, L, EPS))
    cfg = e2f.make_norm_cfg(L, C, xt, "f32", EPS)
    args = (cfg, dev, w.cuda(), mean.cuda(), rstd.cuda(), gy.cuda())
    g = e2f.e2f_layer_norm_backward(*args, x_scales=scales)
    ref = (h, w.double(), mean.double(), rstd.double(), gy.double(), L)
    for name, want, bound in zip(("x", "weight", "bias"), R.norm_backward(*ref), R.norm_backward_bound(*ref)):
        _within(g[name], want, bound, name)
    # a gradient that joins: one more fp32 sum; in place over it, without weight gradients, the same bits
    j = e2f.e2f_layer_norm_backward(*args, grad_skip=skip.cuda(), x_scales=scales)
    assert torch.equal(j["weight"], g["weight"]) and torch.equal(j["bias"], g["bias"])
    want = R.norm_backward(*ref)[0] + skip.double()
    _within(j["x"], want, R.norm_backward_bound(*ref)[0] + 2 * R.U * (want.abs() + skip.abs()), "x with skip")
    at = skip.cuda()
    k = e2f.e2f_layer_norm_backward(*args, grad_skip=at, x_scales=scales, want_weights=False, out={"x": at})
    assert k["x"] is at and set(k) == {"x"} and torch.equal(at, j["x"])
    at = gy.cuda()
    e2f.e2f_layer_norm_backward(*args[:5], at, x_scales=scales, out={"x": at})
    assert torch.equal(at, g["x"])


@pytest.mark.parametrize("xt", ["f32", "bf16", "mxi8"])
@pytest.mark.parametrize("n,L,C", LONG)
def test_long_batches(n, L, C, xt):
    """Forward with the residual and the checkpoint where x is no checkpoint, and backward. The weight gradient's
    longest chain is still below 1024: a lane's rows of its units, then the block's lanes, then the blocks."""
    x, w, b, r = _x(n, L, C, "f32" if xt == "mxi8" else xt, seed=n + C + 4)
    gy = torch.randn(x.shape, generator=torch.Generator().manual_seed(6))
    cfg = e2f.make_norm_cfg(L, C, xt, "bf16", EPS)
    if xt == "mxi8":
        h, code, byte = R.coded(x)
        dev, scales = code.cuda(), byte.cuda()
        f = e2f.e2f_layer_norm(cfg, dev, w.cuda(), b.cuda(), x_scales=scales)
    else:
        f = e2f.e2f_layer_norm(cfg, x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), checkpoint=True)
        h, scales, dev = (x.float() + r).to(x.dtype), None, f["sum"]
        assert torch.equal(dev.cpu(), h)
        _, code, byte = R.coded(h)
        assert torch.equal(f["codes"].cpu(), code) and torch.equal(f["scales"].cpu(), byte)
        h = h.double()
    _check_forward((xt, "bf16"), f, h, w, b, L)
    mean, rstd = f["mean"].cpu().double(), f["rstd"].cpu().double()
    g = e2f.e2f_layer_norm_backward(cfg, dev, w.cuda(), f["mean"], f["rstd"], gy.cuda(), x_scales=scales)
    ref = (h, w.double(), mean, rstd, gy.double(), L)
    for name, want, bound in zip(("x", "weight", "bias"), R.norm_backward(*ref), R.norm_backward_bound(*ref)):
        _within(g[name], want, bound, name)


@pytest.mark.parametrize("yt", ["f32", "bf16"])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("n,L,C", [(5000, 0, 1001), (900, 0, 259), (1200, 0, 2049), (1500, 0, 5001), (700, 0, 8190),
                                   (400, 0, 9001), (2000, 2, 100), (2000, 2, 101), (1500, 0, 4096), (400, 1, 300)])
def test_residual_without_a_checkpoint(n, L, C, xt, yt):
    """Several rows a block, the stream updated in place or not: the same bits, within the forward's bounds."""
    x, w, b, r = _x(n, L, C, xt, seed=n + C + 5)
    cfg = e2f.make_norm_cfg(L, C, xt, yt, EPS)
    f = e2f.e2f_layer_norm(cfg, x.cuda(), w.cuda(), b.cuda(), residual=r.cuda())
    h = (x.float() + r).to(x.dtype)
    assert torch.equal(f["sum"].cpu(), h)
    _check_forward((xt, yt), f, h, w, b, L)
    at = x.cuda()
    g = e2f.e2f_layer_norm(cfg, at, w.cuda(), b.cuda(), residual=r.cuda(), out={"sum": at})
    assert all(torch.equal(f[k], g[k]) for k in f)
    p = e2f.e2f_layer_norm(cfg, f["sum"], w.cuda(), None)
    _check_forward((xt, yt), p, h, w, None, L)


@pytest.mark.parametrize("n,L,C", [(9, 4, 128), (20, 0, 1000), (6, 2, 33)])
def test_gradient_against_differences(n, L, C):
    """The kernel's gradients along a random direction against a central difference of the 64-bit forward (which
    is off by its own h^2 and 2^-52 / h terms: below 1e-8 of the value's scale)."""
    x, w, b, _ = _x(n, L, C, "f32", seed=8)
    gen = torch.Generator().manual_seed(9)
    gy = torch.randn(x.shape, generator=gen)
    cfg = e2f.make_norm_cfg(L, C, "f32", "f32", EPS)
    f = e2f.e2f_layer_norm(cfg, x.cuda(), w.cuda(), b.cuda())
    g = e2f.e2f_layer_norm_backward(cfg, x.cuda(), w.cuda(), f["mean"], f["rstd"], gy.cuda())
    t = [v.double() for v in (x, w, b)]
    for k, name in enumerate(("x", "weight", "bias")):
        dirn = torch.randn(t[k].shape, generator=gen, dtype=torch.float64)
        at = lambda s: (gy.double() * R.norm(*[v + s * dirn if i == k else v for i, v in enumerate(t)], L, EPS)[0]).sum()
        diff = (at(1e-5) - at(-1e-5)) / 2e-5
        got = (g[name].cpu().double() * dirn).sum()
        scale = (g[name].cpu().double() * dirn).abs().sum()
        assert abs(got - diff) <= (2 * R.CHAIN * R.U + 1e-7) * scale


def test_large_mean_constant_rows_and_tiny_values():
    L, C = 1, 128
    x, w, b, _ = _x(6, L, C, "f32")
    x[0, 0] = 1000 + 0.01 * x[0, 0]
    x[1] = 3.0
    x[2] = 0.0
    x[3] *= 1e-20
    x[4] *= 1e15
    f = e2f.e2f_layer_norm(e2f.make_norm_cfg(L, C, "f32", "f32", EPS), x.cuda(), w.cuda(), b.cuda())
    _check_forward(("f32", "f32"), f, x, w, b, L)
    assert torch.equal(f["y"][2, 0].cpu(), b) and (f["y"][2, 1:] == 0).all()


@pytest.mark.parametrize("L,C", [(4, 128), (4, 16), (0, 1001), (2, 33)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_stay_in_their_group(L, C, bad):
    x, w, b, _ = _x(8, L, C, "f32")
    cfg = e2f.make_norm_cfg(L, C, "f32", "f32", EPS)
    clean = e2f.e2f_layer_norm(cfg, x.cuda(), w.cuda(), b.cuda(), checkpoint=True)
    t = x.clone()
    t[3, -1, C // 2] = bad
    f = e2f.e2f_layer_norm(cfg, t.cuda(), w.cuda(), b.cuda(), checkpoint=True)
    rows = R.degrees(L)[-1]
    keep = torch.ones(x.shape, dtype=torch.bool)
    keep[3, rows] = False
    assert torch.equal(f["y"].cpu()[keep], clean["y"].cpu()[keep])
    assert torch.isnan(f["y"][3, -1, C // 2])
    blk = C // 2 // 32
    assert f["scales"][3, -1, blk] == 255
    back = e2f.e2f_checkpoint_load(f["codes"], f["scales"]).cpu()
    good = torch.ones(x.shape, dtype=torch.bool)
    good[3, -1, 32 * blk:32 * blk + 32] = False
    assert torch.isnan(back[~good]).all() and torch.isfinite(back[good]).all()
    gy = torch.randn(x.shape)
    a = e2f.e2f_layer_norm_backward(cfg, x.cuda(), w.cuda(), clean["mean"], clean["rstd"], gy.cuda())
    g = e2f.e2f_layer_norm_backward(cfg, t.cuda(), w.cuda(), f["mean"], f["rstd"], gy.cuda())
    assert torch.equal(g["x"].cpu()[keep], a["x"].cpu()[keep])


@pytest.mark.parametrize("n,L,C", [(37, 4, 128), (37, 2, 33), (5, 0, 1001)])
def test_only_the_given_rows_are_written(n, L, C):
    """Buffers longer than the call: what lies behind the last atom stays as it was."""
    x, w, b, r = _x(n, L, C, "f32")
    K, nb = (L + 1) ** 2, (C + 31) // 32
    full = {"sum": ((n + 3, K, C), torch.float32), "y": ((n + 3, K, C), torch.bfloat16), "mean": ((n + 3,), torch.float32),
            "rstd": ((n + 3, L + 1), torch.float32), "codes": ((n + 3, K, C), torch.int8),
            "scales": ((n + 3, K, nb), torch.uint8)}
    full = {k: torch.full(s, 77, dtype=d, device="cuda") for k, (s, d) in full.items()}
    cfg = e2f.make_norm_cfg(L, C, "f32", "bf16", EPS)
    f = e2f.e2f_layer_norm(cfg, x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), checkpoint=True,
                           out={k: v[:n] for k, v in full.items()})
    for k, v in full.items():
        assert (v[n:] == 77).all(), k
        assert f[k].data_ptr() == v.data_ptr()
    gx = torch.full((n + 3, K, C), 77.0, device="cuda")
    e2f.e2f_layer_norm_backward(cfg, f["sum"], w.cuda(), f["mean"], f["rstd"], r.cuda(), out={"x": gx[:n]})
    assert (gx[n:] == 77).all()


@pytest.mark.parametrize("n,L,C", [(64, 4, 128), (2000, 3, 100), (500, 2, 101), (300, 0, 1001), (90, 0, 4096), (40, 1, 300)])
def test_the_residual_stream_in_place(n, L, C):
    x, w, b, r = _x(n, L, C, "bf16")
    cfg = e2f.make_norm_cfg(L, C, "bf16", "bf16", EPS)
    want = e2f.e2f_layer_norm(cfg, x.cuda(), w.cuda(), b.cuda(), residual=r.cuda(), checkpoint=True)
    at = x.cuda()
    got = e2f.e2f_layer_norm(cfg, at, w.cuda(), b.cuda(), residual=r.cuda(), checkpoint=True, out={"sum": at})
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_no_atoms():
    cfg = e2f.make_norm_cfg(2, 16, "f32", "f32", EPS)
    z = torch.zeros(0, 9, 16, device="cuda")
    w, b = torch.ones(3, 16, device="cuda"), torch.zeros(16, device="cuda")
    f = e2f.e2f_layer_norm(cfg, z, w, b, residual=z.clone(), checkpoint=True)
    assert f["y"].shape == (0, 9, 16)
    g = e2f.e2f_layer_norm_backward(cfg, z, w, f["mean"], f["rstd"], z.clone(),
                                    out={"weight": torch.ones(3, 16, device="cuda")})
    assert (g["weight"] == 0).all() and (g["bias"] == 0).all()


@pytest.mark.parametrize("L,C,n", [(4, 128, 2000), (0, 1001, 700), (4, 100, 300)])
def test_repeats_bit_for_bit_and_runs_on_another_stream(L, C, n):
    x, w, b, gy = (t.cuda() for t in _x(n, L, C, "f32"))
    cfg = e2f.make_norm_cfg(L, C, "f32", "bf16", EPS)
    ref = e2f.e2f_layer_norm(cfg, x, w, b)
    gref = e2f.e2f_layer_norm_backward(cfg, x, w, ref["mean"], ref["rstd"], gy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    f = e2f.e2f_layer_norm(cfg, x, w, b, stream=s)
    g = e2f.e2f_layer_norm_backward(cfg, x, w, f["mean"], f["rstd"], gy, stream=s)
    s.synchronize()
    assert all(torch.equal(f[k], ref[k]) for k in ref) and all(torch.equal(g[k], gref[k]) for k in gref)


def test_captured_and_replayed_on_new_inputs():
    L, C, n = 4, 128, 500
    x, w, b, gy = (t.cuda() for t in _x(n, L, C, "f32"))
    cfg = e2f.make_norm_cfg(L, C, "f32", "bf16", EPS)

    def step():
        f = e2f.e2f_layer_norm(cfg, x, w, b, residual=gy, checkpoint=True)
        return f, e2f.e2f_layer_norm_backward(cfg, f["sum"], w, f["mean"], f["rstd"], gy)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, g = step()
    for seed in (1, 2):
        new = _x(n, L, C, "f32", seed=seed)
        x.copy_(new[0])
        gy.copy_(new[3])
        graph.replay()
        torch.cuda.synchronize()
        f2, g2 = step()
        assert all(torch.equal(f[k], f2[k]) for k in f2) and all(torch.equal(g[k], g2[k]) for k in g2)


def test_refusals():
    x, w, b, r = (t.cuda() for t in _x(4, 1, 16, "f32"))
    cfg = e2f.make_norm_cfg(1, 16, "f32", "f32", EPS)
    for kw in (dict(out={"y": x}), dict(out={"y": torch.empty(4, 4, 16, device="cuda", dtype=torch.bfloat16)}),
               dict(residual=r[:3]), dict(residual=r.cpu()), dict(bias=b[:8])):
        with pytest.raises((ValueError, e2f.E2FError)):
            e2f.e2f_layer_norm(cfg, x, w, **kw)
    with pytest.raises(ValueError):
        e2f.e2f_layer_norm(e2f.make_norm_cfg(1, 16, "mxi8"), x.to(torch.int8), w)
    with pytest.raises(e2f.E2FError) as e:
        e2f.e2f_layer_norm(cfg, torch.zeros(4 * 4 * 16 + 1, device="cuda")[1:].view(4, 4, 16), w)
    assert e.value.code == 4


AROUND_48_KB = """
import sys
sys.path[:0] = %r
import torch, atomistic_cell_list_b200 as e2f, feature_ref as R, test_gpu_norm as T
n, L, failed = 2, 1, []
for xt in ("f32", "bf16", "mxi8"):
    for C in (6128, 6129, 6144):
        x, w, b, gy = T._x(n, L, C, "f32" if xt == "mxi8" else xt, seed=C)
        h, dev, scales = x.double(), x.cuda(), None
        if xt == "mxi8":
            h, code, byte = R.coded(x)
            dev, scales = code.cuda(), byte.cuda()
        _, mean, rstd = (t.float() for t in R.norm(h, w.double(), None, L, T.EPS))
        try:
            g = e2f.e2f_layer_norm_backward(e2f.make_norm_cfg(L, C, xt, "f32", T.EPS), dev, w.cuda(), mean.cuda(),
                                            rstd.cuda(), gy.cuda(), x_scales=scales)
        except e2f.E2FError as e:
            failed.append((xt, C, str(e)))
            continue
        ref = (h, w.double(), mean.double(), rstd.double(), gy.double(), L)
        for name, want, bound in zip(("x", "weight", "bias"), R.norm_backward(*ref), R.norm_backward_bound(*ref)):
            T._within(g[name], want, bound, name)
assert not failed, failed
"""


def test_weight_gradients_around_48_kb_of_shared_memory():
    """A row's weight and bias sums (8 C bytes) and the block's own 128 bytes together pass, at 6,129 channels, the
    shared memory that a launch has without asking. In a process of its own, in this order: a call with more
    channels raises the limit for all later ones."""
    r = subprocess.run([sys.executable, "-c", AROUND_48_KB % sys.path], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("C", [4, 8, 96, 192])
def test_backward_of_equal_channels_near_the_largest_value(C):
    """Channels of equal, huge values (a power of two, whose sum and mean are exact): xh is zero and the gradient
    finite, though mean x rstd, which no value of the row stands for, leaves the fp32 range."""
    n, top = 5, 2.0 ** 120
    x = torch.full((n, 1, C), top)
    _, w, b, gy = _x(n, 0, C, "f32")
    cfg = e2f.make_norm_cfg(0, C, "f32", "f32", EPS)
    f = e2f.e2f_layer_norm(cfg, x.cuda(), w.cuda(), b.cuda())
    mean, rstd = torch.full((n,), top), torch.full((n, 1), EPS, dtype=torch.float64).rsqrt().float()
    assert torch.equal(f["mean"].cpu(), mean)
    assert ((f["rstd"].cpu() - rstd).abs() <= 4 * R.U * rstd).all()
    g = e2f.e2f_layer_norm_backward(cfg, x.cuda(), w.cuda(), mean.cuda(), rstd.cuda(), gy.cuda())
    ref = (x.double(), w.double(), mean.double(), rstd.double(), gy.double(), 0)
    for name, want, bound in zip(("x", "weight", "bias"), R.norm_backward(*ref), R.norm_backward_bound(*ref)):
        _within(g[name], want, bound, name)


@pytest.mark.parametrize("n,L,xt", [(2000000, 0, "f32"), (100000, 4, "bf16"), (30000, 2, "f32")])
def test_weight_gradients_of_many_rows(n, L, xt):
    """Equal terms, whose roundings all fall to one side. The chain of additions behind one weight of degree l: the
    rows of a warp's unit (9, 3, 1, .. nodes), the units of a warp (296 blocks of 4 warps, shared among the degrees by
    their rows and half a row more each), the block's warps, the blocks of a join's warp and its 5 levels."""
    C, K, v = 128, (L + 1) ** 2, 1 + 2.0 ** -14 - 2.0 ** -23
    cfg = e2f.make_norm_cfg(L, C, xt, "f32", EPS)
    x = torch.ones(n, K, C, device="cuda", dtype=R.DT[xt])
    w, g = torch.ones(L + 1, C, device="cuda"), torch.full((n, K, C), v, device="cuda")
    got = e2f.e2f_layer_norm_backward(cfg, x, w, torch.zeros(n, device="cuda"), torch.ones(n, L + 1, device="cuda"), g,
                                      out={"x": g})
    for l in range(L + 1):
        rows, nodes = 2 * l + 1, (9, 3, 1, 1, 1)[l]
        blocks = int(296 * (rows + 0.5) / (K + 0.5 * (L + 1)))
        chain = nodes * rows + -(-n // (nodes * blocks * 4)) + 4 + -(-blocks // 32) + 5
        want = torch.full((C,), n * rows * v, dtype=torch.float64)
        _within(got["weight"][l], want, chain * R.U * want, f"weight {l}")
        if l == 0:
            _within(got["bias"], want, chain * R.U * want, "bias")
