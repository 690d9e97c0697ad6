"""e2f_embedding and e2f_embedding_backward against the plain 64-bit implementation: token distributions from
one species to many rare ones, padding, tokens beyond the table, odd widths."""
import pytest
import torch

import atomistic_cell_list_b200 as e2f
import feature_ref as R

pytestmark = pytest.mark.gpu


def _tokens(n, V, kind, seed=0, pad=0.1):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        t = torch.full((n,), V - 1)
    elif kind == "two":
        t = torch.where(torch.rand(n, generator=g) < 0.7, 0, V - 1)
    elif kind == "sorted":
        t = torch.sort(torch.randint(0, V, (n,), generator=g))[0]
    elif kind == "skewed":
        t = (V ** torch.rand(n, generator=g, dtype=torch.float64)).long().clamp(max=V) - 1
    else:
        t = torch.randint(0, V, (n,), generator=g)
    t[torch.rand(n, generator=g) < pad] = -1
    return t.to(torch.int32)


@pytest.mark.parametrize("tt,yt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("n,V,L,C", [(1, 1, 0, 1), (64, 100, 2, 16), (33, 10, 4, 128), (1000, 5, 0, 33), (17, 50000, 1, 512),
                                     (5, 3, 0, 5001)])
def test_lookup(n, V, L, C, tt, yt):
    tok = _tokens(n, V, "uniform")
    table = torch.randn(V, C, generator=torch.Generator().manual_seed(1)).to(R.DT[tt])
    scale = 2.3
    out = e2f.e2f_embedding(e2f.make_embed_cfg(V, C, L, scale, tt, yt), tok.cuda(), table.cuda())
    want = R.embedding(tok, table, scale, L)
    # the scale's and the product's rounding, then the output's
    bound = want.abs() * (2 * R.U + R.HALF[yt] * (1 + 2 ** -7))
    assert ((out.cpu().double() - want).abs() <= bound).all()


# longest chain of additions behind one table row: 64 of a chunk, then at most 32 of a join's warp, then 32 warps
CHAIN = 160


@pytest.mark.parametrize("kind", ["uniform", "one", "two", "sorted", "skewed"])
@pytest.mark.parametrize("n,V,L,C", [(1, 1, 0, 1), (2, 300, 1, 16), (64, 100, 2, 16), (63, 7, 0, 4), (65, 255, 0, 20),
                                     (1000, 256, 4, 128), (1025, 257, 0, 33), (5000, 100, 1, 64), (20000, 9, 0, 128),
                                     (3000, 70000, 0, 8), (4097, 3, 0, 257), (300, 16777300, 0, 1), (50, 5, 0, 5001),
                                     (700, 2, 0, 16384), (60000, 90, 0, 5)])
def test_gradient(n, V, L, C, kind):
    tok = _tokens(n, V, kind, seed=n)
    g = torch.randn(n, (L + 1) ** 2, C, generator=torch.Generator().manual_seed(2))
    cfg = e2f.make_embed_cfg(V, C, L, 0.7)
    got = e2f.e2f_embedding_backward(cfg, tok.cuda(), g.cuda(), out=torch.full((V, C), 77.0, device="cuda"))
    want, mag = R.embedding_backward(tok, g, V, 0.7)
    assert ((got.cpu().double() - want).abs() <= (CHAIN + 4) * R.U * mag).all()
    assert torch.equal(got, e2f.e2f_embedding_backward(cfg, tok.cuda(), g.cuda()))  # bit for bit


def test_gradient_against_differences():
    """Linear in the table: a unit step of one entry changes the loss by its gradient, but for rounding."""
    n, V, L, C = 200, 6, 1, 24
    tok = _tokens(n, V, "uniform")
    g = torch.randn(n, 4, C, dtype=torch.float32)
    cfg = e2f.make_embed_cfg(V, C, L, 1.25)
    grad = e2f.e2f_embedding_backward(cfg, tok.cuda(), g.cuda()).cpu().double()
    table = torch.randn(V, C, dtype=torch.float64)
    for v, c in ((0, 0), (5, 23), (2, 7)):
        step = torch.zeros(V, C, dtype=torch.float64)
        step[v, c] = 0.5
        at = lambda t: (R.embedding(tok, t, 1.25, L) * g.double()).sum()
        mag = 1.25 * g[tok == v, 0, c].abs().sum().double()
        assert abs((at(table + step) - at(table - step)) - grad[v, c]) <= (CHAIN + 4) * R.U * mag + 1e-9


def test_nothing_but_padding_and_no_atoms():
    cfg = e2f.make_embed_cfg(5, 16, 1)
    tok = torch.full((70,), -3, dtype=torch.int32, device="cuda")
    assert (e2f.e2f_embedding(cfg, tok, torch.ones(5, 16, device="cuda")) == 0).all()
    for n in (70, 0):
        out = torch.full((5, 16), 77.0, device="cuda")
        e2f.e2f_embedding_backward(cfg, tok[:n], torch.ones(n, 4, 16, device="cuda"), out=out)
        assert (out == 0).all()
    assert e2f.e2f_embedding(cfg, tok[:0], torch.ones(5, 16, device="cuda")).shape == (0, 4, 16)


def test_non_finite_gradients_reach_their_token_only():
    tok = _tokens(500, 4, "uniform", pad=0.2)
    g = torch.randn(500, 1, 16)
    i = int((tok == 2).nonzero()[3])
    g[i, 0, 5] = float("nan")
    g[(tok == -1).nonzero()[0], 0] = float("inf")  # padding is not read into any sum
    got = e2f.e2f_embedding_backward(e2f.make_embed_cfg(4, 16), tok.cuda(), g.cuda()).cpu()
    want = torch.zeros(4, 16, dtype=torch.bool)
    want[2, 5] = True
    assert torch.equal(~torch.isfinite(got), want)


def test_tokens_beyond_the_table_are_reported():
    cfg = e2f.make_embed_cfg(5, 16)
    tok = torch.tensor([0, 5, 4, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    table, g = torch.ones(5, 16, device="cuda"), torch.ones(5, 1, 16, device="cuda")
    for call in (lambda **k: e2f.e2f_embedding(cfg, tok, table, **k),
                 lambda **k: e2f.e2f_embedding_backward(cfg, tok, g, **k)):
        with pytest.raises(e2f.E2FError) as e:
            call()
        assert e.value.code == 1
    out = e2f.e2f_embedding(cfg, tok, table, check=False)
    assert out[:, 0, 0].tolist() == [1, 0, 1, 0, 0]
    grad = e2f.e2f_embedding_backward(cfg, tok, g, check=False)
    assert grad[:, 0].tolist() == [1, 0, 0, 0, 1]
    ok = tok[:1]
    assert e2f.e2f_embedding(cfg, ok, table)[0, 0, 0] == 1  # the next call starts clean
    e2f.e2f_embedding_backward(cfg, ok, g[:1])


@pytest.mark.parametrize("n,V", [(300, 5), (30000, 5), (30000, 256), (300, 3000), (30000, 3000), (30000, 70000)])
def test_one_token_beyond_the_table_among_many(n, V):
    """Found wherever it lies, in one tile or many, and gone from the status in the next call."""
    tok = _tokens(n, V, "uniform").cuda()
    g = torch.randn(n, 1, 8, device="cuda")
    cfg = e2f.make_embed_cfg(V, 8)
    ws = torch.empty(e2f.e2f_embedding_backward_workspace_size(n, cfg), dtype=torch.uint8, device="cuda")
    bad = tok.clone()
    bad[2 * n // 3] = V
    tok[2 * n // 3] = -1
    want = e2f.e2f_embedding_backward(cfg, tok, g, workspace=ws)
    with pytest.raises(e2f.E2FError) as e:
        e2f.e2f_embedding_backward(cfg, bad, g, workspace=ws)
    assert e.value.code == 1
    assert torch.equal(e2f.e2f_embedding_backward(cfg, bad, g, workspace=ws, check=False), want)
    assert torch.equal(e2f.e2f_embedding_backward(cfg, tok, g, workspace=ws), want)


@pytest.mark.parametrize("V", [90, 3000])
def test_streams_capture_and_rows_behind(V):
    n, C = 3000, 64
    tok, g = _tokens(n, V, "skewed").cuda(), torch.randn(n, 4, C, device="cuda")
    table = torch.randn(V, C, device="cuda")
    cfg = e2f.make_embed_cfg(V, C, 1, 1.0)
    ws = torch.empty(e2f.e2f_embedding_backward_workspace_size(n, cfg), dtype=torch.uint8, device="cuda")

    def step():
        return (e2f.e2f_embedding(cfg, tok, table, check=False),
                e2f.e2f_embedding_backward(cfg, tok, g, workspace=ws, check=False))

    ref = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = e2f.e2f_embedding(cfg, tok, table, stream=s, check=False)
    grad = e2f.e2f_embedding_backward(cfg, tok, g, stream=s, check=False)
    s.synchronize()
    assert torch.equal(out, ref[0]) and torch.equal(grad, ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    tok.copy_(_tokens(n, V, "two", seed=3))
    graph.replay()
    torch.cuda.synchronize()
    now = step()
    assert torch.equal(held[0], now[0]) and torch.equal(held[1], now[1])
    big, tall = torch.full((n + 2, 4, C), 77.0, device="cuda"), torch.full((V + 2, C), 77.0, device="cuda")
    e2f.e2f_embedding(cfg, tok, table, out=big[:n])
    e2f.e2f_embedding_backward(cfg, tok, g, out=tall[:V])
    assert (big[n:] == 77).all() and (tall[V:] == 77).all() and torch.equal(tall[:V], now[1])
    with pytest.raises(ValueError):
        e2f.e2f_embedding_backward(cfg, tok, g[:, :1])


@pytest.mark.parametrize("V,C", [(1229, 20), (6145, 4), (8193, 3), (4337, 17), (69121, 8), (70042, 20)])
def test_rows_without_tokens_are_zero_to_the_end_of_the_table(V, C):
    """Tables of which the zeroing kernels' equal shares leave a remainder; the tokens are all below V/2, so that
    nothing but the zeroing writes the last rows."""
    n = 300
    tok = _tokens(n, V // 2, "uniform", seed=V)
    g = torch.randn(n, 1, C, generator=torch.Generator().manual_seed(3))
    got = e2f.e2f_embedding_backward(e2f.make_embed_cfg(V, C, 0, 0.7), tok.cuda(), g.cuda(),
                                     out=torch.full((V, C), 77.0, device="cuda"))
    want, mag = R.embedding_backward(tok, g, V, 0.7)
    assert (got[V // 2:] == 0).all()
    assert ((got.cpu().double() - want).abs() <= (CHAIN + 4) * R.U * mag).all()


@pytest.mark.parametrize("V", [100, 300])
def test_a_small_batch_in_the_workspace_of_a_large_one(V):
    """The status word of every call lies in the caller's workspace, whichever batch it was made for."""
    C, most = 128, 19000
    cfg = e2f.make_embed_cfg(V, C)
    ws = torch.empty(e2f.e2f_embedding_backward_workspace_size(most, cfg), dtype=torch.uint8, device="cuda")
    for n in (18945, 18944, 513, 512, 1):
        tok, g = _tokens(n, V, "uniform", seed=n, pad=0.0), torch.randn(n, 1, C)
        tok[n // 2] = V
        ws[:4] = 77
        got = e2f.e2f_embedding_backward(cfg, tok.cuda(), g.cuda(), workspace=ws, check=False)
        assert e2f.lib().e2f_attention_status(ws.data_ptr(), ws.numel(), None) == 1
        want, mag = R.embedding_backward(tok, g, V, 1.0)
        assert ((got.cpu().double() - want).abs() <= (CHAIN + 4) * R.U * mag).all()


# the same for batches whose tiles grow to 2,048 tokens: tile/teams rows of a team, the first and last runs of the
# tile's teams, the tiles of a join's warp, 16 warps. C = 128: 256 + 2 x 8 + 19 + 16; C = 16: 32 + 2 x 64 + 19 + 16
LONG_CHAIN = 310


@pytest.mark.parametrize("kind", ["uniform", "two", "skewed"])
@pytest.mark.parametrize("n,V,C", [(100000, 100, 128), (300000, 300, 128), (620000, 7, 128), (620000, 5000, 128),
                                   (610000, 3, 16), (30000, 256, 1024)])
def test_gradient_of_long_tiles(n, V, C, kind):
    tok = _tokens(n, V, kind, seed=n)
    g = torch.randn(n, 1, C, generator=torch.Generator().manual_seed(4))
    cfg = e2f.make_embed_cfg(V, C, 0, 0.7)
    got = e2f.e2f_embedding_backward(cfg, tok.cuda(), g.cuda(), out=torch.full((V, C), 77.0, device="cuda"))
    want, mag = R.embedding_backward(tok, g, V, 0.7)
    assert ((got.cpu().double() - want).abs() <= (LONG_CHAIN + 4) * R.U * mag).all()
