"""The operators as a program uses them: species embedding, then norm -> attention -> residual sum for each
layer, with only 8-bit checkpoints kept for the backward pass, down to the gradients of the table, of the norms,
of the attention weights and of the positions."""
import numpy as np
import pytest
import torch

import atomistic_cell_list_b200 as e2f
import feature_ref as R
import workloads as W
from gpu_util import TOL, dev
from oracle.grad import layer_t
from oracle.neighbors import neighbors_bruteforce

pytestmark = pytest.mark.gpu

V, EPS, CUTOFF, N_RBF, SCALE = 5, 1e-5, 5.0, 16, 1.5
# the attention's backward against its oracle: 1e-5 fp32, 2e-3 with fp16 operands; the norm's own error and the
# statistics' add a few hundred fp32 roundings (3e-5)
GRAD_TOL = {"f32": 1e-4, "bf16": 3e-3}


class Stack:
    """Two layers with seeded weights on 24 atoms."""

    def __init__(self, dtype, L, C, H, seed=0, n=24, layers=2):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dtype, self.L, self.C, self.H, self.n, self.layers = dtype, L, C, H, n, layers
        pos = rng.uniform(0, 7.0, (n, 3))
        self.pos = torch.from_numpy(pos.astype(np.float32))
        self.rp, self.col = neighbors_bruteforce(self.pos.numpy(), None, CUTOFF)
        self.tok = torch.randint(0, V, (n,), generator=g).to(torch.int32)
        self.tok[3] = -1
        self.table = torch.randn(V, C, generator=g)
        n_so2 = sum(W.so2_block_sizes(L, C))
        s = C ** -0.5
        self.p = [dict(weight=1 + 0.1 * torch.randn(L + 1, C, generator=g), bias=0.1 * torch.randn(C, generator=g),
                       Wq=s * torch.randn(C, C, generator=g), Wk=s * torch.randn(C, C, generator=g),
                       Wrad=s * torch.randn(N_RBF, (L + 1) * C + H, generator=g),
                       Wso2=(s * torch.randn(n_so2, generator=g)).to(R.DT[dtype])) for _ in range(layers)]
        self.G = torch.randn(n, (L + 1) ** 2, C, generator=g)
        self.acfg = e2f.make_cfg(L, C, H, N_RBF, CUTOFF, dtype)
        self.ncfg = e2f.make_norm_cfg(L, C, "f32", dtype, EPS)
        self.qcfg = e2f.make_norm_cfg(L, C, "mxi8", dtype, EPS)
        self.ecfg = e2f.make_embed_cfg(V, C, L, SCALE, "f32", "f32")
        d = dev()
        self.dpos, self.drp, self.dcol = self.pos.to(d), torch.as_tensor(np.asarray(self.rp, np.int32)).to(d), \
            torch.as_tensor(np.asarray(self.col, np.int32)).to(d)
        self.dtok, self.dtable, self.dG = self.tok.to(d), self.table.to(d), self.G.to(d)
        self.dp = [{k: v.to(d) for k, v in p.items()} for p in self.p]

    def forward(self, check=True):
        """The residual stream after the last layer; per layer the stream, the features and the checkpoint."""
        h = e2f.e2f_embedding(self.ecfg, self.dtok, self.dtable, check=check)
        kept, res = [], None
        for p in self.dp:
            f = e2f.e2f_layer_norm(self.ncfg, h, p["weight"], p["bias"], residual=res, checkpoint=True)
            h = f.get("sum", h)
            res = e2f.e2f_onfly_attention(self.acfg, self.dpos, None, self.drp, self.dcol, f["y"], p["Wq"], p["Wk"],
                                          p["Wrad"], p["Wso2"], check=check)
            kept.append(dict(f, h=h, attn=res))
        return h + res, kept

    def backward(self, kept, check=True):
        """Gradients of sum(G * stream) from the checkpoints alone."""
        G, out = self.dG, []
        for p, k in zip(reversed(self.dp), reversed(kept)):
            r = e2f.e2f_layer_norm(self.qcfg, k["codes"], p["weight"], p["bias"], x_scales=k["scales"])
            a = e2f.e2f_onfly_attention_backward(self.acfg, self.dpos, None, self.drp, self.dcol, r["y"], p["Wq"],
                                                 p["Wk"], p["Wrad"], p["Wso2"], G, check=check)
            g = e2f.e2f_layer_norm_backward(self.qcfg, k["codes"], p["weight"], r["mean"], r["rstd"], a["x"],
                                            grad_skip=G, x_scales=k["scales"])
            out.append(dict(a=a, g=g, r=r, G=G))
            G = g["x"]
        table = e2f.e2f_embedding_backward(self.ecfg, self.dtok, G, check=check)
        return table, out[::-1]

    def attention64(self, p, y, pos=None):
        return layer_t(self.L, self.C, self.H, N_RBF, CUTOFF, self.pos.double() if pos is None else pos, None, self.rp,
                       self.col, y, *[p[k].double() for k in ("Wq", "Wk", "Wrad", "Wso2")])


def _near(got, want, tol, what):
    got, want = got.detach().cpu().double().reshape(want.shape), want.detach()
    err = float((got - want).abs().max() / want.abs().max())
    assert err <= tol, f"{what}: {err:.2e} > {tol:.0e}"


@pytest.mark.parametrize("dtype,L,C,H", [("f32", 2, 16, 2), ("f32", 1, 32, 4), ("bf16", 2, 64, 4), ("bf16", 3, 32, 4)])
def test_each_stage_against_64_bits(dtype, L, C, H):
    s = Stack(dtype, L, C, H)
    _, kept = s.forward()
    table, back = s.backward(kept)
    h64 = R.embedding(s.tok, s.table, SCALE, L)
    for p, k, b in zip(s.p, kept, back):
        _near(k["h"], h64, 1e-6, "stream")
        y64 = R.norm(k["h"].cpu().double(), p["weight"].double(), p["bias"].double(), L, EPS)[0]
        _near(k["y"], y64, 1e-5 if dtype == "f32" else 2 * R.HALF["bf16"], "features")
        _near(k["attn"], s.attention64(p, k["y"].cpu().double()), TOL[dtype], "attention")
        # backward of this layer, at the checkpoint, for the gradient that reached it
        q = e2f.e2f_checkpoint_load(k["codes"], k["scales"]).cpu().double().requires_grad_()
        w = p["weight"].double().requires_grad_()
        bias = p["bias"].double().requires_grad_()
        pos = s.pos.double().requires_grad_()
        pw = {n: p[n].double().requires_grad_() for n in ("Wq", "Wk", "Wrad", "Wso2")}
        y = R.norm(q, w, bias, L, EPS)[0]
        if dtype == "bf16":  # the rounding of the features passes its gradient through
            y = y + (b["r"]["y"].cpu().double() - y).detach()
        out = s.attention64(pw, y, pos) + q
        (out * b["G"].cpu().double()).sum().backward()
        tol = GRAD_TOL[dtype]
        for name, ref in (("x", q), ("weight", w), ("bias", bias)):
            _near(b["g"][name], ref.grad, tol, f"norm {name}")
        for name, ref in (("pos", pos), ("W_rad", pw["Wrad"]), ("W_so2", pw["Wso2"])):
            _near(b["a"][name], ref.grad, tol, f"attention {name}")
        h64 = k["h"].cpu().double() + k["attn"].cpu().double()
    _near(table, R.embedding_backward(s.tok, back[0]["g"]["x"].cpu(), V, SCALE)[0], 1e-5, "table")


def test_the_whole_stack_in_fp32_against_autograd():
    """Without checkpoints, the gradients of two layers against autograd through the 64-bit layers."""
    s = Stack("f32", 2, 16, 2, seed=1)
    out, kept = s.forward()
    table = s.table.double().requires_grad_()
    h = torch.cat([torch.where((s.tok >= 0)[:, None], SCALE * table[s.tok.clamp(min=0).long()], 0.0)[:, None],
                   torch.zeros(s.n, (s.L + 1) ** 2 - 1, s.C, dtype=torch.float64)], 1)
    for p in s.p:
        h = h + s.attention64(p, R.norm(h, p["weight"].double(), p["bias"].double(), s.L, EPS)[0])
    _near(out, h, TOL["f32"], "output")
    (h * s.G.double()).sum().backward()
    G = s.dG
    for p, k in zip(reversed(s.dp), reversed(kept)):
        a = e2f.e2f_onfly_attention_backward(s.acfg, s.dpos, None, s.drp, s.dcol, k["y"], p["Wq"], p["Wk"], p["Wrad"],
                                             p["Wso2"], G)
        G = e2f.e2f_layer_norm_backward(s.ncfg, k["h"], p["weight"], k["mean"], k["rstd"], a["x"], grad_skip=G)["x"]
    _near(e2f.e2f_embedding_backward(s.ecfg, s.dtok, G), table.grad, 2 * GRAD_TOL["f32"], "table")


def test_forward_captured_and_replayed():
    s = Stack("bf16", 2, 64, 4)
    s.forward(check=False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held, kept = s.forward(check=False)
    s.dtok.copy_(torch.flip(s.dtok, [0]))
    s.dpos.add_(1.0)  # a translation keeps the list
    graph.replay()
    torch.cuda.synchronize()
    now, kept2 = s.forward(check=False)
    # the attention sums in a fixed order: the same bits
    assert torch.equal(held, now) and all(torch.equal(a["codes"], b["codes"]) for a, b in zip(kept, kept2))


def test_offsets_beyond_32_bits():
    """700,000 atoms at L = 4, C = 128: 2.24 G values. The last atoms come out as they do alone."""
    n, L, C, V = 700_000, 4, 128, 7
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(n, 25, C, dtype=torch.bfloat16, device=dev()).normal_(generator=gen)
    gy = torch.zeros(n, 25, C, device=dev())
    gy[-40:].normal_(generator=gen)
    w, b = torch.randn(L + 1, C, device=dev()), torch.randn(C, device=dev())
    cfg = e2f.make_norm_cfg(L, C, "bf16", "bf16", EPS)
    big = e2f.e2f_layer_norm(cfg, x, w, b, checkpoint=True)
    end = x[-40:].contiguous()
    small = e2f.e2f_layer_norm(cfg, end, w, b, checkpoint=True)
    for k in small:
        assert torch.equal(big[k][-40:], small[k]), k
    g = e2f.e2f_layer_norm_backward(cfg, x, w, big["mean"], big["rstd"], gy)
    gs = e2f.e2f_layer_norm_backward(cfg, end, w, small["mean"], small["rstd"], gy[-40:].contiguous())
    assert torch.equal(g["x"][-40:], gs["x"]) and (g["x"][:-40] == 0).all()
    # the weight sums differ in their order only: 40 nodes' rows, the rest adds zeros
    xh = R.norm(end.cpu().double(), torch.ones(L + 1, C, dtype=torch.float64), None, L, EPS)[0]
    for l, rows in enumerate(R.degrees(L)):
        mag = (gy[-40:, rows].cpu().double() * xh[:, rows]).abs().sum((0, 1))
        assert ((g["weight"][l] - gs["weight"][l]).cpu().double().abs() <= 2 * 1024 * R.U * mag).all()
    del g, big
    codes, scales = e2f.e2f_checkpoint_store(x)
    assert torch.equal(codes[-40:], small["codes"]) and torch.equal(scales[-40:], small["scales"])
    back = e2f.e2f_checkpoint_load(codes, scales, "bf16")
    assert torch.equal(back[-40:], e2f.e2f_checkpoint_load(small["codes"], small["scales"], "bf16"))
    del codes, scales, back, x
    tok = torch.randint(0, V, (n,), dtype=torch.int32, device=dev(), generator=gen)
    for rows in (V, 1000):  # both ways of sorting
        ecfg = e2f.make_embed_cfg(rows, C, L, 1.0, "f32", "bf16")
        grad = e2f.e2f_embedding_backward(ecfg, tok, gy)
        want, mag = R.embedding_backward(tok[-40:].cpu(), gy[-40:].cpu(), rows, 1.0)
        assert ((grad.cpu().double() - want).abs() <= 1024 * R.U * mag).all()
        table = torch.randn(rows, C, device=dev())
        out = e2f.e2f_embedding(ecfg, tok, table)
        assert torch.equal(out[-40:], e2f.e2f_embedding(ecfg, tok[-40:].contiguous(), table))
        del out
