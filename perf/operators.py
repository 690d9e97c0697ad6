"""Measured cases of the operators around the attention layer: layer norm of irreducible features, the
species embedding, and 8-bit activation checkpoints, each with its backward pass.

`run` computes a case in plain torch operations, or, with `own`, through the library's entry points.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-5


def listed():
    return [
        # one norm of a 64-atom cluster in fp32: the smallest system, launch latency only
        {"name": "norm tiny", "kind": "norm", "n": 64, "L": 2, "C": 16, "x": "f32", "y": "f32", "res": False},
        # between two attention layers on a 3,000-atom water box: the fp32 attention output joins the residual
        # stream, the bf16 features of the next layer come out
        {"name": "norm water 3k", "kind": "norm", "n": 3000, "L": 4, "C": 128, "x": "f32", "y": "bf16", "res": True},
        # plain layer norm of long odd rows (a feed-forward width that no vector load divides)
        {"name": "norm rows odd", "kind": "norm", "n": 4099, "L": 0, "C": 5001, "x": "bf16", "y": "bf16", "res": False},
        # the gradient of one norm on the 30,000-atom box, with the residual stream's gradient joined
        {"name": "norm bwd 30k", "kind": "norm_bwd", "n": 30000, "L": 4, "C": 128, "x": "f32", "skip": True},
        # the gradient of one norm on a batch of 256 molecules with bf16 features
        {"name": "norm bwd molecules", "kind": "norm_bwd", "n": 10027, "L": 4, "C": 64, "x": "bf16", "skip": False},
        # a whole norm under checkpointing on a 100,000-atom box: forward with the residual and the 8-bit
        # checkpoint, then from the checkpoint the recomputed features and the gradients
        {"name": "step 100k", "kind": "step", "n": 100000, "L": 4, "C": 128, "x": "f32", "y": "bf16"},
        # the same on the 3,000-atom box with a bf16 residual stream
        {"name": "step 3k", "kind": "step", "n": 3000, "L": 4, "C": 128, "x": "bf16", "y": "bf16"},
        # features of the 30,000-atom box put away in 8 bits and fetched again
        {"name": "checkpoint 30k", "kind": "checkpoint", "n": 30000, "L": 4, "C": 128, "x": "bf16"},
        # species of a 100,000-atom box to the first layer's features
        {"name": "embed 100k", "kind": "embed", "n": 100000, "L": 4, "C": 128, "V": 100, "table": "f32", "y": "bf16",
         "tokens": "water", "pad": 0.0},
        # the embedding's gradient of a 64-atom cluster: launch latency only
        {"name": "embed bwd tiny", "kind": "embed_bwd", "n": 64, "L": 2, "C": 16, "V": 100, "tokens": "uniform",
         "pad": 0.0},
        # water: two species over 100,000 atoms, two long segments of sorted tokens
        {"name": "embed bwd water", "kind": "embed_bwd", "n": 100000, "L": 4, "C": 128, "V": 100, "tokens": "water",
         "pad": 0.0},
        # a large vocabulary with few frequent and many rare tokens, and a padded batch
        {"name": "embed bwd zipf", "kind": "embed_bwd", "n": 65536, "L": 0, "C": 512, "V": 32003, "tokens": "zipf",
         "pad": 0.05},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm_bwd", "step", "checkpoint", "embed", "embed_bwd"])
    L = rng.choice([0, 0, 1, 2, 3, 4, 4])
    K = (L + 1) ** 2
    if L:
        C = rng.choice([16 * rng.randint(1, 16), 16 * rng.randint(1, 16), rng.randint(16, 256)])
    else:
        C = _log(rng, 16, 8192)
        C = rng.choice([C, (C + 15) // 16 * 16])
    n = _log(rng, 1, max(2, min(100000, 160_000_000 // (K * C))))
    case = {"kind": kind, "n": n, "L": L, "C": C}
    if kind in ("norm", "norm_bwd", "step", "checkpoint"):
        case["x"] = rng.choice(["f32", "bf16"])
    if kind in ("norm", "step"):
        case["y"] = rng.choice(["f32", "bf16"])
    if kind == "norm":
        case["res"] = rng.random() < 0.5
    if kind == "norm_bwd":
        case["skip"] = rng.random() < 0.5
    if kind in ("embed", "embed_bwd"):
        case["V"] = _log(rng, 2, max(4, min(262144, 64_000_000 // C)))
        case["tokens"] = rng.choice(["water", "uniform", "zipf"])
        case["pad"] = rng.choice([0.0, 0.1])
    if kind == "embed":
        case["table"] = rng.choice(["f32", "bf16"])
        case["y"] = rng.choice(["f32", "bf16"])
    return case


def _tokens(case, gen):
    """Species or vocabulary indices; a share `pad` of them is -1 (padding)."""
    n, V, dev = case["n"], case["V"], "cuda"
    u = torch.rand(n, generator=gen, device=dev, dtype=torch.float64)
    if case["tokens"] == "water":  # two species of the table, two thirds and one third of the atoms
        t = torch.where(u < 2.0 / 3.0, min(1, V - 1), min(8, V - 1)).to(torch.int32)
    elif case["tokens"] == "zipf":  # frequency about 1 / rank
        t = (torch.exp(u * math.log(V + 1.0)) - 1.0).to(torch.int32).clamp_(0, V - 1)
    else:
        t = (u * V).to(torch.int32).clamp_(0, V - 1)
    if case["pad"]:
        t[torch.rand(n, generator=gen, device=dev) < case["pad"]] = -1
    return t


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    n, L, C = case["n"], case["L"], case["C"]
    K = (L + 1) ** 2

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale)

    s = {"case": case}
    if case["kind"] in ("norm", "norm_bwd", "step", "checkpoint"):
        # a residual stream: atoms of differing magnitude, a channel mean on the invariants
        x = randn(n, K, C)
        x[:, 0] += 0.5
        x *= torch.exp(randn(n, 1, 1, scale=0.5))
        s["x"] = x.to(DT[case["x"]])
        s["weight"] = 1.0 + randn(L + 1, C, scale=0.1)
        s["bias"] = randn(C, scale=0.1)
    if case["kind"] == "step" or case.get("res"):
        s["residual"] = randn(n, K, C, scale=0.3)
    if case["kind"] in ("norm_bwd", "step"):
        s["grad_y"] = randn(n, K, C, scale=1e-2)
    if case["kind"] == "step" or case.get("skip"):
        s["grad_skip"] = randn(n, K, C, scale=1e-2)
    if case["kind"] == "norm_bwd":  # the statistics that the forward call left
        s["mean"], s["rstd"] = (t.float() for t in _stats64(s["x"], L))
    if case["kind"] in ("embed", "embed_bwd"):
        s["tokens"] = _tokens(case, gen)
    if case["kind"] == "embed":
        s["table"] = randn(case["V"], C).to(DT[case["table"]])
    if case["kind"] == "embed_bwd":
        s["grad_out"] = randn(n, K, C, scale=1e-2)
    return s


def work(case):
    n, L, C = case["n"], case["L"], case["C"]
    K = (L + 1) ** 2
    e, kind, x, y = n * K * C, case["kind"], SIZE.get(case.get("x"), 0), SIZE.get(case.get("y"), 0)
    code = n * K * (C + (C + 31) // 32)
    stats, par = 4 * n * (L + 2), 4 * C * (L + 2)
    if kind == "norm":
        return {"bytes": e * (x + y + (4 + x if case["res"] else 0)) + stats + par, "flops": 8 * e}
    if kind == "norm_bwd":
        return {"bytes": e * (x + 8 + (4 if case["skip"] else 0)) + stats + 2 * par, "flops": 14 * e}
    if kind == "step":  # forward: x, residual, sum, y, checkpoint; then checkpoint, y; then checkpoint, 3 gradients
        return {"bytes": e * (2 * x + 4 + 2 * y + 12) + 3 * code + stats + 4 * par, "flops": 40 * e}
    if kind == "checkpoint":
        return {"bytes": 2 * e * x + 2 * code, "flops": 6 * e}
    V = case["V"]
    if kind == "embed":
        rows = min(V, n, 2 if case["tokens"] == "water" else V)
        return {"bytes": 4 * n + rows * C * SIZE[case["table"]] + e * y, "flops": n * C}
    return {"bytes": 4 * n + 4 * n * C + 4 * V * C, "flops": n * C + V * C}


# ---- the plain form ------------------------------------------------------------------------------------------


def _members(L, device):
    """[K, L+1]: 1 where row k belongs to degree l; and the degree of each row."""
    deg = torch.arange((L + 1) ** 2, device=device).sqrt().floor().long()
    return (deg[:, None] == torch.arange(L + 1, device=device)).float(), deg


def _norm(h, weight, bias, L):
    """y, mean, rstd and the normalised features of fp32 h [n, K, C]."""
    onehot, deg = _members(L, h.device)
    first = (torch.arange(h.shape[1], device=h.device) == 0).float()[:, None]
    mean = h[:, 0].mean(-1)
    d = h - mean[:, None, None] * first
    per_row = (d * d).sum(-1)
    rstd = 1.0 / torch.sqrt(per_row @ onehot / (onehot.sum(0) * h.shape[2]) + EPS)
    xh = d * rstd[:, deg, None]
    return xh * weight[deg] + bias * first, mean, rstd, xh


def _norm_bwd(h, weight, mean, rstd, gy, skip, L):
    onehot, deg = _members(L, h.device)
    first = (torch.arange(h.shape[1], device=h.device) == 0).float()[:, None]
    xh = (h - mean[:, None, None] * first) * rstd[:, deg, None]
    u = gy * weight[deg]
    dot = ((u * xh).sum(-1) @ onehot / (onehot.sum(0) * h.shape[2]))[:, deg, None]
    dx = (u - xh * dot - u[:, :1].mean(-1, keepdim=True) * first) * rstd[:, deg, None]
    if skip is not None:
        dx = dx + skip
    dw = onehot.t().double() @ (gy * xh).sum(0, dtype=torch.float64)
    return {"x": dx, "weight": dw.float(), "bias": gy[:, 0].sum(0, dtype=torch.float64).float()}


def _pow2(e):
    """2^e in fp32 for integers -126 <= e <= 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _coded(x):
    """What an 8-bit checkpoint of x stands for: blocks of 32 channels share a power of two, codes are whole numbers."""
    n, K, C = x.shape
    b = torch.zeros(n, K, (C + 31) // 32 * 32, device=x.device)
    b[..., :C] = x.float()
    b = b.view(n, K, -1, 32)
    e = (torch.frexp(b.abs().amax(-1, keepdim=True))[1] - 1).clamp(min=-120)
    v = torch.round(b * _pow2(6 - e)).clamp(-127, 127) * _pow2(e - 6)
    return v.view(n, K, -1)[..., :C].contiguous()


def _plain(s):
    case = s["case"]
    L, kind = case["L"], case["kind"]
    if kind == "norm":
        h = s["x"].float()
        out = {}
        if case["res"]:
            out["sum"] = (h + s["residual"]).to(s["x"].dtype)
            h = out["sum"].float()
        y, out["mean"], out["rstd"], _ = _norm(h, s["weight"], s["bias"], L)
        return {"y": y.to(DT[case["y"]]), **out}
    if kind == "norm_bwd":
        return _norm_bwd(s["x"].float(), s["weight"], s["mean"], s["rstd"], s["grad_y"], s.get("grad_skip"), L)
    if kind == "step":
        h = (s["x"].float() + s["residual"]).to(s["x"].dtype)
        y = _norm(h.float(), s["weight"], s["bias"], L)[0].to(DT[case["y"]])
        q = _coded(h)
        again, mean, rstd, _ = _norm(q, s["weight"], s["bias"], L)
        g = _norm_bwd(q, s["weight"], mean, rstd, s["grad_y"], s["grad_skip"], L)
        return {"sum": h, "y": y, "again": again.to(DT[case["y"]]), **g}
    if kind == "checkpoint":
        return _coded(s["x"]).to(s["x"].dtype)
    t = s["tokens"].long()
    ok = t >= 0
    if kind == "embed":
        out = torch.zeros(case["n"], (L + 1) ** 2, case["C"], dtype=DT[case["y"]], device=t.device)
        row = math.sqrt(case["C"]) * s["table"][t.clamp(min=0)].float()
        out[:, 0] = torch.where(ok[:, None], row, 0.0).to(out.dtype)
        return out
    g = torch.zeros(case["V"], case["C"], dtype=torch.float64, device=t.device)
    g.index_add_(0, t[ok], s["grad_out"][:, 0][ok].double())
    return (math.sqrt(case["C"]) * g).float()


# ---- the library's entry points ------------------------------------------------------------------------------


def _plan(s):
    """The descriptors and the workspace that a program keeps between calls."""
    import atomistic_cell_list_b200 as e2f

    case = s["case"]
    L, C, kind = case["L"], case["C"], case["kind"]
    p = {"lib": e2f}
    if kind in ("norm", "norm_bwd", "step"):
        p["cfg"] = e2f.make_norm_cfg(L, C, case["x"], case.get("y", "f32"), EPS)
        p["cfg8"] = e2f.make_norm_cfg(L, C, "mxi8", case.get("y", "f32"), EPS)
        ws = e2f.e2f_layer_norm_backward_workspace_size(case["n"], p["cfg"])
    elif kind in ("embed", "embed_bwd"):
        p["cfg"] = e2f.make_embed_cfg(case["V"], C, L, math.sqrt(C), case.get("table", "f32"), case.get("y", "f32"))
        ws = e2f.e2f_embedding_backward_workspace_size(case["n"], p["cfg"])
    else:
        ws = 0
    p["ws"] = torch.empty(max(ws, 256), dtype=torch.uint8, device="cuda")
    return p


def _own(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    case, p = s["case"], s["plan"]
    e2f, kind = p["lib"], case["kind"]
    if kind == "norm":
        return e2f.e2f_layer_norm(p["cfg"], s["x"], s["weight"], s["bias"], residual=s.get("residual"))
    if kind == "norm_bwd":
        return e2f.e2f_layer_norm_backward(p["cfg"], s["x"], s["weight"], s["mean"], s["rstd"], s["grad_y"],
                                           grad_skip=s.get("grad_skip"), workspace=p["ws"])
    if kind == "step":
        f = e2f.e2f_layer_norm(p["cfg"], s["x"], s["weight"], s["bias"], residual=s["residual"], checkpoint=True,
                               stats=False)
        r = e2f.e2f_layer_norm(p["cfg8"], f["codes"], s["weight"], s["bias"], x_scales=f["scales"])
        g = e2f.e2f_layer_norm_backward(p["cfg8"], f["codes"], s["weight"], r["mean"], r["rstd"], s["grad_y"],
                                        grad_skip=s["grad_skip"], x_scales=f["scales"], workspace=p["ws"])
        return {"sum": f["sum"], "y": f["y"], "again": r["y"], **g}
    if kind == "checkpoint":
        codes, scales = e2f.e2f_checkpoint_store(s["x"])
        return e2f.e2f_checkpoint_load(codes, scales, dtype=case["x"])
    if kind == "embed":
        return e2f.e2f_embedding(p["cfg"], s["tokens"], s["table"], check=False)
    return e2f.e2f_embedding_backward(p["cfg"], s["tokens"], s["grad_out"], workspace=p["ws"], check=False)


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits -------------------------------------------------------------------------------


def _stats64(x, L):
    """mean [n] and 1/sqrt(mean square + eps) [n, L+1], degree by degree."""
    mean = x[:, 0].double().mean(1)
    cols = []
    for l in range(L + 1):
        part = x[:, l * l:(l + 1) ** 2].double()
        if l == 0:
            part = part - mean[:, None, None]
        cols.append((part.pow(2).mean((1, 2)) + EPS).rsqrt())
    return mean, torch.stack(cols, 1)


def _forward64(h, s, L):
    mean, rstd = _stats64(h, L)
    y = torch.empty(h.shape, dtype=torch.float64, device=h.device)
    for l in range(L + 1):
        rows = slice(l * l, (l + 1) ** 2)
        d = h[:, rows].double() - (mean[:, None, None] if l == 0 else 0.0)
        y[:, rows] = d * rstd[:, l, None, None] * s["weight"][l].double() + (s["bias"].double() if l == 0 else 0.0)
    return y, mean, rstd


def _backward64(h, s, mean, rstd, L):
    dx = torch.empty(h.shape, dtype=torch.float64, device=h.device)
    dw = []
    for l in range(L + 1):
        rows = slice(l * l, (l + 1) ** 2)
        r = rstd[:, l, None, None].double()
        xh = (h[:, rows].double() - (mean[:, None, None].double() if l == 0 else 0.0)) * r
        g = s["grad_y"][:, rows].double()
        dw.append((g * xh).sum((0, 1)))
        u = g * s["weight"][l].double()
        proj = u - xh * (u * xh).mean((1, 2), keepdim=True)
        if l == 0:
            proj = proj - u.mean((1, 2), keepdim=True)
        dx[:, rows] = r * proj
    if "grad_skip" in s:
        dx += s["grad_skip"]
    return {"x": dx, "weight": torch.stack(dw), "bias": s["grad_y"][:, 0].double().sum(0)}


def _coded64(x):
    """The checkpoint's values, block by block of 32 channels."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c in range(0, x.shape[2], 32):
        b = x[..., c:c + 32].double()
        top = b.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -120)
        e = torch.round(torch.log2(top))  # then down to the power of two at or below the largest magnitude
        unit = torch.exp2(torch.where(torch.exp2(e) > top, e - 1.0, e) - 6.0)
        out[..., c:c + 32] = torch.round(b / unit).clamp(-127.0, 127.0) * unit
    return out


def exact(case, seed):
    s = prepare(case, seed)
    L, kind = case["L"], case["kind"]
    h = s.get("x")
    if "residual" in s:  # the sum is formed in fp32 and stored in x's type
        h = (h.float() + s["residual"]).to(h.dtype)
    if kind == "norm":
        y, mean, rstd = _forward64(h, s, L)
        return {"y": y, "mean": mean, "rstd": rstd, **({"sum": h.double()} if case["res"] else {})}
    if kind == "norm_bwd":
        return _backward64(h, s, s["mean"], s["rstd"], L)
    if kind == "step":
        y = _forward64(h, s, L)[0]
        q = _coded64(h)
        again, mean, rstd = _forward64(q, s, L)
        return {"sum": h, "y": y, "again": again, **_backward64(q, s, mean, rstd, L)}
    if kind == "checkpoint":
        return _coded64(h)
    t = s["tokens"].long()
    scale = math.sqrt(case["C"])
    if kind == "embed":
        out = torch.zeros(case["n"], (L + 1) ** 2, case["C"], dtype=torch.float64, device=t.device)
        at = torch.nonzero(t >= 0)[:, 0]
        out[at, 0] = scale * s["table"].double()[t[at]]
        return out
    # every token's sum as the difference of two running sums over the sorted tokens
    at = torch.argsort(t, stable=True)
    run_sum = torch.zeros(case["n"] + 1, case["C"], dtype=torch.float64, device=t.device)
    run_sum[1:] = torch.cumsum(s["grad_out"][at, 0].double(), 0)
    edge = torch.searchsorted(t[at].contiguous(), torch.arange(case["V"] + 1, device=t.device))
    return scale * (run_sum[edge[1:]] - run_sum[edge[:-1]])
