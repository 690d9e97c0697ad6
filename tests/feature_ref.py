"""Plain 64-bit implementations of the operators around the attention layer (norm of irreducible features,
8-bit checkpoint, species embedding), and rounding bounds of an fp32 evaluation of them. Torch double on the
CPU, differentiable where a gradient is tested."""
import torch

U = 2.0 ** -24   # half a step of fp32
HALF = {"f32": U, "bf16": 2.0 ** -8}
# longest chain of fp32 additions behind one sum of a (node, degree) group, at the tested sizes: at most 96
# values added by one thread, then at most 12 tree levels
CHAIN = 128
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def degrees(L):
    return [slice(l * l, (l + 1) ** 2) for l in range(L + 1)]


def norm(h, weight, bias, L, eps):
    """y, mean [N], rstd [N, L+1] of h [N, K, C]."""
    parts, rstd = [], []
    mean = h[:, 0].mean(-1)
    for l, rows in enumerate(degrees(L)):
        d = h[:, rows] - (mean[:, None, None] if l == 0 else 0.0)
        r = 1.0 / torch.sqrt((d * d).mean((1, 2)) + eps)
        y = d * r[:, None, None] * weight[l]
        parts.append(y + bias if l == 0 and bias is not None else y)
        rstd.append(r)
    return torch.cat(parts, 1), mean, torch.stack(rstd, 1)


def norm_bound(h, weight, bias, L, eps, y_dtype):
    """(bound on y, bound on mean, relative bound on rstd [N, L+1]) of an fp32 evaluation.

    mean: a sum in chains of at most CHAIN additions, off by e = CHAIN U mean|h|. d = h - mean is off by e + U |d|.
    The mean square is off by CHAIN U (its sum) + 2 U (d's own rounding) + 2 e mean|d| + e^2, relative to
    mean square + eps; rstd by half of that plus 3 U (sum, root, division). y adds three roundings and the bias."""
    mean = h[:, 0].mean(-1)
    e = CHAIN * U * h[:, 0].abs().mean(-1)
    parts, rel = [], []
    for l, rows in enumerate(degrees(L)):
        em = e if l == 0 else torch.zeros_like(e)
        d = h[:, rows] - (mean[:, None, None] if l == 0 else 0.0)
        ms = (d * d).mean((1, 2)) + eps
        rr = 0.5 * ((CHAIN + 4) * U + (2 * em * d.abs().mean((1, 2)) + em * em) / ms) + 3 * U
        r = 1.0 / torch.sqrt(ms)
        y = (d * r[:, None, None] * weight[l]).abs()
        b = y * (rr[:, None, None] + 4 * U) + em[:, None, None] * r[:, None, None] * weight[l].abs()
        if l == 0 and bias is not None:
            y = (d * r[:, None, None] * weight[l] + bias).abs()
        parts.append(b + y * HALF[y_dtype] * (1 + 2 ** -7))
        rel.append(rr)
    return torch.cat(parts, 1) + 1e-37, e + 1e-37, torch.stack(rel, 1)


def norm_backward(h, weight, mean, rstd, gy, L):
    """grad_x, grad_weight, grad_bias by the formula, for the given statistics."""
    gx, gw = [], []
    for l, rows in enumerate(degrees(L)):
        r = rstd[:, l, None, None]
        xh = (h[:, rows] - (mean[:, None, None] if l == 0 else 0.0)) * r
        u = gy[:, rows] * weight[l]
        p = u - xh * (u * xh).mean((1, 2), keepdim=True)
        gx.append(r * (p - u.mean((1, 2), keepdim=True) if l == 0 else p))
        gw.append((gy[:, rows] * xh).sum((0, 1)))
    return torch.cat(gx, 1), torch.stack(gw), gy[:, 0].sum(0)


def norm_backward_bound(h, weight, mean, rstd, gy, L):
    """Bounds on grad_x, grad_weight, grad_bias: group sums in chains of CHAIN additions of terms that carry at
    most 5 roundings; xh carries 2; the last expression 4 more. The weight sums run in chains of at most 1024
    additions (the longest at the tested sizes: rows of a block's nodes, then the blocks)."""
    gx, gw = [], []
    for l, rows in enumerate(degrees(L)):
        r = rstd[:, l, None, None]
        xh = ((h[:, rows] - (mean[:, None, None] if l == 0 else 0.0)) * r).abs()
        u = (gy[:, rows] * weight[l]).abs()
        m2 = (u * xh).mean((1, 2), keepdim=True)
        m1 = u.mean((1, 2), keepdim=True) if l == 0 else 0.0
        gx.append(r * ((CHAIN + 12) * U * (m1 + xh * m2) + 6 * U * u))
        gw.append((1024 + 4) * U * (gy[:, rows].abs() * xh).sum((0, 1)))
    return torch.cat(gx, 1) + 1e-37, torch.stack(gw) + 1e-37, 1024 * U * gy[:, 0].abs().sum(0) + 1e-37


def coded(x):
    """(values, codes, scale bytes) of the 8-bit checkpoint of x [..., C], in blocks of 32 channels."""
    C = x.shape[-1]
    nb = (C + 31) // 32
    b = torch.zeros(x.shape[:-1] + (32 * nb,), dtype=torch.float64)
    b[..., :C] = x.double()
    b = b.reshape(x.shape[:-1] + (nb, 32))
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    b = torch.where(bad, 0.0, b)
    e = torch.frexp(b.abs().amax(-1, keepdim=True))[1] - 1
    e = torch.where(b.abs().amax(-1, keepdim=True) > 0, e, -120).clamp(min=-120)
    code = torch.round(torch.ldexp(b, 6 - e)).clamp(-127, 127)
    val = torch.where(bad, float("nan"), torch.ldexp(code, e - 6))
    cut = lambda t: t.reshape(x.shape[:-1] + (32 * nb,))[..., :C].contiguous()
    return cut(val), cut(code).to(torch.int8), torch.where(bad, 255, e + 127)[..., 0].to(torch.uint8)


def embedding(tokens, table, scale, L):
    n, (V, C) = tokens.shape[0], table.shape
    first = torch.zeros(n, C, dtype=torch.float64)
    ok = (tokens >= 0) & (tokens < V)
    first[ok] = scale * table.double()[tokens[ok].long()]
    return torch.cat([first[:, None], torch.zeros(n, (L + 1) ** 2 - 1, C, dtype=torch.float64)], 1)


def embedding_backward(tokens, grad_out, V, scale):
    """grad_table and the sum of magnitudes behind each value."""
    out = torch.zeros(V, grad_out.shape[-1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    ok = (tokens >= 0) & (tokens < V)
    out.index_add_(0, tokens[ok].long(), grad_out[ok, 0].double())
    mag.index_add_(0, tokens[ok].long(), grad_out[ok, 0].double().abs())
    return scale * out, abs(scale) * mag
