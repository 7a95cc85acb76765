"""Plain fp64 forms (torch on the CPU) of the operators around the routed
experts, written from their formulas, for the tests of the GPU kernels."""
import torch

F64 = torch.float64
INF = float("inf")
U24 = 2.0 ** -24   # half a step of fp32
U8 = 2.0 ** -8     # half a step of bf16


def rmsnorm(x, residual, weight, eps):
    """(h, rstd, y) of bf16 CPU tensors: h rounded to bf16, the rest in fp64."""
    h = x if residual is None else (x.double() + residual.double()).to(torch.bfloat16)
    d = h.double()
    r = 1.0 / torch.sqrt((d * d).mean(-1) + eps)
    return h, r, d * r[:, None] * weight.double()


def rmsnorm_backward(dy, h, weight, rstd, dh):
    """(dx, dweight, size): `size` is the sum of the magnitudes that make dx."""
    dy, h, w, r = dy.double(), h.double(), weight.double(), rstd.double()[:, None]
    g, n = dy * w, h * r
    c = (g * n).mean(-1, keepdim=True)
    dx = r * (g - n * c)
    size = r * (g.abs() + n.abs() * (g * n).abs().mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        size = size + dh.double().abs()
    return dx, (dy * n).sum(0), size


def clean(logits):
    l = logits.double()
    l = torch.where(torch.isnan(l), -INF, l)
    return l.clamp(max=torch.finfo(torch.float32).max)


def scores(logits, sigmoid):
    """(score, probability) rows; experts at -inf have neither."""
    l = clean(logits)
    on = l > -INF
    if sigmoid:
        # relative to the row's largest, as a sum of tiny scores keeps its quotients
        ref = l.amax(-1, keepdim=True).clamp(max=0.0, min=-1e300)
        rel = torch.exp(l.clamp(max=0.0) - ref) / (1 + torch.exp(-l.abs()))
        score = 1 / (1 + torch.exp(-l))
    else:
        rel = torch.exp(l - l.amax(-1, keepdim=True).clamp(min=-1e300))
        score = rel / rel.sum(-1, keepdim=True).clamp(min=1e-300)
    rel, score = torch.where(on, rel, 0.0), torch.where(on, score, 0.0)
    return score, rel / rel.sum(-1, keepdim=True).clamp(min=1e-300)


def chosen_weights(logits, ids, sigmoid, renormalize):
    """Weights of given ids (-1: none, weight 0)."""
    l = clean(logits)
    score, _ = scores(logits, sigmoid)
    at = ids.clamp(min=0).long()
    ok = ids >= 0
    if not renormalize:
        return torch.where(ok, score.gather(1, at), 0.0)
    c = torch.where(ok, l.gather(1, at), -INF)
    top = c.amax(-1, keepdim=True).clamp(min=-1e300)
    if sigmoid:
        rel = torch.exp(c.clamp(max=0.0) - top.clamp(max=0.0)) / (1 + torch.exp(-c.abs()))
    else:
        rel = torch.exp(c - top)
    rel = torch.where(ok & (c > -INF), rel, 0.0)
    return rel / rel.sum(-1, keepdim=True).clamp(min=1e-300)


def router_topk(logits, k, sigmoid, renormalize, bias=None, mask=None):
    """(ids int32, weights fp64), by a full sort of (key descending, id ascending)."""
    l = clean(logits)
    key = l if bias is None else scores(logits, sigmoid)[0] + bias.double()
    key = torch.where((l > -INF) & ~torch.isnan(key), key, -INF)
    order = torch.sort(key, dim=-1, descending=True, stable=True)
    ids = torch.where(order.values[:, :k] > -INF, order.indices[:, :k], -1)
    if mask is not None:
        ids = torch.where(mask.bool()[:, None], ids, -1)
    return ids.to(torch.int32), chosen_weights(logits, ids, sigmoid, renormalize)


def balance(logits, ids, k, sigmoid, coef, mask=None):
    """(counts, mean_probs, prob_grad, loss)"""
    M, E = logits.shape
    on = torch.ones(M, dtype=torch.bool) if mask is None else mask.bool()
    T = int(on.sum())
    _, p = scores(logits, sigmoid)
    flat = ids[on].reshape(-1).long()
    counts = torch.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
    if T == 0:
        z = torch.zeros(E, dtype=F64)
        return counts, z, z, torch.zeros((), dtype=F64)
    mean = (p * on[:, None]).sum(0) / T
    f = counts.double() / (T * k)
    return counts, mean, coef * E / T * (f - 1.0 / E), coef * E * (f * mean).sum()


def router_backward(logits, ids, sigmoid, renormalize, dw=None, grad=None, dloss=1.0, mask=None):
    """d_logits, and the size of what was added up to it."""
    M, E = logits.shape
    l = clean(logits)
    score, p = scores(logits, sigmoid)
    keep = 1 / (1 + torch.exp(l)) if sigmoid else torch.ones_like(l)
    d, size = torch.zeros(M, E, dtype=F64), torch.zeros(M, E, dtype=F64)
    if grad is not None:
        u = grad.double() * dloss
        dot, mag = (p * u).sum(-1, keepdim=True), (p * u.abs()).sum(-1, keepdim=True)
        d += p * keep * (u - dot)
        size += p * keep * (u.abs() + mag)
    if dw is not None:
        ids = torch.where((ids >= 0) & (ids < E), ids, -1)
        at, ok = ids.clamp(min=0).long(), ids >= 0
        g = torch.where(ok, dw.double(), 0.0)
        w = chosen_weights(logits, ids, sigmoid, renormalize)
        dot, mag = (g * w).sum(-1, keepdim=True), (g * w).abs().sum(-1, keepdim=True)
        if renormalize:
            v, s = w * (g - dot), w * (g.abs() + mag)
        else:
            v, s = w * g, w * g.abs()
        kj = keep.gather(1, at)
        d.scatter_add_(1, at, torch.where(ok, v * kj, 0.0))
        size.scatter_add_(1, at, torch.where(ok, s * kj, 0.0))
        if not renormalize and not sigmoid:
            d -= p * dot
            size += p * mag
    if mask is not None:
        d *= mask.bool()[:, None]
    return d, size


E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=F64)


def e2m1_values(q):
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2).long()
    return torch.cat((E2M1, -E2M1))[c]


def mx_values(q, sf, elem):
    """fp64 values of MX codes (uint8 CPU tensors)."""
    v = e2m1_values(q) if elem == 1 else q.view(torch.float8_e4m3fn).double()
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(sf.double() - 127)[..., None]).flatten(-2)
