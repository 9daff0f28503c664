"""Plain 64-bit definitions of the training step's operators for the tests, written from the
formulas in numpy (the linear ones in torch), sharing no code with the package.  Beside each result stands the sum of the
magnitudes that went into it, which the tests' error bounds are multiples of."""
import numpy as np
import torch


def block_norm(x, y, w_post, gate, w_pre, row_gate, skip, branch, eps):
    """(z, h, rstd_post, rstd_pre, magnitude of z); None where there is none."""
    n, d = x.shape
    z, size, r1 = skip * x, np.abs(skip * x), None
    if y is not None:
        u = y
        if w_post is not None:
            r1 = 1 / np.sqrt((y ** 2).mean(1) + eps)
            u = y * r1[:, None] * w_post
        u = branch * u * (1 if gate is None else gate) * (1 if row_gate is None else row_gate[:, None])
        z, size = z + u, size + np.abs(u)
    r2 = h = None
    if w_pre is not None:
        r2 = 1 / np.sqrt((z ** 2).mean(1) + eps)
        h = z * r2[:, None] * w_pre
    return z, h, r1, r2, size


def block_norm_bwd(dh, d_out, z, y, w_post, gate, w_pre, row_gate, skip, branch, r1, r2):
    """Dict of gradients, and a dict of the magnitudes in them."""
    out, size = {}, {}
    ref = dh if dh is not None else d_out
    n, d = ref.shape
    dz = np.zeros((n, d)) if d_out is None else d_out.copy()
    big = np.abs(dz)
    if dh is not None:
        v = z * r2[:, None]
        a = dh * w_pre
        dz = dz + r2[:, None] * (a - v * (a * v).mean(1, keepdims=True))
        big = big + np.abs(r2)[:, None] * (np.abs(a) + np.abs(v) * np.abs(a * v).mean(1, keepdims=True))
        out["dw_pre"], size["dw_pre"] = (dh * v).sum(0), np.abs(dh * v).sum(0)
    out["dx"], size["dx"] = skip * dz, np.abs(skip) * big
    if y is None:
        return out, size
    s = y if w_post is None else y * r1[:, None]
    g = np.ones(d) if gate is None else gate
    w = np.ones(d) if w_post is None else w_post
    rho = np.ones(n) if row_gate is None else row_gate
    if w_post is not None:
        out["dw_post"] = (branch * rho[:, None] * g * dz * s).sum(0)
        size["dw_post"] = np.abs(branch * rho[:, None] * g * big * s).sum(0)
    if gate is not None:
        out["dgate"] = (branch * rho[:, None] * w * dz * s).sum(0)
        size["dgate"] = np.abs(branch * rho[:, None] * w * big * s).sum(0)
    if row_gate is not None:
        out["drow_gate"] = (branch * g * w * dz * s).sum(1)
        size["drow_gate"] = np.abs(branch * g * w * big * s).sum(1)
    t, bt = branch * rho[:, None] * g * w * dz, np.abs(branch * rho[:, None] * g * w) * big
    if w_post is not None:
        t = r1[:, None] * (t - s * (t * s).mean(1, keepdims=True))
        bt = np.abs(r1)[:, None] * (bt + np.abs(s) * (bt * np.abs(s)).mean(1, keepdims=True))
    out["dy"], size["dy"] = t, bt
    return out, size


def linear_logits(h, w, inv_t):
    """(scaled logits, the magnitudes in them) of 64-bit torch tensors"""
    return inv_t * (h @ w.T), inv_t * (h.abs() @ w.abs().T)


def linear_logprobs(x, targets):
    """(logprob, entropy, lse) of scaled logits"""
    m = x.amax(1)
    m0 = torch.where(torch.isinf(m), 0.0, m)[:, None]
    e = torch.exp(x - m0)
    total = e.sum(1)
    lse = m0[:, 0] + torch.log(total)
    shifted = torch.where(e > 0, e * (x - m0), 0.0).sum(1)
    entropy = torch.where(total > 0, torch.log(total) - shifted / total, 0.0)
    has = (targets >= 0) & (targets < x.shape[1])
    of = x.gather(1, torch.where(has, targets, 0).long()[:, None])[:, 0]
    return torch.where(has, of - lse, 0.0), entropy, lse


def linear_grad(x, targets, inv_t, lse, entropy, g, ge):
    """(gradient of the unscaled logits, the magnitudes in it)"""
    logp = x - lse[:, None]
    p = torch.exp(logp)
    has = (targets >= 0) & (targets < x.shape[1])
    g = torch.where(has, 0.0 if g is None else g, 0.0)
    d, size = -p * g[:, None], p * g.abs()[:, None]
    if ge is not None:
        shift = torch.where(p > 0, logp + entropy[:, None], 0.0)
        d = d - ge[:, None] * p * shift
        size = size + ge.abs()[:, None] * p * (torch.where(p > 0, logp.abs(), 0.0) + entropy[:, None] + 1)
    rows = torch.arange(len(x), device=x.device)[has]
    d[rows, targets[has].long()] += g[has]
    size[rows, targets[has].long()] += g[has].abs()
    return inv_t * d, inv_t * size
