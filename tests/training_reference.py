"""Plain 64-bit definitions of the training step's operators for the tests, written from the
formulas in numpy, sharing no code with the package.  Beside each result stands the sum of the
magnitudes that went into it, which the tests' error bounds are multiples of."""
import numpy as np


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


def linear_logprobs(h, w, targets, inv_t):
    """(logprob, entropy, lse, scaled logits)"""
    x = inv_t * (h @ w.T)
    with np.errstate(over="ignore", invalid="ignore"):
        m = x.max(1)
        m0 = np.where(np.isinf(m), 0, m)
        e = np.exp(x - m0[:, None])
        total = e.sum(1)
        lse = m0 + np.log(total)
        shifted = np.where(e > 0, e * (x - m0[:, None]), 0).sum(1)
        entropy = np.log(total) - shifted / total
    has = (targets >= 0) & (targets < w.shape[0])
    of = x[np.arange(len(x)), np.where(has, targets, 0)]
    return np.where(has, of - lse, 0.0), entropy, lse, x


def linear_logprobs_bwd(h, w, targets, inv_t, lse, entropy, g, ge):
    """(d_hidden, d_weight, gradient of the unscaled logits)"""
    x = inv_t * (h @ w.T)
    logp = x - lse[:, None]
    p = np.exp(logp)
    has = (targets >= 0) & (targets < w.shape[0])
    g = np.where(has, 0.0 if g is None else g, 0.0)
    d = -p * g[:, None]
    if ge is not None:
        d -= ge[:, None] * p * (logp + entropy[:, None])
    d[np.arange(len(x))[has], targets[has]] += g[has]
    d *= inv_t
    return d @ w, d.T @ h, d
