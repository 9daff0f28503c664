"""Cases of the operators of a training step around the sparse feed-forward layer: the norms before and
after a block with its gate and residual scale, and the log probabilities of tokens straight from hidden
rows and output weights (a softmax over a large vocabulary whose logits are never stored), each with its
gradient.

`run` computes an operator in its plain form (elementary torch operations in 32 bits) or, where
`own` is set, by the package's kernels.  `exact` states the definition in 64 bits.

    norm      u = y r1 w_post (or u = y),  z = skip x + branch row_gate gate u,  h = z r2 w_pre,
              r1 = (mean y^2 + eps)^-1/2,  r2 = (mean z^2 + eps)^-1/2
    linear    x = inv_temperature hidden weight^T,  lse, logprob = x[target] - lse, entropy of softmax(x)
"""
import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the decode batch of 16 tokens at d_model 4096, a norm before the next block only: pure latency
        dict(name="norm_decode_16", op="norm", rows=16, dim=4096, stream="bfloat16", post=False, gate=False,
             row_gate=False, pre=True, wide=False),
        # a residual stream kept in 32 bits, an odd number of rows, row widths of no power of two, block outputs that
        # are slices of wider rows, a weight for each row (tokens routed past the block)
        dict(name="norm_odd_f32", op="norm", rows=2999, dim=1352, stream="float32", post=True, gate=False, row_gate=True,
             pre=True, wide=True),
        # the training shape's tokens (8192 x 2048), norms on both sides and a gate for each channel
        dict(name="norm_train", op="norm", rows=8192, dim=2048, stream="bfloat16", post=True, gate=True, row_gate=False,
             pre=True, wide=False),
        # a short batch's gradients with everything there is, odd sizes
        dict(name="norm_bwd_odd", op="norm_bwd", rows=333, dim=4104, stream="float32", post=True, gate=True,
             row_gate=True, pre=True, wide=False),
        # the training shape's gradients
        dict(name="norm_bwd_train", op="norm_bwd", rows=8192, dim=2048, stream="bfloat16", post=True, gate=True,
             row_gate=False, pre=True, wide=False),
        # log probabilities of the decode batch's 16 tokens: the output weights' bytes
        dict(name="linear_decode_16", op="linear", rows=16, dim=4096, vocab=131072, wide=False),
        # a small batch, a vocabulary of odd size, hidden rows that are slices of wider ones
        dict(name="linear_odd", op="linear", rows=413, dim=1032, vocab=50001, wide=True),
        # the training shape's token log probabilities and entropies
        dict(name="linear_train", op="linear", rows=8192, dim=2048, vocab=32768, wide=False),
        # gradients of a few rows over a vocabulary of odd size: the weights' gradient is what there is to write
        dict(name="linear_bwd_odd", op="linear_bwd", rows=77, dim=1032, vocab=50001, wide=False),
        # gradients of the training shape
        dict(name="linear_bwd_train", op="linear_bwd", rows=8192, dim=2048, vocab=32768, wide=False),
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "linear", "linear_bwd"])
    if op in ("norm", "norm_bwd"):
        c = dict(op=op, rows=_log_int(rng, 1, 40000), dim=8 * _log_int(rng, 8, 1024),
                 stream=rng.choice(["bfloat16", "bfloat16", "float32"]), post=rng.random() < 0.7,
                 gate=rng.random() < 0.5, row_gate=rng.random() < 0.3, pre=rng.random() < 0.9,
                 wide=rng.random() < 0.3)
        while c["rows"] * c["dim"] > 1 << 26:
            c["rows"] = c["rows"] * 2 // 3
        return c
    c = dict(op=op, rows=_log_int(rng, 1, 12000), dim=8 * _log_int(rng, 16, 512), vocab=_log_int(rng, 40, 140000),
             wide=rng.random() < 0.3)
    most = (8192 * 2048 * 32768) // (1 if op == "linear" else 2)
    while c["rows"] * c["dim"] * c["vocab"] > most or c["rows"] * c["vocab"] > 1 << 28:
        c["rows"] = max(1, c["rows"] * 2 // 3)
    return c


# ---------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _slice_of_wider(x, extra):
    """The same values as a slice of rows that are `extra` elements longer."""
    wider = torch.zeros((x.shape[0], x.shape[1] + extra), dtype=x.dtype, device=x.device)
    wider[:, :x.shape[1]] = x
    return wider[:, :x.shape[1]]


def _prepare_norm(s, case, g):
    n, d = case["rows"], case["dim"]
    stream = getattr(torch, case["stream"])
    # a residual stream with a few large channels and rows of different size, a block's output of another size
    x = _randn(g, n, d) * torch.exp(0.7 * _randn(g, 1, d)) * torch.exp(0.3 * _randn(g, n, 1))
    y = 0.4 * _randn(g, n, d) * torch.exp(0.4 * _randn(g, n, 1))
    s["y"] = y.to(torch.bfloat16)
    for name, used in (("w_post", case["post"]), ("gate", case["gate"]), ("w_pre", case["pre"])):
        w = (0.3 if name == "gate" else 1.0) * (1 + 0.2 * _randn(g, d))
        s[name] = w.to(torch.bfloat16) if used else None
    s["row_gate"] = None
    if case["row_gate"]:  # a router's weight of each token, some of them routed past the block
        r = torch.rand(n, generator=g, device="cuda")
        s["row_gate"] = torch.where(r < 0.1, 0.0, r)
    s["skip"], s["branch"] = (1.0, 1.0) if n % 2 == 0 else (0.8, 0.35)
    s["x"] = x.to(stream)
    if case["wide"]:
        s["x"], s["y"] = _slice_of_wider(s["x"], 24), _slice_of_wider(s["y"], 40)
    if case["op"] == "norm":
        return
    # what the forward pass left, and the upstream gradients
    z, _, s["rstd_post"], s["rstd_pre"] = _norm_forward(s)
    s["x_out"] = z.to(stream)
    s["d_h"] = (0.1 * _randn(g, n, d) * torch.exp(0.5 * _randn(g, n, 1))).to(torch.bfloat16) if case["pre"] else None
    s["d_out"] = (0.2 * _randn(g, n, d)).to(stream)
    del s["x"]


def _prepare_linear(s, case, g):
    n, d, v = case["rows"], case["dim"], case["vocab"]
    # hidden rows behind a norm; output rows of a size that spreads the logits by about 2.5, and a share of the
    # rows' own token in each hidden row, as a trained model has it
    w = _randn(g, v, d) * (2.5 / math.sqrt(d)) * torch.exp(0.2 * _randn(g, v, 1))
    hot = torch.randint(v, (n,), generator=g, device="cuda")
    of_hot = w[hot]
    h = _randn(g, n, d) + of_hot * (12 * torch.rand((n, 1), generator=g, device="cuda")
                                    / of_hot.square().sum(1, keepdim=True))
    s["hidden"], s["weight"] = h.to(torch.bfloat16), w.to(torch.bfloat16)
    del w, of_hot
    t = torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, hot,
                    torch.randint(v, (n,), generator=g, device="cuda"))
    # prompt tokens and padding have no target
    s["targets"] = torch.where(torch.rand(n, generator=g, device="cuda") < 0.05, -1, t).to(torch.int32)
    s["inv_temperature"] = 1.0 if n % 2 == 0 else 1.25
    if case["wide"]:
        s["hidden"], s["weight"] = _slice_of_wider(s["hidden"], 64), _slice_of_wider(s["weight"], 8)
    if case["op"] == "linear":
        return
    # what the forward pass left, and the upstream gradients: a policy gradient's weights, a little entropy
    out = _plain_linear(s)
    s["lse"], s["entropy"] = out["lse"], out["entropy"]
    s["g_logprob"] = _randn(g, n) / n
    s["g_entropy"] = 0.05 * _randn(g, n) / n


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    (_prepare_norm if case["op"] in ("norm", "norm_bwd") else _prepare_linear)(s, case, g)
    return s


# ---------------------------------------------------------------- the plain forms
def _wide(t):
    return None if t is None else t.float()


def _norm_forward(s):
    """(z, h or None, rstd_post or None, rstd_pre or None) in 32 bits"""
    u, r1, r2, h = s["y"].float(), None, None, None
    if s["w_post"] is not None:
        r1 = torch.rsqrt(u.square().mean(1) + EPS)
        u = u * r1[:, None] * s["w_post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    if s["row_gate"] is not None:
        u = u * s["row_gate"][:, None]
    z = s["skip"] * s["x"].float() + s["branch"] * u
    if s["w_pre"] is not None:
        r2 = torch.rsqrt(z.square().mean(1) + EPS)
        h = z * r2[:, None] * s["w_pre"].float()
    return z, h, r1, r2


def _plain_norm(s):
    z, h, r1, r2 = _norm_forward(s)
    out = {"x_out": z.to(s["x"].dtype)}
    if h is not None:
        out["h"], out["rstd_pre"] = h.to(torch.bfloat16), r2
    if r1 is not None:
        out["rstd_post"] = r1
    return out


def _plain_norm_bwd(s):
    out, dz = {}, s["d_out"].float()
    if s["w_pre"] is not None:
        zh = s["x_out"].float() * s["rstd_pre"][:, None]
        dh = s["d_h"].float()
        a = dh * s["w_pre"].float()
        dz = dz + s["rstd_pre"][:, None] * (a - zh * (a * zh).mean(1, keepdim=True))
        out["dw_pre"] = (dh * zh).sum(0)
    out["dx"] = (s["skip"] * dz).to(s["d_out"].dtype)
    yh = s["y"].float()
    if s["w_post"] is not None:
        yh = yh * s["rstd_post"][:, None]
    w_post, gate = _wide(s["w_post"]), _wide(s["gate"])
    row = s["row_gate"][:, None] if s["row_gate"] is not None else 1.0
    e = s["branch"] * dz
    u = yh if w_post is None else yh * w_post
    if gate is not None:
        out["dgate"] = (e * row * u).sum(0)
        e = e * gate
    if s["row_gate"] is not None:
        out["drow_gate"] = (e * u).sum(1)
        e = e * row
    if w_post is not None:
        out["dw_post"] = (e * yh).sum(0)
        f = e * w_post
        e = s["rstd_post"][:, None] * (f - yh * (f * yh).mean(1, keepdim=True))
    out["dy"] = e.to(torch.bfloat16)
    return out


def _scaled_logits(s):
    return torch.matmul(s["hidden"].float(), s["weight"].float().t()).mul_(s["inv_temperature"])


def _plain_linear(s):
    x = _scaled_logits(s)
    t = s["targets"].long()
    of_target = x.gather(1, t.clamp(min=0)[:, None])[:, 0]
    top = x.amax(1, keepdim=True)
    x.sub_(top)
    e = torch.exp(x)
    total = e.sum(1)
    lse = top[:, 0] + torch.log(total)
    entropy = torch.log(total) - e.mul_(x).sum(1) / total
    return {"logprob": torch.where(t >= 0, of_target - lse, 0.0), "entropy": entropy, "lse": lse}


def _plain_linear_bwd(s):
    logp = _scaled_logits(s).sub_(s["lse"][:, None])
    t = s["targets"].long()
    g = torch.where(t >= 0, s["g_logprob"], 0.0)[:, None]
    p = torch.exp(logp)
    d = logp.add_(s["entropy"][:, None]).mul_(s["g_entropy"][:, None]).add_(g).mul_(p).neg_()
    d.scatter_add_(1, t.clamp(min=0)[:, None], g)
    d.mul_(s["inv_temperature"])
    return {"d_hidden": torch.matmul(d, s["weight"].float()).to(torch.bfloat16),
            "d_weight": torch.matmul(d.t(), s["hidden"].float()).to(torch.bfloat16)}


# ---------------------------------------------------------------- the package's operators
def _handles(tw, s):
    """What a program keeps between steps: output buffers and workspaces."""
    if "kept" in s:
        return s["kept"]
    case, kept = s["case"], {}
    n, d = case["rows"], case["dim"]

    def new(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if case["op"] == "norm":
        kept["x_out"] = new(n, d, dtype=s["x"].dtype)
        if case["pre"]:
            kept["h"], kept["rstd_pre"] = new(n, d, dtype=torch.bfloat16), new(n)
        if case["post"]:
            kept["rstd_post"] = new(n)
    elif case["op"] == "norm_bwd":
        kept["dx"], kept["dy"] = new(n, d, dtype=s["d_out"].dtype), new(n, d, dtype=torch.bfloat16)
        for name, used in (("dw_post", case["post"]), ("dgate", case["gate"]), ("dw_pre", case["pre"])):
            if used:
                kept[name] = new(d)
        if case["row_gate"]:
            kept["drow_gate"] = new(n)
        s["workspace"] = new(tw.block_norm_bwd_workspace_bytes(n, d), dtype=torch.uint8)
    else:
        s["status"] = torch.zeros(4, dtype=torch.int32, device="cuda")
        if case["op"] == "linear":
            kept = {name: new(n) for name in ("logprob", "entropy", "lse")}
            need = tw.linear_logprobs_workspace_bytes(n, d, case["vocab"])
        else:
            kept["d_hidden"] = new(n, d, dtype=torch.bfloat16)
            kept["d_weight"] = new(case["vocab"], d, dtype=torch.bfloat16)
            need = tw.linear_logprobs_bwd_workspace_bytes(n, d, case["vocab"])
        s["workspace"] = new(need, dtype=torch.uint8)
    s["kept"] = kept
    return kept


def _own(s):
    import activation_sparse_transformer_gb300 as tw
    kept, op = _handles(tw, s), s["case"]["op"]
    if op == "norm":
        tw.twell_block_norm(s["x"], s["y"], kept["x_out"], kept.get("h"), w_post=s["w_post"], gate=s["gate"],
                            w_pre=s["w_pre"], row_gate=s["row_gate"], skip_scale=s["skip"], branch_scale=s["branch"],
                            eps=EPS, rstd_post=kept.get("rstd_post"), rstd_pre=kept.get("rstd_pre"))
    elif op == "norm_bwd":
        tw.twell_block_norm_bwd(s["d_h"], s["d_out"], s["x_out"], s["y"], kept["dx"], kept["dy"],
                                w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"], row_gate=s["row_gate"],
                                skip_scale=s["skip"], branch_scale=s["branch"], rstd_post=s["rstd_post"],
                                rstd_pre=s["rstd_pre"], dw_post=kept.get("dw_post"), dgate=kept.get("dgate"),
                                dw_pre=kept.get("dw_pre"), drow_gate=kept.get("drow_gate"), workspace=s["workspace"])
    elif op == "linear":
        tw.twell_linear_logprobs(s["hidden"], s["weight"], s["targets"], s["inv_temperature"], kept["logprob"],
                                 kept["entropy"], kept["lse"], s["workspace"], s["status"])
    else:
        tw.twell_linear_logprobs_bwd(s["hidden"], s["weight"], s["targets"], s["inv_temperature"], s["lse"],
                                     s["entropy"], s["g_logprob"], s["g_entropy"], kept["d_hidden"],
                                     kept["d_weight"], s["workspace"], s["status"])
    return kept


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "linear": _plain_linear,
            "linear_bwd": _plain_linear_bwd}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    n, d = case["rows"], case["dim"]
    if case["op"] in ("norm", "norm_bwd"):
        wide = 2 if case["stream"] == "bfloat16" else 4
        vectors = case["post"] + case["gate"] + case["pre"]
        if case["op"] == "norm":
            return {"bytes": n * d * (2 * wide + 2 + 2 * case["pre"]) + 2 * d * vectors
                    + 4 * n * (case["post"] + case["pre"] + case["row_gate"]), "flops": 10 * n * d}
        return {"bytes": n * d * (2 * wide + 4 + (wide + 2) * case["pre"]) + 6 * d * vectors
                + 4 * n * (case["post"] + case["pre"] + 2 * case["row_gate"]), "flops": 25 * n * d}
    v = case["vocab"]
    if case["op"] == "linear":
        return {"bytes": 2 * d * (n + v) + 16 * n, "flops": 2 * n * d * v}
    return {"bytes": 4 * d * (n + v) + 20 * n, "flops": 6 * n * d * v}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_norm(s):
    d = s["x"].shape[1]
    one = torch.ones((), dtype=torch.float64, device="cuda")
    w_post, gate, w_pre, row = (one if s[k] is None else s[k].double() for k in ("w_post", "gate", "w_pre", "row_gate"))
    y, out = s["y"].double(), {}
    if s["w_post"] is not None:
        out["rstd_post"] = 1 / torch.sqrt((y * y).sum(1) / d + EPS)
        y = torch.einsum("nd,n->nd", y, out["rstd_post"])
    factor = s["branch"] * row.reshape(-1, 1) * (gate * w_post)
    out["x_out"] = s["skip"] * s["x"].double() + factor * y
    if s["w_pre"] is not None:
        out["rstd_pre"] = 1 / torch.sqrt(torch.einsum("nd,nd->n", out["x_out"], out["x_out"]) / d + EPS)
        out["h"] = torch.einsum("nd,n,d->nd", out["x_out"], out["rstd_pre"], w_pre)
    return out


def _exact_norm_bwd(s):
    """By products with the norms' Jacobians, row by row: J = r (I - v v^T / d), v the normed row."""
    n, d = s["y"].shape
    double = {k: (None if s[k] is None else s[k].double()) for k in
              ("w_post", "gate", "w_pre", "row_gate", "rstd_post", "rstd_pre", "x_out", "y", "d_h", "d_out")}

    def through_norm(v, r, upstream):
        return r[:, None] * (upstream - v * (torch.einsum("nd,nd->n", v, upstream) / d)[:, None])

    out, dz = {}, double["d_out"]
    if s["w_pre"] is not None:
        v = double["x_out"] * double["rstd_pre"][:, None]
        out["dw_pre"] = torch.einsum("nd,nd->d", double["d_h"], v)
        dz = dz + through_norm(v, double["rstd_pre"], double["d_h"] * double["w_pre"])
    out["dx"] = s["skip"] * dz
    ones_d, ones_n = torch.ones(d, dtype=torch.float64, device="cuda"), torch.ones(n, dtype=torch.float64, device="cuda")
    w, gate, row = (o if t is None else t for t, o in ((double["w_post"], ones_d), (double["gate"], ones_d),
                                                       (double["row_gate"], ones_n)))
    v = double["y"] if s["w_post"] is None else double["y"] * double["rstd_post"][:, None]
    both = dz * v * s["branch"]  # the branch's z is branch * row * gate * w * v: each factor's gradient leaves it out
    if s["gate"] is not None:
        out["dgate"] = torch.einsum("nd,n,d->d", both, row, w)
    if s["row_gate"] is not None:
        out["drow_gate"] = torch.einsum("nd,d->n", both, gate * w)
    if s["w_post"] is not None:
        out["dw_post"] = torch.einsum("nd,n,d->d", both, row, gate)
    up = s["branch"] * torch.einsum("nd,n,d->nd", dz, row, gate * w)
    out["dy"] = up if s["w_post"] is None else through_norm(v, double["rstd_post"], up)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "norm_bwd":
        return _exact_norm_bwd(s)
    if case["rows"] * case["dim"] * case["vocab"] * (1 if case["op"] == "linear" else 3) > 4e12:
        return None
    h, w = s["hidden"].double(), s["weight"].double()
    x = torch.einsum("nd,vd->nv", h, w) * s["inv_temperature"]
    t = s["targets"].long()
    if case["op"] == "linear":
        lse = torch.logsumexp(x, 1)
        p = torch.softmax(x, 1)
        own_logit = x[torch.arange(len(t), device="cuda"), t.clamp(min=0)]
        return {"logprob": torch.where(t < 0, torch.zeros_like(lse), own_logit - lse),
                "entropy": torch.special.entr(p).sum(1), "lse": lse}
    # by the chain rule through the softmax: the loss's gradient to each log probability, w, then
    # d = p (w - <p, w>) beside the target's own; lse and entropy of these inputs, in 64 bits
    x -= torch.logsumexp(x, 1, keepdim=True)
    p = torch.exp(x)
    up = -(x + 1) * s["g_entropy"].double()[:, None]
    d = p * (up - (p * up).sum(1, keepdim=True))
    g = s["g_logprob"].double() * (t >= 0)
    d -= g[:, None] * p
    d[torch.arange(len(t), device="cuda"), t.clamp(min=0)] += g
    d *= s["inv_temperature"]
    return {"d_hidden": d @ w, "d_weight": d.t() @ h}
