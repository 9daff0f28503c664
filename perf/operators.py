"""Cases of the operators around the sparse feed-forward layer in a decode step, and of the loss on
its answers: the step's block tables and slot maps, the append to an 8-bit cache, the attention that
reads it, the log probabilities of the answer, and their gradient.

`run` computes an operator in its plain form (elementary torch operations in 32 bits) or, where
`own` is set, by the package's kernels.  `exact` states the definition in 64 bits.

A cache is paged: page p, key head h holds `page` tokens of `dim` 8-bit codes (e4m3 or int8) and one
scale, a power of two.  A request's i-th page is block_table[request][i].
"""
import math

import numpy as np
import torch

own = False

MIN_EXP = -100  # the smallest scale is 2^-100, also that of a page of zeros


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the step's bookkeeping for the decode batch of 16 requests: pure latency
        dict(name="plan_decode_16", op="plan", requests=16, page=64, max_len=4096, max_new=1, finished=0.0),
        # a busy server's step: 1000 requests, some of them prompts, some finished
        dict(name="plan_mixed_1000", op="plan", requests=1000, page=16, max_len=32768, max_new=900, finished=0.05),
        # the decode batch's new tokens: one per request, pages that hold earlier tokens
        dict(name="append_decode_16", op="append", requests=16, heads=8, dim=128, page=64, max_len=4096, max_new=1,
             fmt="e4m3"),
        # prompts of ragged lengths, int8 codes
        dict(name="append_prompts_int8", op="append", requests=24, heads=8, dim=128, page=32, max_len=6000,
             max_new=4000, fmt="int8"),
        # the decode batch (16 tokens, d_model 4096 as 32 heads of 128), short caches: latency counts
        dict(name="attn_decode_16", op="attn", requests=16, q_heads=32, kv_heads=8, dim=128, page=64, max_len=1000,
             lengths="even", max_new=1, fmt="e4m3"),
        # few requests with very long caches: the cache's bytes, split over the long axis
        dict(name="attn_decode_long", op="attn", requests=4, q_heads=32, kv_heads=8, dim=128, page=128,
             max_len=131072, lengths="even", max_new=1, fmt="e4m3"),
        # a large ragged batch with heads of 64 (d_model 2048), a head of its own for each query head, int8,
        # idle and refused requests among them
        dict(name="attn_decode_ragged", op="attn", requests=250, q_heads=32, kv_heads=32, dim=64, page=16,
             max_len=4001, lengths="tail", max_new=1, fmt="int8"),
        # prompts taken in chunks over caches that hold earlier chunks: many rows for each cached token
        dict(name="attn_chunk", op="attn", requests=4, q_heads=32, kv_heads=8, dim=128, page=64, max_len=8192,
             lengths="even", max_new=1024, fmt="e4m3"),
        # the answer of the decode batch: 16 rows of a large vocabulary with 20 alternatives
        dict(name="logprobs_decode_16", op="logprobs", rows=16, vocab=131072, dtype="float32", top=20, masked=0.0),
        # a training batch's token log probabilities and entropies
        dict(name="logprobs_train", op="logprobs", rows=8192, vocab=32768, dtype="bfloat16", top=0, masked=0.0),
        # a small batch with a vocabulary of odd size, fp32 logits
        dict(name="logprobs_bwd_odd", op="logprobs_bwd", rows=64, vocab=50001, dtype="float32", masked=0.01),
        # the training batch's gradient
        dict(name="logprobs_bwd_train", op="logprobs_bwd", rows=8192, vocab=32768, dtype="bfloat16", masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn", "chunk", "logprobs", "logprobs", "logprobs_bwd"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        c = dict(op=op, requests=_log_int(rng, 1, 1500), page=page, max_len=_log_int(rng, 1, 32768),
                 max_new=_log_int(rng, 1, 900), finished=rng.choice([0.0, 0.05, 0.3]))
        while c["requests"] * c["max_new"] > 900000:
            c["requests"] //= 2
        return c
    if op == "append":
        c = dict(op=op, requests=_log_int(rng, 1, 300), heads=_log_int(rng, 1, 16), dim=rng.choice([64, 128]),
                 page=page, max_len=_log_int(rng, 1, 8000), max_new=rng.choice([1, 1, 5, _log_int(rng, 2, 4000)]),
                 fmt=rng.choice(["e4m3", "int8"]))
        while c["requests"] * c["heads"] * c["dim"] * (c["max_len"] + 128) > 24 * 8 * 128 * 6000:
            c["requests"], c["max_len"] = max(1, c["requests"] * 2 // 3), max(1, c["max_len"] * 3 // 4)
        return c
    if op in ("attn", "chunk"):
        kv = rng.choice([1, 2, 3, 4, 8, 16])
        c = dict(op="attn", requests=_log_int(rng, 1, 256), q_heads=kv * rng.choice([1, 2, 4, 5, 8]), kv_heads=kv,
                 dim=rng.choice([64, 128]), page=page, max_len=_log_int(rng, 1, 131072),
                 lengths=rng.choice(["even", "tail"]),
                 max_new=_log_int(rng, 16, 1024) if op == "chunk" else rng.choice([1, 1, 1, 2, 5]),
                 fmt=rng.choice(["e4m3", "int8"]))
        c["requests"] = min(c["requests"], 16) if op == "chunk" else c["requests"]
        while (c["requests"] * c["max_len"] * c["kv_heads"] * c["dim"] > 4 * 131072 * 8 * 64
               or c["requests"] * c["max_new"] * c["q_heads"] * c["max_len"] * c["dim"] > 4 * 1024 * 32 * 4096 * 128):
            c["requests"], c["max_len"] = max(1, c["requests"] * 2 // 3), max(1, c["max_len"] * 3 // 4)
        return c
    c = dict(op=op, rows=_log_int(rng, 1, 8192), vocab=_log_int(rng, 40, 140000),
             dtype=rng.choice(["bfloat16", "float32"]), masked=rng.choice([0.0, 0.01, 0.5]))
    if op == "logprobs":
        c["top"] = rng.choice([0, 1, 5, 20, 32])
    while c["rows"] * c["vocab"] > (1 << 27):
        c["rows"] = max(1, c["rows"] // 2)
    return c


# ---------------------------------------------------------------- what a case's requests look like
def _requests(case):
    """Old and new token counts of each request, by the case alone (new = -1: the request is finished)."""
    r, n = np.random.RandomState((case["requests"] * 7919 + case["max_len"] * 31 + case["max_new"]) % (1 << 31)), \
        case["requests"]
    if case["op"] == "attn":
        total = (np.exp(r.rand(n) * math.log(case["max_len"])) if case["lengths"] == "tail"
                 else case["max_len"] * (0.5 + 0.5 * r.rand(n)))
        total = np.maximum(1, total.astype(np.int64))
        total[r.randint(n)] = case["max_len"]
        new = np.full(n, 1) if case["max_new"] == 1 else np.maximum(1, (case["max_new"] * (0.5 + 0.5 * r.rand(n))))
        new = np.minimum(new.astype(np.int64), total)
        if n >= 8:  # a request that takes no part in the step
            total[1], new[1] = 0, 0
        return total - new, new
    old = (case["max_len"] * r.rand(n)).astype(np.int64)
    many = case["max_new"] if case["max_new"] > 1 else 0
    new = np.where(r.rand(n) < 0.5, 1 + (many * r.rand(n) ** 2).astype(np.int64), 1)
    if case["op"] == "append":
        new = np.minimum(new + (many * r.rand(n)).astype(np.int64), max(1, case["max_new"]))
        old = np.minimum(old, np.maximum(0, case["max_len"] - new))
    else:
        new = np.where(r.rand(n) < case["finished"], -1, new)
    return old, new


def _blocks(case, old, new):
    """(pages of each request after the step, width of its block table)"""
    need = -(-(old + np.maximum(new, 0)) // case["page"])
    return need, max(1, int(need.max()))


def _i32(a, device="cuda"):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=device)


def _codes_type(fmt):
    return torch.float8_e4m3fn if fmt == "e4m3" else torch.int8


def _exponent(amax, fmt):
    """The least e with amax <= largest code * 2^e, from the bits of a 32-bit amax, at least MIN_EXP."""
    bits = amax.contiguous().view(torch.int32)
    k, frac = (bits >> 23) - 127, bits & 0x7FFFFF
    top, over = (8, 0x600000) if fmt == "e4m3" else (6, 0x7E0000)  # 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6
    return (k - top + (frac > over).to(torch.int32)).clamp(min=MIN_EXP)


def _two_to(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _encode(x, fmt):
    """32-bit values already divided by their scale -> codes, to nearest even."""
    return x.to(torch.float8_e4m3fn) if fmt == "e4m3" else torch.round(x).to(torch.int8)


def _cache(case, g, heads, need, width):
    """A block table over shuffled pages and a cache full of keys or values: [pages][heads][page][dim]."""
    n_pages, page, dim = int(need.sum()) + 3, case["page"], case["dim"]
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = np.concatenate([[0], np.cumsum(need)])
    at = first[:-1, None] + np.arange(width)[None]
    at = torch.tensor(np.where(np.arange(width)[None] < need[:, None], at, -1), device="cuda")
    table = torch.where(at >= 0, order[at.clamp(min=0)], torch.full_like(order[:1], -1))
    made = []
    for _ in range(2):
        # channels of unequal size and a size for each page, as keys and values have
        x = torch.randn((n_pages, heads, page, dim), generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn((heads, 1, dim), generator=g, device="cuda"))
        x *= torch.exp(0.3 * torch.randn((n_pages, heads, 1, 1), generator=g, device="cuda"))
        scale = _two_to(_exponent(x.abs().amax((-1, -2)), case["fmt"]))
        x /= scale[..., None, None]
        made += [_encode(x, case["fmt"]), scale]
        del x
    return table.contiguous(), made


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] in ("logprobs", "logprobs_bwd"):
        n, v = case["rows"], case["vocab"]
        x = torch.randn((n, v), generator=g, device="cuda") * 2.5
        hot = torch.randint(v, (n, 1), generator=g, device="cuda")
        x.scatter_add_(1, hot, 12 * torch.rand((n, 1), generator=g, device="cuda"))
        if case["masked"]:
            x.masked_fill_(torch.rand((n, v), generator=g, device="cuda") < case["masked"], float("-inf"))
        s["logits"] = x.to(getattr(torch, case["dtype"]))
        t = torch.randint(v, (n,), generator=g, device="cuda")
        t = torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, hot[:, 0], t)
        # a masked token is no target of a training batch, and some rows have none
        t = torch.where(torch.isinf(s["logits"].gather(1, t[:, None])[:, 0]), -1, t)
        s["targets"] = torch.where(torch.rand(n, generator=g, device="cuda") < 0.05, -1, t).to(torch.int32)
        s["inv_temperature"] = 1.0 if case["rows"] % 2 else 1.25
        if case["op"] == "logprobs_bwd":  # what the forward pass left, and the upstream gradients
            y = s["logits"].float() * s["inv_temperature"]
            s["lse"] = torch.logsumexp(y, 1)
            p = torch.exp(y - s["lse"][:, None])
            s["entropy"] = s["lse"] - torch.where(p > 0, p * y, 0.0).sum(1)
            s["g_logprob"] = torch.randn(n, generator=g, device="cuda")
            s["g_entropy"] = 0.1 * torch.randn(n, generator=g, device="cuda")
        return s
    old, new = _requests(case)
    need, width = _blocks(case, old, new)
    s["page"] = case["page"]
    if case["op"] == "plan":
        have = -(-old // case["page"])
        n_pages = int(need.sum()) + 40
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        # pages in use are the order's first ones; the free ones wait in the ring from some place on
        first = np.concatenate([[0], np.cumsum(have)])
        at = np.where(np.arange(width)[None] < have[:, None], first[:-1, None] + np.arange(width)[None], -1)
        at = torch.tensor(at, device="cuda")
        s["table"] = torch.where(at >= 0, order[at.clamp(min=0)], torch.full_like(order[:1], -1)).contiguous()
        used, head = int(have.sum()), n_pages * 2 // 3
        s["ring"] = torch.roll(torch.cat([order[used:], torch.full_like(order[:used], -1)]), head).contiguous()
        s["pool"] = _i32([head, n_pages - used])
        s["lens"], s["new"] = _i32(old), _i32(new)
        s["tokens"] = int(np.maximum(new, 0).sum()) + 5  # a step is padded to a few tokens more
        return s
    heads = case["heads"] if case["op"] == "append" else case["kv_heads"]
    s["table"], (s["k"], s["k_scale"], s["v"], s["v_scale"]) = _cache(case, g, heads, need, width)
    cu = np.concatenate([[0], np.cumsum(new)])
    s["cu_q"] = _i32(cu)
    n = int(cu[-1])
    r = torch.repeat_interleave(torch.arange(len(new), device="cuda"), torch.tensor(new, device="cuda"))
    pos = torch.tensor(old, device="cuda")[r] + torch.arange(n, device="cuda") - torch.tensor(cu, device="cuda")[r]
    s["positions"] = pos.to(torch.int32)
    s["slots"] = s["table"][r, pos // case["page"]].long() * case["page"] + pos % case["page"]
    s["lens"] = _i32(old + new)
    if case["op"] == "append":
        # slices of one fused projection's output: rows further apart than they are long
        both = torch.randn((n, heads * 3 * case["dim"]), generator=g, device="cuda")
        both *= torch.exp(0.5 * torch.randn((n, 1), generator=g, device="cuda"))
        both = both.to(torch.bfloat16).view(n, 3 * heads, case["dim"])
        s["new_k"], s["new_v"] = both[:, heads:2 * heads], both[:, 2 * heads:]
        return s
    if len(new) >= 16:  # a request that had no room in the cache: its rows see nothing
        s["positions"][int(cu[2]):int(cu[3])] = -1
    s["q"] = (1.5 * torch.randn((n, case["q_heads"], case["dim"]), generator=g, device="cuda")).to(torch.bfloat16)
    s["softmax_scale"] = case["dim"] ** -0.5
    return s


# ---------------------------------------------------------------- the plain forms
def _plain_plan(s):
    lens, new, table, ring, page = s["lens"].long(), s["new"].long(), s["table"], s["ring"].long(), s["page"]
    n_pages, width = ring.numel(), table.shape[1]
    head, free = s["pool"][0].long(), s["pool"][1].long()
    done, add = new < 0, new.clamp(min=0)
    cu = torch.cat([add.new_zeros(1), add.cumsum(0)])
    have = (lens + page - 1) // page
    need = torch.where(done, 0, (lens + add + page - 1) // page - have)
    upto = need.cumsum(0)
    refused = (add > 0) & (((need > 0) & (upto > free)) | (have + need > width) | (cu[1:] > s["tokens"]))
    need_ok = torch.where(refused, 0, need)
    taken = torch.where(refused | (need == 0), 0, upto).max()
    j = torch.arange(width, device="cuda")[None]
    fresh = (j >= have[:, None]) & (j < (have + need_ok)[:, None])
    from_ring = ring[(head + (upto - need)[:, None] + j - have[:, None]) % n_pages]
    new_table = torch.where(fresh, from_ring, table.long())
    # the pages of finished requests, in order, behind the free ones
    back = torch.where(done, have, 0)
    back_upto = back.cumsum(0)
    i = (torch.arange(n_pages, device="cuda") - head - free) % n_pages
    of = torch.searchsorted(back_upto, i, right=True).clamp(max=lens.numel() - 1)
    page_back = table[of, (i - (back_upto - back)[of]).clamp(0, width - 1)].long()
    new_ring = torch.where(i < back_upto[-1], page_back, ring)
    t = torch.arange(s["tokens"], device="cuda")
    of = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=lens.numel() - 1)
    pos = lens[of] + t - cu[of]
    live = (t < cu[-1]) & ~refused[of]
    at = new_table[of, (pos // page).clamp(0, width - 1)] * page + pos % page
    return {"kv_lens": torch.where(done, 0, torch.where(refused, lens, lens + add)).to(torch.int32),
            "cu_q": cu.clamp(max=s["tokens"]).to(torch.int32), "slots": torch.where(live, at, -1),
            "positions": torch.where(live, pos, -1).to(torch.int32),
            "pool": torch.stack([(head + taken) % n_pages, free - taken + back_upto[-1]]).to(torch.int32),
            "table": new_table.to(torch.int32), "ring": new_ring.to(torch.int32)}


def _plain_append(s):
    fmt, page, out = s["case"]["fmt"], s["page"], {}
    touched, of = torch.unique(s["slots"] // page, return_inverse=True)
    offset = s["slots"] % page
    first = torch.full_like(touched, page).scatter_reduce(0, of, offset, "amin")
    for name, x in (("k", s["new_k"].float()), ("v", s["new_v"].float())):
        amax = x.abs().amax(-1)
        most = torch.zeros((touched.numel(), amax.shape[1]), device="cuda")
        most = most.scatter_reduce(0, of[:, None].expand_as(amax), amax, "amax")
        was = s[name + "_scale"][touched]
        scale = _two_to(_exponent(most, fmt))
        scale = torch.where((first > 0)[:, None], torch.maximum(scale, was), scale)
        codes = s[name].view(torch.int8)[touched].view(_codes_type(fmt))
        moved = _encode(codes.float() * (was / scale)[..., None, None], fmt)
        grew = (torch.arange(page, device="cuda")[None, None] < first[:, None, None]) & (scale != was)[..., None]
        codes = torch.where(grew[..., None], moved.view(torch.int8), codes.view(torch.int8))
        codes[of, :, offset] = _encode(x / scale[of][..., None], fmt).view(torch.int8)
        s[name].view(torch.int8)[touched] = codes
        s[name + "_scale"][touched] = scale
        out[name], out[name + "_scale"] = s[name], s[name + "_scale"]
    return out


def _plain_attn(s):
    case = s["case"]
    cu, lens, heads = s["cu_q"].long(), s["lens"].long(), case["kv_heads"]
    requests, group, dim, n = lens.numel(), case["q_heads"] // heads, case["dim"], s["q"].shape[0]
    most = case["max_new"]
    pages = s["table"].clamp(min=0).long()

    def dense(codes, scale):  # [requests, heads, tokens, dim]
        x = codes.view(torch.int8)[pages].view(_codes_type(case["fmt"])).float() * scale[pages][..., None, None]
        return x.transpose(1, 2).reshape(requests, heads, -1, dim)

    i = torch.arange(most, device="cuda")[None]
    live = i < (cu[1:] - cu[:-1])[:, None]
    token = torch.where(live, cu[:-1, None] + i, 0)
    limit = torch.where(live, torch.minimum(s["positions"].long()[token] + 1, lens[:, None]), 0)
    q = s["q"].float()[token].view(requests, most, heads, group, dim).permute(0, 2, 3, 1, 4)
    q = q.reshape(requests, heads, group * most, dim)
    x = torch.matmul(q, dense(s["k"], s["k_scale"]).transpose(2, 3)).mul_(s["softmax_scale"])
    x = x.view(requests, heads, group, most, -1)
    hidden = torch.arange(x.shape[-1], device="cuda") >= limit[:, None, None, :, None]
    x.masked_fill_(hidden, float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(requests, heads, group * most, -1), dense(s["v"], s["v_scale"]))
    o = o.view(requests, heads, group, most, dim) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    back = torch.where(live, token, n)  # rows of no token go to a row past the end
    out = torch.zeros((n + 1, case["q_heads"], dim), device="cuda")
    out[back] = o.permute(0, 3, 1, 2, 4).reshape(requests, most, -1, dim)
    out_lse = torch.full((n + 1, case["q_heads"]), float("-inf"), device="cuda")
    out_lse[back] = lse.permute(0, 3, 1, 2).reshape(requests, most, -1)
    return {"o": out[:n].to(torch.bfloat16), "lse": out_lse[:n]}


def _plain_logprobs(s):
    x = s["logits"].float() * s["inv_temperature"]
    v, k = x.shape[1], s["case"]["top"]
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    shifted = torch.where(e > 0, e * (x - top), 0.0).sum(1)
    t = s["targets"].long()
    has = (t >= 0) & (t < v)
    logprob = torch.where(has, x.gather(1, t.clamp(0, v - 1)[:, None])[:, 0] - lse, 0.0)
    out = {"logprob": logprob, "entropy": torch.log(total[:, 0]) - shifted / total[:, 0], "lse": lse}
    if k:  # a stable sort leaves ties in the order of their index
        best, index = torch.sort(x, dim=1, descending=True, stable=True)
        out["top_logprob"], out["top_index"] = best[:, :k] - lse[:, None], index[:, :k].to(torch.int32)
    return out


def _plain_logprobs_bwd(s):
    x = s["logits"].float() * s["inv_temperature"]
    v, t = x.shape[1], s["targets"].long()
    has = (t >= 0) & (t < v)
    logp = x - s["lse"][:, None]
    p = torch.exp(logp)
    g = torch.where(has, s["g_logprob"], 0.0)[:, None]
    d = -p * g - torch.where(p > 0, s["g_entropy"][:, None] * p * (logp + s["entropy"][:, None]), 0.0)
    d.scatter_add_(1, t.clamp(0, v - 1)[:, None], g)
    return {"d_logits": (d * s["inv_temperature"]).to(s["logits"].dtype)}


# ---------------------------------------------------------------- the package's operators
def _handles(tw, s):
    """What a program keeps between steps: output buffers, workspaces and the cache's handle."""
    if "kept" in s:
        return s["kept"]
    op, case = s["case"]["op"], s["case"]
    if op == "plan":
        kept = tw.alloc_kv_plan(s["lens"].numel(), s["tokens"], "cuda")
    elif op in ("append", "attn"):
        kept = {"cache": tw.KVCache(k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                    status=torch.zeros(4, dtype=torch.int32, device="cuda"))}
        if op == "attn":
            n, heads = s["q"].shape[0], case["q_heads"]
            kept["o"] = torch.empty((n, heads, case["dim"]), dtype=torch.bfloat16, device="cuda")
            kept["lse"] = torch.empty((n, heads), dtype=torch.float32, device="cuda")
            kept["workspace"] = torch.empty(
                tw.kv_attention_workspace_bytes(n, s["lens"].numel(), heads, case["kv_heads"], case["dim"]),
                dtype=torch.uint8, device="cuda")
    elif op == "logprobs":
        n, k = case["rows"], case["top"]
        kept = {name: torch.empty(n, dtype=torch.float32, device="cuda") for name in ("logprob", "entropy", "lse")}
        if k:
            kept["top_logprob"] = torch.empty((n, k), dtype=torch.float32, device="cuda")
            kept["top_index"] = torch.empty((n, k), dtype=torch.int32, device="cuda")
    else:
        kept = {"d_logits": torch.empty_like(s["logits"])}
    s["kept"] = kept
    return kept


def _own(s):
    import activation_sparse_transformer_gb300 as tw
    kept, case = _handles(tw, s), s["case"]
    if case["op"] == "plan":
        tw.twell_kv_plan(s["lens"], s["new"], s["table"], s["ring"], s["pool"], s["page"], kept)
        return {"kv_lens": kept.kv_lens, "cu_q": kept.cu_q, "slots": kept.slots, "positions": kept.positions,
                "pool": kept.pool, "table": s["table"], "ring": s["ring"]}
    if case["op"] == "append":
        tw.twell_kv_append(s["new_k"], s["new_v"], s["cu_q"], s["slots"], kept["cache"])
        return {name: s[name] for name in ("k", "k_scale", "v", "v_scale")}
    if case["op"] == "attn":
        tw.twell_kv_attention(s["q"], kept["cache"], s["table"], s["cu_q"], s["positions"], s["lens"],
                              case["max_len"], case["max_new"], s["softmax_scale"], kept["o"], kept["workspace"],
                              lse=kept["lse"])
        return {"o": kept["o"], "lse": kept["lse"]}
    if case["op"] == "logprobs":
        tw.twell_logprobs(s["logits"], s["targets"], s["inv_temperature"], kept["logprob"], kept["entropy"],
                          kept["lse"], kept.get("top_logprob"), kept.get("top_index"))
        return kept
    tw.twell_logprobs_bwd(s["logits"], s["targets"], s["inv_temperature"], s["lse"], s["entropy"], s["g_logprob"],
                          s["g_entropy"], kept["d_logits"])
    return kept


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn, "logprobs": _plain_logprobs,
            "logprobs_bwd": _plain_logprobs_bwd}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] in ("logprobs", "logprobs_bwd"):
        size, n = (2 if case["dtype"] == "bfloat16" else 4), case["rows"]
        passes = 1 if case["op"] == "logprobs" else 2
        return {"bytes": passes * size * n * case["vocab"] + n * (16 + 8 * case.get("top", 0)),
                "flops": 6 * n * case["vocab"]}
    old, new = _requests(case)
    need, _ = _blocks(case, old, new)
    add = np.maximum(new, 0)
    if case["op"] == "plan":
        fresh = int((need - -(-old // case["page"]))[new >= 0].sum())
        back = int((-(-old // case["page"]))[new < 0].sum())
        return {"bytes": 16 * len(old) + 8 * (fresh + back) + 12 * int(add.sum()), "flops": 0}
    if case["op"] == "append":
        pages = -(-(old + new) // case["page"]) - old // case["page"]
        each = case["heads"] * case["dim"]
        return {"bytes": int(add.sum()) * (2 * each * 3 + 8) + int(pages.sum()) * case["heads"] * 2 * 8,
                "flops": int(add.sum()) * each * 4}
    seen = sum(int((np.arange(a, a + b) + 1).sum()) for a, b in zip(old, add))  # cached tokens of all new ones
    cached = int((old + new)[new > 0].sum())
    pages = int(need[new > 0].sum())
    tokens = int(add.sum())
    return {"bytes": cached * case["kv_heads"] * case["dim"] * 2 + pages * (case["kv_heads"] * 8 + 4)
            + tokens * case["q_heads"] * (case["dim"] * 4 + 4),
            "flops": 4 * case["dim"] * case["q_heads"] * seen}


# ---------------------------------------------------------------- the definitions in 64 bits
def _e4m3_numpy(x):
    """The nearest value with 3 fraction bits, least exponent -6, ties to even, of float64 x."""
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -30))), -6) - 3)
    return np.clip(np.rint(x / step) * step, -448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None  # whole numbers
    if case["op"] == "append":
        most = 448.0 if case["fmt"] == "e4m3" else 127.0
        slots, page, out = s["slots"].cpu().numpy(), case["page"], {}
        for name in ("k", "v"):
            x = s["new_" + name].double().cpu().numpy()
            scale = s[name + "_scale"].double().cpu().numpy()
            codes = s[name].view(_codes_type(case["fmt"])).float().double().cpu().numpy()
            cut = np.flatnonzero(np.concatenate([[True], slots[1:] // page != slots[:-1] // page]))
            for a, b in zip(cut, np.append(cut[1:], len(slots))):
                p, at = slots[a] // page, slots[a] % page
                amax = np.maximum(np.abs(x[a:b]).max((0, 2)), 2.0 ** (MIN_EXP - 1))
                new = np.exp2(np.maximum(np.ceil(np.log2(amax / most)), MIN_EXP))
                now = np.maximum(new, scale[p]) if at else new
                rounded = _e4m3_numpy if case["fmt"] == "e4m3" else np.rint
                codes[p, :, :at] = rounded(codes[p, :, :at] * (scale[p] / now)[:, None, None])
                codes[p, :, at:at + b - a] = rounded((x[a:b] / now[None, :, None]).transpose(1, 0, 2))
                scale[p] = now
            out[name], out[name + "_scale"] = (codes if case["fmt"] == "e4m3" else None), scale
        return out
    if case["op"] == "attn":
        n, dim, heads = s["q"].shape[0], case["dim"], case["kv_heads"]
        group = case["q_heads"] // heads
        o = torch.zeros((n, case["q_heads"], dim), dtype=torch.float64, device="cuda")
        lse = torch.full((n, case["q_heads"]), float("-inf"), dtype=torch.float64, device="cuda")
        cu, lens, positions = s["cu_q"].tolist(), s["lens"].tolist(), s["positions"].tolist()
        if sum((b - a) * t for a, b, t in zip(cu, cu[1:], lens)) * case["q_heads"] * dim > 2e11:
            return None
        for r, length in enumerate(lens):
            seen = [min(p + 1, length) for p in positions[cu[r]:cu[r + 1]]]
            if not seen or max(seen) <= 0:
                continue
            pages = s["table"][r, :-(-length // case["page"])].long()
            for h in range(heads):
                k, v = ((s[w][pages, h].float().double() * s[w + "_scale"][pages, h].double()[:, None, None])
                        .reshape(-1, dim)[:length] for w in ("k", "v"))
                q = s["q"][cu[r]:cu[r + 1], h * group:(h + 1) * group].double()
                x = torch.einsum("tgd,jd->tgj", q, k) * s["softmax_scale"]
                seen_t = torch.tensor(seen, device="cuda")[:, None, None]
                x = x.masked_fill(torch.arange(length, device="cuda") >= seen_t, float("-inf"))
                lse[cu[r]:cu[r + 1], h * group:(h + 1) * group] = torch.logsumexp(x, -1)
                o[cu[r]:cu[r + 1], h * group:(h + 1) * group] = torch.einsum("tgj,jd->tgd", x.softmax(-1), v)
        o[torch.isnan(o)] = 0
        return {"o": o, "lse": lse}
    if case["rows"] * case["vocab"] > 1 << 28:
        return None
    x = s["logits"].double() * s["inv_temperature"]
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    entropy = lse - torch.where(p > 0, p * x, 0.0).sum(1)
    t = s["targets"].long()
    has = (t >= 0).double()
    if case["op"] == "logprobs":
        out = {"logprob": torch.where(t >= 0, x.gather(1, t.clamp(min=0)[:, None])[:, 0] - lse, 0.0),
               "entropy": entropy, "lse": lse}
        if case["top"]:
            out["top_logprob"] = torch.topk(x, case["top"], 1).values - lse[:, None]
            out["top_index"] = None
        return out
    # by the chain rule through the softmax: dL/dx = p * (w - <p, w>), w = dL/dlogp of each entry
    g, gh = s["g_logprob"].double() * has, s["g_entropy"].double()
    logp = x - lse[:, None]
    w = torch.where(p > 0, -gh[:, None] * (logp + 1), 0.0)
    d = p * (w - (p * w).sum(1, keepdim=True)) - g[:, None] * p
    d[torch.arange(len(t), device="cuda"), t.clamp(min=0)] += g
    return {"d_logits": d * s["inv_temperature"]}
