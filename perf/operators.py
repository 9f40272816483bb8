"""Cases, plain forms and exact values of the vocabulary operators.

``logprobs``: log probabilities of given tokens with entropy, log-sum-exp, rank and the top
alternatives; ``logprobs_bwd``: its gradient; ``distill``: the loss against a teacher's top
logits and its gradient in one call.  ``own`` selects the framework's calls; otherwise the
operators are computed by elementary torch operations in 32 bits.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One token decoded by a server that returns the 20 most likely alternatives.
        dict(name="lp_token", op="logprobs", dtype="bf16", rows=1, V=131072, ld=131072, top=20, ranks=True, scale=1.0),
        # A decode step of 64 requests, the same options, sampled at temperature 0.8.
        dict(name="lp_step", op="logprobs", dtype="bf16", rows=64, V=131072, ld=131072, top=20, ranks=True, scale=1.25),
        # A policy update's forward: the chosen tokens' log probabilities and the entropy over
        # GPT-2's 50257 words in rows padded to 50304.
        dict(name="lp_policy", op="logprobs", dtype="bf16", rows=4096, V=50257, ld=50304, top=0, ranks=False, scale=1.0),
        # A teacher writes down the 64 largest logits of every position.
        dict(name="lp_teacher", op="logprobs", dtype="bf16", rows=2048, V=131072, ld=131072, top=64, ranks=False, scale=1.0),
        # Evaluation in fp32 over an odd vocabulary.
        dict(name="lp_f32_odd", op="logprobs", dtype="f32", rows=333, V=32001, ld=32001, top=5, ranks=True, scale=1.0),
        # The policy update's backward, with an entropy bonus.
        dict(name="lpb_policy", op="logprobs_bwd", dtype="bf16", rows=4096, V=50257, ld=50304, entropy=True, scale=1.0),
        # A small batch's backward in fp32, rows of odd length one after another.
        dict(name="lpb_f32_odd", op="logprobs_bwd", dtype="f32", rows=200, V=50257, ld=50257, entropy=False, scale=0.5),
        # A distillation step of 8 x 1024 tokens over GPT-2's padded vocabulary.
        dict(name="ds_train", op="distill", dtype="bf16", rows=8192, V=50304, ld=50304, K=64, masked=0.0, scale=1.0),
        # Instruction tuning: the first quarter of the positions is the prompt, of weight 0.
        dict(name="ds_masked", op="distill", dtype="bf16", rows=1024, V=131072, ld=131072, K=128, masked=0.25, scale=0.5),
        # fp32 logits of an odd vocabulary.
        dict(name="ds_f32_odd", op="distill", dtype="f32", rows=130, V=32001, ld=32001, K=17, masked=0.0, scale=1.0),
        # A handful of positions: the smallest distillation call.
        dict(name="ds_small", op="distill", dtype="bf16", rows=8, V=50257, ld=50257, K=8, masked=0.0, scale=1.0),
        # On-line distillation: the teacher's top 32 go straight into the student's loss.
        dict(name="teach", op="chain", dtype="bf16", rows=512, V=65536, ld=65536, K=32, scale=0.5),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_bwd", "distill", "distill", "chain"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    V = _spread(rng, 256, 262144)
    if rng.random() < 0.5:
        V = max(256, V // 64 * 64)
    ld = V if rng.random() < 0.6 else V + rng.choice([1, 7, 47, 64])
    rows = max(1, min(_spread(rng, 1, 8192), (1 << 28) // V // (2 if op == "chain" else 1)))
    case = dict(op=op, dtype=dtype, rows=rows, V=V, ld=ld, scale=round(rng.uniform(0.3, 1.5), 3))
    if op == "logprobs":
        case.update(top=rng.choice([0, 1, _spread(rng, 2, 256), _spread(rng, 2, 64)]), ranks=rng.random() < 0.5)
    elif op == "logprobs_bwd":
        case.update(entropy=rng.random() < 0.5)
    elif op == "distill":
        case.update(K=_spread(rng, 1, 256), masked=rng.choice([0.0, 0.0, 0.25, 0.6]))
    else:
        case.update(K=_spread(rng, 1, 256))
    return case


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _distinct(rows, V, n, g):
    """[rows, n] distinct words a row, in no order: one from each n-th of the vocabulary."""
    start = torch.arange(n, device="cuda") * V // n
    ids = start + (torch.rand(rows, n, generator=g, device="cuda") * (V // n)).long().clamp_(max=V // n - 1)
    return ids.gather(1, torch.rand(rows, n, generator=g, device="cuda").argsort(dim=1))


def _logits(case, g, ids=None, peaks=None):
    """[rows, V] logits in rows of ld values: N(0, 2) with a few likely words a row standing out."""
    rows, V, ld = case["rows"], case["V"], case["ld"]
    x = torch.empty(rows, ld, dtype=_DTYPES[case["dtype"]], device="cuda")
    x.normal_(0.0, 2.0, generator=g)
    if ids is None:
        ids = _distinct(rows, V, 16, g)
        peaks = 4.0 + 6.0 * torch.rand(rows, 16, generator=g, device="cuda")
    x.scatter_(1, ids, peaks.to(x.dtype))
    return x[:, :V], ids


def _tokens(case, g, ids):
    """Half of them likely words, half any word."""
    rows = case["rows"]
    any_word = torch.randint(0, case["V"], (rows,), generator=g, device="cuda")
    likely = torch.rand(rows, generator=g, device="cuda") < 0.5
    return torch.where(likely, ids[:, 0], any_word).to(torch.int32)


def _teacher(case, g):
    """Distinct words in no order, their logits falling along the list; some lists are shorter."""
    rows, V, K = case["rows"], case["V"], case["K"]
    ids = _distinct(rows, V, K, g)
    fall = 9.0 - 1.2 * torch.arange(1, K + 1, device="cuda", dtype=torch.float32).log()
    t = fall + 0.5 * torch.randn(rows, K, generator=g, device="cuda")
    length = torch.randint((K + 1) // 2, K + 1, (rows, 1), generator=g, device="cuda")
    t, _ = t.sort(dim=1, descending=True)
    kept = torch.arange(K, device="cuda") < length
    return ids, torch.where(kept, ids, -1).to(torch.int32), t


def _rows_at_a_time(V):
    return max(1, (1 << 26) // V)


def _lse_entropy64(x, scale):
    """(lse, entropy) in 64 bits, a few rows at a time."""
    lse, ent = [], []
    for part in x.split(_rows_at_a_time(x.shape[1])):
        z = part.double() * scale
        l = torch.logsumexp(z, dim=1)
        logq = z - l[:, None]
        lse.append(l)
        ent.append(-(logq.exp() * logq).sum(dim=1))
    return torch.cat(lse), torch.cat(ent)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    op, rows = case["op"], case["rows"]
    if op in ("logprobs", "logprobs_bwd"):
        s["x"], ids = _logits(case, g)
        s["tokens"] = _tokens(case, g, ids)
        if op == "logprobs_bwd":  # what the forward left, and the upstream gradients
            lse, ent = _lse_entropy64(s["x"], case["scale"])
            s["lse"], s["ent"] = lse.float(), ent.float()
            s["dlogp"] = torch.randn(rows, generator=g, device="cuda") / rows
            s["dent"] = -0.01 * torch.rand(rows, generator=g, device="cuda") / rows if case["entropy"] else None
    elif op == "distill":
        at, s["ids"], s["t"] = _teacher(case, g)
        peaks = s["t"] + 0.7 * torch.randn(rows, case["K"], generator=g, device="cuda")
        s["x"], _ = _logits(case, g, at, peaks)
        s["w"] = (torch.arange(rows, device="cuda") >= int(case["masked"] * rows)).float() if case["masked"] else None
    else:
        s["teacher"], ids = _logits(case, g)
        peaks = s["teacher"].gather(1, ids).float() + 0.7 * torch.randn(ids.shape, generator=g, device="cuda")
        s["x"], _ = _logits(case, g, ids, peaks)
    return s


def work(case):
    rows, V, es = case["rows"], case["V"], 2 if case["dtype"] == "bf16" else 4
    n = rows * V
    if case["op"] == "logprobs":
        return {"bytes": n * es + rows * (4 + 12 + 4 * case["ranks"] + 8 * case["top"]), "flops": 8 * n}
    if case["op"] == "logprobs_bwd":
        return {"bytes": 2 * n * es + rows * (12 + 8 * case["entropy"]), "flops": 8 * n}
    if case["op"] == "distill":
        read = rows - int(case["masked"] * rows)
        return {"bytes": (read * V + n) * es + rows * 4 + read * 8 * case["K"] + rows * 4 * bool(case["masked"]), "flops": 8 * read * V}
    return {"bytes": 3 * n * es + rows * (8 + 16 * case["K"]), "flops": 16 * n}


# --- the plain forms -----------------------------------------------------------------


def _plain_logprobs(x, tokens, scale, top, ranks, entropy=True):
    z = x.float() * scale
    m = z.amax(dim=1, keepdim=True)
    d = z - m
    e = d.exp()
    total = e.sum(dim=1, keepdim=True)
    log_total = total.log()
    out = {"lse": (m + log_total)[:, 0]}
    if entropy:
        out["entropy"] = log_total[:, 0] - (e * torch.where(e > 0, d, 0.0)).sum(dim=1) / total[:, 0]
    if tokens is not None:
        at = tokens.long()[:, None]
        out["logp"] = (d.gather(1, at) - log_total)[:, 0]
        if ranks:
            out["ranks"] = ((x > x.gather(1, at)).sum(dim=1) + 1).to(torch.int32)
    if top:
        bits = (x.float() + 0.0).view(torch.int32).long()  # keys in the order of the values, ties by the lowest index
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 32) - torch.arange(x.shape[1], device=x.device)
        ids = key.topk(top, dim=1).indices
        out["top_ids"] = ids.to(torch.int32)
        out["top_logp"] = d.gather(1, ids) - log_total
    return out


def _plain_logprobs_bwd(x, tokens, lse, ent, dlogp, dent, scale):
    logq = x.float() * scale - lse[:, None]
    q = logq.exp()
    g = -dlogp[:, None] * q
    if dent is not None:
        g = g - dent[:, None] * q * (torch.where(q > 0, logq, 0.0) + ent[:, None])
    g.scatter_add_(1, tokens.long()[:, None], dlogp[:, None])
    return (g * scale).to(x.dtype)


def _plain_distill(x, ids, t, w, scale, dloss):
    kept = ids >= 0
    at = ids.long().clamp(min=0)
    u = torch.where(kept, t * scale, -math.inf)
    u = u - u.amax(dim=1, keepdim=True)
    pe = u.exp()
    ps = pe.sum(dim=1, keepdim=True)
    p = pe / ps
    d = x.float() * scale
    d = d - d.amax(dim=1, keepdim=True)
    e = d.exp()
    total = e.sum(dim=1, keepdim=True)
    logp = torch.where(kept, u - ps.log(), 0.0)
    losses = (p * (logp - (d.gather(1, at) - total.log()))).sum(dim=1)
    g = (e / total).scatter_add_(1, at, -p) * (scale * dloss)
    if w is not None:
        losses = torch.where(w != 0, losses * w, 0.0)
        g = torch.where(w[:, None] != 0, g * w[:, None], 0.0)
    return losses, g.to(x.dtype)


def run(s):
    c = s["case"]
    op, scale = c["op"], c["scale"]
    if op == "logprobs":
        if own:
            import layernorm_ln_fwd_gb300 as ln
            logp, entropy, lse, ranks, top_ids, top_logp = ln.logprobs(s["x"], s["tokens"], scale, top=c["top"], want_ranks=c["ranks"])
            out = {"lse": lse, "entropy": entropy, "logp": logp}
            if c["ranks"]:
                out["ranks"] = ranks
            if c["top"]:
                out["top_ids"], out["top_logp"] = top_ids, top_logp
            return out
        return _plain_logprobs(s["x"], s["tokens"], scale, c["top"], c["ranks"])
    if op == "logprobs_bwd":
        if own:
            import layernorm_ln_fwd_gb300 as ln
            return ln.logprobs_bwd(s["x"], s["tokens"], s["lse"], s["ent"], s["dlogp"], s["dent"], scale)
        return _plain_logprobs_bwd(s["x"], s["tokens"], s["lse"], s["ent"], s["dlogp"], s["dent"], scale)
    dloss = 1.0 / c["rows"]
    if op == "distill":
        if own:
            import layernorm_ln_fwd_gb300 as ln
            return ln.distill(s["x"], s["ids"], s["t"], s["w"], scale, dloss)
        return _plain_distill(s["x"], s["ids"], s["t"], s["w"], scale, dloss)
    if own:
        import layernorm_ln_fwd_gb300 as ln
        _, _, _, _, ids, t = ln.logprobs(s["teacher"], top=c["K"], want_entropy=False)
        return (*ln.distill(s["x"], ids, t, None, scale, dloss), ids)
    teacher = _plain_logprobs(s["teacher"], None, 1.0, c["K"], False, entropy=False)
    return (*_plain_distill(s["x"], teacher["top_ids"], teacher["top_logp"], None, scale, dloss), teacher["top_ids"])


# --- the definitions in 64 bits --------------------------------------------------------


def _exact_distill(x, ids, t, w, scale, dloss):
    losses, grads = [], []
    n = _rows_at_a_time(x.shape[1])
    for r in range(0, x.shape[0], n):
        xr, ir, tr = x[r:r + n].double() * scale, ids[r:r + n].long(), t[r:r + n].double() * scale
        log_p = torch.log_softmax(torch.where(ir >= 0, tr, -math.inf), dim=1)
        p = log_p.exp()
        log_q = torch.log_softmax(xr, dim=1)
        at = torch.where(ir >= 0, ir, 0)
        loss = torch.where(p > 0, p * (log_p - log_q.gather(1, at)), 0.0).sum(dim=1)
        dense = torch.zeros_like(xr).scatter_add(1, at, p)
        grad = (log_q.exp() - dense) * (dloss * scale)
        if w is not None:
            loss, grad = loss * w[r:r + n].double(), grad * w[r:r + n, None].double()
        losses.append(loss)
        grads.append(grad)
    return torch.cat(losses), torch.cat(grads)


def exact(case, seed):
    s = prepare(case, seed)
    op, scale, x = case["op"], case["scale"], s["x"]
    if op == "logprobs":
        lse, ent = _lse_entropy64(x, scale)
        at = s["tokens"].long()[:, None]
        out = {"lse": lse, "entropy": ent, "logp": x.gather(1, at)[:, 0].double() * scale - lse}
        if case["ranks"]:
            out["ranks"] = None
        if case["top"]:
            out["top_ids"] = None
            out["top_logp"] = x.topk(case["top"], dim=1).values.double() * scale - lse[:, None]
        return out
    if op == "logprobs_bwd":
        grads = []
        n = _rows_at_a_time(x.shape[1])
        for r in range(0, x.shape[0], n):
            log_q = torch.log_softmax(x[r:r + n].double() * scale, dim=1)
            q = log_q.exp()
            dlogp = s["dlogp"][r:r + n, None].double()
            g = -dlogp * q
            if s["dent"] is not None:
                g = g - s["dent"][r:r + n, None].double() * q * (log_q - (q * log_q).sum(dim=1, keepdim=True))
            at = s["tokens"][r:r + n].long()[:, None]
            grads.append(g.scatter_add(1, at, dlogp) * scale)
        return torch.cat(grads)
    dloss = 1.0 / case["rows"]
    if op == "distill":
        return _exact_distill(x, s["ids"], s["t"], s["w"], scale, dloss)
    values, ids = s["teacher"].float().sort(dim=1, descending=True, stable=True)
    values, ids = values[:, :case["K"]].double(), ids[:, :case["K"]]
    return (*_exact_distill(x, ids, values, None, scale, dloss), None)
