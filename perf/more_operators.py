"""Cases, plain forms and exact values of the softmax with a learned relative position bias and of
the 8-bit activation checkpoints.

``rel_fwd``: softmax of attention scores plus a bias that a table gives by the bucket of the distance
between key and query; ``rel_bwd``: its gradients for scores and table; ``rel_step``: both, the
probabilities between them kept in 8 bits; ``ckpt``: an activation kept in 8 bits and taken back;
``norm_bwd``: the LayerNorm's and RMSNorm's backward from an input kept in 8 bits.  ``own`` selects the
framework's calls; otherwise the operators are computed by elementary torch operations.

A checkpoint keeps each 32 columns of a row as integers of -127..127 and one power of two, the least
2^e for which the largest magnitude rounds to at most 127.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BLOCK = 32


def listed():
    return [
        # One request decoded: its token against the 1000 keys so far, in a cache of 1024.
        dict(name="rel_token", op="rel_fwd", dtype="bf16", B=1, H=16, Lq=1, Lk=1024, buckets=32, span=128, both=False, causal=False, ragged=True, masked=False, scale=0.125),
        # A decode step of 64 requests of different lengths in a cache of 4096.
        dict(name="rel_decode", op="rel_fwd", dtype="bf16", B=64, H=16, Lq=1, Lk=4096, buckets=32, span=128, both=False, causal=False, ragged=True, masked=False, scale=0.125),
        # An encoder's forward over a padded batch.
        dict(name="rel_encode", op="rel_fwd", dtype="bf16", B=16, H=12, Lq=512, Lk=512, buckets=32, span=128, both=True, causal=False, ragged=True, masked=False, scale=1.0),
        # Documents packed into rows of odd length, in fp32, kept apart by an additive mask.
        dict(name="rel_packed_odd", op="rel_fwd", dtype="f32", B=4, H=6, Lq=333, Lk=333, buckets=32, span=128, both=True, causal=False, ragged=False, masked=True, scale=0.125),
        # The encoder's backward.
        dict(name="relb_encode", op="rel_bwd", dtype="bf16", B=16, H=12, Lq=512, Lk=512, buckets=32, span=128, both=True, causal=False, ragged=True, masked=False, kept=False, scale=1.0),
        # A causal backward of odd length in fp32.
        dict(name="relb_f32_odd", op="rel_bwd", dtype="f32", B=2, H=8, Lq=501, Lk=501, buckets=64, span=256, both=False, causal=True, ragged=False, masked=False, kept=False, scale=0.125),
        # A long causal backward whose probabilities were kept in 8 bits.
        dict(name="relb_long_kept", op="rel_bwd", dtype="bf16", B=2, H=16, Lq=4096, Lk=4096, buckets=32, span=512, both=False, causal=True, ragged=False, masked=False, kept=True, scale=0.125),
        # A causal layer's forward and backward, the probabilities kept in 8 bits between them.
        dict(name="rel_step", op="rel_step", dtype="bf16", B=8, H=16, Lq=1024, Lk=1024, buckets=32, span=128, both=False, causal=True, ragged=False, masked=False, scale=0.125),
        # A hidden layer's activations of 8192 tokens, kept and taken back.
        dict(name="ckpt_hidden", op="ckpt", dtype="bf16", rows=8192, cols=4096),
        # fp32 rows of odd length.
        dict(name="ckpt_f32_odd", op="ckpt", dtype="f32", rows=1003, cols=1001),
        # The LayerNorm's backward at GPT-2's width.
        dict(name="ln_bwd_kept", op="norm_bwd", dtype="bf16", rows=8192, cols=768, rms=False),
        # The RMSNorm's backward over wide rows.
        dict(name="rms_bwd_kept", op="norm_bwd", dtype="bf16", rows=4096, cols=8192, rms=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rel_fwd", "rel_fwd", "rel_bwd", "rel_bwd", "rel_step", "ckpt", "norm_bwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("ckpt", "norm_bwd"):
        cols = _spread(rng, 32, 16384)
        if rng.random() < 0.6:
            cols = cols // 32 * 32
        rows = max(1, min(_spread(rng, 1, 65536), (1 << 27) // cols))
        case = dict(op=op, dtype=dtype, rows=rows, cols=cols)
        if op == "norm_bwd":
            case.update(rms=rng.random() < 0.5)
        return case
    H = rng.choice([1, 5, 6, 8, 12, 16, 20, 32])
    if op == "rel_fwd" and rng.random() < 0.35:  # single tokens against a cache
        Lq, Lk = rng.choice([1, 1, 1, 4]), _spread(rng, 16, 16384)
        B, causal, ragged = _spread(rng, 1, 256), Lq > 1, True
    else:
        Lk = _spread(rng, 16, 4096)
        if rng.random() < 0.6:
            Lk = max(16, Lk // 16 * 16)
        causal = rng.random() < 0.5
        Lq = Lk if causal or rng.random() < 0.7 else _spread(rng, 16, 2048)
        B, ragged = _spread(rng, 1, 32), not causal and rng.random() < 0.5
    H = max(1, min(H, (1 << 27) // (Lq * Lk)))
    B = max(1, min(B, (1 << 27) // (H * Lq * Lk)))
    both = not causal and rng.random() < 0.6
    buckets = rng.choice([16, 32, 32, 64])
    case = dict(op=op, dtype=dtype, B=B, H=H, Lq=Lq, Lk=Lk, buckets=buckets, span=rng.choice([64, 128, 128, 256, 800]), both=both,
                causal=causal, ragged=ragged, masked=op == "rel_fwd" and not ragged and rng.random() < 0.25, scale=rng.choice([1.0, 0.125, 0.0884]))
    if op == "rel_bwd":
        case.update(kept=rng.random() < 0.5)
    if op == "rel_step":
        case.update(dtype="bf16")
    return case


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# --- the checkpoint's format ------------------------------------------------------------


def _quantise(x):
    """(integers as int8 [rows, whole blocks], exponents + 127 as uint8 [rows, blocks]) of x [rows, cols]."""
    rows, cols = x.shape
    blocks = -(-cols // _BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, blocks * _BLOCK - cols)).view(rows, blocks, _BLOCK)
    largest = v.abs().amax(dim=2).view(torch.int32)
    k = (((largest + 0x10000) >> 23) - 6).clamp_(min=1)  # 127.5 / 128 of a power of two and more: the next one
    q = (v * ((254 - k) << 23).view(torch.float32)[:, :, None]).round().to(torch.int8)
    return q.view(rows, blocks * _BLOCK), k.to(torch.uint8)


def _values(q, k, cols):
    """fp32 [rows, cols] that a checkpoint stands for."""
    rows, blocks = k.shape
    step = (k.to(torch.int32) << 23).view(torch.float32)
    return (q.view(rows, blocks, _BLOCK) * step[:, :, None]).view(rows, blocks * _BLOCK)[:, :cols]


# --- positions, buckets and removed keys --------------------------------------------------


def _edges(buckets, span, both):
    """The distances at which a side's buckets 1, 2, ... begin: every distance has its own up to half of
    the side's buckets, then they grow by equal factors up to ``span``."""
    side = buckets // 2 if both else buckets
    near = side // 2
    far = side - near
    found, n = list(range(1, near + 1)), near
    for k in range(1, far):  # the least n with (n / near)^far >= (span / near)^k
        while n ** far * near ** k < span ** k * near ** far:
            n += 1
        found.append(n)
    return found


def _bucket(d, s):
    """Bucket of each distance d = key - query."""
    c = s["case"]
    n = d.abs() if c["both"] else (-d).clamp(min=0)
    found = (n[..., None] >= s["edges"]).sum(dim=-1)
    return found + (d > 0) * (c["buckets"] // 2) if c["both"] else found


def _positions(s):
    """Distance key - query, [B or 1, Lq, Lk]."""
    c = s["case"]
    at = torch.arange(c["Lq"], device="cuda")[None, :, None]
    if s["q_pos"] is not None:
        at = at + s["q_pos"].long()[:, None, None]
    return torch.arange(c["Lk"], device="cuda") - at


def _removed(s):
    """[B or 1, 1, Lq or 1, Lk], true where a key takes no part, or None."""
    c, gone = s["case"], None
    if c["causal"]:
        gone = (_positions(s) > 0)[:, None]
    if s["lens"] is not None:
        behind = torch.arange(c["Lk"], device="cuda") >= s["lens"][:, None, None, None]
        gone = behind if gone is None else gone | behind
    return gone


def _bias(s, table):
    """[B or 1, H, Lq, Lk] of the table's type."""
    d = _positions(s)
    lo, hi = 1 - s["case"]["Lq"] - s["furthest"], s["case"]["Lk"]
    by_distance = table[_bucket(torch.arange(lo, hi, device="cuda"), s)]
    return by_distance.t()[:, d - lo].transpose(0, 1)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    c, dt = case, _DTYPES[case["dtype"]]
    rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    if c["op"] in ("ckpt", "norm_bwd"):
        x = rnd(c["rows"], c["cols"])
        x[:, :: max(1, c["cols"] // 7)] *= 20  # the few columns of a residual stream that stand out
        if c["op"] == "ckpt":
            s["x"] = x.to(dt)
            return s
        s["q"], s["k"] = _quantise(x.to(dt))
        x = x.to(dt).float()
        if not c["rms"]:
            s["mean"] = x.mean(dim=1)
            x -= s["mean"][:, None]
        s["rstd"] = (x.square().mean(dim=1) + 1e-5).rsqrt()
        s["gamma"] = (1 + 0.1 * rnd(c["cols"])).to(dt)
        s["dy"] = rnd(c["rows"], c["cols"]).to(dt)
        return s
    B, H, Lq, Lk = c["B"], c["H"], c["Lq"], c["Lk"]
    s["table"] = (0.5 * rnd(c["buckets"], H)).to(dt)
    s["edges"] = torch.tensor(_edges(c["buckets"], c["span"], c["both"]), device="cuda")
    s["lens"] = s["q_pos"] = s["mask"] = None
    s["furthest"] = 0  # of the first query, as a program knows its cache's size
    if c["ragged"]:
        s["lens"] = torch.randint((3 * Lk + 3) // 4, Lk + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        if Lq < 16:  # the last tokens of each sequence
            s["lens"].clamp_(min=Lq)
            s["q_pos"], s["furthest"] = s["lens"] - Lq, Lk
    if c["masked"]:  # four documents
        cuts = torch.randint(1, Lk, (3,), generator=g, device="cuda")
        doc = (torch.arange(max(Lq, Lk), device="cuda")[:, None] >= cuts).sum(dim=1)
        s["mask"] = torch.where(doc[:Lq, None] == doc[:Lk], 0.0, -math.inf).to(dt)
    if c["op"] in ("rel_fwd", "rel_step"):
        s["x"] = (rnd(B, H, Lq, Lk) * (2.0 / c["scale"])).to(dt)
    if c["op"] == "rel_bwd":
        y = rnd(B, H, Lq, Lk).mul_(2.0)
        gone = _removed(s)
        if gone is not None:
            y.masked_fill_(gone, -math.inf)
        y = torch.softmax(y, dim=3).to(dt)
        if c["kept"]:
            s["q"], s["k"] = _quantise(y.view(-1, Lk))
        else:
            s["y"] = y
    if c["op"] != "rel_fwd":
        s["dy"] = rnd(B, H, Lq, Lk).to(dt)
    return s


def _pairs(c):
    """Scores that take part (those of padded batches about seven eighths of their keys)."""
    n = c["B"] * c["H"]
    if c["causal"]:
        per = sum(min(c["Lk"], i + 1) for i in range(c["Lq"])) if not c["ragged"] else c["Lq"] * c["Lk"] * 7 // 8
        return n * per
    return n * c["Lq"] * c["Lk"] * (7 if c["ragged"] else 8) // 8


def work(case):
    c, es = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "ckpt":  # read, kept; read back, written
        n = c["rows"] * c["cols"]
        return {"bytes": 2 * n * es + 2 * n + 2 * c["rows"] * -(-c["cols"] // _BLOCK), "flops": 4 * n}
    if c["op"] == "norm_bwd":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (2 * es + 1) + c["rows"] * (-(-c["cols"] // _BLOCK) + 4 + 4 * (not c["rms"])) + c["cols"] * es * (2 + (not c["rms"])), "flops": 12 * n}
    n, part = c["B"] * c["H"] * c["Lq"] * c["Lk"], _pairs(c)
    kept = 1 + 1 / _BLOCK
    table = c["buckets"] * c["H"] * es
    if c["op"] == "rel_fwd":
        return {"bytes": (part + n) * es + table + c["masked"] * c["Lq"] * c["Lk"] * es, "flops": 8 * part}
    back = part * (es + (kept if c.get("kept", True) else es)) + n * es + table
    if c["op"] == "rel_bwd":
        return {"bytes": back, "flops": 6 * part}
    return {"bytes": (part + n) * es + n * kept + table + back, "flops": 14 * part}


# --- the plain forms -----------------------------------------------------------------


def _plain_rel_fwd(s):
    c = s["case"]
    z = s["x"].float() * c["scale"] + _bias(s, s["table"].float())
    if s["mask"] is not None:
        z = z + s["mask"].float()
    gone = _removed(s)
    if gone is not None:
        z = z.masked_fill_(gone, -math.inf)
    m = z.amax(dim=3, keepdim=True)
    e = (z - torch.where(m == -math.inf, 0.0, m)).exp_()
    total = e.sum(dim=3, keepdim=True)
    return (e / torch.where(total == 0, 1.0, total)).to(s["x"].dtype)


def _plain_rel_bwd(s, y):
    """(gradient of the scores, of the table) for y in 32 bits."""
    c = s["case"]
    dy = s["dy"].float()
    ds = y * (dy - (dy * y).sum(dim=3, keepdim=True))
    # Every diagonal's sum: row i, taken in reverse, moved i columns to the right by its padding.
    Lq, Lk = c["Lq"], c["Lk"]
    d = torch.nn.functional.pad(ds.sum(dim=0).flip(1), (0, Lq)).flatten(1)[:, :Lq * (Lk + Lq - 1)]
    d = d.view(c["H"], Lq, Lk + Lq - 1).sum(dim=1, dtype=torch.float64)
    at = _bucket(torch.arange(1 - Lq, Lk, device="cuda"), s)
    dtable = torch.zeros(c["buckets"], c["H"], dtype=torch.float64, device="cuda").index_add_(0, at, d.t())
    return (ds * c["scale"]).to(s["dy"].dtype), dtable.to(s["dy"].dtype)


def _plain_norm_bwd(s):
    c, cols = s["case"], s["case"]["cols"]
    x = _values(s["q"], s["k"], cols)
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (x if c["rms"] else x - s["mean"][:, None]) * rstd
    g = dy * s["gamma"].float()
    inner = xhat * ((g * xhat).sum(dim=1, keepdim=True) / cols)
    if not c["rms"]:
        inner = inner + g.sum(dim=1, keepdim=True) / cols
    dx = ((g - inner) * rstd).to(s["dy"].dtype)
    sums = [(dy * xhat).sum(dim=0)] if c["rms"] else [(dy * xhat).sum(dim=0), dy.sum(dim=0)]
    return [dx] + [t.to(s["dy"].dtype) for t in sums]


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import layernorm_ln_fwd_gb300 as ln
        if op == "ckpt":
            return ln.ckpt8_load(ln.ckpt8_store(s["x"]), s["x"].dtype)
        if op == "norm_bwd":
            kept = ln.Ckpt8(s["q"], s["k"], c["cols"])
            if c["rms"]:
                return ln.rms_bwd_ckpt8(s["dy"], kept, s["gamma"], s["rstd"])
            return ln.bwd_ckpt8(s["dy"], kept, s["gamma"], s["mean"], s["rstd"])
        how = dict(max_distance=c["span"], bidirectional=c["both"], scale=c["scale"], causal=c["causal"], lens=s["lens"], q_pos=s["q_pos"])
        if op == "rel_fwd":
            return ln.softmax_rel_fwd(s["x"], s["table"], mask=s["mask"], **how)[0]
        if op == "rel_bwd":
            y = ln.Ckpt8(s["q"], s["k"], c["Lk"]) if c["kept"] else s["y"]
            return ln.softmax_rel_bwd(s["dy"], y, s["table"], **how)
        y, kept = ln.softmax_rel_fwd(s["x"], s["table"], ckpt=True, **how)
        return (y, *ln.softmax_rel_bwd(s["dy"], kept, s["table"], **how))
    if op == "ckpt":
        return _values(*_quantise(s["x"]), c["cols"]).to(s["x"].dtype)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    if op == "rel_fwd":
        return _plain_rel_fwd(s)
    shape = (c["B"], c["H"], c["Lq"], c["Lk"])
    if op == "rel_bwd":
        y = _values(s["q"], s["k"], c["Lk"]).view(shape) if c["kept"] else s["y"].float()
        return _plain_rel_bwd(s, y)
    y = _plain_rel_fwd(s)
    return (y, *_plain_rel_bwd(s, _values(*_quantise(y.view(-1, c["Lk"])), c["Lk"]).view(shape)))


# --- the definitions in 64 bits --------------------------------------------------------


def _power_of_two(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_kept(x):
    """What a checkpoint of x [rows, cols] gives back."""
    rows, cols = x.shape
    v = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, -1, 32)
    part, power = torch.frexp(v.abs().amax(dim=2, keepdim=True))  # part * 2^power, 0.5 <= part < 1
    e = torch.where(part * 128 < 127.5, power - 7, power - 6).clamp(min=-126)
    step = _power_of_two(e)
    return (torch.round(v / step) * step).view(rows, -1)[:, :cols]


def _exact_buckets(c):
    """{distance key - query: bucket}, each by its own comparison of whole numbers."""
    side = c["buckets"] // 2 if c["both"] else c["buckets"]
    near = side // 2
    far, found = side - near, {}
    for n in range(c["span"] + 1):
        if n < near:
            b = n
        else:
            k = 0
            while k < far - 1 and (n ** far) * near ** (k + 1) >= c["span"] ** (k + 1) * near ** far:
                k += 1
            b = near + k
        found[-n] = b
        if n:
            found[n] = side + b if c["both"] else 0
    return found


def _exact_bucket_of(d, c):
    found = _exact_buckets(c)
    at = torch.tensor([found[n] for n in range(-c["span"], c["span"] + 1)], device=d.device)
    return at[d.clamp(-c["span"], c["span"]) + c["span"]]


def _exact_rel_fwd(s, b):
    """Sequence b's probabilities, and the bucket of every pair."""
    c = s["case"]
    start = 0 if s["q_pos"] is None else int(s["q_pos"][b])
    q = torch.arange(c["Lq"], device="cuda")[:, None] + start
    k = torch.arange(c["Lk"], device="cuda")[None, :]
    bucket = _exact_bucket_of(k - q, c)
    out = torch.zeros(c["Lq"], c["Lk"], dtype=torch.bool, device="cuda")
    if c["causal"]:
        out |= k > q
    if s["lens"] is not None:
        out |= k >= s["lens"][b]
    if "x" not in s:
        return None, bucket
    z = s["x"][b].double() * c["scale"] + s["table"].double().t()[:, bucket]
    if s["mask"] is not None:
        z = z + s["mask"].double()
    z = z.masked_fill(out, -math.inf)
    return torch.nan_to_num(torch.softmax(z, dim=2), nan=0.0), bucket


def _exact_rel_bwd(s, b, y, bucket, dtable):
    c = s["case"]
    dy = s["dy"][b].double()
    ds = y * dy - y * (y * dy).sum(dim=2, keepdim=True)
    for h in range(c["H"]):
        dtable[:, h] += torch.bincount(bucket.flatten(), ds[h].flatten(), minlength=c["buckets"])
    return ds * c["scale"]


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "ckpt":
        return _exact_kept(s["x"].double())
    if op == "norm_bwd":
        step = _power_of_two(s["k"].int() - 127)
        x = (s["q"].double() * step.repeat_interleave(32, dim=1))[:, :c["cols"]]
        rstd, dy = s["rstd"].double()[:, None], s["dy"].double()
        xhat = x * rstd if c["rms"] else (x - s["mean"].double()[:, None]) * rstd
        g = dy * s["gamma"].double()
        dx = rstd * (g - xhat * (g * xhat).mean(dim=1, keepdim=True) - (0 if c["rms"] else g.mean(dim=1, keepdim=True)))
        return [dx, (dy * xhat).sum(dim=0)] + ([] if c["rms"] else [dy.sum(dim=0)])
    rows, cols = c["H"] * c["Lq"], c["Lk"]
    ys, dxs = [], []
    dtable = torch.zeros(c["buckets"], c["H"], dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        y, bucket = _exact_rel_fwd(s, b)
        if op == "rel_bwd":
            if c["kept"]:
                at = slice(b * rows, (b + 1) * rows)
                step = _power_of_two(s["k"][at].int() - 127)
                y = (s["q"][at].double() * step.repeat_interleave(32, dim=1))[:, :cols].reshape(c["H"], c["Lq"], cols)
            else:
                y = s["y"][b].double()
        if op != "rel_bwd":
            ys.append(y)
        if op == "rel_step":  # kept as it is stored, rounded to the scores' type
            y = _exact_kept(y.to(s["x"].dtype).double().view(-1, cols)).view(y.shape)
        if op != "rel_fwd":
            dxs.append(_exact_rel_bwd(s, b, y, bucket, dtable))
    if op == "rel_fwd":
        return torch.stack(ys)
    if op == "rel_bwd":
        return torch.stack(dxs), dtable
    return torch.stack(ys), torch.stack(dxs), dtable
