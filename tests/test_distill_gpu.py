"""Distillation from a teacher's top logits (distill) on the GPU against the float64 oracle:
losses and gradients over odd sizes and alignments, short, empty and repeated entries, weights,
masks, in place, and a run of the operators over logits together.  Tolerances: vocabref.py."""
import numpy as np
import pytest
import torch

import layernorm_ln_fwd_gb300 as ln
import oracle
import vocabref as R

pytestmark = pytest.mark.gpu


def teacher_of(rows, V, K, seed, short=True, repeat=False):
    """ids [rows, K] (different columns unless `repeat`), teacher logits, some lists short."""
    g = torch.Generator().manual_seed(seed + 5)
    if repeat or K > V:
        ids = torch.randint(0, V, (rows, K), generator=g)
    else:
        ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(rows)])
    if short and K > 1:
        cut = torch.randint(1, K + 1, (rows, 1), generator=g)
        ids = torch.where(torch.arange(K) < cut, ids, -1)
    t = 2 * torch.randn(rows, K, generator=g)
    return ids.to(torch.int32).cuda(), t.cuda()


def check(x, ids, t, w=None, scale=1.0, dloss=1.0, dtype="f32", **kw):
    x64 = R.to64(x)
    losses, dx = ln.distill(x, ids, t, w, scale, dloss, **kw)
    torch.cuda.synchronize()
    scale, dloss = R.f32(scale), R.f32(dloss)
    wn = None if w is None else R.to64(w)
    ref = oracle.distill(x64, ids.cpu().numpy(), R.to64(t), wn, scale, dloss)
    tl, tg = R.tol_distill(x64, ids.cpu().numpy(), R.to64(t), np.ones(len(x64)) if wn is None else wn,
                           scale, dloss, ref, dtype)
    if losses is not None:
        R.close("loss", R.to64(losses), ref["loss"], tl)
    if dx is not None:
        R.close("gradient", R.to64(dx), ref["dx"], tg)
    return losses, dx


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 255, 1000, 1001, 4097, 50257, 50304])
@pytest.mark.parametrize("K", [1, 5, 64, 256])
def test_widths(dtype, V, K):
    rows = 6
    check(R.logits(rows, V, dtype, V + K), *teacher_of(rows, V, K, V), scale=0.7, dloss=0.3, dtype=dtype)


@pytest.mark.parametrize("dtype,V", [("bf16", 131072), ("f32", 131072), ("f32", 262147), ("bf16", 262144),
                                     ("bf16", 1 << 20), ("f32", 1 << 21)])
@pytest.mark.parametrize("rows", [1, 3])
def test_long_rows(dtype, V, rows):
    check(R.logits(rows, V, dtype, V), *teacher_of(rows, V, 33, V), dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 19, 151, 153, 305, 700])
def test_row_counts(dtype, rows):
    g = torch.Generator().manual_seed(rows)
    w = torch.rand(rows, generator=g)
    w[::3] = 0
    check(R.logits(rows, 2049, dtype, rows), *teacher_of(rows, 2049, 16, rows), w=w.cuda(), dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", range(0, 9))
@pytest.mark.parametrize("ld", [1003, 1008, 1011])
def test_alignments_and_row_distances(dtype, offset, ld):
    x = R.logits(5, 1003, dtype, offset, ld=ld, offset=offset)
    ids, t = teacher_of(5, 1003, 9, offset)
    _, a = check(x, ids, t, dtype=dtype)
    buf = torch.full((5 * 1013 + 5,), 7.0, dtype=x.dtype, device="cuda")
    out = buf[5:].view(5, 1013)[:, :1003]
    _, b = ln.distill(x, ids, t, dlogits=out)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and (buf[5:].view(5, 1013)[:, 1003:] == 7).all() and (buf[:5] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,K", [(3, 40), (50, 256), (1000, 200)])
def test_repeated_columns(dtype, V, K):
    check(R.logits(8, V, dtype, V), *teacher_of(8, V, K, 3, repeat=True), dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place(dtype):
    for V, ld in ((5000, 5000), (1003, 1024), (50257, 50257), (131072, 131072)):
        x = R.logits(9, V, dtype, V, ld=ld)
        ids, t = teacher_of(9, V, 20, V)
        la, a = ln.distill(x, ids, t, scale=0.5)
        lb, b = ln.distill(x, ids, t, scale=0.5, in_place=True)
        torch.cuda.synchronize()
        assert b.data_ptr() == x.data_ptr() and torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("dtype,rows,V,K", [("bf16", 700, 20003, 40), ("f32", 500, 10007, 70), ("bf16", 200, 50304, 256),
                                            ("bf16", 340, 66001, 9)])
def test_many_rows_of_all_kinds(dtype, rows, V, K):
    """Blocks that take several rows each: rows of weight 0 and without entries, one after another and
    between others, short lists, repeated columns and a column outside the row, next to each other."""
    x = R.logits(rows, V, dtype, V)
    ids, t = teacher_of(rows, V, K, V)
    g = torch.Generator().manual_seed(V)
    kind = torch.randint(0, 7, (rows,), generator=g).cuda()
    w = torch.where(kind == 0, 0.0, torch.rand(rows, generator=g).cuda() + 0.5)
    w[rows // 3: rows // 2] = 0
    ids[kind == 1] = -1
    t[kind == 2] = -float("inf")
    twice = kind == 3
    ids[twice, K // 2:] = ids[twice, : K - K // 2]
    ids[kind == 4, -1] = ids[kind == 4, 0]
    ids[(kind == 5) & (torch.arange(rows).cuda() % 5 == 0), 0] = V
    check(x, ids, t, w, scale=0.6, dtype=dtype)


@pytest.mark.parametrize("V,rows", [(1000, 5), (5000, 5), (50304, 200), (131072, 3)])
@pytest.mark.parametrize("step", [256, 1024, 2048])
def test_columns_at_equal_distances(V, rows, step):
    """Lists whose columns meet in a table by their low bits, if it goes by those."""
    K = min(200, V // step)
    ids = (torch.arange(K) * step).flip(0).repeat(rows, 1).to(torch.int32).cuda()
    t = torch.randn(rows, K, generator=torch.Generator().manual_seed(V)).cuda()
    check(R.logits(rows, V, "bf16", V), ids, t, dtype="bf16") if K else None


@pytest.mark.parametrize("dtype,V,rows", [("bf16", 131072, 160), ("bf16", 65537, 333), ("f32", 150001, 80),
                                          ("f32", 262144, 155)])
def test_wide_rows_of_a_batch_in_place(dtype, V, rows):
    """Rows that do not fit a block's shared memory whole, in place and not, against torch in 64 bits."""
    x = R.logits(rows, V, dtype, rows)
    g = torch.Generator().manual_seed(V)
    ids = (torch.randint(0, V // 12, (rows, 12), generator=g) * 12 + torch.arange(12)).to(torch.int32).cuda()
    t = torch.randn(rows, 12, generator=g).cuda()
    la, a = ln.distill(x, ids, t, dloss=1.0 / rows)
    full = x.clone()
    lb, b = ln.distill(full, ids, t, dloss=1.0 / rows, in_place=True)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb) and b.data_ptr() == full.data_ptr()
    for r in (0, 1, rows // 2, rows - 1):
        xr = x[r].double()
        p = torch.softmax(t[r].double(), 0)
        lq = torch.log_softmax(xr, 0)
        want = (p * (p.log() - lq[ids[r].long()])).sum()
        grad = (lq.exp().index_add(0, ids[r].long(), -p)) / rows
        # the entropy of such a row is ~10: E of vocabref.py with A = 12 and a chain of V / 256
        E = R.U * (136 + V / 256)
        assert abs(la[r].double() - want) <= E + 400 * R.U
        err = (a[r].double() - grad).abs()
        assert (err <= R.HALF[dtype] * grad.abs() + (lq.exp() + 1e-3) * (E + 100 * R.U) / rows + 1e-30).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_teach_nothing(dtype):
    V = 700
    x = R.logits(7, V, dtype, 3)
    x[:4] = float("nan")  # not read
    ids, t = teacher_of(7, V, 8, 3, short=False)
    ids[0] = -1
    t[1] = -float("inf")
    w = torch.ones(7, device="cuda")
    w[2:4] = 0
    t[4, 2] = -float("inf")  # weight 0 within a list
    t[5, :] = float("nan")
    ids[5, :] = -5  # what stands at no entry is not looked at
    losses, dx = check(x[4:], ids[4:], t[4:], w[4:], dtype=dtype)
    losses, dx = ln.distill(x, ids, t, w)
    torch.cuda.synchronize()
    assert (losses[:4] == 0).all() and (dx[:4] == 0).all() and losses[5] == 0 and (dx[5] == 0).all()
    assert torch.isfinite(dx).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [60, 50257])
def test_masked_students(dtype, V):
    x = R.logits(4, V, dtype, 5)
    ids, t = teacher_of(4, V, 6, 5, short=False)
    x[0, V // 2:] = -float("inf")
    x[1] = torch.finfo(x.dtype).min
    x[1, ids[1, 0].item()] = 1.0
    x[2, ids[2, 3].item()] = -float("inf")  # a teacher's word the student has removed
    x[3, ids[3, 3].item()] = -float("inf")  # ... which has no weight
    t[3, 3] = -float("inf")
    ids[0] = ids[0] % (V // 2)
    ids[0, 1:] = torch.where(ids[0, 1:] == ids[0, :1], -1, ids[0, 1:])
    losses, dx = check(x, ids, t, dtype=dtype)
    assert torch.isinf(losses[2]) and torch.isfinite(losses[[0, 1, 3]]).all() and torch.isfinite(dx).all()


def test_rows_without_a_distribution():
    x = R.logits(5, 90, "f32", 6)
    ids, t = teacher_of(5, 90, 4, 6, short=False)
    x[1] = -float("inf")
    x[2, 3] = float("nan")
    ids[3, 2] = 90
    ids[4, 0] = 2**31 - 1
    losses, dx = ln.distill(x, ids, t)
    torch.cuda.synchronize()
    assert torch.isnan(losses[1:]).all() and torch.isfinite(losses[0])
    assert torch.isnan(dx[2:]).all() and torch.isfinite(dx[0]).all() and torch.isnan(dx[1]).any()


def test_losses_or_gradient_alone_and_repeatable():
    x = R.logits(40, 50304, "bf16", 7)
    ids, t = teacher_of(40, 50304, 64, 7)
    a = ln.distill(x, ids, t)
    b = ln.distill(x, ids, t, want_grad=False)
    c = ln.distill(x, ids, t, want_losses=False)
    torch.cuda.synchronize()
    assert b[1] is None and c[0] is None and torch.equal(a[0], b[0]) and torch.equal(a[1], c[1])
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d = ln.distill(x, ids, t, losses=torch.empty(40, device="cuda"), dlogits=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):  # at once: a graph, an eager call, another stream
        g.replay()
        e = ln.distill(x, ids, t)
        f = ln.distill(x, ids, t, stream=s)
    torch.cuda.synchronize()
    for o in (d, e, f):
        assert torch.equal(o[0], a[0]) and torch.equal(o[1], a[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_teacher_to_student_to_policy(dtype):
    """The operators together: a teacher's alternatives go into the student's loss; the gradient is
    autograd's; then the student's token log probabilities and their gradient."""
    rows, V, K, scale = 12, 3001, 24, 0.5
    teacher, student = R.logits(rows, V, dtype, 1), R.logits(rows, V, dtype, 2)
    _, _, _, _, ids, lp = ln.logprobs(teacher, top=K, want_entropy=False)
    losses, dx = check(student, ids, lp, scale=scale, dloss=1.0 / rows, dtype=dtype)
    xs = student.double().requires_grad_()
    tk = teacher.double().topk(K, dim=1)
    p = torch.softmax(tk.values * scale, dim=1)
    logq = torch.log_softmax(xs * scale, dim=1).gather(1, tk.indices)
    kl = (p * (p.log() - logq)).sum(dim=1)
    kl.mean().backward()
    # a column that ties with the K-th largest may be another one there: such rows are left out
    same = (tk.indices.sort(1).values == ids.long().sort(1).values).all(dim=1)
    assert same.any()
    # the loss sums 24 terms of up to ~10 in fp32
    assert (losses.double() - kl.detach()).abs()[same].max() < 1e-4
    err = (dx.double() - xs.grad).abs()[same]
    assert (err <= R.HALF[dtype] * xs.grad.abs()[same] + 1e-5 / rows).all()
    logp, ent, lse, ranks, top_ids, _ = ln.logprobs(student, ids[:, 0].contiguous(), top=K, want_ranks=True)
    place = (top_ids == ids[:, :1])
    r = ranks.long()
    torch.cuda.synchronize()
    # the token's rank is its place among the alternatives, ties before it aside
    for i in range(rows):
        if place[i].any():
            assert r[i].item() <= place[i].nonzero()[0, 0].item() + 1
    one = torch.full((rows,), -1.0, device="cuda")
    g = ln.logprobs_bwd(student, ids[:, 0].contiguous(), lse, dlogp=one)
    hard, _ = ln.distill(student, ids[:, :1].contiguous(), lp[:, :1].contiguous(), want_grad=False)
    _, gh = ln.distill(student, ids[:, :1].contiguous(), lp[:, :1].contiguous())
    xl, xg = ln.xent(student, ids[:, 0].contiguous())
    torch.cuda.synchronize()
    # one entry is the cross-entropy, and minus the token's log probability
    assert (hard + logp).abs().max() < 2e-5 and (hard - xl).abs().max() < 2e-5
    step = 2 * R.HALF[dtype] * xg.float().abs() + 2e-6
    assert ((g.float() - xg.float()).abs() <= step).all() and ((gh.float() - xg.float()).abs() <= step).all()


def test_operators_in_a_captured_chain():
    """Teacher to student to policy, captured once and replayed on new logits, the same as eager calls."""
    rows, V, K = 60, 40001, 20
    teacher, student = R.logits(rows, V, "bf16", 1), R.logits(rows, V, "bf16", 2)
    dl = torch.full((rows,), -1.0 / rows, device="cuda")

    def chain():
        _, _, _, _, ids, lp = ln.logprobs(teacher, top=K, want_entropy=False)
        losses, dx = ln.distill(student, ids, lp, scale=0.5)
        tok = ids[:, 0].contiguous()
        logp, ent, lse, ranks, _, _ = ln.logprobs(student, tok, want_ranks=True)
        return losses, dx, logp, ent, ranks, ln.logprobs_bwd(student, tok, lse, ent, dl, dl)

    chain()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = chain()
    for seed in (3, 4):
        teacher.copy_(R.logits(rows, V, "bf16", seed))
        student.copy_(R.logits(rows, V, "bf16", seed + 10))
        for _ in range(5):
            g.replay()
        eager = chain()
        torch.cuda.synchronize()
        for u, v in zip(out, eager):
            assert torch.equal(u, v)
    assert ln.device_check() == 0


def test_refusals():
    x = R.logits(4, 16, "f32", 1)
    ids, t = teacher_of(4, 16, 3, 1)
    f = torch.zeros(4, device="cuda")
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(dloss=float("inf")),
               dict(want_losses=False, want_grad=False)):
        with pytest.raises(ln.LnError):
            ln.distill(x, ids, t, **kw)
    many = torch.zeros(4, 257, dtype=torch.int32, device="cuda")
    with pytest.raises(ln.LnError):
        ln.distill(x, many, many.float())
    with pytest.raises(ln.LnError):
        ln.distill(x, ids[:, :0], t[:, :0])
    with pytest.raises(TypeError):
        ln.distill(x, ids.long(), t)
    with pytest.raises(TypeError):
        ln.distill(x, ids, t.double())
    for call in (lambda: ln.distill(x, ids[:3], t), lambda: ln.distill(x, ids, t[:, :2]),
                 lambda: ln.distill(x, ids[0], t[0]), lambda: ln.distill(x.t(), ids, t),
                 lambda: ln.distill(x, ids, t, f[:2]), lambda: ln.distill(x, ids.cpu(), t),
                 lambda: ln.distill(x, ids, t, dlogits=x[:3])):
        with pytest.raises(ValueError):
            call()
    l, g = ln.distill(x[:0], ids[:0], t[:0])
    assert l.shape == (0,) and g.shape == (0, 16)
