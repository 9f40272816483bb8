"""Token log probabilities (logprobs) and their gradient (logprobs_bwd) on the GPU against the
float64 oracle: sizes from one word to a long vocabulary, odd lengths and row distances, every
alignment, ties, masks, rows without a distribution, the selection of the top among rows made
against it, and the calls' refusals.  Tolerances: vocabref.py."""
import numpy as np
import pytest
import torch

import layernorm_ln_fwd_gb300 as ln
import oracle
import vocabref as R

pytestmark = pytest.mark.gpu


def tokens_of(rows, V, seed):
    g = torch.Generator().manual_seed(seed + 77)
    return torch.randint(0, V, (rows,), generator=g, dtype=torch.int32).cuda()


def run(x, t, scale=1.0, top=0, **kw):
    out = ln.logprobs(x, t, scale, top=top, want_ranks=t is not None, **kw)
    torch.cuda.synchronize()
    return R.check_logprobs(out, R.to64(x), t, scale, top), out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 255, 256, 1000, 1001, 4096, 4097, 8191, 20000, 50257])
@pytest.mark.parametrize("top", [0, 1, 20, 256])
def test_widths(dtype, V, top):
    rows = 9
    run(R.logits(rows, V, dtype, V + top), tokens_of(rows, V, V), 1.0, top)


@pytest.mark.parametrize("dtype,V", [("bf16", 131072), ("f32", 131072), ("bf16", 262144), ("f32", 262147),
                                     ("bf16", 1 << 20)])
@pytest.mark.parametrize("rows,top", [(1, 20), (3, 64), (2, 256)])
def test_long_rows(dtype, V, rows, top):
    run(R.logits(rows, V, dtype, V + rows), tokens_of(rows, V, rows), 0.8, top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 5, 17, 64, 151, 153, 400])
def test_row_counts(dtype, rows):
    run(R.logits(rows, 5003, dtype, rows), tokens_of(rows, 5003, rows), 1.3, 11)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", range(0, 9))
@pytest.mark.parametrize("ld", [1003, 1008, 1011])
def test_alignments_and_row_distances(dtype, offset, ld):
    x = R.logits(6, 1003, dtype, offset, ld=ld, offset=offset)
    t = tokens_of(6, 1003, offset)
    _, out = run(x, t, 1.0, 7)
    dl, de = torch.randn(6).cuda(), torch.randn(6).cuda()
    check_bwd(x, t, out[2], out[1], dl, de, 1.0, dtype)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 3.0, 40.0])
@pytest.mark.parametrize("spread", [0.0, 1e-3, 2.0, 200.0])
def test_scales_and_spreads(scale, spread):
    x = R.logits(8, 3001, "f32", 5, spread=spread)
    run(x, tokens_of(8, 3001, 5), scale, 5)


def test_parts_of_the_results():
    x, t = R.logits(4, 999, "bf16", 3), tokens_of(4, 999, 3)
    full = ln.logprobs(x, t, top=3, want_ranks=True)
    a = ln.logprobs(x, want_entropy=False)
    assert a[0] is None and a[1] is None and a[3] is None and a[4] is None and a[5] is None
    b = ln.logprobs(x, t, want_entropy=False, top=3)
    torch.cuda.synchronize()
    assert torch.equal(a[2], full[2]) and torch.equal(b[0], full[0]) and torch.equal(b[4], full[4])
    assert torch.equal(b[5], full[5]) and b[3] is None
    # Outputs given by the caller are used.
    lse = torch.empty(4, device="cuda")
    ids = torch.empty(4, 3, dtype=torch.int32, device="cuda")
    c = ln.logprobs(x, t, top=3, lse=lse, top_ids=ids)
    assert c[2] is lse and c[4] is ids and torch.equal(lse, full[2]) and torch.equal(ids, full[4])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 4096, 50257, 131072])
@pytest.mark.parametrize("top", [1, 20, 256])
def test_ties_go_to_the_lowest_column(dtype, V, top):
    g = torch.Generator().manual_seed(V)
    few = torch.randint(-2, 3, (4, V), generator=g).float()
    few[1] = 0.0
    few[2] = torch.where(few[2] > 0, -0.0, 0.0)  # -0 and +0 are equal
    few[3] = torch.finfo(torch.bfloat16).min
    run(few.to(R.TYPES[dtype]).cuda(), tokens_of(4, V, top), 1.0, top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 1000, 50257, 131072])
@pytest.mark.parametrize("gone", [-float("inf"), "lowest"])
def test_masked_rows(dtype, V, gone):
    """Rows with all, all but one, all but five, and half of their logits masked."""
    dt = R.TYPES[dtype]
    gone = torch.finfo(dt).min if gone == "lowest" else gone
    x = torch.randn(5, V, generator=torch.Generator().manual_seed(1)).to(dt)
    g = torch.Generator().manual_seed(V)
    keep = torch.zeros(5, V, dtype=torch.bool)
    keep[1, V - 1] = True
    keep[2, torch.randperm(V, generator=g)[:5]] = True
    keep[3, V // 2:] = True
    keep[4, : V // 2] = True
    x = torch.where(keep, x, torch.tensor(gone, dtype=dt)).cuda()
    t = torch.tensor([0, V - 1, 0, V - 1, 0], dtype=torch.int32).cuda()
    _, out = run(x, t, 1.0, 20)
    _, out256 = run(x, t, 1.0, 256)
    dl, de = torch.ones(5).cuda(), torch.full((5,), 0.5).cuda()
    if gone != -float("inf"):
        check_bwd(x, t, out[2], out[1], dl, de, 1.0, dtype)
    else:  # a mask that leaves something: finite everywhere
        check_bwd(x[1:], t[1:], out[2][1:], out[1][1:], dl[1:], de[1:], 1.0, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 5000])
def test_rows_without_a_distribution(dtype, V):
    x = R.logits(6, V, dtype, 8)
    x[1, V // 3] = float("nan")
    x[2, V - 1] = float("inf")
    x[3, :] = float("nan")
    x[4, :] = -float("inf")
    x[4, 2] = float("nan")
    t = tokens_of(6, V, 8)
    out = ln.logprobs(x, t, top=4, want_ranks=True)
    torch.cuda.synchronize()
    for r in (1, 2, 3, 4):
        assert torch.isnan(out[0][r]) and torch.isnan(out[1][r]) and not torch.isfinite(out[2][r])
    assert out[4][2, 0].item() == V - 1  # +inf is the largest
    assert out[4][3].tolist() == [-1] * 4 and out[4][4].tolist() == [-1] * 4
    ref = oracle.logprobs(R.to64(x), None, 1.0, 4)
    np.testing.assert_array_equal(out[4].cpu().numpy(), ref["top_ids"])
    good = [0, 5]
    R.check_logprobs(tuple(o[good] for o in out), R.to64(x)[good], t[good], 1.0, 4)


def test_tokens_that_are_none():
    x = R.logits(5, 300, "bf16", 9)
    t = torch.tensor([3, -1, -100, 300, 2**31 - 1], dtype=torch.int32).cuda()
    _, out = run(x, t, 1.0, 0)
    assert out[3].tolist()[1:] == [0, 0, 0, 0] and out[0].tolist()[1:3] == [0.0, 0.0]
    dl = torch.ones(5).cuda()
    g = ln.logprobs_bwd(x, t, out[2], dlogp=dl)
    torch.cuda.synchronize()
    assert (g[1:3] == 0).all() and torch.isnan(g[3:]).all() and torch.isfinite(g[0]).all()


def adversarial(V, kind, seed):
    """fp32 rows made against the selection of the top by segments."""
    g = torch.Generator().manual_seed(seed)
    if kind == "rising":
        return torch.arange(V).float()[None] / 64
    if kind == "falling":
        return -torch.arange(V).float()[None] / 64
    if kind == "one_stripe":  # every large value in the columns of one thread
        x = torch.randn(1, V, generator=g)
        at = (torch.arange(V) // 4 % 512) == 3
        x[0, at] += 50 + torch.arange(int(at.sum())).float() / 1024
        return x
    # Levels of whole segments: all values of the largest segments above all others.
    nvec, nt = V // 4, 512
    per = -(-nvec // nt)
    seglen = max(1, -(-per * nt // 2048))
    v = torch.arange(V) // 4
    seg = (v // nt // seglen) * nt + v % nt
    level = torch.randperm(int(seg.max()) + 1, generator=g).float()
    return (level[seg] + 0.5 * torch.rand(V, generator=g))[None]


@pytest.mark.parametrize("V", [4096, 50304, 131072, 262144, 1 << 21])
@pytest.mark.parametrize("kind", ["rising", "falling", "one_stripe", "levels"])
def test_rows_made_against_the_selection(V, kind):
    x = adversarial(V, kind, V) * 0.01
    if kind == "levels" and V > (1 << 18):
        x = x.double().float()
    x = torch.cat([x, x.flip(1)]).cuda()
    for top in (1, 20, 256):
        run(x, tokens_of(2, V, 1), 1.0, top)


def check_bwd(x, t, lse, ent, dl, de, scale, dtype, **kw):
    x64 = R.to64(x)
    g = ln.logprobs_bwd(x, t, lse, ent, dl, de, scale, **kw)
    torch.cuda.synchronize()
    scale = R.f32(scale)
    np_ = lambda v: None if v is None else R.to64(v)  # noqa: E731
    tn = None if t is None else t.cpu().numpy()
    want = oracle.logprobs_bwd(x64, tn, np_(lse), np_(ent), np_(dl), np_(de), scale)
    R.close("gradient", R.to64(g), want,
            R.tol_bwd(x64, tn, np_(lse), np_(ent), np_(dl), np_(de), scale, want, dtype))
    return g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 7, 8, 9, 129, 1000, 1001, 4096, 50257, 131072])
@pytest.mark.parametrize("which", ["logp", "entropy", "both"])
def test_gradient_widths(dtype, V, which):
    rows, scale = 7, 0.7
    x, t = R.logits(rows, V, dtype, V), tokens_of(rows, V, V)
    out = ln.logprobs(x, t, scale)
    dl = torch.randn(rows).cuda() if which != "entropy" else None
    de = torch.randn(rows).cuda() if which != "logp" else None
    if dl is not None:
        dl[2] = 0.0
    check_bwd(x, t if dl is not None else None, out[2], out[1], dl, de, scale, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_in_place_padded_and_elsewhere(dtype):
    rows, V, ld = 11, 1003, 1024
    x = R.logits(rows, V, dtype, 2, ld=ld)
    t = tokens_of(rows, V, 2)
    lse = ln.logprobs(x, t)[2]
    dl = torch.randn(rows).cuda()
    a = check_bwd(x, t, lse, None, dl, None, 1.0, dtype)
    assert a.stride() == (ld, 1)
    # into rows at another place of a vector; the columns behind V stay as they are
    buf = torch.full((rows * 1031 + 3,), 7.0, dtype=x.dtype, device="cuda")
    out = buf[3:].view(rows, 1031)[:, :V]
    b = ln.logprobs_bwd(x, t, lse, dlogp=dl, dlogits=out)
    assert torch.equal(a, b) and (buf[3:].view(rows, 1031)[:, V:] == 7).all() and (buf[:3] == 7).all()
    full = torch.full((rows, ld), 7.0, dtype=x.dtype, device="cuda")
    full[:, :V] = x
    c = ln.logprobs_bwd(full[:, :V], t, lse, dlogp=dl, in_place=True)
    torch.cuda.synchronize()
    assert c.data_ptr() == full.data_ptr() and torch.equal(c, a) and (full[:, V:] == 7).all()


def test_gradient_is_that_of_differences_and_rows_left_out():
    x = R.logits(4, 50, "f32", 6)
    x[2, 5] = float("nan")
    x[3, :] = -float("inf")
    t = tokens_of(4, 50, 6)
    out = ln.logprobs(x, t)
    dl, de = torch.tensor([0.7, -0.4, 0.0, 0.0]).cuda(), torch.tensor([0.3, 0.0, 0.0, 0.0]).cuda()
    g = ln.logprobs_bwd(x, t, out[2], out[1], dl, de)
    torch.cuda.synchronize()
    assert (g[2:] == 0).all()
    x64 = R.to64(x)
    h = 1e-5
    for r in range(2):
        for j in range(50):
            up, dn = x64.copy(), x64.copy()
            up[r, j] += h
            dn[r, j] -= h
            tn = t.cpu().numpy()
            a, b = oracle.logprobs(up[r:r + 1], tn[r:r + 1]), oracle.logprobs(dn[r:r + 1], tn[r:r + 1])
            num = (dl[r].item() * (a["logp"] - b["logp"]) + de[r].item() * (a["entropy"] - b["entropy"])) / (2 * h)
            # differences: h^2 of the third derivative and 1e-16 / h; the kernel: some tens of u
            assert abs(g[r, j].item() - num[0]) < 1e-5


def test_repeatable_on_streams_and_in_graphs():
    rows, V = 37, 50257
    x, t = R.logits(rows, V, "bf16", 4), tokens_of(rows, V, 4)
    dl = torch.randn(rows).cuda()
    first = ln.logprobs(x, t, top=20, want_ranks=True)
    grad = ln.logprobs_bwd(x, t, first[2], dlogp=dl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):  # two streams at once
        a = ln.logprobs(x, t, top=20, want_ranks=True)
        b = ln.logprobs(x, t, top=20, want_ranks=True, stream=s)
    torch.cuda.synchronize()
    for u, v, w in zip(first, a, b):
        assert torch.equal(u, v) and torch.equal(u, w)
    out = ln.logprobs(x, t, top=20, want_ranks=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ln.logprobs(x, t, 1.0, 20, True, True, *out)
        gr = ln.logprobs_bwd(x, t, out[2], dlogp=dl)
    for o in out:
        o.zero_()
    g.replay()
    torch.cuda.synchronize()
    for u, v in zip(first, out):
        assert torch.equal(u, v)
    assert torch.equal(gr, grad)
    x.copy_(x.flip(0))  # new inputs, the same graph
    t.copy_(t.flip(0))
    g.replay()
    torch.cuda.synchronize()
    # (A row's sums follow its place in memory: rows of odd length start elsewhere in a vector.)
    again = ln.logprobs(x, t, top=20, want_ranks=True)
    torch.cuda.synchronize()
    for u, v in zip(again, out):
        assert torch.equal(u, v)
    assert torch.equal(first[4].flip(0), out[4]) and torch.equal(first[3].flip(0), out[3])


def test_rows_past_32_bits_of_elements():
    """17000 rows of 131072: the last ones lie more than 2^31 elements behind the first."""
    rows, V, K = 17000, 131072, 4
    x = torch.empty(rows, V, dtype=torch.bfloat16, device="cuda").normal_()
    last = slice(rows - 3, rows)
    t = tokens_of(rows, V, 0)
    out = ln.logprobs(x, t, top=5, want_ranks=True)
    torch.cuda.synchronize()
    R.check_logprobs(tuple(o[last] for o in out), R.to64(x[last]), t[last], 1.0, 5)
    dl = torch.ones(rows, device="cuda")
    g = ln.logprobs_bwd(x, t, out[2], dlogp=dl)
    few = ln.logprobs_bwd(x[last].contiguous(), t[last].contiguous(), out[2][last].contiguous(), dlogp=dl[last].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(g[last], few)
    del few
    losses, d = ln.distill(x, out[4][:, :K].contiguous(), out[5][:, :K].contiguous(), dlogits=g)
    small, ds = ln.distill(x[last].contiguous(), out[4][last, :K].contiguous(), out[5][last, :K].contiguous())
    torch.cuda.synchronize()
    # the same rows, split otherwise over blocks: sums in another order
    assert (losses[last] - small).abs().max() < 2e-5
    assert (d[last].float() - ds.float()).abs().max() <= 2.0 ** -8 and (d[last] != ds).float().mean() < 0.01


def test_refusals():
    x, t = R.logits(4, 16, "f32", 1), tokens_of(4, 16, 1)
    f = torch.zeros(4, device="cuda")
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(ln.LnError):
            ln.logprobs(x, t, bad)
        with pytest.raises(ln.LnError):
            ln.logprobs_bwd(x, t, f, dlogp=f, scale=bad)
    with pytest.raises(ln.LnError):
        ln.logprobs(x, t, top=257)
    with pytest.raises(ln.LnError):
        ln.logprobs(x[:, :0], t)
    with pytest.raises(TypeError):
        ln.logprobs(x, t.long())
    with pytest.raises(TypeError):
        ln.logprobs(x.half(), t)
    for call in (lambda: ln.logprobs(x.t()), lambda: ln.logprobs(x[:1].expand(4, 16)),
                 lambda: ln.logprobs(x, t[:3]), lambda: ln.logprobs(x, want_ranks=True),
                 lambda: ln.logprobs(x, t, top=-1), lambda: ln.logprobs(x, t, top_ids=t),
                 lambda: ln.logprobs(x, t.cpu()), lambda: ln.logprobs_bwd(x, t, f),
                 lambda: ln.logprobs_bwd(x, None, f, dlogp=f), lambda: ln.logprobs_bwd(x, t, None, dlogp=f),
                 lambda: ln.logprobs_bwd(x, t, f, dentropy=f),
                 lambda: ln.logprobs_bwd(x, t, f, dlogp=f, dlogits=x.t()),
                 lambda: ln.logprobs_bwd(x, t, f, dlogp=f, dlogits=x.clone(), in_place=True)):
        with pytest.raises(ValueError):
            call()
    assert [None if o is None else tuple(o.shape) for o in ln.logprobs(x[:0], t[:0], top=3)] == [
        (0,), (0,), (0,), None, (0, 3), (0, 3)]
    assert ln.logprobs_bwd(x[:0], t[:0], f[:0], dlogp=f[:0]).shape == (0, 16)
