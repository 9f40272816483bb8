"""Forms of the token log probabilities' calls beside those of test_logprobs_gpu.py: the gradient of rows of
large logits and of masked words, against the softmax in 64 bits and not by the forward's log-sum, and of
views.  Tolerances: vocabref.py, and at each test."""
import numpy as np
import pytest
import torch

import layernorm_ln_fwd_gb300 as ln
import vocabref as R

pytestmark = pytest.mark.gpu


def true_gradient(x64, tokens, dl, de, scale):
    """From the logits alone: log q = z - max z - log Z."""
    z = scale * x64
    d = z - z.max(axis=1, keepdims=True)
    logq = d - np.log(np.exp(d).sum(axis=1, keepdims=True))
    q = np.exp(logq)
    logq = np.where(q > 0, logq, 0.0)
    H = -(q * logq).sum(axis=1, keepdims=True)
    g = -dl[:, None] * q - de[:, None] * q * (logq + H)
    g[np.arange(len(q)), tokens] += dl
    return scale * g, q, logq, H


def check_true_gradient(x, tokens, dl, de, scale, dtype, **kw):
    """log q errs by 3 u |log q| of the products, E of the sums (the row's own, or the forward's, which is
    then rounded to fp32: half a step of |lse| < 512, 2^-16, and 4 u of its last steps), and the weight by 8 u;
    the entropy by E (2 + A) + 6 u B (vocabref.py); the store rounds."""
    x64 = R.to64(x)
    _, ent, lse, _, _, _ = ln.logprobs(x, tokens, scale)
    got = ln.logprobs_bwd(x, tokens, lse, ent, dl, de, scale, **kw)
    torch.cuda.synchronize()
    scale = R.f32(scale)
    dl, de = R.to64(dl), R.to64(de)
    want, q, logq, H = true_gradient(x64, tokens.cpu().numpy(), dl, de, scale)
    _, d, _, A, B, E = R.row_stats(x64, scale)
    coarse = np.abs(R.to64(lse))
    E, A, B = E[:, None], A[:, None], B[:, None]
    with np.errstate(all="ignore"):
        half = np.where(coarse < 512, np.exp2(np.floor(np.log2(np.maximum(coarse, 1)))) * R.U, 0.0)[:, None]
    eq = q * (R.U * (3 * (np.abs(logq) + 6) + 12) + E + half) + 2.0 ** -125
    hit = np.zeros_like(q)
    hit[np.arange(len(q)), tokens.cpu().numpy()] = 1
    size = np.abs(logq) + H
    eH = E * (2 + A) + 6 * R.U * B + 4 * R.U * H
    err = np.abs(dl)[:, None] * (eq + 4 * R.U * (q + hit))
    err += np.abs(de)[:, None] * (eq * (size + 1) + q * (4 * R.U * size + eH))
    err *= scale
    R.close("gradient", R.to64(got), want, err + R.HALF[dtype] * (np.abs(want) + err) + 2.0 ** -133)
    return got, want


def upstream(rows, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, generator=g).cuda(), torch.randn(rows, generator=g).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 5, 130, 1000, 1001, 50257])
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_gradient_of_rows_of_the_lowest_value(dtype, V, scale):
    """Every word masked by the type's lowest value: uniform, by definition and by the forward."""
    rows = 5
    x = torch.full((rows, V), torch.finfo(R.TYPES[dtype]).min, dtype=R.TYPES[dtype], device="cuda")
    x[1] = R.logits(1, V, dtype, V)  # next to a row of ordinary logits
    t = torch.tensor([0, V - 1, V // 2, V // 3, 0], dtype=torch.int32).cuda()
    got, want = check_true_gradient(x, t, *upstream(rows, V), scale, dtype)
    dl = torch.ones(rows, device="cuda")
    _, ent, lse, _, _, _ = ln.logprobs(x, t, scale)
    one = ln.logprobs_bwd(x, t, lse, dlogp=dl, scale=scale).double()
    torch.cuda.synchronize()
    for r in (0, 2, 3, 4):
        uniform = torch.full((V,), -scale / V, dtype=torch.float64, device="cuda")
        uniform[t[r].item()] += scale
        assert ((one[r] - uniform).abs() <= R.HALF[dtype] * uniform.abs() + 2.0 ** -12 / V + 2.0 ** -22).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [-1e30, -3e4, -600.0, -500.0, 300.0, 511.0, 1e4, 1e6])
@pytest.mark.parametrize("V", [33, 4001, 50304])
def test_gradient_of_shifted_rows(dtype, shift, V):
    rows = 6
    x = (R.logits(rows, V, "f32", V) + shift).to(R.TYPES[dtype])
    x[2] = R.logits(1, V, dtype, 1)[0]
    g = torch.Generator().manual_seed(V)
    t = torch.randint(0, V, (rows,), generator=g, dtype=torch.int32).cuda()
    dl, de = upstream(rows, V)
    dl[3], de[3] = 0.0, 0.0  # nothing flows back
    check_true_gradient(x, t, dl, de, 0.9, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_of_large_logits_in_place_and_elsewhere(dtype):
    rows, V, ld = 40, 5003, 5009
    x = R.logits(rows, V, dtype, 3, ld=ld)
    x[::3] = x[::3] * 500
    x[1] = -float("inf")
    x[1, 7] = -2000.0
    g = torch.Generator().manual_seed(1)
    t = torch.randint(0, V, (rows,), generator=g, dtype=torch.int32).cuda()
    t[1] = 7
    dl, de = upstream(rows, 5)
    _, ent, lse, _, _, _ = ln.logprobs(x, t)
    a, _ = check_true_gradient(x, t, dl, de, 1.0, dtype)
    buf = torch.full((rows * 5011 + 1,), 7.0, dtype=x.dtype, device="cuda")
    out = buf[1:].view(rows, 5011)[:, :V]
    b = ln.logprobs_bwd(x, t, lse, ent, dl, de, dlogits=out)
    full = torch.full((rows, ld), 7.0, dtype=x.dtype, device="cuda")
    full[:, :V] = x
    c = ln.logprobs_bwd(full[:, :V], t, lse, ent, dl, de, in_place=True)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    assert (buf[1:].view(rows, 5011)[:, V:] == 7).all() and (full[:, V:] == 7).all() and buf[0] == 7


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_where_the_log_sum_overflows(dtype):
    """scale * logits past fp32: lse is +-inf, the distribution is not lost."""
    x = torch.tensor([[3e38, 3e38, 1.0], [-3e38, -3e38, -3e38], [3e38, 0.0, -3e38]]).to(R.TYPES[dtype]).cuda()
    t = torch.tensor([0, 2, 1], dtype=torch.int32).cuda()
    logp, ent, lse, _, _, _ = ln.logprobs(x, t, 2.0)
    g = ln.logprobs_bwd(x, t, lse, ent, torch.ones(3).cuda(), torch.ones(3).cuda(), 2.0)
    torch.cuda.synchronize()
    assert torch.isinf(lse[:2]).all()
    want = torch.tensor([[1.0, -1.0, 0.0], [-2 / 3, -2 / 3, 4 / 3], [-2.0, 2.0, 0.0]], device="cuda")
    assert (g.float() - want).abs().max() <= 2 * R.HALF[dtype] * 2 + 1e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 1000, 40003])
@pytest.mark.parametrize("size", [1e3, 1e10, 1e30])
def test_gradient_of_masked_words_with_large_upstream_gradients(dtype, V, size):
    """A word without probability has no gradient, however large the entropy's (a scaled loss, say)."""
    rows = 6
    x = R.logits(rows, V, dtype, V)
    x[1:3, ::2] = -float("inf")
    x[3:5, 1::3] = torch.finfo(x.dtype).min
    x[5, : V - 1] = -float("inf")
    t = torch.tensor([0, 1, 3, 0, 3, V - 1], dtype=torch.int32).cuda()
    dl, de = upstream(rows, V)
    got, want = check_true_gradient(x, t, dl, de * size, 1.0, dtype)
    assert torch.isfinite(got).all() and (got[torch.isinf(x)] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("view", ["last position", "every second row", "some columns", "padding"])
def test_gradient_of_a_view_is_no_larger_than_its_rows(dtype, view):
    V = 1003
    wide = R.logits(6 * 40, 1024, dtype, 2).view(6, 40, 1024)
    x = {"last position": wide[:, -1], "every second row": wide[0, ::2, :V], "some columns": wide[0, :, 5:105],
         "padding": wide[0, :, :V]}[view]
    rows, V = x.shape
    t = torch.arange(rows, dtype=torch.int32, device="cuda")
    dl = torch.randn(rows, generator=torch.Generator().manual_seed(1)).cuda()
    lse = ln.logprobs(x, t)[2]
    g = ln.logprobs_bwd(x, t, lse, dlogp=dl)
    losses, d = ln.distill(x, t[:, None], dl[:, None].contiguous())
    packed = x.contiguous()
    g2 = ln.logprobs_bwd(packed, t, lse, dlogp=dl)
    l2, d2 = ln.distill(packed, t[:, None], dl[:, None].contiguous())
    torch.cuda.synchronize()
    for a, b in ((g, g2), (d, d2)):
        assert a.shape == x.shape and a.untyped_storage().nbytes() <= rows * (V + max(V // 8, 64)) * x.element_size()
        assert (a.stride(0) - x.stride(0)) * x.element_size() % 16 == 0
        # sums in another order may round to the neighbouring value
        assert ((a.double() - b.double()).abs() <= 2.01 * R.HALF[dtype] * b.double().abs() + 1e-5).all()
    assert (g.stride(0) == x.stride(0)) == (view == "padding") and (losses - l2).abs().max() <= 1e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V,ld", [(5, 1003, 1003), (300, 20001, 20003), (3, 131072, 131072), (2, 70001, 70001)])
def test_repeatable_where_the_header_says_so(dtype, rows, V, ld):
    """Copies of the logits at addresses that are equal modulo 32 (logprobs) and modulo 16 (its gradient, distill)."""
    size = R.TYPES[dtype].itemsize
    x = R.logits(rows, V, dtype, V, ld=ld)
    t = torch.randint(0, V, (rows,), generator=torch.Generator().manual_seed(V), dtype=torch.int32).cuda()
    ids = ((t[:, None] + torch.arange(7, device="cuda") * 3) % V).to(torch.int32)
    teacher = torch.randn(rows, 7, generator=torch.Generator().manual_seed(3)).cuda()
    dl = torch.randn(rows, generator=torch.Generator().manual_seed(4)).cuda()

    def copy(offset_bytes):
        flat = torch.empty(offset_bytes // size + rows * ld, dtype=x.dtype, device="cuda")
        assert flat.data_ptr() % 256 == 0
        c = flat[offset_bytes // size:].view(rows, ld)[:, :V]
        return c.copy_(x)

    def all_of(a, b):
        torch.cuda.synchronize()
        for u, v in zip(a, b):
            assert torch.equal(u, v)

    for at in (0, 4, 24):
        p, q = copy(at), copy(at + 96)
        all_of(ln.logprobs(p, t, 0.8, 9, True, True), ln.logprobs(q, t, 0.8, 9, True, True))
        q = copy(at + 48)
        for k in (1.0, 3e4):  # the forward's log-sum, and one beyond 512
            lse = torch.full((rows,), 12.0, device="cuda") * k
            all_of([ln.logprobs_bwd(p, t, lse, dlogp=dl)], [ln.logprobs_bwd(q, t, lse, dlogp=dl)])
        all_of(ln.distill(p, ids, teacher), ln.distill(q, ids, teacher))


def segments(rows, V, top):
    """The segment of every column of an aligned fp32 row, whose largest values the selection of the top begins
    with: launch_logprobs_t's cut of a row into slices, threads, pairs of vectors and batches, restated."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    nvec, blocks = V // 4, 1
    while blocks < 8 and rows * blocks * 2 <= 2 * sms and nvec // (blocks * 2) >= 2048:
        blocks *= 2
    piece = (-(-nvec // blocks) + 1) & ~1
    few = rows <= 8 * sms
    nt = 128 if few else 32
    while nt < (256 if few else 128) and nt * 4 < piece:
        nt *= 2
    per = max(1, -(-piece // (nt * 4)))
    seglen = 1
    while per * nt > seglen * min(max(32 * top, 512), 2048):
        seglen *= 2
    v = torch.arange(V) // 4
    rank, i = v // piece, v % piece
    tid, batch = i % (2 * nt) // 2, i // (4 * nt)
    return rank * (per * nt) + (batch // seglen) * nt + tid


@pytest.mark.parametrize("V", [4096, 50304, 131072, 262144, 1 << 21])
@pytest.mark.parametrize("order", ["random", "rising", "falling"])
@pytest.mark.parametrize("top", [1, 20, 256])
@pytest.mark.parametrize("rows", [1, 400])
def test_rows_of_levels_of_whole_segments(V, order, top, rows):
    """Every value of a segment above all those of a lower one: few segments hold very many large values, and
    all of them are candidates of the top."""
    rows = min(rows, (1 << 28) // V)
    g = torch.Generator().manual_seed(V + top)
    seg = segments(rows, V, top)
    count = int(seg.max()) + 1
    level = {"random": torch.randperm(count, generator=g), "rising": torch.arange(count),
             "falling": torch.arange(count).flip(0)}[order]
    x = (level[seg] + 0.5 * torch.rand(V, generator=g)) * (20.0 / count)
    x = x.repeat(rows, 1).cuda()
    x[rows // 2] = x[0].flip(0)
    t = torch.randint(0, V, (rows,), generator=g, dtype=torch.int32).cuda()
    out = ln.logprobs(x, t, 1.0, top, True, True)
    torch.cuda.synchronize()
    some = sorted({0, rows // 2, rows - 1})
    R.check_logprobs(tuple(o[some] for o in out), R.to64(x[some]), t[some], 1.0, top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,infs", [(900, 3), (5000, 2000), (50257, 700), (50257, 40000), (131072, 130000)])
@pytest.mark.parametrize("top", [1, 20, 256])
def test_top_of_rows_from_the_lowest_value_to_infinity(dtype, V, infs, top):
    """Values over the type's whole range, most of the large ones equal: the lowest columns of +inf first."""
    g = torch.Generator().manual_seed(V + infs)
    x = torch.full((3, V), torch.finfo(R.TYPES[dtype]).min, dtype=R.TYPES[dtype])
    x[1] = torch.randn(V, generator=g).to(x.dtype)
    x[2, ::2] = torch.finfo(R.TYPES[dtype]).max
    for r in range(3):
        x[r, torch.randperm(V, generator=g)[:infs]] = float("inf")
    out = ln.logprobs(x.cuda(), top=top)
    torch.cuda.synchronize()
    want = x.float().sort(dim=1, descending=True, stable=True).indices[:, :top]
    np.testing.assert_array_equal(out[4].cpu().numpy(), want.numpy())
    assert torch.isnan(out[1]).all() and not torch.isfinite(out[2]).any()
