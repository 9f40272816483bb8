"""8-bit checkpoints and the norms' backwards from them on the GPU (relref has the definition in 64 bits and where
the tolerances come from)."""
import numpy as np
import pytest
import torch

import layernorm_ln_fwd_gb300 as ln
import relref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def to64(t):
    return t.detach().double().cpu().numpy()


def values(rows, cols, dtype, seed, pad=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    flat = torch.randn(offset + rows * (cols + pad), generator=g)
    flat *= torch.exp2(torch.randint(-6, 6, (flat.numel(),), generator=g).float())
    return flat.to(TYPES[dtype]).cuda()[offset:].view(rows, cols + pad)[:, :cols]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 32), (4, 33), (700, 64), (64, 768), (9, 1001), (33, 4096),
                                       (2, 16385), (1, 100003), (3000, 40), (301, 130),
                                       (77, 249), (301, 310), (77, 511)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (0, 1), (5, 0), (8, 3)])
def test_store_and_load(dtype, rows, cols, pad, offset):
    x = values(rows, cols, dtype, cols, pad, offset)
    ck = ln.ckpt8_store(x)
    q, k, want = relref.quantise(to64(x))
    np.testing.assert_array_equal(ck.q.cpu().numpy(), q)
    np.testing.assert_array_equal(ck.k.cpu().numpy(), k)
    for t in TYPES.values():
        np.testing.assert_array_equal(to64(ln.ckpt8_load(ck, t)), want)
    whole = torch.full((rows, cols + 6), 9.0, dtype=TYPES[dtype], device="cuda")
    assert ln.ckpt8_load(ck, out=whole[:, 1:1 + cols]).dtype == TYPES[dtype]
    np.testing.assert_array_equal(to64(whole[:, 1:1 + cols]), want)
    assert (whole[:, 0] == 9).all() and (whole[:, 1 + cols:] == 9).all()
    again = ln.ckpt8_store(ln.ckpt8_load(ck, TYPES[dtype]), out=ln.Ckpt8(torch.empty_like(ck.q), torch.empty_like(ck.k), cols))
    np.testing.assert_array_equal(to64(ln.ckpt8_load(again, torch.float32)), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_of_all_sizes(dtype):
    t = TYPES[dtype]
    big, tiny = torch.finfo(t).max, torch.finfo(t).smallest_normal
    rows = [[0.0] * 40, [big, -big, 1.0] + [0.0] * 37, [tiny, -tiny / 2, tiny / 128] + [0.0] * 37, [-0.0] * 40,
            [127.5, 63.5, 64.5, -0.5, 1.5] + [0.25] * 35, [1.9921875, 1.984375] + [1e-3] * 38,
            [float("nan")] + [1.0] * 39, [1.0] * 33 + [float("inf")] + [2.0] * 6, [-float("inf")] * 40]
    x = torch.tensor(rows, dtype=torch.float64).to(t).cuda()
    ck = ln.ckpt8_store(x)
    q, k, want = relref.quantise(to64(x))
    np.testing.assert_array_equal(ck.q.cpu().numpy(), q)
    np.testing.assert_array_equal(ck.k.cpu().numpy(), k)
    np.testing.assert_array_equal(to64(ln.ckpt8_load(ck, t)), want)
    assert np.isnan(want[6, :32]).all() and (want[6, 32:] == 1).all() and np.isnan(want[7, 32:]).all()


def norm_case(dtype, rows, cols, rms, seed=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    x = torch.randn(rows, cols, generator=g) + 0.5
    x[:, :: max(1, cols // 5)] *= 20
    x = x.to(t).cuda()
    gamma = (1 + 0.1 * torch.randn(offset + cols, generator=g)).to(t).cuda()[offset:]
    dy = torch.randn(offset + rows * cols, generator=g).to(t).cuda()[offset:].view(rows, cols)
    if rms:
        _, _, rstd = ln.rms_fwd(x, None, gamma)
        mean = None
    else:
        _, _, mean, rstd = ln.fwd(x, None, gamma, torch.zeros_like(gamma))
    return x, gamma, dy, mean, rstd


def check_norm(dtype, out, dy, x64, gamma, mean, rstd):
    want = relref.norm_bwd(to64(dy), x64, to64(gamma), None if mean is None else to64(mean), to64(rstd))
    assert len(out) == len(want)
    for name, got, (w, tol) in zip(("dx", "dgamma", "dbeta"), out, want):
        relref.close(name, to64(got), w, relref.stored(tol, w, dtype))


def call(rms, dy, ck, gamma, mean, rstd, **more):
    return ln.rms_bwd_ckpt8(dy, ck, gamma, rstd, **more) if rms else ln.bwd_ckpt8(dy, ck, gamma, mean, rstd, **more)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 7), (40, 96), (700, 768), (2500, 100), (5, 1001), (64, 1024),
                                       (30, 1280), (33, 2049), (9, 4096), (7, 5000), (5, 8192), (3, 12001), (3, 16384)])
def test_norm_backwards(dtype, rms, rows, cols):
    x, gamma, dy, mean, rstd = norm_case(dtype, rows, cols, rms, seed=cols)
    ck = ln.ckpt8_store(x)
    out = call(rms, dy, ck, gamma, mean, rstd)
    check_norm(dtype, out, dy, to64(ln.ckpt8_load(ck, torch.float32)), gamma, mean, rstd)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("cols", [96, 333, 1500, 4100])
def test_norm_backwards_at_any_address_and_in_place(dtype, rms, cols):
    x, gamma, dy, mean, rstd = norm_case(dtype, 21, cols, rms, seed=1, offset=3)
    ck = ln.ckpt8_store(x)
    out = call(rms, dy, ck, gamma, mean, rstd)
    check_norm(dtype, out, dy, to64(ln.ckpt8_load(ck, torch.float32)), gamma, mean, rstd)
    d = dy.clone()  # (at another address: its rows may be cut up elsewhere, and their sums formed in another order)
    out = call(rms, d, ck, gamma, mean, rstd)
    check_norm(dtype, out, dy, to64(ln.ckpt8_load(ck, torch.float32)), gamma, mean, rstd)
    again = call(rms, d, ck, gamma, mean, rstd, dx=d)
    assert again[0] is d and all(torch.equal(a, b) for a, b in zip(again, out))
    d = dy.reshape(-1)  # and in place where it was
    want = call(rms, d.view(21, cols), ck, gamma, mean, rstd)
    again = call(rms, d.view(21, cols), ck, gamma, mean, rstd, dx=d.view(21, cols))
    assert all(torch.equal(a, b) for a, b in zip(again, want))


@pytest.mark.parametrize("rms", [False, True])
def test_norm_backwards_of_many_rows(rms):
    x, gamma, dy, mean, rstd = norm_case("bf16", 20000, 256, rms, seed=2)
    ck = ln.ckpt8_store(x)
    out = call(rms, dy, ck, gamma, mean, rstd)
    check_norm("bf16", out, dy, to64(ln.ckpt8_load(ck, torch.float32)), gamma, mean, rstd)
    ws = torch.full((ln.ckpt8_workspace_bytes(20000, 256),), 255, dtype=torch.uint8, device="cuda")
    again = call(rms, dy, ck, gamma, mean, rstd, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(again, out))
    with pytest.raises(ln.LnError, match="ENOSPACE"):
        call(rms, dy, ck, gamma, mean, rstd, workspace=ws[:256])


@pytest.mark.parametrize("rms", [False, True])
def test_no_rows(rms):
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    ck = ln.ckpt8_store(e(0, 40))
    assert ck.q.shape == (0, 64) and ln.ckpt8_load(ck).shape == (0, 40)
    out = call(rms, e(0, 40), ck, e(40), e(0), e(0))
    assert out[0].shape == (0, 40) and all((t == 0).all() for t in out[1:])


def test_a_block_that_is_not_finite_reaches_its_row_and_columns():
    x, gamma, dy, mean, rstd = norm_case("f32", 6, 96, False, seed=3)
    x[2, 40] = float("inf")
    dx, dgamma, dbeta = ln.bwd_ckpt8(dy, ln.ckpt8_store(x), gamma, mean, rstd)
    assert dx[2].isnan().all() and dx[[0, 1, 3, 4, 5]].isfinite().all()
    assert dgamma[32:64].isnan().all() and dgamma[:32].isfinite().all() and dgamma[64:].isfinite().all()
    assert dbeta.isfinite().all()


def test_layer_kept_in_8_bits_end_to_end():
    """The framework's forwards and these backwards as a layer has them: an RMSNorm's input and the attention's
    probabilities kept in 8 bits, on another stream, captured and replayed."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(2 * 64, 256, generator=g).bfloat16().cuda()
    res = torch.randn(2 * 64, 256, generator=g).bfloat16().cuda()
    gamma = torch.ones(256).bfloat16().cuda()
    table = torch.randn(32, 4, generator=g).bfloat16().cuda()
    dout = torch.randn(2 * 64, 256, generator=g).bfloat16().cuda()

    def step():
        out, s, rrms = ln.rms_fwd(x, res, gamma)
        kept = ln.ckpt8_store(s)
        h = out.view(2, 64, 4, 64).transpose(1, 2)
        scores = torch.matmul(h, h.transpose(2, 3))
        probs, kept_probs = ln.softmax_rel_fwd(scores, table, scale=0.125, ckpt=True)
        dprobs = torch.matmul(dout.view(2, 64, 4, 64).transpose(1, 2), h.transpose(2, 3))
        dscores, dtable = ln.softmax_rel_bwd(dprobs, kept_probs, table, scale=0.125)
        dh = torch.matmul(dscores, h) + torch.matmul(dscores.transpose(2, 3), h)
        dh += torch.matmul(ln.ckpt8_load(kept_probs).view(2, 4, 64, 64).transpose(2, 3),
                           dout.view(2, 64, 4, 64).transpose(1, 2))
        dx, dgamma = ln.rms_bwd_ckpt8(dh.transpose(1, 2).reshape(128, 256), kept, gamma, rrms)
        return probs, dtable, dx, dgamma, s, rrms, dh
    want = step()
    probs, dtable, dx, dgamma, s, rrms, dh = (t.clone() for t in want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dy64 = dh.transpose(1, 2).reshape(128, 256)
    x64 = relref.quantise(to64(s))[2]
    check_norm("bf16", (dx, dgamma), dy64, x64, gamma, None, rrms)
