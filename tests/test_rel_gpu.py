"""The softmax with a learned relative position bias on the GPU, against 64 bits (relref has the reference and
where the tolerances come from)."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import layernorm_ln_fwd_gb300 as ln
import relref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def to64(t):
    return t.detach().double().cpu().numpy()


def rows_of(shape, dtype, g, spread=1.0, pad=0, offset=0):
    """A CUDA tensor of that shape, rows `pad` elements wider, `offset` elements behind an aligned address."""
    B, H, Lq, Lk = shape
    ld = Lk + pad
    flat = torch.randn(offset + B * H * Lq * ld, generator=g) * spread
    return flat.to(TYPES[dtype]).cuda()[offset:].view(B, H, Lq, ld)[..., :Lk]


class Case:
    def __init__(self, dtype, shape, buckets=32, span=128, both=True, scale=0.7, causal=False, lens=None, q_pos=None,
                 mask=None, table_f32=False, pad=0, offset=0, spread=2.0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.shape, self.buckets = dtype, shape, buckets
        self.x = rows_of(shape, dtype, g, spread, pad, offset)
        self.dy = rows_of(shape, dtype, g, 1.0, pad, offset)
        self.table = torch.randn(buckets, shape[1], generator=g).to(torch.float32 if table_f32 else TYPES[dtype]).cuda()
        ints = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        self.how = dict(max_distance=span, bidirectional=both, scale=scale, causal=causal, lens=ints(lens), q_pos=ints(q_pos))
        self.mask = None if mask is None else mask.to(TYPES[dtype]).cuda()
        scale = float(np.float32(scale))
        edges = relref.edges_of(buckets, span, both)
        self.y64, self.tol, self.bk, self.kept = relref.fwd(
            to64(self.x), to64(self.table), edges, both, scale, causal, lens, q_pos,
            None if mask is None else to64(self.mask))
        self.scale = scale

    def check_fwd(self, y):
        want = self.y64
        relref.close("y", to64(y), want, relref.stored(self.tol, want, self.dtype))
        assert (to64(y)[~self.kept] == 0).all()

    def check_bwd(self, out, y64, name=""):
        dx, tdx, dt, tdt = relref.bwd(to64(self.dy), y64, self.bk, self.kept, self.buckets, self.scale)
        relref.close(name + "dx", to64(out[0]), dx, relref.stored(tdx, dx, self.dtype))
        ttype = "f32" if self.table.dtype == torch.float32 else self.dtype
        relref.close(name + "dtable", to64(out[1]), dt, relref.stored(tdt, dt, ttype))
        assert (to64(out[0])[~self.kept] == 0).all()

    def check(self):
        y, ck = ln.softmax_rel_fwd(self.x, self.table, mask=self.mask, ckpt=True, **self.how)
        self.check_fwd(y)
        plain = ln.softmax_rel_fwd(self.x, self.table, mask=self.mask, **self.how)
        assert plain[1] is None
        self.check_fwd(plain[0])  # (rows that start elsewhere in 16 bytes are cut up elsewhere without a checkpoint)
        rows = y.reshape(-1, self.shape[3])
        q, k, values = relref.quantise(to64(rows))
        np.testing.assert_array_equal(ck.q.cpu().numpy(), q)
        np.testing.assert_array_equal(ck.k.cpu().numpy(), k)
        self.check_bwd(ln.softmax_rel_bwd(self.dy, y, self.table, **self.how), to64(y))
        out = ln.softmax_rel_bwd(self.dy, ck, self.table, **self.how)
        self.check_bwd(out, values.reshape(self.shape), "kept ")
        dx, none = ln.softmax_rel_bwd(self.dy, ck, self.table, want_table=False, **self.how)
        assert none is None and torch.equal(dx, out[0])


SHAPES = [(1, 1, 1, 1), (2, 3, 1, 77), (2, 2, 5, 8), (1, 2, 33, 33), (2, 3, 17, 100), (1, 2, 40, 256), (1, 2, 24, 333),
          (1, 1, 9, 513), (2, 1, 7, 1000), (1, 2, 5, 1032), (1, 2, 6, 2500), (1, 1, 3, 5001), (1, 1, 5, 8192),
          (1, 1, 4, 16384), (2, 1, 1, 4099), (1, 3, 130, 40), (1, 2, 7, 3600), (1, 1, 9, 2049)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("both", [True, False])
def test_shapes(dtype, shape, both):
    Case(dtype, shape, both=both, seed=shape[3]).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 2, 1, 1), (2, 2, 37, 37), (1, 2, 128, 128), (1, 1, 65, 301), (1, 1, 4, 1100),
                                   (1, 1, 300, 520), (1, 2, 9, 4000), (1, 1, 6, 2111)])
def test_causal(dtype, shape):
    Case(dtype, shape, both=False, causal=True, seed=3).check()
    Case(dtype, shape, both=False, causal=True, q_pos=[shape[3] - shape[2]] * shape[0], seed=4).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lq,Lk", [(1, 200), (6, 200), (1, 2000), (1, 5000), (20, 61)])
def test_sequences_of_their_own_lengths_and_positions(dtype, Lq, Lk):
    lens = [0, 1, Lk, Lk // 2 + 1, Lk + 7, -3]
    Case(dtype, (6, 2, Lq, Lk), lens=lens, q_pos=[max(0, n - Lq) for n in lens], both=False, seed=5).check()
    Case(dtype, (6, 2, Lq, Lk), lens=lens, q_pos=[-Lk, -1, 3 * Lk, 2**31 - 1, -2**31, 40], seed=6).check()
    Case(dtype, (6, 2, Lq, Lk), lens=lens, q_pos=[-Lk, -1, 3 * Lk, 2**31 - 1 - Lq, -2**31, 40], both=False, causal=True,
         seed=7).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lk", [16385, 20000, 33001])
def test_rows_longer_than_the_registers_hold(dtype, Lk):
    Case(dtype, (1, 1, 2, Lk), span=800, seed=8).check()
    Case(dtype, (2, 1, 1, Lk), both=False, lens=[Lk - 5, 3], q_pos=[Lk - 6, 2], seed=9).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("span", [400, 800, 1200, 2500, 6000, 16384])
@pytest.mark.parametrize("shape", [(1, 2, 9, 527), (1, 1, 5, 1501), (2, 1, 1, 331), (1, 1, 40, 101), (1, 1, 6, 1504)])
def test_wide_windows(dtype, span, shape):
    q_pos = [shape[3] // 2] * shape[0]  # (the whole window, whatever the rows' length)
    Case(dtype, shape, span=span, q_pos=q_pos, seed=13).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lq,Lk", [(1, 17), (1, 256), (3, 200), (1, 251)])
@pytest.mark.parametrize("span", [128, 700])
def test_many_single_queries(dtype, Lq, Lk, span):
    lens = [(37 * b) % (Lk + 3) for b in range(100)]
    Case(dtype, (100, 8, Lq, Lk), span=span, both=False, lens=lens, q_pos=[n - Lq for n in lens], seed=11).check()
    Case(dtype, (100, 8, Lq, Lk), span=span, both=False, causal=True, seed=12, pad=3, offset=1).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 3, 1, 70001), (2, 1, 1, 140000), (1, 80, 1, 16400), (1, 2, 90, 16600)])
def test_few_long_rows(dtype, shape):
    B, H, Lq, Lk = shape
    g = torch.Generator().manual_seed(1)
    mask = torch.where(torch.rand(1, Lk, generator=g) < 0.3, -torch.inf, 0.5)
    case = Case(dtype, shape, both=False, lens=[Lk - 1000, 17][:B], q_pos=[Lk - 1001, 16][:B], mask=mask, seed=10)
    y, ck = ln.softmax_rel_fwd(case.x, case.table, mask=case.mask, ckpt=True, **case.how)
    case.check_fwd(y)
    q, k, _ = relref.quantise(to64(y.view(-1, Lk)))
    assert (ck.q.cpu().numpy() == q).all() and (ck.k.cpu().numpy() == k).all()
    again = ln.softmax_rel_fwd(case.x, case.table, mask=case.mask, **case.how)[0]
    assert torch.equal(y, again)
    ln.softmax_rel_fwd(case.x, case.table, mask=case.mask, y=case.x, **case.how)
    assert torch.equal(y, case.x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("buckets,span,both", [(4, 2, True), (2, 5, False), (16, 64, True), (64, 800, False),
                                               (256, 16384, False), (512, 16384, True), (32, 17, True), (3, 2, False)])
def test_buckets(dtype, buckets, span, both):
    Case(dtype, (1, 2, 70, 230), buckets, span, both, seed=10).check()
    Case(dtype, (1, 1, 3, 6000), buckets, span, both, q_pos=[2500], seed=11).check()
    Case(dtype, (1, 1, 1, 17001), buckets, span, both, q_pos=[16999], seed=12).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 1), (3, 5), (13, 2), (64, 7)])
@pytest.mark.parametrize("Lk", [40, 333, 1500])
def test_rows_at_any_distance_and_address(dtype, pad, offset, Lk):
    c = Case(dtype, (2, 2, 5, Lk), pad=pad, offset=offset, seed=13)
    c.check()
    # Outputs into such rows, what lies between them left as it was.
    whole = torch.full((2, 2, 5, Lk + 11), 7.0, dtype=TYPES[dtype], device="cuda")
    y, _ = ln.softmax_rel_fwd(c.x, c.table, y=whole[..., 3:3 + Lk], **c.how)
    c.check_fwd(y)
    dx = torch.full((2, 2, 5, Lk + 11), 7.0, dtype=TYPES[dtype], device="cuda")
    c.check_bwd(ln.softmax_rel_bwd(c.dy, y, c.table, dx=dx[..., 5:5 + Lk], **c.how), to64(y))
    assert (whole[..., :3] == 7).all() and (whole[..., 3 + Lk:] == 7).all()
    assert (dx[..., :5] == 7).all() and (dx[..., 5 + Lk:] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 2, 9, 96), (1, 2, 7, 333), (1, 1, 3, 3001), (1, 1, 2, 17001)])
def test_in_place(dtype, shape):
    c = Case(dtype, shape, seed=14)
    y, _ = ln.softmax_rel_fwd(c.x, c.table, **c.how)
    want = ln.softmax_rel_bwd(c.dy, y, c.table, **c.how)
    x, dy = c.x.clone(), c.dy.clone()
    assert ln.softmax_rel_fwd(x, c.table, y=x, **c.how)[0] is x and torch.equal(x, y)
    got = ln.softmax_rel_bwd(dy, x, c.table, dx=dy, **c.how)
    assert got[0] is dy and torch.equal(dy, want[0]) and torch.equal(got[1], want[1])


def test_table_of_fp32_beside_bf16():
    Case("bf16", (2, 3, 50, 120), table_f32=True, seed=15).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lk", [64, 77, 1500])
def test_masks(dtype, Lk):
    g = torch.Generator().manual_seed(16)
    mask = torch.randn(3, Lk, generator=g)
    mask[:, ::3] = -np.inf
    mask[1] = -np.inf  # a row with nothing left
    Case(dtype, (1, 2, 6, Lk), mask=mask, seed=17).check()
    # The type's lowest value throughout: a softmax of equal scores; in half the row: nothing of that half.
    low = torch.zeros(2, Lk)
    low[0] = torch.finfo(TYPES[dtype]).min
    low[1, ::2] = torch.finfo(TYPES[dtype]).min
    c = Case(dtype, (1, 1, 4, Lk), mask=low, seed=18)
    c.check()
    np.testing.assert_allclose(c.y64[0, 0, 0], 1 / Lk, rtol=1e-12)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lk", [48, 99, 1200, 20001])
def test_what_takes_no_part_is_not_used(dtype, Lk):
    lens = [Lk - 9]
    c = Case(dtype, (1, 2, 3, Lk), lens=lens, seed=19)
    x, dy = c.x.clone(), c.dy.clone()
    x[..., Lk - 9:] = float("nan")
    dy[..., Lk - 9:] = float("inf")
    y, ck = ln.softmax_rel_fwd(x, c.table, ckpt=True, **c.how)
    c.check_fwd(y)
    c.check_bwd(ln.softmax_rel_bwd(dy, y, c.table, **c.how), to64(y))
    # A mask of -inf, whatever the score; a probability of 0, whatever dy.
    mask = torch.zeros(1, Lk, dtype=TYPES[dtype], device="cuda")
    mask[:, 5::7] = -float("inf")
    how = dict(c.how, lens=None)
    m = Case(dtype, (1, 2, 3, Lk), mask=mask.cpu(), seed=19)
    for value in (float("nan"), float("inf"), -float("inf")):
        x, dy = c.x.clone(), c.dy.clone()
        x[..., 5::7] = value
        dy[..., 5::7] = value
        y, ck = ln.softmax_rel_fwd(x, c.table, mask=mask, ckpt=True, **how)
        m.check_fwd(y)
        m.check_bwd(ln.softmax_rel_bwd(dy, y, c.table, **how), to64(y))
        m.check_bwd(ln.softmax_rel_bwd(dy, ck, c.table, **how), to64(ln.ckpt8_load(ck, torch.float32)).reshape(m.shape))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lk", [40, 1500, 20001])
def test_rows_that_are_not_finite(dtype, Lk):
    c = Case(dtype, (1, 1, 4, Lk), seed=20)
    x = c.x.clone()
    x[0, 0, 0, 3] = float("nan")
    x[0, 0, 1, 5] = float("inf")
    x[0, 0, 2] = -float("inf")
    y, ck = ln.softmax_rel_fwd(x, c.table, ckpt=True, **c.how)
    assert y[0, 0, :2].isnan().all() and (y[0, 0, 2] == 0).all()
    relref.close("y", to64(y)[0, 0, 3], c.y64[0, 0, 3], relref.stored(c.tol, c.y64, dtype)[0, 0, 3])
    x[0, 0, 0] = float("nan")
    assert ln.softmax_rel_fwd(x, c.table, **c.how)[0][0, 0, 0].isnan().all()
    back = ln.ckpt8_load(ck, torch.float32)
    assert back[:2].isnan().all() and (back[2] == 0).all()
    for p in (y, ck):
        dx, dt = ln.softmax_rel_bwd(c.dy, p, c.table, **c.how)
        assert dx[0, 0, :2].isnan().all() and (dx[0, 0, 2] == 0).all() and dx[0, 0, 3].isfinite().all()


def test_a_table_that_removes_a_bucket():
    c = Case("f32", (1, 2, 20, 50), seed=21)
    c.table[3, 0] = -float("inf")
    y, _ = ln.softmax_rel_fwd(c.x, c.table, **c.how)
    gone = (c.bk[0] == 3)
    assert (to64(y)[0, 0][gone] == 0).all() and y.isfinite().all()
    dx, dt = ln.softmax_rel_bwd(c.dy, y, c.table, **c.how)
    assert dt[3, 0] == 0 and dt.isfinite().all()


def test_gradients_against_differences():
    """Central differences of the kernel's own forward in fp32: its y errs by at most `tol`, so that a quotient over
    2 eps errs by sum |dy| tol / eps, and by eps^2 / 6 of a third derivative of at most 8 times sum |dy| y."""
    c = Case("f32", (1, 2, 6, 23), buckets=8, span=7, scale=1.0, seed=22)
    y, _ = ln.softmax_rel_fwd(c.x, c.table, **c.how)
    dx, dt = ln.softmax_rel_bwd(c.dy, y, c.table, **c.how)
    eps = 2.0 ** -7
    dy64 = to64(c.dy)
    noise = (np.abs(dy64) * relref.stored(c.tol, c.y64, "f32") * 1.1).sum() / eps + 8 * eps**2 / 6 * np.abs(dy64).sum()
    for grad, t, at in [(dx, c.x, (0, 0, 2, 4)), (dx, c.x, (0, 1, 5, 22)), (dt, c.table, (0, 0)), (dt, c.table, (5, 1))]:
        old = t[at].item()
        ends = []
        for step in (eps, -eps):
            t[at] = old + step
            ends.append((to64(ln.softmax_rel_fwd(c.x, c.table, **c.how)[0]) * dy64).sum())
            width = t[at].item() - old if step > 0 else width - (t[at].item() - old)
        t[at] = old
        assert abs((ends[0] - ends[1]) / width - grad[at].item()) <= noise


def test_no_rows():
    table = torch.randn(32, 2).cuda()
    for shape in ((0, 2, 4, 8), (2, 2, 0, 8)):
        x = torch.empty(shape, device="cuda")
        y, ck = ln.softmax_rel_fwd(x, table, ckpt=True)
        assert y.shape == shape and ck.q.shape == (0, 32)
        dx, dt = ln.softmax_rel_bwd(x, ck, table)
        assert dx.shape == shape and (dt == 0).all()


def test_bitwise_repeatable_whatever_the_workspace_holds():
    c = Case("bf16", (3, 4, 200, 700), lens=[700, 300, 1], seed=23)
    y, ck = ln.softmax_rel_fwd(c.x, c.table, ckpt=True, **c.how)
    want = ln.softmax_rel_bwd(c.dy, ck, c.table, **c.how)
    for fill in (0, 255):
        ws = torch.full((1 << 20,), fill, dtype=torch.uint8, device="cuda")
        got = ln.softmax_rel_bwd(c.dy, ck, c.table, workspace=ws, **c.how)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ln.LnError, match="ENOSPACE"):
        ln.softmax_rel_bwd(c.dy, ck, c.table, workspace=ws[:256], **c.how)
    with pytest.raises(ln.LnError, match="EALIGN"):
        ln.softmax_rel_bwd(c.dy, ck, c.table, workspace=ws[16:], **c.how)


def test_given_streams_and_graphs():
    """A step captured and replayed with new inputs, another on a stream of its own meanwhile."""
    c, d = (Case("bf16", (2, 3, 90, 161), both=False, causal=True, seed=s) for s in (24, 25))

    def step(x, dy, stream=None):
        y, ck = ln.softmax_rel_fwd(x, c.table, ckpt=True, stream=stream, **c.how)
        return (y, *ln.softmax_rel_bwd(dy, ck, c.table, stream=stream, **c.how))
    want_c, want_d = step(c.x, c.dy), step(d.x, d.dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x, dy = c.x.clone(), c.dy.clone()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(x, dy)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for inputs, want in ((c, want_c), (d, want_d), (c, want_c)):
        x.copy_(inputs.x)
        dy.copy_(inputs.dy)
        graph.replay()
        eager = step(d.x, d.dy, other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(eager, want_d))


def test_rows_past_two_to_the_thirty_two_bytes():
    """The last rows of a call whose scores end behind 4 GB."""
    B, H, Lq, Lk = 9, 4, 2048, 16384 + 8
    x = torch.empty((B, H, Lq, Lk), dtype=torch.bfloat16, device="cuda")
    x.view(-1)[:1 << 20].normal_()
    for b in range(B):
        x[b] = x.view(-1)[:1 << 20].repeat(H * Lq * Lk // (1 << 20) + 1)[:H * Lq * Lk].view(H, Lq, Lk)
    x[-1, -1, -3:].normal_()
    table = torch.randn(32, H).bfloat16().cuda()
    last = to64(x[-1:, -1:, -3:])
    y64, tol, bk, kept = relref.fwd(last, to64(table)[:, -1:], relref.edges_of(32, 128, True), True, q_pos=[Lq - 3])
    y, ck = ln.softmax_rel_fwd(x, table, y=x, ckpt=True)
    mine = y[-1:, -1:, -3:].clone()
    relref.close("y", to64(mine), y64, relref.stored(tol, y64, "bf16"))
    q, k, values = relref.quantise(to64(mine.view(3, Lk)))
    assert (ck.q[-3:].cpu().numpy() == q).all() and (ck.k[-3:].cpu().numpy() == k).all()
    y[-1, -1, -3:] = torch.from_numpy(last[0, 0]).to(torch.bfloat16).cuda()
    dx, _ = ln.softmax_rel_bwd(y, ck, table, dx=y)
    want, tol = relref.bwd(last, values.reshape(last.shape), bk, kept, 32)[:2]
    relref.close("dx", to64(dx[-1:, -1:, -3:]), want, relref.stored(tol, want, "bf16"))


@pytest.mark.parametrize("dtype,widths", [("bf16", (*range(57, 65), *range(121, 129), *range(249, 257), *range(377, 385))),
                                          ("f32", (*range(29, 33), *range(61, 65), *range(125, 129), *range(189, 193)))])
def test_rows_that_end_around_a_piece_and_share_a_warp(dtype, widths):
    """Rows held by parts of a warp, their ends on either side of a piece by where in 16 bytes they start."""
    for Lk in widths:
        for pad, how in ((0, {}), (1, dict(lens=[Lk, Lk - 2])), (3, dict(both=False, causal=True, q_pos=[Lk - 9, Lk - 3]))):
            c = Case(dtype, (2, 3, 9, Lk), span=24, pad=pad, seed=Lk, **how)
            whole = torch.full((2, 3, 9, Lk + pad), 7.0, dtype=TYPES[dtype], device="cuda")
            y, _ = ln.softmax_rel_fwd(c.x, c.table, y=whole[..., :Lk], **c.how)
            c.check_fwd(y)
            assert (whole[..., Lk:] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 2, 6, 100), (1, 2, 7, 333), (1, 2, 5, 1000), (1, 1, 9, 1501), (1, 1, 4, 2048), (1, 1, 3, 4096),
                                   (1, 1, 5, 4001), (1, 1, 2, 8192), (1, 1, 2, 20001), (1, 1, 1, 70001)])
def test_scores_of_large_magnitude(dtype, shape):
    """Scores a few units apart around a common offset, as an additive mask gives it or the scores themselves have it,
    exact in fp32: the probabilities are those of the scores without it, at any magnitude and any number of warps."""
    B, H, Lq, Lk = shape
    g = torch.Generator().manual_seed(Lk)
    for offset in (0.0, 1000.0, -9984.0, 99840.0, -999424.0, 8126464.0, 2.0 ** 24, -2.0 ** 24, 2.0 ** 26):
        step = max(0.125, 2.0 ** -23 * 2.0 ** np.ceil(np.log2(2 * abs(offset) + 1)))
        units = lambda n, *s: torch.randint(-n, n + 1, s, generator=g) * step  # noqa: E731
        span = max(2, int(6 / step))
        x = units(span, *shape).to(TYPES[dtype])
        x[..., :Lk // 3] -= 4 * step  # (the warps' largest differ)
        table = units(2, 32, H).to(TYPES[dtype])
        mask = torch.full((1, Lk), offset)
        mask[:, 5::11] = -torch.inf
        z = to64(x) + np.moveaxis(to64(table)[relref.buckets_of(relref.taking_part(B, Lq, Lk, False, None, None)[0],
                                                                relref.edges_of(32, 128, True), True)], 3, 1)
        z = z + mask.double().numpy()
        assert (z == z.astype(np.float32)).all()
        e = np.exp(z - z.max(axis=3, keepdims=True))
        want = e / e.sum(axis=3, keepdims=True)
        tol = relref.stored(relref.exact_scores_tol(want, z, Lk), want, dtype)
        got = ln.softmax_rel_fwd(x.cuda(), table.cuda(), mask=mask.to(TYPES[dtype]).cuda())[0]
        relref.close(f"offset {offset}", to64(got), want, tol)
        if dtype == "f32":
            moved = (x.double() + mask.double()).float().cuda()
            got = ln.softmax_rel_fwd(moved, table.cuda())[0]
            relref.close(f"scores around {offset}", to64(got), want, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Lk", [48, 99, 203, 1200, 20001])
def test_gradients_near_the_types_largest(dtype, Lk):
    """dy - sum dy y passes fp32's range, at keys of probability 0, where it counts for nothing, and at others, where
    its product with y does not."""
    mask = torch.zeros(1, Lk)
    mask[:, 5::7] = -float("inf")
    c = Case(dtype, (1, 2, 5, Lk), mask=mask, seed=26)
    c.dy[..., :3] *= 2.0 ** 100
    c.dy[:, :, 1:3] = c.dy[:, :, 1:3].abs().clamp(1, 2) * -2.0 ** 126
    c.dy[..., 5::7] = 3e38
    c.dy[:, :, 2, 7] = 3e38
    y, ck = ln.softmax_rel_fwd(c.x, c.table, mask=c.mask, ckpt=True, **c.how)
    c.check_bwd(ln.softmax_rel_bwd(c.dy, y, c.table, **c.how), to64(y))
    kept = relref.quantise(to64(y).reshape(-1, Lk))[2].reshape(c.shape)
    c.check_bwd(ln.softmax_rel_bwd(c.dy, ck, c.table, **c.how), kept, "kept ")
    dx, dt = ln.softmax_rel_bwd(c.dy, y, c.table, **c.how)
    assert dx.isfinite().all() and dt.isfinite().all()


def test_the_same_without_the_extension_module(monkeypatch):
    c = Case("bf16", (2, 3, 50, 161), lens=[161, 90], seed=27)

    def calls():
        y, ck = ln.softmax_rel_fwd(c.x, c.table, ckpt=True, **c.how)
        mean = rstd = torch.ones(300, device="cuda")
        norm = ln.bwd_ckpt8(c.dy.view(300, 161), ck, c.x[0, 0, 0], mean, rstd)
        rms = ln.rms_bwd_ckpt8(c.dy.view(300, 161), ck, c.x[0, 0, 0], rstd)
        return [y, ck.q, ck.k, *ln.softmax_rel_bwd(c.dy, ck, c.table, **c.how), *ln.softmax_rel_bwd(c.dy, y, c.table, **c.how),
                ln.ckpt8_load(ck), *ln.ckpt8_store(c.x.view(300, 161))[:2], *norm, *rms]
    want = calls()
    assert ln._binding is not ln._NoBinding
    monkeypatch.setattr(ln, "_binding", ln._NoBinding)
    got = calls()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("buckets,both", [(32, True), (7, False), (256, False), (512, True)])
def test_workspace_of_the_size_asked_for(buckets, both):
    c = Case("f32", (2, 3, 60, 130), buckets, 600, both, seed=28)
    y, _ = ln.softmax_rel_fwd(c.x, c.table, **c.how)
    nbytes = ln.softmax_rel_workspace_bytes(buckets, 3, both)
    guard = torch.full((nbytes + 256,), 171, dtype=torch.uint8, device="cuda")
    c.check_bwd(ln.softmax_rel_bwd(c.dy, y, c.table, workspace=guard[:nbytes], **c.how), to64(y))
    assert (guard[nbytes:] == 171).all()
    with pytest.raises(ln.LnError, match="ENOSPACE"):
        ln.softmax_rel_bwd(c.dy, y, c.table, workspace=guard[:nbytes - 1], **c.how)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("edges", [(), (1,), (1, 1, 5, 5, 7), (40, 40), (3, 100, 16384)])
def test_edges_of_any_kind_through_the_c_abi(dtype, both, edges):
    """No edges, edges that fall together (buckets without a distance), and ones behind all rows."""
    B, H, Lq, Lk = 2, 3, 21, 90
    g = torch.Generator().manual_seed(29)
    x, dy = (rows_of((B, H, Lq, Lk), dtype, g) for _ in range(2))
    buckets = (len(edges) + 1) * (2 if both else 1)
    table = torch.randn(buckets, H, generator=g).to(TYPES[dtype]).cuda()
    q_pos = torch.tensor([0, 60], dtype=torch.int32).cuda()
    array = (ctypes.c_int32 * max(1, len(edges)))(*edges)
    rel = ln._REL.pack(B, H, Lq, Lk, table.data_ptr(), ctypes.addressof(array) if edges else 0, 0, q_pos.data_ptr(),
                       len(edges), dtype == "f32", both, 0, 0.5)
    y, dx, dt = torch.empty_like(x), torch.empty_like(dy), torch.empty_like(table)
    lib, stream = ln.lib(), torch.cuda.current_stream().cuda_stream
    nbytes = getattr(lib, f"ln_softmax_rel_workspace_bytes_{dtype}")(rel)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    assert getattr(lib, f"ln_softmax_rel_fwd_{dtype}")(rel, x.data_ptr(), Lk, None, 1, y.data_ptr(), Lk, None, None, stream) == 0
    assert getattr(lib, f"ln_softmax_rel_bwd_{dtype}")(rel, dy.data_ptr(), Lk, y.data_ptr(), Lk, None, None, dx.data_ptr(), Lk,
                                                       dt.data_ptr(), ws.data_ptr(), nbytes, stream) == 0
    y64, tol, bk, kept = relref.fwd(to64(x), to64(table), edges, both, 0.5, q_pos=[0, 60])
    relref.close("y", to64(y), y64, relref.stored(tol, y64, dtype))
    want = relref.bwd(to64(dy), to64(y), bk, kept, buckets, 0.5)
    relref.close("dx", to64(dx), want[0], relref.stored(want[1], want[0], dtype))
    relref.close("dtable", to64(dt), want[2], relref.stored(want[3], want[2], dtype))


def test_a_first_call_captured():
    """A process whose first calls are captured into a graph."""
    code = """
import torch, layernorm_ln_fwd_gb300 as ln
x = torch.randn(2, 3, 40, 300, device="cuda"); table = torch.randn(32, 3, device="cuda")
long = torch.randn(1, 1, 1, 70001, device="cuda")
gamma, stats = torch.ones(300, device="cuda"), torch.ones(240, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
def step():
    y, ck = ln.softmax_rel_fwd(x, table, ckpt=True)
    return (y, *ln.softmax_rel_bwd(x, ck, table), *ln.softmax_rel_bwd(x, y, table), ln.softmax_rel_fwd(long, table[:, :1].contiguous())[0],
            ln.ckpt8_load(ln.ckpt8_store(x.view(240, 300))), *ln.bwd_ckpt8(x.view(240, 300), ck, gamma, stats, stats),
            *ln.rms_bwd_ckpt8(x.view(240, 300), ck, gamma, stats))
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
print("same")
"""
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                          cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert done.returncode == 0 and done.stdout.strip().endswith("same"), done.stderr[-2000:]
