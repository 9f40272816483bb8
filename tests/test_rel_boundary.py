"""The softmax with a relative position bias and the 8-bit checkpoints without a GPU: the buckets, the
references' own checks, and refusals of the C ABI and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

import relref
import layernorm_ln_fwd_gb300 as ln
from layernorm_ln_fwd_gb300 import build as lnbuild

N = None
P = ctypes.c_void_p(256)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    lnbuild.build()
    return ln.lib()


@pytest.mark.parametrize("buckets,span,both", [(32, 128, True), (32, 128, False), (64, 256, False), (16, 64, True),
                                               (64, 800, False), (64, 64, True), (4, 2, True), (2, 5, False),
                                               (10, 17, True), (7, 100, False)])
def test_edges_are_exact(buckets, span, both):
    edges = ln.rel_edges(buckets, span, both)
    assert list(edges) == relref.edges_of(buckets, span, both)
    assert len(edges) + 1 == (buckets // 2 if both else buckets)


def test_edges_of_the_customary_table():
    assert ln.rel_edges(32, 128, True) == (1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 23, 32, 46, 64, 91)


@pytest.mark.parametrize("args", [(31, 128, True), (2, 128, True), (1, 128, False), (600, 1000, True), (32, 8, True),
                                  (32, 16385, True)])
def test_edges_refuse(args):
    with pytest.raises(ValueError):
        ln.rel_edges(*args)


def test_edges_are_of_whole_numbers():
    for bad in ((32, 200.0), (32.0, 200), (32, "200")):
        with pytest.raises(TypeError):
            ln.rel_edges(*bad)
    assert all(type(e) is int for e in ln.rel_edges(32, 200)) and len(ln.rel_edges(32, 200)) == 15


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(1)
    B, H, Lq, Lk = 2, 2, 5, 9
    edges = ln.rel_edges(8, 6, True)
    x, table, dy = rng.normal(size=(B, H, Lq, Lk)), rng.normal(size=(8, H)), rng.normal(size=(B, H, Lq, Lk))
    how = dict(scale=0.7, lens=[9, 4], q_pos=[0, 2])
    y, _, bk, kept = relref.fwd(x, table, edges, True, **how)
    dx, _, dt, _ = relref.bwd(dy, y, bk, kept, 8, scale=0.7)
    eps = 1e-6
    for i in [(0, 0, 0, 0), (1, 1, 4, 3), (0, 1, 2, 8), (1, 0, 3, 6)]:
        hi, lo = x.copy(), x.copy()
        hi[i] += eps
        lo[i] -= eps
        diff = ((relref.fwd(hi, table, edges, True, **how)[0] - relref.fwd(lo, table, edges, True, **how)[0]) * dy).sum()
        assert abs(diff / (2 * eps) - dx[i]) < 1e-8
    for i in np.ndindex(8, H):
        hi, lo = table.copy(), table.copy()
        hi[i] += eps
        lo[i] -= eps
        diff = ((relref.fwd(x, hi, edges, True, **how)[0] - relref.fwd(x, lo, edges, True, **how)[0]) * dy).sum()
        assert abs(diff / (2 * eps) - dt[i]) < 1e-8


def test_reference_probabilities_against_torch():
    rng = np.random.default_rng(2)
    x, table = rng.normal(size=(2, 3, 4, 7)), rng.normal(size=(4, 3))
    edges = ln.rel_edges(4, 5, False)
    y, _, bk, _ = relref.fwd(x, table, edges, False, scale=1.3, causal=True, q_pos=[3, 0])
    at = torch.arange(4)[None, :, None] + torch.tensor([3, 0])[:, None, None]
    d = torch.arange(7) - at
    bias = torch.tensor(table)[torch.tensor(bk)].permute(0, 3, 1, 2)
    z = (torch.tensor(x) * 1.3 + bias).masked_fill((d > 0)[:, None], -np.inf)
    np.testing.assert_allclose(y, torch.softmax(z, dim=3).numpy(), rtol=1e-12)


def test_reference_checkpoint():
    x = np.array([[127.0, 1.0, 0.5, -0.5, 1.5, 2.5] + [0.0] * 26 + [127.5, 3.0], [1.0] * 34])
    q, k, v = relref.quantise(x)
    assert k.tolist() == [[127, 128], [121, 121]] and q[0, :6].tolist() == [127, 1, 0, 0, 2, 2]
    assert q[0, 32:34].tolist() == [64, 2] and (v[1] == 1.0).all()
    assert (relref.quantise(v)[2] == v).all()
    assert np.isnan(relref.quantise(np.array([[1.0, np.inf]]))[2]).all()
    assert (relref.quantise(np.array([[2.0 ** -126, 2.0 ** -128]]))[2] == [[2.0 ** -126, 0]]).all()


class Packed:
    """The binding's ln_rel with some of its fields changed."""
    names = ("B", "H", "Lq", "Lk", "table", "edges", "lens", "q_pos", "n_edges", "table_f32", "bidirectional", "causal",
             "scale")

    def __init__(self, edge=(1, 2, 4), **over):
        self.held = (ctypes.c_int32 * max(len(edge), 1))(*edge)
        a = dict(B=2, H=2, Lq=3, Lk=8, table=256, edges=ctypes.addressof(self.held), lens=0, q_pos=0, n_edges=len(edge),
                 table_f32=0, bidirectional=0, causal=0, scale=1.0)
        a.update(over)
        self.bytes = ln._REL.pack(*(a[n] for n in self.names))


BAD = [(dict(B=-1), 1), (dict(H=0), 1), (dict(Lq=-1), 1), (dict(Lk=0), 1), (dict(scale=float("nan")), 1),
       (dict(scale=float("inf")), 1), (dict(n_edges=-1), 1), (dict(edges=0), 1), (dict(edge=(0, 1)), 1),
       (dict(edge=(3, 2)), 1), (dict(edge=(1, 16385)), 3), (dict(Lk=(1 << 20) + 1), 3), (dict(H=65537), 3),
       (dict(n_edges=256), 3), (dict(Lq=2**29 + 1, H=1, B=1), 3), (dict(Lq=2**31 - 2**16, H=2), 3), (dict(B=2**40), 3)]


@pytest.mark.parametrize("over,status", BAD)
def test_rel_sizes(lib, over, status):
    rel = Packed(**over)
    r = rel.bytes
    ld = 1 << 21
    for s in ("f32", "bf16"):
        assert getattr(lib, f"ln_softmax_rel_fwd_{s}")(r, P, ld, N, 1, P, ld, N, N, N) == status
        assert getattr(lib, f"ln_softmax_rel_bwd_{s}")(r, P, ld, P, ld, N, N, P, ld, P, P, 1 << 30, N) == status
        assert getattr(lib, f"ln_softmax_rel_workspace_bytes_{s}")(r) == 0


def test_rel_fwd_arguments(lib):
    rel = Packed()
    other = ctypes.c_void_p(512)
    for f in (lib.ln_softmax_rel_fwd_f32, lib.ln_softmax_rel_fwd_bf16):
        def call(r=rel, x=P, ldx=8, mask=N, mask_rows=1, y=other, ldy=8, q=N, k=N):
            return f(r and r.bytes, x, ldx, mask, mask_rows, y, ldy, q, k, N)
        assert call(r=None) == 1 and call(x=N) == 1 and call(y=N) == 1
        assert call(ldx=7) == 1 and call(ldy=7) == 1 and call(ldx=2**29 + 1) == 3 and call(ldy=2**62) == 3
        assert call(mask=P, mask_rows=0) == 1 and call(q=P) == 1 and call(k=P) == 1
        assert call(y=P, ldy=9) == 1  # in place, but rows elsewhere
        assert call(r=Packed(table=0)) == 1
        assert call(q=ctypes.c_void_p(264), k=P) == 2
        assert call(r=Packed(B=0), x=N, y=N) == 0 and call(r=Packed(Lq=0), x=N, y=N) == 0
    assert lib.ln_last_launch_count() == 0


def test_rel_bwd_arguments(lib):
    rel = Packed()
    other = ctypes.c_void_p(512)
    for f in (lib.ln_softmax_rel_bwd_f32, lib.ln_softmax_rel_bwd_bf16):
        def call(r=rel, dy=P, ldd=8, y=P, ldy=8, q=N, k=N, dx=other, ldx=8, dt=N, ws=N, n=0):
            return f(r and r.bytes, dy, ldd, y, ldy, q, k, dx, ldx, dt, ws, n, N)
        assert call(r=None) == 1 and call(dy=N) == 1 and call(y=N) == 1 and call(dx=N) == 1
        assert call(ldd=7) == 1 and call(ldy=7) == 1 and call(ldx=7) == 1
        assert call(ldd=2**30) == 3 and call(ldy=2**30) == 3 and call(ldx=2**30) == 3
        assert call(q=P, k=P) == 1 and call(y=N, q=P) == 1  # both, or half a checkpoint
        assert call(y=N, q=ctypes.c_void_p(264), k=P) == 2
        assert call(dt=P) == 1 and call(dt=P, ws=ctypes.c_void_p(272), n=1 << 20) == 2
        assert call(dx=P, ldx=9) == 1
        assert call(r=Packed(B=0), dy=N, y=N, dx=N) == 0
    assert lib.ln_last_launch_count() == 0


def test_ckpt8_arguments(lib):
    for s in ("f32", "bf16"):
        store, load = getattr(lib, f"ln_ckpt8_store_{s}"), getattr(lib, f"ln_ckpt8_load_{s}")
        assert store(N, 8, 4, 8, P, P, N) == 1 and store(P, 8, 4, 8, N, P, N) == 1 and store(P, 8, 4, 8, P, N, N) == 1
        assert store(P, 7, 4, 8, P, P, N) == 1 and store(P, 8, -1, 8, P, P, N) == 1 and store(P, 8, 4, 0, P, P, N) == 1
        assert store(P, 1 << 21, 4, (1 << 20) + 1, P, P, N) == 3 and store(P, 2**62, 4, 8, P, P, N) == 1
        assert store(P, 8, 4, 8, ctypes.c_void_p(264), P, N) == 2 and store(N, 8, 0, 8, N, N, N) == 0
        assert load(N, P, 4, 8, P, 8, N) == 1 and load(P, N, 4, 8, P, 8, N) == 1 and load(P, P, 4, 8, N, 8, N) == 1
        assert load(P, P, 4, 8, P, 7, N) == 1 and load(ctypes.c_void_p(264), P, 4, 8, P, 8, N) == 2
        assert load(N, N, 0, 8, N, 8, N) == 0
        b, r = getattr(lib, f"ln_bwd_ckpt8_{s}"), getattr(lib, f"ln_rms_bwd_ckpt8_{s}")

        def call(dy=P, q=P, k=P, g=P, m=P, rs=P, dx=P, dg=P, db=P, rows=4, cols=8, ws=P, n=1 << 20):
            return b(dy, q, k, g, m, rs, dx, dg, db, rows, cols, ws, n, N)

        def rms(dy=P, q=P, k=P, g=P, rs=P, dx=P, dg=P, rows=4, cols=8, ws=P, n=1 << 20):
            return r(dy, q, k, g, rs, dx, dg, rows, cols, ws, n, N)
        for f, names in ((call, ("dy", "q", "k", "g", "m", "rs", "dx", "dg", "db", "ws")),
                         (rms, ("dy", "q", "k", "g", "rs", "dx", "dg", "ws"))):
            for what in names:
                assert f(**{what: N}) == 1, what
            assert f(rows=-1) == 1 and f(cols=0) == 1 and f(cols=ln.MAX_COLS + 1) == 3
            assert f(ws=ctypes.c_void_p(272)) == 2 and f(q=ctypes.c_void_p(264)) == 2
    assert lib.ln_bwd_ckpt8_workspace_bytes(4, 0) == 0 and lib.ln_bwd_ckpt8_workspace_bytes(-1, 4) == 0
    assert lib.ln_last_launch_count() == 0


def test_binding_refuses():
    x, table = torch.zeros(2, 3, 4, 8), torch.zeros(8, 3)
    ck = ln.Ckpt8(torch.zeros(24, 32, dtype=torch.int8), torch.zeros(24, 1, dtype=torch.uint8), 8)
    for call in (lambda: ln.softmax_rel_fwd(x, table), lambda: ln.softmax_rel_bwd(x, x, table),
                 lambda: ln.softmax_rel_bwd(x, ck, table), lambda: ln.ckpt8_store(x[0, 0]), lambda: ln.ckpt8_load(ck)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for bad in (lambda: ln.softmax_rel_fwd(x[0], table), lambda: ln.softmax_rel_fwd(x, table[:, :2]),
                lambda: ln.softmax_rel_fwd(x, table, lens=torch.zeros(3, dtype=torch.int32)),
                lambda: ln.softmax_rel_fwd(x, table, mask=torch.zeros(4, 7)),
                lambda: ln.softmax_rel_fwd(x.transpose(1, 2), torch.zeros(8, 4)),
                lambda: ln.softmax_rel_fwd(x.transpose(2, 3), table),
                lambda: ln.softmax_rel_fwd(x, torch.zeros(7, 3)),
                lambda: ln.softmax_rel_fwd(x, table, max_distance=2),
                lambda: ln.softmax_rel_bwd(x, x[:, :, :3], table),
                lambda: ln.softmax_rel_bwd(x, ck._replace(cols=9), table),
                lambda: ln.softmax_rel_bwd(x, ck._replace(q=ck.q[:23]), table),
                lambda: ln.ckpt8_store(x), lambda: ln.ckpt8_load(ck._replace(cols=40)),
                lambda: ln.ckpt8_load(ck, out=torch.zeros(24, 9)),
                lambda: ln.bwd_ckpt8(x[0, 0], ck, table[0], table[0], table[0])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ln.softmax_rel_fwd(x.double(), table), lambda: ln.softmax_rel_fwd(x, table.bfloat16()),
                lambda: ln.softmax_rel_fwd(x, table, lens=torch.zeros(2, dtype=torch.int64)),
                lambda: ln.ckpt8_load((1, 2, 3)), lambda: ln.ckpt8_load(ck, torch.float16),
                lambda: ln.softmax_rel_bwd(x, x.bfloat16(), table)):
        with pytest.raises(TypeError):
            bad()


@pytest.mark.parametrize("content", [None, b"not a module"])
def test_calls_without_the_extension_module(monkeypatch, tmp_path, content):
    """Where it was not built, or for another torch, a call goes through ctypes and says so once."""
    path = tmp_path / "_binding_other.so"
    if content:
        path.write_bytes(content)
    monkeypatch.setattr(lnbuild, "binding_path", lambda: str(path))
    monkeypatch.setattr(ln, "_binding", None)
    x, table = torch.zeros(2, 3, 4, 8), torch.zeros(8, 3)
    with pytest.warns(RuntimeWarning, match="ctypes"), pytest.raises(ValueError, match="CUDA"):
        ln.ckpt8_store(x[0, 0])
    ck = ln.Ckpt8(torch.zeros(24, 32, dtype=torch.int8), torch.zeros(24, 1, dtype=torch.uint8), 8)
    for call in (lambda: ln.softmax_rel_fwd(x, table), lambda: ln.softmax_rel_bwd(x, ck, table, 40), lambda: ln.ckpt8_load(ck),
                 lambda: ln.rms_bwd_ckpt8(x.view(24, 8), ck, x[0, 0, 0], torch.zeros(24))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_the_extension_module_is_of_this_torch(lib, monkeypatch, tmp_path):
    mine = lnbuild.binding_path()
    assert lnbuild.up_to_date() and lnbuild._built() == [lnbuild.LIB, mine]
    (tmp_path / "__init__.py").write_text("")
    (tmp_path / "version.py").write_text("from typing import Optional\n__version__ = '99.1.0+cu999'\n")
    spec = lnbuild.importlib.util.spec_from_file_location("torch", str(tmp_path / "__init__.py"))
    with monkeypatch.context() as m:  # another torch
        m.setattr(lnbuild.importlib.util, "find_spec", lambda name: spec)
        assert "99_1_0_cu999" in lnbuild.binding_path() and lnbuild.binding_path() != mine and not lnbuild.up_to_date()
    with monkeypatch.context() as m:  # none, or no compiler of C++: the library alone
        m.setattr(lnbuild.importlib.util, "find_spec", lambda name: None)
        assert lnbuild.binding_path() is None and lnbuild._built() == [lnbuild.LIB] and lnbuild.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(lnbuild.shutil, "which", lambda name: None)
        assert lnbuild._built() == [lnbuild.LIB] and lnbuild.up_to_date()


def test_the_library_is_built_whatever_comes_of_the_module(monkeypatch, tmp_path):
    monkeypatch.setattr(lnbuild, "LIB", str(tmp_path / "libln.so"))
    monkeypatch.setattr(lnbuild, "BUILD", str(tmp_path))
    monkeypatch.setattr(lnbuild, "_compile", lambda src: (src + ".o", ""))
    monkeypatch.setattr(lnbuild, "nvcc", lambda: "nvcc")

    def link(cmd, **_):
        open(cmd[cmd.index("-o") + 1], "w").close()
        return lnbuild.subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(lnbuild.subprocess, "run", link)

    def fails(path):
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(lnbuild, "_compile_binding", fails)
    with pytest.raises(RuntimeError, match=r"g\+\+ failed"):
        lnbuild.build(force=True)
    assert (tmp_path / "libln.so").exists()
    (tmp_path / "libln.so").unlink()
    monkeypatch.setattr(lnbuild.shutil, "which", lambda name: None)
    assert lnbuild.build(force=True) == str(tmp_path / "libln.so") and (tmp_path / "libln.so").exists()


def test_workspace_size_refuses(lib):
    with pytest.raises(ValueError):
        ln.softmax_rel_workspace_bytes(31, 4)
    for buckets, heads, both in ((0, 4, True), (32, 0, True), (514, 4, True), (257, 4, False), (32, 65537, False)):
        assert ln.softmax_rel_workspace_bytes(buckets, heads, both) == 0
