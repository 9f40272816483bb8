"""Forms of the distillation call beside those of test_distill_gpu.py: rows of an odd distance whose slices
differ in their number of copies, gradients at another place of a vector than the logits, lists of columns at
equal distances.  Tolerances: vocabref.py."""
import pytest
import torch

import layernorm_ln_fwd_gb300 as ln
import vocabref as R
from test_distill_gpu import check, teacher_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,rows,V,ld", [
    ("bf16", 950, 16 * 1025 // 2, 8203), ("bf16", 700, 32777, 32777), ("bf16", 620, 49161, 49163),
    ("f32", 700, 16389, 16389), ("f32", 640, 24581, 24585), ("bf16", 330, 65545, 65545), ("f32", 500, 32775, 32777)])
def test_slices_of_one_vector_more_than_whole_copies(dtype, rows, V, ld):
    """1025, 4097, 6145 and twice 4097 vectors: the last copy of a row is one vector, or there is none, by the
    place in memory that the row starts at.  Every block takes several rows, some of weight 0 between."""
    x = R.logits(rows, V, dtype, V, ld=ld)
    ids, t = teacher_of(rows, V, 12, V)
    w = torch.rand(rows, generator=torch.Generator().manual_seed(V)) + 0.5
    w[::5] = 0
    check(x, ids, t, w.cuda(), scale=0.6, dtype=dtype)
    assert ln.device_check() == 0


@pytest.mark.parametrize("dtype,rows,V,ld", [
    ("bf16", 340, 9001, 9001),     # one block of 256 threads a row, several rows a block
    ("bf16", 330, 50257, 50264),   # 512 threads
    ("f32", 330, 9003, 9003), ("f32", 320, 25001, 25005),
    ("bf16", 9, 50257, 50257), ("f32", 20, 40001, 40001),    # clusters, a row each
    ("bf16", 170, 70001, 70003), ("f32", 160, 30011, 30011),  # two blocks a row
    ("bf16", 5, 300001, 300001), ("f32", 155, 131075, 131077)])  # rows that are read again in part
def test_gradient_at_another_place_of_a_vector(dtype, rows, V, ld):
    """The staged kernel's stores of single words: the gradient's rows start elsewhere in 16 bytes than the
    logits', with rows of weight 0, without entries, of repeated columns and with a column outside."""
    x = R.logits(rows, V, dtype, V, ld=ld)
    ids, t = teacher_of(rows, V, 40, V)
    w = torch.rand(rows, generator=torch.Generator().manual_seed(V)) + 0.5
    w[2::7] = 0
    ids[1::5] = -1
    ids[3::6, 20:] = ids[3::6, :20]
    ids[4::40, 0] = V
    w = w.cuda()
    ldd = ld + 3
    for dloss in (1.0 / rows, 1.0):
        buf = torch.full((rows * ldd + 5,), 7.0, dtype=x.dtype, device="cuda")
        out = buf[5:].view(rows, ldd)[:, :V]
        losses, a = check(x, ids, t, w, scale=0.8, dloss=dloss, dtype=dtype, dlogits=out)
        assert a is out and (buf[:5] == 7).all() and (buf[5:].view(rows, ldd)[:, V:] == 7).all()
    same, b = ln.distill(x, ids, t, w, 0.8, 1.0)
    only, none = ln.distill(x, ids, t, w, 0.8, 1.0, want_grad=False)
    torch.cuda.synchronize()
    # the same arithmetic, whichever way it is stored
    assert torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0)) and none is None
    for l in (same, only):
        assert torch.equal(losses.nan_to_num(9.0), l.nan_to_num(9.0))
    assert ln.device_check() == 0


@pytest.mark.parametrize("V,step", [(1000, 64), (1000, 128), (5000, 256), (5000, 512), (50304, 256), (50304, 2048),
                                    (131072, 1024), (131072, 4096)])
def test_columns_at_equal_distances_of_many(V, step):
    """Lists of at least 7 columns whose low bits are equal."""
    K = min(200, V // step)
    assert K >= 7
    ids = (torch.arange(K) * step).flip(0).repeat(30, 1).to(torch.int32).cuda()
    t = torch.randn(30, K, generator=torch.Generator().manual_seed(V)).cuda()
    check(R.logits(30, V, "bf16", V), ids, t, dtype="bf16")
