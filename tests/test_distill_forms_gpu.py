"""Forms of the distillation call beside those of test_distill_gpu.py: rows of an odd distance whose
slices differ in their number of copies.  Tolerances: vocabref.py."""
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
