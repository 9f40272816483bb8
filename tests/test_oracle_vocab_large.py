"""The float64 oracle of the log probabilities' gradient for rows whose log-sum does not fit fp32, as the forward
leaves it (CPU only): pinned to torch's float64 autograd, which takes the logits alone, and to the uniform row."""
import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("shift", [0.0, 300.0, 1e4, -1e6])
@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_gradient_from_a_rounded_log_sum_is_autograd(shift, scale):
    rng = np.random.default_rng(3)
    x = rng.normal(0, 3, (5, 23)) + shift
    t = rng.integers(0, 23, 5)
    dl, de = rng.normal(size=5), rng.normal(size=5)
    f = oracle.logprobs(x, t, scale)
    lse = f["lse"].astype(np.float32)
    g = oracle.logprobs_bwd(x, t, lse, f["entropy"], dl, de, scale)
    xt = torch.tensor(x, requires_grad=True)
    logq = torch.log_softmax(xt * scale, dim=1)
    H = -(logq.exp() * logq).sum(dim=1)
    logp = logq.gather(1, torch.tensor(t)[:, None])[:, 0]
    (logp * torch.tensor(dl) + H * torch.tensor(de)).sum().backward()
    # below 512 the oracle goes by the given lse: half a step, 2^-16, of every weight and its log
    # (weights of at most 1, logs of at most 25); beyond it by the logits
    tol = 2.0 ** -16 * scale * (np.abs(dl) + 30 * np.abs(de))[:, None] if abs(shift) < 512 else 1e-8
    assert (np.abs(g - xt.grad.numpy()) <= tol).all()


def test_gradient_of_a_row_of_the_lowest_value_is_uniform():
    low = np.full((2, 64), float(np.finfo(np.float32).min))
    f = oracle.logprobs(low, np.array([3, 60]))
    g = oracle.logprobs_bwd(low, np.array([3, 60]), f["lse"].astype(np.float32), f["entropy"], np.ones(2), np.ones(2))
    want = np.full((2, 64), -1 / 64)
    want[0, 3] += 1
    want[1, 60] += 1
    np.testing.assert_allclose(g, want, atol=1e-12)
