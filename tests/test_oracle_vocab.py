"""Pins for the float64 oracle of the operators over rows of logits (CPU only): token log
probabilities with entropy, rank and top alternatives, their gradient, and distillation from a
teacher's top logits.  Pinned to torch's float64 log_softmax, kl_div and autograd, to finite
differences, to closed forms (uniform rows), and against planted mistakes."""
import numpy as np
import pytest
import torch

import oracle


def _case(rows, V, seed, spread=3.0):
    rng = np.random.default_rng(seed)
    return rng.normal(0, spread, (rows, V)), rng.integers(0, V, rows), rng


@pytest.mark.parametrize("scale", [1.0, 0.4, 1.7])
def test_logprobs_match_torch(scale):
    x, t, _ = _case(7, 53, 1)
    r = oracle.logprobs(x, t, scale, top=5)
    logq = torch.log_softmax(torch.tensor(x) * scale, dim=1)
    at = torch.tensor(t)[:, None]
    np.testing.assert_allclose(r["logp"], logq.gather(1, at)[:, 0].numpy(), rtol=1e-13, atol=1e-14)
    np.testing.assert_allclose(r["lse"], torch.logsumexp(torch.tensor(x) * scale, 1).numpy(), rtol=1e-13)
    np.testing.assert_allclose(r["entropy"], torch.distributions.Categorical(logits=logq).entropy().numpy(),
                               rtol=1e-12)
    v, i = logq.topk(5, dim=1)
    np.testing.assert_array_equal(r["top_ids"], i.numpy())
    np.testing.assert_allclose(r["top_logp"], v.numpy(), rtol=1e-13, atol=1e-14)
    order = np.argsort(-x, axis=1)
    np.testing.assert_array_equal(r["ranks"], 1 + np.argmax(order == t[:, None], axis=1))


def test_logprobs_closed_forms_ties_and_masks():
    x = np.full((3, 64), 2.5)
    r = oracle.logprobs(x, np.array([0, 63, 5]), 0.3, top=4)
    np.testing.assert_allclose(r["logp"], -np.log(64), rtol=1e-13)
    np.testing.assert_allclose(r["entropy"], np.log(64), rtol=1e-13)
    np.testing.assert_array_equal(r["top_ids"], [[0, 1, 2, 3]] * 3)  # ties: the lowest column
    np.testing.assert_array_equal(r["ranks"], 1)
    low = oracle.logprobs(np.full((1, 64), -3.39e38), np.array([9]))  # masked throughout: uniform
    np.testing.assert_allclose([low["entropy"][0], -low["logp"][0]], np.log(64), rtol=1e-13)
    x[0, 3:] = -np.inf
    x[1] = -np.inf
    x[2, 7] = np.nan
    r = oracle.logprobs(x, np.array([5, -1, 64]), 1.0, top=4)
    np.testing.assert_array_equal(r["top_ids"][0], [0, 1, 2, -1])
    np.testing.assert_array_equal(r["top_ids"][1], -1)
    np.testing.assert_allclose(r["entropy"][0], np.log(3), rtol=1e-13)
    assert r["logp"][0] == -np.inf and r["logp"][1] == 0 and np.isnan(r["logp"][2])
    assert np.isnan(r["entropy"][1]) and r["lse"][1] == -np.inf and np.isnan(r["entropy"][2])
    np.testing.assert_array_equal(r["ranks"], [4, 0, 0])


@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_logprobs_gradient_is_autograd_and_differences(scale):
    x, t, rng = _case(5, 17, 2)
    dl, de = rng.normal(size=5), rng.normal(size=5)
    f = oracle.logprobs(x, t, scale)
    g = oracle.logprobs_bwd(x, t, f["lse"], f["entropy"], dl, de, scale)
    xt = torch.tensor(x, requires_grad=True)
    logq = torch.log_softmax(xt * scale, dim=1)
    H = -(logq.exp() * logq).sum(dim=1)
    logp = logq.gather(1, torch.tensor(t)[:, None])[:, 0]
    (logp * torch.tensor(dl) + H * torch.tensor(de)).sum().backward()
    np.testing.assert_allclose(g, xt.grad.numpy(), rtol=1e-11, atol=1e-14)
    np.testing.assert_allclose(g.sum(axis=1), 0, atol=1e-13)
    h = 1e-6
    for j in range(17):
        up, dn = x.copy(), x.copy()
        up[0, j] += h
        dn[0, j] -= h
        a, b = oracle.logprobs(up, t, scale), oracle.logprobs(dn, t, scale)
        num = (dl[0] * (a["logp"][0] - b["logp"][0]) + de[0] * (a["entropy"][0] - b["entropy"][0])) / (2 * h)
        assert abs(num - g[0, j]) < 1e-7


def test_logprobs_gradient_rows_left_out():
    x, t, _ = _case(4, 9, 3)
    x[2] = np.nan
    t = np.array([1, -1, 3, 9])
    f = oracle.logprobs(x, t)
    g = oracle.logprobs_bwd(x, t, f["lse"], dlogp=np.array([1.0, 1.0, 0.0, 1.0]))
    assert np.all(g[1] == 0) and np.all(g[2] == 0) and np.all(np.isnan(g[3])) and np.all(np.isfinite(g[0]))


@pytest.mark.parametrize("scale", [1.0, 0.5])
def test_distill_matches_torch_kl_and_autograd(scale):
    x, _, rng = _case(6, 31, 4)
    ids = np.stack([rng.permutation(31)[:5] for _ in range(6)])
    t = rng.normal(0, 2, (6, 5))
    w = rng.uniform(0.5, 2, 6)
    r = oracle.distill(x, ids, t, w, scale, dloss=0.25)
    xt = torch.tensor(x, requires_grad=True)
    dense = torch.full((6, 31), -np.inf, dtype=torch.float64).scatter(1, torch.tensor(ids), torch.tensor(t) * scale)
    logq = torch.log_softmax(xt * scale, dim=1)
    kl = torch.nn.functional.kl_div(logq, torch.softmax(dense, dim=1), reduction="none").sum(dim=1)
    np.testing.assert_allclose(r["loss"], (kl * torch.tensor(w)).detach().numpy(), rtol=1e-12)
    (0.25 * (kl * torch.tensor(w)).sum()).backward()
    np.testing.assert_allclose(r["dx"], xt.grad.numpy(), rtol=1e-11, atol=1e-14)
    # Log probabilities in place of logits: a constant per row does not matter.
    lp = t - np.log(np.exp(t).sum(axis=1, keepdims=True))
    np.testing.assert_allclose(oracle.distill(x, ids, lp, w, scale)["loss"], r["loss"], rtol=1e-12)


def test_distill_differences_short_lists_and_repeated_columns():
    x, _, rng = _case(3, 11, 5)
    ids = np.array([[4, 4, 0, -1], [2, -1, -1, -1], [-1, -1, -1, -1]])
    t = rng.normal(size=(3, 4))
    r = oracle.distill(x, ids, t)
    assert r["loss"][2] == 0 and np.all(r["dx"][2] == 0)
    h = 1e-6
    for i in range(2):
        for j in range(11):
            up, dn = x.copy(), x.copy()
            up[i, j] += h
            dn[i, j] -= h
            num = (oracle.distill(up, ids, t)["loss"][i] - oracle.distill(dn, ids, t)["loss"][i]) / (2 * h)
            assert abs(num - r["dx"][i, j]) < 1e-8
    # A single entry is the cross-entropy of that column.
    np.testing.assert_allclose(r["loss"][1], -oracle.logprobs(x, np.array([0, 2, 0]))["logp"][1], rtol=1e-13)
    # Left out by weight, out of range, and weight 0 next to a student's -inf.
    x[0, 3] = -np.inf
    r = oracle.distill(x, np.array([[3, 1], [11, 0], [0, 1]]), np.array([[-np.inf, 0.0], [0, 0], [0, 0]]),
                       np.array([1.0, 1.0, 0.0]))
    assert np.isfinite(r["loss"][0]) and np.isnan(r["loss"][1]) and np.all(np.isnan(r["dx"][1]))
    assert r["loss"][2] == 0 and np.all(r["dx"][2] == 0)


@pytest.mark.parametrize("kind", ["reverse", "no_renormalisation", "no_scale"])
def test_pins_catch_planted_mistakes(kind):
    x, _, rng = _case(4, 20, 6)
    ids = np.stack([rng.permutation(20)[:4] for _ in range(4)])
    t = rng.normal(size=(4, 4))
    scale = 0.5
    logq = oracle.logprobs(x, scale=scale)["logq"]
    lq = np.take_along_axis(logq, ids, 1)
    u = scale * t
    lp = u - np.log(np.exp(u).sum(axis=1, keepdims=True))
    good = oracle.distill(x, ids, t, scale=scale)["loss"]
    np.testing.assert_allclose((np.exp(lp) * (lp - lq)).sum(axis=1), good, rtol=1e-12)
    if kind == "reverse":
        bad = (np.exp(lq) * (lq - lp)).sum(axis=1)
    elif kind == "no_renormalisation":
        bad = (np.exp(u) * (u - lq)).sum(axis=1)
    else:
        raw = t - np.log(np.exp(t).sum(axis=1, keepdims=True))
        bad = (np.exp(raw) * (raw - lq)).sum(axis=1)
    assert not np.allclose(bad, good, rtol=1e-3)
