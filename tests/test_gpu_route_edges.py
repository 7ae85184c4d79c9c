"""Weights of finite logits whose scores are beyond FP32, some of them beyond 64 bits: the reference takes their logarithms.

The bound is that of test_gpu_route.py: (spread + 48) u before normalising, twice that and 7 u after; logarithms up to
1100 in 64 bits add 2^-42.
"""
import numpy as np
import pytest
import torch

import dense_gemm_13_gb300 as g13
from tests import blocks_ref as ref
from tests.test_gpu_route import DT, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


def check(z, k, bias=None, scores="softmax", normalize=True, scale=1.0, **kw):
    kw = dict(kw, scores=scores, normalize=normalize, scale=scale)
    ids, w = g13.route(z, k, bias=None if bias is None else torch.from_numpy(bias).cuda(), **kw)
    z64 = z.double().cpu().numpy()
    rid = ref.route(z64, k, bias=None if bias is None else bias.astype(np.float64), **kw)[0]
    assert np.array_equal(ids.cpu().numpy(), rid)
    log = z64 - np.logaddexp.reduce(z64, 1, keepdims=True) if scores == "softmax" else -np.logaddexp(0, -z64)
    log = np.take_along_axis(log, rid, 1)
    tol = np.full(log.shape, 48.0)
    if scores == "softmax":
        tol += 2 * (z64.max(1, keepdims=True) - np.take_along_axis(z64, rid, 1))
    if normalize:
        log = log - np.logaddexp.reduce(log, 1, keepdims=True)
        tol = tol + tol.max(1, keepdims=True) + 7
    want = np.exp(log) * scale
    err = np.abs(w.double().cpu().numpy() - want)
    assert (err <= (tol * 2.0 ** -24 + 2.0 ** -42) * want + 1e-37).all()
    return ids, w


@pytest.mark.parametrize("E,k", [(4, 2), (64, 6), (200, 8), (512, 32)])
@pytest.mark.parametrize("at", [0, -80, -89, -95, -100, -104, -200, -600])
@pytest.mark.parametrize("dtype", list(DT))
def test_sigmoid_far_below_zero(E, k, at, dtype):
    # all logits near `at`, and one token with a single chosen one far above the rest
    r = rng("sigmoid", E, at)
    z = at + r.standard_normal((40, E)).astype(np.float32)
    z[1, E // 2] += 150
    z[2] -= np.arange(E)
    z = torch.from_numpy(z).to(DT[dtype]).cuda()
    ids, w = check(z, k, scores="sigmoid")
    assert bool(torch.isfinite(w).all()) and bool(((w.double().sum(1) - 1).abs() < 1e-5).all())
    check(z, k, scores="sigmoid", scale=2.5, groups=2 if k < E // 2 else 1, top_groups=1)
    bias = (r.permutation(E) / E).astype(np.float32)  # what decides among scores of zero
    check(z, k, bias, scores="sigmoid")
    _, w = check(z, k, scores="sigmoid", normalize=False)
    assert bool(torch.isfinite(w).all())


@pytest.mark.parametrize("below", [60, 88, 104, 120, 300])
@pytest.mark.parametrize("dtype", list(DT))
def test_softmax_of_experts_far_below_the_largest(below, dtype):
    # the bias chooses only experts whose scores FP32 cannot hold
    E, k = 96, 5
    r = rng("softmax", below)
    z = r.standard_normal((30, E)).astype(np.float32) * 2
    z[:, 48:] -= below
    z = torch.from_numpy(z).to(DT[dtype]).cuda()
    bias = np.where(np.arange(E) < 48, -4.0, r.permutation(E) / E).astype(np.float32)
    ids, w = check(z, k, bias)
    assert bool((ids >= 48).all()) and bool(torch.isfinite(w).all())
    check(z, k, bias, scale=16.0)
    _, w = check(z, k, bias, normalize=False)
    assert bool(torch.isfinite(w).all())


def test_scores_of_zero():
    # what has no weights: chosen scores that are all exactly zero, normalised
    inf = float("inf")
    z = torch.tensor([[-inf, -inf, 1.0, 2.0], [-inf, 0.0, 1.0, 2.0]], device="cuda")
    bias = torch.tensor([9.0, 8.0, 0.0, 0.0], device="cuda")
    for scores in ("softmax", "sigmoid"):
        ids, w = g13.route(z, 2, bias=bias, scores=scores)
        assert ids.tolist() == [[0, 1]] * 2 and bool(w[0].isnan().all()) and w[1].tolist() == [0.0, 1.0]
        ids, w = g13.route(z, 2, bias=bias, scores=scores, normalize=False)
        assert w[0].tolist() == [0.0, 0.0] and float(w[1, 0]) == 0 and float(w[1, 1]) > 0


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [1.0, 30.0, 1e3, 1e5])
@pytest.mark.parametrize("groups,per", [(16, 2), (32, 2), (8, 8), (4, 60)])
def test_group_scores_of_biases_that_cancel(scores, size, groups, per):
    # the two best of a group have biases of opposite sign, whose sum FP32 rounds far more coarsely than its own size
    # allows
    r = rng("cancel", scores, size, groups)
    z = torch.from_numpy(r.standard_normal((1500, groups * per)).astype(np.float32) * 2).cuda()
    bias = np.full((groups, per), -3 * size, np.float32)
    bias[:, 0] = size * (1 + r.random(groups))
    bias[:, 1] = -bias[:, 0]
    bias = np.take_along_axis(bias, r.permuted(np.tile(np.arange(per), (groups, 1)), axis=1), 1).reshape(-1)
    for top in (1, 3):
        check(z, 2, bias, scores=scores, groups=groups, top_groups=top, group_score="top2")


def test_group_scores_with_experts_that_are_masked():
    # a bias of -infinity takes experts out: some of a group, all but one, all
    inf, r = float("inf"), rng("masked")
    z = torch.from_numpy(r.standard_normal((400, 64)).astype(np.float32)).cuda()
    bias = (r.standard_normal(64) * 0.1).astype(np.float32)
    bias[:8], bias[9:16], bias[20:22] = -inf, -inf, -inf
    for kw in (dict(), dict(groups=8, top_groups=3, group_score="top2"), dict(groups=8, top_groups=3)):
        check(z, 6, bias, scores="sigmoid", **kw)
