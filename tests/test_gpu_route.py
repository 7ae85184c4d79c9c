"""Routing on the GPU against 64 bits, and a layer on a choice made beforehand.

The experts have to be those of the exact order.  Weights, relative, u = 2^-24: softmax: both exponents' arguments
round (u |z - max| each), expf is off by 2 units (4 u), the sum of E exponentials by at most 22 additions, two divisions;
sigmoid: expf and two roundings; normalising: at most 6 additions and a division of sums as exact; the scale once:
    (2 |z - max| + 48) u   before normalising, twice that and 7 u after.
"""
import zlib

import numpy as np
import pytest
import torch

import dense_gemm_13_gb300 as g13
from tests import blocks_ref as ref
from tests import moe_ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


def rng(*key):
    return np.random.default_rng(zlib.crc32(repr(key).encode()))


def check(z, k, bias=None, **kw):
    """z: a CUDA tensor; bias: float32 numpy or None."""
    ids, w = g13.route(z, k, bias=None if bias is None else torch.from_numpy(bias).cuda(), **kw)
    z64 = z.double().cpu().numpy()
    rid, rw = ref.route(z64, k, bias=None if bias is None else bias.astype(np.float64), **kw)
    got = ids.cpu().numpy()
    assert np.array_equal(got, rid), f"{np.sum((got != rid).any(1))} of {len(rid)} tokens"
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    spread = 2 * (z64.max(1, keepdims=True) - np.take_along_axis(z64, rid, 1)) if kw.get("scores", "softmax") == "softmax" else 0
    tol = (spread + 48) * 2.0 ** -24
    if kw.get("normalize", True):
        tol = (tol + np.max(tol, axis=-1, keepdims=True) if np.ndim(tol) else 2 * tol) + 7 * 2.0 ** -24
    err = np.abs(w.double().cpu().numpy() - rw)
    assert (err <= tol * np.abs(rw) + 1e-37).all()
    return ids, w


CASES = [  # T, E, k, options
    (1, 1, 1, {}), (3, 8, 2, {}), (7, 32, 32, dict(normalize=False)), (1, 64, 6, dict(scale=2.5)),
    (100, 33, 5, dict(scores="sigmoid")), (50, 512, 8, {}), (20, 512, 32, dict(scores="sigmoid", normalize=False)),
    (300, 160, 6, dict(groups=8, top_groups=3)), (64, 256, 8, dict(groups=8, top_groups=4, group_score="top2", scores="sigmoid")),
    (40, 96, 4, dict(groups=32, top_groups=5)), (40, 32, 3, dict(groups=32, top_groups=3, group_score="top2")),
    (30, 30, 4, dict(groups=3, top_groups=1, group_score="top2")), (30, 30, 4, dict(groups=5, top_groups=5, group_score="top2")),
    (25, 500, 12, dict(groups=20, top_groups=7, group_score="top2", scores="sigmoid")), (3000, 24, 4, dict(groups=2, top_groups=1))]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:3])) + "".join(f"-{v}" for v in c[3].values()))
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("biased", [False, True])
def test_route(case, dtype, biased):
    T, E, k, kw = case
    r = rng(case, dtype, biased)
    z = torch.from_numpy(r.standard_normal((T, E)).astype(np.float32) * 2).to(DT[dtype]).cuda()
    bias = (r.standard_normal(E) * (0.1 if kw.get("scores") == "sigmoid" else 0.02)).astype(np.float32) if biased else None
    ids, w = check(z, k, bias, **kw)
    for _ in range(2):
        ids2, w2 = g13.route(z, k, bias=None if bias is None else torch.from_numpy(bias).cuda(), **kw)
        assert torch.equal(ids, ids2) and torch.equal(w, w2)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(scores):
    r = rng("ties", scores)
    z = torch.from_numpy(r.integers(-1, 2, (200, 96)).astype(np.float32)).cuda()
    check(z, 10, scores=scores)
    check(z, 10, np.zeros(96, np.float32), scores=scores)
    check(z, 10, scores=scores, groups=8, top_groups=3)
    check(z, 10, scores=scores, groups=8, top_groups=3, group_score="top2")
    check(z, 10, r.integers(0, 2, 96).astype(np.float32), scores=scores, groups=12, top_groups=5, group_score="top2")
    check(z * 0, 32, scores=scores, groups=2, top_groups=1)
    check(torch.cat([z * 0, -z.abs() * 0], 1), 20, scores=scores)  # -0 and +0 are equal


def test_near_ties_are_told_apart():
    # a bias that leaves every expert's sum near one value: closer than FP32 can compute them, wide apart for 64 bits
    E, T = 256, 300
    for scores in ("sigmoid", "softmax"):
        r = rng("near", scores)
        base = r.standard_normal(E)
        s = 1 / (1 + np.exp(-base)) if scores == "sigmoid" else np.exp(base) / np.exp(base).sum()
        bias = (0.5 - s).astype(np.float32)  # its rounding is all that is left
        z = (base[None] + np.zeros((T, 1))).astype(np.float32)
        z[1:] += (r.standard_normal((T - 1, E)) * 1e-7).astype(np.float32)
        for kw in (dict(), dict(groups=8, top_groups=4, group_score="top2"), dict(groups=16, top_groups=3)):
            check(torch.from_numpy(z).cuda(), 8, bias, scores=scores, **kw)


def test_groups_in_doubt():
    # group scores that agree to FP32's accuracy, and scores within a group that do: the exact ones decide
    T, G, per = 400, 8, 32
    for scores, group_score in (("sigmoid", "top2"), ("sigmoid", "max"), ("softmax", "top2"), ("softmax", "max")):
        r = rng("groups", scores, group_score)
        z = r.standard_normal((T, G, per)).astype(np.float32)
        z = np.sort(z, 2)
        z[:, :, -3:] = np.array([0.5, 1.0, 2.0], np.float32) + (r.standard_normal((T, G, 3)) * 2e-7).astype(np.float32)
        z[:, 5, -1], z[:, 6, -3:] = 3.0, 1.0
        z = np.take_along_axis(z, r.permuted(np.tile(np.arange(per), (T, G, 1)), axis=2), 2).reshape(T, G * per)
        bias = (r.standard_normal(G * per) * 1e-7).astype(np.float32)
        for b in (None, bias):
            for top in (2, 4, 7):
                check(torch.from_numpy(z).cuda(), 6, b, scores=scores, groups=G, top_groups=top, group_score=group_score)


def test_many_in_doubt():
    # more experts than a warp has lanes within FP32's accuracy of one another
    r = rng("many")
    z = (1.0 + r.standard_normal((50, 300)) * 1e-7).astype(np.float32)
    bias = (r.standard_normal(300) * 1e-8).astype(np.float32)
    for scores in ("sigmoid", "softmax"):
        check(torch.from_numpy(z).cuda(), 20, bias, scores=scores)
        check(torch.from_numpy(z).cuda(), 20, None, scores=scores)
        check(torch.from_numpy(z).cuda(), 32, bias, scores=scores, groups=10, top_groups=4, group_score="top2")


def test_not_finite_logits():
    nan, inf = float("nan"), float("inf")
    z = torch.tensor([[1.0, nan, 3.0, 2.0], [1.0, inf, 3.0, 2.0], [-inf, -inf, 5.0, -inf], [-inf] * 4, [nan] * 4,
                      [0.0, -inf, nan, inf]], device="cuda")
    ids, w = g13.route(z, 3)
    assert ids.tolist() == [[2, 3, 0], [1, 2, 3], [2, 0, 1], [0, 1, 2], [0, 1, 2], [3, 0, 1]]
    for t in (0, 1, 3, 4, 5):
        assert bool(torch.isnan(w[t]).all())
    assert w[2].tolist() == [1.0, 0.0, 0.0]
    ids, w = g13.route(z, 3, scores="sigmoid", normalize=False)
    assert ids.tolist() == [[2, 3, 0], [1, 2, 3], [2, 0, 1], [0, 1, 2], [0, 1, 2], [3, 0, 1]]
    assert float(w[1, 0]) == 1 and w[3].tolist() == [0.0] * 3 and bool(torch.isnan(w[4]).all())
    # a bias: NaN last as well, in 64 bits as in 32
    ids, _ = g13.route(z, 3, scores="sigmoid", bias=torch.tensor([0.0, 0.0, 0.0, 1.0], device="cuda"))
    assert ids.tolist() == [[3, 2, 0], [3, 1, 2], [3, 2, 0], [3, 0, 1], [0, 1, 2], [3, 0, 1]]
    # groups: one of NaN only comes last
    ids, _ = g13.route(torch.tensor([[nan, nan, -9.0, -8.0, 1.0, 2.0]], device="cuda"), 2, scores="sigmoid", groups=3,
                       top_groups=2, group_score="top2")
    assert ids.tolist() == [[5, 4]]
    ids, _ = g13.route(torch.tensor([[nan, nan, -9.0, nan, nan, nan]], device="cuda"), 2, scores="sigmoid", groups=3,
                       top_groups=1)
    assert ids.tolist() == [[2, 3]]


def test_strides_many_tokens_and_empty():
    r = rng("strides")
    big = torch.from_numpy(r.standard_normal((70001, 45)).astype(np.float32)).cuda()
    check(big[:, 3:40], 4, scores="sigmoid")
    check(big[:500].bfloat16()[:, 1:42], 4)
    ids, w = g13.route(big[:0], 4)
    assert tuple(ids.shape) == tuple(w.shape) == (0, 4)


def test_refusals():
    z = torch.randn(4, 64, device="cuda")
    b = torch.zeros(64, device="cuda")
    E = g13.GemmError
    for args, kw in (((z.cpu(), 2), {}), ((z.double(), 2), {}), ((z[0], 2), {}), ((z.t(), 2), {}), ((z, 0), {}), ((z, 65), {}),
                     ((z, 33), {}), ((z, 2), dict(scores="tanh")), ((z, 2), dict(group_score="sum")),
                     ((z, 2), dict(bias=b[:60])), ((z, 2), dict(bias=b.bfloat16())), ((z, 2), dict(bias=b.cpu())),
                     ((z, 2), dict(groups=5)), ((z, 2), dict(groups=4, top_groups=5)), ((z, 2), dict(groups=0)),
                     ((z, 17), dict(groups=4, top_groups=1)), ((z, 2), dict(scale=float("nan"))),
                     ((z[:1].expand(4, 64), 2), {}), ((torch.zeros(2, 513, device="cuda"), 2), {})):
        with pytest.raises(E):
            g13.route(*args, **kw)


def test_streams_and_graphs():
    z = torch.randn(300, 128, device="cuda")
    kw = dict(scores="sigmoid", bias=torch.randn(128, device="cuda") * 0.1, groups=4, top_groups=2, group_score="top2")
    want = g13.route(z, 6, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = g13.route(z, 6, stream=s, **kw)
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = g13.route(z, 6, **kw)
    z.copy_(torch.randn(300, 128, device="cuda"))
    for _ in range(3):
        gr.replay()
    want = g13.route(z, 6, **kw)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ a layer on a choice made beforehand
def experts_ref(x, w1, w2, ids, weights, act, u):
    """(y, bound): moe_ref.layer's sums and bounds for given experts and FP32 weights."""
    T, H = x.shape
    I = w2.shape[2]
    y, b = np.zeros((T, H)), np.zeros((T, H))
    n1, n2 = (H + 64) * 2.0 ** -23, (2 * I + 64) * 2.0 ** -23
    for t in range(T):
        for e, w in zip(ids[t], weights[t]):
            if not 0 <= e < len(w1):
                continue
            a, da = x[t] @ w1[e].T, n1 * (np.abs(x[t]) @ np.abs(w1[e]).T)
            if act == "swiglu":
                g, up, dg, dup = a[:I], a[I:], da[:I], da[I:]
                sg = g / (1 + np.exp(-g))
                h, dh = sg * up, 1.1 * dg * np.abs(up) + np.abs(sg) * dup + 1.1 * dg * dup + 2.0 ** -20 * np.abs(sg * up)
            else:
                h, dh = np.maximum(a, 0), da
            dh = dh + u * u * (np.abs(h) + dh) + 2.0 ** -24
            o = h @ w2[e].T
            do = dh @ np.abs(w2[e]).T + n2 * ((np.abs(h) + dh) @ np.abs(w2[e]).T)
            y[t] += w * o
            b[t] += abs(w) * (do + 2.0 ** -22 * np.abs(o))
    return y, b + u * (np.abs(y) + b) + 2.0 ** -24


def layer_inputs(key, T, E, H, I, act, dtype):
    r = rng(key)
    def t(std, *shape):
        return torch.from_numpy(r.standard_normal(shape).astype(np.float32) * std).to(DT[dtype]).cuda()
    return r, t(1, T, H), t(H ** -0.5, E, 2 * I if act == "swiglu" else I, H), t(I ** -0.5, E, H, I)


def check_experts(y, x, w1, w2, ids, wts, act):
    u = torch.finfo(x.dtype).eps / 2
    want, bound = experts_ref(*(t.double().cpu().numpy() for t in (x, w1, w2)), ids.cpu().numpy(),
                              wts.double().cpu().numpy(), act, u)
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= bound).all(), f"max err/bound {np.max(err / bound):.3g}"


@pytest.mark.parametrize("case", [(1, 1, 1, 8, 8), (1, 8, 2, 64, 32), (5, 7, 3, 100, 33), (16, 64, 6, 512, 96), (40, 6, 2, 264, 40),
                                  (64, 300, 8, 128, 24)], ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("act", ["swiglu", "relu"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_moe_experts(case, act, dtype):
    T, E, k, H, I = case
    r, x, w1, w2 = layer_inputs((case, act, dtype), T, E, H, I, act, dtype)
    ids = torch.from_numpy(np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).cuda()
    wts = torch.from_numpy(r.standard_normal((T, k)).astype(np.float32)).cuda()
    y = g13.moe_experts(x, w1, w2, ids, wts, act=act)
    check_experts(y, x, w1, w2, ids, wts, act)
    for _ in range(2):
        assert torch.equal(y, g13.moe_experts(x, w1, w2, ids, wts, act=act))


def test_moe_experts_as_moe_layer():
    # the layer's own choice, handed over: the same experts and weights, so the same sums
    r, x, w1, w2 = layer_inputs("same", 20, 12, 256, 64, "swiglu", "bf16")
    router = torch.randn(12, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    y, ids, wts = g13.moe_layer(x, router, w1, w2, 4, return_routing=True)
    assert torch.equal(y, g13.moe_experts(x, w1, w2, ids, wts))


def test_moe_experts_unusual_choices():
    # ids out of range take no part, an expert named twice counts with both weights, a token without experts gets zeros
    r, x, w1, w2 = layer_inputs("odd", 9, 5, 120, 40, "swiglu", "bf16")
    ids = torch.from_numpy(r.integers(0, 5, (9, 4)).astype(np.int32)).cuda()
    ids[0] = torch.tensor([-1, 5, 2, 1 << 30])
    ids[3] = -7
    ids[4] = 3
    wts = torch.rand(9, 4, device="cuda")
    wts[0, 0] = float("nan")
    y = g13.moe_experts(x, w1, w2, ids, wts)
    fixed = torch.where((ids >= 0) & (ids < 5), wts, torch.zeros_like(wts))
    check_experts(y, x, w1, w2, ids, fixed, "swiglu")
    assert bool((y[3] == 0).all())
    # nobody has an expert: zeros, around which nothing is written
    room = torch.full((11, 130), 7.0, dtype=torch.bfloat16, device="cuda")
    g13.moe_experts(x, w1, w2, torch.full_like(ids, -1), wts, out=room[1:-1, 5:125])
    assert bool((room[1:-1, 5:125] == 0).all())
    room[1:-1, 5:125] = 7
    assert bool((room == 7).all())
    wts[5, 0] = float("nan")
    y2 = g13.moe_experts(x, w1, w2, ids, wts)
    rest = [0, 1, 2, 3, 4, 6, 7, 8]
    assert bool(torch.isnan(y2[5]).all()) and torch.equal(y2[rest], y[rest])


def test_moe_experts_refusals():
    r, x, w1, w2 = layer_inputs("refuse", 3, 4, 32, 16, "swiglu", "bf16")
    ids, wts = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, 2, device="cuda")
    E = g13.GemmError
    for args, kw in (((x.float(), w1, w2, ids, wts), {}), ((x, w1, w2, ids.long(), wts), {}), ((x, w1, w2, ids, wts.half()), {}),
                     ((x, w1, w2, ids[:2], wts[:2]), {}), ((x, w1, w2, ids, wts[:, :1]), {}), ((x, w1, w2, ids.cpu(), wts), {}),
                     ((x, w1, w2, ids, wts), dict(act="tanh")), ((x, w1, w2, ids, wts), dict(act="gelu")),
                     ((x, w1, w2, ids, wts), dict(out=x[:2])), ((x, w1[:2], w2, ids, wts), {}),
                     ((x, w1, w2, ids.t().contiguous().t(), wts), {}),
                     ((x, w1, w2, torch.zeros(3, 5, dtype=torch.int32, device="cuda"), torch.zeros(3, 5, device="cuda")), {})):
        with pytest.raises(E):
            g13.moe_experts(*args, **kw)
    plan = g13.gemm_moe_plan("bf16", 3, 4, 2, 32, 16)
    y = torch.empty_like(x)
    with pytest.raises(E):
        g13.gemm_moe_run_routed(plan, x, ids, wts, w1, w2, y, torch.empty(16, dtype=torch.uint8, device="cuda"))
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    g13.gemm_moe_run_routed(plan, x, ids, wts, w1, w2, y, ws)
    assert g13.gemm_moe_status(plan) == 0 and bool((y == 0).all())
