"""The mixture-of-experts layer on the GPU against 64-bit sums (tests/moe_ref.py has the bound)."""
import zlib

import numpy as np
import pytest
import torch

import dense_gemm_13_gb300 as g13
from tests import moe_ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


def inputs(key, T, E, H, I, act, dtype, pad=(0, 0), top_k=2):
    """x, router, w1, w2 on the CPU; pad: extra elements in front of and behind each row of the weights."""
    r = np.random.default_rng(zlib.crc32(repr(key).encode()))
    rows = 2 * I if act == "swiglu" else I

    def t(std, *shape):
        return torch.from_numpy(r.standard_normal(shape).astype(np.float32) * std).to(DT[dtype])

    full = t(H ** -0.5, E, rows, H + sum(pad)), t(I ** -0.5, E, H, I + sum(pad))
    w1, w2 = full[0][..., pad[0]: pad[0] + H], full[1][..., pad[0]: pad[0] + I]
    while True:  # a choice of experts that no rounding can change
        x, router = t(1, T, H), t(3 * H ** -0.5, E, H)
        if moe_ref.routing(x.double().numpy(), router.double().numpy(), top_k)[3] > 0:
            return x, router, w1, w2


def check(x, router, w1, w2, k, act, normalize, y, ids=None, weights=None):
    u = torch.finfo(x.dtype).eps / 2
    args = [t.double().cpu().numpy() for t in (x, router, w1, w2)]
    ref, bound, rid, rw, gap = moe_ref.layer(*args, k, act, normalize, u)
    assert gap > 0, "the inputs leave a choice of experts open"
    if ids is not None:
        assert np.array_equal(ids.cpu().numpy(), rid)
        assert np.allclose(weights.cpu().numpy(), rw, rtol=1e-4, atol=1e-7)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= bound).all(), f"max err/bound {np.nanmax(err / bound):.3g}"


def on_gpu(ts):
    """Copies with the same strides and offsets."""
    out = []
    for t in ts:
        base = t._base if t._base is not None else t
        b = base.cuda()
        out.append(b.as_strided(t.shape, t.stride(), t.storage_offset()))
    return out


CASES = [(1, 1, 1, 1, 1), (1, 8, 2, 64, 32), (3, 5, 5, 40, 24), (8, 16, 4, 256, 128), (9, 7, 3, 1001, 333),
         (16, 64, 6, 512, 96), (17, 33, 2, 130, 77), (33, 4, 4, 264, 40), (64, 64, 8, 512, 64), (64, 3, 1, 96, 520),
         (60, 400, 32, 64, 16), (5, 300, 3, 2048, 16), (2, 4, 2, 16384, 8), (1, 3, 1, 33, 5000), (24, 2, 2, 2000, 9)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("act", list(g13.MOE_ACTS))
def test_layer(case, act):
    T, E, k, H, I = case
    for dtype, normalize in (("bf16", True), ("f16", False)):
        ts = on_gpu(inputs((case, act, dtype), T, E, H, I, act, dtype, top_k=k))
        y, ids, wts = g13.moe_layer(*ts, k, act=act, normalize=normalize, return_routing=True)
        check(*ts, k, act, normalize, y, ids, wts)
        # the same bits again: no sum depends on timing
        for _ in range(3):
            assert torch.equal(y, g13.moe_layer(*ts, k, act=act, normalize=normalize))


@pytest.mark.parametrize("case", [(17, 9, 2, 160, 72), (40, 70, 3, 96, 33), (64, 5, 1, 264, 200), (64, 300, 2, 64, 8)],
                         ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("act", ["relu", "swiglu"])
def test_busy_experts(case, act):
    # one expert that many tokens choose, one that no token chooses, few tokens for the others
    T, E, k, H, I = case
    for n in range(20):
        x, router, w1, w2 = inputs(("busy", case, act, n), T, E, H, I, act, "bf16", top_k=k)
        x[:, 0], router[:, 0] = 4, 0
        router[E // 2, 0], router[E - 1, 0] = 1.5, -8
        if moe_ref.routing(x.double().numpy(), router.double().numpy(), k)[3] > 0:
            break
    ts = on_gpu((x, router, w1, w2))
    y, ids, wts = g13.moe_layer(*ts, k, act=act, return_routing=True)
    per = torch.bincount(ids.flatten().long().cpu(), minlength=E)
    assert per.max() >= T // 4 and per.min() == 0  # (of 300 experts others are liked as much)
    check(*ts, k, act, True, y, ids, wts)


@pytest.mark.parametrize("pad", [(8, 8), (1, 0), (3, 2), (0, 8), (6, 1)])
@pytest.mark.parametrize("T", [2, 20, 50])
def test_strides(T, pad):
    # weights inside larger rows at every kind of alignment, strided x and out whose surroundings stay
    H, I, E, k = 200, 104, 6, 3
    _, router, w1, w2 = inputs((T, pad), T, E, H, I, "swiglu", "bf16", pad, k)
    big = torch.randn(T, H + 13, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    x, router, w1, w2 = on_gpu((big[:, 5: 5 + H], router, w1, w2))
    room = torch.full((T + 2, H + 7), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[1:-1, 3: 3 + H]
    g13.moe_layer(x, router, w1, w2, k, out=out)
    check(x, router, w1, w2, k, "swiglu", True, out)
    out[:] = 7
    assert bool((room == 7).all()), "store outside Y"
    # experts taken from a larger tensor in another order of axes
    w1t = w1.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(g13.moe_layer(x, router, w1t, w2, k), g13.moe_layer(x, router, w1, w2, k))


@pytest.mark.parametrize("case", [(64, 2, 2, 16384, 24), (8, 3, 2, 16384, 17), (1, 1, 1, 16, 100000),
                                  (9, 2, 1, 40, 30001), (64, 512, 32, 48, 8), (1, 512, 32, 8, 640)],
                         ids=lambda c: "x".join(map(str, c)))
def test_extremes(case):
    T, E, k, H, I = case
    ts = on_gpu(inputs((case, "ends"), T, E, H, I, "swiglu", "bf16", top_k=k))
    y, ids, wts = g13.moe_layer(*ts, k, return_routing=True)
    check(*ts, k, "swiglu", True, y, ids, wts)
    assert torch.equal(y, g13.moe_layer(*ts, k))


def test_ties_go_to_the_lowest_index():
    T, E, k, H, I = 6, 40, 5, 96, 16
    x, router, w1, w2 = on_gpu(inputs("ties", T, E, H, I, "gelu", "bf16"))
    router[:] = router[0]  # every expert the same logit
    _, ids, wts = g13.moe_layer(x, router, w1, w2, k, act="gelu", normalize=False, return_routing=True)
    assert (ids.cpu() == torch.arange(k)).all()
    assert torch.allclose(wts.cpu(), torch.full((T, k), 1 / E), rtol=1e-5)
    router.zero_()
    router[1::2] = -0.0
    _, ids, _ = g13.moe_layer(x, router, w1, w2, k, act="gelu", return_routing=True)
    assert (ids.cpu() == torch.arange(k)).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_token_stays_alone(bad):
    T, E, k, H, I = 20, 8, 2, 128, 64
    x, router, w1, w2 = on_gpu(inputs("bad", T, E, H, I, "swiglu", "f16"))
    good = g13.moe_layer(x, router, w1, w2, k)
    y = x.clone()
    y[7, 3] = bad
    out, ids, _ = g13.moe_layer(y, router, w1, w2, k, return_routing=True)
    assert bool(torch.isnan(out[7]).all())
    keep = torch.arange(T) != 7
    assert torch.equal(out[keep], good[keep])
    assert bool(((ids >= 0) & (ids < E)).all()) and len(set(ids[7].tolist())) == k


def test_all_nan_and_no_tokens():
    x, router, w1, w2 = on_gpu(inputs("nan", 3, 5, 64, 32, "relu", "bf16"))
    out, ids, _ = g13.moe_layer(x * float("nan"), router, w1, w2, 5, act="relu", return_routing=True)
    assert bool(torch.isnan(out).all()) and (ids.cpu().sort(1).values == torch.arange(5)).all()
    assert tuple(g13.moe_layer(x[:0], router, w1, w2, 2, act="relu").shape) == (0, 64)


def test_large_stride_between_experts():
    # experts further apart than 2^31 elements
    T, E, k, H, I = 3, 2, 2, 64, 32
    x, router, w1, w2 = on_gpu(inputs("far", T, E, H, I, "gelu", "bf16"))
    far = torch.empty(2 ** 31 + 8192, dtype=torch.bfloat16, device="cuda")
    a = far.as_strided((E, I, H), (2 ** 31 + 4096, H, 1))
    b = far.as_strided((E, H, I), (2 ** 31 + 4096, I, 1), 2048)
    a.copy_(w1)
    b.copy_(w2)
    y = g13.moe_layer(x, router, a, b, k, act="gelu")
    assert torch.equal(y, g13.moe_layer(x, router, w1, w2, k, act="gelu"))


def test_graphs_and_streams():
    # two captured layers and eager ones at the same time: every call has its own workspace
    T, E, k, H, I = 12, 16, 4, 512, 256
    sets = [on_gpu(inputs(("g", i), T, E, H, I, "swiglu", "bf16", top_k=k)) for i in range(2)]
    want = [g13.moe_layer(*s, k) for s in sets]
    graphs, outs = [], [torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in sets]
    for s, o in zip(sets, outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            g13.moe_layer(*s, k, out=o)
        graphs.append(gr)
    st = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    eager = []
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(st[i]):
                graphs[i].replay()
        with torch.cuda.stream(st[2]):
            eager.append(g13.moe_layer(*sets[0], k))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert all(torch.equal(o, want[0]) for o in eager)
    on = torch.cuda.Stream()
    on.wait_stream(torch.cuda.current_stream())
    y = g13.moe_layer(*sets[1], k, stream=on)
    on.synchronize()
    assert torch.equal(y, want[1])


def test_timeout_is_reported():
    T, E, k, H, I = 4, 8, 2, 128, 64
    x, router, w1, w2 = on_gpu(inputs("stall", T, E, H, I, "swiglu", "bf16"))
    y = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    for flags, want in ((g13.FLAG_TEST_STALL, -5), (0, 0)):
        plan = g13.gemm_moe_plan("bf16", T, E, k, H, I, flags=flags, timeout_ms=50)
        ws = torch.full((plan.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")  # any contents
        g13.gemm_moe_run(plan, x, router, w1, w2, y, ws)
        assert g13.gemm_moe_status(plan) == want
    check(x, router, w1, w2, k, "swiglu", True, y)


def test_with_4bit_layers():
    # a layer as it is used: a 4-bit linear, then the experts on its output, captured together
    T, E, k, H, I = 7, 8, 2, 256, 128
    x, router, w1, w2 = on_gpu(inputs("chain", T, E, H, I, "swiglu", "bf16"))
    W = g13.fp4_quantize(torch.randn(H, H, device="cuda") / 16, "nvfp4")

    def step(out=None):
        mid = g13.fp4_matmul(g13.fp4_quantize(x, "nvfp4"), W, out_dtype="bf16")
        return mid, g13.moe_layer(mid, router, w1, w2, k, out=out)

    mid, y = step()
    check(mid, router, w1, w2, k, "swiglu", True, y)
    out = torch.zeros_like(y)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step(out)
    for _ in range(5):
        gr.replay()
    assert torch.equal(out, y)


def test_first_call_in_a_capture_is_refused():
    # a plan allocates: the call is refused, and the capture goes on
    x, router, w1, w2 = on_gpu(inputs("capture", 3, 4, 88, 24, "relu", "f16"))
    q = g13.fp4_quantize(torch.randn(3, 88, device="cuda"))
    gr, y = torch.cuda.CUDAGraph(), torch.zeros(4, device="cuda")
    with torch.cuda.graph(gr):
        with pytest.raises(g13.GemmError, match="before capturing"):
            g13.moe_layer(x, router, w1, w2, 2, act="relu")
        with pytest.raises(g13.GemmError, match="before capturing"):
            g13.fp4_matmul(q, q, act="relu")
        y += 1
    gr.replay()
    torch.cuda.synchronize()
    assert bool((y == 1).all())
    assert g13.moe_layer(x, router, w1, w2, 2, act="relu").shape == (3, 88)


def test_stream_argument():
    T, E, k, H, I = 6, 8, 3, 200, 64
    s = on_gpu(inputs("stream", T, E, H, I, "swiglu", "bf16", top_k=k))
    want = g13.moe_layer(*s, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for st in (side, side.cuda_stream):
        ys = [g13.moe_layer(*s, k, stream=st) for _ in range(4)]
        side.synchronize()
        assert all(torch.equal(y, want) for y in ys)


@pytest.mark.parametrize("T", [5, 30])
def test_relu_of_nan_is_nan(T):
    # a NaN among an expert's weights reaches every output of its tokens, and no other
    E, k, H, I = 6, 2, 96, 48
    x, router, w1, w2 = on_gpu(inputs(("relu nan", T), T, E, H, I, "relu", "bf16"))
    y, ids, _ = g13.moe_layer(x, router, w1, w2, k, act="relu", return_routing=True)
    e = int(ids[0, 0])
    w1[e, 7, 11] = float("nan")
    got = g13.moe_layer(x, router, w1, w2, k, act="relu")
    hit = (ids == e).any(1)
    assert bool(got[hit].isnan().all()) and torch.equal(got[~hit], y[~hit])


def check_beyond_fp16(key, act, T, E, k, H, I, pad=(0, 0)):
    # one expert's h lies beyond 65504, its output does not
    x, router, w1, w2 = inputs(key, T, E, H, I, act, "f16", pad, k)
    e = int(moe_ref.routing(x.double().numpy(), router.double().numpy(), k)[2][0, 0])
    w1[e] *= 300 if act == "swiglu" else 40000
    w2[e] *= 2.0 ** -10
    ts = on_gpu((x, router, w1, w2))
    a = torch.einsum("th,ih->ti", x.double(), w1[e].double())
    h = a[:, :I] * torch.sigmoid(a[:, :I]) * a[:, I:] if act == "swiglu" else a.clamp(min=0)
    assert h.abs().max() > 65504 and h.abs().max() < 2 ** 32
    y = g13.moe_layer(*ts, k, act=act)
    assert bool(y.isfinite().all())
    check(*ts, k, act, True, y)
    assert torch.equal(y, g13.moe_layer(*ts, k, act=act))


@pytest.mark.parametrize("pad", [(0, 0), (1, 0)])
@pytest.mark.parametrize("T", [3, 12, 30, 60])
@pytest.mark.parametrize("act", list(g13.MOE_ACTS))
def test_values_between_the_products_beyond_fp16(act, T, pad):
    check_beyond_fp16(("big", act, T, pad), act, T, 5, 2, 200, 72, pad)


@pytest.mark.parametrize("case", [(12, 8, 3, 4096, 200), (40, 8, 3, 4096, 333), (2, 2, 2, 16384, 520)],
                         ids=lambda c: "x".join(map(str, c)))
def test_values_beyond_fp16_in_blocks_cut_between_teams(case):
    # several steps a team, output blocks that begin and end inside its share
    check_beyond_fp16(("big cut", case), "swiglu", *case)
