"""Gradients of the many-token products with an epilogue
(gptq_dequant_gemm_linear_backward, gptq_dequant_gemm_gated_backward) against
the formulas in float64 and against differences."""
import numpy as np
import pytest
import torch

import linear_testlib as lt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _q():
    import post_weight_quantization_gptq_b200 as q
    return q


def _up8(n):
    return -(-n // 8) * 8


# n_tok, d_col, d_row, bits, g, perm, activation, bias
LINEAR = [
    (1, 64, 1, 4, -1, False, "gelu", True),                 # smallest
    (256, 512, 256, 4, 128, True, "none", True),
    (128, 256, 72, 4, 64, False, "relu", True),
    (129, 320, 257, 4, 32, True, "silu", True),
    (300, 1024, 100, 4, 16, False, "gelu", False),
    (77, 192, 600, 4, 8, True, "gelu_tanh", True),
    (500, 256, 4096, 4, 128, True, "none", False),          # split contraction
    (50, 70 * 64, 8, 4, 128, False, "silu", True),
    (2600, 4096, 1024, 4, 128, False, "none", True),        # whole and split tiles
    (200, 576, 130, 2, 64, True, "silu", True),
    (90, 320, 304, 2, 8, False, "none", True),
    (33, 128, 5, 3, -1, False, "gelu", True),
    (270, 2176, 300, 3, 128, True, "gelu", True),
    (150, 384, 260, 3, 16, False, "relu", False),
    (100, 64, 3, 8, 64, False, "silu", True),
    (333, 512, 2048, 8, 128, True, "gelu", True),
    (140, 448, 260, 8, 8, False, "silu", True),
    (40, 70016, 16, 4, 128, True, "none", False),           # rows too wide for shared memory
]


@pytest.mark.parametrize("n,d_col,d_row,bits,g,with_perm,activation,with_bias", LINEAR)
def test_linear_backward_matches_float64(n, d_col, d_row, bits, g, with_perm, activation, with_bias):
    q = _q()
    rng = lt.rng_of(n, d_col, d_row, bits, g + 2, 6)
    layer = lt.Layer(d_row, d_col, bits, g, rng)
    perm = rng.permutation(d_col).astype(np.int32) if with_perm else None
    dY, pre = lt.bf16(rng, n, d_row, std=1e-2), lt.bf16(rng, n, d_row, std=1.5)
    need = activation != "none" or d_row % 8 != 0
    pbuf, dPre = lt.blank(n, d_row, _up8(d_row) + 8)
    xbuf, dX = lt.blank(n, d_col)
    dbias = torch.full((d_row,), float("nan"), device="cuda") if with_bias else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.gptq_dequant_gemm_linear_backward(dY.cuda(), *layer.cuda(), lt.cuda(perm), bits, g, dX,
                                        lt.workspace(q.gptq_dequant_gemm_linear_backward_workspace_size(n, d_col, d_row)),
                                        activation=activation, pre=pre.cuda() if activation != "none" else None,
                                        dPre=dPre if need else None, dbias=dbias, dev_status=st)
    assert q.gptq_sync_status(st) == 0
    p, pb = lt.slopes_linear(dY, pre, activation)
    if need:
        lt.check(dPre, p, pb, "dPre")
        lt.untouched(pbuf, d_row)
    x, xb = lt.back_product([dPre if need else dY], [layer], perm)
    lt.check(dX, x, xb, "dX")
    lt.untouched(xbuf, d_col)
    if with_bias:
        # a column's sum: a chain of at most n / 8 terms of a slab, 8 and the slabs' joins
        mags = np.abs(p).sum(0)
        lt.check(dbias, p.sum(0), (n / 8 + 80) * lt.EPS32 * mags + lt.ACT_EPS * np.abs(lt.f64(dY)).sum(0) + 1e-30, "dbias")


GATED = [
    (1, 64, 1, 4, -1, False, "silu"),
    (256, 512, 128, 4, 128, False, "silu"),
    (130, 256, 300, 4, 64, True, "gelu"),
    (300, 1024, 129, 4, 32, True, "silu"),
    (70, 320, 257, 4, 8, False, "gelu_tanh"),
    (500, 256, 2048, 4, 128, True, "silu"),
    (1300, 4096, 600, 4, -1, False, "none"),
    (40, 192, 65, 4, 16, True, "relu"),
    (150, 576, 200, 2, 64, True, "gelu_tanh"),
    (77, 1024, 500, 3, 128, False, "silu"),
    (129, 448, 140, 8, 32, False, "silu"),
]


@pytest.mark.parametrize("n,d_col,d_row,bits,g,with_perm,activation", GATED)
def test_gated_backward_matches_float64(n, d_col, d_row, bits, g, with_perm, activation):
    q = _q()
    rng = lt.rng_of(n, d_col, d_row, bits, g + 3, 6)
    layers = [lt.Layer(d_row, d_col, bits, g, rng) for _ in range(2)]
    perm = rng.permutation(d_col).astype(np.int32) if with_perm else None
    dY, gate, up = (lt.bf16(rng, n, d_row, std=s) for s in (1e-2, 1.5, 1.5))
    bufs = [lt.blank(n, d_row, _up8(d_row) + 8) for _ in range(2)]
    xbuf, dX = lt.blank(n, d_col)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.gptq_dequant_gemm_gated_backward(dY.cuda(), gate.cuda(), up.cuda(), *layers[0].cuda(), *layers[1].cuda(),
                                       lt.cuda(perm), bits, g, activation, bufs[0][1], bufs[1][1], dX,
                                       lt.workspace(q.gptq_dequant_gemm_gated_backward_workspace_size(n, d_col, d_row)),
                                       dev_status=st)
    assert q.gptq_sync_status(st) == 0
    for (buf, v), (w, b), name in zip(bufs, lt.slopes_gated(dY, gate, up, activation), ("dGate", "dUp")):
        lt.check(v, w, b, name)
        lt.untouched(buf, d_row)
    x, xb = lt.back_product([bufs[0][1], bufs[1][1]], layers, perm)
    lt.check(dX, x, xb, "dX")
    lt.untouched(xbuf, d_col)


def test_in_place_and_misaligned_inputs():
    """dPre over pre, dGate over gate and dUp over up; the other inputs at odd
    offsets and pitches."""
    q = _q()
    rng = lt.rng_of(3, 2, 1)
    n, d_col, d_row = 140, 320, 96
    layers = [lt.Layer(d_row, d_col, 4, 64, rng) for _ in range(2)]
    dY, gate, up = (lt.bf16(rng, n, d_row) for _ in range(3))
    _, dYv = lt.padded(dY, d_row + 3, offset=1)
    dX = torch.empty(n, d_col, dtype=torch.bfloat16, device="cuda")
    P = gate.cuda()
    q.gptq_dequant_gemm_linear_backward(dYv, *layers[0].cuda(), None, 4, 64, dX,
                                        lt.workspace(q.gptq_dequant_gemm_linear_backward_workspace_size(n, d_col, d_row)),
                                        activation="gelu", pre=P, dPre=P)
    p, pb = lt.slopes_linear(dY, gate, "gelu")
    lt.check(P, p, pb, "dPre")
    x, xb = lt.back_product([P], layers[:1], None)
    lt.check(dX, x, xb, "dX")
    G, U = gate.cuda(), up.cuda()
    q.gptq_dequant_gemm_gated_backward(dYv, G, U, *layers[0].cuda(), *layers[1].cuda(), None, 4, 64, "silu", G, U, dX,
                                       lt.workspace(q.gptq_dequant_gemm_gated_backward_workspace_size(n, d_col, d_row)))
    (gw, gb), (uw, ub) = lt.slopes_gated(dY, gate, up, "silu")
    lt.check(G, gw, gb, "dGate")
    lt.check(U, uw, ub, "dUp")
    x, xb = lt.back_product([G, U], layers, None)
    lt.check(dX, x, xb, "dX")


@pytest.mark.parametrize("op,activation", [("linear", "gelu"), ("linear", "silu"), ("gated", "silu"),
                                           ("gated", "gelu_tanh")])
def test_gradient_agrees_with_differences(op, activation):
    """<dX, V> against a central difference of L(X) = sum dY * Y(X) in float64
    along V, from the calls' own saved pre-activations.  Bounds: the saved
    values and the products' gradient are rounded to bf16 (half a step each,
    slopes change by at most 1.2 per unit), dX once more; the difference's own
    error is O(h^2) and rounding O(1e-16 / h), both below 1e-8."""
    q = _q()
    rng = lt.rng_of(len(op), len(activation))
    n, d_col, d_row, bits, g = 40, 256, 96, 4, 64
    layers = [lt.Layer(d_row, d_col, bits, g, rng) for _ in range(2 if op == "gated" else 1)]
    perm = rng.permutation(d_col).astype(np.int32)
    X, dY = lt.bf16(rng, n, d_col), lt.bf16(rng, n, d_row)
    mats = [l.weights(True) for l in layers]

    def sums(x):
        return [x[:, perm] @ w.T for w in mats]

    def loss(x):
        s = sums(x)
        y = lt.act(s[0], activation)[0]
        return float((lt.f64(dY) * (y * s[1] if op == "gated" else y)).sum())

    args = [t for l in layers for t in l.cuda()] + [lt.cuda(perm), bits, g]
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    Y, P, Q, dP, dQ, dX = e(n, d_row), e(n, d_row), e(n, d_row), e(n, d_row), e(n, d_row), e(n, d_col)
    if op == "linear":
        q.gptq_dequant_gemm_linear(X.cuda(), *args, Y, lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(n, d_col, d_row)),
                                   activation=activation, pre=P)
        q.gptq_dequant_gemm_linear_backward(dY.cuda(), *args, dX,
                                            lt.workspace(q.gptq_dequant_gemm_linear_backward_workspace_size(n, d_col, d_row)),
                                            activation=activation, pre=P, dPre=dP)
    else:
        q.gptq_dequant_gemm_gated(X.cuda(), *args, activation, Y,
                                  lt.workspace(q.gptq_dequant_gemm_gated_workspace_size(n, d_col, d_row)), gate=P, up=Q)
        q.gptq_dequant_gemm_gated_backward(dY.cuda(), P, Q, *args, activation, dP, dQ, dX,
                                           lt.workspace(q.gptq_dequant_gemm_gated_backward_workspace_size(n, d_col, d_row)))
    V = rng.standard_normal((n, d_col))
    x, h = lt.f64(X), 1e-5
    want = (loss(x + h * V) - loss(x - h * V)) / (2 * h)
    got = float((lt.f64(dX) * V).sum())
    # magnitudes: |dP| errors through |W|, |V|
    s = sums(x)
    d, half = np.abs(lt.f64(dY)), lt.HALF_BF16
    v, sl = (np.abs(t) for t in lt.act(s[0], activation))
    if op == "linear":
        errs = [d * (half * 1.2 * np.abs(s[0]) + half * sl)]
    else:
        u = np.abs(s[1])
        errs = [d * (half * u * sl + u * half * 1.2 * np.abs(s[0]) + half * u * sl),
                d * (half * lt.LIPSCHITZ * np.abs(s[0]) + half * v)]
    bound = sum(float((e_ @ np.abs(w) * np.abs(V[:, perm])).sum()) for e_, w in zip(errs, mats))
    bound += half * float((np.abs(lt.f64(dX)) * np.abs(V)).sum())
    # every rounding error has its own sign: a sum of N independent terms stays
    # within the bound over sqrt(N) times six, N > 1000 terms here
    assert abs(got - want) <= 6 * bound / np.sqrt(n * d_col), (got, want, bound)


def test_backward_in_a_graph_and_the_same_bits():
    q = _q()
    rng = lt.rng_of(7, 7, 7)
    n, d_col, d_row = 140, 256, 2048
    layer = lt.Layer(d_row, d_col, 4, 128, rng)
    dev = layer.cuda()
    perm = lt.cuda(rng.permutation(d_col).astype(np.int32))
    size = q.gptq_dequant_gemm_linear_backward_workspace_size(n, d_col, d_row)
    pre = lt.bf16(rng, n, d_row).cuda()
    g1, g2 = lt.bf16(rng, n, d_row).cuda(), lt.bf16(rng, n, d_row).cuda()
    sets = [dict(ws=lt.workspace(size), dPre=torch.empty_like(pre), dbias=torch.empty(d_row, device="cuda"),
                 dX=torch.empty(n, d_col, dtype=torch.bfloat16, device="cuda")) for _ in range(2)]

    def call(dY, s):
        q.gptq_dequant_gemm_linear_backward(dY, *dev, perm, 4, 128, s["dX"], s["ws"], activation="silu", pre=pre,
                                            dPre=s["dPre"], dbias=s["dbias"])

    def eager(dY):
        call(dY, sets[1])
        return [sets[1][k].clone() for k in ("dX", "dPre", "dbias")]

    a, b = eager(g1), eager(g2)
    assert all(torch.equal(x, y) for x, y in zip(a, eager(g1)))
    dY = g1.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            call(dY, sets[0])
    torch.cuda.synchronize()
    for x, want in ((g1, a), (g2, b)):
        dY.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(sets[0][k], w) for k, w in zip(("dX", "dPre", "dbias"), want))


def test_no_tokens():
    """An empty batch is a no-op; its bias gradient is zero."""
    q = _q()
    rng = lt.rng_of(1)
    layer = lt.Layer(16, 64, 4, 64, rng)
    e = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    dbias = torch.full((16,), 3.0, device="cuda")
    q.gptq_dequant_matmul_linear(x, *layer.cuda(), None, 4, 64, e)
    q.gptq_dequant_gemm_linear(x, *layer.cuda(), None, 4, 64, e)
    q.gptq_dequant_gemm_linear_backward(e, *layer.cuda(), None, 4, 64, x, dbias=dbias)
    assert torch.all(dbias == 0)
