"""The many-token form of the products with an epilogue (gptq_dequant_gemm_linear,
gptq_dequant_gemm_gated) against float64, through the Python entry points."""
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


# n_tok, d_col, d_row, bits, g, perm, activation, bias, residual, keep pre
LINEAR = [
    (1, 64, 1, 4, -1, False, "none", False, False, False),      # smallest
    (256, 512, 256, 4, 128, True, "none", True, True, False),   # one whole tile
    (128, 256, 300, 4, 64, False, "relu", True, False, True),   # one half tile
    (129, 1024, 257, 4, 32, True, "silu", False, True, True),   # second half of one token
    (300, 320, 100, 4, 16, False, "gelu", True, True, True),
    (77, 192, 600, 4, 8, True, "gelu_tanh", True, True, False),
    (500, 4096, 512, 4, 128, True, "none", True, True, False),  # split contraction
    (50, 16448, 70, 4, 128, False, "silu", True, False, True),  # long contraction, few tiles
    (2600, 1024, 4096, 4, 128, False, "none", False, True, False),  # whole and split tiles
    (200, 576, 130, 2, 64, True, "none", True, True, True),
    (90, 320, 300, 2, 8, False, "silu", False, False, False),
    (33, 128, 5, 3, -1, False, "none", True, False, False),
    (270, 2176, 300, 3, 128, True, "gelu", True, True, True),   # odd split of slots of two stages
    (150, 384, 260, 3, 16, False, "none", False, True, False),
    (400, 640, 129, 3, 32, True, "relu", True, False, False),
    (100, 64, 3, 8, 64, False, "none", True, True, False),
    (333, 2048, 520, 8, 128, True, "gelu", True, True, True),
    (140, 448, 260, 8, 8, False, "silu", False, True, False),
    (64, 448, 60, 8, 32, True, "none", False, False, False),
    (130, 1024, 64, 4, 256, False, "none", True, True, False),
]


@pytest.mark.parametrize("n,d_col,d_row,bits,g,with_perm,activation,with_bias,with_res,keep", LINEAR)
def test_linear_matches_float64(n, d_col, d_row, bits, g, with_perm, activation, with_bias, with_res, keep):
    q = _q()
    rng = lt.rng_of(n, d_col, d_row, bits, g + 2, 5)
    layer = lt.Layer(d_row, d_col, bits, g, rng)
    X = lt.bf16(rng, n, d_col)
    perm = rng.permutation(d_col).astype(np.int32) if with_perm else None
    bias = rng.standard_normal(d_row).astype(np.float32) if with_bias else None
    res = lt.bf16(rng, n, d_row) if with_res else None
    want, bound, pw, pb = lt.linear(X, layer, perm, "many", bias, activation, res)
    buf, Y = lt.blank(n, d_row)
    pbuf, pre = lt.blank(n, d_row, d_row + 5)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.gptq_dequant_gemm_linear(X.cuda(), *layer.cuda(), lt.cuda(perm), bits, g, Y,
                               lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(n, d_col, d_row)),
                               bias=lt.cuda(bias), activation=activation, residual=lt.cuda(res),
                               pre=pre if keep else None, dev_status=st)
    assert q.gptq_sync_status(st) == 0
    lt.check(Y, want, bound, "Y")
    lt.untouched(buf, d_row)
    if keep:
        lt.check(pre, pw, pb, "pre")
        lt.untouched(pbuf, d_row)


GATED = [
    (1, 64, 1, 4, -1, False, "none", False),
    (256, 512, 128, 4, 128, False, "silu", True),
    (130, 256, 300, 4, 64, True, "gelu", True),
    (300, 1024, 129, 4, 32, True, "silu", False),
    (70, 320, 257, 4, 8, False, "gelu_tanh", True),
    (500, 4096, 256, 4, 128, True, "silu", True),           # split contraction
    (1300, 1088, 4096, 4, -1, False, "silu", False),        # whole and split tiles
    (40, 192, 65, 4, 16, True, "relu", True),
    (150, 576, 200, 2, 64, True, "silu", True),
    (77, 1024, 500, 3, 128, False, "silu", True),
    (260, 384, 70, 3, 8, True, "gelu", False),
    (129, 448, 140, 8, 32, False, "silu", True),
    (200, 1024, 100, 8, 128, True, "gelu_tanh", False),
]


@pytest.mark.parametrize("n,d_col,d_row,bits,g,with_perm,activation,keep", GATED)
def test_gated_matches_float64(n, d_col, d_row, bits, g, with_perm, activation, keep):
    q = _q()
    rng = lt.rng_of(n, d_col, d_row, bits, g + 3, 5)
    gate, up = (lt.Layer(d_row, d_col, bits, g, rng) for _ in range(2))
    X = lt.bf16(rng, n, d_col)
    perm = rng.permutation(d_col).astype(np.int32) if with_perm else None
    want, bound, (gw, gb), (uw, ub) = lt.gated(X, gate, up, perm, "many", activation)
    buf, Y = lt.blank(n, d_row)
    gbuf, G = lt.blank(n, d_row, d_row + 5)
    ubuf, U = lt.blank(n, d_row, -(-d_row // 8) * 8 + 8)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.gptq_dequant_gemm_gated(X.cuda(), *gate.cuda(), *up.cuda(), lt.cuda(perm), bits, g, activation, Y,
                              lt.workspace(q.gptq_dequant_gemm_gated_workspace_size(n, d_col, d_row)),
                              gate=G if keep else None, up=U if keep else None, dev_status=st)
    assert q.gptq_sync_status(st) == 0
    lt.check(Y, want, bound, "Y")
    lt.untouched(buf, d_row)
    if keep:
        lt.check(G, gw, gb, "gate")
        lt.check(U, uw, ub, "up")
        lt.untouched(gbuf, d_row)
        lt.untouched(ubuf, d_row)


@pytest.mark.parametrize("n,offset,pad", [(5, 1, 0), (140, 0, 3), (300, 3, 5), (200, 0, 8)])
def test_strided_and_misaligned_operands(n, offset, pad):
    """Rows of any alignment and pitch; values beside them are NaN and reach no sum."""
    q = _q()
    rng = lt.rng_of(n, offset, pad, 2)
    layer = lt.Layer(70, 320, 4, 64, rng)
    X, res = lt.bf16(rng, n, 320), lt.bf16(rng, n, 70)
    _, Xv = lt.padded(X, 320 + pad, offset=offset)
    _, Rv = lt.padded(res, 70 + pad, offset=offset)
    want, bound, _, _ = lt.linear(X, layer, None, "many", None, "silu", res)
    buf, Y = lt.blank(n, 70, 70 + pad)
    q.gptq_dequant_gemm_linear(Xv, *layer.cuda(), None, 4, 64, Y,
                               lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(n, 320, 70)),
                               activation="silu", residual=Rv)
    lt.check(Y, want, bound, "Y")
    lt.untouched(buf, 70)


@pytest.mark.parametrize("n,d_col,d_row", [(150, 512, 130), (60, 4096, 130)])   # whole and split tiles
def test_residual_in_place(n, d_col, d_row):
    q = _q()
    rng = lt.rng_of(n, d_col, d_row, 1)
    layer = lt.Layer(d_row, d_col, 4, 128, rng)
    X, res = lt.bf16(rng, n, d_col), lt.bf16(rng, n, d_row)
    want, bound, _, _ = lt.linear(X, layer, None, "many", None, "none", res)
    Y = res.cuda()
    q.gptq_dequant_gemm_linear(X.cuda(), *layer.cuda(), None, 4, 128, Y,
                               lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(n, d_col, d_row)), residual=Y)
    lt.check(Y, want, bound, "Y")


def test_same_bits_every_call_and_in_a_graph():
    """Deterministic, also with a split contraction; a captured call replays on
    new inputs while an eager call uses a workspace of its own."""
    q = _q()
    rng = lt.rng_of(5, 5, 6)
    n, d_col, d_row = 140, 4096, 300
    layer = lt.Layer(d_row, d_col, 4, 128, rng)
    dev = layer.cuda()
    perm = lt.cuda(rng.permutation(d_col).astype(np.int32))
    X1, X2 = lt.bf16(rng, n, d_col).cuda(), lt.bf16(rng, n, d_col).cuda()
    size = q.gptq_dequant_gemm_linear_workspace_size(n, d_col, d_row)
    ws = [lt.workspace(size) for _ in range(2)]
    X, Y = X1.clone(), torch.empty(n, d_row, dtype=torch.bfloat16, device="cuda")
    E = torch.empty_like(Y)

    def eager(x):
        q.gptq_dequant_gemm_linear(x, *dev, perm, 4, 128, E, ws[1], activation="gelu")
        return E.clone()

    a, b = eager(X1), eager(X2)
    assert torch.equal(a, eager(X1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            q.gptq_dequant_gemm_linear(X, *dev, perm, 4, 128, Y, ws[0], activation="gelu")
    torch.cuda.synchronize()
    for x, want in ((X1, a), (X2, b)):
        X.copy_(x)
        graph.replay()
        assert torch.equal(eager(X1), a)
        torch.cuda.synchronize()
        assert torch.equal(Y, want)


def test_nonfinite_tokens_stay_in_their_rows():
    q = _q()
    rng = lt.rng_of(8, 9)
    layer = lt.Layer(90, 256, 4, 32, rng)
    X = lt.bf16(rng, 140, 256)
    want, bound, _, _ = lt.linear(X, layer, None, "many")
    bad = X.clone()
    bad[3, 77], bad[139, 0] = float("nan"), float("inf")
    Y = torch.empty(140, 90, dtype=torch.bfloat16, device="cuda")
    q.gptq_dequant_gemm_linear(bad.cuda(), *layer.cuda(), None, 4, 32, Y,
                               lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(140, 256, 90)))
    keep = [i for i in range(140) if i not in (3, 139)]
    lt.check(Y[keep], want[keep], bound[keep], "Y")
    assert torch.isnan(Y[3]).all()
    # infinity times a nonzero weight, NaN where the weight is 0
    assert not torch.isfinite(Y[139]).any()


def test_zero_points_far_outside_the_codes():
    q = _q()
    rng = lt.rng_of(9, 10)
    for bits in (4, 8):
        layer = lt.Layer(40, 512, bits, 128, rng, scale=1e-5)
        layer.zeros[:] = rng.integers(-(1 << 20), 1 << 20, size=layer.zeros.shape)
        X = lt.bf16(rng, 150, 512)
        want, bound, _, _ = lt.linear(X, layer, None, "many")
        Y = torch.empty(150, 40, dtype=torch.bfloat16, device="cuda")
        q.gptq_dequant_gemm_linear(X.cuda(), *layer.cuda(), None, bits, 128, Y,
                                   lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(150, 512, 40)))
        lt.check(Y, want, bound, f"Y {bits} bits")


def test_agrees_with_the_plain_many_token_product():
    """The same sums as gptq_dequant_gemm, rounded to bf16 at the end (whole
    tiles, so the contraction runs in the same order)."""
    q = _q()
    rng = lt.rng_of(12, 1)
    layer = lt.Layer(512, 448, 4, 64, rng)   # 7 stages: never split
    X = lt.bf16(rng, 200, 448).cuda()
    Y = torch.empty(200, 512, dtype=torch.bfloat16, device="cuda")
    F = torch.empty(200, 512, dtype=torch.float32, device="cuda")
    q.gptq_dequant_gemm(X, *layer.cuda(), None, 4, 64, F)
    q.gptq_dequant_gemm_linear(X, *layer.cuda(), None, 4, 64, Y)
    assert torch.equal(F.to(torch.bfloat16), Y)


def test_feed_forward_block():
    """The operators as a block uses them: x + down(silu(gate x) * up x), the
    prompt on the tensor cores and its last token again in the decode form,
    each against float64 from the call's own bf16 input."""
    q = _q()
    rng = lt.rng_of(4, 4, 4)
    d, f, n = 256, 704, 150
    gate, up = (lt.Layer(f, d, 3, 128, rng, scale=0.05) for _ in range(2))
    down = lt.Layer(d, f, 4, 64, rng)
    p_in, p_mid = (rng.permutation(k).astype(np.int32) for k in (d, f))
    x = lt.bf16(rng, n, d)
    xd = x.cuda()
    H = torch.empty(n, f, dtype=torch.bfloat16, device="cuda")
    Y = xd.clone()
    q.gptq_dequant_gemm_gated(xd, *gate.cuda(), *up.cuda(), lt.cuda(p_in), 3, 128, "silu", H,
                              lt.workspace(q.gptq_dequant_gemm_gated_workspace_size(n, d, f)))
    q.gptq_dequant_gemm_linear(H, *down.cuda(), lt.cuda(p_mid), 4, 64, Y,
                               lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(n, f, d)), residual=Y)
    h, hb, _, _ = lt.gated(x, gate, up, p_in, "many", "silu")
    lt.check(H, h, hb, "H")
    y, yb, _, _ = lt.linear(H.cpu(), down, p_mid, "many", residual=x)
    lt.check(Y, y, yb, "Y")
    h1 = torch.empty(1, f, dtype=torch.bfloat16, device="cuda")
    y1 = xd[-1:].clone()
    ws = lt.workspace(max(q.gptq_dequant_matmul_gated_workspace_size(1, d),
                          q.gptq_dequant_matmul_linear_workspace_size(1, f)))
    q.gptq_dequant_matmul_gated(xd[-1:], *gate.cuda(), *up.cuda(), lt.cuda(p_in), 3, 128, "silu", h1, ws)
    q.gptq_dequant_matmul_linear(h1, *down.cuda(), lt.cuda(p_mid), 4, 64, y1, ws, residual=y1)
    h, hb, _, _ = lt.gated(x[-1:], gate, up, p_in, "decode", "silu")
    lt.check(h1, h, hb, "decode H")
    y, yb, _, _ = lt.linear(h1.cpu(), down, p_mid, "decode", residual=x[-1:])
    lt.check(y1, y, yb, "decode Y")
