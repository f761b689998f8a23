"""The decode form of the products with an epilogue (gptq_dequant_matmul_linear,
gptq_dequant_matmul_gated) against float64, through the Python entry points."""
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


# n_tok, d_col, d_row, bits, g, perm, activation, bias, residual
LINEAR = [
    (1, 64, 1, 4, -1, False, "none", False, False),        # smallest
    (1, 4096, 4096, 4, 128, False, "none", True, True),
    (3, 192, 33, 4, 64, True, "relu", True, True),         # K tail inside a 128-code block
    (8, 1024, 257, 4, 32, True, "silu", False, True),
    (9, 512, 100, 4, 16, False, "gelu", True, False),      # second token tile
    (16, 320, 47, 4, 8, True, "gelu_tanh", True, True),
    (17, 2048, 130, 4, 256, False, "none", True, True),    # several blocks per group
    (32, 1088, 300, 4, -1, True, "silu", True, True),      # one group, not a multiple of 128
    (33, 256, 65, 4, 128, True, "none", False, True),      # a second launch of one token
    (70, 384, 40, 4, 64, False, "gelu", True, True),       # three launches
    (2, 128, 31, 2, 128, False, "none", True, False),
    (11, 576, 64, 2, 32, True, "silu", False, True),
    (30, 320, 70, 2, 8, False, "relu", True, True),
    (1, 128, 5, 3, -1, False, "none", False, False),
    (5, 4096, 95, 3, 128, True, "none", True, True),
    (12, 384, 77, 3, 16, False, "gelu_tanh", True, True),
    (32, 640, 129, 3, 32, True, "silu", True, False),
    (1, 64, 3, 8, 64, False, "none", True, True),
    (8, 1024, 200, 8, 128, True, "gelu", True, True),
    (10, 192, 50, 8, 8, True, "none", False, True),
    (25, 448, 66, 8, 32, False, "silu", True, True),
    (4, 16448, 64, 4, 128, True, "none", False, True),     # long K, few rows: K over a cluster
]


@pytest.mark.parametrize("n,d_col,d_row,bits,g,with_perm,activation,with_bias,with_res", LINEAR)
def test_linear_matches_float64(n, d_col, d_row, bits, g, with_perm, activation, with_bias, with_res):
    q = _q()
    rng = lt.rng_of(n, d_col, d_row, bits, g + 2)
    layer = lt.Layer(d_row, d_col, bits, g, rng)
    X = lt.bf16(rng, n, d_col)
    perm = rng.permutation(d_col).astype(np.int32) if with_perm else None
    bias = rng.standard_normal(d_row).astype(np.float32) if with_bias else None
    res = lt.bf16(rng, n, d_row) if with_res else None
    want, bound, _, _ = lt.linear(X, layer, perm, "decode", bias, activation, res)
    buf, Y = lt.blank(n, d_row)
    ws = torch.full((q.gptq_dequant_matmul_linear_workspace_size(n, d_col),), 255, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.gptq_dequant_matmul_linear(X.cuda(), *layer.cuda(), lt.cuda(perm), bits, g, Y, ws, bias=lt.cuda(bias),
                                 activation=activation, residual=lt.cuda(res), dev_status=st)
    assert q.gptq_sync_status(st) == 0
    lt.check(Y, want, bound, "Y")
    lt.untouched(buf, d_row)


GATED = [
    (1, 64, 1, 4, -1, False, "none"),
    (1, 4096, 1000, 4, 128, False, "silu"),
    (7, 192, 33, 4, 64, True, "gelu"),
    (8, 512, 130, 4, 32, True, "silu"),
    (13, 320, 18, 4, 8, False, "gelu_tanh"),
    (32, 1024, 257, 4, 128, True, "silu"),
    (40, 256, 65, 4, 16, True, "relu"),
    (3, 576, 50, 2, 64, True, "silu"),
    (20, 128, 40, 2, -1, False, "gelu"),
    (1, 1024, 500, 3, 128, False, "silu"),
    (18, 384, 70, 3, 64, True, "silu"),
    (6, 448, 64, 8, 32, False, "silu"),
    (24, 1024, 100, 8, 128, True, "gelu_tanh"),
]


@pytest.mark.parametrize("n,d_col,d_row,bits,g,with_perm,activation", GATED)
def test_gated_matches_float64(n, d_col, d_row, bits, g, with_perm, activation):
    q = _q()
    rng = lt.rng_of(n, d_col, d_row, bits, g + 3)
    gate, up = (lt.Layer(d_row, d_col, bits, g, rng) for _ in range(2))
    X = lt.bf16(rng, n, d_col)
    perm = rng.permutation(d_col).astype(np.int32) if with_perm else None
    want, bound, _, _ = lt.gated(X, gate, up, perm, "decode", activation)
    buf, Y = lt.blank(n, d_row)
    ws = torch.full((q.gptq_dequant_matmul_gated_workspace_size(n, d_col),), 255, dtype=torch.uint8, device="cuda")
    q.gptq_dequant_matmul_gated(X.cuda(), *gate.cuda(), *up.cuda(),
                                None if perm is None else torch.from_numpy(perm).cuda(), bits, g, activation, Y, ws)
    lt.check(Y, want, bound, "Y")
    lt.untouched(buf, d_row)


@pytest.mark.parametrize("n,offset,pad", [(1, 1, 0), (5, 0, 3), (8, 3, 5), (20, 0, 8)])
def test_strided_and_misaligned_inputs(n, offset, pad):
    """X and residual rows of any alignment and pitch (X then passes through
    the workspace unless its rows start on 16 bytes); values beside the rows
    are NaN and are not read into any sum."""
    q = _q()
    rng = lt.rng_of(n, offset, pad)
    layer = lt.Layer(70, 320, 4, 64, rng)
    X, res = lt.bf16(rng, n, 320), lt.bf16(rng, n, 70)
    _, Xv = lt.padded(X, 320 + pad, offset=offset)
    _, Rv = lt.padded(res, 70 + pad, offset=offset)
    want, bound, _, _ = lt.linear(X, layer, None, "decode", None, "silu", res)
    Y = torch.empty(n, 70, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(q.gptq_dequant_matmul_linear_workspace_size(n, 320), dtype=torch.uint8, device="cuda")
    q.gptq_dequant_matmul_linear(Xv, *layer.cuda(), None, 4, 64, Y, ws, activation="silu", residual=Rv)
    lt.check(Y, want, bound, "Y")


def test_residual_in_place_and_no_workspace_without_a_gather():
    q = _q()
    rng = lt.rng_of(1, 2, 3)
    layer = lt.Layer(130, 512, 4, 128, rng)
    X, res = lt.bf16(rng, 12, 512), lt.bf16(rng, 12, 130)
    want, bound, _, _ = lt.linear(X, layer, None, "decode", None, "none", res)
    Y = res.cuda()
    q.gptq_dequant_matmul_linear(X.cuda(), *layer.cuda(), None, 4, 128, Y, residual=Y)
    lt.check(Y, want, bound, "Y")


def test_same_bits_every_call_and_in_a_graph():
    """Deterministic; a captured call replays on new inputs, beside an eager
    call with a workspace of its own."""
    q = _q()
    rng = lt.rng_of(5, 5, 5)
    layer = lt.Layer(300, 1024, 4, 128, rng)
    dev = layer.cuda()
    perm = torch.from_numpy(rng.permutation(1024).astype(np.int32)).cuda()
    X1, X2 = lt.bf16(rng, 6, 1024).cuda(), lt.bf16(rng, 6, 1024).cuda()
    size = q.gptq_dequant_matmul_linear_workspace_size(6, 1024)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    X, Y = X1.clone(), torch.empty(6, 300, dtype=torch.bfloat16, device="cuda")
    E = torch.empty_like(Y)

    def eager(x):
        q.gptq_dequant_matmul_linear(x, *dev, perm, 4, 128, E, ws[1], activation="gelu")
        return E.clone()

    a, b = eager(X1), eager(X2)
    assert torch.equal(a, eager(X1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            q.gptq_dequant_matmul_linear(X, *dev, perm, 4, 128, Y, ws[0], activation="gelu")
    torch.cuda.synchronize()
    for x, want in ((X1, a), (X2, b)):
        X.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)


def test_nonfinite_tokens_stay_in_their_rows():
    """A NaN or infinite activation spoils its own token's outputs only."""
    q = _q()
    rng = lt.rng_of(8, 8)
    layer = lt.Layer(90, 256, 4, 32, rng)
    X = lt.bf16(rng, 10, 256)
    want, bound, _, _ = lt.linear(X, layer, None, "decode")
    bad = X.clone()
    bad[3, 77], bad[9, 0] = float("nan"), float("inf")
    Y = torch.empty(10, 90, dtype=torch.bfloat16, device="cuda")
    q.gptq_dequant_matmul_linear(bad.cuda(), *layer.cuda(), None, 4, 32, Y)
    keep = [i for i in range(10) if i not in (3, 9)]
    lt.check(Y[keep], want[keep], bound[keep], "Y")
    assert torch.isnan(Y[3]).all() and not torch.isfinite(Y[9]).any()


def test_zero_points_far_outside_the_codes():
    """The pure min-max range allows zero points up to 2^20 levels away."""
    q = _q()
    rng = lt.rng_of(9, 9)
    layer = lt.Layer(40, 512, 4, 128, rng, scale=1e-5)
    layer.zeros[:] = rng.integers(-(1 << 20), 1 << 20, size=layer.zeros.shape)
    X = lt.bf16(rng, 5, 512)
    want, bound, _, _ = lt.linear(X, layer, None, "decode")
    Y = torch.empty(5, 40, dtype=torch.bfloat16, device="cuda")
    q.gptq_dequant_matmul_linear(X.cuda(), *layer.cuda(), None, 4, 128, Y)
    lt.check(Y, want, bound, "Y")
