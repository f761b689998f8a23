"""The bounded waits of the products with an epilogue run out: the lanes of a
warp, the warps of a CTA and the CTAs of a pair or a cluster wind down together,
the call reports GPTQ_ERR_TIMEOUT, and the next call is right.

gptq_debug_arm_wait_probe makes the next launch wait, with a short limit, on a
barrier that nothing completes; no other wait is shortened.  The kernels' other
waits end by the abort word, and in a pair's second CTA by their own limit."""
import numpy as np
import pytest
import torch

import linear_testlib as lt

pytestmark = pytest.mark.gpu

PROBE_NS = 200_000  # 0.2 ms
DECODE, SINGLE, PAIR = 4, 5, 6


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _q():
    import post_weight_quantization_gptq_b200 as q
    return q


def _expires(q, kind, call, outputs):
    """The armed call reports its timeout and leaves what lies beside its
    outputs; the same call again is right."""
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.gptq_debug_arm_wait_probe(kind, PROBE_NS)
    call(st)
    assert q.gptq_sync_status(st) == 4
    for buf, cols in outputs:
        lt.untouched(buf, cols)
    st.zero_()
    call(st)
    assert q.gptq_sync_status(st) == 0


# one tile; K split over a cluster; more tiles than CTAs; tokens gathered first
@pytest.mark.parametrize("n,d_col,d_row,with_perm", [(1, 512, 64, False), (4, 16448, 64, False), (2, 256, 38001, False),
                                                     (32, 1024, 300, True)])
def test_decode_form(n, d_col, d_row, with_perm):
    q = _q()
    rng = lt.rng_of(n, d_col, d_row, 31)
    layers = [lt.Layer(d_row, d_col, 4, 128, rng) for _ in range(2)]
    dev = [l.cuda() for l in layers]
    X, perm = lt.bf16(rng, n, d_col), rng.permutation(d_col).astype(np.int32) if with_perm else None
    Xd, pd, ws = X.cuda(), lt.cuda(perm), lt.workspace(q.gptq_dequant_matmul_linear_workspace_size(n, d_col))
    buf, Y = lt.blank(n, d_row)
    _expires(q, DECODE, lambda st: q.gptq_dequant_matmul_linear(Xd, *dev[0], pd, 4, 128, Y, ws, dev_status=st),
             [(buf, d_row)])
    want, bound, _, _ = lt.linear(X, layers[0], perm, "decode")
    lt.check(Y, want, bound, "Y")
    _expires(q, DECODE, lambda st: q.gptq_dequant_matmul_gated(Xd, *dev[0], *dev[1], pd, 4, 128, "silu", Y, ws, dev_status=st),
             [(buf, d_row)])
    want, bound, _, _ = lt.gated(X, *layers, perm, "decode", "silu")
    lt.check(Y, want, bound, "gated Y")


# few stages; a split contraction; more tiles than SMs
@pytest.mark.parametrize("kind,n,d_col,d_row,bits,g", [
    (SINGLE, 100, 128, 300, 4, 128), (SINGLE, 70, 4096, 260, 3, 32), (SINGLE, 250, 1024, 19001, 8, 64),
    (PAIR, 300, 128, 300, 4, 128), (PAIR, 600, 4096, 260, 3, 32), (PAIR, 1030, 1024, 9601, 8, 64)])
def test_many_token_form(kind, n, d_col, d_row, bits, g):
    q = _q()
    rng = lt.rng_of(n, d_col, d_row, bits, g, 32)
    layers = [lt.Layer(d_row, d_col, bits, g, rng) for _ in range(2)]
    dev = [l.cuda() for l in layers]
    X, dY = lt.bf16(rng, n, d_col), lt.bf16(rng, n, d_row)
    Xd = X.cuda()
    buf, Y = lt.blank(n, d_row)
    ws = lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(n, d_col, d_row))
    _expires(q, kind, lambda st: q.gptq_dequant_gemm_linear(Xd, *dev[0], None, bits, g, Y, ws, activation="gelu", dev_status=st),
             [(buf, d_row)])
    rows = rng.choice(n, size=min(n, 40), replace=False)   # (the reference takes a while)
    want, bound, _, _ = lt.linear(X[rows], layers[0], None, "many", None, "gelu")
    lt.check(Y[rows], want, bound, "Y")
    ws = lt.workspace(q.gptq_dequant_gemm_gated_workspace_size(n, d_col, d_row))
    _expires(q, kind, lambda st: q.gptq_dequant_gemm_gated(Xd, *dev[0], *dev[1], None, bits, g, "silu", Y, ws, dev_status=st),
             [(buf, d_row)])
    want, bound, _, _ = lt.gated(X[rows], *layers, None, "many", "silu")
    lt.check(Y[rows], want, bound, "gated Y")
    xbuf, dX = lt.blank(n, d_col)
    pbuf, dP = lt.blank(n, d_row, -(-d_row // 8) * 8 + 8)
    dYd, ws = dY.cuda(), lt.workspace(q.gptq_dequant_gemm_linear_backward_workspace_size(n, d_col, d_row))
    _expires(q, kind, lambda st: q.gptq_dequant_gemm_linear_backward(dYd, *dev[0], None, bits, g, dX, ws, dPre=dP, dev_status=st),
             [(xbuf, d_col), (pbuf, d_row)])
    want, bound = lt.back_product([dP[rows]], layers[:1], None)
    lt.check(dX[rows], want, bound, "dX")
