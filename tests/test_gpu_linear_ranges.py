"""Scales and tokens far from one: the products with an epilogue keep the
result's accuracy where the result is in range."""
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


@pytest.mark.parametrize("tokens,scales", [(-50, -30), (-20, -55), (0, -60), (60, -100), (-56, -20), (50, 60), (-50, 90)])
@pytest.mark.parametrize("n,bits,g,d_row", [(1, 4, 128, 48), (8, 4, -1, 4101), (5, 4, 32, 70), (32, 4, 64, 70),
                                            (12, 4, 8, 40), (20, 3, 128, 33), (3, 2, 16, 33), (17, 8, 128, 40)])
def test_small_and_large_results_of_the_decode_form(n, bits, g, d_row, tokens, scales):
    """Tokens of 2^tokens (inside the documented 2^-57 to 2^64), scales of
    2^scales: results from about 2^-80 to 2^120, all of them normal bf16
    numbers.  The bound is relative to the sum of magnitudes; its absolute part
    of 1e-30 is below 2^-99."""
    q = _q()
    rng = lt.rng_of(n, bits, g + 2, d_row, tokens + 200, scales + 200)
    layer = lt.Layer(d_row, 384, bits, g, rng, scale=2.0 ** scales)
    X = (lt.bf16(rng, n, 384).float() * 2.0 ** tokens).to(torch.bfloat16)
    want, bound, _, _ = lt.linear(X, layer, None, "decode")
    Y = torch.empty(n, d_row, dtype=torch.bfloat16, device="cuda")
    q.gptq_dequant_matmul_linear(X.cuda(), *layer.cuda(), None, bits, g, Y)
    lt.check(Y, want, bound, "Y")
    # gated, with an up matrix whose product is near one
    up = lt.Layer(d_row, 384, bits, g, rng, scale=2.0 ** -tokens)
    if tokens + scales < 100:
        want, bound, _, _ = lt.gated(X, layer, up, None, "decode", "none")
        q.gptq_dequant_matmul_gated(X.cuda(), *layer.cuda(), *up.cuda(), None, bits, g, "none", Y)
        lt.check(Y, want, bound, "gated Y")


def test_tokens_below_the_range_lose_in_proportion_to_the_scale():
    """Below 2^-57 each of the two sums' products loses at most fp32's smallest
    step, 2^-149, scaled back by 2^69: 2^-80 (1 + |z|) times the scale."""
    q = _q()
    rng = lt.rng_of(5, 66)
    for scale in (2.0 ** -12, 2.0 ** 12):
        layer = lt.Layer(48, 512, 4, 128, rng, scale=scale)
        X = (lt.bf16(rng, 4, 512).float() * 2.0 ** -66).to(torch.bfloat16)
        want, bound, _, _ = lt.linear(X, layer, None, "decode")
        Y = torch.empty(4, 48, dtype=torch.bfloat16, device="cuda")
        q.gptq_dequant_matmul_linear(X.cuda(), *layer.cuda(), None, 4, 128, Y)
        loss = 2.0 ** -80 * 512 * (1 + np.abs(layer.zeros).max()) * layer.scales.max()
        lt.check(Y, want, bound + loss, f"scale {scale}")


@pytest.mark.parametrize("tokens,scales", [(-60, -20), (60, -105), (90, 10), (-90, 100)])
@pytest.mark.parametrize("n,bits,g", [(40, 4, 128), (300, 4, 32), (20, 3, 128), (130, 8, 64), (9, 2, 16)])
def test_small_and_large_results_of_the_many_token_form(n, bits, g, tokens, scales):
    q = _q()
    rng = lt.rng_of(n, bits, g, tokens + 200, scales + 200)
    layer = lt.Layer(70, 384, bits, g, rng, scale=2.0 ** scales)
    X = (lt.bf16(rng, n, 384).float() * 2.0 ** tokens).to(torch.bfloat16)
    want, bound, _, _ = lt.linear(X, layer, None, "many")
    Y = torch.empty(n, 70, dtype=torch.bfloat16, device="cuda")
    q.gptq_dequant_gemm_linear(X.cuda(), *layer.cuda(), None, bits, g, Y,
                               lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(n, 384, 70)))
    lt.check(Y, want, bound, "Y")
