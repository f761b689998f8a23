"""The activations' slopes in fp32: the bias gradient of a single token is
dY act'(pre) unrounded, here at every finite bf16 pre-activation."""
import math

import numpy as np
import pytest
import torch

import linear_testlib as lt

pytestmark = pytest.mark.gpu

U = lt.EPS32   # 2^-23; a rounding is at most U / 2 relative


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _bound(x, activation):
    """Absolute error of a slope a + b in fp32: a the share 1 / (1 + 2^y) (or the
    normal distribution's), b the term with x.

    2^y: the exponent's own roundings (k of U / 2 each) times ln 2 |y|, and two
    units of the approximate instruction.  a: that times 1 - a, and one and a half
    units for 1 + e and the reciprocal.  b = x a (1 - a) ...: a twice, e once, and
    as many roundings as it has factors (twelve allowed).  GELU: erfc to 4 units
    and its argument's rounding (times the density: at most |b|), exp to
    2 + 1.173 times its argument and the argument's rounding."""
    if activation == "gelu":
        a = np.vectorize(lambda v: 0.5 * math.erfc(-v / math.sqrt(2)))(x)
        b = np.abs(x) * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        err = 5 * U * a + U * b + b * U * (8 + 1.673 * x * x / 2)
    elif activation == "relu":
        a = b = err = np.zeros_like(x)
    else:
        c = math.sqrt(2 / math.pi)
        if activation == "silu":
            y, k, factor = -x * math.log2(math.e), 2, np.ones_like(x)
        else:
            y, k, factor = -2 * math.log2(math.e) * c * (x + 0.044715 * x ** 3), 5, 2 * c * (1 + 3 * 0.044715 * x * x)
        e = np.exp2(np.clip(y, -1000, 1000))
        a, rest = 1 / (1 + e), 1 / (1 + 1 / e)
        b = np.abs(x) * a * rest * factor
        ee = k * U / 2 * math.log(2) * np.abs(y) + 2 * U
        err = a * (rest * ee + 1.5 * U) + b * (3 * ee + 6 * U)
    return err + U * (np.abs(a) + b) + 2.0 ** -100   # the sum; what underflows


@pytest.mark.parametrize("activation", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_to_fp32_accuracy(activation):
    import post_weight_quantization_gptq_b200 as q
    x = torch.from_numpy(np.arange(65536, dtype=np.uint16).view(np.int16)).view(torch.bfloat16)
    x = x[torch.isfinite(x)]
    d = len(x) // 8 * 8
    x = x[-d:]
    layer = lt.Layer(d, 64, 4, 64, lt.rng_of(41)).cuda()
    dY, dP = torch.ones(1, d, dtype=torch.bfloat16, device="cuda"), torch.empty(1, d, dtype=torch.bfloat16, device="cuda")
    dbias, dX = torch.empty(d, device="cuda"), torch.empty(1, 64, dtype=torch.bfloat16, device="cuda")
    q.gptq_dequant_gemm_linear_backward(dY, *layer, None, 4, 64, dX,
                                        lt.workspace(q.gptq_dequant_gemm_linear_backward_workspace_size(1, 64, d)),
                                        activation=activation, pre=x[None].cuda(), dPre=dP, dbias=dbias)
    v = np.clip(lt.f64(x), -100, 100)   # beyond: 0 or 1 to fp32's accuracy
    # SILU's slope in a form without cancellation; the others as the formulas have them
    s = 1 / (1 + np.exp(-v))
    want = s + v * s / (1 + np.exp(v)) if activation == "silu" else lt.act(v, activation)[1]
    if activation == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        h, rest = 1 / (1 + np.exp(np.clip(-2 * u, -700, 700))), 1 / (1 + np.exp(np.clip(2 * u, -700, 700)))
        want = h + 2 * v * h * rest * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v * v)
    lt.check(dbias, want, _bound(v, activation), activation)
    print(f"{activation}: max |err| {np.abs(lt.f64(dbias) - want).max() * 2 ** 24:.2f} units of 2^-24")
