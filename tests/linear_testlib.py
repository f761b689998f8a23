"""Inputs and float64 references of the products with packed layers that carry
their epilogue (gptq_dequant_matmul_linear / _gated and their tensor-core and
backward forms), with error bounds per output derived from the arithmetic the
header states.

Everything is computed on the CPU in float64 from the packed words themselves.
"""
import math

import numpy as np
import torch

import oracle

# a value in [2^e, 2^(e+1)) rounds by at most half a step: eps / 2 relative
HALF_BF16 = 2.0 ** -8
EPS32 = 2.0 ** -23


class Layer:
    """A packed layer: random words (every code equally likely), scales of both
    signs' worth of magnitudes and zero points inside and outside the code
    range."""

    def __init__(self, d_row, d_col, bits, g, rng, scale=0.02):
        self.bits, self.g, self.d_col, self.d_row = bits, g, d_col, d_row
        words = d_col * bits // 32
        self.packed = rng.integers(0, 1 << 32, size=(d_row, words), dtype=np.uint64).astype(np.uint32)
        self.gg = d_col if g == -1 or g > d_col else g
        ng = -(-d_col // self.gg)
        self.scales = (scale * (rng.random((ng, d_row)) + 0.1)).astype(np.float32)
        self.zeros = rng.integers(-2, (1 << bits) + 2, size=(ng, d_row)).astype(np.int32)

    def codes(self):
        return oracle.unpack(self.packed, self.d_col, self.bits)

    def weights(self, rounded):
        """W_hat in quantization order, float64."""
        gi = np.arange(self.d_col) // self.gg
        s = self.scales[gi, :].T
        m = self.codes().astype(np.float64) - self.zeros[gi, :].T
        if rounded:
            return oracle.bf16_round((s * m.astype(np.float32)).astype(np.float32)).astype(np.float64)
        return s.astype(np.float64) * m

    def magnitudes(self):
        """s (q + |z|), the magnitudes that the decode form's per-group sums
        (of x q and of z x) pass through, float64."""
        gi = np.arange(self.d_col) // self.gg
        s = self.scales[gi, :].T.astype(np.float64)
        return s * (self.codes().astype(np.float64) + np.abs(self.zeros[gi, :].T))

    def cuda(self):
        return (torch.from_numpy(self.packed.view(np.int32)).cuda(), torch.from_numpy(self.scales).cuda(),
                torch.from_numpy(self.zeros).cuda())


def rng_of(*key):
    return np.random.default_rng(sum((i + 1) * 7919 * int(k) for i, k in enumerate(key)) + 11)


def bf16(rng, *shape, std=1.0):
    return torch.from_numpy((std * rng.standard_normal(shape)).astype(np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(x, name):
    """(value, slope) in float64."""
    x = np.asarray(x, dtype=np.float64)
    if name == "none":
        return x, np.ones_like(x)
    if name == "relu":
        return np.maximum(x, 0), (x > 0).astype(np.float64)
    if name == "silu":
        s = 1 / (1 + np.exp(-np.clip(x, -700, 700)))
        return x * s, s * (1 + x * (1 - s))
    if name == "gelu":
        cdf = 0.5 * _erfc(-x / math.sqrt(2))
        return x * cdf, cdf + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = np.tanh(c * (x + 0.044715 * x ** 3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


# Largest slope of any of the activations (GELU: 1 + 0.129).
LIPSCHITZ = 1.13
# Relative error of an activation and absolute error of a slope (at most 1.13)
# in fp32: exp's argument y carries a rounding of |y| 2^-24, |y| < 104 where
# the result has not underflowed, so 52 units of 2^-23, and a dozen roundings.
ACT_EPS = 64 * EPS32


def ordered(X, perm):
    x = f64(X)
    return x if perm is None else x[:, perm]


def product(X, layer, perm, form):
    """(sum, bound of its fp32 error) of one product in float64.

    decode: per 16 codes one tensor-core step, whose rounding is at most one
    unit of 2^-23 of the running magnitude, which stays below
    sum_k |x_k| s (q + |z|); per group three more roundings, per 128-code
    block one, plus the joins: K / 16 + 3 K / 8 (groups of 8) + 64 of them
    cover every group size.
    many: at most one rounding per 16 terms plus the sums inside a step, each
    within 2^-23 of sum_k |x_k w_k| (twice that allowed), plus the joins of a
    split K."""
    x = ordered(X, perm)
    K = x.shape[1]
    w = layer.weights(form != "decode")
    y = x @ w.T
    if form == "decode":
        bound = (K / 16 + 3 * K / min(128, layer.gg) + 64) * EPS32 * (np.abs(x) @ layer.magnitudes().T)
    else:
        bound = 2 * (K / 16 + 64) * EPS32 * (np.abs(x) @ np.abs(w).T)
    return y, bound


def rounded_bound(y, err):
    """Bound of |bf16(y') - y| where |y' - y| <= err."""
    return err + HALF_BF16 * (np.abs(y) + err)


def linear(X, layer, perm, form, bias=None, activation="none", residual=None):
    """(Y, bound, pre, pre bound) in float64."""
    p, e = product(X, layer, perm, form)
    if bias is not None:
        p = p + bias.astype(np.float64)
        e = e + EPS32 * np.abs(p)
    y = act(p, activation)[0]
    ey = LIPSCHITZ * e + ACT_EPS * np.abs(y) + 1e-30
    if residual is not None:
        y = y + f64(residual)
        ey = ey + EPS32 * np.abs(y)
    return y, rounded_bound(y, ey), p, rounded_bound(p, e)


def gated(X, gate, up, perm, form, activation):
    """(Y, bound, (gate, bound), (up, bound)) in float64."""
    (pg, eg), (pu, eu) = product(X, gate, perm, form), product(X, up, perm, form)
    a = act(pg, activation)[0]
    ea = LIPSCHITZ * eg + ACT_EPS * np.abs(a)
    y = a * pu
    ey = ea * np.abs(pu) + np.abs(a) * eu + ea * eu + EPS32 * np.abs(y) + 1e-30
    return y, rounded_bound(y, ey), (pg, rounded_bound(pg, eg)), (pu, rounded_bound(pu, eu))


def check(got, want, bound, what):
    g = f64(got) if isinstance(got, torch.Tensor) else got
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    err = np.abs(g - want)
    worst = np.max(err / bound)
    print(f"{what}: max |err| / bound {worst:.3f}")
    assert worst <= 1.0, f"{what}: {worst} at {np.unravel_index(np.argmax(err / bound), err.shape)}"


def slopes_linear(dY, pre, activation):
    """(dP, bound) in float64."""
    d = f64(dY)
    if activation == "none":
        return d, HALF_BF16 * np.abs(d)
    p = d * act(f64(pre), activation)[1]
    return p, rounded_bound(p, np.abs(d) * ACT_EPS)


def slopes_gated(dY, gate, up, activation):
    """((dG, bound), (dU, bound)) in float64."""
    d, u = f64(dY), f64(up)
    v, sl = act(f64(gate), activation)
    dg, du = d * u * sl, d * v
    return ((dg, rounded_bound(dg, np.abs(d * u) * ACT_EPS)),
            (du, rounded_bound(du, np.abs(du) * ACT_EPS + 1e-30)))


def back_product(dPs, layers, perm):
    """(dX, bound) in float64 from the bf16 gradients that the call wrote: at
    most one rounding per 16 terms plus the sums inside a step, each within
    2^-23 of the sum of magnitudes (twice that allowed), plus the joins."""
    y = e = 0
    for d, layer in zip(dPs, layers):
        w = layer.weights(True)
        y = y + f64(d) @ w
        e = e + np.abs(f64(d)) @ np.abs(w)
    terms = sum(d.shape[1] for d in dPs)
    bound = rounded_bound(y, 2 * (terms / 16 + 64) * EPS32 * e)
    if perm is not None:
        out, ob = np.empty_like(y), np.empty_like(y)
        out[:, perm], ob[:, perm] = y, bound
        return out, ob
    return y, bound


def padded(t, ld, fill=float("nan"), offset=0):
    """t's values as a view of a wider CUDA buffer whose other entries are `fill`."""
    n, c = t.shape
    buf = torch.full((n * ld + offset,), fill, dtype=t.dtype, device="cuda")
    v = buf[offset:offset + n * ld].view(n, ld)[:, :c]
    v.copy_(t)
    return buf, v


def blank(n, c, ld=None):
    """An n x c bf16 output of NaNs in a buffer whose other entries are 7."""
    ld = c + 3 if ld is None else ld
    buf = torch.full((n, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    v = buf[:, :c]
    v.fill_(float("nan"))
    return buf, v


def untouched(buf, c):
    assert torch.all(buf[:, c:] == 7.0), "written outside the output"


def cuda(x):
    if x is None:
        return None
    return x.cuda() if isinstance(x, torch.Tensor) else torch.from_numpy(x).cuda()


def workspace(size):
    """A workspace of exactly `size` bytes full of NaN bit patterns."""
    return torch.full((size,), 255, dtype=torch.uint8, device="cuda") if size else None
