"""Calls of the products with an epilogue at the edges of their contract:
streams, other devices, bad permutations, extreme magnitudes, shared layers,
shapes that the Python entry points refuse."""
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


def _sizes(q, form, n, d_col, d_row):
    return (q.gptq_dequant_matmul_linear_workspace_size(n, d_col) if form == "decode"
            else q.gptq_dequant_gemm_linear_workspace_size(n, d_col, d_row))


def _linear(q, form):
    return q.gptq_dequant_matmul_linear if form == "decode" else q.gptq_dequant_gemm_linear


@pytest.mark.parametrize("form,n", [("decode", 7), ("many", 90), ("many", 300)])
def test_two_streams_at_once(form, n):
    """Two calls in flight on two streams, each with its workspace, the second
    one through the stream argument."""
    q = _q()
    rng = lt.rng_of(n, 1)
    d_col, d_row = 2048, 300
    layers = [lt.Layer(d_row, d_col, 4, 128, rng) for _ in range(2)]
    devs = [l.cuda() for l in layers]
    perm = rng.permutation(d_col).astype(np.int32)
    pd = lt.cuda(perm)
    X = [lt.bf16(rng, n, d_col) for _ in range(2)]
    Xd = [x.cuda() for x in X]
    Y = [torch.empty(n, d_row, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = [lt.workspace(_sizes(q, form, n, d_col, d_row)) for _ in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        _linear(q, form)(Xd[0], *devs[0], pd, 4, 128, Y[0], ws[0])
        _linear(q, form)(Xd[1], *devs[1], pd, 4, 128, Y[1], ws[1], stream=side)
    torch.cuda.synchronize()
    for x, l, y in zip(X, layers, Y):
        want, bound, _, _ = lt.linear(x, l, perm, form)
        lt.check(y, want, bound, "Y")


@pytest.mark.parametrize("form,n", [("decode", 5), ("many", 70)])
def test_a_bad_permutation_entry_is_read_as_its_position(form, n):
    """No access leaves the row."""
    q = _q()
    rng = lt.rng_of(n, 2)
    layer = lt.Layer(64, 256, 4, 64, rng)
    X = lt.bf16(rng, n, 256)
    perm = np.arange(256, dtype=np.int32)
    bad = perm.copy()
    bad[[3, 100, 255]] = [-1, 256, 1 << 30]
    want, bound, _, _ = lt.linear(X, layer, perm, form)
    Y = torch.empty(n, 64, dtype=torch.bfloat16, device="cuda")
    _linear(q, form)(X.cuda(), *layer.cuda(), lt.cuda(bad), 4, 64, Y, lt.workspace(_sizes(q, form, n, 256, 64)))
    lt.check(Y, want, bound, "Y")


def test_a_bad_permutation_entry_in_the_backward_pass():
    q = _q()
    rng = lt.rng_of(2, 2)
    n, d_col, d_row = 40, 256, 64
    layer = lt.Layer(d_row, d_col, 4, 64, rng)
    dY = lt.bf16(rng, n, d_row)
    bad = np.arange(d_col, dtype=np.int32)
    bad[[0, 77]] = [-5, d_col]
    buf, dX = lt.blank(n, d_col)
    q.gptq_dequant_gemm_linear_backward(dY.cuda(), *layer.cuda(), lt.cuda(bad), 4, 64, dX,
                                        lt.workspace(q.gptq_dequant_gemm_linear_backward_workspace_size(n, d_col, d_row)))
    x, xb = lt.back_product([dY], [layer], None)
    lt.check(dX, x, xb, "dX")
    lt.untouched(buf, d_col)


def test_magnitudes_of_the_decode_form():
    """Tokens from 2^-50 to 2^60 keep the result's relative accuracy; tokens
    below 2^-57 lose an absolute 2^-80 per product; from 2^64 on they may
    count as infinite: a token is multiplied by 2^(64 - j) for the position j of
    its code in the packed word's byte, 0 to 6, and bf16 ends below 2^128.  So
    2^64 does at j = 0 (column 0 of 4-bit codes), not at j = 4 (column 5), and
    2^70 everywhere."""
    q = _q()
    rng = lt.rng_of(6, 6)
    layer = lt.Layer(48, 512, 4, 128, rng)
    base = lt.bf16(rng, 4, 512)
    for e in (-50, 0, 60):
        X = (base.float() * 2.0 ** e).to(torch.bfloat16)
        # a normal deviate stays below 2^3, so the scaled tokens below 2^63
        want, bound, _, _ = lt.linear(X, layer, None, "decode")
        Y = torch.empty(4, 48, dtype=torch.bfloat16, device="cuda")
        q.gptq_dequant_matmul_linear(X.cuda(), *layer.cuda(), None, 4, 128, Y)
        lt.check(Y, want, bound, f"2^{e}")
    X = (base.float() * 2.0 ** -66).to(torch.bfloat16)
    want, bound, _, _ = lt.linear(X, layer, None, "decode")
    Y = torch.empty(4, 48, dtype=torch.bfloat16, device="cuda")
    q.gptq_dequant_matmul_linear(X.cuda(), *layer.cuda(), None, 4, 128, Y)
    # fp32's smallest step 2^-149 scaled back by 2^69, for each of the two sums'
    # products (512 codes and 512 ones times |z|), times the scale
    loss = 2.0 ** -80 * 512 * (1 + np.abs(layer.zeros).max()) * layer.scales.max()
    lt.check(Y, want, bound + loss, "2^-66")
    X = base.clone()
    X[2, 5] = 2.0 ** 63
    want, bound, _, _ = lt.linear(X, layer, None, "decode")
    q.gptq_dequant_matmul_linear(X.cuda(), *layer.cuda(), None, 4, 128, Y)
    lt.check(Y, want, bound, "2^63")
    X[2, 5] = 2.0 ** 64
    want, bound, _, _ = lt.linear(X, layer, None, "decode")
    q.gptq_dequant_matmul_linear(X.cuda(), *layer.cuda(), None, 4, 128, Y)
    lt.check(Y, want, bound, "2^64, j = 4")
    for col, e in ((0, 64), (5, 70)):
        X = base.clone()
        X[2, col] = 2.0 ** e
        q.gptq_dequant_matmul_linear(X.cuda(), *layer.cuda(), None, 4, 128, Y)
        assert not torch.isfinite(Y[2]).any() and torch.isfinite(Y[[0, 1, 3]]).all()


def test_large_magnitudes_of_the_many_token_form():
    """No such limit on the tensor cores' side: products up to fp32's range."""
    q = _q()
    rng = lt.rng_of(6, 7)
    layer = lt.Layer(48, 512, 4, 128, rng)
    for e in (-60, 100):
        X = (lt.bf16(rng, 150, 512).float() * 2.0 ** e).to(torch.bfloat16)
        want, bound, _, _ = lt.linear(X, layer, None, "many")
        Y = torch.empty(150, 48, dtype=torch.bfloat16, device="cuda")
        q.gptq_dequant_gemm_linear(X.cuda(), *layer.cuda(), None, 4, 128, Y,
                                   lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(150, 512, 48)))
        lt.check(Y, want, bound, f"2^{e}")


@pytest.mark.parametrize("activation", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activations_far_from_zero(activation):
    """Large positive and negative sums: no NaN from an overflowing exponential,
    forward and backward."""
    q = _q()
    rng = lt.rng_of(3, 9)
    n, d = 6, 64
    layer = lt.Layer(16, d, 4, 64, rng)
    X = lt.bf16(rng, n, d)
    bias = np.array([0, -1e4, 1e4, -100, 100, -40, 40, -12, 12, -1e30, 1e30, 3e38, -3e38, 1e-30, -6, 6], np.float32)
    for form in ("decode", "many"):
        want, bound, _, _ = lt.linear(X, layer, None, form, bias, activation)
        Y = torch.empty(n, 16, dtype=torch.bfloat16, device="cuda")
        _linear(q, form)(X.cuda(), *layer.cuda(), None, 4, 64, Y, lt.workspace(_sizes(q, form, n, d, 16)),
                         bias=lt.cuda(bias), activation=activation)
        got = lt.f64(Y)
        assert not np.isnan(got).any()
        keep = np.abs(want) < 3.3e38                  # bf16's largest is 3.39e38
        assert np.all(np.abs(got - want)[keep] <= bound[keep])
    pre = torch.from_numpy(np.tile(bias, (n, 1))).to(torch.bfloat16)
    dY = lt.bf16(rng, n, 16)
    dP = torch.empty(n, 16, dtype=torch.bfloat16, device="cuda")
    dX = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
    q.gptq_dequant_gemm_linear_backward(dY.cuda(), *layer.cuda(), None, 4, 64, dX,
                                        lt.workspace(q.gptq_dequant_gemm_linear_backward_workspace_size(n, d, 16)),
                                        activation=activation, pre=pre.cuda(), dPre=dP)
    # slopes beyond |x| = 100 are 0 or 1 to fp32's accuracy
    x = np.clip(lt.f64(pre), -100, 100)
    w = lt.f64(dY) * lt.act(x, activation)[1]
    lt.check(dP, w, lt.rounded_bound(w, np.abs(lt.f64(dY)) * lt.ACT_EPS), "dPre")


def test_one_layer_as_gate_and_up_and_an_inner_view():
    """The same packed layer in both places; X a column slice of a wider buffer."""
    q = _q()
    rng = lt.rng_of(11)
    layer = lt.Layer(100, 256, 2, 32, rng)
    wide = lt.bf16(rng, 30, 512).cuda()
    X = wide[:, 128:384]
    for form, n in (("decode", 30), ("many", 30)):
        Y = torch.empty(30, 100, dtype=torch.bfloat16, device="cuda")
        want, bound, _, _ = lt.gated(X.cpu(), layer, layer, None, form, "gelu")
        if form == "decode":
            q.gptq_dequant_matmul_gated(X, *layer.cuda(), *layer.cuda(), None, 2, 32, "gelu", Y)
        else:
            q.gptq_dequant_gemm_gated(X, *layer.cuda(), *layer.cuda(), None, 2, 32, "gelu", Y,
                                      lt.workspace(q.gptq_dequant_gemm_gated_workspace_size(30, 256, 100)))
        lt.check(Y, want, bound, form)


@pytest.mark.parametrize("form", ["decode", "many"])
def test_offsets_past_32_bits(form):
    """Rows of X, residual and Y more than 2^31 elements apart in all."""
    q = _q()
    rng = lt.rng_of(13)
    n, d_col, d_row, pitch = 40, 128, 72, 60_000_000
    layer = lt.Layer(d_row, d_col, 4, 64, rng)
    X, res = lt.bf16(rng, n, d_col), lt.bf16(rng, n, d_row)
    buf = torch.empty(n * pitch, dtype=torch.bfloat16, device="cuda").view(n, pitch)
    Xv, Rv, Y = buf[:, :d_col], buf[:, 1000:1000 + d_row], buf[:, 2000:2000 + d_row]
    Xv.copy_(X)
    Rv.copy_(res)
    want, bound, _, _ = lt.linear(X, layer, None, form, residual=res)
    _linear(q, form)(Xv, *layer.cuda(), None, 4, 64, Y, lt.workspace(_sizes(q, form, n, d_col, d_row)), residual=Rv)
    lt.check(Y, want, bound, "Y")


@pytest.mark.parametrize("bits,d_col", [(2, 64), (3, 128), (4, 64), (8, 64)])
def test_narrowest_layers(bits, d_col):
    """Packed rows of 16 to 64 bytes: every copy is wider than the layer."""
    q = _q()
    rng = lt.rng_of(bits, d_col, 14)
    layers = [lt.Layer(17, d_col, bits, 8, rng) for _ in range(2)]
    dev = [t for l in layers for t in l.cuda()]
    for n in (1, 20, 140, 300):
        X = lt.bf16(rng, n, d_col)
        Y = torch.empty(n, 17, dtype=torch.bfloat16, device="cuda")
        if n <= 20:
            want, bound, _, _ = lt.gated(X, *layers, None, "decode", "silu")
            q.gptq_dequant_matmul_gated(X.cuda(), *dev, None, bits, 8, "silu", Y)
            lt.check(Y, want, bound, f"decode {n}")
        want, bound, _, _ = lt.gated(X, *layers, None, "many", "silu")
        q.gptq_dequant_gemm_gated(X.cuda(), *dev, None, bits, 8, "silu", Y,
                                  lt.workspace(q.gptq_dequant_gemm_gated_workspace_size(n, d_col, 17)))
        lt.check(Y, want, bound, f"many {n}")
        dY, g, u = (lt.bf16(rng, n, 17) for _ in range(3))
        (_, dG), (_, dU) = lt.blank(n, 17, 24), lt.blank(n, 17, 24)
        dX = torch.empty(n, d_col, dtype=torch.bfloat16, device="cuda")
        q.gptq_dequant_gemm_gated_backward(dY.cuda(), g.cuda(), u.cuda(), *dev, None, bits, 8, "silu", dG, dU, dX,
                                           lt.workspace(q.gptq_dequant_gemm_gated_backward_workspace_size(n, d_col, 17)))
        x, xb = lt.back_product([dG, dU], layers, None)
        lt.check(dX, x, xb, f"dX {n}")


# Layers of at least 4096 weight rows take 64 rows per CTA unless two blocks of
# the rings then leave one CTA per SM; above 148 x 2 x 64 rows a CTA goes through
# several tiles.  K tails of 64 end inside a block of 128 codes.
@pytest.mark.parametrize("n,d_col,d_row,bits,g", [
    (1, 320, 4101, 4, 64), (5, 320, 4101, 4, 64), (8, 4160, 4096, 4, 64), (1, 320, 4101, 4, 32), (4, 2112, 4097, 4, 32),
    (5, 2112, 4097, 4, 32), (8, 320, 19001, 4, 32), (8, 320, 19001, 4, 64), (2, 256, 38001, 4, -1), (8, 384, 4101, 3, 32),
    (3, 384, 19001, 3, 64), (8, 320, 4101, 2, 32), (6, 320, 19001, 2, 64), (8, 320, 4101, 8, 128), (1, 320, 19001, 8, 64),
    (7, 320, 4101, 8, 32), (4, 192, 4101, 4, 16), (8, 192, 4101, 2, 8), (16, 320, 9601, 4, 64), (31, 320, 9601, 4, 32)])
def test_many_rows_few_tokens(n, d_col, d_row, bits, g):
    q = _q()
    rng = lt.rng_of(n, d_col, d_row, bits, g + 2, 15)
    layers = [lt.Layer(d_row, d_col, bits, g, rng) for _ in range(2)]
    X, res = lt.bf16(rng, n, d_col), lt.bf16(rng, n, d_row)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, bound, _, _ = lt.linear(X, layers[0], None, "decode", None, "gelu", res)
    buf, Y = lt.blank(n, d_row)
    q.gptq_dequant_matmul_linear(X.cuda(), *layers[0].cuda(), None, bits, g, Y, activation="gelu", residual=res.cuda(),
                                 dev_status=st)
    lt.check(Y, want, bound, "Y")
    lt.untouched(buf, d_row)
    want, bound, _, _ = lt.gated(X, *layers, None, "decode", "silu")
    buf, Y = lt.blank(n, d_row)
    q.gptq_dequant_matmul_gated(X.cuda(), *layers[0].cuda(), *layers[1].cuda(), None, bits, g, "silu", Y, dev_status=st)
    lt.check(Y, want, bound, "gated Y")
    lt.untouched(buf, d_row)
    assert q.gptq_sync_status(st) == 0


@pytest.mark.parametrize("n,d_col,d_row,bits", [(27, 512, 109, 4), (128, 576, 261, 8), (200, 640, 33, 3), (300, 512, 70, 2),
                                                (700, 1024, 515, 8), (5, 4096, 19, 4)])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_rows_off_their_boundaries(n, d_col, d_row, bits, offset):
    """Outputs and a residual updated in place whose rows start on 2, 16 or 32
    bytes, in whole tiles and in tiles whose contraction is split; what lies
    beside the rows stays."""
    q = _q()
    rng = lt.rng_of(n, d_col, d_row, bits, offset, 16)
    layer = lt.Layer(d_row, d_col, bits, 64, rng)
    X, res = lt.bf16(rng, n, d_col), lt.bf16(rng, n, d_row)
    bias = rng.standard_normal(d_row).astype(np.float32)
    want, bound, pw, pb = lt.linear(X, layer, None, "many", bias, "silu", res)
    ld = -(-(d_row + 9) // 16) * 16 + (offset & 1)
    bufs = [torch.full((n, ld), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    Y, pre = (b[:, offset:offset + d_row] for b in bufs)
    Y.copy_(res)
    ws = lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(n, d_col, d_row))
    q.gptq_dequant_gemm_linear(X.cuda(), *layer.cuda(), None, bits, 64, Y, ws, bias=lt.cuda(bias), activation="silu",
                               residual=Y, pre=pre)
    lt.check(Y, want, bound, "Y")
    lt.check(pre, pw, pb, "pre")
    for b in bufs:
        assert bool((b[:, :offset] == 7).all()) and bool((b[:, offset + d_row:] == 7).all())


def test_python_refusals():
    q = _q()
    rng = lt.rng_of(12)
    layer = lt.Layer(40, 256, 4, 64, rng).cuda()
    X = lt.bf16(rng, 6, 256).cuda()
    Y = torch.empty(6, 40, dtype=torch.bfloat16, device="cuda")

    def call(**kw):
        v = dict(X=X, layer=layer, perm=None, bits=4, g=64, Y=Y, ws=None, kw={})
        v.update(kw)
        q.gptq_dequant_matmul_linear(v["X"], *v["layer"], v["perm"], v["bits"], v["g"], v["Y"], v["ws"], **v["kw"])

    call()
    for err, kw in [
        (TypeError, dict(X=X.float())), (TypeError, dict(X=X.cpu())), (TypeError, dict(X=None)),
        (TypeError, dict(Y=Y.float())), (TypeError, dict(Y=Y.cpu())),
        (TypeError, dict(layer=(layer[0].float(), *layer[1:]))), (TypeError, dict(layer=(layer[0].cpu(), *layer[1:]))),
        (ValueError, dict(X=X[0])), (ValueError, dict(X=X.t().contiguous().t())), (ValueError, dict(X=X[:1].expand(6, 256))),
        (ValueError, dict(Y=Y[:5])), (ValueError, dict(Y=Y[:, :39])), (ValueError, dict(Y=torch.empty_like(Y).t().contiguous().t())),
        (ValueError, dict(layer=(layer[0][:, :-1].contiguous(), *layer[1:]))),
        (ValueError, dict(layer=(layer[0], layer[1][:3].contiguous(), layer[2]))),
        (ValueError, dict(layer=(layer[0], layer[1].t().contiguous().t(), layer[2]))),
        (ValueError, dict(perm=torch.arange(255, dtype=torch.int32, device="cuda"))),
        (TypeError, dict(perm=torch.arange(256, device="cuda"))),
        (ValueError, dict(kw=dict(bias=torch.zeros(39, device="cuda")))),
        (TypeError, dict(kw=dict(bias=torch.zeros(40, dtype=torch.bfloat16, device="cuda")))),
        (ValueError, dict(kw=dict(residual=Y[:, :20]))), (ValueError, dict(kw=dict(activation="swish"))),
        (TypeError, dict(kw=dict(dev_status=torch.zeros(1, device="cuda")))),
    ]:
        with pytest.raises(err):
            call(**kw)
    for status, kw in [(2, dict(g=48, layer=(layer[0], torch.zeros(6, 40, device="cuda"),
                                             torch.zeros(6, 40, dtype=torch.int32, device="cuda")))),
                       (6, dict(perm=torch.arange(256, dtype=torch.int32, device="cuda"))),
                       (1, dict(Y=None)), (1, dict(g=0))]:
        with pytest.raises(q.GPTQError) as e:
            call(**kw)
        assert e.value.status == status
