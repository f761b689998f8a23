"""Workspaces of the tensor-core products with an epilogue: one that serves a
batch serves every smaller one, and a call needs no more than it uses."""
import numpy as np
import pytest
import torch

import linear_testlib as lt


@pytest.fixture(scope="module")
def q():
    import post_weight_quantization_gptq_b200 as pkg
    return pkg


FORMS = ["gptq_dequant_gemm_linear", "gptq_dequant_gemm_gated", "gptq_dequant_gemm_linear_backward",
         "gptq_dequant_gemm_gated_backward"]


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("d_col,d_row", [(64, 1), (1024, 4096), (4096, 1024), (4096, 11008), (11008, 4096),
                                         (8192, 8192), (320, 19001), (16384, 100)])
def test_sizes_do_not_fall_as_tokens_are_added(q, name, d_col, d_row):
    size = getattr(q, name + "_workspace_size")
    ns = sorted(set(range(1, 1100)) | {k * 128 + i for k in range(8, 200) for i in (-1, 0, 1)})
    sizes = [size(n, d_col, d_row) for n in ns]
    assert sizes[0] > 0 and all(s % 256 == 0 for s in sizes)
    falls = [(n, a, b) for n, a, b in zip(ns[1:], sizes, sizes[1:]) if b < a]
    assert not falls, falls[:3]
    # the tokens, the split tiles of at most one wave, and 256 slabs of bias sums
    most = ns[-1] * d_col * 2 + 74 * 512 * 256 * 4 + 256 * d_row * 4 + 1024
    assert sizes[-1] <= most


def _setup(n, d_col, d_row, with_perm):
    rng = lt.rng_of(n, d_col, d_row, with_perm, 21)
    layers = [lt.Layer(d_row, d_col, 4, 128, rng) for _ in range(2)]
    perm = rng.permutation(d_col).astype(np.int32) if with_perm else None
    return rng, layers, perm


def _e(*shape):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("name", FORMS)
def test_a_workspace_of_the_largest_batch_serves_the_smaller_ones(q, name):
    """Guard bytes behind the workspace stay."""
    d_col, d_row, most = 512, 1152, 3000
    rng, layers, perm = _setup(most, d_col, d_row, True)
    dev, pd = [l.cuda() for l in layers], lt.cuda(perm)
    size = getattr(q, name + "_workspace_size")(most, d_col, d_row)
    buf = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    ws = buf[:size]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n in (1, 60, 128, 129, 200, 256, 257, 300, 512, 513, 700, 1024, 2048, 2049):
        X, dY = lt.bf16(rng, n, d_col), lt.bf16(rng, n, d_row)
        if name == "gptq_dequant_gemm_linear":
            Y = _e(n, d_row)
            q.gptq_dequant_gemm_linear(X.cuda(), *dev[0], pd, 4, 128, Y, ws, dev_status=st)
            want = lt.linear(X, layers[0], perm, "many")
        elif name == "gptq_dequant_gemm_gated":
            Y = _e(n, d_row)
            q.gptq_dequant_gemm_gated(X.cuda(), *dev[0], *dev[1], pd, 4, 128, "silu", Y, ws, dev_status=st)
            want = lt.gated(X, *layers, perm, "many", "silu")
        elif name == "gptq_dequant_gemm_linear_backward":
            Y, dbias = _e(n, d_col), torch.empty(d_row, device="cuda")
            q.gptq_dequant_gemm_linear_backward(dY.cuda(), *dev[0], pd, 4, 128, Y, ws, dbias=dbias, dev_status=st)
            want = lt.back_product([dY], layers[:1], perm)
            # a chain of at most n / 8 terms, 8 and the slabs' joins
            lt.check(dbias, lt.f64(dY).sum(0), (n / 8 + 80) * lt.EPS32 * np.abs(lt.f64(dY)).sum(0), f"dbias {n}")
        else:
            Y, dG, dU = _e(n, d_col), _e(n, d_row), _e(n, d_row)
            q.gptq_dequant_gemm_gated_backward(dY.cuda(), lt.bf16(rng, n, d_row).cuda(), lt.bf16(rng, n, d_row).cuda(),
                                               *dev[0], *dev[1], pd, 4, 128, "silu", dG, dU, Y, ws, dev_status=st)
            want = lt.back_product([dG, dU], layers, perm)
        lt.check(Y, want[0], want[1], f"{n} tokens")
        assert q.gptq_sync_status(st) == 0
        assert bool((buf[size:] == 255).all())


@pytest.mark.gpu
@pytest.mark.parametrize("n,d_col,d_row", [(300, 4096, 300), (90, 2048, 260)])
def test_a_call_that_only_splits_needs_no_room_for_its_tokens(q, n, d_col, d_row):
    """Without a permutation the tokens are read where they are; with one the
    same workspace is refused."""
    rng, layers, _ = _setup(n, d_col, d_row, False)
    perm = lt.cuda(rng.permutation(d_col).astype(np.int32))
    dev = layers[0].cuda()
    X, Y = lt.bf16(rng, n, d_col), _e(n, d_row)
    ws = lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(n, d_col, d_row) - n * d_col * 2)
    q.gptq_dequant_gemm_linear(X.cuda(), *dev, None, 4, 128, Y, ws)
    want = lt.linear(X, layers[0], None, "many")
    lt.check(Y, want[0], want[1], "Y")
    with pytest.raises(q.GPTQError) as e:
        q.gptq_dequant_gemm_linear(X.cuda(), *dev, perm, 4, 128, Y, ws)
    assert e.value.status == 6
    # backward: the roles of the widths change places
    layer = lt.Layer(d_col, 320, 4, 64, rng)
    dY, dX = lt.bf16(rng, n, d_col), _e(n, 320)
    size = q.gptq_dequant_gemm_linear_backward_workspace_size(n, 320, d_col)
    slabs = -(-n // 8) * d_col * 4
    ws = lt.workspace((size - n * 320 * 2 - slabs) // 256 * 256)
    q.gptq_dequant_gemm_linear_backward(dY.cuda(), *layer.cuda(), None, 4, 64, dX, ws)
    want = lt.back_product([dY], [layer], None)
    lt.check(dX, want[0], want[1], "dX")
    with pytest.raises(q.GPTQError) as e:
        q.gptq_dequant_gemm_linear_backward(dY.cuda(), *layer.cuda(), None, 4, 64, dX, ws,
                                            dbias=torch.empty(d_col, device="cuda"))
    assert e.value.status == 6
