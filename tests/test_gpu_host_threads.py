"""Two host threads that call the library at the same time, each with its own
stream and workspace: a narrow and a wide layer through the same kernels, whose
launches need different amounts of shared memory."""
import threading

import numpy as np
import pytest
import torch

import linear_testlib as lt

pytestmark = pytest.mark.gpu

CALLS = 4000


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _q():
    import post_weight_quantization_gptq_b200 as q
    return q


def _recorded(q, name, call):
    """(entry point of the library, arguments without the stream) of the one
    call of `name` that `call` makes: repeated below without the Python entry
    point's work, which would keep the threads apart most of the time."""
    entry, got = getattr(q._lib, name), []
    try:
        setattr(q._lib, name, lambda *args: got.append(args) or entry(*args))
        call()
    finally:
        setattr(q._lib, name, entry)
    assert len(got) == 1
    return entry, got[0][:-1]


def _at_once(q, jobs, calls=CALLS):
    """Each job's call, `calls` times in a thread of its own; no call may fail,
    and the outputs are those of a call alone, bit for bit."""
    alone, recorded = [], []
    for name, call, outputs in jobs:
        recorded.append(_recorded(q, name, call))
        alone.append([t.clone() for t in outputs])
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(jobs)), []

    def work(entry, args, stream):
        torch.cuda.set_device(0)
        start.wait()
        for _ in range(calls):
            status = entry(*args, stream.cuda_stream)
            if status != 0:
                failed.append(status)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(*r, torch.cuda.Stream())) for r in recorded]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, f"{len(failed)} of {calls * len(jobs)} calls: {set(failed)}"
    for (name, call, outputs), want in zip(jobs, alone):
        assert name == "gptq_quantize_layer" or all(torch.equal(a, b) for a, b in zip(outputs, want))
        for t in outputs:
            t.zero_()
        call()
        assert all(torch.equal(a, b) for a, b in zip(outputs, want))


def _layer(d_col, d_row, seed):
    rng = lt.rng_of(d_col, d_row, seed)
    return rng, lt.Layer(d_row, d_col, 4, 128, rng).cuda(), lt.cuda(rng.permutation(d_col).astype(np.int32))


def _e(*shape):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda")


def test_decode_form():
    q = _q()

    def job(n, d_col, d_row):
        rng, layer, _ = _layer(d_col, d_row, 1)
        X, Y = lt.bf16(rng, n, d_col).cuda(), _e(n, d_row)
        return "gptq_dequant_matmul_linear", lambda: q.gptq_dequant_matmul_linear(X, *layer, None, 4, 128, Y), [Y]

    _at_once(q, [job(1, 128, 64), job(8, 8192, 64)])


def test_gather_of_the_many_token_forms():
    """Aligned rows, then rows that are not, with a permutation."""
    q = _q()

    def job(d_col, pad, linear):
        rng, layer, perm = _layer(d_col, 64, 2)
        _, X = lt.padded(lt.bf16(rng, 4, d_col), d_col + pad)
        if linear:
            Y, ws = _e(4, 64), lt.workspace(q.gptq_dequant_gemm_linear_workspace_size(4, d_col, 64))
            return "gptq_dequant_gemm_linear", lambda: q.gptq_dequant_gemm_linear(X, *layer, perm, 4, 128, Y, ws), [Y]
        Y = torch.empty(4, 64, device="cuda")
        ws = lt.workspace(q.gptq_dequant_gemm_workspace_size(4, d_col))
        return "gptq_dequant_gemm", lambda: q.gptq_dequant_gemm(X, *layer, perm, 4, 128, Y, ws), [Y]

    for pad in (0, 1):
        _at_once(q, [job(512, pad, True), job(16384, pad, True)])
        _at_once(q, [job(512, pad, False), job(16384, pad, True)])


def test_scatter_of_the_backward_pass():
    q = _q()

    def job(d_col):
        rng, layer, perm = _layer(d_col, 64, 3)
        dY, dX = lt.bf16(rng, 4, 64).cuda(), _e(4, d_col)
        ws = lt.workspace(q.gptq_dequant_gemm_linear_backward_workspace_size(4, d_col, 64))
        return "gptq_dequant_gemm_linear_backward", lambda: q.gptq_dequant_gemm_linear_backward(dY, *layer, perm, 4, 128, dX, ws), [dX]

    _at_once(q, [job(512), job(16384)])


def test_act_order_column_walk():
    """gptq_quantize_layer with act-order: the pass that permutes W's rows
    (which a call overwrites, so only a call on a fresh W is compared)."""
    q = _q()

    def job(d):
        rng = lt.rng_of(d, 4)
        W0 = torch.from_numpy(rng.standard_normal((4, d)).astype(np.float32)).cuda()
        W, U = torch.empty_like(W0), torch.eye(d, device="cuda")
        perm = lt.cuda(rng.permutation(d).astype(np.int32))
        dead = torch.zeros(d, dtype=torch.uint8, device="cuda")
        cfg = q.GPTQConfig(bits=4, group_size=128, desc_act=True)
        ng = q.n_groups(d, 128)
        codes = torch.empty(4, d, dtype=torch.uint8, device="cuda")
        scales, zeros = torch.empty(ng, 4, device="cuda"), torch.empty(ng, 4, dtype=torch.int32, device="cuda")
        ws = lt.workspace(q.gptq_workspace_size(cfg, 4, d))

        def call():
            W.copy_(W0)
            q.gptq_quantize_layer(W, U, perm, dead, cfg, codes, scales, zeros, None, ws)
        return "gptq_quantize_layer", call, [codes, scales, zeros]

    _at_once(q, [job(512), job(16384)], calls=200)
