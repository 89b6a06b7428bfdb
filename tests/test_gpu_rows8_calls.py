"""GPU: the 8-bit rows and projections in calls that are allowed, or refused,
and that no other test makes."""
import ctypes

import numpy as np
import pytest
import torch

from deepseek_sparse_attention_dsa_gb300 import dsa
from deepseek_sparse_attention_dsa_gb300 import workloads as W
from tests.test_gpu_rows8 import placed, rand

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def ctx():
    from deepseek_sparse_attention_dsa_gb300 import build
    build.build()
    return dsa.Context(W.DSAShape(**W.DEEPSEEK), 0)


def test_a_launch_that_is_refused_spoils_no_later_call(ctx):
    """A launch into the default stream while another stream is captured is
    refused by the runtime; the calls after it are not told of that error."""
    x = placed(rand(1, 4, 256), BF16)
    codes, scales = ctx.quantize_rows(x)
    want = codes.clone()
    plan = ctx.plan([W.Span(0, 0, 3, 0, np.zeros(1, np.int32))], 1)
    keys = torch.zeros(3, 128, dtype=BF16, device="cuda")
    cache = torch.zeros(1, 64, 128, dtype=BF16, device="cuda")
    L = dsa.load()
    shape = dsa._Rows(rows=4, width=256, x_type=0, x_stride=256, codes_stride=256, scales_stride=2)
    args = [ctypes.c_void_p(t.data_ptr()) for t in (x, codes, scales)]
    store = [ctypes.c_void_p(t.data_ptr()) for t in (keys, cache)]
    cudart = ctypes.CDLL("libcudart.so.13")
    own, graph, other = ctypes.c_void_p(), ctypes.c_void_p(), torch.cuda.Stream()
    assert cudart.cudaStreamCreate(ctypes.byref(own)) == 0           # one that the default stream waits for
    torch.cuda.synchronize()
    assert cudart.cudaStreamBeginCapture(own, 0) == 0                # global mode
    refused = L.dsa_quantize_rows(ctx.handle, None, ctypes.byref(shape), *args, ctypes.c_void_p(1))   # cudaStreamLegacy
    after = L.dsa_store_keys(ctx.handle, plan.handle, *store, ctypes.c_void_p(other.cuda_stream))     # on a stream of its own
    cudart.cudaStreamEndCapture(own, ctypes.byref(graph))            # (no graph: the capture ended with the refused call)
    cudart.cudaGetLastError()
    assert refused == 4 and b"cudaErrorStreamCapture" in L.dsa_last_cuda_error(ctx.handle)
    assert after == dsa.DSA_OK
    torch.cuda.synchronize()
    assert cudart.cudaStreamDestroy(own) == 0
    assert torch.equal(ctx.quantize_rows(x)[0], want)
    ctx.get_error()


def test_pointers_off_their_type_are_refused(ctx):
    """Through the C calls (a tensor is always on its type's size): each pointer in turn one byte, or half a float, off."""
    L = dsa.load()
    store = torch.zeros(16 * 4096, dtype=U8, device="cuda")
    base = store.data_ptr()
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    norm = dsa._Norm(rows=2, width=128, x_type=0, weight_type=1, residual_type=1, out_type=0, eps=1e-6, x_stride=128, residual_stride=128,
                     residual_out_stride=128, out_stride=128, codes_stride=128, scales_stride=1)
    rows = dsa._Rows(rows=2, width=128, x_type=1, x_stride=128, codes_stride=128, scales_stride=1)
    weight = dsa._Weight(batch=1, n=2, k=128, w_type=0, w_stride=128, codes_stride=128, scales_stride=1)
    project = dsa._Project(rows=2, batch=1, n=2, k=128, out_type=0, a_stride=128, a_scale_stride=1, w_stride=128, w_scale_stride=1, out_stride=2)
    # the call with its tensors in order, and the bytes that each has to be on
    calls = ((lambda *p: L.dsa_rmsnorm(ctx.handle, None, ctypes.byref(norm), *p, stream), (2, 4, 4, 4, 2, 1, 4)),
             (lambda *p: L.dsa_quantize_rows(ctx.handle, None, ctypes.byref(rows), *p, stream), (4, 1, 4)),
             (lambda *p: L.dsa_quantize_weight(ctx.handle, ctypes.byref(weight), *p, stream), (2, 1, 4)),
             (lambda *p: L.dsa_project_fp8(ctx.handle, None, ctypes.byref(project), *p, stream), (1, 4, 1, 4, 2)))
    for call, on in calls:
        at = [base + 4096 * i for i in range(len(on))]
        assert call(*map(ctypes.c_void_p, at)) == dsa.DSA_OK
        for i, size in enumerate(on):
            for off in {1, size // 2, size - 1} - {0}:
                moved = at[:i] + [at[i] + off] + at[i + 1:]
                got = call(*map(ctypes.c_void_p, moved))
                assert got == (1 if size > 1 else dsa.DSA_OK), (i, off)
    ctx.get_error()


def test_a_captured_fork_and_join(ctx):
    """Two streams in one graph whose launches overlap with each other's: the
    norm's codes go into two projections on two streams, whose outputs are
    quantised after the join; replayed over new inputs in the same buffers."""
    g = torch.Generator().manual_seed(4)
    ws = [ctx.quantize_weight((torch.randn(n, 1024, generator=g) / 32).to(BF16).cuda()) for n in (512, 2048)]
    x, res = (torch.zeros(70, 1024, dtype=BF16, device="cuda") for _ in range(2))

    def step(main, side):
        codes, scales, h = ctx.rmsnorm_quantize(x, None, residual=res)
        fork, join = torch.cuda.Event(), torch.cuda.Event()
        fork.record(main)
        side.wait_event(fork)
        with torch.cuda.stream(side):
            b = ctx.project_fp8(codes, scales, *ws[1])
            bq = ctx.quantize_rows(b)
            join.record(side)
        a = ctx.project_fp8(codes, scales, *ws[0])
        main.wait_event(join)
        return [codes, scales, h, a, b, *bq, *ctx.quantize_rows(a), ctx.rmsnorm(b, None)]

    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(main):
        step(main, side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        got = step(main, side)
    for seed in range(5, 9):
        x.copy_(rand(seed, 70, 1024))
        res.copy_(rand(seed + 50, 70, 1024))
        torch.cuda.synchronize()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        with torch.cuda.stream(main):
            want = step(main, side)
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(kept, want)):
            assert torch.equal(p, q), (seed, i)
    ctx.get_error()


def test_the_same_tensor_as_both_operands(ctx):
    """A product of codes with themselves: whole numbers, so exact."""
    g = torch.Generator().manual_seed(5)
    for rows in (1, 40, 200):
        codes = torch.randint(-3, 4, (rows, 384), generator=g).float().to(torch.float8_e4m3fn).cuda()
        ones = torch.ones(rows, 3, device="cuda")
        out = ctx.project_fp8(codes, ones, codes, torch.ones(-(-rows // 128), 3, device="cuda"), out_dtype=F32)
        v = codes.float()
        assert torch.equal(out, v @ v.t()) or torch.equal(out.double(), v.double() @ v.double().t())
    ctx.get_error()


def test_no_rows_and_rows_that_are_all_padding(ctx):
    """Nothing to do, with and without a plan: nothing is written, nothing is wrong."""
    from tests.test_gpu_rows8 import capturable
    plan = capturable(ctx, 0)
    empty = ctx.plan([], 1)
    w = torch.zeros(128, 256, dtype=U8, device="cuda"), torch.ones(1, 2, device="cuda")
    for rows, p in ((0, None), (0, empty), (0, plan), (8, plan), (64, plan)):
        x = torch.full((rows, 256), float("nan"), dtype=BF16, device="cuda")
        out, codes = torch.full((rows, 256), 7.0, dtype=BF16, device="cuda"), torch.full((rows, 256), 9, dtype=U8, device="cuda")
        scales, y = torch.full((rows, 2), 5.0, device="cuda"), torch.full((rows, 128), 3.0, dtype=BF16, device="cuda")
        ctx.rmsnorm(x, None, out=out, plan=p)
        ctx.quantize_rows(x, codes, scales, plan=p)
        ctx.project_fp8(codes, scales, *w, out=y, plan=p)
        assert (out == 7).all() and (codes == 9).all() and (scales == 5).all() and (y == 3).all()
    ctx.get_error()
