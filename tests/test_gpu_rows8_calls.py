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
