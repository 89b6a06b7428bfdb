"""The 8-bit rows and projections on the host (no GPU): the binding's checks
of shapes, types and layouts, and the statuses of the C entry points for sizes
that they refuse before they look at a device."""
import ctypes

import pytest
import torch

from deepseek_sparse_attention_dsa_gb300 import build as dsa_build
from deepseek_sparse_attention_dsa_gb300 import dsa
from deepseek_sparse_attention_dsa_gb300 import workloads as W

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def ctx():
    dsa_build.build()
    return dsa.Context(W.DSAShape(**W.DEEPSEEK), device=-1)   # its tensors are the host's


@pytest.fixture()
def lib(ctx):
    return dsa.load()


def test_norm_checks_its_tensors(ctx):
    x = torch.zeros(4, 256, dtype=BF16)
    with pytest.raises(ValueError):
        ctx.rmsnorm(x[0], None)                                     # one dimension
    with pytest.raises(TypeError):
        ctx.rmsnorm(x.half(), None)
    with pytest.raises(ValueError):
        ctx.rmsnorm(x, torch.zeros(255, dtype=BF16))
    with pytest.raises(ValueError):
        ctx.rmsnorm(x, torch.zeros(512, dtype=BF16)[::2])           # values not adjacent
    with pytest.raises(ValueError):
        ctx.rmsnorm(x, None, residual=x[:3])
    with pytest.raises(TypeError):
        ctx.rmsnorm(x, None, residual=x, residual_out=x.float())    # the residual's own type
    with pytest.raises(ValueError):
        ctx.rmsnorm(x, None, residual_out=x)
    with pytest.raises(ValueError):
        ctx.rmsnorm(torch.zeros(256, 4, dtype=BF16).t(), None)
    with pytest.raises(ValueError):
        ctx.rmsnorm_quantize(x, None, scales=torch.zeros(4, 3))
    with pytest.raises(TypeError):
        ctx.rmsnorm_quantize(x, None, codes=torch.zeros(4, 256, dtype=torch.int8))


def test_quantisers_check_their_tensors(ctx):
    x = torch.zeros(4, 256, dtype=BF16)
    with pytest.raises((TypeError, KeyError)):
        ctx.quantize_rows(x.double())
    with pytest.raises(ValueError):
        ctx.quantize_rows(x.view(2, 2, 256))
    with pytest.raises(ValueError):
        ctx.quantize_rows(x, codes=torch.zeros(4, 255, dtype=U8))
    with pytest.raises(ValueError):
        ctx.quantize_weight(x[0])
    with pytest.raises(ValueError):
        ctx.quantize_weight(x, scales=torch.zeros(2, 2))


def test_project_checks_its_tensors(ctx):
    a, asc = torch.zeros(4, 256, dtype=U8), torch.zeros(4, 2)
    w, wsc = torch.zeros(130, 256, dtype=U8), torch.zeros(2, 2)
    for bad in ((a.to(torch.int8), asc, w, wsc), (a, asc.double(), w, wsc)):
        with pytest.raises(TypeError):
            ctx.project_fp8(*bad)
    for bad in ((a[:, :255], asc, w, wsc), (a, asc[:, :1], w, wsc), (a, asc, w, wsc[:1]), (a[0], asc, w, wsc),
                (a.view(4, 1, 256), asc, w, wsc), (a.view(2, 2, 256), asc.view(2, 2, 2), w.view(1, 130, 256), wsc[None])):
        with pytest.raises(ValueError):
            ctx.project_fp8(*bad)
    with pytest.raises(TypeError):
        ctx.project_fp8(a, asc, w, wsc, out=torch.zeros(4, 130, dtype=torch.float16))


def test_calls_refuse_a_host_only_context(ctx):
    x = torch.zeros(4, 256, dtype=BF16)
    for call in (lambda: ctx.rmsnorm(x, None), lambda: ctx.quantize_rows(x), lambda: ctx.quantize_weight(x),
                 lambda: ctx.project_fp8(x.to(U8), torch.zeros(4, 2), x.to(U8), torch.zeros(1, 2))):
        with pytest.raises(dsa.DSAError) as e:
            call()
        assert e.value.status == 1


def test_calls_refuse_closed_contexts_and_plans():
    c = dsa.Context(W.DSAShape(**W.DEEPSEEK), device=-1)
    plan = c.plan([], 1)
    x = torch.zeros(4, 256, dtype=BF16)
    calls = [lambda p: c.rmsnorm(x, None, plan=p), lambda p: c.rmsnorm_quantize(x, None, plan=p),
             lambda p: c.quantize_rows(x, plan=p),
             lambda p: c.project_fp8(x.to(U8), torch.zeros(4, 2), x.to(U8), torch.zeros(1, 2), plan=p)]
    plan.close()
    for call in calls:      # not taken for a call without a plan
        with pytest.raises(dsa.DSAError, match="plan"):
            call(plan)
    c.close()
    for call in calls + [lambda p: c.quantize_weight(x)]:
        with pytest.raises(dsa.DSAError) as e:
            call(None)
        assert e.value.status == 1


def _norm(**kw):
    base = dict(rows=4, width=256, eps=1e-6, x_stride=256, residual_stride=256, residual_out_stride=256, out_stride=256,
                codes_stride=256, scales_stride=2)
    base.update(kw)
    return dsa._Norm(**base)


def test_sizes_beyond_the_limits_are_told_from_bad_ones(ctx, lib):
    """Statuses that do not depend on a device: 7 (unsupported) for sizes, 1 for what no call can mean."""
    one = ctypes.c_void_p(16)

    def norm(**kw):
        return lib.dsa_rmsnorm(ctx.handle, None, _norm(**kw), one, None, None, None, one, None, None, None)

    assert norm(width=32769) == 7 and norm(width=32768) == 1   # the latter for the host-only context
    for bad in (dict(width=0), dict(x_type=2), dict(out_type=-1), dict(eps=-1e-9), dict(x_stride=-1), dict(rows=-1)):
        assert norm(**bad) == 1
    w = dict(batch=1, n=128, k=128, w_stride=128, codes_stride=128, scales_stride=1)

    def weight(**kw):
        return lib.dsa_quantize_weight(ctx.handle, dsa._Weight(**dict(w, **kw)), one, one, one, None)

    assert weight() == 1 and weight(k=0) == 1 and weight(batch=0) == 1
    p = dict(rows=1, batch=1, n=128, k=128, a_stride=128, a_scale_stride=1, w_stride=128, w_scale_stride=1, out_stride=128)

    def project(**kw):
        return lib.dsa_project_fp8(ctx.handle, None, dsa._Project(**dict(p, **kw)), one, one, one, one, one, None)

    assert project() == 1 and project(n=0) == 1 and project(k=-1) == 1
    assert project(batch=65536) == 7 and project(n=64 * 65535 + 1) == 7
    assert lib.dsa_rmsnorm(ctx.handle, None, None, one, None, None, None, one, None, None, None) == 1
    assert lib.dsa_project_on_tensor_cores(None, one, one) == 0


def test_new_entry_points_are_exported(lib):
    for name in ("dsa_rmsnorm", "dsa_quantize_rows", "dsa_quantize_weight", "dsa_project_fp8", "dsa_project_on_tensor_cores"):
        assert name in dsa.EXPORTED and hasattr(lib, name)


def test_views_that_negate_their_memory_are_refused(ctx):
    """The imaginary part of a conjugate: its memory holds the other sign."""
    c = torch.conj(torch.randn(4, 1, dtype=torch.complex64))
    x = c.imag
    assert x.is_neg() and x.dtype == F32
    for call in (lambda: ctx.rmsnorm(x, None), lambda: ctx.quantize_rows(x), lambda: ctx.quantize_weight(x),
                 lambda: ctx.rmsnorm(torch.zeros(4, 1), None, residual=x),
                 lambda: ctx.project_fp8(torch.zeros(4, 1, dtype=U8), x, torch.zeros(1, 1, dtype=U8), torch.zeros(1, 1))):
        with pytest.raises(ValueError, match="negates"):
            call()
    with pytest.raises(dsa.DSAError):       # written out it goes as far as the host-only context
        ctx.quantize_rows(x.resolve_neg())
