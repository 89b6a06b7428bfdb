"""Rotary tables, rotations, appends and prefix plans on the host (no GPU): the
binding's checks, the statuses of the C entry points, which prefixes are found,
and which are refused."""
import ctypes

import numpy as np
import pytest
import torch

from deepseek_sparse_attention_dsa_gb300 import build as dsa_build
from deepseek_sparse_attention_dsa_gb300 import dsa
from deepseek_sparse_attention_dsa_gb300 import workloads as W

BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def span(q_start, q_len, ctx_start, pages, page_start=0):
    return W.Span(0, q_start, q_len, ctx_start, np.asarray(pages, np.int32), page_start)


@pytest.fixture(scope="module")
def ctx():
    dsa_build.build()
    return dsa.Context(W.DSAShape(**W.DEEPSEEK), device=-1)   # its tensors are the host's


@pytest.fixture()
def plan(ctx):
    return ctx.plan([span(0, 1, 5, [0]), span(1, 3, 62, [1, 2])], 3)


def status(call):
    with pytest.raises(dsa.DSAError) as e:
        call()
    return e.value.status


@pytest.mark.parametrize("bad", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=1026), dict(base=1.0), dict(base=float("inf")),
                                 dict(scaling="linear", factor=0.0), dict(scaling="yarn", factor=-1.0), dict(amplitude=float("nan")),
                                 dict(scaling="yarn", original_context=0), dict(scaling="yarn", beta_fast=0.5), dict(scaling="yarn", beta_slow=0.0),
                                 dict(rot_dim=4, frequencies=[1.0, float("inf")])])
def test_tables_refuse(ctx, bad):
    args = dict(dict(rot_dim=64), **bad)
    assert status(lambda: ctx.rotary_table(**args)) == 1


def test_tables_refuse_amplitudes_beyond_fp32(ctx):
    """They are applied in fp32: one that is infinite there would make every value so."""
    for bad in (3.5e38, -1e39, 1.7e308):
        assert status(lambda: ctx.rotary_table(64, amplitude=bad)) == 1
    for good in (3.4e38, -3.4e38, 0.0, 1e-60):
        ctx.rotary_table(64, amplitude=good).close()


def test_tables_check_their_arguments(ctx):
    with pytest.raises(ValueError):
        ctx.rotary_table(64, scaling="cubic")
    with pytest.raises(ValueError):
        ctx.rotary_table(64, frequencies=[1.0] * 31)
    with pytest.raises(ValueError):
        ctx.rotary_table(4, frequencies=[1.0, 2.0], scaling="yarn")
    t = ctx.rotary_table(4, frequencies=[-7.5, 100.0])      # turns back, and more than one a position
    t.close()
    t.close()


def test_rotary_checks_its_tensors(ctx, plan):
    t = ctx.rotary_table(64)
    x, p = torch.zeros(4, 2, 64, dtype=BF16), torch.zeros(4, dtype=I32)
    for bad in (dict(x=x.half()), dict(x=x.to(torch.float64)), dict(positions=p.long()), dict(positions=p.float()), dict(out=x.float())):
        a = dict(dict(x=x, positions=p), **bad)
        with pytest.raises(TypeError):
            ctx.rotary(t, a["x"], a["positions"], out=a.get("out"))
    for bad in (dict(x=x[0, 0]), dict(x=x[None]), dict(positions=p[:3]), dict(out=x[:, :1]), dict(x=torch.zeros(4, 2, 128, dtype=BF16)[..., ::2])):
        a = dict(dict(x=x, positions=p), **bad)
        with pytest.raises(ValueError):
            ctx.rotary(t, a["x"], a["positions"], out=a.get("out"))
    with pytest.raises(ValueError):
        ctx.rotary(t, x, p, layout="neox")
    with pytest.raises(TypeError):
        ctx.rotary(None, x, p)
    t.close()
    assert status(lambda: ctx.rotary(t, x, p)) == 1


def test_rotate_statuses(ctx, plan):
    """Before the host-only context is looked at: all are 1, but none may be taken for a call."""
    lib, t = dsa.load(), ctx.rotary_table(64)
    one = ctypes.c_void_p(16)
    base = dict(rows=4, heads=2, width=64, offset=0, layout=0, inverse=0, type=0, x_stride=128, x_head=64, out_stride=128, out_head=64)

    def call(p=None, pos=one, **kw):
        return lib.dsa_rotate(ctx.handle, p, t.handle, ctypes.byref(dsa._Rotate(**dict(base, **kw))), one, pos, one, None)

    for bad in (dict(rows=-1), dict(heads=0), dict(width=0), dict(offset=-1), dict(offset=1), dict(width=63), dict(layout=2), dict(inverse=2),
                dict(type=2), dict(x_stride=-1), dict(out_head=-1), dict(p=plan.handle), dict(pos=None), dict(p=plan.handle, pos=None, rows=5)):
        assert call(**bad) == 1, bad
    assert lib.dsa_rotate(ctx.handle, None, None, ctypes.byref(dsa._Rotate(**base)), one, one, one, None) == 1
    assert lib.dsa_rotate(ctx.handle, None, t.handle, None, one, one, one, None) == 1


def test_appends_check_their_tensors(ctx, plan):
    t = ctx.rotary_table(64)
    c, k_pe, keys = torch.zeros(4, 512, dtype=BF16), torch.zeros(4, 64, dtype=BF16), torch.zeros(4, 128, dtype=BF16)
    lat, idx = torch.zeros(3, 64, 576, dtype=BF16), torch.zeros(3, 64, 128, dtype=BF16)
    good = dict(c=c, k_pe=k_pe, latent_cache=lat, keys=keys, index_cache=idx)

    def call(table=t, **kw):
        return ctx.append_latents(plan, table, **dict(good, **kw))

    for bad in (dict(c=c.half()), dict(latent_cache=lat.view(U8)), dict(index_cache=idx.float()), dict(k_pe=None), dict(keys=None), dict(c=[0])):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(c=c[:3]), dict(c=c[:, :511]), dict(k_pe=k_pe[:, :63]), dict(keys=keys[:, :64]), dict(latent_cache=lat[:2]),
                dict(index_cache=idx[:, :63]), dict(latent_cache=torch.zeros(3, 64, 1152, dtype=BF16)[..., ::2])):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError):
        call(layout="both")
    assert status(call) == 1                                           # host-only
    assert status(lambda: call(table=ctx.rotary_table(32))) == 1       # not rope_dim
    assert status(lambda: call(key_offset=65)) == 1
    k, kv = torch.zeros(4, 4, 128, dtype=BF16), torch.zeros(3, 64, 1024, dtype=BF16)
    msa = W.MSAShape()
    with pytest.raises(ValueError):
        ctx.append_kv(plan, msa, t, k, k[:, :3], kv)
    with pytest.raises(TypeError):
        ctx.append_kv(plan, msa, t, k, k.float(), kv)
    with pytest.raises(ValueError):
        ctx.append_kv(plan, msa, t, k, k, kv[:2])
    assert status(lambda: ctx.append_kv(plan, msa, t, k, k, kv, offset=65)) == 1
    plan.close()
    assert status(lambda: ctx.append_kv(plan, msa, t, k, k, kv)) == 1


def shared_spans(lengths, shared_pages, q_len=1, page_start=0, groups=1):
    """Spans of `lengths` own tokens (new ones among them) behind shared_pages pages, a group after another."""
    out, q, at = [], 0, groups * shared_pages
    for i, n in enumerate(lengths):
        g = i * groups // len(lengths)
        own = -(-n // 64)
        out.append(span(q, q_len, shared_pages * 64 - page_start + n - q_len, list(range(g * shared_pages, (g + 1) * shared_pages)) +
                        list(range(at, at + own)), page_start))
        q += q_len
        at += own
    return out, at


def read(ctx, spans, pages, prefixes=None):
    plan = ctx.plan(spans, pages)
    pp = ctx.plan_prefix(plan, W.MSAShape(), prefixes)
    return pp.info.num_prefixes, pp.info.tokens_read


def test_prefixes_are_found(ctx):
    spans, pages = shared_spans([10, 70, 1, 64], 4)
    assert read(ctx, spans, pages) == (1, 256 + 145)
    assert read(ctx, spans, pages, []) == (0, 4 * 256 + 145)
    assert read(ctx, spans, pages, [(1, 2, 100)]) == (1, 4 * 256 + 145 - 100)
    spans, pages = shared_spans([10, 70, 1, 64, 9, 3], 4, groups=3)
    assert read(ctx, spans, pages) == (3, 3 * 256 + 157)
    spans, pages = shared_spans([40, 50], 4, page_start=37)
    assert read(ctx, spans, pages) == (1, 219 + 90)
    spans[1].page_start = 36                                  # the same pages, other slots
    assert read(ctx, spans, pages)[0] == 0
    spans, pages = shared_spans([10, 20, 30], 1)              # shorter than a tile
    assert read(ctx, spans, pages) == (0, 3 * 64 + 60)
    # a run ends where a shorter common part would save less
    a, b = list(range(100)), list(range(2)) + list(range(100, 110))
    spans = [span(0, 1, 6399, a), span(1, 1, 6398, a), span(2, 1, 200, b)]
    assert read(ctx, spans, 120) == (1, 6400 + 6399 + 201 - 6398)
    # the new rows of a step are never shared, whatever the pages say
    spans = [span(0, 8, 200, [0, 1, 2, 3]), span(8, 8, 150, [0, 1, 2, 3])]
    assert read(ctx, spans, 4) == (1, 208 + 158 - 150)
    assert read(ctx, [], 4) == (0, 0)


def test_prefixes_that_do_not_hold_are_refused(ctx):
    spans, pages = shared_spans([10, 70, 1, 64], 4)
    plan = ctx.plan(spans, pages)
    msa = W.MSAShape()
    for bad in ([(0, 2, 257)], [(0, 5, 64)], [(-1, 2, 64)], [(0, 0, 64)], [(0, 2, -1)], [(0, 2, 64), (1, 2, 64)], [(2, 2, 64), (0, 2, 64)]):
        assert status(lambda: ctx.plan_prefix(plan, msa, bad)) == 1, bad
    assert ctx.plan_prefix(plan, msa, [(0, 2, 256), (2, 2, 1)]).info.num_prefixes == 2
    assert ctx.plan_prefix(plan, msa, [(0, 4, 0)]).info.num_prefixes == 0
    for bad, st in ((dict(q_heads=63), 1), (dict(kv_heads=0), 1), (dict(q_heads=2048, kv_heads=4), 7), (dict(head_dim=513), 7)):
        assert status(lambda: ctx.plan_prefix(plan, W.MSAShape(**bad))) == st, bad
    lib = dsa.load()
    h = ctypes.c_void_p()
    ms = dsa._msa_shape(msa)
    assert lib.dsa_prefix_plan(ctx.handle, plan.handle, ctypes.byref(ms), None, 1, None, ctypes.byref(h)) == 1
    assert lib.dsa_prefix_plan(ctx.handle, plan.handle, ctypes.byref(ms), None, -2, None, ctypes.byref(h)) == 1
    assert lib.dsa_prefix_plan(ctx.handle, plan.handle, None, None, 0, None, ctypes.byref(h)) == 1
    assert lib.dsa_prefix_plan(ctx.handle, plan.handle, ctypes.byref(ms), None, 0, None, None) == 1
    x = (dsa._Prefix * 1)(dsa._Prefix(0, 2, 64, 1))
    assert lib.dsa_prefix_plan(ctx.handle, plan.handle, ctypes.byref(ms), x, 1, None, ctypes.byref(h)) == 1


def test_numbers_that_do_not_fit_are_refused(ctx):
    """Not taken modulo 2^32."""
    spans, pages = shared_spans([10, 70, 1, 64], 4)
    plan = ctx.plan(spans, pages)
    for bad in (2 ** 32 + 64, 2 ** 63 + 64, -2 ** 32 + 64):
        assert status(lambda: ctx.rotary_table(bad)) == 1, bad
        for prefix in ((bad, 2, 64), (0, bad, 64), (0, 2, bad)):
            assert status(lambda: ctx.plan_prefix(plan, W.MSAShape(), [prefix])) == 1, prefix
        for field in ("q_heads", "kv_heads", "head_dim"):
            assert status(lambda: ctx.plan_prefix(plan, W.MSAShape(**{field: bad}))) in (1, 7), field


def test_prefix_attend_checks_its_tensors(ctx):
    spans, pages = shared_spans([10, 70], 4)
    plan = ctx.plan(spans, pages)
    pp = ctx.plan_prefix(plan, W.MSAShape())
    q, kv = torch.zeros(2, 64, 128, dtype=BF16), torch.zeros(pages, 64, 1024, dtype=BF16)
    for bad in ((q.float(), kv), (q.half(), kv), (q, kv.float())):
        with pytest.raises(TypeError):
            ctx.prefix_attend(pp, *bad)
    for bad in ((q[:1], kv), (q[:, :63], kv), (q, kv[1:]), (torch.zeros(2, 64, 256, dtype=BF16)[..., ::2], kv),
                (torch.zeros(64, 2, 128, dtype=BF16).transpose(0, 1), kv)):
        with pytest.raises(ValueError):
            ctx.prefix_attend(pp, *bad)
    with pytest.raises(ValueError):
        ctx.prefix_attend(pp, q, kv, out=torch.zeros(64, 2, 128, dtype=BF16).transpose(0, 1))
    assert status(lambda: ctx.prefix_attend(pp, q, kv)) == 1           # host-only
    plan.close()
    assert status(lambda: ctx.prefix_attend(pp, q, kv)) == 1
    pp.close()
    assert status(lambda: ctx.prefix_attend(pp, q, kv)) == 1
