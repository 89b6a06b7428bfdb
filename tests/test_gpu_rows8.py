"""GPU: the 8-bit rows (rmsnorm with residual, quantize_rows, quantize_weight)
against their definitions in 64 bits: odd and ragged widths, strided and
unaligned rows, every type, rows that are zero or not finite, padding rows of a
capturable plan, graph capture, and the calls they refuse."""
import numpy as np
import pytest
import torch

from deepseek_sparse_attention_dsa_gb300 import dsa
from deepseek_sparse_attention_dsa_gb300 import workloads as W
from tests import rows_reference as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    from deepseek_sparse_attention_dsa_gb300 import build
    build.build()
    return dsa.Context(W.DSAShape(**W.DEEPSEEK), 0)


def rand(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g) * std


def placed(values, dtype, stride=None, offset=0):
    """The values on the GPU as rows at a stride, `offset` elements into their storage."""
    r, w = values.shape
    stride = w if stride is None else stride
    store = torch.full((offset + r * stride,), 7.0, dtype=dtype, device="cuda")
    out = store[offset:].view(r, stride)[:, :w]
    out.copy_(values)
    return out


WIDTHS = [1, 7, 64, 127, 128, 129, 255, 512, 520, 576, 1000, 1024, 1032, 2048, 2056, 4096, 5120, 8191, 8192, 16384, 32768]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_widths(ctx, width, residual):
    rows = 3
    x = placed(rand(width, rows, width), BF16)
    w = (1 + 0.3 * rand(width + 1, width)).to(BF16).cuda()
    res = placed(rand(width + 2, rows, width, std=3.0), BF16) if residual else None
    y, h = R.rmsnorm(x, w, 1e-6, res)
    rel = R.norm_error(width)
    got = ctx.rmsnorm(x, w, 1e-6, residual=res)
    out = got[0] if residual else got
    assert out.dtype == BF16 and ((out.cpu().double() - y).abs() <= (2.0 ** -8 + 2 * rel) * y.abs()).all()
    got = ctx.rmsnorm_quantize(x, w, 1e-6, residual=res)
    R.check_codes(got[0], got[1], y, rel)
    if residual:   # h is a sum of two bf16 values, rounded to fp32 and to bf16
        assert ((got[2].cpu().double() - h).abs() <= (2.0 ** -8 + 2 * R.EPS32) * h.abs()).all()


@pytest.mark.parametrize("x_type", [BF16, F32])
@pytest.mark.parametrize("residual_type", [BF16, F32])
@pytest.mark.parametrize("weight_type", [BF16, F32, None])
@pytest.mark.parametrize("out_type", [BF16, F32])
def test_rmsnorm_types_strides_and_both_outputs(ctx, x_type, residual_type, weight_type, out_type):
    rows, width = 5, 704
    x = placed(rand(1, rows, width), x_type, stride=760, offset=8)
    res = placed(rand(2, rows, width), residual_type, stride=711, offset=1)   # odd: no row but the first on 16 bytes
    w = None if weight_type is None else (1 + 0.3 * rand(3, width)).to(weight_type).cuda()
    y, h = R.rmsnorm(x, w, 1e-5, res)
    rel = R.norm_error(width)
    store = torch.full((rows, 800), -5.0, dtype=out_type, device="cuda")
    out = store[:, 3:3 + width]
    cstore = torch.full((rows, 731), 99, dtype=torch.uint8, device="cuda")
    codes = cstore[:, 1:1 + width]
    sstore = torch.full((rows, 9), -3.0, device="cuda")
    c, s, ro = ctx.rmsnorm_quantize(x, w, 1e-5, residual=res, out=out, codes=codes, scales=sstore[:, :6])
    assert c is codes and ro.dtype == residual_type
    R.check_codes(codes, s, y, rel)
    assert ((out.cpu().double() - y).abs() <= (R.HALF_STEP[out_type] + 2 * rel) * y.abs()).all()
    assert ((ro.cpu().double() - h).abs() <= (R.HALF_STEP[residual_type] + 2 * R.EPS32) * h.abs()).all()
    # nothing beside the rows was written
    assert (store[:, :3] == -5).all() and (store[:, 3 + width:] == -5).all()
    assert (cstore[:, :1] == 99).all() and (cstore[:, 1 + width:] == 99).all() and (sstore[:, 6:] == -3).all()


def test_rmsnorm_in_place(ctx):
    """residual_out over residual, and out over x, as a decode step keeps its buffers."""
    x0, r0 = rand(4, 6, 2056).to(BF16), rand(5, 6, 2056).to(BF16)
    w = (1 + 0.3 * rand(6, 2056)).to(BF16).cuda()
    want, want_r = ctx.rmsnorm(x0.cuda(), w, residual=r0.cuda())
    x, r = x0.cuda(), r0.cuda()
    out, ro = ctx.rmsnorm(x, w, residual=r, residual_out=r, out=x)
    assert out is x and ro is r and torch.equal(x, want) and torch.equal(r, want_r)


def test_rmsnorm_many_rows_and_zero_rows(ctx):
    for rows, width in ((0, 512), (1, 512), (2113, 136), (1031, 1280)):
        x = placed(rand(rows + 7, rows, width), BF16)
        if rows > 10:
            x[5] = 0   # mean 0: only eps is under the root, every value 0, every scale 1
        y, _ = R.rmsnorm(x, None, 1e-6)
        codes, scales = ctx.rmsnorm_quantize(x, None, 1e-6)
        assert ctx.last_launch_count() == (1 if rows else 0)
        if rows:
            R.check_codes(codes, scales, y, R.norm_error(width))
        if rows > 10:
            assert (codes[5] == 0).all() and (scales[5] == 1).all()
    ctx.get_error()


def test_rows_that_are_not_finite_stay_where_they_are(ctx):
    """A NaN or an infinity spoils its own row (norm) or group (quantiser) visibly, and no other."""
    x = rand(8, 4, 640)
    clean = x.clone()
    x[1, 130] = float("nan")
    x[2, 400] = float("-inf")
    out = ctx.rmsnorm(placed(x, BF16), None).cpu()
    ref = ctx.rmsnorm(placed(clean, BF16), None).cpu()
    assert torch.equal(out[0], ref[0]) and torch.equal(out[3], ref[3])
    assert out[1].isnan().all() and out[2, 400].isnan() and (out[2, :400] == 0).all()
    for t in (BF16, F32):
        codes, scales = ctx.quantize_rows(placed(x, t))
        cc, cs = ctx.quantize_rows(placed(clean, t))
        back = R.e4m3_values(codes) * scales.cpu().double().repeat_interleave(128, 1)
        spoilt = torch.zeros(4, 640, dtype=torch.bool)
        spoilt[1, 128:256] = spoilt[2, 384:512] = True
        assert not back[spoilt].isfinite().any()
        assert torch.equal(codes.cpu()[~spoilt], cc.cpu()[~spoilt]) and back[~spoilt].isfinite().all()


def _exact(codes, scales, ref):
    assert torch.equal(scales.cpu(), ref[1])
    assert torch.equal(codes.cpu(), ref[0]), int((codes.cpu() != ref[0]).sum())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,width,stride,offset", [
    (1, 1, 1, 0), (1, 128, 128, 0), (3, 127, 127, 0), (5, 129, 131, 1), (7, 576, 704, 0), (2, 1024, 1024, 8),
    (9, 1000, 1000, 0), (2, 2056, 2060, 4), (257, 128, 128, 0), (33, 512, 512, 0), (4, 4224, 4224, 3)])
def test_quantize_rows_is_exact(ctx, dtype, rows, width, stride, offset):
    v = rand(rows * 31 + width, rows, width) * torch.exp(rand(9, rows, 1))
    if rows > 2:
        v[2] = 0
    v[0, ::5] *= 1e-4      # codes that are subnormal or zero
    x = placed(v, dtype, stride, offset)
    _exact(*ctx.quantize_rows(x), R.quantize(x, 1))


def test_quantize_rows_boundaries(ctx):
    """Quotients on and beside every rounding border of e4m3, and the smallest and largest scales."""
    every = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()   # 0 .. 448
    mid = (every[1:] + every[:-1]) / 2
    near = torch.cat([every, mid, mid * (1 + 2.0 ** -22), mid * (1 - 2.0 ** -22), -mid])
    near = torch.cat([near, torch.full((-len(near) % 127,), 0.5)]).view(-1, 127)
    v = torch.cat([torch.full((near.shape[0], 1), 448.0), near], 1)   # each group's maximum is 448: the scale is 1
    for scale in (1.0, 3.0, 1 + 2.0 ** -23, 2 - 2.0 ** -23, 2.0 ** -60, 1.7 * 2.0 ** -79, 1.3 * 2.0 ** -81, 2.0 ** -126 / 448,
                  2.0 ** 118 * 1.9):
        x = (v * scale).cuda()
        _exact(*ctx.quantize_rows(x), R.quantize(x, 1))
    # every bf16 mantissa under every bf16 maximum, where quotients on a border are common
    m = torch.arange(128, 256).float()
    v = torch.cat([(m / 256).expand(128, 128) * torch.cat([m.new_full((64,), -1.0), m.new_full((64,), 1.0)]), m[:, None].expand(128, 128) / 128], 1)
    for shift in (0, 3, -20):
        x = (v * torch.where(torch.arange(256) % 128 == 7, 1.0, 2.0 ** (shift % 5))).contiguous()
        x[:, 5] = x[:, 128 + 5] = m / 16
        _exact(*ctx.quantize_rows(x.to(BF16).cuda()), R.quantize(x.to(BF16), 1))
    # a maximum whose 448th part is below fp32's range: the group counts as zero
    x = torch.zeros(2, 128)
    x[0, 3], x[1, 7] = 2.0 ** -142, -(2.0 ** -149)
    codes, scales = ctx.quantize_rows(x.cuda())
    assert (scales == 1).all() and ((codes & 127) == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (129, 127), (64, 576), (300, 1000), (704, 520), (3, 200, 136)])
def test_quantize_weight_is_exact(ctx, dtype, shape):
    v = rand(sum(shape), *shape)
    if shape[-1] > 128:
        v[..., :128, :128] = 0
    w = v.to(dtype).cuda()
    codes, scales = ctx.quantize_weight(w)
    for b in range(shape[0] if len(shape) == 3 else 1):
        at = (b,) if len(shape) == 3 else ()
        _exact(codes[at] if at else codes, scales[at] if at else scales, R.quantize(w[at] if at else w, 128))


def test_quantize_weight_strided(ctx):
    big = rand(11, 2, 200, 300).to(BF16).cuda()
    w = big[:, 3:190, 5:260]
    codes = torch.full((2, 190, 280), 99, dtype=torch.uint8, device="cuda")
    c, s = ctx.quantize_weight(w, codes=codes[:, 1:188, 3:258])
    for b in range(2):
        _exact(c[b], s[b], R.quantize(w[b], 128))
    codes[:, 1:188, 3:258] = 99
    assert (codes == 99).all()


def capturable(ctx, live, cap=8):
    """A capturable plan of `cap` rows whose update holds `live` single-row spans."""
    plan = ctx.plan_capturable(cap, cap, 64 * cap, 64)
    set_rows(ctx, plan, live, cap)
    return plan


def set_rows(ctx, plan, live, cap=8):
    sp = np.zeros((cap, 6), np.int32)
    for i in range(live):
        sp[i] = [1, i, 0, i, 1, 0]
    plan._n = torch.tensor([live], dtype=torch.int32, device="cuda")
    plan._spans = torch.from_numpy(sp).cuda()
    plan._pages = torch.arange(cap, dtype=torch.int32, device="cuda")
    ctx.plan_update(plan, plan._n, plan._spans, plan._pages)


def test_padding_rows_of_a_capturable_plan_are_left(ctx):
    for live in (0, 3, 8):
        plan = capturable(ctx, live)
        for m in (1, 4):   # rows for each of the plan's
            rows, width = 8 * m, 640
            x = placed(rand(12, rows, width), BF16)
            x[live * m:] = float("nan")
            res = placed(rand(13, rows, width), BF16)
            fresh = lambda *s, t: torch.full(s, 77, dtype=t, device="cuda")   # noqa: E731
            codes, scales, ro, out = (fresh(rows, width, t=torch.uint8), fresh(rows, 5, t=F32),
                                      fresh(rows, width, t=BF16), fresh(rows, width, t=BF16))
            ctx.rmsnorm_quantize(x, None, residual=res, residual_out=ro, out=out, codes=codes, scales=scales, plan=plan)
            full = ctx.rmsnorm_quantize(x, None, residual=res)
            for got, want in ((codes, full[0]), (scales, full[1]), (ro, full[2])):
                assert torch.equal(got[:live * m], want[:live * m]) and (got[live * m:] == 77).all()
            assert (out[live * m:] == 77).all()
            codes, scales = fresh(rows, width, t=torch.uint8), fresh(rows, 5, t=F32)
            ctx.quantize_rows(x, codes, scales, plan=plan)
            full = ctx.quantize_rows(x)
            assert torch.equal(codes[:live * m], full[0][:live * m]) and (codes[live * m:] == 77).all()
            assert torch.equal(scales[:live * m], full[1][:live * m]) and (scales[live * m:] == 77).all()
            wide = fresh(rows, 650, t=torch.uint8)   # rows that are not dense
            ctx.quantize_rows(x, wide[:, :width], plan=plan)
            assert torch.equal(wide[:live * m, :width], full[0][:live * m]) and (wide[live * m:] == 77).all()
    ctx.get_error()


def test_captured_and_replayed_on_new_data(ctx):
    x = placed(rand(14, 6, 1280), BF16)
    w = (1 + 0.3 * rand(15, 1280)).to(BF16).cuda()
    res = placed(rand(16, 6, 1280), BF16)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ctx.rmsnorm_quantize(x, w, residual=res)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = ctx.rmsnorm_quantize(x, w, residual=res)
        q = ctx.quantize_rows(got[2])
        wq = ctx.quantize_weight(got[2])
    for seed in (17, 18):
        x.copy_(rand(seed, 6, 1280))
        g.replay()
        torch.cuda.synchronize()
        want = ctx.rmsnorm_quantize(x, w, residual=res)
        for a, b in zip(list(got) + list(q) + list(wq),
                        list(want) + list(ctx.quantize_rows(want[2])) + list(ctx.quantize_weight(want[2]))):
            assert torch.equal(a, b)


def test_new_outputs_belong_to_the_stream_of_the_call(ctx):
    """Memory that the current stream has given back but still has work on is not
    handed to a call on another stream."""
    x = placed(rand(22, 64, 4096), BF16)
    want = [t.clone() for t in ctx.quantize_rows(x)]
    a = torch.zeros(64, 4096, dtype=torch.uint8, device="cuda")
    asc, w, wsc = torch.ones(64, 32, device="cuda"), torch.zeros(4096, 4096, dtype=torch.uint8, device="cuda"), torch.ones(32, 32, device="cuda")
    side = torch.cuda.Stream()
    for given in (side, side.cuda_stream):
        for call, like in ((lambda: ctx.quantize_rows(x, stream=given)[0], torch.uint8),
                           (lambda: ctx.project_fp8(a, asc, w, wsc, stream=given), BF16),
                           (lambda: ctx.rmsnorm(x, None, stream=given), BF16)):
            for _ in range(2):
                torch.cuda.synchronize()
                torch.cuda.empty_cache()
                held = torch.empty(64, 4096, dtype=like, device="cuda")
                at = held.data_ptr()
                torch.cuda._sleep(20_000_000)      # some 10 ms on the current stream
                held.fill_(7)
                del held
                out = call()
                assert out.data_ptr() != at
                side.synchronize()
                kept = out.clone()
                torch.cuda.synchronize()
                assert torch.equal(out, kept)
                if like == torch.uint8:
                    assert torch.equal(out, want[0])


def test_refused_calls_leave_the_context_usable(ctx):
    x = placed(rand(19, 4, 256), BF16)
    plan3 = ctx.plan([W.Span(0, 0, 3, 0, np.zeros(1, np.int32))], 1)

    def status(fn):
        with pytest.raises(dsa.DSAError) as e:
            fn()
        return e.value.status

    assert status(lambda: ctx.rmsnorm(x, None, eps=-1.0)) == 1
    assert status(lambda: ctx.rmsnorm(x, None, eps=float("nan"))) == 1
    assert status(lambda: ctx.rmsnorm(placed(rand(20, 1, 32769), BF16), None)) == 7
    assert status(lambda: ctx.rmsnorm(x, None, plan=plan3)) == 1          # 4 rows, a plan of 3
    assert status(lambda: ctx.quantize_rows(x, plan=plan3)) == 1
    other = dsa.Context(W.DSAShape(**W.DEEPSEEK), 0)
    assert status(lambda: other.quantize_rows(x[:3], plan=plan3)) == 1    # another context's plan
    # rows that would be written over one another
    flat = torch.empty(600, dtype=torch.uint8, device="cuda")
    assert status(lambda: ctx.quantize_rows(x, codes=flat.as_strided((4, 256), (100, 1)))) == 1
    assert status(lambda: ctx.rmsnorm(x, None, out=torch.empty(256, dtype=BF16, device="cuda").expand(4, 256))) == 1
    _exact(*ctx.quantize_rows(x[:3], plan=plan3), R.quantize(x[:3], 1))
    ctx.get_error()


def test_norm_at_the_ends_of_the_sum_of_squares(ctx):
    """Beyond fp32's range the sum gives zeros; an all-zero row gives zeros with an eps and NaN without."""
    x = torch.zeros(3, 640, dtype=BF16, device="cuda")
    x[1] = 1e20
    x[2] = 1.0
    for dt in (BF16, F32):
        out = ctx.rmsnorm(x.to(dt), None, eps=1e-6, out_dtype=F32)
        assert (out[:2] == 0).all() and ((out[2] - 1).abs() < 1e-6).all()
        out = ctx.rmsnorm(x.to(dt), None, eps=0.0, out_dtype=F32)
        assert out[0].isnan().all() and (out[1] == 0).all() and (out[2] == 1).all()
