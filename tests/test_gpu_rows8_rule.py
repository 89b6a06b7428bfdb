"""GPU: the codes of the 8-bit rows byte for byte where a value says nothing
about them: zeros of both signs, values far below their group's scale, and
groups that hold an infinity or a NaN.  The reference is the rule itself, scale
= amax / 448 and code = E4M3(x / scale) with fp32 divisions, and for bf16 the
oracle's and the quantise-on-store kernels'."""
import numpy as np
import pytest
import torch

import oracle
from deepseek_sparse_attention_dsa_gb300 import dsa
from deepseek_sparse_attention_dsa_gb300 import workloads as W
from tests import rows_reference as R
from tests.test_gpu_rows8 import placed, rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    from deepseek_sparse_attention_dsa_gb300 import build
    build.build()
    return dsa.Context(W.DSAShape(**W.DEEPSEEK), 0)


def same_bytes(got, want):
    codes, scales = got
    assert torch.equal(scales.cpu(), want[1])
    assert torch.equal(codes.cpu(), want[0]), int((codes.cpu() != want[0]).sum())


def with_zeros(rows, width):
    """Values with zeros of both signs among them, in groups of their own, and beside values of every size."""
    v = rand(rows + width, rows, width)
    v[:, 1::7] = -0.0
    v[:, 3::7] = 0.0
    v[0, :128] = -0.0          # a group of nothing else: its scale is 1
    v[1, ::2], v[1, 1::2] = -0.0, 0.0
    return v


# rows on 16 bytes, end to end and at a stride; rows off them; rows cut inside a piece of eight
LAYOUTS = [(8, 512, 512, 0), (8, 512, 640, 8), (8, 512, 515, 1), (8, 333, 333, 0)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,width,stride,offset", LAYOUTS)
def test_negative_zeros_keep_their_sign(ctx, dtype, rows, width, stride, offset):
    v = with_zeros(rows, width)
    x = placed(v, dtype, stride, offset)
    assert int((x.signbit() & (x == 0)).sum()) > rows
    want = R.quantize(x, 1)
    assert (want[0] == 0x80).any()
    same_bytes(ctx.quantize_rows(x), want)
    same_bytes(ctx.quantize_weight(x), R.quantize(x, 128))


def test_negative_zeros_beside_the_smallest_and_largest_values(ctx):
    """Scales on both sides of where the quotient becomes a division."""
    v = with_zeros(8, 512)
    for scale in (2.0 ** -100, 1.5 * 2.0 ** -81, 2.0 ** -73, 2.0 ** -70, 2.0 ** 100):
        x = (v * scale).cuda()
        same_bytes(ctx.quantize_rows(x), R.quantize(x, 1))


def test_the_norm_keeps_the_signs_of_zeros(ctx):
    """y = h * weight / root is a zero of the sign of h times the weight's."""
    for width in (512, 515):      # both norm kernels
        x = placed(with_zeros(8, width), BF16)
        w = (1 + 0.3 * rand(1, width)).to(BF16)
        w[::3] *= -1
        for residual in (None, placed(-torch.zeros(8, width), BF16)):     # -0 + -0 = -0, x + -0 = x
            codes = ctx.rmsnorm_quantize(x, w.cuda(), 1e-6, residual=residual)[0].cpu()
            zero = x.cpu() == 0
            negative = x.cpu().signbit() ^ w.signbit()
            assert torch.equal(codes[zero], torch.where(negative, 0x80, 0).to(torch.uint8)[zero])


def test_the_quantisers_agree_byte_for_byte(ctx):
    """quantize_rows, quantize_q and the oracle on the same bf16 rows."""
    heads, width = ctx.shape.index_heads, ctx.shape.index_dim
    x = placed(with_zeros(3 * heads, width), BF16)
    codes, scales = ctx.quantize_rows(x)
    plan = ctx.plan([W.Span(0, 0, 3, 0, np.zeros(1, np.int32))], 1)
    q_codes, q_scales = ctx.quantize_q(plan, x.view(3, heads, width))
    assert torch.equal(codes.view(-1), q_codes.view(torch.uint8).view(-1)) and torch.equal(scales.view(-1), q_scales.view(-1))
    o_codes, o_scales = oracle.quantize_rows(x.cpu(), width)
    assert np.array_equal(codes.cpu().numpy().reshape(-1), o_codes) and np.array_equal(scales.cpu().numpy().reshape(-1), o_scales)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,width,stride,offset", LAYOUTS)
def test_groups_that_are_not_finite_follow_the_rule(ctx, dtype, rows, width, stride, offset):
    """Over an infinite scale a finite value is a zero of its sign and an infinity NaN (0x7F); over NaN all is NaN."""
    v = with_zeros(rows, width)
    v[2, 5], v[3, 130], v[3, 131] = float("inf"), float("-inf"), float("inf")
    v[4, 200], v[5, 300] = float("nan"), -float("nan")
    v[6, 10], v[6, 20] = float("inf"), float("nan")
    x = placed(v, dtype, stride, offset)
    codes, scales = (t.cpu() for t in ctx.quantize_rows(x))
    x = x.cpu().float()
    for j in range(scales.shape[1]):
        at = slice(128 * j, 128 * j + 128)
        group = x[:, at]
        bad = ~group.isfinite().all(dim=1)
        amax = group.abs().amax(dim=1)      # (NaN where there is one)
        assert torch.equal(scales[bad, j].isnan(), amax[bad].isnan())
        assert (scales[bad, j][~amax[bad].isnan()] == float("inf")).all()
        q = group[bad] / scales[bad, j:j + 1]
        want = torch.where(q.isnan(), 0x7F, torch.where(q.signbit(), 0x80, 0)).to(torch.uint8)
        assert torch.equal(codes[bad, at], want), j
        good, want = ~bad, R.quantize(group[~bad], 1)
        assert torch.equal(codes[good, at], want[0]) and torch.equal(scales[good, j:j + 1], want[1])
    # a matrix's block of 128 x 128 holds all rows: every one of these blocks is spoilt by its own values
    w_codes, w_scales = (t.cpu() for t in ctx.quantize_weight(placed(v, dtype, stride, offset)))
    for j in range(w_scales.shape[1]):
        at = slice(128 * j, 128 * j + 128)
        block, s = x[:, at], w_scales[0, j]
        if block.isfinite().all():
            continue
        assert s.isnan() if block.isnan().any() else s == float("inf")
        q = block / s
        assert torch.equal(w_codes[:, at], torch.where(q.isnan(), 0x7F, torch.where(q.signbit(), 0x80, 0)).to(torch.uint8)), j


def test_values_far_below_their_scale(ctx):
    """Subnormal and tiny values beside large ones keep their signs as zeros."""
    v = torch.zeros(4, 128)
    v[:, 0] = torch.tensor([1.0, 448.0, 2.0 ** 127, 2.0 ** -60])
    tiny = torch.tensor([2.0 ** -149, 2.0 ** -127, 2.0 ** -126, 2.0 ** -103, 2.0 ** -102, 2.0 ** -101, 3 * 2.0 ** -73, 2.0 ** -72])
    v[:, 1:9], v[:, 9:17] = tiny, -tiny
    same_bytes(ctx.quantize_rows(v.cuda()), R.quantize(v, 1))


def test_an_infinite_norm_follows_the_rule(ctx):
    """The norm's codes where y overflows: the value NaN, its group's others zeros of their signs."""
    for width in (512, 515):
        x = placed(rand(3, 3, width), BF16)
        w = torch.ones(width)
        w[5], w[300] = 3e38, -3e38
        x[:, 5] = x[:, 300] = 16.0          # some 4 to 16 after the norm: beyond fp32 times these weights
        codes, scales = (t.cpu() for t in ctx.rmsnorm_quantize(x, w.to(BF16).cuda(), 1e-6))
        assert (scales[:, [0, 2]] == float("inf")).all() and scales[:, [1, 3]].isfinite().all()
        for group in (0, 2):
            at = slice(128 * group, 128 * group + 128)
            want = torch.where(x.cpu()[:, at].signbit(), 0x80, 0).to(torch.uint8)
            want[:, 5 if group == 0 else 300 - 256] = 0x7F
            assert torch.equal(codes[:, at], want)


@pytest.mark.parametrize("k", [2 ** 31 - 8, 2 ** 30 + 1032])
def test_long_rows_in_whole_pieces(ctx, k):
    """bf16 rows of whole 16-byte pieces whose bytes, or columns, come up to 32 bits: the packed kernels' offsets."""
    x = torch.zeros(1, k, dtype=BF16, device="cuda")
    at = torch.tensor([0, 127, 128, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 129, k - 8, k - 1], device="cuda")
    x[0, at] = torch.tensor([1.0, -2.0, 3.0, -4.0, 5.0, -6.0, 7.0, -3.5], dtype=BF16, device="cuda")
    for codes, scales in (ctx.quantize_rows(x), ctx.quantize_weight(x)):
        groups = torch.unique(at // 128)
        assert int((codes != 0).sum()) == len(at) and int((scales != 1).sum()) == len(groups)
        cols = (groups[:, None] * 128 + torch.arange(128, device="cuda")).clamp(max=k - 1)
        want = R.quantize(torch.where(groups[:, None] * 128 + torch.arange(128, device="cuda") < k, x[0, cols], 0), 1)
        assert torch.equal(scales[0, groups].cpu(), want[1][:, 0])
        inside = groups[:, None].cpu() * 128 + torch.arange(128) < k
        assert torch.equal(codes[0, cols].cpu()[inside], want[0][inside])
        del codes, scales
