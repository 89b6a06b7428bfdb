"""GPU: the codes of the 8-bit rows byte for byte where a value says nothing
about them: zeros of both signs.  The reference is the rule itself, scale = amax / 448 and code = E4M3(x / scale)
with fp32 divisions, and for bf16 the oracle's and the quantise-on-store kernels'."""
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
