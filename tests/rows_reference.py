"""The 8-bit rows and projections written out plainly, in 64 bits on the host
(the quantisers in the 32-bit arithmetic that defines their codes), and the
error bounds that the tests hold the kernels to."""
from __future__ import annotations

import torch

GROUP = 128
EPS32 = 2.0 ** -24       # half a step of fp32, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: EPS32}


def groups(n: int) -> int:
    return -(-n // GROUP)


def e4m3_values(codes: torch.Tensor) -> torch.Tensor:
    """float64 values of uint8 codes."""
    return codes.cpu().view(torch.float8_e4m3fn).to(torch.float32).double()


def quantize(x: torch.Tensor, group_rows: int):
    """Codes (uint8) and scales of x (rows, width), fp32, finite: per group of
    group_rows x 128 scale = amax / 448 in fp32 (1 where that is zero), code = E4M3 of
    the fp32 quotient."""
    x = x.cpu().float()
    r, w = x.shape
    codes = torch.empty(r, w, dtype=torch.uint8)
    scales = torch.empty(-(-r // group_rows), groups(w), dtype=torch.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = (slice(i * group_rows, (i + 1) * group_rows), slice(j * GROUP, (j + 1) * GROUP))
            amax = x[at].abs().max()
            s = amax / torch.tensor(448.0)
            s = s if s > 0 else torch.tensor(1.0)
            scales[i, j] = s
            codes[at] = (x[at] / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scales


def rmsnorm(x, weight, eps, residual=None):
    """(y, h) in float64."""
    h = x.cpu().double()
    if residual is not None:
        h = h + residual.cpu().double()
    y = h / (h.square().mean(dim=1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * weight.cpu().double()
    return y, h


def norm_error(width: int) -> float:
    """Relative error of a normed value in fp32 before its last rounding: the
    sum of squares adds `width` positive terms, at most 32 of them one after
    another in a thread, then 5 + 32 steps over lanes and warps, each off by
    half a step (as is each square); the root halves what the sum is off; the
    addition of the residual, the mean, its sum with eps, the root, the
    division and two products add half a step each."""
    return (0.5 * (32 + 37 + 1) + 8) * EPS32


def check_codes(codes, scales, y, rel):
    """Codes and scales of float64 values y that the kernel knew to `rel`."""
    r, w = y.shape
    scales = scales.cpu().double()
    assert scales.shape == (r, groups(w))
    for j in range(groups(w)):
        sl = slice(j * GROUP, (j + 1) * GROUP)
        amax = y[:, sl].abs().amax(dim=1)
        want = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        # the quotient is one more rounding; a zero group is exactly 1
        assert ((scales[:, j] - want).abs() <= (rel + 2 * EPS32) * want).all(), j
        got = e4m3_values(codes[:, sl].contiguous()) * scales[:, j:j + 1]
        # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale where the
        # code is subnormal; the quotient and the scale are off by rel and two steps each
        bound = (2.0 ** -4) * y[:, sl].abs() + (2.0 ** -10) * want[:, None] + 4 * (rel + 2 * EPS32) * y[:, sl].abs()
        assert ((got - y[:, sl]).abs() <= bound).all(), j


def project(a, a_scale, w, w_scale):
    """float64 (out, sum of the products' magnitudes): a (rows, batch, k)
    codes, w (batch, n, k) codes; scales (rows, batch, kb) and (batch, nb, kb)."""
    m, b, k = a.shape
    n = w.shape[1]
    col = torch.arange(k) // GROUP
    av = e4m3_values(a) * a_scale.cpu().double()[:, :, col]
    wv = e4m3_values(w) * w_scale.cpu().double()[:, torch.arange(n) // GROUP][:, :, col]
    return torch.einsum("mbk,bnk->mbn", av, wv), torch.einsum("mbk,bnk->mbn", av.abs(), wv.abs())


def project_error(k: int) -> float:
    """Error of a product's sum relative to the sum of its terms' magnitudes:
    a block adds up to 128 exact products in fp32, each addition off by at most
    a whole step (2 half steps: the tensor core may cut rather than round);
    the blocks' sums take the scales' product (2 half steps) and are added one
    after another, in up to 16 runs whose sums are added last."""
    return (2 * 128 + 2 + groups(k) + 16) * EPS32


def check_project(out, want, mag, k):
    got = out.cpu().double()
    bound = project_error(k) * mag + HALF_STEP[out.dtype] * want.abs() * (1 + 2.0 ** -7)
    bad = (got - want).abs() > bound + HALF_STEP[out.dtype] * project_error(k) * mag
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() - bound).max()))
