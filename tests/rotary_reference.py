"""Rotary positions, appends and the attention over a shared prefix written out
plainly in 64 bits on the host, and the error bounds that the tests hold the
kernels to."""
from __future__ import annotations

import math

import numpy as np
import torch

EPS32 = 2.0 ** -24                                            # half a step of fp32, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: EPS32}


def frequencies(rot, base=10000.0, scaling=None, factor=1.0, original_context=4096, beta_fast=32.0, beta_slow=1.0):
    """Radians a position of pairs 0 .. rot / 2 - 1, one at a time."""
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            def pair(turns):
                return rot * math.log(original_context / (2 * math.pi * turns)) / (2 * math.log(base))
            low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot - 1)
            r = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            f = f * (1 - r) + f / factor * r
        out.append(f)
    return out


def rotate(x, positions, freqs, offset=0, layout="interleaved", inverse=False, amplitude=1.0):
    """(float64 result, magnitude of each value's terms) of x (rows, heads, width), pair by pair."""
    y = x.cpu().double().clone()
    mag = y.abs()
    rot = 2 * len(freqs)
    p = positions.cpu().double()
    for i, f in enumerate(freqs):
        a, b = (offset + 2 * i, offset + 2 * i + 1) if layout == "interleaved" else (offset + i, offset + i + rot // 2)
        t = p * f * (-1 if inverse else 1)
        c, s = (amplitude * torch.cos(t))[:, None], (amplitude * torch.sin(t))[:, None]
        u, v = x[..., a].cpu().double(), x[..., b].cpu().double()
        y[..., a], y[..., b] = u * c - v * s, u * s + v * c
        mag[..., a], mag[..., b] = (u * c).abs() + (v * s).abs(), (u * s).abs() + (v * c).abs()
    return y, mag


def rotated_error() -> float:
    """Error of a rotated value in fp32 before its last rounding, relative to its
    terms' magnitudes, in half steps.  Sine and cosine of the rounded angle by
    their sums: the sine's last coefficient is off by 0.5, its last addition and
    the product with x by 1 each, the sum before them (0.1 of the value, 2.5)
    by 0.3: 2.8 in all; the cosine's last addition by 1, and x x and the sum before it
    (at most 0.44 of the value) by 1 and 1.5: 2.1 in all.  The angle, off by half a
    step of at most pi, moves them by pi half steps of 1, which is not relative
    to a small sine or cosine (see rotate_bound).  The amplitude (itself
    rounded), its product, the term's product and the sum add half a step each."""
    return (3 + 1 + 1 + 1 + 1) * EPS32


def rotate_bound(x, y, mag, offset, rot, layout, amplitude=1.0):
    """Elementwise bound of the rotated columns' error before the output's rounding; 0 for the copied ones."""
    bound = torch.zeros_like(y)
    half = rot // 2
    for i in range(half):
        a, b = (offset + 2 * i, offset + 2 * i + 1) if layout == "interleaved" else (offset + i, offset + i + half)
        size = x[..., a].cpu().double().abs() + x[..., b].cpu().double().abs()
        turn = abs(amplitude) * math.pi * (EPS32 + 2.0 ** -40) * size       # the angle's own error (table: 2^-40 and less)
        for k in (a, b):
            bound[..., k] = rotated_error() * mag[..., k] + turn
    return bound


def close(got, want, bound, dtype):
    """Whether got is `want` known to `bound` and rounded once to dtype."""
    got, half = got.cpu().double(), HALF_STEP[dtype]
    off = (got - want).abs()
    allowed = bound + half * (want.abs() + bound) + torch.finfo(dtype).tiny
    bad = off > allowed
    assert not bad.any(), (int(bad.sum()), float((off - allowed).max()))


def slots(spans, page_size):
    """(physical cache row, position) of every row of the plan, as int64 arrays."""
    where, pos = [], []
    for s in spans:
        for r in range(s.q_len):
            p = s.ctx_start + r
            slot = getattr(s, "page_start", 0) + p
            where.append(int(s.pages[slot // page_size]) * page_size + slot % page_size)
            pos.append(p)
    return np.asarray(where, np.int64), np.asarray(pos, np.int64)


def prefix_attend(spans, page_size, q, kv_cache, kv_heads, scale):
    """float64 (out, sum of the weights times |v|, log2 of the span of each row's
    logits) of dense causal GQA: q (T, q_heads, dim), cache (pages, page_size, 2 * kv_heads * dim)."""
    q = q.cpu().double()
    T, Hq, D = q.shape
    cache = kv_cache.cpu().view(-1, 2, kv_heads, D)
    out, mag, top = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(T, Hq, dtype=torch.float64)
    group = Hq // kv_heads
    for s in spans:
        start = getattr(s, "page_start", 0)
        for r in range(s.q_len):
            slot = start + np.arange(s.ctx_start + r + 1)
            rows = torch.from_numpy(np.asarray(s.pages, np.int64)[slot // page_size] * page_size + slot % page_size)
            k, v = cache[rows, 0].double(), cache[rows, 1].double()       # (keys, kv_heads, D)
            for h in range(Hq):
                logits = (k[:, h // group] @ q[s.q_start + r, h]) * scale
                size = (k[:, h // group].abs() @ q[s.q_start + r, h].abs()) * abs(scale)
                w = torch.softmax(logits, 0)
                out[s.q_start + r, h] = w @ v[:, h // group]
                mag[s.q_start + r, h] = w @ v[:, h // group].abs()
                top[s.q_start + r, h] = size.max()
    return out, mag, top


def attend_error(dim: int, keys: int, top, tensor_cores: bool):
    """Error of an output relative to sum(w |v|).  A logit (natural units) is a sum
    of `dim` products, each addition off by at most a whole step of the terms' sum
    `top` (2 half steps: the tensor core may cut), then scaled, in log2 units, minus
    the reference maximum (3 half steps of 2 * top); an absolute error e of the
    logits moves a weight by e^e - 1 relative to it, and so does the sum of the
    weights: twice in all.  The exponential is off by 2^-22, twice.  Weights rounded
    to bf16 on the tensor cores are off by 2^-8 in what they add to the values, not
    in their own sum.  The sums over the keys add at most a whole step for each of
    their terms one after another (128 in a tile, then the tiles), and the parts'
    joining a few more."""
    logit = (2 * dim + 8) * EPS32 * top
    sums = (2 * 128 + 2 * (keys / 128 + 1) + 64) * EPS32 if tensor_cores else (2 * (keys / 8 + 1) + 64) * EPS32
    return 2 * torch.expm1(logit) + 4 * 2.0 ** -22 + 2 * sums + (2.0 ** -8 if tensor_cores else 0.0)


def check_attend(got, ref, dim, keys, tensor_cores):
    out, mag, top = ref
    got = got.cpu().double()
    bound = attend_error(dim, keys, top, tensor_cores)[..., None] * mag
    off = (got - out).abs()
    allowed = bound + 2.0 ** -8 * (out.abs() + bound)
    assert not (off > allowed).any(), (int((off > allowed).sum()), float((off / allowed.clamp_min(1e-30)).max()))
