"""GPU: appends of hundreds to thousands of rows, where a CTA takes several rows side by side and a thread several in
turn, against their definitions in 64 bits, slot by slot."""
import numpy as np
import pytest
import torch

from deepseek_sparse_attention_dsa_gb300 import dsa
from deepseek_sparse_attention_dsa_gb300 import workloads as W
from tests import rotary_reference as ref
from tests.rows_reference import e4m3_values, quantize

pytestmark = pytest.mark.gpu
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
YARN = dict(scaling="yarn", factor=40.0, original_context=4096, beta_fast=32.0, beta_slow=1.0)


@pytest.fixture(scope="module")
def contexts():
    from deepseek_sparse_attention_dsa_gb300 import build
    build.build()
    made = {}

    def get(**kw):
        key = tuple(sorted(kw.items()))
        if key not in made:
            made[key] = dsa.Context(W.DSAShape(**dict(W.DEEPSEEK, **kw)), 0)
        return made[key]
    return get


def rand(seed, *shape, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def spans_of(rows, page, start=37):
    """A decode row and two chunks of unlike lengths, their pages in no order and some of them nobody's."""
    lengths = [1, rows // 3, rows - 1 - rows // 3]
    contexts = [3 * page + 2, 0, 5 * page - 7]
    need = [-(-(start + c + n) // page) for c, n in zip(contexts, lengths)]
    pool = np.random.default_rng(rows).permutation(sum(need) + 3).astype(np.int32)
    spans, at, q = [], 0, 0
    for c, n, k in zip(contexts, lengths, need):
        spans.append(W.Span(0, q, n, c, pool[at:at + k], start))
        at += k
        q += n
    return spans, len(pool)


def turned(x, pos, freqs, offset, layout, amplitude=1.0):
    """(values in 64 bits, bound) of x (rows, heads, width) rotated."""
    y, mag = ref.rotate(x, torch.from_numpy(pos), freqs, offset, layout, amplitude=amplitude)
    return y, ref.rotate_bound(x, y, mag, offset, 2 * len(freqs), layout, amplitude)


# Rows for one, two, three and four rows a thread where 152 SMs take 5 of these rows side by side (32-bit sources: two at most).
@pytest.mark.parametrize("rows", [304, 3001, 4999, 8197, 12001])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (F32, BF16, F32), (F32, F32, F32)])
def test_latents_and_keys(contexts, rows, fp8, types):
    c = contexts(latent_fmt=W.LATENT_FP8_656 if fp8 else W.LATENT_BF16, index_fmt=W.INDEX_FP8_132 if fp8 else W.INDEX_BF16)
    layout, key_layout = ("interleaved", "half") if rows % 3 else ("half", "interleaved")
    spans, pages = spans_of(rows, 64)
    plan = c.plan(spans, pages)
    table = c.rotary_table(64, amplitude=1.1, **YARN)
    lat, k_pe, keys = (rand(i, rows, n, dtype=t) for i, n, t in zip((1, 2, 3), (512, 64, 128), types))
    where, pos = ref.slots(spans, 64)
    freqs = ref.frequencies(64, **YARN)
    pe, pe_bound = (t[:, 0] for t in turned(k_pe[:, None], pos, freqs, 0, layout, 1.1))
    ky, ky_bound = (t[:, 0] for t in turned(keys[:, None], pos, freqs, 64, key_layout, 1.1))
    others = np.setdiff1d(np.arange(pages * 64), where)
    args = dict(layout=layout, key_layout=key_layout, key_offset=64)
    if not fp8:
        lc = torch.full((pages, 64, 576), 9.0, dtype=BF16, device="cuda")
        ic = torch.full((pages, 64, 128), 9.0, dtype=BF16, device="cuda")
        c.append_latents(plan, table, lat.cuda(), k_pe.cuda(), lc, keys.cuda(), ic, **args)
        c.get_error()
        l, i = lc.view(-1, 576).cpu(), ic.view(-1, 128).cpu()
        assert torch.equal(l[where][:, :512], lat.to(BF16))
        ref.close(l[where][:, 512:], pe, pe_bound, BF16)
        ref.close(i[where], ky, ky_bound, BF16)
        assert bool((l[others] == 9.0).all()) and bool((i[others] == 9.0).all())
        return
    lc = torch.full((pages, 64, 656), 77, dtype=U8, device="cuda")
    ic = torch.full((pages, 64 * 132), 77, dtype=U8, device="cuda")
    c.append_latents(plan, table, lat.cuda(), k_pe.cuda(), lc, keys.cuda(), ic, **args)
    c.get_error()
    l = lc.view(-1, 656).cpu()
    codes = ic[:, :64 * 128].reshape(-1, 128).cpu()
    scales = ic[:, 64 * 128:].contiguous().view(F32).view(-1).cpu()
    assert bool((l[others] == 77).all()) and bool((codes[others] == 77).all())
    assert bool((scales.view(I32)[others] == 0x4D4D4D4D).all())
    want, want_scale = quantize(lat, 1)
    assert torch.equal(l[where][:, :512], want)
    assert torch.equal(l[where][:, 512:528].contiguous().view(F32), want_scale)
    ref.close(l[where][:, 528:].contiguous().view(BF16), pe, pe_bound, BF16)
    # a rotated key is known to its bound, so its group's scale is too, and a code to half a step beside that
    got_scale = scales[where].double()
    amax, slack = ky.abs().amax(1), ky_bound.amax(1)
    assert ((got_scale * 448 - amax).abs() <= slack + 2 * ref.EPS32 * amax).all()
    got = e4m3_values(codes[where].contiguous()) * got_scale[:, None]
    bound = 2.0 ** -4 * ky.abs() + 2.0 ** -10 * got_scale[:, None] + 2 * ky_bound + 4 * ref.EPS32 * amax[:, None]
    assert ((got - ky).abs() <= bound).all()


@pytest.mark.parametrize("rows", [304, 1501, 8197])
@pytest.mark.parametrize("heads,dim,rot,with_keys", [(1, 128, 128, False), (4, 128, 64, False), (8, 128, 128, True), (4, 64, 32, True), (3, 96, 32, True)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_keys_and_values(contexts, rows, heads, dim, rot, with_keys, dtype):
    c = contexts()
    layout = "half" if rows % 2 else "interleaved"
    offset = dim - rot
    spans, pages = spans_of(rows, 64)
    plan = c.plan(spans, pages)
    table = c.rotary_table(rot, base=500000.0)
    both, keys = rand(4, rows, 2, heads, dim, dtype=dtype), rand(5, rows, 128, dtype=F32 if dtype == BF16 else BF16)
    k, v = both[:, 0], both[:, 1]
    msa = W.MSAShape(kv_heads=heads, q_heads=heads, head_dim=dim)
    kv = torch.full((pages, 64, 2 * heads * dim), 9.0, dtype=BF16, device="cuda")
    ic = torch.full((pages, 64, 128), 9.0, dtype=BF16, device="cuda")
    on = both.cuda()
    c.append_kv(plan, msa, table, on[:, 0], on[:, 1], kv, *((keys.cuda(), ic) if with_keys else ()), layout=layout, offset=offset)
    c.get_error()
    where, pos = ref.slots(spans, 64)
    freqs = ref.frequencies(rot, 500000.0)
    want, bound = turned(k, pos, freqs, offset, layout)
    got = kv.view(-1, 2, heads, dim).cpu()
    ref.close(got[where][:, 0], want, bound, BF16)
    assert torch.equal(got[where][:, 1], v.to(BF16))
    others = np.setdiff1d(np.arange(pages * 64), where)
    assert bool((got[others] == 9.0).all())
    i = ic.view(-1, 128).cpu()
    if with_keys:
        want, bound = turned(keys[:, None], pos, freqs, 0, "half")
        ref.close(i[where], want[:, 0], bound[:, 0], BF16)
        i = i[others]
    assert bool((i == 9.0).all())


@pytest.mark.parametrize("live", [4111, 5000, 1, 0])
@pytest.mark.parametrize("fp8", [False, True])
def test_padding_among_the_rows_of_a_thread(contexts, live, fp8):
    """A capturable plan of 5000 rows: those behind `live` hold NaN and are not written; the others as a host plan's."""
    c = contexts(latent_fmt=W.LATENT_FP8_656 if fp8 else W.LATENT_BF16, index_fmt=W.INDEX_FP8_132 if fp8 else W.INDEX_BF16)
    msa, table = W.MSAShape(), c.rotary_table(64)
    lengths = [n for n in (live // 2, live - live // 2) if n]
    pages = np.random.default_rng(1).permutation(100).astype(np.int32)
    spans, dev, q = [], [], 0
    for i, n in enumerate(lengths):
        spans.append(W.Span(0, q, n, 3, pages[50 * i:50 * i + 50]))
        dev.append([n, 3, 0, 50 * i, 50, 0])
        q += n
    cap = c.plan_capturable(5000, 2, 5000 * 3000, 100)
    on = dict(device="cuda", dtype=I32)
    c.plan_update(cap, torch.tensor([len(lengths)], **on), torch.tensor(dev + [[0] * 6] * (2 - len(dev)), **on), torch.from_numpy(pages).cuda())
    lat, k_pe, keys, k, v = (rand(i, 5000, *n).cuda() for i, n in enumerate([(512,), (64,), (128,), (4, 128), (4, 128)]))
    for t in (lat, k_pe, keys, k, v):
        t[live:] = float("nan")

    def caches():
        wide = torch.full((100, 64, 1024), 7.0, dtype=BF16, device="cuda")
        if fp8:
            return torch.full((100, 64, 656), 7, dtype=U8, device="cuda"), torch.full((100, 64 * 132), 7, dtype=U8, device="cuda"), wide
        return torch.full((100, 64, 576), 7.0, dtype=BF16, device="cuda"), torch.full((100, 64, 128), 7.0, dtype=BF16, device="cuda"), wide

    got, want = caches(), caches()
    c.append_latents(cap, table, lat, k_pe, got[0], keys, got[1])
    c.append_kv(cap, msa, table, k, v, got[2])
    c.get_error()
    # the host plan's rows, a hundred at a time: one row a thread
    for s in spans:
        for r in range(0, s.q_len, 100):
            n = min(100, s.q_len - r)
            rows = slice(s.q_start + r, s.q_start + r + n)
            plan = c.plan([W.Span(0, 0, n, s.ctx_start + r, s.pages)], 100)
            c.append_latents(plan, table, lat[rows], k_pe[rows], want[0], keys[rows], want[1])
            c.append_kv(plan, msa, table, k[rows], v[rows], want[2])
    c.get_error()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [12, 4999])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift", [0, 1])
def test_codes_of_any_values(contexts, rows, dtype, shift):
    """NaN, infinities, zeros of both signs, values at both ends of the type's range: the codes and scales of the 8-bit rows,
    to the byte, on 16 bytes and off them."""
    c = contexts(latent_fmt=W.LATENT_FP8_656, index_fmt=W.INDEX_FP8_132)
    spans, pages = spans_of(rows, 64)
    plan = c.plan(spans, pages)
    x = torch.randn(rows, 512 + 128, generator=torch.Generator().manual_seed(6))
    special = [float("nan"), float("inf"), -float("inf"), -0.0, 0.0, 1e-38, -3e-41, 3e38, 1e-45, 448.0]
    for i, v in enumerate(special):
        x[i::12, 17 + 50 * i] = v                  # one such value in a group
    x[10::12] = torch.where(x[10::12] > 0, 1e-30, -0.0)
    x[11::12, :300] *= 1e-39
    x[9::12, 128:256], x[9::12, 512:] = -0.0, 0.0
    x = x.to(dtype)
    lat, keys = (torch.empty(rows * n + shift, dtype=dtype, device="cuda")[shift:].view(rows, n) for n in (512, 128))
    lat.copy_(x[:, :512])
    keys.copy_(x[:, 512:])
    k_pe = torch.zeros(rows, 64, dtype=dtype, device="cuda")
    lc = torch.full((pages, 64, 656), 77, dtype=U8, device="cuda")
    ic = torch.full((pages, 64 * 132), 77, dtype=U8, device="cuda")
    c.append_latents(plan, None, lat, k_pe, lc, keys, ic)
    c.get_error()
    where = torch.from_numpy(ref.slots(spans, 64)[0]).cuda()
    l = lc.view(-1, 656)[where]
    codes, scales = c.quantize_rows(lat.clone())
    assert torch.equal(l[:, :512], codes) and bool((l[:, 528:] == 0).all())
    torch.testing.assert_close(l[:, 512:528].contiguous().view(F32), scales, rtol=0, atol=0, equal_nan=True)
    codes, scales = c.quantize_rows(keys.clone())
    assert torch.equal(ic[:, :64 * 128].reshape(-1, 128)[where], codes)
    torch.testing.assert_close(ic[:, 64 * 128:].contiguous().view(F32).view(-1)[where], scales[:, 0], rtol=0, atol=0, equal_nan=True)
