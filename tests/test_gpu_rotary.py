"""GPU: rotations and appends against their definitions in 64 bits."""
import math
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

from deepseek_sparse_attention_dsa_gb300 import dsa
from deepseek_sparse_attention_dsa_gb300 import workloads as W
from tests import rotary_reference as ref

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


@pytest.fixture(scope="module")
def ctx(contexts):
    return contexts()


def rand(seed, *shape, dtype=BF16, stride=None, shift=0):
    """Values on the GPU; rows `stride` elements apart, the first `shift` elements into its memory."""
    x = torch.randn(*shape, generator=torch.Generator().manual_seed(seed))
    if stride is None and shift == 0:
        return x.to(dtype).cuda()
    inner = 1
    for n in shape[1:]:
        inner *= n
    stride = stride or inner
    store = torch.zeros(shift + shape[0] * stride, dtype=dtype, device="cuda")
    view = store.as_strided(shape, (stride,) + torch.empty(shape).stride()[1:], shift)
    view.copy_(x)
    return view


def positions(*values):
    return torch.tensor(values, dtype=I32, device="cuda")


FAR = (0, 1, 131071, 1000003, 2147483647, -5, -2147483648)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,width,offset,rot,stride,shift", [
    (128, 64, 0, 64, 128 * 192, 0),    # a view of wider heads is below; rows far apart
    (1, 128, 0, 64, None, 0),          # one head: the columns behind are copied
    (3, 128, 64, 64, None, 0),         # the last columns
    (5, 200, 8, 96, None, 0),          # columns before and behind
    (2, 99, 33, 64, None, 0),          # off 16 bytes
    (7, 64, 0, 64, 64 * 7 + 8, 1),     # first value off 16 bytes
    (64, 2, 0, 2, None, 0),            # one pair
    (3, 70, 1, 68, 221, 3),            # half of 34 pairs: cut pieces
    (1, 1024, 0, 1024, None, 0),       # the widest table
    (2, 2100, 20, 1000, None, 0),      # more pieces a head than threads
])
def test_rotary(ctx, layout, dtype, heads, width, offset, rot, stride, shift):
    table = ctx.rotary_table(rot)
    x = rand(1, len(FAR), heads, width, dtype=dtype, stride=stride, shift=shift)
    pos = positions(*FAR)
    freqs = ref.frequencies(rot)
    for inverse in (False, True):
        got = ctx.rotary(table, x, pos, offset=offset, layout=layout, inverse=inverse)
        assert got.is_contiguous() and got.dtype == dtype
        want, mag = ref.rotate(x, pos, freqs, offset, layout, inverse)
        # the definition's own angle, position * frequency in 64 bits, is off by 2^-53 of it
        slack = 2.0 ** -53 * 2.0 ** 32
        bound = ref.rotate_bound(x, want, mag, offset, rot, layout) + slack * 4 * x.cpu().double().abs().amax()
        ref.close(got, want, bound, dtype)
        kept = torch.ones(width, dtype=torch.bool)
        kept[offset:offset + rot] = False
        assert torch.equal(got[..., kept], x[..., kept])
    ctx.get_error()


@pytest.mark.parametrize("rows,heads,rot", [(1, 1, 2), (1, 128, 64), (1, 300, 64), (1031, 1, 64), (513, 3, 32), (4, 7, 16), (3000, 2, 2), (70, 64, 128)])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotary_sizes(ctx, rows, heads, rot, layout):
    """Every row and head where a CTA's items cross rows."""
    table = ctx.rotary_table(rot, base=500000.0, scaling="linear", factor=8.0, amplitude=1.3)
    x = rand(2, rows, heads, rot, dtype=F32)
    pos = torch.randint(0, 200000, (rows,), generator=torch.Generator().manual_seed(3), dtype=I32).cuda()
    got = ctx.rotary(table, x, pos, layout=layout)
    want, mag = ref.rotate(x, pos, ref.frequencies(rot, 500000.0, "linear", 8.0), 0, layout, amplitude=1.3)
    ref.close(got, want, ref.rotate_bound(x, want, mag, 0, rot, layout, 1.3), F32)


@pytest.mark.parametrize("form", [dict(), dict(scaling="linear", factor=4.0), YARN, dict(base=1.5, scaling="yarn", factor=3.0, original_context=64),
                                  dict(scaling="yarn", factor=2.0, original_context=1e9, beta_fast=1.0, beta_slow=1.0)])
@pytest.mark.parametrize("rot", [2, 64, 128])
def test_frequencies(ctx, form, rot):
    """Each form's frequencies, seen through unit pairs at far positions; the same as given ones."""
    freqs = ref.frequencies(rot, **form)
    x = torch.zeros(3, 1, rot, device="cuda")
    x[..., 0::2] = 1.0
    pos = positions(1, 4097, 1048576)
    got = ctx.rotary(ctx.rotary_table(rot, **form), x, pos)
    given = ctx.rotary(ctx.rotary_table(rot, frequencies=freqs), x, pos)
    want, mag = ref.rotate(x, pos, freqs)
    # the two computations of a frequency may differ in its last bits of 64: 2^-50 of 2^20 positions
    bound = ref.rotate_bound(x, want, mag, 0, rot, "interleaved") + 2.0 ** -50 * 2.0 ** 20 * 1.0
    ref.close(got, want, bound, F32)
    ref.close(given, want, bound, F32)


def test_frequencies_beyond_a_turn(ctx):
    freqs = [-7.5, 100.0, 0.0, 6.283185307179586]
    x = rand(5, 4, 2, 8, dtype=F32)
    pos = positions(0, 3, 1001, -17)
    got = ctx.rotary(ctx.rotary_table(8, frequencies=freqs), x, pos)
    want, mag = ref.rotate(x, pos, freqs)
    ref.close(got, want, ref.rotate_bound(x, want, mag, 0, 8, "interleaved") + 2.0 ** -52 * 1001 * 100 * 4, F32)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_angles_hold_at_any_position(ctx, layout):
    """The fraction of a turn of position x frequency, the frequency as the double it is, in 60 digits."""
    freqs = [100.0, 0.9, 730000.5, -12345.678, 1.0, 1e9 + 0.1, 2.5e-7, -0.1, 3.3e11, 6.283185307179586, 1e-19, 0.75, 5e-324, -1e-300, 41.5, 0.3]
    far = FAR + (2147483646, 1073741789, -1999999973)
    x = rand(15, len(far), 3, 32, dtype=F32)
    got = ctx.rotary(ctx.rotary_table(32, frequencies=freqs), x, positions(*far), layout=layout)
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    want, mag = x.cpu().double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    with localcontext() as digits:
        digits.prec = 80
        for r, p in enumerate(far):
            for i, f in enumerate(freqs):
                turns = p * Decimal(f) / two_pi
                t = 2 * math.pi * float(turns - turns.to_integral_value())
                a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + 16)
                u, v, c, s = x[r, :, a].cpu().double(), x[r, :, b].cpu().double(), math.cos(t), math.sin(t)
                want[r, :, a], want[r, :, b] = u * c - v * s, u * s + v * c
                mag[r, :, a], mag[r, :, b] = (u * c).abs() + (v * s).abs(), (u * s).abs() + (v * c).abs()
    # a table is off by 2^-65 of a turn a position, half a unit (and 2^-106 of the turns, here below 2^36)
    bound = ref.rotate_bound(x, want, mag, 0, 32, layout) + 2 * math.pi * 2.0 ** -34 * 2 * x.cpu().double().abs().amax()
    ref.close(got, want, bound, F32)


def test_small_angles_keep_their_sine(ctx):
    """x e1 turned by 1e-9: the second value is that, to a few steps, not to a part of a turn."""
    x = torch.zeros(1, 1, 2, device="cuda")
    x[..., 0] = 1.0
    got = ctx.rotary(ctx.rotary_table(2, frequencies=[1e-9]), x, positions(1))
    assert abs(float(got[0, 0, 1]) / 1e-9 - 1) < 1e-6


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rotary_in_place_and_inverse(ctx, layout, dtype):
    """In place the columns beside are not touched; turning back gives the values, and is the gradient."""
    table = ctx.rotary_table(64)
    store = rand(6, 9, 4, 192, dtype=dtype)
    x, before = store[..., 128:], store.clone()
    pos = torch.arange(100000, 100009, dtype=I32, device="cuda")
    want = ctx.rotary(table, x, pos, layout=layout)
    got = ctx.rotary(table, x, pos, layout=layout, out=x)
    assert got is x and torch.equal(x, want) and torch.equal(store[..., :128], before[..., :128])
    back = ctx.rotary(table, x, pos, layout=layout, inverse=True, out=x)
    first, mag = ref.rotate(want, pos, ref.frequencies(64), 0, layout, inverse=True)
    ref.close(back, first, ref.rotate_bound(want, first, mag, 0, 64, layout), dtype)
    if dtype == F32:
        # the gradient of sum(w * rotate(x)) by differences is rotate^T w = the inverse of w
        w = rand(7, 9, 4, 64, dtype=F32)
        grad = ctx.rotary(table, w, pos, layout=layout, inverse=True)
        e = rand(8, 9, 4, 64, dtype=F32)
        plus, minus = (ctx.rotary(table, want + s * e, pos, layout=layout) for s in (1.0, -1.0))   # linear: any step will do
        d = ((plus.double() - minus.double()) / 2 * w.double()).sum()
        size = float((e.double().abs() * 2 * w.double().abs()).sum() + (want.double().abs() * 2 * w.double().abs()).sum())
        assert abs(float(d - (grad.double() * e.double()).sum())) <= 16 * ref.EPS32 * size


def test_rotary_rows_of_a_plan(ctx):
    spans = [W.Span(0, 0, 3, 70, np.array([1, 0]), 5), W.Span(1, 3, 1, 8191, np.arange(129), 0), W.Span(2, 4, 2, 0, np.array([2]), 0)]
    plan = ctx.plan(spans, 129)
    table = ctx.rotary_table(64, **YARN)
    x = rand(9, 6, 12, 192)[..., 128:]
    want = ctx.rotary(table, x, positions(70, 71, 72, 8191, 0, 1))
    assert torch.equal(ctx.rotary(table, x, plan), want)
    # a capturable plan's padding is neither read nor written
    cap = ctx.plan_capturable(9, 4, 20000, 129)
    pages = torch.from_numpy(np.concatenate([s.pages for s in spans]).astype(np.int32)).cuda()
    dev, off = [], 0
    for s in spans:
        dev.append([s.q_len, s.ctx_start, s.page_start, off, len(s.pages), 0])
        off += len(s.pages)
    ctx.plan_update(cap, positions(3), torch.tensor(dev + [[0] * 6], dtype=I32, device="cuda"), pages)
    padded = torch.full((9, 12, 64), float("nan"), dtype=BF16, device="cuda")
    padded[:6] = x
    out = torch.full((9, 12, 64), 7.0, dtype=BF16, device="cuda")
    assert ctx.rotary(table, padded, cap, out=out) is out
    assert torch.equal(out[:6], want) and bool((out[6:] == 7.0).all())
    ctx.get_error()


def test_a_table_is_there_when_its_call_returns(ctx):
    """Used at once on a stream that waits for nothing, table after table in the memory of the last one."""
    x, pos, side = rand(16, 1, 1, 1024, dtype=F32), positions(1), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for i in range(50):
        table = ctx.rotary_table(1024, frequencies=[0.01 * (i + 1)] * 512)
        got.append(ctx.rotary(table, x, pos, stream=side))
        side.synchronize()
        table.close()
    for i, y in enumerate(got):
        want, mag = ref.rotate(x, pos, [0.01 * (i + 1)] * 512)
        ref.close(y, want, ref.rotate_bound(x, want, mag, 0, 1024, "interleaved"), F32)


@pytest.mark.parametrize("width,offset,rot", [(2 ** 31 - 1, 0, 2), (2 ** 31 - 1, 2 ** 31 - 3, 2), (2 ** 31 - 1, 2 ** 31 - 1 - 64, 64), (2 ** 31 - 8, 0, 64)])
def test_the_widest_row(ctx, width, offset, rot):
    """Counts of its pieces stay below 2^31."""
    table, pos = ctx.rotary_table(rot), positions(1000)
    x = torch.empty(1, width, dtype=BF16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(17))
    got = ctx.rotary(table, x, pos, offset=offset)
    ctx.get_error()
    end = offset + rot
    assert torch.equal(got[:, :offset], x[:, :offset]) and torch.equal(got[:, end:], x[:, end:])
    assert torch.equal(got[:, offset:end], ctx.rotary(table, x[:, offset:end].clone(), pos))


def test_rotary_refuses(ctx):
    table = ctx.rotary_table(64)
    x = rand(1, 4, 2, 64)
    pos = positions(0, 1, 2, 3)
    wide = torch.zeros(4, 2, 128, dtype=BF16, device="cuda")
    plan = ctx.plan([W.Span(0, 0, 3, 0, np.zeros(1, np.int32))], 1)
    for bad in (lambda: ctx.rotary(table, x, pos, offset=1), lambda: ctx.rotary(table, x, pos, offset=-1),
                lambda: ctx.rotary(table, x[..., :32], pos), lambda: ctx.rotary(table, x, plan),
                lambda: ctx.rotary(table, x, pos, offset=2 ** 40),
                lambda: ctx.rotary(table, x, pos, out=x[:, :1].expand(4, 2, 64)), lambda: ctx.rotary(table, x[:, :1].expand(4, 2, 64), pos, out=x[:, :1].expand(4, 2, 64))):
        with pytest.raises(dsa.DSAError) as e:
            bad()
        assert e.value.status == 1
    assert ctx.rotary(table, x[:0], pos[:0]).shape == (0, 2, 64)
    got = ctx.rotary(table, x[:, :1].expand(4, 2, 64), pos)     # an input may repeat
    assert torch.equal(got[:, 0], got[:, 1])
    assert torch.equal(ctx.rotary(table, x, pos, out=wide[..., 64:]), ctx.rotary(table, x, pos)) and bool((wide[..., :64] == 0).all())
    with pytest.raises(ValueError):
        ctx.rotary(table, x, pos.cpu())
    ctx.get_error()


def test_nothing_spreads_beyond_its_pair(ctx):
    table = ctx.rotary_table(64)
    x = rand(3, 2, 2, 64, dtype=F32)
    want = ctx.rotary(table, x, positions(3, 9))
    x[0, 1, 10] = float("nan")
    x[1, 0, 3] = float("inf")
    got = ctx.rotary(table, x, positions(3, 9))
    hit = torch.zeros(2, 2, 64, dtype=torch.bool, device="cuda")
    hit[0, 1, 10:12] = hit[1, 0, 2:4] = True
    assert torch.equal(got[~hit], want[~hit]) and not torch.isfinite(got[hit]).any()


# ---------------------------------------------------------------- appends
def spans_for(P, start=0):
    """A decode row, a chunk that crosses pages, one that begins a request: pages in no order."""
    a = W.Span(0, 0, 1, 3 * P - start - 1, np.array([7, 3, 9], np.int32), start)
    b = W.Span(1, 1, P + 3, P - 2, np.array([1, 8, 0, 5], np.int32), start)
    c = W.Span(2, P + 4, 2, 0, np.array([2], np.int32) if start + 2 <= P else np.array([2, 6], np.int32), start)
    return [a, b, c], 11


def key_offsets(layout):
    return 64 if layout == "half" else 33


@pytest.mark.parametrize("page,start", [(64, 0), (64, 63), (16, 5), (7, 3)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout,key_layout,aligned", [("interleaved", "half", True), ("half", "interleaved", False)])
def test_append_latents(contexts, page, start, fp8, dtype, layout, key_layout, aligned):
    c = contexts(page_size=page, latent_fmt=W.LATENT_FP8_656 if fp8 else W.LATENT_BF16, index_fmt=W.INDEX_FP8_132 if fp8 else W.INDEX_BF16)
    spans, pages = spans_for(page, start)
    plan = c.plan(spans, pages)
    T = plan.num_rows
    table = c.rotary_table(64, amplitude=1.1, **YARN)
    shift = 0 if aligned else 1
    lat = rand(1, T, 512, dtype=dtype, stride=None if aligned else 515, shift=shift)
    k_pe = rand(2, T, 64, dtype=dtype, stride=None if aligned else 67, shift=shift)
    keys = rand(3, T, 128, dtype=dtype, stride=None if aligned else 131, shift=shift)
    offset = 0 if aligned else key_offsets(key_layout)
    where, pos = ref.slots(spans, page)
    pt = torch.from_numpy(pos).to(torch.int32)
    pe, pe_mag = ref.rotate(k_pe[:, None], pt, ref.frequencies(64, **YARN), 0, layout, amplitude=1.1)
    pe_bound = ref.rotate_bound(k_pe[:, None], pe, pe_mag, 0, 64, layout, 1.1)[:, 0]
    ky, ky_mag = ref.rotate(keys[:, None], pt, ref.frequencies(64, **YARN), offset, key_layout, amplitude=1.1)
    ky_bound = ref.rotate_bound(keys[:, None], ky, ky_mag, offset, 64, key_layout, 1.1)[:, 0]
    pe, ky = pe[:, 0], ky[:, 0]
    others = np.setdiff1d(np.arange(pages * page), where)
    if not fp8:
        lc = torch.full((pages, page, 576), 9.0, dtype=BF16, device="cuda")
        ic = torch.full((pages, page, 128), 9.0, dtype=BF16, device="cuda")
        c.append_latents(plan, table, lat, k_pe, lc, keys, ic, layout=layout, key_layout=key_layout, key_offset=offset)
        assert c.last_launch_count() == 1
        c.get_error()
        l, i = lc.view(-1, 576).cpu(), ic.view(-1, 128).cpu()
        assert torch.equal(l[where][:, :512], lat.cpu().to(BF16))
        ref.close(l[where][:, 512:], pe, pe_bound, BF16)
        ref.close(i[where], ky, ky_bound, BF16)
        assert bool((l[others] == 9.0).all()) and bool((i[others] == 9.0).all())
        # one at a time: the same rows
        l2, i2 = torch.full_like(lc, 9.0), torch.full_like(ic, 9.0)
        c.append_latents(plan, table, lat, k_pe, l2, layout=layout)
        c.append_latents(plan, table, keys=keys, index_cache=i2, key_layout=key_layout, key_offset=offset)
        assert torch.equal(l2, lc) and torch.equal(i2, ic)
        return
    lc = torch.full((pages, page, 656), 77, dtype=U8, device="cuda")
    ic = torch.full((pages, page * 132), 77, dtype=U8, device="cuda")
    c.append_latents(plan, table, lat, k_pe, lc, keys, ic, layout=layout, key_layout=key_layout, key_offset=offset)
    c.get_error()
    l = lc.view(-1, 656).cpu()
    codes = ic[:, :page * 128].reshape(-1, 128).cpu()
    scales = ic[:, page * 128:].contiguous().view(F32).view(-1).cpu()
    assert bool((l[others] == 77).all()) and bool((codes[others] == 77).all()) and bool((scales.view(torch.int32)[others] == 0x4D4D4D4D).all())
    from tests.rows_reference import check_codes, e4m3_values, quantize
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


@pytest.mark.parametrize("lora,rope,dim,rot", [(512, 0, 128, 64), (256, 16, 64, 16), (136, 8, 128, 8), (64, 32, 64, 32), (512, 64, 128, 64)])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("turned", [True, False])
def test_append_widths(contexts, lora, rope, dim, rot, aligned, turned):
    """Other widths of the caches' rows, down to no rope at all (the table is the key's alone then)."""
    c = contexts(kv_lora_rank=lora, rope_dim=rope, index_dim=dim)
    spans, pages = spans_for(64, 3)
    plan = c.plan(spans, pages)
    T = plan.num_rows
    table = c.rotary_table(rot) if turned else None
    stride = (lambda n: None) if aligned else (lambda n: n + 3)
    lat, keys = rand(1, T, lora, stride=stride(lora)), rand(3, T, dim, stride=stride(dim))
    k_pe = rand(2, T, rope, stride=stride(rope)) if rope else None
    where, pos = ref.slots(spans, 64)
    lc = torch.full((pages, 64, lora + rope), 9.0, dtype=BF16, device="cuda")
    ic = torch.full((pages, 64, dim), 9.0, dtype=BF16, device="cuda")
    c.append_latents(plan, table, lat, k_pe, lc, keys, ic, layout="half", key_layout="interleaved", key_offset=dim - rot)
    c.get_error()
    l, i = lc.view(-1, lora + rope).cpu(), ic.view(-1, dim).cpu()
    others = np.setdiff1d(np.arange(pages * 64), where)
    assert torch.equal(l[where][:, :lora], lat.cpu()) and bool((l[others] == 9.0).all()) and bool((i[others] == 9.0).all())
    pt, freqs = torch.from_numpy(pos).to(torch.int32), ref.frequencies(rot)
    for x, got, offset, layout in ((k_pe, l[where][:, lora:], 0, "half"), (keys, i[where], dim - rot, "interleaved")):
        if x is None:
            continue
        if not turned:
            assert torch.equal(got, x.cpu())
            continue
        y, mag = ref.rotate(x[:, None], pt, freqs, offset, layout)
        ref.close(got, y[:, 0], ref.rotate_bound(x[:, None], y, mag, offset, rot, layout)[:, 0], BF16)


@pytest.mark.parametrize("lora,rot,rows", [(128, 1024, 1672), (256, 1024, 4999), (128, 512, 3344), (128, 1024, 70), (136, 1024, 4999)])
def test_append_without_a_rope_ignores_a_wide_table(contexts, lora, rot, rows):
    """Nothing of such a latent turns: a table of any width leaves it as it is, however many rows there are."""
    c = contexts(kv_lora_rank=lora, rope_dim=0)
    pages = rows // 64 + 2
    order = np.random.default_rng(rows).permutation(pages).astype(np.int32)
    plan = c.plan([W.Span(0, 0, rows, 5, order)], pages)
    lat = rand(1, rows, lora)
    lc = torch.full((pages, 64, lora), 9.0, dtype=BF16, device="cuda")
    c.append_latents(plan, c.rotary_table(rot), lat, None, lc)
    c.get_error()
    slot = np.arange(5, 5 + rows)
    where = order[slot // 64].astype(np.int64) * 64 + slot % 64
    want = torch.full((pages * 64, lora), 9.0, dtype=BF16)
    want[where] = lat.cpu()
    assert torch.equal(lc.view(-1, lora).cpu(), want)


@pytest.mark.parametrize("page", [64, 16])
def test_append_without_a_table_is_the_store(contexts, page):
    """Unrotated bf16 rows: byte for byte what the stores write."""
    c = contexts(page_size=page, latent_fmt=W.LATENT_FP8_656, index_fmt=W.INDEX_FP8_132)
    spans, pages = spans_for(page, 5)
    plan = c.plan(spans, pages)
    lat, keys = rand(1, plan.num_rows, 576), rand(2, plan.num_rows, 128)
    a, b = (torch.zeros(pages, page, 656, dtype=U8, device="cuda") for _ in range(2))
    x, y = (torch.zeros(pages, page * 132, dtype=U8, device="cuda") for _ in range(2))
    c.quantize_store_latents(plan, lat, a)
    c.quantize_store_keys(plan, keys, x)
    c.append_latents(plan, None, lat[:, :512], lat[:, 512:], b, keys, y)
    assert torch.equal(a, b) and torch.equal(x, y)
    c = contexts(page_size=page)
    plan = c.plan(spans, pages)
    x, y = (torch.zeros(pages, page, 128, dtype=BF16, device="cuda") for _ in range(2))
    c.store_keys(plan, keys, x)
    c.append_latents(plan, None, keys=keys, index_cache=y)
    assert torch.equal(x, y)


@pytest.mark.parametrize("heads,dim,offset,rot,dtype,page", [(4, 128, 0, 128, BF16, 64), (1, 64, 0, 32, F32, 16), (8, 128, 64, 64, BF16, 7),
                                                             (3, 96, 10, 70, F32, 64), (2, 576, 8, 512, BF16, 64), (5, 3, 1, 2, BF16, 64)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_append_kv(contexts, heads, dim, offset, rot, dtype, page, layout):
    c = contexts(page_size=page)
    spans, pages = spans_for(page, 2)
    plan = c.plan(spans, pages)
    T = plan.num_rows
    both = rand(4, T, 2, heads, dim, dtype=dtype)      # a fused projection's halves
    k, v = both[:, 0], both[:, 1]
    keys = rand(5, T, 128)
    table = c.rotary_table(rot)
    msa = W.MSAShape(kv_heads=heads, q_heads=heads, head_dim=dim, page_size=page)
    kv = torch.full((pages, page, 2 * heads * dim), 9.0, dtype=BF16, device="cuda")
    ic, want_ic = (torch.zeros(pages, page, 128, dtype=BF16, device="cuda") for _ in range(2))
    with_keys = rot <= 128
    c.append_kv(plan, msa, table, k, v, kv, *((keys, ic) if with_keys else ()), layout=layout, offset=offset)
    c.get_error()
    where, pos = ref.slots(spans, page)
    got = kv.view(-1, 2, heads, dim).cpu()
    want, mag = ref.rotate(k, torch.from_numpy(pos).int(), ref.frequencies(rot), offset, layout)
    ref.close(got[where][:, 0], want, ref.rotate_bound(k, want, mag, offset, rot, layout), BF16)
    assert torch.equal(got[where][:, 1], v.cpu().to(BF16))
    others = np.setdiff1d(np.arange(pages * page), where)
    assert bool((got[others] == 9.0).all())
    if with_keys:
        c.append_latents(plan, table, keys=keys, index_cache=want_ic)
        assert torch.equal(ic, want_ic)


def test_append_through_a_capturable_plan(contexts):
    """Captured with its re-plan, replayed over other spans: padding rows neither read nor written."""
    c = contexts()
    msa = W.MSAShape()
    table = c.rotary_table(64)
    cap = c.plan_capturable(8, 4, 4000, 12)
    num, dev = positions(0), torch.zeros(4, 6, dtype=I32, device="cuda")
    pages = torch.arange(12, dtype=I32, device="cuda").flip(0).contiguous()
    lat, k_pe, keys, k, v = rand(1, 8, 512), rand(2, 8, 64), rand(3, 8, 128), rand(4, 8, 4, 128), rand(5, 8, 4, 128)
    lc, ic, kv = (torch.zeros(12, 64, n, dtype=BF16, device="cuda") for n in (576, 128, 1024))

    def step():
        c.plan_update(cap, num, dev, pages)
        c.append_latents(cap, table, lat, k_pe, lc, keys, ic)
        c.append_kv(cap, msa, table, k, v, kv)
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for spans in ([[1, 100, 0, 0, 2, 0], [3, 62, 7, 2, 3, 0]], [[5, 0, 0, 6, 1, 0]], []):
        for t in (lc, ic, kv):
            t.fill_(5.0)
        for t, s in ((lat, 1), (k_pe, 2), (keys, 3), (k, 4), (v, 5)):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(s + len(spans))))
        rows = sum(s[0] for s in spans)
        for t in (lat, k_pe, keys, k, v):
            t[rows:] = float("nan")
        num.fill_(len(spans))
        dev.zero_()
        for i, s in enumerate(spans):
            dev[i] = torch.tensor(s, dtype=I32)
        graph.replay()
        c.get_error()
        host, q = [], 0
        for s in spans:
            host.append(W.Span(0, q, s[0], s[1], pages.cpu().numpy()[s[3]:s[3] + s[4]], s[2]))
            q += s[0]
        plan = c.plan(host, 12)
        want = [torch.full_like(t, 5.0) for t in (lc, ic, kv)]
        if rows:
            c.append_latents(plan, table, lat[:rows], k_pe[:rows], want[0], keys[:rows], want[1])
            c.append_kv(plan, msa, table, k[:rows], v[:rows], want[2])
        for a, b in zip((lc, ic, kv), want):
            assert torch.equal(a, b)


def test_append_reports_pages_outside_the_cache(contexts):
    """Only a capturable plan can hold one; its row is skipped."""
    c = contexts()
    cap = c.plan_capturable(4, 2, 400, 3)
    dev = torch.tensor([[1, 0, 0, 0, 1, 0], [1, 64, 0, 0, 2, 0]], dtype=I32, device="cuda")
    c.plan_update(cap, positions(2), dev, positions(1, 3))
    ic = torch.full((3, 64, 128), 9.0, dtype=BF16, device="cuda")
    c.append_latents(cap, None, keys=rand(1, 4, 128), index_cache=ic)
    with pytest.raises(dsa.DSAError) as e:
        c.get_error()
    assert e.value.status == 5
    assert torch.equal(ic[1, 0], rand(1, 4, 128)[0])
    ic[1, 0] = 9.0
    assert bool((ic == 9.0).all())
    c.get_error()


def test_append_refuses(contexts):
    c = contexts()
    plan = c.plan([W.Span(0, 0, 4, 0, np.zeros(1, np.int32))], 1)
    lat, k_pe, keys = rand(1, 4, 512), rand(2, 4, 64), rand(3, 4, 128)
    lc, ic = torch.zeros(1, 64, 576, dtype=BF16, device="cuda"), torch.zeros(1, 64, 128, dtype=BF16, device="cuda")
    t64, t32 = c.rotary_table(64), c.rotary_table(32)
    for bad in (lambda: c.append_latents(plan, t32, lat, k_pe, lc), lambda: c.append_latents(plan, t64, keys=keys, index_cache=ic, key_offset=65),
                lambda: c.append_latents(plan, t64, keys=keys, index_cache=ic, key_offset=-1), lambda: c.append_latents(plan, t64)):
        with pytest.raises(dsa.DSAError) as e:
            bad()
        assert e.value.status == 1
    c.append_latents(plan, t32, keys=keys, index_cache=ic, key_offset=96)
    empty = c.plan([], 1)
    c.append_latents(empty, t64, lat[:0], k_pe[:0], lc)
    assert c.last_launch_count() == 0
    c.get_error()


def test_long_caches(contexts):
    """Rows past 2^31 bytes, and past 2^31 elements, of their cache."""
    c = contexts(page_size=64)
    pages = 2 ** 31 // (64 * 576) + 100                      # 5.0 GB of bf16 latents
    lc = torch.zeros(pages, 64, 576, dtype=BF16, device="cuda")
    last = pages - 1
    plan = c.plan([W.Span(0, 0, 1, 64, np.array([0, last], np.int32)), W.Span(0, 1, 1, 3, np.array([pages // 2 + 7], np.int32))], pages)
    lat, k_pe = rand(1, 2, 512), rand(2, 2, 64)
    c.append_latents(plan, None, lat, k_pe, lc)
    c.get_error()
    assert torch.equal(lc[last, 0], torch.cat((lat[0], k_pe[0]))) and torch.equal(lc[pages // 2 + 7, 3], torch.cat((lat[1], k_pe[1])))
    lc[last, 0] = 0
    lc[pages // 2 + 7, 3] = 0
    assert int(torch.count_nonzero(lc)) == 0


def test_on_another_stream_and_back_to_back(contexts):
    """The rotation's output goes straight into the append on a stream that is not the current one."""
    c = contexts()
    table = c.rotary_table(64)
    plan = c.plan([W.Span(0, 0, 64, 64, np.array([1, 2], np.int32))], 3)
    torch.cuda.synchronize()
    x, other = rand(1, 64, 1, 64), torch.cuda.Stream()
    lat = rand(2, 64, 512)
    a, b = (torch.zeros(3, 64, 576, dtype=BF16, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    r = c.rotary(table, x, plan, stream=other)
    c.append_latents(plan, None, lat, r[:, 0], a, stream=other)
    other.synchronize()
    c.append_latents(plan, table, lat, x[:, 0], b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("layout,key_layout", [("interleaved", "half"), ("half", "interleaved")])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_sparse_layer(contexts, layout, key_layout, fp8):
    """Rotations, one append and the sparse attention: the same bits as with rows that were rotated first and stored
    by the calls without a rotation."""
    c = contexts(topk=64, latent_fmt=W.LATENT_FP8_656 if fp8 else W.LATENT_BF16, index_fmt=W.INDEX_FP8_132 if fp8 else W.INDEX_BF16)
    spans = [W.Span(0, 0, 150, 0, np.array([4, 1, 3], np.int32)), W.Span(1, 150, 70, 0, np.array([5, 0], np.int32))]
    plan = c.plan(spans, 6)
    T = plan.num_rows
    table = c.rotary_table(64, **YARN)
    down = rand(1, T, 704)
    lat, k_pe, keys = rand(2, T, 512), down[:, 512:576], down[:, 576:]
    q_nope, q, qi, w = rand(3, T, 128, 512), rand(4, T, 128, 192), rand(5, T, 64, 128), rand(6, T, 64, dtype=F32).abs()
    if fp8:
        caches = [(torch.zeros(6, 64, 656, dtype=U8, device="cuda"), torch.zeros(6, 64 * 132, dtype=U8, device="cuda")) for _ in range(2)]
    else:
        caches = [(torch.zeros(6, 64, 576, dtype=BF16, device="cuda"), torch.zeros(6, 64, 128, dtype=BF16, device="cuda")) for _ in range(2)]
    q_pe = c.rotary(table, q[..., 128:], plan, layout=layout)
    q_idx = c.rotary(table, qi, plan, layout=key_layout)

    def rest(lc, ic):
        sel = c.index_topk(plan, q_idx, w, ic)
        return sel, c.attend(plan, sel, q_nope, q_pe, lc, None, 192 ** -0.5)
    c.append_latents(plan, table, lat, k_pe, caches[0][0], keys, caches[0][1], layout=layout, key_layout=key_layout)
    sel, out = rest(*caches[0])
    pe, ky = c.rotary(table, k_pe, plan, layout=layout), c.rotary(table, keys, plan, layout=key_layout)
    if fp8:      # (the append rounds a rotated key once, to its code: compared from the append's own keys)
        c.quantize_store_latents(plan, torch.cat((lat, pe), dim=1), caches[1][0])
        assert torch.equal(caches[0][0], caches[1][0])
        caches[1][1].copy_(caches[0][1])
    else:
        where, _ = ref.slots(spans, 64)
        rows = torch.from_numpy(where).cuda()
        caches[1][0].view(-1, 576)[rows] = torch.cat((lat, pe), dim=1)
        c.store_keys(plan, ky, caches[1][1])
        assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    sel2, out2 = rest(*caches[1])
    assert torch.equal(sel, sel2) and torch.equal(out, out2) and bool(torch.isfinite(out).all())
    c.get_error()
