"""GPU: the projection of e4m3 codes with a scale for each block of 128, against
its definition in 64 bits: row counts from one to several tiles, odd and ragged
sizes, heads, strided and unaligned layouts on both kernels, scales of every
size, codes that are NaN, padding rows, capture, streams, and a layer's run of
the operators around the sparse attention."""
import numpy as np
import pytest
import torch

from deepseek_sparse_attention_dsa_gb300 import dsa
from deepseek_sparse_attention_dsa_gb300 import workloads as W
from tests import rows_reference as R
from tests.test_gpu_rows8 import capturable, set_rows

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def ctx():
    from deepseek_sparse_attention_dsa_gb300 import build
    build.build()
    return dsa.Context(W.DSAShape(**W.DEEPSEEK), 0)


def make(seed, rows, n, k, batch=0):
    """Codes of every finite value and scales over six powers of ten, on the GPU; batch 0: without the dimension."""
    g = torch.Generator().manual_seed(seed)
    b = max(1, batch)

    def codes(*shape):
        c = torch.randint(0, 254, shape, generator=g)       # 254 finite codes: 0x7F and 0xFF are NaN
        return (c + (c >= 127)).to(U8)

    def scales(*shape):
        return torch.exp(torch.randn(*shape, generator=g) * 2.0)

    a, w = codes(rows, b, k), codes(b, n, k)
    asc, wsc = scales(rows, b, R.groups(k)), scales(b, R.groups(n), R.groups(k))
    if not batch:
        a, w, asc, wsc = a[:, 0], w[0], asc[:, 0], wsc[0]
    return [t.contiguous().cuda() for t in (a, asc, w, wsc)]


def check(out, a, asc, w, wsc, rows=None):
    k = a.shape[-1]
    if w.dim() == 2:
        a, asc, w, wsc, out = a[:, None], asc[:, None], w[None], wsc[None], out[:, None]
    rows = a.shape[0] if rows is None else rows
    want, mag = R.project(a[:rows], asc[:rows], w, wsc)
    R.check_project(out[:rows], want, mag, k)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 200, 257, 300])
@pytest.mark.parametrize("n,k", [(128, 128), (704, 576), (200, 1040)])
def test_row_counts(ctx, rows, n, k):
    t = make(rows * 7 + n, rows, n, k)
    out = ctx.project_fp8(*t)
    check(out, *t)
    check(ctx.project_fp8(*t, out_dtype=F32), *t)
    ctx.get_error()


@pytest.mark.parametrize("rows,n,k", [(1, 1, 16), (3, 1, 1), (1, 129, 16), (5, 127, 144), (20, 8, 112), (70, 513, 400), (130, 255, 272),
                                      (9, 300, 130), (7, 64, 77), (1, 8192, 2048), (40, 128, 8192), (600, 1000, 256)])
def test_odd_and_ragged_sizes(ctx, rows, n, k):
    t = make(rows + n + k, rows, n, k)
    for dt in (BF16, F32):
        check(ctx.project_fp8(*t, out_dtype=dt), *t)
    ctx.get_error()


@pytest.mark.parametrize("rows,n,k", [(256, 20000, 128), (300, 10000, 144), (1031, 8192, 576), (2600, 2000, 272), (600, 6503, 16), (700, 6500, 1100)])
def test_many_rows(ctx, rows, n, k):
    """Shapes with a tile of 256 x 256 for every two SMs and more: whole and ragged tiles, one tile after another."""
    t = make(rows + n + k, rows, n, k)
    for dt in (BF16, F32):
        check(ctx.project_fp8(*t, out_dtype=dt), *t)
    ctx.get_error()


def test_many_rows_and_heads(ctx):
    for rows, batch, n, k in ((300, 40, 520, 128), (260, 128, 192, 576)):
        t = make(rows, rows, n, k, batch)
        check(ctx.project_fp8(*t), *t)
    ctx.get_error()


@pytest.mark.parametrize("rows,batch,n,k", [(1, 16, 128, 512), (3, 5, 512, 128), (17, 3, 65, 192), (140, 2, 128, 512), (300, 3, 192, 576),
                                            (2, 130, 64, 64)])
def test_heads(ctx, rows, batch, n, k):
    t = make(rows + batch, rows, n, k, batch)
    out = ctx.project_fp8(*t)
    assert out.shape == (rows, batch, n)
    check(out, *t)
    ctx.get_error()


@pytest.mark.parametrize("pad,shift,fast", [(16, 0, True), (32, 16, True), (8, 0, False), (16, 4, False)])
def test_strided_and_unaligned_layouts(ctx, pad, shift, fast):
    """Rows and heads at strides beyond their length: on 16 bytes for the tensor cores, off them for the other kernel."""
    rows, batch, n, k = 37, 3, 136, 272
    a, asc, w, wsc = make(5, rows, n, k, batch)

    abig = torch.full((rows, batch, k + pad), 0x7F, dtype=U8, device="cuda").view(-1)
    abig = torch.cat([torch.full((shift,), 0x7F, dtype=U8, device="cuda"), abig])
    a2 = abig[shift:].view(rows, batch, k + pad)[:, :, :k]
    a2.copy_(a)
    wbig = torch.full((batch, n + 2, k + pad), 0x7F, dtype=U8, device="cuda")
    w2 = wbig[:, 1:n + 1, :k]
    w2.copy_(w)
    as2 = torch.full((batch, rows, 7), float("nan"), device="cuda")[:, :, 2:5].transpose(0, 1)    # heads outermost
    as2.copy_(asc)
    ws2 = torch.full((batch, 4, 5), float("nan"), device="cuda")[:, 1:3, :3]
    ws2.copy_(wsc)
    for dt in (BF16, F32):
        store = torch.full((batch, rows + 2, n + 5), 77.0, dtype=dt, device="cuda")
        out = store[:, 1:rows + 1, 3:n + 3].transpose(0, 1)
        assert ctx.project_on_tensor_cores(a2, as2, w2, ws2, out) == fast
        ctx.project_fp8(a2, as2, w2, ws2, out=out)
        check(out, a, asc, w, wsc)
        out.fill_(77.0)
        assert (store == 77).all()      # nothing beside the rows was written
    ctx.get_error()


@pytest.mark.parametrize("rows,batch,n,k", [(20, 3, 136, 272), (300, 3, 136, 272), (300, 40, 520, 128)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_heads_outermost_output(ctx, rows, batch, n, k, dt):
    """out as [batch][rows][n] in a larger buffer, on 16 bytes: whole boxes are stored at permuted strides."""
    t = make(21, rows, n, k, batch)
    store = torch.full((batch, rows + 1, n + 8), 77.0, dtype=dt, device="cuda")
    out = store[:, :rows, :n].transpose(0, 1)
    ctx.project_fp8(*t, out=out)
    check(out, *t)
    out.fill_(77.0)
    assert (store == 77).all()


def test_one_weight_for_every_head(ctx):
    """w expanded over the batch (a stride of zero)."""
    a, asc, w, wsc = make(6, 20, 128, 256, 4)
    t = (a, asc, w[:1].expand(4, -1, -1), wsc[:1].expand(4, -1, -1))
    check(ctx.project_fp8(*t), *[x.contiguous() for x in t])


def test_both_kernels_give_what_the_definition_gives_for_integers(ctx):
    """Small whole codes and scales of powers of two: every sum is exact, so the
    two kernels, every split and the definition agree to the bit."""
    for rows, n, k in ((1, 256, 2048), (16, 384, 1024), (100, 256, 512), (300, 136, 1152), (300, 9992, 384)):
        g = torch.Generator().manual_seed(rows)
        a = torch.randint(-3, 4, (rows, k), generator=g).float().to(torch.float8_e4m3fn).view(U8)
        w = torch.randint(-3, 4, (n, k), generator=g).float().to(torch.float8_e4m3fn).view(U8)
        asc = 2.0 ** torch.randint(-2, 3, (rows, R.groups(k)), generator=g).float()
        wsc = 2.0 ** torch.randint(-2, 3, (R.groups(n), R.groups(k)), generator=g).float()
        want, _ = R.project(a[:, None], asc[:, None], w[None], wsc[None])
        a, asc, w, wsc = a.cuda(), asc.cuda(), w.cuda(), wsc.cuda()
        got = ctx.project_fp8(a, asc, w, wsc, out_dtype=F32)
        off = torch.empty(rows, k + 1, dtype=U8, device="cuda")[:, :k]
        off.copy_(a)
        assert torch.equal(got.cpu().double(), want[:, 0])
        assert torch.equal(ctx.project_fp8(off, asc, w, wsc, out_dtype=F32), got)


def test_a_nan_stays_in_its_row_or_column(ctx):
    a, asc, w, wsc = make(8, 40, 200, 384)
    ref = ctx.project_fp8(a, asc, w, wsc)
    a[7, 200] = 0x7F
    asc[9, 1] = float("inf")
    w[150, 3] = 0xFF
    out = ctx.project_fp8(a, asc, w, wsc)
    clean = torch.ones(40, 200, dtype=torch.bool)
    clean[7] = clean[9] = clean[:, 150] = False
    assert torch.equal(out.cpu()[clean], ref.cpu()[clean])
    assert out[7].isnan().all() and not out[9].isfinite().any() and out[:, 150].isnan().all()


def test_no_rows_launch_nothing(ctx):
    a, asc, w, wsc = make(9, 1, 128, 128)
    out = ctx.project_fp8(a[:0], asc[:0], w, wsc)
    assert out.shape == (0, 128) and ctx.last_launch_count() == 0
    ctx.project_fp8(a, asc, w, wsc)
    assert ctx.last_launch_count() == 1


@pytest.mark.parametrize("m,n", [(1, 264), (40, 264), (80, 9000)])
def test_padding_rows_of_a_capturable_plan_are_left(ctx, m, n):
    rows = 8 * m
    t = make(10, rows, n, 320)
    full = ctx.project_fp8(*t)
    plan = None
    for live in (8, 0, 5):
        if plan is None:
            plan = capturable(ctx, live)
        else:
            set_rows(ctx, plan, live)
        a, asc, w, wsc = (x.clone() for x in t)
        a[live * m:] = 0x7F
        asc[live * m:] = float("nan")
        out = torch.full((rows, n), 77.0, dtype=BF16, device="cuda")
        ctx.project_fp8(a, asc, w, wsc, out=out, plan=plan)
        assert torch.equal(out[:live * m], full[:live * m]) and (out[live * m:] == 77).all()
    ctx.get_error()


def test_equal_calls_give_equal_bits_on_any_stream(ctx):
    for rows, n, k in ((1, 1024, 4096), (24, 512, 2048), (520, 384, 512), (520, 9000, 512)):
        t = make(11, rows, n, k)
        ref = ctx.project_fp8(*t, out_dtype=F32)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        outs = []
        for i in range(6):    # calls that run side by side share nothing
            outs.append(ctx.project_fp8(*t, out_dtype=F32, stream=streams[i % 3]))
        torch.cuda.synchronize()
        assert all(torch.equal(o, ref) for o in outs)


def test_captured_and_replayed_on_new_data(ctx):
    a, asc, w, wsc = make(12, 18, 512, 1024)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ctx.project_fp8(a, asc, w, wsc)
    s.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=s):
        out1 = ctx.project_fp8(a, asc, w, wsc)
    with torch.cuda.graph(g2, stream=s):
        out2 = ctx.project_fp8(a, asc, w, wsc, out_dtype=F32)
    for seed in (13, 14):
        a.copy_(make(seed, 18, 512, 1024)[0])
        torch.cuda.synchronize()
        s1 = torch.cuda.Stream()
        g1.replay()
        with torch.cuda.stream(s1):
            g2.replay()
        torch.cuda.synchronize()
        check(out1, a, asc, w, wsc)
        check(out2, a, asc, w, wsc)
    ctx.get_error()


def test_refused_calls_leave_the_context_usable(ctx):
    a, asc, w, wsc = make(15, 4, 128, 128)

    def status(fn):
        with pytest.raises(dsa.DSAError) as e:
            fn()
        return e.value.status

    plan3 = ctx.plan([W.Span(0, 0, 3, 0, np.zeros(1, np.int32))], 1)
    assert status(lambda: ctx.project_fp8(a, asc, w, wsc, plan=plan3)) == 1
    assert status(lambda: ctx.project_fp8(a, asc, w, wsc, out=torch.empty(128, dtype=BF16, device="cuda").expand(4, 128))) == 1
    check(ctx.project_fp8(a[:3], asc[:3], w, wsc, plan=plan3), a[:3], asc[:3], w, wsc)
    with pytest.raises(ValueError):
        ctx.project_fp8(a.cpu(), asc, w, wsc)
    ctx.get_error()


@pytest.mark.parametrize("rows", [5, 70, 130, 700])
def test_inputs_may_overlap_or_repeat(ctx, rows):
    """Rows 16 codes apart (windows of one sequence) on the tensor cores; one row, or one matrix, for all (stride 0) off them."""
    n, k = 1024, 272
    a, asc, w, wsc = make(rows, rows, n, k)
    windows = make(rows + 1, 1, 128, 16 * rows + k)[0].view(-1).as_strided((rows, k), (16, 1))
    for x, ws, fast in ((windows, w, True), (a, make(3, 1, 128, 16 * n + k)[0].view(-1).as_strided((n, k), (16, 1)), True),
                        (a[:1].expand(rows, k), w, False), (a, w[:1].expand(n, k), False)):
        out = torch.empty(rows, n, dtype=F32, device="cuda")
        assert ctx.project_on_tensor_cores(x, asc, ws, wsc, out) is fast
        check(ctx.project_fp8(x, asc, ws, wsc, out=out), x, asc, ws, wsc)
    ctx.get_error()


def test_heads_share_a_matrix_or_their_rows(ctx):
    rows, batch, n, k = 40, 6, 200, 272
    a, asc, w, wsc = make(8, rows, n, k, batch)
    for x, xs, m, ms in ((a, asc, w[:1].expand_as(w), wsc[:1].expand_as(wsc)), (a[:, :1].expand_as(a), asc[:, :1].expand_as(asc), w, wsc)):
        check(ctx.project_fp8(x, xs, m, ms), x, xs, m, ms)
    ctx.get_error()


def test_the_longest_rows(ctx):
    """k up to the last block of 32 bits."""
    k = 2 ** 31 - 16
    a = torch.zeros(1, k, dtype=U8, device="cuda")
    w = torch.zeros(1, k, dtype=U8, device="cuda")
    at = torch.tensor([0, 127, 128, 2 ** 24 + 5, 2 ** 30, k - 129, k - 128, k - 1], device="cuda")
    a[0, at] = 0x38            # 1.0
    w[0, at] = 0x40            # 2.0
    asc = torch.full((1, R.groups(k)), 0.5, device="cuda")
    wsc = torch.full((1, R.groups(k)), 0.25, device="cuda")
    wsc[0, at // 128] = 3.0
    out = ctx.project_fp8(a, asc, w, wsc, out_dtype=F32)
    assert ctx.project_on_tensor_cores(a, asc, w, wsc, out)
    assert out.item() == 0.5 * 3.0 * 2.0 * 8
    ctx.get_error()


def test_the_longest_rows_quantised(ctx):
    """One row: its groups of 128 columns are its blocks too."""
    k = 2 ** 31 - 1
    x = torch.zeros(1, k, dtype=BF16, device="cuda")
    x[0, ::1000003] = 3.5
    x[0, -5:] = -7.0
    codes, scales = ctx.quantize_rows(x)
    assert codes[0, -5:].tolist() == [0xFE] * 5 and scales[0, -1].item() == 7.0 / 448
    w_codes, w_scales = ctx.quantize_weight(x)
    assert torch.equal(codes, w_codes) and torch.equal(scales, w_scales)
    assert int((codes != 0).sum()) == int((x != 0).sum())


@pytest.mark.parametrize("n", [136, 700, 20000])
def test_padding_begins_at_any_row(ctx, n):
    """Inside, at the start and at the end of the 32 rows that are stored together, in whole and in cut columns."""
    cap = 300
    t = make(14, cap, n, 160)
    plan = ctx.plan_capturable(cap, cap, cap, 1)
    spans = torch.tensor([[1, 0, 0, 0, 1, 0]] * cap, dtype=torch.int32, device="cuda")   # one token each, all in page 0
    pages = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt in (BF16, F32):
        full = ctx.project_fp8(*t, out_dtype=dt)
        for live in (1, 31, 32, 33, 100, 128, 160, 256, 289, 299, 300):
            count = torch.tensor([live], dtype=torch.int32, device="cuda")
            ctx.plan_update(plan, count, spans, pages)
            out = torch.full((cap, n), 77.0, dtype=dt, device="cuda")
            ctx.project_fp8(*t, out=out, plan=plan)
            assert torch.equal(out[:live], full[:live]) and (out[live:] == 77).all()
    ctx.get_error()


@pytest.mark.parametrize("rows,n,k", [(200, 4096, 4096), (1031, 704, 5120), (130, 200, 1040), (300, 520, 3000), (256, 2048, 1152)])
def test_pairs_that_split_k(ctx, rows, n, k):
    """Few tiles of many tokens: two pairs of CTAs share one, with even and odd numbers of blocks."""
    t = make(rows + n, rows, n, k)
    for dt in (BF16, F32):
        out = ctx.project_fp8(*t, out_dtype=dt)
        check(out, *t)
        assert torch.equal(out, ctx.project_fp8(*t, out_dtype=dt))
    ctx.get_error()


def test_threads_share_a_context(ctx):
    """Calls from several threads at once, each on a stream of its own, from the first call of a size on."""
    import threading
    sizes = [(1, 1032, 2048), (48, 1032, 2064), (200, 1032, 2080), (600, 1032, 2096)]
    ts = [make(30 + i, *s) for i, s in enumerate(sizes)]
    x = torch.randn(70, 1032, device="cuda").to(BF16)
    got, failed = {}, []
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for j in range(20):
                    a = (i + j) % len(ts)
                    got[i, j] = a, ctx.project_fp8(*ts[a], out_dtype=F32), ctx.rmsnorm(x, None), ctx.quantize_rows(x)
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    outs = [ctx.project_fp8(*t, out_dtype=F32) for t in ts]
    y, (codes, scales) = ctx.rmsnorm(x, None), ctx.quantize_rows(x)
    for a, out, yi, (ci, si) in got.values():
        assert torch.equal(out, outs[a]) and torch.equal(yi, y) and torch.equal(ci, codes) and torch.equal(si, scales)
    ctx.get_error()


@pytest.mark.parametrize("rows,n,k", [(1, 1032, 8192), (16, 2048, 4096), (30, 1032, 8192), (60, 520, 8192), (128, 8192, 4096), (200, 4096, 4096),
                                      (1031, 704, 5120)])
def test_sums_that_cross_ctas_are_whole(ctx, rows, n, k):
    """Every form that splits k, again and again on other numbers: whole codes and
    scales of powers of two, so that a sum read before it is there, or read from
    the call before, is off by more than a rounding."""
    g = torch.Generator().manual_seed(rows)
    w = torch.randint(-3, 4, (n, k), generator=g).float()
    ts = []
    for i in range(4):
        a = torch.randint(-3, 4, (rows, k), generator=g).float()
        asc = 2.0 ** torch.randint(-2, 3, (rows, R.groups(k)), generator=g).float()
        ts.append((a.to(torch.float8_e4m3fn).cuda(), asc.cuda()))
    wc, wsc = w.to(torch.float8_e4m3fn).cuda(), 2.0 ** torch.randint(-2, 3, (R.groups(n), R.groups(k)), generator=g).float().cuda()
    col, row = torch.arange(k, device="cuda") // R.GROUP, torch.arange(n, device="cuda") // R.GROUP
    wv = wc.float().double() * wsc.double()[row][:, col]
    want = [((a.float().double() * s.double()[:, col]) @ wv.t()).float() for a, s in ts]
    outs = []
    for i in range(80):
        outs.append(ctx.project_fp8(*ts[i % 4], wc, wsc, out_dtype=F32))
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 4]), i
    ctx.get_error()


def test_threads_leave_a_launch_count_of_one_call(ctx):
    """One launch a call: the count that a call leaves is one, also where another
    thread's calls begin and end while it waits for room in its stream."""
    import threading
    import time
    x = torch.randn(3, 256, device="cuda").to(BF16)
    codes, scales = ctx.quantize_rows(x)
    full, free = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    seen, done = set(), threading.Event()

    def fill():     # more calls than a stream takes while its first kernel runs: one of them waits
        with torch.cuda.stream(full):
            torch.cuda._sleep(600_000_000)      # some 0.3 s
            for _ in range(3000):
                ctx.quantize_rows(x, codes, scales)
                seen.add(ctx.last_launch_count())
        done.set()

    filler = threading.Thread(target=fill)
    filler.start()
    while not done.is_set():
        ctx.quantize_rows(x, stream=free)
        seen.add(ctx.last_launch_count())
        time.sleep(0.002)
    filler.join()
    torch.cuda.synchronize()
    assert seen == {1}
    assert dsa.load().dsa_last_cuda_error(ctx.handle) == b""
    ctx.get_error()
