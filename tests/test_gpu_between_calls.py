"""GPU: calls of the rotations, appends and the attention over a shared prefix next to one another: new inputs from call to
call without a wait, host threads, sources that repeat, and mixed batches of every head layout."""
import random
import threading

import numpy as np
import pytest
import torch

from deepseek_sparse_attention_dsa_gb300 import dsa
from deepseek_sparse_attention_dsa_gb300 import workloads as W
from tests import rotary_reference as ref
from tests.test_gpu_prefix import batch, inputs, shape

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def contexts():
    from deepseek_sparse_attention_dsa_gb300 import build
    build.build()
    made = {}

    def get(page=64):
        if page not in made:
            made[page] = dsa.Context(W.DSAShape(**dict(W.DEEPSEEK, page_size=page)), 0)
        return made[page]
    return get


def rand(seed, *shape, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("rows,q_heads,kv_heads,dim", [(4, 64, 4, 128), (33, 64, 4, 64), (3, 6, 2, 96)])
def test_other_queries_from_call_to_call(contexts, rows, q_heads, kv_heads, dim):
    """One plan's calls back to back, each launched while the one before runs: its partial results are its own."""
    ctx = contexts()
    spans, pages = batch(1, 64, [(1280 + 5 * i, 1) for i in range(rows)], 20)
    _, kv = inputs(2, spans, pages, 64, q_heads, kv_heads, dim)
    pp, kv = ctx.plan_prefix(ctx.plan(spans, pages), shape(q_heads, kv_heads, dim)), kv.cuda()
    qs = [rand(10 + i, rows, q_heads, dim) for i in range(7)]
    want = []
    for q in qs:
        want.append(ctx.prefix_attend(pp, q, kv))
        torch.cuda.synchronize()
    for _ in range(10):
        got = [ctx.prefix_attend(pp, q, kv) for q in qs]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.zeros_like(q) for q in qs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for q, out in zip(qs, outs):
                ctx.prefix_attend(pp, q, kv, out=out)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    ctx.get_error()


def test_layers_with_a_turn_in_place(contexts):
    """Eight layers in a row through the same buffers, nothing waited for: queries turned in place and attended, the next
    layer's written over them."""
    ctx = contexts()
    msa, table = shape(64, 4), ctx.rotary_table(128)
    spans, pages = batch(3, 64, [(640 + 3 * i, 1 + i % 3) for i in range(9)], 10)
    plan = ctx.plan(spans, pages)
    pp, T = ctx.plan_prefix(plan, msa), plan.num_rows
    _, kv0 = inputs(4, spans, pages, 64, 64, 4, 128)
    layers = [(rand(20 + 3 * i, T, 64, 128), rand(21 + 3 * i, T, 4, 128), rand(22 + 3 * i, T, 4, 128), kv0.cuda()) for i in range(8)]

    def run(wait):
        x, out, got = torch.zeros(T, 64, 128, dtype=BF16, device="cuda"), torch.zeros(T, 64, 128, dtype=BF16, device="cuda"), []
        for q, k, v, kv in layers:
            for call in (lambda: x.copy_(q), lambda: ctx.rotary(table, x, plan, layout="half", out=x),
                         lambda: ctx.append_kv(plan, msa, table, k, v, kv), lambda: ctx.prefix_attend(pp, x, kv, out=out)):
                call()
                if wait:
                    torch.cuda.synchronize()
            got.append(out.clone())
        return got
    want = run(True)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))
    ctx.get_error()


def test_host_threads(contexts):
    """A context's calls from four threads, each with a plan and a stream of its own."""
    ctx = contexts()
    msa, table = shape(16, 2), ctx.rotary_table(64)
    work, failed = [], []
    for t in range(4):
        spans, pages = batch(40 + t, 64, [(256 + 7 * i, 1 + t) for i in range(5 + t)], 4)
        _, kv = inputs(50 + t, spans, pages, 64, 16, 2, 128)
        T = sum(s.q_len for s in spans)
        work.append((ctx.plan(spans, pages), kv.cuda(), rand(60 + t, T, 16, 128), rand(70 + t, T, 2, 128), rand(80 + t, T, 2, 128)))

    def step(plan, kv, q, k, v):
        pp, kv = ctx.plan_prefix(plan, msa), kv.clone()
        rq = ctx.rotary(table, q, plan, layout="half")
        ctx.append_kv(plan, msa, table, k, v, kv)
        out = ctx.prefix_attend(pp, rq, kv)
        torch.cuda.current_stream().synchronize()
        return out

    want = [step(*w) for w in work]
    torch.cuda.synchronize()

    def thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    assert torch.equal(step(*work[i]), want[i])
        except BaseException as e:      # noqa: BLE001 (handed to the test's own thread)
            failed.append(e)
    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    ctx.get_error()


@pytest.mark.parametrize("rows", [5, 700])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sources_that_repeat(contexts, rows, dtype):
    """One row for all of a step, one head for all of a row: strides of 0 are read, and give what copies give."""
    ctx = contexts()
    msa, table = W.MSAShape(kv_heads=4, q_heads=4), ctx.rotary_table(64)
    pages = rows // 64 + 2
    plan = ctx.plan([W.Span(0, 0, rows, 9, np.arange(pages, dtype=np.int32))], pages)
    lat, k_pe, keys, k = (rand(i, 1, *n, dtype=dtype) for i, n in enumerate([(512,), (64,), (128,), (1, 128)]))
    lat, k_pe, keys, k = lat.expand(rows, -1), k_pe.expand(rows, -1), keys.expand(rows, -1), k.expand(rows, 4, -1)
    v = rand(9, rows, 1, 128, dtype=dtype).expand(rows, 4, 128)
    got, want = ([torch.zeros(pages, 64, n, dtype=BF16, device="cuda") for n in (576, 128, 1024)] for _ in range(2))
    for caches, f in ((got, lambda t: t), (want, lambda t: t.contiguous())):
        ctx.append_latents(plan, table, f(lat), f(k_pe), caches[0], f(keys), caches[1])
        ctx.append_kv(plan, msa, table, f(k), f(v), caches[2])
    for a, b in zip(got, want):
        assert torch.equal(a, b) and bool(a.any())
    assert torch.equal(ctx.rotary(table, k, plan), ctx.rotary(table, k.contiguous(), plan))
    ctx.get_error()


def defined(spans, page, q, kv, kv_heads, scale):
    """What rotary_reference.prefix_attend gives, on the GPU a kv head at a time."""
    T, heads, dim = q.shape
    cache, group = kv.view(-1, 2, kv_heads, dim), heads // kv_heads
    out, mag, top = (torch.empty(*s, dtype=torch.float64, device="cuda") for s in (q.shape, q.shape, q.shape[:2]))
    for s in spans:
        end, rows = s.ctx_start + s.q_len, slice(s.q_start, s.q_start + s.q_len)
        slot = s.page_start + np.arange(end)
        at = torch.from_numpy(s.pages.astype(np.int64)[slot // page] * page + slot % page).cuda()
        late = torch.arange(end, device="cuda")[None] > s.ctx_start + torch.arange(s.q_len, device="cuda")[:, None]
        for g in range(kv_heads):
            hs = slice(g * group, (g + 1) * group)
            k, v, x = cache[at, 0, g].double(), cache[at, 1, g].double(), q[rows, hs].double()
            w = torch.softmax((torch.einsum("nhd,td->hnt", x, k) * scale).masked_fill(late, -float("inf")), dim=-1)
            out[rows, hs], mag[rows, hs] = torch.einsum("hnt,td->nhd", w, v), torch.einsum("hnt,td->nhd", w, v.abs())
            top[rows, hs] = (torch.einsum("nhd,td->hnt", x.abs(), k.abs()) * scale).masked_fill(late, 0.0).amax(-1).t()
    return out.cpu(), mag.cpu(), top.cpu()


@pytest.mark.parametrize("seed", range(26))
def test_mixed_batches(contexts, seed):
    """Runs of requests behind prefixes of any length and requests alone, of one to some hundred rows each, every layout of
    heads twice; cache rows that nobody sees hold NaN."""
    rng = random.Random(seed)
    q_heads, kv_heads, dim = [(64, 4, 128), (64, 4, 64), (40, 8, 64), (96, 1, 128), (8, 8, 64), (12, 4, 128), (16, 1, 64), (128, 1, 64),
                              (7, 7, 128), (66, 2, 128), (127, 1, 64), (4, 2, 96), (6, 2, 33)][seed % 13]
    page = rng.choice([8, 24, 48, 64, 64, 128, 256])
    start = rng.choice([0, rng.randrange(3 * page)])
    runs, cost = [], 0
    for _ in range(rng.randint(1, 4)):
        shared = rng.choice([0, 1, int(2 ** rng.uniform(1, 12)) // page + 1])
        requests = []
        for _ in range(int(2 ** rng.uniform(0, 5))):
            context, new = max(shared * page - start, 0) + int(2 ** rng.uniform(0, 10)) - 1, rng.choice([1, 1, 1, 2, 5, 17, 64, 130])
            cost += new * (context + new)
            if cost < 1500000:
                requests.append((context, new))
        runs.append((shared, requests))
    need = sum(n + sum(-(-(start + c + m) // page) - n for c, m in requests) for n, requests in runs)
    pool, spans, at, q0, given = np.random.default_rng(seed).permutation(need + 3).astype(np.int32), [], 0, 0, []
    for n, requests in runs:
        common = pool[at:at + n]
        at += n
        tokens = min([n * page - start] + [c for c, _ in requests])
        if len(requests) and tokens > 3:
            given.append((len(spans), len(requests), tokens - rng.choice([0, 3])))
        for c, m in requests:
            k = -(-(start + c + m) // page) - n
            spans.append(W.Span(0, q0, m, c, np.concatenate((common, pool[at:at + k])), start))
            at += k
            q0 += m
    ctx, msa = contexts(page), shape(q_heads, kv_heads, dim, page)
    q, kv = (t.cuda() for t in inputs(seed, spans, need + 3, page, q_heads, kv_heads, dim))
    plan, want = ctx.plan(spans, need + 3), defined(spans, page, q, kv, kv_heads, msa.sm_scale)
    for prefixes in (None, given, []):
        pp = ctx.plan_prefix(plan, msa, prefixes)
        out = ctx.prefix_attend(pp, q, kv)
        ctx.get_error()
        ref.check_attend(out, want, dim, max(s.ctx_end for s in spans), pp.on_tensor_cores)
