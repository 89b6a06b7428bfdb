"""GPU: the 8-bit rows and projections together with the sparse attention, as a
layer runs them: norm with residual -> down projection (latents, rope, index
keys), latents' norm, quantise-on-store, indexer query and weights, selection,
absorbed queries by head, sparse attention, its output's codes, values by head,
output projection, next norm.  Each operator is held to its definition on the
inputs that the one before it made, the attention to the oracle; the same step
back to back without a wait, captured with a capturable plan and replayed gives
the same bits."""
import numpy as np
import pytest
import torch

import oracle
from deepseek_sparse_attention_dsa_gb300 import dsa
from deepseek_sparse_attention_dsa_gb300 import workloads as W
from tests import harness as H
from tests import rows_reference as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
D, HEAD = 1024, 128            # hidden width; columns of a head's query and value


@pytest.fixture(scope="module")
def built():
    from deepseek_sparse_attention_dsa_gb300 import build
    build.build()


class Layer:
    """One layer's quantised weights, made by the library once."""

    def __init__(self, ctx, seed):
        g = torch.Generator().manual_seed(seed)
        sh = ctx.shape
        L, Rp, Hm, Hi = sh.kv_lora_rank, sh.rope_dim, sh.heads, sh.index_heads

        def weight(*shape):
            return ctx.quantize_weight((torch.randn(*shape, generator=g) / shape[-1] ** 0.5).to(BF16).cuda())

        self.norm1, self.norm2, self.norm_latent = ((1 + 0.2 * torch.randn(n, generator=g)).to(BF16).cuda() for n in (D, D, L))
        self.down = weight(L + Rp + sh.index_dim, D)
        self.index_q = weight(Hi * sh.index_dim, D)
        self.index_w = weight(Hi, D)
        self.q = weight(Hm * HEAD, D)
        self.q_pe = weight(Hm * Rp, D)
        self.absorb_k = weight(Hm, L, HEAD)
        self.absorb_v = weight(Hm, HEAD, L)
        self.out = weight(D, Hm * HEAD)


def step(ctx, layer, plan, T, x, residual, index_cache, latent_cache, padded=None):
    """One layer's pass; every intermediate by name.  padded: the plan, where its rows may be padding."""
    sh = ctx.shape
    L, Rp, Hm, Hi, Di = sh.kv_lora_rank, sh.rope_dim, sh.heads, sh.index_heads, sh.index_dim
    s = {}
    s["c1"], s["s1"], s["res1"] = ctx.rmsnorm_quantize(x, layer.norm1, residual=residual, plan=padded)
    s["down"] = ctx.project_fp8(s["c1"], s["s1"], *layer.down, plan=padded)
    s["lat"] = torch.zeros(T, L + Rp, dtype=BF16, device="cuda")
    ctx.rmsnorm(s["down"][:, :L], layer.norm_latent, out=s["lat"][:, :L], plan=padded)      # strided in and out
    s["lat"][:, L:] = s["down"][:, L:L + Rp]
    ctx.quantize_store_latents(plan, s["lat"], latent_cache)
    ctx.quantize_store_keys(plan, s["down"][:, L + Rp:].contiguous(), index_cache)
    s["iq"] = ctx.project_fp8(s["c1"], s["s1"], *layer.index_q, plan=padded)
    s["iw"] = ctx.project_fp8(s["c1"], s["s1"], *layer.index_w, out_dtype=F32, plan=padded)
    s["iqc"], s["iqs"] = ctx.quantize_rows(s["iq"].view(T * Hi, Di), plan=padded)
    s["sel"] = ctx.index_topk_fp8q(plan, s["iqc"].view(T, Hi, Di), s["iqs"].view(T, Hi), s["iw"], index_cache)
    s["q"] = ctx.project_fp8(s["c1"], s["s1"], *layer.q, plan=padded)
    s["q_pe"] = ctx.project_fp8(s["c1"], s["s1"], *layer.q_pe, plan=padded)
    s["qc"], s["qs"] = ctx.quantize_rows(s["q"], plan=padded)
    s["q_nope"] = ctx.project_fp8(s["qc"].view(T, Hm, HEAD), s["qs"].view(T, Hm, 1), *layer.absorb_k, plan=padded)
    s["att"] = ctx.attend(plan, s["sel"], s["q_nope"], s["q_pe"].view(T, Hm, Rp), latent_cache, None, sh.sm_scale)
    s["ac"], s["as"] = ctx.quantize_rows(s["att"].view(T, Hm * L), plan=padded)
    s["v"] = ctx.project_fp8(s["ac"].view(T, Hm, L), s["as"].view(T, Hm, L // 128), *layer.absorb_v, plan=padded)
    s["vc"], s["vs"] = ctx.quantize_rows(s["v"].view(T, Hm * HEAD), plan=padded)
    s["y"] = ctx.project_fp8(s["vc"], s["vs"], *layer.out, plan=padded)
    s["c2"], s["s2"], s["res2"] = ctx.rmsnorm_quantize(s["y"], layer.norm2, residual=s["res1"], plan=padded)
    return s


def inputs(T, seed):
    g = torch.Generator().manual_seed(seed)
    return ((2 * torch.randn(T, D, generator=g)).to(BF16).cuda(), (4 * torch.randn(T, D, generator=g)).to(BF16).cuda())


def workload():
    # decode rows and a chunk that crosses topk
    return H.deepseek_small(seed=71, fp8=True, decode_ctx=(2500, 300, 4001), chunk=(2040, 20))


def check_project(out, codes, scales, weight, k):
    w, ws = weight
    if w.dim() == 2:
        codes, scales, w, ws, out = codes[:, None], scales[:, None], w[None], ws[None], out[:, None]
    want, mag = R.project(codes, scales, w, ws)
    R.check_project(out, want, mag, k)


def test_a_layer_holds_each_operator_to_its_definition(built):
    wl = workload()
    sh = wl.shape
    ctx = dsa.Context(sh, 0)
    plan = ctx.plan(wl.spans, wl.num_pages)
    T = plan.num_rows
    layer = Layer(ctx, 1)
    x, residual = inputs(T, 2)
    ic, lc = W.make_index_cache(wl).cuda(), W.make_latent_cache(wl).cuda()
    s = step(ctx, layer, plan, T, x, residual, ic, lc)
    ctx.get_error()
    L, Rp, Hm, Hi, Di = sh.kv_lora_rank, sh.rope_dim, sh.heads, sh.index_heads, sh.index_dim
    y, h = R.rmsnorm(x, layer.norm1, 1e-6, residual)
    R.check_codes(s["c1"], s["s1"], y, R.norm_error(D))
    assert ((s["res1"].cpu().double() - h).abs() <= (2.0 ** -8 + 2 * R.EPS32) * h.abs()).all()
    for name, weight in (("down", layer.down), ("iq", layer.index_q), ("iw", layer.index_w), ("q", layer.q), ("q_pe", layer.q_pe)):
        check_project(s[name], s["c1"], s["s1"], weight, D)
    y, _ = R.rmsnorm(s["down"][:, :L], layer.norm_latent, 1e-6)
    assert ((s["lat"][:, :L].cpu().double() - y).abs() <= (2.0 ** -8 + 2 * R.norm_error(L)) * y.abs()).all()
    ref_codes, ref_scales = oracle.quantize_rows(s["iq"].cpu(), Di)     # the quantise-on-store rule, byte for byte
    assert np.array_equal(s["iqc"].cpu().numpy().reshape(-1), ref_codes)
    assert np.array_equal(s["iqs"].cpu().numpy().reshape(-1), ref_scales)
    check_project(s["q_nope"], s["qc"].view(T, Hm, HEAD), s["qs"].view(T, Hm, 1), layer.absorb_k, HEAD)
    # selection and attention against the oracle, on the caches as the step left them
    scores, off = oracle.index_scores_fp8q(sh, wl.spans, wl.num_pages, ref_codes, ref_scales, s["iw"].cpu(), ic.cpu())
    H.check_selection(s["sel"].cpu().numpy(), oracle.topk(sh, wl.spans, scores, off), scores, off, sh.topk)
    ref = oracle.attend(sh, wl.spans, wl.num_pages, s["sel"].cpu().numpy(), s["q_nope"].cpu(), s["q_pe"].view(T, Hm, Rp).cpu(),
                        lc.cpu(), None)
    H.check_attention(s["att"].float().cpu().numpy(), ref, fp8=True)
    rc, rs = oracle.quantize_rows(s["att"].cpu(), 128)
    assert np.array_equal(s["ac"].cpu().numpy().reshape(-1), rc) and np.array_equal(s["as"].cpu().numpy().reshape(-1), rs)
    check_project(s["v"], s["ac"].view(T, Hm, L), s["as"].view(T, Hm, L // 128), layer.absorb_v, L)
    check_project(s["y"], s["vc"], s["vs"], layer.out, Hm * HEAD)
    y, h = R.rmsnorm(s["y"], layer.norm2, 1e-6, s["res1"])
    R.check_codes(s["c2"], s["s2"], y, R.norm_error(D))
    assert ((s["res2"].cpu().double() - h).abs() <= (2.0 ** -8 + 2 * R.EPS32) * h.abs()).all()


def test_steps_back_to_back_equal_steps_with_a_wait_between_the_calls(built):
    """Launches of these operators overlap with the kernel before them: the
    outputs are those of calls that wait for one another."""
    wl = workload()
    ctx = dsa.Context(wl.shape, 0)
    plan = ctx.plan(wl.spans, wl.num_pages)
    T = plan.num_rows
    layer = Layer(ctx, 3)
    ic, lc = W.make_index_cache(wl).cuda(), W.make_latent_cache(wl).cuda()

    def run(wait):
        # three layers over the same buffers, the residual in place
        x, residual = inputs(T, 4)
        outs = []
        codes, scales = (torch.empty(T, D, dtype=torch.uint8, device="cuda"), torch.empty(T, D // 128, device="cuda"))
        y = x.clone()
        for _ in range(12):
            ctx.rmsnorm_quantize(y, layer.norm1, residual=residual, residual_out=residual, codes=codes, scales=scales)
            if wait:
                torch.cuda.synchronize()
            q = ctx.project_fp8(codes, scales, *layer.q)
            if wait:
                torch.cuda.synchronize()
            qc, qs = ctx.quantize_rows(q)
            if wait:
                torch.cuda.synchronize()
            ctx.project_fp8(qc, qs, *layer.out, out=y)
            if wait:
                torch.cuda.synchronize()
            outs.append(y.clone())
        s = step(ctx, layer, plan, T, y, residual, ic.clone(), lc.clone())
        torch.cuda.synchronize()
        return outs + [residual, s["y"], s["c2"], s["res2"]]

    want = run(True)
    for _ in range(5):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [3, 40, 100, 300])
def test_buffers_rewritten_call_after_call(built, rows):
    """Codes, scales and rows written and read again and again in the same
    buffers by launches that overlap, on few enough CTAs for three of them to be
    on the card at once."""
    ctx = dsa.Context(W.DSAShape(**W.DEEPSEEK), 0)
    g = torch.Generator().manual_seed(rows)
    w = ctx.quantize_weight((torch.randn(256, 1024, generator=g) / 32).to(BF16).cuda())
    back = ctx.quantize_weight((torch.randn(1024, 256, generator=g) / 16).to(BF16).cuda())
    xs = [(torch.randn(rows, 1024, generator=g) * (i + 1)).to(BF16).cuda() for i in range(8)]

    codes, scales = torch.empty(rows, 1024, dtype=torch.uint8, device="cuda"), torch.empty(rows, 8, device="cuda")
    yc, ys = torch.empty(rows, 256, dtype=torch.uint8, device="cuda"), torch.empty(rows, 2, device="cuda")
    y, h = torch.empty(rows, 256, dtype=F32, device="cuda"), torch.empty(rows, 1024, dtype=BF16, device="cuda")
    res = torch.empty(rows, 1024, dtype=BF16, device="cuda")
    outs = [torch.empty(rows, 256, dtype=F32, device="cuda") for _ in range(64)]

    def body(wait=False):
        h.zero_()
        res.zero_()
        for i in range(64):
            for call in (lambda: ctx.rmsnorm_quantize(xs[i % 8] if i % 3 else h, None, residual=res if i % 8 else xs[i % 8],
                                                      residual_out=res, codes=codes, scales=scales),
                         lambda: ctx.project_fp8(codes, scales, *w, out=y),
                         lambda: ctx.quantize_rows(y, yc, ys),
                         lambda: ctx.project_fp8(yc, ys, *back, out=h),
                         lambda: ctx.project_fp8(codes, scales, *w, out=outs[i])):
                call()
                if wait:
                    torch.cuda.synchronize()

    def results():
        torch.cuda.synchronize()
        ctx.get_error()
        return [t.clone() for t in outs + [res, h]]

    body(wait=True)
    want = results()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        body()
    for go in [body] * 4 + [g.replay] * 4:
        for t in outs:
            t.fill_(-1)
        go()
        for i, (a, b) in enumerate(zip(results(), want)):
            assert torch.equal(a, b), (go, i)


def test_a_captured_layer_replays_over_rewritten_spans(built):
    """The whole step on a capturable plan in one graph: replays over two
    different steps (fewer rows, then more) equal the eager calls, and the rows
    behind the step's last stay as they were."""
    wl = H.deepseek_small(seed=73, fp8=True, decode_ctx=(2500, 300, 4001, 900, 2049), chunk=None)
    ctx = dsa.Context(wl.shape, 0)
    cap = 8
    layer = Layer(ctx, 5)
    total = 8 * 6000
    plan = ctx.plan_capturable(cap, cap, total, wl.num_pages)
    pages = torch.from_numpy(np.concatenate([np.asarray(s.pages, np.int32) for s in wl.spans])).cuda()
    offs = np.cumsum([0] + [len(s.pages) for s in wl.spans])
    table = np.zeros((cap, 6), np.int32)
    for i, s in enumerate(wl.spans):
        table[i] = [1, s.ctx_start, s.page_start, offs[i], len(s.pages), 0]
    count = torch.tensor([5], dtype=torch.int32, device="cuda")
    spans = torch.from_numpy(table).cuda()
    x, residual = inputs(cap, 6)
    ic0, lc0 = W.make_index_cache(wl).cuda(), W.make_latent_cache(wl).cuda()
    ic, lc = ic0.clone(), lc0.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ctx.plan_update(plan, count, spans, pages)
        step(ctx, layer, plan, cap, x, residual, ic, lc, padded=plan)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ctx.plan_update(plan, count, spans, pages)
        got = step(ctx, layer, plan, cap, x, residual, ic, lc, padded=plan)
    for live, seed in ((5, 7), (2, 8), (4, 9)):
        count.fill_(live)
        nx, nr = inputs(cap, seed)
        x.copy_(nx)
        residual.copy_(nr)
        ic.copy_(ic0)
        lc.copy_(lc0)
        for t in (got["y"], got["c2"], got["res2"], got["v"]):
            t.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        ctx.get_error()
        kept = {k: got[k].clone() for k in ("y", "c2", "s2", "res2", "v")}
        ic.copy_(ic0)
        lc.copy_(lc0)
        want = step(ctx, layer, plan, cap, x, residual, ic, lc, padded=plan)
        for k in kept:
            assert torch.equal(kept[k][:live], want[k][:live]), k
        for k in ("y", "c2", "res2", "v"):
            assert (kept[k][live:] == 77).all(), k
    ctx.get_error()
