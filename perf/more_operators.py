"""Cases for the operators between a layer's projections and its paged caches:
the rotation of queries by their positions (``rotary``), the append of a step's
latents, index keys, keys and values to the caches with the rotation applied on
the way (``append_latents``, ``append_kv``), and the attention of a batch whose
requests share a long prefix, which reads the shared pages once for all of them
(``prefix_attend``).

A rotation takes pairs of columns (x, y) to (x cos t - y sin t, x sin t + y cos t)
with t = position * frequency: neighbouring columns where the layout is
"interleaved", columns half the rotated width apart where it is "half".
Frequencies are base ** (-2 i / rot), or that stretched for long contexts by
YaRN: slow pairs divided by a factor, fast ones kept, and a linear ramp between.
Index rows and latents in 8 bits are e4m3 codes with an fp32 scale (amax / 448,
or 1) for each 128 columns; codes are returned as float8 tensors, beside their
scales.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
BASE = 10000.0
FP8 = torch.float8_e4m3fn
YARN = dict(factor=40.0, original_context=4096, beta_fast=32.0, beta_slow=1.0)
AMPLITUDE = 0.1 * math.log(40.0) + 1.0


def listed():
    return [
        # the queries of one token: the 64 rotated columns behind each head's 128 others, 128 heads
        dict(name="rotate one token", op="rotary", rows=1, heads=128, width=64, stride=192, offset=0, rot=64,
             layout="interleaved", scaled=True, far=131072, type="bf16", inverse=False),
        # the same of a prefill chunk
        dict(name="rotate prefill", op="rotary", rows=8192, heads=128, width=64, stride=192, offset=0, rot=64,
             layout="interleaved", scaled=True, far=16384, type="bf16", inverse=False),
        # the indexer's queries of a prefill chunk: the first 64 of 128 columns, the others carried over
        dict(name="rotate index queries", op="rotary", rows=4096, heads=64, width=128, stride=128, offset=0, rot=64,
             layout="half", scaled=True, far=16384, type="bf16", inverse=False),
        # a ragged step's projected queries still in 32 bits, turned back
        dict(name="rotate back ragged", op="rotary", rows=1031, heads=64, width=128, stride=128, offset=0, rot=128,
             layout="half", scaled=False, far=1000000, type="fp32", inverse=True),
        # a decode step of 128 sequences: latent and index key of each
        dict(name="append decode", op="latents", requests=128, new=1, far=131072, fp8=False, scaled=True),
        # a prefill chunk into the 8-bit caches
        dict(name="append prefill 8 bit", op="latents", requests=2, new=4096, far=16384, fp8=True, scaled=True),
        # keys and values of a step of ragged chunks, 4 heads of 128
        dict(name="append keys and values", op="kv", requests=7, new=1171, far=32768, kv_heads=4, rot=128,
             layout="half", scaled=False),
        # a few sequences that decode after a short common prompt: latency
        dict(name="prefix few", op="prefix", groups=1, requests=4, new=1, prefix=1024, own_lo=1, own_hi=200,
             q_heads=64, kv_heads=4),
        # a decode step of 32 sequences after a long system prompt
        dict(name="prefix decode", op="prefix", groups=1, requests=32, new=1, prefix=8192, own_lo=64, own_hi=1024,
             q_heads=64, kv_heads=4),
        # two long documents with 128 sequences on each
        dict(name="prefix batch", op="prefix", groups=2, requests=256, new=1, prefix=32768, own_lo=128, own_hi=2048,
             q_heads=64, kv_heads=4),
        # the questions to a long document, prefilled together
        dict(name="prefix prefill", op="prefix", groups=1, requests=16, new=128, prefix=16384, own_lo=128, own_hi=300,
             q_heads=64, kv_heads=4),
    ]


def _log(rng, lo, hi):
    """An integer of lo .. hi, spread over its logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "latents", "kv", "prefix", "prefix", "prefix"])
    if op == "rotary":
        rows, heads, rot = _log(rng, 1, 8192), _log(rng, 1, 128), rng.choice([16, 32, 64, 64, 96, 128])
        offset = rng.choice([0, 0, 8, 32, 33])
        width = offset + rot + rng.choice([0, 0, 32, 64, 1])
        while rows * heads * width > 8192 * 128 * 64:
            rows //= 2
        return dict(op=op, rows=rows, heads=heads, width=width, stride=width + rng.choice([0, 0, 64, 128, 3]), offset=offset,
                    rot=rot, layout=rng.choice(["interleaved", "half"]), scaled=rng.random() < 0.5,
                    far=_log(rng, 1024, 1000000), type=rng.choice(["bf16", "bf16", "fp32"]), inverse=rng.random() < 0.25)
    if op in ("latents", "kv"):
        requests = _log(rng, 1, 256)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, 8192 // requests))
        case = dict(op=op, requests=requests, new=new, far=_log(rng, 8192, 131072), scaled=rng.random() < 0.5)
        if op == "latents":
            case["fp8"] = rng.random() < 0.5
        else:
            case.update(kv_heads=rng.choice([1, 2, 4, 8]), rot=rng.choice([32, 64, 128]), layout=rng.choice(["interleaved", "half"]))
        return case
    q_heads, kv_heads = rng.choice([(64, 4), (64, 4), (64, 8), (32, 8), (16, 1), (12, 4), (8, 8), (40, 8)])
    requests, new = _log(rng, 1, 256), rng.choice([1, 1, 1, 1, 2, 5, 16, 64, 128])
    prefix, own_lo = 64 * _log(rng, 1, 512), _log(rng, 1, 512)
    own_hi = own_lo + _log(rng, 1, 2048)
    while requests * new * q_heads * (prefix + own_hi + new) > 2048 * 64 * 16384:
        requests = max(1, requests // 2)
        prefix = max(64, prefix // 128 * 64)
    return dict(op=op, groups=rng.choice([1, 1, 2, 3]) if requests >= 6 else 1, requests=requests, new=new, prefix=prefix,
                own_lo=own_lo, own_hi=own_hi, q_heads=q_heads, kv_heads=kv_heads)


def _own_lengths(c):
    """Each request's tokens behind the shared prefix before this step's, spread over own_lo - 1 .. own_hi."""
    return [c["own_lo"] - 1 + int((c["own_hi"] - c["own_lo"] + 1) * ((i * 0.6180339887 + 0.37) % 1.0)) for i in range(c["requests"])]


def _contexts(c):
    """Each request's tokens before this step's, up to `far`."""
    top = c["far"] - c["new"]
    return [int(top * (1.0 - 0.5 * ((i * 0.6180339887) % 1.0))) for i in range(c["requests"])]


def work(case):
    c = case
    if c["op"] == "rotary":
        values = c["rows"] * c["heads"] * c["width"]
        return {"bytes": (4 if c["type"] == "bf16" else 8) * values, "flops": 3 * c["rows"] * c["heads"] * c["rot"]}
    if c["op"] == "latents":
        rows = c["requests"] * c["new"]
        read = 2 * (512 + 64 + 128)
        return {"bytes": rows * (read + (656 + 132 if c["fp8"] else read)), "flops": rows * (3 * 128 + (4 * 640 if c["fp8"] else 0))}
    if c["op"] == "kv":
        rows = c["requests"] * c["new"]
        return {"bytes": rows * 2 * 2 * 2 * c["kv_heads"] * 128, "flops": rows * 3 * c["kv_heads"] * c["rot"]}
    rows, n = c["requests"] * c["new"], c["new"]
    lengths = _own_lengths(c)
    tokens = c["groups"] * c["prefix"] + sum(l + n for l in lengths)
    seen = rows * c["prefix"] + sum(n * l + n * (n + 1) // 2 for l in lengths)
    return {"bytes": 2 * 2 * rows * c["q_heads"] * 128 + tokens * 2 * 2 * c["kv_heads"] * 128,
            "flops": 4 * c["q_heads"] * 128 * seen}


# ---------------------------------------------------------------- inputs
class _Span:
    def __init__(self, q_start, q_len, ctx_start, pages):
        self.q_start, self.q_len, self.ctx_start, self.pages = q_start, q_len, ctx_start, pages


def _randn(rng, *shape):
    return torch.randn(*shape, device="cuda", generator=rng)


def _append_pages(rng, c):
    """Spans whose new rows lie in pages of their own; the pages of what came before are not touched, and all stand for page 0."""
    spans, where, used = [], [], 1
    contexts, q = _contexts(c), 0
    needed = sum((t + c["new"] - 1) // PAGE - t // PAGE + 1 for t in contexts)
    mixed = (torch.randperm(needed, device="cuda", generator=rng) + 1).cpu().numpy().astype(np.int32)
    for t in contexts:
        first, last = t // PAGE, (t + c["new"] - 1) // PAGE
        pages = np.zeros(last + 1, dtype=np.int32)
        pages[first:] = mixed[used - 1:used + last - first]
        used += last - first + 1
        spans.append(_Span(q, c["new"], t, pages))
        q += c["new"]
        at = np.arange(t, t + c["new"])
        where.append(np.stack((pages[at // PAGE], at % PAGE, at)))
    return spans, torch.from_numpy(np.concatenate(where, axis=1).astype(np.int64)).cuda(), needed + 1


def _prefix_pages(rng, c):
    """Spans in groups that share their first pages, the physical pages in any order."""
    shared, lengths = c["prefix"] // PAGE, _own_lengths(c)
    owned = [(l + c["new"] + PAGE - 1) // PAGE for l in lengths]
    total = c["groups"] * shared + sum(owned)
    mixed = torch.randperm(total, device="cuda", generator=rng).cpu().numpy().astype(np.int32)
    spans, at, q = [], c["groups"] * shared, 0
    for i, l in enumerate(lengths):
        g = i * c["groups"] // c["requests"]
        pages = np.concatenate((mixed[g * shared:(g + 1) * shared], mixed[at:at + owned[i]]))
        spans.append(_Span(q, c["new"], c["prefix"] + l, pages))
        at += owned[i]
        q += c["new"]
    return spans, total


def prepare(case, seed):
    c = case
    rng = torch.Generator(device="cuda")
    rng.manual_seed(seed)
    s = {"case": c}
    bf16 = torch.bfloat16
    if c["op"] == "rotary":
        x = _randn(rng, c["rows"], c["heads"], c["stride"])
        x = x.to(bf16) if c["type"] == "bf16" else x
        s["x"] = x[..., c["stride"] - c["width"]:]
        start = c["far"] - c["rows"] if c["far"] > c["rows"] else 0
        s["positions"] = torch.arange(start, start + c["rows"], device="cuda", dtype=torch.int32)
        if c["rows"] < 512:   # a decode step's: each of its own sequence
            s["positions"] = torch.randint(0, c["far"], (c["rows"],), device="cuda", generator=rng, dtype=torch.int32)
    elif c["op"] in ("latents", "kv"):
        s["spans"], where, s["pages"] = _append_pages(rng, c)
        s["page"], s["slot"], s["positions"] = where
        rows = c["requests"] * c["new"]
        if c["op"] == "kv":
            h = c["kv_heads"]
            s["k"], s["v"] = _randn(rng, rows, h, 128).to(bf16), _randn(rng, rows, h, 128).to(bf16)
            s["cache"] = torch.zeros(s["pages"], PAGE, 2 * h * 128, device="cuda", dtype=bf16)
            s["held"] = (s["cache"],)
        else:
            # the fused down projection's columns: latent (normed into a tensor of its own), rope, index key
            s["c"] = (0.5 * _randn(rng, rows, 512)).to(bf16)
            down = _randn(rng, rows, 704).to(bf16)
            s["k_pe"], s["keys"] = down[:, 512:576], down[:, 576:]
            if c["fp8"]:
                lat = torch.zeros(s["pages"], PAGE, 656, device="cuda", dtype=torch.uint8)
                idx = torch.zeros(s["pages"], PAGE * 132, device="cuda", dtype=torch.uint8)
                s["held"] = (lat[..., :512].view(FP8), lat[..., 512:528].view(torch.float32), lat[..., 528:].view(bf16),
                             idx[:, :PAGE * 128].view(FP8).unflatten(1, (PAGE, 128)), idx[:, PAGE * 128:].view(torch.float32))
            else:
                lat = torch.zeros(s["pages"], PAGE, 576, device="cuda", dtype=bf16)
                idx = torch.zeros(s["pages"], PAGE, 128, device="cuda", dtype=bf16)
                s["held"] = (lat, idx)
            s["cache"], s["index_cache"] = lat, idx
    else:
        s["spans"], s["pages"] = _prefix_pages(rng, c)
        s["q"] = _randn(rng, c["requests"] * c["new"], c["q_heads"], 128).to(bf16)
        s["cache"] = torch.empty(s["pages"], PAGE, 2 * c["kv_heads"] * 128, device="cuda", dtype=bf16).normal_(0, 0.5, generator=rng)
        shared, n = c["prefix"] // PAGE, c["requests"]
        heads = [s["spans"][-(-g * n // c["groups"])] for g in range(c["groups"])]
        s["shared_pages"] = torch.from_numpy(np.stack([h.pages[:shared] for h in heads])).cuda().long()
        most = max(len(sp.pages) for sp in s["spans"])
        padded = np.stack([np.pad(sp.pages, (0, most - len(sp.pages)), mode="edge")[shared:] for sp in s["spans"]])
        s["own_pages"] = torch.from_numpy(padded).cuda().long()
        s["own_start"] = torch.tensor([sp.ctx_start - c["prefix"] for sp in s["spans"]], device="cuda")
    if own:
        _plan(s)
    return s


# ---------------------------------------------------------------- the framework's operators
_held = {}


def _context(fp8=False):
    """The program's context of these cache formats, made once and kept."""
    if fp8 not in _held:
        from deepseek_sparse_attention_dsa_gb300 import dsa, workloads
        shape = workloads.DSAShape(**dict(workloads.DEEPSEEK, page_size=PAGE))
        if fp8:
            shape.latent_fmt, shape.index_fmt = workloads.LATENT_FP8_656, workloads.INDEX_FP8_132
        _held[fp8] = dsa.Context(shape, 0)
    return _held[fp8]


def _table(rot, scaled):
    """A model's frequencies, laid out once."""
    if (rot, scaled) not in _held:
        ctx = _context()
        _held[rot, scaled] = (ctx.rotary_table(rot, base=BASE, scaling="yarn", amplitude=AMPLITUDE, **YARN) if scaled
                              else ctx.rotary_table(rot, base=BASE))
    return _held[rot, scaled]


def _msa(q_heads, kv_heads):
    from deepseek_sparse_attention_dsa_gb300 import workloads
    return workloads.MSAShape(page_size=PAGE, q_heads=q_heads, kv_heads=kv_heads)


def _plan(s):
    """The step's plan, made once for all of a model's layers."""
    c = s["case"]
    if "spans" in s and "plan" not in s:
        ctx = _context(c.get("fp8", False))
        s["ctx"], s["plan"] = ctx, ctx.plan(s["spans"], s["pages"])
        if c["op"] == "prefix":
            s["prefixes"] = ctx.plan_prefix(s["plan"], _msa(c["q_heads"], c["kv_heads"]))
        elif c["op"] == "kv":
            s["msa"] = _msa(c["kv_heads"], c["kv_heads"])


def _run_own(s):
    c = s["case"]
    if c["op"] == "rotary":
        return _context().rotary(_table(c["rot"], c["scaled"]), s["x"], s["positions"], offset=c["offset"],
                                 layout=c["layout"], inverse=c["inverse"])
    if "plan" not in s:
        _plan(s)
    if c["op"] == "latents":
        s["ctx"].append_latents(s["plan"], _table(64, c["scaled"]), s["c"], s["k_pe"], s["cache"], keys=s["keys"],
                                index_cache=s["index_cache"], layout="interleaved", key_layout="half")
        return s["held"]
    if c["op"] == "kv":
        s["ctx"].append_kv(s["plan"], s["msa"], _table(c["rot"], c["scaled"]), s["k"], s["v"], s["cache"], layout=c["layout"])
        return s["held"]
    return s["ctx"].prefix_attend(s["prefixes"], s["q"], s["cache"])


# ---------------------------------------------------------------- the plain forms
def _frequencies(rot, scaled):
    """The rot / 2 frequencies in 64 bits."""
    f = torch.arange(0, rot, 2, device="cuda", dtype=torch.float64)
    f = BASE ** (-f / rot)
    if not scaled:
        return f
    # the pair that turns `turns` times over the original context
    low, high = (rot * math.log(YARN["original_context"] / (turns * 2 * math.pi)) / (2 * math.log(BASE))
                 for turns in (YARN["beta_fast"], YARN["beta_slow"]))
    low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
    ramp = ((torch.arange(rot // 2, device="cuda", dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
    return f * (1 - ramp) + f / YARN["factor"] * ramp


def _turned(x, positions, offset, rot, layout, scaled, inverse=False):
    """x (rows, heads, width) in 32 bits with its columns offset .. offset + rot rotated; angles in 64 bits."""
    angle = positions.double()[:, None] * _frequencies(rot, scaled)
    amplitude = AMPLITUDE if scaled else 1.0
    cos, sin = (torch.cos(angle) * amplitude).float()[:, None], (torch.sin(angle) * amplitude).float()[:, None]
    if inverse:
        sin = -sin
    part = x[..., offset:offset + rot].float()
    if layout == "interleaved":
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((x[..., :offset].float(), part, x[..., offset + rot:].float()), dim=-1)


def _plain_codes(x):
    """(codes, scales) of x (rows, whole groups of 128)."""
    t = x.unflatten(1, (-1, 128))
    amax = t.abs().amax(dim=2)
    scale = torch.where(amax > 0, amax / 448.0, 1.0)
    return (t / scale[..., None]).to(FP8).flatten(1), scale


def _run_plain(s):
    c = s["case"]
    if c["op"] == "rotary":
        return _turned(s["x"], s["positions"], c["offset"], c["rot"], c["layout"], c["scaled"], c["inverse"]).to(s["x"].dtype)
    if c["op"] == "kv":
        k = _turned(s["k"], s["positions"], 0, c["rot"], c["layout"], c["scaled"])
        s["cache"][s["page"], s["slot"]] = torch.cat((k.flatten(1).to(torch.bfloat16), s["v"].flatten(1)), dim=1)
        return s["held"]
    if c["op"] == "latents":
        k_pe = _turned(s["k_pe"][:, None], s["positions"], 0, 64, "interleaved", c["scaled"])[:, 0]
        keys = _turned(s["keys"][:, None], s["positions"], 0, 64, "half", c["scaled"])[:, 0]
        at = s["page"], s["slot"]
        if not c["fp8"]:
            s["cache"][at] = torch.cat((s["c"], k_pe.to(torch.bfloat16)), dim=1)
            s["index_cache"][at] = keys.to(torch.bfloat16)
            return s["held"]
        codes, scale = _plain_codes(s["c"].float())
        key_codes, key_scale = _plain_codes(keys)
        lat, lat_scale, rope, idx, idx_scale = s["held"]
        lat.view(torch.uint8)[at], lat_scale[at], rope[at] = codes.view(torch.uint8), scale, k_pe.to(torch.bfloat16)
        idx.view(torch.uint8)[at], idx_scale[at] = key_codes.view(torch.uint8), key_scale[:, 0]
        return s["held"]
    # attention: the logits of the shared prefix for all of a group's rows in one product, those of each request's own
    # tokens in a padded batch, one softmax over both
    n, h, group = c["new"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    scale, parts = 128 ** -0.5, []
    for g in range(c["groups"]):
        lo, hi = -(-g * c["requests"] // c["groups"]), -(-(g + 1) * c["requests"] // c["groups"])
        b = hi - lo
        if b == 0:
            continue
        q = s["q"].view(c["requests"], n, h, group, 128)[lo:hi].float()
        own_kv = s["cache"][s["own_pages"][lo:hi]].flatten(1, 2).unflatten(2, (2, h, 128))      # (b, own, 2, h, 128)
        seen = s["own_start"][lo:hi, None] + torch.arange(n, device="cuda")                    # (b, n)
        hidden = torch.arange(own_kv.shape[1], device="cuda") > seen[..., None]                # (b, n, own)
        shared_kv = s["cache"][s["shared_pages"][g]].flatten(0, 1).unflatten(1, (2, h, 128))
        out = torch.empty(b, n, h, group, 128, device="cuda", dtype=torch.bfloat16)
        for i in range(h):
            qi = q[:, :, i]                                                                   # (b, n, group, 128)
            ks, vs = shared_kv[:, 0, i].float(), shared_kv[:, 1, i].float()
            ko, vo = own_kv[:, :, 0, i].float(), own_kv[:, :, 1, i].float()
            ls = (qi.reshape(-1, 128) @ ks.t() * scale).view(b, n, group, -1)
            lo_ = torch.bmm(qi.reshape(b, n * group, 128), ko.transpose(1, 2)).view(b, n, group, -1) * scale
            lo_ = lo_.masked_fill(hidden[:, :, None], float("-inf"))
            top = torch.maximum(ls.amax(-1), lo_.amax(-1))[..., None]
            ls, lo_ = torch.exp(ls - top), torch.exp(lo_ - top)
            total = ls.sum(-1) + lo_.sum(-1)
            o = (ls.view(-1, ls.shape[-1]) @ vs).view(b, n, group, 128)
            o = o + torch.bmm(lo_.view(b, n * group, -1), vo).view(b, n, group, 128)
            out[:, :, i] = (o / total[..., None]).to(torch.bfloat16)
        parts.append(out.view(b * n, c["q_heads"], 128))
    return torch.cat(parts)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- the definitions, in 64 bits
def _exact_turn(x, positions, offset, rot, layout, scaled, sign=1.0):
    """The rotation as a complex product, pair by pair."""
    y = x.double().clone()
    for i in range(rot // 2):
        f = BASE ** (-2.0 * i / rot)
        if scaled:
            def border(turns):
                return rot * math.log(YARN["original_context"] / (turns * 2 * math.pi)) / (2 * math.log(BASE))
            a, b = max(math.floor(border(YARN["beta_fast"])), 0), min(math.ceil(border(YARN["beta_slow"])), rot - 1)
            slow = min(max((i - a) / ((b - a) or 0.001), 0.0), 1.0)
            f = slow * f / YARN["factor"] + (1.0 - slow) * f
        one, two = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rot // 2)
        z = torch.complex(x[..., offset + one].double(), x[..., offset + two].double())
        t = sign * f * positions.double()
        w = torch.polar(torch.full_like(t, AMPLITUDE if scaled else 1.0), t)
        z = z * w.view(-1, *[1] * (z.dim() - 1))
        y[..., offset + one], y[..., offset + two] = z.real, z.imag
    return y


def _exact_codes(y):
    """The quotients that the codes round, and the scales."""
    scale = torch.stack([y[:, j:j + 128].abs().amax(1) for j in range(0, y.shape[1], 128)], dim=1) / 448.0
    scale[scale == 0] = 1.0
    return y / scale.repeat_interleave(128, dim=1), scale


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rotary":
        return _exact_turn(s["x"], s["positions"], c["offset"], c["rot"], c["layout"], c["scaled"], -1.0 if c["inverse"] else 1.0)
    if c["op"] == "prefix":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        group, n = c["q_heads"] // c["kv_heads"], c["new"]
        for sp in s["spans"]:
            end = sp.ctx_start + n
            kv = s["cache"][torch.from_numpy(sp.pages).cuda().long()].view(-1, 2, c["kv_heads"], 128)[:end]
            late = torch.arange(end, device="cuda")[None] > sp.ctx_start + torch.arange(n, device="cuda")[:, None]
            for i in range(c["kv_heads"]):
                rows = slice(sp.q_start, sp.q_start + n), slice(i * group, (i + 1) * group)
                logits = torch.einsum("nhd,td->hnt", s["q"][rows].double(), kv[:, 0, i].double()) / math.sqrt(128.0)
                weights = torch.softmax(logits.masked_fill_(late, -math.inf), dim=-1)
                out[rows] = torch.einsum("hnt,td->nhd", weights, kv[:, 1, i].double())
        return out
    where = s["page"] * PAGE + s["slot"]
    held = [torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in s["held"]]

    def put(i, rows):
        held[i].view(s["pages"] * PAGE, -1)[where] = rows

    if c["op"] == "kv":
        k = _exact_turn(s["k"], s["positions"], 0, c["rot"], c["layout"], c["scaled"])
        put(0, torch.cat((k.flatten(1), s["v"].double().flatten(1)), dim=1))
        return tuple(held)
    k_pe = _exact_turn(s["k_pe"], s["positions"], 0, 64, "interleaved", c["scaled"])
    keys = _exact_turn(s["keys"], s["positions"], 0, 64, "half", c["scaled"])
    if not c["fp8"]:
        put(0, torch.cat((s["c"].double(), k_pe), dim=1))
        put(1, keys)
        return tuple(held)
    codes, scale = _exact_codes(s["c"].double())
    key_codes, key_scale = _exact_codes(keys)
    for i, rows in enumerate((codes, scale, k_pe, key_codes, key_scale)):
        put(i, rows)
    return tuple(held)
