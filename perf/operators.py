"""Cases for the operators around the sparse attention that work in 8 bits: the
root-mean-square norm with the residual's addition (``rmsnorm``), the matrix
product of e4m3 codes with a scale for each block of 128 (``project_fp8``), and
the two quantisers that feed it (``quantize_rows``, ``quantize_weight``).

An 8-bit value is an e4m3 code times the fp32 scale of its group: 128 columns
of a row for activations, a block of 128 x 128 for weights.  A group's scale is
amax / 448, or 1 where the group is all zero; a code is the quotient by it
rounded to nearest even.  Codes are returned as float8 tensors, beside their
scales.
"""
import torch

own = False

GROUP = 128
FP8 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # the norm before a layer's projections, one sequence decoding: one launch's latency
        dict(name="norm one token", op="norm", rows=1, width=5120, stride=5120, residual=True, out="codes"),
        # the latents' norm of a prefill chunk: 512 columns inside the rows of the fused down projection (512 + 64
        # latent and rope columns, 128 index key columns)
        dict(name="norm latents", op="norm", rows=4096, width=512, stride=704, residual=False, out="bf16"),
        # a prefill chunk's norm with its residual
        dict(name="norm prefill", op="norm", rows=8192, width=4096, stride=4096, residual=True, out="codes"),
        # the indexer's query of one token (64 heads of 128)
        dict(name="project one token", op="project", rows=1, batch=1, n=8192, k=2048, out="bf16"),
        # the same projection of a decode step of 128 sequences
        dict(name="project decode", op="project", rows=128, batch=1, n=8192, k=4096, out="bf16"),
        # the fused down projection (latent, rope and index key columns) of a ragged chunk, kept in 32 bits
        dict(name="project ragged", op="project", rows=1031, batch=1, n=704, k=5120, out="fp32"),
        # each of 128 heads' values out of its 512 latent columns
        dict(name="project heads", op="project", rows=256, batch=128, n=128, k=512, out="bf16"),
        # a prefill chunk
        dict(name="project prefill", op="project", rows=8192, batch=1, n=8192, k=4096, out="bf16"),
        # the attention's output (128 heads of 512) of a decode step, on its way into a projection
        dict(name="quantize decode rows", op="rows", rows=128, width=65536, stride=65536),
        # and of a prefill chunk
        dict(name="quantize prefill rows", op="rows", rows=2048, width=65536, stride=65536),
        # a layer's weights when a model is loaded
        dict(name="quantize weight", op="weight", n=8192, k=4096, source="bf16"),
        # the fused down projection's, from a 32-bit checkpoint
        dict(name="quantize ragged weight", op="weight", n=704, k=5120, source="fp32"),
    ]


def _log(rng, lo, hi):
    """An integer of lo .. hi, spread over its logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["norm", "project", "project", "heads", "rows", "weight"])
    if op == "norm":
        rows = _log(rng, 1, 8192)
        width = _log(rng, 128, 8192)
        width -= rng.choice([0, width % 8, width % 128])   # any width, whole 16-byte pieces, whole groups
        while rows * width > 8192 * 4096:
            rows //= 2
        return dict(op=op, rows=rows, width=width, stride=width + rng.choice([0, 0, 64, 3]),
                    residual=rng.random() < 0.6, out=rng.choice(["codes", "codes", "bf16"]))
    if op == "project":
        n, k = _log(rng, 64, 8192), _log(rng, 128, 8192)
        n -= rng.choice([0, n % 8, n % 64])
        k -= k % 16 if k < 256 else rng.choice([k % 16, k % 128])
        rows = _log(rng, 1, 8192)
        while rows * n * k > 8192 * 8192 * 4096:
            rows //= 2
        return dict(op=op, rows=rows, batch=1, n=n, k=k, out=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "heads":
        n, k = rng.choice([(128, 512), (512, 128), (64, 256), (256, 64), (192, 576)])
        return dict(op="project", rows=_log(rng, 1, 1024), batch=rng.choice([8, 16, 31, 64, 128]), n=n, k=k, out="bf16")
    if op == "rows":
        rows, width = _log(rng, 1, 4096), _log(rng, 128, 65536)
        width -= rng.choice([0, width % 8, width % 128])
        while rows * width > 2048 * 65536:
            rows //= 2
        return dict(op=op, rows=rows, width=width, stride=width + rng.choice([0, 0, 64, 5]))
    n, k = _log(rng, 64, 8192), _log(rng, 128, 8192)
    k -= rng.choice([0, k % 8, k % 128])
    return dict(op=op, n=n, k=k, source=rng.choice(["bf16", "bf16", "fp32"]))


def _groups(k):
    return (k + GROUP - 1) // GROUP


def _work_codes(rows, width):
    return rows * width + 4 * rows * _groups(width)


def work(case):
    c = case
    if c["op"] == "norm":
        values = c["rows"] * c["width"]
        moved = 2 * values + 2 * c["width"] + (4 * values if c["residual"] else 0)
        moved += _work_codes(c["rows"], c["width"]) if c["out"] == "codes" else 2 * values
        return {"bytes": moved, "flops": 6 * values}
    if c["op"] == "project":
        m, b, n, k = c["rows"], c["batch"], c["n"], c["k"]
        moved = _work_codes(m * b, k) + b * (n * k + 4 * _groups(n) * _groups(k))
        moved += m * b * n * (2 if c["out"] == "bf16" else 4)
        return {"bytes": moved, "flops": 2 * m * b * n * k}
    if c["op"] == "rows":
        values = c["rows"] * c["width"]
        return {"bytes": 2 * values + _work_codes(c["rows"], c["width"]), "flops": 4 * values}
    values = c["n"] * c["k"]
    read = (2 if c["source"] == "bf16" else 4) * values
    return {"bytes": read + values + 4 * _groups(c["n"]) * _groups(c["k"]), "flops": 4 * values}


def _activations(rng, rows, width):
    """Activations as a layer sees them: each row of its own size, some columns far larger than the others."""
    x = torch.randn(rows, width, device="cuda", generator=rng)
    x *= torch.rand(rows, 1, device="cuda", generator=rng) + 0.5
    x *= torch.where(torch.rand(width, device="cuda", generator=rng) < 0.01, 20.0, 1.0)
    return x


def _made_codes(x, group_rows):
    """Codes and scales of x (batch, rows, width) in groups of group_rows x 128, as a program holds them."""
    b, r, w = x.shape
    pad_r, pad_w = -r % group_rows, -w % GROUP
    t = torch.nn.functional.pad(x, (0, pad_w, 0, pad_r))
    t = t.view(b, (r + pad_r) // group_rows, group_rows, (w + pad_w) // GROUP, GROUP)
    amax = t.abs().amax(dim=(2, 4), keepdim=True)
    scale = torch.where(amax > 0, amax / 448.0, 1.0)
    codes = (t / scale).clamp(-448.0, 448.0).to(FP8).view(b, r + pad_r, w + pad_w)[:, :r, :w].contiguous()
    return codes, scale.view(b, (r + pad_r) // group_rows, (w + pad_w) // GROUP).contiguous()


def prepare(case, seed):
    c = case
    rng = torch.Generator(device="cuda")
    rng.manual_seed(seed)
    state = {"case": c}
    if c["op"] == "norm":
        wide = _activations(rng, c["rows"], c["stride"]).to(torch.bfloat16)
        state["x"] = wide[:, :c["width"]]
        state["weight"] = (1.0 + 0.2 * torch.randn(c["width"], device="cuda", generator=rng)).to(torch.bfloat16)
        if c["residual"]:
            state["residual"] = (4.0 * _activations(rng, c["rows"], c["width"])).to(torch.bfloat16)
    elif c["op"] == "project":
        m, b, n, k = c["rows"], c["batch"], c["n"], c["k"]
        a, a_scale = _made_codes(_activations(rng, m * b, k).view(1, m * b, k), 1)
        w, w_scale = _made_codes(torch.randn(b, n, k, device="cuda", generator=rng) / k ** 0.5, GROUP)
        if b > 1:
            state.update(a=a.view(m, b, k), a_scale=a_scale.view(m, b, -1), w=w, w_scale=w_scale)
        else:
            state.update(a=a.view(m, k), a_scale=a_scale.view(m, -1), w=w[0], w_scale=w_scale[0])
    elif c["op"] == "rows":
        state["x"] = _activations(rng, c["rows"], c["stride"]).to(torch.bfloat16)[:, :c["width"]]
    else:
        w = torch.randn(c["n"], c["k"], device="cuda", generator=rng) / c["k"] ** 0.5
        state["w"] = w.to(torch.bfloat16) if c["source"] == "bf16" else w
    return state


# ---------------------------------------------------------------- the framework's operators
_held = []


def _context():
    """The program's context, made once and kept."""
    if not _held:
        from deepseek_sparse_attention_dsa_gb300 import dsa, workloads
        _held.append(dsa.Context(workloads.DSAShape(**workloads.DEEPSEEK), 0))
    return _held[0]


def _run_own(s):
    ctx, c = _context(), s["case"]
    if c["op"] == "norm":
        if c["out"] == "bf16":
            got = ctx.rmsnorm(s["x"], s["weight"], EPS, residual=s.get("residual"))
        else:
            got = ctx.rmsnorm_quantize(s["x"], s["weight"], EPS, residual=s.get("residual"))
            got = (got[0].view(FP8),) + got[1:]
        return got
    if c["op"] == "project":
        return ctx.project_fp8(s["a"], s["a_scale"], s["w"], s["w_scale"],
                               out_dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    codes, scale = ctx.quantize_rows(s["x"]) if c["op"] == "rows" else ctx.quantize_weight(s["w"])
    return codes.view(FP8), scale


# ---------------------------------------------------------------- the plain forms, in 32 bits
def _plain_codes(y, group_rows):
    """(codes, scales) of y (rows, width) in groups of group_rows x 128."""
    r, w = y.shape
    if r % group_rows or w % GROUP:
        whole = y.new_zeros(r + -r % group_rows, w + -w % GROUP)
        whole[:r, :w] = y
    else:
        whole = y
    t = whole.view(whole.shape[0] // group_rows, group_rows, whole.shape[1] // GROUP, GROUP)
    amax = t.abs().amax(dim=(1, 3))
    scale = torch.where(amax > 0, amax / 448.0, 1.0)
    codes = (t / scale[:, None, :, None]).to(FP8).view(whole.shape)[:r, :w].contiguous()
    return codes, scale


def _plain_values(codes, scale, group_rows):
    """The 32-bit values of codes (..., rows, width)."""
    spread = scale.repeat_interleave(GROUP, dim=-1)[..., :codes.shape[-1]]
    if group_rows > 1:
        spread = spread.repeat_interleave(group_rows, dim=-2)[..., :codes.shape[-2], :]
    return codes.float() * spread


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        h = s["x"].float()
        if c["residual"]:
            h = h + s["residual"].float()
        y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
        got = _plain_codes(y, 1) if c["out"] == "codes" else (y.to(torch.bfloat16),)
        if c["residual"]:
            return got + (h.to(torch.bfloat16),)
        return got if c["out"] == "codes" else got[0]
    if c["op"] == "project":
        a, w = _plain_values(s["a"], s["a_scale"], 1), _plain_values(s["w"], s["w_scale"], GROUP)
        if c["batch"] > 1:
            out = torch.bmm(a.transpose(0, 1), w.transpose(1, 2)).transpose(0, 1).contiguous()
        else:
            out = a @ w.t()
        return out.to(torch.bfloat16) if c["out"] == "bf16" else out
    if c["op"] == "rows":
        return _plain_codes(s["x"].float(), 1)
    return _plain_codes(s["w"].float(), GROUP)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- the definitions, in 64 bits
def _exact_codes(y, rows_of, cols_of):
    """The quotients that the codes round, and the scales; rows_of and cols_of say which group each row and column is in."""
    top = y.new_zeros(int(rows_of[-1]) + 1, y.shape[1])
    top.scatter_reduce_(0, rows_of[:, None].expand_as(y), y.abs(), "amax")
    amax = top.new_zeros(top.shape[0], int(cols_of[-1]) + 1)
    amax.scatter_reduce_(1, cols_of[None, :].expand_as(top), top, "amax")
    scale = amax / 448.0
    scale[amax == 0] = 1.0
    return y / scale[rows_of][:, cols_of], scale


def _index(n, group):
    return torch.arange(n, device="cuda") // group


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        h = s["x"].double()
        if c["residual"]:
            h += s["residual"].double()
        y = h / torch.sqrt((h * h).sum(1) / c["width"] + EPS)[:, None]
        y *= s["weight"].double()
        got = _exact_codes(y, _index(c["rows"], 1), _index(c["width"], GROUP)) if c["out"] == "codes" else (y,)
        if c["residual"]:
            return got + (h,)
        return got if c["out"] == "codes" else got[0]
    if c["op"] == "project":
        m, b, n, k = c["rows"], c["batch"], c["n"], c["k"]
        a, w = s["a"].double().view(m, b, k), s["w"].double().view(b, n, k)
        a_scale, w_scale = s["a_scale"].double().view(m, b, -1), s["w_scale"].double().view(b, _groups(n), -1)
        out = torch.zeros(m, b, n, dtype=torch.float64, device="cuda")
        for kb in range(_groups(k)):
            cols = slice(kb * GROUP, min(k, (kb + 1) * GROUP))
            part = torch.einsum("mbk,bnk->mbn", a[:, :, cols], w[:, :, cols])
            out += part * a_scale[:, :, kb, None] * w_scale[:, _index(n, GROUP), kb][None]
        return out if b > 1 else out[:, 0]
    if c["op"] == "rows":
        return _exact_codes(s["x"].double(), _index(c["rows"], 1), _index(c["width"], GROUP))
    return _exact_codes(s["w"].double(), _index(c["n"], GROUP), _index(c["k"], GROUP))
