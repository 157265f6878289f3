"""Measured cases of the operators in 8-bit floating point with a scale for each block of 128.

Codes are e4m3 (largest value 448).  Rows of activations have a scale for every 128 consecutive
columns, matrices one for every 128 x 128 elements; a block that ends at an edge is smaller.  A
block's scale is its largest magnitude / 448 (2^-126 at least), its codes value / scale rounded.

  norm     s = x + residual, y = s / rms(s) * gain with rms(s) = sqrt(mean(s^2) + eps), y rounded to
           16 bits or written as blocks; and its backward pass from dy and the gradient of s
  blocks   activations, or a matrix, written as blocks
  linear   y = x W^T with W held as blocks and x written as blocks in the call, or held so already;
           its input gradient dy W, with dy written as blocks
  grouped  the same with a matrix per expert, over rows sorted by expert (ragged groups)

``run`` computes them in elementary torch operations in 32 bits, or, where ``own`` is true,
through the package's entry points.  ``exact`` computes them in 64 bits by another route.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn


def _case(name, op, form, n, rows, cols, dtype, experts=1):
    c = {"op": op, "form": form, "n": n, "rows": rows, "cols": cols, "dtype": dtype,
         "experts": experts}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one sequence being generated, before a projection in 8 bits: the smallest call
        _case("norm 1x4096 blocks", "norm", "blocks", 1, 0, 4096, "bf16"),
        # a long prompt, before a projection in 8 bits
        _case("norm 8200x4096 blocks", "norm", "blocks", 8200, 0, 4096, "bf16"),
        # a training step, through the norm and the residual
        _case("norm grad 2000x4096", "norm", "backward", 2000, 0, 4096, "bf16"),
        # a long prompt's activations between two projections of an MLP
        _case("blocks 4096x12288", "blocks", "rows", 4096, 0, 12288, "bf16"),
        # a checkpoint's matrix, written as blocks once when it is loaded
        _case("blocks of 12288x4096", "blocks", "matrix", 0, 12288, 4096, "bf16"),
        # one sequence being generated, an MLP projection
        _case("linear 1x12288x4096", "linear", "forward", 1, 12288, 4096, "fp16"),
        # a batch of sequences being generated, an MLP's second projection, blocks in hand
        _case("linear 24x4096x12288", "linear", "forward blocks", 24, 4096, 12288, "bf16"),
        # a short prompt of an odd length
        _case("linear 333x4096x4096", "linear", "forward", 333, 4096, 4096, "fp16"),
        # a long prompt through an MLP projection after the norm's 8 bits: the largest call
        _case("linear 4096x12288x4096", "linear", "forward blocks", 4096, 12288, 4096, "bf16"),
        # a training step through a frozen projection
        _case("linear grad 2000x4096x4096", "linear", "backward", 2000, 4096, 4096, "bf16"),
        # eight tokens with eight experts each: few rows an expert, some experts none
        _case("grouped 64x1408x2048 E64", "grouped", "forward", 64, 1408, 2048, "bf16",
              experts=64),
        # a prompt through the same experts, groups of uneven sizes
        _case("grouped 8200x1408x2048 E64", "grouped", "forward", 8200, 1408, 2048, "bf16",
              experts=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "blocks", "linear", "linear", "grouped"])
    dtype = rng.choice(["bf16", "fp16"])

    def side(lo, hi):
        step = rng.choice([1, 8, 128])
        return max(step, _log_int(rng, lo, hi) // step * step)

    if op == "norm":
        cols = side(64, 16384)
        return _case(None, op, rng.choice(["blocks", "16 bits", "backward"]),
                     min(_log_int(rng, 1, 8200), 2 ** 25 // cols), 0, cols, dtype)
    if op == "blocks":
        cols = side(64, 16384)
        if rng.random() < 0.5:
            return _case(None, op, "rows", min(_log_int(rng, 1, 8200), 2 ** 25 // cols), 0, cols,
                         dtype)
        return _case(None, op, "matrix", 0, min(side(64, 16384), 2 ** 25 // cols), cols, dtype)
    form = rng.choice(["forward", "forward blocks", "backward"])
    if op == "grouped":
        return _case(None, op, form, _log_int(rng, 1, 8200), side(256, 2048), side(256, 2048),
                     dtype, experts=rng.randint(4, 64))
    cols = side(256, 12288)
    return _case(None, op, form, _log_int(rng, 1, 4096), min(side(256, 12288), 2 ** 25 // cols),
                 cols, dtype)


def _blocks(n):
    return (n + 127) // 128


def work(case):
    c = case
    n, R, C, E = c["n"], c["rows"], c["cols"], c["experts"]
    if c["op"] == "norm":
        if c["form"] == "backward":          # s, dy and ds; dx, the gain and its gradient
            return {"bytes": 8.0 * n * C + 4 * C, "flops": 12.0 * n * C}
        y = n * (C + 4 * _blocks(C)) if c["form"] == "blocks" else 2.0 * n * C
        return {"bytes": 6.0 * n * C + 2 * C + y, "flops": 8.0 * n * C}
    if c["op"] == "blocks":
        if c["form"] == "rows":
            return {"bytes": 3.0 * n * C + 4 * n * _blocks(C), "flops": 3.0 * n * C}
        return {"bytes": 3.0 * R * C + 4 * _blocks(R) * _blocks(C), "flops": 3.0 * R * C}
    wide, tall = (R, C) if c["form"] == "backward" else (C, R)
    # experts that some row goes to, each row's expert drawn from _expert_share
    used = float((1 - (1 - _expert_share(E)) ** n).sum()) if E > 1 else 1.0
    x = n * (wide + 4 * _blocks(wide)) if c["form"] == "forward blocks" else 2.0 * n * wide
    return {"bytes": used * (R * C + 4.0 * _blocks(R) * _blocks(C)) + x + 2.0 * n * tall,
            "flops": 2.0 * n * R * C}


def _expert_share(E):
    """How often each expert is chosen: the busiest about six times as often as the median."""
    p = 1.0 / (1.0 + np.arange(E)) ** 0.5 if E > 1 else np.ones(1)
    return p / p.sum()


def _padded(v, rows):
    """v [..., R, C] with zeros up to whole blocks of `rows` x 128."""
    r, c = -v.shape[-2] % rows, -v.shape[-1] % 128
    return torch.nn.functional.pad(v, (0, c, 0, r)) if r or c else v


def _to_blocks(v, rows=1):
    """v [..., R, C] in 32 bits -> codes [..., R, C] and scales, a scale for `rows` x 128."""
    p = _padded(v, rows)
    p = p.reshape(p.shape[:-2] + (p.shape[-2] // rows, rows, p.shape[-1] // 128, 128))
    scale = torch.clamp(p.abs().amax(dim=(-3, -1)) / 448.0, min=2.0 ** -126)
    q = (p / scale[..., None, :, None]).to(E4M3)
    q = q.reshape(v.shape[:-2] + (-(-v.shape[-2] // rows) * rows, scale.shape[-1] * 128))
    return q[..., :v.shape[-2], :v.shape[-1]].contiguous(), scale


def _from_blocks(q, scale, rows=1, dtype=torch.float32):
    """The values [..., R, C] that codes and scales stand for."""
    s = scale.to(dtype).repeat_interleave(128, dim=-1)
    if rows > 1:
        s = s.repeat_interleave(rows, dim=-2)
    return q.to(dtype) * s[..., :q.shape[-2], :q.shape[-1]]


_contexts = []


def _context():
    """The context a program keeps."""
    if not _contexts:
        import trellis_coded_weight_amd as T
        _contexts.append(T.Context(0))
    return _contexts[0]


def _inputs(case, seed):
    c = case
    n, R, C, E = c["n"], c["rows"], c["cols"], c["experts"]
    dt = TYPES[c["dtype"]]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def channels(k):                          # a few channels are large
        return torch.where(torch.rand(k, generator=g, device=DEV) < 0.004, 12.0, 1.0)

    s = dict(c)
    if c["op"] == "norm":
        s["gain"] = (1.0 + 0.2 * normal(C)).to(dt)
        if c["form"] == "backward":
            s["s"] = (3.0 * normal(n, C) * channels(C)).to(dt)
            s["dy"], s["ds"] = (0.01 * normal(n, C)).to(dt), (0.01 * normal(n, C)).to(dt)
        else:                                 # the residual stream has grown, x is one layer's
            s["x"] = normal(n, C).to(dt)
            s["residual"] = (3.0 * normal(n, C) * channels(C)).to(dt)
        return s
    if c["op"] == "blocks" and c["form"] == "rows":
        # an activation function's products: heavy tails
        s["x"] = (normal(n, C) * normal(n, C) * channels(C)).to(dt)
        return s
    # rows of different sizes, as output channels have; a few are dead
    rms = 0.02 * torch.exp(0.4 * normal(E, R, 1))
    rms = torch.where(torch.rand(E, R, 1, generator=g, device=DEV) < 0.002, 0.0, rms)
    if c["op"] == "blocks":
        s["w"] = (normal(R, C) * rms[0]).to(dt)
        return s
    s["q"], s["scale"] = _to_blocks(normal(E, R, C) * rms, 128)
    wide = R if c["form"] == "backward" else C
    x = 0.01 * normal(n, wide) if c["form"] == "backward" else normal(n, wide) * channels(wide)
    s["x"] = x.to(dt)
    if c["form"] == "forward blocks":
        s["xq"], s["xs"] = _to_blocks(s["x"].float())
    if c["op"] == "grouped":
        host = np.random.Generator(np.random.PCG64(seed + 5))
        sizes = host.multinomial(n, host.permutation(_expert_share(E)))
        s["largest"] = int(sizes.max())
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).to(DEV)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import trellis_coded_weight_amd as T
        s["context"] = _context()
        if "q" in s:
            one = case["op"] == "linear"
            s["weight"] = T.BlockWeight(s["q"][0], s["scale"][0]) if one else \
                T.BlockWeight(s["q"], s["scale"])
        if "xq" in s:
            s["x"] = T.BlockRows(s["xq"], s["xs"])
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    ctx, form = s["context"], s["form"]
    if s["op"] == "norm":
        if form == "backward":
            return ctx.rms_norm_backward(s["dy"], s["s"], s["gain"], eps=1e-6, ds=s["ds"])
        y, total = ctx.rms_norm(s["x"], s["gain"], eps=1e-6, residual=s["residual"],
                                blocks=form == "blocks")
        return (y.q, y.scale, total) if form == "blocks" else (y, total)
    if s["op"] == "blocks":
        b = ctx.block_quantize(s["x"]) if form == "rows" else ctx.block_quantize_weight(s["w"])
        return b.q, b.scale
    back, dt = form == "backward", TYPES[s["dtype"]]
    if s["op"] == "linear":
        return ctx.block_linear(s["x"], s["weight"], transpose=back, dtype=dt)
    return ctx.block_grouped_linear(s["x"], s["weight"], s["offsets"], transpose=back, dtype=dt)


def _plain_grouped(x, w, offsets, largest):
    """x's rows times their group's matrix w [experts, in, out], in 32 bits."""
    row = torch.arange(x.shape[0], device=DEV)
    expert = torch.searchsorted(offsets[1:].contiguous(), row.to(torch.int32), right=True)
    slot = row - offsets[expert]
    padded = torch.zeros(w.shape[0], largest, x.shape[1], device=DEV)
    padded[expert, slot] = x
    return torch.bmm(padded, w.contiguous())[expert, slot]


def _run_plain(s):
    dt, form = TYPES[s["dtype"]], s["form"]
    if s["op"] == "norm":
        gain = s["gain"].float()
        t = s["s"].float() if form == "backward" else s["x"].float() + s["residual"].float()
        r = 1.0 / torch.sqrt(t.square().mean(dim=1, keepdim=True) + 1e-6)
        unit = t * r
        if form == "backward":
            dy = s["dy"].float()
            du = dy * gain
            dx = s["ds"].float() + r * (du - unit * (du * unit).mean(dim=1, keepdim=True))
            return dx.to(dt), (dy * unit).sum(dim=0).to(dt)
        if form == "blocks":
            return _to_blocks(unit * gain) + (t.to(dt),)
        return (unit * gain).to(dt), t.to(dt)
    if s["op"] == "blocks":
        return _to_blocks(s["x"].float()) if form == "rows" else _to_blocks(s["w"].float(), 128)
    w = _from_blocks(s["q"], s["scale"], 128)
    x = _from_blocks(s["xq"], s["xs"]) if form == "forward blocks" else \
        _from_blocks(*_to_blocks(s["x"].float()))
    if form != "backward":
        w = w.transpose(1, 2)
    if s["op"] == "linear":
        return torch.matmul(x, w[0]).to(dt)
    return _plain_grouped(x, w, s["offsets"], s["largest"]).to(dt)


def _exact_e4m3(t):
    """t rounded to the nearest e4m3 value, ties to even, in 64 bits: four significant bits, or
    the spacing 2^-9 below 2^-6."""
    exponent = torch.clamp(torch.frexp(t)[1].double() - 1, min=-6.0)
    step = torch.exp2(exponent - 3)
    return torch.round(t / step) * step


def _exact_rows(v):
    """(codes, scales) of rows in 64 bits, block after block."""
    q, scale = torch.empty_like(v), []
    for c in range(0, v.shape[1], 128):
        part = v[:, c:c + 128]
        s = part.abs().max(dim=1).values.div(448.0).clamp(min=2.0 ** -126)
        q[:, c:c + 128] = _exact_e4m3(part / s[:, None])
        scale.append(s)
    return q, torch.stack(scale, dim=1)


def exact(case, seed):
    s = _inputs(case, seed)
    form = s["form"]
    if s["op"] == "norm":
        gain = s["gain"].double()
        t = s["s"].double() if form == "backward" else s["x"].double() + s["residual"].double()
        rms = torch.sqrt((t * t).sum(dim=1) / t.shape[1] + 1e-6)[:, None]
        if form != "backward":
            y = t / rms * gain
            return _exact_rows(y) + (t,) if form == "blocks" else (y, t)
        dy = s["dy"].double()
        inner = (dy * gain * t).sum(dim=1)[:, None] / t.shape[1]
        return s["ds"].double() + dy * gain / rms - t * inner / rms ** 3, (dy * t / rms).sum(dim=0)
    if s["op"] == "blocks":
        if form == "rows":
            return _exact_rows(s["x"].double())
        w = s["w"].double()
        q, scale = torch.empty_like(w), []
        for r in range(0, w.shape[0], 128):
            strip = w[r:r + 128]
            big = [strip[:, c:c + 128].abs().max() for c in range(0, w.shape[1], 128)]
            line = (torch.stack(big) / 448.0).clamp(min=2.0 ** -126)
            q[r:r + 128] = _exact_e4m3(strip / line.repeat_interleave(128)[:w.shape[1]])
            scale.append(line)
        return q, torch.stack(scale)
    if form == "forward blocks":
        xq, xs = s["xq"].double(), s["xs"].double()
    else:
        xq, xs = _exact_rows(s["x"].double())
    cut = s["offsets"].tolist() if s["op"] == "grouped" else [0, s["n"]]
    out = []
    for e in range(s["experts"]):
        a, b = cut[e], cut[e + 1]
        if a == b:
            continue
        wq, ws = s["q"][e].double(), s["scale"][e].double()
        ws = ws.repeat_interleave(128, dim=0)[:s["rows"]]
        if form == "backward":     # every 128 rows of W are one block of the contraction
            ws = ws.repeat_interleave(128, dim=1)[:, :s["cols"]]
            y = (xq[a:b] * xs[a:b].repeat_interleave(128, dim=1)[:, :s["rows"]]) @ (wq * ws)
        else:                      # the sum over blocks of the codes' products, scaled
            y = torch.zeros(b - a, s["rows"], dtype=torch.float64, device=DEV)
            for k in range(ws.shape[1]):
                at = slice(128 * k, 128 * k + 128)
                y += (xq[a:b, at] @ wq[:, at].t()) * xs[a:b, k:k + 1] * ws[:, k]
        out.append(y)
    return torch.cat(out)
